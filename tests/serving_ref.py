"""64-bit numpy forms of the operators around the products (norm with codes,
low-rank adapters, sampling), for the tests; no code of the library's."""
import numpy as np


def bf16_round(v):
    """Nearest bf16 (ties to even) of float32 values, as float32."""
    b = np.asarray(v, np.float32).view(np.uint32).astype(np.uint64)
    return (((b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16) & 0xFFFFFFFF).astype(np.uint32).view(np.float32)


def rmsnorm_quant(x, residual, w, eps, bf16):
    """(q, s, h, y, clear): the definition with its binary32 roundings; float32 arrays hold bf16 values when bf16.
    clear[m]: the row's factor lies further than 2^-40 from a rounding border, so the codes are determined."""
    rnd = bf16_round if bf16 else (lambda v: v)
    h = x if residual is None else rnd((x + residual).astype(np.float32))
    mean = (h.astype(np.float64) ** 2).mean(1) + np.float64(np.float32(eps))
    with np.errstate(divide="ignore"):
        r64 = np.where(mean > 0, 1 / np.sqrt(mean), 0.0)
    r = r64.astype(np.float32)
    up, down = np.nextafter(r, np.float32(np.inf)).astype(np.float64), np.nextafter(r, np.float32(0)).astype(np.float64)
    r32 = r.astype(np.float64)
    border = np.minimum(np.abs(r64 - (r32 + up) / 2), np.abs(r64 - (r32 + down) / 2))
    v = ((h * r[:, None]).astype(np.float32) * w).astype(np.float32)
    amax = np.abs(v).max(1)
    with np.errstate(divide="ignore", invalid="ignore"):
        inv = np.where(amax > 0, np.float32(127) / amax, np.float32(0)).astype(np.float32)
    q = np.clip(np.rint((v * inv[:, None]).astype(np.float32)), -127, 127).astype(np.int8)
    s = (amax / np.float32(127)).astype(np.float32)
    return q, s, h, rnd(v), border > r64 * 2.0 ** -40


def lora_add(x, adapter, a, b, scale, base):
    """(y, cond): cond is the sum of the absolute products of each output."""
    y, cond = base.astype(np.float64).copy(), np.abs(base).astype(np.float64)
    for m in range(x.shape[0]):
        l = adapter[m]
        if 0 <= l < a.shape[0]:
            low = a[l].astype(np.float64) @ x[m].astype(np.float64)
            y[m] += np.float64(scale[l]) * (b[l].astype(np.float64) @ low)
            low = np.abs(a[l]).astype(np.float64) @ np.abs(x[m]).astype(np.float64)
            cond[m] += abs(np.float64(scale[l])) * (np.abs(b[l]).astype(np.float64) @ low)
    return y, cond


def sample_row(l, u, t=1.0, k=0, p=1.0, mp=0.0):
    """(token, prob, margin, near): margin is how far (relative to the weight that stays) the nearest decision that
    the token rests on is from going the other way (equality of exact weights is decided exactly and does not count);
    near[i] is how far token i's interval of cumulative weights is from the goal, relative to the same."""
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64)) + 0.0
    order = np.argsort(-l, kind="stable")
    z = l[order]
    if z[0] == -np.inf:
        return -1, 0.0, 1.0, np.full(len(z), np.inf)
    w = np.zeros(len(z))
    w[z == z[0]] = 1.0
    if t >= np.float32(1e-5) and np.isfinite(z[0]):
        low = (z < z[0]) & (z > -np.inf)
        w[low] = np.exp((z[low] - z[0]) / np.float64(t))
    n = len(z) if k <= 0 else min(int(k), len(z))
    margin = 1.0
    exact = lambda v: float(v) == round(float(v) * 2 ** 20) / 2 ** 20  # noqa: E731
    if p < 1:
        mass = np.cumsum(w[:n])
        limit = max(float(p), 0.0) * mass[-1]
        before = mass - w[:n]
        stay = before < limit
        if not (np.all((w == 0) | (w == 1)) and exact(limit)):
            margin = min(margin, np.abs(before[1:] - limit).min(initial=np.inf) / mass[-1])
        n = max(1, int(stay.sum()))
    if mp > 0:
        stay = w[:n] >= min(float(mp), 1.0)
        stay[0] = True
        if mp < 1:
            margin = min(margin, np.abs(w[:n] - float(mp)).min())
        n = int(stay.sum())
    mass = np.cumsum(w[:n])
    uu = min(float(u), 0.99999994) if u > 0 else 0.0
    goal = uu * mass[-1]
    at = min(int((mass <= goal).sum()), n - 1)
    if not (np.all((w == 0) | (w == 1)) and exact(goal)) and uu > 0:
        margin = min(margin, np.abs(mass - goal).min() / mass[-1])
    near = np.full(len(z), np.inf)
    near[order[:n]] = np.maximum(0, np.maximum(goal - mass, mass - w[:n] - goal)) / mass[-1]
    return int(order[at]), w[at] / mass[-1], margin, near
