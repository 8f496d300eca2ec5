"""64-bit numpy forms of the operators over a paged key-value cache (page maps, rotary positions with the cache's rows,
attention of new tokens, verification of drafted tokens), for the tests; no code of the library's."""
import numpy as np


def page_map(length, count, table, owned, free, free_count, page, tokens):
    """The step of bl_page_map, one page and one token at a time: (start, position, slot, length, owned, left) and whether
    anything was out of range; table and free are changed in place."""
    R, W = table.shape
    pages = len(free)
    bad = not 0 <= free_count <= pages
    left = min(max(free_count, 0), pages)
    start, position, slot, length_out, owned_out = [0], [], [], [], []
    for r in range(R):
        have = min(max(int(owned[r]), 0), W)
        bad |= length[r] < 0 or have != owned[r]
        if count[r] < 0:
            length_out.append(0)
            owned_out.append(0)
            start.append(start[-1])
            continue
        total = max(int(length[r]), 0) + int(count[r])
        need = -(-total // page)
        bad |= need > W
        got = have
        for i in range(have, min(need, W)):
            if left > 0:
                left -= 1
                table[r, i] = free[left]
                got += 1
            else:
                table[r, i] = -1
                bad = True
        for i in range(int(count[r])):
            at = total - int(count[r]) + i
            entry = table[r, at // page] if at // page < W else -1
            bad |= entry >= pages
            position.append(at)
            slot.append(entry * page + at % page if 0 <= entry < pages else -1)
        length_out.append(total)
        owned_out.append(got)
        start.append(start[-1] + int(count[r]))
    for r in range(R):
        if count[r] < 0:
            for i in range(min(max(int(owned[r]), 0), W)):
                if left < pages:
                    free[left] = table[r, i]
                    left += 1
                else:
                    bad = True
    bad |= start[-1] > tokens
    position = (position + [-1] * tokens)[:tokens]
    slot = (slot + [-1] * tokens)[:tokens]
    return np.minimum(start, tokens), np.array(position), np.array(slot), np.array(length_out), np.array(owned_out), left, bad


def rope(x, cos, sin, position):
    """Heads x [M, heads, D] turned by the tables' rows [positions, rotary / 2]: (values, sums of absolute terms)."""
    half = cos.shape[1]
    y, cond = x.astype(np.float64).copy(), np.abs(x).astype(np.float64)
    c, s = cos[position][:, None, :].astype(np.float64), sin[position][:, None, :].astype(np.float64)
    a, b = x[..., :half].astype(np.float64), x[..., half:2 * half].astype(np.float64)
    y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    cond[..., :half], cond[..., half:2 * half] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return y, cond


def attention_row(q, k, v, seen, scale):
    """(out, cond, size): out [D] of one row over the tokens of k, v [n, D] that are seen; cond = sum_j p_j |v_j|; size: the
    largest sum of absolute products in a score that has weight, times scale."""
    D = v.shape[1]
    if not seen.any():
        return np.zeros(D), np.zeros(D), 0.0
    k, v, q = k[seen].astype(np.float64), v[seen].astype(np.float64), q.astype(np.float64)
    z = k @ q * scale
    w = np.exp(z - z.max())
    p = w / w.sum()
    size = (np.abs(k) @ np.abs(q)).max() * abs(scale)
    return p @ v, p @ np.abs(v), size


def seen_by(position, n, window, sinks):
    j = np.arange(n)
    return (j <= position) & ((j > position - window) | (j < sinks) if window else np.ones(n, bool))


def weights(l, t):
    """exp((l - max) / t), unnormalised; zeros for a row without a logit above -inf."""
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64)) + 0.0
    top = l.max()
    if top == -np.inf:
        return np.zeros(len(l))
    w = (l == top).astype(np.float64)
    if t >= np.float32(1e-5):
        low = (l < top) & (l > -np.inf) if top < np.inf else np.zeros(len(l), bool)
        w[low] = np.exp((l[low] - top) / np.float64(t))
    return w


def verify(logits, drafts, token, u, us, t):
    """One request's rows: (accepted, next token, margin, weights): margin is how far, relative to p, the nearest test of
    acceptance is from going the other way; weights: what the token is drawn from."""
    margin, V = 1.0, logits.shape[1]
    clamp = lambda v: min(float(v), float(np.float32(0.99999994))) if v > 0 else 0.0  # noqa: E731
    for i in range(len(logits) - 1):
        p, x = weights(logits[i], t), int(token[i + 1])
        p = p / p.sum() if p.sum() else p
        if drafts is None:
            q = np.zeros(V)
            if 0 <= x < V:
                q[x] = 1
        else:
            q = weights(drafts[i], t)
            q = q / q.sum() if q.sum() else q
        px, qx = (p[x], q[x]) if 0 <= x < V else (0.0, 1.0)
        gap = px - clamp(u[i]) * qx
        if gap != 0 and 0 <= x < V and px > 0 and clamp(u[i]) * qx > 0 and not (set(np.unique(p)) <= {0.0, p.max()} and drafts is None):
            margin = min(margin, abs(gap) / px)
        if gap > 0:
            continue
        rest = np.maximum(p - q, 0)
        if rest.sum() <= 0:
            rest = p
        return i, draw(rest, clamp(us)), margin, rest
    p = weights(logits[-1], t)
    return len(logits) - 1, draw(p, clamp(us)), margin, p


def draw(w, u):
    mass = np.cumsum(w)
    if not mass[-1] > 0:
        return -1
    return min(int(np.searchsorted(mass, u * mass[-1], side="right")), int(np.nonzero(w)[0][-1]))
