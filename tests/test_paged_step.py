"""The operators of a decode step over a paged key-value cache (bl_page_map, bl_rope_append, bl_attn_paged, bl_verify)
against 64-bit forms.

Maps, counts and tokens are compared exactly; the tolerances of the other
outputs are derived beside each test."""
import ctypes

import numpy as np
import pytest
import torch

import paged_ref as R
from serving_ref import bf16_round

gpu = pytest.mark.gpu
BF16_HALF_STEP, F32_HALF_STEP = 2.0 ** -8, 2.0 ** -24
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def B():
    from gemm_bl_gemv_gb300 import build
    build.build()
    from gemm_bl_gemv_gb300 import binding
    yield binding


@pytest.fixture(autouse=True)
def no_device_error(request):
    if "gpu" not in request.keywords:
        yield
        return
    from gemm_bl_gemv_gb300 import binding
    binding.set_overlap(False)
    binding.device_error(clear=True)
    yield
    torch.cuda.synchronize()
    assert binding.device_error(clear=True) == 0


def rng(*seed):
    return np.random.Generator(np.random.PCG64(list(seed)))


def dev(v, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(v)).cuda()
    return t if dtype is None else t.to(dtype)


def ints(v):
    return torch.tensor(np.asarray(v).tolist(), dtype=I32).reshape(np.asarray(v).shape).cuda()


def host(t):
    return t.float().cpu().numpy()


def range_error(B):
    torch.cuda.synchronize()
    return B.device_error(clear=True) == B.BL_DEVERR_RANGE


# ---------------------------------------------------------------------------
# refusals (host checks: no GPU)
# ---------------------------------------------------------------------------

def test_refusals_without_gpu(B):
    L = B.lib()
    P = ctypes.c_void_p
    a, o1, o2, o8, o16 = (P((1 << 14) + n) for n in (0, 1, 2, 8, 16))
    NULL, SHAPE, AL, DT, UN = B.BL_ERR_NULL, B.BL_ERR_SHAPE, B.BL_ERR_ALIGN, B.BL_ERR_DTYPE, B.BL_ERR_UNSUPPORTED
    F, H = B.BL_F32, B.BL_BF16
    cases = []

    def case(fn, good, want, **bad):  # `good` by name, in order; one or more replaced
        cases.append((fn, tuple({**good, **bad}.values()), want))

    m = dict(length=a, count=a, table=a, owned=a, free=a, fc=a, R=2, W=4, pages=8, page=16, M=3, start=a, position=a, slot=a,
             length_out=a, owned_out=a, left=a, stream=None)
    f = L.bl_page_map
    for n in ("length", "count", "table", "owned", "free", "fc", "start", "position", "slot", "length_out", "owned_out", "left"):
        case(f, m, NULL, **{n: None})
        case(f, m, AL, **{n: o2})
    for n in ("R", "W", "pages", "page", "M"):
        case(f, m, SHAPE, **{n: 0})
    case(f, m, SHAPE, M=1 << 31)
    case(f, m, UN, pages=1 << 28)

    e = dict(qkv=a, xt=F, cos=a, sin=a, position=a, slot=a, M=2, H=4, Hk=2, D=64, rotary=64, positions=10, q=a, k=a, v=a,
             pages=8, page=16, stream=None)
    f = L.bl_rope_append
    for n in ("qkv", "cos", "sin", "position", "slot", "q", "k", "v"):
        case(f, e, NULL, **{n: None})
        case(f, e, AL, **{n: o2})
    for n in ("qkv", "q", "k", "v"):
        case(f, e, AL, **{n: o8})
    case(f, e, DT, xt=2)
    for n in ("M", "H", "Hk", "D", "rotary", "positions", "pages", "page"):
        case(f, e, SHAPE, **{n: 0})
    case(f, e, SHAPE, D=60)
    case(f, e, SHAPE, rotary=7)
    case(f, e, SHAPE, rotary=66)
    case(f, e, UN, D=1032, rotary=64)
    case(f, e, UN, pages=1 << 28)

    ws = L.bl_attn_paged_workspace(3, 8, 2, 128)
    assert ws > 0 and L.bl_attn_paged_workspace(0, 8, 2, 128) == 0 and L.bl_attn_paged_workspace(3, 8, 3, 128) == 0
    t = dict(q=a, k=a, v=a, table=a, length=a, start=a, scale=0.1, window=0, sinks=0, M=3, R=2, H=8, Hk=2, D=128, pages=8,
             page=16, W=4, out=a, ot=F, ws=a, bytes=ws, stream=None)
    f = L.bl_attn_paged
    for n in ("q", "k", "v", "table", "length", "start", "out", "ws"):
        case(f, t, NULL, **{n: None})
        case(f, t, AL, **{n: o2})
    for n in ("q", "k", "v", "out"):
        case(f, t, AL, **{n: o8})
    case(f, t, AL, ws=o16)
    case(f, t, DT, ot=2)
    for n in ("M", "R", "H", "Hk", "D", "pages", "page", "W"):
        case(f, t, SHAPE, **{n: 0})
    case(f, t, SHAPE, Hk=3)
    case(f, t, SHAPE, D=12)
    case(f, t, SHAPE, window=-1)
    case(f, t, SHAPE, sinks=-1)
    case(f, t, SHAPE, bytes=ws - 1)
    case(f, t, UN, D=264)
    case(f, t, UN, pages=1 << 28)

    ws = L.bl_verify_workspace(3)
    assert ws > 0 and L.bl_verify_workspace(0) == 0
    y = dict(logits=a, drafts=a, lt=F, token=a, start=a, temperature=a, u=a, us=a, M=3, R=2, V=100, accepted=a, next=a, ws=a,
             bytes=ws, stream=None)
    f = L.bl_verify
    for n in ("logits", "token", "start", "u", "us", "accepted", "next", "ws"):
        case(f, y, NULL, **{n: None})
    for n in ("logits", "drafts", "token", "start", "temperature", "u", "us", "accepted", "next", "ws"):
        case(f, y, AL, **{n: o2})
    case(f, y, AL, logits=o1, lt=H)
    case(f, y, DT, lt=2)
    for n in ("M", "R", "V"):
        case(f, y, SHAPE, **{n: 0})
    case(f, y, SHAPE, bytes=ws - 1)
    case(f, y, UN, V=524289)
    case(f, y, UN, M=1 << 26)
    for fn, args, want in cases:
        got = fn(*args)
        assert got == want, (fn.__name__, args, B.status_name(got), B.status_name(want))
        assert fn.__name__.encode() in L.bl_last_error()


def test_binding_refuses_host_tensors(B):
    x, i = torch.zeros(2, 8), torch.zeros(2, dtype=I32)
    c = torch.zeros(2, 1, 4, 8, dtype=BF)
    for call in (lambda: B.bl_page_map(i, i, i.reshape(1, 2), i, i, i, 16, 2), lambda: B.bl_rope_append(x, x, x, i, i, c, c, 1),
                 lambda: B.bl_attn_paged(x.reshape(2, 1, 8), c, c, i.reshape(1, 2), i, i, 1.0), lambda: B.bl_verify(x, i, i, x[0], x[0])):
        with pytest.raises(TypeError):
            call()


def test_reference_forms():
    """The 64-bit forms on hand-worked values."""
    table, free = np.full((3, 3), -1), np.array([7, 5, 3, 1, 0, 0, 0, 0])
    table[1, 0] = 6
    got = R.page_map([0, 3, 4], [5, 2, -1], table, [0, 1, 0], free, 4, 4, 9)
    assert got[0].tolist() == [0, 5, 7, 7] and got[1].tolist() == [0, 1, 2, 3, 4, 3, 4, -1, -1]
    assert table.tolist() == [[1, 3, -1], [6, 5, -1], [-1, -1, -1]] and got[5] == 1 and not got[6]
    assert got[2].tolist() == [4, 5, 6, 7, 12, 27, 20, -1, -1] and got[3].tolist() == [5, 5, 0] and got[4].tolist() == [2, 2, 0]
    y, _ = R.rope(np.array([[[1.0, 2.0, 3.0, 4.0, 9.0]]]), np.array([[0.0, 1.0]]), np.array([[1.0, 0.0]]), np.array([0]))
    assert y[0, 0].tolist() == [-3.0, 2.0, 1.0, 4.0, 9.0]
    o, _, _ = R.attention_row(np.array([1.0]), np.array([[0.0], [np.log(3.0)], [9.0]]), np.array([[4.0], [8.0], [0.0]]), np.array([1, 1, 0], bool), 1.0)
    assert np.allclose(o, 7.0)
    assert R.seen_by(5, 8, 2, 1).tolist() == [True, False, False, False, True, True, False, False]
    l = np.log(np.array([[1.0, 2.0, 1.0], [3.0, 1.0, 4.0]]))
    assert R.verify(l, None, [0, 1], [0.49, 0], 0.4, 1.0)[:2] == (1, 1)  # 3 of 8 lies below 0.4
    assert R.verify(l, None, [0, 1], [0.5, 0], 0.6, 1.0)[:2] == (0, 2)   # without token 1
    q = np.log(np.array([[1.0, 1.0, 2.0], [1.0, 1.0, 1.0]]))
    assert R.verify(l, q, [0, 2], [0.6, 0], 0.9, 1.0)[:2] == (0, 1)      # p - q = 0, 1/4, -1/4


# ---------------------------------------------------------------------------
# page maps: exact
# ---------------------------------------------------------------------------

def page_inputs(requests, page, W, longest, most_new, seed, ended=0.2, ahead=0.3):
    g = rng(requests, page, seed)
    length = g.integers(0, longest + 1, requests)
    count = g.integers(0, most_new + 1, requests)
    owned = np.minimum(-(-length // page) + (g.random(requests) < ahead), W)
    count[g.random(requests) < ended] = -1
    pages = int(owned.sum() + (-(-np.maximum(count, 0) // page) + 1).sum())
    pool = g.permutation(pages)
    table = np.full((requests, W), -1)
    table[np.arange(W) < owned[:, None]] = pool[: owned.sum()]
    free = np.zeros(pages, int)
    free[: pages - owned.sum()] = pool[owned.sum():]
    return length, count, table, owned, free, int(pages - owned.sum())


def check_page_map(B, length, count, table, owned, free, free_count, page, tokens, bad=False, in_place=False):
    t = [ints(v) for v in (length, count, table, owned, free, [free_count])]
    outs = dict(length_out=t[0], owned_out=t[3], free_left=t[5]) if in_place else {}
    want_table, want_free = table.copy(), free.copy()
    want = R.page_map(length, count, want_table, owned, want_free, free_count, page, tokens)
    assert want[6] == bad
    got = B.bl_page_map(*t, page, tokens, **outs)
    for name, a, b in zip(("start", "position", "slot", "length", "owned", "left"), got, want):
        assert np.array_equal(a.cpu().numpy().reshape(-1), np.asarray(b).reshape(-1)), name
    assert np.array_equal(t[2].cpu().numpy(), want_table)
    left = want[5]
    assert np.array_equal(t[4].cpu().numpy()[:left], want_free[:left])
    if bad:
        assert range_error(B)
    return got


@gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("requests,page,longest,most_new", [
    (1, 16, 0, 1), (1, 1, 3, 5), (3, 16, 40, 40), (64, 16, 1000, 1), (33, 7, 300, 9), (1500, 16, 200, 3), (5, 128, 1000, 4000),
    (2100, 8, 60, 2), (40, 16, 100, 600)])
def test_page_map(B, requests, page, longest, most_new, in_place):
    W = -(-(longest + most_new) // page) + 1
    v = page_inputs(requests, page, W, longest, most_new, 1)
    tokens = int(np.maximum(v[1], 0).sum())
    for padding in (0, 5):
        check_page_map(B, *v, page, max(tokens + padding, 1), in_place=in_place)


@gpu
def test_page_map_ended_requests_only_and_idle_ones(B):
    v = list(page_inputs(9, 16, 10, 100, 3, 2, ended=0.0))
    check_page_map(B, v[0], np.full(9, -1), *v[2:], 16, 4)
    check_page_map(B, v[0], np.zeros(9, int), *v[2:], 16, 4)
    check_page_map(B, np.zeros(9, int), np.zeros(9, int), v[2], np.zeros(9, int), *v[4:], 16, 4)


@gpu
def test_page_map_out_of_range(B):
    length, count, table, owned, free, n = page_inputs(12, 16, 30, 200, 60, 3, ended=0.1)
    tokens = int(np.maximum(count, 0).sum())
    check_page_map(B, length, count, table, owned, free, 4, 16, tokens, bad=True)                # the stack runs empty
    check_page_map(B, length, count, table, owned, free, 0, 16, tokens, bad=True)
    check_page_map(B, length, count, table[:, :8].copy(), np.minimum(owned, 8), free, n, 16, tokens, bad=True)  # too few entries
    check_page_map(B, length, count, table, owned, free, n, 16, tokens - 7, bad=True)            # more tokens than rows
    odd = length.copy()
    odd[3] = -5
    check_page_map(B, odd, count, table, owned, free, n, 16, 3000, bad=True)
    odd = owned.copy()
    odd[4] = -1
    check_page_map(B, length, np.maximum(count, 1), table, odd, free, n, 16, 3000, bad=True)
    check_page_map(B, length, count, table, owned, free, len(free) + 3, 16, 3000, bad=True)
    odd = table.copy()
    odd[5, :owned[5]] = len(free)
    check_page_map(B, np.maximum(length, 1), np.zeros(12, int) + (np.arange(12) == 5), odd, np.maximum(owned, 2), free, n, 16, 3,
                   bad=bool(owned[5] * 16 > max(length[5], 1)))


@gpu
def test_page_map_steps(B):
    """A run of steps in place: requests come, grow, lose drafts and end; no page is ever held twice."""
    g = rng(7)
    requests, page, W, pages = 20, 4, 16, 120
    length, owned, fc = ints(np.zeros(requests)), ints(np.zeros(requests)), ints([pages])
    table, free = ints(np.full((requests, W), -1)), ints(g.permutation(pages))
    for step in range(40):
        n, have = length.cpu().numpy(), owned.cpu().numpy()
        count = np.where(n == 0, g.integers(0, 20, requests), g.integers(1, 6, requests))
        count[(n + count > W * page) | (g.random(requests) < 0.05)] = -1
        if np.maximum(-(-(n + np.maximum(count, 0)) // page) - have, 0).sum() > int(fc):
            count[g.random(requests) < 0.7] = -1
            if np.maximum(-(-(n + np.maximum(count, 0)) // page) - have, 0).sum() > int(fc):
                count[:] = -1
        ct = ints(count)
        B.bl_page_map(length, ct, table, owned, free, fc, page, 300, length_out=length, owned_out=owned, free_left=fc)
        held = [int(p) for r in range(requests) for p in table[r, : int(owned[r])]] + free[: int(fc)].tolist()
        assert sorted(held) == list(range(pages)), step
        refused = np.minimum(g.integers(0, 4, requests), np.maximum(count - 1, 0))
        length -= ints(refused)


# ---------------------------------------------------------------------------
# rotary positions and the cache's rows.  A term's product is rounded once, their
# sum once more: 2^-23 of the sum of absolute terms, then half a step of bf16.
# What is copied is rounded once, exactly.
# ---------------------------------------------------------------------------

def rope_inputs(M, H, Hk, D, rotary, page, xb, seed):
    g = rng(M, H, D, rotary, seed)
    x = g.standard_normal((M, H + 2 * Hk, D)).astype(np.float32) * g.uniform(0.1, 10, (M, 1, 1)).astype(np.float32)
    angle = np.arange(500)[:, None] * 10000.0 ** -(np.arange(rotary // 2) * 2 / rotary)
    pages = M // page + 3
    slot = g.permutation(pages * page)[:M]
    return (bf16_round(x) if xb else x), np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32), g.integers(0, 500, M), slot, pages


def check_rope(B, v, H, Hk, page, xb, place=lambda t: t):
    x, cos, sin, position, slot, pages = v
    M, _, D = x.shape
    k, w = (torch.full((pages, Hk, page, D), 7.0, dtype=BF, device="cuda") for _ in range(2))
    q0 = torch.full((M, H, D), 7.0, dtype=BF, device="cuda")
    q = B.bl_rope_append(dev(x.reshape(M, -1), BF if xb else F32), place(dev(cos)), place(dev(sin)), ints(position), ints(slot), k, w, H, q=q0)
    assert q is q0
    token = (position >= 0) & (position < len(cos))
    ref, cond = R.rope(x[:, : H + Hk], cos, sin, np.where(token, position, 0))
    slack = BF16_HALF_STEP * np.abs(ref) + 2.0 ** -22 * cond  # the last half step of a value next to a border included
    half = cos.shape[1]
    err = np.abs(host(q) - ref[:, :H])
    assert np.all(err[token] <= slack[token, :H]) and np.all(host(q)[~token] == 7)
    assert np.array_equal(host(q)[token][..., 2 * half:], bf16_round(x[token][:, :H, 2 * half:]))
    for cache, rows, bound in ((k, ref[:, H:], slack[:, H:]), (w, bf16_round(x[:, H + Hk:]), 0 * x[:, H + Hk:])):
        flat = host(cache).transpose(0, 2, 1, 3).reshape(-1, Hk, D)
        stored = token & (slot >= 0) & (slot < len(flat))
        assert np.all(np.abs(flat[slot[stored]] - rows[stored]) <= bound[stored])
        rest = np.ones(len(flat), bool)
        rest[slot[stored]] = False
        assert np.all(flat[rest] == 7)


@gpu
@pytest.mark.parametrize("xb", [True, False])
@pytest.mark.parametrize("M,H,Hk,D,rotary,page", [
    (1, 1, 1, 8, 8, 16), (1, 20, 5, 128, 128, 16), (3, 4, 4, 64, 64, 1), (37, 6, 2, 80, 80, 7), (5, 8, 1, 96, 48, 16), (9, 3, 3, 128, 20, 32),
    (311, 40, 8, 128, 128, 16), (2000, 8, 2, 256, 128, 64), (1300, 5, 5, 72, 2, 16)])
def test_rope_append(B, M, H, Hk, D, rotary, page, xb):
    v = rope_inputs(M, H, Hk, D, rotary, page, xb, 1)
    check_rope(B, v, H, Hk, page, xb)


@gpu
@pytest.mark.parametrize("xb", [True, False])
@pytest.mark.parametrize("M,D,rotary", [(1301, 1024, 1024), (1217, 1024, 1022), (1250, 136, 136), (2001, 8, 2)])
def test_rope_append_many_tokens_with_long_and_short_heads(B, M, D, rotary, xb):
    check_rope(B, rope_inputs(M, 2, 1, D, rotary, 16, xb, 3), 2, 1, 16, xb)


@gpu
def test_rope_append_unaligned_tables(B):
    def off(t):
        buf = torch.empty(t.numel() + 1, device="cuda")
        out = buf[1:].view(t.shape)
        out.copy_(t)
        return out
    check_rope(B, rope_inputs(20, 4, 2, 64, 64, 16, True, 2), 4, 2, 16, True, place=off)


@gpu
@pytest.mark.parametrize("rotary", [64, 4])
def test_rope_append_rows_without_a_token_or_slot(B, rotary):
    x, cos, sin, position, slot, pages = rope_inputs(50, 4, 2, 64, rotary, 16, True, 3)
    position[[3, 48, 49]] = -1
    slot[[5, 6]] = -1
    check_rope(B, (x, cos, sin, position, slot, pages), 4, 2, 16, True)
    position[7] = 500
    check_rope(B, (x, cos, sin, position, slot, pages), 4, 2, 16, True)
    assert range_error(B)
    position[7], slot[8] = 0, pages * 16
    check_rope(B, (x, cos, sin, position, slot, pages), 4, 2, 16, True)
    assert range_error(B)


@gpu
def test_rope_append_infinities_stay_in_their_head(B):
    x, cos, sin, position, slot, pages = rope_inputs(6, 4, 2, 64, 64, 16, False, 4)
    y = x.copy()
    y[2, 1, 5], y[3, 5, 9], y[4, 6, 9] = np.inf, np.nan, -np.inf

    def run(x):
        k, v = (torch.zeros((pages, 2, 16, 64), dtype=BF, device="cuda") for _ in range(2))
        q = B.bl_rope_append(dev(x.reshape(6, -1)), dev(cos), dev(sin), ints(position), ints(slot), k, v, 4)
        rows = [host(c).transpose(0, 2, 1, 3).reshape(-1, 2, 64)[slot] for c in (k, v)]
        return np.concatenate([host(q)] + rows, 1)
    a, b = run(x), run(y)
    for m, h in ((2, 1), (3, 5), (4, 6)):
        assert not np.isfinite(b[m, h]).all()
        b[m, h] = a[m, h]
    assert np.array_equal(a, b)


# ---------------------------------------------------------------------------
# attention.  With z the scores (scale included), s = the largest sum of absolute
# products of a score, cond = sum_j p_j |v_j|, the errors are
#   of a score: the tensor core's sums over D, D / 16 + 2 additions that cut off at
#     2^-22 of s at most; a rounding by scale and one by the subtraction of the
#     maximum, 2^-23 |z| <= 2^-23 s each; exp2's 2^-22;  it moves p by as much,
#     and the sum of the weights once more: twice all this, times cond
#   of a weight on its way into the second product: 2^-17 (bf16), 2^-24 (fp32)
#   of the sums over tokens: an addition per tile of 16 tokens and per part, each
#     with its multiplication, and the sum of the weights: 2^-22 (n / 16 + 40)
# and half a step of the result.
# ---------------------------------------------------------------------------

class Cache:
    """Requests of the given lengths on randomly placed pages; what no request owns, and the rest of their pages, is NaN."""

    def __init__(self, lengths, Hk, D, page, seed, spare=3, wide=False, k_scale=1.0):
        g = rng(Hk, D, page, seed, len(lengths))
        extra_w = -(-4096 // page) if wide else 1  # tables for 4096 tokens and more: tiles of 128 tokens where D is 104..128
        self.lengths, self.page, self.Hk, self.D = list(lengths), page, Hk, D
        need = [-(-n // page) for n in lengths]
        self.pages = sum(need) + spare
        W = max(need + [0]) + extra_w
        order = g.permutation(self.pages)
        self.table = np.full((len(lengths), W), -1)
        self.k, self.v = (np.full((self.pages, Hk, page, D), np.nan, np.float32) for _ in range(2))
        self.rows, at = [], 0
        for r, n in enumerate(lengths):
            mine = order[at:at + need[r]]
            at += need[r]
            self.table[r, :need[r]] = mine
            k = bf16_round((g.standard_normal((n, Hk, D)) * k_scale + g.standard_normal((1, Hk, D)) * 0.5).astype(np.float32))
            v = bf16_round(g.standard_normal((n, Hk, D)).astype(np.float32))
            self.rows.append((k, v))
            for j in range(n):
                self.k[mine[j // page], :, j % page], self.v[mine[j // page], :, j % page] = k[j], v[j]

    def gpu(self):
        return dev(self.k, BF), dev(self.v, BF), ints(self.table), ints(self.lengths)


def attn_ref(q, cache, counts, scale, window, sinks):
    """(out, cond, size) of all rows; size [M, H]."""
    M, H, D = q.shape
    out, cond, size, at = np.zeros((M, H, D)), np.zeros((M, H, D)), np.zeros((M, H)), 0
    for (k, v), n, c in zip(cache.rows, cache.lengths, counts):
        for t in range(c):
            seen = R.seen_by(n - c + t, n, window, sinks)
            for h in range(H):
                kv = h // (H // cache.Hk)
                out[at, h], cond[at, h], size[at, h] = R.attention_row(q[at, h], k[:, kv], v[:, kv], seen, scale)
            at += 1
    return out, cond, size


def attn_bound(ref, cond, size, longest, D, f32):
    score = ((D / 16 + 2) * 2.0 ** -22 + 2 * 2.0 ** -23) * size + 2.0 ** -22
    rel = 2 * score[..., None] + (2.0 ** -24 if f32 else 2.0 ** -17) + 2.0 ** -22 * (longest / 16 + 40)
    return rel * cond + (F32_HALF_STEP if f32 else BF16_HALF_STEP) * (np.abs(ref) + rel * cond)


def check_attn(B, cache, counts, H, f32, window=0, sinks=0, scale=None, seed=0, padding=0, q=None, **kw):
    M, D = sum(counts), cache.D
    scale = D ** -0.5 if scale is None else scale
    q = bf16_round(1.3 * rng(H, D, M, seed).standard_normal((M, H, D)).astype(np.float32)) if q is None else q
    k, v, table, length = cache.gpu()
    start = np.concatenate([[0], np.cumsum(counts)])
    qt = torch.full((M + padding, H, D), float("nan"), dtype=BF, device="cuda")
    qt[:M] = dev(q, BF)
    out = torch.full((M + padding, H, D), 5.0, dtype=F32 if f32 else BF, device="cuda")
    got = B.bl_attn_paged(qt, k, v, table, length, ints(start), scale, window=window, sinks=sinks, out=out, **kw)
    assert got is out
    ref, cond, size = attn_ref(q, cache, counts, scale, window, sinks)
    err = np.abs(host(out)[:M].astype(np.float64) - ref)
    bound = attn_bound(ref, cond, size, max(cache.lengths + [1]), D, f32)
    assert np.all(err <= bound), float(np.nanmax(err / np.maximum(bound, 1e-30)))
    assert np.all(host(out)[M:] == 5)
    return out


@gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("lengths,H,Hk,D,page", [
    ([1], 1, 1, 8, 16), ([2, 15, 16, 17], 4, 4, 64, 16), ([33, 100, 1], 10, 2, 128, 16), ([700], 20, 5, 128, 16), ([31, 32, 33, 64], 3, 1, 40, 32),
    ([129, 5], 8, 1, 80, 7), ([90, 300], 6, 2, 256, 16), ([50, 1, 2], 2, 2, 136, 1), ([400, 3, 77], 40, 8, 128, 128), ([65], 17, 1, 96, 8),
    ([140, 20], 40, 1, 64, 16), ([1500, 40, 900], 8, 2, 64, 64)])
def test_attn_one_token(B, lengths, H, Hk, D, page, f32, wide):
    check_attn(B, Cache(lengths, Hk, D, page, 1, wide=wide), [1] * len(lengths), H, f32)


@gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("lengths,counts,H,Hk,D,page", [
    ([40, 100, 17], [5, 2, 1], 10, 2, 128, 16), ([5, 9, 200], [5, 8, 3], 8, 8, 64, 16), ([70, 16, 30], [9, 16, 0], 6, 3, 128, 7), ([300], [33], 4, 1, 128, 16),
    ([130, 60], [4, 7], 16, 1, 256, 32), ([64, 40], [40, 40], 5, 1, 80, 16), ([20, 8, 100, 1], [0, 8, 0, 1], 4, 2, 64, 16),
    ([500, 3, 130, 128, 129], [5, 3, 8, 4, 1], 10, 2, 128, 16), ([1000, 127], [8, 7], 8, 1, 128, 64), ([260, 255, 40], [5, 6, 5], 8, 2, 72, 16), ([90, 4, 385], [17, 4, 9], 3, 1, 128, 1)])
def test_attn_drafts(B, lengths, counts, H, Hk, D, page, f32, wide):
    """Several new tokens, each of which sees those before it; requests without any; rows behind the last request."""
    check_attn(B, Cache(lengths, Hk, D, page, 2, wide=wide), counts, H, f32, padding=3)


@gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (16, 4), (100, 1), (5, 64), (33, 17), (1000, 4), (40, 1000), (1, 1)])
@pytest.mark.parametrize("lengths,counts,H,Hk,D", [([300, 17, 64, 1], [1, 1, 1, 1], 10, 2, 128), ([260, 40, 90], [5, 3, 8], 4, 2, 64), ([150, 33], [4, 2], 6, 2, 256),
                                                   ([700, 140, 9], [5, 8, 9], 8, 1, 128), ([400, 130], [7, 6], 8, 2, 64)])
def test_attn_window(B, lengths, counts, H, Hk, D, window, sinks, wide):
    check_attn(B, Cache(lengths, Hk, D, 16, 3, wide=wide), counts, H, True, window=window, sinks=sinks)


@gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("window,sinks", [(1 << 31, 0), ((1 << 63) - 1, 0), ((1 << 63) - 1, (1 << 63) - 1), (50, (1 << 63) - 1), (0, (1 << 63) - 1)])
def test_attn_windows_wider_than_any_request(B, window, sinks, wide):
    check_attn(B, Cache([300, 17, 129], 2, 128, 16, 17, wide=wide), [5, 1, 3], 10, True, window=window, sinks=sinks)


@gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("f32", [False, True])
def test_attn_many_requests_and_long_ones(B, f32, wide):
    g = rng(11)
    lengths = [int(n) for n in g.integers(1, 60, 300)]
    check_attn(B, Cache(lengths, 1, 64, 16, 4, wide=wide), [1] * 300, 2, f32)
    check_attn(B, Cache([6000, 3, 2500], 1, 128, 16, 5, wide=wide), [1, 1, 2], 2, f32)
    check_attn(B, Cache([6000, 5, 2500], 1, 128, 16, 5, wide=wide), [3, 5, 6], 5, f32)
    check_attn(B, Cache([max(n, 4) for n in lengths], 1, 128, 16, 4, wide=wide), [4] * 300, 5, f32)


@gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("page,window,sinks", [(32, 0, 0), (16, 1000, 4), (256, 0, 0), (8, 300, 200), (64, 0, 0), (128, 100, 0), (384, 700, 1)])
def test_attn_units_that_follow_each_other(B, page, window, sinks, wide):
    """Many units of many rows and a few tiles each, one after the other in a CTA."""
    lengths = [int(n) for n in rng(page).integers(200, 1500, 20)]
    check_attn(B, Cache(lengths, 8, 128, page, 15, wide=wide), [1 + r % 5 for r in range(20)], 40, True, window=window, sinks=sinks)


@gpu
@pytest.mark.parametrize("wide", [False, True])
def test_attn_rows_that_see_nothing(B, wide):
    """A length of zero, new tokens before the beginning, an empty table: 0."""
    cache = Cache([0, 3, 40], 2, 128, 16, 6, wide=wide)
    check_attn(B, cache, [2, 5, 1], 4, True)
    k, v, table, length = cache.gpu()
    q = torch.ones(3, 4, 128, dtype=BF, device="cuda")
    out = B.bl_attn_paged(q, k, v, table, ints([0, 0, 0]), ints([0, 1, 2, 3]), 1.0, out_dtype=F32)
    assert torch.equal(out, torch.zeros_like(out))


@gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_attn_scale_and_peaked_scores(B, scale, wide):
    check_attn(B, Cache([200, 31, 700], 2, 112, 16, 7, k_scale=2.0, wide=wide), [1, 3, 9], 4, True, scale=scale)


@gpu
@pytest.mark.parametrize("wide", [False, True])
def test_attn_scores_of_minus_infinity(B, wide):
    """Keys with an infinity against the query have no weight; a row with no other key gives 0."""
    cache = Cache([40, 20], 1, 128, 16, 8, wide=wide)
    q = np.abs(bf16_round(rng(1).standard_normal((2, 2, 128)).astype(np.float32))) + np.float32(0.125)
    q = bf16_round(q)
    for k, _ in cache.rows[1:]:
        k[:, :, 3] = -np.inf
    k0 = cache.rows[0][0]
    k0[5:30, :, 7] = -np.inf
    for r, n in enumerate(cache.lengths):
        for j in range(n):
            cache.k[cache.table[r, j // 16], :, j % 16] = cache.rows[r][0][j]
    kt, vt, table, length = cache.gpu()
    out = host(B.bl_attn_paged(dev(q, BF), kt, vt, table, length, ints([0, 1, 2]), 0.125, out_dtype=F32))
    assert np.all(out[1] == 0)
    keep = np.r_[0:5, 30:40]
    for h in range(2):
        ref, cond, size = R.attention_row(q[0, h], k0[keep, 0], cache.rows[0][1][keep, 0], np.ones(15, bool), 0.125)
        assert np.all(np.abs(out[0, h] - ref) <= attn_bound(ref[None], cond[None], np.array([size]), 40, 128, True)[0])


@gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("what", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("D,H", [(64, 4), (128, 4), (256, 2), (128, 12), (80, 12)])
def test_attn_infinities_stay_where_they_are_seen(B, what, D, H, wide):
    """A key or value that is not finite reaches the rows that see it and no others: later drafts, other windows, other
    requests, other heads."""
    lengths, counts = [70, 50], [6, 2]
    cache = Cache(lengths, 2, D, 16, 9, wide=wide)
    base = host(check_attn(B, cache, counts, H, True, window=20, sinks=3))
    G = H // 2
    for name, r, j, first, last in (("v", 0, 67, 3, 6), ("v", 0, 46, 0, 2), ("k", 0, 67, 3, 6), ("v", 1, 49, 7, 8), ("v", 0, 1, 0, 6), ("v", 0, 30, 0, 0)):
        c = {"k": cache.k.copy(), "v": cache.v.copy()}
        c[name][cache.table[r, j // 16], 1, j % 16, 2] = what
        q = bf16_round(1.3 * rng(H, D, 8, 0).standard_normal((8, H, D)).astype(np.float32))
        out = host(B.bl_attn_paged(dev(q, BF), dev(c["k"], BF), dev(c["v"], BF), ints(cache.table), ints(lengths), ints([0, 6, 8]), D ** -0.5,
                                   window=20, sinks=3, out_dtype=F32))
        hit = np.zeros(out.shape[:2], bool)
        hit[first:last, G:] = True
        if r == 0 and j == 46:  # the window of row t begins at 70 - 6 + t + 1 - 20 = 45 + t
            assert first == 0 and last == 2
        close = np.abs(out - base) <= 1e-4  # a tile with an infinity is added up in another order
        assert close[~hit].all(), (name, r, j)
        if name == "v":
            assert not np.isfinite(out[hit][:, 2]).any() and close[hit][:, 3:].all(), (name, r, j)
        elif not (what == -np.inf or what == np.inf):
            assert np.isnan(out[hit]).all()


@gpu
@pytest.mark.parametrize("wide", [False, True])
def test_attn_bad_pages_are_left_out(B, wide):
    cache = Cache([100, 40], 2, 128, 16, 10, wide=wide)
    q = bf16_round(rng(3).standard_normal((2, 4, 128)).astype(np.float32))
    for entry in (cache.pages, 1 << 30, -1, -(1 << 31)):
        k, v, table, length = cache.gpu()
        table[0, 2] = entry
        out = B.bl_attn_paged(dev(q, BF), k, v, table, length, ints([0, 1, 2]), 0.125, out_dtype=F32)
        assert range_error(B)
        seen = np.ones(100, bool)
        seen[32:48] = False
        for h in range(4):
            ref, cond, size = R.attention_row(q[0, h], cache.rows[0][0][:, h // 2], cache.rows[0][1][:, h // 2], seen, 0.125)
            assert np.all(np.abs(host(out)[0, h] - ref) <= attn_bound(ref[None], cond[None], np.array([size]), 100, 128, True)[0])
    k, v, table, length = cache.gpu()
    # lengths beyond the table, negative ones, starts outside the rows or falling
    for length, start in (([1 << 20, 40], [0, 1, 2]), ([-3, 40], [0, 1, 2]), ([100, 40], [0, 1, 9]), ([100, 40], [-2, 1, 2]), ([100, 40], [0, 2, 1]),
                          ([100, 40], [0, 1 << 31 - 1, 2])):
        out = B.bl_attn_paged(dev(q, BF), k, v, table, ints(length), ints(start), 0.125, out_dtype=F32)
        assert range_error(B), (length, start)


@gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("H,Hk,counts", [(10, 2, [1, 1, 1]), (16, 2, [3, 5, 1])])
def test_attn_repeats_bit_for_bit_and_shares_a_workspace(B, H, Hk, counts, wide):
    cache = Cache([900, 17, 2000], Hk, 128, 16, 11, wide=wide)
    ws = B.attn_paged_workspace(sum(counts), H, Hk, 128)
    ws.fill_(255)
    first = check_attn(B, cache, counts, H, False, workspace=ws)
    other = Cache([30, 1200], Hk, 128, 16, 12, wide=wide)
    check_attn(B, other, [1, 1], H, True, workspace=ws)
    again = check_attn(B, cache, counts, H, False, workspace=ws)
    assert torch.equal(first, again)


@gpu
def test_attn_offsets_beyond_32_bits(B):
    """A cache of more than 2^32 elements; the request lies at its end and its beginning."""
    page, Hk, D = 64, 4, 128
    pages = (1 << 32) // (Hk * page * D) + 9
    small = Cache([150], Hk, D, page, 13)
    k, v = (torch.empty((pages, Hk, page, D), dtype=BF, device="cuda") for _ in range(2))
    place = [pages - 1, 0, pages - 2]
    for c, s in ((k, small.k), (v, small.v)):
        for i, p in enumerate(place):
            c[p] = dev(s[small.table[0, i]], BF)
    q = bf16_round(rng(4).standard_normal((1, 8, D)).astype(np.float32))
    ref, cond, size = attn_ref(q, small, [1], 0.1, 0, 0)
    for table in (place, place + [-1] * 61):
        out = B.bl_attn_paged(dev(q, BF), k, v, ints([table]), ints([150]), ints([0, 1]), 0.1, out_dtype=F32)
        assert np.all(np.abs(host(out) - ref) <= attn_bound(ref, cond, size, 150, D, True))
    x = rng(5).standard_normal((1, (8 + 2 * Hk) * D)).astype(np.float32)
    one, none = np.ones((1, D // 2), np.float32), np.zeros((1, D // 2), np.float32)
    at = (pages - 1) * page + 5
    B.bl_rope_append(dev(x), dev(one), dev(none), ints([0]), ints([at]), k, v, 8)
    rows = bf16_round(x).reshape(1, -1, D)[0, 8:]
    assert np.array_equal(host(k[pages - 1, :, 5]), rows[:Hk]) and np.array_equal(host(v[pages - 1, :, 5]), rows[Hk:])


# ---------------------------------------------------------------------------
# verification: exact, where no decision lies within the stated accuracy of going
# the other way: 2^-19 of p for a test of acceptance (p and q are within 2^-20);
# 2^-20 of the mass for the token (weights within 2^-21, in a sum and in the total)
# ---------------------------------------------------------------------------

def verify_inputs(counts, V, bf16, model, seed, t=None):
    g = rng(len(counts), V, seed)
    M = sum(counts)
    logits = (2.5 * g.standard_normal((M, V))).astype(np.float32)
    logits[np.arange(M)[:, None], g.integers(0, V, (M, 5))] += 6
    drafts = (logits + 0.8 * g.standard_normal((M, V))).astype(np.float32) if model else None
    if bf16:
        logits, drafts = bf16_round(logits), bf16_round(drafts) if model else None
    t = g.uniform(0.4, 1.6, len(counts)).astype(np.float32) if t is None else np.full(len(counts), t, np.float32)
    each = np.repeat(t, counts)
    token = g.integers(0, V, M)
    for i in range(M - 1):
        w = R.weights((drafts if model else logits)[i], each[i])
        token[i + 1] = g.choice(V, p=w / w.sum())
    return logits, drafts, token, g.random(M).astype(np.float32), g.random(len(counts)).astype(np.float32), t


def check_verify(B, counts, v, bf16, padding=0, clear=0.9, **kw):
    logits, drafts, token, u, us, t = v
    M, V = logits.shape
    start = np.concatenate([[0], np.cumsum(counts)])
    x = BF if bf16 else F32

    def pad(a, fill=np.nan):
        return np.concatenate([a, np.full((padding, *a.shape[1:]), fill, a.dtype)])
    got = B.bl_verify(dev(pad(logits), x), ints(pad(token, 3)), ints(start), dev(pad(u)), dev(us), temperature=None if t is None else dev(t),
                      draft_logits=None if drafts is None else dev(pad(drafts), x), **kw)
    accepted, token_out = (a.cpu().numpy() for a in got)
    sure = 0
    for r, (a, b) in enumerate(zip(start[:-1], start[1:])):
        if a == b:
            assert (accepted[r], token_out[r]) == (0, -1)
            continue
        n, x, margin, w = R.verify(logits[a:b], None if drafts is None else drafts[a:b], token[a:b], u[a:b], us[r], 1.0 if t is None else t[r])
        if margin > 2.0 ** -19:
            assert accepted[r] == n, (r, margin)
            sure += 1
            got_x = token_out[r]
            assert (got_x < 0) == (x < 0)
            if x >= 0:  # the number lies in the token's stretch of the mass, up to the weights' accuracy
                mass = np.cumsum(w) / w.sum()
                u1 = min(float(us[r]), float(np.float32(0.99999994)))
                assert w[got_x] > 0 and mass[got_x] - w[got_x] / w.sum() - 2.0 ** -20 <= u1 <= mass[got_x] + 2.0 ** -20, r
                live = mass[:-1][w[:-1] > 0]
                if u1 == 0 or np.abs(live - u1).min(initial=1.0) > 2.0 ** -20:
                    assert got_x == x, r
    assert sure >= clear * sum(c > 0 for c in counts)
    return got


@gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("model", [True, False])
@pytest.mark.parametrize("counts,V", [([5], 1000), ([1], 7), ([2], 1), ([1, 2, 3, 4, 5, 6], 4099), ([3, 1, 0, 9], 513), ([4] * 40, 3001), ([2, 5], 50000),
                                      ([1] * 9, 20011), ([30], 300)])
def test_verify(B, counts, V, model, bf16):
    check_verify(B, counts, verify_inputs(counts, V, bf16, model, 1), bf16, padding=2)


@gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("model", [True, False])
def test_verify_largest_vocabularies(B, model, bf16):
    counts = [3, 1]
    check_verify(B, counts, verify_inputs(counts, 248320, bf16, model, 2), bf16)
    check_verify(B, counts, verify_inputs(counts, 524288, bf16, model, 3), bf16)


@gpu
@pytest.mark.parametrize("model", [True, False])
def test_verify_greedy_and_flat(B, model):
    """Temperature 0 accepts what is the largest logit; ties share; a large temperature makes all weights alike."""
    counts = [3, 4, 1, 2]
    for t in (0.0, 1e30, np.inf, np.nan, 0.02):
        v = verify_inputs(counts, 2000, True, model, 4, t=0.0 if not t >= 1e-5 else min(t, 1e30))
        check_verify(B, counts, (*v[:5], np.full(4, t, np.float32)), True)
    v = verify_inputs(counts, 2000, True, model, 5)
    check_verify(B, counts, (*v[:5], None), True)


@gpu
def test_verify_ties_and_ends_of_the_numbers(B):
    l = np.zeros((4, 8), np.float32)
    l[0, [2, 5]] = 3
    t = np.zeros(2, np.float32)
    for u, x, want in ((0.49, 2, 1), (0.5, 2, 0), (0.0, 5, 1), (0.0, 3, 0), (np.nan, 5, 1), (-1.0, 2, 1), (2.0, 2, 0)):
        v = (l, None, np.array([0, x, 0, 0]), np.float32([u, 0, 0, 0]), np.float32([0.0, 1.0]), t)
        a, n = (o.tolist() for o in check_verify(B, [2, 2], v, False))  # 1.0 lies at the last border
        assert a[0] == want
        # row 1 and 3 are flat: the first and the last token; a refused 2 leaves 5, a refused 3 both
        assert n[1] == 7 and n[0] == (0 if want else 5 if x == 2 else 2)


@gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("model", [True, False])
def test_verify_infinities_and_masks(B, model, bf16):
    counts, V = [3, 2, 2, 3, 2, 1], 3000
    logits, drafts, token, u, us, t = verify_inputs(counts, V, bf16, model, 6)
    logits[0, : V // 2] = -np.inf                     # a grammar's mask
    logits[1, 17] = np.nan
    logits[3] = -np.inf                               # nothing is left: refused, no token
    logits[5, 40], logits[5, 41], token[6] = np.inf, np.inf, 40   # infinities share the mass
    logits[9, :] = np.finfo(np.float32).min if not bf16 else -3.3895313892515355e38
    logits[9, 100] = 0                                # masked by the type's lowest value
    logits[12] = -np.inf
    if model:
        drafts[0, V // 3:] = -np.inf
        drafts[8] = -np.inf                           # q is 0: any draft that p has is accepted
        drafts[9, 5] = np.nan
    check_verify(B, counts, (logits, drafts, token, u, us, t), bf16)


@gpu
def test_verify_drafts_out_of_range(B):
    counts = [3, 3, 2]
    v = verify_inputs(counts, 500, True, True, 7)
    for x in (-1, 500, 1 << 30):
        v[2][4] = x
        check_verify(B, counts, v, True)
        assert range_error(B)
    v[2][4] = 0
    logits, drafts, token, u, us, t = v
    args = (dev(logits, BF), ints(token), None, dev(u), dev(us))
    for start in ([0, 3, 6, 9], [-1, 3, 6, 8], [0, 5, 3, 8]):
        B.bl_verify(*args[:2], ints(start), *args[3:], temperature=dev(t))
        assert range_error(B)


@gpu
def test_verify_equal_distributions_accept_and_certain_drafts(B):
    """p = q accepts for every u; q(x) = 1 with p(x) = 1 too; equal rows whose draft is impossible under both refuse and draw from p."""
    v = list(verify_inputs([4] * 8, 1000, True, True, 8))
    v[1] = v[0].copy()
    v[3] = np.full(32, 0.9999, np.float32)
    got = check_verify(B, [4] * 8, tuple(v), True)
    assert got[0].tolist() == [3] * 8
    l = np.full((2, 64), -np.inf, np.float32)
    l[:, 9] = 1
    l[:, 20] = 1
    for x, a in ((9, 1), (3, 0)):
        out = check_verify(B, [2], (l, l.copy(), np.array([0, x]), np.float32([0.3, 0]), np.float32([0.7]), None), False)
        assert out[0].item() == a and out[1].item() == 20


@gpu
def test_verify_distribution(B):
    """Over many draws accepted and resampled tokens follow p (the point of the procedure): 20000 requests of one draft."""
    V, n = 12, 20000
    g = rng(99)
    l, d = (g.standard_normal(V).astype(np.float32) for _ in range(2))
    q = R.weights(d, 1.0)
    x = g.choice(V, n, p=q / q.sum())
    token = np.zeros(2 * n, int)
    token[1::2] = x
    a, t = B.bl_verify(dev(np.tile(l, (2 * n, 1))), ints(token), ints(np.arange(0, 2 * n + 1, 2)), dev(g.random(2 * n).astype(np.float32)),
                       dev(g.random(n).astype(np.float32)), draft_logits=dev(np.tile(d, (2 * n, 1))))
    a, t = a.cpu().numpy(), t.cpu().numpy()
    first = np.where(a == 1, x, t)
    p = R.weights(l, 1.0)
    p /= p.sum()
    # a count of n p has a deviation of sqrt(n p (1 - p)); six of them
    assert np.all(np.abs(np.bincount(first, minlength=V) - n * p) <= 6 * np.sqrt(n * p * (1 - p)))


# ---------------------------------------------------------------------------
# streams, graphs, and the operators together
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("D,wide", [(64, False), (128, False), (128, True)])
def test_calls_on_another_stream_and_captured(B, D, wide):
    """The same results on a side stream, and from a graph that is replayed with other contents in its tensors."""
    H, Hk, page = 8, 2, 16
    cache = Cache([100, 33, 260], Hk, D, page, 14, wide=wide)
    k, v, table, length = cache.gpu()
    q = torch.randn(5, H, D, device="cuda").to(BF)
    start = ints([0, 1, 3, 5])
    ws, out = B.attn_paged_workspace(5, H, Hk, D), torch.empty(5, H, D, dtype=BF, device="cuda")
    vi = verify_inputs([1, 2, 2], 3000, True, True, 9)
    vt = [dev(vi[0], BF), ints(vi[2]), start, dev(vi[3]), dev(vi[4])]
    vw, acc, nxt = B.verify_workspace(5), torch.empty(3, dtype=I32, device="cuda"), torch.empty(3, dtype=I32, device="cuda")

    def step(stream=None):
        B.bl_attn_paged(q, k, v, table, length, start, 0.125, out=out, workspace=ws, stream=stream)
        B.bl_verify(*vt, draft_logits=dl, temperature=tt, accepted=acc, next_token=nxt, workspace=vw, stream=stream)
    dl, tt = dev(vi[1], BF), dev(vi[5])
    step()
    want = [t.clone() for t in (out, acc, nxt)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in (out, acc, nxt):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (out, acc, nxt)))
    for overlap in (False, True):
        B.set_overlap(overlap)
        graphs = []
        for _ in range(2):  # two graphs that share the workspaces
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
                step()
            graphs.append(g)
        for lengths in ([100, 33, 260], [90, 30, 7], [100, 33, 260]):
            length.copy_(ints(lengths))
            for g in graphs:
                out.zero_()
                g.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in (out, acc, nxt)]
            B.set_overlap(False)
            step()
            assert all(torch.equal(a, b) for a, b in zip(got, (out, acc, nxt))), lengths
            B.set_overlap(overlap)
        B.set_overlap(False)


@gpu
def test_steps_of_a_paged_cache_together(B):
    """Maps, rotary rows, attention and verification over several steps with refused drafts and ended requests, against
    attention over the tokens kept in order on the host."""
    requests, H, Hk, D, page, W, pages, V = 5, 4, 2, 64, 8, 12, 40, 400
    g = rng(21)
    angle = np.arange(W * page)[:, None] * 100.0 ** -(np.arange(D // 2) * 2 / D)
    cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    k, v = (torch.full((pages, Hk, page, D), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    length, owned, fc = ints(np.zeros(requests)), ints(np.zeros(requests)), ints([pages])
    table, free = ints(np.full((requests, W), -1)), ints(g.permutation(pages))
    rows = [([], []) for _ in range(requests)]
    for step in range(12):
        count = g.integers(1, 6, requests) if step else g.integers(1, 20, requests)
        if step in (4, 8):
            count[step % requests] = -1
            rows[step % requests] = ([], [])
        n = np.maximum(count, 0)
        M = int(n.sum())
        pad = 3
        start, position, slot, length, owned, fc = B.bl_page_map(length, ints(count), table, owned, free, fc, page, M + pad)
        x = g.standard_normal((M + pad, (H + 2 * Hk) * D)).astype(np.float32)
        q = B.bl_rope_append(dev(x), dev(cos), dev(sin), position, slot, k, v, H)
        out = B.bl_attn_paged(q, k, v, table, length, start, D ** -0.5, out_dtype=F32)
        # the host's copy: k as the library rounded it (checked on its own elsewhere)
        heads, at = x.reshape(M + pad, -1, D), start.cpu().numpy()
        lens = length.cpu().numpy()
        kt, _ = R.rope(heads[:M, H:H + Hk], cos, sin, position.cpu().numpy()[:M])
        kt = bf16_round(kt.astype(np.float32))
        for r in range(requests):
            for i in range(at[r], at[r + 1]):
                rows[r][0].append(kt[i])
                rows[r][1].append(bf16_round(heads[i, H + Hk:]))
            assert len(rows[r][0]) == lens[r]
            for t in range(n[r]):
                seen = R.seen_by(lens[r] - n[r] + t, lens[r], 0, 0)
                for h in range(H):
                    ref, cond, size = R.attention_row(host(q)[at[r] + t, h], np.array(rows[r][0])[:, h // 2], np.array(rows[r][1])[:, h // 2], seen, D ** -0.5)
                    # a key next to a rounding border may be stored a step off: 2^-7 of a few products
                    tol = attn_bound(ref[None], cond[None], np.array([size]), 100, D, True)[0] + 2.0 ** -7 * size / 8 * cond
                    assert np.all(np.abs(host(out)[at[r] + t, h] - ref) <= tol), (step, r, t, h)
        logits = dev((3 * g.standard_normal((M + pad, V))).astype(np.float32), BF)
        token = logits.float().argmax(1).roll(1).to(I32)  # drafts: the largest logit of the row before
        token[g.integers(0, M, M // 2)] = 0
        acc, nxt = B.bl_verify(logits, token, start, dev(g.random(M + pad).astype(np.float32)), dev(g.random(requests).astype(np.float32)))
        acc = acc.cpu().numpy()
        assert np.all((acc >= 0) & (acc <= np.maximum(n - 1, 0))) and np.all((nxt.cpu().numpy() >= 0) == (n > 0))
        gone = np.maximum(n - 1, 0) - acc
        length = length - ints(gone)
        for r in range(requests):
            for lst in rows[r]:
                del lst[len(lst) - gone[r]:]


@gpu
def test_memory_of_calls_on_another_stream(B):
    """What a call allocates is not handed out again to the current stream while the call waits on its own."""
    H, Hk, D = 40, 8, 128
    cache = Cache([900, 1300], Hk, D, 16, 18, wide=True)
    k, v, table, length = cache.gpu()
    q, start = torch.randn(9, H, D, device="cuda").to(BF), ints([0, 5, 9])
    vi = verify_inputs([5, 4], 40000, True, True, 10)
    vt = [dev(vi[0], BF), ints(vi[2]), start, dev(vi[3]), dev(vi[4])]
    dl, tt = dev(vi[1], BF), dev(vi[5])
    side = torch.cuda.Stream()
    want = (B.bl_attn_paged(q, k, v, table, length, start, D ** -0.5), *B.bl_verify(*vt, draft_logits=dl, temperature=tt))
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # 10 ms
        got = (B.bl_attn_paged(q, k, v, table, length, start, D ** -0.5, stream=side), *B.bl_verify(*vt, draft_logits=dl, temperature=tt, stream=side))
        sizes = (B.attn_paged_workspace(9, H, Hk, D).numel(), B.verify_workspace(9).numel(), 2 * 9 * H * D, 8)
        kept = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert all(bool((t == 0).all()) for t in kept)


@gpu
def test_two_calls_at_once_and_a_cache_that_is_shared(B):
    """Calls on two streams with a workspace each; requests whose tables hold the same pages (a common prefix)."""
    H, Hk, D, page = 40, 8, 128, 16
    cache = Cache([640, 1000, 333], Hk, D, page, 16, wide=True)
    cache.table[1, :20] = cache.table[0, :20]  # 320 tokens
    for i in range(2):
        cache.rows[1][i][:320] = cache.rows[0][i][:320]
    want = [check_attn(B, cache, counts, H, True) for counts in ([5, 4, 3], [1, 1, 1])]
    k, v, table, length = cache.gpu()
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = []
    for counts, w in zip(([5, 4, 3], [1, 1, 1]), want):
        q = dev(bf16_round(1.3 * rng(H, D, sum(counts), 0).standard_normal((sum(counts), H, D)).astype(np.float32)), BF)
        work.append((q, ints(np.concatenate([[0], np.cumsum(counts)])), torch.empty(sum(counts), H, D, device="cuda"),
                     B.attn_paged_workspace(sum(counts), H, Hk, D)))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (q, start, out, ws) in zip(streams, work):
            B.bl_attn_paged(q, k, v, table, length, start, D ** -0.5, out=out, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for w, (_, _, out, _) in zip(want, work):
        assert torch.equal(out, w[:len(out)])


@gpu
@pytest.mark.parametrize("requests,drafts", [(1, 3), (5, 0), (7, 4)])
def test_example_paged_step(B, requests, drafts):
    """The example runs, eagerly and captured, with the same tokens; lengths and pages add up."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_step.py")
    spec = importlib.util.spec_from_file_location("paged_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    model = example.Model(5001, heads=4, kv_heads=2, dim=128, positions=512)
    g = torch.Generator(device="cuda").manual_seed(3)
    tokens = torch.randint(0, 5001, (requests, 20), generator=g, device="cuda", dtype=I32)
    numbers = [(torch.rand(requests * (drafts + 1), generator=g, device="cuda"), torch.rand(requests, generator=g, device="cuda")) for _ in range(6)]
    temperature = torch.full((requests,), 0.8, device="cuda")
    u, us = (torch.empty_like(t) for t in numbers[0])
    runs = []
    for captured in (False, True):
        req = example.Requests(model, requests, 100)
        example.prompt(model, req, tokens)
        u.copy_(numbers[0][0]), us.copy_(numbers[0][1])
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                example.step(model, req, drafts, u, us, temperature)
        seen = []
        for n in numbers:
            u.copy_(n[0]), us.copy_(n[1])
            graph.replay() if captured else example.step(model, req, drafts, u, us, temperature)
            seen.append((req.accepted.clone(), req.next.clone()))
        runs.append(seen)
        accepted, nxt = (torch.stack(t) for t in zip(*seen))
        assert bool(((accepted >= 0) & (accepted <= drafts) & (nxt >= 0) & (nxt < 5001)).all())
        assert torch.equal(req.length, 19 + (accepted + 1).sum(0).to(I32))
        assert int(req.free_count) + int(req.owned.sum()) == len(req.free)
        assert bool((req.owned * req.page >= req.length).all())
    assert all(torch.equal(x, y) for a, b in zip(*runs) for x, y in zip(a, b))
