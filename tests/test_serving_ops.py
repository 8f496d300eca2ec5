"""The operators around the products (bl_rmsnorm_quant_int8, bl_lora_add, bl_sample) against 64-bit forms.

Codes, scales and tokens are compared exactly; the tolerances of the other
outputs are derived beside each test."""
import ctypes

import numpy as np
import pytest
import torch

import serving_ref as R

gpu = pytest.mark.gpu
BF16_HALF_STEP, F32_HALF_STEP = 2.0 ** -8, 2.0 ** -24


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


def host(t):
    return t.float().cpu().numpy()


def shifted(t, n):
    """The same values in a tensor that starts n elements into an allocation."""
    buf = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)
    out = buf[n:].view(t.shape)
    out.copy_(t)
    return out


# ---------------------------------------------------------------------------
# refusals (host checks: no GPU)
# ---------------------------------------------------------------------------

def test_refusals_without_gpu(B):
    L = B.lib()
    P = ctypes.c_void_p
    a, o1, o2, o8 = P(1 << 14), P((1 << 14) + 1), P((1 << 14) + 2), P((1 << 14) + 8)
    other = P(1 << 15)
    NULL, SHAPE, AL, DT, UN = B.BL_ERR_NULL, B.BL_ERR_SHAPE, B.BL_ERR_ALIGN, B.BL_ERR_DTYPE, B.BL_ERR_UNSUPPORTED
    F, H = B.BL_F32, B.BL_BF16
    n, l, s = L.bl_rmsnorm_quant_int8, L.bl_lora_add, L.bl_sample
    cases = [
        (n, (None, None, F, a, 1e-5, 1, 8, None, None, a, a, None), NULL),
        (n, (a, None, F, None, 1e-5, 1, 8, None, None, a, a, None), NULL),
        (n, (a, None, F, a, 1e-5, 1, 8, None, None, None, a, None), NULL),
        (n, (a, None, F, a, 1e-5, 1, 8, None, None, a, None, None), NULL),
        (n, (a, a, F, a, 1e-5, 1, 8, None, None, a, a, None), NULL),          # a residual without h
        (n, (a, None, 2, a, 1e-5, 1, 8, None, None, a, a, None), DT),
        (n, (a, None, F, a, 1e-5, 0, 8, None, None, a, a, None), SHAPE),
        (n, (a, None, F, a, 1e-5, 1, 0, None, None, a, a, None), SHAPE),
        (n, (a, None, F, a, 1e-5, 1 << 31, 8, None, None, a, a, None), SHAPE),
        (n, (a, None, F, a, -1.0, 1, 8, None, None, a, a, None), SHAPE),
        (n, (a, None, F, a, float("nan"), 1, 8, None, None, a, a, None), SHAPE),
        (n, (a, None, F, a, 1e-5, 1, 8, other, other, a, a, None), SHAPE),    # y is h
        (n, (o2, None, F, a, 1e-5, 1, 8, None, None, a, a, None), AL),
        (n, (a, None, H, o1, 1e-5, 1, 8, None, None, a, a, None), AL),
        (n, (a, o2, F, a, 1e-5, 1, 8, a, None, a, a, None), AL),
        (n, (a, None, F, a, 1e-5, 1, 8, o2, None, a, a, None), AL),
        (n, (a, None, F, a, 1e-5, 1, 8, None, o2, a, a, None), AL),
        (n, (a, None, F, a, 1e-5, 1, 8, None, None, a, o2, None), AL),
        (l, (None, F, a, a, a, a, a, a, F, 1, 4, 8, 1, 8, None), NULL),
        (l, (a, F, None, a, a, a, a, a, F, 1, 4, 8, 1, 8, None), NULL),
        (l, (a, F, a, a, a, None, a, a, F, 1, 4, 8, 1, 8, None), NULL),
        (l, (a, F, a, a, a, a, None, a, F, 1, 4, 8, 1, 8, None), NULL),
        (l, (a, 2, a, a, a, a, a, a, F, 1, 4, 8, 1, 8, None), DT),
        (l, (a, F, a, a, a, a, a, a, 5, 1, 4, 8, 1, 8, None), DT),
        (l, (a, F, a, a, a, a, a, a, F, 0, 4, 8, 1, 8, None), SHAPE),
        (l, (a, F, a, a, a, a, a, a, F, 1, 0, 8, 1, 8, None), SHAPE),
        (l, (a, F, a, a, a, a, a, a, F, 1, 4, 12, 1, 8, None), SHAPE),
        (l, (a, F, a, a, a, a, a, a, F, 1, 4, 8, 0, 8, None), SHAPE),
        (l, (a, F, a, a, a, a, a, a, F, 1, 4, 8, 1, 0, None), SHAPE),
        (l, (a, F, a, a, a, a, a, a, F, 1, 4, 8, 1, 12, None), SHAPE),
        (l, (a, F, a, a, a, a, a, a, F, 1, 4, 8, 1, 136, None), UN),
        (l, (a, F, a, a, a, a, a, a, F, 1, 4, 65544, 1, 8, None), UN),
        (l, (o8, F, a, a, a, a, a, a, F, 1, 4, 8, 1, 8, None), AL),
        (l, (a, F, a, o8, a, a, a, a, F, 1, 4, 8, 1, 8, None), AL),
        (l, (a, F, a, a, o8, a, a, a, F, 1, 4, 8, 1, 8, None), AL),
        (l, (a, F, o2, a, a, a, a, a, F, 1, 4, 8, 1, 8, None), AL),
        (l, (a, F, a, a, a, a, o2, a, F, 1, 4, 8, 1, 8, None), AL),
        (l, (a, F, a, a, a, a, a, o1, H, 1, 4, 8, 1, 8, None), AL),
        (s, (None, F, None, None, None, None, a, 1, 8, a, None, None), NULL),
        (s, (a, F, None, None, None, None, None, 1, 8, a, None, None), NULL),
        (s, (a, F, None, None, None, None, a, 1, 8, None, None, None), NULL),
        (s, (a, 3, None, None, None, None, a, 1, 8, a, None, None), DT),
        (s, (a, F, None, None, None, None, a, 0, 8, a, None, None), SHAPE),
        (s, (a, F, None, None, None, None, a, 1, 0, a, None, None), SHAPE),
        (s, (a, F, None, None, None, None, a, 1, 524289, a, None, None), UN),
        (s, (o2, F, None, None, None, None, a, 1, 8, a, None, None), AL),
        (s, (o1, H, None, None, None, None, a, 1, 8, a, None, None), AL),
        (s, (a, F, o2, None, None, None, a, 1, 8, a, None, None), AL),
        (s, (a, F, None, o2, None, None, a, 1, 8, a, None, None), AL),
        (s, (a, F, None, None, o2, None, a, 1, 8, a, None, None), AL),
        (s, (a, F, None, None, None, o2, a, 1, 8, a, None, None), AL),
        (s, (a, F, None, None, None, None, o2, 1, 8, a, None, None), AL),
        (s, (a, F, None, None, None, None, a, 1, 8, o2, None, None), AL),
        (s, (a, F, None, None, None, None, a, 1, 8, a, o2, None), AL),
    ]
    for fn, args, want in cases:
        got = fn(*args)
        assert got == want, (fn.__name__, args, B.status_name(got), B.status_name(want))
        assert fn.__name__.encode() in L.bl_last_error()


def test_binding_refuses_host_tensors(B):
    x, w = torch.zeros(2, 8), torch.ones(8)
    for call in (lambda: B.bl_rmsnorm_quant_int8(x, w), lambda: B.bl_sample(x, torch.zeros(2)),
                 lambda: B.bl_lora_add(x, torch.zeros(2, dtype=torch.int32), x, x, w, x)):
        with pytest.raises(TypeError):
            call()


def test_reference_rounding_and_order():
    """The 64-bit forms on hand-worked values."""
    assert R.bf16_round(np.float32(1 + 2.0 ** -8)) == 1.0 and R.bf16_round(np.float32(1 + 3 * 2.0 ** -8)) == 1 + 2.0 ** -6
    q, s, h, y, _ = R.rmsnorm_quant(np.float32([[3, -1, 1, 1]]), None, np.float32([1, 1, 2, 1]), 1.0, False)
    assert y.tolist() == [[1.5, -0.5, 1.0, 0.5]] and q.tolist() == [[127, -42, 85, 42]] and s[0] == np.float32(1.5) / 127
    l = np.float32([1, 2, 2, -np.inf, np.nan, 0])  # order: 1, 2, 0, 5; the others have no weight
    assert [R.sample_row(l, u, p=0.0)[0] for u in (0, 0.9)] == [1, 1]
    assert [R.sample_row(l, u, k=2)[0] for u in (0, 0.49, 0.5, 1)] == [1, 1, 2, 2]
    assert R.sample_row(l, 0.999999)[0] == 5 and R.sample_row(l, 0.3, t=0.0)[0] == 1
    assert R.sample_row(np.float32([-np.inf, np.nan]), 0.5)[:2] == (-1, 0.0)


# ---------------------------------------------------------------------------
# norm with codes: bit for bit (the factor of a row is determined unless its
# 64-bit value lies within 2^-40 of a rounding border, which the seeds avoid)
# ---------------------------------------------------------------------------

def norm_inputs(M, K, bf16, residual, seed):
    g = rng(M, K, seed)
    x = g.standard_normal((M, K)).astype(np.float32) * g.uniform(0.01, 30, (M, 1)).astype(np.float32)
    x[:, :: 97] *= 40
    if M > 2:
        x[1] = 0
        x[2] = np.float32(2.0 ** -30) * np.sign(x[2])
    r = g.standard_normal((M, K)).astype(np.float32) * 5 if residual else None
    w = (1 + 0.3 * g.standard_normal(K)).astype(np.float32)
    if bf16:
        x, w, r = R.bf16_round(x), R.bf16_round(w), R.bf16_round(r) if residual else None
    return x, r, w


def check_norm(B, x, r, w, bf16, eps, place=lambda t: t, **out):
    t = torch.bfloat16 if bf16 else torch.float32
    up = lambda v: None if v is None else place(dev(v, t))  # noqa: E731
    q, s, h, y = B.bl_rmsnorm_quant_int8(up(x), up(w), eps, residual=up(r), y=True, **out)
    rq, rs, rh, ry, clear = R.rmsnorm_quant(x, r, w, eps, bf16)
    assert clear.all()
    if r is not None:
        assert np.array_equal(host(h), rh)
    else:
        assert h is None
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(host(y), ry)


@gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 7), (3, 8), (5, 129), (4, 1000), (1, 2560), (37, 2561), (130, 2560), (9, 5120),
                                 (3, 6912), (2, 13824), (2, 32768), (2, 32776), (1, 70001)])
def test_norm_codes_bit_exact(B, M, K, residual, bf16):
    check_norm(B, *norm_inputs(M, K, bf16, residual, 1), bf16, 1e-5)


@gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 3.0])
def test_norm_eps_and_alignment(B, bf16, eps):
    x, r, w = norm_inputs(6, 1024, bf16, True, 2)
    check_norm(B, x, r, w, bf16, eps)
    check_norm(B, x, r, w, bf16, eps, place=lambda t: shifted(t, 1))
    q = torch.empty(6 * 1024 + 3, dtype=torch.int8, device="cuda")[3:].view(6, 1024)
    check_norm(B, x, r, w, bf16, eps, q=q)


@gpu
@pytest.mark.parametrize("K", [2560, 2563])
def test_norm_in_place_and_repeated(B, K):
    """h in the residual's or x's place, y in x's place; the same bits on every call."""
    x, r, w = norm_inputs(20, K, True, True, 3)
    t = torch.bfloat16
    want = B.bl_rmsnorm_quant_int8(dev(x, t), dev(w, t), residual=dev(r, t), y=True)
    for _ in range(3):
        xg, rg = dev(x, t), dev(r, t)
        got = B.bl_rmsnorm_quant_int8(xg, dev(w, t), residual=rg, h=rg, y=xg)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        xg, rg = dev(x, t), dev(r, t)
        got = B.bl_rmsnorm_quant_int8(xg, dev(w, t), residual=rg, h=xg, y=rg)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    plain = B.bl_rmsnorm_quant_int8(want[2], dev(w, t), y=True)  # the stored h, without a residual
    assert torch.equal(plain[0], want[0]) and torch.equal(plain[1], want[1]) and torch.equal(plain[3], want[3])


@gpu
def test_norm_infinite_row_stays_in_its_row(B):
    x, r, w = norm_inputs(8, 640, True, True, 4)
    t = torch.bfloat16
    want = B.bl_rmsnorm_quant_int8(dev(x, t), dev(w, t), residual=dev(r, t), y=True)
    x[3, 5], x[3, 7] = np.inf, np.nan
    got = B.bl_rmsnorm_quant_int8(dev(x, t), dev(w, t), residual=dev(r, t), y=True)
    rest = [0, 1, 2, 4, 5, 6, 7]
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip(want, got))


# ---------------------------------------------------------------------------
# low-rank adapters.  The worst case of fp32 sums over K and then rank terms
# is (K + rank + 8) 2^-24 of the sum of absolute products; a bf16 output adds
# half a step, and the rank values may be carried in 16 bits for it (2^-16).
# In the 2-norm the errors add up like independent ones: 1e-6 of the
# condition's size covers fp32 outputs, half a step of the values bf16 ones.
# ---------------------------------------------------------------------------

def lora_inputs(M, N, K, rank, adapters, xb, yb, seed, index=None):
    g = rng(M, N, K, rank, seed)
    x = g.standard_normal((M, K)).astype(np.float32)
    a = R.bf16_round(g.standard_normal((adapters, rank, K)) / np.sqrt(K))
    b = R.bf16_round(g.standard_normal((adapters, N, rank)) * 0.1)
    scale = g.uniform(0.25, 4, adapters).astype(np.float32)
    base = g.standard_normal((M, N)).astype(np.float32)
    if index is None:
        index = g.integers(-1, adapters, M)
    return (R.bf16_round(x) if xb else x, np.asarray(index, np.int32), a, b, scale, R.bf16_round(base) if yb else base)


def run_lora(B, v, xb, yb, **kw):
    x, index, a, b, scale, base = v
    bf, f = torch.bfloat16, torch.float32
    return B.bl_lora_add(dev(x, bf if xb else f), dev(index), dev(a, bf), dev(b, bf), dev(scale), dev(base, bf if yb else f),
                         **kw)


def check_lora(y, v, yb):
    ref, cond = R.lora_add(*v)
    K, rank = v[2].shape[2], v[2].shape[1]
    err = np.abs(host(y).astype(np.float64) - ref)
    bound = (K + rank + 8) * 2.0 ** -24 * cond + (BF16_HALF_STEP if yb else F32_HALF_STEP) * np.abs(ref)
    assert np.all(err <= bound + (2.0 ** -16 * cond if yb else 0)), float((err / bound).max())
    norm = np.linalg.norm
    assert norm(err) <= (BF16_HALF_STEP if yb else F32_HALF_STEP) * norm(ref) + 1e-6 * norm(cond)
    none = v[1] < 0
    assert np.array_equal(host(y)[none], v[5][none])  # without an adapter the base passes through


@gpu
@pytest.mark.parametrize("xb,yb", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("M,N,K,rank,adapters", [
    (1, 1, 8, 8, 1), (1, 6912, 2560, 16, 3), (2, 33, 264, 24, 2), (7, 129, 1000, 40, 3), (9, 2560, 6912, 64, 4),
    (64, 515, 512, 32, 40), (33, 257, 2560, 128, 5), (65, 100, 136, 8, 64)])
def test_lora_scattered_tokens(B, M, N, K, rank, adapters, xb, yb):
    v = lora_inputs(M, N, K, rank, adapters, xb, yb, 1)
    check_lora(run_lora(B, v, xb, yb), v, yb)


@gpu
@pytest.mark.parametrize("xb,yb", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("N,K,rank,lengths", [
    (300, 512, 16, [300]), (257, 264, 64, [1, 127, 128, 129, 5]), (128, 1024, 128, [64, 17, 200, 16, 15, 1, 90]),
    (1000, 2560, 24, [511, 1, 1, 1, 2, 30]), (96, 72, 8, [1000, 24]), (131, 640, 32, [8] * 40), (2560, 320, 96, [260])])
def test_lora_runs_of_tokens(B, N, K, rank, lengths, xb, yb):
    """Runs of tokens of one request, some requests without an adapter, two runs of one adapter apart."""
    index = np.repeat([[0, 2, -1, 1, 0, 3, -1][i % 7] for i in range(len(lengths))], lengths)
    v = lora_inputs(len(index), N, K, rank, 4, xb, yb, 2, index)
    check_lora(run_lora(B, v, xb, yb), v, yb)


@gpu
@pytest.mark.parametrize("M", [3, 200])
def test_lora_in_place_repeated_and_without_adapters(B, M):
    v = lora_inputs(M, 389, 512, 16, 4, True, True, 3)
    want = run_lora(B, v, True, True)
    x, index, a, b, scale, base = v
    bf = torch.bfloat16
    for _ in range(3):
        y = dev(base, bf)
        got = B.bl_lora_add(dev(x, bf), dev(index), dev(a, bf), dev(b, bf), dev(scale), y, y=y)
        assert got is y and torch.equal(got, want)
    y = B.bl_lora_add(dev(x, bf), dev(np.full(M, -1, np.int32)), dev(a, bf), dev(b, bf), dev(scale), dev(base, bf))
    assert np.array_equal(host(y), base)
    # base and y off a 16-byte boundary
    got = B.bl_lora_add(dev(x, bf), dev(index), dev(a, bf), dev(b, bf), dev(scale), shifted(dev(base, bf), 1),
                        y=shifted(torch.zeros_like(want), 3))
    assert torch.equal(got, want)


@gpu
@pytest.mark.parametrize("M", [4, 300])
def test_lora_reports_an_adapter_out_of_range(B, M):
    index = np.arange(M) % 3
    index[M // 2] = 3
    v = lora_inputs(M, 64, 256, 8, 3, True, False, 4, index)
    y = run_lora(B, v, True, False)
    torch.cuda.synchronize()
    assert B.device_error(clear=True) == B.BL_DEVERR_RANGE
    assert np.array_equal(host(y)[M // 2], v[5][M // 2])
    v[1][M // 2] = -1
    check_lora(y, v, False)


@gpu
def test_lora_a_bad_row_stays_in_its_row(B):
    """Infinities and NaN of one token (with or without an adapter) leave the others' bits."""
    index = np.repeat([0, -1, 1], [150, 20, 60])
    v = lora_inputs(230, 200, 256, 16, 2, True, True, 5, index)
    want = run_lora(B, v, True, True)
    for bad in (3, 155, 229):
        v[0][bad, 7], v[0][bad, 9] = np.nan, np.inf
    got = run_lora(B, v, True, True)
    rest = [m for m in range(230) if m not in (3, 229)]  # 155 has no adapter: its x is not used
    assert torch.equal(got[rest], want[rest]) and bool(torch.isnan(got[3]).all())


def tile_case(lengths, N, K, rank, yb, seed):
    """Enough work and tokens for the tensor-core kernel: runs of one adapter, some of none."""
    index = np.repeat([[0, 2, -1, 1, 0, 3, -1][i % 7] for i in range(len(lengths))], lengths)
    assert len(index) * rank * (N + K) > 3e8
    return lora_inputs(len(index), N, K, rank, 4, True, yb, seed, index)


def check_lora_rows(y, v, yb, rows):
    x, index, a, b, scale, base = v
    check_lora(y[torch.from_numpy(rows).cuda()], (x[rows], index[rows], a, b, scale, base[rows]), yb)


@gpu
@pytest.mark.parametrize("yb", [True, False])
@pytest.mark.parametrize("N,K,rank,lengths", [
    (1537, 4096, 64, [1, 127, 128, 129, 5, 250, 384]), (2048, 4096, 64, [1, 127, 128, 129, 5, 250, 260]),
    (3000, 2056, 128, [64, 17, 200, 16, 15, 1, 190]), (2051, 4096, 24, [511, 1, 1, 1, 2, 30, 1600]),
    (2600, 5000, 8, [1000, 24, 4000]), (9000, 264, 96, [260, 140]), (2049, 2048, 72, [300, 300, 500]),
    (2560, 4096, 32, [200] + [1] * 140 + [300, 800]), (5000, 1000, 40, [8] * 160), (4104, 2048, 16, [3200])])
def test_lora_tiles(B, N, K, rank, lengths, yb):
    """Tiles of one run, of several, of none, and tiles of many runs (the other kernel's) in one call."""
    v = tile_case(lengths, N, K, rank, yb, 7)
    M = len(v[1])
    edges = np.cumsum([0] + lengths)
    rows = np.unique(np.clip(np.concatenate([edges[:30], edges[:30] - 1, [0, 127, 128, 255, 256, M - 1],
                                             rng(M).integers(0, M, 20)]), 0, M - 1))
    y = run_lora(B, v, True, yb)
    check_lora_rows(y, v, yb, rows)
    # every row, against the library's kernel for scattered tokens (one token a call cannot reach the tiles)
    bf = torch.bfloat16
    x, index, a, b, scale, base = [dev(t, d) for t, d in zip(v, (bf, None, bf, bf, None, bf if yb else None))]
    part = torch.cat([B.bl_lora_add(x[i:i + 32], index[i:i + 32], a, b, scale, base[i:i + 32]) for i in range(0, M, 32)])
    far = (y.float() - part.float()).abs()
    step = 2.0 ** -8 if yb else 2.0 ** -16  # one rounding of the output each; fp32: sums in another order
    assert bool((far <= 2 * step * part.float().abs() + 2.0 ** -12).all())
    same = run_lora(B, v, True, yb)
    assert torch.equal(y, same)


@gpu
@pytest.mark.parametrize("yb", [True, False])
@pytest.mark.parametrize("N,K,rank,lengths", [
    (1537, 4096, 64, [1, 127, 128, 129, 5, 250, 384]), (3000, 2056, 128, [64, 17, 200, 16, 15, 1, 190]),
    (2051, 4096, 24, [511, 1, 1, 1, 2, 30, 1600]), (2600, 5000, 8, [1000, 24, 4000]), (9000, 264, 96, [260, 140]),
    (2560, 4096, 32, [200] + [1] * 140 + [300, 800]), (5000, 1000, 40, [8] * 160), (4104, 2048, 16, [3200])])
def test_lora_tiles_fp32_activations(B, N, K, rank, lengths, yb):
    """fp32 x enters the tensor cores as three bf16 terms (24 bits): the same bounds as everywhere."""
    x, index, a, b, scale, base = tile_case(lengths, N, K, rank, yb, 9)
    x = rng(len(index), K, 10).standard_normal(x.shape).astype(np.float32)
    x[::7] *= np.float32(2.0 ** 40)  # rows of other magnitudes
    x[3::7] *= np.float32(2.0 ** -40)
    v = (x, index, a, b, scale, base)
    M = len(index)
    edges = np.cumsum([0] + lengths)
    rows = np.unique(np.clip(np.concatenate([edges[:30], edges[:30] - 1, [0, 127, 128, 255, 256, M - 1],
                                             rng(M).integers(0, M, 20)]), 0, M - 1))
    y = run_lora(B, v, False, yb)
    for size in (0, 3, 1):  # each magnitude by itself, for the 2-norm
        some = rows[rows % 7 == size]
        if len(some):
            check_lora_rows(y, v, yb, some)
    check_lora_rows(y, v, yb, rows)
    assert torch.equal(run_lora(B, v, False, yb), y)
    x[5, 3], x[M - 2, 7] = np.nan, np.inf
    got = run_lora(B, v, False, yb)
    rest = np.array([m for m in range(M) if m not in (5, M - 2)])
    assert torch.equal(got[rest], y[rest])


@gpu
@pytest.mark.parametrize("xb,yb", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("N,K,rank,lengths", [
    (8, 8, 8, [100, 1, 300]), (1, 8, 8, [257]), (33, 72, 16, [5, 400, 2]), (129, 264, 128, [256, 1, 1, 200]),
    (64, 520, 40, [300]), (1000, 136, 56, [1] * 9 + [300]), (6912, 64, 64, [128] * 5)])
def test_lora_tiles_of_small_shapes(B, N, K, rank, lengths, xb, yb):
    """Parts of K without a block, clusters without a tile of outputs, boxes wider than the tensors."""
    index = np.repeat([[0, 2, -1, 1, 0, 3, -1][i % 7] for i in range(len(lengths))], lengths)
    v = lora_inputs(len(index), N, K, rank, 4, xb, yb, 12, index)
    y = run_lora(B, v, xb, yb)
    check_lora(y, v, yb)
    assert torch.equal(run_lora(B, v, xb, yb), y)


@gpu
@pytest.mark.parametrize("yb", [True, False])
@pytest.mark.parametrize("M,longest", [(3000, 200), (4500, 400), (6000, 90), (9600, 300), (10000, 2000), (13000, 60),
                                       (25000, 500)])
def test_lora_tiles_with_helpers(B, M, longest, yb):
    """Idle SMs take half of the outputs of tiles with several runs: fewer and more of them than helpers."""
    lengths = rng(M, longest).integers(1, longest + 1, M // 4 + 1)
    index = np.repeat([[0, 2, -1, 1, 0, 3, -1][i % 7] for i in range(len(lengths))], lengths)[:M]
    v = lora_inputs(M, 1032, 136, 16, 4, True, yb, 13, index)
    y = run_lora(B, v, True, yb)
    check_lora(y, v, yb)
    x, index, a, b, scale, base = v
    bf = torch.bfloat16
    at = dev(base, bf if yb else None)
    assert torch.equal(B.bl_lora_add(dev(x, bf), dev(index), dev(a, bf), dev(b, bf), dev(scale), at, y=at), y)


@gpu
@pytest.mark.parametrize("xb", [True, False])
def test_lora_scattered_tiles_far_behind_long_runs(B, xb):
    """Tiles of many runs among more than 256 tiles, the first, some in the middle and the last ones."""
    lengths = [1] * 200 + [20000] + [3] * 100 + [12500] + [2] * 301
    index = np.repeat([[0, 2, -1, 1, 0, 3, -1][i % 7] for i in range(len(lengths))], lengths)
    v = lora_inputs(len(index), 72, 64, 16, 4, xb, True, 14, index)
    check_lora(run_lora(B, v, xb, True), v, True)


@gpu
def test_lora_tiles_in_place_out_of_range_and_bad_rows(B):
    v = tile_case([300, 200, 400, 300], 2048, 3000, 64, True, 8)
    x, index, a, b, scale, base = v
    bf = torch.bfloat16
    want = run_lora(B, v, True, True)
    y = dev(base, bf)
    assert torch.equal(B.bl_lora_add(dev(x, bf), dev(index), dev(a, bf), dev(b, bf), dev(scale), y, y=y), want)
    x[5, 3], x[450, 7], x[1100, 9] = np.nan, np.inf, -np.inf  # 300..499 have adapter 2, 500..899 none
    x[600, 0] = np.nan
    index[1150] = 4
    got = run_lora(B, v, True, True)
    torch.cuda.synchronize()
    assert B.device_error(clear=True) == B.BL_DEVERR_RANGE
    rest = [m for m in range(1200) if m not in (5, 450, 1100, 1150)]
    assert torch.equal(got[rest], want[rest]) and np.array_equal(host(got)[1150], base[1150])
    assert bool(torch.isnan(got[5]).all())


# ---------------------------------------------------------------------------
# sampling: tokens exactly, unless a decision lies within 2^-28 of going the
# other way (weights are within 2^-30): then the token's interval has to reach
# within 2^-28 of the goal.  Probabilities within 2^-23 (their own rounding,
# and the weights').
# ---------------------------------------------------------------------------

def check_sample(B, logits, u, bf16, t=None, k=None, p=None, mp=None):
    f = lambda v, d: None if v is None else dev(np.asarray(v, d))  # noqa: E731
    lg = dev(logits, torch.bfloat16 if bf16 else torch.float32)
    token, prob = B.bl_sample(lg, f(u, np.float32), f(t, np.float32), f(k, np.int32), f(p, np.float32), f(mp, np.float32),
                              prob=True)
    token, prob, seen = token.cpu().numpy(), prob.cpu().numpy(), host(lg)
    at = lambda v, m, d, none: none if v is None else d(v[m])  # noqa: E731
    for m in range(len(logits)):
        want, pr, margin, near = R.sample_row(seen[m], np.float32(u[m]), at(t, m, np.float32, 1.0), at(k, m, int, 0),
                                              at(p, m, np.float32, 1.0), at(mp, m, np.float32, 0.0))
        if margin < 2.0 ** -28:
            assert near[token[m]] < 2.0 ** -28, (m, token[m], want)
            continue
        assert token[m] == want, (m, token[m], want, margin)
        assert abs(prob[m] - pr) <= 2.0 ** -23 * pr, (m, prob[m], pr)
    return lg, token


def bulk(g, M, V, bf16, spread=2.0):
    l = (g.standard_normal((M, V)) * spread - 2).astype(np.float32)
    for m in range(M):
        l[m, g.integers(0, V, 12)] = 7 + 3 * g.standard_normal(12)
    return R.bf16_round(l) if bf16 else l


@gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("M,V", [(3, 1), (4, 2), (9, 31), (16, 1000), (40, 4099), (24, 65537), (5, 248320), (2, 524288)])
def test_sample_filters(B, M, V, bf16):
    g = rng(M, V)
    l = bulk(g, M, V, bf16)
    u = g.random(M).astype(np.float32)
    t = g.uniform(0.3, 2, M).astype(np.float32)
    check_sample(B, l, u, bf16)
    check_sample(B, l, u, bf16, t=t)
    check_sample(B, l, u, bf16, t=t, k=g.integers(0, 60, M))
    check_sample(B, l, u, bf16, t=t, p=g.uniform(0.2, 1.05, M).astype(np.float32))
    check_sample(B, l, u, bf16, t=t, mp=g.uniform(0, 0.3, M).astype(np.float32))
    check_sample(B, l, u, bf16, t=t, k=g.integers(-1, V + 2, M), p=g.uniform(0.5, 1, M).astype(np.float32),
                 mp=g.choice([0, 0.001, 0.05], M).astype(np.float32))


@gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("V", [7, 3000, 70000])
def test_sample_ties_and_equal_rows(B, V, bf16):
    """Equal logits: the order is that of the indices, weights are exact, so the place is known exactly."""
    g = rng(V, 5)
    u = np.float32([0, 0.25, 0.5, 0.75, 0.999, 1.0, 0.5, 0.125])
    same = np.full((8, V), -3.25, np.float32)
    lg, token = check_sample(B, same, u, bf16)
    assert token.tolist() == [min(int(np.float64(min(v, np.float32(0.99999994))) * V), V - 1) for v in u]
    check_sample(B, same, u, bf16, k=[1, 2, 3, 5, 0, 7, V, 4], p=np.float32([1, 0.5, 0.5, 0.75, 0.25, 1, 0.5, 0]))
    few = g.choice(np.float32([2, 2, 1, -1, -30, 0, -0.0]), (8, V))
    check_sample(B, few, u, bf16, t=np.float32([1, 0.5, 2, 0, 1e-6, 50, 1, 3]), k=[0, 3, V // 2, 1, 2, 0, 5, V - 1])
    few[:] = np.where(g.random((8, V)) < 0.5, np.float32(0.0), np.float32(-0.0))
    check_sample(B, few, u, bf16, k=[0, 3, V // 2, 1, 2, 0, 5, V - 1])


@gpu
@pytest.mark.parametrize("bf16", [True, False])
def test_sample_is_the_same_for_every_number_of_rows(B, bf16):
    """The number of rows chooses the CTAs of a row; the row's token and probability do not depend on it."""
    g, n, V = rng(41), 200, 40001
    l = dev((3 * g.standard_normal((n, V))).astype(np.float32), torch.bfloat16 if bf16 else None)
    u, t = dev(g.random(n).astype(np.float32)), dev(g.uniform(0.5, 1.5, n).astype(np.float32))
    k, p = dev(np.where(g.random(n) < 0.5, 40, 0).astype(np.int32)), dev(g.uniform(0.8, 1.1, n).astype(np.float32))
    token, prob = B.bl_sample(l, u, t, k, p, prob=True)
    for m in (1, 16, 19, 36, 38, 74, 76, 77, 152, 153):
        a, b = B.bl_sample(l[:m], u[:m], t[:m], k[:m], p[:m], prob=True)
        assert torch.equal(a, token[:m]) and torch.equal(b, prob[:m]), m


@gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("V", [5, 1025, 40000])
def test_sample_masks_infinities_and_odd_parameters(B, V, bf16):
    g = rng(V, 6)
    l = bulk(g, 14, V, bf16)
    lowest = np.float32(torch.finfo(torch.bfloat16 if bf16 else torch.float32).min)
    l[0] = -np.inf                                  # nothing left
    l[1] = np.nan
    l[2], l[2, V - 1] = -np.inf, -50                # one left
    l[3, g.random(V) < 0.95] = -np.inf
    l[4, g.random(V) < 0.95] = lowest
    l[5] = lowest                                   # a mask of the lowest value over everything: uniform
    l[6, ::2] = np.nan
    l[7, 1], l[7, 3] = np.inf, np.inf
    l[8] = np.inf
    l[9] = np.float32(2.0 ** -140) * np.sign(l[9]) if not bf16 else l[9]
    l[10] *= 1000
    l[11] *= 1e-4
    u = g.random(14).astype(np.float32)
    check_sample(B, l, u, bf16)
    nan, inf = np.float32("nan"), np.float32("inf")
    u[3:10] = [nan, -1, 2, 0, 0.5, 0.99999994, inf]
    check_sample(B, l, u, bf16, t=np.float32([1, 1, 1, 1, 1, 1, 0, nan, 1, -2, 1e-5, 1e6, 9e-6, 0.7]))
    check_sample(B, l, u, bf16, k=[-5, 0, 3, V + 9, 2 ** 31 - 1, 2, 1, 1, 4, -2 ** 31, 6, 7, 8, 9])
    check_sample(B, l, u, bf16, p=np.float32([nan, 0, 0.5, 0.9, -1, 0.3, 0.9, 0.5, 2, inf, 0.9, 0.5, 1e-9, 0.99999]))
    check_sample(B, l, u, bf16, mp=np.float32([nan, 0.1, 0.5, 0.01, 1, 1, 2, 0.5, 0.2, -1, 1e-9, 0.9, inf, 0.03]))


@gpu
@pytest.mark.parametrize("spread", [0.01, 30.0])
def test_sample_f32_close_logits(B, spread):
    """fp32 logits that differ in their last bits only, and a sharp distribution."""
    g = rng(77)
    l = (5 + spread * 1e-3 * g.standard_normal((16, 5000))).astype(np.float32) if spread < 1 else bulk(g, 16, 5000, False, spread)
    u = g.random(16).astype(np.float32)
    check_sample(B, l, u, False)
    check_sample(B, l, u, False, k=g.integers(1, 4000, 16), p=g.uniform(0.2, 1, 16).astype(np.float32))


@gpu
@pytest.mark.parametrize("bf16", [True, False])
def test_sample_alignment_and_repeats(B, bf16):
    g = rng(9)
    l = bulk(g, 6, 5003, bf16)
    u, k = dev(g.random(6).astype(np.float32)), dev(np.int32([0, 50, 3, 0, 900, 1]))
    t = torch.bfloat16 if bf16 else torch.float32
    want = B.bl_sample(dev(l, t), u, top_k=k, prob=True)
    for n in (1, 2, 3, 5):
        got = B.bl_sample(shifted(dev(l, t), n), u, top_k=k, prob=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(B.bl_sample(dev(l, t), u, top_k=k), want[0])


@gpu
def test_sample_follows_the_distribution(B):
    """10000 uniform numbers on one distribution: shares within five standard deviations."""
    n = 10000
    l = np.float32([0.0, 1.0, 2.0, -1.0, 3.0])
    p = np.exp(l.astype(np.float64)) / np.exp(l.astype(np.float64)).sum()
    u = (np.arange(n) + 0.5) / n
    token = B.bl_sample(dev(np.tile(l, (n, 1))), dev(u.astype(np.float32))).cpu().numpy()
    share = np.bincount(token, minlength=5) / n
    assert np.all(np.abs(share - p) <= 5 * np.sqrt(p * (1 - p) / n))


# ---------------------------------------------------------------------------
# streams, overlap, graphs
# ---------------------------------------------------------------------------

def serving_step(B, v, stream=None):
    x, res, w, index, a, b, scale, base, u, k = v
    q, s, h, y = B.bl_rmsnorm_quant_int8(x, w, residual=res, y=True, stream=stream)
    z = B.bl_lora_add(y, index, a, b, scale, base, stream=stream)
    token, prob = B.bl_sample(z, u, top_k=k, prob=True, stream=stream)
    return q, s, h, y, z, token, prob


@gpu
@pytest.mark.parametrize("M", [1, 5, 300])
def test_streams_overlap_and_graphs(B, M):
    g = rng(M, 11)
    K, N, bf = 1024, 4000, torch.bfloat16
    lora = lora_inputs(M, N, K, 16, 3, True, True, 6, np.arange(M) // 20 % 4 - 1)
    v = [dev(t, bf) for t in norm_inputs(M, K, True, True, 7)]
    v += [dev(lora[1]), dev(lora[2], bf), dev(lora[3], bf), dev(lora[4]), dev(lora[5] * 4, bf)]
    v += [dev(g.random(M).astype(np.float32)), dev(g.integers(0, 50, M).astype(np.int32))]
    want = serving_step(B, v)
    torch.cuda.synchronize()
    same = lambda got: all(torch.equal(p, q) for p, q in zip(want, got))  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = serving_step(B, v, stream=side)
    side.synchronize()
    assert same(got)
    B.set_overlap(True)
    try:
        got = serving_step(B, v)
        torch.cuda.synchronize()
        assert same(got)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            serving_step(B, v)
            side.synchronize()
            with torch.cuda.graph(graph, stream=side):
                got = serving_step(B, v)
        for _ in range(3):
            for t in got:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert same(got)
    finally:
        B.set_overlap(False)


# ---------------------------------------------------------------------------
# the operators together, as the example runs them
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("requests", [1, 7, 40])
def test_example_serving_step(B, requests):
    """The step's tokens are those of its logits, and an adapter changes the logits of its own requests only."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serving_step.py")
    spec = importlib.util.spec_from_file_location("serving_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    model = example.Model(256, 512, 4000, adapters=4, rank=16)
    v = list(example.inputs(requests, 256, 4))
    token, prob, logits = example.step(model, *v)
    rows = host(logits)
    args = [t.cpu().numpy() for t in v[3:]]
    for m in range(requests):
        u, t, k, p, mp = (a[m] for a in args)
        want, pr, margin, near = R.sample_row(rows[m], u, t, int(k), p, mp)
        assert token[m].item() == want or (margin < 2.0 ** -28 and near[token[m].item()] < 2.0 ** -28)
    none = v[2] < 0
    v[2] = torch.full_like(v[2], -1)
    plain = example.step(model, *v)[2]
    assert torch.equal(plain[none], logits[none])
    assert bool((plain != logits).any(1)[~none].all())
