"""Edges of the operators around the products: limits of their parameters, values at the ends of their types, and
the precision of fp32 results.  Tolerances are derived beside each test."""
import numpy as np
import pytest
import torch

import serving_ref as R
from test_serving_ops import B, dev, host, no_device_error, rng, run_lora  # noqa: F401

gpu = pytest.mark.gpu


# ---------------------------------------------------------------------------
# sampling
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("V", [2, 5, 3000, 70000, 248320])
def test_sample_min_p_above_one_keeps_the_first_token_alone(B, V, bf16):
    """No weight reaches a min_p above 1, so only the first token stays, whatever ties with it; at 1 all maxima stay."""
    g = rng(V, 21)
    l = g.choice(np.float32([2, 2, 1, 0.5, -3]), (10, V))
    l[:, [0, V - 1]] = 2
    l[9] = [-np.inf] * (V - 1) + [-7]
    above = np.nextafter(np.float32(1), np.float32(2))
    mp = np.float32([above, 1.5, 2, 1e30, np.inf, 1, 1, np.inf, 1.5, 3])
    k = np.int32([0, 0, V, 1, 0, 0, 2, 7, 0, 0])
    p = np.float32([1, 1, 0.9, 1, 1, 1, 1, 0.5, 0.99, 1])
    t = np.float32([1, 0.7, 1, 1, 2, 1, 1, 0, 1, 1])
    u = np.float32([0.9, 0.5, 0.999, 0.99999994, 0.75, 0.9, 0.75, 0.9, 0.9, 0.9])
    token, prob = B.bl_sample(dev(l, torch.bfloat16 if bf16 else None), dev(u), dev(t), dev(k), dev(p), dev(mp), prob=True)
    token, prob = token.cpu().numpy(), prob.cpu().numpy()
    for m in range(10):
        ties = np.nonzero(l[m] == l[m].max())[0]
        if mp[m] > 1:
            ties = ties[:1]
        if k[m] > 0:
            ties = ties[:k[m]]
        assert token[m] == ties[int(np.float64(u[m]) * len(ties))], (m, token[m])
        assert prob[m] == np.float32(1 / len(ties)), (m, prob[m])


# ---------------------------------------------------------------------------
# norm with codes
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("M,K", [(3, 256), (2, 2560), (2, 2561), (400, 5120), (3, 6912), (2, 13824), (2, 32776)])
def test_norm_codes_where_the_inverse_scale_overflows(B, M, K, bf16):
    """127 / max|v| beyond binary32: the steps of the quantization give +-127 for what is not 0, for every shape."""
    g = rng(M, K, 22)
    x = (np.sign(g.standard_normal((M, K))) * g.uniform(0.5, 2, (M, K))).astype(np.float32)
    w = np.full(K, 2.0 ** -125, np.float32) * g.choice(np.float32([1, 0.5, 0.75]), K)
    if bf16:
        x, w = R.bf16_round(x), R.bf16_round(w)
    x[0] *= np.float32(2.0 ** 10)  # the factor of a row undoes it
    t = torch.bfloat16 if bf16 else torch.float32
    with np.errstate(over="ignore"):
        rq, rs, _, ry, clear = R.rmsnorm_quant(x, None, w, 1e-5, bf16)
    assert clear.all() and np.all(np.abs(rq) == 127) and np.all(rs > 0)
    q, s, _, y = B.bl_rmsnorm_quant_int8(dev(x, t), dev(w, t), 1e-5, y=True)
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(host(y), ry)
    assert np.array_equal(q.cpu().numpy(), rq)
    if not bf16:
        assert torch.equal(B.bl_quantize_act_absmax_int8(y)[0], q)


@gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("K", [256, 2560, 2561, 32768])
def test_norm_codes_at_the_ends_of_their_range(B, K, bf16):
    """Rows from just above 2^-50 to just below 2^50, with zeros among them: codes bit for bit."""
    g, M = rng(K, 27), 48
    x = (np.sign(g.standard_normal((M, K))) * g.uniform(1.1, 1.9, (M, K))).astype(np.float32)
    x *= np.float32(2.0) ** np.where(np.arange(M) % 2, np.linspace(-50, -1, M), np.linspace(49, 1, M)).round().astype(np.float32)[:, None]
    x[:, :: 5] = 0
    w = (1 + 0.3 * g.standard_normal(K)).astype(np.float32)
    if bf16:
        x, w = R.bf16_round(x), R.bf16_round(w)
    t = torch.bfloat16 if bf16 else torch.float32
    for eps in (0.0, 1e-5):
        rq, rs, _, ry, clear = R.rmsnorm_quant(x, None, w, eps, bf16)
        q, s, _, y = B.bl_rmsnorm_quant_int8(dev(x, t), dev(w, t), eps, y=True)
        assert clear.sum() > M - 4
        assert np.array_equal(s.cpu().numpy()[clear], rs[clear]) and np.array_equal(host(y)[clear], ry[clear])
        assert np.array_equal(q.cpu().numpy()[clear], rq[clear])


# ---------------------------------------------------------------------------
# adapters
# ---------------------------------------------------------------------------

def run_edge(B, x, index, a, b, scale, base, xb, yb):
    return host(run_lora(B, (x, index, a, b, scale, base), xb, yb))


@gpu
@pytest.mark.parametrize("xb", [True, False])
@pytest.mark.parametrize("M,N,K,rank", [(300, 136, 8200, 64), (300, 72, 13824, 16), (2000, 136, 13824, 64), (11000, 72, 8200, 64),
                                        (11000, 40, 13824, 16), (10500, 40, 8200, 128)])
def test_lora_fp32_outputs_of_long_sums(B, M, N, K, rank, xb):
    """The 2-norm of a row block's error against that of its result, without a base.  The tensor core cuts off up to a
    step (2^-23) in each of 16 additions (fp32 x: 24, of which the first eight are of far smaller terms) to a sum that
    grows with the square root of their number: 11 steps.  Then it is added up in binary32, K / 128 times half a step
    at most, of either sign; the operand's rounding and rank / 16 steps of the second product follow."""
    g = rng(M, N, K, rank, 25)
    x = g.standard_normal((M, K)).astype(np.float32)
    x = R.bf16_round(x) if xb else x
    a = R.bf16_round(g.standard_normal((2, rank, K)) / np.sqrt(K))
    b = R.bf16_round(g.standard_normal((2, N, rank)) * 0.1)
    scale = np.float32([1.3, 0.7])
    index = (np.arange(M) * 2 // M).astype(np.int32)
    y = run_edge(B, x, index, a, b, scale, np.zeros((M, N), np.float32), xb, False)
    rows = np.arange(0, M, max(1, M // 60))
    ref = R.lora_add(x[rows], index[rows], a, b, scale, np.zeros((len(rows), N), np.float32))[0]
    off = np.linalg.norm(y[rows] - ref) / np.linalg.norm(ref)
    assert off <= (11 + np.sqrt(K / 128) / 2 + rank / 16 + 2) * 2.0 ** -23, off * 2 ** 23


@gpu
@pytest.mark.parametrize("xb", [True, False])
@pytest.mark.parametrize("M,N,K,rank", [(9, 1000, 512, 16), (300, 1000, 512, 64), (700, 1537, 1000, 128), (2500, 520, 2560, 16),
                                        (4225, 648, 384, 128)])
def test_lora_bf16_outputs_are_the_rounded_sums(B, M, N, K, rank, xb):
    """A bf16 output is another than its exact value's rounding only where a border lies within the error of the fp32
    sums, at most 2^-20 of a value of the usual size: for 2 2^-20 / 2^-8 = 2^-11 of such values, and, as the smaller ones
    have finer steps, for no more than 2^-10 of all."""
    g = rng(M, N, K, rank, 26)
    index = np.repeat([0, 1, 2, 1], [M // 4] * 3 + [M - M // 4 * 3]).astype(np.int32)
    x = g.standard_normal((M, K)).astype(np.float32)
    a, b = R.bf16_round(g.standard_normal((3, rank, K)) / np.sqrt(K)), R.bf16_round(g.standard_normal((3, N, rank)) * 0.1)
    base = R.bf16_round(g.standard_normal((M, N)))
    v = (R.bf16_round(x) if xb else x, index, a, b, g.uniform(0.25, 4, 3).astype(np.float32), base)
    y = run_edge(B, *v, xb, True)
    rows = np.arange(0, M, max(1, M // 300))
    ref = R.lora_add(v[0][rows], index[rows], a, b, v[4], base[rows])[0]
    assert (y[rows] != R.bf16_round(ref)).mean() <= 2.0 ** -10


def one_hot(M, N, K, rank, adapters, xb, seed):
    """One product per inner product and per output: no sums, so a term that is lost shows in full."""
    g = rng(M, N, K, rank, seed)
    x = g.standard_normal((M, K)).astype(np.float32)
    x[np.abs(x) < 0.01] = 1.2345678
    if xb:
        x = R.bf16_round(x)
    a, b = np.zeros((adapters, rank, K), np.float32), np.zeros((adapters, N, rank), np.float32)
    for l in range(adapters):
        a[l, np.arange(rank), g.integers(0, K, rank)] = R.bf16_round(g.uniform(0.5, 2, rank))
        b[l, np.arange(N), g.integers(0, rank, N)] = R.bf16_round(g.uniform(0.5, 2, N))
    return x, a, b, g.uniform(0.25, 4, adapters).astype(np.float32)


@gpu
@pytest.mark.parametrize("xb", [True, False])
@pytest.mark.parametrize("M,N,K,rank", [(9, 300, 520, 16), (300, 136, 264, 8), (700, 1537, 1000, 64), (1300, 260, 2056, 128),
                                        (11000, 72, 520, 24), (6000, 1032, 264, 72)])
def test_lora_fp32_outputs_keep_24_bits(B, M, N, K, rank, xb):
    """x, the inner product and its product with the scale are rounded to binary32 at most, the last two and the
    output by up to a step each where the tensor core truncates, and the terms that they are split into are added up
    with as many: 2^-21 in all."""
    x, a, b, scale = one_hot(M, N, K, rank, 3, xb, 24)
    index = np.repeat([0, 1, -1, 2], [M // 4] * 3 + [M - M // 4 * 3]).astype(np.int32)
    y = run_edge(B, x, index, a, b, scale, np.zeros((M, N), np.float32), xb, False)
    rows = np.unique(np.concatenate([np.arange(0, M, max(1, M // 300)), [M - 1]]))
    for m in rows:
        l = index[m]
        ref = np.zeros(N) if l < 0 else np.float64(scale[l]) * (b[l].astype(np.float64) @ (a[l].astype(np.float64) @ x[m]))
        assert np.all(np.abs(y[m] - ref) <= 2.0 ** -21 * np.abs(ref)), (m, np.abs(y[m] / ref - 1).max() * 2 ** 21)


@gpu
@pytest.mark.parametrize("yb", [True, False])
@pytest.mark.parametrize("xb", [True, False])
@pytest.mark.parametrize("M,N,rank", [(10, 200, 16), (300, 200, 16), (300, 203, 72), (1500, 1032, 64)])
def test_lora_infinities_and_values_near_the_largest(B, M, N, rank, xb, yb):
    """Infinite inner products stay infinite, and finite ones beyond the largest bf16 stay finite, by both kernels."""
    K, big = 256, np.float32(3.4e38)  # above the largest bf16, 3.3895e38
    g = rng(M, N, 23)
    x = np.zeros((M, K), np.float32)
    x[:, 0] = 1
    a = np.zeros((4, rank, K), np.float32)
    a[:, :, 0] = 1
    a[1, 0, 0], a[1, 1:, 0] = 2.0 ** -80, 0  # a finite inner product of a huge x
    a[2, 1:, 0] = 0
    b = R.bf16_round(g.uniform(0.5, 2, (4, N, rank)))
    b[1] *= np.float32(2.0 ** -20)
    b[2] *= np.float32(2.0 ** -100)
    index = np.repeat([0, 1, 2, 3, -1], [M // 5] * 4 + [M - M // 5 * 4]).astype(np.int32)
    at = [np.nonzero(index == i)[0] for i in range(4)]
    x[at[0][0], 0] = np.inf
    x[at[3][0], 0] = -np.inf
    x[at[1], 0] = R.bf16_round(np.float32(3.3e38)) if xb else big
    x[at[2], 0] = 2.0 ** 126
    a[2, 0, 0] = R.bf16_round(np.float32(3.99))
    base = R.bf16_round(g.standard_normal((M, N)))
    scale = np.float32([1, 1, 1.003, 1])  # the third inner product passes the largest bf16 by its scale
    y = run_edge(B, x, index, a, b, scale, base, xb, yb)
    assert np.all(y[at[0][0]] == np.inf) and np.all(y[at[3][0]] == -np.inf)
    rows = np.setdiff1d(np.arange(M), [at[0][0], at[3][0]])
    ref, cond = R.lora_add(x[rows], index[rows], a, b, scale, base[rows])
    assert np.all(np.isfinite(ref)) and ref.max() < 1e38
    # a single product of K; rank + 8 additions; bf16 outputs: half a step, and 16 bits of the inner product
    bound = (rank + 8) * 2.0 ** -23 * cond + (2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * cond if yb else 0)
    assert np.all(np.abs(y[rows] - ref) <= bound)
    x[at[0][0], 0], x[at[3][0], 0] = 1, 1
    x[at[0][1], 0] = np.uint32(0x7F800001).view(np.float32)  # a NaN that a truncation would make an infinity
    y = run_edge(B, x, index, a, b, scale, base, xb, yb)
    assert np.all(np.isnan(y[at[0][1]])) and np.all(np.isfinite(np.delete(y, at[0][1], 0)))


def test_lora_refuses_more_tokens_than_a_grid_has_clusters(B):
    """The header's limit on M is refused before any CUDA call; so are counts and sizes beyond 32 bits."""
    import ctypes
    P, f = ctypes.c_void_p, B.lib().bl_lora_add
    a = P(1 << 14)
    for M, N, L, want in ((2 ** 30 - 3, 4, 1, B.BL_ERR_UNSUPPORTED), (2 ** 31 - 1, 4, 1, B.BL_ERR_UNSUPPORTED),
                          (2 ** 31, 4, 1, B.BL_ERR_SHAPE), (1, 2 ** 31, 1, B.BL_ERR_SHAPE), (1, 4, 2 ** 31, B.BL_ERR_SHAPE)):
        assert f(a, B.BL_BF16, a, a, a, a, a, a, B.BL_F32, M, N, 8, L, 8, None) == want, (M, N, L)


@gpu
def test_binding_names_the_tensor_that_does_not_fit(B):
    bf = torch.bfloat16
    x, index = torch.zeros(3, 16, device="cuda", dtype=bf), torch.zeros(3, dtype=torch.int32, device="cuda")
    a, b = torch.zeros(2, 8, 16, device="cuda", dtype=bf), torch.zeros(2, 5, 8, device="cuda", dtype=bf)
    scale, base = torch.ones(2, device="cuda"), torch.zeros(3, 5, device="cuda")
    B.bl_lora_add(x, index, a, b, scale, base)
    for bad in ((x, index, a[0], b, scale, base), (x, index, a, b, scale, base[0]), (x, index, a, b[0], scale, base),
                (x, index, a[:, :, :8].contiguous(), b, scale, base), (x, index, a, b, scale, base[:2])):
        with pytest.raises(ValueError):
            B.bl_lora_add(*bad)
    for bad in ((x, index, None, b, scale, base), (x, index, a, b, scale, None), (x, index, a, b, scale, base.cpu()),
                (x, index, a.float(), b, scale, base), (x, index.long(), a, b, scale, base)):
        with pytest.raises(TypeError):
            B.bl_lora_add(*bad)
