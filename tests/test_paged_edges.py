"""Edges of the operators over a paged key-value cache: rows that see nothing of a tile, parts of a row without weight, values
at the ends of their types, the precision of unlikely tokens.  Tolerances are derived beside each test."""
import numpy as np
import pytest
import torch

import paged_ref as R
from serving_ref import bf16_round
from test_paged_step import (BF, F32, I32, B, Cache, attn_bound, attn_ref, check_attn, dev, host, ints,  # noqa: F401
                             no_device_error, range_error, rng)

gpu = pytest.mark.gpu


# ---------------------------------------------------------------------------
# attention: rows that see no token in a unit's first tile, or in the first tile of a CTA's stretch.  The bound is that of
# the other attention tests.
# ---------------------------------------------------------------------------

def spread_queries(M, H, D, deviation, shift, seed):
    """Queries whose scores (times D ** -0.5, against keys of deviation 1 around a common part of 0.5) have about this
    deviation; with `shift` the first coordinate is kept for it."""
    q = deviation / 1.25 ** 0.5 * rng(M, H, D, seed).standard_normal((M, H, D)).astype(np.float32)
    if shift:
        q[..., 0] = 8
    return bf16_round(q)


def shift_scores(cache, by):
    """All scores by about `by`, through the first coordinate (the queries have 8 there)."""
    value = bf16_round(np.float32([by * cache.D ** 0.5 / 8]))[0]
    for k, _ in cache.rows:
        k[:, :, 0] = value
    real = ~np.isnan(cache.k)
    cache.k[..., 0] = np.where(real[..., 0], value, cache.k[..., 0])


@gpu
@pytest.mark.parametrize("window,new", [(300, 2), (512, 5), (1000, 8), (400, 5)])
@pytest.mark.parametrize("deviation,shift", [(0.8, 0), (1.2, 0), (1.5, 0), (2.0, 0), (1.2, -100), (1.2, 100), (2.0, -300)])
def test_attn_window_that_begins_in_a_tiles_last_tokens(B, window, new, deviation, shift):
    lengths = [128 * (r % 4) + 120 + r % 8 + new - 1 + window for r in range(24)]
    cache = Cache(lengths, 2, 128, 16, 31)
    if shift:
        shift_scores(cache, shift)
    q = spread_queries(24 * new, 10, 128, deviation, shift, window)
    check_attn(B, cache, [new] * 24, 10, True, window=window, q=q)


@gpu
@pytest.mark.parametrize("length,new,window", [(300, 300, 64), (700, 700, 512), (900, 300, 256), (640, 200, 100), (1500, 640, 128)])
@pytest.mark.parametrize("D,page,f32", [(128, 16, True), (80, 64, False)])
def test_attn_prompt_chunks_with_a_window(B, length, new, window, D, page, f32):
    cache = Cache([length, 40], 1, D, page, 32)
    q = spread_queries(new + 3, 4, D, 1.0, 0, length)
    check_attn(B, cache, [new, 3], 4, f32, window=window, q=q)


@gpu
@pytest.mark.parametrize("sinks", [0, 4])
@pytest.mark.parametrize("deviation,shift", [(0.5, 0), (1.5, 0), (1.0, -200)])
def test_attn_windows_cut_between_ctas(B, deviation, shift, sinks):
    """Units of 33 tiles, of which a CTA has some 14."""
    new, window = 5, 4096
    lengths = [128 * (1 + r) + 124 + r % 4 + new - 1 + window for r in range(8)]
    cache = Cache(lengths, 8, 128, 64, 33)
    if shift:
        shift_scores(cache, shift)
    q = spread_queries(8 * new, 16, 128, deviation, shift, sinks)
    check_attn(B, cache, [new] * 8, 16, True, window=window, sinks=sinks, q=q)


@gpu
@pytest.mark.parametrize("new", [1, 6])
@pytest.mark.parametrize("deviation,shift", [(0.5, 0), (1.5, 0), (1.0, -200)])
def test_attn_first_tiles_on_bad_pages_or_without_weight(B, new, deviation, shift):
    """A request's first tile has no pages, or keys whose scores are all -inf: its rows have seen nothing when the next comes."""
    lengths, H, D, scale = [300, 1000, 2900, 260] * 3, 24, 128, 128 ** -0.5  # some 900 tiles: a CTA has several
    cache = Cache(lengths, 8, D, 16, 34, wide=True)
    if shift:
        shift_scores(cache, shift)
    q = spread_queries(12 * new, H, D, deviation, shift, 7)
    q[..., 1] = 1
    first = [128, 256, 1280, 128] * 3  # hidden tokens of each request
    for how in ("pages", "scores"):
        k, v, table, length = cache.gpu()
        for r, n in enumerate(first):
            if how == "pages":
                table[r, :n // 16] = -1
            else:
                k[table[r, :n // 16].long(), :, :, 1] = -float("inf")
        out = host(B.bl_attn_paged(dev(q, BF), k, v, table, length, ints(np.arange(13) * new), scale, out_dtype=F32))
        assert range_error(B) == (how == "pages")
        for r, n in enumerate(lengths):
            for t in range(new):
                seen = R.seen_by(n - new + t, n, 0, 0) & (np.arange(n) >= first[r])
                for h in range(H):
                    kr, vr = (c[:, h // 3] for c in cache.rows[r])
                    ref, cond, size = R.attention_row(q[r * new + t, h], kr, vr, seen, scale)
                    assert np.all(np.abs(out[r * new + t, h] - ref) <= attn_bound(ref[None], cond[None], np.array([size]), n, D, True)[0]), (how, r, t, h)


# ---------------------------------------------------------------------------
# verification: what is drawn from lies in many tokens below the sums' units (2^-44 of a weight, 2^-60 of p - q).  The sums
# are within 2^-20 of the mass.
# ---------------------------------------------------------------------------

NUMBERS = [0.0, float("nan"), -1.0, 1e-12, 1e-7, 0.3, 0.5, 0.99, 0.99999994, 2.0]


def tail_rows(rows, V, tail, bf16):
    """Logits of 0 at V - 5, nothing at V - 1, `tail` elsewhere."""
    l = torch.full((rows, V), tail, dtype=BF if bf16 else F32, device="cuda")
    l[:, V - 5] = 0
    l[:, V - 1] = -float("inf")
    return l


@gpu
@pytest.mark.parametrize("requests", [1, 64, 200])
@pytest.mark.parametrize("tail", [-31.0, -34.0, -35.0, -38.0, -42.0, -45.0])
def test_verify_tails_below_the_unit_of_the_sums(B, tail, requests):
    V = 248320
    us = np.resize(np.float32(NUMBERS), requests)
    if requests == 1:
        us = np.float32([0])
    for bf16 in (True, False):
        _, got = B.bl_verify(tail_rows(requests, V, tail, bf16), ints(np.zeros(requests)), ints(np.arange(requests + 1)), dev(us), dev(us))
        got = got.cpu().numpy()
        w = np.full(V, np.exp(tail))
        w[V - 5], w[V - 1] = 1, 0
        mass = np.cumsum(w) / w.sum()
        u = np.clip(np.nan_to_num(us), 0, np.float32(0.99999994))
        assert np.all((got >= 0) & (got < V - 1)), got
        assert np.all((mass[got] - w[got] / w.sum() <= u + 2.0 ** -20) & (mass[got] >= u - 2.0 ** -20)), got


@gpu
@pytest.mark.parametrize("requests", [1, 64, 200])
@pytest.mark.parametrize("tail", [-31.0, -38.0, -42.0, -43.0, -44.0, -45.0])
def test_verify_tails_below_the_unit_of_what_is_left(B, tail, requests):
    """A draft that both models mask is refused, and the draft's model has all but the tail: the tail is what is left."""
    V = 248320
    us = np.resize(np.float32(NUMBERS), requests)
    if requests == 1:
        us = np.float32([0])
    u = np.full(2 * requests, 0.5, np.float32)
    token = np.resize([0, V - 1], 2 * requests)
    for bf16 in (True, False):
        drafts = tail_rows(2 * requests, V, -float("inf"), bf16)
        accepted, got = B.bl_verify(tail_rows(2 * requests, V, tail, bf16), ints(token), ints(2 * np.arange(requests + 1)), dev(u), dev(us), draft_logits=drafts)
        got = got.cpu().numpy()
        assert not accepted.any()
        assert np.all((got >= 0) & (got < V - 1)), got


def near(us, w, got, slack=2.0 ** -20):
    """Whether `got` is a token whose stretch of the weights w holds the number, up to `slack` of the mass."""
    mass = np.cumsum(w) / w.sum()
    u = min(max(float(np.nan_to_num(us)), 0.0), float(np.float32(0.99999994)))
    return w[got] > 0 and mass[got] - w[got] / w.sum() - slack <= u <= mass[got] + slack


@gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("requests,V", [(3, 20000), (40, 20001), (70, 100000)])
def test_verify_equal_rows_leave_nothing_of_their_difference(B, requests, V, apart, bf16):
    """p = q in every token, light and heavy ones: nothing is left, so p is taken.  `apart`: rows at other addresses modulo 16."""
    g = rng(V, requests, 41)
    l = (2.5 * g.standard_normal((2 * requests, V))).astype(np.float32)
    l[np.arange(2 * requests)[:, None], g.integers(0, V, (2 * requests, 5))] += 6
    l = bf16_round(l) if bf16 else l
    x = g.integers(0, V, requests)
    l[2 * np.arange(requests), x] = -np.inf
    t, us = g.uniform(0.4, 1.6, requests).astype(np.float32), g.random(requests).astype(np.float32)
    token = np.stack([x * 0, x], 1).reshape(-1)
    lt = dev(l, BF if bf16 else F32)
    drafts = lt.clone()
    if apart:
        buf = torch.empty(lt.numel() + 1, dtype=lt.dtype, device="cuda")
        drafts = buf[1:].view(lt.shape)
        drafts.copy_(lt)
    accepted, got = B.bl_verify(lt, ints(token), ints(2 * np.arange(requests + 1)), dev(np.full(2 * requests, 0.3, np.float32)), dev(us),
                                temperature=dev(t), draft_logits=drafts)
    assert not accepted.any()
    for r, n in enumerate(got.tolist()):
        assert near(us[r], R.weights(l[2 * r], t[r]), n), r


@gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("model", [False, True])
def test_verify_tokens_without_a_share_are_not_drawn(B, model, bf16):
    """The tokens that hold the number have each less than a unit (2^-44 of the largest weight, 2^-60 of the mass of p - q); among
    them lies the refused draft, which is far likelier and has no share."""
    V, end = 30000, 29000
    for x in (96, 100, 103, 110):
        # the other tokens of the first part: a fifth of a unit each, four of them above half of one
        tail = np.float32(np.log(0.2 * 1.66) - 60 * np.log(2) if model else np.log(0.2) - 44 * np.log(2))
        l = np.full((2, V), -np.inf, np.float32)
        l[:, :300], l[:, x], l[:, end] = tail, np.log(np.float32(0.66)), 0
        q = np.full((2, V), -np.inf, np.float32)
        q[:, x], q[:, end] = 0, np.log(np.float32(0.66))
        if bf16:
            l, q = bf16_round(l), bf16_round(q)
        u = np.float32([0.9, 0])  # p(x) = 0.4, q(x) = 0.6 or 1
        for us in (0.0, -1.0, 1e-30):
            accepted, got = B.bl_verify(dev(l, BF if bf16 else F32), ints([0, x]), ints([0, 2]), dev(u), dev(np.float32([us])),
                                        draft_logits=dev(q, BF if bf16 else F32) if model else None)
            w = R.weights(l[0], 1.0)
            w[x] = 0
            if model:
                w = np.maximum(R.weights(l[0], 1.0) / R.weights(l[0], 1.0).sum() - R.weights(q[0], 1.0) / R.weights(q[0], 1.0).sum(), 0)
            assert accepted.item() == 0 and w[got.item()] > 0 and near(us, w, got.item()), (x, us, got.item())


# ---------------------------------------------------------------------------
# verification: logits and temperatures at the ends of their types
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("model", [False, True])
@pytest.mark.parametrize("temperature", [0.0, 1e-4, 0.7, 1.4, 1.5, 1.7, 2.0, 3.0, 5.0, 100.0, 1e10, 1e17, 1e19, 1e30, 1e36, 1e37, 1e38, 3e38, np.inf])
def test_verify_masks_of_the_lowest_value(B, temperature, model, bf16):
    """Logits of the type's lowest value have the weight that the temperature leaves them, -inf none at any; whole words, threads
    and stretches of them."""
    low = np.float32(-3.3895313892515355e38) if bf16 else np.finfo(np.float32).min
    for V, live in ((96, slice(0, 32)), (9000, slice(40, 90)), (9000, slice(8000, 9000, 7))):
        n = 40
        l = np.full((2 * n, V), low, np.float32)
        l[:, live] = 0
        l[:, V - V // 3:V - V // 4] = -np.inf
        x = V - V // 3
        us = ((np.arange(n) + 0.5) / n).astype(np.float32)
        q = l.copy()
        q[:, :60] = -np.inf
        _, got = B.bl_verify(dev(l, BF if bf16 else F32), ints(np.resize([0, x], 2 * n)), ints(2 * np.arange(n + 1)), dev(np.resize(us, 2 * n)), dev(us),
                             temperature=dev(np.full(n, temperature, np.float32)), draft_logits=dev(q, BF if bf16 else F32) if model else None)

        def weights(row):
            if temperature < 1e-5:
                return (row == row.max()) * 1.0
            z = (np.where(row > -np.inf, row, low).astype(np.float64) - row.max()) / np.float64(np.float32(temperature))
            return np.where(row > -np.inf, np.exp(z), 0)
        w, slack = weights(l[0]), 2.0 ** -20
        if model:  # each share is rounded to a unit of 2^-60 of the mass; below that nothing is left, and p is taken
            rest = np.maximum(w / w.sum() - weights(q[0]) / weights(q[0]).sum(), 0)
            if rest.max() > 2.0 ** -60:
                w, slack = rest, slack + (rest > 0).sum() * 2.0 ** -61 / rest.sum()
        for r in range(n):
            assert near(us[r], w, got[r].item(), slack), (V, r, got[r].item())


@gpu
@pytest.mark.parametrize("model", [False, True])
@pytest.mark.parametrize("top,temperature", [(1000.0, 2e-5), (-1000.0, 2e-5), (60.0, 1e-5), (1e6, 0.03), (-1e6, 0.03), (3e7, 1.0), (-3e8, 20.0), (5e9, 300.0), (1e12, 0.5), (-1e20, 1e12)])
def test_verify_large_exponents(B, top, temperature, model):
    """Logits whose differences are steps of fp32 and whose exponents have no fraction any more: the weights are those of the
    differences, in tests of acceptance too."""
    V, n = 5000, 64
    step = abs(np.spacing(np.float32(top)))
    g = rng(71, int(abs(top)))
    l = (np.float32(top) - step * g.integers(0, 6, (2 * n, V))).astype(np.float32)
    l[:, 17] = top
    q = (np.float32(top) - step * g.integers(0, 6, (2 * n, V))).astype(np.float32) if model else None
    t = np.full(n, temperature, np.float32)
    us, u = g.random(n).astype(np.float32), g.random(2 * n).astype(np.float32)
    token = g.integers(0, V, 2 * n)
    accepted, got = B.bl_verify(dev(l), ints(token), ints(2 * np.arange(n + 1)), dev(u), dev(us), temperature=dev(t), draft_logits=dev(q) if model else None)
    for r in range(n):
        a, x, margin, w = R.verify(l[2 * r:2 * r + 2], q[2 * r:2 * r + 2] if model else None, token[2 * r:2 * r + 2], u[2 * r:2 * r + 2], us[r], t[r])
        if margin > 2.0 ** -15:
            assert accepted[r].item() == a, (r, margin)
            assert near(us[r], w, got[r].item()), (r, got[r].item())


# ---------------------------------------------------------------------------
# verification: unlikely drafts.  p and q are within 2^-17 of their value each (include/bl.h), so tests of acceptance that are
# 2^-16 of p away from going the other way are sure.
# ---------------------------------------------------------------------------

def acceptance(l, q, x, t):
    """p(x) / q(x) in 64 bits, of rows with an own temperature."""
    def share(a):
        z = (a.astype(np.float64) - a.max()) / np.float64(t)
        return np.exp(z[x]) / np.exp(z).sum()
    return share(l) / (share(q) if q is not None else 1.0)


@gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("z", [2, 20, 60, 100, 140, 400, 900])
def test_verify_unlikely_drafts(B, z, bf16):
    """Drafts whose weights under both models are about 2^-z of the largest, tested by numbers just beside p / q."""
    V, requests = 700, 64
    g = rng(61, z, bf16)
    t = g.uniform(0.02, 0.2, requests).astype(np.float32)
    l, q = ((0.2 * g.standard_normal((2 * requests, V))).astype(np.float32) for _ in range(2))
    x = g.integers(0, V, requests)
    for r in range(requests):
        for a in (l, q):
            a[2 * r, (x[r] + 5) % V] = 4 + g.random()
            a[2 * r, x[r]] = a[2 * r].max() - t[r] * z * np.log(2) * g.uniform(0.99, 1)
        q[2 * r, x[r]] += t[r] * g.uniform(1, 3) + (0.1 if bf16 else 0)
    if bf16:
        l, q = bf16_round(l), bf16_round(q)
    u, want, sure = np.zeros(2 * requests, np.float32), np.zeros(requests, int), 0
    for r in range(requests):
        ratio = acceptance(l[2 * r], q[2 * r], x[r], t[r])
        want[r] = r % 2
        u[2 * r] = np.float32(ratio * (1 - 2.0 ** -15.9 if want[r] else 1 + 2.0 ** -15.9))  # (the number's own rounding: 2^-24)
        if not 0 < u[2 * r] < 0.9999:  # q no likelier than p: accepted whatever the number
            u[2 * r], want[r] = 0.5, ratio > 0.5
            assert abs(ratio - 0.5) > 1e-3
        else:
            sure += 1
    assert sure >= requests // 2
    accepted, _ = B.bl_verify(dev(l, BF if bf16 else F32), ints(np.stack([0 * x, x], 1).reshape(-1)), ints(2 * np.arange(requests + 1)), dev(u),
                              dev(u[:requests]), temperature=dev(t), draft_logits=dev(q, BF if bf16 else F32))
    assert np.array_equal(accepted.cpu().numpy(), want), np.nonzero(accepted.cpu().numpy() != want)


@gpu
@pytest.mark.parametrize("temperature", [1.0, 0.05])
def test_verify_a_number_of_zero_accepts_what_the_model_can_say(B, temperature):
    """u = 0 accepts every draft with p(x) > 0, given ones and a model's, and none without."""
    V = 5000
    l = np.zeros((8, V), np.float32)
    l[:, 30] = -20
    l[:, 40] = -np.inf
    l[:, 50] = -0.5 * 700 * temperature
    token = np.array([0, 30, 0, 40, 0, 50, 0, 60])
    q = np.zeros((8, V), np.float32)
    q[:, 50] = 30
    zero, t = np.zeros(8, np.float32), np.full(4, temperature, np.float32)
    for drafts in (None, dev(q)):
        accepted, _ = B.bl_verify(dev(l), ints(token), ints([0, 2, 4, 6, 8]), dev(zero), dev(zero[:4]), temperature=dev(t), draft_logits=drafts)
        assert accepted.tolist() == [1, 0, 1, 1]


# ---------------------------------------------------------------------------
# attention: waits that give up
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("f32", [True, False])
def test_attn_waits_that_run_out(B, f32):
    """With a test limit the roles give up: the call returns, says so, writes no row but its own (whatever an earlier
    call has left in the workspace), and the next one is right."""
    H, Hk, D = 40, 8, 128
    t = F32 if f32 else BF
    big, small = Cache([3000, 900, 2000, 1700, 2500, 1100], Hk, D, 16, 81), Cache([700, 1300], Hk, D, 16, 82)
    ws = B.attn_paged_workspace(60, H, Hk, D)
    buf = torch.empty(70, H, D, dtype=t, device="cuda")
    out = buf[:10]

    def call(cache, new, out):
        k, v, table, length = cache.gpu()
        n = len(cache.lengths)
        q = dev(bf16_round(rng(n, 83).standard_normal((n * new, H, D)).astype(np.float32)), BF)
        return B.bl_attn_paged(q, k, v, table, length, ints(np.arange(n + 1) * new), D ** -0.5, out=out, workspace=ws)
    want = call(small, 5, torch.empty(10, H, D, dtype=t, device="cuda"))
    for _ in range(2):
        call(big, 10, torch.empty(60, H, D, dtype=t, device="cuda"))  # leaves units of 60 rows that go on in other CTAs
        buf.fill_(5)
        torch.cuda.synchronize()
        B.set_wait_limit(1)
        try:
            call(small, 5, out)
            torch.cuda.synchronize()
        finally:
            B.set_wait_limit(0)
        assert B.device_error(clear=True) == B.BL_DEVERR_WAIT_TIMEOUT
        assert bool((buf[10:] == 5).all())
        assert torch.equal(call(small, 5, out), want)
        assert bool((buf[10:] == 5).all())


# ---------------------------------------------------------------------------
# attention: precision
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("H,Hk,D,new", [(10, 2, 128, 1), (10, 2, 128, 6), (8, 2, 64, 1), (40, 8, 80, 3), (16, 4, 256, 1)])
def test_attn_bf16_results_are_the_fp32_ones_rounded_once(B, H, Hk, D, new, wide):
    cache = Cache([900, 40, 2000, 333], Hk, D, 16, 91, wide=wide)
    k, v, table, length = cache.gpu()
    q = dev(bf16_round(1.3 * rng(H, D, new, 92).standard_normal((4 * new, H, D)).astype(np.float32)), BF)
    full, short = (B.bl_attn_paged(q, k, v, table, length, ints(np.arange(5) * new), D ** -0.5, out_dtype=t) for t in (F32, BF))
    assert torch.equal(full.to(BF), short)


# ---------------------------------------------------------------------------
# page maps: requests whose positions do not fit
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("requests", [3, 2100])
@pytest.mark.parametrize("tokens", [40, 5000])
def test_page_map_lengths_next_to_the_largest(B, requests, tokens):
    """New tokens of a request that comes to 2^31 - 1 tokens or more get no slot (they took those of earlier tokens)."""
    page, pages, W, most = 1 << 20, 2047, 2049, (1 << 31) - 1
    length, count, owned = np.zeros(requests, int), np.zeros(requests, int), np.zeros(requests, int)
    length[:3], count[:3], owned[:3] = (most - 7, most - 3, 5), (6, 5, 2), (2048, 2048, 1)
    table = torch.full((requests, W), -1, dtype=I32, device="cuda")
    table[:2] = torch.arange(W, device="cuda", dtype=I32) % pages
    table[2, 0] = 7
    start, position, slot, length_out, owned_out, left = B.bl_page_map(ints(length), ints(count), table, ints(owned), ints(np.arange(pages)), ints([4]), page, tokens)
    assert range_error(B)
    assert position[:6].tolist() == list(range(most - 7, most - 1))
    assert slot[:6].tolist() == [(p // page) % pages * page + p % page for p in range(most - 7, most - 1)]
    assert position[6:11].tolist() == [-1] * 5 and slot[6:11].tolist() == [-1] * 5
    assert position[11:13].tolist() == [5, 6] and slot[11:13].tolist() == [7 * page + 5, 7 * page + 6]
    assert length_out[:3].tolist() == [most - 1, most, 7] and bool((position[13:] == -1).all()) and bool((slot[13:] == -1).all())


# ---------------------------------------------------------------------------
# attention: scores that are large against the steps of fp32.  The keys' first coordinate alone makes them, in numbers that
# bf16, the products and their sums hold exactly, so the weights are 1 at the largest and 0 elsewhere: the values at the
# largest come out to 2^-21 (a weight's three terms and its sum, 2^-23 each, 1 / sum and the product, 2^-24 each; several
# equal ones add up in fp32, 2^-22).
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 20, 2.0 ** 24, 2.0 ** 28, 2.0 ** 29])
@pytest.mark.parametrize("H,Hk,D,new", [(10, 2, 128, 1), (10, 2, 128, 6), (8, 2, 64, 2), (4, 2, 256, 1)])
def test_attn_large_scores(B, H, Hk, D, new, size, sign, wide):
    g = rng(H, D, new, int(np.log2(size)))
    lengths = [300, 40, 1000]
    cache = Cache(lengths, Hk, D, 16, 95, wide=wide)
    level = [g.integers(0, 100, (n, Hk)) for n in lengths]  # of 128: (1 + level / 128) times the size
    for (k, _), l in zip(cache.rows, level):
        k[:] = 0
        k[:, :, 0] = sign * 64 * (1 + l / 128)
    for r, n in enumerate(lengths):
        for j in range(n):
            cache.k[cache.table[r, j // 16], :, j % 16] = cache.rows[r][0][j]
    k, v, table, length = cache.gpu()
    q = np.zeros((3 * new, H, D), np.float32)
    q[..., 0] = size / 64
    out = host(B.bl_attn_paged(dev(q, BF), k, v, table, length, ints(np.arange(4) * new), 1.0, out_dtype=F32))
    for r, n in enumerate(lengths):
        for t in range(new):
            for h in range(H):
                l = level[r][:n - new + t + 1, h // (H // Hk)] * sign
                best = cache.rows[r][1][:len(l), h // (H // Hk)][l == l.max()].astype(np.float64)
                assert np.all(np.abs(out[r * new + t, h] - best.mean(0)) <= 2.0 ** -21 * np.abs(best).mean(0)), (r, t, h)


# ---------------------------------------------------------------------------
# more requests than a CTA has threads; rows before the first request's; flat rows of the largest vocabulary
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("H,Hk,D,wide,most_new", [(2, 1, 64, False, 1), (4, 1, 128, True, 1), (12, 1, 128, False, 2), (2, 1, 256, False, 1)])
def test_attn_more_requests_than_threads(B, H, Hk, D, wide, most_new):
    g = rng(H, D, 101)
    lengths = [int(n) for n in g.integers(0, 40, 1700)]
    counts = [int(min(n, c)) for n, c in zip(lengths, g.integers(0, most_new + 1, 1700))]
    check_attn(B, Cache(lengths, Hk, D, 8, 102, wide=wide), counts, H, True, padding=2)


@gpu
@pytest.mark.parametrize("H,wide", [(4, False), (12, False), (2, True)])
def test_rows_before_the_first_request_are_left_alone(B, H, wide):
    D, before, counts = 128, 3, [2, 1, 4]
    cache = Cache([50, 300, 140], 1, D, 16, 103, wide=wide)
    k, v, table, length = cache.gpu()
    q = bf16_round(rng(H, 104).standard_normal((before + 7, H, D)).astype(np.float32))
    start = before + np.concatenate([[0], np.cumsum(counts)])
    out = torch.full((before + 7, H, D), 5.0, device="cuda")
    B.bl_attn_paged(dev(q, BF), k, v, table, length, ints(start), D ** -0.5, out=out)
    ref, cond, size = attn_ref(q[before:], cache, counts, D ** -0.5, 0, 0)
    assert bool((out[:before] == 5).all()) and np.all(np.abs(host(out)[before:] - ref) <= attn_bound(ref, cond, size, 300, D, True))
    l = (3 * rng(105).standard_normal((before + 7, 2000))).astype(np.float32)
    l[:before] = np.nan
    token, u, us = rng(106).integers(0, 2000, before + 7), np.full(before + 7, 1e-3, np.float32), np.float32([0.2, 0.5, 0.9])
    a = B.bl_verify(dev(l), ints(token), ints(start), dev(u), dev(us), draft_logits=dev(l[::-1]))
    b = B.bl_verify(dev(l[before:]), ints(token[before:]), ints(start - before), dev(u[before:]), dev(us), draft_logits=dev(l[::-1][before:]))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@gpu
@pytest.mark.parametrize("requests", [1, 9, 80])
@pytest.mark.parametrize("bf16", [True, False])
def test_verify_flat_rows_of_the_largest_vocabulary(B, requests, bf16):
    """The sums reach 2^63: token u V, from p alone and where nothing is left of p - q."""
    V = 524288
    l = torch.full((2 * requests, V), 1.5, dtype=BF if bf16 else F32, device="cuda")
    us = ((np.arange(requests) + 0.5) / requests).astype(np.float32)
    us[-1] = 0.99999994
    u, token = np.zeros(2 * requests, np.float32), np.resize([0, V], 2 * requests)  # out of range: refused
    for drafts in (None, l.clone()):
        accepted, got = B.bl_verify(l, ints(token), ints(2 * np.arange(requests + 1)), dev(u), dev(us), draft_logits=drafts)
        assert range_error(B)
        assert not accepted.any() and got.tolist() == [int(np.float64(x) * V) for x in us]
    _, got = B.bl_verify(l[:requests].contiguous(), ints(token[:requests] * 0), ints(np.arange(requests + 1)), dev(u[:requests]), dev(us))
    assert got.tolist() == [int(np.float64(x) * V) for x in us]


@gpu
@pytest.mark.parametrize("model", [False, True])
@pytest.mark.parametrize("top,temperature", [(20.0, 0.01), (20.0, 1e-3), (-20.0, 1e-3), (20.0, 1e-4), (-300.0, 1e-3), (5.0, 2e-5), (100.0, 3e-4), (1000.0, 0.01), (1e5, 1.0), (-4e5, 0.3)])
def test_verify_low_temperatures_beside_large_logits(B, top, temperature, model):
    """Exponents of 2^11 to 2^21, whose fractions are steps of fp32 still: the likely tokens lie within a few temperatures."""
    V, n = 5000, 64
    g = rng(72, int(abs(top)), int(1 / temperature))
    l, q = ((top - temperature * g.uniform(0, 9, (2 * n, V))).astype(np.float32) for _ in range(2))
    t = np.full(n, temperature, np.float32)
    us, u = g.random(n).astype(np.float32), g.random(2 * n).astype(np.float32)
    token = g.integers(0, V, 2 * n)
    accepted, got = B.bl_verify(dev(l), ints(token), ints(2 * np.arange(n + 1)), dev(u), dev(us), temperature=dev(t), draft_logits=dev(q) if model else None)
    for r in range(n):
        a, x, margin, w = R.verify(l[2 * r:2 * r + 2], q[2 * r:2 * r + 2] if model else None, token[2 * r:2 * r + 2], u[2 * r:2 * r + 2], us[r], t[r])
        if margin > 2.0 ** -15:
            assert accepted[r].item() == a, (r, margin)
            assert near(us[r], w, got[r].item()), (r, got[r].item())


# ---------------------------------------------------------------------------
# verification: the precision of light weights.  A row of one likely token and many with one light logit: all of these have
# the same error, so the border behind the first token shows it, times its distances to both ends.  Between 2^-8 and 2^-16 of the
# largest it is two roundings of an exponent, up to 2^-22 each, times ln 2; exp2's 2^-22; and six additions of fp32, 2^-24 each:
# 2^-20 in all, and, the roundings spread evenly, 2^-20 sqrt(0.14^2 + 0.25^2 + 0.09^2) = 0.30 2^-20 in the mean of the squares.
# The numbers' own steps are a tenth of 2^-20 there.
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("bf16", [True, False])
def test_verify_light_weights_move_no_border(B, bf16):
    n, V = 64, 20000
    tail = -rng(111).uniform(5.6, 9.6, n).astype(np.float32)
    tail = bf16_round(tail) if bf16 else tail
    l = dev(np.zeros((n, V), np.float32) + tail[:, None], BF if bf16 else F32)
    l[:, 0] = 0
    border = 1 / (1 + (V - 1) * np.exp(tail.astype(np.float64)))
    low = border.astype(np.float32).view(np.int32) - 200  # numbers as their bits: token 0 below, others above
    high = low + 400
    zero = dev(np.zeros(n, np.float32))
    while np.any(high - low > 1):
        mid = (low + high) // 2
        _, got = B.bl_verify(l, ints(np.zeros(n)), ints(np.arange(n + 1)), zero, dev(mid.view(np.float32)))
        first = got.cpu().numpy() == 0
        low, high = np.where(first, mid, low), np.where(first, high, mid)
    off = ((low.view(np.float32).astype(np.float64) + high.view(np.float32)) / 2 - border) / (border * (1 - border)) * 2.0 ** 20
    assert np.all(np.abs(off) <= 1.1) and np.sqrt(np.mean(off ** 2)) <= 0.33, (np.abs(off).max(), np.sqrt(np.mean(off ** 2)))
