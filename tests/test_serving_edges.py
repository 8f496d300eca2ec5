"""Edges of the operators around the products: limits of their parameters, values at the ends of their types, and
the precision of fp32 results.  Tolerances are derived beside each test."""
import numpy as np
import pytest
import torch

import serving_ref as R
from test_serving_ops import B, dev, host, no_device_error, rng, run_lora  # noqa: F401

gpu = pytest.mark.gpu


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
