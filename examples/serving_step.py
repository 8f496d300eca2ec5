"""One decode step of several requests through a ternary MLP block and a binary LM head, each request with its own
low-rank adapter and its own sampling parameters.

    python examples/serving_step.py [--requests 8] [--hidden 2560] [--inner 6912] [--vocab 248320]

The base weights are shared and stay packed (i2_s for the MLP, W1A8 for the head); random weights stand in for a model's.
Per step: residual + RMSNorm + int8 codes in one call, the packed products on the codes, the requests' adapters beside the
up projection, a second norm, the head, and a token per request.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from gemm_bl_gemv_gb300 import binding as B  # noqa: E402


class Model:
    """The shared packed weights, and the stacked adapters of the up projection."""

    def __init__(self, hidden, inner, vocab, adapters, rank, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        ternary = lambda n, k: torch.randint(-1, 2, (n, k), generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.hidden, self.inner, self.vocab = hidden, inner, vocab
        self.gate, self.up = (B.bl_pack_i2s(ternary(inner, hidden), hidden ** -0.5) for _ in range(2))
        self.down = B.bl_pack_i2s(ternary(hidden, inner), inner ** -0.5)
        self.head = B.bl_pack_w1(torch.where(randn(vocab, hidden) > 0, 1, -1).to(torch.int8))
        self.head_scale = torch.full((vocab, hidden // 128), 2 * hidden ** -0.5, device="cuda", dtype=torch.float16)
        self.norm, self.inner_norm, self.final_norm = (
            (1 + 0.1 * randn(n)).to(torch.bfloat16) for n in (hidden, inner, hidden))
        self.lora_a = (randn(adapters, rank, hidden) * hidden ** -0.5).to(torch.bfloat16)
        self.lora_b = (randn(adapters, inner, rank) * 0.1).to(torch.bfloat16)
        self.lora_scale = torch.full((adapters,), 2.0 / rank, device="cuda")


def step(model, x, residual, adapter, u, temperature, top_k, top_p, min_p):
    """(token, prob, logits): one token per request.  x and residual bf16 [requests, hidden]; adapter int32 (-1: none)."""
    q, s, h, y = B.bl_rmsnorm_quant_int8(x, model.norm, residual=residual, y=True)
    gate = B.bl_gemm_i2s_int8(q, s, model.gate, model.inner)
    up = B.bl_gemm_i2s_int8(q, s, model.up, model.inner)
    B.bl_lora_add(y, adapter, model.lora_a, model.lora_b, model.lora_scale, up, y=up)  # in place, beside the shared product
    inner = torch.relu(gate).square_().mul_(up).to(torch.bfloat16)
    q, s, _, _ = B.bl_rmsnorm_quant_int8(inner, model.inner_norm)
    mlp = B.bl_gemm_i2s_int8(q, s, model.down, model.hidden).to(torch.bfloat16)
    q, s, h, _ = B.bl_rmsnorm_quant_int8(mlp, model.final_norm, residual=h)
    logits = B.bl_gemm_w1a8(q, s, model.head, model.head_scale.view(torch.uint16))
    token, prob = B.bl_sample(logits, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p, prob=True)
    return token, prob, logits


def inputs(requests, hidden, adapters, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, residual = (torch.randn(requests, hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    i = torch.arange(requests, device="cuda")
    adapter = torch.where(i % 4 == 3, -1, i % adapters).to(torch.int32)
    u = torch.rand(requests, generator=g, device="cuda")
    temperature = torch.where(i % 5 == 4, 0.0, 0.7 + 0.1 * (i % 3))  # every fifth request is greedy
    top_k = torch.where(i % 2 == 0, 50, 0).to(torch.int32)
    top_p = torch.where(i % 3 == 0, 0.9, 1.0)
    min_p = torch.where(i % 3 == 1, 0.05, 0.0)
    return x, residual, adapter, u, temperature, top_k, top_p, min_p


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=2560)
    ap.add_argument("--inner", type=int, default=6912)
    ap.add_argument("--vocab", type=int, default=248320)
    a = ap.parse_args()
    model = Model(a.hidden, a.inner, a.vocab, adapters=4, rank=16)
    v = inputs(a.requests, a.hidden, 4)
    token, prob, _ = step(model, *v)
    for r in range(a.requests):
        print("request %d: adapter %2d  temperature %.1f  token %6d  prob %.4f" % (r, v[2][r], v[4][r], token[r], prob[r]))


if __name__ == "__main__":
    main()
