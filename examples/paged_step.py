"""Decoding with drafted tokens over a paged key-value cache: one attention layer and a binary LM head.

    python examples/paged_step.py [--requests 8] [--drafts 3] [--steps 16] [--vocab 248320] [--temperature 0.2]

The weights are packed (i2_s for the products, W1A8 for the head); random weights stand in for a model's, and a table of
followers for whatever drafts tokens.  Per step and request the last known token and its drafts go in: pages and cache slots
for them, norm + int8 codes, the packed qkv product, rotary positions and the cache's new rows, attention over the pages, the
output product, the head, and the verification.  The step is captured in a CUDA graph: lengths, counts and tokens stay on
the device, and of refused drafts only the length is taken back.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from gemm_bl_gemv_gb300 import binding as B  # noqa: E402

I32 = dict(dtype=torch.int32, device="cuda")


class Model:
    """The packed weights, the embedding, the angles and the drafts' table of followers."""

    def __init__(self, vocab, heads=20, kv_heads=5, dim=128, positions=8192, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        pack = lambda n, k: B.bl_pack_i2s(torch.randint(-1, 2, (n, k), generator=g, device="cuda", dtype=torch.int8), k ** -0.5)  # noqa: E731
        self.vocab, self.heads, self.kv_heads, self.dim, self.hidden = vocab, heads, kv_heads, dim, heads * dim
        self.rows = (heads + 2 * kv_heads) * dim
        self.qkv, self.out = pack(self.rows, self.hidden), pack(self.hidden, self.hidden)
        self.head = B.bl_pack_w1(torch.where(randn(vocab, self.hidden) > 0, 1, -1).to(torch.int8))
        self.head_scale = torch.full((vocab, self.hidden // 128), 2 * self.hidden ** -0.5, device="cuda", dtype=torch.float16)
        self.embedding = randn(vocab, self.hidden).to(torch.bfloat16)
        self.norm, self.out_norm, self.final_norm = ((1 + 0.1 * randn(self.hidden)).to(torch.bfloat16) for _ in range(3))
        angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2 * torch.arange(dim // 2, device="cuda") / dim)
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        # what the head makes of a token's embedding alone: often what the whole model answers
        self.follower = torch.cat([self.logits(self.embedding[i:i + 2048]).argmax(1) for i in range(0, vocab, 2048)]).to(torch.int32)

    def logits(self, x, residual=None):
        q, s, _, _ = B.bl_rmsnorm_quant_int8(x, self.final_norm, residual=residual)
        return B.bl_gemm_w1a8(q, s, self.head, self.head_scale.view(torch.uint16))


class Requests:
    """The caches, the block tables and what is known of each request."""

    def __init__(self, model, requests, longest, page=16):
        per = -(-longest // page)
        self.page, pages = page, requests * per
        self.k, self.v = (torch.zeros(pages, model.kv_heads, page, model.dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.table = torch.full((requests, per), -1, **I32)
        self.free, self.free_count = torch.arange(pages, **I32), torch.full((1,), pages, **I32)
        self.length, self.owned = torch.zeros(requests, **I32), torch.zeros(requests, **I32)
        self.last = torch.zeros(requests, **I32)
        self.accepted, self.next = torch.zeros(requests, **I32), torch.zeros(requests, **I32)


def forward(model, req, token, count):
    """(start, logits) of the new tokens (int32 [rows], count[r] of them for request r); their k and v are in the cache."""
    M = token.shape[0]
    start, position, slot, _, _, _ = B.bl_page_map(req.length, count, req.table, req.owned, req.free, req.free_count, req.page, M,
                                                   length_out=req.length, owned_out=req.owned, free_left=req.free_count)
    x = model.embedding[token.long()]
    q, s, _, _ = B.bl_rmsnorm_quant_int8(x, model.norm)
    qkv = B.bl_gemm_i2s_int8(q, s, model.qkv, model.rows)
    q = B.bl_rope_append(qkv, model.cos, model.sin, position, slot, req.k, req.v, model.heads)
    o = B.bl_attn_paged(q, req.k, req.v, req.table, req.length, start, model.dim ** -0.5)
    q, s, _, _ = B.bl_rmsnorm_quant_int8(o.view(M, model.hidden), model.out_norm)
    y = B.bl_gemm_i2s_int8(q, s, model.out, model.hidden).to(torch.bfloat16)
    return start, model.logits(y, residual=x)


def prompt(model, req, tokens):
    """The requests' first tokens (int32 [requests, n]); the last one is left to the first step."""
    R, n = tokens.shape
    forward(model, req, tokens[:, :-1].reshape(-1).contiguous(), torch.full((R,), n - 1, **I32))
    req.last.copy_(tokens[:, -1])


def step(model, req, drafts, u, u_sample, temperature):
    """One step of all requests: accepted[r] drafts and one token more (req.accepted, req.next)."""
    token = [req.last]
    for _ in range(drafts):
        token.append(model.follower[token[-1].long()])
    token = torch.stack(token, 1).reshape(-1)
    count = torch.full_like(req.length, drafts + 1)
    start, logits = forward(model, req, token, count)
    B.bl_verify(logits, token, start, u, u_sample, temperature=temperature, accepted=req.accepted, next_token=req.next)
    req.length.sub_(drafts - req.accepted)  # refused drafts leave; their pages stay owned for the tokens to come
    req.last.copy_(req.next)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=3)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--vocab", type=int, default=248320)
    ap.add_argument("--temperature", type=float, default=0.2)
    a = ap.parse_args()
    model = Model(a.vocab)
    req = Requests(model, a.requests, 64 + (a.steps + 3) * (a.drafts + 1))
    g = torch.Generator(device="cuda").manual_seed(1)
    prompt(model, req, torch.randint(0, a.vocab, (a.requests, 32), generator=g, **I32))
    u, u_sample = torch.empty(a.requests * (a.drafts + 1), device="cuda"), torch.empty(a.requests, device="cuda")
    temperature = torch.full((a.requests,), a.temperature, device="cuda")

    def numbers():
        u.uniform_(generator=g)
        u_sample.uniform_(generator=g)

    numbers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(model, req, a.drafts, u, u_sample, temperature)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(model, req, a.drafts, u, u_sample, temperature)
    for i in range(a.steps):
        numbers()
        graph.replay()
        print("step %2d: accepted %s  next %s" % (i, req.accepted.tolist(), req.next.tolist()))
    print("lengths %s, %d pages free, device error %d" % (req.length.tolist(), req.free_count.item(), B.device_error()))


if __name__ == "__main__":
    main()
