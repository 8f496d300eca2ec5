"""Workloads of a decode step over a paged key-value cache: page maps, rotary positions with the cache's rows, attention of
the new tokens, verification of drafted tokens.

Each case is one call as a serving loop makes it.  ``run`` computes it in
elementary torch operations, or, with ``own`` true, by the library's entry
points.  ``exact`` gives the outputs from the definitions in 64 bits.

  pages   from the requests' lengths and counts of new tokens: pages from a stack of free ones into the block tables, the
          new tokens' positions and cache slots (page * page size + offset).
  rope    the heads of q and k turned by their token's position, k and v stored at the token's slot of the paged cache.
  attn    softmax(scale q k^T) v of each request's new tokens over its cached ones, causal, with an optional window and
          first tokens that stay visible; a row that sees nothing is 0.
  verify  of each request's drafted tokens, accepted from the left while u q(x) < p(x); then one token from max(p - q, 0)
          where a draft was refused, from p after the last draft (p, q: softmax of logits / temperature; q is 1 at the
          draft where no draft logits are given).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GREEDY_BELOW = 1e-5  # temperatures under this leave the largest logits


def listed():
    return [
        # a decode step: one token for each of 64 requests, pages of 16 tokens
        {"name": "pages_decode", "op": "pages", "requests": 64, "longest": 8192, "page": 16, "new": 1, "prompts": 0, "prompt": 0, "padding": 0},
        # chunked prompts beside decoding requests, in a batch padded to a captured size
        {"name": "pages_mixed", "op": "pages", "requests": 256, "longest": 32768, "page": 16, "new": 5, "prompts": 12, "prompt": 640, "padding": 77},
        # one token of one request, 2560 wide
        {"name": "rope_token", "op": "rope", "tokens": 1, "heads": 20, "kv_heads": 5, "dim": 128, "rotary": 128, "page": 16, "dtype": "bf16"},
        # drafted tokens of 64 requests after the int8 products, whose results are fp32; 5120 wide
        {"name": "rope_drafts_f32", "op": "rope", "tokens": 311, "heads": 40, "kv_heads": 8, "dim": 128, "rotary": 128, "page": 32, "dtype": "f32"},
        # several long prompts at once
        {"name": "rope_prompts", "op": "rope", "tokens": 8192, "heads": 20, "kv_heads": 5, "dim": 128, "rotary": 128, "page": 16, "dtype": "bf16"},
        # one request with a middling context, one token
        {"name": "attn_token", "op": "attn", "requests": 1, "longest": 4096, "heads": 20, "kv_heads": 5, "dim": 128, "page": 16, "new": 1,
         "window": 0, "sinks": 0, "out": "bf16"},
        # a decode batch of uneven lengths, 5120 wide
        {"name": "attn_batch", "op": "attn", "requests": 64, "longest": 8192, "heads": 40, "kv_heads": 8, "dim": 128, "page": 16, "new": 1,
         "window": 0, "sinks": 0, "out": "bf16"},
        # few requests with very long contexts: the work has to be split over the length
        {"name": "attn_long", "op": "attn", "requests": 3, "longest": 131072, "heads": 20, "kv_heads": 5, "dim": 128, "page": 64, "new": 1,
         "window": 0, "sinks": 0, "out": "bf16"},
        # drafted tokens beside the last one, a window with the first tokens kept, fp32 results for a norm with codes
        {"name": "attn_drafts_window", "op": "attn", "requests": 48, "longest": 20000, "heads": 40, "kv_heads": 8, "dim": 128, "page": 32,
         "new": 5, "window": 4096, "sinks": 4, "out": "f32"},
        # one request with four tokens drafted by lookup, against the LM head's logits
        {"name": "verify_token", "op": "verify", "requests": 1, "drafts": 4, "even": True, "vocab": 248320, "dtype": "bf16", "model": False},
        # a batch whose requests have none to four tokens from a draft model
        {"name": "verify_batch", "op": "verify", "requests": 64, "drafts": 4, "even": False, "vocab": 248320, "dtype": "bf16", "model": True},
        # fp32 logits and an odd vocabulary
        {"name": "verify_f32", "op": "verify", "requests": 32, "drafts": 7, "even": False, "vocab": 100003, "dtype": "f32", "model": True},
    ]


def _spread(rng, lo, hi):
    """An integer in [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["pages", "rope", "attn", "attn", "verify"])
    if op == "pages":
        case = {"op": op, "requests": _spread(rng, 1, 256), "longest": _spread(rng, 1, 32768), "page": rng.choice([8, 16, 16, 32, 64, 128]),
                "new": _spread(rng, 1, 8), "prompts": 0, "prompt": 0, "padding": rng.choice([0, _spread(rng, 1, 256)])}
        if rng.random() < 0.5:
            case["prompts"], case["prompt"] = rng.randint(1, min(12, case["requests"])), _spread(rng, 1, 640)
        shrink, most = ("requests", "longest", "prompt"), listed()[1]
    elif op == "rope":
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        kv = rng.choice([1, 2, 4, 5, 8])
        case = {"op": op, "tokens": _spread(rng, 1, 8192), "heads": kv * rng.choice([1, 2, 4, 5, 8]), "kv_heads": kv, "dim": dim,
                "rotary": dim if rng.random() < 0.7 else dim // 2, "page": rng.choice([8, 16, 16, 32, 64, 128]), "dtype": rng.choice(["bf16", "f32"])}
        shrink, most = ("tokens",), listed()[4]
    elif op == "attn":
        kv = rng.choice([1, 2, 4, 5, 8])
        case = {"op": op, "requests": _spread(rng, 1, 64), "longest": _spread(rng, 1, 131072), "heads": kv * rng.choice([1, 2, 4, 5, 8]),
                "kv_heads": kv, "dim": rng.choice([64, 80, 96, 128, 128, 128, 256]), "page": rng.choice([8, 16, 16, 32, 64, 128]),
                "new": rng.choice([1, 1, 1, _spread(rng, 2, 8)]), "window": 0, "sinks": 0, "out": rng.choice(["bf16", "bf16", "f32"])}
        if rng.random() < 0.3:
            case["window"], case["sinks"] = _spread(rng, 16, 8192), rng.choice([0, 1, 4, 64])
        shrink, most = ("longest",), listed()[8 if case["new"] > 1 else 6]
    else:
        case = {"op": op, "requests": _spread(rng, 1, 64), "drafts": _spread(rng, 1, 8), "even": rng.random() < 0.3,
                "vocab": _spread(rng, 1000, 262144), "dtype": rng.choice(["bf16", "bf16", "f32"]), "model": rng.random() < 0.6}
        shrink, most = ("requests",), listed()[10]
    limit = work(most)
    while any(work(case)[k] > limit[k] for k in ("bytes", "flops")):
        for name in shrink:
            case[name] = max(case[name] * 3 // 4, min(case[name], 1))
        if op == "pages":
            case["prompts"] = min(case["prompts"], case["requests"])
    return case


def _lengths(case):
    """Tokens in the cache before the step: spread evenly over (0, longest], the first request's the longest."""
    n = case["requests"]
    return [max(1, case["longest"] - case["longest"] * ((r * 19) % n) // n) for r in range(n)]


def _counts(case):
    """New tokens of each request."""
    if case["op"] == "pages":
        n = case["requests"]
        prompt = {n * i // max(case["prompts"], 1) for i in range(case["prompts"])}
        return [case["prompt"] - 13 * (r % 7) % case["prompt"] if r in prompt else 1 + r % case["new"] for r in range(n)]
    if case["op"] == "attn":  # of those that decode drafts, some have fewer
        return [min(length, 1 + (case["new"] - 1 if r % 4 else (case["new"] - 1) // 2)) for r, length in enumerate(_lengths(case))]
    return [1 + (case["drafts"] if case["even"] else (r * 3 + 2) % (case["drafts"] + 1)) for r in range(case["requests"])]


def _starts(case):
    return [0] + [int(s) for s in np.cumsum(_counts(case))]


def _visible(case, length, count):
    """(first tokens, from, tokens): a request's new tokens see [0, first) and [from, tokens) between them."""
    w = case["window"]
    low = max(0, length - count + 1 - w) if w else 0
    return min(case["sinks"], low) if w else 0, low, length


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    rand = lambda *shape: torch.rand(*shape, generator=g, device="cuda")  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    empty = lambda *shape: torch.empty(*shape, dtype=torch.int32, device="cuda")  # noqa: E731
    permuted = lambda n: torch.randperm(n, generator=g, device="cuda").to(torch.int32)  # noqa: E731
    state = {"case": case}
    if case["op"] == "pages":
        R, P = case["requests"], case["page"]
        length, count = _lengths(case), _counts(case)
        # the seed moves the lengths within a page; some requests own a page ahead, left by refused drafts
        move = np.random.default_rng(seed).integers(0, P, R)
        length = [n + int(m) for n, m in zip(length, move)]
        owned = [-(-n // P) + (r % 5 == 3) for r, n in enumerate(length)]
        # the same for every seed
        W = max(-(-(n + c) // P) for n, c in zip(_lengths(case), count)) + 3
        pages = sum(-(-n // P) + 2 for n in _lengths(case)) + sum(-(-c // P) + 1 for c in count)
        pool = permuted(pages)
        table = torch.full((R, W), -1, dtype=torch.int32, device="cuda")
        mine = torch.arange(W, device="cuda") < torch.tensor(owned, device="cuda")[:, None]
        table[mine] = pool[: sum(owned)]
        free = torch.zeros(pages, dtype=torch.int32, device="cuda")
        free[: pages - sum(owned)] = pool[sum(owned):]
        M = sum(count) + case["padding"]
        state.update(length=ints(length), count=ints(count), owned=ints(owned), table=table, free=free,
                     free_count=ints([pages - sum(owned)]), tokens=M,
                     out=dict(start=empty(R + 1), position=empty(M), slot=empty(M), length_out=empty(R), owned_out=empty(R), free_left=empty(1)))
    elif case["op"] == "rope":
        M, H, Hk, D, P = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "page"))
        most = 32768
        angle = torch.arange(most, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** -(
            torch.arange(case["rotary"] // 2, device="cuda", dtype=torch.float64) * 2 / case["rotary"])
        state["cos"], state["sin"] = torch.cos(angle).float(), torch.sin(angle).float()
        state["qkv"] = randn(M, (H + 2 * Hk) * D).to(DTYPES[case["dtype"]])
        state["position"] = torch.randint(0, most, (M,), generator=g, device="cuda", dtype=torch.int32)
        pages = -(-M // P) * 2 + 3
        state["slot"] = permuted(pages * P)[:M].contiguous()
        state["k_cache"], state["v_cache"] = (randn(pages, Hk, P, D).to(torch.bfloat16) for _ in range(2))
        state["q"] = torch.empty(M, H, D, dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "attn":
        R, H, Hk, D, P = (case[k] for k in ("requests", "heads", "kv_heads", "dim", "page"))
        length = _lengths(case)
        state["lengths"], state["starts"] = length, _starts(case)
        M = state["starts"][-1]
        W = -(-max(length) // P) + 1
        owned = [-(-n // P) for n in length]
        pages = sum(owned) + 5
        table = torch.full((R, W), -1, dtype=torch.int32, device="cuda")
        mine = torch.arange(W, device="cuda") < torch.tensor(owned, device="cuda")[:, None]
        table[mine] = permuted(pages)[: sum(owned)]
        state.update(table=table, length=ints(length), start=ints(state["starts"]))
        # keys with a common part and queries that look for some of them, so that weights are uneven as a model's are
        state["k_cache"] = (randn(pages, Hk, P, D) + randn(Hk, 1, D)).to(torch.bfloat16)
        state["v_cache"] = randn(pages, Hk, P, D).to(torch.bfloat16)
        state["q"] = (1.5 * randn(M, H, D)).to(torch.bfloat16)
        state["scale"] = D ** -0.5
        state["out"] = torch.empty(M, H, D, dtype=DTYPES[case["out"]], device="cuda")
        if own:
            from gemm_bl_gemv_gb300 import binding as B
            state["workspace"] = B.attn_paged_workspace(M, H, Hk, D)
    else:
        R, V = case["requests"], case["vocab"]
        state["starts"] = starts = _starts(case)
        M = starts[-1]
        request = np.repeat(np.arange(R), np.diff(starts))
        # a model's logits: a broad bulk, and a short head of likely tokens that differs by row
        logits = 2.0 * randn(M, V) - 2.0
        head = torch.arange(40, device="cuda") * (V // 40) + torch.randint(0, V // 40, (M, 40), generator=g, device="cuda")
        logits.scatter_(1, head, 9.0 + 3.0 * randn(M, 40))
        t = 0.5 + rand(R)
        t = torch.where(torch.randint(0, 8, (R,), generator=g, device="cuda") == 7, 0.0, t)
        each = t[torch.from_numpy(request).cuda()]
        state["temperature"] = t
        state["logits"] = logits.to(DTYPES[case["dtype"]])
        if case["model"]:  # a smaller model's logits are near the target's
            drafts = logits + 0.7 * randn(M, V)
            state["draft_logits"] = drafts.to(DTYPES[case["dtype"]])
            noise = -torch.log(-torch.log(rand(M, V).clamp(1e-7, 1 - 1e-7)))
            drafted = (state["draft_logits"].float() + each[:, None] * noise).argmax(1)
        else:  # a lookup is often right
            state["draft_logits"] = None
            drafted = torch.where(rand(M) < 0.7, state["logits"].float().argmax(1), head[:, 0])
        token = torch.randint(0, V, (M,), generator=g, device="cuda")
        token[1:] = torch.where(torch.from_numpy(request[1:] == request[:-1]).cuda(), drafted[:-1], token[1:])
        state.update(token=token.to(torch.int32), start=ints(starts), u=rand(M), u_sample=rand(R), accepted=empty(R), next_token=empty(R))
        if own:
            from gemm_bl_gemv_gb300 import binding as B
            state["workspace"] = B.verify_workspace(M)
    return state


# ---- plain forms -------------------------------------------------------------

def _pages_plain(s):
    P, M = s["case"]["page"], s["tokens"]
    R, W = s["table"].shape
    length, count, owned = s["length"].long(), s["count"].long(), s["owned"].long()
    total = length + count
    ask = ((total + P - 1) // P - owned).clamp(min=0)
    before = torch.cumsum(ask, 0) - ask
    left = s["free_count"].long()
    j = torch.arange(W, device="cuda") - owned[:, None]  # [R, W]: which of the asked pages an entry is
    k = before[:, None] + j
    fresh = (j >= 0) & (j < ask[:, None])
    page = torch.where(k < left, s["free"].long()[(left - 1 - k).clamp(0, s["free"].numel() - 1)], -1)
    table = torch.where(fresh, page, s["table"].long())
    start = torch.nn.functional.pad(torch.cumsum(count, 0), (1, 0))
    i = torch.arange(M, device="cuda")
    r = torch.searchsorted(start, i, right=True) - 1
    live = r < R
    r = r.clamp(max=R - 1)
    position = length[r] + i - start[r]
    page = table[r, (position // P).clamp(max=W - 1)]
    slot = torch.where(page >= 0, page * P + position % P, -1)
    s["table"].copy_(table)
    return {"start": start.int(), "position": torch.where(live, position, -1).int(), "slot": torch.where(live, slot, -1).int(),
            "length": total.int(), "owned": (owned + torch.minimum(ask, (left - before).clamp(min=0))).int(),
            "free_left": (left - torch.minimum(ask.sum(), left)).int(), "table": s["table"]}


def _rope_plain(s):
    M, H, Hk, D, P = (s["case"][k] for k in ("tokens", "heads", "kv_heads", "dim", "page"))
    x = s["qkv"].float().reshape(M, H + 2 * Hk, D)
    half = s["cos"].shape[1]
    cos, sin = (s[n][s["position"].long()][:, None, :] for n in ("cos", "sin"))
    a, b = x[:, : H + Hk, :half], x[:, : H + Hk, half: 2 * half]
    turned = torch.cat([a * cos - b * sin, b * cos + a * sin, x[:, : H + Hk, 2 * half:]], 2).to(torch.bfloat16)
    page, at = s["slot"].long() // P, s["slot"].long() % P
    s["k_cache"][page, :, at] = turned[:, H:]
    s["v_cache"][page, :, at] = x[:, H + Hk:].to(torch.bfloat16)
    return {"q": turned[:, :H].contiguous(), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attn_plain(s):
    case = s["case"]
    H, Hk, D, P = (case[k] for k in ("heads", "kv_heads", "dim", "page"))
    for r, n in enumerate(s["lengths"]):
        a, b = s["starts"][r], s["starts"][r + 1]
        pages = s["table"][r, : -(-n // P)].long()
        k, v = (s[c][pages].permute(1, 0, 2, 3).reshape(Hk, -1, D)[:, :n].float() for c in ("k_cache", "v_cache"))
        q = s["q"][a:b].float().reshape(b - a, Hk, H // Hk, D).permute(1, 0, 2, 3)  # [Hk, t, G, D]
        z = (q.reshape(Hk, -1, D) @ k.transpose(1, 2)).reshape(Hk, b - a, H // Hk, n) * s["scale"]
        at = torch.arange(n, device="cuda")
        mine = torch.arange(n - (b - a), n, device="cuda")[:, None]
        seen = at <= mine
        if case["window"]:
            seen = seen & ((mine - at < case["window"]) | (at < case["sinks"]))
        z = torch.where(seen[:, None, :], z, -math.inf)
        w = torch.exp(z - z.amax(3, keepdim=True))
        o = (w.reshape(Hk, -1, n) @ v).reshape(Hk, b - a, H // Hk, D) / w.sum(3, keepdim=True)
        s["out"][a:b] = o.permute(1, 0, 2, 3).reshape(b - a, H, D).to(s["out"].dtype)
    return s["out"]


def _shares(logits, t):
    """softmax(logits / t) by row in 64 bits (cumulative masses lie next to borders); 0 for a row of -inf."""
    z = logits.double()
    z = torch.where(torch.isnan(z), -math.inf, z)
    top = z.amax(1, keepdim=True)
    w = torch.exp((z - top) / t.double()[:, None])
    w = torch.where(z == top, 1.0, torch.where(t[:, None] >= GREEDY_BELOW, w, 0.0))
    w = torch.where(z > -math.inf, w, 0.0)
    mass = w.sum(1, keepdim=True)
    return torch.where(mass > 0, w / mass, 0.0)


def _verify_plain(s):
    case = s["case"]
    R = case["requests"]
    start, token = s["start"].long(), s["token"].long()
    drafts = start[1:] - start[:-1] - 1
    M = token.numel()
    request = torch.repeat_interleave(torch.arange(R, device="cuda"), drafts + 1, output_size=M)
    t = s["temperature"][request]
    p = _shares(s["logits"], t)
    x = torch.cat([token[1:], token[:1]])[:, None]  # row i is asked about token i + 1
    px = torch.gather(p, 1, x)[:, 0]
    if s["draft_logits"] is None:
        qx = torch.ones_like(px)
    else:
        q = _shares(s["draft_logits"], t)
        qx = torch.gather(q, 1, x)[:, 0]
    good = s["u"].double() * qx < px
    most = case["drafts"]
    j = torch.arange(most, device="cuda")
    at = (start[:-1, None] + j).clamp(max=M - 1)
    accepted = torch.cumprod((good[at] & (j < drafts[:, None])).long(), 1).sum(1)
    stop = start[:-1] + accepted
    refused = accepted < drafts
    share = p[stop]
    if s["draft_logits"] is None:
        other = torch.zeros_like(share).scatter_(1, x[stop], math.inf)
    else:
        other = q[stop]
    rest = (share - torch.where(refused[:, None], other, 0.0)).clamp(min=0)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, share)
    mass = torch.cumsum(rest, 1)
    place = (mass <= s["u_sample"].double()[:, None] * mass[:, -1:]).sum(1)
    last = (torch.where(rest > 0, torch.arange(rest.shape[1], device="cuda"), -1)).amax(1)
    return {"accepted": accepted.int(), "next_token": torch.minimum(place, last).int()}


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"pages": _pages_plain, "rope": _rope_plain, "attn": _attn_plain, "verify": _verify_plain}[op](state)
    from gemm_bl_gemv_gb300 import binding as B
    s = state
    if op == "pages":
        start, position, slot, length, owned, left = B.bl_page_map(
            s["length"], s["count"], s["table"], s["owned"], s["free"], s["free_count"], s["case"]["page"], s["tokens"], **s["out"])
        return {"start": start, "position": position, "slot": slot, "length": length, "owned": owned, "free_left": left, "table": s["table"]}
    if op == "rope":
        q = B.bl_rope_append(s["qkv"], s["cos"], s["sin"], s["position"], s["slot"], s["k_cache"], s["v_cache"], s["case"]["heads"], q=s["q"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "attn":
        return B.bl_attn_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["length"], s["start"], s["scale"], window=s["case"]["window"],
                               sinks=s["case"]["sinks"], out=s["out"], workspace=s["workspace"])
    accepted, token = B.bl_verify(s["logits"], s["token"], s["start"], s["u"], s["u_sample"], draft_logits=s["draft_logits"],
                                  temperature=s["temperature"], accepted=s["accepted"], next_token=s["next_token"], workspace=s["workspace"])
    return {"accepted": accepted, "next_token": token}


def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "pages":
        M = sum(_counts(case)) + case["padding"]
        R, P = case["requests"], case["page"]
        fresh = sum(-(-c // P) for c in _counts(case))
        # lengths, counts, owned and what becomes of them, starts; positions and slots; fresh entries and where they come from
        return {"bytes": 24 * R + 8 * M + 8 * fresh, "flops": 10 * (R + M)}
    if case["op"] == "rope":
        M, H, Hk, D = (case[k] for k in ("tokens", "heads", "kv_heads", "dim"))
        return {"bytes": M * (H + 2 * Hk) * D * (size[case["dtype"]] + 2) + M * (8 + 4 * case["rotary"]), "flops": 3 * M * (H + Hk) * D}
    if case["op"] == "attn":
        H, Hk, D = (case[k] for k in ("heads", "kv_heads", "dim"))
        out = {"bytes": 0, "flops": 0}
        for n, c in zip(_lengths(case), _counts(case)):
            first, low, high = _visible(case, n, c)
            out["bytes"] += (first + high - low) * (Hk * D * 4 + 4 / case["page"]) + c * H * D * (2 + size[case["out"]]) + 8
            out["flops"] += 4 * c * H * D * (first + high - low)
        return {k: int(v) for k, v in out.items()}
    rows = sum(_counts(case))
    drafted = rows - case["requests"]
    logits = rows + (drafted if case["model"] else 0)
    return {"bytes": logits * case["vocab"] * size[case["dtype"]] + 8 * rows + 20 * case["requests"], "flops": 4 * logits * case["vocab"]}


# ---- the definitions in 64 bits -----------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pages":
        host = lambda n: s[n].cpu().numpy().astype(np.int64)  # noqa: E731
        length, count, owned, table, free = (host(n) for n in ("length", "count", "owned", "table", "free"))
        left, P, M = int(host("free_count")[0]), case["page"], s["tokens"]
        start, position, slot = [0], [], []
        for r in range(case["requests"]):
            while owned[r] * P < length[r] + count[r] and left > 0:
                left -= 1
                table[r, owned[r]] = free[left]
                owned[r] += 1
            for i in range(count[r]):
                at = int(length[r]) + i
                position.append(at)
                slot.append(int(table[r, at // P]) * P + at % P if at // P < owned[r] else -1)
            start.append(start[-1] + int(count[r]))
        position += [-1] * (M - len(position))
        slot += [-1] * (M - len(slot))
        return {"start": np.asarray(start, np.int32), "position": np.asarray(position, np.int32), "slot": np.asarray(slot, np.int32),
                "length": (length + count).astype(np.int32), "owned": owned.astype(np.int32), "free_left": np.asarray([left], np.int32),
                "table": table.astype(np.int32)}
    if case["op"] == "rope":
        M, H, Hk, D, P = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "page"))
        x = s["qkv"].double().reshape(M, H + 2 * Hk, D)
        half = case["rotary"] // 2
        # a pair of coordinates as a complex number, turned by the table's angle
        turn = torch.complex(s["cos"].double(), s["sin"].double()).index_select(0, s["position"].long())
        z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * turn.unsqueeze(1)
        turned = x.clone()
        turned[:, : H + Hk, :half], turned[:, : H + Hk, half:2 * half] = z.real[:, : H + Hk], z.imag[:, : H + Hk]
        caches = []
        for name, rows in (("k_cache", turned[:, H:H + Hk]), ("v_cache", x[:, H + Hk:])):
            flat = s[name].double().transpose(1, 2).reshape(-1, Hk, D)
            flat.index_copy_(0, s["slot"].long(), rows)
            caches.append(flat.reshape(-1, P, Hk, D).transpose(1, 2))
        return {"q": turned[:, :H], "k_cache": caches[0], "v_cache": caches[1]}
    if case["op"] == "attn":
        H, Hk, D, P = (case[k] for k in ("heads", "kv_heads", "dim", "page"))
        G = H // Hk
        out = torch.zeros(s["starts"][-1], H, D, dtype=torch.float64, device="cuda")
        for r, (n, count) in enumerate(zip(_lengths(case), _counts(case))):
            token = torch.arange(n, device="cuda")
            slot = s["table"][r].long()[token // P] * P + token % P
            rows = slice(s["starts"][r], s["starts"][r + 1])
            for h in range(Hk):
                k, v = (s[c][:, h].reshape(-1, D)[slot].double() for c in ("k_cache", "v_cache"))
                z = torch.einsum("tgd,jd->tgj", s["q"][rows, h * G:(h + 1) * G].double(), k) * s["scale"]
                for t in range(count):
                    mine = n - count + t
                    hidden = token > mine
                    if case["window"]:
                        hidden = hidden | ((token <= mine - case["window"]) & (token >= case["sinks"]))
                    z[t, :, hidden] = -math.inf
                out[rows, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", torch.softmax(z, -1), v)
        return out
    accepted, tokens = [], []

    def weights(logits, row, t):
        z = torch.nan_to_num(logits[row].double(), nan=-math.inf, posinf=math.inf, neginf=-math.inf)
        best = z.max()
        if best == -math.inf:
            return torch.zeros_like(z)
        w = (z == best).double()
        if t >= GREEDY_BELOW:
            lower = z < best
            w[lower] = torch.exp((z[lower] - best) / t)
        return w

    for r in range(case["requests"]):
        first, last = s["starts"][r], s["starts"][r + 1] - 1
        t, row, rest = s["temperature"][r].item(), first, None
        while row < last:
            x, u = s["token"][row + 1].item(), s["u"][row].item()
            p = weights(s["logits"], row, t)
            if s["draft_logits"] is None:
                q = torch.zeros_like(p)
                q[x] = 1.0
            else:
                q = weights(s["draft_logits"], row, t)
            P, Q = p.sum(), q.sum()
            if not (u * q[x] * P < p[x] * Q).item():
                rest = torch.relu(p / P - q / Q)
                if s["draft_logits"] is None:
                    rest[x] = 0.0
                if not rest.any():
                    rest = p
                break
            row += 1
        rest = weights(s["logits"], row, t) if rest is None else rest
        rest = rest.cpu().numpy()
        mass = np.cumsum(rest)
        accepted.append(row - first)
        tokens.append(min(int(np.searchsorted(mass, s["u_sample"][r].item() * mass[-1], side="right")), int(np.nonzero(rest)[0][-1])) if mass[-1] > 0 else -1)
    return {"accepted": np.asarray(accepted, np.int32), "next_token": np.asarray(tokens, np.int32)}
