"""Workloads of the operators around the packed products: RMSNorm with int8 codes, low-rank adapters, sampling.

Each case is one call as a serving loop makes it.  ``run`` computes it in
elementary torch operations, or, with ``own`` true, by the library's entry
points.  ``exact`` gives the outputs from the definitions in 64 bits.

  norm    h = x + residual; v = h * rsqrt(mean(h^2) + eps) * weight; int8 codes of v with one scale per token.
  lora    y = base + scale[a] * B[a] (A[a] x) with a = adapter[token]; a negative index means no adapter.
  sample  temperature, top-k, top-p and min-p over rows of logits; the token is found from a given uniform number
          by the cumulative probabilities in the order of falling logits (ties: lowest index first).
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GREEDY_BELOW = 1e-5  # temperatures under this take the largest logit


def listed():
    return [
        # one token of a decode step: residual added, 2560 wide (the MLP's input)
        {"name": "norm_token", "op": "norm", "tokens": 1, "width": 2560, "dtype": "bf16", "residual": True, "normed": False},
        # a decode batch before the down projection: 6912 wide, fp32 activations, no residual
        {"name": "norm_batch_f32", "op": "norm", "tokens": 37, "width": 6912, "dtype": "f32", "residual": False, "normed": True},
        # the 512-token prefill; the normed values go to the adapters as well
        {"name": "norm_prefill", "op": "norm", "tokens": 512, "width": 2560, "dtype": "bf16", "residual": True, "normed": True},
        # several long prompts at once, 5120 wide
        {"name": "norm_long", "op": "norm", "tokens": 8192, "width": 5120, "dtype": "bf16", "residual": True, "normed": False},
        # one request with an adapter, one token, beside the gate projection
        {"name": "lora_token", "op": "lora", "tokens": 1, "requests": 1, "adapters": 4, "rank": 16, "width_in": 2560,
         "width_out": 6912, "xt": "bf16", "yt": "bf16"},
        # a decode step of 64 requests over 40 adapters, an eighth of them without one
        {"name": "lora_batch", "op": "lora", "tokens": 64, "requests": 64, "adapters": 40, "rank": 32, "width_in": 5120,
         "width_out": 13824, "xt": "bf16", "yt": "bf16"},
        # nine requests of uneven lengths beside the i2_s prefill, whose result is fp32
        {"name": "lora_ragged_f32", "op": "lora", "tokens": 517, "requests": 9, "adapters": 5, "rank": 24, "width_in": 2560,
         "width_out": 2560, "xt": "bf16", "yt": "f32"},
        # twelve long prompts beside the gate projection, high rank
        {"name": "lora_prompts", "op": "lora", "tokens": 8192, "requests": 12, "adapters": 6, "rank": 64, "width_in": 2560,
         "width_out": 6912, "xt": "bf16", "yt": "bf16"},
        # the LM head's logits of one token
        {"name": "sample_token", "op": "sample", "rows": 1, "vocab": 248320, "dtype": "bf16", "filters": "mixed"},
        # a decode batch whose requests ask for different filters, some with a grammar's mask
        {"name": "sample_batch", "op": "sample", "rows": 64, "vocab": 248320, "dtype": "bf16", "filters": "mixed"},
        # fp32 logits and an odd vocabulary
        {"name": "sample_f32", "op": "sample", "rows": 32, "vocab": 100003, "dtype": "f32", "filters": "mixed"},
        # many samples by temperature alone (rollouts): the whole vocabulary stays in
        {"name": "sample_rollout", "op": "sample", "rows": 256, "vocab": 248320, "dtype": "bf16", "filters": "none"},
    ]


def _spread(rng, lo, hi):
    """An integer in [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "lora", "sample"])
    if op == "norm":
        width = _spread(rng, 128, 13824)
        if rng.random() < 0.7:
            width = (width + 7) // 8 * 8
        case = {"op": op, "tokens": _spread(rng, 1, 8192), "width": width, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "residual": rng.random() < 0.7, "normed": rng.random() < 0.5}
        size, most = "tokens", listed()[3]
    elif op == "lora":
        tokens = _spread(rng, 1, 8192)
        requests = tokens if tokens <= 256 and rng.random() < 0.5 else min(tokens, _spread(rng, 1, 32))
        case = {"op": op, "tokens": tokens, "requests": requests, "adapters": _spread(rng, 1, 48),
                "rank": rng.choice([8, 16, 24, 32, 64, 128]), "width_in": 8 * _spread(rng, 32, 1728),
                "width_out": _spread(rng, 128, 13824), "xt": rng.choice(["bf16", "bf16", "bf16", "f32"]),
                "yt": rng.choice(["bf16", "f32"])}
        size, most = "tokens", listed()[7]
    else:
        case = {"op": op, "rows": _spread(rng, 1, 256), "vocab": _spread(rng, 1000, 262144),
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "filters": rng.choice(["mixed", "none"])}
        size, most = "rows", listed()[11]
    limit = work(most)
    while case[size] > 1 and any(work(case)[k] > limit[k] for k in ("bytes", "flops")):
        case[size] = case[size] * 3 // 4
        if op == "lora":
            case["requests"] = min(case["requests"], case["tokens"])
    return case


def _adapter_of_request(case):
    """Request i uses adapter i mod adapters; of eight requests the last has none."""
    return [-1 if i % 8 == 7 else i % case["adapters"] for i in range(case["requests"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    rand = lambda *shape: torch.rand(*shape, generator=g, device="cuda")  # noqa: E731
    state = {"case": case}
    if case["op"] == "norm":
        M, K, t = case["tokens"], case["width"], DTYPES[case["dtype"]]
        state["x"] = randn(M, K).to(t)
        if case["residual"]:  # a residual stream: a few channels are far larger than the rest
            channel = torch.where(rand(K) < 0.005, 20.0, 1.0)
            state["residual"] = (randn(M, K) * channel * (0.5 + 3 * rand(M, 1))).to(t)
        state["weight"] = (1 + 0.2 * randn(K)).to(t)
        state["values"] = torch.empty(M, K, device="cuda")
        state["q"] = torch.empty(M, K, dtype=torch.int8, device="cuda")
        state["s"] = torch.empty(M, device="cuda")
        state["h"] = torch.empty(M, K, dtype=t, device="cuda") if case["residual"] else None
        state["y"] = torch.empty(M, K, dtype=t, device="cuda") if case["normed"] else False
    elif case["op"] == "lora":
        M, K, N, R, L = case["tokens"], case["width_in"], case["width_out"], case["rank"], case["adapters"]
        index = _adapter_of_request(case)
        cuts = np.random.default_rng(seed).choice(np.arange(1, M), case["requests"] - 1, replace=False) if M > 1 else []
        bounds = np.concatenate([[0], np.sort(np.asarray(cuts, dtype=np.int64)), [M]])
        state["adapter"] = torch.from_numpy(np.repeat(np.asarray(index, np.int32), np.diff(bounds))).cuda()
        state["x"] = randn(M, K).to(DTYPES[case["xt"]])
        state["a"] = (randn(L, R, K) / math.sqrt(K)).to(torch.bfloat16)
        state["b"] = (randn(L, N, R) * 0.1).to(torch.bfloat16)
        state["scale"] = 2 ** (4 * rand(L) - 2)
        state["base"] = randn(M, N).to(DTYPES[case["yt"]])
        state["y"] = torch.empty_like(state["base"])
    else:
        M, V = case["rows"], case["vocab"]
        # a model's logits: a broad bulk, and a short head of likely tokens that differs by row
        logits = 2.0 * randn(M, V) - 2.0
        head = torch.arange(40, device="cuda") * (V // 40) + torch.randint(0, V // 40, (M, 40), generator=g, device="cuda")
        logits.scatter_(1, head, 9.0 + 3.0 * randn(M, 40))
        state["u"] = rand(M)
        state["temperature"] = 0.5 + rand(M)
        state["top_k"] = state["top_p"] = state["min_p"] = None
        if case["filters"] == "mixed":
            pick = torch.randint(0, 8, (M,), generator=g, device="cuda")
            state["temperature"] = torch.where(pick == 7, 0.0, state["temperature"])
            k = torch.randint(1, 200, (M,), generator=g, device="cuda", dtype=torch.int32)
            state["top_k"] = torch.where((pick == 0) | (pick == 1) | (pick == 4), k, 0).to(torch.int32)
            state["top_p"] = torch.where((pick == 1) | (pick == 2) | (pick == 5), 0.7 + 0.29 * rand(M), 1.0)
            state["min_p"] = torch.where((pick == 3) | (pick == 4), 0.01 + 0.1 * rand(M), 0.0)
            masked = (rand(M, V) < 0.9) & ((pick == 5) | (pick == 6))[:, None]
            logits.masked_fill_(masked, -math.inf)
        state["logits"] = logits.to(DTYPES[case["dtype"]])
        state["token"] = torch.empty(M, dtype=torch.int32, device="cuda")
        state["prob"] = torch.empty(M, device="cuda")
    return state


# ---- plain forms -------------------------------------------------------------

def _norm_plain(s):
    t = s["x"].dtype
    out = {}
    h = s["x"].float()
    if "residual" in s:
        out["h"] = (h + s["residual"].float()).to(t)
        h = out["h"].float()
    mean = (h.double() * h.double()).mean(1, keepdim=True)  # 64 bits: the codes lie next to borders
    r = (1 / torch.sqrt(mean + float(np.float32(EPS)))).float()
    v = h * r * s["weight"].float()
    if s["case"]["normed"]:
        out["y"] = v.to(t)
    amax = v.abs().amax(1, keepdim=True)
    most = torch.full_like(amax, 127.0)  # a division by a number would be a product with its reciprocal
    q = torch.clamp(torch.round(v * torch.where(amax > 0, most / amax, 0.0)), -127, 127).to(torch.int8)
    out["scale"] = (amax / most)[:, 0]
    out["values"] = torch.mul(q, out["scale"][:, None], out=s["values"])
    return out


def _lora_plain(s):
    L, R, K = s["a"].shape
    N = s["b"].shape[1]
    M = s["x"].shape[0]
    mine = s["adapter"][:, None] == torch.arange(L, device="cuda", dtype=torch.int32)  # [M, L]
    low = (s["x"].float() @ s["a"].float().reshape(L * R, K).T).reshape(M, L, R)
    low = torch.where(mine[:, :, None], low * s["scale"][None, :, None], 0.0)
    wide = s["b"].float().transpose(1, 2).reshape(L * R, N)
    return (s["base"].float() + low.reshape(M, L * R) @ wide).to(s["base"].dtype)


def _sample_plain(s):
    logits = s["logits"].float()
    M, V = logits.shape
    logits = torch.where(torch.isnan(logits), -math.inf, logits) + 0.0
    z, order = torch.sort(logits, dim=1, descending=True, stable=True)
    top = z[:, :1]
    t = s["temperature"][:, None]
    w = torch.exp((z.double() - top.double()) / t.double())  # 64 bits: cumulative masses lie next to borders
    w = torch.where(z == top, 1.0, torch.where(t >= GREEDY_BELOW, w, 0.0))
    w = torch.where(z > -math.inf, w, 0.0)
    place = torch.arange(V, device="cuda")
    keep = w > -1
    if s["top_k"] is not None:
        keep = (place < s["top_k"][:, None]) | (s["top_k"][:, None] <= 0)
    if s["top_p"] is not None:
        mass = torch.cumsum(torch.where(keep, w, 0.0), 1)
        before = torch.nn.functional.pad(mass[:, :-1], (1, 0))
        keep = keep & ((before < s["top_p"][:, None].double() * mass[:, -1:]) | (s["top_p"][:, None] >= 1) | (place == 0))
    if s["min_p"] is not None:
        keep = keep & ((w >= s["min_p"][:, None].double()) | (place == 0))
    w = torch.where(keep, w, 0.0)
    mass = torch.cumsum(w, 1)
    at = (mass <= s["u"][:, None].double() * mass[:, -1:]).sum(1, keepdim=True)
    at = torch.minimum(at, keep.sum(1, keepdim=True) - 1)
    empty = top[:, 0] == -math.inf
    token = torch.where(empty, -1, torch.gather(order, 1, at)[:, 0]).to(torch.int32)
    prob = torch.where(empty, 0.0, torch.gather(w, 1, at)[:, 0] / mass[:, -1]).float()
    return {"token": token, "prob": prob}


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"norm": _norm_plain, "lora": _lora_plain, "sample": _sample_plain}[op](state)
    from gemm_bl_gemv_gb300 import binding as B
    if op == "norm":
        q, s, h, y = B.bl_rmsnorm_quant_int8(state["x"], state["weight"], EPS, residual=state.get("residual"), h=state["h"],
                                             y=state["y"], q=state["q"], s=state["s"])
        out = {"scale": s, "values": torch.mul(q, s[:, None], out=state["values"])}
        if h is not None:
            out["h"] = h
        if y is not None:
            out["y"] = y
        return out
    if op == "lora":
        return B.bl_lora_add(state["x"], state["adapter"], state["a"], state["b"], state["scale"], state["base"], y=state["y"])
    token, prob = B.bl_sample(state["logits"], state["u"], temperature=state["temperature"], top_k=state["top_k"],
                              top_p=state["top_p"], min_p=state["min_p"], token=state["token"], prob=state["prob"])
    return {"token": token, "prob": prob}


def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "norm":
        M, K, e = case["tokens"], case["width"], size[case["dtype"]]
        tensors = 1 + 2 * case["residual"] + case["normed"]  # x; residual and h; y
        return {"bytes": M * K * (tensors * e + 1) + K * e + 4 * M, "flops": 9 * M * K}
    if case["op"] == "lora":
        M, K, N, R = case["tokens"], case["width_in"], case["width_out"], case["rank"]
        index = _adapter_of_request(case)
        used = len({a for a in index if a >= 0})
        share = sum(a >= 0 for a in index) / len(index)
        return {"bytes": M * K * size[case["xt"]] + 2 * M * N * size[case["yt"]] + used * R * (K + N) * 2 + 4 * M + 4 * used,
                "flops": 2 * share * M * R * (K + N) + M * N}
    M, V = case["rows"], case["vocab"]
    return {"bytes": M * V * size[case["dtype"]] + 32 * M, "flops": 4 * M * V}


# ---- the definitions in 64 bits -----------------------------------------------

def _f32(v):
    """A binary32 rounding step of the definition, kept in 64 bits."""
    return v.to(torch.float32).to(torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        out = {}
        t = s["x"].dtype
        h = s["x"].double()
        if case["residual"]:
            h = h + s["residual"].double()
            out["h"] = h
            h = _f32(h).to(t).double()  # the residual stream is stored in its own type
        # the definition's roundings: the row's factor once, each product once, as the codes are defined by them
        r = _f32(torch.rsqrt(torch.einsum("mk,mk->m", h, h) / h.shape[1] + float(np.float32(EPS))))
        v = _f32(_f32(torch.einsum("mk,m->mk", h, r)) * s["weight"].double())
        amax = torch.max(v.max(1).values, -v.min(1).values)
        out["scale"] = amax / 127.0
        codes = torch.zeros_like(v)
        live = amax > 0
        codes[live] = torch.round(_f32(v[live] * _f32(127.0 / amax[live])[:, None]))
        out["values"] = codes * out["scale"][:, None]
        if case["normed"]:
            out["y"] = v
        return out
    if case["op"] == "lora":
        y = s["base"].double()
        for a in sorted(set(s["adapter"].tolist()) - {-1}):
            rows = torch.nonzero(s["adapter"] == a)[:, 0]
            low = s["x"][rows].double() @ s["a"][a].double().T
            y[rows] += float(s["scale"][a]) * (low @ s["b"][a].double().T)
        return y
    tokens, probs = [], []
    at = lambda name, m, none: none if s[name] is None else s[name][m].item()  # noqa: E731
    for m in range(case["rows"]):
        row = torch.nan_to_num(s["logits"][m].double(), nan=-math.inf, posinf=math.inf, neginf=-math.inf)
        value, count = torch.unique(row, return_counts=True)  # rising; -0 and 0 are one value
        value, count = value.flip(0).cpu().numpy(), count.flip(0).cpu().numpy().astype(np.float64)
        live = value > -math.inf
        value, count = value[live], count[live]
        if not len(value):
            tokens.append(-1)
            probs.append(0.0)
            continue
        t, k, p, low, u = (at(n, m, d) for n, d in (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0), ("min_p", 0.0), ("u", None)))
        w = np.zeros(len(value))
        w[0] = 1.0
        if t >= GREEDY_BELOW:
            w[1:] = np.exp((value[1:] - value[0]) / t)
        if k > 0:  # how many of each value stay
            count = np.clip(k - (np.cumsum(count) - count), 0, count)
        if p < 1:
            mass = np.cumsum(w * count)
            room = p * mass[-1] - (mass - w * count)  # mass that may still lie before a token of this value
            first = np.where(w > 0, np.ceil(room / np.where(w > 0, w, 1.0)), 0)
            count = np.minimum(count, np.maximum(first, 0))
            count[0] = max(count[0], 1)
        if low > 0:
            count[1:][w[1:] < low] = 0
            if w[0] < low:
                count[0] = 1
        mass = np.cumsum(w * count)
        i = min(int(np.searchsorted(mass, u * mass[-1], side="right")), int(np.nonzero(count)[0][-1]))
        j = min(int((u * mass[-1] - (mass[i] - w[i] * count[i])) / w[i]), int(count[i]) - 1) if w[i] > 0 else 0
        tokens.append(int(torch.nonzero(row == value[i])[max(j, 0), 0]))
        probs.append(w[i] / mass[-1])
    return {"token": np.asarray(tokens, np.int32), "prob": np.asarray(probs)}
