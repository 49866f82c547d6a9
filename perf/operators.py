"""Timed cases of the FP8 linear-layer operators: what is measured, on which inputs,
and the operators' plain forms.

    fp8_quant_act   BF16 activation -> E4M3 codes, one FP32 scale per 128 elements of a row
    fp8_gemm        y = sum_b sx[b,m] sw[n/128,b] (xq[m,:] . wq[n,:])_b over blocks b of 128 along K
    block_norm      h' = a h + gate * norm(y; w_post), x = norm(h'; w_pre), x in BF16 or as FP8 blocks
    fp8_moe         router, top-k, gated FP8 experts and the weighted sum, for a few tokens

`own = False` computes each in elementary torch operations in 32 bits (the router's
scores in 64, where two experts can be close), `own = True` calls the package.
"""

from __future__ import annotations

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -100          # smallest block maximum that the scale follows
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token through a square projection: the call whose latency a decode step waits for
        {"name": "gemm_token", "op": "gemm", "M": 1, "N": 5120, "K": 5120, "out": "bf16"},
        # a decode batch through the MLP's up projection
        {"name": "gemm_batch", "op": "gemm", "M": 16, "N": 13824, "K": 5120, "out": "bf16"},
        # a short ragged prompt through an odd head: no size is a multiple of a tile, K ends inside a block
        {"name": "gemm_ragged", "op": "gemm", "M": 333, "N": 1000, "K": 2064, "out": "f32"},
        # a long prompt through the MLP's up projection: bound by the tensor cores
        {"name": "gemm_prompt", "op": "gemm", "M": 4096, "N": 13824, "K": 5120, "out": "bf16"},
        # activation of a decode batch before the MLP's down projection
        {"name": "quant_batch", "op": "quant", "M": 32, "K": 13824},
        # activation of a long prompt
        {"name": "quant_prompt", "op": "quant", "M": 8192, "K": 5120},
        # one token between two blocks, residual stream held in 32 bits
        {"name": "norm_token", "op": "norm", "M": 1, "D": 5120, "h": "f32", "post": True, "gate": 1, "quant": False},
        # a prompt of several sequences with a gate for each of them, odd width
        {"name": "norm_gated", "op": "norm", "M": 777, "D": 1160, "h": "bf16", "post": True, "gate": 7, "quant": False},
        # a long prompt between two blocks, the next block's FP8 activation written at once
        {"name": "norm_prompt", "op": "norm", "M": 8192, "D": 5120, "h": "bf16", "post": True, "gate": 0, "quant": True},
        # one token through a small mixture of experts
        {"name": "moe_token", "op": "moe", "T": 1, "D": 2048, "F": 1024, "E": 64, "k": 8, "shared": 0, "score": "softmax"},
        # a decode batch in which most experts get a token or two
        {"name": "moe_batch", "op": "moe", "T": 16, "D": 4096, "F": 2048, "E": 32, "k": 4, "shared": 1, "score": "sigmoid"},
        # the largest batch of the few-token form: every expert is read
        {"name": "moe_full", "op": "moe", "T": 64, "D": 5120, "F": 2048, "E": 64, "k": 8, "shared": 1, "score": "softmax"},
    ]


def _log(rng, lo, hi, step=1):
    """Spread over the logarithm of [lo, hi], a multiple of `step`."""
    v = lo * (hi / lo) ** rng.random()
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "quant", "norm", "moe"])
    if op == "gemm":
        while True:
            c = {"op": "gemm", "M": _log(rng, 1, 4096), "N": _log(rng, 40, 13824), "K": _log(rng, 64, 13824, 16),
                 "out": rng.choice(["bf16", "bf16", "f32"])}
            if c["M"] * c["N"] * c["K"] <= 4096 * 13824 * 5120:
                return c
    if op == "quant":
        while True:
            c = {"op": "quant", "M": _log(rng, 1, 8192), "K": _log(rng, 64, 13824, 16)}
            if c["M"] * c["K"] <= 8192 * 5120:
                return c
    if op == "norm":
        M, quant = _log(rng, 1, 8192), rng.random() < 0.5
        D = _log(rng, 256, 5120, 16)
        gate = rng.choice([0, 1, 2])
        return {"op": "norm", "M": M, "D": D, "h": rng.choice(["bf16", "f32"]), "post": rng.random() < 0.7,
                "gate": gate if gate < 2 or M % 2 == 0 else 1, "quant": quant}
    while True:
        E = rng.choice([8, 16, 32, 60, 64])
        c = {"op": "moe", "T": _log(rng, 1, 64), "D": _log(rng, 512, 5120, 16), "F": _log(rng, 256, 2048, 16), "E": E,
             "k": rng.choice([1, 2, 4, 6, 8]), "shared": rng.choice([0, 0, 1]), "score": rng.choice(["softmax", "sigmoid"])}
        if (E + c["shared"]) * c["D"] * c["F"] <= 65 * 5120 * 2048:
            return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activation(g, M, K):
    """N(0, 1) with one channel in a hundred twenty times as large, in BF16."""
    x = torch.randn((M, K), generator=g, device="cuda")
    big = torch.randperm(K, generator=g, device="cuda")[: max(1, K // 100)]
    x[:, big] *= 20.0
    return x.to(torch.bfloat16)


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _quant_rows(x):
    """FP32 [M, K] -> (E4M3 codes [M, K], scales FP32 [ceil(K/128), M])."""
    M, K = x.shape
    kb = _blocks(K)
    v = torch.nn.functional.pad(x, (0, kb * BLOCK - K)).view(M, kb, BLOCK)
    amax = v.abs().amax(-1).clamp_min(TINY)
    inv = E4M3_MAX / amax
    codes = (v * inv.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).view(M, kb * BLOCK)[:, :K].to(torch.float8_e4m3fn)
    return codes.contiguous(), (amax / E4M3_MAX).t().contiguous()


def _quant_tiles(w):
    """FP32 [N, K] -> (E4M3 codes [N, K], scales FP32 [ceil(N/128), ceil(K/128)])."""
    N, K = w.shape
    nb, kb = _blocks(N), _blocks(K)
    v = torch.nn.functional.pad(w, (0, kb * BLOCK - K, 0, nb * BLOCK - N)).view(nb, BLOCK, kb, BLOCK)
    amax = v.abs().amax((1, 3)).clamp_min(TINY)
    codes = (v * (E4M3_MAX / amax)[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(nb * BLOCK, kb * BLOCK)[:N, :K]
    return codes.to(torch.float8_e4m3fn).contiguous(), amax / E4M3_MAX


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    if op == "gemm":
        st["x"], st["sx"] = _quant_rows(_activation(g, case["M"], case["K"]).float())
        st["w"], st["sw"] = _quant_tiles(torch.randn((case["N"], case["K"]), generator=g, device="cuda") * 0.02)
    elif op == "quant":
        st["x"] = _activation(g, case["M"], case["K"])
    elif op == "norm":
        M, D = case["M"], case["D"]
        st["y"] = _activation(g, M, D)
        st["h"] = (_activation(g, M, D).float() * 3.0).to(DT[case["h"]])
        st["w_post"] = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16) if case["post"] else None
        st["w_pre"] = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
        st["gate"] = torch.randn((case["gate"], D), generator=g, device="cuda").to(torch.bfloat16) if case["gate"] else None
    else:
        T, D, F, n = case["T"], case["D"], case["F"], case["E"] + case["shared"]
        st["x"] = _activation(g, T, D)
        st["router"] = (torch.randn((case["E"], D), generator=g, device="cuda") * 0.02).to(torch.bfloat16)
        st["bias"] = 0.05 * torch.randn(case["E"], generator=g, device="cuda") if case["score"] == "sigmoid" else None
        st["w13"] = torch.empty((n, 2 * F, D), dtype=torch.float8_e4m3fn, device="cuda")
        st["s13"] = torch.empty((n, _blocks(2 * F), _blocks(D)), device="cuda")
        st["w2"] = torch.empty((n, D, F), dtype=torch.float8_e4m3fn, device="cuda")
        st["s2"] = torch.empty((n, _blocks(D), _blocks(F)), device="cuda")
        for e in range(n):
            st["w13"][e], st["s13"][e] = _quant_tiles(torch.randn((2 * F, D), generator=g, device="cuda") * 0.02)
            st["w2"][e], st["s2"][e] = _quant_tiles(torch.randn((D, F), generator=g, device="cuda") * 0.02)
    return st


# ------------------------------------------------------------------ plain forms

EPS = 1e-6
RES_SCALE = 0.9
ROUTE_SCALE = 2.5


def _tiles_out(codes, scales):
    """FP8 weight tiles [..., N, K] with scales [..., N/128, K/128] -> FP32 [..., N, K]."""
    N, K = codes.shape[-2:]
    s = scales.repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)[..., :K]
    return codes.float() * s


def _gemm(st):
    M, K = st["x"].shape
    x = st["x"].float() * st["sx"].t().repeat_interleave(BLOCK, 1)[:, :K]
    return (x @ _tiles_out(st["w"], st["sw"]).t()).to(DT[st["case"]["out"]])


def _rms(v, w):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * w.float()


def _norm(st):
    y, h, gate = st["y"].float(), st["h"].float(), st["gate"]
    u = y if st["w_post"] is None else _rms(y, st["w_post"])
    if gate is not None:
        u = u * gate.float().repeat_interleave(y.shape[0] // gate.shape[0], 0)
    h2 = RES_SCALE * h + u
    x = _rms(h2, st["w_pre"])
    if st["case"]["quant"]:
        return (h2.to(st["h"].dtype), *_quant_rows(x))
    return h2.to(st["h"].dtype), x.to(torch.bfloat16)


def _moe(st):
    c = st["case"]
    T, E, k, F = c["T"], c["E"], c["k"], c["F"]
    logits = st["x"].double() @ st["router"].double().t()
    p = torch.softmax(logits, -1) if c["score"] == "softmax" else torch.sigmoid(logits)
    key = logits if st["bias"] is None else p + st["bias"].double()
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :k]      # ties: the lowest index
    w = p.gather(1, ids)
    w = (w / w.sum(-1, keepdim=True) * ROUTE_SCALE).float()
    share = torch.zeros((T, E + c["shared"]), device="cuda").scatter_(1, ids, w)
    share[:, E:] = 1.0
    x = st["x"].float()
    gu = x @ _tiles_out(st["w13"], st["s13"]).transpose(1, 2)                   # [experts, T, 2F]
    a = gu[..., :F]
    a = a / (1.0 + torch.exp(-a)) * gu[..., F:]
    y = a @ _tiles_out(st["w2"], st["s2"]).transpose(1, 2)                      # [experts, T, D]
    y = (y * share.t().unsqueeze(-1)).sum(0)
    return y.to(torch.bfloat16), ids.to(torch.int32), w


def run(state):
    op = state["case"]["op"]
    if own:
        import nvfp4_binary_rank_b200 as nb
        if op == "gemm":
            return nb.fp8_gemm(state["x"], state["sx"], state["w"], state["sw"], out_dtype=DT[state["case"]["out"]])
        if op == "quant":
            return nb.fp8_quant_act(state["x"])
        if op == "norm":
            return nb.block_norm(state["y"], state["h"], post_weight=state["w_post"], gate=state["gate"],
                                 res_scale=RES_SCALE, pre_weight=state["w_pre"], eps=EPS, quant=state["case"]["quant"])
        return nb.fp8_moe(state["x"], state["router"], state["w13"], state["s13"], state["w2"], state["s2"],
                          state["case"]["k"], score=state["case"]["score"], bias=state["bias"], renorm=True,
                          route_scale=ROUTE_SCALE)
    if op == "gemm":
        return _gemm(state)
    if op == "quant":
        return _quant_rows(state["x"].float())
    if op == "norm":
        return _norm(state)
    return _moe(state)


# ------------------------------------------------------------------ work

def _expected_experts(E, picks):
    """Experts that get a token when each of `picks` choices falls on any of E alike."""
    return E * (1.0 - (1.0 - 1.0 / E) ** picks)


def work(case):
    op = case["op"]
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 4 * _blocks(K) * (M + _blocks(N)) + M * N * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * M * N * K}
    if op == "quant":
        M, K = case["M"], case["K"]
        return {"bytes": 3 * M * K + 4 * M * _blocks(K), "flops": 3 * M * K}
    if op == "norm":
        M, D = case["M"], case["D"]
        hb = 2 if case["h"] == "bf16" else 4
        out = M * D + 4 * M * _blocks(D) if case["quant"] else 2 * M * D
        return {"bytes": 2 * M * D + 2 * hb * M * D + out + 2 * D * (1 + int(case["post"]) + case["gate"]), "flops": 10 * M * D}
    T, D, F, E, k, s = (case[n] for n in ("T", "D", "F", "E", "k", "shared"))
    read = (k if T == 1 else _expected_experts(E, T * k)) + s
    return {"bytes": read * 3 * D * F + 2 * E * D + 4 * T * D + 8 * T * k, "flops": 6 * T * (k + s) * D * F + 2 * T * E * D}


# ------------------------------------------------------------------ 64 bits

def _e4m3(v):
    """FP64 values rounded to E4M3 (four significant bits, ties to even, at most 448)."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -20))).clamp_min(-6.0)
    e = torch.where(v.abs() < torch.exp2(e), e - 1, e).clamp_min(-6.0)
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_blocks(x):
    codes, scales = [], []
    for b in range(0, x.shape[1], BLOCK):
        v = x[:, b:b + BLOCK]
        top = torch.clamp(v.abs().max(1).values, min=TINY)
        codes.append(_e4m3(v * (E4M3_MAX / top)[:, None]))
        scales.append(top / E4M3_MAX)
    return torch.cat(codes, 1), torch.stack(scales)


def _exact_gemm(x, sx, w, sw):
    """Block by block, in FP64."""
    N, K = w.shape
    y = torch.zeros((x.shape[0], N), dtype=torch.float64, device=x.device)
    col = torch.arange(N, device=x.device) // BLOCK
    for b in range(_blocks(K)):
        at = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
        part = x[:, at].double() @ w[:, at].double().T
        y += part * sx[b].double()[:, None] * sw[:, b].double()[col][None, :]
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        return _exact_gemm(st["x"], st["sx"], st["w"], st["sw"])
    if op == "quant":
        return _exact_blocks(st["x"].double())
    if op == "norm":
        y, h = st["y"].double(), st["h"].double()
        M, D = y.shape
        if st["w_post"] is not None:
            y = y / torch.sqrt((y * y).sum(1, keepdim=True) / D + EPS) * st["w_post"].double()
        if st["gate"] is not None:
            G = st["gate"].shape[0]
            y = (y.view(G, M // G, D) * st["gate"].double()[:, None, :]).view(M, D)
        h = h * RES_SCALE + y
        x = h / torch.sqrt((h * h).sum(1, keepdim=True) / D + EPS) * st["w_pre"].double()
        return (h, *_exact_blocks(x)) if case["quant"] else (h, x)
    T, E, k, F = (case[n] for n in ("T", "E", "k", "F"))
    x = st["x"].double()
    logits = torch.stack([(x * r.double()).sum(1) for r in st["router"]], 1)
    p = torch.softmax(logits, 1) if case["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-logits))
    key = (p + st["bias"].double() if st["bias"] is not None else logits).clone()
    picked = []
    for _ in range(k):
        picked.append(key.argmax(1))
        key.scatter_(1, picked[-1][:, None], -float("inf"))
    ids = torch.stack(picked, 1)
    w = p.gather(1, ids)
    w = w / w.sum(1, keepdim=True) * ROUTE_SCALE
    y = torch.zeros_like(x)
    for e in range(E + case["shared"]):
        share = torch.where(ids == e, w, torch.zeros_like(w)).sum(1) if e < E else torch.ones(T, dtype=torch.float64, device="cuda")
        at = share.nonzero().flatten()
        if at.numel():
            ones = torch.ones((_blocks(x.shape[1]), at.numel()), device="cuda")
            gu = _exact_gemm(x[at], ones, st["w13"][e], st["s13"][e])
            a = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
            ones = torch.ones((_blocks(F), at.numel()), device="cuda")
            y[at] += _exact_gemm(a, ones, st["w2"][e], st["s2"][e]) * share[at][:, None]
    return y, None, w
