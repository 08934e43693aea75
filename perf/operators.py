"""Cases for the router, the combine's gradient and the dense FP8 product of the MoE layer.

The operators (names as in include/moe.h):

  router        moe_router_topk: router logits -> topk_ids and topk_weights of every token
  router_bwd    moe_router_topk_bwd: d topk_weights -> d logits
  combine_bwd   moe_unpermute_combine_bwd: d Z -> d Y (packed rows) and d topk_weights
  gemm          moe_gemm_fp8: dense FP8 product, one fp32 scale per 1x128 / 128x128 block
  quant_t       moe_quant_act_t: the transposing quantiser behind the weight gradient's product

``own`` selects what run() computes: the plain form (elementary torch operations) or the calls of
int4_weights_amd.  Shapes are those of the repository's DeepSeek-V3-shaped and Qwen3-shaped layers, or generic.
"""

from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # One decode step of the 16-token, 128-expert layer: softmax scores, renormalised top-8.  Latency counts.
        {"name": "router_decode", "op": "router", "T": 16, "E": 128, "k": 8, "dtype": "bf16", "score": "softmax",
         "bias": False, "groups": 1, "topk_group": 1, "group_top": 1, "norm": True, "scale": 1.0, "masked": 0},
        # A prefill batch of the 256-expert layer: sigmoid scores, balance bias, the best 4 of 8 groups.
        {"name": "router_prefill", "op": "router", "T": 4096, "E": 256, "k": 8, "dtype": "fp32", "score": "sigmoid",
         "bias": True, "groups": 8, "topk_group": 4, "group_top": 2, "norm": True, "scale": 2.5, "masked": 0},
        # Training step of the same router: the gradient reaches the selected experts only.
        {"name": "router_bwd_sigmoid", "op": "router_bwd", "T": 4096, "E": 256, "k": 8, "dtype": "fp32",
         "score": "sigmoid", "norm": True, "scale": 2.5, "masked": 0},
        # Softmax weights that are not renormalised: every expert's logit gets a gradient; an odd batch in bf16.
        {"name": "router_bwd_softmax", "op": "router_bwd", "T": 8191, "E": 128, "k": 8, "dtype": "bf16",
         "score": "softmax", "norm": False, "scale": 1.0, "masked": 3},
        # Gradient of the combine for a short, ragged batch (some routes dropped by a full expert).
        {"name": "combine_bwd_small", "op": "combine_bwd", "T": 61, "k": 8, "N": 7168, "dropped": 9},
        # Gradient of the combine for the Qwen3-shaped training batch: the longest stream of packed rows.
        {"name": "combine_bwd_large", "op": "combine_bwd", "T": 8192, "k": 8, "N": 4096, "dropped": 0},
        # The dense (every-token) expert's up-projection for a single decoded token.
        {"name": "gemm_decode", "op": "gemm", "M": 1, "N": 4096, "K": 7168, "gran_n": 128, "out": "bf16",
         "add": False, "pad": 0},
        # Its down-projection for a small mixed batch; an odd number of rows, rows inside a wider output.
        {"name": "gemm_batch", "op": "gemm", "M": 131, "N": 7168, "K": 2048, "gran_n": 128, "out": "bf16",
         "add": False, "pad": 16},
        # Its up-projection for a prefill batch.
        {"name": "gemm_prefill", "op": "gemm", "M": 4096, "N": 4096, "K": 7168, "gran_n": 128, "out": "bf16",
         "add": False, "pad": 0},
        # Its weight gradient over 4096 tokens (both operands scaled 1x128 along the tokens), added to the
        # fp32 gradient of the step so far.
        {"name": "gemm_wgrad", "op": "gemm", "M": 4096, "N": 7168, "K": 4096, "gran_n": 1, "out": "fp32",
         "add": True, "pad": 0},
        # Quantising the operands of that weight gradient: a short odd batch, and the whole batch.
        {"name": "quant_t_small", "op": "quant_t", "M": 333, "K": 1536},
        {"name": "quant_t_large", "op": "quant_t", "M": 4096, "K": 7168},
    ]


def _logrand(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router", "router", "router_bwd", "combine_bwd", "gemm", "gemm", "gemm", "quant_t"])
    if op in ("router", "router_bwd"):
        T = _logrand(rng, 1, 8192)
        score = rng.choice(["softmax", "sigmoid"])
        c = {"op": op, "T": T, "dtype": rng.choice(["fp32", "bf16"]), "score": score,
             "norm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]), "masked": rng.choice([0, 0, 1, 5])}
        if op == "router":
            groups = rng.choice([1, 1, 4, 8])
            c["E"] = groups * rng.randint(max(2, 16 // groups), 256 // groups)
            c["topk_group"] = 1 if groups == 1 else rng.randint(2, groups)
            c["groups"] = groups
            c["group_top"] = rng.choice([1, 2])
            c["bias"] = rng.random() < 0.6
            c["k"] = rng.randint(1, min(12, c["E"] // groups * c["topk_group"]))
        else:
            c["E"] = rng.randint(16, 256)
            c["k"] = rng.randint(1, 12)
        return c
    if op == "combine_bwd":
        N = 8 * rng.randint(16, 896)
        T = _logrand(rng, 1, max(1, 8192 * 4096 // N))
        return {"op": op, "T": min(T, 8192), "k": rng.randint(1, 8), "N": N, "dropped": rng.choice([0, 1, 7])}
    if op == "gemm":
        K = 128 * rng.randint(1, 56)
        N = _logrand(rng, 64, 7168)
        M = _logrand(rng, 1, max(1, min(8192, 4096 * 4096 * 7168 // (N * K))))
        out = rng.choice(["bf16", "bf16", "fp32"])
        return {"op": op, "M": M, "N": N, "K": K, "gran_n": rng.choice([128, 128, 1]), "out": out,
                "add": out == "fp32" and rng.random() < 0.5, "pad": rng.choice([0, 0, 16])}
    return {"op": op, "M": _logrand(rng, 1, 4096), "K": 8 * _logrand(rng, 4, 896)}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _logits(case, g):
    x = torch.randn(case["T"], case["E"], generator=g, device=DEV) * 1.5
    x = x.to(torch.float32 if case["dtype"] == "fp32" else torch.bfloat16)
    if case["masked"]:  # experts this token may not use
        off = torch.rand(case["T"], case["E"], generator=g, device=DEV).argsort(1)[:, :case["masked"]]
        x.scatter_(1, off, float("-inf"))
    return x


def _codes(rows, K, gran, g):
    """Codes and scales of a normal matrix: scale = amax / 448 of each gran x 128 block, no power of two."""
    x = torch.randn(rows, K, generator=g, device=DEV)
    nb = -(-rows // gran)
    p = torch.zeros(nb * gran, K, device=DEV)
    p[:rows] = x
    s = (p.view(nb, gran, K // 128, 128).abs().amax((1, 3)) / 448.0).clamp_min(1e-12)
    s = s * torch.empty_like(s).uniform_(0.01, 0.04, generator=g)  # magnitudes differ from block to block
    unit = p.view(nb, gran, K // 128, 128) / (p.view(nb, gran, K // 128, 128).abs().amax((1, 3), keepdim=True) / 448.0)
    q = unit.view(nb * gran, K)[:rows].to(torch.float8_e4m3fn)
    return q.contiguous().view(torch.uint8), s.contiguous()


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": dict(case)}
    op = case["op"]
    if op == "router":
        s["logits"] = _logits(case, g)
        s["bias"] = torch.randn(case["E"], generator=g, device=DEV) * 0.05 if case["bias"] else None
        s["ids"] = torch.empty(case["T"], case["k"], dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty(case["T"], case["k"], dtype=torch.float32, device=DEV)
    elif op == "router_bwd":
        s["logits"] = _logits(case, g)
        top = torch.topk(s["logits"].float(), case["k"], dim=1)
        s["ids"] = torch.where(top.values > float("-inf"), top.indices, torch.full_like(top.indices, -1)).to(torch.int32)
        s["dweights"] = torch.randn(case["T"], case["k"], generator=g, device=DEV)
        s["dlogits"] = torch.empty_like(s["logits"])
    elif op == "combine_bwd":
        T, k, N = case["T"], case["k"], case["N"]
        rows = T * k + 37  # padding rows that no route names
        s["dZ"] = torch.randn(T, N, generator=g, device=DEV).to(torch.bfloat16)
        s["Y"] = torch.randn(rows, N, generator=g, device=DEV, dtype=torch.bfloat16)
        oi = torch.randperm(rows, generator=g, device=DEV)[:T * k].to(torch.int32)
        drop = torch.randperm(T * k, generator=g, device=DEV)[:min(case["dropped"], T * k - 1)]
        oi[drop] = -1
        s["output_index"] = oi.view(T, k)
        s["topk_weights"] = torch.softmax(torch.randn(T, k, generator=g, device=DEV), 1)
        s["dY_and_spare"] = torch.zeros(rows + 1, N, dtype=torch.bfloat16, device=DEV)
        s["dY"] = s["dY_and_spare"][:rows]
        s["dweights"] = torch.empty(T, k, dtype=torch.float32, device=DEV)
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s["A"], s["SFA"] = _codes(M, K, 1, g)
        s["W"], s["SFW"] = _codes(N, K, case["gran_n"], g)
        dt = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        s["D"] = torch.zeros(M, N + case["pad"], dtype=dt, device=DEV)[:, :N]
        s["C"] = torch.randn(M, N + case["pad"], generator=g, device=DEV)[:, :N] if case["add"] else None
    elif op == "quant_t":
        M, K = case["M"], case["K"]
        x = torch.randn(M, K, generator=g, device=DEV) * torch.exp2(torch.randint(-6, 7, (M, 1), generator=g, device=DEV))
        s["x"] = x.to(torch.bfloat16)
        mb = -(-M // 128)
        s["q"] = torch.empty(K, 128 * mb, dtype=torch.uint8, device=DEV)
        s["sf"] = torch.empty(K, mb, dtype=torch.float32, device=DEV)
    return s


# ------------------------------------------------------------------------------------------------- plain form --


def _scores(x, score):
    """Scores of the available experts (0 elsewhere); x has -inf where an expert is not available."""
    ok = x > float("-inf")
    if score == "sigmoid":
        return torch.where(ok, 1 / (1 + torch.exp(-x)), torch.zeros_like(x))
    m = x.max(1, keepdim=True).values
    e = torch.where(ok, torch.exp(torch.where(x == m, torch.zeros_like(x), x - m)), torch.zeros_like(x))
    return e / e.sum(1, keepdim=True).clamp_min(1e-300)


def _selected_weights(x, ids, score, norm, scale):
    """(weights before scaling, scores) of the selected slots, in x's precision; -1 slots give 0."""
    on = ids >= 0
    at = ids.clamp_min(0).long()
    xs = torch.where(on, x.gather(1, at), torch.full_like(x[:, :1], float("-inf")))
    s = _scores(xs if score == "sigmoid" or norm else x, score)
    if not norm:
        s = s if score == "sigmoid" else torch.where(on, s.gather(1, at), torch.zeros_like(xs))
        return s, s
    return s / s.sum(1, keepdim=True).clamp_min(1e-30), s


def _plain_router(c, logits, bias):
    x = logits.float()
    x = torch.where(x.isnan(), torch.full_like(x, float("-inf")), x)
    x64 = x.double()
    T, E, G = c["T"], c["E"], c["groups"]
    none = torch.full_like(x64, float("-inf"))
    # who is chosen is decided in 64 bits: scores of two experts may lie closer together than 32 bits tell apart
    s = torch.where(x > float("-inf"), _scores(x64, c["score"]), none)
    key = x64 if bias is None else s + bias.double()
    if G > 1:
        gk = key if c["group_top"] == 1 else (s if bias is None else key)
        top = gk.view(T, G, E // G).sort(2, descending=True).values[:, :, :c["group_top"]]
        some = top[:, :, 0] > float("-inf")
        gs = torch.where(some, torch.where(top > float("-inf"), top, torch.zeros_like(top)).sum(2),
                         torch.full_like(top[:, :, 0], float("-inf")))
        keep = gs.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        gm = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, keep, True)
        key = torch.where(gm.repeat_interleave(E // G, 1), key, none)
    val, idx = key.sort(dim=1, descending=True, stable=True)
    ids = torch.where(val[:, :c["k"]] > float("-inf"), idx[:, :c["k"]], torch.full_like(idx[:, :1], -1)).to(torch.int32)
    w, _ = _selected_weights(x, ids, c["score"], c["norm"], c["scale"])
    return {"ids": ids, "weights": w * c["scale"]}


def _plain_router_bwd(c, logits, ids, dw):
    x = logits.float()
    w, s = _selected_weights(x, ids, c["score"], c["norm"], c["scale"])
    at = ids.clamp_min(0).long()
    on = ids >= 0
    g = torch.where(on, dw, torch.zeros_like(dw)) * c["scale"]
    if c["norm"]:
        d = w * (g - (g * w).sum(1, keepdim=True))
        if c["score"] == "sigmoid":
            d = d / (1 + torch.exp(torch.where(on, x.gather(1, at), torch.zeros_like(dw))))
        full = torch.zeros_like(x).scatter_add_(1, at, torch.where(on, d, torch.zeros_like(d)))
    elif c["score"] == "sigmoid":
        d = g * s / (1 + torch.exp(torch.where(on, x.gather(1, at), torch.zeros_like(dw))))
        full = torch.zeros_like(x).scatter_add_(1, at, d)
    else:
        p = _scores(x, "softmax")
        full = torch.zeros_like(x).scatter_add_(1, at, g * s) - p * (g * s).sum(1, keepdim=True)
    return {"dlogits": full.to(logits.dtype)}


def _plain_combine_bwd(dZ, Y, oi, w, dY_and_spare):
    spare = Y.shape[0]  # the row that dropped routes write
    at = oi.clamp_min(0).long()
    on = oi >= 0
    dz = dZ.float()
    dw = (Y[at].float() * dz[:, None, :]).sum(2)
    rows = (w[:, :, None] * dz[:, None, :]).to(torch.bfloat16)
    dY_and_spare.index_copy_(0, torch.where(on, at, torch.full_like(at, spare)).view(-1), rows.view(-1, rows.shape[2]))
    return {"dY": dY_and_spare[:spare], "dweights": torch.where(on, dw, torch.zeros_like(dw))}


def _dequant(codes, sf, gran, dtype):
    rows, K = codes.shape
    s = sf.to(dtype).repeat_interleave(128, 1)
    if gran > 1:
        s = s.repeat_interleave(gran, 0)[:rows]
    return codes.view(torch.float8_e4m3fn).to(dtype) * s


def _plain_gemm(c, A, SFA, W, SFW, C, D):
    d = _dequant(A, SFA, 1, torch.float32) @ _dequant(W, SFW, c["gran_n"], torch.float32).t()
    if C is not None:
        d = d + C
    D.copy_(d)
    return {"D": D}


def _plain_quant_t(x):
    M, K = x.shape
    mb = -(-M // 128)
    p = torch.zeros(128 * mb, K, device=x.device)
    p[:M] = x.float()
    t = p.t().contiguous().view(K, mb, 128)
    amax = t.abs().amax(2)
    man, ex = torch.frexp(amax)
    e = torch.where(man <= 0.875, ex - 9, ex - 8).clamp(-126, 127)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    one = torch.ones_like(amax)
    q = torch.ldexp(t, -e[:, :, None]).to(torch.float8_e4m3fn)
    return {"q": q.view(K, 128 * mb), "sf": torch.ldexp(one, e)}


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        return _run_own(state, c, op)
    if op == "router":
        return _plain_router(c, state["logits"], state["bias"])
    if op == "router_bwd":
        return _plain_router_bwd(c, state["logits"], state["ids"], state["dweights"])
    if op == "combine_bwd":
        return _plain_combine_bwd(state["dZ"], state["Y"], state["output_index"], state["topk_weights"],
                                  state["dY_and_spare"])
    if op == "gemm":
        return _plain_gemm(c, state["A"], state["SFA"], state["W"], state["SFW"], state["C"], state["D"])
    return _plain_quant_t(state["x"])


def _run_own(state, c, op):
    import int4_weights_amd as moe

    if op == "router":
        moe.moe_router_topk(state["logits"], state["ids"], state["weights"], score=c["score"], bias=state["bias"],
                            n_group=c["groups"], topk_group=c["topk_group"], group_top=c["group_top"],
                            renormalize=c["norm"], scale=c["scale"])
        return {"ids": state["ids"], "weights": state["weights"]}
    if op == "router_bwd":
        moe.moe_router_topk_bwd(state["logits"], state["ids"], state["dweights"], state["dlogits"], score=c["score"],
                                renormalize=c["norm"], scale=c["scale"])
        return {"dlogits": state["dlogits"]}
    if op == "combine_bwd":
        if "ws" not in state:  # kept by the program, as a layer keeps its workspace
            n = moe.moe_unpermute_combine_bwd_workspace_bytes(c["T"], c["k"], state["Y"].shape[0])
            state["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        moe.moe_unpermute_combine_bwd(state["dZ"], state["Y"], state["output_index"], state["topk_weights"],
                                      state["dY"], state["dweights"], workspace=state["ws"])
        return {"dY": state["dY"], "dweights": state["dweights"]}
    if op == "gemm":
        if "ws" not in state:
            n = moe.moe_gemm_fp8_workspace_bytes(c["M"], c["N"], c["K"])
            state["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        moe.moe_gemm_fp8(state["A"], state["SFA"], state["W"], state["SFW"], state["D"], C=state["C"],
                         workspace=state["ws"])
        return {"D": state["D"]}
    moe.moe_quant_act_t(state["x"], state["q"], state["sf"])
    return {"q": state["q"].view(torch.float8_e4m3fn), "sf": state["sf"]}


def work(case):
    op = case["op"]
    if op in ("router", "router_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "fp32" else 2
        if op == "router":  # logits and bias in, ids and weights out; a few operations on each score
            return {"bytes": T * E * size + T * k * 8 + (E * 4 if case["bias"] else 0), "flops": 8 * T * E}
        # the whole row is read only where its softmax is needed; d logits are always written whole
        read = E * size if case["score"] == "softmax" and not case["norm"] else k * size
        return {"bytes": T * (read + 8 * k + E * size), "flops": T * (8 * E if read > k * size else 12 * k)}
    if op == "combine_bwd":
        T, k, N = case["T"], case["k"], case["N"]
        R = T * k - min(case["dropped"], T * k - 1)
        return {"bytes": 2 * T * N + 4 * R * N + 12 * T * k, "flops": 3 * R * N}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        size = 2 if case["out"] == "bf16" else 4
        scales = 4 * (K // 128) * (M + -(-N // case["gran_n"]))
        return {"bytes": (M + N) * K + scales + M * N * (size + (4 if case["add"] else 0)), "flops": 2 * M * N * K}
    M, K = case["M"], case["K"]
    mb = -(-M // 128)
    return {"bytes": 2 * M * K + K * 128 * mb + 4 * K * mb, "flops": 2 * M * K}


# ------------------------------------------------------------------------------------------------------ exact --


def _exact_select(c, x, bias):
    """The router's choice, one slot after another, in 64 bits: (ids, on)."""
    T, E, G = c["T"], c["E"], c["groups"]
    rows = torch.arange(T, device=x.device)
    ninf = float("-inf")
    if c["score"] == "sigmoid":
        s = torch.sigmoid(x)
    else:
        s = torch.softmax(x, 1)
    s = torch.where(x == ninf, torch.full_like(x, ninf), s)
    if bias is not None:
        s = s + bias.double()
        order = s
    else:
        order = x
    if G > 1:
        left = (order if c["group_top"] == 1 else s).reshape(T, G, E // G).clone()
        total = torch.zeros(T, G, dtype=torch.float64, device=x.device)
        for i in range(c["group_top"]):
            v, a = left.max(2)
            total += v if i == 0 else torch.where(v == ninf, torch.zeros_like(v), v)
            left.scatter_(2, a[:, :, None], ninf)
        allowed = torch.zeros(T, G, dtype=torch.bool, device=x.device)
        for _ in range(c["topk_group"]):
            a = torch.where(allowed, torch.full_like(total, ninf), total).argmax(1)
            allowed[rows, a] = True
        order = torch.where(allowed[:, :, None].expand(T, G, E // G).reshape(T, E), order, torch.full_like(order, ninf))
    order = order.clone()
    ids, on = [], []
    for _ in range(c["k"]):
        v, a = order.max(1)
        # max() may name any of several equal experts; the lowest one counts
        a = (order == v[:, None]).to(torch.int8).argmax(1)
        ids.append(a)
        on.append(v > ninf)
        order[rows, a] = ninf
    return torch.stack(ids, 1), torch.stack(on, 1)


def _exact_weights(c, x, ids, on):
    """Weights (unscaled) of the slots as a function of x [T, E] in 64 bits."""
    chosen = x.gather(1, ids)
    if c["score"] == "softmax":
        log_s = torch.log_softmax(x, 1).gather(1, ids)
    else:
        log_s = torch.nn.functional.logsigmoid(chosen)
    log_s = torch.where(on, log_s, torch.full_like(log_s, float("-inf")))
    return torch.where(on, torch.softmax(log_s, 1) if c["norm"] else log_s.exp(), torch.zeros_like(log_s))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "router":
        x = s["logits"].double()
        ids, on = _exact_select(case, x, s["bias"])
        return {"ids": None, "weights": case["scale"] * _exact_weights(case, x, ids, on)}
    if op == "router_bwd":
        x = s["logits"].double().requires_grad_(True)
        ids, on = s["ids"].long().clamp_min(0), s["ids"] >= 0
        with torch.enable_grad():
            w = case["scale"] * _exact_weights(case, x, ids, on)
            (dx,) = torch.autograd.grad((w * s["dweights"].double()).sum(), x)
        return {"dlogits": dx}
    if op == "combine_bwd":
        T, k, N = case["T"], case["k"], case["N"]
        dY = torch.zeros(s["Y"].shape, dtype=torch.float64, device=DEV)
        dw = torch.zeros(T, k, dtype=torch.float64, device=DEV)
        dz = s["dZ"].double()
        for r in range(k):
            i = s["output_index"][:, r].long()
            t = (i >= 0).nonzero()[:, 0]
            dY[i[t]] = s["topk_weights"][t, r].double()[:, None] * dz[t]
            dw[t, r] = torch.linalg.vecdot(s["Y"][i[t]].double(), dz[t])
        return {"dY": dY, "dweights": dw}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        d = torch.zeros(M, N, dtype=torch.float64, device=DEV) if s["C"] is None else s["C"].double()
        a = s["A"].view(torch.float8_e4m3fn).double().view(M, K // 128, 128) * s["SFA"].double()[:, :, None]
        rows = torch.arange(N, device=DEV) // case["gran_n"]
        w = s["W"].view(torch.float8_e4m3fn).double().view(N, K // 128, 128) * s["SFW"].double()[rows][:, :, None]
        return {"D": torch.addmm(d, a.view(M, K), w.view(N, K).t())}
    # the scaled values that the codes stand for (before their rounding), and the scales
    x = s["x"].double()
    M, K = x.shape
    mb = -(-M // 128)
    blocks = torch.nn.functional.pad(x, (0, 0, 0, 128 * mb - M)).view(mb, 128, K)
    amax = blocks.abs().amax(1)
    sf = torch.where(amax > 0, torch.exp2(torch.ceil(torch.log2(amax / 448)).clamp(-126, 127)), torch.ones_like(amax))
    return {"q": (blocks / sf[:, None, :]).view(128 * mb, K).t(), "sf": sf.t()}
