"""Cases for the few-token expert layer and the dense bf16 product with its epilogue and gradient.

The operators (names as in include/moe.h):

  experts      moe_experts_decode: up-projection, SwiGLU, down-projection and weighted sum of every token's experts
  linear       moe_gemm_bf16: D = C + act(A W^T + bias), optionally with the pre-activation kept
  linear_grad  moe_gemm_bf16 with operands in their stored order: dX = dP W and dW += dP^T X
  act_grad     moe_act_bwd: dP = dD * act'(pre), and the bias's gradient

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
        # One token through the DeepSeek-V3-shaped layer: the latency of a single decode stream, FP8 weights.
        {"name": "experts_one_fp8", "op": "experts", "T": 1, "E": 256, "k": 8, "H": 7168, "I": 2048, "weights": "fp8",
         "packed": False, "residual": True, "dropped": 0},
        # The 16-token, 128-expert decode step with 4-bit weights, in the order the grouped product reads fastest.
        {"name": "experts_16_int4", "op": "experts", "T": 16, "E": 128, "k": 8, "H": 4096, "I": 768, "weights": "int4",
         "packed": True, "residual": False, "dropped": 0},
        # Three tokens of a small layer, one route dropped by a full expert: launches and latency count.
        {"name": "experts_3_bf16", "op": "experts", "T": 3, "E": 64, "k": 6, "H": 2048, "I": 1408, "weights": "bf16",
         "packed": False, "residual": False, "dropped": 1},
        # A batch of 61 decode streams over the Qwen3-shaped layer in bf16: nearly every expert is active.
        {"name": "experts_61_bf16", "op": "experts", "T": 61, "E": 128, "k": 8, "H": 4096, "I": 1536, "weights": "bf16",
         "packed": False, "residual": True, "dropped": 0},
        # The router's gate projection in a decode step: fp32 logits of 256 experts for 16 tokens.
        {"name": "linear_gate", "op": "linear", "M": 16, "N": 256, "K": 7168, "act": "none", "gated": False,
         "bias": False, "residual": "", "out": "fp32", "pre": False},
        # The shared expert's up-projection with SwiGLU for one token.
        {"name": "linear_one_swiglu", "op": "linear", "M": 1, "N": 4096, "K": 7168, "act": "silu", "gated": True,
         "bias": False, "residual": "", "out": "bf16", "pre": False},
        # Its down-projection added to the routed experts' result, an odd mixed batch.
        {"name": "linear_131_residual", "op": "linear", "M": 131, "N": 7168, "K": 2048, "act": "none", "gated": False,
         "bias": False, "residual": "bf16", "out": "bf16", "pre": False},
        # A training batch through a GELU layer with bias, the pre-activation kept for the gradient.
        {"name": "linear_4096_gelu", "op": "linear", "M": 4096, "N": 4096, "K": 7168, "act": "gelu", "gated": False,
         "bias": True, "residual": "", "out": "bf16", "pre": True},
        # Gradients of a small projection over an odd number of tokens.
        {"name": "linear_grad_333", "op": "linear_grad", "M": 333, "N": 1536, "K": 2048, "residual": False},
        # Gradients of the large one over the training batch, dX joined with the gradient of another branch.
        {"name": "linear_grad_4096", "op": "linear_grad", "M": 4096, "N": 4096, "K": 7168, "residual": True},
        # Activation's and bias's gradient: a small odd batch with GELU, the training batch with SwiGLU.
        {"name": "act_grad_333_gelu", "op": "act_grad", "M": 333, "N": 1536, "act": "gelu", "gated": False},
        {"name": "act_grad_4096_swiglu", "op": "act_grad", "M": 4096, "N": 4096, "act": "silu", "gated": True},
    ]


ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def _logrand(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["experts", "experts", "experts", "linear", "linear", "linear", "linear_grad", "act_grad"])
    if op == "experts":
        weights = rng.choice(["bf16", "fp8", "int4"])
        H, I = 128 * rng.randint(4, 32), 128 * rng.randint(1, 12)
        E = _logrand(rng, 4, 128)
        k = rng.randint(1, min(8, E))
        T = _logrand(rng, 1, 61)
        return {"op": op, "T": T, "E": E, "k": k, "H": H, "I": I, "weights": weights, "packed": rng.random() < 0.5,
                "residual": rng.random() < 0.5, "dropped": rng.choice([0, 0, 1, 3])}
    if op == "act_grad":
        N = 8 * _logrand(rng, 8, 512)
        return {"op": op, "M": _logrand(rng, 1, 4096), "N": N, "act": rng.choice(ACTS), "gated": rng.random() < 0.5}
    K = 8 * rng.randint(8, 896)
    N = 8 * _logrand(rng, 4, 896)
    M = _logrand(rng, 1, max(1, min(8192, 4096 * 4096 * 7168 // (N * K))))
    if op == "linear_grad":
        return {"op": op, "M": M, "N": N, "K": K, "residual": rng.random() < 0.5}
    gated = rng.random() < 0.3
    return {"op": op, "M": M, "N": 2 * N if gated and N <= 3584 else N, "K": K, "act": rng.choice(ACTS),
            "gated": gated and N <= 3584, "bias": rng.random() < 0.5, "residual": rng.choice(["", "bf16", "fp32"]),
            "out": rng.choice(["bf16", "bf16", "fp32"]), "pre": rng.random() < 0.3}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16).mul_(std)


def _weights(kind, E, N, K, g):
    """Expert weights N(0, 0.02) as a checkpoint of this format holds them: (values or codes, scales or None)."""
    if kind == "bf16":
        return _normal(g, E, N, K, std=0.02), None
    if kind == "fp8":  # codes that fill the format's range block by block, one fp32 scale per 128x128
        q = _normal(g, E, N, K, std=100.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s = torch.empty(E, N // 128, K // 128, device=DEV).uniform_(1.5e-4, 2.5e-4, generator=g)
        return q, s
    q = _normal(g, E, N, K, std=2.3).round_().add_(8).clamp_(0, 15).to(torch.uint8)
    s = torch.empty(E, N, K // 128, device=DEV).uniform_(7e-3, 1.1e-2, generator=g)
    return q[:, :, 0::2] | (q[:, :, 1::2] << 4), s.to(torch.float16)


def _packed(kind, w, s):
    """The weights in the order that the framework's products read fastest, laid out once by the program; s too."""
    E, N = w.shape[:2]
    if kind == "int4":
        K = 2 * w.shape[2]
        c = _int4_codes(w).view(E, N // 16, 16, K // 128, 4, 4, 8)  # cb, c16, g, d, h, k
        c = c[..., [0, 2, 4, 6, 1, 3, 5, 7]].permute(0, 3, 1, 5, 2, 4, 6)  # g, cb, h, c16, d, nibble
        sp = s.view(E, N // 64, 4, 16, K // 128).permute(0, 4, 1, 3, 2)
        return (c[..., 0::2] | (c[..., 1::2] << 4)).reshape(w.shape), sp.reshape(s.shape).contiguous()
    b = w.view(torch.uint8) if kind == "fp8" else w.view(torch.uint8).view(E, N, -1)
    p = b.view(E, N // 16, 16, b.shape[2] // 128, 2, 4, 16).permute(0, 3, 1, 4, 5, 2, 6).contiguous()
    return (p.view(w.shape) if kind == "fp8" else p.view(torch.bfloat16).view(w.shape)), s


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": dict(case)}
    op = case["op"]
    if op == "experts":
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        s["x"] = _normal(g, T, H)
        s["ids"] = torch.randn(T, E, generator=g, device=DEV).topk(k, dim=1).indices.to(torch.int32)
        drop = torch.randperm(T * k, generator=g, device=DEV)[:min(case["dropped"], T * k - 1)]
        s["ids"].view(-1)[drop] = -1
        s["p"] = torch.softmax(torch.randn(T, k, generator=g, device=DEV), 1)
        for name, n, kk in (("13", 2 * I, H), ("2", H, I)):
            w, sc = _weights(case["weights"], E, n, kk, g)
            s["plain_w" + name], s["plain_s" + name] = w, sc
            s["w" + name], s["s" + name] = _packed(case["weights"], w, sc) if case["packed"] else (w, sc)
        s["C"] = _normal(g, T, H) if case["residual"] else None
        s["Z"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
        return s
    M, N = case["M"], case["N"]
    if op == "linear":
        K = case["K"]
        half = N // 2 if case["gated"] else N
        s["A"], s["W"] = _normal(g, M, K), _normal(g, N, K, std=0.02)
        s["bias"] = torch.randn(N, generator=g, device=DEV) * 0.1 if case["bias"] else None
        s["C"] = _normal(g, M, half) if case["residual"] else None
        if case["residual"] == "fp32":
            s["C"] = s["C"].float()
        s["D"] = torch.empty(M, half, dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16, device=DEV)
        s["pre"] = torch.empty(M, N, dtype=torch.bfloat16, device=DEV) if case["pre"] else None
    elif op == "linear_grad":
        K = case["K"]
        s["X"], s["W"], s["dP"] = _normal(g, M, K), _normal(g, N, K, std=0.02), _normal(g, M, N)
        s["C"] = _normal(g, M, K) if case["residual"] else None
        s["dX"] = torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
        s["before"] = torch.randn(N, K, generator=g, device=DEV)  # the gradient of the step so far
        s["dW"] = torch.empty(N, K, device=DEV)
    else:
        half = N // 2 if case["gated"] else N
        s["dD"], s["pre"] = _normal(g, M, half), _normal(g, M, N, std=1.5)
        s["dP"] = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        s["dbias"] = torch.empty(N, device=DEV)
    return s


# ------------------------------------------------------------------------------------------------- plain form --


def _int4_codes(q):
    return torch.stack((q & 15, q >> 4), -1).view(q.shape[0], q.shape[1], 2 * q.shape[2])


def _values(kind, w, s, dtype):
    """The numbers that weights of shape [n, N, K] stand for."""
    if kind == "bf16":
        return w.to(dtype)
    if kind == "fp8":
        n, N, K = w.shape
        v = w.view(torch.float8_e4m3fn).to(dtype).view(n, N // 128, 128, K // 128, 128)
        return (v * s.to(dtype)[:, :, None, :, None]).view(n, N, K)
    v = (_int4_codes(w).to(dtype) - 8).view(w.shape[0], w.shape[1], -1, 128)
    return (v * s.to(dtype)[..., None]).view(w.shape[0], w.shape[1], -1)


def _act(name, v):
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _slope(name, v):
    """The derivative of _act."""
    if name == "relu":
        return (v > 0).to(v.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-v))
        return s * (1 + v * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) * (1 / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-c * (v + 0.044715 * v * v * v)))
        return s + v * s * (1 - s) * c * (1 + 3 * 0.044715 * v * v)
    return torch.ones_like(v)


def _plain_experts(c, st):
    T, E, k, H, I, kind = (c[n] for n in ("T", "E", "k", "H", "I", "weights"))
    x, on = st["x"].float(), st["ids"] >= 0
    at = st["ids"].clamp_min(0).long()
    p = torch.where(on, st["p"], torch.zeros_like(st["p"]))
    some = (lambda w: None if w is None else w[at.view(-1)]) if T * k <= E else (lambda w: w)
    w13 = _values(kind, some(st["plain_w13"]), some(st["plain_s13"]), torch.float32)
    if T * k <= E:  # every route's own expert
        gu = torch.bmm(w13, x.repeat_interleave(k, 0)[:, :, None])[:, :, 0]
        del w13
        h = _act("silu", gu[:, :I]) * gu[:, I:] * p.view(-1, 1)
        w2 = _values(kind, some(st["plain_w2"]), some(st["plain_s2"]), torch.float32)
        z = torch.bmm(w2, h[:, :, None])[:, :, 0].view(T, k, H).sum(1)
    else:  # every expert for every token, weighted by what the token gives it
        share = torch.zeros(T, E, device=x.device).scatter_add_(1, at, p)
        gu = (x @ w13.view(E * 2 * I, H).t()).view(T, E, 2 * I)
        del w13
        h = _act("silu", gu[:, :, :I]) * gu[:, :, I:] * share[:, :, None]
        w2 = _values(kind, some(st["plain_w2"]), some(st["plain_s2"]), torch.float32)
        z = h.view(T, E * I) @ w2.transpose(1, 2).reshape(E * I, H)
    if st["C"] is not None:
        z = z + st["C"].float()
    return {"Z": z.to(torch.bfloat16)}


def _plain_linear(c, st):
    v = st["A"].float() @ st["W"].float().t()
    if st["bias"] is not None:
        v = v + st["bias"]
    half = st["D"].shape[1]
    d = _act(c["act"], v[:, :half]) * v[:, half:] if c["gated"] else _act(c["act"], v)
    if st["C"] is not None:
        d = d + st["C"].float()
    return {"D": d.to(st["D"].dtype), "pre": v.to(torch.bfloat16) if c["pre"] else None}


def _plain_linear_grad(st):
    dP = st["dP"].float()
    dX = dP @ st["W"].float()
    if st["C"] is not None:
        dX = dX + st["C"].float()
    return {"dX": dX.to(torch.bfloat16), "dW": st["before"] + dP.t() @ st["X"].float()}


def _plain_act_grad(c, st):
    dD, pre = st["dD"].float(), st["pre"].float()
    if c["gated"]:
        gate, up = pre[:, :dD.shape[1]], pre[:, dD.shape[1]:]
        d = torch.cat((dD * up * _slope(c["act"], gate), dD * _act(c["act"], gate)), 1)
    else:
        d = dD * _slope(c["act"], pre)
    return {"dP": d.to(torch.bfloat16), "dbias": d.sum(0)}


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        return _run_own(state, c, op)
    if op == "experts":
        return _plain_experts(c, state)
    if op == "linear":
        return _plain_linear(c, state)
    if op == "linear_grad":
        return _plain_linear_grad(state)
    return _plain_act_grad(c, state)


def _workspace(state, nbytes):
    """Kept by the program, as a layer keeps its workspace."""
    if "ws" not in state:
        state["ws"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=DEV)
    return state["ws"]


def _run_own(state, c, op):
    import int4_weights_amd as moe

    if op == "experts":
        ws = _workspace(state, moe.moe_experts_decode_workspace_bytes(c["T"], c["k"], c["I"]))
        moe.moe_experts_decode(state["x"], state["ids"], state["p"], state["w13"], state["w2"], state["Z"],
                               weights=c["weights"], s13=state["s13"], s2=state["s2"], packed=c["packed"],
                               residual=state["C"], workspace=ws)
        return {"Z": state["Z"]}
    if op == "linear":
        ws = _workspace(state, moe.moe_gemm_bf16_workspace_bytes(c["M"], c["N"], c["K"]))
        moe.moe_gemm_bf16(state["A"], state["W"], state["D"], bias=state["bias"], act=c["act"], gated=c["gated"],
                          C=state["C"], pre=state["pre"], workspace=ws)
        return {"D": state["D"], "pre": state["pre"]}
    if op == "linear_grad":
        M, N, K = c["M"], c["N"], c["K"]
        ws = _workspace(state, max(moe.moe_gemm_bf16_workspace_bytes(M, K, N), moe.moe_gemm_bf16_workspace_bytes(N, K, M)))
        moe.moe_gemm_bf16(state["dP"], state["W"], state["dX"], C=state["C"], trans_w=True, workspace=ws)
        moe.moe_gemm_bf16(state["dP"], state["X"], state["dW"], C=state["before"], trans_a=True, trans_w=True, workspace=ws)
        return {"dX": state["dX"], "dW": state["dW"]}
    ws = _workspace(state, moe.moe_act_bwd_workspace_bytes(c["M"], c["N"]))
    moe.moe_act_bwd(state["dD"], state["pre"], state["dP"], dbias=state["dbias"], act=c["act"], gated=c["gated"],
                    workspace=ws)
    return {"dP": state["dP"], "dbias": state["dbias"]}


def work(case):
    op = case["op"]
    if op == "experts":
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        R = T * k - min(case["dropped"], T * k - 1)
        active = E * (1 - (1 - k / E) ** T)  # expected, of distinct random experts per token
        each = {"bf16": 2.0, "fp8": 1.0 + 4 / 16384, "int4": 0.5 + 2 / 128}[case["weights"]]
        return {"bytes": active * 3 * I * H * each + 2 * T * H * (3 if case["residual"] else 2) + 8 * T * k,
                "flops": 6 * R * I * H}
    M, N = case["M"], case["N"]
    if op == "linear":
        K = case["K"]
        half = N // 2 if case["gated"] else N
        b = 2 * (M * K + N * K) + M * half * (4 if case["out"] == "fp32" else 2) + (4 * N if case["bias"] else 0)
        b += {"": 0, "bf16": 2, "fp32": 4}[case["residual"]] * M * half + (2 * M * N if case["pre"] else 0)
        return {"bytes": b, "flops": 2 * M * N * K}
    if op == "linear_grad":
        K = case["K"]
        return {"bytes": 2 * (M * N + M * K + N * K) + 2 * M * K * (2 if case["residual"] else 1) + 8 * N * K,
                "flops": 4 * M * N * K}
    half = N // 2 if case["gated"] else N
    return {"bytes": 2 * M * half + 4 * M * N + 4 * N, "flops": 12 * M * N}


# ------------------------------------------------------------------------------------------------------ exact --


def _exact_act(name, v):
    F = torch.nn.functional
    return {"none": lambda: v, "relu": lambda: F.relu(v), "silu": lambda: F.silu(v), "gelu": lambda: F.gelu(v),
            "gelu_tanh": lambda: F.gelu(v, approximate="tanh")}[name]()


def _exact_expert(case, s, e, which):
    """Expert e's matrix in 64 bits, from the row-major weights."""
    w, sc = s["plain_w" + which][e], s["plain_s" + which]
    if case["weights"] == "bf16":
        return w.double()
    if case["weights"] == "fp8":
        return w.view(torch.float8_e4m3fn).double() * sc[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    q = torch.empty(w.shape[0], 2 * w.shape[1], dtype=torch.float64, device=w.device)
    q[:, 0::2], q[:, 1::2] = (w % 16).double(), torch.div(w, 16, rounding_mode="floor").double()
    return (q - 8) * sc[e].double().repeat_interleave(128, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "experts":
        I = case["I"]
        z = torch.zeros(case["T"], case["H"], dtype=torch.float64, device=DEV)
        if s["C"] is not None:
            z += s["C"].double()
        x = s["x"].double()
        for e in sorted(set(s["ids"].view(-1).tolist()) - {-1}):
            t, r = (s["ids"] == e).nonzero(as_tuple=True)
            gu = torch.nn.functional.linear(x[t], _exact_expert(case, s, e, "13"))
            h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
            z.index_add_(0, t, s["p"][t, r].double()[:, None] * torch.nn.functional.linear(h, _exact_expert(case, s, e, "2")))
        return {"Z": z}
    if op == "linear":
        v = torch.nn.functional.linear(s["A"].double(), s["W"].double(), None if s["bias"] is None else s["bias"].double())
        half = s["D"].shape[1]
        d = _exact_act(case["act"], v[:, :half]) * (v[:, half:] if case["gated"] else 1)
        return {"D": d if s["C"] is None else d + s["C"].double(), "pre": v if case["pre"] else None}
    if op == "linear_grad":
        X, W = s["X"].double().requires_grad_(True), s["W"].double().requires_grad_(True)
        with torch.enable_grad():
            dX, dW = torch.autograd.grad(torch.nn.functional.linear(X, W), (X, W), s["dP"].double())
        return {"dX": dX if s["C"] is None else dX + s["C"].double(), "dW": dW + s["before"].double()}
    pre = s["pre"].double().requires_grad_(True)
    half = s["dD"].shape[1]
    with torch.enable_grad():
        d = _exact_act(case["act"], pre[:, :half]) * (pre[:, half:] if case["gated"] else 1)
        (dP,) = torch.autograd.grad(d, pre, s["dD"].double())
    return {"dP": dP, "dbias": dP.sum(0)}
