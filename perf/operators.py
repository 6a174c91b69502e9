"""Timing cases of the dense projections around the MoE layer and of the
layer's form for a few tokens.

Two operators, each in a plain form (elementary torch operations in 32 bits)
and, where ``own`` is true, through this package:

  linear   out = act(x W^T + bias) [* (x W_up^T + bias_up)] [+ residual]
           the router's logits, a shared expert's gate/up and down projections,
           and the projections before and after the layer, for one token up to
           a long prefill batch
  decode   the whole MoE layer for a few tokens: top-k routing of f32 logits,
           the experts' SwiGLU FFNs, the weighted combine, plus the residual;
           bf16 experts, or e4m3 experts with one scale per matrix

A case is a dict of plain values; ``listed`` and ``draw`` give cases,
``prepare`` their inputs, ``run`` one pass, ``exact`` the result in 64 bits.
"""
import math

import torch

own = False

F32, BF16 = "f32", "bf16"


def _linear(name, M, K, N, act="none", gated=False, bias="", residual=False, out=BF16, pad=0):
    return {"name": name, "op": "linear", "M": M, "K": K, "N": N, "act": act, "gated": gated,
            "bias": bias, "residual": residual, "out": out, "pad": pad}


def _decode(name, T, H, I, E, k, weights=BF16, zipf=False, residual=True):
    return {"name": name, "op": "decode", "T": T, "H": H, "I": I, "E": E, "k": k,
            "weights": weights, "zipf": zipf, "residual": residual}


def listed():
    return [
        # router logits of one token, 8 experts: pure latency
        _linear("router 1 token E8", 1, 4096, 8, out=F32),
        # router logits of a prefill batch over 128 experts, with a selection bias
        _linear("router 4096 tokens E128", 4096, 2048, 128, bias=F32, out=F32),
        # a shared expert's gate/up (SwiGLU) for one token: the weights' stream
        _linear("shared gate/up 1 token", 1, 7168, 2048, act="silu", gated=True),
        # its down projection onto the residual stream, an odd decode batch
        _linear("shared down 13 tokens", 13, 2048, 7168, residual=True),
        # a projection with bias and GELU, a batch too large to stream weights for free
        _linear("project 77 tokens", 77, 2880, 2880, act="gelu", bias=BF16, pad=64),
        # prefill: a shared expert's gate/up, and a dense FFN's down projection
        _linear("shared gate/up 8192 tokens", 8192, 7168, 2048, act="silu", gated=True),
        _linear("dense down 4096 tokens", 4096, 14336, 4096, residual=True),
        # one token through few large experts: bound by the weights' stream
        _decode("layer 1 token E8", 1, 4096, 14336, 8, 2),
        # one token through many small experts: latency and stream matter alike
        _decode("layer 1 token E128", 1, 2048, 768, 128, 8),
        # a small batch with popular experts shared between tokens
        _decode("layer 6 tokens E64", 6, 7168, 2048, 64, 8, zipf=True),
        # e4m3 experts: one token, and an odd batch
        _decode("layer e4m3 1 token E32", 1, 2880, 2880, 32, 4, weights="e4m3"),
        _decode("layer e4m3 13 tokens E32", 13, 2880, 2880, 32, 4, weights="e4m3"),
    ]


def _log(rng, lo, hi, step=1):
    """An integer in [lo, hi], even over the logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    if rng.random() < 0.55:
        most_flops = 2 * 8192 * 7168 * 4096
        while True:
            M = rng.randint(1, 16) if rng.random() < 0.5 else _log(rng, 17, 8192)
            K, N = _log(rng, 64, 14336, 8), _log(rng, 8, 14336)
            gated = rng.random() < 0.4
            if 2 * M * K * N * (2 if gated else 1) <= most_flops:
                break
        out = F32 if N <= 256 and not gated else BF16
        act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"]) if gated or rng.random() < 0.4 \
            else "none"
        c = _linear("", M, K, N, act=act, gated=gated, bias=rng.choice(["", BF16, F32]),
                    residual=rng.random() < 0.4, out=out, pad=rng.choice([0, 0, 8, 64]))
    else:
        weights = rng.choice([BF16, "e4m3"])
        while True:
            T = rng.randint(1, 16)
            E = rng.choice([8, 16, 32, 60, 64, 128])
            k = min(E, rng.choice([1, 2, 4, 6, 8]))
            H, I = _log(rng, 512, 7168, 64), _log(rng, 256, 14336, 64)
            # the assignments' weights (the plain form gathers them) and all experts'
            if T * k * H * I <= 48 * 7168 * 2048 and E * H * I <= 64 * 7168 * 2048:
                break
        c = _decode("", T, H, I, E, k, weights=weights, zipf=rng.random() < 0.3,
                    residual=rng.random() < 0.7)
    c.pop("name")
    return c


def _rand(gen, shape, std, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(std)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _e4m3(W):
    """(codes, scale) of one expert matrix: scale = amax / 448, nearest even."""
    amax = W.float().abs().amax()
    s = amax / torch.full_like(amax, 448.0)      # by a Python number it is not the rounded quotient
    return (W.float() / s).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn), s


def _inputs(case, seed):
    """Every tensor of a case, from the seed alone."""
    g = _gen(seed)
    c = case
    if c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        rows = 2 * N if c["gated"] else N
        out = torch.float32 if c["out"] == F32 else torch.bfloat16
        # rows of a wider buffer where pad > 0 (a slice of a fused projection)
        return {
            "x": _rand(g, (M, K + c["pad"]), 1.0)[:, :K],
            "w": _rand(g, (rows, K), 1.0 / math.sqrt(K)),
            "bias": _rand(g, (rows,), 0.1, torch.float32 if c["bias"] == F32 else torch.bfloat16)
            if c["bias"] else None,
            "residual": _rand(g, (M, N), 1.0, out) if c["residual"] else None,
        }
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    x = _rand(g, (T, H), 1.0)
    logits = (x.float() @ _rand(g, (H, E), 1.0 / math.sqrt(H), torch.float32))
    if c["zipf"]:
        rank = torch.randperm(E, generator=g, device="cuda").float() + 1.0
        logits = logits - 1.2 * rank.log()
    s = {"x": x, "logits": logits,
         "residual": _rand(g, (T, H), 1.0) if c["residual"] else None,
         "Wg": _rand(g, (E, H, I), 1.0 / math.sqrt(H)),
         "Wu": _rand(g, (E, H, I), 1.0 / math.sqrt(H)),
         "Wd": _rand(g, (E, I, H), 1.0 / math.sqrt(I))}
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "decode":
        if own:
            import mixture_experts_expert_route_b200 as moe
            s["layer"] = moe.MoELayer(
                s["Wg"], s["Wu"], s["Wd"], case["k"],
                dtype=moe.FP8_E4M3 if case["weights"] == "e4m3" else moe.BF16)
        if case["weights"] == "e4m3":
            for n in ("Wg", "Wu", "Wd"):
                W = s.pop(n)
                pairs = [_e4m3(W[e]) for e in range(W.shape[0])]
                s[n] = torch.stack([p[0].view(torch.uint8) for p in pairs])
                s[n + "_scale"] = torch.stack([p[1] for p in pairs])
    return s


def _act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.7071067811865476))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    return z


def _plain_linear(s):
    c = s["case"]
    y = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if c["gated"]:
        y = _act(y[:, :c["N"]], c["act"]) * y[:, c["N"]:]
    else:
        y = _act(y, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y if c["out"] == F32 else y.to(torch.bfloat16)


def _picked(s, name, ids):
    """The selected experts' matrices in 32 bits, one per assignment."""
    W = s[name][ids]
    if s["case"]["weights"] == "e4m3":
        return W.view(torch.float8_e4m3fn).float() * s[name + "_scale"][ids][..., None, None]
    return W.float()


def _plain_decode(s):
    c = s["case"]
    T, H, I, k = c["T"], c["H"], c["I"], c["k"]
    top, ids = torch.sort(s["logits"], dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    w = torch.exp(top - top[:, :1])
    w = w / w.sum(dim=1, keepdim=True)
    x = s["x"].float()[:, None, None, :].expand(T, k, 1, H)
    g = x @ _picked(s, "Wg", ids)
    u = x @ _picked(s, "Wu", ids)
    h = g / (1.0 + torch.exp(-g)) * u
    y = ((h @ _picked(s, "Wd", ids)).squeeze(2) * w[..., None]).sum(dim=1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"out": y.to(torch.bfloat16), "ids": ids.int(), "w": w}


def _own_linear(s):
    import mixture_experts_expert_route_b200 as moe
    c = s["case"]
    act = {"none": moe.ACT_NONE, "relu": moe.ACT_RELU, "silu": moe.ACT_SILU,
           "gelu": moe.ACT_GELU, "gelu_tanh": moe.ACT_GELU_TANH}[c["act"]]
    return moe.linear(s["x"], s["w"], bias=s["bias"], act=act, gated=c["gated"],
                      residual=s["residual"],
                      out_dtype=torch.float32 if c["out"] == F32 else torch.bfloat16)


def _own_decode(s):
    c = s["case"]
    ids = torch.empty((c["T"], c["k"]), dtype=torch.int32, device=s["x"].device)
    w = torch.empty((c["T"], c["k"]), dtype=torch.float32, device=s["x"].device)
    out = s["layer"].decode(s["x"], s["logits"], residual=s["residual"], ids=ids, w=w)
    return {"out": out, "ids": ids, "w": w}


def run(state):
    if state["case"]["op"] == "linear":
        return _own_linear(state) if own else _plain_linear(state)
    return _own_decode(state) if own else _plain_decode(state)


def work(case):
    c = case
    if c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        rows = 2 * N if c["gated"] else N
        ob = 4 if c["out"] == F32 else 2
        b = 2 * M * K + 2 * rows * K + ob * M * N * (2 if c["residual"] else 1)
        b += {"": 0, BF16: 2, F32: 4}[c["bias"]] * rows
        return {"bytes": b, "flops": 2 * M * rows * K}
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    experts = E * (1.0 - (1.0 - k / E) ** T)      # distinct ones, of even popularity
    b = experts * 3 * H * I * (1 if c["weights"] == "e4m3" else 2)
    b += 2 * T * H * (3 if c["residual"] else 2) + 4 * T * E + 8 * T * k
    return {"bytes": b, "flops": 2 * T * k * 3 * H * I}


def exact(case, seed):
    s = _inputs(case, seed)
    d = torch.float64
    if case["op"] == "linear":
        x, W = s["x"].to(d), s["w"].to(d)
        z = torch.addmm(torch.zeros((), dtype=d, device="cuda"), x, W.T)
        if s["bias"] is not None:
            z += s["bias"].to(d)
        up = None
        if case["gated"]:
            z, up = z.chunk(2, dim=1)
        f = {"none": lambda v: v, "relu": lambda v: v.clamp(min=0.0),
             "silu": lambda v: v * torch.sigmoid(v),
             "gelu": lambda v: v * torch.special.ndtr(v),
             "gelu_tanh": lambda v: v * torch.sigmoid(
                 2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))}[case["act"]]
        z = f(z) if up is None else f(z) * up
        return z if s["residual"] is None else z + s["residual"].to(d)
    T, k = case["T"], case["k"]
    lg = s["logits"].to(d).cpu()
    ids = torch.tensor([sorted(range(case["E"]), key=lambda e: (-float(r[e]), e))[:k] for r in lg])
    w = torch.softmax(lg.gather(1, ids), dim=1)

    def mat(name, e):
        if case["weights"] != "e4m3":
            return s[name][e].to(d)
        codes, scale = _e4m3(s[name][e])
        return codes.to(d) * scale.to(d)

    y = torch.zeros_like(s["x"], dtype=d) if s["residual"] is None else s["residual"].to(d)
    for e in sorted(set(ids.reshape(-1).tolist())):
        t, j = (ids == e).nonzero(as_tuple=True)
        xt = s["x"][t.cuda()].to(d)
        gate, up = xt @ mat("Wg", e), xt @ mat("Wu", e)
        y[t.cuda()] += w[t, j].cuda()[:, None] * ((gate * torch.sigmoid(gate) * up) @ mat("Wd", e))
    return {"out": y, "ids": ids.int(), "w": w}
