"""Cases that measure the operators of a mixture-of-experts feed-forward block.

Four operators, each in the directions it is used in:

  linear    Y = act(X W + b) + R, and its gradients dX, dW, db
  grouped   the same product for rows sorted by expert, one weight matrix an expert
  route     top-k of softmax(logits), the rows sorted by expert, and dlogits
  combine   rows copied to their experts' order, and the weighted sum that brings the experts' rows back,
            with their gradients

`own` selects between the plain form (elementary torch operations in 32 bits, rounded once at the end) and the
library's calls.  `exact` gives the same results from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

_handle = None


def _lib():
    """The library handle a user's program creates once."""
    global _handle
    if _handle is None:
        import programming_tiled_gemm_gb300 as g
        _handle = g.Gemm(0)
    return _handle


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token through one projection of a small model: the smallest call, launch latency counts
        {"name": "linear one token", "op": "linear", "way": "fwd", "M": 1, "K": 2048, "N": 2048, "dtype": "bf16",
         "act": "silu", "bias": True, "residual": False, "save": False},
        # a short ragged prompt, fp16, sizes that fill no tile, residual added in the epilogue, activation's input kept
        {"name": "linear odd f16", "op": "linear", "way": "fwd", "M": 77, "K": 1000, "N": 4104, "dtype": "f16",
         "act": "gelu", "bias": True, "residual": True, "save": True},
        # the largest product of the benchmark with a full epilogue: prefill of a large layer
        {"name": "linear large", "op": "linear", "way": "fwd", "M": 8192, "K": 8192, "N": 8192, "dtype": "bf16",
         "act": "gelu_tanh", "bias": True, "residual": True, "save": False},
        # gradients of a training step's feed-forward projection
        {"name": "linear backward", "op": "linear", "way": "bwd", "M": 4096, "K": 4096, "N": 4096, "dtype": "bf16",
         "act": "gelu_tanh", "bias": True},
        # the same for a small ragged batch: an adapter or a head
        {"name": "linear backward odd", "op": "linear", "way": "bwd", "M": 333, "K": 1032, "N": 776, "dtype": "f16",
         "act": "silu", "bias": True},
        # eight tokens of a decode batch, two experts each: the active experts' weights are streamed once
        {"name": "experts decode", "op": "grouped", "way": "fwd", "rows": 16, "E": 16, "K": 2048, "N": 1024,
         "dtype": "bf16", "act": "swiglu", "bias": False, "save": False, "skew": 0.5},
        # a prefill batch over 32 experts of unequal load, gated up projection
        {"name": "experts prefill", "op": "grouped", "way": "fwd", "rows": 16384, "E": 32, "K": 2048, "N": 2048,
         "dtype": "bf16", "act": "swiglu", "bias": True, "save": True, "skew": 1.0},
        # gradients of the experts' gated projection
        {"name": "experts backward", "op": "grouped", "way": "bwd", "rows": 8192, "E": 16, "K": 2048, "N": 1024,
         "dtype": "bf16", "act": "swiglu", "bias": True, "skew": 1.0},
        # routing of a decode batch from 16-bit logits (many ties), some experts switched off
        {"name": "route decode", "op": "route", "way": "fwd", "T": 16, "E": 64, "k": 4, "dtype": "bf16",
         "renormalize": True, "masked": 0.1},
        # routing of a training batch and its gradient
        {"name": "route train", "op": "route", "way": "train", "T": 16384, "E": 128, "k": 8, "dtype": "f32",
         "renormalize": True, "masked": 0.0},
        # rows out to their experts and back for a decode batch, residual added
        {"name": "combine decode", "op": "combine", "way": "fwd", "T": 16, "N": 2048, "E": 64, "k": 4, "dtype": "bf16",
         "residual": True, "dropped": 0.0},
        # the same for a training batch, with the gradients of rows and weights
        {"name": "combine train", "op": "combine", "way": "train", "T": 8192, "N": 4096, "E": 64, "k": 4,
         "dtype": "bf16", "residual": False, "dropped": 0.0},
    ]


def _log(rng, lo, hi, step=1):
    """An odd multiple of `step` up to `hi`, spread over the logarithm: drawn sizes fill no tile."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return (int(v / step) - 1 | 1) * step if v >= 2 * step else step


def draw(rng):
    op = rng.choice(["linear", "linear", "grouped", "grouped", "route", "combine"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "linear":
        if rng.random() < 0.5:
            return {"op": op, "way": "fwd", "M": _log(rng, 1, 8192), "K": _log(rng, 256, 8192, 8),
                    "N": _log(rng, 256, 8192, 8), "dtype": dtype,
                    "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"]),
                    "bias": rng.random() < 0.5, "residual": rng.random() < 0.5, "save": rng.random() < 0.5}
        return {"op": op, "way": "bwd", "M": _log(rng, 64, 8192), "K": _log(rng, 256, 4096, 8),
                "N": _log(rng, 256, 4096, 8), "dtype": dtype,
                "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"]), "bias": rng.random() < 0.5}
    if op == "grouped":
        way = rng.choice(["fwd", "bwd"])
        c = {"op": op, "way": way, "rows": _log(rng, 4 if way == "fwd" else 128, 16384), "E": rng.randint(4, 64),
             "K": _log(rng, 256, 2048, 8), "N": _log(rng, 256, 2048, 8), "dtype": dtype,
             "act": rng.choice(["none", "gelu", "silu", "swiglu"]), "bias": rng.random() < 0.5,
             "skew": rng.choice([0.0, 0.5, 1.0, 2.0])}
        if way == "fwd":
            c["save"] = rng.random() < 0.5
        return c
    if op == "route":
        E = rng.randint(4, 256)
        return {"op": op, "way": rng.choice(["fwd", "train"]), "T": _log(rng, 1, 32768), "E": E,
                "k": rng.randint(1, min(8, E)), "dtype": rng.choice(["bf16", "f16", "f32"]),
                "renormalize": rng.random() < 0.7, "masked": rng.choice([0.0, 0.2])}
    return {"op": op, "way": rng.choice(["fwd", "train"]), "T": _log(rng, 1, 8192), "N": _log(rng, 256, 4096, 8),
            "E": rng.randint(8, 64), "k": rng.randint(1, 4), "dtype": dtype, "residual": rng.random() < 0.5,
            "dropped": rng.choice([0.0, 0.1])}


def work(case):
    c = case
    if c["op"] in ("linear", "grouped"):
        M, K, N = c["M"] if c["op"] == "linear" else c["rows"], c["K"], c["N"]
        Nw = 2 * N if c["act"] == "swiglu" else N
        # an expert without rows is not read: the expected number of others
        E = 1 if c["op"] == "linear" else c["E"] * (1 - (1 - 1 / c["E"]) ** M)
        w = E * (K * Nw + (Nw if c["bias"] else 0))
        flops = 2.0 * M * K * Nw
        if c["way"] == "fwd":
            vals = M * K + w + M * N * (2 if c.get("residual") else 1) + (M * Nw if c["save"] else 0)
            return {"bytes": 2.0 * vals, "flops": flops}
        E_out = 1 if c["op"] == "linear" else c["E"]  # an expert without rows still has its (zero) gradient written
        vals = M * N + 2 * M * K + (M * Nw if c["act"] != "none" else 0) + (E + E_out) * K * Nw
        return {"bytes": 2.0 * vals + (4.0 * E_out * Nw if c["bias"] else 0), "flops": 2 * flops}
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        b = 2 if c["dtype"] != "f32" else 4
        fwd = T * E * b + T * k * 16 + 4 * (E + 1)
        return {"bytes": float(fwd + (T * E * 2 * b + T * k * 8 if c["way"] == "train" else 0)), "flops": 5.0 * T * E}
    T, N, k = c["T"], c["N"], c["k"]
    rows = T * k
    fwd = T * N + rows * N + rows * N + T * N * (2 if c["residual"] else 1)
    bwd = rows * N + T * N + T * N + 2 * rows * N
    vals = fwd + (bwd if c["way"] == "train" else 0)
    return {"bytes": 2.0 * vals + 12.0 * rows, "flops": (6.0 if c["way"] == "train" else 2.0) * rows * N}


# ------------------------------------------------------------------------------------------------ inputs

def _counts(E, rows, skew, seed):
    """Rows an expert gets: loads with a log-normal spread, as an untrained router gives them."""
    g = torch.Generator().manual_seed(seed)
    p = torch.exp(skew * torch.randn(E, generator=g, dtype=torch.float64))
    pick = torch.multinomial(p / p.sum(), rows, replacement=True, generator=g)
    return torch.bincount(pick, minlength=E).tolist()


def _sorted_rows(experts, E):
    """(slots [T, k], rows [T * k]): each assignment's place in the order by expert, and the assignment at each place;
    -1 where there is none."""
    flat = experts.reshape(-1).long()
    routed = flat >= 0
    order = torch.argsort(torch.where(routed, flat, torch.full_like(flat, E)), stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(flat.numel(), device=flat.device)
    slots = torch.where(routed, place, torch.full_like(place, -1)).reshape(experts.shape)
    rows = torch.where(torch.arange(flat.numel(), device=flat.device) < routed.sum(), order, torch.full_like(order, -1))
    return slots.to(torch.int32), rows.to(torch.int32)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dtype)

    s = {"case": c}
    if c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        Nw = 2 * N if c["act"] == "swiglu" else N
        s["x"], s["w"] = normal(M, K), normal(K, Nw, scale=K ** -0.5)
        if c["way"] == "fwd":
            s["bias"] = normal(Nw, scale=0.1) if c["bias"] else None
            s["residual"] = normal(M, N) if c["residual"] else None
        else:
            s["dy"] = normal(M, N)
            s["z"] = normal(M, Nw) if c["act"] != "none" else None
        return s
    if c["op"] == "grouped":
        R, E, K, N = c["rows"], c["E"], c["K"], c["N"]
        Nw = 2 * N if c["act"] == "swiglu" else N
        s["counts"] = _counts(E, R, c["skew"], seed)
        s["offsets"] = torch.tensor([0] + s["counts"]).cumsum(0).to(torch.int32).to(dev)
        s["x"], s["w"] = normal(R, K), normal(E, K, Nw, scale=K ** -0.5)
        if c["way"] == "fwd":
            s["bias"] = normal(E, Nw, scale=0.1) if c["bias"] else None
        else:
            s["dy"] = normal(R, N)
            s["z"] = normal(R, Nw) if c["act"] != "none" else None
        return s
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        s["logits"] = normal(T, E, scale=1.5)
        if c["masked"]:
            off = torch.rand(T, E, generator=g, device=dev) < c["masked"]
            s["logits"] = s["logits"].masked_fill(off, float("-inf"))
            s["logits"][::7] = float("-inf")  # padding tokens go to no expert
        s["dweights"] = normal(T, k, dtype=torch.float32)
        return s
    T, N, E, k = c["T"], c["N"], c["E"], c["k"]
    scores = torch.rand(T, E, generator=g, device=dev)
    experts = torch.topk(scores, k, dim=1).indices
    if c["dropped"]:
        experts = experts.masked_fill(torch.rand(T, k, generator=g, device=dev) < c["dropped"], -1)
    s["slots"], s["rows"] = _sorted_rows(experts, E)
    s["weights"] = torch.softmax(normal(T, k, dtype=torch.float32), dim=1).masked_fill(experts < 0, 0.0)
    s["x"], s["y"] = normal(T, N), normal(T * k, N)
    s["residual"] = normal(T, N) if c["residual"] else None
    s["dout"], s["dxr"] = normal(T, N), normal(T * k, N)
    return s


# ------------------------------------------------------------------------------------------------ plain forms

GELU_C = math.sqrt(2.0 / math.pi)


def _activate(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(GELU_C * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "swiglu":
        gate, up = z.chunk(2, dim=1)
        return gate / (1 + torch.exp(-gate)) * up
    return z


def _activate_backward(dy, z, act):
    """dZ = dY act'(Z)."""
    if act == "none":
        return dy
    if act == "relu":
        return torch.where(z > 0, dy, torch.zeros_like(dy))
    if act == "gelu":
        return dy * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        t = torch.tanh(GELU_C * (z + 0.044715 * z * z * z))
        return dy * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * GELU_C * (1 + 3 * 0.044715 * z * z))
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return dy * p * (1 + z * (1 - p))
    gate, up = z.chunk(2, dim=1)
    p = 1 / (1 + torch.exp(-gate))
    return torch.cat([dy * up * p * (1 + gate * (1 - p)), dy * gate * p], dim=1)


def _plain_linear(s):
    c, dt = s["case"], s["x"].dtype
    if c["way"] == "fwd":
        z = s["x"].float() @ s["w"].float()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _activate(z, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(dt), "z": z.to(dt)} if c["save"] else {"y": y.to(dt)}
    dz = _activate_backward(s["dy"].float(), s["z"].float() if s["z"] is not None else None, c["act"])
    out = {"dx": (dz @ s["w"].float().t()).to(dt), "dw": (s["x"].float().t() @ dz).to(dt)}
    if c["bias"]:
        out["db"] = dz.sum(0)
    return out


def _plain_grouped(s):
    c, dt, n = s["case"], s["x"].dtype, s["counts"]
    w = s["w"].float()
    x = s["x"].float().split(n)
    if c["way"] == "fwd":
        z = torch.cat([a @ b for a, b in zip(x, w)])
        if s["bias"] is not None:
            z = z + torch.cat([b.expand(m, -1) for m, b in zip(n, s["bias"].float())])
        y = _activate(z, c["act"])
        return {"y": y.to(dt), "z": z.to(dt)} if c["save"] else {"y": y.to(dt)}
    dz = _activate_backward(s["dy"].float(), s["z"].float() if s["z"] is not None else None, c["act"]).split(n)
    out = {"dx": torch.cat([a @ b.t() for a, b in zip(dz, w)]).to(dt),
           "dw": torch.stack([a.t() @ b for a, b in zip(x, dz)]).to(dt)}
    if c["bias"]:
        out["db"] = torch.stack([a.sum(0) for a in dz])
    return out


def _plain_route(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    l = s["logits"].float()
    top, pick = torch.sort(l, dim=1, descending=True, stable=True)
    top, pick = top[:, :k], pick[:, :k]
    here = top != float("-inf")
    m = l.amax(dim=1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(l - m)
    total = torch.exp(top - m).sum(1, keepdim=True) if c["renormalize"] else p.sum(1, keepdim=True)
    weights = torch.where(here, torch.exp(top - m) / total, torch.zeros_like(top))
    experts = torch.where(here, pick, torch.full_like(pick, -1))
    slots, rows = _sorted_rows(experts, E)
    counts = (experts.reshape(-1, 1) == torch.arange(E, device=l.device)).sum(0)
    offsets = torch.cat([torch.zeros_like(counts[:1]), counts.cumsum(0)]).to(torch.int32)
    out = {"weights": weights, "experts": experts.to(torch.int32), "slots": slots, "rows": rows, "offsets": offsets}
    if c["way"] == "train":
        dw = torch.where(here, s["dweights"], torch.zeros_like(weights))
        mean = (weights * dw).sum(1, keepdim=True)
        grad = torch.zeros_like(l) if c["renormalize"] else torch.nan_to_num(-p / total * mean)
        out["dlogits"] = grad.scatter_add(1, pick, weights * (dw - mean if c["renormalize"] else dw)).to(s["logits"].dtype)
    return out


def _plain_combine(s):
    c, dt, T, N, k = s["case"], s["x"].dtype, s["case"]["T"], s["case"]["N"], s["case"]["k"]
    slots, rows = s["slots"].long(), s["rows"].long()
    there, used = (slots >= 0)[:, :, None], (rows >= 0)[:, None]
    at = slots.clamp(min=0)
    token = rows.clamp(min=0) // k
    xr = torch.where(used, s["x"][token], torch.zeros((), dtype=dt, device=rows.device))
    y = torch.where(there, s["y"].float()[at], torch.zeros((), device=rows.device))
    o = (s["weights"][:, :, None] * y).sum(1)
    if s["residual"] is not None:
        o = o + s["residual"].float()
    out = {"xr": xr, "out": o.to(dt)}
    if c["way"] == "train":
        w = s["weights"].reshape(-1)[rows.clamp(min=0)][:, None]
        dout = s["dout"].float()
        out["dy"] = torch.where(used, w * dout[token], torch.zeros((), device=rows.device)).to(dt)
        out["dweights"] = (y * dout[:, None, :]).sum(2)
        out["dx"] = torch.where(there, s["dxr"].float()[at], torch.zeros((), device=rows.device)).sum(1).to(dt)
    return out


# ------------------------------------------------------------------------------------------------ the library's calls

def _own(s):
    c, lib = s["case"], _lib()
    if c["op"] in ("linear", "grouped"):
        if c["way"] == "fwd":
            if c["op"] == "linear":
                got = lib.linear(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"],
                                 save_preact=c["save"])
            else:
                got = lib.grouped_linear(s["x"], s["w"], s["offsets"], bias=s["bias"], act=c["act"],
                                         save_preact=c["save"])
            return {"y": got[0], "z": got[1]} if c["save"] else {"y": got}
        if c["op"] == "linear":
            dx, dw, db = lib.linear_backward(s["dy"], s["x"], s["w"], z=s["z"], act=c["act"], bias=c["bias"])
        else:
            dx, dw, db = lib.grouped_linear_backward(s["dy"], s["x"], s["w"], s["offsets"], z=s["z"], act=c["act"],
                                                     bias=c["bias"])
        return {"dx": dx, "dw": dw, "db": db} if c["bias"] else {"dx": dx, "dw": dw}
    if c["op"] == "route":
        r = lib.moe_route(s["logits"], c["k"], renormalize=c["renormalize"])
        out = {"weights": r.weights, "experts": r.experts, "slots": r.slots, "rows": r.rows, "offsets": r.offsets}
        if c["way"] == "train":
            out["dlogits"] = lib.moe_route_backward(s["dweights"], s["logits"], r.experts, renormalize=c["renormalize"])
        return out
    out = {"xr": lib.moe_dispatch(s["x"], s["rows"], c["k"]),
           "out": lib.moe_combine(s["y"], s["slots"], s["weights"], residual=s["residual"])}
    if c["way"] == "train":
        out["dy"], out["dweights"] = lib.moe_combine_backward(s["dout"], s["y"], s["slots"], s["rows"], s["weights"])
        out["dx"] = lib.moe_combine(s["dxr"], s["slots"])
    return out


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "grouped": _plain_grouped, "route": _plain_route,
            "combine": _plain_combine}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------ 64 bits

def _exact_act(z, act):
    """(act(z), z -> dy -> dz) by the derivative of each formula; sigmoid(z) = 1 / (1 + e^-z)."""
    sig = torch.sigmoid
    if act == "none":
        return z, lambda dy: dy
    if act == "relu":
        return z.clamp(min=0), lambda dy: dy * (z > 0)
    if act == "silu":
        return z * sig(z), lambda dy: dy * (sig(z) + z * sig(z) * sig(-z))
    if act == "gelu":  # z Phi(z), with Phi' the normal density
        cdf = 0.5 * torch.special.erfc(-z * 2 ** -0.5)
        return z * cdf, lambda dy: dy * (cdf + z * torch.exp(-z ** 2 / 2) * (2 * math.pi) ** -0.5)
    if act == "gelu_tanh":  # 0.5 (1 + tanh u) = sigmoid(2 u)
        u2 = 2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)
        slope = 2 * (2 / math.pi) ** 0.5 * (1 + 0.134145 * z ** 2)
        return z * sig(u2), lambda dy: dy * (sig(u2) + z * sig(u2) * sig(-u2) * slope)
    n = z.shape[1] // 2
    a, b = z[:, :n], z[:, n:]
    return a * sig(a) * b, lambda dy: torch.cat([dy * b * (sig(a) + a * sig(a) * sig(-a)), dy * a * sig(a)], 1)


def _exact_part(c, x, w, bias, residual, dy, z):
    """One weight matrix's share."""
    if c["way"] == "fwd":
        z = torch.einsum("mk,kn->mn", x.double(), w.double())
        if bias is not None:
            z += bias.double()
        y = _exact_act(z, c["act"])[0]
        return {"y": y + residual.double() if residual is not None else y, "z": z}
    dz = _exact_act(z.double() if z is not None else None, c["act"])[1](dy.double())
    return {"dx": torch.einsum("mn,kn->mk", dz, w.double()), "dw": torch.einsum("mk,mn->kn", x.double(), dz),
            "db": torch.einsum("mn->n", dz)}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "linear":
        got = _exact_part(c, s["x"], s["w"], s.get("bias"), s.get("residual"), s.get("dy"), s.get("z"))
    elif c["op"] == "grouped":
        parts, at = [], 0
        for e, n in enumerate(s["counts"]):
            sl = slice(at, at + n)
            parts.append(_exact_part(c, s["x"][sl], s["w"][e], s["bias"][e] if s.get("bias") is not None else None,
                                     None, s["dy"][sl] if "dy" in s else None,
                                     s["z"][sl] if s.get("z") is not None else None))
            at += n
        got = {name: (torch.stack if name in ("dw", "db") else torch.cat)([p[name] for p in parts])
               for name in parts[0]}
    elif c["op"] == "route":
        return _exact_route(c, s)
    else:
        return _exact_combine(c, s)
    if c["way"] == "fwd":
        return got if c["save"] else {"y": got["y"]}
    return got if c["bias"] else {"dx": got["dx"], "dw": got["dw"]}


def _exact_route(c, s):
    l, k = s["logits"].double(), c["k"]
    # the softmax's logarithm with the top-k taken from it one by one, lowest index first
    left, picks = l.clone(), []
    for _ in range(k):
        best = left.max(1, keepdim=True).values
        first = torch.where(left == best, torch.arange(c["E"], device=l.device), c["E"]).min(1, keepdim=True).values
        picks.append(torch.where(best > -math.inf, first, -1))
        left.scatter_(1, first, -math.inf)
    pick = torch.cat(picks, 1)
    on = torch.zeros_like(l).scatter_add(1, pick.clamp(min=0), (pick >= 0).double()) > 0
    live = on if c["renormalize"] else l > -math.inf
    p = torch.exp(l - torch.logsumexp(torch.where(live, l, -math.inf), 1, keepdim=True))
    p = torch.where(live, p, 0.0)
    weights = torch.where(pick >= 0, p.gather(1, pick.clamp(min=0)), 0.0)
    out = {"weights": weights, "experts": None, "slots": None, "rows": None, "offsets": None}
    if c["way"] == "train":
        up = torch.zeros_like(l).scatter_add(1, pick.clamp(min=0), torch.where(pick >= 0, s["dweights"].double(), 0.0))
        out["dlogits"] = p * (up - (p * up).sum(1, keepdim=True))
    return out


def _exact_combine(c, s):
    T, N, k = c["T"], c["N"], c["k"]
    slots = s["slots"].cpu().long()
    n = T * k
    # the exchange as one sparse matrix: assignment -> place
    a = torch.nonzero(slots.reshape(-1) >= 0).reshape(-1)
    place, token = slots.reshape(-1)[a].to(s["x"].device), (a // k).to(s["x"].device)
    w = s["weights"].double().reshape(-1)[a.to(s["x"].device)][:, None]
    zero = torch.zeros(n, N, dtype=torch.float64, device=s["x"].device)
    xr = zero.index_copy(0, place, s["x"].double()[token])
    o = torch.zeros(T, N, dtype=torch.float64, device=xr.device).index_add_(0, token, w * s["y"].double()[place])
    out = {"xr": xr, "out": o + s["residual"].double() if s["residual"] is not None else o}
    if c["way"] == "train":
        up = s["dout"].double()[token]
        out["dy"] = zero.index_copy(0, place, w * up)
        dots = torch.zeros(n, dtype=torch.float64, device=xr.device)
        dots[a.to(xr.device)] = torch.einsum("an,an->a", up, s["y"].double()[place])
        out["dweights"] = dots.reshape(T, k)
        out["dx"] = torch.zeros_like(o).index_add_(0, token, s["dxr"].double()[place])
    return out
