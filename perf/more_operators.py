"""Cases that measure the operators of a served and fine-tuned language model's step around its linear layers.

Three operators, each in the directions it is used in:

  adapted    Y = act(X W + s_i (X A_i) B_i + b) + R: a shared projection with every row's own low-rank adapter i
  layer      a whole mixture-of-experts layer for a few tokens: top-k of softmax(logits), the picked experts' two
             products and their weighted sum
  logprobs   log probabilities of given tokens, the entropy and the best alternatives, and the logits' gradient

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
        # one token of one request through a small model's projection with its adapter: launch latency counts
        {"name": "adapted one token", "op": "adapted", "M": 1, "K": 2048, "N": 2048, "n": 8, "r": 16, "requests": 0,
         "dtype": "bf16", "act": "none", "bias": True, "residual": False},
        # a decode batch, every row a request with an adapter of its own choice, some with none
        {"name": "adapted decode", "op": "adapted", "M": 32, "K": 4096, "N": 4096, "n": 16, "r": 16, "requests": 0,
         "dtype": "bf16", "act": "none", "bias": False, "residual": True},
        # sizes that fill no tile, fp16, a rank that is no power of two, a few short prompts
        {"name": "adapted odd f16", "op": "adapted", "M": 77, "K": 1000, "N": 4104, "n": 5, "r": 24, "requests": 4,
         "dtype": "f16", "act": "gelu", "bias": True, "residual": True},
        # prompts of eight requests in one batch, gated up projection
        {"name": "adapted prefill", "op": "adapted", "M": 8192, "K": 4096, "N": 2048, "n": 8, "r": 64, "requests": 8,
         "dtype": "bf16", "act": "swiglu", "bias": False, "residual": False},
        # one token through a layer of 64 experts: four experts' weights are read
        {"name": "layer one token", "op": "layer", "T": 1, "D": 2048, "F": 1024, "E": 64, "k": 4, "dtype": "bf16",
         "act": "swiglu", "bias": False, "residual": True, "masked": 0.0},
        # a decode batch through the same layer: most experts are picked by a token or two
        {"name": "layer decode", "op": "layer", "T": 16, "D": 2048, "F": 1024, "E": 64, "k": 4, "dtype": "bf16",
         "act": "swiglu", "bias": False, "residual": True, "masked": 0.0},
        # more tokens than experts, fp16, odd sizes, plain activation with biases, experts switched off and padding
        {"name": "layer odd f16", "op": "layer", "T": 48, "D": 1032, "F": 776, "E": 16, "k": 2, "dtype": "f16",
         "act": "gelu", "bias": True, "residual": False, "masked": 0.2},
        # a decode batch through experts as large as the benchmark's product, eight or so tokens each
        {"name": "layer large", "op": "layer", "T": 64, "D": 4096, "F": 4096, "E": 16, "k": 2, "dtype": "bf16",
         "act": "swiglu", "bias": False, "residual": True, "masked": 0.0},
        # sampling of one request: fp32 logits of a small vocabulary, five alternatives
        {"name": "logprobs one row", "op": "logprobs", "way": "fwd", "rows": 1, "V": 32000, "ld": 32000, "top": 5,
         "entropy": True, "temperature": 1.0, "dtype": "f32", "masked": 0.0},
        # a decode batch over a large vocabulary, twenty alternatives, constrained decoding masks a part
        {"name": "logprobs decode", "op": "logprobs", "way": "fwd", "rows": 64, "V": 131072, "ld": 131072, "top": 20,
         "entropy": True, "temperature": 0.7, "dtype": "bf16", "masked": 0.3},
        # a training batch over an odd vocabulary in rows that start on no 16-byte boundary: log probabilities and
        # entropy forward, the logits' gradient backward, prompt tokens left out
        {"name": "logprobs train odd", "op": "logprobs", "way": "train", "rows": 1000, "V": 50257, "ld": 50257,
         "top": 0, "entropy": True, "temperature": 1.0, "dtype": "bf16", "masked": 0.0},
        # the largest training batch: 4096 tokens of a large vocabulary, no entropy
        {"name": "logprobs train", "op": "logprobs", "way": "train", "rows": 4096, "V": 131072, "ld": 131072, "top": 0,
         "entropy": False, "temperature": 1.0, "dtype": "bf16", "masked": 0.0},
    ]


def _log(rng, lo, hi, step=1):
    """An odd multiple of `step` up to `hi`, spread over the logarithm: drawn sizes fill no tile."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return (int(v / step) - 1 | 1) * step if v >= 2 * step else step


def draw(rng):
    op = rng.choice(["adapted", "layer", "logprobs"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "adapted":
        M = _log(rng, 1, 8192)
        return {"op": op, "M": M, "K": _log(rng, 256, 4096, 8), "N": _log(rng, 256, 4096, 8), "n": rng.randint(1, 32),
                "r": 8 * rng.randint(1, 8), "requests": 0 if M <= 64 else rng.randint(1, 16), "dtype": dtype,
                "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), "bias": rng.random() < 0.5,
                "residual": rng.random() < 0.5}
    if op == "layer":
        E = rng.randint(4, 64)
        return {"op": op, "T": _log(rng, 1, 64), "D": _log(rng, 256, 4096, 8), "F": _log(rng, 256, 2048, 8), "E": E,
                "k": rng.randint(1, min(8, E)), "dtype": dtype, "act": rng.choice(["silu", "gelu", "relu", "swiglu"]),
                "bias": rng.random() < 0.5, "residual": rng.random() < 0.5, "masked": rng.choice([0.0, 0.2])}
    way = rng.choice(["fwd", "train"])
    V = _log(rng, 1000, 131072)
    return {"op": op, "way": way, "rows": _log(rng, 1, 2048 if way == "train" else 256), "V": V,
            "ld": rng.choice([V, (V + 127) // 128 * 128]), "top": rng.randint(0, 20) if way == "fwd" else 0,
            "entropy": rng.random() < 0.5, "temperature": rng.choice([1.0, 0.7, 1.3]),
            "dtype": rng.choice(["bf16", "f16", "f32"]), "masked": rng.choice([0.0, 0.3])}


def _picked(c):
    """Experts that T tokens pick, on average, of those left on."""
    left = max(c["E"] * (1 - c["masked"]), c["k"])
    return left * (1 - (1 - c["k"] / left) ** c["T"])


def work(case):
    c = case
    if c["op"] == "adapted":
        M, K, N, r = c["M"], c["K"], c["N"], c["r"]
        Nw = 2 * N if c["act"] == "swiglu" else N
        picks = c["requests"] or M
        used = c["n"] * (1 - (1 - 1 / (c["n"] + 1)) ** picks)  # adapters that some row uses
        vals = M * K + K * Nw + used * r * (K + Nw) + (Nw if c["bias"] else 0) + M * N * (2 if c["residual"] else 1)
        with_one = M * c["n"] / (c["n"] + 1)
        return {"bytes": 2.0 * vals + 4.0 * M, "flops": 2.0 * M * K * Nw + 2.0 * with_one * r * (K + Nw)}
    if c["op"] == "layer":
        T, D, F, E, k = c["T"], c["D"], c["F"], c["E"], c["k"]
        Fw = 2 * F if c["act"] == "swiglu" else F
        vals = _picked(c) * (D * Fw + F * D + (Fw + D if c["bias"] else 0)) + T * D * (3 if c["residual"] else 2)
        return {"bytes": 2.0 * vals + 4.0 * T * E, "flops": 2.0 * T * k * (D * Fw + F * D)}
    b = 4 if c["dtype"] == "f32" else 2
    logits = c["rows"] * c["V"] * b
    small = c["rows"] * (8 + 4 + (4 if c["entropy"] else 0) + c["top"] * 12)
    if c["way"] == "fwd":
        return {"bytes": float(logits + small), "flops": 5.0 * c["rows"] * c["V"]}
    return {"bytes": float(3 * logits + 2 * small), "flops": 11.0 * c["rows"] * c["V"]}


# ------------------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    c = case
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dtype)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device=dev)

    s = {"case": c}
    if c["op"] == "adapted":
        M, K, N, n, r = c["M"], c["K"], c["N"], c["n"], c["r"]
        Nw = 2 * N if c["act"] == "swiglu" else N
        s["x"], s["w"] = normal(M, K), normal(K, Nw, scale=K ** -0.5)
        s["a"], s["b"] = normal(n, K, r, scale=K ** -0.5), normal(n, r, Nw, scale=0.25 * r ** -0.5)
        s["scales"] = 1.0 + torch.rand(n, generator=g, device=dev)
        if c["requests"]:  # the rows of a request lie together
            cuts = whole(0, M + 1, c["requests"] - 1).sort().values
            request = (torch.arange(M, device=dev)[:, None] >= cuts[None, :]).sum(1)
            s["adapters"] = whole(-1, n, c["requests"])[request].to(torch.int32)
        else:
            s["adapters"] = whole(-1, n, M).to(torch.int32)
            if M == 1:
                s["adapters"].clamp_(min=0)
        s["bias"] = normal(Nw, scale=0.1) if c["bias"] else None
        s["residual"] = normal(M, N) if c["residual"] else None
        return s
    if c["op"] == "layer":
        T, D, F, E, k = c["T"], c["D"], c["F"], c["E"], c["k"]
        Fw = 2 * F if c["act"] == "swiglu" else F
        s["x"], s["logits"] = normal(T, D), normal(T, E, scale=1.5, dtype=torch.float32)
        if c["masked"]:
            off = torch.rand(T, E, generator=g, device=dev) < c["masked"]
            s["logits"] = s["logits"].masked_fill(off, float("-inf"))
            s["logits"][5::7] = float("-inf")  # padding tokens go to no expert
        s["w1"], s["w2"] = normal(E, D, Fw, scale=D ** -0.5), normal(E, F, D, scale=F ** -0.5)
        s["b1"] = normal(E, Fw, scale=0.1) if c["bias"] else None
        s["b2"] = normal(E, D, scale=0.1) if c["bias"] else None
        s["residual"] = normal(T, D) if c["residual"] else None
        return s
    rows, V = c["rows"], c["V"]
    s["logits"] = normal(rows, c["ld"], scale=2.0)[:, :V]
    s["tokens"] = whole(0, V, rows)
    if c["masked"]:
        off = torch.rand(rows, V, generator=g, device=dev) < c["masked"]
        off.scatter_(1, s["tokens"][:, None], False)
        s["logits"].masked_fill_(off, float("-inf"))
    if c["way"] == "train":
        s["tokens"][: rows // 8] = -100  # the prompt's tokens are given, not learnt
        s["dlogprobs"] = normal(rows, dtype=torch.float32)
        s["dentropy"] = normal(rows, scale=0.1, dtype=torch.float32) if c["entropy"] else None
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _activate(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "swiglu":
        gate, up = z.chunk(2, dim=-1)
        return gate / (1 + torch.exp(-gate)) * up
    return z


def _plain_adapted(s):
    c, x, adapters = s["case"], s["x"].float(), s["adapters"].long()
    z = x @ s["w"].float()
    a, b, on = s["a"].float(), s["b"].float(), (adapters >= 0)[:, None]
    if c["M"] <= c["n"]:  # a few rows: each one's own matrices
        at = adapters.clamp(min=0)
        u = (x[:, None, :] @ a[at])[:, 0] * s["scales"][at][:, None]
        z = z + torch.where(on, (u[:, None, :] @ b[at])[:, 0], torch.zeros((), device=x.device))
    else:  # all adapters of all rows, those not the row's own set to zero
        n, r = c["n"], c["r"]
        u = (x @ a.permute(1, 0, 2).reshape(c["K"], n * r)).reshape(-1, n, r)
        mine = (adapters[:, None] == torch.arange(n, device=x.device)) * s["scales"]
        z = z + (u * mine[:, :, None]).reshape(-1, n * r) @ b.reshape(n * r, -1)
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _activate(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(s["x"].dtype)}


def _plain_layer(s):
    c, T, E, k = s["case"], s["case"]["T"], s["case"]["E"], s["case"]["k"]
    x, l = s["x"].float(), s["logits"]
    top, pick = torch.sort(l, dim=1, descending=True, stable=True)
    top, pick = top[:, :k], pick[:, :k]
    here = top != float("-inf")
    m = torch.where(here[:, :1], top[:, :1], torch.zeros_like(top[:, :1]))
    e = torch.where(here, torch.exp(top - m), torch.zeros_like(top))
    weights = e / e.sum(1, keepdim=True).clamp(min=1e-30)
    if T * k < E:  # fewer picks than experts: each pick's own matrices
        z = (x[:, None, None, :] @ s["w1"][pick].float())[:, :, 0]
        if s["b1"] is not None:
            z = z + s["b1"][pick].float()
        y = (_activate(z, c["act"])[:, :, None, :] @ s["w2"][pick].float())[:, :, 0]
        if s["b2"] is not None:
            y = y + s["b2"][pick].float()
        out = (weights[:, :, None] * y).sum(1)
    else:  # every expert for every token, weighted by zero where it was not picked
        z = x @ s["w1"].float()
        if s["b1"] is not None:
            z = z + s["b1"].float()[:, None, :]
        y = _activate(z, c["act"]) @ s["w2"].float()
        if s["b2"] is not None:
            y = y + s["b2"].float()[:, None, :]
        dense = torch.zeros_like(l).scatter_add(1, pick, weights)
        out = (dense.t()[:, :, None] * y).sum(0)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return {"out": out.to(s["x"].dtype)}


def _plain_logprobs(s):
    c, tokens = s["case"], s["tokens"]
    l = s["logits"].float()
    z = (l - l.amax(dim=1, keepdim=True)) / c["temperature"]
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    logp = z - torch.log(total)
    given = tokens >= 0
    at = tokens.clamp(min=0)[:, None]
    out = {"logprobs": torch.where(given, logp.gather(1, at)[:, 0], torch.zeros_like(total[:, 0]))}
    p = e / total
    zero = torch.zeros((), device=l.device)
    if c["entropy"]:
        plogp = torch.where(p > 0, p * logp, zero)
        out["entropy"] = -plogp.sum(1)
    if c["top"]:
        top, pick = torch.sort(l, dim=1, descending=True, stable=True)
        top, pick = top[:, :c["top"]], pick[:, :c["top"]]
        out["top_logprobs"] = logp.gather(1, pick)
        out["top_tokens"] = torch.where(top > float("-inf"), pick, torch.full_like(pick, -1))
    if c["way"] == "train":
        gain = torch.where(given, s["dlogprobs"], zero)[:, None]
        d = (-gain * p).scatter_add(1, at, gain)
        if c["entropy"]:
            d = d - s["dentropy"][:, None] * (plogp + p * out["entropy"][:, None])
        out["dlogits"] = (d / c["temperature"]).to(s["logits"].dtype)
    return out


# ------------------------------------------------------------------------------------------------ the library's calls

def _own(s):
    c, lib = s["case"], _lib()
    if c["op"] == "adapted":
        return {"y": lib.adapted_linear(s["x"], s["w"], s["a"], s["b"], s["adapters"], scales=s["scales"],
                                        bias=s["bias"], act=c["act"], residual=s["residual"])}
    if c["op"] == "layer":
        return {"out": lib.moe_layer(s["x"], s["logits"], s["w1"], s["w2"], c["k"], act=c["act"], b1=s["b1"],
                                     b2=s["b2"], residual=s["residual"])}
    r = lib.token_logprobs(s["logits"], s["tokens"], top=c["top"], entropy=c["entropy"], temperature=c["temperature"])
    out = {"logprobs": r.logprobs}
    if c["entropy"]:
        out["entropy"] = r.entropy
    if c["top"]:
        out["top_logprobs"], out["top_tokens"] = r.top_logprobs, r.top_tokens
    if c["way"] == "train":
        out["dlogits"] = lib.token_logprobs_backward(s["dlogprobs"], s["logits"], s["tokens"], r,
                                                     dentropy=s["dentropy"], temperature=c["temperature"])
    return out


def run(state):
    if own:
        return _own(state)
    return {"adapted": _plain_adapted, "layer": _plain_layer, "logprobs": _plain_logprobs}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------ 64 bits

def _exact_act(z, act):
    """Each formula by another route: sigmoid(z) = 1 / (1 + e^-z)."""
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":  # z Phi(z)
        return z * 0.5 * torch.special.erfc(-z * 2 ** -0.5)
    if act == "gelu_tanh":  # 0.5 (1 + tanh u) = sigmoid(2 u)
        return z * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    if act == "swiglu":
        n = z.shape[-1] // 2
        return z[..., :n] * torch.sigmoid(z[..., :n]) * z[..., n:]
    return z


def _exact_adapted(c, s):
    x = s["x"].double()
    z = torch.einsum("mk,kn->mn", x, s["w"].double())
    for i in range(c["n"]):
        rows = torch.nonzero(s["adapters"] == i)[:, 0]
        if rows.numel():
            u = torch.einsum("mk,kr->mr", x[rows], s["a"][i].double())
            z[rows] += s["scales"][i].double() * torch.einsum("mr,rn->mn", u, s["b"][i].double())
    if s["bias"] is not None:
        z += s["bias"].double()
    y = _exact_act(z, c["act"])
    return {"y": y + s["residual"].double() if s["residual"] is not None else y}


def _exact_layer(c, s):
    out = s["residual"].double() if s["residual"] is not None else torch.zeros_like(s["x"], dtype=torch.float64)
    l = s["logits"].double().tolist()
    for t in range(c["T"]):
        order = sorted(range(c["E"]), key=lambda i: (-l[t][i], i))[:c["k"]]
        order = [i for i in order if l[t][i] > -math.inf]
        total = sum(math.exp(l[t][i] - l[t][order[0]]) for i in order)
        for i in order:
            z = torch.einsum("d,df->f", s["x"][t].double(), s["w1"][i].double())
            if s["b1"] is not None:
                z += s["b1"][i].double()
            y = torch.einsum("f,fd->d", _exact_act(z, c["act"]), s["w2"][i].double())
            if s["b2"] is not None:
                y += s["b2"][i].double()
            out[t] += math.exp(l[t][i] - l[t][order[0]]) / total * y
    return {"out": out}


def _exact_logprobs(c, s):
    names = ["logprobs"] + ["entropy"] * c["entropy"] + ["top_logprobs", "top_tokens"] * (c["top"] > 0)
    got = {n: [] for n in names + ["dlogits"] * (c["way"] == "train")}
    for r0 in range(0, c["rows"], 256):  # (a batch in 64 bits at a time)
        sl = slice(r0, min(r0 + 256, c["rows"]))
        z = s["logits"][sl].double() / c["temperature"]
        tok = s["tokens"][sl].tolist()
        logp = z - torch.logsumexp(z, 1, keepdim=True)
        p = torch.exp(logp)
        h = torch.special.entr(p).sum(1)
        got["logprobs"].append(torch.stack([logp[i, t] if t >= 0 else torch.zeros_like(h[0])
                                            for i, t in enumerate(tok)]))
        if c["entropy"]:
            got["entropy"].append(h)
        if c["top"]:
            got["top_logprobs"].append(torch.topk(logp, c["top"], dim=1).values)
        if c["way"] == "train":
            d = torch.zeros_like(p)
            for i, t in enumerate(tok):
                if t >= 0:
                    d[i] = -s["dlogprobs"][r0 + i].double() * p[i]
                    d[i, t] += s["dlogprobs"][r0 + i].double()
            if c["entropy"]:  # dH/dz_j = entr(p_j) - p_j H
                d += s["dentropy"][sl].double()[:, None] * (torch.special.entr(p) - p * h[:, None])
            got["dlogits"].append(d / c["temperature"])
    if c["way"] == "train" and c["rows"] * c["V"] > 1 << 28:
        got["dlogits"] = []  # (too large to be kept in 64 bits)
    return {n: torch.cat(v) if v else None for n, v in got.items()}


def exact(case, seed):
    s = prepare(case, seed)
    return {"adapted": _exact_adapted, "layer": _exact_layer, "logprobs": _exact_logprobs}[case["op"]](case, s)
