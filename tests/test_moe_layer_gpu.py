"""A whole mixture-of-experts layer for a few tokens, against the formula in 64 bits.

Tolerance, element by element, with u = eps / 2 of the 16-bit type: z = x W1 + b1 is off by the tensor
core's truncation, 2^-23 of the partial sums for each 16 of D, and a few fp32 roundings: dz = (D / 16 + 8) 2^-23
(|x| |W1| + |b1|).  The activation passes that on by its slope (at most 1.13; swiglu: the product's two
terms) and adds 2^-20 (1 + |z|) of itself (exp and its argument); H is rounded once: u |H|, and 2^-25 where fp16 is
subnormal.  The second product is off by the same rule over F and by H's error times |W2|; the weights by
2^-20, the sum over j by fp32 roundings, and the result by its own rounding.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def g():
    import programming_tiled_gemm_gb300 as g
    return g


@pytest.fixture(scope="module")
def lib(g):
    lib = g.Gemm(0)
    yield lib
    assert lib.device_status() == g.GEMM_OK
    lib.close()


def make(seed, T, E, D, F, dtype, act="swiglu", bias=False, residual=False, logits_dtype=F32):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dt=dtype):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dt)

    Fw = 2 * F if act == "swiglu" else F
    s = {"x": normal(T, D), "logits": normal(T, E, scale=1.5, dt=logits_dtype), "w1": normal(E, D, Fw, scale=D ** -0.5),
         "w2": normal(E, F, D, scale=F ** -0.5)}
    s["b1"] = normal(E, Fw, scale=0.3) if bias else None
    s["b2"] = normal(E, D, scale=0.3) if bias else None
    s["residual"] = normal(T, D) if residual else None
    return s


def activation(z, act):
    """(act(z), the bound of its slope)"""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), torch.ones_like(z)
    if act == "silu":
        return z * torch.sigmoid(z), torch.full_like(z, 1.13)
    if act == "gelu":
        return z * 0.5 * torch.special.erfc(-z * 2 ** -0.5), torch.full_like(z, 1.13)
    return z * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)), torch.full_like(z, 1.13)


def picks_of(logits, k, renormalize):
    out = []
    for row in logits.double().tolist():
        order = sorted((e for e in range(len(row)) if row[e] != -math.inf), key=lambda e: (-row[e], e))
        pick = order[:k]
        over = pick if renormalize else order
        total = sum(math.exp(row[e] - row[pick[0]]) for e in over) if pick else 1.0
        out.append([(e, math.exp(row[e] - row[pick[0]]) / total) for e in pick])
    return out


def reference(s, k, act, renormalize=True, out_dtype=None):
    """(result, tolerance) in 64 bits"""
    x, dt = s["x"].double(), s["x"].dtype
    T, D = x.shape
    F = s["w2"].shape[1]
    u, sub = torch.finfo(dt).eps / 2, 2.0 ** -25 if dt is F16 else 0.0
    want, tol = torch.zeros_like(x), torch.zeros_like(x)
    experts = {}
    for t, pick in enumerate(picks_of(s["logits"], k, renormalize)):
        for e, w in pick:
            experts.setdefault(e, []).append((t, w))
    for e, rows in experts.items():
        t = torch.tensor([r[0] for r in rows], device=x.device)
        w = torch.tensor([r[1] for r in rows], device=x.device, dtype=torch.float64)[:, None]
        w1, w2 = s["w1"][e].double(), s["w2"][e].double()
        z, dz = x[t] @ w1, x[t].abs() @ w1.abs()
        if s["b1"] is not None:
            z, dz = z + s["b1"][e].double(), dz + s["b1"][e].double().abs()
        dz = dz * (D / 16 + 8) * 2.0 ** -23
        if act == "swiglu":
            a, up = z[:, :F], z[:, F:]
            si, slope = activation(a, "silu")
            h = si * up
            dh = dz[:, :F] * slope * (up.abs() + dz[:, F:]) + dz[:, F:] * si.abs() + 2.0 ** -20 * (1 + a.abs()) * h.abs()
        else:
            h, slope = activation(z, act)
            dh = dz * slope + 2.0 ** -20 * (1 + z.abs()) * (h.abs() + (2.0 ** -20 if act.startswith("gelu") else 0.0))
        dh = dh + u * (h.abs() + dh) + sub
        y = h @ w2
        dy = dh @ w2.abs() + (F / 16 + 8) * 2.0 ** -23 * ((h.abs() + dh) @ w2.abs())
        if s["b2"] is not None:
            y = y + s["b2"][e].double()
        dy = dy + y.abs() * 2.0 ** -19
        want.index_add_(0, t, w * y)
        tol.index_add_(0, t, w * dy)
    if s["residual"] is not None:
        want = want + s["residual"].double()
    tol = tol + want.abs() * 2.0 ** -22
    if (out_dtype or dt) is not F32:
        tol = tol + (want.abs() + tol) * u + sub
    return want, tol


def check(got, s, k, act, **kw):
    want, tol = reference(s, k, act, out_dtype=got.dtype, **kw)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), got[bad][:4], want[bad][:4], tol[bad][:4])


@pytest.mark.parametrize("T,E,k,D,F,act,bias,residual,dtype", [
    (1, 1, 1, 8, 8, "swiglu", False, False, BF16),
    (1, 4, 2, 64, 32, "swiglu", True, True, BF16),
    (1, 64, 4, 520, 264, "swiglu", False, True, BF16),
    (2, 8, 8, 136, 72, "silu", True, False, F16),
    (7, 5, 3, 200, 104, "gelu", True, True, F16),
    (8, 16, 2, 1032, 776, "swiglu", True, False, BF16),
    (9, 33, 5, 72, 1000, "relu", False, False, BF16),
    (16, 64, 4, 512, 256, "swiglu", False, True, BF16),
    (17, 3, 1, 264, 40, "none", False, True, F16),
    (33, 100, 7, 128, 128, "gelu_tanh", True, False, BF16),
    (48, 16, 2, 1032, 776, "gelu", True, False, F16),
    (63, 300, 3, 96, 48, "swiglu", False, False, BF16),
    (64, 2, 2, 320, 192, "swiglu", True, True, BF16),
    (64, 1024, 32, 64, 64, "swiglu", False, False, F16),
    (64, 8, 1, 2048, 1024, "swiglu", False, True, BF16),
])
def test_layer(lib, T, E, k, D, F, act, bias, residual, dtype):
    s = make(T * E + D, T, E, D, F, dtype, act, bias, residual)
    got = lib.moe_layer(s["x"], s["logits"], s["w1"], s["w2"], k, act=act, b1=s["b1"], b2=s["b2"], residual=s["residual"])
    assert got.dtype is dtype
    check(got, s, k, act)
    again = lib.moe_layer(s["x"], s["logits"], s["w1"], s["w2"], k, act=act, b1=s["b1"], b2=s["b2"], residual=s["residual"])
    assert torch.equal(got, again)
    if residual:  # the residual's own buffer
        r = s["residual"].clone()
        lib.moe_layer(s["x"], s["logits"], s["w1"], s["w2"], k, act=act, b1=s["b1"], b2=s["b2"], residual=r, out=r)
        assert torch.equal(r, got)


@pytest.mark.parametrize("N,D,F", [(1, 12, 7), (3, 13, 9), (20, 100, 33)])
def test_odd_columns_in_padded_rows(lib, N, D, F):
    """widths that are no multiple of 8, in rows that are; NaN between the rows"""
    dt, E, k = BF16, 6, 2
    s = make(N, N, E, D, F, dt, "silu", True, True)

    def pad(t):
        shape = list(t.shape)
        wide = torch.full(shape[:-1] + [(shape[-1] + 15) // 8 * 8], math.nan, device="cuda", dtype=t.dtype)
        wide[..., :shape[-1]] = t
        return wide[..., :shape[-1]]

    out = torch.full((N, D + 3), 5.0, device="cuda", dtype=dt)
    got = lib.moe_layer(pad(s["x"]), pad(s["logits"]), pad(s["w1"]), pad(s["w2"]), k, act="silu", b1=s["b1"], b2=s["b2"],
                        residual=pad(s["residual"]), out=out[:, 1:D + 1])
    check(got, s, k, "silu")
    assert bool((out[:, 0] == 5).all()) and bool((out[:, D + 1:] == 5).all())


@pytest.mark.parametrize("logits_dtype", [F32, BF16, F16])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_routing_as_moe_route(lib, logits_dtype, renormalize, out_dtype):
    """ties, experts that are not there, tokens without any: the picks of moe_route, and the five calls' result"""
    T, E, k, D, F = 40, 24, 4, 128, 64
    s = make(3, T, E, D, F, BF16, "swiglu", False, False, logits_dtype)
    l = (s["logits"].float() * 2).round() / 2  # many equal ones
    l[::3, ::2] = -math.inf
    l[5] = -math.inf
    l[6, 1:] = -math.inf
    l[7, 2:] = -math.inf
    l[8] = torch.finfo(logits_dtype).min
    l[9, 1::2] = torch.finfo(logits_dtype).min
    s["logits"] = l.to(logits_dtype)
    got = lib.moe_layer(s["x"], s["logits"], s["w1"], s["w2"], k, renormalize=renormalize, out_dtype=out_dtype)
    assert got.dtype is out_dtype
    check(got, s, k, "swiglu", renormalize=renormalize)
    assert bool((got[5] == 0).all())
    r = lib.moe_route(s["logits"], k, renormalize=renormalize)
    y = lib.grouped_linear(lib.moe_dispatch(s["x"], r.rows, k), s["w1"], r.offsets, act="swiglu")
    five = lib.moe_combine(lib.grouped_linear(y, s["w2"], r.offsets, out_dtype=F32), r.slots, r.weights)
    _, tol = reference(s, k, "swiglu", renormalize=renormalize)
    assert bool(((five.double() - got.double()).abs() <= 2 * tol).all())


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(3, 50, 6), (10, 64, 32), (11, 9, 9), (41, 64, 20), (64, 40, 11), (12, 65, 5),
                                   (50, 256, 12), (30, 257, 9)])
def test_routing_whatever_lanes_a_token_has(lib, T, E, k, renormalize):
    """both sides of the limits at which a token has 8 or 32 lanes, keys in registers or not: ties, experts that
    are not there, more picks than experts that are, tokens without any"""
    s = make(T + E, T, E, 64, 32, BF16, "swiglu")
    l = (s["logits"].float() * 2).round() / 2
    l[::2, 1::3] = -math.inf
    l[1::4, 3:] = -math.inf
    l[2] = -math.inf
    s["logits"] = l
    got = lib.moe_layer(s["x"], l, s["w1"], s["w2"], k, renormalize=renormalize, out_dtype=F32)
    check(got, s, k, "swiglu", renormalize=renormalize)
    assert bool((got[2] == 0).all())
    l[0, 5], l[-1, 0] = math.nan, math.inf  # a NaN is picked first, and the row is NaN; so is inf's, as inf - inf
    got = lib.moe_layer(s["x"], l, s["w1"], s["w2"], k, renormalize=renormalize, out_dtype=F32)
    assert bool(got[0].isnan().all()) and bool(got[-1].isnan().all()) and not bool(got[1:-1].isnan().any())


def test_no_token_goes_anywhere(lib, g):
    s = make(1, 5, 8, 64, 32, BF16, residual=True)
    s["logits"][:] = -math.inf
    got = lib.moe_layer(s["x"], s["logits"], s["w1"], s["w2"], 2, residual=s["residual"])
    assert torch.equal(got, s["residual"])
    got = lib.moe_layer(s["x"], s["logits"], s["w1"], s["w2"], 2, out=torch.full_like(s["x"], 7.0))
    assert bool((got == 0).all())
    empty = lib.moe_layer(s["x"][:0], s["logits"][:0], s["w1"], s["w2"], 2)
    assert empty.shape == (0, 64)


def test_nan_stays_with_its_token_and_expert(lib):
    T, E, k, D, F = 12, 6, 2, 96, 64
    s = make(11, T, E, D, F, BF16)
    clean = lib.moe_layer(s["x"], s["logits"], s["w1"], s["w2"], k)
    picks = [[e for e, _ in p] for p in picks_of(s["logits"], k, True)]
    s["x"][3] = math.nan
    s["w1"][4] = math.inf
    got = lib.moe_layer(s["x"], s["logits"], s["w1"], s["w2"], k)
    for t in range(T):
        if t == 3 or 4 in picks[t]:
            assert not bool(got[t].isfinite().all())
        else:
            assert torch.equal(got[t], clean[t])
    # a NaN logit is picked first, and its weights are NaN
    s = make(11, T, E, D, F, BF16)
    s["logits"][2, 1] = math.nan
    got = lib.moe_layer(s["x"], s["logits"], s["w1"], s["w2"], k)
    assert bool(got[2].isnan().all()) and torch.equal(got[3:], clean[3:]) and torch.equal(got[:2], clean[:2])


def test_strided_experts(lib):
    """every second expert of a larger stack, columns of wider matrices, rows of a wider x"""
    T, E, k, D, F = 10, 5, 2, 72, 40
    s = make(2, T, 2 * E, D + 16, F + 8, BF16)
    w1, w2 = s["w1"][::2, 8:D + 8, :2 * F], s["w2"][::2, 8:F + 8, 8:D + 8]
    x = s["x"][:, 8:D + 8]
    v = {"x": x, "logits": s["logits"][:, :E], "w1": w1, "w2": w2, "b1": None, "b2": None, "residual": None}
    check(lib.moe_layer(x, v["logits"], w1, w2, k), v, k, "swiglu")


def test_streams_and_graphs_share_the_workspace(lib, g):
    own = g.Gemm(0)
    small = make(5, 3, 8, 128, 64, BF16, residual=True)
    large = make(6, 64, 8, 512, 384, BF16)

    def call(s, k):
        return own.moe_layer(s["x"], s["logits"], s["w1"], s["w2"], k, residual=s["residual"])

    want_small = call(small, 2).clone()
    with pytest.raises(g.GemmError):  # more workspace than there is: refused whole under capture
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            call(large, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept_small = call(small, 2)
    want_large = call(large, 4).clone()  # outgrows what the first graph holds
    graph2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph2):
        kept_large = call(large, 4)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        other = call(large, 4)
    s.synchronize()
    assert torch.equal(other, want_large)
    for _ in range(3):
        kept_small.zero_(), kept_large.zero_()
        graph.replay()
        graph2.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept_small, want_small) and torch.equal(kept_large, want_large)
    assert own.device_status() == g.GEMM_OK
    own.close()


def test_back_to_back_calls_read_the_last_ones_results(lib):
    """layer after layer without a wait between: the second kernel's early start sees the first's inputs whole"""
    T, E, k, D, F = 4, 16, 2, 256, 128
    s = make(8, T, E, D, F, BF16)
    wr = (torch.randn(D, E, device="cuda") * D ** -0.5).to(BF16)
    x = s["x"]
    xs, ls = [x], []
    for _ in range(20):
        ls.append(lib.linear(xs[-1], wr, out_dtype=F32))
        xs.append(lib.moe_layer(xs[-1], ls[-1], s["w1"], s["w2"], k, residual=xs[-1]))
    torch.cuda.synchronize()
    checked = 0
    for i in range(20):
        # (swiglu squares the magnitude: |x| grows to 1e19, whose square times a weight leaves fp32's range of
        # 3.4e38 and has no result to compare; rows below 1e17 stay within it)
        if float(xs[i].double().abs().nan_to_num(math.inf).max()) > 1e17:
            break
        step = dict(s, x=xs[i], logits=ls[i], residual=xs[i])
        check(xs[i + 1], step, k, "swiglu")
        checked += 1
    assert checked >= 4


def test_wait_limit_is_none_of_the_first_kernels_time(g):
    """the second kernel starts early, and may wait for the first for longer than its waits' limit"""
    lib = g.Gemm(0)
    s = make(7, 8, 16, 4096, 4096, BF16)
    want = lib.moe_layer(s["x"], s["logits"], s["w1"], s["w2"], 8)
    lib.set_option(g.GEMM_OPT_WAIT_LIMIT_US, 40)  # (the first kernel takes some 150)
    for _ in range(3):
        assert torch.equal(lib.moe_layer(s["x"], s["logits"], s["w1"], s["w2"], 8), want)
    assert lib.device_status() == g.GEMM_OK
    lib.close()


def test_refusals(lib, g):
    s = make(1, 4, 8, 64, 32, BF16)
    x, l, w1, w2 = s["x"], s["logits"], s["w1"], s["w2"]
    with pytest.raises(g.GemmError):
        lib.moe_layer(x.repeat(17, 1), l.repeat(17, 1), w1, w2, 2)  # 68 tokens
    for k in (0, 9):
        with pytest.raises(ValueError):
            lib.moe_layer(x, l, w1, w2, k)
    for bad in (dict(w1=w1[:, :, :60]), dict(w2=w2[:, :, :56]), dict(x=x[:, :56]), dict(l=l[:3]), dict(w1=w1[:7]),
                dict(b1=torch.zeros(8, 32, device="cuda", dtype=BF16)), dict(b2=torch.zeros(8, 64, device="cuda")),
                dict(w1=w1.transpose(1, 2)), dict(x=x.cpu())):
        a = dict(x=x, l=l, w1=w1, w2=w2)
        b = {n: bad[n] for n in ("b1", "b2") if n in bad}
        a.update({n: v for n, v in bad.items() if n in a})
        with pytest.raises(ValueError):
            lib.moe_layer(a["x"], a["l"], a["w1"], a["w2"], 2, **b)
    with pytest.raises(TypeError):
        lib.moe_layer(x.half(), l, w1, w2, 2)
    with pytest.raises(KeyError):
        lib.moe_layer(x, l, w1, w2, 2, act="tanh")
    with pytest.raises(g.GemmError):  # no tensor cores for these
        lib.moe_layer(x.float(), l, w1.float(), w2.float(), 2)
    with pytest.raises(g.GemmError):  # rows that start off 16 bytes
        lib.moe_layer(s["x"][:, 4:36], l, w1[:, :32], w2[:, :, :32], 2)
    odd = torch.empty(8, 64, 24, device="cuda", dtype=BF16)  # swiglu's up columns off 16 bytes
    with pytest.raises(g.GemmError):
        lib.moe_layer(x, l, odd, torch.empty(8, 12, 64, device="cuda", dtype=BF16), 2)
    n = lib.launch_count()
    a = g.MoeLayerArgs(T=4, E=8, k=2, D=64, F=32, logits=l.data_ptr(), ldl=8, X=x.data_ptr(), ldx=64, W1=w1.data_ptr(),
                       ldw1=64, w1_stride=64 * 64, W2=w2.data_ptr(), ldw2=64, w2_stride=32 * 64, Y=x.data_ptr(), ldy=64,
                       dtype=g.GEMM_BF16, logits_dtype=g.GEMM_F32, y_dtype=g.GEMM_BF16, act=g.ACTIVATIONS["swiglu"])

    def call(**kw):
        b = g.MoeLayerArgs.from_buffer_copy(a)
        for name, v in kw.items():
            setattr(b, name, v)
        return g.moe_layer(lib.handle, b)

    for kw in (dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(D=-1), dict(F=0), dict(logits=None), dict(ldx=63),
               dict(W1=None), dict(ldw2=32), dict(Y=None), dict(w1_stride=64), dict(w2_stride=8), dict(act=6),
               dict(dtype=9), dict(logits_dtype=4), dict(y_dtype=g.GEMM_F16)):
        assert call(**kw) == g.GEMM_ERR_INVALID_ARG, kw
    for kw in (dict(dtype=g.GEMM_F32), dict(E=1025, ldl=1025), dict(E=64, ldl=64, k=33), dict(F=(1 << 24) + 8, ldw1=1 << 26,
                                                                                              w1_stride=1 << 32,
                                                                                              w2_stride=1 << 32)):
        assert call(**kw) == g.GEMM_ERR_UNSUPPORTED, kw
    for kw in (dict(X=x.data_ptr() + 2), dict(ldx=65), dict(W2=w2.data_ptr() + 8), dict(w1_stride=64 * 64 + 4),
               dict(F=28, ldw1=64), dict(logits=l.data_ptr() + 2), dict(b1=x.data_ptr() + 1), dict(Y=x.data_ptr() + 1)):
        assert call(**kw) == g.GEMM_ERR_ALIGNMENT, kw
    assert lib.launch_count() == n


def test_a_wait_that_runs_out_is_reported(g):
    lib = g.Gemm(0)
    s = make(4, 6, 8, 256, 128, BF16)
    want = lib.moe_layer(s["x"], s["logits"], s["w1"], s["w2"], 2)
    lib.set_option(g.GEMM_OPT_WAIT_LIMIT_US, 20000)
    lib.set_option(g.GEMM_OPT_TEST_STALL, 1)
    out = torch.full_like(want, 3.0)
    lib.moe_layer(s["x"], s["logits"], s["w1"], s["w2"], 2, out=out)
    assert lib.device_status() == g.GEMM_ERR_DEVICE_TIMEOUT
    assert bool((out == 3).all())
    lib.set_option(g.GEMM_OPT_TEST_STALL, 0)
    for _ in range(2):  # (and the counters are zero again)
        assert torch.equal(lib.moe_layer(s["x"], s["logits"], s["w1"], s["w2"], 2), want)
    assert lib.device_status() == g.GEMM_OK
    lib.close()
