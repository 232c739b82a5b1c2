"""Linear layers with a low-rank adapter of each row's choice, against the formula in 64 bits.

Tolerance, element by element, with u = eps / 2 of the type: the accumulators truncate 2^-23 of their partial
sum for each 16 of the reduced dimension, so U = s X A is off by dU = (K / 16 + 16) 2^-23 |s| |X| |A| and its own
rounding u |U| (2^-25 where fp16 is subnormal), and z = X W + U B + bias by that times |B| and (K / 16 + 8 r + 16)
2^-23 (|X| |W| + |U| |B|) (a tile has up to 8 r / 16 blocks of other adapters' zeros and more; zeros lose
nothing).  The activation passes it on by its slope (at most 1.13; swiglu: the product's two terms) and adds
2^-20 (1 + |z|) of itself; the residual and the result's own rounding follow.
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


def make(seed, M, K, N, n, r, dtype, act="none", bias=False, residual=False, order="random"):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dt=dtype):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dt)

    Nw = 2 * N if act == "swiglu" else N
    s = {"x": normal(M, K), "w": normal(K, Nw, scale=K ** -0.5), "a": normal(n, K, r, scale=K ** -0.5),
         "b": normal(n, r, Nw, scale=r ** -0.5), "scales": 0.5 + torch.rand(n, generator=gen, device="cuda")}
    s["bias"] = normal(Nw, scale=0.3) if bias else None
    s["residual"] = normal(M, N) if residual else None
    if order == "random":
        s["adapters"] = torch.randint(-1, n, (M,), generator=gen, device="cuda").to(torch.int32)
    elif order == "requests":  # rows of an adapter together, the last adapter twice
        cuts = torch.randint(0, M + 1, (n,), generator=gen, device="cuda").sort().values
        s["adapters"] = ((torch.arange(M, device="cuda")[:, None] >= cuts[None]).sum(1) - 1).to(torch.int32)
        s["adapters"][: M // 5] = n - 1
    elif order == "none":
        s["adapters"] = torch.full((M,), -1, device="cuda", dtype=torch.int32)
    else:
        s["adapters"] = torch.full((M,), n - 1, device="cuda", dtype=torch.int32)
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


def reference(s, act):
    """(result, tolerance) in 64 bits"""
    x, w, dt = s["x"].double(), s["w"].double(), s["x"].dtype
    (M, K), n, r = x.shape, s["a"].shape[0], s["a"].shape[2]
    u, sub = torch.finfo(dt).eps / 2, 2.0 ** -25 if dt is F16 else 0.0
    z, size = x @ w, x.abs() @ w.abs()
    dz = torch.zeros_like(z)
    for i in range(n):
        rows = torch.nonzero(s["adapters"] == i)[:, 0]
        if rows.numel() == 0:
            continue
        a, b = s["a"][i].double(), s["b"][i].double()
        sc = float(s["scales"][i]) if s["scales"] is not None else 1.0
        uu, du = sc * (x[rows] @ a), abs(sc) * (x[rows].abs() @ a.abs()) * (K / 16 + 16) * 2.0 ** -23
        du = du + u * (uu.abs() + du) + sub
        z[rows] += uu @ b
        size[rows] += (uu.abs() + du) @ b.abs()
        dz[rows] += du @ b.abs()
    if s["bias"] is not None:
        z, size = z + s["bias"].double(), size + s["bias"].double().abs()
    dz = dz + (K / 16 + 8 * r + 16) * 2.0 ** -23 * size
    if act == "swiglu":
        N = z.shape[1] // 2
        gate, up = z[:, :N], z[:, N:]
        si, slope = activation(gate, "silu")
        y = si * up
        dy = dz[:, :N] * slope * (up.abs() + dz[:, N:]) + dz[:, N:] * si.abs() + 2.0 ** -20 * (1 + gate.abs()) * y.abs()
    else:
        y, slope = activation(z, act)
        dy = dz * slope + 2.0 ** -20 * (1 + z.abs()) * (y.abs() + (2.0 ** -20 if act.startswith("gelu") else 0.0))
    if s["residual"] is not None:
        y = y + s["residual"].double()
    dy = dy + y.abs() * 2.0 ** -22
    return y, dy + (y.abs() + dy) * u + sub


def run(lib, s, act, **kw):
    return lib.adapted_linear(s["x"], s["w"], s["a"], s["b"], s["adapters"], scales=s["scales"], bias=s["bias"], act=act,
                              residual=s["residual"], **kw)


def check(got, s, act, rows=slice(None)):
    want, tol = reference(s, act)
    bad = ~((got.double() - want).abs() <= tol)[rows]
    assert not bool(bad.any()), (int(bad.sum()), got[rows][bad][:4], want[rows][bad][:4], tol[rows][bad][:4])


@pytest.mark.parametrize("M,K,N,n,r,act,bias,residual,dtype,order", [
    # the few-row kernel
    (1, 64, 64, 1, 8, "none", False, False, BF16, "one"),
    (1, 2048, 2048, 8, 16, "none", True, False, BF16, "one"),
    (2, 1000, 264, 3, 24, "gelu", True, True, F16, "random"),
    (3, 520, 72, 5, 64, "swiglu", True, True, BF16, "random"),
    (5, 8, 8, 2, 8, "relu", False, False, F16, "random"),
    (8, 4096, 512, 40, 16, "silu", False, True, BF16, "random"),
    (7, 136, 1032, 3, 128, "none", True, False, F16, "one"),
    (4, 256, 256, 3, 16, "none", False, False, BF16, "none"),
    # the tensor-core kernel, a cluster a row
    (9, 64, 64, 4, 8, "none", False, False, BF16, "random"),
    (16, 2048, 2048, 16, 16, "none", False, True, BF16, "random"),
    (33, 4096, 1024, 64, 16, "swiglu", False, False, BF16, "random"),
    (64, 1024, 776, 100, 8, "gelu_tanh", True, True, F16, "random"),
    (77, 1000, 4104, 5, 24, "gelu", True, True, F16, "requests"),
    (100, 72, 40, 7, 40, "silu", True, False, BF16, "random"),
    (130, 512, 512, 300, 16, "none", False, False, BF16, "random"),
    (40, 512, 256, 3, 128, "none", False, False, F16, "random"),
    (50, 512, 256, 3, 72, "swiglu", True, True, BF16, "requests"),
    # the tensor-core kernel, groups of 64 rows
    (300, 4096, 512, 6, 64, "none", False, False, BF16, "requests"),
    (1000, 2000, 1032, 8, 16, "silu", True, True, BF16, "requests"),
    (777, 1032, 776, 20, 48, "gelu", True, False, F16, "random"),
    (2048, 4096, 256, 9, 128, "none", False, True, BF16, "requests"),
    (520, 16384, 128, 2, 32, "none", False, False, BF16, "requests"),
    (4100, 1024, 2048, 8, 64, "swiglu", False, False, BF16, "requests"),
    (700, 1024, 512, 4, 16, "none", False, False, BF16, "none"),
    # more groups than are under way at once, most of them small; none of any adapter but one
    (5000, 512, 64, 600, 16, "none", False, False, BF16, "random"),
    (300, 2048, 128, 8192, 8, "none", False, False, F16, "random"),
    (1500, 1024, 256, 3, 32, "none", False, False, BF16, "one"),
])
def test_adapted(lib, M, K, N, n, r, act, bias, residual, dtype, order):
    s = make(M + K + N, M, K, N, n, r, dtype, act, bias, residual, order)
    got = run(lib, s, act)
    assert got.dtype is dtype
    check(got, s, act)
    assert torch.equal(run(lib, s, act), got)
    if order == "none":
        s["adapters"][::2] = n  # past the last: none either
        assert torch.equal(run(lib, s, act), got)
        plain = lib.linear(s["x"], s["w"], bias=s["bias"], act=act, residual=s["residual"])
        assert torch.equal(got, plain)
    if residual:
        buf = s["residual"].clone()
        keep = dict(s, residual=buf)
        run(lib, keep, act, out=buf)
        assert torch.equal(buf, got)


@pytest.mark.parametrize("M", [3, 20, 400])
def test_padded_rows_and_strided_adapters(lib, M):
    """widths that are no multiple of 8 in rows that are, NaN between them, every second adapter of a larger stack"""
    K, N, n, r = 100, 77, 4, 16
    s = make(M, M, K, N, n, r, BF16, "silu", True, True)

    def pad(t, wide=8):
        shape = list(t.shape)
        big = torch.full(shape[:-1] + [(shape[-1] + 7) // 8 * 8 + wide], math.nan, device="cuda", dtype=t.dtype)
        big[..., :shape[-1]] = t
        return big[..., :shape[-1]]

    def every_second(t):
        big = torch.full([2 * n, t.shape[1] + 3, (t.shape[2] + 15) // 8 * 8], math.nan, device="cuda", dtype=t.dtype)
        v = big[::2, :t.shape[1], :t.shape[2]]
        v.copy_(t)
        return v

    v = dict(s, x=pad(s["x"]), w=pad(s["w"]), a=every_second(s["a"]), b=every_second(s["b"]), residual=pad(s["residual"], 0))
    out = torch.full((M, N + 3), 5.0, device="cuda", dtype=BF16)
    got = run(lib, v, "silu", out=out[:, 1:N + 1])
    check(got, s, "silu")
    assert bool((out[:, 0] == 5).all()) and bool((out[:, N + 1:] == 5).all())


@pytest.mark.parametrize("M,order", [(1, "one"), (6, "random"), (24, "random"), (90, "requests"), (600, "requests"),
                                     (600, "random")])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_nan_stays_with_its_rows(lib, M, order, value):
    """in a row of X; in an adapter's A; in an adapter's B (one entry); in an adapter no row has"""
    K, N, n, r = 256, 200, 6, 16
    s = make(M, M, K, N, n, r, BF16, order=order)
    s["adapters"][s["adapters"] == 4] = 3
    s["a"][4], s["b"][4] = value, value
    clean = run(lib, s, "none")
    check(clean, s, "none")
    assert not bool(clean.isnan().any())
    x = dict(s, x=s["x"].clone())
    x["x"][M // 2, 7] = value
    got = run(lib, x, "none")
    others = torch.arange(M, device="cuda") != M // 2
    assert not bool(got[M // 2].isfinite().any()) and torch.equal(got[others], clean[others])
    for name, at in (("a", (5, 3, 2)), ("b", (5, 1, 130))):
        y = dict(s, **{name: s[name].clone()})
        y[name][at] = value
        got = run(lib, y, "none")
        mine = s["adapters"] == 5
        assert torch.equal(got[~mine], clean[~mine]), name
        if bool(mine.any()):
            assert not bool((got if name == "a" else got[:, 130])[mine].isfinite().any()), name


def test_indices_that_start_anywhere(lib):
    """rows' indices off every 16-byte boundary: the same results"""
    s = make(8, 1001, 1024, 128, 5, 16, BF16, order="requests")
    want = run(lib, s, "none")
    check(want, s, "none")
    for off in (1, 2, 3):
        big = torch.full((1001 + 8,), 77, device="cuda", dtype=torch.int32)
        big[off:off + 1001] = s["adapters"]
        assert torch.equal(run(lib, dict(s, adapters=big[off:off + 1001]), "none"), want)


@pytest.mark.parametrize("scales", [True, False])
def test_scales(lib, scales):
    s = make(3, 20, 512, 128, 4, 16, BF16)
    if not scales:
        s["scales"] = None
    else:
        s["scales"] = torch.tensor([0.0, -2.0, 16.0, 1.0], device="cuda")
    check(run(lib, s, "none"), s, "none")
    s["x"], s["adapters"] = s["x"][:4], s["adapters"][:4].contiguous()
    check(run(lib, s, "none"), s, "none")


def test_no_adapters_at_all(lib):
    s = make(3, 20, 512, 128, 1, 16, BF16, "silu", True, True)
    want = lib.linear(s["x"], s["w"], bias=s["bias"], act="silu", residual=s["residual"])
    got = lib.adapted_linear(s["x"], s["w"], s["a"][:0], s["b"][:0], s["adapters"], bias=s["bias"], act="silu",
                             residual=s["residual"])
    assert torch.equal(got, want)
    empty = lib.adapted_linear(s["x"][:0], s["w"], s["a"], s["b"], s["adapters"][:0])
    assert empty.shape == (0, 128)


def test_a_row_of_integers_is_exact(lib):
    """small whole numbers: every product and sum is exact, whatever order or block they lie in"""
    gen = torch.Generator(device="cuda").manual_seed(1)

    def ints(*shape, m=2):
        return torch.randint(-m, m + 1, shape, generator=gen, device="cuda").to(BF16)

    for M, n, r in ((3, 5, 8), (64, 64, 16), (256, 200, 16), (200, 3, 128), (1500, 7, 24)):
        K, N = 96, 264
        # (|U| <= 96 * 4 fits bf16's 8 bits up to 256: one nonzero column of A in eight)
        x, w, a, b = ints(M, K, m=1), ints(K, N, m=1), ints(n, K, r, m=1), ints(n, r, N, m=1)
        a[:, 32:] = 0
        adapters = torch.randint(-1, n, (M,), generator=gen, device="cuda").to(torch.int32)
        got = lib.adapted_linear(x, w, a, b, adapters)
        want = x.double() @ w.double()
        for i in range(n):
            rows = torch.nonzero(adapters == i)[:, 0]
            want[rows] += (x[rows].double() @ a[i].double()) @ b[i].double()
        assert torch.equal(got, want.float().to(BF16)), (M, n, r)


def test_streams_graphs_and_other_calls_between(g):
    lib = g.Gemm(0)
    cases = [make(1, 2, 512, 256, 4, 16, BF16), make(2, 40, 1024, 512, 16, 16, BF16), make(3, 600, 1024, 512, 5, 64, BF16,
                                                                                      order="requests")]
    want, graphs, kept = [], [], []
    big = make(4, 3000, 2048, 1024, 50, 128, BF16)
    with pytest.raises(g.GemmError):  # (no workspace yet)
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            run(lib, cases[2], "none")
    for s in cases:
        want.append(run(lib, s, "none").clone())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kept.append(run(lib, s, "none"))
        graphs.append(graph)
    run(lib, big, "none")  # outgrows what the graphs hold
    lib.linear(big["x"], big["w"])
    filler = [torch.full((1 << 20,), 7, device="cuda", dtype=torch.int32) for _ in range(32)]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        others = [run(lib, s, "none") for s in cases]
    st.synchronize()
    for _ in range(3):
        for k in kept:
            k.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(want, kept, others):
            assert torch.equal(a, b) and torch.equal(a, c)
    del filler
    assert lib.device_status() == g.GEMM_OK
    lib.close()


def test_back_to_back_layers(lib):
    """each call's input is the last one's output: the product starts before its adapters' part is there"""
    for M in (1, 4, 24, 200):
        K = 512
        s = make(M, M, K, K, 6, 16, BF16)
        xs = [s["x"]]
        for _ in range(12):
            xs.append(run(lib, dict(s, x=xs[-1]), "none"))
            xs[-1] = (xs[-1].float() * 0.5).to(BF16)
        y = s["x"]
        for i in range(12):
            y = (run(lib, dict(s, x=y), "none").float() * 0.5).to(BF16)
            torch.cuda.synchronize()
            assert torch.equal(y, xs[i + 1])
        chain = [s["x"]]
        for _ in range(12):
            chain.append(run(lib, dict(s, x=chain[-1]), "relu"))
        torch.cuda.synchronize()
        for i in range(12):
            check(chain[i + 1], dict(s, x=chain[i]), "relu")


def test_a_wait_that_runs_out_is_reported(g):
    lib = g.Gemm(0)
    s = make(2, 40, 1024, 512, 16, 16, BF16)
    want = run(lib, s, "none")
    lib.set_option(g.GEMM_OPT_WAIT_LIMIT_US, 20000)
    lib.set_option(g.GEMM_OPT_TEST_STALL, 1)
    out = torch.full_like(want, 3.0)
    run(lib, s, "none", out=out)
    assert lib.device_status() == g.GEMM_ERR_DEVICE_TIMEOUT
    assert bool((out == 3).all())
    lib.set_option(g.GEMM_OPT_TEST_STALL, 0)
    assert torch.equal(run(lib, s, "none"), want)
    assert lib.device_status() == g.GEMM_OK
    lib.close()


def test_wait_limit_is_none_of_the_first_kernels_time(g):
    """the product's waits may begin while the kernel that makes U is busy for longer than their limit"""
    lib = g.Gemm(0)
    s = make(5, 65536, 2048, 256, 6, 128, BF16, order="requests")
    want = run(lib, s, "none")
    lib.set_option(g.GEMM_OPT_WAIT_LIMIT_US, 60)
    for _ in range(3):
        assert torch.equal(run(lib, s, "none"), want)
    assert lib.device_status() == g.GEMM_OK
    lib.close()


def test_refusals(lib, g):
    s = make(1, 12, 64, 64, 3, 16, BF16)
    x, w, a, b, ad = s["x"], s["w"], s["a"], s["b"], s["adapters"]
    for bad in (dict(a=a[:, :56]), dict(b=b[:, :8]), dict(b=b[:, :, :56]), dict(ad=ad[:5]), dict(ad=ad.long()),
                dict(w=w[:56]), dict(b=b[:2]), dict(ad=ad.cpu()), dict(a=a.transpose(1, 2))):
        v = dict(x=x, w=w, a=a, b=b, ad=ad)
        v.update(bad)
        with pytest.raises(ValueError):
            lib.adapted_linear(v["x"], v["w"], v["a"], v["b"], v["ad"])
    with pytest.raises(ValueError):
        lib.adapted_linear(x, w, a, b, ad, scales=torch.ones(2, device="cuda"))
    with pytest.raises(TypeError):
        lib.adapted_linear(x, w, a.half(), b, ad)
    with pytest.raises(TypeError):
        lib.adapted_linear(x, w, a, b, ad, out=torch.empty(12, 64, device="cuda"))
    with pytest.raises(g.GemmError):  # a rank that is no multiple of 8
        lib.adapted_linear(x, w, a[:, :, :12].contiguous(), b[:, :12].contiguous(), ad)
    with pytest.raises(g.GemmError):  # no tensor cores
        lib.adapted_linear(x.float(), w.float(), a.float(), b.float(), ad)
    n = lib.launch_count()
    la = g.LinearArgs(M=12, K=64, N=64, X=x.data_ptr(), ldx=64, W=w.data_ptr(), ldw=64, Y=x.data_ptr(), ldy=64,
                      dtype=g.GEMM_BF16, y_dtype=g.GEMM_BF16)
    aa = g.AdapterArgs(n=3, r=16, A=a.data_ptr(), lda=16, a_stride=64 * 16, B=b.data_ptr(), ldb=64, b_stride=16 * 64,
                       adapters=ad.data_ptr())

    def call(lin=(), **kw):
        l, d = g.LinearArgs.from_buffer_copy(la), g.AdapterArgs.from_buffer_copy(aa)
        for name, v in dict(lin).items():
            setattr(l, name, v)
        for name, v in kw.items():
            setattr(d, name, v)
        return g.gemm_linear_adapted(lib.handle, l, d)

    for kw in (dict(n=-1), dict(r=0), dict(A=None), dict(B=None), dict(adapters=None), dict(lda=8), dict(ldb=56),
               dict(a_stride=64), dict(b_stride=64), dict(lin=dict(groups=1, offsets=ad.data_ptr())),
               dict(lin=dict(Z=x.data_ptr(), ldz=64))):
        assert call(**kw) == g.GEMM_ERR_INVALID_ARG, kw
    for kw in (dict(lin=dict(y_dtype=g.GEMM_F32)), dict(lin=dict(K=16392, ldx=16392), a_stride=1 << 30), dict(n=8193),
               dict(r=136, lda=136, a_stride=1 << 20, b_stride=1 << 20)):
        assert call(**kw) == g.GEMM_ERR_UNSUPPORTED, kw
    for kw in (dict(A=a.data_ptr() + 8), dict(B=b.data_ptr() + 2), dict(lda=20, a_stride=2048), dict(ldb=68, b_stride=2048),
               dict(a_stride=64 * 16 + 4), dict(adapters=ad.data_ptr() + 2), dict(scales=ad.data_ptr() + 2), dict(r=12)):
        assert call(**kw) == g.GEMM_ERR_ALIGNMENT, kw
    assert g.library().gemm_linear_adapted(lib.handle, la, None, None) == g.GEMM_ERR_INVALID_ARG
    assert lib.launch_count() == n


def test_rows_near_the_end_of_32_bits_are_refused(lib, g):
    """The kernels look some rows past the last, in 32 bits: 2^31 - 1025 rows pass gemm_linear's own limit."""
    s = make(1, 12, 64, 64, 3, 16, BF16)
    la = g.LinearArgs(M=12, K=64, N=64, X=s["x"].data_ptr(), ldx=64, W=s["w"].data_ptr(), ldw=64, Y=s["x"].data_ptr(),
                      ldy=64, dtype=g.GEMM_BF16, y_dtype=g.GEMM_BF16)
    aa = g.AdapterArgs(n=3, r=16, A=s["a"].data_ptr(), lda=16, a_stride=64 * 16, B=s["b"].data_ptr(), ldb=64,
                       b_stride=16 * 64, adapters=s["adapters"].data_ptr())
    n = lib.launch_count()
    for rows in (2 ** 31 - 1025, 2 ** 31 - 2 ** 16):
        la.M = rows
        assert g.gemm_linear_adapted(lib.handle, la, aa) == g.GEMM_ERR_UNSUPPORTED
    assert lib.launch_count() == n
