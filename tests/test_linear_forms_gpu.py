"""Linear layers in the forms that sizes or options select: sums cut into chunks for each of the three
products, groups in both types with residuals and fp32 gradients, gated groups cut along K.

Against the formulas in 64 bits.  Tolerances, elementwise, with u the unit roundoff of a
result's type and S the sum of the magnitudes that a product adds:
  * the tensor core truncates its accumulator once every 16 of the reduced dimension, 2^-23 of the
    partial sum at most (which S bounds); accumulators restart every L (1024 where sums are cut
    into chunks, else the whole length or a slice's), and their sums are added in fp32:
        acc(n, L) = (min(n, L) / 16 2^-23 + (n / L + 4) 2^-24) S;
  * the activation, its derivative, dZ's rounding and the result's as in test_linear_gpu.py.
Integers whose sums stay below 2^24 are exact in fp32 results.
"""
import pytest
import torch

from test_linear_gpu import UNIT, act64, assert_within, grads64, offsets_of

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def g():
    import programming_tiled_gemm_gb300 as g
    return g


@pytest.fixture()
def lib(g):
    lib = g.Gemm(0)
    yield lib
    assert lib.device_status() == g.GEMM_OK
    lib.close()


def randn(seed, *shape, dtype=torch.float32, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def ints(seed, *shape, dtype, top=4):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=gen, device="cuda").to(dtype)


def acc(n, S, L=None):
    L = L or max(n, 1)
    return (min(n, L) / 16 * 2.0 ** -23 + (n / L + 4) * 2.0 ** -24) * S


def rounded(got, ref, tol):
    assert_within(got, ref, tol + UNIT[got.dtype] * (ref.abs() + tol) + 2.0 ** -25)


def check_forward(y, z_out, x, w, b, act, r, L=None):
    z = x.double() @ w.double()
    S = x.double().abs() @ w.double().abs()
    if b is not None:
        z, S = z + b.double(), S + b.double().abs()
    zt = acc(x.shape[1], S, L)
    if z_out is not None:
        rounded(z_out, z, zt)
    ref = act64(z, act)
    if act == "swiglu":
        a, u = z.chunk(2, dim=1)
        at, ut = zt.chunk(2, dim=1)
        tol = 1.13 * at * (u.abs() + ut) + ut * a.abs() + 2.0 ** -19 * (1 + a.abs()) * u.abs()
    else:
        tol = 1.13 * zt + (0 if act in ("none", "relu") else 2.0 ** -19 * (1 + z.abs()))
    if r is not None:
        ref = ref + r.double()
        tol = tol + 2.0 ** -23 * ref.abs()
    rounded(y, ref, tol)


def check_grads(dx, dw, dy, x, w, z, act, L=None):
    dz, rx, rw, _ = grads64(dy, x, w, z, act)
    u, scale = UNIT[x.dtype], dy.double().abs()
    if act == "swiglu":
        a, b = z.double().chunk(2, dim=1)
        own = 2.0 ** -18 * torch.cat([scale * b.abs() * (1 + a.abs()), scale * a.abs()], 1)
    elif act in ("none", "relu"):
        own = torch.zeros_like(dz)
    else:
        own = 2.0 ** -18 * scale * (1 + z.double().abs()) ** 2
    zt = own + (0 if act == "none" else u * (dz.abs() + own) + 2.0 ** -25)
    aw, ax = w.double().abs(), x.double().abs()
    if dx is not None:
        rounded(dx, rx, zt @ aw.t() + acc(w.shape[1], (dz.abs() + zt) @ aw.t(), L))
    if dw is not None:
        rounded(dw, rw, ax.t() @ zt + acc(x.shape[0], ax.t() @ (dz.abs() + zt), L))


# ------------------------------------------------------------------------------------------------ chunks

@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("chunk", [1, 3, 16, 4096])
def test_chunk_option(g, lib, chunk, dt):
    """GEMM_OPT_TC_CHUNK: every product's 16-bit results from chunks of that many k-blocks, an odd number
    being the next even one's."""
    dtype = DTYPES[dt]
    x, w, dy = randn(1, 300, 1100, dtype=dtype)[:, :1096], randn(2, 1096, 520, dtype=dtype, scale=0.03), randn(3, 300, 520, dtype=dtype)
    x = x.contiguous()
    z = randn(4, 300, 520, dtype=dtype)
    lib.set_option(g.GEMM_OPT_TC_CHUNK, chunk)
    y = lib.linear(x, w, act="relu")
    y32 = lib.linear(x, w, out_dtype=torch.float32)
    dx, dw, _ = lib.linear_backward(dy, x, w, z=z, act="silu")
    L = (chunk + 1) // 2 * 2 * 64
    check_forward(y, None, x, w, None, "relu", None, L)
    check_forward(y32, None, x, w, None, "none", None, L)
    check_grads(dx, dw, dy, x, w, z, "silu", L)
    if chunk % 2:
        lib.set_option(g.GEMM_OPT_TC_CHUNK, chunk + 1)
        assert torch.equal(lib.linear(x, w, out_dtype=torch.float32), y32)
        for a, b in zip(lib.linear_backward(dy, x, w, z=z, act="silu"), (dx, dw)):
            assert torch.equal(a, b)
    lib.set_option(g.GEMM_OPT_TC_CHUNK, 0)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N,act", [(40, 264, 16648, "none"), (300, 136, 8328, "swiglu"), (9, 2048, 20000, "gelu")])
def test_dx_over_many_columns(lib, M, K, N, act, dt):
    """dX reduces over W's columns: beyond 16384 of them in chunks."""
    dtype = DTYPES[dt]
    Nw = 2 * N if act == "swiglu" else N
    x, w = randn(1, M, K, dtype=dtype), randn(2, K, Nw, dtype=dtype, scale=K ** -0.5)
    dy, z = randn(3, M, N, dtype=dtype), randn(4, M, Nw, dtype=dtype)
    dx, dw, db = lib.linear_backward(dy, x, w, z=z, act=act, bias=True)
    check_grads(dx, dw, dy, x, w, z, act)
    only, _, _ = lib.linear_backward(dy, x, w, z=z, act=act, need_dw=False)
    assert torch.equal(only, dx)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N", [(16392, 136, 264), (20001, 72, 8), (32768, 264, 136)])
def test_dw_over_many_rows(lib, M, K, N, dt):
    """dW reduces over the rows: beyond 16384 of them in chunks, results of 16 and of 32 bits."""
    dtype = DTYPES[dt]
    x, w, dy = randn(1, M, K, dtype=dtype), randn(2, K, N, dtype=dtype), randn(3, M, N, dtype=dtype, scale=0.1)
    for dw_dtype in (dtype, torch.float32):
        _, dw, _ = lib.linear_backward(dy, x, w, need_dx=False, dw_dtype=dw_dtype)
        check_grads(None, dw, dy, x, w, dy, "none")


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("way", ["forward", "dx", "dw"])
def test_chunked_sums_are_exact_on_integers(g, lib, way, dt):
    dtype = DTYPES[dt]
    n = 17000  # of the reduced dimension
    a, b = ints(1, 72, n, dtype=dtype), ints(2, n, 136, dtype=dtype)
    want = a.double() @ b.double()
    if way == "forward":
        got = lib.linear(a, b, out_dtype=torch.float32)
    elif way == "dw":
        _, got, _ = lib.linear_backward(b, a.t().contiguous(), b[:72].contiguous(), need_dx=False, dw_dtype=torch.float32)
    else:  # (a 16-bit result: small sums, each exact)
        a, b = a * (torch.arange(n, device="cuda") % 97 == 0), b
        want = a.double() @ b.double()
        want = want.to(dtype).double()
        w = b.t().contiguous()
        got, _, _ = lib.linear_backward(a.contiguous(), torch.zeros(72, 136, device="cuda", dtype=dtype), w, need_dw=False)
    assert torch.equal(got.double(), want)


# ------------------------------------------------------------------------------------------------ groups

COUNTS = [130, 0, 1, 64, 700, 63, 257, 0]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
def test_grouped_residual(lib, act, out, dt):
    """act(x w[g] + b[g]) + r over groups, in both types of operands and of results."""
    dtype = DTYPES[dt]
    M, K, N, G = sum(COUNTS), 136, 264, len(COUNTS)
    Nw = 2 * N if act == "swiglu" else N
    x, w = randn(1, M, K, dtype=dtype), randn(2, G, K, Nw, dtype=dtype, scale=K ** -0.5)
    b, r = randn(3, G, Nw, dtype=dtype), randn(4, M + 3, N, dtype=dtype if out == "same" else torch.float32)
    want_tail = r[M:].clone()
    x = torch.cat([x, x.new_full((3, K), float("nan"))])  # rows of no group
    y = r.clone()
    got, z = lib.grouped_linear(x, w, offsets_of(COUNTS), bias=b, act=act, residual=y, out=y, save_preact=True)
    at = 0
    for e, n in enumerate(COUNTS):
        sl = slice(at, at + n)
        at += n
        if n:
            check_forward(got[sl], z[sl], x[sl], w[e], b[e], act, r[sl])
    assert torch.equal(got[M:], want_tail)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dw_dtype", ["same", "f32"])
@pytest.mark.parametrize("act", ["none", "silu", "swiglu"])
def test_grouped_gradients_in_both_types(lib, act, dw_dtype, dt):
    dtype = DTYPES[dt]
    M, K, N, G = sum(COUNTS), 200, 136, len(COUNTS)
    Nw = 2 * N if act == "swiglu" else N
    x, w = randn(1, M, K, dtype=dtype), randn(2, G, K, Nw, dtype=dtype, scale=K ** -0.5)
    dy, z = randn(3, M, N, dtype=dtype), randn(4, M, Nw, dtype=dtype)
    dx, dw, db = lib.grouped_linear_backward(dy, x, w, offsets_of(COUNTS), z=z, act=act, bias=True,
                                             dw_dtype=dtype if dw_dtype == "same" else torch.float32)
    at = 0
    for e, n in enumerate(COUNTS):
        sl = slice(at, at + n)
        at += n
        if n:
            check_grads(dx[sl], dw[e], dy[sl], x[sl], w[e], z[sl], act)
        else:
            assert (dw[e] == 0).all() and (db[e] == 0).all()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_grouped_fp32_dw_is_exact_on_integers(lib, dt):
    """Chunks of a group's rows and the group's cut last k-block together, next to NaN neighbours."""
    dtype = DTYPES[dt]
    counts = [1500, 7, 0, 2100, 33]
    M, K, N = sum(counts), 136, 264
    x, dy, w = ints(1, M, K, dtype=dtype), ints(2, M, N, dtype=dtype), ints(3, 5, K, N, dtype=dtype)
    x[1500:1507] = float("nan")
    _, dw, _ = lib.grouped_linear_backward(dy, x, w, offsets_of(counts), need_dx=False, dw_dtype=torch.float32)
    at = 0
    for e, n in enumerate(counts):
        if e != 1:
            assert torch.equal(dw[e].double(), x[at:at + n].double().t() @ dy[at:at + n].double()), e
        at += n


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["silu", "swiglu"])
@pytest.mark.parametrize("counts", [[1, 0, 2, 1, 0, 0, 3, 1], [16, 3, 0, 40], [300, 20, 64, 1]])
def test_groups_cut_along_k(lib, counts, act, dt):
    """Few tiles and a long K, as in a decode batch: the last wave's tiles are cut into slices."""
    dtype = DTYPES[dt]
    M, K, N, G = sum(counts), 2048, 264, len(counts)
    Nw = 2 * N if act == "swiglu" else N
    x, w = randn(1, M, K, dtype=dtype), randn(2, G, K, Nw, dtype=dtype, scale=K ** -0.5)
    b, off = randn(3, G, Nw, dtype=dtype), offsets_of(counts)
    for out_dtype in (dtype, torch.float32):
        y, z = lib.grouped_linear(x, w, off, bias=b, act=act, out_dtype=out_dtype, save_preact=True)
        at = 0
        for e, n in enumerate(counts):
            sl = slice(at, at + n)
            at += n
            if n:
                check_forward(y[sl], z[sl], x[sl], w[e], b[e], act, None)
        again = lib.grouped_linear(x, w, off, bias=b, act=act, out_dtype=out_dtype)
        assert torch.equal(again, y)


# ------------------------------------------------------------------------------------------------ long sums

@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("signs", ["same", "halves cancel"])
def test_one_accumulator_over_16384(g, lib, signs, dt):
    """16-bit results of whole tiles keep one accumulator over all of K: off by 2^-23 of the largest
    partial sum at most every 16 of K, however small the sum ends.  Largest partial sum: the sum
    itself, or of a first half that the second takes back.  In chunks of 1024: the same of each
    chunk's own partial sums, and one fp32 addition a chunk."""
    dtype, K = DTYPES[dt], 16384
    gen = torch.Generator(device="cuda").manual_seed(17)
    x = (torch.rand(1024, K, generator=gen, device="cuda") * 0.5 + 0.5).to(dtype)
    w = ((torch.rand(K, 4864, generator=gen, device="cuda") * 0.5 + 0.5) / K).to(dtype)
    if signs != "same":
        w[K // 2:] *= -1
    z = x.double() @ w.double()
    largest = z if signs == "same" else x[:, :K // 2].double() @ w[:K // 2].double()
    rounded(lib.linear(x, w), z, K / 16 * 2.0 ** -23 * largest)
    lib.set_option(g.GEMM_OPT_TC_CHUNK, 16)
    chunk = x[:, :1024].double() @ w[:1024].double() * 2  # (twice the first's: every chunk's, by the factors' range)
    rounded(lib.linear(x, w), z, K / 16 * 2.0 ** -23 * chunk + 16 * 2.0 ** -24 * largest)
    lib.set_option(g.GEMM_OPT_TC_CHUNK, 0)
