"""Linear layers with fused epilogues, dense and grouped, and their gradients, against the
formulas in 64 bits.

Tolerances, elementwise, with u the unit roundoff of the 16-bit type (2^-8 bf16, 2^-11 fp16)
and S = |X||W| + |b| the sum of the magnitudes that a product adds:
  * the sum: the tensor core truncates its fp32 accumulator once every 16 of K, 2^-23 of the
    partial sum at most each time.  Counting 2048 of K in full, with S for every partial sum
    (sums of random signs stay far below it), and one fp32 addition for each 2048 more:
    sum_tol = (min(K, 2048) / 16 + K / 2048 + 4) 2^-23 S;
  * the activation: its slope (at most 1.13; swiglu: the other factor's size) times the
    error of its input, and 2^-19 (1 + |z|) of its own (the fast exponential);
  * one rounding of the result: u |y|;
  * gradients: dZ is rounded once (u |dZ|) before the products, which then add as above.
Integer inputs whose sums stay below 2^24 are exact in fp32 results.
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"]


@pytest.fixture(scope="module")
def g():
    import programming_tiled_gemm_gb300 as g
    return g


@pytest.fixture(scope="module")
def lib(g):
    lib = g.Gemm(0)
    yield lib
    lib.close()


def randn(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def gen_of(*key):
    return torch.Generator(device="cuda").manual_seed(hash(key) % (1 << 31))


def act64(z, act):
    if act == "relu":
        return torch.relu(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "swiglu":
        a, b = z.chunk(2, dim=-1)
        return a * torch.sigmoid(a) * b
    return z


def sum_tol(K, S):
    return (min(K, 2048) / 16 + K / 2048 + 4) * 2.0 ** -23 * S


def check_forward(y, z_out, x, w, b, act, r):
    """y (and the kept z) of one weight matrix against 64 bits."""
    z = x.double() @ w.double()
    S = x.double().abs() @ w.double().abs()
    if b is not None:
        z, S = z + b.double(), S + b.double().abs()
    zt = sum_tol(x.shape[1], S)
    if z_out is not None:
        assert_within(z_out, z, zt + UNIT[z_out.dtype] * (z.abs() + zt) + 2.0 ** -25)
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
    assert_within(y, ref, tol + UNIT[y.dtype] * (ref.abs() + tol) + 2.0 ** -25)


def assert_within(got, ref, tol):
    assert got.shape == ref.shape
    if got.numel() == 0:
        return
    d = (got.double() - ref).abs()
    assert torch.isfinite(got.float()).all()
    worst = (d - tol).max().item()
    assert worst <= 0, "off by %g beyond its tolerance (max |diff| %g)" % (worst, d.max().item())


FORWARD = [
    # M, K, N: one token, few tokens (K split over the pairs), tile edges, several tiles
    (1, 64, 128), (1, 2048, 2048), (2, 8, 8), (15, 520, 72), (16, 1024, 256), (17, 200, 264), (33, 4096, 512),
    (64, 264, 1000), (129, 136, 136), (256, 512, 256), (257, 72, 520), (300, 2560, 776), (1000, 1032, 1000),
]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,K,N", FORWARD)
def test_forward(lib, M, K, N, act, dt):
    gen, dtype = gen_of(M, K, N), DTYPES[dt]
    Nw = 2 * N if act == "swiglu" else N
    x, w = randn(gen, M, K, dtype=dtype), randn(gen, K, Nw, dtype=dtype, scale=K ** -0.5)
    b, r = randn(gen, Nw, dtype=dtype), randn(gen, M, N, dtype=dtype)
    y, z = lib.linear(x, w, bias=b, act=act, residual=r, save_preact=True)
    check_forward(y, z, x, w, b, act, r)
    check_forward(lib.linear(x, w, act=act, out_dtype=torch.float32), None, x, w, None, act, None)
    assert lib.device_status() == 0


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9])
def test_few_rows(lib, M, dt):
    """One to nine rows over sizes on both sides of the kernels' rule: K below and above a warp's
    and a cluster's share, ends inside eight columns, padded rows, fp32 and 16-bit results."""
    dtype = DTYPES[dt]
    for K, N, act in ((1, 1, "none"), (7, 9, "relu"), (31, 65, "silu"), (33, 64, "gelu"), (257, 130, "none"),
                      (300, 8, "swiglu"), (1000, 40, "swiglu"), (2048, 31, "gelu_tanh"), (4099, 77, "none"),
                      (520, 8200, "silu"), (9000, 72, "swiglu"), (5000, 4104, "none")):
        gen = gen_of(M, K, N)
        Nw = 2 * N if act == "swiglu" else N
        pad = lambda n: (n + 7) // 8 * 8
        # what lies between the rows is NaN: it must not count
        x = torch.full((M, pad(K) + 8), float("nan"), dtype=dtype, device="cuda")[:, :K]
        w = torch.full((K, pad(Nw) + 8), float("nan"), dtype=dtype, device="cuda")[:, :Nw]
        x.copy_(randn(gen, M, K))
        w.copy_(randn(gen, K, Nw, scale=K ** -0.5))
        b = randn(gen, Nw, dtype=dtype)
        for out_dtype in (dtype, torch.float32):
            r = randn(gen, M, N + 3, dtype=out_dtype)[:, 1:N + 1]
            out = torch.full((M + 1, N + 2), 7.0, dtype=out_dtype, device="cuda")
            y, z = lib.linear(x, w, bias=b, act=act, residual=r, out=out[:M, :N], save_preact=True)
            check_forward(y, z, x, w, b, act, r)
            assert (out[M] == 7).all() and (out[:, N:] == 7).all()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N", [(1, 512, 256), (77, 1000, 136), (260, 4096, 264), (700, 640, 1032)])
def test_forward_is_exact_on_integers(lib, M, K, N, dt):
    """Products of integers in [-4, 4] add without rounding."""
    gen, dtype = gen_of(M, K, N), DTYPES[dt]
    x, w, b = (torch.randint(-4, 5, s, generator=gen, device="cuda").to(dtype) for s in ((M, K), (K, N), (N,)))
    r = torch.randint(-100, 100, (M, N), generator=gen, device="cuda").float()
    got = lib.linear(x, w, bias=b, act="relu", residual=r)
    ref = torch.relu(x.double() @ w.double() + b.double()) + r.double()
    assert got.dtype == torch.float32 and torch.equal(got.double(), ref)


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_strides_and_alignment(lib, act):
    """Padded rows (the padding NaN, never read or written), a result at an odd address, the
    residual in place."""
    gen = gen_of(1)
    M, K, N = 70, 136, 200
    Nw = 2 * N if act == "swiglu" else N
    X = torch.full((M, K + 24), math.nan, device="cuda", dtype=torch.bfloat16)
    W = torch.full((K, Nw + 8), math.nan, device="cuda", dtype=torch.bfloat16)
    X[:, :K], W[:, :Nw] = randn(gen, M, K), randn(gen, K, Nw, scale=K ** -0.5)
    x, w = X[:, :K], W[:, :Nw]
    for shift, pad in ((0, 0), (0, 5), (1, 3), (3, 8)):
        buf = torch.full((M * (N + pad) + shift,), -7.0, device="cuda", dtype=torch.bfloat16)
        out = buf[shift:].view(M, N + pad)[:, :N]
        r = randn(gen, M, N, dtype=torch.bfloat16)
        out.copy_(r)
        got = lib.linear(x, w, act=act, residual=out, out=out)
        assert got.data_ptr() == out.data_ptr()
        check_forward(out.contiguous(), None, x, w, None, act, r)
        assert (buf[:shift] == -7).all() and (buf[shift:].view(M, N + pad)[:, N:] == -7).all()
    assert lib.device_status() == 0


@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (33, 13, 21), (300, 67, 259)])
def test_odd_sizes_in_padded_rows(lib, M, K, N):
    """K and N that are no multiples of anything: only the rows' starts are aligned."""
    gen = gen_of(M, K, N, 2)

    def padded(rows, cols, scale=1.0):
        t = torch.full((rows, (cols + 7) // 8 * 8), math.nan, device="cuda", dtype=torch.float16)
        t[:, :cols] = randn(gen, rows, cols, scale=scale)
        return t[:, :cols]

    x, w, z, dy = padded(M, K), padded(K, N, K ** -0.5), padded(M, N), padded(M, N)
    b, r = randn(gen, N, dtype=torch.float16), randn(gen, M, N, dtype=torch.float16)
    y, zk = lib.linear(x, w, bias=b, act="silu", residual=r, save_preact=True)
    check_forward(y, zk, x, w, b, "silu", r)
    dx, dw, db = lib.linear_backward(dy, x, w, z=z, act="silu", bias=True)
    check_grads(dx, dw, db, dy, x, w, z, "silu")
    assert lib.device_status() == 0


def test_offsets_past_32_bits(lib):
    """Results and weights of more than 2^31 elements: the last rows and the last group."""
    gen = gen_of(10)
    M, K, N = 270_000, 64, 8192
    x, w = randn(gen, M, K, dtype=torch.bfloat16), randn(gen, K, N, dtype=torch.bfloat16, scale=K ** -0.5)
    y, z = lib.linear(x, w, act="silu", save_preact=True)
    assert y.numel() > 2 ** 31
    check_forward(y[-300:], z[-300:], x[-300:], w, None, "silu", None)
    dx, _, _ = lib.linear_backward(y, x, w, z=z, act="silu", need_dw=False)
    check_grads(dx[-300:], None, None, y[-300:], x[-300:], w, z[-300:], "silu")
    del y, z, dx
    G, K, N = 36, 8192, 8192
    counts = [1] * (G - 1) + [70]
    x, dy = randn(gen, sum(counts), K, dtype=torch.bfloat16), randn(gen, sum(counts), N, dtype=torch.bfloat16)
    w = torch.zeros(G, K, N, device="cuda", dtype=torch.bfloat16)
    w[-1] = randn(gen, K, N, dtype=torch.bfloat16, scale=K ** -0.5)
    assert w.numel() > 2 ** 31
    y = lib.grouped_linear(x, w, offsets_of(counts))
    check_forward(y[-70:], None, x[-70:], w[-1], None, "none", None)
    dx, dw, _ = lib.grouped_linear_backward(dy, x, w, offsets_of(counts))
    check_grads(dx[-70:], dw[-1], None, dy[-70:], x[-70:], w[-1], y[-70:], "none")
    check_grads(dx[:1], dw[0], None, dy[:1], x[:1], w[0], y[:1], "none")
    assert lib.device_status() == 0


def test_long_reductions(lib):
    """Beyond 16384 of K the sum is cut into chunks for 16-bit results too."""
    gen = gen_of(11)
    for M, K, N in ((24, 20000, 264), (200, 16384, 72), (130, 16392, 72)):
        x, w = randn(gen, M, K, dtype=torch.float16), randn(gen, K, N, dtype=torch.float16, scale=K ** -0.5)
        y, z = lib.linear(x, w, act="gelu", save_preact=True)
        check_forward_any(y, z, x, w, "gelu")


def check_forward_any(y, z_out, x, w, act):
    """check_forward for a sum in one accumulator: 2^-23 of S lost at most every 16 of K."""
    z = x.double() @ w.double()
    zt = (x.shape[1] / 16 + 4) * 2.0 ** -23 * (x.double().abs() @ w.double().abs())
    assert_within(z_out, z, zt + UNIT[z_out.dtype] * (z.abs() + zt) + 2.0 ** -25)
    ref, tol = act64(z, act), 1.13 * zt + 2.0 ** -19 * (1 + z.abs())
    assert_within(y, ref, tol + UNIT[y.dtype] * (ref.abs() + tol) + 2.0 ** -25)


def test_groups_without_rows(lib):
    """All offsets zero: nothing is written but the gradients' zeros."""
    gen = gen_of(12)
    x, w = randn(gen, 20, 64, dtype=torch.bfloat16), randn(gen, 3, 64, 32, dtype=torch.bfloat16)
    off = torch.zeros(4, device="cuda", dtype=torch.int32)
    out = torch.full((20, 32), 2.0, device="cuda", dtype=torch.bfloat16)
    lib.grouped_linear(x, w, off, out=out)
    assert (out == 2).all()
    _, dw, db = lib.grouped_linear_backward(out, x, w, off, bias=True)
    assert (dw == 0).all() and (db == 0).all()
    assert lib.device_status() == 0


def test_empty_sizes(lib):
    x, w = torch.zeros(0, 64, device="cuda", dtype=torch.bfloat16), torch.ones(64, 32, device="cuda", dtype=torch.bfloat16)
    assert lib.linear(x, w).shape == (0, 32)
    dx, dw, db = lib.linear_backward(torch.zeros(0, 32, device="cuda", dtype=torch.bfloat16), x, w, bias=True)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    # K = 0: the activation of the bias
    b = torch.arange(8, device="cuda", dtype=torch.bfloat16) - 4
    y = lib.linear(torch.empty(5, 0, device="cuda", dtype=torch.bfloat16),
                   torch.empty(0, 8, device="cuda", dtype=torch.bfloat16), bias=b, act="relu")
    assert torch.equal(y, torch.relu(b).expand(5, 8))


def counts_of(kind, gen):
    if kind == "empty and single":
        return [0, 1, 0, 0, 3, 1, 0]
    if kind == "one has all":
        return [0, 0, 517, 0]
    if kind == "tile edges":
        return [16, 15, 17, 64, 63, 65, 256, 255, 257]
    if kind == "many":
        return torch.randint(0, 4, (1024,), generator=torch.Generator().manual_seed(3)).tolist()
    return [300, 1, 70, 0, 33]


def offsets_of(counts):
    return torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()


KINDS = ["empty and single", "one has all", "tile edges", "many", "mixed"]


@pytest.mark.parametrize("act", ["none", "silu", "swiglu"])
@pytest.mark.parametrize("kind", KINDS)
def test_grouped_forward(lib, kind, act):
    gen = gen_of(2)
    counts = counts_of(kind, gen)
    G, M, K, N = len(counts), sum(counts), 136, 72
    Nw = 2 * N if act == "swiglu" else N
    x = randn(gen, M + 9, K, dtype=torch.bfloat16)
    w, b = randn(gen, G, K, Nw, dtype=torch.bfloat16, scale=K ** -0.5), randn(gen, G, Nw, dtype=torch.bfloat16)
    x[M:] = math.nan  # rows past the last group: not read into a result, not written
    out = torch.full((M + 9, N), 5.0, device="cuda", dtype=torch.bfloat16)
    _, z = lib.grouped_linear(x, w, offsets_of(counts), bias=b, act=act, out=out, save_preact=True)
    at = 0
    for e, n in enumerate(counts):
        if n:
            check_forward(out[at:at + n], z[at:at + n], x[at:at + n], w[e], b[e], act, None)
        at += n
    assert (out[M:] == 5).all()
    assert lib.device_status() == 0


@pytest.mark.parametrize("way", ["fwd", "bwd"])
def test_groups_do_not_touch_each_other(lib, way):
    """NaN and infinities in one group's rows or weights stay in that group."""
    gen = gen_of(3)
    counts, K, N = [70, 5, 130, 64], 72, 136
    off = offsets_of(counts)
    M = sum(counts)
    x, w = randn(gen, M, K, dtype=torch.float16), randn(gen, 4, K, N, dtype=torch.float16)
    dy = randn(gen, M, N, dtype=torch.float16)

    def all_of(x, w, dy):
        if way == "fwd":
            return list(lib.grouped_linear(x, w, off).split(counts))
        dx, dw, db = lib.grouped_linear_backward(dy, x, w, off, bias=True)
        return [torch.cat([a.reshape(-1), b.reshape(-1).to(a.dtype), c.to(a.dtype)])
                for a, b, c in zip(dx.split(counts), dw, db)]

    clean = all_of(x, w, dy)
    at = 0
    for e, n in enumerate(counts):
        bx, bw, bdy = x.clone(), w.clone(), dy.clone()
        bx[at:at + n] = math.nan
        bw[e] = math.inf
        bdy[at:at + n] = math.nan
        at += n
        got = all_of(bx, bw, bdy)
        for o in range(4):
            if o != e:
                assert torch.equal(got[o], clean[o]), (e, o)


def grads64(dy, x, w, z, act):
    """dZ and, from the operands' own values, dX, dW, db in 64 bits."""
    zz = z.double().requires_grad_()
    act64(zz, act).backward(dy.double())
    dz = zz.grad
    return dz, dz @ w.double().t(), x.double().t() @ dz, dz.sum(0)


def check_grads(dx, dw, db, dy, x, w, z, act):
    M, K = x.shape
    dz, rx, rw, rb = grads64(dy, x, w, z, act)
    u = UNIT[x.dtype]
    # dZ: the derivative's own evaluation, then one rounding
    scale = dy.double().abs()
    if act == "swiglu":
        a, b = z.double().chunk(2, dim=1)
        own = 2.0 ** -18 * torch.cat([scale * b.abs() * (1 + a.abs()), scale * a.abs()], 1)
    elif act in ("none", "relu"):
        own = torch.zeros_like(dz)
    else:
        own = 2.0 ** -18 * scale * (1 + z.double().abs()) ** 2
    zt = own + (0 if act == "none" else u * (dz.abs() + own) + 2.0 ** -25)
    aw, ax = w.double().abs(), x.double().abs()
    tol = zt @ aw.t() + sum_tol(w.shape[1], dz.abs() @ aw.t())
    assert_within(dx, rx, tol + u * (rx.abs() + tol) + 2.0 ** -25)
    if dw is None:
        return
    tol = ax.t() @ zt + sum_tol(M, ax.t() @ dz.abs())
    assert_within(dw, rw, tol + UNIT[dw.dtype] * (rw.abs() + tol) + 2.0 ** -25)
    if db is not None:
        assert_within(db, rb, own.sum(0) + (M + 4) * 2.0 ** -24 * dz.abs().sum(0) + 1e-30)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,K,N", [(1, 64, 64), (5, 72, 136), (63, 256, 8), (64, 64, 256), (333, 200, 264),
                                   (1000, 264, 72), (4100, 136, 72)])
def test_backward(lib, M, K, N, act, dt):
    gen, dtype = gen_of(M, K, N, 1), DTYPES[dt]
    Nw = 2 * N if act == "swiglu" else N
    x, w = randn(gen, M, K, dtype=dtype), randn(gen, K, Nw, dtype=dtype, scale=K ** -0.5)
    dy, z = randn(gen, M, N, dtype=dtype), randn(gen, M, Nw, dtype=dtype, scale=2.0)
    dx, dw, db = lib.linear_backward(dy, x, w, z=z, act=act, bias=True, dw_dtype=torch.float32)
    check_grads(dx, dw, db, dy, x, w, z, act)
    dx2, dw2, none = lib.linear_backward(dy, x, w, z=z, act=act)
    assert torch.equal(dx2, dx) and none is None
    check_grads(dx2, dw2, None, dy, x, w, z, act)
    assert lib.device_status() == 0


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("kind", KINDS)
def test_grouped_backward(lib, kind, act):
    gen = gen_of(4)
    counts = counts_of(kind, gen)
    G, M, K, N = len(counts), sum(counts), 72, 136
    Nw = 2 * N if act == "swiglu" else N
    x, w = randn(gen, M, K, dtype=torch.bfloat16), randn(gen, G, K, Nw, dtype=torch.bfloat16, scale=K ** -0.5)
    dy, z = randn(gen, M, N, dtype=torch.bfloat16), randn(gen, M, Nw, dtype=torch.bfloat16)
    dx, dw, db = lib.grouped_linear_backward(dy, x, w, offsets_of(counts), z=z, act=act, bias=True)
    at = 0
    for e, n in enumerate(counts):
        sl = slice(at, at + n)
        at += n
        if n:
            check_grads(dx[sl], dw[e], db[e], dy[sl], x[sl], w[e], z[sl], act)
        else:
            assert (dw[e] == 0).all() and (db[e] == 0).all()
    assert lib.device_status() == 0


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu", "swiglu"])
def test_activations_saturate(lib, act, dt):
    """Far from zero act(z) is z or 0 and act'(z) is 1 or 0: from |z| = 128 on the sigmoid and the
    normal distribution are 0 or 1 in fp32 exactly.  So is the result but for the roundings of
    two products in fp32 (2^-22 of it) and, forward, of the result (u); no step may overflow."""
    dtype = DTYPES[dt]
    size = [128.0, 1024.0, 2.0 ** 15]
    if dtype == torch.bfloat16:
        size += [2.0 ** 40, 2.0 ** 62, 2.0 ** 65, 2.0 ** 100, 2.0 ** 124]
    v = torch.tensor(size + [-a for a in size] + ([-1.5 * 2.0 ** 127] if dtype == torch.bfloat16 else []))
    v = v.to(dtype).cuda()
    M = v.numel()
    on = torch.where(v > 0, 1.0, 0.0).double()
    # forward: z is the one value of its row
    x = torch.zeros(M, 8, dtype=dtype, device="cuda")
    x[:, 0], x[:, 1] = v, 1.0
    w = torch.zeros(8, 16 if act == "swiglu" else 8, dtype=dtype, device="cuda")
    w[0, :8] = 1.0
    w[1, 8:] = 0.5
    y = lib.linear(x, w, act=act)
    ref = (on * v.double() * (0.5 if act == "swiglu" else 1.0))[:, None].expand(M, 8)
    assert_within(y, ref, (UNIT[dtype] + 2.0 ** -22) * ref.abs() + 2.0 ** -25)
    # backward: each row a group of its own, whose db is the row of dZ
    z = x.double() @ w.double()
    dy = torch.full((M, 8), 4.0, dtype=dtype, device="cuda")
    off = torch.arange(M + 1, dtype=torch.int32, device="cuda")
    _, _, db = lib.grouped_linear_backward(dy, x, w.expand(M, *w.shape).contiguous(), off, z=z.to(dtype), act=act,
                                           bias=True, need_dx=False, need_dw=False)
    ref = 4.0 * on[:, None].expand(M, 8)
    if act == "swiglu":
        ref = torch.cat([0.5 * ref, ref * v.double()[:, None]], dim=1)
    assert_within(db, ref, 2.0 ** -22 * ref.abs() + 2.0 ** -25)


@pytest.mark.parametrize("M,K,N,counts", [(1, 64, 72, None), (333, 200, 264, None), (2100, 1032, 1000, None),
                                          (5000, 8, 4104, None), (700, 136, 40, [0, 300, 1, 0, 390, 0, 9]),
                                          (90, 520, 264, [3] * 30)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_bias_gradient_with_and_without_dx(lib, M, K, N, counts, act):
    """db does not depend on whether dX is wanted, to the bit, and is the sum of dZ's rows: n fp32
    additions at most for n rows, and dZ's own error (swiglu: 2^-19 (1 + |z|) of |dY u|)."""
    gen, dtype = gen_of(M, K, N), torch.bfloat16
    G, Nw = len(counts) if counts else 1, 2 * N if act == "swiglu" else N
    dy, x = randn(gen, M, N, dtype=dtype), randn(gen, M, K, dtype=dtype)
    w = randn(gen, *((G, K, Nw) if counts else (K, Nw)), dtype=dtype, scale=K ** -0.5)
    z = randn(gen, M, Nw, dtype=dtype) if act != "none" else None
    off = torch.tensor([0] + counts).cumsum(0).int().cuda() if counts else None
    got = []
    for need in (True, False):
        if counts:
            got.append(lib.grouped_linear_backward(dy, x, w, off, z=z, act=act, bias=True, need_dx=need)[2])
        else:
            got.append(lib.linear_backward(dy, x, w, z=z, act=act, bias=True, need_dx=need)[2])
    assert torch.equal(*got)
    dz, own = dy.double(), 0
    if act == "swiglu":
        a, u = z.double().chunk(2, dim=1)
        s = torch.sigmoid(a)
        dz, own = (torch.cat([dz * u * (s + a * s * (1 - s)), dz * a * s], dim=1),
                   2.0 ** -19 * torch.cat([(1 + a.abs()) * (dz * u).abs(), (1 + a.abs()) * dz.abs()], dim=1))
    size = dz.abs() * M * 2.0 ** -24 + own
    parts = lambda t: torch.stack([r.sum(0) for r in t.split(counts)]) if counts else t.sum(0)
    assert_within(got[0], parts(dz), parts(size) + 2.0 ** -25)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "swiglu"])
def test_gradients_against_differences(lib, act):
    """<dX, V> and <dW, V> against central differences of <dY, Y> along V.

    Inputs are multiples of 2^-6 below 2 and V is +-1, so X +- hV with h = 2^-6 is exact in
    fp16.  The difference's own error is h^2 / 6 times the third derivative along V; the
    step h is small against the activations' scale of 1, and Richardson's combination of h
    and 2 h removes that term.  What is left is the fp16 rounding of Z, dZ, dX and dW:
    2^-11 each of terms whose signs are random, so that 0.5 % of the gradient's norm times
    that of V over the square root of its size covers it many times over."""
    gen = gen_of(5)
    M, K, N = 48, 64, 72
    Nw = 2 * N if act == "swiglu" else N

    def grid(*s, top):
        return (torch.randint(-top, top + 1, s, generator=gen, device="cuda").float() / 64).half()

    x, w, dy = grid(M, K, top=64), grid(K, Nw, top=16), grid(M, N, top=64)
    _, z = lib.linear(x, w, act=act, save_preact=True)
    dx, dw, _ = lib.linear_backward(dy, x, w, z=z, act=act)

    def loss(x, w):
        return (lib.linear(x, w, act=act, out_dtype=torch.float32).double() * dy.double()).sum().item()

    for which, grad, t in (("x", dx, x), ("w", dw, w)):
        for _ in range(4):
            v = (torch.randint(0, 2, t.shape, generator=gen, device="cuda") * 2 - 1).half()

            def diff(h):
                a, b = t + h * v, t - h * v
                return (loss(a, w) - loss(b, w)) / (2 * h) if which == "x" else (loss(x, a) - loss(x, b)) / (2 * h)

            d = (4 * diff(2.0 ** -6) - diff(2.0 ** -5)) / 3
            got = (grad.double() * v.double()).sum().item()
            # one direction: the products' norm is |grad| for a random V
            assert abs(got - d) <= 0.005 * grad.double().norm().item() + 1e-6 * abs(d), (which, got, d)


def test_repeats_bit_for_bit(lib):
    """K slices are added in order whoever finishes last."""
    gen = gen_of(6)
    x, w = randn(gen, 24, 4096, dtype=torch.bfloat16), randn(gen, 4096, 512, dtype=torch.bfloat16)
    first = lib.linear(x, w, out_dtype=torch.float32)
    for _ in range(20):
        assert torch.equal(lib.linear(x, w, out_dtype=torch.float32), first)
    dy = randn(gen, 24, 512, dtype=torch.bfloat16)
    a = lib.linear_backward(dy, x, w, bias=True)
    for _ in range(5):
        for p, q in zip(a, lib.linear_backward(dy, x, w, bias=True)):
            assert torch.equal(p, q)


def test_other_stream_and_graph(lib):
    """On a stream of its own, and replayed from a graph (nothing is left over between calls)."""
    gen = gen_of(7)
    x, w = randn(gen, 40, 2048, dtype=torch.bfloat16), randn(gen, 2048, 256, dtype=torch.bfloat16)
    out = torch.empty(40, 256, device="cuda", dtype=torch.bfloat16)
    want = lib.linear(x, w, act="silu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = lib.linear(x, w, act="silu", stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.linear(x, w, act="silu", out=out)
    x2 = randn(gen, 40, 2048, dtype=torch.bfloat16)
    for src in (x, x2, x):
        keep = src.clone()
        x.copy_(keep)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, lib.linear(keep, w, act="silu"))


def test_bounded_wait_reports(g):
    """A wait that runs out is reported, and the next calls work."""
    lib = g.Gemm(0)
    gen = gen_of(8)
    x, w = randn(gen, 24, 4096, dtype=torch.bfloat16), randn(gen, 4096, 512, dtype=torch.bfloat16)
    want = lib.linear(x, w)
    lib.set_option(g.GEMM_OPT_WAIT_LIMIT_US, 20000)
    lib.set_option(g.GEMM_OPT_TEST_STALL, 1)
    lib.linear(x, w)
    assert lib.device_status() == g.GEMM_ERR_DEVICE_TIMEOUT
    lib.set_option(g.GEMM_OPT_TEST_STALL, 0)
    lib.set_option(g.GEMM_OPT_WAIT_LIMIT_US, 0)
    assert torch.equal(lib.linear(x, w), want)
    assert lib.device_status() == 0
    lib.close()


def test_refusals(g, lib):
    x = torch.zeros(16, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(64, 32, device="cuda", dtype=torch.bfloat16)
    off = torch.tensor([0, 8, 16], device="cuda", dtype=torch.int32)
    w3 = torch.zeros(2, 64, 32, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(g.GemmError) as e:
        lib.linear(x.float(), w.float())
    assert e.value.status == g.GEMM_ERR_UNSUPPORTED
    with pytest.raises(TypeError):
        lib.linear(x, w.half())
    with pytest.raises(ValueError):
        lib.linear(x, w[:32])
    with pytest.raises(ValueError):
        lib.linear(x, w.t().contiguous().t())
    with pytest.raises(KeyError):
        lib.linear(x, w, act="softmax")
    with pytest.raises(ValueError):
        lib.linear(x.cpu(), w)
    with pytest.raises(ValueError):
        lib.linear(x, w, bias=torch.zeros(31, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        lib.linear(x, w[:, :31].contiguous(), act="swiglu")
    for bad in (lambda: lib.linear(x, w[:, :20].contiguous()),           # ldw % 8
                lambda: lib.linear(x.reshape(-1)[1:961].view(15, 64), w),  # x not 16-byte aligned
                lambda: lib.linear(x, w[:, :24].contiguous(), act="swiglu")):  # N = 12
        with pytest.raises(g.GemmError) as e:
            bad()
        assert e.value.status == g.GEMM_ERR_ALIGNMENT
    with pytest.raises(ValueError):
        lib.grouped_linear(x, w3, None)
    with pytest.raises(ValueError):
        lib.grouped_linear(x, w3, off.long())
    with pytest.raises(ValueError):
        lib.grouped_linear(x, w3, off[:2])
    with pytest.raises(ValueError):
        lib.linear_backward(x[:, :32].contiguous(), x, w, act="gelu")  # no z
    many = torch.zeros(1025, 8, 8, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(g.GemmError) as e:
        lib.grouped_linear(torch.zeros(4, 8, device="cuda", dtype=torch.bfloat16), many,
                           torch.zeros(1026, device="cuda", dtype=torch.int32))
    assert e.value.status == g.GEMM_ERR_UNSUPPORTED
    a = g.LinearArgs(4, 8, 8, x.data_ptr(), 64, w.data_ptr(), 32, 0, None, None, 0, None, 0, x.data_ptr(), 64, 0, None,
                     g.GEMM_BF16, g.GEMM_F16, 0)
    assert g.gemm_linear(lib.handle, a) == g.GEMM_ERR_INVALID_ARG  # bf16 operands, fp16 result
    a.y_dtype, a.ldx = g.GEMM_BF16, 7
    assert g.gemm_linear(lib.handle, a) == g.GEMM_ERR_INVALID_ARG
    a.ldx, a.act = 64, 6
    assert g.gemm_linear(lib.handle, a) == g.GEMM_ERR_INVALID_ARG
    assert lib.device_status() == 0


def test_wrong_offsets_stay_inside(lib):
    """Offsets out of range or out of order give wrong results, not accesses outside: they are
    clamped to the rows there are."""
    gen = gen_of(9)
    x, w = randn(gen, 40, 64, dtype=torch.bfloat16), randn(gen, 3, 64, 64, dtype=torch.bfloat16)
    buf = torch.full((60, 64), 3.0, device="cuda", dtype=torch.bfloat16)
    out = buf[10:50]
    for off in ([0, 30, 10, 40], [-5, 100, 200, 300], [0, 0, 0, 1000]):
        lib.grouped_linear(x, w, torch.tensor(off, device="cuda", dtype=torch.int32), out=out)
        assert (buf[:10] == 3).all() and (buf[50:] == 3).all()
    assert lib.device_status() == 0


def test_moe_block_example():
    """The operators together; each step rounds to bf16 (2^-9 of it on average), six to eight
    roundings deep for the gradients."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import moe_block
    for shape in (dict(), dict(tokens=1, k=3), dict(tokens=515, hidden=136, inner=72, experts=5, k=5)):
        for name, err in moe_block.compare(**shape).items():
            assert err < 8 * 2.0 ** -9, (shape, name, err)


DEBUG_SCRIPT = r"""
import torch
import programming_tiled_gemm_gb300 as g
assert g.DEBUG
lib = g.Gemm(0)
for M, K, N in ((1, 2048, 256), (300, 136, 264), (1000, 512, 72)):
    x, w = torch.randn(M, K, device="cuda").bfloat16(), torch.randn(K, 2 * N, device="cuda").bfloat16()
    y, z = lib.linear(x, w, act="swiglu", save_preact=True)
    lib.linear_backward(y, x, w, z=z, act="swiglu", bias=True)
    off = torch.tensor([0, M // 3, M // 3, M], device="cuda", dtype=torch.int32)
    w3 = w.expand(3, K, 2 * N).contiguous()
    y, z = lib.grouped_linear(x, w3, off, act="swiglu", save_preact=True)
    lib.grouped_linear_backward(y, x, w3, off, z=z, act="swiglu", bias=True)
    r = lib.moe_route(torch.randn(M, 40, device="cuda"), 3)
    lib.moe_combine(lib.moe_dispatch(x, r.rows, 3), r.slots, r.weights)
assert lib.device_status() == g.GEMM_OK
print("clean")
"""


def test_debug_build_finds_no_index_out_of_range():
    env = dict(os.environ, GEMM_GB300_DEBUG="1")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", DEBUG_SCRIPT], cwd=root, env=env, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "clean" in out.stdout, out.stdout + out.stderr
