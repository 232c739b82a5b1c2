"""Routing to experts and the exchange of rows, against plain forms in 64 bits.

Whole numbers are equal.  weights: the exponential (2 ulp of fp32) of each logit's distance
from the largest, and a sum of n of them: (n + 8) 2^-24 relative, plus 2^-24 |distance| for the
rounded difference.  Exchange: fp32 sums of k terms (k 2^-24 of their magnitudes), one rounding.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def g():
    import programming_tiled_gemm_gb300 as g
    return g


@pytest.fixture(scope="module")
def lib(g):
    lib = g.Gemm(0)
    yield lib
    lib.close()


def gen_of(*key):
    return torch.Generator(device="cuda").manual_seed(hash(key) % (1 << 31))


def route64(logits, k, renormalize):
    """weights, experts, slots, rows, offsets with numpy, one token at a time."""
    l = logits.double().cpu().numpy()
    T, E = l.shape
    weights, experts = np.zeros((T, k)), np.full((T, k), -1, np.int64)
    for t in range(T):
        # NaN first, then descending, lower index first; -inf is not there
        order = sorted((e for e in range(E) if not l[t, e] == -math.inf),
                       key=lambda e: (0 if math.isnan(l[t, e]) else 1, 0.0 if math.isnan(l[t, e]) else -l[t, e], e))
        pick = order[:k]
        experts[t, :len(pick)] = pick
        if pick:
            over = pick if renormalize else order
            with np.errstate(invalid="ignore"):
                top = max(l[t, over]) if not any(math.isnan(l[t, e]) for e in over) else math.nan
                p = np.exp(l[t, over] - top)
                weights[t, :len(pick)] = (p / p.sum())[:len(pick)]
    flat = experts.reshape(-1)
    place = np.argsort(np.where(flat < 0, E, flat), kind="stable")
    n = int((flat >= 0).sum())
    slots, rows = np.full(T * k, -1, np.int64), np.full(T * k, -1, np.int64)
    rows[:n] = place[:n]
    slots[place[:n]] = np.arange(n)
    offsets = np.concatenate([[0], np.bincount(flat[flat >= 0], minlength=E).cumsum()])
    return weights, experts, slots.reshape(T, k), rows, offsets


def check_route(lib, logits, k, renormalize=True):
    r = lib.moe_route(logits, k, renormalize=renormalize)
    weights, experts, slots, rows, offsets = route64(logits, k, renormalize)
    for got, ref in ((r.experts, experts), (r.slots, slots), (r.rows, rows), (r.offsets, offsets)):
        assert np.array_equal(got.cpu().numpy(), ref)
    got = r.weights.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(weights))
    n = logits.shape[1] if not renormalize else k
    finite = logits.double().cpu().numpy()
    finite = finite[np.isfinite(finite)]
    spread = float(finite.max() - finite.min()) if finite.size else 0.0
    ok = ~np.isnan(weights)
    assert (np.abs(got - weights)[ok] <= ((n + 8) + spread) * 2.0 ** -23 * weights[ok] + 1e-37).all()
    return r


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (7, 5, 5), (16, 64, 4), (33, 32, 1), (100, 33, 8),
                                   (128, 128, 8), (129, 60, 6), (300, 256, 8), (515, 512, 3), (200, 1024, 32),
                                   (1000, 16, 2)])
def test_route(lib, T, E, k, dt):
    gen = gen_of(T, E, k)
    logits = (torch.randn(T, E, generator=gen, device="cuda") * 2).to(DTYPES[dt])
    for renormalize in (True, False):
        check_route(lib, logits, k, renormalize)


@pytest.mark.parametrize("T", [40, 400])
def test_route_ties_masks_and_specials(lib, T):
    gen = gen_of(T)
    E, k = 24, 4
    l = torch.randint(-2, 3, (T, E), generator=gen, device="cuda").float()  # many ties
    l[1] = 0.0
    l[2, ::2] = -0.0  # equal to +0
    l[2, 1::2] = 0.0
    l[3] = -math.inf  # nobody is there
    l[4, 2:] = -math.inf  # two experts for four picks
    l[5, 7] = math.inf
    l[6, 9] = math.nan
    l[7] = torch.finfo(torch.float32).min  # the lowest finite value is there
    l[8, :5] = -math.inf
    l[9, 3] = -math.nan
    for renormalize in (True, False):
        check_route(lib, l, k, renormalize)
        check_route(lib, l[torch.arange(T) % 10 != 5].half(), k, renormalize)
    none = torch.full((T, E), -math.inf, device="cuda")
    r = check_route(lib, none, k)
    assert (r.offsets == 0).all() and (r.weights == 0).all()


def test_route_skew_strides_and_empty(lib):
    """All tokens to the same experts; padded rows; no token."""
    l = torch.zeros(700, 48, device="cuda")
    l[:, 10], l[:, 40] = 5.0, 4.0
    check_route(lib, l, 2)
    wide = torch.full((200, 70), math.nan, device="cuda", dtype=torch.bfloat16)
    wide[:, :61] = torch.randn(200, 61, generator=gen_of(1), device="cuda")
    check_route(lib, wide[:, :61], 3)
    r = lib.moe_route(torch.zeros(0, 12, device="cuda"), 2)
    assert r.experts.shape == (0, 2) and torch.equal(r.offsets, torch.zeros(13, device="cuda", dtype=torch.int32))
    assert lib.device_status() == 0


def grad64(logits, experts, dw, renormalize):
    """The formula through autograd in 64 bits."""
    l = logits.double().detach().requires_grad_()
    here = experts >= 0
    at = experts.clamp(min=0).long()
    if renormalize:
        z = torch.where(here, l.gather(1, at), torch.full((), -1e300, dtype=torch.float64, device=l.device))
        w = torch.softmax(z, 1)
    else:
        w = torch.softmax(torch.where(l == -math.inf, torch.full_like(l, -1e300), l), 1).gather(1, at)
    (w * torch.where(here, dw.double(), torch.zeros_like(w))).sum().backward()
    return l.grad


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (50, 33, 5), (300, 128, 8), (20, 1024, 32)])
def test_route_backward(lib, T, E, k, renormalize, dt):
    gen = gen_of(T, E, 2)
    logits = (torch.randn(T, E, generator=gen, device="cuda") * 2).to(DTYPES[dt])
    if T > 1:
        logits[torch.rand(T, E, generator=gen, device="cuda") < 0.2] = -math.inf
        logits[3] = -math.inf
        logits[4, 1:] = -math.inf
    r = lib.moe_route(logits, k, renormalize=renormalize)
    dw = torch.randn(T, k, generator=gen, device="cuda")
    got = lib.moe_route_backward(dw, logits, r.experts, renormalize=renormalize)
    ref = grad64(logits, r.experts, dw, renormalize)
    ref[(r.experts < 0).all(1)] = 0
    assert got.dtype == logits.dtype
    # p (g - mean): each factor as the weights, the difference of magnitudes up to max |dw|
    p = (ref.abs() + r.weights.double().max(1, keepdim=True).values) * dw.abs().max().item()
    tol = (E + 24) * 2.0 ** -23 * p + UNIT[got.dtype] * ref.abs() + (2.0 ** -25 if dt == "f16" else 1e-37)
    assert ((got.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_against_differences(lib, renormalize):
    """Central differences of the weights, h = 2^-5, with the h^2 term removed by a second step
    of 2 h; the picks of well separated logits do not change.  What is left: h^4 / 30 of fifth
    derivatives (below 20 for a softmax) and fp32 rounding over h, 1e-5 together."""
    gen = gen_of(3)
    T, E, k = 40, 12, 3
    logits = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t)) for t in range(T)]).cuda() * 0.5
    dw = torch.randn(T, k, generator=gen, device="cuda")
    r = lib.moe_route(logits, k, renormalize=renormalize)
    got = lib.moe_route_backward(dw, logits, r.experts, renormalize=renormalize)
    for e in range(E):
        step = torch.zeros(T, E, device="cuda")
        step[:, e] = 1.0

        def diff(h):
            a, b = (lib.moe_route(logits + s * step, k, renormalize=renormalize) for s in (h, -h))
            assert torch.equal(a.experts, r.experts) and torch.equal(b.experts, r.experts)
            return ((a.weights - b.weights) * dw).sum(1) / (2 * h)

        d = (4 * diff(2.0 ** -5) - diff(2.0 ** -4)) / 3
        assert (got[:, e] - d).abs().max() < 2e-5 * (1 + dw.abs().max())


def routing(T, E, k, gen, drop):
    experts = torch.topk(torch.rand(T, E, generator=gen, device="cuda"), k, dim=1).indices
    if drop:
        experts[torch.rand(T, k, generator=gen, device="cuda") < drop] = -1
    flat = experts.reshape(-1).cpu().numpy()
    place = np.argsort(np.where(flat < 0, E, flat), kind="stable")
    n = int((flat >= 0).sum())
    slots, rows = np.full(T * k, -1, np.int32), np.full(T * k, -1, np.int32)
    rows[:n] = place[:n]
    slots[place[:n]] = np.arange(n)
    return torch.from_numpy(slots).view(T, k).cuda(), torch.from_numpy(rows).cuda(), n


def close(got, ref, mags, k):
    u = UNIT[got.dtype]
    tol = (k + 1) * 2.0 ** -23 * mags + u * ref.abs() + 2.0 ** -25
    assert ((got.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,N,k,drop", [(1, 8, 1, 0), (5, 7, 2, 0.3), (64, 256, 4, 0), (33, 2056, 3, 0.2),
                                        (200, 1001, 6, 0.1), (40, 64, 32, 0.5)])
def test_exchange(lib, T, N, k, drop, dt):
    gen = gen_of(T, N, k)
    dtype = DTYPES[dt]
    slots, rows, n = routing(T, 64, k, gen, drop)
    x, dout, r = (torch.randn(T, N, generator=gen, device="cuda").to(dtype) for _ in range(3))
    y = torch.randn(T * k, N, generator=gen, device="cuda").to(dtype)
    y[n:] = math.nan  # rows that hold nothing are not read
    w = torch.rand(T, k, generator=gen, device="cuda")
    xr = lib.moe_dispatch(x, rows, k)
    want = torch.zeros_like(xr)
    want[:n] = x[rows[:n].long() // k]
    assert torch.equal(xr, want)
    there = (slots >= 0)[:, :, None]
    rowsof = torch.where(there, y.double()[slots.clamp(min=0).long()], torch.zeros((), dtype=torch.float64, device="cuda"))
    terms = w.double()[:, :, None] * rowsof
    close(lib.moe_combine(y, slots, w, residual=r), terms.sum(1) + r.double(), terms.abs().sum(1) + r.double().abs(), k)
    close(lib.moe_combine(y, slots), rowsof.sum(1), rowsof.abs().sum(1), k)
    dy, dw = lib.moe_combine_backward(dout, y, slots, rows, w)
    ref = torch.zeros(T * k, N, dtype=torch.float64, device="cuda")
    a = rows[:n].long()
    ref[:n] = w.reshape(-1).double()[a][:, None] * dout.double()[a // k]
    close(dy, ref, ref.abs(), 1)
    prod = rowsof * dout.double()[:, None, :]
    # dots of N products
    assert ((dw.double() - prod.sum(2)).abs() <= (N + 8) * 2.0 ** -24 * prod.abs().sum(2) + 1e-30).all()
    assert lib.device_status() == 0


def test_exchange_strides_and_in_place(lib):
    gen = gen_of(4)
    T, N, k = 30, 72, 2
    slots, rows, n = routing(T, 16, k, gen, 0.0)
    for pad, shift in ((8, 0), (3, 0), (8, 1)):
        X = torch.full((T * (N + pad) + shift,), math.nan, device="cuda", dtype=torch.bfloat16)
        x = X[shift:].view(T, N + pad)[:, :N]
        x.copy_(torch.randn(T, N, generator=gen, device="cuda"))
        xr = lib.moe_dispatch(x, rows, k)
        assert torch.equal(xr, x[rows.long() // k])
        was = x.clone()
        got = lib.moe_combine(xr, slots, residual=x, out=x)
        assert got.data_ptr() == x.data_ptr()
        close(x, 3 * was.double(), 3 * was.double().abs(), k)
        assert torch.isnan(X[shift:].view(T, N + pad)[:, N:]).all()


def test_exchange_past_32_bits(lib):
    """More than 2^31 elements on the experts' side: the last rows."""
    T, N, k = 140_000, 8192, 2
    x = torch.zeros(T, N, device="cuda", dtype=torch.bfloat16)
    x[-2:] = torch.randn(2, N, generator=gen_of(6), device="cuda")
    rows = torch.arange(T * k, device="cuda", dtype=torch.int32)  # each pick at its own place
    slots = rows.view(T, k)
    xr = lib.moe_dispatch(x, rows, k)
    assert xr.numel() > 2 ** 31 and torch.equal(xr[-4:], x[-2:].repeat_interleave(2, 0)) and (xr[:4] == 0).all()
    w = torch.ones(T, k, device="cuda")
    out = lib.moe_combine(xr, slots, w)
    assert torch.equal(out[-2:], (2 * x[-2:].float()).bfloat16())
    dy, dw = lib.moe_combine_backward(x, xr, slots, rows, w)
    assert torch.equal(dy[-4:], xr[-4:])
    ref = (x[-2:].double() ** 2).sum(1, keepdim=True).expand(2, k)
    assert ((dw[-2:].double() - ref).abs() <= (N + 8) * 2.0 ** -24 * ref).all()
    assert lib.device_status() == 0


def test_empty_and_refusals(g, lib):
    e = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    i32 = dict(dtype=torch.int32)
    assert lib.moe_dispatch(e(0, 16), e(0, **i32), 2).shape == (0, 16)
    assert lib.moe_combine(e(0, 16), e(0, 2, **i32)).shape == (0, 16)
    dy, dw = lib.moe_combine_backward(e(3, 0), e(6, 0), e(3, 2, **i32), e(6, **i32), e(3, 2))
    assert dy.shape == (6, 0) and (dw == 0).all()
    with pytest.raises(ValueError):
        lib.moe_route(e(4, 8), 9)
    with pytest.raises(ValueError):
        lib.moe_route(e(4, 8), 0)
    with pytest.raises(TypeError):
        lib.moe_route(e(4, 8, dtype=torch.float64), 2)
    with pytest.raises(g.GemmError) as err:
        lib.moe_route(e(4, 1025), 2)
    assert err.value.status == g.GEMM_ERR_UNSUPPORTED
    with pytest.raises(g.GemmError) as err:
        lib.moe_route(e(4, 64), 33)
    assert err.value.status == g.GEMM_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        lib.moe_dispatch(e(4, 8), e(7, **i32), 2)
    with pytest.raises(ValueError):
        lib.moe_dispatch(e(4, 8), e(8, dtype=torch.int64), 2)
    with pytest.raises(ValueError):
        lib.moe_combine(e(8, 8), e(4, 2, **i32), weights=e(4, 2, dtype=torch.float64))
    with pytest.raises(ValueError):
        lib.moe_combine_backward(e(4, 8), e(7, 8), e(4, 2, **i32), e(8, **i32), e(4, 2))
    # row numbers out of range are left out
    wild = torch.full((4, 2), 1 << 30, device="cuda", **i32)
    assert (lib.moe_combine(torch.ones(8, 8, device="cuda"), wild) == 0).all()
    assert lib.device_status() == 0


def test_graph(lib):
    """Replayed routing leaves its counter as it found it."""
    gen = gen_of(5)
    l = torch.randn(300, 40, generator=gen, device="cuda")
    lib.moe_route(l, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = lib.moe_route(l, 4)
    for seed in range(3):
        l.copy_(torch.randn(300, 40, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = lib.moe_route(l, 4)
        for a, b in zip(r, want):
            assert torch.equal(a, b)
