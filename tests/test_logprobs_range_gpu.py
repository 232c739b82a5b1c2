"""Token log probabilities wherever the finite logits lie: finite masks, rows of nothing else, offsets at which
neighbouring logits are far apart, temperatures down to the smallest; forward and backward, against 64 bits.

The tolerances are those of test_logprobs_gpu.py: they count roundings of u = (z - m) / T, which has the same number
whatever the magnitude of z and m.  Temperatures are fp32 values, so that both sides take the same one.
"""
import math

import numpy as np
import pytest
import torch

from test_logprobs_gpu import DTYPES, check_backward, check_forward, make

pytestmark = pytest.mark.gpu

LOWEST = {"bf16": -3.3895313892515355e38, "f16": -65504.0, "f32": -3.4028234663852886e38}
# fp16 has no larger mask than its lowest value; colder temperatures take it as far
MASKED = ([("f32", v, t) for v in (-1e9, -1e10, -1e12, -1e20, -1e30, LOWEST["f32"]) for t in (0.1, 0.3, 1.0, 5.0, 30.0)] +
          [("bf16", v, t) for v in (-1e9, -1e10, -1e12, -1e20, -1e30, LOWEST["bf16"]) for t in (0.1, 1.0, 5.0, 10.0)] +
          [("f16", v, t) for v in (-6e4, LOWEST["f16"]) for t in (1e-6, 1e-4, 0.1, 1.0)])


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


def f32(v):
    return float(np.float32(v))


def masked_rows(dtype, value, rows, V):
    """rows whose masked stretches leave: all but the first part, all but the last, one in the middle, one at either
    end, a few, none, every other one"""
    logits, tokens = make(rows + V, rows, V, DTYPES[dtype])
    free = torch.zeros(rows, V, dtype=torch.bool, device="cuda")
    at = torch.arange(V, device="cuda")
    kinds = [at >= V * 3 // 4, at < V // 4, at == V // 2, at == 0, at == V - 1, (at > V // 3) & (at < V // 3 + 40),
             at < 0, at % 2 == 0]
    for r in range(rows):
        free[r] = kinds[r % len(kinds)]
    logits.masked_fill_(~free, value)
    # a token that is left, where there is one, and a masked one in every third row
    first = torch.where(free.any(1), free.float().argmax(1), torch.full_like(tokens, 3))
    tokens = torch.where(torch.arange(rows, device="cuda") % 3 == 1, tokens, first)
    return logits, tokens



# (rows, V): a row over eight CTAs; threads with several batches; a row a CTA
SHAPES = [(16, 20011), (8, 40000), (1400, 6007)]


@pytest.mark.parametrize("rows,V", SHAPES)
@pytest.mark.parametrize("dtype,value,temperature", MASKED)
def test_finite_masks(lib, dtype, value, temperature, rows, V):
    t = f32(temperature)
    logits, tokens = masked_rows(dtype, value, rows, V)
    r = lib.token_logprobs(logits, tokens, top=8, entropy=True, temperature=t)
    check_forward(logits, tokens, t, 8, r)
    plain = lib.token_logprobs(logits, tokens, temperature=t)
    check_forward(logits, tokens, t, 0, plain)


OFFSETS = [("f32", 1e8, 8.0), ("f32", -3e9, 256.0), ("f32", 1e20, 2.0 ** 43), ("f32", -1e30, 2.0 ** 76),
           ("bf16", 1e8, 2.0 ** 19), ("bf16", -1e20, 2.0 ** 59), ("f16", 6e4, 32.0), ("f16", -6e4, 32.0)]


def offset_rows(dtype, base, step, rows=12, V=5003):
    """logits a few of the type's steps from each other, far from zero"""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    k = torch.randint(-8, 9, (rows, V), generator=gen, device="cuda")
    k[::4] = 0  # rows of one value only
    logits = (base + k.double() * step).to(DTYPES[dtype])
    return logits, torch.randint(0, V, (rows,), generator=gen, device="cuda")


@pytest.mark.parametrize("dtype,base,step", OFFSETS)
@pytest.mark.parametrize("of_step", [0.01, 0.5, 4.0])
def test_far_from_zero(lib, dtype, base, step, of_step):
    """the distribution of offsets of some `step`s at temperatures about as large"""
    t = f32(step * of_step)
    logits, tokens = offset_rows(dtype, base, step)
    r = lib.token_logprobs(logits, tokens, top=8, entropy=True, temperature=t)
    check_forward(logits, tokens, t, 8, r)


COLD = [1e-3, 1e-6, 1e-9, 1e-12, 1e-30]


def tied_rows(dtype, rows=10, V=9001):
    """ordinary logits, the largest of them n times in the n-th row"""
    logits, tokens = make(31, rows, V, DTYPES[dtype])
    for n in range(rows):
        logits[n, torch.arange(n + 1, device="cuda") * 811] = 17.75
    tokens[::2] = 0
    return logits, tokens


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("temperature", COLD)
def test_cold(lib, dtype, temperature):
    t = f32(temperature)
    logits, tokens = tied_rows(dtype)
    r = lib.token_logprobs(logits, tokens, top=12, entropy=True, temperature=t)
    check_forward(logits, tokens, t, 12, r)
    n = torch.arange(1, 11, device="cuda").double()
    if t < 1e-5:
        assert bool(((r.entropy.double() - torch.log(n)).abs() <= 2.0 ** -20).all())


HOT = [1.0, 1.5, 3.0, 2e38, 3.4e38]


def rows_of_extremes(dtype):
    """largest and lowest values side by side: their difference has no fp32 value, its product with 1 / T has"""
    low = LOWEST[dtype]
    logits, tokens = make(77, 6, 3001, DTYPES[dtype])
    logits[0] = low
    logits[0, 7::3] = -low
    logits[1, ::2] = low
    logits[1, 1::2] = -low
    logits[2] = low
    logits[2, 2222] = -low
    logits[3] = -low
    logits[4, ::5] = low
    tokens[:4] = torch.tensor([8, 1, 2222, 0], device="cuda")
    return logits, tokens


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("temperature", HOT)
def test_differences_beyond_the_range(lib, dtype, temperature):
    t = f32(temperature)
    logits, tokens = rows_of_extremes(dtype)
    r = lib.token_logprobs(logits, tokens, top=5, entropy=True, temperature=t)
    check_forward(logits, tokens, t, 5, r)


def check_gradients(lib, logits, tokens, t, r):
    gen = torch.Generator(device="cuda").manual_seed(len(logits))
    # (no larger than the temperature: the logits' gradients stay in the types' range)
    gain, dh = (torch.randn(len(logits), generator=gen, device="cuda") * min(1.0, t) for _ in range(2))
    for g_, h_ in ((gain, dh), (gain, None)):
        dl = lib.token_logprobs_backward(g_, logits, tokens, r, dentropy=h_, temperature=t)
        assert not bool(dl.isnan().any())
        check_backward(logits, tokens, t, g_, h_, dl)


@pytest.mark.parametrize("rows,V", SHAPES[:2])
@pytest.mark.parametrize("dtype,value,temperature", MASKED)
def test_gradient_of_finite_masks(lib, dtype, value, temperature, rows, V):
    t = f32(temperature)
    logits, tokens = masked_rows(dtype, value, rows, V)
    check_gradients(lib, logits, tokens, t, lib.token_logprobs(logits, tokens, entropy=True, temperature=t))


@pytest.mark.parametrize("dtype,base,step", OFFSETS)
@pytest.mark.parametrize("of_step", [0.01, 0.5, 4.0])
def test_gradient_far_from_zero(lib, dtype, base, step, of_step):
    t = f32(step * of_step)
    logits, tokens = offset_rows(dtype, base, step)
    check_gradients(lib, logits, tokens, t, lib.token_logprobs(logits, tokens, entropy=True, temperature=t))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("temperature", COLD)
def test_gradient_of_ties_in_the_cold(lib, dtype, temperature):
    """n equal largest logits have 1 / n each, however cold"""
    t = f32(temperature)
    logits, tokens = tied_rows(dtype)
    r = lib.token_logprobs(logits, tokens, entropy=True, temperature=t)
    check_gradients(lib, logits, tokens, t, r)
    dl = lib.token_logprobs_backward(torch.full((10,), -t, device="cuda"), logits, torch.full_like(tokens, 5), r,
                                     temperature=t)
    if t < 1e-5:
        share = 1.0 / torch.arange(1, 11, device="cuda")
        assert bool(((dl[:, 0].float() - share).abs() <= share * (torch.finfo(dl.dtype).eps / 2 + 2.0 ** -19)).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("temperature", HOT)
def test_gradient_of_differences_beyond_the_range(lib, dtype, temperature):
    t = f32(temperature)
    logits, tokens = rows_of_extremes(dtype)
    check_gradients(lib, logits, tokens, t, lib.token_logprobs(logits, tokens, entropy=True, temperature=t))


@pytest.mark.parametrize("temperature", [2.95e-39, 3.5e-39, 4.23e-39])
def test_temperatures_without_a_finite_exponent_scale_are_refused(lib, g, temperature):
    """1 / T is finite there, 1 / (T ln 2) is not"""
    t = f32(temperature)
    logits, tokens = make(1, 4, 100, torch.float32)
    ok = lib.token_logprobs(logits, tokens)
    n = lib.launch_count()
    with pytest.raises(g.GemmError) as e:
        lib.token_logprobs(logits, tokens, temperature=t)
    assert e.value.status == g.GEMM_ERR_INVALID_ARG
    with pytest.raises(g.GemmError) as e:
        lib.token_logprobs_backward(None, logits, tokens, ok, temperature=t)
    assert e.value.status == g.GEMM_ERR_INVALID_ARG
    assert lib.launch_count() == n


@pytest.mark.parametrize("temperature", [4.3e-39, 8.4e-39, 1e-38])
def test_smallest_temperatures(lib, temperature):
    """the largest logits share all, the others come to nothing; rows of zeros among them"""
    t = f32(temperature)
    logits, tokens = tied_rows("f32")
    logits[3] = 0.0
    r = lib.token_logprobs(logits, tokens, top=12, entropy=True, temperature=t)
    check_forward(logits, tokens, t, 12, r)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("temperature,size", [(1e-38, 10.0), (1e-30, 3e8), (5e-39, 1.0), (1e-20, 1e30)])
@pytest.mark.parametrize("entropy", [False, True])
def test_gradient_where_g_over_t_overflows(lib, dtype, temperature, size, entropy):
    """g / T has no fp32 value; g p / T is 0 nearly everywhere, and may be in range at the largest logits.
    Equal to the formula as it rounds to the type, or off by the exponential's and the products' errors, 2^-19
    (the entropy's part is a difference of two such), and the type's own rounding."""
    t = f32(temperature)
    logits, tokens = tied_rows(dtype)
    rows = len(logits)
    r = lib.token_logprobs(logits, tokens, entropy=True, temperature=t)
    gain = torch.linspace(-1.0, 1.0, rows, device="cuda") * size
    dh = gain.flip(0) if entropy else None
    dl = lib.token_logprobs_backward(gain, logits, tokens, r, dentropy=dh, temperature=t)
    n = torch.arange(1, rows + 1, device="cuda").double()[:, None]
    p = (logits == 17.75).double() / n
    delta = torch.zeros_like(p).scatter_(1, tokens[:, None], 1.0)
    want = gain.double()[:, None] * (delta - p) / t  # (n equal ones: ln p + H = 0)
    tol = 2.0 ** -19 * (gain.double().abs()[:, None] * (delta + p) + (dh.double().abs()[:, None] * p if entropy else 0)) / t
    tol = tol + torch.finfo(dl.dtype).eps / 2 * want.abs()
    top = torch.finfo(dl.dtype).max
    got = dl.double()
    over = want.abs() - tol > top  # (no value of the type)
    assert bool(torch.where(over, got == want.sign() * math.inf, (got - want).abs() <= tol).logical_or(
        (want.abs() + tol > top) & (got == want.sign() * math.inf)).all())
    assert not bool(dl.isnan().any()) and bool((dl[p == 0][delta[p == 0] == 0] == 0).all())
