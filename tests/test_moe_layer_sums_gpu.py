"""Long sums of one sign in the expert layer's products.

An MMA truncates up to 2^-23 of the partial sum it adds 16 products to: over a stretch of 4096, in four accumulators, 64
times in each, 2^-17 of the stretch in all; the stretches are added with a rounding of 2^-24 each, two a stretch.  So a
product over F is off by at most (2^-17 + (F / 2048 + 8) 2^-24) |h| |W2|, whatever F.
"""
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


def positive(seed, *shape, dt=BF16, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(*shape, generator=gen, device="cuda") * scale).to(dt)


@pytest.mark.parametrize("T", [1, 9, 40])
@pytest.mark.parametrize("F", [4096, 4100, 8192, 16392, 65536, 262144, 1 << 20])
def test_second_product(lib, T, F):
    """token t takes row t % 8 of W1 as it is: H is exact"""
    D = 72
    x = torch.zeros(T, D, device="cuda", dtype=BF16)
    x[torch.arange(T), torch.arange(T) % 8] = 1.0
    ld = (F + 7) // 8 * 8
    w1 = positive(F, 1, D, ld)[:, :, :F]
    w2 = positive(F + 1, 1, F, D, scale=F ** -0.5)
    got = lib.moe_layer(x, torch.zeros(T, 1, device="cuda"), w1, w2, 1, act="none", out_dtype=F32)
    want = w1[0, :8].double()[torch.arange(T) % 8] @ w2[0].double()
    tol = (2.0 ** -17 + (F / 2048 + 8) * 2.0 ** -24) * want
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), float(((got.double() - want).abs() / want).max())
    # rows of both signs, which cancel: the same bound on the magnitudes
    w2 = w2 * torch.where(torch.arange(F, device="cuda") % 3 == 0, -1.0, 1.0)[:, None].to(BF16)
    got = lib.moe_layer(x, torch.zeros(T, 1, device="cuda"), w1, w2, 1, act="none", out_dtype=F32)
    want = w1[0, :8].double()[torch.arange(T) % 8] @ w2[0].double()
    assert bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,act", [(5000, "swiglu"), (20000, "relu"), (262144, "swiglu")])
def test_first_product(lib, D, act, dtype):
    """several experts, gated and not; W2 passes H's columns on: the results are H, rounded once to its type"""
    T, E, k, F = 20, 6, 2, 16
    x = positive(D, T, D, dt=dtype)
    w1 = positive(D + 1, E, D, 2 * F if act == "swiglu" else F, dt=dtype, scale=2.0 / D)
    w2 = torch.zeros(E, F, D, device="cuda", dtype=dtype)
    w2[:, torch.arange(F), torch.arange(F)] = 1.0
    logits = torch.full((T, E), float("-inf"), device="cuda")
    pick = torch.arange(T, device="cuda") % E
    logits[torch.arange(T), pick] = 0.0
    got = lib.moe_layer(x, logits, w1, w2, k, act=act, out_dtype=F32)
    z = torch.stack([x[t].double() @ w1[t % E].double() for t in range(T)])
    rel = 2.0 ** -17 + (D / 2048 + 8) * 2.0 ** -24  # (every term is positive: of z itself)
    if act == "swiglu":
        gate, up = z[:, :F], z[:, F:]
        want, rel = gate * torch.sigmoid(gate) * up, 2.13 * rel + 2.0 ** -19
    else:
        want = z
    tol = want * (rel + torch.finfo(dtype).eps / 2 * (1 + rel))
    assert bool(((got[:, :F].double() - want).abs() <= tol).all())
    assert bool((got[:, F:] == 0).all())
