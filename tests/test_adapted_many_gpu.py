"""Tiles with more adapters than a warp has lanes, at every width that a rank is rounded to: their list is read 32 at
a time, and a block of the reduction holds four of them, one, or half of one.  Tolerances as in test_adapted_gpu.py."""
import math

import pytest
import torch

from test_adapted_gpu import BF16, F16, check, make, run

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("M,K,N,n,r,act,dtype", [
    (48, 512, 256, 48, 64, "none", BF16), (100, 256, 264, 90, 40, "silu", F16), (100, 256, 264, 90, 128, "none", BF16),
    (200, 1024, 520, 70, 72, "swiglu", BF16), (256, 512, 136, 256, 64, "none", BF16), (256, 512, 136, 256, 128, "none", F16),
    (256, 520, 1032, 200, 32, "gelu", BF16), (3000, 2048, 1024, 50, 128, "none", BF16), (900, 1024, 2048, 300, 48, "none", F16)])
def test_tiles_with_many_adapters(lib, M, K, N, n, r, act, dtype):
    s = make(M + n + r, M, K, N, n, r, dtype, act, bias=True, residual=True)
    if n >= M:  # as many as there are rows
        s["adapters"] = torch.randperm(n, device="cuda")[:M].to(torch.int32)
    got = run(lib, s, act)
    check(got, s, act)
    assert torch.equal(run(lib, s, act), got)


@pytest.mark.parametrize("r", [16, 64, 128])
def test_bad_adapters_among_many(lib, r):
    """NaN and infinities in the B of some adapters, on both sides of the 32nd: their own rows only"""
    s = make(5, 120, 512, 200, 100, r, BF16)
    s["adapters"] = torch.randperm(100, device="cuda")[torch.arange(120, device="cuda") % 100].to(torch.int32)
    clean = run(lib, s, "none")
    check(clean, s, "none")
    bad = s["adapters"][[0, 31, 32, 33, 64, 99]].long()
    b = s["b"].clone()
    b[bad, r - 1, 77] = math.nan
    b[bad[::2], 0, 199] = -math.inf
    got = run(lib, dict(s, b=b), "none")
    mine = (s["adapters"].long()[:, None] == bad[None]).any(1)
    assert torch.equal(got[~mine], clean[~mine])
    assert not bool(got[mine][:, 77].isfinite().any())
