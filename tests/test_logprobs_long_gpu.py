"""Token log probabilities of long rows: eight warps a CTA (more than 65536 logits of a CTA and fewer CTAs than
fill the SMs eight times), and alternatives from units over several batches (more than 32768 16-bit or 16384 fp32 logits
of a CTA).  Tolerances as in test_logprobs_gpu.py.
"""
import math

import pytest
import torch

from test_logprobs_gpu import DTYPES, check_backward, check_forward, make

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


# logits of a CTA: the row's, over as many CTAs as have two batches and fit nine an SM
LONG = [(1, 600001, "bf16"),    # 8 CTAs of 8 warps, units of 3 batches
        (2, 2100007, "f32"),    # 8 CTAs of 8 warps, units of 17 batches
        (400, 140003, "bf16"),  # 2 CTAs of 8 warps
        (700, 66001, "f16"),    # 1 CTA of 8 warps
        (700, 66001, "f32"),
        (1300, 40001, "bf16"),  # 1 CTA of 4 warps, units of 2 batches
        (1400, 20011, "f32"),
        (1250, 131072, "bf16")]  # units of 4


@pytest.mark.parametrize("rows,V,dtype", LONG)
@pytest.mark.parametrize("entropy", [False, True])
def test_long_rows(lib, rows, V, dtype, entropy):
    logits, tokens = make(rows + V, rows, V, DTYPES[dtype])
    for top in (0, 1, 20, 32):
        r = lib.token_logprobs(logits, tokens, top=top, entropy=entropy)
        check_forward(logits, tokens, 1.0, top, r)


@pytest.mark.parametrize("rows,V,dtype", [(1, 600001, "bf16"), (3, 600001, "f32"), (1300, 40001, "f16")])
def test_where_the_best_lie(lib, rows, V, dtype):
    """rising and falling rows, equal ones, a few levels, the best in one stretch, at the ends, masked elsewhere"""
    at = torch.arange(V, device="cuda")
    base, _ = make(3, 1, V, DTYPES[dtype])
    base = base[0].float()
    kinds = [at / V, -at / V, torch.zeros(V, device="cuda"), (at % 7).float(), -(at // 1000 % 5).float(),
             torch.where((at > V // 2) & (at < V // 2 + 60), 9.0 + at % 3, base),
             torch.where((at < 3) | (at >= V - 3), torch.full_like(base, 12.0), base),
             torch.where(at % 4099 == 5, base, torch.full_like(base, -math.inf)),
             torch.where(at == V - 7, base, torch.full_like(base, -math.inf)), torch.full_like(base, -math.inf)]
    for k in range(0, len(kinds), rows if rows < 4 else len(kinds)):
        mine = [kinds[(k + i) % len(kinds)] for i in range(min(rows, len(kinds)))]
        few = torch.stack(mine).to(DTYPES[dtype])
        logits = few[torch.arange(rows, device="cuda") % len(mine)]
        tokens = torch.full((rows,), V - 7, device="cuda")
        r = lib.token_logprobs(logits, tokens, top=32, entropy=True)
        check_forward(logits, tokens, 1.0, 32, r)


@pytest.mark.parametrize("rows,V,dtype", [(1, 600001, "bf16"), (2, 300007, "f32"), (700, 66001, "f16")])
def test_gradient_of_long_rows(lib, rows, V, dtype):
    logits, tokens = make(rows + V, rows, V, DTYPES[dtype])
    gen = torch.Generator(device="cuda").manual_seed(1)
    gain, dh = (torch.randn(rows, generator=gen, device="cuda") for _ in range(2))
    r = lib.token_logprobs(logits, tokens, entropy=True)
    dl = lib.token_logprobs_backward(gain, logits, tokens, r, dentropy=dh)
    check_backward(logits, tokens, 1.0, gain, dh, dl)
