"""The limits that gemm_linear_adapted's contract names, at the values themselves.  Nothing is launched: a call within
a limit is refused for what is checked after it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


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


@pytest.fixture(scope="module")
def call(g, lib):
    """gemm_linear_adapted with fields of its two structures replaced"""
    keep = [torch.zeros(n, device="cuda", dtype=BF16) for n in (12 * 64, 64 * 64, 3 * 64 * 16, 3 * 16 * 64)]
    ids = torch.zeros(12, device="cuda", dtype=torch.int32)
    x, w, a, b = keep

    def call(lin=(), **kw):
        la = g.LinearArgs(M=12, K=64, N=64, X=x.data_ptr(), ldx=64, W=w.data_ptr(), ldw=64, Y=x.data_ptr(), ldy=64,
                          dtype=g.GEMM_BF16, y_dtype=g.GEMM_BF16)
        aa = g.AdapterArgs(n=3, r=16, A=a.data_ptr(), lda=16, a_stride=64 * 16, B=b.data_ptr(), ldb=64, b_stride=16 * 64,
                           adapters=ids.data_ptr())
        for name, v in dict(lin).items():
            setattr(la, name, v)
        for name, v in kw.items():
            setattr(aa, name, v)
        n = lib.launch_count()
        rc = g.gemm_linear_adapted(lib.handle, la, aa)
        assert rc == g.GEMM_OK or lib.launch_count() == n
        return rc

    call.ids, call.keep = ids, keep
    return call


def test_row_limit(g, call):
    limit = 2 ** 31 - 2 ** 17
    off = call.ids.data_ptr() + 2  # indices off their 4-byte boundary: looked at behind the limits
    for rows in (limit + 1, limit + 2 ** 16, 2 ** 31 - 1025):
        assert call(lin=dict(M=rows), adapters=off) == g.GEMM_ERR_UNSUPPORTED, rows
    assert call(lin=dict(M=limit), adapters=off) == g.GEMM_ERR_ALIGNMENT


def test_other_limits(g, call):
    off, wide = call.ids.data_ptr() + 2, dict(a_stride=1 << 30, b_stride=1 << 30)
    assert call(lin=dict(K=16384, ldx=16384), adapters=off, **wide) == g.GEMM_ERR_ALIGNMENT
    assert call(lin=dict(K=16385, ldx=16392), adapters=off, **wide) == g.GEMM_ERR_UNSUPPORTED
    assert call(n=8192, adapters=off) == g.GEMM_ERR_ALIGNMENT
    assert call(n=8193, adapters=off) == g.GEMM_ERR_UNSUPPORTED
    assert call(r=128, lda=128, adapters=off, **wide) == g.GEMM_ERR_ALIGNMENT
    assert call(r=129, lda=136, adapters=off, **wide) == g.GEMM_ERR_UNSUPPORTED


@pytest.mark.parametrize("M,K,f32", [(3, 64, False), (3, 16400, False), (40, 20000, False), (40, 64, True), (2, 64, True)])
def test_without_adapters_it_is_the_linear_layer(g, lib, M, K, f32):
    """n = 0 and nothing else in the adapters' structure: K and types that only the layer itself takes"""
    gen = torch.Generator(device="cuda").manual_seed(K + M)
    x, w = (torch.randn(*s, generator=gen, device="cuda").to(BF16) for s in ((M, K), (K, 72)))
    out_dtype = torch.float32 if f32 else BF16
    want = lib.linear(x, w, out_dtype=out_dtype)
    got = torch.full_like(want, 3.0)
    la = g.LinearArgs(M=M, K=K, N=72, X=x.data_ptr(), ldx=K, W=w.data_ptr(), ldw=72, Y=got.data_ptr(), ldy=72,
                      dtype=g.GEMM_BF16, y_dtype=g.GEMM_F32 if f32 else g.GEMM_BF16)
    stream = torch.cuda.current_stream().cuda_stream
    assert g.gemm_linear_adapted(lib.handle, la, g.AdapterArgs(), stream) == g.GEMM_OK
    assert torch.equal(got, want)
    if not f32:  # and through the binding, with a stack of no adapters
        for r in (0, 16):
            none = torch.empty(0, K, r, device="cuda", dtype=BF16), torch.empty(0, r, 72, device="cuda", dtype=BF16)
            ids = torch.full((M,), -1, device="cuda", dtype=torch.int32)
            assert torch.equal(lib.adapted_linear(x, w, none[0], none[1], ids), want)
