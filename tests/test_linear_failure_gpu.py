"""Linear layers of which one CTA pair gives up on a wait, and what the handle does afterwards.

The test hooks let that pair wait on a barrier nothing arrives on; the wait runs out after
its limit, the pair drains and returns, and a status word is left.  Nothing faults."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture()
def g():
    import programming_tiled_gemm_gb300 as g
    return g


@pytest.fixture()
def lib(g):
    lib = g.Gemm(0)
    lib.set_option(g.GEMM_OPT_WAIT_LIMIT_US, 5000)
    yield lib
    lib.close()


def randn(seed, *shape, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def stalled(g, lib, pair, call):
    lib.set_option(g.GEMM_OPT_TEST_STALL_PAIR, pair)
    lib.set_option(g.GEMM_OPT_TEST_STALL, 1)
    call()
    lib.set_option(g.GEMM_OPT_TEST_STALL, 0)
    lib.set_option(g.GEMM_OPT_TEST_STALL_PAIR, 0)


class Groups:
    """A grouped product whose last four tiles are cut along K (one tile a group, 76 pairs).  The
    pairs that share such a tile come to it at different times: before it they have a tile
    of one row or of 256."""

    def __init__(self, seed):
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        rows = [1, 256] * (sms // 4) + [64] * 4
        self.x = randn(seed, sum(rows), 4096)
        self.other = randn(seed + 1, sum(rows), 4096)
        self.w = randn(seed + 2, len(rows), 4096, 256)
        ends = torch.tensor([0] + rows).cumsum(0)
        self.offsets = ends.to(torch.int32).cuda()
        self.cut = slice(int(ends[-5]), int(ends[-4]))  # the first of the four: pair 1 has a slice of it


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_products_after_one_that_gave_up_half_way(g, lib, out_dtype):
    """Slices count their arrivals.  Where one pair gave up and the others counted, the next launch
    is right all the same, with the status still unread."""
    s = Groups(1)
    want = lib.grouped_linear(s.x, s.w, s.offsets, out_dtype=out_dtype)
    assert lib.device_status() == g.GEMM_OK
    for pair in (1, 2, 3, 7):
        stalled(g, lib, pair, lambda: lib.grouped_linear(s.other, s.w, s.offsets, out_dtype=out_dtype))
        for _ in range(2):
            assert torch.equal(lib.grouped_linear(s.x, s.w, s.offsets, out_dtype=out_dtype), want), pair
    # (the hook did what it is there for)
    assert lib.device_status() == g.GEMM_ERR_DEVICE_TIMEOUT
    assert lib.device_status() == g.GEMM_OK
    assert torch.equal(lib.grouped_linear(s.x, s.w, s.offsets, out_dtype=out_dtype), want)


def test_replays_after_launches_that_gave_up_half_way(g, lib):
    """The same for a graph, whose launches all carry the same arguments: a replay may be the one
    that gave up."""
    s = Groups(4)
    x, y = s.x.clone(), torch.empty(s.x.shape[0], 256, device="cuda", dtype=torch.bfloat16)
    want = lib.grouped_linear(x, s.w, s.offsets, out=y).clone()
    graphs = []
    for pair in (0, 2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            if pair:
                stalled(g, lib, pair, lambda: lib.grouped_linear(x, s.w, s.offsets, out=y))
            else:
                lib.grouped_linear(x, s.w, s.offsets, out=y)
        graphs.append(graph)
    for _ in range(3):
        x.copy_(s.other)
        graphs[1].replay()
        x.copy_(s.x)
        y.zero_()
        graphs[0].replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert lib.device_status() == g.GEMM_ERR_DEVICE_TIMEOUT


def test_a_tile_with_a_slice_missing_is_not_written(g, lib):
    """Its other slices' sums are not a result."""
    s = Groups(7)
    y = lib.grouped_linear(s.x, s.w, s.offsets)
    y.fill_(3.0)
    stalled(g, lib, 1, lambda: lib.grouped_linear(s.x, s.w, s.offsets, out=y))
    assert lib.device_status() == g.GEMM_ERR_DEVICE_TIMEOUT
    assert (y[s.cut] == 3).all()
    assert (y[s.cut.stop:] != 3).any()  # the other tiles were


def test_stall_hook_refuses_other_values(g, lib):
    for v in (-1, 1025):
        assert g.gemm_set_option(lib.handle, g.GEMM_OPT_TEST_STALL_PAIR, v) == g.GEMM_ERR_INVALID_ARG


def test_status_waits_for_its_own_stream_only(g, lib):
    """The status is read and cleared in the order of the stream it is asked for: not behind work of
    the default stream, where it would also not be ordered before what that stream's caller runs next."""
    x, w = randn(31, 24, 4096), randn(32, 4096, 512)
    stream = torch.cuda.Stream()  # (does not wait for the default stream)
    torch.cuda.synchronize()
    stalled(g, lib, 1, lambda: lib.linear(x, w, stream=stream.cuda_stream))
    torch.cuda._sleep(1_000_000_000)  # half a second of the default stream
    busy = torch.cuda.Event()
    busy.record()
    assert lib.device_status(stream=stream.cuda_stream) == g.GEMM_ERR_DEVICE_TIMEOUT
    assert lib.device_status(stream=stream.cuda_stream) == g.GEMM_OK
    assert not busy.query()
    torch.cuda.synchronize()


def test_wait_limit_is_none_of_the_launch(g, lib):
    """A launch may last far longer than the limit as long as its tiles come along.  Forward: one of the
    pair's CTAs has a warp that waits for the whole launch.  Gradient of W over groups: the
    groups' last rows are waited for past every whole tile."""
    x, w = randn(41, 16384, 8192), randn(42, 8192, 16384)
    lib.set_option(g.GEMM_OPT_WAIT_LIMIT_US, 0)
    off = torch.tensor([0, 16384 - 64, 16384 - 31], dtype=torch.int32, device="cuda")
    want = lib.linear(x, w)
    _, want_dw, _ = lib.grouped_linear_backward(want, x, w.view(1, 8192, 16384).expand(2, -1, -1).contiguous(), off,
                                                need_dx=False)
    w2 = torch.empty(2, 8192, 16384, device="cuda", dtype=torch.bfloat16)
    assert lib.device_status() == g.GEMM_OK
    lib.set_option(g.GEMM_OPT_WAIT_LIMIT_US, 400)
    y = lib.linear(x, w)
    assert lib.device_status() == g.GEMM_OK
    assert torch.equal(y, want)
    _, dw, _ = lib.grouped_linear_backward(want, x, w2, off, need_dx=False)
    assert lib.device_status() == g.GEMM_OK
    assert torch.equal(dw, want_dw)
