"""The handle's workspace under CUDA graphs: a graph's replays do not depend on what the handle
is used for between them, and a capture that would need more workspace is refused whole."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture()
def g():
    import programming_tiled_gemm_gb300 as g
    return g


def randn(seed, *shape, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def captured(call):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    return graph


def test_replays_after_other_operators_and_larger_calls(g):
    """A product cut along K, a gradient with db and a routing of several blocks, captured on a
    handle that has run just these; then every operator at larger sizes."""
    lib = g.Gemm(0)
    x, w = randn(1, 24, 4096), randn(2, 4096, 512)
    dy, z = randn(3, 24, 512), randn(4, 24, 512)
    logits = randn(5, 5000, 64, dtype=torch.float32)
    y = torch.empty(24, 512, device="cuda", dtype=torch.bfloat16)
    got = {}

    def linear():
        lib.linear(x, w, act="silu", out=y)

    def backward():
        got["grads"] = lib.linear_backward(dy, x, w, z=z, act="gelu", bias=True)

    def route():
        got["routing"] = lib.moe_route(logits, 4)

    want, graphs = {}, {}
    for name, call in (("y", linear), ("grads", backward), ("routing", route)):
        call()
        torch.cuda.synchronize()
        want[name] = y.clone() if name == "y" else [t.clone() for t in got[name]]
        graphs[name] = captured(call)
    # larger calls: every workspace outgrows what the graphs hold
    lib.moe_route(randn(6, 60000, 256, dtype=torch.float32), 8)
    big_x, big_w = randn(7, 4096, 2048), randn(8, 2048, 4096)
    big_y, big_z = lib.linear(big_x, big_w, act="gelu", save_preact=True)
    lib.linear(big_x[:300], big_w, out_dtype=torch.float32)
    lib.linear_backward(big_y, big_x, big_w, z=big_z, act="gelu", bias=True)
    # what the allocator hands out next may lie where outgrown buffers lay
    filler = [torch.full((1 << 20,), 7, device="cuda", dtype=torch.int32) for _ in range(64)]
    for _ in range(3):
        y.zero_()
        for name in graphs:
            graphs[name].replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want["y"])
        for name in ("grads", "routing"):
            for a, b in zip(got[name], want[name]):
                assert torch.equal(a, b)
    assert all(int(t.min()) == 7 and int(t.max()) == 7 for t in filler)
    assert lib.device_status() == 0
    lib.close()


def test_first_route_of_a_handle_leaves_products_graphs_alone(g):
    """Products and the router count arrivals in words that never move."""
    lib = g.Gemm(0)
    x, w = randn(11, 24, 4096), randn(12, 4096, 512)
    y = torch.empty(24, 512, device="cuda", dtype=torch.float32)
    want = lib.linear(x, w, out=y).clone()
    graph = captured(lambda: lib.linear(x, w, out=y))
    lib.moe_route(randn(13, 16, 64), 4)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    lib.close()


def test_capture_that_would_grow_the_workspace_is_refused(g):
    """The larger call raises; the capture goes on and its graph is right."""
    lib = g.Gemm(0)
    x, w = randn(21, 24, 4096), randn(22, 4096, 512)
    y = torch.empty(24, 512, device="cuda", dtype=torch.bfloat16)
    want = lib.linear(x, w, out=y).clone()
    logits, dy = randn(23, 5000, 64, dtype=torch.float32), randn(24, 24, 512)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        before = lib.launch_count()
        with pytest.raises(g.GemmError) as e:
            lib.moe_route(logits, 4)
        assert e.value.status == g.GEMM_ERR_CUDA and lib.launch_count() == before
        with pytest.raises(g.GemmError) as e:
            lib.linear_backward(dy, x, w, z=dy, act="silu", bias=True)
        assert e.value.status == g.GEMM_ERR_CUDA and lib.launch_count() == before
        lib.linear(x, w, out=y)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    # and the refused calls run outside
    lib.linear_backward(dy, x, w, z=dy, act="silu", bias=True)
    r = lib.moe_route(logits, 4)
    assert int(r.offsets[-1]) == 5000 * 4 and lib.device_status() == 0
    lib.close()
