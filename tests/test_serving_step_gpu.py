"""The operators of a served step one after the other, as a server runs them: against 64 bits, in a graph, on
another stream, and in the debug build."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import decode_step
    finally:
        sys.path.pop(0)
    return decode_step


@pytest.mark.parametrize("shape", [dict(), dict(tokens=1), dict(tokens=64, hidden=512, inner=264, experts=7, k=3),
                                   dict(tokens=5, vocabulary=50257, rank=64, adapters=40)])
def test_step_and_head_gradient(example, shape):
    """Each part against 64 bits on the part's own inputs.  In the 2-norm a rounding to bf16 is at most u = 2^-8 of what
    it rounds: h and y have two (an operand of the second product and the result), dy and dhead too; fp32 results
    none, sums of up to 512 lose 512 / 16 2^-23 of their magnitudes, 40 times their values' here at most."""
    u = 2.0 ** -8
    for name, err in example.compare(**shape).items():
        assert err < (2 * u if name in ("h", "y", "dy", "dhead") else 2e-4), (name, err)


def test_a_captured_step_replays_new_inputs(example):
    import programming_tiled_gemm_gb300 as g
    lib = g.Gemm(0)
    T, hidden, V, n = 24, 256, 1003, 6
    step = example.DecodeStep(lib, hidden, 128, 12, 2, V, n, 16)
    gen = torch.Generator(device="cuda").manual_seed(3)

    def inputs():
        return (torch.randn(T, hidden, generator=gen, device="cuda").bfloat16(),
                torch.randint(-1, n, (T,), generator=gen, device="cuda").int(),
                torch.randint(-1, V, (T,), generator=gen, device="cuda"))

    def run(x, ids, tok):
        out = step.forward(x, ids, tok, top=8)
        gain = torch.ones(T, device="cuda")
        return out + step.head_gradient(out[2], out[3], tok, out[4], gain, gain)

    def flat(r):
        return [t for v in r for t in (v if isinstance(v, tuple) else (v,))]

    static = inputs()
    run(*static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run(*static)
    side = torch.cuda.Stream()
    for _ in range(3):
        new = inputs()
        for dst, src in zip(static, new):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in flat(kept)]
        want = run(*new)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            other = run(*new)
        side.synchronize()
        for a, b, c in zip(got, flat(want), flat(other)):
            assert torch.equal(a, b) and torch.equal(b, c)
    assert lib.device_status() == g.GEMM_OK
    lib.close()


CLEAN = r"""
import torch
import programming_tiled_gemm_gb300 as g
assert g.DEBUG
lib = g.Gemm(0)
gen = torch.Generator(device="cuda").manual_seed(5)
def randn(*shape):
    return torch.randn(*shape, generator=gen, device="cuda")
def ok(name):
    assert lib.device_status() == g.GEMM_OK, name

for dt in (torch.bfloat16, torch.float16):
    for M, K, N, n, r in ((1, 64, 80, 1, 8), (5, 1000, 272, 3, 24), (40, 520, 784, 50, 16), (300, 2048, 272, 4, 64),
                          (700, 1032, 1040, 9, 128)):
        x, w, a, b = randn(M, K).to(dt), randn(K, N).to(dt), randn(n, K, r).to(dt), randn(n, r, N).to(dt)
        ids = torch.randint(-2, n + 2, (M,), generator=gen, device="cuda").int()
        for act in ("gelu", "swiglu"):
            lib.adapted_linear(x, w, a, b, ids, scales=randn(n), bias=randn(N).to(dt), act=act)
            ok(("adapted", M, K, N, act))
    for T, E, k, D, F in ((1, 3, 3, 40, 24), (16, 64, 4, 264, 136), (64, 300, 8, 72, 200), (50, 2, 1, 520, 64)):
        x, l, w1, w2 = randn(T, D).to(dt), randn(T, E), randn(E, D, 2 * F).to(dt), randn(E, F, D).to(dt)
        l[::3] = float("-inf")
        for act, w in (("swiglu", w1), ("relu", w1[:, :, :F])):
            b1, b2 = randn(E, 2 * F if act == "swiglu" else F).to(dt), randn(E, D).to(dt)
            lib.moe_layer(x, l, w, w2, k, act=act, b1=b1, b2=b2, residual=x, renormalize=False)
            ok(("layer", T, E, act))
for dt in (torch.float32, torch.bfloat16):
    for rows, V in ((1, 5), (3, 4099), (200, 1001), (2, 131073)):
        l, t = randn(rows, V).to(dt), torch.randint(-1, V + 1, (rows,), generator=gen, device="cuda")
        q = lib.token_logprobs(l, t, top=7, entropy=True)
        lib.token_logprobs_backward(randn(rows), l, t, q, dentropy=randn(rows), out=l)
        ok(("logprobs", rows, V))
print("clean")
"""


def test_debug_build_raises_no_check():
    env = dict(os.environ, GEMM_GB300_DEBUG="1", PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    p = subprocess.run([sys.executable, "-c", CLEAN], capture_output=True, text=True, env=env, cwd=ROOT, timeout=600)
    assert p.returncode == 0 and "clean" in p.stdout, p.stdout + p.stderr
