"""The debug build's index checks in the kernels of the linear layers and of the routing: silent on
every kernel's ordinary calls, and raised by slots, rows and experts that are out of range (the
access is skipped, in this build and in the release one)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

COMMON = r"""
import torch
import programming_tiled_gemm_gb300 as g
assert g.DEBUG
lib = g.Gemm(0)
gen = torch.Generator(device="cuda").manual_seed(5)
def randn(*shape):
    return torch.randn(*shape, generator=gen, device="cuda")
"""

CLEAN = COMMON + r"""
def ok(name):
    assert lib.device_status() == g.GEMM_OK, name

for dt in (torch.bfloat16, torch.float16):
    for M in (1, 2, 3, 8, 9, 200):
        for K, N in ((520, 72), (8, 1000), (2048, 264)):
            x, w, b, r = randn(M, K).to(dt), randn(K, N).to(dt), randn(N).to(dt), randn(M, N).to(dt)
            y, z = lib.linear(x, w, bias=b, act="gelu", residual=r, save_preact=True)
            lib.linear(x, w, bias=b, out_dtype=torch.float32)
            lib.linear_backward(y, x, w, z=z, act="gelu", bias=True)
            lib.linear_backward(y, x, w, z=z, act="gelu", bias=True, need_dx=False, dw_dtype=torch.float32)
            ok(("linear", M, K, N))
    x, w, off = randn(300, 2048).to(dt), randn(4, 2048, 528).to(dt), torch.tensor([0, 100, 100, 290, 300], device="cuda").int()
    for act in ("silu", "swiglu"):
        b = randn(4, 528).to(dt)
        y, z = lib.grouped_linear(x, w, off, bias=b, act=act, save_preact=True)
        lib.grouped_linear_backward(y, x, w, off, z=z, act=act, bias=True)
        lib.grouped_linear_backward(y, x, w, off, z=z, act=act, bias=True, need_dx=False)
        ok(("grouped", act))
for dt in (torch.float32, torch.bfloat16):
    for T, E, k in ((1, 5, 5), (100, 64, 4), (3000, 64, 8), (900, 700, 3)):
        l = randn(T, E).to(dt)
        l[::3] = float("-inf")
        for renormalize in (True, False):
            r = lib.moe_route(l, k, renormalize=renormalize)
            lib.moe_route_backward(randn(T, k), l, r.experts, renormalize=renormalize)
        for N in (8, 100, 2056):
            x = randn(T, N).to(dt)
            y = lib.moe_dispatch(x, r.rows, k)
            lib.moe_combine(y, r.slots, r.weights, residual=x)
            lib.moe_combine(y, r.slots)
            lib.moe_combine_backward(x, y, r.slots, r.rows, r.weights)
        ok(("routing", T, E, k))
print("clean")
"""

CAUGHT = COMMON + r"""
T, E, k, N = 12, 6, 2, 40
x, logits = randn(T, N), randn(T, E)
r = lib.moe_route(logits, k)
y = lib.moe_dispatch(x, r.rows, k)
dw = randn(T, k)
lib.moe_route_backward(dw, logits, r.experts)
lib.moe_combine_backward(x, y, r.slots, r.rows, r.weights)
lib.moe_combine(y, r.slots, r.weights)
assert lib.device_status() == g.GEMM_OK

def bad(t, v):
    t = t.clone()
    t.view(-1)[3] = v
    return t

calls = {
    "dispatch rows": lambda: lib.moe_dispatch(x, bad(r.rows, T * k), k),
    "combine slots": lambda: lib.moe_combine(y, bad(r.slots, T * k), r.weights),
    "combine gradient slots": lambda: lib.moe_combine_backward(x, y, bad(r.slots, T * k), r.rows, r.weights),
    "combine gradient rows": lambda: lib.moe_combine_backward(x, y, r.slots, bad(r.rows, T * k), r.weights),
    "route gradient experts": lambda: lib.moe_route_backward(dw, logits, bad(r.experts, E)),
}
for name, call in calls.items():
    call()
    assert lib.device_status() == g.GEMM_ERR_DEVICE_BOUNDS, name
    assert lib.device_status() == g.GEMM_OK, name
print("caught", len(calls))
"""


def child(script):
    env = dict(os.environ, GEMM_GB300_DEBUG="1", PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    p = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, env=env, cwd=ROOT, timeout=600)
    assert p.returncode == 0, p.stdout + p.stderr
    return p.stdout


def test_ordinary_calls_raise_no_check():
    assert "clean" in child(CLEAN)


def test_indices_out_of_range_are_caught():
    assert "caught 5" in child(CAUGHT)
