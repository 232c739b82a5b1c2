"""A mixture-of-experts feed-forward block, forward and backward, on the library's operators.

    h   = router(x)                       moe_route: top-k experts, weights, rows sorted by expert
    xr  = x in the experts' order         moe_dispatch
    a   = swiglu(xr W1[e] + b1[e])        grouped_linear, the activation's input kept
    y   = a W2[e]                         grouped_linear, kept in fp32: the router's gradient takes
                                          differences of its products with dout
    out = x + sum_j weight_j y_j          moe_combine with the residual

    python examples/moe_block.py          # one training step, checked against 64-bit autograd
"""
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import programming_tiled_gemm_gb300 as g  # noqa: E402


class MoEBlock:
    """The block's weights on one device and its two passes.  All matrices are K x N row-major."""

    def __init__(self, lib, hidden, inner, experts, k, dtype=torch.bfloat16, seed=0):
        self.lib, self.k = lib, k
        dev = torch.device("cuda", lib.device)
        gen = torch.Generator(device=dev).manual_seed(seed)

        def init(*shape, scale):
            return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype)

        # (rows of 16-bit operands start on 16-byte boundaries: the router's are padded)
        self.wr = init(hidden, (experts + 7) // 8 * 8, scale=hidden ** -0.5)[:, :experts]
        self.w1 = init(experts, hidden, 2 * inner, scale=hidden ** -0.5)
        self.b1 = init(experts, 2 * inner, scale=0.1)
        self.w2 = init(experts, inner, hidden, scale=inner ** -0.5)

    def forward(self, x):
        """(out, what backward needs)"""
        lib = self.lib
        logits = lib.linear(x, self.wr, out_dtype=torch.float32)
        r = lib.moe_route(logits, self.k)
        xr = lib.moe_dispatch(x, r.rows, self.k)
        a, z = lib.grouped_linear(xr, self.w1, r.offsets, bias=self.b1, act="swiglu", save_preact=True)
        y = lib.grouped_linear(a, self.w2, r.offsets, out_dtype=torch.float32)
        out = lib.moe_combine(y, r.slots, r.weights, residual=x.float())
        return out.to(x.dtype), (x, logits, r, xr, z, a, y)

    def backward(self, dout, saved):
        """Gradients of x and of the weights: {"x", "wr", "w1", "b1", "w2"}."""
        lib = self.lib
        x, logits, r, xr, z, a, y = saved
        dy, dweights = lib.moe_combine_backward(dout.float(), y, r.slots, r.rows, r.weights)
        da, dw2, _ = lib.grouped_linear_backward(dy.to(x.dtype), a, self.w2, r.offsets)
        dxr, dw1, db1 = lib.grouped_linear_backward(da, xr, self.w1, r.offsets, z=z, act="swiglu", bias=True)
        T, E = logits.shape
        dlogits = x.new_empty(T, (E + 7) // 8 * 8)[:, :E]
        dlogits.copy_(lib.moe_route_backward(dweights, logits, r.experts))
        dx_router, dwr, _ = lib.linear_backward(dlogits, x, self.wr)
        # the residual's gradient is dout itself; the experts' rows come back unweighted
        dx = lib.moe_combine(dxr, r.slots, residual=dout)
        return {"x": dx + dx_router, "wr": dwr, "w1": dw1, "b1": db1, "w2": dw2}


def reference(block, x, dout, experts):
    """The same step in 64 bits with autograd, for the experts the block's router chose."""
    x, wr, w1, b1, w2 = (t.double().detach().requires_grad_() for t in (x, block.wr, block.w1, block.b1, block.w2))
    picked = experts.long()
    weights = torch.softmax((x @ wr).gather(1, picked), dim=1)
    out = x
    for e in range(block.w1.shape[0]):
        t, j = torch.nonzero(picked == e, as_tuple=True)
        gate, up = (x[t] @ w1[e] + b1[e]).chunk(2, dim=1)
        y = (torch.nn.functional.silu(gate) * up) @ w2[e]
        out = out.index_add(0, t, weights[t, j][:, None] * y)
    out.backward(dout.double())
    return out.detach(), {"x": x.grad, "wr": wr.grad, "w1": w1.grad, "b1": b1.grad, "w2": w2.grad}


def compare(tokens=300, hidden=256, inner=192, experts=8, k=2, seed=0):
    """Relative errors (2-norm) of one step against the 64-bit reference."""
    lib = g.Gemm(torch.cuda.current_device())
    block = MoEBlock(lib, hidden, inner, experts, k, seed=seed)
    gen = torch.Generator(device=block.wr.device).manual_seed(seed + 1)
    x, dout = (torch.randn(tokens, hidden, generator=gen, device=block.wr.device).bfloat16() for _ in range(2))
    out, saved = block.forward(x)
    grads = block.backward(dout, saved)
    status = lib.device_status()
    if status != g.GEMM_OK:
        raise g.GemmError(status, "moe_block")
    want_out, want = reference(block, x, dout, saved[2].experts)

    def off(got, ref):
        return float((got.double() - ref).norm() / ref.norm())

    return {"out": off(out, want_out), **{n: off(grads[n], want[n]) for n in want}}


if __name__ == "__main__":
    for name, err in compare().items():
        print("%-4s relative error %.1e" % (name, err))
