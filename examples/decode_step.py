"""One step of a served model's tokens through the library's operators for few rows.

    h      = x + silu(x W + s_i (x A_i) B_i)          adapted_linear: every request's own adapter
    y      = h + sum_j w_j swiglu(h W1[e_j]) W2[e_j]  linear for the router's logits, then moe_layer
    logits = y W_head                                 linear, kept in fp32
    what is asked of them                             token_logprobs: given tokens, entropy, alternatives

and, for a head that is trained on the tokens' log probabilities, its gradient (token_logprobs_backward, then
linear_backward).

    python examples/decode_step.py        # one step, checked against 64 bits
"""
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import programming_tiled_gemm_gb300 as g  # noqa: E402


class DecodeStep:
    """The step's weights on one device.  All matrices are K x N row-major."""

    def __init__(self, lib, hidden, inner, experts, k, vocabulary, adapters, rank, dtype=torch.bfloat16, seed=0):
        self.lib, self.k = lib, k
        dev = torch.device("cuda", lib.device)
        gen = torch.Generator(device=dev).manual_seed(seed)

        def init(*shape, scale):
            return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype)

        def padded(n):  # (rows of 16-bit operands start on 16-byte boundaries)
            return (n + 7) // 8 * 8

        self.w = init(hidden, hidden, scale=hidden ** -0.5)
        self.a = init(adapters, hidden, rank, scale=hidden ** -0.5)
        self.b = init(adapters, rank, hidden, scale=rank ** -0.5)
        self.scales = torch.full((adapters,), 0.5, device=dev)
        self.wr = init(hidden, padded(experts), scale=hidden ** -0.5)[:, :experts]
        self.w1 = init(experts, hidden, 2 * inner, scale=hidden ** -0.5)
        self.w2 = init(experts, inner, hidden, scale=inner ** -0.5)
        self.head = init(hidden, padded(vocabulary), scale=hidden ** -0.5)[:, :vocabulary]

    def forward(self, x, adapters, tokens, top=0):
        """(h, router logits, y, logits, TokenLogprobs)"""
        lib = self.lib
        h = lib.adapted_linear(x, self.w, self.a, self.b, adapters, scales=self.scales, act="silu", residual=x)
        scores = lib.linear(h, self.wr, out_dtype=torch.float32)
        y = lib.moe_layer(h, scores, self.w1, self.w2, self.k, residual=h)
        logits = lib.linear(y, self.head, out_dtype=torch.float32)
        return h, scores, y, logits, lib.token_logprobs(logits, tokens, top=top, entropy=True)

    def head_gradient(self, y, logits, tokens, result, dlogprobs, dentropy):
        """(dy, dhead) of the tokens' log probabilities and the rows' entropy."""
        lib = self.lib
        dlogits = lib.token_logprobs_backward(dlogprobs, logits, tokens, result, dentropy=dentropy)
        wide = y.new_empty(y.shape[0], (logits.shape[1] + 7) // 8 * 8)[:, :logits.shape[1]]
        dy, dhead, _ = lib.linear_backward(wide.copy_(dlogits), y, self.head)
        return dy, dhead


def reference(step, x, adapters, tokens, given, dlogprobs, dentropy):
    """The same step in 64 bits, each part from what the library's parts before it gave (`given`)."""
    h, scores, y, logits, _ = given
    d = torch.double
    z = x.to(d) @ step.w.to(d)
    for i in range(step.a.shape[0]):
        rows = torch.nonzero(adapters == i)[:, 0]
        z[rows] += step.scales[i].to(d) * (x[rows].to(d) @ step.a[i].to(d)) @ step.b[i].to(d)
    want = {"h": x.to(d) + z * torch.sigmoid(z), "scores": h.to(d) @ step.wr.to(d)}
    top, pick = torch.topk(scores.to(d), step.k, dim=1)
    weights, out = torch.softmax(top, dim=1), h.to(d)
    for e in range(step.w1.shape[0]):
        t, j = torch.nonzero(pick == e, as_tuple=True)
        gate, up = (h[t].to(d) @ step.w1[e].to(d)).chunk(2, dim=1)
        out = out.index_add(0, t, weights[t, j][:, None] * ((gate * torch.sigmoid(gate) * up) @ step.w2[e].to(d)))
    want["y"], want["logits"] = out, y.to(d) @ step.head.to(d)
    yy, hh = y.to(d).requires_grad_(), step.head.to(d).requires_grad_()
    lp = torch.log_softmax(logits.to(d) + (yy @ hh - (yy @ hh).detach()), dim=1)
    given_lp, entropy = lp.gather(1, tokens[:, None])[:, 0], -(lp.exp() * lp).sum(1)
    ((dlogprobs.to(d) * given_lp).sum() + (dentropy.to(d) * entropy).sum()).backward()
    want.update(logprobs=given_lp.detach(), entropy=entropy.detach(), dy=yy.grad, dhead=hh.grad)
    return want


def compare(tokens=12, hidden=256, inner=192, experts=16, k=2, vocabulary=1001, adapters=5, rank=16, seed=0):
    """Relative errors (2-norm) of every part of one step against 64 bits."""
    lib = g.Gemm(torch.cuda.current_device())
    step = DecodeStep(lib, hidden, inner, experts, k, vocabulary, adapters, rank, seed=seed)
    dev = step.w.device
    gen = torch.Generator(device=dev).manual_seed(seed + 1)
    x = torch.randn(tokens, hidden, generator=gen, device=dev).bfloat16()
    ids = torch.randint(-1, adapters, (tokens,), generator=gen, device=dev).int()
    next_token = torch.randint(0, vocabulary, (tokens,), generator=gen, device=dev)
    dlogprobs, dentropy = (torch.randn(tokens, generator=gen, device=dev) for _ in range(2))
    got = step.forward(x, ids, next_token, top=5)
    h, scores, y, logits, result = got
    dy, dhead = step.head_gradient(y, logits, next_token, result, dlogprobs, dentropy)
    status = lib.device_status()
    if status != g.GEMM_OK:
        raise g.GemmError(status, "decode_step")
    want = reference(step, x, ids, next_token, got, dlogprobs, dentropy)
    have = {"h": h, "scores": scores, "y": y, "logits": logits, "logprobs": result.logprobs, "entropy": result.entropy,
            "dy": dy, "dhead": dhead}
    return {n: float((have[n].double() - want[n]).norm() / want[n].norm()) for n in have}


if __name__ == "__main__":
    for name, err in compare().items():
        print("%-8s relative error %.1e" % (name, err))
