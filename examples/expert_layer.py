"""A mixture-of-experts layer with 8-bit experts, from router logits to the
combined output, and the router's gradient.

    python examples/expert_layer.py [tokens [hidden [width [experts [topk]]]]]

Serving: route -> plan -> quantise the tokens -> gate and up product of the rows
the plan gathers -> gated quantisation -> down product -> combine.  No token is
copied per expert: the first product reads its rows from the tokens.  Training
the router: combine_backward gives the weights' gradient, route_backward takes
it to the logits.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import combine_ep_plan_gb300 as ep  # noqa: E402


def quantize_weights(w):
    """[E,N,K] -> 8-bit codes and a scale for each output channel."""
    codes, scales = ep.quantize_int8(w.reshape(-1, w.shape[-1]))
    return codes.view(w.shape), scales.view(w.shape[:-1])


class ExpertLayer:
    """Experts w2 (silu(w1_gate x) * (w1_up x)), w1 [E, 2F, H], w2 [E, H, F]."""

    def __init__(self, w1, w2, topk, num_ranks=1, expert_alignment=1, score="softmax", bias=None):
        self.w1, self.s1 = quantize_weights(w1)
        self.w2, self.s2 = quantize_weights(w2)
        self.topk, self.score, self.bias = topk, score, bias
        self.ranks, self.align = num_ranks, expert_alignment
        self.handle = self.planned = None  # the plan, and the routing it was made from

    def _plan(self, idx):
        """The handle, planned for this routing."""
        if self.planned is not idx:
            if self.handle is None or self.handle.T != idx.shape[0]:
                self.handle = ep.plan(idx, self.ranks, self.w1.shape[0], self.align)
            else:
                self.handle.replan(idx)
            self.planned = idx
        return self.handle

    def __call__(self, x, logits):
        """x [T,H] bf16, logits [T,E] -> ([T,H] bf16, what the backward needs)."""
        idx, weights = ep.route(logits, self.topk, self.score, self.bias)
        h = self._plan(idx)
        rows = h.field("expert_offsets")[-1:]  # read on the device: no host wait
        q, qs = ep.quantize_int8(x)
        gate_up = ep.expert_matmul_int8(h, q, qs, self.w1, self.s1, gather=True)
        m, ms = ep.quantize_int8(gate_up, gated=True, num_rows=rows)
        y = ep.expert_matmul_int8(h, m, ms, self.w2, self.s2)
        return ep.combine(h, y, weights), (logits, idx, weights, y)

    def router_gradient(self, saved, grad_out):
        """The gradient of the logits of the call that `saved` is from, whichever calls came after it."""
        logits, idx, weights, y = saved
        _, grad_weights = ep.combine_backward(self._plan(idx), grad_out, y, weights)
        return ep.route_backward(logits, idx, grad_weights, self.score)


def reference(x, w1, w2, idx, weights):
    """The layer in fp32, token by token over its experts."""
    out = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
    for e in range(w1.shape[0]):
        t, k = (idx == e).nonzero(as_tuple=True)
        v = x[t].float() @ w1[e].float().t()
        gate, up = v.chunk(2, 1)
        out.index_add_(0, t, weights[t, k][:, None] * ((torch.nn.functional.silu(gate) * up) @ w2[e].float().t()))
    return out


def main(tokens=512, hidden=1024, width=512, experts=16, topk=4):
    g = torch.Generator("cuda").manual_seed(0)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(torch.bfloat16)

    w1, w2 = normal(experts, 2 * width, hidden, scale=hidden ** -0.5), normal(experts, hidden, width, scale=width ** -0.5)
    x, logits = normal(tokens, hidden), torch.randn(tokens, experts, device="cuda", generator=g)
    layer = ExpertLayer(w1, w2, topk)
    out, saved = layer(x, logits)
    grad = layer.router_gradient(saved, normal(tokens, hidden))
    layer.handle.check()
    want = reference(x, w1, w2, saved[1], saved[2])
    error = ((out.float() - want).norm() / want.norm()).item()
    print(f"{tokens} tokens, {experts} experts top-{topk}, {hidden} -> {width} -> {hidden}: relative error of 8-bit "
          f"experts {error:.4f}, |gradient of the logits| {grad.norm().item():.3f}")
    return error, grad


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:]))
