"""One hyper-connection sublayer with a mixture of experts, from streams to streams.

    python examples/moe_sublayer.py [--rows 256] [--width 512] [--experts 16] [--top 2] [--steps 20]

Every step but the experts' own matrix products runs in the library's kernels:

    hc_mix_fused            pre, post, comb from the streams x[M, 4 * D]
    hc_mix_collapse_norm    the sublayer's normalised input
    hc_mix_expert_sort      the (token, choice) pairs by expert
    hc_mix_expert_dispatch  the tokens' rows at their experts
    (experts)               one torch matrix product for each expert
    hc_mix_expert_combine   the weighted rows back at their tokens
    hc_mix_expand           the next streams

The script trains the experts, the norm and the expert weights' scores on a fixed target for a few
steps with the gradients of each operator (pre, post and comb are taken as given: the library has no
gradient of the mix statistics), and then serves single rows with the trained weights.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from hyper_connection_mix_gb300 import binding, sublayer as sub

HC = 4


class Sublayer:
    """Parameters of one sublayer, seeded."""

    def __init__(self, width: int, experts: int, top: int, device="cuda", seed: int = 0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        rand = lambda *s, std=1.0: torch.randn(*s, generator=g, device=device) * std  # noqa: E731
        K = HC * width
        self.width, self.n_experts, self.top = width, experts, top
        self.mix = rand(24, K, std=K ** -0.5)
        self.hc_scale = torch.ones(3, device=device)
        self.hc_base = rand(24, std=0.1)
        self.router = rand(width, experts, std=width ** -0.5)
        self.weight, self.bias = torch.ones(width, device=device), torch.zeros(width, device=device)
        self.up = rand(experts, width, width, std=width ** -0.5)

    def experts(self, xs, offsets, f):
        """f(expert, its rows) for every expert that has rows; where they are is read once."""
        at = offsets.tolist()
        for e in range(self.n_experts):
            if at[e] < at[e + 1]:
                f(e, slice(at[e], at[e + 1]))

    def forward(self, x, keep: bool = False):
        """The next streams [M, 4 * width], and with `keep` what backward needs."""
        pre, post, comb = binding.hc_mix_fused(x, self.mix, self.hc_scale, self.hc_base)
        n, h, mean, rstd = sub.hc_mix_collapse_norm(x, pre, self.weight, self.bias, want_saved=True)
        scores, ids = torch.topk(n.float() @ self.router, self.top, dim=1)
        chosen = torch.softmax(scores, 1)
        offsets, slots, _ = sub.hc_mix_expert_sort(ids, self.n_experts)
        xs = sub.hc_mix_expert_dispatch(n, slots, offsets)
        ys = torch.zeros_like(xs)

        def product(e, rows):
            ys[rows] = xs[rows] @ self.up[e].to(xs.dtype)

        self.experts(xs, offsets, product)
        y = sub.hc_mix_expert_combine(ys, slots, chosen)
        out = sub.hc_mix_expand(x, y, post, comb)
        return (out, (x, pre, post, comb, h, mean, rstd, n, ids, chosen, offsets, slots, xs, ys, y)
                ) if keep else out

    def backward(self, dout, kept):
        """Gradients of x, up, weight, bias and router for the gradient of forward's result, with
        pre, post and comb held: x's lacks its way through them."""
        x, pre, post, comb, h, mean, rstd, n, ids, chosen, offsets, slots, xs, ys, y = kept
        dx, dy, _, _ = sub.hc_mix_expand_backward(dout, x, y, post, comb)
        dys, dchosen = sub.hc_mix_expert_combine_backward(dy, ys, slots, offsets, chosen)
        dup, dxs = torch.zeros_like(self.up), torch.zeros_like(xs)

        def product(e, rows):
            dup[e] = xs[rows].float().t() @ dys[rows].float()
            dxs[rows] = dys[rows] @ self.up[e].to(xs.dtype).t()

        self.experts(xs, offsets, product)
        dscores = chosen * (dchosen - (chosen * dchosen).sum(1, keepdim=True))
        dlogits = torch.zeros(x.shape[0], self.n_experts, device=x.device).scatter_(1, ids, dscores)
        drouter = n.float().t() @ dlogits
        # the norm's result went to the experts and to the router
        dn = sub.hc_mix_expert_combine(dxs, slots) + (dlogits @ self.router.t()).to(n.dtype)
        dh, dweight, dbias = sub.hc_mix_layer_norm_backward(dn, h, mean, rstd, self.weight)
        dx, _ = sub.hc_mix_collapse_backward(dh, x, pre, dx_add=dx, out=dx)
        return {"x": dx, "up": dup, "weight": dweight, "bias": dbias, "router": drouter}


def train(layer: Sublayer, x, target, steps: int, rate: float = 0.5):
    """Losses of `steps` steps of gradient descent on the mean squared error to `target`."""
    losses = []
    for _ in range(steps):
        out, kept = layer.forward(x, keep=True)
        d = out.float() - target
        losses.append(float(d.square().mean()))
        grads = layer.backward((d * (2 / layer.width)).to(out.dtype), kept)
        for name in ("up", "weight", "bias", "router"):
            getattr(layer, name).sub_(grads[name] * (rate / x.shape[0]))
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--rows", type=int, default=256)
    ap.add_argument("--width", type=int, default=512, help="of one stream, a multiple of 64")
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top", type=int, default=2)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    layer = Sublayer(a.width, a.experts, a.top)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(a.rows, HC * a.width, generator=g, device="cuda").to(torch.bfloat16)
    target = torch.randn(a.rows, HC * a.width, generator=g, device="cuda")
    losses = train(layer, x, target, a.steps)
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")
    whole = layer.forward(x)
    one = torch.cat([layer.forward(x[i:i + 1]) for i in range(4)])
    print(f"serving: rows on their own differ from the batch's by at most "
          f"{float((one.float() - whole[:4].float()).abs().max()):.3g}")


if __name__ == "__main__":
    main()
