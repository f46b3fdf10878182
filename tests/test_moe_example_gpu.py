"""The example's sublayer: its gradients against torch's differentiation of the same chain in 64
bits, and a training run whose loss falls."""
import importlib.util
import os

import pytest
import torch

from hyper_connection_mix_gb300 import binding

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HC = 4


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_sublayer",
                                                  os.path.join(ROOT, "examples", "moe_sublayer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(layer, x, ids, dout):
    """out and gradients in 64 bits, with the experts that the layer chose."""
    pre, post, comb = (t.double() for t in binding.hc_mix_fused(x, layer.mix, layer.hc_scale,
                                                                layer.hc_base))
    M, D = x.shape[0], layer.width
    leaf = lambda t: t.double().requires_grad_()  # noqa: E731
    xs = leaf(x)
    up, weight, bias, router = (leaf(t) for t in (layer.up, layer.weight, layer.bias, layer.router))
    streams = xs.view(M, HC, D)
    h = (pre[:, :, None] * streams).sum(1)
    n = torch.nn.functional.layer_norm(h, (D,), weight, bias, 1e-5)
    chosen = torch.softmax((n @ router).gather(1, ids), 1)
    y = sum(chosen[:, j, None] * torch.einsum("md,mde->me", n, up[ids[:, j]])
            for j in range(layer.top))
    out = (post[:, :, None] * y[:, None] + torch.matmul(comb, streams)).view(M, HC * D)
    return out, torch.autograd.grad(out, (xs, up, weight, bias, router), dout.double())


def test_gradients_of_the_sublayer(example):
    """bf16 rounds each of the chain's six intermediate rows once (2^-8 of their size each), so
    whole gradients agree to a few per cent of their norm; a wrong formula is off by its norm."""
    layer = example.Sublayer(128, 6, 2, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.randn(50, HC * 128, generator=g, device="cuda").to(torch.bfloat16)
    dout = torch.randn(50, HC * 128, generator=g, device="cuda").to(torch.bfloat16)
    out, kept = layer.forward(x, keep=True)
    got = layer.backward(dout, kept)
    want_out, want = reference(layer, x, kept[8], dout)
    assert (out.double() - want_out).norm() <= 0.02 * want_out.norm()
    for name, w in zip(("x", "up", "weight", "bias", "router"), want):
        assert (got[name].double() - w).norm() <= 0.04 * w.norm(), name


def test_training_and_serving(example):
    layer = example.Sublayer(256, 8, 2, seed=1)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn(96, HC * 256, generator=g, device="cuda").to(torch.bfloat16)
    target = torch.randn(96, HC * 256, generator=g, device="cuda")
    losses = example.train(layer, x, target, 12)
    assert losses[-1] < losses[0] and all(b < a * 1.001 for a, b in zip(losses, losses[1:]))
    one = layer.forward(x[5:6])
    whole = layer.forward(x)[5:6]
    assert (one.float() - whole.float()).abs().max() <= 2 ** -6 * whole.float().abs().max()
