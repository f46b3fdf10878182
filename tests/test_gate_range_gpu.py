"""The gate and its gradient where 1 + exp(-g) leaves the range that a division holds (g below -87.3)
or fp32 itself (below -88.7): silu(g) is then small, but a normal number, or one that a large u makes
large.  g and u (dh) are exact, so that only the gate's own error is left; helpers and its bound,
(8 + 2 |g|) 2^-23 of silu(g), are those of test_experts_gpu.

The bound: with e = exp(-|g| / 2) off by (2 + 0.59 |g|) 2^-23 of itself, e^2 is by twice that, the
quotient by 2 steps and the four products by half a step each.  The gradient's are those of
test_gate_backward: (8 + 2 |g|) 2^-23 of du, (12 + 2 |g|) 2^-23 of dg's terms.
"""
import pytest
import torch

from hyper_connection_mix_gb300 import experts
from test_experts_gpu import BF16, F32, STEP, close, offsets_of

pytestmark = pytest.mark.gpu

INF = float("inf")
# all of them are bf16 values
G = [-180, -150, -120, -104, -100, -95, -90, -89, -88.5, -88, -87.5, -87, -86, -60, -20, -3, -0.5, 0, 0.5, 3, 20, 60, 88, 120]
U = [1.0, -1.5, 2.0 ** 60, -2.0 ** 100, 1.25 * 2.0 ** 118]


def column(values, dtype=BF16):
    return torch.tensor(values, device="cuda").to(dtype)


def check(h):
    g, u = column(G).double()[:, None], column(U).double()
    s = g / (1 + torch.exp(-g))
    close(h[:, :len(U)], s * u, (8 + 2 * g.abs()) * STEP * (s * u).abs(), "h")
    # an infinite u: the sign is g's
    last = h[:, len(U)].double()
    assert torch.equal(last[g[:, 0] < 0], torch.full_like(last[g[:, 0] < 0], -INF))
    assert torch.equal(last[g[:, 0] > 0], torch.full_like(last[g[:, 0] > 0], INF))


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("pad", [0, 1])
def test_gated_product(pad, transposed):
    """pad: rows that start on no 16 bytes."""
    K, F = 16 + pad, len(U) + 3
    xs = torch.zeros(len(G), K, dtype=BF16, device="cuda")
    xs[:, 0], xs[:, 1] = column(G), 1
    w = torch.zeros(1, 2 * F, K, dtype=BF16, device="cuda")
    w[0, :F, 0], w[0, F:, 1] = 1, column(U + [INF, 0, 0])
    w = w.transpose(1, 2).contiguous() if transposed else w
    check(experts.hc_mix_expert_product_gated(xs, w, offsets_of([len(G)]), transposed))


@pytest.mark.parametrize("apart", [False, True])
def test_gated_product_q4(apart):
    """A scale holds u; codes of 8 are zeros, and of an infinite scale no code is used but 9.  apart: one
    row an expert, else all of one."""
    F, E = len(U) + 3, len(G) if apart else 1
    xs = torch.zeros(len(G), 64, dtype=BF16, device="cuda")
    xs[:, 0], xs[:, 32:] = column(G), 1
    codes = torch.full((E, 2 * F, 32), 0x88, dtype=torch.uint8, device="cuda")
    codes[:, :F, 0], codes[:, F:, 16] = 0x89, 0x89  # k = 0 and k = 32
    scales = torch.ones(E, 2 * F, 2, dtype=BF16, device="cuda")
    scales[:, F:, 1] = column(U + [INF, 0, 0])
    check(experts.hc_mix_expert_product_q4(xs, codes, scales, offsets_of([1] * E if apart else [len(G)]), gated=True))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad", [0, 1])
def test_gate_backward(pad, dtype):
    """dh and u large, one at a time: dg and du stay in range, whatever their factors' order."""
    for size in (1.0, 2.0 ** 60, 2.0 ** 110):
        for of_dh in (False, True):
            F = len(G) + pad
            g = torch.zeros(F, dtype=dtype, device="cuda")
            g[:len(G)] = column(G, dtype)
            dh = torch.full((3, F), size if of_dh else 1.25, dtype=dtype, device="cuda")
            gu = torch.cat([g, torch.full_like(g, -1.5 if of_dh else size)]).expand(3, -1).contiguous()
            got = experts.hc_mix_expert_gate_backward(dh, gu)
            g, u, d = gu.double()[:, :F], gu.double()[:, F:], dh.double()
            q = 1 / (1 + torch.exp(-g))
            want = torch.cat([d * u * q * (1 + g * (1 - q)), d * g * q], 1)
            err = torch.cat([d * u.abs() * q * (1 + g.abs()) * (12 + 2 * g.abs()), d * g.abs() * q * (8 + 2 * g.abs())], 1)
            close(got, want, err * STEP, f"dgu, {size}")
