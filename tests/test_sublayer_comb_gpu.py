"""Which index of comb the expand operators sum over, and how the other reading is had: with
comb's two indices exchanged."""
import pytest
import torch

from hyper_connection_mix_gb300 import sublayer as sub

pytestmark = pytest.mark.gpu
M, HC, D = 5, 4, 64


def randn(*shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def test_one_weight_moves_one_stream():
    """comb with the single entry [i][j]: stream j comes out as stream i."""
    x, y, post = randn(M, HC * D, seed=1), randn(M, D, seed=2), torch.zeros(M, HC, device="cuda")
    for i in range(HC):
        for j in range(HC):
            comb = torch.zeros(M, HC, HC, device="cuda")
            comb[:, i, j] = 1
            out = sub.hc_mix_expand(x, y, post, comb).view(M, HC, D)
            assert torch.equal(out[:, i], x.view(M, HC, D)[:, j])
            assert not out[:, [k for k in range(HC) if k != i]].any()
            dx, _, _, _ = sub.hc_mix_expand_backward(x, x, y, post, comb)
            assert torch.equal(dx.view(M, HC, D)[:, j], x.view(M, HC, D)[:, i])


def test_the_sum_over_the_first_index():
    """Of small whole numbers, so that every result is exact."""
    x, y, dout = (randn(M, n, seed=s).mul(4).round() for n, s in ((HC * D, 1), (D, 2), (HC * D, 3)))
    post, comb = randn(M, HC, seed=4).mul(4).round(), randn(M, HC, HC, seed=5).mul(4).round()
    s = x.view(M, HC, D).double().requires_grad_()
    c, d = comb.double().requires_grad_(), dout.view(M, HC, D).double()
    want = torch.einsum("mij,mid->mjd", c, s) + post.double()[:, :, None] * y.double()[:, None]
    ds, dc = torch.autograd.grad(want, (s, c), d)
    turned = comb.transpose(1, 2).contiguous()
    assert torch.equal(sub.hc_mix_expand(x, y, post, turned).view(M, HC, D).double(), want.detach())
    dx, _, _, dcomb = sub.hc_mix_expand_backward(dout, x, y, post, turned)
    assert torch.equal(dx.view(M, HC, D).double(), ds)
    assert torch.equal(dcomb.transpose(1, 2).double(), dc)
