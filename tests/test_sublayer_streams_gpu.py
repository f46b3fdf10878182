"""Calls on a given stream while other streams work: what each call allocates, reads and
returns stays its own.  The given stream is held back by ordinary matrix products, so that
its kernels run after the host has gone on."""
import pytest
import torch

from hyper_connection_mix_gb300 import sublayer as sub

pytestmark = pytest.mark.gpu


@pytest.fixture
def side():
    """A stream with a few milliseconds of work ahead of whatever comes next."""
    stream = torch.cuda.Stream()
    a = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for _ in range(100):
            a = torch.mm(a, a)
    return stream


def randn(*shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def refill(kinds):
    """New allocations of the current stream of these shapes and types, overwritten."""
    return [torch.empty(shape, dtype=dtype, device="cuda").fill_(99)
            for shape, dtype in kinds for _ in range(3)]


@pytest.mark.parametrize("rows,width", [(700, 512), (4096, 5120), (64, 40000)])
@pytest.mark.parametrize("raw", [False, True])
def test_norm_backward_on_a_given_stream(side, rows, width, raw):
    dy, x = randn(rows, width, seed=1), randn(rows, width, seed=2)
    weight = randn(width, seed=3, dtype=torch.float32)
    _, mean, rstd = sub.hc_mix_layer_norm(x, weight, want_stats=True)
    want = sub.hc_mix_layer_norm_backward(dy, x, mean, rstd, weight)
    inputs = [t.clone() for t in (dy, x, mean, rstd, weight)]
    torch.cuda.synchronize()
    got = sub.hc_mix_layer_norm_backward(*inputs, stream=side.cuda_stream if raw else side)
    kinds = [(t.shape, t.dtype) for t in (*inputs, *got)]
    kinds.append((sub.layer_norm_workspace_bytes(rows, width, x.dtype), torch.uint8))
    del inputs
    kept = refill(kinds)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    del kept


def test_outputs_may_be_let_go_while_the_current_stream_reads_them(side):
    x = randn(4096, 1024, seed=1)
    others = [randn(4096, 1024, seed=5 + i) for i in range(4)]
    want = sub.hc_mix_layer_norm(x).float().sum(1)
    torch.cuda.synchronize()
    y = sub.hc_mix_layer_norm(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    a = torch.randn(4096, 4096, device="cuda")
    for _ in range(50):
        a = torch.mm(a, a)
    got = y.float().sum(1)
    del y
    for other in others:  # would be given y's memory, and write it before it is read
        sub.hc_mix_layer_norm(other, stream=side)
    assert torch.equal(got, want)


def test_the_default_stream_by_its_handle(side):
    """Handle 0 is the default stream, also where another one is current."""
    x = randn(64, 1024, seed=1)
    want = sub.hc_mix_layer_norm(x)
    with torch.cuda.stream(side):  # held back: what went there would not be done in time
        got = sub.hc_mix_layer_norm(x, stream=0)
    torch.cuda.default_stream().synchronize()
    assert torch.equal(got, want)
