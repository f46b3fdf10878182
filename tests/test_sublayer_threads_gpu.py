"""Two host threads that call the same kernels with different sizes, each on its own stream:
every call is launched and every result right.  The threads call the C entry points with
arguments made ahead, so that most of their time is spent inside the library at once."""
import threading

import pytest
import torch

from hyper_connection_mix_gb300 import sublayer as sub

pytestmark = pytest.mark.gpu
CALLS = 20000
BF16 = sub.TYPES[torch.bfloat16]


def together(*calls):
    """The statuses other than 0 of CALLS calls of each (function, arguments but the stream), a
    thread and a stream for each."""
    streams = [torch.cuda.Stream() for _ in calls]
    bad, start = [], threading.Barrier(len(calls))

    def work(f, args, stream):
        handle = stream.cuda_stream
        start.wait(30)
        for i in range(CALLS):
            status = f(*args, handle)
            if status:
                bad.append(status)
            if i % 512 == 0:
                stream.synchronize()

    threads = [threading.Thread(target=work, args=(*call, s)) for call, s in zip(calls, streams)]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return bad


# rows that make teams of one, of some and of all of a block's threads: less and more shared memory
@pytest.mark.parametrize("few,many", [(2280, 4000), (456, 4000)])
def test_norm(few, many):
    calls, checks = [], []
    for rows in (few, many):
        x = torch.randn(rows, 512, device="cuda").to(torch.bfloat16)
        y = torch.empty_like(x)
        calls.append((sub.lib().hc_mix_layer_norm, (x.data_ptr(), 512, BF16, rows, 512, None, None, BF16,
                                                    1e-5, y.data_ptr(), None, None)))
        checks.append((x, y))
    assert not together(*calls)
    assert all(torch.equal(y, sub.hc_mix_layer_norm(x)) for x, y in checks)


def test_norm_backward():
    calls, checks = [], []
    for rows in (1824, 5000):
        x = torch.randn(rows, 512, device="cuda").to(torch.bfloat16)
        _, mean, rstd = sub.hc_mix_layer_norm(x, want_stats=True)
        dx, dweight, dbias = (torch.empty_like(t) for t in sub.hc_mix_layer_norm_backward(x, x, mean, rstd))
        n = sub.layer_norm_workspace_bytes(rows, 512, x.dtype)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        calls.append((sub.lib().hc_mix_layer_norm_backward, (
            x.data_ptr(), 512, x.data_ptr(), 512, BF16, rows, 512, mean.data_ptr(), rstd.data_ptr(), None,
            BF16, dx.data_ptr(), dweight.data_ptr(), dbias.data_ptr(), ws.data_ptr(), n)))
        checks.append(((x, x, mean, rstd), (dx, dweight, dbias), ws))
    assert not together(*calls)
    for args, got, _ in checks:
        want = sub.hc_mix_layer_norm_backward(*args)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("few,many,experts", [(600, 20000, 1024), (600, 8000, 128), (600, 5000, 4096)])
def test_sort(few, many, experts):
    calls, checks = [], []
    for n in (few, many):
        ids = torch.randint(0, experts, (n, 1), device="cuda")
        got = [torch.empty_like(t) for t in sub.hc_mix_expert_sort(ids, experts)]
        calls.append((sub.lib().hc_mix_expert_sort,
                      (ids.data_ptr(), 8, n, 1, experts, *(t.data_ptr() for t in got))))
        checks.append((ids, got))
    assert not together(*calls)
    for ids, got in checks:
        assert all(torch.equal(a, b) for a, b in zip(got, sub.hc_mix_expert_sort(ids, experts)))
