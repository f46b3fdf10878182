"""The experts' products at sizes where their kernels take other ways (clusters of four blocks,
many tiles, more than 2^31 elements), on given streams, from several host threads, and what is left
as it was.  Helpers and tolerances are those of test_experts_gpu."""
import threading

import pytest
import torch

from hyper_connection_mix_gb300 import experts
from test_experts_gpu import (BF16, F16, F32, NAN, chain, close, gate_of, offsets_of, product_of, quantised, randn, rows_of,
                              strided, weights)

pytestmark = pytest.mark.gpu

MANY = {"one": [16389], "few": [5000, 0, 7001, 3, 4100], "ragged": [(i * 37) % 300 for i in range(96)]}


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("counts", MANY)
@pytest.mark.parametrize("K,N", [(136, 1024), (64, 1000), (200, 2056)])
def test_many_tiles(counts, K, N, transposed):
    counts = MANY[counts]
    xs, w = rows_of(counts, K, BF16, 1), weights(len(counts), N, K, BF16, transposed)
    y, size = product_of(xs, w, counts, transposed)
    offsets = offsets_of(counts)
    close(experts.hc_mix_expert_product(xs, w, offsets, transposed), y, chain(K) * size, "ys")
    h, gu = experts.hc_mix_expert_product_gated(xs, w, offsets, transposed, want_saved=True)
    close(gu, y, chain(K) * size, "gu")
    close(h, *gate_of(y, size, K), "h")


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("counts,K,N", [([327], 5120, 4096), ([64, 1, 0, 63, 129], 2304, 2056), ([1] * 300, 264, 520),
                                        ([64 * 7] * 3 + [5], 1288, 4104)])
def test_many_tiles_of_weight_gradients(counts, K, N, transposed):
    xs, dys = rows_of(counts, K, BF16, 2), rows_of(counts, N, BF16, 3)
    got = experts.hc_mix_expert_product_weight_backward(dys, xs, offsets_of(counts), transposed)
    at = 0
    for e, n in enumerate(counts):
        x, d = xs[at:at + n].double(), dys[at:at + n].double()
        a, b = (x, d) if transposed else (d, x)
        close(got[e], a.t() @ b, chain(n) * (a.t().abs() @ b.abs()), f"dweight[{e}] of {n} rows")
        at += n


def test_rows_results_do_not_depend_on_the_others():
    """A row on its own, among few and among many: the same bits, whatever kernel takes them."""
    K, N = 520, 1032
    xs, w = randn(9000, K, dtype=BF16, seed=4), weights(1, N, K, BF16, False)
    whole = experts.hc_mix_expert_product(xs, w, offsets_of([9000]))
    for n in (1, 7, 300):
        assert torch.equal(experts.hc_mix_expert_product(xs[:n], w, offsets_of([n])), whole[:n])
    other = experts.hc_mix_expert_product(strided(xs[:300], 3), w, offsets_of([300]))
    assert torch.equal(other, whole[:300])


def test_more_than_2_to_31_elements():
    """Weights, results, gradients and codes whose offsets pass 32 bits, checked at their far ends."""
    K, N, far = 32768, 40000, slice(39900, 40000)
    w = torch.zeros(2, N, K, dtype=BF16, device="cuda")
    w[1, far] = randn(100, K, dtype=BF16, seed=5, std=K ** -0.5)
    xs = randn(5, K, dtype=BF16, seed=6)
    got = experts.hc_mix_expert_product(xs, w, offsets_of([2, 3]))
    want, size = product_of(xs, w[:, far], [2, 3], False)
    close(got[:, far], want, chain(K) * size, "ys")
    assert not got[:, :39900].any()
    dys = randn(5, N, dtype=BF16, seed=7)
    dw = experts.hc_mix_expert_product_weight_backward(dys, xs, offsets_of([2, 3]), out=w)
    assert dw is w
    a, b = dys[2:, far].double(), xs[2:].double()
    close(dw[1, far], a.t() @ b, chain(3) * (a.t().abs() @ b.abs()), "dweight")
    del w, dw, got
    xs, w = randn(70001, 16, dtype=BF16, seed=8), randn(1, 32768, 16, dtype=BF16, seed=9)
    got = experts.hc_mix_expert_product(xs, w, offsets_of([70001]))[69900:]
    want, size = product_of(xs[69900:], w, [101], False)
    close(got, want, chain(16) * size, "far rows")
    del got
    gu = torch.zeros(70001, 32768, dtype=BF16, device="cuda")
    gu[-1] = randn(32768, dtype=BF16, seed=10)
    dh = torch.ones(70001, 16384, dtype=BF16, device="cuda")
    dgu = experts.hc_mix_expert_gate_backward(dh, gu)
    assert torch.equal(dgu[-1:], experts.hc_mix_expert_gate_backward(dh[-1:], gu[-1:]))
    assert not dgu[:-1].any()
    del gu, dh, dgu
    N, K = 70000, 65536
    codes = torch.full((2, N, K // 2), 0x88, dtype=torch.uint8, device="cuda")
    scales = torch.ones(2, N, K // 128, dtype=BF16, device="cuda")
    c, s, q = quantised(1, 100, K, 128, BF16)
    codes[1, -100:], scales[1, -100:] = c[0], s[0]
    xs = randn(3, K, dtype=BF16, seed=11)
    got = experts.hc_mix_expert_product_q4(xs, codes, scales, offsets_of([1, 2]))
    want, size = product_of(xs[1:], q, [2], False)
    close(got[1:, -100:], want, chain(K) * size, "4 bits")
    assert not got[:, :-100].any() and not got[0].any()  # codes of 8 are zeros, exactly


@pytest.mark.parametrize("raw", [False, True])
def test_on_a_given_stream(raw):
    """Held back behind other work: what a call allocates, reads and returns stays its own."""
    counts, K, N = [40, 0, 333], 264, 136
    xs, w = rows_of(counts, K, BF16, 12), weights(3, N, K, BF16, False)
    offsets = offsets_of(counts)
    h, gu = experts.hc_mix_expert_product_gated(xs, w, offsets, want_saved=True)
    dxs, dw = experts.hc_mix_expert_product_backward(gu, xs, w, offsets)
    side = torch.cuda.Stream()
    a = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(60):
            a = torch.mm(a, a)
    on = side.cuda_stream if raw else side
    inputs = [t.clone() for t in (xs, w, offsets, gu)]
    side.wait_stream(torch.cuda.current_stream())
    got = experts.hc_mix_expert_product_gated(inputs[0], inputs[1], inputs[2], want_saved=True, stream=on)
    back = experts.hc_mix_expert_product_backward(inputs[3], inputs[0], inputs[1], inputs[2], stream=on)
    shapes = [(t.shape, t.dtype) for t in (*inputs, *got, *back)]
    del inputs
    kept = [torch.empty(s, dtype=d, device="cuda").fill_(99) for s, d in shapes for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    for g, x in zip((*got, *back), (h, gu, dxs, dw)):
        assert torch.equal(g, x)
    del kept


def test_host_threads():
    """Calls of different sizes and kernels from several threads at once."""
    counts, offsets = [3, 100, 0, 29], offsets_of([3, 100, 0, 29])
    cases = []
    for i, (K, N) in enumerate([(64, 128), (67, 130), (1024, 512), (2048, 66)]):
        xs, w = rows_of(counts, K, BF16, 20 + i), weights(4, N, K, BF16, False)
        cases.append((xs, w, *experts.hc_mix_expert_product_backward(
            experts.hc_mix_expert_product(xs, w, offsets), xs, w, offsets)))
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        xs, w, dxs, dw = cases[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                ys = experts.hc_mix_expert_product(xs, w, offsets)
                got = experts.hc_mix_expert_product_backward(ys, xs, w, offsets)
            torch.cuda.current_stream().synchronize()
            if not (torch.equal(got[0], dxs) and torch.equal(got[1], dw)):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong
    assert experts.hc_mix_expert_device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_memory_beside_the_operands_is_left_alone(dtype):
    """Outputs between guards, at every alignment that a type has."""
    counts, K, N = [5, 0, 70], 72, 40
    xs, w = rows_of(counts, K, dtype, 30), weights(3, N, K, dtype, False)
    R, offsets = xs.shape[0], offsets_of(counts)
    dys = rows_of(counts, N, dtype, 31)
    codes, scales, _ = quantised(3, N, 64, 32, dtype)
    calls = [((R, N), dtype, lambda o: experts.hc_mix_expert_product(xs, w, offsets, out=o)),
             ((R, N // 2), dtype, lambda o: experts.hc_mix_expert_product_gated(xs, w, offsets, out=o)),
             ((3, N, K), dtype, lambda o: experts.hc_mix_expert_product_weight_backward(dys, xs, offsets, out=o)),
             ((3, N, K), F32, lambda o: experts.hc_mix_expert_product_weight_backward(dys, xs, offsets, weight_dtype=F32, out=o)),
             ((R, N), dtype, lambda o: experts.hc_mix_expert_gate_backward(dys[:, :N // 2], dys, out=o)),
             ((R, N), dtype, lambda o: experts.hc_mix_expert_product_q4(xs[:, :64], codes, scales, offsets, out=o))]
    for shape, t, call in calls:
        n = torch.Size(shape).numel()
        want = call(torch.empty(shape, dtype=t, device="cuda"))
        for shift in (0, 1, 2, 8):
            buf = torch.full((n + 64 + shift,), NAN, dtype=t, device="cuda")
            out = buf[32 + shift:32 + shift + n].view(shape)
            call(out)
            assert torch.equal(out.nan_to_num(), want.nan_to_num())
            assert buf[:32 + shift].isnan().all() and buf[32 + shift + n:].isnan().all()


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("K,N", [(365, 1824), (1824, 365), (368, 1824)])
@pytest.mark.parametrize("every", [1, 3, 11])
def test_weight_gradients_of_experts_without_rows(K, N, every, transposed):
    """Runs of tiles that have nothing to multiply, longer than the tiles that are told ahead."""
    counts = [i % 3 + 1 if i % every == 0 else 0 for i in range(24)]
    xs, dys = rows_of(counts, K, F16, 60), rows_of(counts, N, F16, 61)
    got = experts.hc_mix_expert_product_weight_backward(dys, xs, offsets_of(counts), transposed)
    at = 0
    for e, n in enumerate(counts):
        x, d = xs[at:at + n].double(), dys[at:at + n].double()
        a, b = (x, d) if transposed else (d, x)
        close(got[e], a.t() @ b, chain(n) * (a.t().abs() @ b.abs()), f"dweight[{e}] of {n} rows")
        at += n
    assert experts.hc_mix_expert_device_status() == 0


@pytest.mark.parametrize("K,N", [(64, 24), (33, 17)])
def test_the_most_experts(K, N):
    """4096 experts, most of few rows and many of none: more of them than threads."""
    counts = [(i * 7) % 3 for i in range(4095)] + [41]
    offsets, E = offsets_of(counts), 4096
    xs, w = rows_of(counts, K, BF16, 40), weights(E, N, K, BF16, False)
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.tensor(counts, device="cuda"))
    x = xs[:expert.numel()].double()
    y, size = ((a[:, None] @ b[expert].mT).squeeze(1) for a, b in ((x, w.double()), (x.abs(), w.double().abs())))
    close(experts.hc_mix_expert_product(xs, w, offsets)[:expert.numel()], y, chain(K) * size, "ys")
    dys = rows_of(counts, N, BF16, 41)
    d = dys[:expert.numel()].double()
    dw, dsize = (torch.zeros(E, N, K, dtype=torch.float64, device="cuda").index_add(0, expert, a[:, :, None] * b[:, None])
                 for a, b in ((d, x), (d.abs(), x.abs())))
    close(experts.hc_mix_expert_product_weight_backward(dys, xs, offsets), dw, chain(41) * dsize, "dweight")
    codes, scales, q = quantised(E, N, 64, 32, BF16)
    xs = rows_of(counts, 64, BF16, 42)
    x = xs[:expert.numel()].double()
    y, size = ((a[:, None] @ b[expert].mT).squeeze(1) for a, b in ((x, q), (x.abs(), q.abs())))
    close(experts.hc_mix_expert_product_q4(xs, codes, scales, offsets)[:expert.numel()], y, chain(64) * size, "4 bits")
