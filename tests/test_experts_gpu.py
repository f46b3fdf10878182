"""GPU parity of the experts' feed-forward network with plain 64-bit implementations.

Tolerances follow from the arithmetic, not from observed errors.  A product's n terms are exact in
fp32 (two 16-bit factors) and are added in fp32, 16 at a time: each step drops less than 2^-23 of
the running sum, which is at most sum |terms|, once for the group of 16 and once for the sum so far.
So the sum is off by at most (n / 8 + 16) 2^-23 sum |terms|; a result of a 16-bit type is rounded
once more (half a step: 2^-8, 2^-11).  The gate's exponential and division are within
(8 + 2 |g|) 2^-23 of silu(g), and |silu'| < 1.1.
"""
import pytest
import torch

from hyper_connection_mix_gb300 import experts, sublayer as sub

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
TINY = {BF16: 2.0 ** -134, F16: 2.0 ** -25, F32: 2.0 ** -149}
STEP = 2.0 ** -23
NAN = float("nan")

# rows of each expert: none, one, the tile sizes and one around them, several tiles
COUNTS = {"mixed": [0, 1, 5, 0, 300, 16, 17, 256, 257, 0], "one": [7], "none": [0, 0, 0],
          "long": [0, 1030], "many": [i % 4 for i in range(100)]}


def chain(n):
    return (n / 8 + 16) * STEP


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(*shape, dtype=F32, seed=0, std=1.0):
    return (torch.randn(*shape, generator=generator(seed), device="cuda") * std).to(dtype)


def offsets_of(counts):
    return torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)


def rows_of(counts, width, dtype, seed, tail=3, std=1.0, fill=NAN):
    """Rows of the experts, and `tail` ones behind them that hold `fill`."""
    x = randn(sum(counts) + tail, width, dtype=dtype, seed=seed, std=std)
    x[sum(counts):] = fill
    return x


def strided(t, pad, shift=0):
    """`t`'s values with rows `pad` elements further apart, `shift` elements into a buffer of NaN."""
    if pad == 0 and shift == 0:
        return t
    rows, width = t.numel() // t.shape[-1], t.shape[-1]
    buf = torch.full((shift + rows * (width + pad) + 64,), NAN, dtype=t.dtype, device="cuda")
    v = buf[shift:shift + rows * (width + pad)].view(*t.shape[:-1], width + pad)[..., :width]
    v.copy_(t)
    return v


def close(got, want, err, what):
    assert got.shape == want.shape, what
    tol = U[got.dtype] * (want.abs() + err) + TINY[got.dtype] + err
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at "
                           f"{bad.nonzero()[0].tolist()}, worst ratio "
                           f"{float(((got.double() - want).abs() / tol)[bad].max())}")


def product_of(xs, weight, counts, transposed):
    """The rows' products and the sums of their terms' sizes, in 64 bits; zeros behind the last."""
    N = weight.shape[2 if transposed else 1]
    y = torch.zeros(xs.shape[0], N, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(y)
    at = 0
    for e, n in enumerate(counts):
        w = weight[e].double()
        w = w if transposed else w.t()
        x = xs[at:at + n].double()
        y[at:at + n], size[at:at + n] = x @ w, x.abs() @ w.abs()
        at += n
    return y, size


def gate_of(y, size, K):
    """h of 64-bit (g, u), and how far an fp32 (g, u) may put it off."""
    g, u = y.chunk(2, 1)
    eg, eu = (chain(K) * s for s in size.chunk(2, 1))
    s = g * torch.sigmoid(g)
    return s * u, (1.1 * eg + s.abs() * (8 + 2 * g.abs()) * STEP) * (u.abs() + eu) + s.abs() * eu


def weights(E, N, K, dtype, transposed, seed=2):
    return randn(*((E, K, N) if transposed else (E, N, K)), dtype=dtype, seed=seed, std=K ** -0.5)


WIDTHS = [(64, 128), (8, 8), (1, 1), (200, 264), (136, 72), (1023, 1001), (67, 130), (514, 66)]


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("K,N", WIDTHS)
def test_product(K, N, dtype, transposed):
    counts = COUNTS["mixed"]
    xs, w = rows_of(counts, K, dtype, 1), weights(len(counts), N, K, dtype, transposed)
    got = experts.hc_mix_expert_product(xs, w, offsets_of(counts), transposed)
    want, size = product_of(xs, w, counts, transposed)
    close(got, want, chain(K) * size, "ys")


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("K,N", [(128, 192), (99, 35)])
def test_product_counts(counts, K, N):
    counts = COUNTS[counts]
    xs, w = rows_of(counts, K, BF16, 3), weights(len(counts), N, K, BF16, False)
    got = experts.hc_mix_expert_product(xs, w, offsets_of(counts))
    want, size = product_of(xs, w, counts, False)
    close(got, want, chain(K) * size, "ys")


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (3, 0), (0, 1), (8, 2)])
def test_product_strides(pad, shift, transposed):
    """Rows further apart and at other alignments; NaN between them."""
    counts, K, N = [3, 0, 40], 96, 80
    xs, w = rows_of(counts, K, BF16, 4), weights(3, N, K, BF16, transposed)
    want, size = product_of(xs, w, counts, transposed)
    for x in (xs, strided(xs, pad, shift)):
        for v in (w, strided(w, pad, shift)):
            got = experts.hc_mix_expert_product(x, v, offsets_of(counts), transposed)
            close(got, want, chain(K) * size, "ys")


def test_experts_further_apart():
    counts, K, N = [3, 5, 40], 64, 48
    both = weights(6, N, K, BF16, False)
    xs = rows_of(counts, K, BF16, 5)
    want, size = product_of(xs, both[::2], counts, False)
    close(experts.hc_mix_expert_product(xs, both[::2], offsets_of(counts)), want, chain(K) * size, "ys")


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("K,F", [(64, 64), (200, 136), (72, 65), (1023, 333), (33, 1), (128, 100)])
def test_gated(K, F, dtype, transposed):
    counts = COUNTS["mixed"]
    xs, w = rows_of(counts, K, dtype, 6), weights(len(counts), 2 * F, K, dtype, transposed)
    h, gu = experts.hc_mix_expert_product_gated(xs, w, offsets_of(counts), transposed, want_saved=True)
    y, size = product_of(xs, w, counts, transposed)
    close(gu, y, chain(K) * size, "gu")
    close(h, *gate_of(y, size, K), "h")
    assert torch.equal(experts.hc_mix_expert_product_gated(xs, w, offsets_of(counts), transposed), h)


def test_gate_of_large_values():
    """exp(-g) past the largest fp32, and results past neither."""
    K, F = 16, 8
    xs = torch.zeros(4, K, dtype=BF16, device="cuda")
    xs[:, 0] = torch.tensor([-300.0, -88.0, 88.0, 300.0], device="cuda")
    w = torch.zeros(1, 2 * F, K, dtype=BF16, device="cuda")
    w[:, :F, 0], w[:, F:, 0] = 1, 2 ** -10
    h = experts.hc_mix_expert_product_gated(xs, w, offsets_of([4]))
    y, size = product_of(xs, w, [4], False)
    close(h, *gate_of(y, size, K), "h")


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype,to", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("K,N", WIDTHS)
def test_weight_gradient(K, N, dtype, to, transposed):
    """Each row is a term of its own expert only: tails of 64 rows hold the next one's."""
    counts = COUNTS["mixed"]
    xs, dys = rows_of(counts, K, dtype, 7), rows_of(counts, N, dtype, 8, std=0.1)
    got = experts.hc_mix_expert_product_weight_backward(dys, xs, offsets_of(counts), transposed, to)
    assert got.dtype is to
    at = 0
    for e, n in enumerate(counts):
        x, d = xs[at:at + n].double(), dys[at:at + n].double()
        a, b = (x, d) if transposed else (d, x)
        close(got[e], a.t() @ b, chain(n) * (a.t().abs() @ b.abs()), f"dweight[{e}] of {n} rows")
        at += n


@pytest.mark.parametrize("K,N", [(128, 64), (65, 30)])
def test_an_experts_rows_reach_no_other(K, N):
    """NaN and infinities in one expert's rows, between others that share its 16 rows."""
    counts = [5, 3, 70, 2]
    xs, dys = rows_of(counts, K, BF16, 9), rows_of(counts, N, BF16, 10)
    xs[5:8], dys[5:7], dys[7:8] = NAN, float("inf"), NAN
    w = weights(4, N, K, BF16, False)
    offsets = offsets_of(counts)
    ys = experts.hc_mix_expert_product(xs, w, offsets)
    dxs, dw = experts.hc_mix_expert_product_backward(dys, xs, w, offsets)
    for t in (ys, dxs):
        assert t[5:8].isnan().all() and t[:5].isfinite().all() and t[8:].isfinite().all()
    assert dw[1].isnan().all() and dw[0].isfinite().all() and dw[2:].isfinite().all()


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("K,N", [(128, 64), (65, 30)])
def test_backward(K, N, transposed):
    """Against torch's differentiation in 64 bits."""
    counts = COUNTS["mixed"]
    xs, dys = rows_of(counts, K, BF16, 11), rows_of(counts, N, BF16, 12, std=0.1)
    w = weights(len(counts), N, K, BF16, transposed)
    dxs, dw = experts.hc_mix_expert_product_backward(dys, xs, w, offsets_of(counts), transposed)
    at = 0
    for e, n in enumerate(counts):
        x, v = xs[at:at + n].double().requires_grad_(), w[e].double().requires_grad_()
        d = dys[at:at + n].double()
        y = x @ (v if transposed else v.t())
        dx, dv = torch.autograd.grad(y, (x, v), d)
        wa = (v.t() if transposed else v).detach().abs()
        close(dxs[at:at + n], dx, chain(N) * (d.abs() @ wa), f"dxs of {e}")
        size = (x.detach().abs().t() @ d.abs()) if transposed else (d.abs().t() @ x.detach().abs())
        close(dw[e], dv, chain(n) * size, f"dweight of {e}")
        at += n
    assert not dxs[at:].any()


# ------------------------------------------------------------------------------- gate backward


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("rows,F,pad,shift", [(1, 1, 0, 0), (3, 8, 0, 0), (37, 64, 8, 0), (65, 66, 2, 0),
                                              (5, 1001, 0, 0), (130, 100, 3, 1), (0, 8, 0, 0)])
def test_gate_backward(rows, F, pad, shift, dtype):
    """Four products and the gate's factors, each within a few steps of fp32; 1 + g (1 - q) is
    the sum of 1 and a number that may be as large as |g|."""
    dh, gu = randn(rows, F, dtype=dtype, seed=13, std=0.1), randn(rows, 2 * F, dtype=dtype, seed=14, std=4.0)
    got = experts.hc_mix_expert_gate_backward(strided(dh, pad, shift), strided(gu, pad, shift))
    v = gu.double().requires_grad_()
    h = v[:, :F] / (1 + torch.exp(-v[:, :F])) * v[:, F:]
    want = torch.autograd.grad(h, v, dh.double())[0]
    g, u = gu.double().chunk(2, 1)
    q, d = torch.sigmoid(g), dh.double().abs()
    err = torch.cat([d * u.abs() * q * (1 + g.abs()) * (12 + 2 * g.abs()), d * g.abs() * q * (8 + 2 * g.abs())], 1)
    close(got, want, err * STEP, "dgu")


def test_gate_backward_against_differences():
    g, u, dh = (randn(1, 33, seed=s).double() for s in (15, 16, 17))
    got = experts.hc_mix_expert_gate_backward(dh.float(), torch.cat([g, u], 1).float()).double()
    f = lambda g, u: g / (1 + torch.exp(-g)) * u * dh  # noqa: E731
    step = 1e-5
    dg, du = (f(g + step, u) - f(g - step, u)) / (2 * step), (f(g, u + step) - f(g, u - step)) / (2 * step)
    assert (got - torch.cat([dg, du], 1)).abs().max() < 1e-5


# ------------------------------------------------------------------------------- 4 bits


def quantised(E, N, K, group, dtype, seed=18):
    codes = torch.randint(0, 256, (E, N, K // 2), generator=generator(seed), device="cuda", dtype=torch.uint8)
    scales = (torch.rand(E, N, K // group, generator=generator(seed + 1), device="cuda") * 0.1 + 0.01).to(dtype)
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(2).double() - 8
    return codes, scales, q * scales.double().repeat_interleave(group, 2)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("K,N,group", [(32, 16, 32), (64, 2, 32), (128, 40, 64), (256, 34, 128), (1280, 66, 256),
                                       (1024, 70, 32), (2112, 514, 64)])
def test_product_q4(K, N, group, dtype, gated):
    """A code less 8 is exact in the kernel, and so is its product with an input in fp32; a group's
    sum is scaled in fp32."""
    counts = [0, 1, 8, 0, 9, 33, 0]
    xs = rows_of(counts, K, dtype, 20)
    codes, scales, w = quantised(len(counts), N, K, group, dtype)
    got = experts.hc_mix_expert_product_q4(xs, codes, scales, offsets_of(counts), gated)
    y, size = product_of(xs, w, counts, False)
    if gated:
        close(got, *gate_of(y, size, K), "h")
    else:
        close(got, y, chain(K) * size, "ys")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("counts", [[9], [40], [33, 1, 64], [1000, 0, 77]])
@pytest.mark.parametrize("K,N,group,pad", [(64, 34, 32, 0), (1152, 66, 64, 3), (2304, 130, 128, 8)])
def test_product_q4_of_many_rows(K, N, group, pad, counts, dtype, gated):
    """More than eight rows an expert on average: four tiles of rows at a time, several times over."""
    xs = rows_of(counts, K, dtype, 50)
    codes, scales, w = quantised(len(counts), N, K, group, dtype)
    got = experts.hc_mix_expert_product_q4(strided(xs, pad), codes, scales, offsets_of(counts), gated)
    y, size = product_of(xs, w, counts, False)
    if gated:
        close(got, *gate_of(y, size, K), "h")
    else:
        close(got, y, chain(K) * size, "ys")
    few = experts.hc_mix_expert_product_q4(xs[:1], codes, scales, offsets_of([1] + [0] * (len(counts) - 1)), gated)
    assert torch.equal(few, got[:1])


@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (8, 4)])
def test_product_q4_strides(pad, shift):
    counts, K, N = [2, 11], 192, 48
    xs = rows_of(counts, K, BF16, 21)
    codes, scales, w = quantised(2, N, K, 64, BF16)
    got = experts.hc_mix_expert_product_q4(strided(xs, pad, shift), codes, scales, offsets_of(counts))
    y, size = product_of(xs, w, counts, False)
    close(got, y, chain(K) * size, "ys")


def test_product_q4_of_infinities():
    """The weight's sign decides, as in the formula: no code is held with an offset that an
    infinity would turn into NaN."""
    xs = torch.zeros(1, 32, dtype=F16, device="cuda")
    xs[0, 5] = float("inf")
    codes = torch.full((1, 3, 16), 0x99, dtype=torch.uint8, device="cuda")
    codes[0, 1, 2], codes[0, 2, 2] = 0x79, 0x89  # k = 5: codes 9, 7 and 8, weights 1, -1 and 0
    scales = torch.ones(1, 3, 1, dtype=F16, device="cuda")
    got = experts.hc_mix_expert_product_q4(xs, codes, scales, offsets_of([1]))[0].tolist()
    assert got[0] == float("inf") and got[1] == float("-inf") and got[2] != got[2]


# ------------------------------------------------------------------------------- together


def test_same_bits_and_graph():
    """The same call twice, into a given output, and replayed from a graph on new values."""
    counts, K, F = COUNTS["mixed"], 136, 72
    xs, w1 = rows_of(counts, K, BF16, 22), weights(len(counts), 2 * F, K, BF16, False)
    w2 = weights(len(counts), K, F, BF16, False, seed=23)
    codes, scales, _ = quantised(len(counts), 34, 64, 64, BF16)
    offsets = offsets_of(counts)

    def chain_of(x):
        h, gu = experts.hc_mix_expert_product_gated(x, w1, offsets, want_saved=True)
        y = experts.hc_mix_expert_product(h, w2, offsets)
        dh, dw2 = experts.hc_mix_expert_product_backward(y, h, w2, offsets)
        dgu = experts.hc_mix_expert_gate_backward(dh, gu)
        q = experts.hc_mix_expert_product_q4(x[:, :64], codes, scales, offsets, gated=True)
        return (h, gu, y, dw2, q, *experts.hc_mix_expert_product_backward(dgu, x, w1, offsets))

    first = chain_of(xs)
    again = chain_of(xs)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    out = torch.full_like(first[2], 5)
    assert experts.hc_mix_expert_product(first[0], w2, offsets, out=out) is out and torch.equal(out, first[2])
    held = torch.zeros_like(xs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain_of(held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = chain_of(held)
    held.copy_(xs)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, captured))
    assert experts.hc_mix_expert_device_status() == 0


@pytest.mark.parametrize("K,N", [(64, 40), (33, 7)])
def test_no_rows_and_rows_of_no_expert(K, N):
    """No rows at all; and many rows that no expert has, whose results are zero."""
    w, codes = weights(3, N, K, BF16, False), quantised(3, 40, 64, 32, BF16)
    for R in (0, 5000):
        xs, offsets = torch.full((R, K), NAN, dtype=BF16, device="cuda"), offsets_of([0, 0, 0])
        ys = experts.hc_mix_expert_product(xs, w, offsets)
        assert ys.shape == (R, N) and not ys.any()
        h, gu = experts.hc_mix_expert_product_gated(xs, weights(3, 2 * N, K, BF16, False), offsets, want_saved=True)
        assert h.shape == (R, N) and gu.shape == (R, 2 * N) and not h.any() and not gu.any()
        dxs, dw = experts.hc_mix_expert_product_backward(torch.full((R, N), NAN, dtype=BF16, device="cuda"), xs, w, offsets)
        assert dxs.shape == xs.shape and dw.shape == w.shape and not dxs.any() and not dw.any()
        q = experts.hc_mix_expert_product_q4(torch.full((R, 64), NAN, dtype=BF16, device="cuda"), *codes[:2], offsets)
        assert q.shape == (R, 40) and not q.any()


def test_offsets_out_of_range_are_safe():
    """Unspecified results, but every access within the operands."""
    K, N = 64, 48
    xs, w = randn(20, K, dtype=BF16), weights(3, N, K, BF16, False)
    codes, scales, _ = quantised(3, N, K, 32, BF16)
    for at in ([0, 5, 3, 20], [-7, 1 << 30, 4, 90], [0, 25, 26, 1 << 30], [20, 10, 5, 0]):
        offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
        experts.hc_mix_expert_product(xs, w, offsets)
        experts.hc_mix_expert_product_gated(xs, w, offsets)
        experts.hc_mix_expert_product_weight_backward(xs, xs, offsets)
        experts.hc_mix_expert_product_q4(xs, codes, scales, offsets)
        torch.cuda.synchronize()


def test_with_the_sublayer_operators():
    """From tokens to tokens: sort, dispatch, gated product, product, combine, with dropped pairs."""
    T, k, E, D, F = 50, 3, 7, 96, 40
    x = randn(T, D, dtype=BF16, seed=24)
    ids = torch.randint(-1, E, (T, k), generator=generator(25), device="cuda")
    share = torch.rand(T, k, generator=generator(26), device="cuda")
    w1, w2 = weights(E, 2 * F, D, BF16, False), weights(E, D, F, BF16, False, seed=27)
    offsets, slots, _ = sub.hc_mix_expert_sort(ids, E)
    xs = sub.hc_mix_expert_dispatch(x, slots, offsets)
    h = experts.hc_mix_expert_product_gated(xs, w1, offsets)
    y = sub.hc_mix_expert_combine(experts.hc_mix_expert_product(h, w2, offsets), slots, share)
    want = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e >= 0:
                g, u = (w1[e].double() @ x[t].double()).chunk(2)
                want[t] += share[t, j].double() * (w2[e].double() @ (g * torch.sigmoid(g) * u))
    # h and ys are rounded to bf16 on the way: 2^-8 of each, against sums of k rows
    assert (y.double() - want).norm() <= 3 * 2 ** -8 * want.norm()
