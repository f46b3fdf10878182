"""The sublayer kernels at the widths where their shapes change, and at the edges of their
operands: rows at every alignment, operands that end with their buffer, outputs between guards.

Tolerances are those of test_sublayer_gpu."""
import pytest
import torch

from hyper_connection_mix_gb300 import sublayer as sub

from test_sublayer_gpu import (EPS, HC, SUM4, TYPES, U32, chain, check_norm, close, coefficients,
                               norm_backward_reference, norm_reference, randn, random_ids)

pytestmark = pytest.mark.gpu

# row bytes at which the ring kernels change shape
BYTES = [512, 1024, 4096, 10240, 20480, 40960, 81920]


def widths():
    for dtype in TYPES:
        n = torch.tensor([], dtype=dtype).element_size()
        for b in BYTES:
            for d in (-1, 0, 1, 16 // n):
                yield pytest.param(b // n + d, dtype, id=f"{b // n + d}-{str(dtype)[6:]}")


@pytest.mark.parametrize("width,dtype", list(widths()))
def test_norm_shapes(width, dtype):
    for rows in (1, 2, 7, 700):
        if rows * width > 6_000_000:
            continue
        x, dy = randn(rows, width, dtype=dtype, mean=0.3), randn(rows, width, dtype=dtype, seed=1)
        weight, bias = randn(width, seed=2, mean=1), randn(width, seed=3)
        got = sub.hc_mix_layer_norm(x, weight, bias, EPS, want_stats=True)
        check_norm(x, weight, bias, got, f"{rows}")
        back = sub.hc_mix_layer_norm_backward(dy, x, got[1], got[2], weight)
        want, err = norm_backward_reference(dy, x, got[1], got[2], weight)
        for g, w, e, name in zip(back, want, err, ("dx", "dweight", "dbias")):
            close(g, w, e, f"{rows} {name}")


@pytest.mark.parametrize("width,dtype", list(widths()))
def test_collapse_norm_shapes(width, dtype):
    for rows in (1, 3, 400):
        if rows * width > 4_000_000:
            continue
        pre, _, _ = coefficients(rows)
        x = randn(rows, HC * width, dtype=dtype)
        weight, bias = randn(width, seed=2, mean=1), randn(width, seed=3)
        y, h, mean, rstd = sub.hc_mix_collapse_norm(x, pre, weight, bias, EPS, want_saved=True)
        terms = pre.double()[:, :, None] * x.double().view(rows, HC, width)
        h64, h_err = terms.sum(1), SUM4 * terms.abs().sum(1)
        close(h, h64, h_err, f"{rows} h")
        (y64, m64, r64), (y_err, m_err, r_err) = norm_reference(h64, weight, bias)
        d = h_err + h_err.mean(1, keepdim=True)
        r = r64[:, None]
        dr = r * r * d.pow(2).mean(1, keepdim=True).sqrt()
        w = weight.double().abs()
        y_err = y_err + w * (d * (r + dr) + (h64 - m64[:, None]).abs() * dr)
        close(y, y64, y_err, f"{rows} y")
        close(mean, m64, m_err + h_err.mean(1), f"{rows} mean")
        close(rstd, r64, r_err + dr[:, 0], f"{rows} rstd")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [5, 96, 1027, 5120, 5126, 20481])
def test_rows_do_not_depend_on_the_call(width, dtype):
    """A row's result is the same bits alone and among many, wherever it stands."""
    rows = 333
    x, dy = randn(rows, HC * width, dtype=dtype), randn(rows, width, dtype=dtype, seed=1)
    pre, post, comb = coefficients(rows)
    _, h, mean, rstd = sub.hc_mix_collapse_norm(x, pre, want_saved=True)
    every = [sub.hc_mix_collapse_norm(x, pre), sub.hc_mix_layer_norm(dy),
             sub.hc_mix_layer_norm_backward(dy, h, mean, rstd)[0],
             sub.hc_mix_collapse_backward(dy, x, pre)[1],
             *sub.hc_mix_expand_backward(x, x, dy, post, comb)[2:]]
    for at in (0, 1, 170, 332):
        s = slice(at, at + 1)
        x1, dy1, pre1 = x[s].contiguous(), dy[s].contiguous(), pre[s].contiguous()
        post1, comb1 = post[s].contiguous(), comb[s].contiguous()
        one = [sub.hc_mix_collapse_norm(x1, pre1), sub.hc_mix_layer_norm(dy1),
               sub.hc_mix_layer_norm_backward(dy1, h[s].contiguous(), mean[s].contiguous(),
                                              rstd[s].contiguous())[0],
               sub.hc_mix_collapse_backward(dy1, x1, pre1)[1],
               *sub.hc_mix_expand_backward(x1, x1, dy1, post1, comb1)[2:]]
        for a, b in zip(every, one):
            assert torch.equal(a[s], b)


def placed(t, shift):
    """`t`'s values `shift` elements into a buffer that ends with them, among NaN."""
    buf = torch.full((shift + t.numel(),), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[shift:].view(t.shape)
    v.copy_(t)
    return v


def guarded(shape, dtype, shift):
    """An output `shift` elements into a buffer of sentinels, and the check of the rest."""
    n = 1
    for d in shape:
        n *= d
    buf = torch.full((shift + n + 64,), 77.0, dtype=dtype, device="cuda")

    def untouched():
        assert (buf[:shift] == 77).all() and (buf[shift + n:] == 77).all()

    return buf[shift:shift + n].view(shape), untouched


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [3, 130, 1029, 5121])
def test_every_alignment(width, dtype):
    """Operands that start at every alignment and end with their buffer; outputs between guards."""
    rows, k, E = 9, 3, 5
    pre, post, comb = coefficients(rows)
    x0, y0 = randn(rows, HC * width, dtype=dtype), randn(rows, width, dtype=dtype, seed=1)
    ids = random_ids(rows, k, E, seed=3, drop=0.2).cuda()
    offsets, slots, _ = sub.hc_mix_expert_sort(ids, E)
    weights = torch.softmax(randn(rows, k, seed=4), 1)
    ys0 = randn(rows * k, width, dtype=dtype, seed=5)
    _, mean, rstd = sub.hc_mix_layer_norm(y0, want_stats=True)

    def calls(x, y, ys, out):
        return [sub.hc_mix_layer_norm(y, out=out(rows, width)),
                sub.hc_mix_layer_norm_backward(x[:, :width], y, mean, rstd, out=out(rows, width))[0],
                sub.hc_mix_collapse(x, pre, out=out(rows, width)),
                sub.hc_mix_collapse_norm(x, pre, out=out(rows, width)),
                sub.hc_mix_collapse_backward(y, x, pre, dx_add=x, out=out(rows, HC * width))[0],
                sub.hc_mix_expand(x, y, post, comb, out=out(rows, HC * width)),
                sub.hc_mix_expand_backward(x, x, y, post, comb, out=out(rows, HC * width))[0],
                sub.hc_mix_expert_dispatch(y, slots, offsets, out=out(rows * k, width)),
                sub.hc_mix_expert_combine(ys, slots, weights, out=out(rows, width)),
                sub.hc_mix_expert_combine_backward(y, ys, slots, offsets, weights,
                                                   out=out(rows * k, width))[0]]

    # against the same values in buffers of their own: a result may differ by what the order of
    # its sums over a row does (a narrower vector adds up in another order)
    want = calls(x0, y0, ys0, lambda *s: None)
    n = torch.tensor([], dtype=dtype).element_size()
    for shift in range(1, 16 // n + 1):
        checks = []

        def out(*shape):
            t, untouched = guarded(shape, dtype, shift)
            checks.append(untouched)
            return t

        got = calls(placed(x0, shift), placed(y0, shift), placed(ys0, shift), out)
        torch.cuda.synchronize()
        for i, (g, w) in enumerate(zip(got, want)):
            if i in (2, 4, 5, 6, 7, 8, 9):  # no sum over a row: the same bits
                assert torch.equal(g, w), (i, shift)
            else:
                # two roundings of values that differ by the sums' errors
                scale = w.double().abs().max()
                u = {2: 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11, 4: U32}[n]
                tol = 2 * u * w.double().abs() + 16 * chain(width) * U32 * (scale + 1)
                assert ((g.double() - w.double()).abs() <= tol).all(), (i, shift)
        for untouched in checks:
            untouched()


@pytest.mark.parametrize("n", [1, 511, 512, 513, 2048, 2049, 40000])
@pytest.mark.parametrize("E", [1, 2, 31, 33, 1024, 1025, 4096])
def test_sort_shapes(n, E):
    g = torch.Generator()
    g.manual_seed(n)
    ids = torch.randint(-1, E, (n, 1), generator=g)
    offsets, slots, source = (t.cpu() for t in sub.hc_mix_expert_sort(ids.cuda(), E))
    flat = ids.reshape(-1)
    keyed, order = torch.sort(torch.where(flat < 0, E, flat), stable=True)
    used = int((flat >= 0).sum())
    assert torch.equal(offsets.long(), torch.searchsorted(keyed, torch.arange(E + 1)))
    assert torch.equal(source[:used].long(), order[:used]) and (source[used:] == -1).all()
    back = torch.full_like(flat, -1)
    back[order[:used]] = torch.arange(used)
    assert torch.equal(slots.reshape(-1).long(), back)


def test_sort_is_the_same_every_time():
    ids = random_ids(9000, 8, 128, seed=0, drop=0.1).cuda()
    first = sub.hc_mix_expert_sort(ids, 128)
    for _ in range(50):
        for a, b in zip(first, sub.hc_mix_expert_sort(ids, 128)):
            assert torch.equal(a, b)


def test_norm_and_experts_past_32_bits():
    """Matrices of more than 2^31 elements: the last rows are right."""
    M, D = 430000, 5120
    x = torch.zeros(M, D, dtype=torch.bfloat16, device="cuda")
    x[-33:] = randn(33, D, dtype=torch.bfloat16)
    tail = slice(M - 33, M)
    y, mean, rstd = sub.hc_mix_layer_norm(x, want_stats=True)
    few = x[tail].clone()  # x is written over below
    y1, mean1, rstd1 = sub.hc_mix_layer_norm(few, want_stats=True)
    assert torch.equal(y[tail], y1) and torch.equal(mean[tail], mean1)
    dx, _, db = sub.hc_mix_layer_norm_backward(y, x, mean, rstd, out=y)
    dx1, _, _ = sub.hc_mix_layer_norm_backward(y1, few, mean1, rstd1)
    assert torch.equal(dx[tail], dx1)
    del y, dx
    # the last rows of the experts' matrix belong to the last tokens, twice in a row
    T = M // 2
    ids = torch.arange(M, device="cuda").view(2, T).t().contiguous() // T  # both experts of each token
    offsets, slots, _ = sub.hc_mix_expert_sort(ids, 2)
    assert offsets.tolist() == [0, T, M] and int(slots[-1, 1]) == M - 1
    xs = sub.hc_mix_expert_dispatch(x[-T:], slots, offsets)
    assert torch.equal(xs[tail], x[tail]) and torch.equal(xs[T - 33:T], x[tail])
    weights = torch.full((T, 2), 0.5, device="cuda")
    back = sub.hc_mix_expert_combine(xs, slots, weights)
    assert torch.equal(back[-33:], x[tail])
    dys, dw = sub.hc_mix_expert_combine_backward(back, xs, slots, offsets, weights, out=x)
    assert torch.equal(dys[tail], back[-33:] * 0.5)
    dots = (few.double() * few.double()).sum(1)
    assert ((dw[-33:, 1].double() - dots).abs() <= chain(D) * U32 * dots).all()
