"""GPU parity of the sublayer operators with plain 64-bit implementations.

Tolerances follow from the arithmetic, not from observed errors.  With u the
unit roundoff of fp32 (2^-24) and of the output type (2^-8, 2^-11, 2^-24):

  * a result of a 16-bit type is rounded once: u_type |result|, plus half the
    type's smallest spacing;
  * a sum of n fp32 terms is formed as at least 32 chains whose results are
    added in a tree or in order, each term with one or two roundings of its
    own, so its error is at most C(n) u sum |terms| with C(n) = n / 32 + 64;
  * sums over rows run in chains of at most n / 4 with up to 1024 chains'
    results added in order: C_rows(n) = n / 4 + 1024.
"""
import pytest
import torch

from hyper_connection_mix_gb300 import binding, sublayer as sub

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
U32 = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16, torch.float32]
HC, EPS = 4, 1e-5


def chain(n):
    return n / 32 + 64


def row_chain(n):
    return n / 4 + 1024


def randn(*shape, dtype=torch.float32, seed=0, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def strided(t, pad, shift=0):
    """`t`'s values with rows `pad` elements further apart, from `shift` elements into a buffer."""
    rows, width = t.shape
    if pad == 0 and shift == 0:
        return t
    buf = torch.full((shift + rows * (width + pad),), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[shift:].view(rows, width + pad)[:, :width]
    v.copy_(t)
    return v


def close(got, want, err, what):
    """|got - want| <= the output type's rounding + err (elementwise, 64 bits)."""
    assert got.shape == want.shape, what
    u = U[got.dtype]
    tol = u * (want.abs() + err) + TINY[got.dtype] + err
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst ratio "
                           f"{float(((got.double() - want).abs() / tol)[bad].max())}")


# layouts: (row padding, elements that the first row is shifted by)
LAYOUTS = [(0, 0), (8, 8), (3, 1)]
# one element; less than a vector; odd; one past a vector, a warp and a block of vectors; the
# workload's stream; wider than the registers of a block
WIDTHS = [1, 2, 7, 8, 64, 257, 1023, 2056, 2051, 5120, 16392, 20480, 36871]


# ---------------------------------------------------------------- layer norm


def norm_reference(x, weight, bias, eps=EPS):
    """y, mean, rstd in 64 bits, and the errors that fp32 arithmetic may leave."""
    x = x.double()
    N = x.shape[1]
    mean = x.mean(1, keepdim=True)
    var = (x - mean).pow(2).mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    w = torch.ones(N, dtype=torch.float64, device="cuda") if weight is None else weight.double()
    b = torch.zeros(N, dtype=torch.float64, device="cuda") if bias is None else bias.double()
    y = (x - mean) * rstd * w + b
    c = chain(N) * U32
    mean_err = c * x.abs().mean(1, keepdim=True)
    # the variance: its own sum, the differences' roundings, and the mean's error, squared
    var_err = 2 * c * var + mean_err ** 2 + 2 * mean_err * 4 * U32 * x.abs().mean(1, keepdim=True)
    rstd_err = rstd * (var_err / (var + eps) + 4 * U32)
    y_err = w.abs() * ((mean_err + U32 * (x - mean).abs()) * (rstd + rstd_err)
                       + (x - mean).abs() * (rstd_err + 2 * U32 * rstd)) + U32 * (b.abs() + y.abs())
    return (y, mean[:, 0], rstd[:, 0]), (y_err, mean_err[:, 0], rstd_err[:, 0])


def check_norm(x, weight, bias, got, what):
    for g, w, e, name in zip(got, *norm_reference(x, weight, bias), ("y", "mean", "rstd")):
        close(g, w, e, f"{what} {name}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("rows", [1, 5, 331])
def test_layer_norm(rows, width, dtype):
    for i, (pad, shift) in enumerate(LAYOUTS):
        at = [torch.float32, dtype, torch.float32][i]
        x = strided(randn(rows, width, dtype=dtype, seed=i, mean=0.5), pad, shift)
        weight, bias = randn(width, seed=7, mean=1, dtype=at), randn(width, seed=8, dtype=at)
        check_norm(x, weight, bias, sub.hc_mix_layer_norm(x, weight, bias, EPS, want_stats=True),
                   f"{rows} {width} {dtype} layout {i}")


@pytest.mark.parametrize("width", [100, 5120, 40000])
def test_layer_norm_optional_parameters(width):
    x = randn(9, width)
    weight, bias = randn(width, seed=1, mean=1), randn(width, seed=2)
    for w, b in ((None, None), (weight, None), (None, bias)):
        check_norm(x, w, b, sub.hc_mix_layer_norm(x, w, b, EPS, want_stats=True), f"{width}")
        out = torch.empty_like(x)
        assert sub.hc_mix_layer_norm(x, w, b, EPS, out=out) is out
        check_norm(x, w, b, (out,), f"{width} out")


@pytest.mark.parametrize("width", [96, 5120, 5121, 40000])
def test_layer_norm_special_rows(width):
    """Constant rows, a large mean, the ends of the range, and NaN or infinity in one row only."""
    x = randn(8, width)
    x[0] = 3.0
    x[1] += 4096.0
    x[2] *= 1e-18
    x[3] *= 1e15
    clean = sub.hc_mix_layer_norm(x, None, None, EPS, want_stats=True)
    check_norm(x, None, None, clean, "special rows")
    assert (clean[0][0].abs() <= 3 * chain(width) * U32 / EPS ** 0.5).all()
    x[5, width // 2] = float("nan")
    x[6, -1] = float("inf")
    got = sub.hc_mix_layer_norm(x, None, None, EPS, want_stats=True)
    for g, c in zip(got, clean):
        keep = [0, 1, 2, 3, 4, 7]
        assert torch.equal(g[keep], c[keep])
        assert torch.isnan(got[0][5]).all() and torch.isnan(got[0][6]).all()


def norm_backward_reference(dy, x, mean, rstd, weight):
    dy, x, m, r = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    M, N = x.shape
    w = torch.ones(N, dtype=torch.float64, device="cuda") if weight is None else weight.double()
    xh, g = (x - m) * r, dy * w
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - c1 - xh * c2)
    c = (chain(N) + 8) * U32
    dx_err = r * (4 * U32 * (g.abs() + c1.abs() + 2 * (xh * c2).abs())
                  + c * g.abs().mean(1, keepdim=True)
                  + xh.abs() * c * (g * xh).abs().mean(1, keepdim=True))
    cr = (row_chain(M) + 8) * U32
    return ((dx, (dy * xh).sum(0), dy.sum(0)),
            (dx_err, cr * (dy * xh).abs().sum(0), cr * dy.abs().sum(0)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("rows", [1, 5, 331])
def test_layer_norm_backward(rows, width, dtype):
    for i, (pad, shift) in enumerate(LAYOUTS):
        at = [torch.float32, dtype, torch.float32][i]
        x = strided(randn(rows, width, dtype=dtype, seed=i, mean=0.5), pad, shift)
        dy = strided(randn(rows, width, dtype=dtype, seed=i + 10, std=0.1), pad, shift)
        weight = None if (width == 257 and i == 0) else randn(width, seed=7, mean=1, dtype=at)
        _, mean, rstd = sub.hc_mix_layer_norm(x, None, None, EPS, want_stats=True)
        got = sub.hc_mix_layer_norm_backward(dy, x, mean, rstd, weight)
        want, err = norm_backward_reference(dy, x, mean, rstd, weight)
        for g, w, e, name in zip(got, want, err, ("dx", "dweight", "dbias")):
            close(g, w, e, f"{rows} {width} {dtype} layout {i} {name}")
        dx = sub.hc_mix_layer_norm_backward(dy, x, mean, rstd, weight, want_params=False)
        close(dx, want[0], err[0], f"{rows} {width} {dtype} layout {i} dx alone")


@pytest.mark.parametrize("rows,width", [(4099, 64), (2500, 1000), (1031, 5120), (700, 20480)])
def test_layer_norm_backward_many_rows(rows, width):
    """More rows than blocks; the same bits twice, and with a workspace full of NaN."""
    x, dy = randn(rows, width, dtype=torch.bfloat16), randn(rows, width, dtype=torch.bfloat16, seed=1)
    weight = randn(width, seed=2, mean=1)
    _, mean, rstd = sub.hc_mix_layer_norm(x, None, None, EPS, want_stats=True)
    got = sub.hc_mix_layer_norm_backward(dy, x, mean, rstd, weight)
    want, err = norm_backward_reference(dy, x, mean, rstd, weight)
    for g, w, e, name in zip(got, want, err, ("dx", "dweight", "dbias")):
        close(g, w, e, f"{rows} {width} {name}")
    ws = torch.full((sub.layer_norm_workspace_bytes(rows, width, x.dtype),), 255,
                    dtype=torch.uint8, device="cuda")
    for g, h in zip(got, sub.hc_mix_layer_norm_backward(dy, x, mean, rstd, weight, workspace=ws)):
        assert torch.equal(g, h)


def test_layer_norm_no_rows():
    x = torch.empty(0, 300, device="cuda")
    y, mean, rstd = sub.hc_mix_layer_norm(x, want_stats=True)
    assert y.shape == (0, 300) and mean.shape == rstd.shape == (0,)
    dx, dw, db = sub.hc_mix_layer_norm_backward(x, x, mean, rstd)
    assert dx.shape == (0, 300)
    assert torch.equal(dw, torch.zeros_like(dw)) and torch.equal(db, torch.zeros_like(db))


# ---------------------------------------------------------------- streams


def coefficients(M, seed=0):
    pre = torch.sigmoid(randn(M, HC, seed=seed))
    post = 2 * torch.sigmoid(randn(M, HC, seed=seed + 1))
    comb = torch.softmax(randn(M, HC, HC, seed=seed + 2), 2)
    return pre, post, comb


def streams(x):
    return x.double().reshape(x.shape[0], HC, -1)


SUM4 = 6 * U32  # four products and their additions, each rounded


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("rows", [1, 3, 130])
def test_collapse(rows, width, dtype):
    pre, _, _ = coefficients(rows)
    for i, (pad, shift) in enumerate(LAYOUTS):
        x = strided(randn(rows, HC * width, dtype=dtype, seed=i), pad, shift)
        terms = pre.double()[:, :, None] * streams(x)
        h, h_err = terms.sum(1), SUM4 * terms.abs().sum(1)
        what = f"{rows} {width} {dtype} layout {i}"
        close(sub.hc_mix_collapse(x, pre), h, h_err, what)
        at = [torch.float32, dtype, torch.float32][i]
        weight, bias = randn(width, seed=7, mean=1, dtype=at), randn(width, seed=8, dtype=at)
        got = sub.hc_mix_collapse_norm(x, pre, weight, bias, EPS, want_saved=True)
        (y, mean, rstd), (y_err, mean_err, rstd_err) = norm_reference(h, weight, bias)
        close(got[1], h, h_err, what + " h")
        # the norm of an h that is off by d has a mean off by at most mean(d), differences by
        # d + mean(d), and an rstd off by at most rstd^2 (root mean square of those)
        d = h_err + h_err.mean(1, keepdim=True)
        r = rstd[:, None]
        dr = r * r * d.pow(2).mean(1, keepdim=True).sqrt()
        w = weight.double().abs()
        y_err = y_err + w * (d * (r + dr) + (h - mean[:, None]).abs() * dr)
        close(got[0], y, y_err, what + " y")
        close(got[2], mean, mean_err + h_err.mean(1), what + " mean")
        close(got[3], rstd, rstd_err + dr[:, 0], what + " rstd")
        assert torch.equal(sub.hc_mix_collapse_norm(x, pre, weight, bias, EPS), got[0])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("rows", [1, 3, 130])
def test_collapse_backward(rows, width, dtype):
    pre, _, _ = coefficients(rows)
    for i, (pad, shift) in enumerate(LAYOUTS):
        x = strided(randn(rows, HC * width, dtype=dtype, seed=i), pad, shift)
        dh = strided(randn(rows, width, dtype=dtype, seed=i + 5, std=0.1), pad, shift)
        add = strided(randn(rows, HC * width, dtype=dtype, seed=i + 6, std=0.1), pad, shift)
        p, g = pre.double()[:, :, None], dh.double()[:, None, :]
        want_dpre, dpre_err = (g * streams(x)).sum(2), (chain(width) * U32) * (g * streams(x)).abs().sum(2)
        for extra in (None, add):
            a = 0 if extra is None else streams(extra)
            want = (p * g + a).reshape(rows, -1)
            err = 2 * U32 * ((p * g).abs() + (0 if extra is None else a.abs())).reshape(rows, -1)
            dx, dpre = sub.hc_mix_collapse_backward(dh, x, pre, dx_add=extra)
            what = f"{rows} {width} {dtype} layout {i} add {extra is not None}"
            close(dx, want, err, what + " dx")
            close(dpre, want_dpre, dpre_err, what + " dpre")
        held = add.contiguous()
        dx2, _ = sub.hc_mix_collapse_backward(dh, x, pre, dx_add=held, out=held)
        assert dx2 is held and torch.equal(held, dx)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("rows", [1, 3, 130])
def test_expand(rows, width, dtype):
    _, post, comb = coefficients(rows)
    for i, (pad, shift) in enumerate(LAYOUTS):
        x = strided(randn(rows, HC * width, dtype=dtype, seed=i), pad, shift)
        y = strided(randn(rows, width, dtype=dtype, seed=i + 5), pad, shift)
        c, s = comb.double(), streams(x)
        p = post.double()[:, :, None] * y.double()[:, None, :]
        want = (torch.matmul(c, s) + p).reshape(rows, -1)
        err = (SUM4 + 2 * U32) * (torch.matmul(c, s.abs()) + p.abs()).reshape(rows, -1)
        out = sub.hc_mix_expand(x, y, post, comb)
        close(out, want, err, f"{rows} {width} {dtype} layout {i}")
        held = x.contiguous().clone()
        assert sub.hc_mix_expand(held, y, post, comb, out=held) is held
        assert torch.equal(held, out)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("rows", [1, 3, 130])
def test_expand_backward(rows, width, dtype):
    _, post, comb = coefficients(rows)
    for i, (pad, shift) in enumerate(LAYOUTS):
        x = strided(randn(rows, HC * width, dtype=dtype, seed=i), pad, shift)
        y = strided(randn(rows, width, dtype=dtype, seed=i + 5), pad, shift)
        dout = strided(randn(rows, HC * width, dtype=dtype, seed=i + 6, std=0.1), pad, shift)
        c, p, d, s = comb.double(), post.double()[:, :, None], streams(dout), streams(x)
        yd = y.double()[:, None, :]
        cs = chain(width) * U32
        want = (torch.matmul(c.transpose(1, 2), d).reshape(rows, -1), (p * d).sum(1),
                (d * yd).sum(2), torch.matmul(d, s.transpose(1, 2)))
        err = (SUM4 * torch.matmul(c.transpose(1, 2), d.abs()).reshape(rows, -1),
               SUM4 * (p * d).abs().sum(1), cs * (d * yd).abs().sum(2),
               cs * torch.matmul(d.abs(), s.abs().transpose(1, 2)))
        got = sub.hc_mix_expand_backward(dout, x, y, post, comb)
        for g, w, e, name in zip(got, want, err, ("dx", "dy", "dpost", "dcomb")):
            close(g, w, e, f"{rows} {width} {dtype} layout {i} {name}")
        held = dout.contiguous().clone()
        again = sub.hc_mix_expand_backward(held, x, y, post, comb, out=held)
        assert all(torch.equal(a, b) for a, b in zip(again, got))


def test_streams_no_rows():
    x, c = torch.empty(0, 4 * 96, device="cuda"), coefficients(0)
    y = torch.empty(0, 96, device="cuda")
    assert sub.hc_mix_collapse(x, c[0]).shape == (0, 96)
    assert sub.hc_mix_collapse_norm(x, c[0], want_saved=True)[0].shape == (0, 96)
    assert sub.hc_mix_expand(x, y, c[1], c[2]).shape == x.shape
    assert sub.hc_mix_collapse_backward(y, x, c[0])[1].shape == (0, 4)
    assert sub.hc_mix_expand_backward(x, x, y, c[1], c[2])[3].shape == (0, 4, 4)


@pytest.mark.parametrize("width", [640, 643])
def test_streams_special_values(width):
    """A NaN or infinity reaches its own row and column only (dots: its own row)."""
    x, y = randn(6, HC * width, dtype=torch.bfloat16), randn(6, width, dtype=torch.bfloat16)
    pre, post, comb = coefficients(6)
    x[2, width + 5] = float("nan")
    y[4, 9] = float("inf")
    out = sub.hc_mix_expand(x, y, post, comb).view(6, HC, width)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[2, :, 5] = True
    want[4, :, 9] = True
    assert torch.equal(bad, want)
    assert torch.equal(~torch.isfinite(sub.hc_mix_collapse(x, pre)).all(1),
                       torch.tensor([False, False, True, False, False, False], device="cuda"))


def test_offsets_past_32_bits():
    """Streams of more than 2^32 bytes and 2^31 elements: the last rows are right."""
    M, D = 110000, 5120
    x = torch.empty(M, HC * D, dtype=torch.bfloat16, device="cuda")
    x[-64:] = randn(64, HC * D, dtype=torch.bfloat16)
    x[:-64] = 0
    pre, post, comb = coefficients(M)
    y = torch.zeros(M, D, dtype=torch.bfloat16, device="cuda")
    y[-64:] = randn(64, D, dtype=torch.bfloat16, seed=3)
    tail = slice(M - 64, M)
    few = [t[tail].contiguous() for t in (x, y, pre, post, comb)]
    assert torch.equal(sub.hc_mix_collapse(x, pre)[tail], sub.hc_mix_collapse(few[0], few[2]))
    assert torch.equal(sub.hc_mix_collapse_norm(x, pre)[tail],
                       sub.hc_mix_collapse_norm(few[0], few[2]))
    assert torch.equal(sub.hc_mix_expand(x, y, post, comb)[tail],
                       sub.hc_mix_expand(few[0], few[1], few[3], few[4]))
    dx, dpre = sub.hc_mix_collapse_backward(y, x, pre)
    dx1, dpre1 = sub.hc_mix_collapse_backward(few[1], few[0], few[2])
    assert torch.equal(dx[tail], dx1) and torch.equal(dpre[tail], dpre1)
    got = sub.hc_mix_expand_backward(x, x, y, post, comb, out=dx)
    for g, h in zip(got, sub.hc_mix_expand_backward(few[0], few[0], few[1], few[3], few[4])):
        assert torch.equal(g[tail], h)


# ---------------------------------------------------------------- experts


def sort_reference(ids, E):
    flat = ids.reshape(-1).tolist()
    lists = [[] for _ in range(E)]
    for pair, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(pair)
    offsets = [0]
    for pairs in lists:
        offsets.append(offsets[-1] + len(pairs))
    source = [p for pairs in lists for p in pairs]
    slots = [-1] * len(flat)
    for row, p in enumerate(source):
        slots[p] = row
    source += [-1] * (len(flat) - len(source))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return i32(offsets), i32(slots).view(ids.shape), i32(source)


def random_ids(T, k, E, seed, drop=0.0, dtype=torch.int64):
    g = torch.Generator()
    g.manual_seed(seed)
    popular = torch.randn(E, generator=g)
    ids = torch.topk(torch.randn(T, E, generator=g) + popular, min(k, E), dim=1).indices
    if ids.shape[1] < k:
        ids = torch.cat([ids, ids[:, : k - ids.shape[1]]], 1)
    if drop:
        off = torch.rand(T, k, generator=g) < drop
        ids[off] = torch.tensor([-1, E, -(2 ** 31), 2 ** 31 - 1])[torch.randint(0, 4, (int(off.sum()),), generator=g)]
    return ids.to(dtype)


SORTS = [(1, 1, 1), (1, 8, 128), (16, 8, 128), (33, 3, 61), (511, 8, 64), (513, 8, 64),
         (1531, 3, 61), (4096, 8, 128), (4097, 7, 509), (700, 2, 1025), (2000, 4, 4096),
         (20000, 1, 2), (30011, 6, 257)]


@pytest.mark.parametrize("T,k,E", SORTS)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
def test_expert_sort(T, k, E, dtype, drop):
    ids = random_ids(T, k, E, seed=T + k, drop=drop, dtype=dtype)
    for g, w in zip(sub.hc_mix_expert_sort(ids.cuda(), E), sort_reference(ids, E)):
        assert torch.equal(g.cpu(), w)


def test_expert_sort_wide_ids_and_one_expert():
    """Ids beyond 32 bits name no expert; all pairs of one expert keep their order."""
    ids = torch.tensor([[2 ** 32, 1], [0, 2 ** 40 + 1], [-(2 ** 32), 2 ** 63 - 1]])
    for g, w in zip(sub.hc_mix_expert_sort(ids.cuda(), 2), sort_reference(ids, 2)):
        assert torch.equal(g.cpu(), w)
    ids = torch.full((9000, 2), 5)
    offsets, slots, source = sub.hc_mix_expert_sort(ids.cuda(), 7)
    assert torch.equal(source.cpu(), torch.arange(18000, dtype=torch.int32))
    assert offsets.tolist() == [0] * 6 + [18000] * 2


@pytest.mark.parametrize("T,k", [(0, 4), (5, 0)])
def test_expert_no_pairs(T, k):
    offsets, slots, source = sub.hc_mix_expert_sort(torch.empty(T, k, dtype=torch.int64, device="cuda"), 6)
    assert offsets.tolist() == [0] * 7 and slots.shape == (T, k) and source.shape == (0,)
    x = randn(T, 40)
    xs = sub.hc_mix_expert_dispatch(x, slots, offsets)
    assert xs.shape == (0, 40)
    y = sub.hc_mix_expert_combine(xs, slots, torch.ones(T, k, device="cuda"))
    assert torch.equal(y, torch.zeros(T, 40, device="cuda"))
    rows = randn(3, 40)  # rows without a pair
    dys, dw = sub.hc_mix_expert_combine_backward(x, rows, slots, offsets, torch.ones(T, k, device="cuda"))
    assert torch.equal(dys, torch.zeros_like(rows)) and dw.shape == (T, k)


EXPERTS = [(1, 1, 4, 0.0), (16, 8, 128, 0.0), (61, 3, 5, 0.3), (333, 8, 40, 0.05), (50, 2, 3, 1.0),
           (20, 17, 33, 0.1)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [1, 7, 64, 1023, 2056, 5120, 9001])
@pytest.mark.parametrize("T,k,E,drop", EXPERTS)
def test_expert_rows(T, k, E, drop, width, dtype):
    ids = random_ids(T, k, E, seed=T, drop=drop).cuda()
    offsets, slots, source = sub.hc_mix_expert_sort(ids, E)
    used = int(offsets[-1])
    held, at = slots >= 0, slots.clamp(min=0).long()
    weights = torch.softmax(randn(T, k, seed=1), 1)
    w64 = torch.where(held, weights.double(), 0.0)
    for i, (pad, shift) in enumerate(LAYOUTS):
        what = f"{T} {k} {E} {width} {dtype} layout {i}"
        x = strided(randn(T, width, dtype=dtype, seed=i), pad, shift)
        xs = sub.hc_mix_expert_dispatch(x, slots, offsets)
        want = torch.zeros_like(xs)
        want[:used] = x[source[:used].long() // k]
        assert torch.equal(xs, want), what
        ys = randn(T * k, width, dtype=dtype, seed=i + 3)
        ys[used:] = float("nan")  # rows that no pair names are not read
        ys = strided(ys, pad, shift)
        rows = torch.where(held[:, :, None], ys.double()[at], 0.0)
        terms = rows * w64[:, :, None]
        close(sub.hc_mix_expert_combine(ys, slots, weights), terms.sum(1),
              (k + 2) * U32 * terms.abs().sum(1), what + " combine")
        close(sub.hc_mix_expert_combine(ys, slots), rows.sum(1), (k + 2) * U32 * rows.abs().sum(1),
              what + " combine of ones")
        dy = strided(randn(T, width, dtype=dtype, seed=i + 4, std=0.1), pad, shift)
        dys, dw = sub.hc_mix_expert_combine_backward(dy, ys, slots, offsets, weights)
        want = torch.zeros(T * k, width, dtype=torch.float64, device="cuda")
        pairs = (w64[:, :, None] * dy.double()[:, None, :]).reshape(T * k, width)
        want[slots.reshape(-1)[held.reshape(-1)].long()] = pairs[held.reshape(-1)]
        close(dys, want, U32 * want.abs(), what + " dys")
        dots = rows * dy.double()[:, None, :]
        close(dw, dots.sum(2), chain(width) * U32 * dots.abs().sum(2), what + " dweights")


def test_expert_slots_outside_are_dropped():
    """Slots that are no rows (a caller's own, or stale ones) are not followed."""
    slots = torch.tensor([[0, 7], [-5, 1], [2 ** 31 - 1, -1]], dtype=torch.int32, device="cuda")
    x, ones = randn(3, 64), torch.ones(3, 2, device="cuda")
    xs = sub.hc_mix_expert_dispatch(x, slots, out=torch.full((6, 64), 9.0, device="cuda"))
    assert torch.equal(xs[:2], x[:2]) and (xs[2:] == 9).all()
    y = sub.hc_mix_expert_combine(xs, slots, ones)
    assert torch.equal(y, torch.cat([x[:2], torch.zeros(1, 64, device="cuda")]))
    keep = torch.full((6, 64), 5.0, device="cuda")
    dys, dw = sub.hc_mix_expert_combine_backward(x, xs, slots, None, ones, out=keep)
    assert torch.equal(dys[:2], x[:2]) and (dys[2:] == 5).all()
    assert (dw[0, 1], dw[1, 0], dw[2, 0], dw[2, 1]) == (0, 0, 0, 0)
    # offsets beyond the rows leave no tail; negative ones make every row tail
    far = torch.tensor([0, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    assert torch.equal(sub.hc_mix_expert_dispatch(x, slots, far)[:2], x[:2])


# ---------------------------------------------------------------- gradients by differences


def test_gradients_by_differences():
    """The whole chain's gradient against central differences of its own forward pass.

    L = <r, out> for a random r, moved by h along a random direction of every input.  In fp32
    with values of order one the forward pass is good to about 1e-6 of sum |r out| terms; the
    difference divides that by 2 h, and its cubic term is h^2 times third derivatives of order
    one: with h = 1e-2 both stay below 1e-3 of the scale |r| |out|, which is the tolerance."""
    T, k, E, D, h = 24, 2, 5, 96, 1e-2
    x, (pre, post, comb) = randn(T, HC * D), coefficients(T)
    weight, bias, weights = randn(D, seed=5, mean=1), randn(D, seed=6), torch.softmax(randn(T, k, seed=7), 1)
    offsets, slots, _ = sub.hc_mix_expert_sort(random_ids(T, k, E, seed=9, drop=0.1).cuda(), E)

    def forward(x, pre, post, comb, weight, bias, weights):
        n, hh, mean, rstd = sub.hc_mix_collapse_norm(x, pre, weight, bias, EPS, want_saved=True)
        xs = sub.hc_mix_expert_dispatch(n, slots, offsets)
        ys = xs * xs  # the experts' own work, with its gradient 2 xs
        y = sub.hc_mix_expert_combine(ys, slots, weights)
        return sub.hc_mix_expand(x, y, post, comb), (hh, mean, rstd, xs, ys, y)

    inputs = [x, pre, post, comb, weight, bias, weights]
    out, (hh, mean, rstd, xs, ys, y) = forward(*inputs)
    r = randn(T, HC * D, seed=11)
    dx, dy, dpost, dcomb = sub.hc_mix_expand_backward(r, x, y, post, comb)
    dys, dweights = sub.hc_mix_expert_combine_backward(dy, ys, slots, offsets, weights)
    dn = sub.hc_mix_expert_combine(2 * xs * dys, slots)
    dh, dweight, dbias = sub.hc_mix_layer_norm_backward(dn, hh, mean, rstd, weight)
    dx, dpre = sub.hc_mix_collapse_backward(dh, x, pre, dx_add=dx)
    grads = [dx, dpre, dpost, dcomb, dweight, dbias, dweights]
    for i, (t, g) in enumerate(zip(inputs, grads)):
        d = randn(*t.shape, seed=20 + i)
        d /= d.norm()
        ends = [forward(*[u + s * h * d if j == i else u for j, u in enumerate(inputs)])[0].double()
                for s in (1, -1)]
        numeric = float((r.double() * (ends[0] - ends[1])).sum()) / (2 * h)
        exact = float((g.double() * d.double()).sum())
        assert abs(numeric - exact) <= 1e-3 * float(g.double().norm() + 1), (i, numeric, exact)


# ---------------------------------------------------------------- streams, graphs, refusals


def chain_of_calls(x, pre, post, comb, ids, weights, weight, bias, E):
    n, hh, mean, rstd = sub.hc_mix_collapse_norm(x, pre, weight, bias, EPS, want_saved=True)
    offsets, slots, source = sub.hc_mix_expert_sort(ids, E)
    xs = sub.hc_mix_expert_dispatch(n, slots, offsets)
    y = sub.hc_mix_expert_combine(xs, slots, weights)
    out = sub.hc_mix_expand(x, y, post, comb)
    dx, dy, dpost, dcomb = sub.hc_mix_expand_backward(out, x, y, post, comb)
    dys, dw = sub.hc_mix_expert_combine_backward(dy, xs, slots, offsets, weights)
    dn = sub.hc_mix_expert_combine(dys, slots)
    dh, dweight, dbias = sub.hc_mix_layer_norm_backward(dn, hh, mean, rstd, weight)
    dx, dpre = sub.hc_mix_collapse_backward(dh, x, pre, dx_add=dx)
    return [out, dx, dpre, dpost, dcomb, dw, dweight, dbias, offsets, slots, source]


def chain_inputs(T=70, k=3, E=11, D=520):
    return (randn(T, HC * D, dtype=torch.bfloat16), *coefficients(T),
            random_ids(T, k, E, seed=1, drop=0.1).cuda(), torch.softmax(randn(T, k, seed=2), 1),
            randn(D, seed=3, mean=1), randn(D, seed=4), E)


def test_other_stream_and_graph_capture():
    """The calls go to the current stream, and replay from a CUDA graph with the same bits."""
    args = chain_inputs()
    want = chain_of_calls(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = chain_of_calls(*args)
    side.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = chain_of_calls(*args)
    for t in held:
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(held, want))


def test_stream_argument():
    x = randn(8, 640)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = sub.hc_mix_layer_norm(x, stream=side)
    side.synchronize()
    assert torch.equal(y, sub.hc_mix_layer_norm(x))


def test_refusals():
    x, (pre, post, comb) = randn(6, HC * 32), coefficients(6)
    y = randn(6, 32)
    slots = torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    bad = [
        lambda: sub.hc_mix_layer_norm(x.t()),                                  # inner stride
        lambda: sub.hc_mix_layer_norm(x.double()),
        lambda: sub.hc_mix_layer_norm(x[0]),
        lambda: sub.hc_mix_layer_norm(x, torch.ones(7, device="cuda")),
        lambda: sub.hc_mix_layer_norm(x, torch.ones(128)),                     # a host weight
        lambda: sub.hc_mix_layer_norm(x, torch.ones(128, device="cuda", dtype=torch.float16)),
        lambda: sub.hc_mix_layer_norm(x, out=torch.empty(6, 127, device="cuda")),
        lambda: sub.hc_mix_layer_norm_backward(x[:5], x, pre[:, 0].contiguous(), pre[:, 0].contiguous()),
        lambda: sub.hc_mix_layer_norm_backward(x, x, pre[:, 0], pre[:, 0].contiguous()),
        lambda: sub.hc_mix_collapse(x[:, :126], pre),                          # not 4 streams
        lambda: sub.hc_mix_collapse(x, pre.half()),
        lambda: sub.hc_mix_collapse(x, pre[:5]),
        lambda: sub.hc_mix_collapse_backward(y.half(), x, pre),
        lambda: sub.hc_mix_collapse_backward(y, x, pre, dx_add=y),
        lambda: sub.hc_mix_expand(x, y[:, :31], post, comb),
        lambda: sub.hc_mix_expand(x, y, post, comb.transpose(1, 2)),
        lambda: sub.hc_mix_expand(x, y, post, comb, out=y),
        lambda: sub.hc_mix_expand_backward(y, x, y, post, comb),
        lambda: sub.hc_mix_expert_sort(slots.float(), 4),
        lambda: sub.hc_mix_expert_sort(slots.t(), 4),
        lambda: sub.hc_mix_expert_dispatch(y, slots.long()),
        lambda: sub.hc_mix_expert_dispatch(y[:5], slots),
        lambda: sub.hc_mix_expert_combine(x, slots, torch.ones(6, 3, device="cuda")),
        lambda: sub.hc_mix_expert_combine_backward(y[:5], y, slots, None, torch.ones(6, 2, device="cuda")),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    for f in (lambda: sub.hc_mix_expert_sort(slots, 0), lambda: sub.hc_mix_expert_sort(slots, 5000),
              lambda: sub.hc_mix_layer_norm(y.expand(6, 32)[:1].expand(6, 32))):  # row stride 0
        with pytest.raises(binding.HcMixError):
            f()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    one = torch.ones(6, device="cuda")
    with pytest.raises(binding.HcMixError):
        sub.hc_mix_layer_norm_backward(x, x, one, one, workspace=ws)  # too small
