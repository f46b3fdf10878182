"""Sums over a long k, of terms of one sign: what each step of the MMAs drops is always to the same side, so
that such a sum shows all of it.  The kernels add up parts of 16384 (1024 for an fp32 result) whose
sums begin at zero: a part is off by at most (n / 8 + 16) 2^-23 of its terms' sum, as in
test_experts_gpu with n the part's length, and each of the additions of parts by half a step, 2^-24.
"""
import pytest
import torch

from hyper_connection_mix_gb300 import experts
from test_experts_gpu import BF16, F16, F32, NAN, chain, close, generator, offsets_of, strided

pytestmark = pytest.mark.gpu


def positive(*shape, dtype, seed, scale=1.0):
    """From a half to one, times scale."""
    return ((torch.rand(*shape, generator=generator(seed), device="cuda") + 1) * (scale / 2)).to(dtype)


def parts(n, of):
    return chain(min(n, of)) + (n // of + 1) * 2.0 ** -24


def weight_gradients(dys, xs, counts, transposed, to):
    """Of the first rows of both, 16384 at a time: widths are small."""
    at = 0
    for n in counts:
        a, b = (xs, dys) if transposed else (dys, xs)
        yield n, sum(a[i:min(i + 16384, at + n)].double().t() @ b[i:min(i + 16384, at + n)].double()
                     for i in range(at, at + n, 16384)) if n else None
        at += n


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype,to", [(BF16, F32), (F16, F32), (F16, F16)])
@pytest.mark.parametrize("K,N,pad", [(72, 40, 0), (264, 520, 0), (67, 33, 0), (64, 48, 3)])
@pytest.mark.parametrize("counts", [[131072], [2048, 2049, 0, 4095, 16384, 1, 16385, 32768 + 37]])
def test_weight_gradients(counts, K, N, pad, dtype, to, transposed):
    R = sum(counts) + 5
    xs, dys = positive(R, K, dtype=dtype, seed=80), positive(R, N, dtype=dtype, seed=81, scale=2.0 ** -3)
    xs[-5:], dys[-5:] = NAN, NAN
    got = experts.hc_mix_expert_product_weight_backward(strided(dys, pad), strided(xs, pad), offsets_of(counts), transposed, to)
    for e, (n, want) in enumerate(weight_gradients(dys, xs, counts, transposed, to)):
        if n == 0:
            assert not got[e].any()
        else:
            close(got[e], want, parts(n, 1024 if to is F32 else 16384) * want, f"dweight[{e}] of {n} rows")
    assert experts.hc_mix_expert_device_status() == 0


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("K", [16383, 16384, 16448, 65537, 1 << 20])
def test_products(K, transposed):
    """fp16: its half step is 2^-11, less than what one sum of 2^20 terms loses."""
    counts, N = [5, 0, 300 if K < 1 << 20 else 33], 40
    xs = positive(sum(counts) + 2, K, dtype=F16, seed=82)
    xs[-2:] = NAN
    w = positive(3, *((K, N) if transposed else (N, K)), dtype=F16, seed=83)
    w *= 2.0 ** -6 * 16384 / (1 << (K.bit_length() - 1))  # exact; results stay below fp16's largest (h not always)
    offsets = offsets_of(counts)
    ys = experts.hc_mix_expert_product(xs, w, offsets, transposed)
    want = torch.zeros(xs.shape[0], N, dtype=torch.float64, device="cuda")
    for e, r in ((0, slice(0, 5)), (2, slice(5, sum(counts)))):
        v = w[e].double()
        want[r] = xs[r].double() @ (v if transposed else v.t())
    close(ys, want, parts(K, 16384) * want, "ys")
    # gated: silu(g) u of numbers that are large, or nearly so
    h, gu = experts.hc_mix_expert_product_gated(xs, w, offsets, transposed, want_saved=True)
    assert torch.equal(gu, ys)
    F, e = N // 2, parts(K, 16384)
    hs = want[:, :F] * want[:, F:]
    # 65520, half a step above fp16's largest, and more is rounded to infinity
    over = hs > 65520 * (1 + 2.0 ** -8)
    assert (h[over] == float("inf")).all() and not (hs[~over] > 65520 * (1 - 2.0 ** -8)).any()
    close(h.masked_fill(over, 0), hs.masked_fill(over, 0), 3 * (e + 24 * 2.0 ** -23) * hs, "h")


def test_same_bits_for_any_rows():
    """Parts are of k alone: a row's bits are the same among few and many, by either kind of loads."""
    K, N = 40000, 72
    xs, w = positive(700, K, dtype=BF16, seed=84), positive(1, N, K, dtype=BF16, seed=85, scale=2.0 ** -6)
    whole = experts.hc_mix_expert_product(xs, w, offsets_of([700]))
    for n in (1, 300):
        assert torch.equal(experts.hc_mix_expert_product(xs[:n], w, offsets_of([n])), whole[:n])
    assert torch.equal(experts.hc_mix_expert_product(strided(xs[:300], 3), w, offsets_of([300])), whole[:300])


@pytest.mark.parametrize("K,N", [(1032, 520), (1001, 333)])
def test_many_tiles_of_parts(K, N):
    """More tiles than blocks, of different numbers of parts, twice with the same bits; random signs."""
    counts = [5000, 0, 2048, 37, 9001, 2049, 1, 12288] * 3
    xs = torch.randn(sum(counts), K, generator=generator(86), device="cuda").to(BF16)
    dys = torch.randn(sum(counts), N, generator=generator(87), device="cuda").to(BF16)
    offsets = offsets_of(counts)
    got = experts.hc_mix_expert_product_weight_backward(dys, xs, offsets, weight_dtype=F32)
    at = 0
    for e, n in enumerate(counts):
        x, d = xs[at:at + n].double(), dys[at:at + n].double()
        close(got[e], d.t() @ x, parts(n, 1024) * (d.t().abs() @ x.abs()), f"dweight[{e}] of {n} rows")
        at += n
    assert torch.equal(experts.hc_mix_expert_product_weight_backward(dys, xs, offsets, weight_dtype=F32), got)
    assert experts.hc_mix_expert_device_status() == 0
