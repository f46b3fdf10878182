"""Where the experts' binding's calls go and what it refuses, checked without a GPU against the
stand-ins of test_sublayer_binding_cpu."""
import pytest
import torch

from hyper_connection_mix_gb300 import experts, sublayer as sub
from test_sublayer_binding_cpu import Stream, Tensor, cuda as sublayer_cuda  # noqa: F401

BF16, F16, F32, I32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8
E, R, K, N, G = 4, 10, 64, 32, 32


class Strided(Tensor):
    """Contiguous, of any number of dimensions."""

    def stride(self):
        steps, at = [], 1
        for n in reversed(self.shape):
            steps.append(at)
            at *= n
        return tuple(reversed(steps))


@pytest.fixture
def cuda(sublayer_cuda, monkeypatch):  # noqa: F811
    c = sublayer_cuda
    monkeypatch.setattr(experts, "lib", lambda: c)
    monkeypatch.setattr(experts, "_empty", c.empty)
    monkeypatch.setattr(experts, "_device", lambda: c.device)
    return c


def entry_points(device):
    t = lambda dtype, *shape: Strided(shape, dtype, device)  # noqa: E731
    xs, dys, at = t(BF16, R, K), t(BF16, R, N), t(I32, E + 1)
    w = t(BF16, E, N, K)
    return {
        "hc_mix_expert_product": ((xs, w, at), {}),
        "hc_mix_expert_product_gated": ((xs, w, at), {"want_saved": True}),
        "hc_mix_expert_product_weight_backward": ((dys, xs, at), {}),
        "hc_mix_expert_gate_backward": ((t(BF16, R, N), t(BF16, R, 2 * N)), {}),
        "hc_mix_expert_product_q4": ((xs, t(U8, E, N, K // 2), t(BF16, E, N, K // G), at), {}),
    }


NAMES = list(entry_points("cuda:0"))


def test_every_entry_point_is_here():
    assert sorted(NAMES) == sorted(n for n in experts.EXPORTS if not n.endswith("_status"))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("device,where", [("cuda:0", (0, 100)), ("cuda:1", (1, 200))])
def test_a_call_goes_to_the_current_stream_of_its_tensors_device(cuda, name, device, where):
    args, kw = entry_points(device)[name]
    getattr(experts, name)(*args, **kw)
    assert cuda.called == [(name, where, where[1])]
    assert {t.device.index for t in cuda.allocated} == {where[0]}
    assert cuda.device == 0


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("stream,handle", [(Stream(300), 300), (301, 301), (0, 0)],
                         ids=["stream", "handle", "default"])
def test_memory_belongs_to_the_stream_that_uses_it(cuda, name, stream, handle):
    args, kw = entry_points("cuda:0")[name]
    result = getattr(experts, name)(*args, **kw, stream=stream)
    assert cuda.called == [(name, (0, handle), handle)]
    assert {t.place for t in cuda.allocated} == {(0, handle)}
    assert {tuple(t.on) for t in args} == {(handle,)}
    outputs = result if isinstance(result, tuple) else (result,)
    assert {tuple(t.on) for t in outputs} == {(100,)}


def test_backward_is_two_calls_on_the_given_stream(cuda):
    t = lambda dtype, *shape: Strided(shape, dtype, "cuda:0")  # noqa: E731
    dxs, dw = experts.hc_mix_expert_product_backward(t(BF16, R, N), t(BF16, R, K), t(BF16, E, N, K),
                                                     t(I32, E + 1), stream=Stream(300))
    assert [c[0] for c in cuda.called] == ["hc_mix_expert_product", "hc_mix_expert_product_weight_backward"]
    assert {c[2] for c in cuda.called} == {300}
    assert dxs.shape == (R, K) and dw.shape == (E, N, K)


def test_shapes_of_transposed_weights(cuda):
    t = lambda dtype, *shape: Strided(shape, dtype, "cuda:0")  # noqa: E731
    xs, at, w = t(BF16, R, K), t(I32, E + 1), t(BF16, E, K, N)
    assert experts.hc_mix_expert_product(xs, w, at, transposed=True).shape == (R, N)
    assert experts.hc_mix_expert_product_gated(xs, w, at, transposed=True).shape == (R, N // 2)
    dw = experts.hc_mix_expert_product_weight_backward(t(BF16, R, N), xs, at, True, F32)
    assert dw.shape == (E, K, N) and dw.dtype is F32


def refused(call, *args, **kw):
    with pytest.raises(ValueError):
        call(*args, **kw)


def test_refusals(cuda):
    t = lambda dtype, *shape, device="cuda:0": Strided(shape, dtype, device)  # noqa: E731
    xs, at, w = t(BF16, R, K), t(I32, E + 1), t(BF16, E, N, K)
    for f in (experts.hc_mix_expert_product, experts.hc_mix_expert_product_gated):
        refused(f, xs, t(F16, E, N, K), at)                    # another type
        refused(f, xs, t(BF16, E, N, K, device="cuda:1"), at)  # another device
        refused(f, xs, t(BF16, N, K), at)
        refused(f, xs, w, at, transposed=True)                 # N is not xs's width
        refused(f, xs, w, t(I32, E))                           # offsets of E - 1 experts
        refused(f, xs, w, t(torch.int64, E + 1))
        refused(f, xs, w, t(I32, E + 1, device="cuda:1"))
        refused(f, xs, w, at, out=t(BF16, R, N + 1))
        refused(f, t(BF16, R, K, 1), w, at)
    refused(experts.hc_mix_expert_product_gated, xs, t(BF16, E, 31, K), at)
    back = experts.hc_mix_expert_product_weight_backward
    refused(back, t(BF16, R + 1, N), xs, at)
    refused(back, t(F16, R, N), xs, at)
    refused(back, t(BF16, R, N), xs, at, weight_dtype=F16)
    refused(back, t(BF16, R, N), xs, t(I32, 1))                # no expert
    refused(experts.hc_mix_expert_product_backward, t(BF16, R, N + 1), xs, w, at)
    refused(experts.hc_mix_expert_gate_backward, t(BF16, R, N), t(BF16, R, N))
    q4, codes, scales = experts.hc_mix_expert_product_q4, t(U8, E, N, K // 2), t(BF16, E, N, 2)
    refused(q4, xs, t(torch.int8, E, N, K // 2), scales, at)
    refused(q4, xs, t(U8, E, N, K), scales, at)                # a code a byte
    refused(q4, xs, codes, t(F32, E, N, 2), at)
    refused(q4, xs, codes, t(BF16, E, N + 1, 2), at)
    refused(q4, xs, codes, t(BF16, E, N, 3), at)               # groups of no whole number
    refused(q4, xs, codes, t(BF16, E, N, 0), at)
    refused(q4, t(BF16, R, 63), codes, scales, at)
    refused(q4, xs, t(U8, E, 31, K // 2), t(BF16, E, 31, 2), at, gated=True)
    assert not cuda.called


def test_rows_without_unit_stride_are_refused(cuda):
    class Columns(Strided):
        def stride(self):
            return tuple(reversed(super().stride()))

    at = Strided((E + 1,), I32, "cuda:0")
    refused(experts.hc_mix_expert_product, Columns((R, K), BF16, "cuda:0"), Strided((E, N, K), BF16, "cuda:0"), at)
    refused(experts.hc_mix_expert_product, Strided((R, K), BF16, "cuda:0"), Columns((E, N, K), BF16, "cuda:0"), at)


def test_the_same_types_as_the_sublayers():
    assert experts.TYPES is sub.TYPES
