"""Where the sublayer binding's calls go, checked without a GPU: stand-ins for CUDA tensors,
streams and the library record the device and the stream under which each thing happens."""
import contextlib

import pytest
import torch

from hyper_connection_mix_gb300 import sublayer as sub

BF16, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
M, D, E, K = 6, 32, 8, 2


class Tensor:
    """As much of a contiguous CUDA tensor as the binding looks at."""
    is_cuda = True

    def __init__(self, shape, dtype, device, place=None):
        shape = (shape,) if isinstance(shape, int) else shape
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)
        self.place = place  # the (device, stream) that it was allocated under
        self.on = []        # the streams that it was recorded on

    def stride(self):
        return (self.shape[1], 1)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return 0x10000

    def record_stream(self, stream):
        self.on.append(stream.cuda_stream)


class Stream:
    def __init__(self, handle, device="cuda:0"):
        self.cuda_stream, self.device = handle, torch.device(device)

    def __eq__(self, other):
        return self.cuda_stream == other.cuda_stream


class Cuda:
    """The current device, each device's current stream, and what happened where."""

    def __init__(self):
        self.device, self.streams = 0, {0: 100, 1: 200}
        self.allocated, self.called = [], []

    def where(self):
        return self.device, self.streams[self.device]

    def empty(self, shape, dtype, device):
        self.allocated.append(Tensor(shape, dtype, device, self.where()))
        return self.allocated[-1]

    def __getattr__(self, name):  # an entry point of the library
        def call(*args):
            if name.endswith("_bytes"):
                return 1024
            self.called.append((name, self.where(), args[-1]))
            return 0
        return call

    @contextlib.contextmanager
    def on_device(self, device):
        before, self.device = self.device, torch.device(device).index
        yield
        self.device = before

    @contextlib.contextmanager
    def on_stream(self, stream):
        at = stream.device.index
        before, self.streams[at] = self.streams[at], stream.cuda_stream
        yield
        self.streams[at] = before


@pytest.fixture
def cuda(monkeypatch):
    c = Cuda()
    monkeypatch.setattr(sub, "lib", lambda: c)
    monkeypatch.setattr(sub, "_empty", c.empty)
    monkeypatch.setattr(sub, "_device", lambda: c.device, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: c.streams[i], raising=False)
    monkeypatch.setattr(torch.cuda, "device", c.on_device)
    monkeypatch.setattr(torch.cuda, "stream", c.on_stream)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch, "Tensor", Tensor)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device: Stream(h, device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: Stream(0, device))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream(c.where()[1], f"cuda:{c.device}"))
    return c


def entry_points(device):
    """Every call of the module on tensors of `device`."""
    t = lambda dtype, *shape: Tensor(shape, dtype, device)  # noqa: E731
    x, y, h = t(BF16, M, 4 * D), t(BF16, M, D), t(BF16, M, D)
    pre, post, comb = t(F32, M, 4), t(F32, M, 4), t(F32, M, 4, 4)
    mean, rstd, weight = t(F32, M), t(F32, M), t(F32, D)
    slots, offsets, weights = t(I32, M, K), t(I32, E + 1), t(F32, M, K)
    ys = t(BF16, M * K, D)
    return {
        "hc_mix_layer_norm": ((y, weight, weight), {"want_stats": True}),
        "hc_mix_layer_norm_backward": ((h, y, mean, rstd, weight), {}),
        "hc_mix_collapse": ((x, pre), {}),
        "hc_mix_collapse_norm": ((x, pre, weight, weight), {"want_saved": True}),
        "hc_mix_collapse_backward": ((h, x, pre), {"dx_add": t(BF16, M, 4 * D)}),
        "hc_mix_expand": ((x, y, post, comb), {}),
        "hc_mix_expand_backward": ((t(BF16, M, 4 * D), x, y, post, comb), {}),
        "hc_mix_expert_sort": ((t(I64, M, K), E), {}),
        "hc_mix_expert_dispatch": ((y, slots, offsets), {}),
        "hc_mix_expert_combine": ((ys, slots, weights), {}),
        "hc_mix_expert_combine_backward": ((y, ys, slots, offsets, weights), {}),
    }


NAMES = list(entry_points("cuda:0"))


def test_every_entry_point_is_here():
    assert sorted(NAMES) == sorted(n for n in sub.EXPORTS if not n.endswith("_bytes"))


@pytest.mark.parametrize("name", NAMES)
def test_a_call_goes_to_the_current_stream(cuda, name):
    args, kw = entry_points("cuda:0")[name]
    getattr(sub, name)(*args, **kw)
    assert cuda.called == [(name, (0, 100), 100)]
    assert {t.place for t in cuda.allocated} == {(0, 100)}


@pytest.mark.parametrize("name", NAMES)
def test_a_call_goes_to_the_device_of_its_tensors(cuda, name):
    """The library launches on the current device: it is the tensors' during the call."""
    args, kw = entry_points("cuda:1")[name]
    getattr(sub, name)(*args, **kw)
    assert cuda.called == [(name, (1, 200), 200)]
    assert {t.device.index for t in cuda.allocated} == {1}
    assert cuda.device == 0


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("stream,handle", [(Stream(300), 300), (301, 301), (0, 0)],
                         ids=["stream", "handle", "default"])
def test_memory_belongs_to_the_stream_that_uses_it(cuda, name, stream, handle):
    """With `stream`, outputs and workspaces are allocated under it; the inputs are recorded on
    it, and the outputs on the stream that the caller goes on with."""
    args, kw = entry_points("cuda:0")[name]
    result = getattr(sub, name)(*args, **kw, stream=stream)
    assert cuda.called == [(name, (0, handle), handle)]
    assert {t.place for t in cuda.allocated} == {(0, handle)}
    inputs = [t for t in (*args, *kw.values()) if isinstance(t, Tensor)]
    assert {tuple(t.on) for t in inputs} <= {(handle,), (handle, handle)}  # weight given as bias too
    outputs = result if isinstance(result, tuple) else (result,)
    assert {tuple(t.on) for t in outputs} == {(100,)}
    assert cuda.where() == (0, 100)


@pytest.mark.parametrize("stream", [Stream(100), 100], ids=["stream", "handle"])
def test_the_current_stream_given_by_name(cuda, stream):
    y = Tensor((M, D), BF16, "cuda:0")
    out = sub.hc_mix_layer_norm(y, stream=stream)
    assert cuda.called == [("hc_mix_layer_norm", (0, 100), 100)]
    assert out.place == (0, 100) and not out.on and not y.on


def test_a_stream_of_another_device_is_refused(cuda):
    with pytest.raises(ValueError):
        sub.hc_mix_layer_norm(Tensor((M, D), BF16, "cuda:0"), stream=Stream(300, "cuda:1"))
    assert not cuda.called


class NonContiguous(Tensor):
    def is_contiguous(self):
        return False


@pytest.mark.parametrize("workspace", [
    Tensor(1 << 20, torch.uint8, "cuda:1"),          # another device's memory
    NonContiguous(1 << 20, torch.uint8, "cuda:0"),   # fewer bytes than elements, or bytes apart
    Tensor(1 << 20, F32, "cuda:0"),                  # elements that are not bytes
], ids=["device", "strided", "type"])
def test_workspaces_that_are_not_bytes_of_the_device_are_refused(cuda, workspace):
    args, _ = entry_points("cuda:0")["hc_mix_layer_norm_backward"]
    with pytest.raises(ValueError):
        sub.hc_mix_layer_norm_backward(*args, workspace=workspace)
    assert not cuda.called


def test_a_host_workspace_is_refused(cuda):
    args, _ = entry_points("cuda:0")["hc_mix_layer_norm_backward"]
    workspace = Tensor(1 << 20, torch.uint8, "cpu")
    with pytest.raises(ValueError):
        sub.hc_mix_layer_norm_backward(*args, workspace=workspace)
    assert not cuda.called


def test_a_workspace_that_is_given_is_used(cuda):
    args, _ = entry_points("cuda:0")["hc_mix_layer_norm_backward"]
    sub.hc_mix_layer_norm_backward(*args, workspace=Tensor(1 << 20, torch.uint8, "cuda:0"))
    assert len(cuda.called) == 1 and torch.uint8 not in {t.dtype for t in cuda.allocated}


@pytest.mark.parametrize("experts", [1 << 40, 4097, 0, -1, -(1 << 40)])
def test_a_number_of_experts_that_the_library_refuses_allocates_little(cuda, experts):
    """The refusal is the library's: it comes before memory for so many offsets is asked for."""
    sub.hc_mix_expert_sort(Tensor((M, K), I64, "cuda:0"), experts)
    assert len(cuda.called) == 1
    assert max(t.numel() for t in cuda.allocated) <= 4097
