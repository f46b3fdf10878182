"""Weights' gradients of experts with so many rows that one tile takes seconds, longer than a wait
without progress may.  Nearly all rows are zeros and the others small whole numbers, so that the
sums are exact.  Helpers are those of test_experts_gpu."""
import pytest
import torch

from hyper_connection_mix_gb300 import experts
from test_experts_gpu import BF16, F16, F32, generator, offsets_of

pytestmark = pytest.mark.gpu


# rows that start on no 16 bytes (plain loads, about 2 us for 64 rows) and such that do (pairs)
@pytest.mark.parametrize("R,width,dtype", [((1 << 27) + 3, 7, F16), ((1 << 30) + 35, 8, BF16)])
def test_weight_gradient_of_one_long_expert(R, width, dtype):
    xs = torch.zeros(R, width, dtype=dtype, device="cuda")
    at = torch.tensor([0, 1, 63, 64, R // 3, R // 2, R - 36, R - 2, R - 1], device="cuda")
    xs[at] = torch.randint(-8, 9, (len(at), width), generator=generator(70), device="cuda").to(dtype)
    offsets = offsets_of([R - 1, 1])
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    dw = experts.hc_mix_expert_product_weight_backward(xs, xs, offsets, weight_dtype=F32)
    end.record()
    assert experts.hc_mix_expert_device_status() == 0
    print(f"{R} rows of {width}: {start.elapsed_time(end):.0f} ms")
    x = xs[at].double()
    want = torch.stack([x[:-1].t() @ x[:-1], x[-1:].t() @ x[-1:]])
    assert torch.equal(dw.double(), want)
