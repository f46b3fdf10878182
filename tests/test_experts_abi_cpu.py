"""Host-side checks of the experts' entry points that need no GPU: exported symbols, and the
refusal of bad arguments before anything is launched, by the library and by the binding."""
import os
import re

import pytest
import torch

from hyper_connection_mix_gb300 import experts
from hyper_connection_mix_gb300 import build as hbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000  # never dereferenced: every call here is refused or empty
OK, INVALID, ALIGNMENT, UNSUPPORTED = 0, 1, 2, 3
BF16, F16, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    hbuild.build()
    return experts.lib()


def test_exports_every_declared_symbol(L):
    src = open(os.path.join(ROOT, "include", "hcmix_experts.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(hc_mix_\w+)\s*\(", src)))
    assert sorted(experts.EXPORTS) == names
    for n in names:
        assert hasattr(L, n), n


def caller(f, **defaults):
    def call(**kw):
        assert set(kw) <= set(defaults)
        return f(*{**defaults, **kw}.values())
    return call


def check_matrix_refusals(call, pointer, stride, width):
    assert call(**{pointer: None}) == INVALID
    assert call(**{stride: width - 1}) == INVALID
    assert call(**{pointer: P + 1}) == ALIGNMENT


def check_common(call):
    assert call(R=-1) == INVALID
    assert call(R=(1 << 31) - 4095) == UNSUPPORTED
    assert call(type=F32) == UNSUPPORTED
    assert call(type=3) == INVALID
    assert call(type=-1) == INVALID
    assert call(offsets=None) == INVALID
    assert call(offsets=P + 2) == ALIGNMENT
    assert call(E=0) == INVALID
    assert call(E=-1) == INVALID
    assert call(E=4097, **({"we": 1 << 30} if "product" in call.__name__ else {})) == UNSUPPORTED


@pytest.mark.parametrize("gated", [False, True])
def test_product_refusals(L, gated):
    N = 32
    args = dict(xs=P, xss=64, type=BF16, R=4, K=64, N=N, w=P, ws=64, we=64 * 64, transposed=0,
                offsets=P, E=8, ys=P)
    if gated:
        call = caller(L.hc_mix_expert_product_gated, **args, gu=P, stream=None)
        assert call(gu=P + 1) == ALIGNMENT
    else:
        call = caller(L.hc_mix_expert_product, **args, stream=None)
    call.__name__ = "product"
    check_common(call)
    check_matrix_refusals(call, "xs", "xss", 64)
    check_matrix_refusals(call, "w", "ws", 64)
    assert call(K=0) == INVALID
    assert call(N=0) == INVALID
    assert call(K=(1 << 24) + 1, xss=1 << 25, ws=1 << 25, we=1 << 40) == UNSUPPORTED
    assert call(N=(1 << 24) + 1, we=1 << 40) == UNSUPPORTED
    features = 2 * N if gated else N
    assert call(we=(features - 1) * 64 + 63) == INVALID     # experts that overlap
    assert call(transposed=1, ws=features - 1) == INVALID   # its rows are of features
    assert call(transposed=1, ws=features, we=63 * features + features - 1) == INVALID
    assert call(ys=None) == INVALID
    assert call(ys=P + 1) == ALIGNMENT
    assert call(R=0, xs=None, ys=None) == OK


def test_the_gates_features_are_counted_twice(L):
    call = caller(L.hc_mix_expert_product_gated, xs=P, xss=64, type=F16, R=4, K=64, F=(1 << 23) + 1,
                  w=P, ws=64, we=1 << 40, transposed=0, offsets=P, E=2, h=P, gu=None, stream=None)
    assert call() == UNSUPPORTED


def test_weight_backward_refusals(L):
    call = caller(L.hc_mix_expert_product_weight_backward, dys=P, ds=32, xs=P, xss=64, type=BF16, R=4,
                  K=64, N=32, transposed=0, offsets=P, E=8, dw=P, dwt=BF16, stream=None)
    check_common(call)
    check_matrix_refusals(call, "xs", "xss", 64)
    check_matrix_refusals(call, "dys", "ds", 32)
    assert call(dwt=F16) == INVALID  # neither fp32 nor the rows' type
    assert call(dwt=5) == INVALID
    assert call(dw=None) == INVALID
    assert call(dw=P + 1) == ALIGNMENT
    assert call(dw=P + 2, dwt=F32) == ALIGNMENT
    assert call(K=0) == INVALID
    assert call(N=(1 << 24) + 1, ds=1 << 25) == UNSUPPORTED


def test_gate_backward_refusals(L):
    call = caller(L.hc_mix_expert_gate_backward, dh=P, ds=32, gu=P, gs=64, type=F32, R=4, F=32, dgu=P,
                  stream=None)
    assert call(R=-1) == INVALID
    assert call(F=0) == INVALID
    assert call(F=(1 << 23) + 1, ds=1 << 25, gs=1 << 25) == UNSUPPORTED
    assert call(type=3) == INVALID
    check_matrix_refusals(call, "dh", "ds", 32)
    check_matrix_refusals(call, "gu", "gs", 64)
    assert call(dgu=None) == INVALID
    assert call(dgu=P + 2) == ALIGNMENT
    assert call(R=0, dh=None, gu=None, dgu=None) == OK


def test_q4_refusals(L):
    call = caller(L.hc_mix_expert_product_q4, xs=P, xss=64, type=F16, R=4, K=64, N=32, codes=P, scales=P,
                  group=32, gated=0, offsets=P, E=8, out=P, stream=None)
    check_common(call)
    check_matrix_refusals(call, "xs", "xss", 64)
    assert call(group=0) == INVALID
    assert call(group=48) == INVALID               # does not divide K
    assert call(group=16) == UNSUPPORTED
    assert call(group=512, K=512, xss=512) == UNSUPPORTED
    assert call(gated=1, N=31) == INVALID
    assert call(codes=None) == INVALID
    assert call(codes=P + 8) == ALIGNMENT
    assert call(scales=None) == INVALID
    assert call(scales=P + 1) == ALIGNMENT
    assert call(out=None) == INVALID
    assert call(out=P + 1) == ALIGNMENT
    assert call(R=0, xs=None, out=None) == OK


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(1, 8, 64, dtype=torch.bfloat16)
    at = torch.zeros(2, dtype=torch.int32)
    for f in (lambda: experts.hc_mix_expert_product(x, w, at),
              lambda: experts.hc_mix_expert_product_gated(x, w, at),
              lambda: experts.hc_mix_expert_product_backward(x, x, w, at),
              lambda: experts.hc_mix_expert_product_weight_backward(x, x, at),
              lambda: experts.hc_mix_expert_gate_backward(x, x),
              lambda: experts.hc_mix_expert_product_q4(x, w, w, at)):
        with pytest.raises(ValueError):
            f()
