"""Host-side checks of the sublayer operators that need no GPU: exported symbols,
workspace size, and the refusal of bad arguments before anything is launched."""
import os
import re

import pytest
import torch

from hyper_connection_mix_gb300 import binding, sublayer
from hyper_connection_mix_gb300 import build as hbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000  # never dereferenced: every call here is refused or empty
OK, INVALID, ALIGNMENT, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4
BF16, F16, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    hbuild.build()
    return sublayer.lib()


def header():
    src = open(os.path.join(ROOT, "include", "hcmix_sublayer.h")).read()
    return re.sub(r"/\*.*?\*/", "", src, flags=re.S)


def test_exports_every_declared_symbol(L):
    names = sorted(set(re.findall(r"\b(hc_mix_\w+)\s*\(", header())))
    assert sorted(sublayer.EXPORTS) == names
    for n in names:
        assert hasattr(L, n), n


def test_type_codes_match_header():
    body = re.search(r"typedef enum \{([^}]*)\} hcmix_type;", header()).group(1)
    codes = {m.group(1): int(m.group(2)) for m in re.finditer(r"HCMIX_(\w+) = (\d)", body)}
    assert codes == {"BF16": sublayer.TYPES[torch.bfloat16], "F16": sublayer.TYPES[torch.float16],
                     "F32": sublayer.TYPES[torch.float32]}


def test_workspace_bytes(L):
    f = L.hc_mix_layer_norm_workspace_bytes
    assert f(BF16, 4096, 5120) >= 2 * 5120 * 4
    assert f(BF16, 4096, 5120) % 256 == 0
    assert f(BF16, 0, 5120) == 0
    assert f(BF16, -1, 5120) == 0 and f(BF16, 4, 0) == 0 and f(7, 4, 16) == 0
    assert f(F32, 4, (1 << 24) + 1) == 0


def caller(f, **defaults):
    def call(**kw):
        assert set(kw) <= set(defaults)
        return f(*{**defaults, **kw}.values())
    return call


def check_matrix_refusals(call, pointer, stride, width):
    assert call(**{pointer: None}) == INVALID
    assert call(**{stride: width - 1}) == INVALID
    assert call(**{pointer: P + 1}) == ALIGNMENT


def test_layer_norm_refusals(L):
    call = caller(L.hc_mix_layer_norm, x=P, xs=64, type=BF16, M=4, N=64, w=P, b=P, wt=F32,
                  eps=1e-5, y=P, mean=P, rstd=P, stream=None)
    assert call(M=-1) == INVALID
    assert call(N=0) == INVALID
    assert call(M=1 << 31) == UNSUPPORTED
    assert call(N=(1 << 24) + 1) == UNSUPPORTED
    assert call(type=3) == INVALID
    assert call(type=-1) == INVALID
    assert call(wt=F16) == INVALID         # neither fp32 nor x's type
    assert call(w=P + 2) == ALIGNMENT
    assert call(b=P + 2) == ALIGNMENT
    assert call(mean=P + 2) == ALIGNMENT
    assert call(y=None) == INVALID
    check_matrix_refusals(call, "x", "xs", 64)
    assert call(M=0, x=None, y=None) == OK


def test_layer_norm_backward_refusals(L):
    need = L.hc_mix_layer_norm_workspace_bytes(F32, 4, 64)
    call = caller(L.hc_mix_layer_norm_backward, dy=P, ds=64, x=P, xs=64, type=F32, M=4, N=64,
                  mean=P, rstd=P, w=P, wt=F32, dx=P, dw=P, db=P, ws=P, bytes=need, stream=None)
    assert call(M=-1) == INVALID
    assert call(db=None) == INVALID        # one of the two gradients alone
    assert call(mean=None) == INVALID
    assert call(rstd=P + 2) == ALIGNMENT
    assert call(wt=BF16) == INVALID
    assert call(ws=None) == INVALID
    assert call(ws=P + 128) == ALIGNMENT
    assert call(bytes=need - 1) == WORKSPACE
    check_matrix_refusals(call, "x", "xs", 64)
    check_matrix_refusals(call, "dy", "ds", 64)
    assert call(M=0, dw=None, db=None, dx=None, x=None) == OK


def test_streams_refusals(L):
    collapse = caller(L.hc_mix_collapse, x=P, xs=256, type=BF16, M=4, D=64, hc=4, pre=P, h=P,
                      stream=None)
    norm = caller(L.hc_mix_collapse_norm, x=P, xs=256, type=BF16, M=4, D=64, hc=4, pre=P, w=P, b=P,
                  wt=BF16, eps=1e-5, y=P, h=P, mean=P, rstd=P, stream=None)
    back = caller(L.hc_mix_collapse_backward, dh=P, ds=64, x=P, xs=256, add=P, adds=256, type=BF16,
                  M=4, D=64, hc=4, pre=P, dx=P, dpre=P, stream=None)
    expand = caller(L.hc_mix_expand, x=P, xs=256, y=P, ys=64, type=BF16, M=4, D=64, hc=4, post=P,
                    comb=P, out=P, stream=None)
    eback = caller(L.hc_mix_expand_backward, do=P, dos=256, x=P, xs=256, y=P, ys=64, type=BF16,
                   M=4, D=64, hc=4, post=P, comb=P, dx=P, dy=P, dpost=P, dcomb=P, stream=None)
    for call in (collapse, norm, back, expand, eback):
        assert call(hc=3) == UNSUPPORTED
        assert call(D=0) == INVALID
        assert call(D=1 << 23, xs=1 << 25) == UNSUPPORTED
        assert call(M=-1) == INVALID
        assert call(type=9) == INVALID
        check_matrix_refusals(call, "x", "xs", 256)
        assert call(M=0, x=None) == OK
    assert collapse(pre=None) == INVALID
    assert collapse(h=P + 1) == ALIGNMENT
    assert norm(wt=F16) == INVALID
    assert norm(y=None) == INVALID
    assert norm(h=P + 1) == ALIGNMENT
    check_matrix_refusals(back, "dh", "ds", 64)
    assert back(adds=255) == INVALID
    assert back(dpre=None) == INVALID
    check_matrix_refusals(expand, "y", "ys", 64)
    assert expand(comb=P + 2) == ALIGNMENT
    check_matrix_refusals(eback, "do", "dos", 256)
    check_matrix_refusals(eback, "y", "ys", 64)
    assert eback(dcomb=None) == INVALID
    assert eback(dy=None) == INVALID


def test_expert_refusals(L):
    sort = caller(L.hc_mix_expert_sort, ids=P, bytes=8, T=4, k=2, E=8, offsets=P, slots=P,
                  source=P, stream=None)
    assert sort(bytes=2) == INVALID
    assert sort(E=0) == INVALID
    assert sort(E=4097) == UNSUPPORTED
    assert sort(T=-1) == INVALID
    assert sort(T=1 << 30, k=2) == UNSUPPORTED
    assert sort(ids=None) == INVALID
    assert sort(ids=P + 4) == ALIGNMENT
    assert sort(offsets=None) == INVALID
    assert sort(slots=P + 2) == ALIGNMENT
    dispatch = caller(L.hc_mix_expert_dispatch, x=P, xs=64, type=BF16, T=4, k=2, D=64, slots=P,
                      offsets=P, E=8, out=P, stream=None)
    combine = caller(L.hc_mix_expert_combine, ys=P, yss=64, type=BF16, rows=8, T=4, k=2, D=64,
                     slots=P, weights=P, y=P, stream=None)
    back = caller(L.hc_mix_expert_combine_backward, dy=P, ds=64, ys=P, yss=64, type=BF16, rows=8,
                  T=4, k=2, D=64, slots=P, offsets=P, E=8, weights=P, dys=P, dw=P, stream=None)
    for call in (dispatch, combine, back):
        assert call(T=-1) == INVALID
        assert call(k=-1) == INVALID
        assert call(D=0) == INVALID
        assert call(T=1 << 30, k=2) == UNSUPPORTED
        assert call(type=5) == INVALID
        assert call(slots=None) == INVALID
        assert call(slots=P + 2) == ALIGNMENT
    check_matrix_refusals(dispatch, "x", "xs", 64)
    assert dispatch(E=-1) == INVALID
    check_matrix_refusals(combine, "ys", "yss", 64)
    assert combine(rows=-1) == INVALID
    assert combine(weights=P + 2) == ALIGNMENT
    check_matrix_refusals(back, "dy", "ds", 64)
    check_matrix_refusals(back, "ys", "yss", 64)
    assert back(weights=None) == INVALID
    assert back(dw=None) == INVALID
    assert back(dys=None) == INVALID
    assert dispatch(T=0, x=None, slots=None, out=None) == OK
    assert dispatch(k=0, x=None, slots=None, out=None) == OK
    assert combine(T=0, ys=None, slots=None, y=None) == OK
    assert back(T=0, rows=0, dy=None, ys=None, slots=None, dys=None) == OK


def test_binding_refuses_cpu_tensors():
    """There is no CPU fallback: host tensors raise before the library is asked."""
    x = torch.zeros(2, 8)
    for f in (lambda: sublayer.hc_mix_layer_norm(x),
              lambda: sublayer.hc_mix_collapse(x, torch.zeros(2, 4)),
              lambda: sublayer.hc_mix_expand(x, x, torch.zeros(2, 4), torch.zeros(2, 4, 4)),
              lambda: sublayer.hc_mix_expert_dispatch(x, torch.zeros(2, 1, dtype=torch.int32)),
              lambda: sublayer.hc_mix_expert_sort(torch.zeros(2, 2, dtype=torch.int64), 4)):
        with pytest.raises(ValueError):
            f()


def test_binding_uses_the_built_library(L):
    assert binding.lib() is L
