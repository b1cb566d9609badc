"""The entry points of the gated projections and the low-rank adapters: exported,
bound one to one, and refusing invalid arguments on the host before any HIP call
(fake, never dereferenced addresses; only where no GPU is visible)."""
import ctypes
import os
import re

import pytest
import torch

import sparse_gemm_layers_amd as sg
from sparse_gemm_layers_amd import _gated, _lora

INCLUDE = os.path.join(os.path.dirname(sg.__file__), "include")
OK, NULL, SHAPE, UNSUP, ALIGN, HIP = range(6)
P = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(16)]
ODD = ctypes.c_void_p(0x100008)     # 8- but not 16-byte aligned
ODD1 = ctypes.c_void_p(0x100001)

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run only without a GPU")


@pytest.mark.parametrize("header,module", [("sg_gated.h", _gated), ("sg_lora.h", _lora)])
def test_header_binding_and_library_agree(header, module):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(INCLUDE, header)).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(sg_[a-z0-9_]+)\s*\(", src)))
    assert names == sorted(module._SIGS)
    for n in names:
        assert hasattr(module._lib(), n), n
        assert n[3:] in sg.__all__


def call(module, name, base, kw):
    a = dict(base, **kw)
    return getattr(module._lib(), name)(*[a[k] for k in base])


GATED = dict(T=3, F=48, D=40, x=P[0], ldx=40, gate=P[1], ldg=40, up=P[2], ldu=48, act=0, ga=P[3], ua=P[4], lda=48, h=P[5],
             dt=1, ldh=48, g=P[6], u=P[7], ldgu=48, st=None)
BIG = 1 << 22
SHARED = [
    *[({n: None}, NULL) for n in ("x", "gate", "up", "g", "u")],
    (dict(act=4), UNSUP), (dict(act=-1), UNSUP), (dict(T=0), SHAPE), (dict(F=0), SHAPE), (dict(D=0), SHAPE),
    (dict(D=36), SHAPE), (dict(F=44), SHAPE), (dict(T=1 << 31), SHAPE), (dict(F=BIG), SHAPE), (dict(D=BIG), SHAPE),
    (dict(T=1 << 30, F=1 << 20), SHAPE), (dict(ldx=32), SHAPE), (dict(ldg=32), SHAPE), (dict(ldu=32), SHAPE),
    (dict(lda=40), SHAPE), (dict(ldgu=40), SHAPE), (dict(ldx=BIG), SHAPE), (dict(ldx=44), ALIGN), (dict(ldg=44), ALIGN),
    (dict(ldu=44), ALIGN), (dict(lda=52), ALIGN), (dict(ldgu=52), ALIGN),
    *[({n: ODD}, ALIGN) for n in ("x", "gate", "up", "ga", "ua", "g", "u")],
]


@no_gpu
@pytest.mark.parametrize("kw,code", [
    *SHARED, (dict(h=None), NULL), (dict(dt=2), UNSUP), (dict(ldh=40), SHAPE), (dict(ldh=52), ALIGN), (dict(h=ODD), ALIGN),
])
def test_gated_refusals(kw, code):
    assert call(_gated, "sg_gated_gemm", GATED, kw) == code


GATED_BACK = dict(T=3, F=48, D=4096, dh=P[8], lddh=48, x=P[0], ldx=4096, gate=P[1], ldg=4096, up=P[2], ldu=4104, act=0,
                  g=P[6], u=P[7], ldgu=48, ga=P[3], ua=P[4], lda=48, dg=P[9], du=P[10], lddgu=48, dx=P[11], lddx=4096,
                  dgate=P[12], dup=P[13], lddw=4096, ws=P[14], wsb=1 << 40, st=None)


@no_gpu
@pytest.mark.parametrize("kw,code", [
    *[(dict(k, **({n: 4100} if (n := next(iter(k))) in ("ldx", "ldg", "ldu") and k[n] == 44 else {})), c) for k, c in SHARED],
    *[({n: None}, NULL) for n in ("dh", "dg", "du", "dgate", "dup")],
    (dict(lddh=40), SHAPE), (dict(lddgu=40), SHAPE), (dict(lddx=4088), SHAPE), (dict(lddw=4088), SHAPE),
    (dict(T=1 << 20, D=1 << 21, ldx=1 << 21, ldg=1 << 21, ldu=1 << 21, lddx=1 << 21, lddw=1 << 21), SHAPE),
    (dict(lddh=52), ALIGN), (dict(lddgu=52), ALIGN), (dict(lddx=4100), ALIGN), (dict(lddw=4100), ALIGN),
    *[({n: ODD}, ALIGN) for n in ("dh", "dg", "du", "dx", "dgate", "dup")],
])
def test_gated_backward_refusals(kw, code):
    assert call(_gated, "sg_gated_gemm_backward", GATED_BACK, kw) == code


def test_gated_backward_workspace():
    need = sg.gated_gemm_backward_workspace
    assert need(333, 2760, 1032) > 0 and need(333, 2760, 1032) % (4 * 333 * 1032) == 0
    for bad in ((0, 8, 8), (1, 0, 8), (1, 8, 0), (1, 12, 8), (1, 8, 12), (1 << 31, 8, 8), (1, BIG, 8), (1, 8, BIG)):
        assert need(*bad) == -1


@no_gpu
def test_gated_backward_checks_its_workspace():
    size = dict(T=333, F=2760, D=1032, lddh=2760, ldx=1032, ldg=1032, ldu=1032, ldgu=2760, lda=2760, lddgu=2760,
                lddx=1032, lddw=1032)
    need = sg.gated_gemm_backward_workspace(333, 2760, 1032)   # the larger of with and without the weights' gradients
    calls = [dict(size, wsb=need - 1), dict(size, wsb=need - 1, dgate=None, dup=None)]
    assert SHAPE in [call(_gated, "sg_gated_gemm_backward", GATED_BACK, c) for c in calls]
    assert call(_gated, "sg_gated_gemm_backward", GATED_BACK, dict(size, wsb=4 * 333 * 1032 - 1)) == SHAPE
    assert call(_gated, "sg_gated_gemm_backward", GATED_BACK, dict(size, ws=None)) == NULL
    assert call(_gated, "sg_gated_gemm_backward", GATED_BACK, dict(size, ws=ODD)) == ALIGN


LORA = dict(T=100, K=40, N=48, r=16, L=5, x=P[0], ldx=40, ids=P[1], a=P[2], b=P[3], scale=P[4], base=P[5], bdt=1, ldb=48, y=P[6],
            dt=0, ldy=48, ws=P[7], wsb=1 << 40, st=None)
LORA_SHARED = [
    *[({n: None}, NULL) for n in ("x", "a", "b", "ws")],
    (dict(T=0), SHAPE), (dict(K=0), SHAPE), (dict(N=0), SHAPE), (dict(r=0), SHAPE), (dict(L=0), SHAPE),
    (dict(K=36), SHAPE), (dict(N=44), SHAPE), (dict(r=12), SHAPE), (dict(r=264), SHAPE), (dict(L=65536), SHAPE),
    (dict(T=BIG), SHAPE), (dict(ldx=32), SHAPE), (dict(ldx=BIG), SHAPE), (dict(wsb=100), SHAPE),
    (dict(ldx=44), ALIGN), *[({n: ODD}, ALIGN) for n in ("x", "a", "b", "base", "ws")], (dict(ids=ODD1), ALIGN),
    (dict(scale=ODD1), ALIGN),
]


@no_gpu
@pytest.mark.parametrize("kw,code", [
    *LORA_SHARED, (dict(y=None), NULL), (dict(dt=2), UNSUP), (dict(bdt=3), UNSUP), (dict(ldy=40), SHAPE),
    (dict(ldb=40), SHAPE), (dict(base=P[6]), SHAPE), (dict(base=P[6], bdt=0, ldb=56), SHAPE), (dict(ldy=52), ALIGN),
    (dict(ldb=52), ALIGN), (dict(y=ODD), ALIGN),
])
def test_lora_refusals(kw, code):
    assert call(_lora, "sg_lora_gemm", LORA, kw) == code


LORA_BACK = dict(T=3, K=40, N=48, r=16, L=5, dy=P[8], lddy=48, x=P[0], ldx=40, ids=P[1], a=P[2], b=P[3], scale=P[4],
                 base=P[5], ldb=40, dx=P[6], lddx=40, da=P[9], db=P[10], dt=0, ws=P[7], wsb=1 << 40, st=None)


@no_gpu
@pytest.mark.parametrize("kw,code", [
    *LORA_SHARED, *[({n: None}, NULL) for n in ("dy", "da", "db")], (dict(dx=None, da=None, db=None), NULL),
    (dict(dt=2), UNSUP), (dict(lddy=40), SHAPE), (dict(lddx=32), SHAPE), (dict(ldb=32), SHAPE),
    (dict(base=P[6], ldb=48), SHAPE), (dict(lddy=52), ALIGN), (dict(lddx=44), ALIGN), (dict(ldb=44), ALIGN),
    *[({n: ODD}, ALIGN) for n in ("dy", "dx", "da", "db")],
])
def test_lora_backward_refusals(kw, code):
    assert call(_lora, "sg_lora_gemm_backward", LORA_BACK, kw) == code


def test_lora_workspaces():
    assert sg.lora_gemm_workspace(1, 4096, 4096, 16, 8) == 0 and sg.lora_gemm_backward_workspace(1, 4096, 4096, 16, 8) > 0
    for need in (sg.lora_gemm_workspace, sg.lora_gemm_backward_workspace):
        assert need(70000, 64, 64, 16, 1) >= 4 * 70000 * 16
        for bad in ((0, 8, 8, 8, 1), (1, 4, 8, 8, 1), (1, 8, 12, 8, 1), (1, 8, 8, 4, 1), (1, 8, 8, 264, 1), (1, 8, 8, 8, 0),
                    (1, 8, 8, 8, 65536), (BIG, 8, 8, 8, 1), (1, BIG, 8, 8, 1)):
            assert need(*bad) == -1
    assert sg.lora_gemm_backward_workspace(80, 64, 64, 16, 1) > sg.lora_gemm_workspace(80, 64, 64, 16, 1) > 0


@pytest.mark.parametrize("call", [
    lambda t: sg.gated_gemm(t(2, 8), t(8, 8), t(8, 8)),
    lambda t: sg.gated_gemm_backward(t(2, 8), t(2, 8), t(8, 8), t(8, 8)),
    lambda t: sg.lora_gemm(t(2, 8), None, t(1, 8, 8), t(1, 8, 8)),
    lambda t: sg.lora_gemm_backward(t(2, 8), t(2, 8), None, t(1, 8, 8), t(1, 8, 8)),
])
def test_host_tensors_are_refused(call):
    with pytest.raises(sg.SgError):
        call(lambda *s: torch.zeros(s, dtype=torch.bfloat16))
