"""The mixture-of-experts entry points: exported, bound one to one, and refusing
invalid arguments on the host before any HIP call (fake, never dereferenced
addresses; only where no GPU is visible)."""
import ctypes
import os
import re

import pytest
import torch

import sparse_gemm_layers_amd as sg
from sparse_gemm_layers_amd import _moe as B

HEADER = os.path.join(os.path.dirname(sg.__file__), "include", "sg_moe.h")
OK, NULL, SHAPE, UNSUP, ALIGN, HIP = range(6)
P, P2, P3, P4, P5, P6, P7, P8 = (ctypes.c_void_p(0x100000 * (i + 1)) for i in range(8))
ODD = ctypes.c_void_p(0x100004)     # 4- but not 16-byte aligned
ODD1 = ctypes.c_void_p(0x100001)

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run only without a GPU")


def test_header_binding_and_library_agree():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(sg_[a-z0-9_]+)\s*\(", src)))
    assert names == sorted(B._SIGS)
    for n in names:
        assert hasattr(B._lib(), n), n
    for n in names:
        assert n[3:] in sg.__all__


def call(name, base, order, kw):
    a = dict(base, **kw)
    return getattr(B._lib(), name)(*[a[k] for k in order])


ROUTE = dict(l=P, dt=0, T=4, E=64, ldl=64, bias=P2, k=8, score=0, ng=8, tg=4, gs=1, rn=1, sc=1.0, ids=P3, w=P4, st=None)


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(l=None), NULL), (dict(ids=None), NULL), (dict(w=None), NULL), (dict(dt=2), UNSUP), (dict(score=2), UNSUP),
    (dict(gs=-1), UNSUP), (dict(T=0), SHAPE), (dict(E=0), SHAPE), (dict(E=1025, ldl=2000, ng=1, tg=1), SHAPE),
    (dict(ldl=63), SHAPE), (dict(k=0), SHAPE), (dict(k=65), SHAPE), (dict(k=33), SHAPE), (dict(ng=7), SHAPE),
    (dict(ng=0), SHAPE), (dict(ng=128, E=256, ldl=256), SHAPE), (dict(tg=0), SHAPE), (dict(tg=9), SHAPE),
    (dict(E=4, ldl=4, ng=1, tg=1, k=5), SHAPE), (dict(l=ODD1), ALIGN), (dict(bias=ODD1), ALIGN),
    (dict(ids=ODD1), ALIGN), (dict(w=ODD1), ALIGN),
])
def test_route_refusals(kw, code):
    assert call("sg_moe_route", ROUTE, list(ROUTE), kw) == code


GRAD = dict(g=P, l=P2, dt=1, T=4, E=64, ldl=64, ids=P3, k=8, score=0, rn=0, sc=1.0, d=P4, ldd=64, st=None)


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(g=None), NULL), (dict(l=None), NULL), (dict(ids=None), NULL), (dict(d=None), NULL), (dict(dt=3), UNSUP),
    (dict(score=-1), UNSUP), (dict(T=-1), SHAPE), (dict(E=1025, ldl=2000, ldd=2000), SHAPE), (dict(ldl=1), SHAPE),
    (dict(ldd=63), SHAPE), (dict(k=0), SHAPE), (dict(k=65), SHAPE), (dict(E=4, k=5), SHAPE), (dict(g=ODD1), ALIGN),
    (dict(l=ODD1), ALIGN), (dict(d=ODD1), ALIGN), (dict(ids=ODD1), ALIGN),
])
def test_route_backward_refusals(kw, code):
    assert call("sg_moe_route_backward", GRAD, list(GRAD), kw) == code


@pytest.mark.parametrize("n,k,gc,want", [
    (16, 128, 128, 1088), (17, 128, 128, 2176), (1, 32, 32, 1280), (100, 192, 64, 7 * 2 * 1152), (16, 128, 16, -1),
    (16, 100, 32, -1), (0, 128, 128, -1), (16, 0, 64, -1), (16, 192, 128, -1), (16, (1 << 24) + 128, 128, -1),
    ((1 << 31) + 1, 128, 128, -1),
])
def test_w4_packed_bytes(n, k, gc, want):
    assert sg.w4_packed_bytes(n, k, gc) == want


PACK = dict(L=2, wq=P, ldw=64, wbs=6400, s=P2, ssn=1, ssk=100, sbs=100, N=100, K=128, gc=128, out=P3, st=None)


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(wq=None), NULL), (dict(s=None), NULL), (dict(out=None), NULL), (dict(gc=16), UNSUP), (dict(L=0), SHAPE),
    (dict(N=0), SHAPE), (dict(K=96), SHAPE), (dict(ldw=60), SHAPE), (dict(ssn=-1), SHAPE), (dict(wbs=-4), SHAPE),
    (dict(L=1 << 40), SHAPE), (dict(ldw=66), ALIGN), (dict(wbs=6402), ALIGN), (dict(wq=ODD1), ALIGN),
    (dict(s=ODD1), ALIGN), (dict(out=ODD), ALIGN),
])
def test_w4_pack_refusals(kw, code):
    assert call("sg_w4_pack", PACK, list(PACK), kw) == code


GEMM = dict(M=3, N=100, K=256, x=P, ldx=256, w=P2, gc=64, bias=P3, y=P4, dt=1, ldy=100, st=None)


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None), NULL), (dict(gc=256), UNSUP), (dict(dt=2), UNSUP),
    (dict(M=0), SHAPE), (dict(N=0), SHAPE), (dict(K=100), SHAPE), (dict(ldx=128), SHAPE), (dict(ldy=99), SHAPE),
    (dict(ldx=1 << 22), SHAPE), (dict(M=1 << 31), SHAPE), (dict(x=ODD), ALIGN), (dict(ldx=260), ALIGN),
    (dict(w=ODD), ALIGN), (dict(bias=ODD1), ALIGN), (dict(y=ODD1), ALIGN),
])
def test_w4a16_gemm_refusals(kw, code):
    assert call("sg_w4a16_gemm_groupwise_packed", GEMM, list(GEMM), kw) == code


MLP = dict(T=3, k=2, E=8, D=128, F=256, x=P, ldx=128, ids=P2, w=P3, gate=P4, up=P5, down=P6, gc=64, y=P7, dt=1, ldy=128,
           ws=P8, wsb=1 << 30, st=None)


@no_gpu
@pytest.mark.parametrize("kw,code", [
    *[({n: None}, NULL) for n in ("x", "ids", "w", "gate", "up", "down", "y", "ws")],
    (dict(gc=100), UNSUP), (dict(dt=3), UNSUP), (dict(T=0), SHAPE), (dict(k=0), SHAPE), (dict(E=0), SHAPE),
    (dict(E=1025), SHAPE), (dict(D=96, ldx=96, ldy=96), SHAPE), (dict(F=96), SHAPE), (dict(F=0), SHAPE),
    (dict(ldx=64), SHAPE), (dict(ldy=64), SHAPE), (dict(ldy=130), SHAPE), (dict(wsb=1000), SHAPE),
    (dict(T=1 << 30), SHAPE), (dict(x=ODD), ALIGN), (dict(ldx=132), ALIGN), (dict(gate=ODD), ALIGN),
    (dict(up=ODD), ALIGN), (dict(down=ODD), ALIGN), (dict(y=ODD), ALIGN), (dict(ws=ODD), ALIGN),
    (dict(ids=ODD1), ALIGN), (dict(w=ODD1), ALIGN),
])
def test_moe_mlp_refusals(kw, code):
    assert call("sg_w4a16_moe_mlp", MLP, list(MLP), kw) == code


def test_moe_mlp_workspace_size():
    ws = sg.w4a16_moe_mlp_workspace
    assert ws(1, 8, 64, 4096, 1024) > 0
    assert ws(2, 8, 64, 4096, 1024) > ws(1, 8, 64, 4096, 1024)
    for bad in ((0, 1, 1, 32, 32), (1, 0, 1, 32, 32), (1, 1, 0, 32, 32), (1, 1, 1025, 32, 32), (1, 1, 1, 33, 32),
                (1, 1, 1, 32, 0), (1 << 30, 2, 1, 32, 32), (1, 1, 1, 1 << 22, 32)):
        assert ws(*bad) == -1


@pytest.mark.parametrize("call", [
    lambda t: sg.moe_route(t(2, 8), 2),
    lambda t: sg.moe_route_backward(t(2, 2), t(2, 8), torch.zeros((2, 2), dtype=torch.int32)),
    lambda t: sg.w4_pack(torch.zeros((4, 64), dtype=torch.uint8), t(4, 1)),
    lambda t: sg.w4a16_gemm_groupwise_packed(t(2, 128).bfloat16(), torch.zeros(1088, dtype=torch.uint8), 4),
    lambda t: sg.w4a16_moe_mlp(t(2, 128).bfloat16(), None, None, None, None, None, 128),
])
def test_host_tensors_are_refused(call):
    with pytest.raises(sg.SgError):
        call(lambda *s: torch.zeros(s))
