"""ctypes binding of the low-rank adapters' entry points of libsg.so
(``sparse_gemm_layers_amd/include/sg_lora.h``).  Argument marshalling only."""

import ctypes
import functools

import torch

from ._binding import SgError, _FB, _check, _i64, _int, _ptr, lib
from ._gated import _at, _launch, _ld, _space
from ._moe import _BF, _CODE, _matrix, _refuse

_SIGS = {
    "sg_lora_gemm_workspace": ([_i64, _i64, _i64, _int, _i64], _i64),
    "sg_lora_gemm": ([_i64, _i64, _i64, _int, _i64, _ptr, _i64, _ptr, _ptr, _ptr, _ptr, _ptr, _int, _i64, _ptr, _int,
                      _i64, _ptr, _i64, _ptr], _int),
    "sg_lora_gemm_backward_workspace": ([_i64, _i64, _i64, _int, _i64], _i64),
    "sg_lora_gemm_backward": ([_i64, _i64, _i64, _int, _i64, _ptr, _i64, _ptr, _i64, _ptr, _ptr, _ptr, _ptr, _ptr, _i64,
                               _ptr, _i64, _ptr, _ptr, _int, _ptr, _i64, _ptr], _int),
    "sg_lora_gemm_plan": ([_i64, _i64, _i64, _int, _i64, _ptr], _int),
    "sg_lora_gemm_backward_plan": ([_i64, _i64, _i64, _int, _i64, _ptr], _int),
}

_typed = None


def _lib():
    """libsg.so with this module's entry points typed too."""
    global _typed
    h = lib()
    if _typed is not h:
        for name, (args, res) in _SIGS.items():
            fn = getattr(h, name)
            fn.argtypes = args
            fn.restype = res
        _typed = h
    return h


def lora_gemm_workspace(t: int, k: int, n: int, r: int, l: int) -> int:
    """Bytes of workspace of a lora_gemm call (-1: sizes out of range)."""
    return int(_lib().sg_lora_gemm_workspace(t, k, n, r, l))


def lora_gemm_backward_workspace(t: int, k: int, n: int, r: int, l: int) -> int:
    """Bytes of workspace of a lora_gemm_backward call (-1: sizes out of range)."""
    return int(_lib().sg_lora_gemm_backward_workspace(t, k, n, r, l))


@functools.lru_cache(maxsize=1024)
def _need(back, t, k, n, r, l):
    need = (lora_gemm_backward_workspace if back else lora_gemm_workspace)(t, k, n, r, l)
    if need < 0:
        more = ", and ceil(max(K, N) / 256) (2 L ceil(r / 64) + ceil(T / 64)) under 2^24 - 4096" if back else ""
        raise SgError(f"low-rank adapters: sizes out of range (T = {t}, K = {k}, N = {n}, r = {r}, L = {l}; K, N and r "
                      f"multiples of 8, r at most 256, L at most 65535, T, K and N under 2^22{more})")
    return need


def _adapters(x, ids, a, b, scale):
    """(T, K, N, r, L, row stride of x, addresses of ids, a, b and scale, index of their GPU)."""
    T, K, ldx = _matrix(x, "x", _BF)
    dev = x.get_device()
    if not isinstance(a, torch.Tensor) or a.dim() != 3 or not isinstance(b, torch.Tensor) or b.dim() != 3:
        raise SgError("a and b must be GPU tensors [L, r, K] and [L, N, r]")
    L, r, _ = a.shape
    N = b.shape[1]
    if L < 1 or r < 1 or N < 1:
        raise SgError(f"L, r and N must be at least 1, got {L}, {r} and {N}")
    pa, pb = _at(a, "a", torch.bfloat16, (L, r, K), dev), _at(b, "b", torch.bfloat16, (L, N, r), dev)
    pi = None if ids is None else _at(ids, "ids", torch.int32, (T,), dev)
    ps = None if scale is None else _at(scale, "scale", torch.float32, (L,), dev)
    return T, K, N, r, L, ldx, pi, pa, pb, ps, dev


def lora_gemm(x, ids, a, b, scale=None, base=None, out_dtype=torch.bfloat16, y=None, workspace=None):
    """y[t] = base[t] + scale[e] (x[t] . a[e]^T) . b[e]^T, e = ids[t].

    x bfloat16 [T, K]; ids int32 [T] (outside [0, L): no adapter, y is base or 0; None:
    adapter 0 for every token); a bfloat16 [L, r, K], b bfloat16 [L, N, r] (a smaller
    rank is padded with zeros); scale float32 [L] or None for 1; base [T, N] float32 or
    bfloat16: the shared projection's output, from any of the library's products, or
    None for 0.  y may be base: then the adapters are added in place.  fp32 sums, the
    inner product included; y is rounded once.  workspace: uint8, at least
    lora_gemm_workspace(T, K, N, r, L) bytes where that is not 0 (allocated if not
    given; keep it to one stream)."""
    T, K, N, r, L, ldx, pi, pa, pb, ps, dev = _adapters(x, ids, a, b, scale)
    ldb = 0 if base is None else _ld(base, "base", _FB, (T, N), dev)
    if y is None:
        if out_dtype not in _CODE:
            raise SgError(f"out_dtype {out_dtype} not supported (float32 or bfloat16)")
        y = x.new_empty((T, N), dtype=out_dtype)
        ldy = N
    else:
        ldy = _ld(y, "y", _FB, (T, N), dev)
    need, pw, wn = _need(False, T, K, N, r, L), None, 0
    if need:
        workspace = _space(workspace, need, x, dev)
        pw, wn = workspace.data_ptr(), workspace.numel()
    st = _launch(dev, _lib().sg_lora_gemm, T, K, N, r, L, x.data_ptr(), ldx, pi, pa, pb, ps,
                 None if base is None else base.data_ptr(), 0 if base is None else _CODE[base.dtype], ldb, y.data_ptr(),
                 _CODE[y.dtype], ldy, pw, wn)
    if st:
        _check(st, "sg_lora_gemm")
    return y


def lora_gemm_backward(dy, x, ids, a, b, scale=None, base=None, need_dx: bool = True, need_dab: bool = True,
                       grad_dtype=torch.bfloat16, dx=None, da=None, db=None, workspace=None):
    """Gradients of lora_gemm for dy bfloat16 [T, N], the gradient of y (and so of its
    base): (dx bfloat16 [T, K], da [L, r, K], db [L, N, r]); None where not needed.

    dx[t] = base[t] + scale[e] (dy[t] . b[e]) . a[e], with base bfloat16 [T, K] what else
    contributes to the gradient of x (None: 0; it may be dx itself); da and db, of
    grad_dtype, are sums over the adapter's own tokens, zeros where it has none.
    workspace: uint8, at least lora_gemm_backward_workspace(T, K, N, r, L) bytes
    (allocated if not given; keep it to one stream)."""
    T, K, N, r, L, ldx, pi, pa, pb, ps, dev = _adapters(x, ids, a, b, scale)
    ld_dy = _ld(dy, "dy", _BF, (T, N), dev)
    ldb = 0 if base is None else _ld(base, "base", _BF, (T, K), dev)
    if grad_dtype not in _CODE:
        raise SgError(f"grad_dtype {grad_dtype} not supported (float32 or bfloat16)")
    pdx, ldd = None, K
    if dx is not None:
        ldd, pdx = _ld(dx, "dx", _BF, (T, K), dev), dx.data_ptr()
    elif need_dx:
        dx = x.new_empty((T, K))
        pdx = dx.data_ptr()
    pda = pdb = None
    if da is not None or db is not None:
        if da is None or db is None:
            raise SgError("da and db go together")
        if not isinstance(da, torch.Tensor) or da.dtype not in _CODE:
            _refuse(da, "da", _FB, (L, r, K), x.device)
        pda = _at(da, "da", da.dtype, (L, r, K), dev)
        pdb = _at(db, "db", da.dtype, (L, N, r), dev)
    elif need_dab:
        da, db = x.new_empty((L, r, K), dtype=grad_dtype), x.new_empty((L, N, r), dtype=grad_dtype)
        pda, pdb = da.data_ptr(), db.data_ptr()
    if pdx is None and pda is None:
        return None, None, None
    workspace = _space(workspace, _need(True, T, K, N, r, L), x, dev)
    st = _launch(dev, _lib().sg_lora_gemm_backward, T, K, N, r, L, dy.data_ptr(), ld_dy, x.data_ptr(), ldx, pi, pa, pb, ps,
                 None if base is None else base.data_ptr(), ldb, pdx, ldd, pda, pdb, 0 if pda is None else _CODE[da.dtype],
                 workspace.data_ptr(), workspace.numel())
    if st:
        _check(st, "sg_lora_gemm_backward")
    return dx, da, db


def _plan(name, fields, t, k, n, r, l):
    out = (ctypes.c_int32 * len(fields))()
    _check(getattr(_lib(), name)(t, k, n, r, l, ctypes.addressof(out)), name)
    return dict(zip(fields, out))


def lora_gemm_plan(t: int, k: int, n: int, r: int, l: int):
    """How lora_gemm goes at these sizes: launches (1: both products in one), tokens of an adapter
    taken at a time, ranks of a workgroup of x . a^T, parts of its sum."""
    return _plan("sg_lora_gemm_plan", ("launches", "tokens", "ranks", "parts"), t, k, n, r, l)


def lora_gemm_backward_plan(t: int, k: int, n: int, r: int, l: int):
    """How lora_gemm_backward goes at these sizes: tokens taken at a time and ranks of a workgroup of
    dy . b and x . a^T, the parts of either sum, ranks of a workgroup of da and db, parts of
    their tokens."""
    return _plan("sg_lora_gemm_backward_plan", ("tokens", "ranks", "parts_v", "parts_u", "sum_ranks", "token_parts"), t, k, n,
                 r, l)
