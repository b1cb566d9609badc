"""ctypes binding of the mixture-of-experts entry points of libsg.so
(``sparse_gemm_layers_amd/include/sg_moe.h``).  Argument marshalling only."""

import ctypes

import torch

from ._binding import (SgError, _FB, _check, _dtype_code, _gpu2d, _i64, _int, _p, _positive, _ptr,
                       _row_stride, _stream, _want, lib)

_f32 = ctypes.c_float

_SIGS = {
    "sg_moe_route": ([_ptr, _int, _i64, _i64, _i64, _ptr, _int, _int, _int, _int, _int, _int, _f32, _ptr, _ptr, _ptr],
                     _int),
    "sg_moe_route_backward": ([_ptr, _ptr, _int, _i64, _i64, _i64, _ptr, _int, _int, _int, _f32, _ptr, _i64, _ptr],
                              _int),
    "sg_w4_packed_bytes": ([_i64, _i64, _int], _i64),
    "sg_w4_pack": ([_i64, _ptr, _i64, _i64, _ptr, _i64, _i64, _i64, _i64, _i64, _int, _ptr, _ptr], _int),
    "sg_w4a16_gemm_groupwise_packed": ([_i64, _i64, _i64, _ptr, _i64, _ptr, _int, _ptr, _ptr, _int, _i64, _ptr], _int),
    "sg_w4a16_moe_mlp_workspace": ([_i64, _int, _i64, _i64, _i64], _i64),
    "sg_w4a16_moe_mlp": ([_i64, _int, _i64, _i64, _i64, _ptr, _i64, _ptr, _ptr, _ptr, _ptr, _ptr, _int, _ptr, _int,
                          _i64, _ptr, _i64, _ptr], _int),
}

_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"max": 0, "top2": 1}
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


def _want_rows(t, name, dtype, shape, device):
    """A contiguous GPU tensor of one dtype and shape (None entries: any size)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise SgError(f"{name} must be a GPU tensor")
    if t.device != device:
        raise SgError(f"{name} is on {t.device}, the operands on {device}")
    if t.dtype != dtype:
        raise SgError(f"{name}: dtype {t.dtype} not supported ({str(dtype).replace('torch.', '')})")
    if t.dim() != len(shape) or any(w is not None and w != h for w, h in zip(shape, t.shape)):
        raise SgError(f"{name} must have shape [{', '.join('*' if w is None else str(w) for w in shape)}], "
                      f"got {list(t.shape)}")
    if not t.is_contiguous():
        raise SgError(f"{name} must be contiguous")
    return t


def _score_code(score):
    if score not in _SCORES:
        raise SgError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    return _SCORES[score]


def moe_route(logits, k: int, score: str = "softmax", bias=None, n_group: int = 1, topk_group: int = 1,
              group_score: str = "max", renormalize: bool = False, scale: float = 1.0, ids=None, weights=None):
    """logits [T, E] float32/bfloat16 -> (ids int32 [T, k], weights float32 [T, k]),
    the experts of each token, best first (-1 and weight 0 where none is left).

    An expert's key is its logit, or score + bias (float32 [E]) where there is a
    bias; with n_group > 1 only the topk_group groups of E / n_group experts with
    the largest value (the group's largest key, "max", or the sum of its two
    largest score + bias, "top2") stay.  Weights are the scores of the chosen,
    divided by their sum if `renormalize`, times `scale`.  Ties go to the lowest
    index; -inf or NaN takes an expert out."""
    _gpu2d(logits, "logits")
    T, E = logits.shape
    _positive(T=T, E=E, k=k)
    dt = _dtype_code(logits, "logits")
    sc = _score_code(score)
    if group_score not in _GROUP_SCORES:
        raise SgError(f"group_score must be 'max' or 'top2', got {group_score!r}")
    if bias is not None:
        _want_rows(bias, "bias", torch.float32, (E,), logits.device)
    if ids is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    if weights is None:
        weights = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _want_rows(ids, "ids", torch.int32, (T, k), logits.device)
    _want_rows(weights, "weights", torch.float32, (T, k), logits.device)
    st = _lib().sg_moe_route(_p(logits), dt, T, E, _row_stride(logits), _p(bias), k, sc, n_group, topk_group,
                             _GROUP_SCORES[group_score], int(bool(renormalize)), scale, _p(ids), _p(weights),
                             _stream(logits))
    _check(st, "sg_moe_route")
    return ids, weights


def moe_route_backward(grad, logits, ids, score: str = "softmax", renormalize: bool = False, scale: float = 1.0,
                       dlogits=None):
    """Gradient of moe_route's weights: grad float32 [T, k], the logits and ids of
    the forward call -> dlogits [T, E] of the logits' dtype (the choice of experts
    held fixed; groups and bias enter through ids alone)."""
    _gpu2d(logits, "logits")
    T, E = logits.shape
    _positive(T=T, E=E)
    dt = _dtype_code(logits, "logits")
    sc = _score_code(score)
    _want_rows(ids, "ids", torch.int32, (T, None), logits.device)
    k = ids.shape[1]
    _positive(k=k)
    _want_rows(grad, "grad", torch.float32, (T, k), logits.device)
    if dlogits is None:
        dlogits = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    _gpu2d(_want(dlogits, "dlogits", (logits.dtype,), (T, E), logits.device), "dlogits")
    st = _lib().sg_moe_route_backward(_p(grad), _p(logits), dt, T, E, _row_stride(logits), _p(ids), k, sc,
                                      int(bool(renormalize)), scale, _p(dlogits), _row_stride(dlogits),
                                      _stream(logits))
    _check(st, "sg_moe_route_backward")
    return dlogits


def w4_packed_bytes(n: int, k: int, gc: int = 128) -> int:
    """Bytes of the packed form of an n x k 4-bit weight (-1: there is none)."""
    return int(_lib().sg_w4_packed_bytes(n, k, gc))


def _packed_bytes(n, k, gc):
    need = w4_packed_bytes(n, k, gc)
    if need < 0:
        raise SgError(f"no packed 4-bit form for N = {n}, K = {k}, gc = {gc} (gc 32, 64 or 128 dividing K)")
    return need


def w4_pack(wq, s, gc: int = 128, packed=None):
    """int4 codes wq uint8 [N, K/2] (element 2j in the low nibble of byte j, as
    int4_quant_groupwise writes them) and scales s float32 [N, K/gc] (any strides)
    -> the packed weight, uint8 [w4_packed_bytes(N, K, gc)].  With a leading
    dimension of L weights: uint8 [L, bytes]."""
    if not isinstance(wq, torch.Tensor) or not wq.is_cuda:
        raise SgError("wq must be a GPU tensor")
    if wq.dim() not in (2, 3) or wq.dtype != torch.uint8 or (wq.shape[-1] > 1 and wq.stride(-1) != 1):
        raise SgError("wq must be uint8 [N, K/2] or [L, N, K/2] with unit column stride")
    batch = wq.shape[:-2]
    L, n, k = (wq.shape[0] if batch else 1), wq.shape[-2], wq.shape[-1] * 2
    _positive(L=L, N=n, K=k)
    need = _packed_bytes(n, k, gc)
    if not isinstance(s, torch.Tensor) or not s.is_cuda or s.dtype != torch.float32 or s.device != wq.device:
        raise SgError("s must be a float32 tensor on wq's GPU")
    if tuple(s.shape) != (*batch, n, k // gc):
        raise SgError(f"s must have shape {[*batch, n, k // gc]}, got {list(s.shape)}")
    if packed is None:
        packed = torch.empty((*batch, need), dtype=torch.uint8, device=wq.device)
    _want_rows(packed, "packed", torch.uint8, (*batch, need), wq.device)
    ldw = wq.stride(-2) if n > 1 else k // 2
    st = _lib().sg_w4_pack(L, _p(wq), ldw, wq.stride(0) if L > 1 else 0, _p(s), s.stride(-2), s.stride(-1),
                           s.stride(0) if L > 1 else 0, n, k, gc, _p(packed), _stream(wq))
    _check(st, "sg_w4_pack")
    return packed


def _want_w4(w, name, need, device, batch=None):
    if not isinstance(w, torch.Tensor) or not w.is_cuda or w.dtype != torch.uint8:
        raise SgError(f"{name} must be a uint8 GPU tensor")
    if w.device != device:
        raise SgError(f"{name} is on {w.device}, the operands on {device}")
    want = (need,) if batch is None else (batch, need)
    if tuple(w.shape) != want or not w.is_contiguous():
        raise SgError(f"{name} must be a contiguous packed weight {list(want)}, got {list(w.shape)}")


def w4a16_gemm_groupwise_packed(x, wpacked, n: int, gc: int = 128, out_dtype=torch.bfloat16, bias=None, y=None):
    """Y [M, n] = X . W^T + bias: x bfloat16 [M, K], wpacked from w4_pack (n rows,
    groups of gc columns), bias float32 [n]; fp32 sums, bf16 or fp32 out."""
    _gpu2d(x, "x")
    if x.dtype != torch.bfloat16:
        raise SgError("x must be bfloat16")
    M, K = x.shape
    _positive(M=M, N=n, K=K)
    _want_w4(wpacked, "wpacked", _packed_bytes(n, K, gc), x.device)
    if bias is not None:
        _want_rows(bias, "bias", torch.float32, (n,), x.device)
    if y is None:
        y = torch.empty((M, n), dtype=out_dtype, device=x.device)
    _gpu2d(_want(y, "y", _FB, (M, n), x.device), "y")
    st = _lib().sg_w4a16_gemm_groupwise_packed(M, n, K, _p(x), _row_stride(x), _p(wpacked), gc, _p(bias), _p(y),
                                               _dtype_code(y, "y"), _row_stride(y), _stream(x))
    _check(st, "sg_w4a16_gemm_groupwise_packed")
    return y


def w4a16_moe_mlp_workspace(t: int, k: int, e: int, d: int, f: int) -> int:
    """Bytes of workspace of a w4a16_moe_mlp call (-1: sizes out of range)."""
    return int(_lib().sg_w4a16_moe_mlp_workspace(t, k, e, d, f))


def w4a16_moe_mlp(x, ids, weights, gate, up, down, f: int, gc: int = 128, out_dtype=torch.bfloat16, y=None,
                  workspace=None):
    """y[t] = sum_j weights[t, j] * Wd_e (silu(Wg_e x_t) * (Wu_e x_t)), e = ids[t, j].

    x bfloat16 [T, D]; ids int32 and weights float32 [T, k] as moe_route gives
    them (an id outside [0, E) contributes nothing); gate, up uint8 [E, bytes] from
    w4_pack of E weights [f, D], down of E weights [D, f].  workspace: uint8, at least
    w4a16_moe_mlp_workspace(T, k, E, D, f) bytes (allocated if not given; keep it
    to one stream)."""
    _gpu2d(x, "x")
    if x.dtype != torch.bfloat16:
        raise SgError("x must be bfloat16")
    T, D = x.shape
    _positive(T=T, D=D, F=f)
    _want_rows(ids, "ids", torch.int32, (T, None), x.device)
    k = ids.shape[1]
    _positive(k=k)
    _want_rows(weights, "weights", torch.float32, (T, k), x.device)
    if not isinstance(gate, torch.Tensor) or gate.dim() != 2:
        raise SgError("gate must be packed weights [E, bytes]")
    E = gate.shape[0]
    _positive(E=E)
    _want_w4(gate, "gate", _packed_bytes(f, D, gc), x.device, E)
    _want_w4(up, "up", _packed_bytes(f, D, gc), x.device, E)
    _want_w4(down, "down", _packed_bytes(D, f, gc), x.device, E)
    need = w4a16_moe_mlp_workspace(T, k, E, D, f)
    if need < 0:
        raise SgError(f"w4a16_moe_mlp: sizes out of range (T = {T}, k = {k}, E = {E}, D = {D}, F = {f})")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 or not workspace.is_contiguous() \
            or workspace.numel() < need or workspace.device != x.device:
        raise SgError(f"workspace must be a contiguous uint8 tensor of at least {need} bytes on {x.device}")
    if y is None:
        y = torch.empty((T, D), dtype=out_dtype, device=x.device)
    _gpu2d(_want(y, "y", _FB, (T, D), x.device), "y")
    st = _lib().sg_w4a16_moe_mlp(T, k, E, D, f, _p(x), _row_stride(x), _p(ids), _p(weights), _p(gate), _p(up),
                                 _p(down), gc, _p(y), _dtype_code(y, "y"), _row_stride(y), _p(workspace), workspace.numel(), _stream(x))
    _check(st, "sg_w4a16_moe_mlp")
    return y
