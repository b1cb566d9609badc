"""ctypes binding of the mixture-of-experts entry points of libsg.so
(``sparse_gemm_layers_amd/include/sg_moe.h``).  Argument marshalling only."""

import ctypes
import functools

import torch

from ._binding import SgError, _FB, _check, _i64, _int, _p, _positive, _ptr, _stream, lib

# A call on a few tokens costs the host more than the GPU (a launch alone is 4 us), so
# operands are checked by one expression each, which names the fault only where there is
# one, and addresses go to ctypes as integers: a one-token linear layer took 12.5 us with
# the other modules' helpers and takes 7.6 us with these.

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


def _refuse(t, name, dtypes, shape, device):
    """Raises with the first thing that is wrong about operand t."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise SgError(f"{name} must be a GPU tensor")
    if t.device != device:
        raise SgError(f"{name} is on {t.device}, the operands on {device}")
    if t.dtype not in dtypes:
        want = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise SgError(f"{name}: dtype {t.dtype} not supported ({want})")
    if tuple(t.shape) != shape:
        raise SgError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    raise SgError(f"{name} must be contiguous")


def _rows(t, name, dtype, shape, device):
    """Address of a contiguous GPU tensor of one dtype and shape."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.shape == shape
            and t.is_contiguous() and t.device == device):
        _refuse(t, name, (dtype,), shape, device)
    return t.data_ptr()


def _matrix(t, name, dtypes):
    """(rows, columns, row stride) of a GPU matrix with unit column stride, none of them 0."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise SgError(f"{name} must be a GPU tensor")
    if t.dim() != 2:
        raise SgError(f"{name} must be 2-D with unit column stride")
    if t.dtype not in dtypes:
        _refuse(t, name, dtypes, None, t.device)
    r, c = t.shape
    ld, one = t.stride()
    if r < 1 or c < 1 or (one != 1 and c > 1):
        raise SgError(f"{name} must be 2-D with unit column stride and no empty side, got {[r, c]}, strides {[ld, one]}")
    return r, c, (ld if r > 1 else c)


def _result(t, name, dtypes, shape, device):
    """Row stride of an output matrix that the caller gave."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.device == device and t.dtype in dtypes and t.shape == shape):
        _refuse(t, name, dtypes, shape, device)
    return _matrix(t, name, dtypes)[2]


def _current_stream(t):
    return torch._C._cuda_getCurrentRawStream(t.get_device())


_CODE = {torch.float32: 0, torch.bfloat16: 1}
_BF = (torch.bfloat16,)


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
    divided by their sum if `renormalize`, times `scale`; softmax weights are within
    32 steps of 2^-24, and may differ by that between calls of few and of many
    tokens.  Ties go to the lowest index; -inf or NaN takes an expert out."""
    T, E, ld = _matrix(logits, "logits", _FB)
    dev = logits.device
    if k < 1:
        raise SgError(f"k must be at least 1, got {k}")
    sc = _score_code(score)
    if group_score not in _GROUP_SCORES:
        raise SgError(f"group_score must be 'max' or 'top2', got {group_score!r}")
    pb = None if bias is None else _rows(bias, "bias", torch.float32, (E,), dev)
    if ids is None:
        ids = logits.new_empty((T, k), dtype=torch.int32)
        pi = ids.data_ptr()
    else:
        pi = _rows(ids, "ids", torch.int32, (T, k), dev)
    if weights is None:
        weights = logits.new_empty((T, k), dtype=torch.float32)
        pw = weights.data_ptr()
    else:
        pw = _rows(weights, "weights", torch.float32, (T, k), dev)
    st = _lib().sg_moe_route(logits.data_ptr(), _CODE[logits.dtype], T, E, ld, pb, k, sc, n_group, topk_group,
                             _GROUP_SCORES[group_score], 1 if renormalize else 0, scale, pi, pw,
                             _current_stream(logits))
    if st:
        _check(st, "sg_moe_route")
    return ids, weights


def moe_route_backward(grad, logits, ids, score: str = "softmax", renormalize: bool = False, scale: float = 1.0,
                       dlogits=None):
    """Gradient of moe_route's weights: grad float32 [T, k], the logits and ids of
    the forward call -> dlogits [T, E] of the logits' dtype (the choice of experts
    held fixed; groups and bias enter through ids alone)."""
    T, E, ld = _matrix(logits, "logits", _FB)
    dev = logits.device
    sc = _score_code(score)
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise SgError("ids must be int32 [T, k]")
    k = ids.shape[1]
    if k < 1:
        raise SgError("k must be at least 1, got 0")
    pi = _rows(ids, "ids", torch.int32, (T, k), dev)
    pg = _rows(grad, "grad", torch.float32, (T, k), dev)
    if dlogits is None:
        dlogits = logits.new_empty((T, E))
        ldd = E
    else:
        ldd = _result(dlogits, "dlogits", (logits.dtype,), (T, E), dev)
    st = _lib().sg_moe_route_backward(pg, logits.data_ptr(), _CODE[logits.dtype], T, E, ld, pi, k, sc,
                                      1 if renormalize else 0, scale, dlogits.data_ptr(), ldd,
                                      _current_stream(logits))
    if st:
        _check(st, "sg_moe_route_backward")
    return dlogits


def w4_packed_bytes(n: int, k: int, gc: int = 128) -> int:
    """Bytes of the packed form of an n x k 4-bit weight (-1: there is none)."""
    return int(_lib().sg_w4_packed_bytes(n, k, gc))


@functools.lru_cache(maxsize=1024)
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
    _rows(packed, "packed", torch.uint8, (*batch, need), wq.device)
    ldw = wq.stride(-2) if n > 1 else k // 2
    st = _lib().sg_w4_pack(L, _p(wq), ldw, wq.stride(0) if L > 1 else 0, _p(s), s.stride(-2), s.stride(-1),
                           s.stride(0) if L > 1 else 0, n, k, gc, _p(packed), _stream(wq))
    _check(st, "sg_w4_pack")
    return packed


def w4a16_gemm_groupwise_packed(x, wpacked, n: int, gc: int = 128, out_dtype=torch.bfloat16, bias=None, y=None):
    """Y [M, n] = X . W^T + bias: x bfloat16 [M, K], wpacked from w4_pack (n rows,
    groups of gc columns), bias float32 [n]; fp32 sums, bf16 or fp32 out."""
    M, K, ldx = _matrix(x, "x", _BF)
    dev = x.device
    pw = _rows(wpacked, "wpacked", torch.uint8, (_packed_bytes(n, K, gc),), dev)
    pb = None if bias is None else _rows(bias, "bias", torch.float32, (n,), dev)
    if y is None:
        if out_dtype not in _CODE:
            raise SgError(f"out_dtype {out_dtype} not supported (float32 or bfloat16)")
        y = x.new_empty((M, n), dtype=out_dtype)
        ldy = n
    else:
        ldy = _result(y, "y", _FB, (M, n), dev)
    st = _lib().sg_w4a16_gemm_groupwise_packed(M, n, K, x.data_ptr(), ldx, pw, gc, pb, y.data_ptr(), _CODE[y.dtype],
                                               ldy, _current_stream(x))
    if st:
        _check(st, "sg_w4a16_gemm_groupwise_packed")
    return y


def w4a16_moe_mlp_workspace(t: int, k: int, e: int, d: int, f: int) -> int:
    """Bytes of workspace of a w4a16_moe_mlp call (-1: sizes out of range)."""
    return int(_lib().sg_w4a16_moe_mlp_workspace(t, k, e, d, f))


@functools.lru_cache(maxsize=1024)
def _moe_need(t, k, e, d, f):
    need = w4a16_moe_mlp_workspace(t, k, e, d, f)
    if need < 0:
        raise SgError(f"w4a16_moe_mlp: sizes out of range (T = {t}, k = {k}, E = {e}, D = {d}, F = {f})")
    return need


def w4a16_moe_mlp(x, ids, weights, gate, up, down, f: int, gc: int = 128, out_dtype=torch.bfloat16, y=None,
                  workspace=None):
    """y[t] = sum_j weights[t, j] * Wd_e (silu(Wg_e x_t) * (Wu_e x_t)), e = ids[t, j].

    x bfloat16 [T, D]; ids int32 and weights float32 [T, k] as moe_route gives
    them (an id outside [0, E) contributes nothing); gate, up uint8 [E, bytes] from
    w4_pack of E weights [f, D], down of E weights [D, f].  fp32 sums; silu(..) * (..)
    is rounded to bf16 once, also for out_dtype float32.  workspace: uint8, at least
    w4a16_moe_mlp_workspace(T, k, E, D, f) bytes (allocated if not given; keep it
    to one stream)."""
    T, D, ldx = _matrix(x, "x", _BF)
    dev = x.device
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise SgError("ids must be int32 [T, k]")
    k = ids.shape[1]
    if k < 1 or f < 1:
        raise SgError(f"k and F must be at least 1, got {k} and {f}")
    pi = _rows(ids, "ids", torch.int32, (T, k), dev)
    pr = _rows(weights, "weights", torch.float32, (T, k), dev)
    if not isinstance(gate, torch.Tensor) or gate.dim() != 2 or gate.shape[0] < 1:
        raise SgError("gate must be packed weights [E, bytes]")
    E = gate.shape[0]
    gu = (E, _packed_bytes(f, D, gc))
    pg = _rows(gate, "gate", torch.uint8, gu, dev)
    pu = _rows(up, "up", torch.uint8, gu, dev)
    pd = _rows(down, "down", torch.uint8, (E, _packed_bytes(D, f, gc)), dev)
    need = _moe_need(T, k, E, D, f)
    if workspace is None:
        workspace = ids.new_empty(need, dtype=torch.uint8)
    elif not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 or not workspace.is_contiguous() \
            or workspace.numel() < need or workspace.device != dev:
        raise SgError(f"workspace must be a contiguous uint8 tensor of at least {need} bytes on {dev}")
    if y is None:
        if out_dtype not in _CODE:
            raise SgError(f"out_dtype {out_dtype} not supported (float32 or bfloat16)")
        y = x.new_empty((T, D), dtype=out_dtype)
        ldy = D
    else:
        ldy = _result(y, "y", _FB, (T, D), dev)
    st = _lib().sg_w4a16_moe_mlp(T, k, E, D, f, x.data_ptr(), ldx, pi, pr, pg, pu, pd, gc, y.data_ptr(),
                                 _CODE[y.dtype], ldy, workspace.data_ptr(), workspace.numel(), _current_stream(x))
    if st:
        _check(st, "sg_w4a16_moe_mlp")
    return y
