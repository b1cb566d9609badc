"""ctypes binding of the gated projections' entry points of libsg.so
(``sparse_gemm_layers_amd/include/sg_gated.h``).  Argument marshalling only."""

import ctypes
import functools

import torch

from ._binding import SgError, _FB, _check, _i64, _int, _ptr, lib
from ._moe import _BF, _CODE, _matrix, _refuse, _result

_SIGS = {
    "sg_gated_gemm": ([_i64, _i64, _i64, _ptr, _i64, _ptr, _i64, _ptr, _i64, _int, _ptr, _ptr, _i64, _ptr, _int, _i64,
                       _ptr, _ptr, _i64, _ptr], _int),
    "sg_gated_gemm_backward_workspace": ([_i64, _i64, _i64], _i64),
    "sg_gated_gemm_backward": ([_i64, _i64, _i64, _ptr, _i64, _ptr, _i64, _ptr, _i64, _ptr, _i64, _int, _ptr, _ptr,
                                _i64, _ptr, _ptr, _i64, _ptr, _ptr, _i64, _ptr, _i64, _ptr, _ptr, _i64, _ptr, _i64,
                                _ptr], _int),
    "sg_gated_gemm_plan": ([_i64, _i64, _i64, _ptr, _ptr], _int),
    "sg_gated_gemm_backward_plan": ([_i64, _i64, _i64, _int, _ptr, _ptr], _int),
}

_ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
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


def _launch(dev, fn, *args):
    """fn(*args, stream) with GPU dev current, on its current stream."""
    if dev == torch._C._cuda_getDevice():
        return fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    with torch.cuda.device(dev):
        return fn(*args, torch._C._cuda_getCurrentRawStream(dev))


# Operands that are as they should be and contiguous, as most are, pass by one expression;
# dev is the index of the GPU that all have to be on.

def _ld(t, name, dtypes, shape, dev):
    """Row stride of a matrix."""
    if isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype in dtypes and t.shape == shape \
            and t.is_contiguous():
        return shape[1]
    return _result(t, name, dtypes, shape, torch.device("cuda", dev))


def _at(t, name, dtype, shape, dev):
    """Address of a contiguous tensor."""
    if isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype is dtype and t.shape == shape \
            and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, (dtype,), shape, torch.device("cuda", dev))


def _space(workspace, need, x, dev):
    """The workspace: as given, or of the bytes that are needed."""
    if workspace is None:
        return x.new_empty(need, dtype=torch.uint8)
    if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 or not workspace.is_contiguous() \
            or workspace.numel() < need or workspace.get_device() != dev:
        raise SgError(f"workspace must be a contiguous uint8 tensor of at least {need} bytes on {x.device}")
    return workspace


def _act_code(act):
    if act not in _ACTS:
        raise SgError(f"act must be one of {', '.join(map(repr, _ACTS))}, got {act!r}")
    return _ACTS[act]


def _weights(x, gate, up):
    """(T, D, F, row strides of x, gate and up, index of their GPU)."""
    T, D, ldx = _matrix(x, "x", _BF)
    dev = x.get_device()
    F = gate.shape[0] if isinstance(gate, torch.Tensor) and gate.dim() == 2 else 0
    if F < 1:
        _matrix(gate, "gate", _BF)
    return T, D, F, ldx, _ld(gate, "gate", _BF, (F, D), dev), _ld(up, "up", _BF, (F, D), dev), dev


def _pair(s, t, names, shape, dev):
    """(addresses, row stride) of two bf16 matrices of one shape that share a row
    stride, or of neither."""
    if s is None and t is None:
        return None, None, 0
    if s is None or t is None:
        raise SgError(f"{names[0]} and {names[1]} go together")
    ld = _ld(s, names[0], _BF, shape, dev)
    if _ld(t, names[1], _BF, shape, dev) != ld:
        raise SgError(f"{names[0]} and {names[1]} must have the same row stride")
    return s.data_ptr(), t.data_ptr(), ld


def _addends(gate_add, up_add, shape, dev):
    if gate_add is not None and up_add is not None:
        return _pair(gate_add, up_add, ("gate_add", "up_add"), shape, dev)
    pg = pu = None
    ld = 0
    if gate_add is not None:
        ld, pg = _ld(gate_add, "gate_add", _BF, shape, dev), gate_add.data_ptr()
    if up_add is not None:
        ld, pu = _ld(up_add, "up_add", _BF, shape, dev), up_add.data_ptr()
    return pg, pu, ld


def gated_gemm(x, gate, up, act: str = "silu", gate_add=None, up_add=None, out_dtype=torch.bfloat16, keep: bool = False,
               h=None, g=None, u=None):
    """h [T, F] = act(G) * U with G = x . gate^T + gate_add, U = x . up^T + up_add.

    x bfloat16 [T, D], gate and up bfloat16 [F, D], the addends (what stands beside a
    projection, an adapter's product for one) bfloat16 [T, F] or None; act "silu",
    "gelu", "gelu_tanh" or "relu".  fp32 sums, rounded once.  With `keep`: (h, G, U),
    the last two rounded to bfloat16, for gated_gemm_backward.  h, g, u: results to
    write to."""
    T, D, F, ldx, ldg, ldu, dev = _weights(x, gate, up)
    code = _act_code(act)
    pga, pua, ld_add = _addends(gate_add, up_add, (T, F), dev)
    if h is None:
        if out_dtype not in _CODE:
            raise SgError(f"out_dtype {out_dtype} not supported (float32 or bfloat16)")
        h = x.new_empty((T, F), dtype=out_dtype)
        ldh = F
    else:
        ldh = _ld(h, "h", _FB, (T, F), dev)
    if keep and g is None and u is None:
        g, u = x.new_empty((T, F)), x.new_empty((T, F))
        pg, pu, ld_gu = g.data_ptr(), u.data_ptr(), F
    else:
        pg, pu, ld_gu = _pair(g, u, ("g", "u"), (T, F), dev)
    st = _launch(dev, _lib().sg_gated_gemm, T, F, D, x.data_ptr(), ldx, gate.data_ptr(), ldg, up.data_ptr(), ldu, code, pga,
                 pua, ld_add, h.data_ptr(), _CODE[h.dtype], ldh, pg, pu, ld_gu)
    if st:
        _check(st, "sg_gated_gemm")
    return (h, g, u) if pg is not None else h


def gated_gemm_backward_workspace(t: int, f: int, d: int) -> int:
    """Bytes of workspace of a gated_gemm_backward call that computes dx (-1: sizes out of range)."""
    return int(_lib().sg_gated_gemm_backward_workspace(t, f, d))


@functools.lru_cache(maxsize=1024)
def _back_need(t, f, d):
    need = gated_gemm_backward_workspace(t, f, d)
    if need < 0:
        raise SgError(f"gated_gemm_backward: sizes out of range (T = {t}, F = {f}, D = {d}; F and D multiples of 8)")
    return need


def gated_gemm_backward(dh, x, gate, up, act: str = "silu", g=None, u=None, gate_add=None, up_add=None,
                        need_dx: bool = True, need_dw: bool = True, dx=None, dgate=None, dup=None, dg=None, du=None,
                        workspace=None):
    """Gradients of gated_gemm for dh bfloat16 [T, F], the gradient of h:
    (dx [T, D], dgate [F, D], dup [F, D], dg [T, F], du [T, F]), all bfloat16; dx and
    the weights' are None where not needed.

    g and u are what the forward call kept; without them G and U are computed again
    from x, the weights and the addends.  dg and du are the gradients of G and U, and
    so of gate_add and up_add; rounded to bfloat16 they are the operands of the other
    three.  workspace: uint8, at least gated_gemm_backward_workspace(T, F, D) bytes
    (allocated if not given; keep it to one stream)."""
    T, D, F, ldx, ldg, ldu, dev = _weights(x, gate, up)
    code = _act_code(act)
    ld_dh = _ld(dh, "dh", _BF, (T, F), dev)
    pg, pu, ld_gu = _pair(g, u, ("g", "u"), (T, F), dev)
    pga, pua, ld_add = _addends(gate_add, up_add, (T, F), dev)
    need = _back_need(T, F, D)
    if dg is None and du is None:
        dg, du = x.new_empty((T, F)), x.new_empty((T, F))
        pdg, pdu, ld_dgu = dg.data_ptr(), du.data_ptr(), F
    else:
        pdg, pdu, ld_dgu = _pair(dg, du, ("dg", "du"), (T, F), dev)
    pdx, ld_dx = None, D
    if dx is not None:
        ld_dx, pdx = _ld(dx, "dx", _BF, (T, D), dev), dx.data_ptr()
    elif need_dx:
        dx = x.new_empty((T, D))
        pdx = dx.data_ptr()
    if need_dw and dgate is None and dup is None:
        dgate, dup = x.new_empty((F, D)), x.new_empty((F, D))
        pwg, pwu, ld_dw = dgate.data_ptr(), dup.data_ptr(), D
    else:
        pwg, pwu, ld_dw = _pair(dgate, dup, ("dgate", "dup"), (F, D), dev)
    pw, wn = None, 0
    if dx is not None and need:
        workspace = _space(workspace, need, x, dev)
        pw, wn = workspace.data_ptr(), workspace.numel()
    st = _launch(dev, _lib().sg_gated_gemm_backward, T, F, D, dh.data_ptr(), ld_dh, x.data_ptr(), ldx, gate.data_ptr(), ldg,
                 up.data_ptr(), ldu, code, pg, pu, ld_gu, pga, pua, ld_add, pdg, pdu, ld_dgu, pdx, ld_dx, pwg, pwu,
                 ld_dw, pw, wn)
    if st:
        _check(st, "sg_gated_gemm_backward")
    return dx, dgate, dup, dg, du


def gated_gemm_plan(t: int, f: int, d: int):
    """(tokens, hidden values) of one workgroup of gated_gemm, and of a gated_gemm_backward call
    that computes G and U again."""
    a, b = ctypes.c_int32(), ctypes.c_int32()
    _check(_lib().sg_gated_gemm_plan(t, f, d, ctypes.addressof(a), ctypes.addressof(b)), "sg_gated_gemm_plan")
    return a.value, b.value


def gated_gemm_backward_plan(t: int, f: int, d: int, need_dw: bool = True):
    """(rows and columns of a gradient that one workgroup computes, parts of dx's sum) of
    gated_gemm_backward; more than one part take 4 parts T D bytes of workspace."""
    a, b = ctypes.c_int32(), ctypes.c_int32()
    _check(_lib().sg_gated_gemm_backward_plan(t, f, d, int(need_dw), ctypes.addressof(a), ctypes.addressof(b)),
           "sg_gated_gemm_backward_plan")
    return a.value, b.value
