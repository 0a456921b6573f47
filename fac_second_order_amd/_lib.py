"""ctypes binding of libkfac (include/kfac.h): argument marshalling only.

Every function has the name of the C entry point it calls and takes torch tensors
that live on the current HIP device; it passes their data pointers, the sizes and
the current torch stream (or the one given) to the library, and raises KfacError
when the library returns a non-zero status. Nothing here computes any part of the
K-FAC step, and there is no fallback: without the built library, import fails.
"""
import array
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkfac.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run `python fac_second_order_amd/build.py` "
        "(hipcc, gfx950) first. There is no CPU fallback.")

_lib = ctypes.CDLL(LIB_PATH)

KFAC_F16 = 0
KFAC_F32 = 1
KFAC_F64 = 2
KFAC_BF16 = 3
_STATUS = {0: "KFAC_OK", -1: "KFAC_ERR_INVALID", -2: "KFAC_ERR_UNSUPPORTED",
           -3: "KFAC_ERR_WORKSPACE", -4: "KFAC_ERR_HIP"}


class KfacError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = _lib.kfac_last_error().decode(errors="replace")
        super().__init__(f"{where}: {_STATUS.get(status, status)}: {msg}")


class kfac_layer(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in
                ("n", "h", "w", "c_in", "h_out", "w_out", "c_out",
                 "kh", "kw", "sh", "sw", "ph", "pw", "bias")]


class kfac_bn(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("hw", ctypes.c_int32), ("c", ctypes.c_int32)]


_c = ctypes
_vp, _i32, _sz, _f32 = _c.c_void_p, _c.c_int32, _c.c_size_t, _c.c_float
_i64 = _c.c_int64
_P = _c.POINTER


def _sig(name, res, *args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


_sig("kfac_version", _i32)
_sig("kfac_status_string", _c.c_char_p, _i32)
_sig("kfac_last_error", _c.c_char_p)
_sig("kfac_factors_workspace", _i32, _P(kfac_layer), _i32, _i32, _P(_sz))
_sig("kfac_factors", _i32, _P(kfac_layer), _i32, _i32, _P(_vp), _P(_vp), _P(_vp), _P(_vp), _f32,
     _vp, _sz, _vp)
_sig("kfac_factors_full", _i32, _P(kfac_layer), _i32, _i32, _P(_vp), _P(_vp), _P(_vp), _P(_vp), _P(_vp),
     _P(_vp), _f32, _vp, _sz, _vp)
_sig("kfac_pack_sym_workspace", _i32, _i32, _P(_i32), _P(_sz))
_sig("kfac_pack_sym", _i32, _i32, _P(_i32), _P(_vp), _P(_vp), _i32, _vp, _sz, _vp)
_sig("kfac_invert_workspace", _i32, _i32, _P(_i32), _P(_sz))
_sig("kfac_invert_schedule", _i32, _P(_i32), _P(_i32))
_sig("kfac_invert", _i32, _i32, _P(_i32), _P(_vp), _P(_vp), _P(_f32), _vp, _P(_vp), _vp, _sz, _vp)
_sig("kfac_invert_refine_workspace", _i32, _i32, _P(_i32), _P(_sz))
_sig("kfac_invert_refine", _i32, _i32, _P(_i32), _P(_vp), _P(_f32), _P(_vp), _vp, _sz, _vp)
_sig("kfac_precondition_workspace", _i32, _i32, _P(_i32), _P(_i32), _P(_sz))
_sig("kfac_precondition", _i32, _i32, _P(_i32), _P(_i32), _P(_vp), _P(_vp), _P(_vp), _i32, _P(_vp),
     _vp, _sz, _vp)
_sig("kfac_precondition_update", _i32, _i32, _P(_i32), _P(_i32), _P(_vp), _P(_vp), _P(_vp), _i32,
     _P(_vp), _P(_vp), _f32, _vp, _sz, _vp)
_sig("kfac_precondition_ex", _i32, _i32, _P(_i32), _P(_i32), _P(_vp), _P(_vp), _P(_vp), _i32,
     _P(_vp), _P(_vp), _f32, _i32, _vp, _sz, _vp)
_sig("kfac_bn_diag_workspace", _i32, _P(kfac_bn), _i32, _P(_sz))
_sig("kfac_bn_diag", _i32, _P(kfac_bn), _i32, _i32, _P(_vp), _P(_vp), _P(_vp), _P(_vp), _f32, _f32,
     _vp, _sz, _vp)
_sig("kfac_bn_update", _i32, _P(kfac_bn), _i32, _i32, _P(_vp), _P(_vp), _P(_vp), _P(_vp), _P(_vp),
     _f32, _f32, _f32, _vp, _sz, _vp)
_sig("kfac_bn_diag_noalloc", _i32, _P(kfac_bn), _i32, _i32, _P(_vp), _P(_vp), _P(_vp), _P(_vp), _P(_vp),
     _f32, _f32, _f32, _vp)
_sig("kfac_grad_norm_workspace", _i32, _i32, _vp, _P(_sz))
_sig("kfac_grad_norm", _i32, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp)
_sig("kfac_grad_clip", _i32, _i32, _vp, _vp, _vp, _vp, _vp, _f32, _vp, _vp, _sz, _vp)
_sig("kfac_trust_update", _i32, _i32, _vp, _vp, _vp, _vp, _vp, _f32, _vp, _f32, _f32, _vp, _vp, _sz, _vp)
_sig("kfac_policy_loss_workspace", _i32, _i32, _i32, _i32, _P(_sz))
_sig("kfac_policy_loss", _i32, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _f32, _f32, _f32,
     _i32, _f32, _vp, _vp, _vp, _i64, _vp, _sz, _vp)
_sig("kfac_preference_loss_workspace", _i32, _i32, _i32, _i32, _P(_sz))
_sig("kfac_preference_loss", _i32, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _i32, _vp, _vp, _f32, _f32, _f32, _vp,
     _vp, _vp, _vp, _i64, _vp, _sz, _vp)
_sig("kfac_timing_kernels", _i32)
_sig("kfac_kernel_name", _c.c_char_p, _i32)
_sig("kfac_timing_enable", _i32, _i32)
_sig("kfac_timing_only", _i32, _i32)
_sig("kfac_timing_reset", _i32)
_sig("kfac_timing_read", _i32, _i32, _P(_c.c_double), _P(_c.c_int64))


def _check(status, where):
    if status != 0:
        raise KfacError(status, where)


def _ptrs(tensors):
    arr = (_vp * max(1, len(tensors)))()
    for i, t in enumerate(tensors):
        arr[i] = None if t is None else t.data_ptr()
    return arr


def _ints(vals):
    arr = (_i32 * max(1, len(vals)))()
    for i, v in enumerate(vals):
        arr[i] = int(v)
    return arr


# The current stream's handle without a Stream object around it, which takes 2.8 us to make (a
# third of a small call); torch versions without it make the object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is not None:
        return _vp(stream.cuda_stream)
    if _raw_stream is not None:
        return _vp(_raw_stream(torch.cuda.current_device()))
    return _vp(torch.cuda.current_stream().cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.float16:
        return KFAC_F16
    if t.dtype == torch.float32:
        return KFAC_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _layers(layers):
    arr = (kfac_layer * max(1, len(layers)))()
    for i, l in enumerate(layers):
        for f, _ in kfac_layer._fields_:
            setattr(arr[i], f, int(getattr(l, f) if not isinstance(l, dict) else l[f]))
    return arr


def _bns(layers):
    arr = (kfac_bn * max(1, len(layers)))()
    for i, l in enumerate(layers):
        for f, _ in kfac_bn._fields_:
            setattr(arr[i], f, int(getattr(l, f) if not isinstance(l, dict) else l[f]))
    return arr


def _ws(workspace, nbytes, device):
    """The caller's workspace, or a fresh torch allocation of nbytes (256-aligned)."""
    if nbytes == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    ptr = workspace.data_ptr()
    pad = (-ptr) % 256
    return _vp(ptr + pad), max(0, workspace.numel() * workspace.element_size() - pad)


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def kfac_version():
    return _lib.kfac_version()


def kfac_factors_workspace(layers, in_dtype=KFAC_F16):
    out = _sz()
    _check(_lib.kfac_factors_workspace(_layers(layers), len(layers), in_dtype, _c.byref(out)),
           "kfac_factors_workspace")
    return out.value


def _factor_call_args(layers, act, gout, workspace):
    first = next(t for t in list(act) + list(gout) if t is not None)
    dt = _dtype_code(first)
    for t in list(act) + list(gout):
        if t is not None and (t.dtype != first.dtype or not t.is_contiguous()):
            raise TypeError("factor inputs must share one dtype and be contiguous")
    need = kfac_factors_workspace(layers, dt)
    ws, wsb = _ws(workspace, need, first.device)
    return dt, ws, wsb


def kfac_factors(layers, act, gout, A_packed, G_packed, ema_decay=0.0, workspace=None, stream=None):
    """A_packed[l], G_packed[l] <- packed factors of layer l (see kfac.h)."""
    dt, ws, wsb = _factor_call_args(layers, act, gout, workspace)
    _check(_lib.kfac_factors(_layers(layers), len(layers), dt, _ptrs(act), _ptrs(gout),
                             _ptrs(A_packed), _ptrs(G_packed), float(ema_decay), ws, wsb,
                             _stream(stream)), "kfac_factors")


def kfac_factors_full(layers, act, gout, A_packed, G_packed, A_full, G_full, ema_decay=0.0, workspace=None,
                      stream=None):
    """kfac_factors that also writes the upper triangle of each factor into A_full[l] /
    G_full[l] (d x d fp32, row-major; None entries skip it; see kfac.h)."""
    dt, ws, wsb = _factor_call_args(layers, act, gout, workspace)
    orders = [(l.c_in * l.kh * l.kw + (1 if l.bias else 0), l.c_out) for l in layers]
    if len(A_full) != len(layers) or len(G_full) != len(layers):
        raise ValueError("A_full and G_full need one entry per layer")
    for (da, dg), fa, fg in zip(orders, A_full, G_full):
        for t, d in ((fa, da), (fg, dg)):
            if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or t.numel() != d * d):
                raise TypeError("full factor outputs must be contiguous float32 d x d")
    _check(_lib.kfac_factors_full(_layers(layers), len(layers), dt, _ptrs(act), _ptrs(gout),
                                  _ptrs(A_packed), _ptrs(G_packed), _ptrs(A_full), _ptrs(G_full),
                                  float(ema_decay), ws, wsb, _stream(stream)), "kfac_factors_full")


def kfac_pack_sym_workspace(n):
    out = _sz()
    _check(_lib.kfac_pack_sym_workspace(len(n), _ints(n), _c.byref(out)), "kfac_pack_sym_workspace")
    return out.value


def kfac_pack_sym(n, full, packed, direction, workspace=None, stream=None):
    """direction 0: packed <- upper(full); 1: full <- symmetric(packed); 2: upper(full)
    <- packed, strict lower triangle of full left as it was."""
    need = kfac_pack_sym_workspace(n)
    ws, wsb = _ws(workspace, need, full[0].device if full else None)
    _check(_lib.kfac_pack_sym(len(n), _ints(n), _ptrs(full), _ptrs(packed), int(direction), ws, wsb,
                              _stream(stream)), "kfac_pack_sym")


def kfac_invert_workspace(n):
    out = _sz()
    _check(_lib.kfac_invert_workspace(len(n), _ints(n), _c.byref(out)), "kfac_invert_workspace")
    return out.value


def kfac_invert_schedule():
    """(block size, block steps per update launch) of kfac_invert."""
    b, g = _i32(), _i32()
    _check(_lib.kfac_invert_schedule(_c.byref(b), _c.byref(g)), "kfac_invert_schedule")
    return b.value, g.value


def kfac_invert_refine_workspace(n):
    out = _sz()
    _check(_lib.kfac_invert_refine_workspace(len(n), _ints(n), _c.byref(out)), "kfac_invert_refine_workspace")
    return out.value


def kfac_invert_refine(n, mat, shift, inv, workspace=None, stream=None):
    """inv[m] <- X + X (I - (mat[m] + shift[m] I) X), X = inv[m] (see kfac.h)."""
    need = kfac_invert_refine_workspace(n)
    ws, wsb = _ws(workspace, need, inv[0].device)
    shifts = (_f32 * len(n))(*[float(v) for v in shift])
    _check(_lib.kfac_invert_refine(len(n), _ints(n), _ptrs(mat), shifts, _ptrs(inv), ws, wsb, _stream(stream)),
           "kfac_invert_refine")


def kfac_invert(n, mat, inv, shift, info, chol=None, workspace=None, stream=None):
    """inv[m] <- (sym(mat[m]) + shift[m] I)^-1; info (int32 device tensor) <- breakdown index."""
    need = kfac_invert_workspace(n)
    ws, wsb = _ws(workspace, need, mat[0].device if mat else None)
    sh = (_f32 * max(1, len(n)))(*[float(s) for s in shift])
    if info.dtype != torch.int32 or info.numel() < len(n):
        raise TypeError("info must be an int32 tensor with one entry per matrix")
    _check(_lib.kfac_invert(len(n), _ints(n), _ptrs(mat), _ptrs(inv), sh, _vp(info.data_ptr()),
                            _ptrs(chol) if chol is not None else None, ws, wsb, _stream(stream)),
           "kfac_invert")


def kfac_precondition_workspace(d_g, d_a):
    out = _sz()
    _check(_lib.kfac_precondition_workspace(len(d_g), _ints(d_g), _ints(d_a), _c.byref(out)),
           "kfac_precondition_workspace")
    return out.value


def kfac_precondition(d_g, d_a, G_inv, A_inv, grad, out, workspace=None, stream=None):
    """out[l] <- G_inv[l] @ grad[l] @ A_inv[l] (fp32)."""
    dt = _dtype_code(grad[0])
    need = kfac_precondition_workspace(d_g, d_a)
    ws, wsb = _ws(workspace, need, grad[0].device)
    _check(_lib.kfac_precondition(len(d_g), _ints(d_g), _ints(d_a), _ptrs(G_inv), _ptrs(A_inv),
                                  _ptrs(grad), dt, _ptrs(out), ws, wsb, _stream(stream)),
           "kfac_precondition")


def kfac_precondition_update(d_g, d_a, G_inv, A_inv, grad, out, w, lr, workspace=None, stream=None):
    """w[l] <- w[l] - lr * G_inv[l] @ grad[l] @ A_inv[l]; out[l] <- the product unless out is None."""
    dt = _dtype_code(grad[0])
    need = kfac_precondition_workspace(d_g, d_a)
    ws, wsb = _ws(workspace, need, grad[0].device)
    _check(_lib.kfac_precondition_update(len(d_g), _ints(d_g), _ints(d_a), _ptrs(G_inv), _ptrs(A_inv),
                                         _ptrs(grad), dt, None if out is None else _ptrs(out), _ptrs(w),
                                         float(lr), ws, wsb, _stream(stream)),
           "kfac_precondition_update")


def kfac_precondition_ex(d_g, d_a, G_inv, A_inv, grad, out, w=None, lr=0.0, accum=KFAC_F32, workspace=None,
                         stream=None):
    """kfac_precondition (w None) or kfac_precondition_update (w given), the products
    summed in fp32 (accum KFAC_F32) or fp64 (KFAC_F64)."""
    dt = _dtype_code(grad[0])
    need = kfac_precondition_workspace(d_g, d_a)
    ws, wsb = _ws(workspace, need, grad[0].device)
    _check(_lib.kfac_precondition_ex(len(d_g), _ints(d_g), _ints(d_a), _ptrs(G_inv), _ptrs(A_inv), _ptrs(grad), dt,
                                     None if out is None else _ptrs(out), None if w is None else _ptrs(w),
                                     float(lr), int(accum), ws, wsb, _stream(stream)), "kfac_precondition_ex")


def kfac_bn_diag_workspace(layers):
    out = _sz()
    _check(_lib.kfac_bn_diag_workspace(_bns(layers), len(layers), _c.byref(out)), "kfac_bn_diag_workspace")
    return out.value


def kfac_bn_diag(layers, xhat, gout, fisher, precond, ema_decay=0.0, shift=1e-3, workspace=None,
                 stream=None):
    """fisher[l], precond[l] ([2, c] fp32) <- BN diagonal Fisher and grad/(F+shift)."""
    dt = _dtype_code(xhat[0])
    need = kfac_bn_diag_workspace(layers)
    ws, wsb = _ws(workspace, need, xhat[0].device)
    _check(_lib.kfac_bn_diag(_bns(layers), len(layers), dt, _ptrs(xhat), _ptrs(gout), _ptrs(fisher),
                             _ptrs(precond), float(ema_decay), float(shift), ws, wsb, _stream(stream)),
           "kfac_bn_diag")


def kfac_bn_update(layers, xhat, gout, fisher, precond, params, lr, ema_decay=0.0, shift=1e-3,
                   workspace=None, stream=None):
    """kfac_bn_diag, then params[l] ([2, c] fp32: gamma, beta) <- params[l] - lr * precond[l]."""
    dt = _dtype_code(xhat[0])
    need = kfac_bn_diag_workspace(layers)
    ws, wsb = _ws(workspace, need, xhat[0].device)
    _check(_lib.kfac_bn_update(_bns(layers), len(layers), dt, _ptrs(xhat), _ptrs(gout), _ptrs(fisher),
                               _ptrs(precond), _ptrs(params), float(lr), float(ema_decay), float(shift),
                               ws, wsb, _stream(stream)), "kfac_bn_update")


KFAC_BN_NOALLOC_SCRATCH_BYTES = 16 << 20


def kfac_bn_diag_noalloc(layers, xhat, gout, fisher, precond, params=None, lr=0.0, ema_decay=0.0, shift=1e-3,
                         stream=None):
    """kfac_bn_diag (params None) or kfac_bn_update (params given) with the library's
    static scratch instead of a workspace: allocates nothing (see kfac.h)."""
    dt = _dtype_code(xhat[0])
    _check(_lib.kfac_bn_diag_noalloc(_bns(layers), len(layers), dt, _ptrs(xhat), _ptrs(gout), _ptrs(fisher),
                                     _ptrs(precond), None if params is None else _ptrs(params), float(lr),
                                     float(ema_decay), float(shift), _stream(stream)), "kfac_bn_diag_noalloc")


# gradient norm, clipping and the bounded update ------------------------------

_ANY_CODE = {torch.float16: KFAC_F16, torch.float32: KFAC_F32, torch.bfloat16: KFAC_BF16}
_device_of = torch.Tensor.get_device


def _on_device(tensors, what):
    """Refuses tensors that are not on the current device: the library launches there."""
    at = set(map(_device_of, tensors))
    if at and (len(at) > 1 or min(at) < 0 or min(at) != torch.cuda.current_device()):
        raise ValueError(f"{what} must be on the current HIP device")


def _listed(tensors, what):
    """(numel, dtype code, addresses) of contiguous tensors on the current device."""
    tensors = list(tensors)  # looked through several times: a generator would be empty after the first
    _on_device(tensors, what)
    if not all(map(torch.Tensor.is_contiguous, tensors)):
        raise TypeError(f"{what} must be contiguous")
    try:
        codes = [_ANY_CODE[t.dtype] for t in tensors]
    except KeyError as e:
        raise TypeError(f"{what}: unsupported dtype {e.args[0]}") from None
    return list(map(torch.Tensor.numel, tensors)), codes, list(map(torch.Tensor.data_ptr, tensors))


# Lists of integers as C arrays; array.array is several times faster to fill than a ctypes one.
def _words(values):
    return array.array("q", values or (0,))


def _halfwords(values):
    return array.array("i", values or (0,))


def _at(arr):
    return arr.buffer_info()[0]


def _scalar_out(t, n, what):
    if t.dtype != torch.float32 or t.numel() < n or not t.is_contiguous():
        raise TypeError(f"{what} must be a contiguous float32 tensor of {n} or more")
    return t.data_ptr()


def _call_ws(workspace, query, sizes, device, stream):
    """Aligned address and bytes of the call's workspace, and the tensor behind it, to be held
    until the call has been made. Without one from the caller, query(*sizes) bytes are
    allocated on the stream that the call runs on: their memory is free there, and goes to
    nothing else before the call's kernels are done. A stream of another device would run
    the call there."""
    if stream is not None and stream.device != device:
        raise ValueError("stream must be of the current HIP device")
    if workspace is None:
        with torch.cuda.stream(stream):
            workspace = torch.empty(query(*sizes) + 256, dtype=torch.uint8, device=device)
    elif workspace.device != device:
        raise ValueError("workspace must be on the current HIP device")
    elif not workspace.is_contiguous():  # numel would count bytes that are not there
        raise TypeError("workspace must be contiguous")
    at = workspace.data_ptr()
    pad = -at % 256
    return at + pad, max(0, workspace.numel() * workspace.element_size() - pad), workspace


def kfac_grad_norm_workspace(numel):
    out = _sz()
    n = _words(numel)
    _check(_lib.kfac_grad_norm_workspace(len(numel), _at(n), _c.byref(out)), "kfac_grad_norm_workspace")
    return out.value


def kfac_grad_norm(grad, norm, workspace=None, stream=None):
    """norm[0] <- sqrt of the sum of squares over all tensors of grad (float16, bfloat16
    or float32, each its own; see kfac.h)."""
    numel, codes, at = _listed(grad, "grad")
    _on_device([norm], "norm")
    out = _scalar_out(norm, 1, "norm")
    ws, wsb, held = _call_ws(workspace, kfac_grad_norm_workspace, (numel,), norm.device, stream)
    n, c, g = _words(numel), _halfwords(codes), _words(at)
    _check(_lib.kfac_grad_norm(len(numel), _at(n), _at(c), _at(g), out, ws, wsb, _stream(stream)), "kfac_grad_norm")


def kfac_grad_clip(grad, out, max_norm, norm, workspace=None, stream=None):
    """out[i] <- grad[i] * min(1, max_norm / norm), norm[0] <- the global norm; out[i] is
    grad[i] or a tensor of its size, of its type or float32 (see kfac.h)."""
    numel, codes, at = _listed(grad, "grad")
    out_numel, out_codes, out_at = _listed(out, "out")
    if out_numel != numel:
        raise ValueError("out must have one tensor of the gradient's size for each gradient")
    _on_device([norm], "norm")
    norm_at = _scalar_out(norm, 1, "norm")
    ws, wsb, held = _call_ws(workspace, kfac_grad_norm_workspace, (numel,), norm.device, stream)
    n, c, g, oc, o = _words(numel), _halfwords(codes), _words(at), _halfwords(out_codes), _words(out_at)
    _check(_lib.kfac_grad_clip(len(numel), _at(n), _at(c), _at(g), _at(oc), _at(o), float(max_norm), norm_at, ws, wsb,
                               _stream(stream)), "kfac_grad_clip")


def kfac_trust_update(precond, grad, w, lr, delta, step, fisher=None, shift=0.0, workspace=None, stream=None):
    """w[i] <- w[i] - s * precond[i], s = min(lr, sqrt(2 delta / |q|)), q = sum of
    <precond[i], grad[i]>; step[:2] <- s, q. Where grad[i] is None, fisher[i] (diagonal)
    and shift give the gradient (see kfac.h)."""
    n = len(precond)
    if len(grad) != n or len(w) != n or (fisher is not None and len(fisher) != n):
        raise ValueError("precond, grad, fisher and w must have one tensor of one size for each entry")
    given = list(grad)  # an entry's gradient, or else its Fisher
    diagonal = [i for i, g in enumerate(given) if g is None]
    for i in diagonal:
        if fisher is None or fisher[i] is None:
            raise ValueError("an entry without a gradient needs its fisher")
        given[i] = fisher[i]
    numel, codes, at = _listed([*precond, *w, *given], "precond, grad, fisher and w")
    if codes[:2 * n] != [KFAC_F32] * (2 * n):
        raise TypeError("precond and w must be float32")
    if numel[n:2 * n] != numel[:n] or numel[2 * n:] != numel[:n]:
        raise ValueError("precond, grad, fisher and w must have one tensor of one size for each entry")
    numel, s_codes, p_at, w_at, g_at, f_at = numel[:n], codes[2 * n:], at[:n], at[n:2 * n], at[2 * n:], [0] * n
    for i in diagonal:
        if s_codes[i] != KFAC_F32:
            raise TypeError("fisher must be float32")
        f_at[i], g_at[i] = g_at[i], 0
    _on_device([step], "step")
    step_at = _scalar_out(step, 2, "step")
    ws, wsb, held = _call_ws(workspace, kfac_grad_norm_workspace, (numel,), step.device, stream)
    counts, c, p, ww = _words(numel), _halfwords(s_codes), _words(p_at), _words(w_at)
    g, f = _words(g_at), _words(f_at)
    _check(_lib.kfac_trust_update(n, _at(counts), _at(p), _at(c), _at(g), _at(f), float(shift), _at(ww), float(lr),
                                  float(delta), step_at, ws, wsb, _stream(stream)), "kfac_trust_update")


# losses over logits -----------------------------------------------------------

def kfac_policy_loss_workspace(rows, vocab, seqs=0):
    out = _sz()
    _check(_lib.kfac_policy_loss_workspace(int(rows), int(vocab), int(seqs), _c.byref(out)),
           "kfac_policy_loss_workspace")
    return out.value


def kfac_preference_loss_workspace(rows, vocab, pairs):
    out = _sz()
    _check(_lib.kfac_preference_loss_workspace(int(rows), int(vocab), int(pairs), _c.byref(out)),
           "kfac_preference_loss_workspace")
    return out.value


def _vector(t, dtype, n, what):
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise TypeError(f"{what} must be a contiguous {dtype} tensor of {n}")
    return t.data_ptr()


def _pitch(t, rows, vocab, what):
    apart, within = t.stride()
    if (vocab > 1 and within != 1) or (rows > 1 and apart < vocab):
        raise TypeError(f"the rows of {what} must be contiguous and apart")
    return apart if rows > 1 else vocab


def _logit_rows(logits, dlogits, token, mask, others):
    """Checks the rows of a loss; (rows, vocab, dtype code, logits pointer and pitch,
    token, mask, dlogits pointer and pitch). Small calls wait for the host, so each tensor
    is asked once for what is needed of it."""
    dtype = logits.dtype
    if logits.dim() != 2 or dtype not in _ANY_CODE:
        raise TypeError("logits must be [rows, vocab] in float16, bfloat16 or float32")
    rows, vocab = shape = logits.shape
    _on_device([t for t in (logits, token, mask, dlogits, *others) if t is not None], "every tensor of the call")
    d = msk = None
    ldd = 0
    ld = _pitch(logits, rows, vocab, "logits")
    if dlogits is not None:
        if dlogits.shape != shape or dlogits.dtype != dtype:
            raise TypeError("dlogits must have the shape and type of logits")
        d, ldd = dlogits.data_ptr(), _pitch(dlogits, rows, vocab, "dlogits")
    if mask is not None:
        if mask.dtype not in (torch.bool, torch.uint8):
            raise TypeError("mask must be bool or uint8")
        msk = _vector(mask, mask.dtype, rows, "mask")
    return (rows, vocab, _ANY_CODE[dtype], logits.data_ptr(), ld, _vector(token, torch.int64, rows, "token"), msk, d,
            ldd)


def kfac_policy_loss(logits, token, old_logp, advantage, logp, stats, dlogits=None, ref_logp=None, mask=None,
                     seq_begin=None, by_sequence=False, clip_low=0.2, clip_high=0.2, kl_coef=0.0, grad_scale=1.0,
                     workspace=None, stream=None):
    """Clipped policy loss with a KL term over logits [rows, vocab]: stats[:4] <- loss,
    its surrogate part, mean KL, clipped share; logp <- the tokens' log-probabilities;
    dlogits <- grad_scale * gradient of the loss (see kfac.h)."""
    rows, vocab, code, z, ld, tok, msk, d, ldd = _logit_rows(
        logits, dlogits, token, mask, (old_logp, advantage, logp, stats, ref_logp, seq_begin))
    seqs = 0 if seq_begin is None else seq_begin.numel() - 1
    if seq_begin is not None and seqs < 1:
        raise ValueError("seq_begin needs one offset more than there are sequences")
    f32 = torch.float32
    stats_at = _scalar_out(stats, 4, "stats")
    ws, wsb, held = _call_ws(workspace, kfac_policy_loss_workspace, (rows, vocab, seqs), logits.device, stream)
    _check(_lib.kfac_policy_loss(
        rows, vocab, code, z, ld, tok, msk, seqs,
        None if seq_begin is None else _vector(seq_begin, torch.int32, seqs + 1, "seq_begin"),
        _vector(old_logp, f32, rows, "old_logp"),
        None if ref_logp is None else _vector(ref_logp, f32, rows, "ref_logp"),
        _vector(advantage, f32, rows, "advantage"), float(clip_low), float(clip_high), float(kl_coef),
        1 if by_sequence else 0, float(grad_scale), _vector(logp, f32, rows, "logp"), stats_at, d, ldd, ws,
        wsb, _stream(stream)), "kfac_policy_loss")


def kfac_preference_loss(logits, token, seq_begin, seq_logp, margin, loss, dlogits=None, ref_logp=None, mask=None,
                         beta=0.1, label_smoothing=0.0, grad_scale=1.0, workspace=None, stream=None):
    """Preference loss over pairs of sequences (i preferred to pairs + i) of logits
    [rows, vocab]: loss[0], margin [pairs], seq_logp [2 * pairs], dlogits <- grad_scale *
    gradient of the loss (see kfac.h)."""
    rows, vocab, code, z, ld, tok, msk, d, ldd = _logit_rows(
        logits, dlogits, token, mask, (seq_begin, seq_logp, margin, loss, ref_logp))
    if seq_begin.numel() % 2 != 1:
        raise ValueError("seq_begin needs one offset more than two for each pair")
    pairs = seq_begin.numel() // 2
    f32 = torch.float32
    loss_at = _scalar_out(loss, 1, "loss")
    ws, wsb, held = _call_ws(workspace, kfac_preference_loss_workspace, (rows, vocab, pairs), logits.device, stream)
    _check(_lib.kfac_preference_loss(
        rows, vocab, code, z, ld, tok, msk, pairs, _vector(seq_begin, torch.int32, 2 * pairs + 1, "seq_begin"),
        None if ref_logp is None else _vector(ref_logp, f32, 2 * pairs, "ref_logp"), float(beta),
        float(label_smoothing), float(grad_scale), _vector(seq_logp, f32, 2 * pairs, "seq_logp"),
        _vector(margin, f32, pairs, "margin"), loss_at, d, ldd, ws, wsb, _stream(stream)),
        "kfac_preference_loss")


# timing -------------------------------------------------------------------

def kfac_timing_kernels():
    return _lib.kfac_timing_kernels()


def kfac_kernel_name(i):
    return _lib.kfac_kernel_name(int(i)).decode()


def kfac_timing_enable(on=True):
    _check(_lib.kfac_timing_enable(1 if on else 0), "kfac_timing_enable")


def kfac_timing_only(i=-1):
    """Time only kernel id i (-1: every kernel)."""
    _check(_lib.kfac_timing_only(int(i)), "kfac_timing_only")


def kfac_timing_reset():
    _check(_lib.kfac_timing_reset(), "kfac_timing_reset")


def kfac_timing_read(i):
    ms = _c.c_double()
    n = _c.c_int64()
    _check(_lib.kfac_timing_read(int(i), _c.byref(ms), _c.byref(n)), "kfac_timing_read")
    return ms.value, n.value
