"""ctypes binding of libgdn (``include/gdn.h``): argument marshalling only.

Each function has the name of its C entry point and takes torch CUDA tensors
(device memory from PyTorch); all computation happens in libgdn's kernels.
There is no fallback: if ``libgdn.so`` is missing, loading it raises.
"""
import ctypes
import math
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# GDN_CHECKS=1: the bounds-checked build (python -m gated_deltanet_mixer_gb300.build --checks)
LIB_PATH = os.path.join(_HERE, "libgdn_checks.so" if os.environ.get("GDN_CHECKS", "0") not in ("", "0")
                        else "libgdn.so")

GDN_OK = 0
GDN_ERR_INVALID_ARG = 1
GDN_ERR_TIMEOUT = 6
STATUS_NAMES = {0: "GDN_OK", 1: "GDN_ERR_INVALID_ARG", 2: "GDN_ERR_UNSUPPORTED_SHAPE",
                3: "GDN_ERR_ALIGNMENT", 4: "GDN_ERR_ALIAS", 5: "GDN_ERR_CUDA",
                6: "GDN_ERR_TIMEOUT", 7: "GDN_ERR_NO_DEVICE", 8: "GDN_ERR_BOUNDS"}
GDN_F32, GDN_BF16 = 0, 1
GDN_STATIC_SCRATCH_BYTES = 512 << 20  # include/gdn.h: the scratch of gdn_prefill_static


class GdnError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s (%s)" % (where, STATUS_NAMES.get(status, status),
                                          gdn_status_str(status)))


class gdn_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("Hk", ctypes.c_int),
                ("Hv", ctypes.c_int), ("Dk", ctypes.c_int), ("Dv", ctypes.c_int),
                ("io_dtype", ctypes.c_int), ("eps_l2", ctypes.c_float),
                ("eps_norm", ctypes.c_float), ("q_scale", ctypes.c_float)]


vp = ctypes.c_void_p


class gdn_raw_gates(ctypes.Structure):
    _fields_ = [("a", vp), ("b", vp), ("A_log", vp), ("dt_bias", vp)]


class gdn_prefill_io(ctypes.Structure):
    _fields_ = [(n, vp) for n in ("qkv_pre", "z", "g", "beta", "raw_gates", "conv_w", "norm_w", "S0",
                                  "conv0", "o", "S_T", "conv_T", "cu_seqlens", "S_snap", "workspace")] + \
               [("workspace_bytes", ctypes.c_size_t)]


class gdn_linear_out(ctypes.Structure):
    _fields_ = [("col_begin", ctypes.c_int), ("col_end", ctypes.c_int), ("ptr", vp), ("ld", ctypes.c_longlong)]


class gdn_decode_io(ctypes.Structure):
    _fields_ = [(n, vp) for n in ("qkv_pre", "z", "g", "beta", "raw_gates", "conv_w", "norm_w", "S",
                                  "S_snap", "conv_in", "conv_out", "o")]


class gdn_linear_ex_out(ctypes.Structure):
    _fields_ = [("col_begin", ctypes.c_int), ("col_end", ctypes.c_int), ("ptr", vp), ("ld", ctypes.c_longlong),
                ("act", ctypes.c_int), ("residual", vp), ("ldr", ctypes.c_longlong)]


class gdn_linear_ex_form(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("tile", ctypes.c_int), ("tiles", ctypes.c_longlong), ("rows_w", ctypes.c_int),
                ("split", ctypes.c_int)]


class gdn_linattn_form(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("chunked", "segments", "parts")]


class gdn_linattn_io(ctypes.Structure):
    _fields_ = [(n, vp) for n in ("q", "k", "v")] + \
               [(n, ctypes.c_longlong) for n in ("ldq", "ldk", "ldv", "ldo")] + \
               [(n, vp) for n in ("g", "log_decay", "S0", "o", "S_T", "cu_seqlens", "workspace")] + \
               [("workspace_bytes", ctypes.c_size_t)]


ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "sigmoid": 3}

_lib = None


def lib():
    """The loaded libgdn (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libgdn.so is not built (%s); run "
                               "`python -m gated_deltanet_mixer_gb300.build`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp = ctypes.c_void_p
        L.gdn_abi_version.restype = ctypes.c_int
        L.gdn_abi_version.argtypes = []
        L.gdn_status_str.restype = ctypes.c_char_p
        L.gdn_status_str.argtypes = [ctypes.c_int]
        L.gdn_prefill.restype = ctypes.c_int
        L.gdn_prefill.argtypes = [ctypes.POINTER(gdn_shape)] + [vp] * 12
        L.gdn_decode_step.restype = ctypes.c_int
        L.gdn_decode_step.argtypes = [ctypes.POINTER(gdn_shape)] + [vp] * 11
        L.gdn_device_status.restype = ctypes.c_int
        L.gdn_device_status.argtypes = [vp, ctypes.c_int]
        L.gdn_prefill_ex.restype = ctypes.c_int
        L.gdn_prefill_ex.argtypes = [ctypes.POINTER(gdn_shape), ctypes.POINTER(gdn_prefill_io), vp]
        L.gdn_decode_ex.restype = ctypes.c_int
        L.gdn_decode_ex.argtypes = [ctypes.POINTER(gdn_shape), ctypes.POINTER(gdn_decode_io), vp]
        L.gdn_linear.restype = ctypes.c_int
        L.gdn_linear.argtypes = [ctypes.c_int] * 3 + [vp, ctypes.c_longlong, vp, ctypes.c_longlong, ctypes.c_int,
                                                      ctypes.POINTER(gdn_linear_out), vp]
        L.gdn_linear_ex.restype = ctypes.c_int
        L.gdn_linear_ex.argtypes = [ctypes.c_int] * 4 + [vp, ctypes.c_longlong, vp, ctypes.c_longlong, vp, ctypes.c_int, vp, vp]
        L.gdn_selftest_linear_ex_form.restype = ctypes.c_int
        L.gdn_selftest_linear_ex_form.argtypes = [ctypes.c_int] * 5 + [ctypes.POINTER(gdn_linear_ex_form)]
        for name in ("gdn_linattn_prefill", "gdn_linattn_decode"):
            getattr(L, name).restype = ctypes.c_int
            getattr(L, name).argtypes = [vp, vp, vp]  # structures by reference, or packed bytes
        L.gdn_selftest_linattn_form.restype = ctypes.c_int
        L.gdn_selftest_linattn_form.argtypes = [ctypes.POINTER(gdn_shape), ctypes.c_int, ctypes.c_int,
                                                ctypes.POINTER(gdn_linattn_form)]
        L.gdn_linattn_workspace_bytes.restype = ctypes.c_size_t
        L.gdn_linattn_workspace_bytes.argtypes = [ctypes.POINTER(gdn_shape), ctypes.c_int]
        L.gdn_selftest_wait_timeout.restype = ctypes.c_int
        L.gdn_selftest_wait_timeout.argtypes = [ctypes.c_int, vp]
        L.gdn_prefill_static.restype = ctypes.c_int
        L.gdn_prefill_static.argtypes = [ctypes.POINTER(gdn_shape), ctypes.POINTER(gdn_prefill_io), vp]
        L.gdn_prefill_workspace_bytes.restype = ctypes.c_size_t
        L.gdn_prefill_workspace_bytes.argtypes = [ctypes.POINTER(gdn_shape), ctypes.c_int]
        L.gdn_prefill_staged_bytes.restype = ctypes.c_size_t
        L.gdn_prefill_staged_bytes.argtypes = [ctypes.POINTER(gdn_shape), ctypes.c_int]
        _lib = L
    return _lib


def gdn_abi_version():
    return lib().gdn_abi_version()


def gdn_status_str(status):
    return lib().gdn_status_str(int(status)).decode()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _io_code(dtype):
    if dtype == torch.bfloat16:
        return GDN_BF16
    if dtype == torch.float32:
        return GDN_F32
    raise TypeError("io tensors must be bfloat16 or float32, not %s" % dtype)


def _head_width(C, Hk, Hv):
    D, rem = divmod(C, 2 * Hk + Hv)
    if rem:
        raise ValueError("channel count %d is not (2*Hk + Hv) * D" % C)
    return D


def make_shape(B, T, Hk, Hv, D, io_dtype, eps_l2=1e-6, eps_norm=1e-6, q_scale=0.0):
    return gdn_shape(B, T, Hk, Hv, D, D, io_dtype, eps_l2, eps_norm, q_scale)


def gdn_prefill(qkv_pre, z, g, beta, conv_w, norm_w, S0, conv0, o, S_T, conv_T, *, Hk, Hv,
                eps_l2=1e-6, eps_norm=1e-6, q_scale=0.0, stream=None):
    """Prefill T tokens of B sequences (layouts as in gdn.h).  S0 / conv0 may
    be None (zeros); S_T may be S0 itself.  Raises GdnError on a non-OK status."""
    B, T, C = qkv_pre.shape
    sh = make_shape(B, T, Hk, Hv, _head_width(C, Hk, Hv), _io_code(qkv_pre.dtype),
                    eps_l2, eps_norm, q_scale)
    st = lib().gdn_prefill(ctypes.byref(sh), _ptr(qkv_pre), _ptr(z), _ptr(g), _ptr(beta),
                           _ptr(conv_w), _ptr(norm_w), _ptr(S0), _ptr(conv0), _ptr(o),
                           _ptr(S_T), _ptr(conv_T), _stream(stream))
    if st != GDN_OK:
        raise GdnError(st, "gdn_prefill")


def gdn_decode_step(qkv_pre, z, g, beta, conv_w, norm_w, S, conv_in, conv_out, o, *, Hk, Hv,
                    eps_l2=1e-6, eps_norm=1e-6, q_scale=0.0, stream=None):
    """One decode token for B sequences; S is updated in place, the new conv
    window goes to conv_out (distinct from conv_in)."""
    B, C = qkv_pre.shape
    sh = make_shape(B, 1, Hk, Hv, _head_width(C, Hk, Hv), _io_code(qkv_pre.dtype),
                    eps_l2, eps_norm, q_scale)
    st = lib().gdn_decode_step(ctypes.byref(sh), _ptr(qkv_pre), _ptr(z), _ptr(g), _ptr(beta),
                               _ptr(conv_w), _ptr(norm_w), _ptr(S), _ptr(conv_in),
                               _ptr(conv_out), _ptr(o), _stream(stream))
    if st != GDN_OK:
        raise GdnError(st, "gdn_decode_step")


def _raw(raw_gates):
    """A gdn_raw_gates struct from dict(a, b, A_log, dt_bias) of tensors, or None."""
    if raw_gates is None:
        return None
    return gdn_raw_gates(*[_ptr(raw_gates[k]) for k in ("a", "b", "A_log", "dt_bias")])


def gdn_prefill_ex(qkv_pre, z, g, beta, conv_w, norm_w, S0, conv0, o, S_T, conv_T, *, Hk, Hv,
                   raw_gates=None, cu_seqlens=None, S_snap=None, workspace=None, eps_l2=1e-6,
                   eps_norm=1e-6, q_scale=0.0, stream=None, _entry="gdn_prefill_ex"):
    """Prefill with the options of gdn_prefill_ex: raw gate projections
    (raw_gates = dict(a, b, A_log, dt_bias), g = beta = None), packed
    sequences (qkv_pre [N, C], z and o [N, Hv*D], cu_seqlens int32 [B+1] on
    the device), per-token state snapshots S_snap [tokens, Hv, D, D], and a
    device workspace (any tensor of at least gdn_prefill_workspace_bytes()
    bytes) for the staged q^ / k^ path."""
    if cu_seqlens is not None:
        N, C = qkv_pre.shape
        B, T = cu_seqlens.numel() - 1, N
    else:
        B, T, C = qkv_pre.shape
    io_dtype = _io_code(qkv_pre.dtype)
    sh = make_shape(B, T, Hk, Hv, _head_width(C, Hk, Hv), io_dtype, eps_l2, eps_norm, q_scale)
    rg = _raw(raw_gates)
    io = gdn_prefill_io(_ptr(qkv_pre), _ptr(z), _ptr(g), _ptr(beta),
                        None if rg is None else ctypes.addressof(rg), _ptr(conv_w), _ptr(norm_w),
                        _ptr(S0), _ptr(conv0), _ptr(o), _ptr(S_T), _ptr(conv_T), _ptr(cu_seqlens),
                        _ptr(S_snap), _ptr(workspace),
                        0 if workspace is None else workspace.numel() * workspace.element_size())
    st = getattr(lib(), _entry)(ctypes.byref(sh), ctypes.byref(io), _stream(stream))
    if st != GDN_OK:
        raise GdnError(st, _entry)


def gdn_prefill_static(qkv_pre, z, g, beta, conv_w, norm_w, S0, conv0, o, S_T, conv_T, *, Hk, Hv, **kw):
    """gdn_prefill_ex in the library's own device scratch (gdn_prefill_static):
    no workspace argument, no allocation; calls that overlap in time race."""
    if kw.get("workspace") is not None:
        raise ValueError("gdn_prefill_static takes no workspace")
    gdn_prefill_ex(qkv_pre, z, g, beta, conv_w, norm_w, S0, conv0, o, S_T, conv_T, Hk=Hk, Hv=Hv,
                   _entry="gdn_prefill_static", **kw)


def gdn_prefill_workspace_bytes(B, T, Hk, Hv, packed=False, D=128, io_dtype=None):
    """Workspace bytes of the chunk-parallel prefill (gdn_prefill_workspace_bytes)."""
    sh = make_shape(B, T, Hk, Hv, D, GDN_BF16 if io_dtype is None else io_dtype)
    return lib().gdn_prefill_workspace_bytes(ctypes.byref(sh), 1 if packed else 0)


def gdn_prefill_staged_bytes(B, T, Hk, Hv, packed=False, D=128, io_dtype=None):
    """Workspace bytes of the staged q^ / k^ form alone (gdn_prefill_staged_bytes)."""
    sh = make_shape(B, T, Hk, Hv, D, GDN_BF16 if io_dtype is None else io_dtype)
    return lib().gdn_prefill_staged_bytes(ctypes.byref(sh), 1 if packed else 0)


def gdn_decode_ex(qkv_pre, z, g, beta, conv_w, norm_w, S, conv_in, conv_out, o, *, Hk, Hv,
                  raw_gates=None, S_snap=None, eps_l2=1e-6, eps_norm=1e-6, q_scale=0.0,
                  stream=None):
    """T new tokens per sequence from the cache (qkv_pre [B, T, C], z and o
    [B, T, Hv*D]); S is updated in place; S_snap [B, T, Hv, D, D] (optional)
    receives the state after every token; the window after the T tokens goes
    to conv_out."""
    B, T, C = qkv_pre.shape
    sh = make_shape(B, T, Hk, Hv, _head_width(C, Hk, Hv), _io_code(qkv_pre.dtype), eps_l2,
                    eps_norm, q_scale)
    rg = _raw(raw_gates)
    io = gdn_decode_io(_ptr(qkv_pre), _ptr(z), _ptr(g), _ptr(beta),
                       None if rg is None else ctypes.addressof(rg), _ptr(conv_w), _ptr(norm_w),
                       _ptr(S), _ptr(S_snap), _ptr(conv_in), _ptr(conv_out), _ptr(o))
    st = lib().gdn_decode_ex(ctypes.byref(sh), ctypes.byref(io), _stream(stream))
    if st != GDN_OK:
        raise GdnError(st, "gdn_decode_ex")


def gdn_linear(x, w, outs, stream=None):
    """y = x w^T for bf16 x [M, K] and w [N, K] (row strides may exceed K);
    ``outs`` lists (col_begin, col_end, tensor) with tensor a bf16 [M, >=
    col_end - col_begin] view (row stride from the tensor) receiving those
    columns of y."""
    M, K = x.shape
    N, K2 = w.shape
    if K2 != K:
        raise ValueError("x and w disagree on K")
    arr = (gdn_linear_out * len(outs))(*[gdn_linear_out(int(b), int(e), _ptr(t), int(t.stride(0)))
                                         for b, e, t in outs])
    st = lib().gdn_linear(M, N, K, _ptr(x), int(x.stride(0)), _ptr(w), int(w.stride(0)), len(outs), arr,
                          _stream(stream))
    if st != GDN_OK:
        raise GdnError(st, "gdn_linear")


def gdn_linear_ex(x, w, outs, *, bias=None, gated=False, stream=None):
    """y = act(x w^T + bias) + residual for bf16 x [M, K] and w [N, K], or,
    gated, y = act(p[:, :N]) * p[:, N:] + residual with w [2N, K] and bias
    [2N].  ``outs`` lists (col_begin, col_end, tensor[, act[, residual]]):
    ranges of the N output columns with their bf16 [M, >= width] tensors (row
    strides from the tensors), act one of ACTIVATIONS (default "none"),
    residual a tensor like the output, or the output itself (added in place)."""
    M, K = x.shape
    N, K2 = w.shape
    if K2 != K:
        raise ValueError("x and w disagree on K")
    if bias is not None:
        if bias.numel() != N or not bias.is_contiguous():
            raise ValueError("bias has one value per row of w")
        if bias.dtype != _BF16:
            raise TypeError("bias must be bfloat16")
    if gated:
        if N % 2:
            raise ValueError("gated: w has 2N rows")
        N //= 2
    packed = []
    for o in outs:
        begin, end, t = o[0], o[1], o[2]
        act = ACTIVATIONS[o[3]] if len(o) > 3 else 0
        res = o[4] if len(o) > 4 else None
        packed.append(_PACK_LINEAR_OUT.pack(
            begin, end, t.data_ptr(), _rows(t, M, end - begin, "output"), act, 0 if res is None else res.data_ptr(),
            0 if res is None else _rows(res, M, end - begin, "residual")))
    st = (_lib or lib()).gdn_linear_ex(M, N, K, 1 if gated else 0, x.data_ptr(), _rows(x, M, K, "x"), w.data_ptr(),
                                       _rows(w, 0, K, "w"), None if bias is None else bias.data_ptr(), len(packed),
                                       b"".join(packed), _raw_stream(stream, x))
    if st != GDN_OK:
        raise GdnError(st, "gdn_linear_ex")


def gdn_selftest_linear_ex_form(M, N, K, gated=False, residual=False):
    """The kernel that gdn_linear_ex takes for these sizes (gdn_selftest_linear_ex_form)."""
    f = gdn_linear_ex_form()
    st = lib().gdn_selftest_linear_ex_form(M, N, K, int(gated), int(residual), ctypes.byref(f))
    if st != GDN_OK:
        raise GdnError(st, "gdn_selftest_linear_ex_form")
    return f


_BF16 = torch.bfloat16
_PACK_LINEAR_OUT = struct.Struct("=2iQqi4xQq")  # gdn_linear_ex_out


def _raw_stream(stream, t):
    """The stream handle of a call on `t`'s device (the current stream if none is given)."""
    if stream is None:
        dev = t.get_device()
        return torch._C._cuda_getCurrentRawStream(dev) if dev >= 0 else None
    return _stream(stream)


def _rows(t, M, cols, what):
    """Elements between the rows of a bf16 matrix of at least M rows of `cols` (one row: at least its width,
    in whole 16 bytes)."""
    shape = t.shape
    if t.dtype != _BF16:
        raise TypeError("%s must be bfloat16" % what)
    if len(shape) != 2 or shape[0] < M or shape[1] < cols:
        raise ValueError("%s is smaller than its columns" % what)
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError("%s: rows must be contiguous" % what)
    return ld if shape[0] > 1 else max(ld, -(-shape[1] // 8) * 8)


def _token_rows(t, what):
    """(tokens per sequence or in all, width, elements between token rows) of [B, T, C] (sequences back to back)
    or [tokens, C]."""
    shape, st = t.shape, t.stride()
    if len(shape) == 3:
        B, T, C = shape
        s0, ld, one = st
        if T == 1:
            ld = s0 if B > 1 else (C + 7) // 8 * 8
        elif B > 1 and s0 != T * ld:
            raise ValueError("%s: sequences must follow each other at the token stride" % what)
    else:
        B, T, C = 0, *shape
        ld, one = st
        if T == 1:
            ld = (C + 7) // 8 * 8
    if one != 1:
        raise ValueError("%s: the last dimension must be contiguous" % what)
    return B, T, C, ld


# The layouts of gdn_shape and gdn_linattn_io, packed in one go: the smallest
# calls take a few microseconds, of which filling the structures would be two.
_PACK_SHAPE = struct.Struct("=7i3f")
_PACK_LINATTN = struct.Struct("=3Q4q8Q")
_F32 = torch.float32
_IO_CODES = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}


def _linattn(entry, q, k, v, o, S0, S_T, Hk, Hv, g, log_decay, cu_seqlens, workspace, scale, stream):
    dtype = q.dtype
    if not (k.dtype == dtype and v.dtype == dtype and o.dtype == dtype) or dtype not in _IO_CODES:
        raise TypeError("q, k, v and o have one dtype, bfloat16 or float32")
    B, T, C, ldq = _token_rows(q, "q")
    Bk, Tk, Ck, ldk = _token_rows(k, "k")
    Bv, Tv, Cv, ldv = _token_rows(v, "v")
    Bo, To, Co, ldo = _token_rows(o, "o")
    D = C // Hk
    if not (B == Bk == Bv == Bo and T == Tk == Tv == To and C == Ck == Hk * D and Cv == Co == Hv * D):
        raise ValueError("q and k are [.., Hk * D], v and o [.., Hv * D], over the same tokens")
    tokens = B * T
    if cu_seqlens is not None:
        if B or cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_contiguous():
            raise ValueError("packed: q is [tokens, Hk * D], cu_seqlens contiguous int32 [B + 1]")
        B, tokens = cu_seqlens.numel() - 1, T
    elif not B:
        raise ValueError("q is [B, T, Hk * D]")
    if g is not None:
        _fp32(g, tokens * Hv, "g")
    if log_decay is not None:
        _fp32(log_decay, Hv, "log_decay")
    n = B * Hv * D * D
    _fp32(S_T, n, "the state")
    if S0 is not None:
        _fp32(S0, n, "S0")
    ws = ws_bytes = 0
    if workspace is not None and workspace.numel():
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = getattr(_lib or lib(), entry)(
        _PACK_SHAPE.pack(B, T, Hk, Hv, D, D, _IO_CODES[dtype], 0.0, 0.0, scale),
        _PACK_LINATTN.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), ldq, ldk, ldv, ldo,
                           0 if g is None else g.data_ptr(), 0 if log_decay is None else log_decay.data_ptr(),
                           0 if S0 is None else S0.data_ptr(), o.data_ptr(), S_T.data_ptr(),
                           0 if cu_seqlens is None else cu_seqlens.data_ptr(), ws, ws_bytes),
        _raw_stream(stream, q))
    if st != GDN_OK:
        raise GdnError(st, entry)


def _fp32(t, n, what):
    if t.dtype != _F32 or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s: %d contiguous float32 values are wanted" % (what, n))


def gdn_linattn_prefill(q, k, v, S0, o, S_T, *, Hk, Hv, g=None, log_decay=None, cu_seqlens=None, workspace=None,
                        scale=0.0, stream=None):
    """Linear attention with decay over prompts (gdn_linattn_prefill): q, k
    [B, T, Hk*D], v and o [B, T, Hv*D] (packed: [tokens, ..] with cu_seqlens
    int32 [B+1]), rows possibly strided; g [.., Hv] or log_decay [Hv]; S0 (or
    None) and S_T [B, Hv, D, D]; a workspace of gdn_linattn_workspace_bytes().
    bf16 prompts run in chunks of 64 tokens, where a log decay acts as -80 at
    least and an output sees at least 2^-58 of the state at its chunk's start."""
    _linattn("gdn_linattn_prefill", q, k, v, o, S0, S_T, Hk, Hv, g, log_decay, cu_seqlens, workspace, scale, stream)


def gdn_linattn_decode(q, k, v, S, o, *, Hk, Hv, g=None, log_decay=None, scale=0.0, stream=None):
    """T >= 1 new tokens per sequence from the cached state S [B, Hv, D, D],
    updated in place (gdn_linattn_decode); q, k [B, T, Hk*D], v, o [B, T, Hv*D]."""
    _linattn("gdn_linattn_decode", q, k, v, o, None, S, Hk, Hv, g, log_decay, None, None, scale, stream)


def gdn_linattn_workspace_bytes(B, T, Hk, Hv, packed=False, D=128, io_dtype=None):
    """Workspace bytes of gdn_linattn_prefill (packed: T is the total token count)."""
    sh = make_shape(B, T, Hk, Hv, D, GDN_BF16 if io_dtype is None else io_dtype)
    return lib().gdn_linattn_workspace_bytes(ctypes.byref(sh), 1 if packed else 0)


def gdn_selftest_linattn_form(B, T, Hk, Hv, packed=False, workspace=True, D=128, io_dtype=None):
    """How gdn_linattn_prefill runs this shape (gdn_selftest_linattn_form)."""
    sh, f = make_shape(B, T, Hk, Hv, D, GDN_BF16 if io_dtype is None else io_dtype), gdn_linattn_form()
    st = lib().gdn_selftest_linattn_form(ctypes.byref(sh), int(packed), int(workspace), ctypes.byref(f))
    if st != GDN_OK:
        raise GdnError(st, "gdn_selftest_linattn_form")
    return f


def gdn_device_status(stream=None, reset=False):
    """Synchronise and return the device-side status code (0 = OK)."""
    return lib().gdn_device_status(_stream(stream), int(bool(reset)))


def gdn_selftest_wait_timeout(wait_us, stream=None):
    """Enqueue the failure-detection self-test: a kernel whose bounded wait
    runs out after `wait_us` microseconds and records a timeout."""
    st = lib().gdn_selftest_wait_timeout(int(wait_us), _stream(stream))
    if st != GDN_OK:
        raise GdnError(st, "gdn_selftest_wait_timeout")


# ---------------------------------------------------------------- helpers
def alloc_prefill_outputs(B, T, Hk, Hv, dtype, device="cuda", D=128):
    """Fresh (o, S_T, conv_T) buffers for a prefill call."""
    C = (2 * Hk + Hv) * D
    o = torch.empty(B, T, Hv * D, dtype=dtype, device=device)
    S_T = torch.empty(B, Hv, D, D, dtype=torch.float32, device=device)
    conv_T = torch.empty(B, 3, C, dtype=dtype, device=device)
    return o, S_T, conv_T


def default_q_scale(D=128):
    return 1.0 / math.sqrt(D)
