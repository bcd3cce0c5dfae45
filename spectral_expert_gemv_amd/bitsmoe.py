"""ctypes binding of libbitsmoe.so (declared in include/bitsmoe.h).

Argument marshalling only: every device step runs in the library's gfx950
kernels.  Device buffers are torch tensors (torch provides memory and
streams); host buffers are numpy arrays.  There is no fallback: if the
library is missing, importing this module raises.
"""
import ctypes
import functools
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbitsmoe.so")

OK, EINVAL, ESHAPE, EBITS, ENOSPC, EFORMAT, EHIP = 0, -1, -2, -3, -4, -5, -6


class BitsMoEError(RuntimeError):
    def __init__(self, status, detail):
        super().__init__("%s (status %d): %s" % (_strerror(status), status, detail))
        self.status = status
        self.detail = detail


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libbitsmoe.so is not built (%s); run "
                          "`python -m spectral_expert_gemv_amd.build`" % LIB_PATH)
    # One HIP runtime per process: torch ships its own libamdhip64 under the
    # same soname as ROCm's, and the library's launches must run in the
    # runtime that owns torch's device memory and streams.  Importing torch
    # first makes the library's libamdhip64.so.7 dependency resolve to
    # torch's copy (loaded the other way round, the library's first launch
    # finds no device).
    import torch  # noqa: F401
    return ctypes.CDLL(LIB_PATH)


_lib = _load()

_vp, _sz, _i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
_i64, _f = ctypes.c_int64, ctypes.c_float
_pi = ctypes.POINTER(ctypes.c_int)
_psz = ctypes.POINTER(ctypes.c_size_t)

_SIGS = {
    "bitsmoe_version": ([], _i),
    "bitsmoe_strerror": ([_i], ctypes.c_char_p),
    "bitsmoe_last_error_detail": ([], ctypes.c_char_p),
    "bitsmoe_pack_size": ([_i, _i, _i, _vp, _psz], _i),
    "bitsmoe_pack": ([_i, _i, _i, _vp, _vp, _vp, _vp, _sz], _i),
    "bitsmoe_blob_check": ([_vp, _sz, _pi, _pi, _pi], _i),
    "bitsmoe_spectral_proj": ([_vp, _vp, _vp, _i, _i, _i, _vp], _i),
    "bitsmoe_expert_apply": ([_vp, _sz, _i, _i, _i, _vp, _i, _vp, _i, _i, _vp, _vp, _sz, _vp], _i),
    "bitsmoe_moe_gateup_workspace_size": ([_i, _i, _i, _i, _i, _i, _psz], _i),
    "bitsmoe_moe_gateup": ([_vp, _sz, _vp, _sz, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i,
                            _vp, _vp, _sz, _vp], _i),
    "bitsmoe_moe_gateup_noalloc": ([_vp, _sz, _vp, _sz, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                                    _i, _vp, _vp], _i),
    "bitsmoe_workspace_init": ([_vp, _sz, _vp], _i),
    "bitsmoe_dump_codes": ([_vp, _sz, _i, _i, _i, _i, _i, _vp, _vp], _i),
    "bitsmoe_debug_set_wait_limit": ([ctypes.c_uint32], ctypes.c_uint32),
    "bitsmoe_wait_timeouts": ([_vp, _sz, ctypes.POINTER(ctypes.c_uint32), _vp], _i),
    "bitsmoe_pack_device_workspace_size": ([_i, _i, _i, _vp, _psz], _i),
    "bitsmoe_pack_device": ([_i, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp, _sz, _vp], _i),
    "bitsmoe_fqcm_distortion": ([_vp, _i, _i, _i, _vp, _vp], _i),
    "bitsmoe_fqcm_beta": ([_vp, _i, _vp, _vp, _i, _i, _i, _i, _vp, _vp], _i),
    "bitsmoe_fqcm_allocate": ([_vp, _vp, _vp, _i, _i, _i, ctypes.c_uint64, _vp,
                               ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_uint64),
                               ctypes.POINTER(ctypes.c_double), _vp, _sz, _vp], _i),
    "bitsmoe_moe_down_workspace_size": ([_i, _i, _i, _i, _i, _i, _psz], _i),
    "bitsmoe_moe_down": ([_vp, _sz, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _sz,
                          _vp], _i),
    "bitsmoe_ssd_workspace_size": ([_i, _i, _i, _i, _psz], _i),
    "bitsmoe_moe_route": ([_i, _vp, _i64, _i, _i, _i, _i, _f, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                           _vp], _i),
    "bitsmoe_moe_route_grad": ([_i, _vp, _i64, _vp, _vp, _i, _i, _i, _i, _f, _vp, _i64, _vp], _i),
    "bitsmoe_moe_group_workspace_size": ([_i, _i, _psz], _i),
    "bitsmoe_moe_group": ([_vp, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp], _i),
    "bitsmoe_grouped_matmul_workspace_size": ([_i, _vp, _i64, _i64, _vp, _i64, _i64, _i, _i, _i,
                                               _i, _i, _psz], _i),
    "bitsmoe_grouped_matmul": ([_i, _vp, _i64, _i, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _vp, _i,
                                _i64, _vp, _sz, _vp], _i),
    "bitsmoe_grouped_matmul_dx": ([_i, _vp, _i64, _vp, _vp, _i, _i, _i, _i, _vp, _i, _i64, _vp,
                                   _sz, _vp], _i),
    "bitsmoe_grouped_matmul_dw": ([_i, _vp, _i64, _vp, _i64, _i, _vp, _i, _vp, _i, _i, _i, _i,
                                   _vp, _i, _vp, _sz, _vp], _i),
    "bitsmoe_silu_mul": ([_i, _vp, _i64, _vp, _i, _i, _i, _vp, _i64, _vp], _i),
    "bitsmoe_silu_mul_grad": ([_i, _vp, _i64, _vp, _i64, _vp, _i, _i, _i, _vp, _i64, _vp], _i),
    "bitsmoe_moe_combine": ([_i, _vp, _i64, _i, _vp, _vp, _i, _i, _i, _vp, _i, _i64, _vp], _i),
    "bitsmoe_moe_combine_grad": ([_vp, _i, _i64, _i, _vp, _i64, _i, _vp, _vp, _i, _i, _i, _vp,
                                  _i64, _vp, _vp], _i),
    "bitsmoe_w4_matmul": ([_i, _vp, _i64, _i, _vp, _i, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i,
                           _vp, _i, _i64, _vp], _i),
    "bitsmoe_w4_pack": ([_vp, _i64, _i, _i, _vp, _vp, _vp], _i),
    "bitsmoe_ssd": ([_vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _pi, _i, _vp, _sz, _vp], _i),
}
FQCM_WS_BYTES = 1024 + 65536 * 24
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res

EXPORTS = tuple(_SIGS)


def _strerror(status):
    return _lib.bitsmoe_strerror(int(status)).decode()


def _check(status):
    if status != OK:
        raise BitsMoEError(status, _lib.bitsmoe_last_error_detail().decode())


def version():
    return _lib.bitsmoe_version()


def _ptr(t):
    """Device pointer of a torch tensor or host pointer of a numpy array."""
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _nbytes(t):
    if isinstance(t, np.ndarray):
        return t.nbytes
    return t.numel() * t.element_size()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ---------------------------------------------------------------- host side

def pack_size(E, dout, r, bits):
    bits = np.ascontiguousarray(bits, dtype=np.uint8)
    out = ctypes.c_size_t(0)
    _check(_lib.bitsmoe_pack_size(E, dout, r, bits.ctypes.data, ctypes.byref(out)))
    return out.value


def pack(p, a, bits):
    """Quantize and pack one linear type (p: E x r x dout, a, bits: E x r)."""
    p = np.ascontiguousarray(p, dtype=np.float32)
    a = np.ascontiguousarray(a, dtype=np.float32)
    bits = np.ascontiguousarray(bits, dtype=np.uint8)
    E, r, dout = p.shape
    if a.shape != (E, r) or bits.shape != (E, r):
        raise ValueError("a and bits must be E x r")
    n = pack_size(E, dout, r, bits)
    out = np.zeros(n, dtype=np.uint8)
    _check(_lib.bitsmoe_pack(E, dout, r, p.ctypes.data, a.ctypes.data, bits.ctypes.data,
                             out.ctypes.data, out.nbytes))
    return out


def blob_check(blob):
    blob = np.ascontiguousarray(blob, dtype=np.uint8)
    E, dout, r = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(_lib.bitsmoe_blob_check(blob.ctypes.data, blob.nbytes, ctypes.byref(E),
                                   ctypes.byref(dout), ctypes.byref(r)))
    return E.value, dout.value, r.value


# -------------------------------------------------------------- device side

def spectral_proj(phi_t, x, z, stream=None):
    """z[T, R] = x[T, din] @ phi_t[R, din]^T (phi_t, x fp16; z float32)."""
    R, din = phi_t.shape
    T = x.shape[0]
    _check(_lib.bitsmoe_spectral_proj(_ptr(phi_t), _ptr(x), _ptr(z), T, din, R,
                                      _stream(stream)))


def expert_apply(packed, E, dout, r, z, ids, y, z_stride=None, ws=None, stream=None):
    T, k = ids.shape
    zs = z.shape[1] if z_stride is None else z_stride
    _check(_lib.bitsmoe_expert_apply(_ptr(packed), _nbytes(packed), E, dout, r, _ptr(z), zs,
                                     _ptr(ids), T, k, _ptr(y), _ptr(ws),
                                     0 if ws is None else _nbytes(ws), _stream(stream)))


def moe_gateup_workspace_size(T, k, E, din, dout, r):
    out = ctypes.c_size_t(0)
    _check(_lib.bitsmoe_moe_gateup_workspace_size(T, k, E, din, dout, r, ctypes.byref(out)))
    return out.value


def moe_gateup(packed_gate, packed_up, phi_t_gateup, x, ids, E, dout, r, h, ws, stream=None):
    T, k = ids.shape
    din = x.shape[1]
    _check(_lib.bitsmoe_moe_gateup(_ptr(packed_gate), _nbytes(packed_gate), _ptr(packed_up),
                                   _nbytes(packed_up), _ptr(phi_t_gateup), _ptr(x), _ptr(ids),
                                   T, k, E, din, dout, r, _ptr(h), _ptr(ws), _nbytes(ws),
                                   _stream(stream)))


# bytes of the static workspace behind moe_gateup_noalloc
GATEUP_NOALLOC_MAX_WS = 64 << 20


def moe_gateup_noalloc(packed_gate, packed_up, phi_t_gateup, x, ids, E, dout, r, h,
                       stream=None):
    """moe_gateup on the library's static per-device workspace (no workspace
    argument; calls that overlap in time on one device race)."""
    T, k = ids.shape
    din = x.shape[1]
    _check(_lib.bitsmoe_moe_gateup_noalloc(_ptr(packed_gate), _nbytes(packed_gate),
                                           _ptr(packed_up), _nbytes(packed_up),
                                           _ptr(phi_t_gateup), _ptr(x), _ptr(ids), T, k, E,
                                           din, dout, r, _ptr(h), _stream(stream)))


def workspace_init(ws, stream=None):
    _check(_lib.bitsmoe_workspace_init(_ptr(ws), _nbytes(ws), _stream(stream)))


def debug_set_wait_limit(spins):
    """Sets the bound on the one-launch gate/up kernel's waits for z (0: give
    up at once, every row NaN); returns the previous bound.  Test hook."""
    return int(_lib.bitsmoe_debug_set_wait_limit(int(spins)))


def wait_timeouts(ws=None, stream=None):
    """Waits of the one-launch gate/up kernels that gave up (rows written as
    NaN) since the workspace was zero-filled; ws=None reads the static
    workspace of moe_gateup_noalloc.  Synchronises the stream."""
    n = ctypes.c_uint32(0)
    if ws is None:
        _check(_lib.bitsmoe_wait_timeouts(None, 0, ctypes.byref(n), _stream(stream)))
    else:
        _check(_lib.bitsmoe_wait_timeouts(_ptr(ws), _nbytes(ws), ctypes.byref(n),
                                          _stream(stream)))
    return int(n.value)


DUMP_I8, DUMP_F16, DUMP_LANE = 0, 1, 2


def dump_codes(packed, E, dout, r, e, codes, path=DUMP_LANE, stream=None):
    """Codes of expert e as decoder `path` builds them (DUMP_I8: int8 operand
    bytes of the one-launch kernel; DUMP_F16: fp16 operands of the batched
    kernel; DUMP_LANE: codes of the lane-per-row kernel)."""
    _check(_lib.bitsmoe_dump_codes(_ptr(packed), _nbytes(packed), E, dout, r, e, path,
                                   _ptr(codes), _stream(stream)))


def pack_device_workspace_size(E, dout, r, bits):
    bits = np.ascontiguousarray(bits, dtype=np.uint8)
    out = ctypes.c_size_t(0)
    _check(_lib.bitsmoe_pack_device_workspace_size(E, dout, r, bits.ctypes.data,
                                                   ctypes.byref(out)))
    return out.value


def pack_device(p, a, bits, out=None, ws=None, stream=None):
    """Quantize and pack one linear type on the GPU.  p: E x r x dout and a:
    E x r float32 device tensors; bits: E x r host widths.  Returns the blob as
    a uint8 device tensor (`out` if given); the call returns once it is
    complete."""
    import torch
    bits = np.ascontiguousarray(bits, dtype=np.uint8)
    E, r, dout = p.shape
    if tuple(a.shape) != (E, r) or bits.shape != (E, r):
        raise ValueError("a and bits must be E x r")
    if p.dtype != torch.float32 or a.dtype != torch.float32:
        raise ValueError("p and a must be float32")
    if not (p.is_contiguous() and a.is_contiguous()):
        raise ValueError("p and a must be contiguous")
    if out is None:
        out = torch.empty(pack_size(E, dout, r, bits), dtype=torch.uint8, device=p.device)
    if ws is None:
        ws = torch.empty(pack_device_workspace_size(E, dout, r, bits), dtype=torch.uint8,
                         device=p.device)
    _check(_lib.bitsmoe_pack_device(E, dout, r, _ptr(p), _ptr(a), bits.ctypes.data, _ptr(out),
                                    _nbytes(out), _ptr(ws), _nbytes(ws), _stream(stream)))
    return out


def fqcm_distortion(p, eps=None, stream=None):
    """eps (E x r x 8 float64 device tensor) of the unit directions p
    (E x r x dout float32 device tensor)."""
    import torch
    E, r, dout = p.shape
    if p.dtype != torch.float32 or not p.is_contiguous():
        raise ValueError("p must be contiguous float32")
    if eps is None:
        eps = torch.empty((E, r, 8), dtype=torch.float64, device=p.device)
    _check(_lib.bitsmoe_fqcm_distortion(_ptr(p), E, r, dout, _ptr(eps), _stream(stream)))
    return eps


def fqcm_beta(z, ids, g, E, beta=None, stream=None):
    """beta (E x r float64) from z (T x r float32, row stride z.stride(0)),
    ids (T x k int32) and routing weights g (T x k float32), device tensors."""
    import torch
    T, r = z.shape
    k = ids.shape[1]
    if z.dtype != torch.float32 or z.stride(1) != 1:
        raise ValueError("z must be float32 with unit column stride")
    if ids.dtype != torch.int32 or g.dtype != torch.float32 or tuple(g.shape) != (T, k):
        raise ValueError("ids must be int32 and g float32, both T x k")
    if beta is None:
        beta = torch.empty((E, r), dtype=torch.float64, device=z.device)
    _check(_lib.bitsmoe_fqcm_beta(_ptr(z), z.stride(0), _ptr(ids.contiguous()),
                                  _ptr(g.contiguous()), T, k, E, r, _ptr(beta), _stream(stream)))
    return beta


def fqcm_allocate(a, beta, eps, dout, budget_bits, bits=None, ws=None, stream=None):
    """Least-loss widths within the bit budget; returns (bits uint8 device
    tensor E x r, the Lagrangian multiplier lam, bits used, loss minus the
    dual bound at lam)."""
    import torch
    E, r = a.shape
    if bits is None:
        bits = torch.empty((E, r), dtype=torch.uint8, device=a.device)
    if ws is None:
        ws = torch.empty(FQCM_WS_BYTES, dtype=torch.uint8, device=a.device)
    lam = ctypes.c_double(0.0)
    used = ctypes.c_uint64(0)
    gap = ctypes.c_double(0.0)
    _check(_lib.bitsmoe_fqcm_allocate(_ptr(a), _ptr(beta), _ptr(eps), E, r, dout,
                                      int(budget_bits), _ptr(bits), ctypes.byref(lam),
                                      ctypes.byref(used), ctypes.byref(gap), _ptr(ws),
                                      _nbytes(ws), _stream(stream)))
    return bits, lam.value, used.value, gap.value


def moe_down_workspace_size(T, k, E, dout, din, r_d):
    out = ctypes.c_size_t(0)
    _check(_lib.bitsmoe_moe_down_workspace_size(T, k, E, dout, din, r_d, ctypes.byref(out)))
    return out.value


def moe_down(packed_down, phi_t_down, h, ids, g, E, din, r_d, out=None, ws=None, stream=None):
    """out (T x din float32) = sum_j g[t, j] * down_e(h[t, j]); h: T x k x
    dout float32, ids: T x k int32, g: T x k float32, phi_t_down: r_d x dout
    fp16, packed_down: the down blob; all device tensors."""
    import torch
    T, k, dout = h.shape
    if h.dtype != torch.float32 or g.dtype != torch.float32 or ids.dtype != torch.int32:
        raise ValueError("h and g must be float32, ids int32")
    h, ids, g = h.contiguous(), ids.contiguous(), g.contiguous()
    if out is None:
        out = torch.empty((T, din), dtype=torch.float32, device=h.device)
    if ws is None:
        ws = torch.empty(moe_down_workspace_size(T, k, E, dout, din, r_d), dtype=torch.uint8,
                         device=h.device)
    _check(_lib.bitsmoe_moe_down(_ptr(packed_down), _nbytes(packed_down), _ptr(phi_t_down),
                                 _ptr(h), _ptr(ids), _ptr(g), T, k, E, dout, din, r_d, _ptr(out),
                                 _ptr(ws), _nbytes(ws), _stream(stream)))
    return out


def ssd_workspace_size(E, dout, din, r):
    out = ctypes.c_size_t(0)
    _check(_lib.bitsmoe_ssd_workspace_size(E, dout, din, r, ctypes.byref(out)))
    return out.value


def ssd(W, r, max_sweeps=30, ws=None, stream=None):
    """Shared-basis decomposition of W (E x dout x din float32 device tensor).
    Returns (phi din x r, a E x r, p E x r x dout) device float32 tensors,
    sigma^2 (numpy float64, r) and the Jacobi sweeps taken."""
    import torch
    E, dout, din = W.shape
    if W.dtype != torch.float32 or not W.is_contiguous():
        raise ValueError("W must be contiguous float32")
    phi = torch.empty((din, r), dtype=torch.float32, device=W.device)
    a = torch.empty((E, r), dtype=torch.float32, device=W.device)
    p = torch.empty((E, r, dout), dtype=torch.float32, device=W.device)
    if ws is None:
        ws = torch.empty(ssd_workspace_size(E, dout, din, r), dtype=torch.uint8, device=W.device)
    s2 = np.zeros(r, dtype=np.float64)
    sw = ctypes.c_int(0)
    _check(_lib.bitsmoe_ssd(_ptr(W), E, dout, din, r, _ptr(phi), _ptr(a), _ptr(p),
                            s2.ctypes.data, ctypes.byref(sw), int(max_sweeps), _ptr(ws),
                            _nbytes(ws), _stream(stream)))
    return phi, a, p, s2, sw.value


# ------------------------------------------------ the expert layer's operators
#
# Routing, products with dense or 4-bit experts, the gated activation and the
# combine, with their gradients.  Sorted rows: the T*k (token, slot) pairs
# grouped by expert; `bounds` (E + 1), `order` (row -> pair) and `slot`
# (pair -> row) come from moe_route or moe_group.  Matrices may have any row
# stride; their rows are contiguous.  Without `stream` a call runs on the
# current stream of its tensors' device.

import torch  # noqa: E402  (after the library: see _load)

ACT = {None: 0, "silu_mul": 1}
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_I32, _F32 = torch.int32, torch.float32


def _dtype(t):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError("unsupported dtype %s" % t.dtype)
    return code


def _matrix(name, t, shape=None):
    """(pointer, row stride) of a 2-d tensor with contiguous rows."""
    have = t.shape
    if len(have) != 2 or (shape is not None and have != shape):
        raise ValueError("%s must be %s, got %s" % (name, "2-d" if shape is None else
                                                    "of shape %s" % (shape,), tuple(have)))
    step, one = t.stride()
    if one != 1 and have[1] > 1:
        raise ValueError("the rows of %s must be contiguous" % name)
    # the stride of a single row says nothing
    return t.data_ptr(), max(step, have[1]) if have[0] <= 1 else step


def _array(name, t, dtype, shape=None):
    """Pointer of a contiguous tensor of that dtype (and shape)."""
    if t.dtype is not dtype or (shape is not None and t.shape != shape):
        raise ValueError("%s must be %s of shape %s, got %s of %s" % (name, dtype, shape, t.dtype,
                                                                      tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _same_device(first, *rest):
    """The index of the tensors' one GPU."""
    index = first.get_device()
    if index < 0:
        raise ValueError("a tensor is on %s, not on a GPU" % first.device)
    for t in rest:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors on %s and %s" % (first.device, t.device))
    return index


def _enqueue(fn, index, stream, *args):
    """Calls fn(*args, stream) with the tensors' device as the current one."""
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return _enqueue(fn, index, stream, *args)
    if stream is None:
        # (the handle alone: a Stream object would take most of a call's time)
        stream = torch._C._cuda_getCurrentRawStream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    status = fn(*args, stream)
    if status:
        _check(status)


def _new(shape, dtype, index, stream, zero=False):
    """A tensor that belongs to the stream the call runs on."""
    make = torch.zeros if zero else torch.empty
    dev = torch.device("cuda", index)
    if stream is None:
        return make(shape, dtype=dtype, device=dev)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=dev)


def _ws_bytes(ws):
    if ws is None:
        return 0
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return _nbytes(ws)


def _scratch(nbytes, dev, stream):
    return _new(nbytes, torch.uint8, dev, stream) if nbytes else None


@functools.lru_cache(maxsize=256)
def moe_group_workspace_size(P, E):
    out = ctypes.c_size_t(0)
    _check(_lib.bitsmoe_moe_group_workspace_size(P, E, ctypes.byref(out)))
    return out.value


def _group_buffers(T, k, E, bounds, order, slot, dev, stream):
    i32 = _I32
    bounds = _new(E + 1, i32, dev, stream) if bounds is None else bounds
    order = _new(T * k, i32, dev, stream) if order is None else order
    slot = _new((T, k), i32, dev, stream) if slot is None else slot
    _array("bounds", bounds, _I32, (E + 1,))
    _array("order", order, _I32, (T * k,))
    _array("slot", slot, _I32, (T, k))
    return bounds, order, slot


def moe_group(ids, E, bounds=None, order=None, slot=None, ws=None, stream=None):
    """(bounds, order, slot) of the pairs of ids (T x k int32) by expert, in
    rising pair order; pairs with an id outside [0, E) come last, with -1."""
    T, k = ids.shape
    dev = _same_device(ids, bounds, order, slot, ws)
    pi = _array("ids", ids, _I32, (T, k))
    bounds, order, slot = _group_buffers(T, k, E, bounds, order, slot, dev, stream)
    if ws is None:
        ws = _scratch(moe_group_workspace_size(T * k, E), dev, stream)
    _enqueue(_lib.bitsmoe_moe_group, dev, stream, pi, T * k, E, bounds.data_ptr(),
             order.data_ptr(), slot.data_ptr(), _ptr(ws), _ws_bytes(ws))
    return bounds, order, slot


def moe_route(logits, k, ids=None, g=None, renorm=False, scale=1.0, bounds=None, order=None,
              slot=None, ws=None, stream=None):
    """(ids T x k int32, g T x k float32) of the k largest logits (T x E) of
    each token: softmax weights over all experts, or over the chosen ones
    (renorm), times scale.  With bounds, order and slot the pairs are grouped
    by expert as well, as by moe_group."""
    T, E = logits.shape
    dev = _same_device(logits, ids, g, bounds, order, slot, ws)
    pl, ld = _matrix("logits", logits)
    if ids is None:
        ids = _new((T, k), _I32, dev, stream)
    if g is None:
        g = _new((T, k), _F32, dev, stream)
    pi, pg = _array("ids", ids, _I32, (T, k)), _array("g", g, _F32, (T, k))
    pb = po = ps = None
    if bounds is not None or order is not None or slot is not None:
        if bounds is None or order is None or slot is None:
            raise ValueError("bounds, order and slot go together")
        pb = _array("bounds", bounds, _I32, (E + 1,))
        po = _array("order", order, _I32, (T * k,))
        ps = _array("slot", slot, _I32, (T, k))
        if ws is None and T * k:
            ws = _scratch(moe_group_workspace_size(T * k, E), dev, stream)
    _enqueue(_lib.bitsmoe_moe_route, dev, stream, _dtype(logits), pl, ld, T, E, k, int(renorm),
             scale, pi, pg, pb, po, ps, _ptr(ws), _ws_bytes(ws))
    return ids, g


def moe_route_grad(logits, ids, dg, dlogits=None, renorm=False, scale=1.0, stream=None):
    """dlogits (T x E, the logits' dtype) from dg (T x k float32) and the ids
    that moe_route gave for these logits."""
    T, E = logits.shape
    k = ids.shape[1]
    dev = _same_device(logits, ids, dg, dlogits)
    pl, ld = _matrix("logits", logits)
    if dlogits is None:
        dlogits = _new((T, E), logits.dtype, dev, stream)
    if dlogits.dtype != logits.dtype:
        raise ValueError("dlogits must have the logits' dtype")
    pd, ldd = _matrix("dlogits", dlogits, (T, E))
    _enqueue(_lib.bitsmoe_moe_route_grad, dev, stream, _dtype(logits), pl, ld,
             _array("ids", ids, _I32, (T, k)), _array("dg", dg, _F32, (T, k)), T,
             E, k, int(renorm), scale, pd, ldd)
    return dlogits


def _gather(x, rows, div, R):
    if rows is None:
        if x.shape[0] < R:
            raise ValueError("x has %d rows, the sorted layout %d" % (x.shape[0], R))
        return None, 1
    return _array("rows", rows, _I32, (R,)), div


def _bounds(bounds, E):
    return _array("bounds", bounds, _I32, (E + 1,))


def _matmul_scratch(op, pa, lda, a_rows, pb, ldb, b_rows, R, E, N, K, act, ws, index, stream):
    """The workspace of a product, or None: the given one, or one for operands
    whose rows are not whole 16-byte pieces."""
    if ws is not None or not ((pa | pb) & 15 or (lda | ldb | N | K) & 7):
        return ws
    out = ctypes.c_size_t(0)
    _check(_lib.bitsmoe_grouped_matmul_workspace_size(op, pa, lda, a_rows, pb, ldb, b_rows, R, E, N,
                                                      K, act, ctypes.byref(out)))
    return _scratch(out.value, index, stream)


def grouped_matmul(x, w, bounds, y=None, rows=None, div=1, act=None, ws=None, stream=None):
    """y (R x N) with y[i] = W_e x[i] for the sorted rows i of expert e.
    w: E x N x K; with act="silu_mul" E x 2N x K (gate rows first) and y =
    SiLU(gate) * up.  rows (R int32): row i reads x[rows[i] // div].  y has
    x's dtype, or float32 where it is given so."""
    E, n2, K = w.shape
    N = n2 // 2 if act else n2
    if act not in ACT or (act and n2 % 2):
        raise ValueError("act=%r with %d rows of w" % (act, n2))
    R = rows.shape[0] if rows is not None else y.shape[0] if y is not None else x.shape[0]
    dev = _same_device(x, w, bounds, y, rows, ws)
    px, ldx = _matrix("x", x, (x.shape[0], K))
    pr, div = _gather(x, rows, div, R)
    if y is None:
        y = _new((R, N), x.dtype, dev, stream)
    py, ldy = _matrix("y", y, (R, N))
    pw, code = _array("w", w, x.dtype), ACT[act]
    ws = _matmul_scratch(0, px, ldx, x.shape[0], pw, K, 0, R, E, N, K, code, ws, dev, stream)
    _enqueue(_lib.bitsmoe_grouped_matmul, dev, stream, _dtype(x), px, ldx, x.shape[0], pr, div, pw,
             _bounds(bounds, E), R, E, N, K, code, py, _dtype(y), ldy, _ptr(ws),
             _ws_bytes(ws))
    return y


def grouped_matmul_dx(dy, w, bounds, dx=None, ws=None, stream=None):
    """dx (R x K) with dx[i] = W_e^T dy[i]: the gradient of grouped_matmul's
    sorted rows (of a gathered x, moe_combine adds up a token's rows)."""
    E, N, K = w.shape
    R = dy.shape[0]
    dev = _same_device(dy, w, bounds, dx, ws)
    pd, ldd = _matrix("dy", dy, (R, N))
    if dx is None:
        dx = _new((R, K), dy.dtype, dev, stream)
    px, ldx = _matrix("dx", dx, (R, K))
    pw = _array("w", w, dy.dtype)
    ws = _matmul_scratch(1, pd, ldd, R, pw, K, 0, R, E, N, K, 0, ws, dev, stream)
    _enqueue(_lib.bitsmoe_grouped_matmul_dx, dev, stream, _dtype(dy), pd, ldd, pw,
             _bounds(bounds, E), R, E, N, K, px, _dtype(dx), ldx, _ptr(ws),
             _ws_bytes(ws))
    return dx


def grouped_matmul_dw(dy, x, bounds, dw=None, rows=None, div=1, ws=None, stream=None):
    """dw (E x N x K) with dw_e = sum of dy[i] x[i]^T over the sorted rows of
    expert e; 0 for an expert without rows.  float32 unless dw is given."""
    R, N = dy.shape
    K = x.shape[1]
    E = bounds.shape[0] - 1
    dev = _same_device(dy, x, bounds, dw, rows, ws)
    pd, ldd = _matrix("dy", dy)
    px, ldx = _matrix("x", x)
    if x.dtype != dy.dtype:
        raise ValueError("x and dy must have one dtype")
    pr, div = _gather(x, rows, div, R)
    if dw is None:
        dw = _new((E, N, K), _F32, dev, stream)
    ws = _matmul_scratch(2, pd, ldd, R, px, ldx, x.shape[0], R, E, N, K, 0, ws, dev, stream)
    _enqueue(_lib.bitsmoe_grouped_matmul_dw, dev, stream, _dtype(dy), pd, ldd, px, ldx, x.shape[0],
             pr, div, _bounds(bounds, E), R, E, N, K, _array("dw", dw, dw.dtype, (E, N, K)),
             _dtype(dw), _ptr(ws), _ws_bytes(ws))
    return dw


def silu_mul(a, h=None, bounds=None, stream=None):
    """h (R x F) = SiLU(gate) * up of rows a = [gate | up] (R x 2F); with
    bounds only the experts' rows."""
    R, F2 = a.shape
    dev = _same_device(a, h, bounds)
    pa, lda = _matrix("a", a)
    if F2 % 2:
        raise ValueError("a has %d columns" % F2)
    if h is None:
        h = _new((R, F2 // 2), a.dtype, dev, stream)
    if h.dtype != a.dtype:
        raise ValueError("h must have a's dtype")
    ph, ldh = _matrix("h", h, (R, F2 // 2))
    E = 0 if bounds is None else bounds.shape[0] - 1
    _enqueue(_lib.bitsmoe_silu_mul, dev, stream, _dtype(a), pa, lda,
             None if bounds is None else _bounds(bounds, E), R, E, F2 // 2, ph, ldh)
    return h


def silu_mul_grad(a, dh, da=None, bounds=None, stream=None):
    """da (R x 2F) from a and dh (R x F); da may be a itself."""
    R, F2 = a.shape
    dev = _same_device(a, dh, da, bounds)
    pa, lda = _matrix("a", a)
    if F2 % 2:
        raise ValueError("a has %d columns" % F2)
    if da is None:
        da = _new((R, F2), a.dtype, dev, stream)
    if dh.dtype != a.dtype or da.dtype != a.dtype:
        raise ValueError("dh and da must have a's dtype")
    pd, ldd = _matrix("dh", dh, (R, F2 // 2))
    po, ldo = _matrix("da", da, (R, F2))
    E = 0 if bounds is None else bounds.shape[0] - 1
    _enqueue(_lib.bitsmoe_silu_mul_grad, dev, stream, _dtype(a), pa, lda, pd, ldd,
             None if bounds is None else _bounds(bounds, E), R, E, F2 // 2, po, ldo)
    return da


def moe_combine(y, slot, g=None, out=None, stream=None):
    """out (T x D) = sum over j of g[t, j] * y[slot[t, j]], in slot order; a
    slot of -1 has a row of zeros.  out has y's dtype, or float32 where given so."""
    T, k = slot.shape
    R, D = y.shape
    dev = _same_device(y, slot, g, out)
    py, ldy = _matrix("y", y)
    if out is None:
        out = _new((T, D), y.dtype, dev, stream)
    po, ldo = _matrix("out", out, (T, D))
    _enqueue(_lib.bitsmoe_moe_combine, dev, stream, _dtype(y), py, ldy, R,
             _array("slot", slot, _I32, (T, k)),
             None if g is None else _array("g", g, _F32, (T, k)), T, k, D, po, _dtype(out),
             ldo)
    return out


def moe_combine_grad(dout, y, slot, g=None, dy=None, dg=None, stream=None):
    """(dy, dg) of moe_combine: dy[slot[t, j]] = g[t, j] * dout[t] (other rows
    as they were), dg[t, j] = <dout[t], y[slot[t, j]]>; the slots differ."""
    T, k = slot.shape
    R, D = y.shape
    dev = _same_device(dout, y, slot, g, dy, dg)
    py, ldy = _matrix("y", y)
    pd, ldd = _matrix("dout", dout, (T, D))
    if dy is None:
        dy = _new((R, D), y.dtype, dev, stream, zero=True)
    if dg is None:
        dg = _new((T, k), _F32, dev, stream)
    if dy.dtype != y.dtype:
        raise ValueError("dy must have y's dtype")
    pdy, lddy = _matrix("dy", dy, (R, D))
    _enqueue(_lib.bitsmoe_moe_combine_grad, dev, stream, pd, _dtype(dout), ldd, _dtype(y), py, ldy,
             R, _array("slot", slot, _I32, (T, k)),
             None if g is None else _array("g", g, _F32, (T, k)), T, k, D, pdy, lddy,
             _array("dg", dg, _F32, (T, k)))
    return dy, dg


def w4_pack(w, group=128):
    """(codes, scales, mins) of dense host weights w (... x K float32), 4 bits
    with a step and a minimum per `group` inputs."""
    w = np.ascontiguousarray(w, dtype=np.float32)
    K = w.shape[-1]
    if group < 1 or K % group:
        raise ValueError("K=%d is not a multiple of the group of %d" % (K, group))
    lead = w.shape[:-1]
    rows = int(np.prod(lead, dtype=np.int64))
    codes = np.empty(lead + (K // 2,), np.uint8)
    scales = np.empty(lead + (K // group,), np.float16)
    mins = np.empty_like(scales)
    _check(_lib.bitsmoe_w4_pack(w.ctypes.data, rows, K, group, codes.ctypes.data,
                                scales.ctypes.data, mins.ctypes.data))
    return codes, scales, mins


def w4_matmul(x, codes, scales, mins=None, y=None, bounds=None, rows=None, div=1, act=None,
              stream=None):
    """y (R x N) = W x with 4-bit weights W = mins + scales * codes, per group
    of K / scales.shape[-1] inputs (mins None: -8 * scales).  codes: E x N x
    K/2 uint8 (or N x K/2 for one dense projection); bounds, rows, div and act
    as for grouped_matmul (bounds may be None when E is 1)."""
    if codes.dim() == 2:
        codes, scales = codes.unsqueeze(0), scales.unsqueeze(0)
        mins = None if mins is None else mins.unsqueeze(0)
    E, n2, half = codes.shape
    K, groups = 2 * half, scales.shape[-1]
    N = n2 // 2 if act else n2
    if act not in ACT or (act and n2 % 2):
        raise ValueError("act=%r with %d rows of codes" % (act, n2))
    if groups < 1 or K % groups:
        raise ValueError("%d inputs in %d groups" % (K, groups))
    R = rows.shape[0] if rows is not None else y.shape[0] if y is not None else x.shape[0]
    dev = _same_device(x, codes, scales, mins, y, bounds, rows)
    px, ldx = _matrix("x", x, (x.shape[0], K))
    pr, div = _gather(x, rows, div, R)
    if y is None:
        y = _new((R, N), x.dtype, dev, stream)
    py, ldy = _matrix("y", y, (R, N))
    _enqueue(_lib.bitsmoe_w4_matmul, dev, stream, _dtype(x), px, ldx, x.shape[0], pr, div,
             _array("codes", codes, torch.uint8),
             _array("scales", scales, torch.float16, (E, n2, groups)),
             None if mins is None else _array("mins", mins, torch.float16, (E, n2, groups)),
             K // groups, None if bounds is None else _bounds(bounds, E), R, E, N, K, ACT[act], py,
             _dtype(y), ldy)
    return y
