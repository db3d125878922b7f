"""Python binding of libbsr: the C-ABI entry points under the same names.

Argument marshalling only -- every step runs in the HIP kernels of libbsr.so.
Tensors must be CUDA (HIP) tensors; their data pointers, sizes derived from
their shapes, and a stream (default: torch's current stream on the tensors'
device) are passed straight through.  A non-zero status raises ``BsrError``.
There is no fallback: if libbsr.so is missing, the first call raises.
"""
import contextlib
import ctypes
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libbsr.so")

BSR_OK, BSR_EINVAL, BSR_ENULL, BSR_EALIGN, BSR_EDEVICE, BSR_ELAUNCH = range(6)
PATH_AUTO, PATH_GEMM, PATH_GEMV, PATH_INVARIANT = 0, 1, 2, 3
GEMV_MAX_ROWS = 16          # any K
GEMV_STREAM_MAX_ROWS = 64   # K a multiple of 256

# Exported symbols and their C signatures (kept in step with include/bsr.h).
_vp, _u32, _f32, _int = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_float, ctypes.c_int
SIGNATURES = {
    "requant_w_nvfp4_int8": (_int, [_vp, _vp, _f32, _vp, _vp, _u32, _u32, _vp]),
    "requant_a_int8": (_int, [_vp, _vp, _vp, _u32, _u32, _vp]),
    "int8_gemm_blockscaled": (_int, [_vp, _vp, _vp, _vp, _vp, _u32, _u32, _u32, _vp]),
    "int8_gemm_blockscaled_ex": (_int, [_vp, _vp, _vp, _vp, _vp, _u32, _u32, _u32, _vp, _int]),
    "silu_mul_requant_int8": (_int, [_vp, _vp, _u32, _vp, _vp, _u32, _u32, _vp]),
    "w4a16_gemv": (_int, [_vp, _vp, _vp, _f32, _vp, _u32, _u32, _u32, _vp]),
    "quantize_act": (_int, [_vp, _vp, _vp, _u32, _u32, _u32, _int, _vp]),
    "int8_gemm_blockscaled_agroup": (_int, [_vp, _vp, _vp, _u32, _vp, _vp, _u32, _u32, _u32, _vp, _int]),
    "int8_gemm_blockscaled_ws_bytes": (ctypes.c_uint64, [_u32, _u32, _u32]),
    "int8_gemm_blockscaled_ws": (_int, [_vp, _vp, _vp, _vp, _vp, _u32, _u32, _u32, _vp, ctypes.c_uint64, _vp]),
    "int8_gemm_blockscaled_noalloc": (_int, [_vp, _vp, _vp, _vp, _vp, _u32, _u32, _u32, _vp]),
    "moe_route_ws_bytes": (ctypes.c_uint64, [_u32, _u32, _u32]),
    "moe_route": (_int, [_vp, _int, _u32, _vp, _vp, _vp, _vp, _vp, _u32, _u32, _u32, _int, _int, _f32, _vp,
                         ctypes.c_uint64, _vp]),
    "int8_grouped_gemm_blockscaled": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _u32, _u32, _u32, _u32, _u32, _vp]),
    "moe_combine": (_int, [_vp, _vp, _vp, _vp, _vp, _u32, _u32, _u32, _u32, _vp]),
    "w4a16_group_gemv": (_int, [_vp, _vp, _vp, _int, _vp, _u32, _vp, _u32, _u32, _u32, _vp]),
    "w4a16_group_gemv_experts": (_int, [_vp, _vp, _vp, _int, _vp, _u32, _vp, _vp, _int, _vp, _u32, _u32, _u32, _u32,
                                        _u32, _vp]),
    "bsr_status_string": (ctypes.c_char_p, [_int]),
}

_LIB = None


class BsrError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


def lib():
    """The loaded libbsr.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -c 'import __graft_entry__ as g; "
                               f"g.build()'` or `python block_scaled_precision_requant_amd/build.py`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def status_string(status: int) -> str:
    return lib().bsr_status_string(int(status)).decode()


def _ptr(t):
    # runs after every argument's shape and element checks
    if t is None:
        return ctypes.c_void_p(0)
    if not t.is_cuda:
        raise ValueError("arguments must be device tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream, like):
    if stream is None:
        stream = torch.cuda.current_stream(like.device)
    return ctypes.c_void_p(stream.cuda_stream)


# Element kinds the kernels read and write: byte codes (int8, packed E2M1,
# E4M3), 16-bit BF16 bits (any 2-byte dtype: torch.bfloat16, int16, uint16; the
# calls that read float16 as such refuse it there) and binary32 scales.
BYTES, BF16, F32, I32 = "1-byte", "2-byte", "float32", "int32"
_USUAL = {BYTES: {torch.int8, torch.uint8}, BF16: {torch.bfloat16, torch.int16}, F32: {torch.float32},
          I32: {torch.int32}}  # what _kind need not look at


def _shape(t, shape, what, kind):
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    if t.dtype not in _USUAL[kind]:
        _kind(t, what, kind)


def _kind(t, what, kind):
    ok = (t.dtype == (torch.float32 if kind == F32 else torch.int32) if kind in (F32, I32) else
          t.element_size() == (1 if kind == BYTES else 2) and not t.dtype.is_complex)
    if not ok:
        raise ValueError(f"{what}: dtype {t.dtype}, expected {kind} elements")


def _done(status, what):
    if status != BSR_OK:
        raise BsrError(status, what)


def requant_w_nvfp4_int8(w_packed, w_e4m3, scale2, w_i8, w_scale, stream=None):
    """NVFP4 weight (w_packed [N,K/2] u8, w_e4m3 [N,K/16] u8, scale2 float) ->
    w_i8 [N,K] int8 and w_scale [N,K/32] float32 (both preallocated)."""
    n, half_k = w_packed.shape
    k = 2 * half_k
    _shape(w_packed, (n, k // 2), "w_packed", BYTES)
    _shape(w_e4m3, (n, k // 16), "w_e4m3", BYTES)
    _shape(w_i8, (n, k), "w_i8", BYTES)
    _shape(w_scale, (n, k // 32), "w_scale", F32)
    st = lib().requant_w_nvfp4_int8(_ptr(w_packed), _ptr(w_e4m3), float(scale2), _ptr(w_i8),
                                    _ptr(w_scale), n, k, _stream(stream, w_i8))
    _done(st, "requant_w_nvfp4_int8")


def requant_a_int8(a_bf16, a_i8, a_scale, stream=None):
    """BF16 activations a_bf16 [M,K] -> a_i8 [M,K] int8 and a_scale [M,K/32] float32."""
    m, k = a_bf16.shape
    _shape(a_bf16, (m, k), "a_bf16", BF16)
    _shape(a_i8, (m, k), "a_i8", BYTES)
    _shape(a_scale, (m, k // 32), "a_scale", F32)
    st = lib().requant_a_int8(_ptr(a_bf16), _ptr(a_i8), _ptr(a_scale), m, k, _stream(stream, a_i8))
    _done(st, "requant_a_int8")


def silu_mul_requant_int8(gate, up, a_i8, a_scale, stream=None):
    """SiLU(gate) * up -> a_i8 [M,K] int8 and a_scale [M,K/32] float32.

    gate and up are [M,K] BF16 (raw 16-bit) views with unit column stride and
    the same row stride (for instance the two halves of one [M, 2K] buffer)."""
    m, k = gate.shape
    if tuple(up.shape) != (m, k):
        raise ValueError(f"up: shape {tuple(up.shape)}, expected {(m, k)}")
    for t, what in ((gate, "gate"), (up, "up")):
        _kind(t, what, BF16)
        if (m > 1 and t.stride(1) != 1) or (m > 1 and t.stride(0) != gate.stride(0)):
            raise ValueError(f"{what}: 16-bit rows with unit column stride and the gate's row stride")
    ld = gate.stride(0) if m > 1 else k
    _shape(a_i8, (m, k), "a_i8", BYTES)
    _shape(a_scale, (m, k // 32), "a_scale", F32)
    st = lib().silu_mul_requant_int8(_ptr(gate), _ptr(up), ld, _ptr(a_i8), _ptr(a_scale), m, k,
                                     _stream(stream, a_i8))
    _done(st, "silu_mul_requant_int8")


def w4a16_gemv(x_bf16, w_packed, w_e4m3, scale2, out, stream=None):
    """out [M,N] BF16 = x_bf16 [M,K] (M <= 16) times the NVFP4 weight (w_packed [N,K/2] u8,
    w_e4m3 [N,K/16] u8, scale2), dequantized on the fly."""
    m, k = x_bf16.shape
    n = w_packed.shape[0]
    _shape(x_bf16, (m, k), "x_bf16", BF16)
    _shape(w_packed, (n, k // 2), "w_packed", BYTES)
    _shape(w_e4m3, (n, k // 16), "w_e4m3", BYTES)
    _shape(out, (m, n), "out", BF16)
    st = lib().w4a16_gemv(_ptr(x_bf16), _ptr(w_packed), _ptr(w_e4m3), float(scale2), _ptr(out), m, n, k,
                          _stream(stream, out))
    _done(st, "w4a16_gemv")


def int8_gemm_blockscaled_ex(a_i8, w_i8, a_scale, w_scale, out, path=PATH_AUTO, stream=None):
    """out [M,N] BF16 = block-scaled int8 GEMM of a_i8 [M,K] and w_i8 [N,K]."""
    m, k = a_i8.shape
    n = w_i8.shape[0]
    _shape(a_i8, (m, k), "a_i8", BYTES)
    _shape(w_i8, (n, k), "w_i8", BYTES)
    _shape(a_scale, (m, k // 32), "a_scale", F32)
    _shape(w_scale, (n, k // 32), "w_scale", F32)
    _shape(out, (m, n), "out", BF16)
    st = lib().int8_gemm_blockscaled_ex(_ptr(a_i8), _ptr(w_i8), _ptr(a_scale), _ptr(w_scale), _ptr(out),
                                        m, n, k, _stream(stream, out), int(path))
    _done(st, "int8_gemm_blockscaled_ex")


def int8_gemm_blockscaled(a_i8, w_i8, a_scale, w_scale, out, stream=None):
    """As int8_gemm_blockscaled_ex with the automatic path (the GEMV for M <= 16, and for
    M <= 48 when K % 256 == 0 and N <= 4096; else the GEMM)."""
    m, k = a_i8.shape
    n = w_i8.shape[0]
    _shape(a_i8, (m, k), "a_i8", BYTES)
    _shape(w_i8, (n, k), "w_i8", BYTES)
    _shape(a_scale, (m, k // 32), "a_scale", F32)
    _shape(w_scale, (n, k // 32), "w_scale", F32)
    _shape(out, (m, n), "out", BF16)
    st = lib().int8_gemm_blockscaled(_ptr(a_i8), _ptr(w_i8), _ptr(a_scale), _ptr(w_scale), _ptr(out),
                                     m, n, k, _stream(stream, out))
    _done(st, "int8_gemm_blockscaled")


def int8_gemm_blockscaled_ws_bytes(m, n, k):
    """Workspace bytes int8_gemm_blockscaled_ws needs for (m, n, k); 0 if it runs without a K split."""
    return int(lib().int8_gemm_blockscaled_ws_bytes(int(m), int(n), int(k)))


def int8_gemm_blockscaled_ws(a_i8, w_i8, a_scale, w_scale, out, workspace, stream=None):
    """int8_gemm_blockscaled with a caller workspace (a 16-byte aligned device
    tensor of at least int8_gemm_blockscaled_ws_bytes(M, N, K) bytes, or None when
    that is 0), which lets small grids split K across workgroups."""
    m, k = a_i8.shape
    n = w_i8.shape[0]
    _shape(a_i8, (m, k), "a_i8", BYTES)
    _shape(w_i8, (n, k), "w_i8", BYTES)
    _shape(a_scale, (m, k // 32), "a_scale", F32)
    _shape(w_scale, (n, k // 32), "w_scale", F32)
    _shape(out, (m, n), "out", BF16)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().int8_gemm_blockscaled_ws(_ptr(a_i8), _ptr(w_i8), _ptr(a_scale), _ptr(w_scale), _ptr(out), m, n, k,
                                        _ptr(workspace), ws_bytes, _stream(stream, out))
    _done(st, "int8_gemm_blockscaled_ws")


def int8_gemm_blockscaled_noalloc(a_i8, w_i8, a_scale, w_scale, out, stream=None):
    """int8_gemm_blockscaled_ws with the library's static per-GPU scratch as the
    workspace: allocates nothing; calls that overlap in time on one GPU race."""
    m, k = a_i8.shape
    n = w_i8.shape[0]
    _shape(a_i8, (m, k), "a_i8", BYTES)
    _shape(w_i8, (n, k), "w_i8", BYTES)
    _shape(a_scale, (m, k // 32), "a_scale", F32)
    _shape(w_scale, (n, k // 32), "w_scale", F32)
    _shape(out, (m, n), "out", BF16)
    st = lib().int8_gemm_blockscaled_noalloc(_ptr(a_i8), _ptr(w_i8), _ptr(a_scale), _ptr(w_scale), _ptr(out),
                                             m, n, k, _stream(stream, out))
    _done(st, "int8_gemm_blockscaled_noalloc")


FMT_INT8, FMT_E4M3 = 0, 1


def _scale_cols(k, group):
    return 1 if group == 0 else k // group


def quantize_act(a_bf16, q, scale, group=32, fmt=FMT_INT8, stream=None):
    """BF16 a_bf16 [M,K] -> codes q [M,K] (uint8: int8 or E4M3 bits) and float32
    scales [M, K/group] (group 32 or 128) or [M, 1] (group 0: one per row)."""
    m, k = a_bf16.shape
    _shape(a_bf16, (m, k), "a_bf16", BF16)
    _shape(q, (m, k), "q", BYTES)
    _shape(scale, (m, _scale_cols(k, group)), "scale", F32)
    st = lib().quantize_act(_ptr(a_bf16), _ptr(q), _ptr(scale), m, k, int(group), int(fmt), _stream(stream, q))
    _done(st, "quantize_act")


def int8_gemm_blockscaled_agroup(a_i8, w_i8, a_scale, a_group, w_scale, out, path=PATH_AUTO, stream=None):
    """int8_gemm_blockscaled_ex with activation scales a_scale [M, K/a_group]
    (a_group 32 or 128) or [M, 1] (a_group 0: one per row)."""
    m, k = a_i8.shape
    n = w_i8.shape[0]
    _shape(a_i8, (m, k), "a_i8", BYTES)
    _shape(w_i8, (n, k), "w_i8", BYTES)
    _shape(a_scale, (m, _scale_cols(k, a_group)), "a_scale", F32)
    _shape(w_scale, (n, k // 32), "w_scale", F32)
    _shape(out, (m, n), "out", BF16)
    st = lib().int8_gemm_blockscaled_agroup(_ptr(a_i8), _ptr(w_i8), _ptr(a_scale), int(a_group), _ptr(w_scale),
                                            _ptr(out), m, n, k, _stream(stream, out), int(path))
    _done(st, "int8_gemm_blockscaled_agroup")


def prefill(a_bf16, w_i8, w_scale, a_i8_scratch, a_scale_scratch, out, stream=None):
    """The two-launch projection: requant_a_int8 then int8_gemm_blockscaled on one stream."""
    requant_a_int8(a_bf16, a_i8_scratch, a_scale_scratch, stream=stream)
    int8_gemm_blockscaled(a_i8_scratch, w_i8, a_scale_scratch, w_scale, out, stream=stream)


# ---- expert layers and integer 4-bit weights --------------------------------

SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
TYPE_BF16, TYPE_F16, TYPE_F32 = 0, 1, 2


_TYPES = {torch.float32: TYPE_F32, torch.float16: TYPE_F16, torch.bfloat16: TYPE_BF16}


def _type(t, what):
    """Element type of an argument that takes three: float32, float16, or BF16 (any
    other 2-byte dtype, as raw bits)."""
    kind = _TYPES.get(t.dtype)
    if kind is None:
        _kind(t, what, BF16)
        kind = TYPE_BF16
    return kind


# Small decode calls last as long as the host takes to issue them, so the calls
# below look at each tensor once and take the short ways: integers for devices
# and pointers.

# (a build of torch without devices has neither; no call reaches them there)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _arg(t, shape, kind, what, dev):
    """Data pointer of a contiguous tensor of this shape and element kind on device `dev`."""
    if t.shape != shape or t.dtype not in _USUAL[kind] or not t.is_contiguous() or t.get_device() != dev:
        _shape(t, shape, what, kind)
        if kind == BF16 and t.dtype == torch.float16:  # a type that other arguments of these calls are read as
            raise ValueError(f"{what}: dtype torch.float16, expected BF16 elements (torch.bfloat16, or raw bits)")
        _same_device(t, what, dev)
    return t.data_ptr()


def _fit(bits):
    """Refuses sizes and strides, or-ed together, that the ABI's 32-bit arguments would cut."""
    if bits >> 32:
        raise ValueError("sizes and strides must fit 32 bits")


def _same_device(t, what, dev):
    if t.get_device() != dev:
        raise ValueError(f"{what}: on {t.device}, the other arguments on "
                         f"{'the CPU' if dev < 0 else f'cuda:{dev}'}: all must be on one device")


def _on(dev):
    """A context in which `dev` is the current device."""
    return contextlib.nullcontext() if dev < 0 or _current_device() == dev else torch.cuda.device(dev)


def _launch(name, dev, stream, *args):
    """Calls an entry point with `args` and a stream (default: torch's current one on device `dev`), `dev` being
    the current device during the call."""
    if dev < 0:
        raise ValueError("arguments must be device tensors")
    fn = getattr(_LIB or lib(), name)
    raw = _current_stream(dev) if stream is None else stream.cuda_stream
    if _current_device() == dev:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    if status != BSR_OK:
        raise BsrError(status, name)


def moe_route_ws_bytes(tokens, experts, top_k):
    """Workspace bytes moe_route needs; 0 for few tokens, at most 1024 * experts."""
    _fit(int(tokens) | int(experts) | int(top_k))
    return int(lib().moe_route_ws_bytes(int(tokens), int(experts), int(top_k)))


def moe_route(logits, ids, weights, offsets, row_token, pos, workspace=None, score=SCORE_SOFTMAX, renorm=True,
              scale=1.0, stream=None):
    """Router: logits [T,E] (BF16, float16 or float32; rows may be strided) -> ids [T,k] int32, weights [T,k]
    float32, and the routed rows in expert order: offsets [E+1], row_token [T*k], pos [T,k] (all int32).
    workspace: a device tensor of at least moe_route_ws_bytes(T, E, k) bytes, or None when that is 0."""
    t, e = logits.shape
    if ids.dim() != 2:
        raise ValueError(f"ids: shape {tuple(ids.shape)}, expected two dimensions")
    k = ids.shape[1]
    kind = _type(logits, "logits")
    if (e > 1 and logits.stride(1) != 1) or (t > 1 and logits.stride(0) < e):
        raise ValueError("logits: rows with unit column stride that do not overlap")
    ld = logits.stride(0) if t > 1 else e
    _fit(t | e | k | ld)
    dev = logits.get_device()
    ptrs = (_arg(ids, (t, k), I32, "ids", dev), _arg(weights, (t, k), F32, "weights", dev),
            _arg(offsets, (e + 1,), I32, "offsets", dev), _arg(row_token, (t * k,), I32, "row_token", dev),
            _arg(pos, (t, k), I32, "pos", dev))
    ws, ws_bytes = None, 0
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace: must be contiguous")
        _same_device(workspace, "workspace", dev)
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _launch("moe_route", dev, stream, logits.data_ptr(), kind, ld, *ptrs, t, e, k, score,
            1 if renorm else 0, scale, ws, ws_bytes)


def _rows_args(offsets, row_index, out, cols, experts, dev):
    """Pointers of (offsets, row_index or NULL, out) of a grouped call, and its row capacity."""
    rows = out.shape[0]
    return (_arg(offsets, (experts + 1,), I32, "offsets", dev),
            None if row_index is None else _arg(row_index, (rows,), I32, "row_index", dev),
            _arg(out, (rows, cols), BF16, "out", dev), rows)


def int8_grouped_gemm_blockscaled(a_i8, w_i8, a_scale, w_scale, offsets, out, row_index=None, stream=None):
    """Products grouped by expert: out[p] (BF16, rows offsets[e]..offsets[e+1]-1) = row row_index[p] (p without it)
    of a_i8 [A,K] / a_scale [A,K/32] times the weight w_i8 [E,N,K] / w_scale [E,N,K/32] of expert e."""
    a_rows, k = a_i8.shape
    e, n, _ = w_i8.shape
    _fit(a_rows | out.shape[0] | e | n | k)
    dev = a_i8.get_device()
    a, w = _arg(a_i8, (a_rows, k), BYTES, "a_i8", dev), _arg(w_i8, (e, n, k), BYTES, "w_i8", dev)
    a_s = _arg(a_scale, (a_rows, k // 32), F32, "a_scale", dev)
    w_s = _arg(w_scale, (e, n, k // 32), F32, "w_scale", dev)
    off, index, o, rows = _rows_args(offsets, row_index, out, n, e, dev)
    _launch("int8_grouped_gemm_blockscaled", dev, stream, a, w, a_s, w_s, off, index, o, a_rows, rows, e, n, k)


def moe_combine(y, pos, weights, out, residual=None, stream=None):
    """out [T,N] BF16 = residual + sum over the slots s of weights[t,s] * y[pos[t,s]] (y [R,N] BF16; a pos outside
    0..R-1 adds nothing)."""
    rows, n = y.shape
    t, k = pos.shape
    _fit(t | k | rows | n)
    dev = y.get_device()
    _launch("moe_combine", dev, stream, _arg(y, (rows, n), BF16, "y", dev), _arg(pos, (t, k), I32, "pos", dev),
            _arg(weights, (t, k), F32, "weights", dev),
            None if residual is None else _arg(residual, (t, n), BF16, "residual", dev),
            _arg(out, (t, n), BF16, "out", dev), t, k, rows, n)


def _w4_args(x, w_packed, scale, zero, lead, dev):
    """Pointers of (x, w_packed, scale), the scale type, the pointer of zero, the group, and (m, n, k), of a 4-bit
    weight w_packed [*lead, K/2] (lead: N, or E and N) for x [M, K]."""
    m, k = x_shape = x.shape
    groups = scale.shape
    n, cols = lead[-1], groups[-1]
    if cols == 0 or k % cols:
        raise ValueError(f"scale: {cols} groups do not divide K = {k}")
    _fit(m | lead[0] | n | k)
    kind, shape = _type(scale, "scale"), (*lead, cols)
    if groups != shape or not scale.is_contiguous():
        raise ValueError(f"scale: shape {tuple(groups)}, expected contiguous {shape}")
    if scale.get_device() != dev:
        _same_device(scale, "scale", dev)
    if zero is not None and zero.dtype != torch.uint8:  # numbers, not raw bytes: -1 would be read as 255
        raise ValueError(f"zero: dtype {zero.dtype}, expected torch.uint8")
    return (_arg(x, x_shape, BF16, "x_bf16", dev), _arg(w_packed, (*lead, k // 2), BYTES, "w_packed", dev),
            scale.data_ptr(), kind, None if zero is None else _arg(zero, shape, BYTES, "zero", dev),
            0 if cols == 1 else k // cols), m, n, k


def w4a16_group_gemv(x_bf16, w_packed, scale, out, zero=None, stream=None):
    """out [M,N] BF16 = x_bf16 [M,K] times the 4-bit weight scale * (code - zero): w_packed [N,K/2] (low nibble
    first), scale [N,K/group] (BF16, float16 or float32; one column: one scale per row), zero [N,K/group] uint8 or
    None (8 throughout)."""
    if w_packed.dim() != 2:
        raise ValueError(f"w_packed: shape {tuple(w_packed.shape)}, expected two dimensions")
    dev, (n, _) = x_bf16.get_device(), w_packed.shape
    ptrs, m, n, k = _w4_args(x_bf16, w_packed, scale, zero, (n,), dev)
    _launch("w4a16_group_gemv", dev, stream, *ptrs, _arg(out, (m, n), BF16, "out", dev), m, n, k)


def w4a16_group_gemv_experts(x_bf16, w_packed, scale, offsets, out, zero=None, row_index=None, silu_mul=False,
                             stream=None):
    """w4a16_group_gemv by expert (w_packed [E,N,K/2], scale and zero [E,N,K/group]); offsets and row_index as
    int8_grouped_gemm_blockscaled.  silu_mul: the first N/2 columns are gates, the others ups, and out [R,N/2] is
    SiLU(gate) * up."""
    dev = x_bf16.get_device()
    if w_packed.dim() != 3:
        raise ValueError(f"w_packed: shape {tuple(w_packed.shape)}, expected three dimensions")
    e, n, _ = w_packed.shape
    ptrs, m, n, k = _w4_args(x_bf16, w_packed, scale, zero, (e, n), dev)
    _fit(out.shape[0])
    off, index, o, rows = _rows_args(offsets, row_index, out, n // 2 if silu_mul else n, e, dev)
    _launch("w4a16_group_gemv_experts", dev, stream, *ptrs, off, index, 1 if silu_mul else 0, o, m, rows,
            e, n, k)


class MoeScratch:
    """What the launches of moe_prefill and moe_decode_w4 pass between them, for up to `tokens` tokens of width
    `hidden`, `experts` experts of which a token takes `top_k`, and expert projections of width `inter`.  Calls that
    may overlap in time need one each.  It holds the buffers of both calls."""

    def __init__(self, tokens, experts, top_k, hidden, inter, device="cuda"):
        def buf(*shape, dtype):
            return torch.zeros(shape, dtype=dtype, device=device)
        rows = tokens * top_k
        i32, f32, i8, bf16 = torch.int32, torch.float32, torch.int8, torch.bfloat16
        self.tokens, self.top_k = tokens, top_k
        self.ids, self.pos = buf(tokens, top_k, dtype=i32), buf(tokens, top_k, dtype=i32)
        self.weights = buf(tokens, top_k, dtype=f32)
        self.offsets, self.row_token = buf(experts + 1, dtype=i32), buf(rows, dtype=i32)
        self.workspace = buf(1024 * experts, dtype=torch.uint8)
        self.a_i8, self.a_scale = buf(tokens, hidden, dtype=i8), buf(tokens, hidden // 32, dtype=f32)
        self.gate_up = buf(rows, 2 * inter, dtype=bf16)
        self.h_i8, self.h_scale = buf(rows, inter, dtype=i8), buf(rows, inter // 32, dtype=f32)
        self.h, self.y = buf(rows, inter, dtype=bf16), buf(rows, hidden, dtype=bf16)

    def route(self, logits, **how):
        """moe_route of len(logits) tokens into these buffers; returns the row capacity, len(logits) * top_k."""
        t = logits.shape[0]
        if t > self.tokens:
            raise ValueError(f"{t} tokens, scratch for {self.tokens}")
        rows = t * self.top_k
        moe_route(logits, self.ids[:t], self.weights[:t], self.offsets, self.row_token[:rows], self.pos[:t],
                  self.workspace, **how)
        return rows


def _layer_tokens(x_bf16, logits, out, residual):
    """Token count of a layer call, whose token tensors are checked before its first launch."""
    t = x_bf16.shape[0]
    if logits.shape[0] != t:  # the rows come from the logits, what they are made of from x_bf16
        raise ValueError(f"logits: {logits.shape[0]} tokens, x_bf16 {t}")
    dev = x_bf16.get_device()
    _same_device(logits, "logits", dev)
    for v, what in ((x_bf16, "x_bf16"), (out, "out"), (residual, "residual")):
        if v is not None:
            _arg(v, x_bf16.shape, BF16, what, dev)
    return t


def moe_prefill(x_bf16, logits, w_gate_up, gate_up_scale, w_down, down_scale, out, scratch, residual=None,
                score=SCORE_SOFTMAX, renorm=True, scale=1.0, stream=None):
    """One expert layer on int8 per-32 weights (requant_w_nvfp4_int8 of each expert): x_bf16 [T,H], router logits
    [T,E], w_gate_up [E,2I,H] (gate rows first), w_down [E,H,I] with their scales -> out [T,H] (+ residual), in six
    steps on one stream: router, activation requant, grouped gate and up, SiLU product requant, grouped down,
    weighted sum."""
    t, inter = _layer_tokens(x_bf16, logits, out, residual), w_down.shape[2]
    s = scratch
    rows = s.route(logits, score=score, renorm=renorm, scale=scale, stream=stream)
    a_i8, a_scale, gate_up, y = s.a_i8[:t], s.a_scale[:t], s.gate_up[:rows], s.y[:rows]
    dev = x_bf16.get_device()
    with _on(dev):  # (the two requants run on the current device)
        requant_a_int8(x_bf16, a_i8, a_scale, stream=stream)
    int8_grouped_gemm_blockscaled(a_i8, w_gate_up, a_scale, gate_up_scale, s.offsets, gate_up,
                                  row_index=s.row_token[:rows], stream=stream)
    with _on(dev):
        silu_mul_requant_int8(gate_up[:, :inter], gate_up[:, inter:], s.h_i8[:rows], s.h_scale[:rows], stream=stream)
    int8_grouped_gemm_blockscaled(s.h_i8[:rows], w_down, s.h_scale[:rows], down_scale, s.offsets, y, stream=stream)
    moe_combine(y, s.pos[:t], s.weights[:t], out, residual=residual, stream=stream)


def moe_decode_w4(x_bf16, logits, w_gate_up, gate_up_scale, gate_up_zero, w_down, down_scale, down_zero, out, scratch,
                  residual=None, score=SCORE_SOFTMAX, renorm=True, scale=1.0, stream=None):
    """One expert layer on 4-bit weights with group scales, for a few tokens: as moe_prefill, with w_gate_up
    [E,2I,H/2] and w_down [E,H,I/2] packed, their scales and zero points (or None), in four steps: router, gate and up
    with the SiLU product, down, weighted sum."""
    t = _layer_tokens(x_bf16, logits, out, residual)
    s = scratch
    rows = s.route(logits, score=score, renorm=renorm, scale=scale, stream=stream)
    h, y = s.h[:rows], s.y[:rows]
    w4a16_group_gemv_experts(x_bf16, w_gate_up, gate_up_scale, s.offsets, h, zero=gate_up_zero,
                             row_index=s.row_token[:rows], silu_mul=True, stream=stream)
    w4a16_group_gemv_experts(h, w_down, down_scale, s.offsets, y, zero=down_zero, stream=stream)
    moe_combine(y, s.pos[:t], s.weights[:t], out, residual=residual, stream=stream)
