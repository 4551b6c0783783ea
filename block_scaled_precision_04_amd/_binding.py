"""Thin ctypes binding over libbsgemm.so (include/bsgemm.h).

Argument marshalling only: torch tensors become device pointers and the
current HIP stream; every step of the computation runs in the library's HIP
kernels.  Outputs that are not passed in are allocated with torch (device
memory plumbing).  A negative status from the library raises BsError.  If the
library is not built, importing the functions fails loudly: there is no
fallback path.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbsgemm.so")

BS_OP_FP8_BLOCK = 1
BS_OP_W4A8_MXFP4 = 2
BS_OP_BF16_SKINNY = 3
BS_OP_W4A4_MXFP4 = 4
BS_OP_MOE_SORT = 5
BS_LAYOUT_FP8_BLOCK = 0x38423631
BS_LAYOUT_MXFP4 = 0x34584D31
BS_WDESC_MAGIC = 0x42534744


class BsError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: {lib().bs_status_string(status).decode()} (status {status})")


class WDesc(ctypes.Structure):
    """Host-side weight descriptor (bs_wdesc)."""
    _fields_ = [("magic", ctypes.c_uint32), ("layout", ctypes.c_uint32), ("N", ctypes.c_int32),
                ("K", ctypes.c_int32), ("codes_bytes", ctypes.c_uint64), ("scales_offset", ctypes.c_uint64),
                ("scales_bytes", ctypes.c_uint64), ("total_bytes", ctypes.c_uint64)]


_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_Z = ctypes.c_size_t
_F = ctypes.c_float
_D = ctypes.POINTER(WDesc)
_FP = ctypes.POINTER(ctypes.c_float)

SIGNATURES = {
    "bs_status_string": (ctypes.c_char_p, [_I]),
    "bs_version": (_I, []),
    "bs_prelayout_fp8_block_bytes": (_Z, [_I, _I]),
    "bs_prelayout_fp8_block": (_I, [_P, _P, _Z, _I, _I, _D, _P]),
    "bs_unprelayout_fp8_block": (_I, [_D, _P, _P, _P]),
    "bs_prelayout_mxfp4_bytes": (_Z, [_I, _I]),
    "bs_prelayout_mxfp4": (_I, [_P, _P, _P, _Z, _I, _I, _D, _P]),
    "bs_unprelayout_mxfp4": (_I, [_D, _P, _P, _P, _P]),
    "bs_workspace_bytes": (_Z, [_I, _I, _I, _I]),
    "bsgemm_fp8_block": (_I, [_P, _L, _P, _L, _L, _D, _P, _P, _P, _L, _I, _I, _I, _P, _Z, _P]),
    "bsgemm_w4a8_mxfp4": (_I, [_P, _L, _P, _D, _P, _P, _L, _I, _I, _I, _P, _Z, _P]),
    "bsgemm_w4a8_mxfp4_atiled": (_I, [_P, _P, _D, _P, _P, _L, _I, _I, _I, _P, _Z, _P]),
    "gemm_bf16_skinny": (_I, [_P, _P, _P, _I, _I, _I, _P, _Z, _P]),
    "gemm_bf16_skinny_noalloc": (_I, [_P, _P, _P, _I, _I, _I, _P]),
    "add_rms_quant_fp8": (_I, [_P, _P, _P, _F, _P, _P, _P, _I, _I, _P]),
    "add_rms_quant_fp8_group128": (_I, [_P, _P, _P, _F, _P, _P, _P, _I, _I, _P]),
    "add_rms_quant_fp8_tiled": (_I, [_P, _P, _P, _F, _P, _P, _P, _I, _I, _P]),
    "silu_mul_quant_fp8": (_I, [_P, _P, _P, _I, _I, _P]),
    "quant_fp8_per_token": (_I, [_P, _P, _P, _I, _I, _P]),
    "quant_fp8_group128": (_I, [_P, _P, _P, _I, _I, _P]),
    "quant_fp8_block128": (_I, [_P, _P, _P, _I, _I, _P]),
    "bsgemm_w4a4_mxfp4": (_I, [_P, _L, _P, _L, _D, _P, _P, _L, _I, _I, _I, _P, _Z, _P]),
    "bsgemm_w4a4_mxfp4_grouped": (_I, [_P, _L, _P, _L, _I, _P, _P, _D, _P, _Z, _P, _L, _I, _I, _I, _I, _P]),
    "quant_mxfp4": (_I, [_P, _L, _P, _P, _I, _I, _P]),
    "silu_mul_quant_mxfp4": (_I, [_P, _P, _P, _P, _I, _I, _P]),
    "dequant_mxfp4": (_I, [_P, _P, _P, _I, _I, _P]),
    "moe_sort": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _Z, _P]),
    "moe_gather": (_I, [_P, _P, _P, _I, _I, _I, _P]),
    "moe_combine": (_I, [_P, _P, _P, _P, _I, _I, _I, _P]),
    "moe_combine_backward": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
}

_LIB = None


def lib():
    """Load libbsgemm.so once and declare every C signature."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run block_scaled_precision_04_amd.build.build() "
                               "(hipcc for gfx950); there is no fallback")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def _check(fn, status):
    if status != 0:
        raise BsError(fn, status)


def _ptr(t):
    return t.data_ptr() if t is not None else None


# The raw handle of a device's current stream; torch's Stream object costs about
# 3 us to build, as much as the whole C call of a small operator.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# torch.cuda.current_device without its check that the GPU is initialised: asked
# only when a tensor lives there
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream():
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def _u8(t):
    return t.view(torch.uint8) if t.dtype != torch.uint8 else t


# ---------------------------------------------------------------- argument checks
# The library sees raw pointers and sizes only, so every tensor's shape, dtype
# and row stride is checked here before the call: a wrong output tensor would
# otherwise be written as if it were a dense [M, N] buffer.
_FP8 = (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8))
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_U8 = (torch.uint8,)
_I32 = (torch.int32,)
_F32 = (torch.float32,)


def _need(cond, fn, msg):
    if not cond:
        raise ValueError(f"{fn}: {msg}")


def _arg(fn, name, t, shape, dtypes, contiguous=False, unit_inner=True, one_row=False):
    """t must have `shape` and one of `dtypes`; its last dimension must be
    unit-stride (rows may be padded) or, with contiguous=True, the tensor dense.
    one_row=True: a single row may have any row stride (the caller passes a dense one on)."""
    # an accepted tensor builds no message: formatting one for every argument
    # took most of a small call's host time
    if not (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape):
        _need(t is not None, fn, f"{name} is required")
        _need(isinstance(t, torch.Tensor), fn, f"{name} must be a torch.Tensor")
        _need(t.dtype in dtypes, fn, f"{name} has dtype {t.dtype}, expected one of {tuple(str(d) for d in dtypes)}")
        _need(tuple(t.shape) == tuple(shape), fn, f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if contiguous:
        if not t.is_contiguous():
            _need(False, fn, f"{name} must be contiguous")
    elif unit_inner and t.dim() >= 2 and t.shape[-1] > 1 and not (one_row and t.is_contiguous()):
        # (is_contiguous() looks at no stride of a dimension of one)
        if t.stride(-1) != 1:
            _need(False, fn, f"{name} must have unit stride along its last dimension")
        if t.stride(0) < t.shape[-1]:
            _need(False, fn, f"{name} rows overlap (stride {t.stride(0)} < {t.shape[-1]})")
    return t


def _on_device(fn, *ts):
    """Every tensor lives on the same GPU (a host tensor would hand the kernels a host address)."""
    first = None
    for t in ts:
        if t is None:
            continue
        if first is None:
            first = t.device
        if t.device != first or first.type != "cuda":
            devs = {u.device for u in ts if u is not None}
            _need(all(d.type == "cuda" for d in devs), fn, f"tensors must be on a GPU, got {sorted(map(str, devs))}")
            _need(False, fn, f"tensors are on different devices: {sorted(map(str, devs))}")
    return first


def _on_current(fn, *ts):
    """Every tensor lives on the current GPU: the launch goes to its current
    stream, whose handle is returned."""
    dev = ts[0].get_device()
    for t in ts:
        if t is not None and (t.get_device() != dev or dev < 0):
            _on_device(fn, *ts)
    cur = _current_device()
    if dev != cur:
        _need(False, fn, f"tensors are on cuda:{dev}, the current device is cuda:{cur}")
    return _raw_stream(cur) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream


def _rows(rows, cols, dtype, device):
    """A fresh dense [rows, cols] tensor (with its strides given, torch takes 0.35 us less)."""
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _row_stride(t):
    """Leading dimension of a [M, C] tensor (with one row any stride is a dense one)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _ws(fn, ws):
    """(pointer, bytes) of an optional workspace tensor (dense, any dtype)."""
    if ws is None:
        return None, 0
    _need(isinstance(ws, torch.Tensor) and ws.is_contiguous(), fn, "ws must be a contiguous tensor")
    return _ptr(ws), ws.numel() * ws.element_size()


def _bits16(t):
    if t.dtype in (torch.bfloat16, torch.int16, torch.uint16):
        return t
    raise TypeError(f"expected bf16 data (bfloat16 or 16-bit bit patterns), got {t.dtype}")


# ------------------------------------------------------------------ layouts
def prelayout_fp8_block(w_e4m3):
    """[N, K] e4m3 codes (uint8 or float8_e4m3fn) -> (pre-laid-out uint8 buffer, WDesc)."""
    w = _u8(w_e4m3).contiguous()
    N, K = w.shape
    nbytes = lib().bs_prelayout_fp8_block_bytes(N, K)
    if nbytes == 0:
        raise BsError("bs_prelayout_fp8_block_bytes", -2)
    out = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
    desc = WDesc()
    _check("bs_prelayout_fp8_block", lib().bs_prelayout_fp8_block(_ptr(w), _ptr(out), nbytes, N, K,
                                                                   ctypes.byref(desc), _stream()))
    return out, desc


def unprelayout_fp8_block(desc, pre):
    w = torch.empty((desc.N, desc.K), dtype=torch.uint8, device=pre.device)
    _check("bs_unprelayout_fp8_block", lib().bs_unprelayout_fp8_block(ctypes.byref(desc), _ptr(pre), _ptr(w),
                                                                       _stream()))
    return w


def prelayout_mxfp4(w_packed, w_e8m0):
    """[N, K/2] packed e2m1 + [N, K/32] e8m0 -> (pre-laid-out uint8 buffer, WDesc)."""
    wp = _u8(w_packed).contiguous()
    e = _u8(w_e8m0).contiguous()
    N, Kh = wp.shape
    K = 2 * Kh
    nbytes = lib().bs_prelayout_mxfp4_bytes(N, K)
    if nbytes == 0:
        raise BsError("bs_prelayout_mxfp4_bytes", -2)
    out = torch.empty(nbytes, dtype=torch.uint8, device=wp.device)
    desc = WDesc()
    _check("bs_prelayout_mxfp4", lib().bs_prelayout_mxfp4(_ptr(wp), _ptr(e), _ptr(out), nbytes, N, K,
                                                           ctypes.byref(desc), _stream()))
    return out, desc


def prelayout_mxfp4_experts(w_packed, w_e8m0):
    """[E, N, K/2] packed e2m1 + [E, N, K/32] e8m0 -> (uint8 [E, total_bytes] with
    every expert's pre-laid-out weight, the WDesc that they share)."""
    fn = "prelayout_mxfp4_experts"
    _need(isinstance(w_packed, torch.Tensor) and w_packed.dim() == 3, fn, "w_packed must be a 3-D tensor [E, N, K/2]")
    E, N, Kh = w_packed.shape
    K = 2 * Kh
    _need(E >= 1, fn, "at least one expert is needed")
    _arg(fn, "w_packed", w_packed, (E, N, Kh), (torch.uint8,), unit_inner=False)
    _arg(fn, "w_e8m0", w_e8m0, (E, N, K // 32), (torch.uint8,), unit_inner=False)
    nbytes = lib().bs_prelayout_mxfp4_bytes(N, K)
    if nbytes == 0:
        raise BsError("bs_prelayout_mxfp4_bytes", -2)
    stream = _on_current(fn, w_packed, w_e8m0)
    out = torch.empty((E, nbytes), dtype=torch.uint8, device=w_packed.device)
    desc = WDesc()
    for e in range(E):
        wp, sc = w_packed[e].contiguous(), w_e8m0[e].contiguous()
        _check(fn, lib().bs_prelayout_mxfp4(_ptr(wp), _ptr(sc), _ptr(out[e]), nbytes, N, K, ctypes.byref(desc),
                                            stream))
    return out, desc


def unprelayout_mxfp4(desc, pre):
    wp = torch.empty((desc.N, desc.K // 2), dtype=torch.uint8, device=pre.device)
    e = torch.empty((desc.N, desc.K // 32), dtype=torch.uint8, device=pre.device)
    _check("bs_unprelayout_mxfp4", lib().bs_unprelayout_mxfp4(ctypes.byref(desc), _ptr(pre), _ptr(wp), _ptr(e),
                                                               _stream()))
    return wp, e


def workspace_bytes(op, M, N, K):
    return int(lib().bs_workspace_bytes(op, M, N, K))


def alloc_workspace(op, M, N, K, device="cuda"):
    """A zero-filled workspace for (op, M, N, K), or None when none is needed.
    Allocate once (outside graph capture) and reuse: the kernels leave it zeroed."""
    n = workspace_bytes(op, M, N, K)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


# ------------------------------------------------------------------ GEMMs
def bsgemm_fp8_block(a, a_scale, desc, w_pre, w_scale, out=None, ws=None):
    """C[M,N] bf16 = block-FP8 GEMM.  a: [M,K] e4m3 (row stride in bytes may be
    padded to a multiple of 16); a_scale: fp32 [M, K/128] with any strides;
    w_scale: fp32 [N/128, K/128] contiguous."""
    fn = "bsgemm_fp8_block"
    _need(isinstance(a, torch.Tensor) and a.dim() == 2, fn, "a must be a 2-D tensor [M, K]")
    M, K = a.shape
    N = desc.N
    _need(desc.K == K, fn, f"a has K = {K}, the weight descriptor K = {desc.K}")
    _arg(fn, "a", a, (M, K), _FP8)
    _arg(fn, "a_scale", a_scale, (M, K // 128), (torch.float32,), unit_inner=False)
    _arg(fn, "w_scale", w_scale, (N // 128, K // 128), (torch.float32,), unit_inner=False)
    _arg(fn, "w_pre", w_pre, (w_pre.numel(),), (torch.uint8,), contiguous=True)
    _need(w_pre.numel() >= desc.total_bytes, fn, f"w_pre holds {w_pre.numel()} bytes, the layout needs "
                                                 f"{desc.total_bytes}")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    _arg(fn, "out", out, (M, N), _BF16)
    _on_device(fn, a, a_scale, w_pre, w_scale, out, ws)
    a8 = _u8(a)
    ws_p, ws_n = _ws(fn, ws)
    _check(fn, lib().bsgemm_fp8_block(
        _ptr(a8), a8.stride(0), _ptr(a_scale), a_scale.stride(0), a_scale.stride(1), ctypes.byref(desc),
        _ptr(w_pre), _ptr(w_scale.contiguous()), _ptr(out), out.stride(0), M, N, K, ws_p, ws_n, _stream()))
    return out


def bsgemm_w4a8_mxfp4(a, a_scale, desc, w_pre, out=None, ws=None):
    """C[M,N] bf16 = MXFP4 W4A8 GEMM.  a: [M,K] e4m3; a_scale: fp32 [M]."""
    fn = "bsgemm_w4a8_mxfp4"
    _need(isinstance(a, torch.Tensor) and a.dim() == 2, fn, "a must be a 2-D tensor [M, K]")
    M, K = a.shape
    N = desc.N
    _need(desc.K == K, fn, f"a has K = {K}, the weight descriptor K = {desc.K}")
    _arg(fn, "a", a, (M, K), _FP8)
    _arg(fn, "a_scale", a_scale, (M,), (torch.float32,), unit_inner=False)
    _arg(fn, "w_pre", w_pre, (w_pre.numel(),), (torch.uint8,), contiguous=True)
    _need(w_pre.numel() >= desc.total_bytes, fn, f"w_pre holds {w_pre.numel()} bytes, the layout needs "
                                                 f"{desc.total_bytes}")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    _arg(fn, "out", out, (M, N), _BF16)
    _on_device(fn, a, a_scale, w_pre, out, ws)
    a8 = _u8(a)
    ws_p, ws_n = _ws(fn, ws)
    _check(fn, lib().bsgemm_w4a8_mxfp4(
        _ptr(a8), a8.stride(0), _ptr(a_scale.contiguous()), ctypes.byref(desc), _ptr(w_pre), _ptr(out),
        out.stride(0), M, N, K, ws_p, ws_n, _stream()))
    return out


def tiled_activation_bytes(M, K):
    """Bytes of an activation-tiled [M, K] e4m3 buffer (rows padded to 32)."""
    return (M + 31) // 32 * 32 * K


def bsgemm_w4a8_mxfp4_atiled(a_tiled, a_scale, desc, w_pre, M, out=None, ws=None):
    """C[M,N] bf16 = MXFP4 W4A8 GEMM on an activation in the activation-tiled
    order (uint8, tiled_activation_bytes(M, K) bytes, from
    add_rms_quant_fp8_tiled); M > 64."""
    fn = "bsgemm_w4a8_mxfp4_atiled"
    N, K = desc.N, desc.K
    _arg(fn, "a_tiled", a_tiled, (tiled_activation_bytes(M, K),), _FP8, contiguous=True)
    _arg(fn, "a_scale", a_scale, (M,), (torch.float32,), unit_inner=False)
    _arg(fn, "w_pre", w_pre, (w_pre.numel(),), (torch.uint8,), contiguous=True)
    _need(w_pre.numel() >= desc.total_bytes, fn, f"w_pre holds {w_pre.numel()} bytes, the layout needs "
                                                 f"{desc.total_bytes}")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a_tiled.device)
    _arg(fn, "out", out, (M, N), _BF16)
    _on_device(fn, a_tiled, a_scale, w_pre, out, ws)
    ws_p, ws_n = _ws(fn, ws)
    _check(fn, lib().bsgemm_w4a8_mxfp4_atiled(
        _ptr(a_tiled), _ptr(a_scale.contiguous()), ctypes.byref(desc), _ptr(w_pre), _ptr(out), out.stride(0),
        M, N, K, ws_p, ws_n, _stream()))
    return out


def _mxfp4_activation(fn, a, a_scale, desc):
    """Checked (a, a_scale, rows, K) of an MXFP4 activation: codes [M, K/2], scales [M, K/32]."""
    _need(isinstance(a, torch.Tensor) and a.dim() == 2, fn, "a must be a 2-D tensor [M, K/2]")
    M, Kh = a.shape
    K = 2 * Kh
    if desc.K != K:
        _need(False, fn, f"a has K = {K}, the weight descriptor K = {desc.K}")
    _arg(fn, "a", a, (M, Kh), _U8, one_row=True)
    _arg(fn, "a_scale", a_scale, (M, K // 32), _U8, one_row=True)
    return M, K


def bsgemm_w4a4_mxfp4(a, a_scale, desc, w_pre, out=None, ws=None):
    """C[M,N] bf16 = MXFP4 W4A4 GEMM.  a: [M, K/2] packed e2m1 (row stride in
    bytes may be padded to a multiple of 16); a_scale: e8m0 [M, K/32] (row
    stride padded to a multiple of 4); ws: alloc_workspace(BS_OP_W4A4_MXFP4, M, N, K)."""
    fn = "bsgemm_w4a4_mxfp4"
    M, K = _mxfp4_activation(fn, a, a_scale, desc)
    N = desc.N
    _need(isinstance(w_pre, torch.Tensor), fn, "w_pre must be a torch.Tensor")
    nw = w_pre.numel()
    _arg(fn, "w_pre", w_pre, (nw,), _U8, contiguous=True)
    if nw < desc.total_bytes:
        _need(False, fn, f"w_pre holds {nw} bytes, the layout needs {desc.total_bytes}")
    if out is None:
        out = _rows(M, N, torch.bfloat16, a.device)
    else:
        _arg(fn, "out", out, (M, N), _BF16, one_row=True)
    stream = _on_current(fn, a, a_scale, w_pre, out, ws)
    ws_p, ws_n = _ws(fn, ws)
    # (with one row any stride is a dense one)
    lda, lds, ldc = (a.stride(0), a_scale.stride(0), out.stride(0)) if M > 1 else (K // 2, K // 32, N)
    _check(fn, lib().bsgemm_w4a4_mxfp4(
        a.data_ptr(), lda, a_scale.data_ptr(), lds, ctypes.byref(desc), w_pre.data_ptr(), out.data_ptr(), ldc, M, N, K,
        ws_p, ws_n, stream))
    return out


def bsgemm_w4a4_mxfp4_grouped(a, a_scale, offsets, desc, w_pre, rows=None, out=None):
    """The experts' W4A4 products over slots sorted by expert (moe_sort):
    out[s] = a[rows[s]] . W_e^T for offsets[e] <= s < offsets[e+1]; bf16 [S, N].
    offsets: int32 [E+1]; rows: int32 [S] (None: slot s is row s of a); desc,
    w_pre: from prelayout_mxfp4_experts.  Rows of out past offsets[E] keep what
    they hold (pass out to choose; a fresh one is not cleared)."""
    fn = "bsgemm_w4a4_mxfp4_grouped"
    Ma, K = _mxfp4_activation(fn, a, a_scale, desc)
    N = desc.N
    _need(isinstance(w_pre, torch.Tensor) and w_pre.dim() == 2, fn, "w_pre must be a 2-D tensor [E, total_bytes]")
    E = w_pre.shape[0]
    _arg(fn, "w_pre", w_pre, (E, w_pre.shape[1]), _U8, one_row=True)
    if w_pre.shape[1] < desc.total_bytes:
        _need(False, fn, f"w_pre holds {w_pre.shape[1]} bytes an expert, the layout needs {desc.total_bytes}")
    _arg(fn, "offsets", offsets, (E + 1,), _I32, contiguous=True)
    S = Ma
    if rows is not None:
        _need(isinstance(rows, torch.Tensor), fn, "rows must be a torch.Tensor")
        S = rows.numel()
        _arg(fn, "rows", rows, (S,), _I32, contiguous=True)
    if out is None:
        out = _rows(S, N, torch.bfloat16, a.device)
    else:
        _arg(fn, "out", out, (S, N), _BF16, one_row=True)
    stream = _on_current(fn, a, a_scale, offsets, w_pre, rows, out)
    _check(fn, lib().bsgemm_w4a4_mxfp4_grouped(
        a.data_ptr(), _row_stride(a), a_scale.data_ptr(), _row_stride(a_scale), Ma, offsets.data_ptr(), _ptr(rows),
        ctypes.byref(desc), w_pre.data_ptr(), _row_stride(w_pre), out.data_ptr(), _row_stride(out), S, E, N, K, stream))
    return out


def gemm_bf16_skinny(x, w, out=None, ws=None):
    """C[M,N] bf16 = x[M,K] . w[N,K]^T (M <= 64).  ws: from alloc_workspace when K is split."""
    fn = "gemm_bf16_skinny"
    _need(isinstance(x, torch.Tensor) and x.dim() == 2 and isinstance(w, torch.Tensor) and w.dim() == 2, fn,
          "x [M, K] and w [N, K] must be 2-D tensors")
    M, K = x.shape
    N = w.shape[0]
    _arg(fn, "x", x, (M, K), _BF16, unit_inner=False)
    _arg(fn, "w", w, (N, K), _BF16, unit_inner=False)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _arg(fn, "out", out, (M, N), _BF16, contiguous=True)    # the C call takes no leading dimension for c
    _on_device(fn, x, w, out, ws)
    x = x.contiguous()
    w = w.contiguous()
    ws_p, ws_n = _ws(fn, ws)
    _check(fn, lib().gemm_bf16_skinny(_ptr(x), _ptr(w), _ptr(out), M, N, K, ws_p, ws_n, _stream()))
    return out


def gemm_bf16_skinny_noalloc(x, w, out=None):
    """gemm_bf16_skinny without a workspace: the library keeps the split-K
    scratch in a static per-GPU array (calls that overlap on one GPU race).
    The C call allocates nothing; pass `out` to allocate nothing here either."""
    fn = "gemm_bf16_skinny_noalloc"
    _need(isinstance(x, torch.Tensor) and x.dim() == 2 and isinstance(w, torch.Tensor) and w.dim() == 2, fn,
          "x [M, K] and w [N, K] must be 2-D tensors")
    M, K = x.shape
    N = w.shape[0]
    _arg(fn, "x", x, (M, K), _BF16, contiguous=True)
    _arg(fn, "w", w, (N, K), _BF16, contiguous=True)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _arg(fn, "out", out, (M, N), _BF16, contiguous=True)
    _on_device(fn, x, w, out)
    _check(fn, lib().gemm_bf16_skinny_noalloc(_ptr(x), _ptr(w), _ptr(out), M, N, K, _stream()))
    return out


# ------------------------------------------------------------------ producers
def _producer_args(fn, y, residual, gamma, q, scale, residual_out, group):
    """Checked (y, residual, gamma, q, scale, residual_out) of the norm
    producers; scale has one value per row (group = 1) or per 128 columns."""
    _need(isinstance(y, torch.Tensor) and y.dim() == 2, fn, "y must be a 2-D tensor [M, K]")
    M, K = y.shape
    dev = y.device
    _arg(fn, "y", y, (M, K), _BF16, unit_inner=False)
    _arg(fn, "residual", residual, (M, K), _BF16, unit_inner=False)
    _arg(fn, "gamma", gamma, (K,), _BF16, unit_inner=False)
    sshape = (M,) if group == 1 else (M, K // 128)
    q = torch.empty((M, K), dtype=torch.uint8, device=dev) if q is None else q
    scale = torch.empty(sshape, dtype=torch.float32, device=dev) if scale is None else scale
    residual_out = torch.empty((M, K), dtype=torch.bfloat16, device=dev) if residual_out is None else residual_out
    _arg(fn, "q", q, (M, K), _FP8, contiguous=True)
    _arg(fn, "scale", scale, sshape, _F32, contiguous=True)
    _arg(fn, "residual_out", residual_out, (M, K), _BF16, contiguous=True)
    _on_device(fn, y, residual, gamma, q, scale, residual_out)
    return y.contiguous(), residual.contiguous(), gamma.contiguous(), q, scale, residual_out


def _quant_args(fn, x, q, scale, qshape, sshape, in_shape=None):
    """Checked (x, q, scale) of the quantizers."""
    _arg(fn, "x", x, in_shape or qshape, _BF16, unit_inner=False)
    q = torch.empty(qshape, dtype=torch.uint8, device=x.device) if q is None else q
    scale = torch.empty(sshape, dtype=torch.float32, device=x.device) if scale is None else scale
    _arg(fn, "q", q, qshape, _FP8, contiguous=True)
    _arg(fn, "scale", scale, sshape, _F32, contiguous=True)
    _on_device(fn, x, q, scale)
    return x.contiguous(), q, scale


def add_rms_quant_fp8(y, residual, gamma, eps=1e-6, q=None, scale=None, residual_out=None):
    """(q e4m3 [M,K] as uint8, scale fp32 [M], residual_out bf16 [M,K])."""
    fn = "add_rms_quant_fp8"
    y, residual, gamma, q, scale, residual_out = _producer_args(fn, y, residual, gamma, q, scale, residual_out, 1)
    M, K = y.shape
    _check(fn, lib().add_rms_quant_fp8(
        _ptr(y), _ptr(residual), _ptr(gamma), ctypes.c_float(eps), _ptr(q), _ptr(scale), _ptr(residual_out),
        M, K, _stream()))
    return q, scale, residual_out


def add_rms_quant_fp8_tiled(y, residual, gamma, eps=1e-6, q=None, scale=None, residual_out=None):
    """(q e4m3 in the activation-tiled order, uint8 [tiled_activation_bytes(M, K)],
    scale fp32 [M], residual_out bf16 [M,K])."""
    fn = "add_rms_quant_fp8_tiled"
    _need(isinstance(y, torch.Tensor) and y.dim() == 2, fn, "y must be a 2-D tensor [M, K]")
    M, K = y.shape
    if q is None:
        q = torch.empty((tiled_activation_bytes(M, K),), dtype=torch.uint8, device=y.device)
    _arg(fn, "q", q, (tiled_activation_bytes(M, K),), _FP8, contiguous=True)
    q2 = q.view(-1)[: M * K].view(M, K)      # shape stand-in for the shared checks only
    y, residual, gamma, _, scale, residual_out = _producer_args(fn, y, residual, gamma, q2, scale, residual_out, 1)
    _check(fn, lib().add_rms_quant_fp8_tiled(
        _ptr(y), _ptr(residual), _ptr(gamma), ctypes.c_float(eps), _ptr(q), _ptr(scale), _ptr(residual_out),
        M, K, _stream()))
    return q, scale, residual_out


def add_rms_quant_fp8_group128(y, residual, gamma, eps=1e-6, q=None, scale=None, residual_out=None):
    """(q e4m3 [M,K] as uint8, scale fp32 [M, K/128], residual_out bf16 [M,K])."""
    fn = "add_rms_quant_fp8_group128"
    y, residual, gamma, q, scale, residual_out = _producer_args(fn, y, residual, gamma, q, scale, residual_out,
                                                                128)
    M, K = y.shape
    _check(fn, lib().add_rms_quant_fp8_group128(
        _ptr(y), _ptr(residual), _ptr(gamma), ctypes.c_float(eps), _ptr(q), _ptr(scale), _ptr(residual_out),
        M, K, _stream()))
    return q, scale, residual_out


def silu_mul_quant_fp8(gu, q=None, scale=None):
    """gu bf16 [M, 2N] (gate half first) -> (q e4m3 [M, N] as uint8, scale fp32 [M])."""
    fn = "silu_mul_quant_fp8"
    _need(isinstance(gu, torch.Tensor) and gu.dim() == 2 and gu.shape[1] % 2 == 0, fn,
          "gu must be a 2-D tensor [M, 2N]")
    M, N2 = gu.shape
    N = N2 // 2
    gu, q, scale = _quant_args(fn, gu, q, scale, (M, N), (M,), in_shape=(M, N2))
    _check(fn, lib().silu_mul_quant_fp8(_ptr(gu), _ptr(q), _ptr(scale), M, N, _stream()))
    return q, scale


def quant_fp8_per_token(x, q=None, scale=None):
    fn = "quant_fp8_per_token"
    _need(isinstance(x, torch.Tensor) and x.dim() == 2, fn, "x must be a 2-D tensor [M, K]")
    M, K = x.shape
    x, q, scale = _quant_args(fn, x, q, scale, (M, K), (M,))
    _check(fn, lib().quant_fp8_per_token(_ptr(x), _ptr(q), _ptr(scale), M, K, _stream()))
    return q, scale


def quant_fp8_group128(x, q=None, scale=None):
    fn = "quant_fp8_group128"
    _need(isinstance(x, torch.Tensor) and x.dim() == 2, fn, "x must be a 2-D tensor [M, K]")
    M, K = x.shape
    x, q, scale = _quant_args(fn, x, q, scale, (M, K), (M, K // 128))
    _check(fn, lib().quant_fp8_group128(_ptr(x), _ptr(q), _ptr(scale), M, K, _stream()))
    return q, scale


def quant_fp8_block128(w, q=None, scale=None):
    fn = "quant_fp8_block128"
    _need(isinstance(w, torch.Tensor) and w.dim() == 2, fn, "w must be a 2-D tensor [N, K]")
    N, K = w.shape
    w, q, scale = _quant_args(fn, w, q, scale, (N, K), (N // 128, K // 128))
    _check(fn, lib().quant_fp8_block128(_ptr(w), _ptr(q), _ptr(scale), N, K, _stream()))
    return q, scale


# ------------------------------------------------------------------ MXFP4 quantizers
def _mxfp4_out(fn, q, scale, M, K, device):
    if q is None:
        q = _rows(M, K // 2, torch.uint8, device)
    else:
        _arg(fn, "q", q, (M, K // 2), _U8, contiguous=True)
    if scale is None:
        scale = _rows(M, K // 32, torch.uint8, device)
    else:
        _arg(fn, "scale", scale, (M, K // 32), _U8, contiguous=True)
    return q, scale


def quant_mxfp4(x, q=None, scale=None):
    """x bf16 [M, K] (row stride may be padded to a multiple of 8) ->
    (q packed e2m1 uint8 [M, K/2], scale e8m0 uint8 [M, K/32])."""
    fn = "quant_mxfp4"
    _need(isinstance(x, torch.Tensor) and x.dim() == 2, fn, "x must be a 2-D tensor [M, K]")
    M, K = x.shape
    if K < 32 or K % 32:
        _need(False, fn, f"K = {K} must be a multiple of 32")
    _arg(fn, "x", x, (M, K), _BF16, unit_inner=False)
    q, scale = _mxfp4_out(fn, q, scale, M, K, x.device)
    stream = _on_current(fn, x, q, scale)
    ldx, inner = x.stride()
    if M == 1:
        ldx = K
    if inner != 1 or ldx < K or ldx % 8 or x.data_ptr() % 16:
        x, ldx = x.clone(memory_format=torch.contiguous_format), K
    _check(fn, lib().quant_mxfp4(x.data_ptr(), ldx, q.data_ptr(), scale.data_ptr(), M, K, stream))
    return q, scale


def silu_mul_quant_mxfp4(gu, q=None, scale=None, rows=None):
    """gu bf16 [M, 2N] (gate half first) -> (q packed e2m1 [M, N/2], scale e8m0
    [M, N/32]) of silu(gate) * up.  rows: optional int32 tensor of one element;
    only the first min(rows, M) rows are computed (e.g. offsets[E:])."""
    fn = "silu_mul_quant_mxfp4"
    _need(isinstance(gu, torch.Tensor) and gu.dim() == 2 and gu.shape[1] % 2 == 0, fn,
          "gu must be a 2-D tensor [M, 2N]")
    M, N = gu.shape[0], gu.shape[1] // 2
    if N < 32 or N % 32:
        _need(False, fn, f"N = {N} must be a multiple of 32")
    _arg(fn, "gu", gu, (M, 2 * N), _BF16, unit_inner=False)
    if rows is not None:
        _arg(fn, "rows", rows, (1,), _I32)
    q, scale = _mxfp4_out(fn, q, scale, M, N, gu.device)
    stream = _on_current(fn, gu, q, scale, rows)
    gu = gu.contiguous()
    _check(fn, lib().silu_mul_quant_mxfp4(_ptr(gu), _ptr(q), _ptr(scale), _ptr(rows), M, N, stream))
    return q, scale


def dequant_mxfp4(q, scale, out=None):
    """(q packed e2m1 [M, K/2], scale e8m0 [M, K/32]) -> the values, bf16 [M, K]."""
    fn = "dequant_mxfp4"
    _need(isinstance(q, torch.Tensor) and q.dim() == 2, fn, "q must be a 2-D tensor [M, K/2]")
    M, K = q.shape[0], 2 * q.shape[1]
    if K < 32 or K % 32:
        _need(False, fn, f"K = {K} must be a multiple of 32")
    _arg(fn, "q", q, (M, K // 2), _U8, unit_inner=False)
    _arg(fn, "scale", scale, (M, K // 32), _U8, unit_inner=False)
    if out is None:
        out = _rows(M, K, torch.bfloat16, q.device)
    else:
        _arg(fn, "out", out, (M, K), _BF16, contiguous=True)
    stream = _on_current(fn, q, scale, out)
    q, scale = q.contiguous(), scale.contiguous()
    _check(fn, lib().dequant_mxfp4(q.data_ptr(), scale.data_ptr(), out.data_ptr(), M, K, stream))
    return out


# ------------------------------------------------------------------ mixture of experts
def moe_sort(ids, E, rows=None, pos=None, offsets=None, ws=None):
    """Sort the (token, expert) pairs by expert.  ids: int32 [T, k], ids outside
    [0, E) are dropped.  -> (rows int32 [T*k]: token of each slot, -1 past the
    kept pairs; pos int32 [T, k]: slot of each pair, -1 if dropped; offsets int32
    [E+1]).  ws: alloc_workspace(BS_OP_MOE_SORT, T, k, E)."""
    fn = "moe_sort"
    _need(isinstance(ids, torch.Tensor) and ids.dim() == 2, fn, "ids must be a 2-D tensor [T, k]")
    T, k = ids.shape
    _arg(fn, "ids", ids, (T, k), _I32, unit_inner=False)
    if not (isinstance(E, int) and E >= 1):
        _need(False, fn, f"E = {E!r} must be a positive int")
    dev = ids.device
    if rows is None:
        rows = torch.empty_strided((T * k,), (1,), dtype=torch.int32, device=dev)
    else:
        _arg(fn, "rows", rows, (T * k,), _I32, contiguous=True)
    if pos is None:
        pos = _rows(T, k, torch.int32, dev)
    else:
        _arg(fn, "pos", pos, (T, k), _I32, contiguous=True)
    if offsets is None:
        offsets = torch.empty_strided((E + 1,), (1,), dtype=torch.int32, device=dev)
    else:
        _arg(fn, "offsets", offsets, (E + 1,), _I32, contiguous=True)
    stream = _on_current(fn, ids, rows, pos, offsets, ws)
    ids = ids.contiguous()
    ws_p, ws_n = _ws(fn, ws)
    _check(fn, lib().moe_sort(ids.data_ptr(), rows.data_ptr(), pos.data_ptr(), offsets.data_ptr(), T, k, E, ws_p, ws_n,
                              stream))
    return rows, pos, offsets


def _moe_pos(fn, pos):
    _need(isinstance(pos, torch.Tensor) and pos.dim() == 2, fn, "pos must be a 2-D tensor [T, k]")
    shape = pos.shape
    _arg(fn, "pos", pos, shape, _I32, contiguous=True)
    return shape


def moe_gather(x, pos, out=None):
    """Token rows in slot order: out[pos[t, j]] = x[t], bf16 [T*k, K].  Rows that
    no pair names keep what they hold.  Gradient: moe_combine(d_out, pos)."""
    fn = "moe_gather"
    T, k = _moe_pos(fn, pos)
    _need(isinstance(x, torch.Tensor) and x.dim() == 2, fn, "x must be a 2-D tensor [T, K]")
    K = x.shape[1]
    _arg(fn, "x", x, (T, K), _BF16, unit_inner=False)
    if out is None:
        out = _rows(T * k, K, torch.bfloat16, x.device)
    else:
        _arg(fn, "out", out, (T * k, K), _BF16, contiguous=True)
    stream = _on_current(fn, x, pos, out)
    x = x.contiguous()
    _check(fn, lib().moe_gather(x.data_ptr(), pos.data_ptr(), out.data_ptr(), T, k, K, stream))
    return out


def moe_combine(y, pos, weights=None, out=None):
    """out[t] = sum_j weights[t, j] * y[pos[t, j]], bf16 [T, K]; weights fp32
    [T, k] or None for ones.  Dropped pairs (pos -1) add nothing."""
    fn = "moe_combine"
    T, k = _moe_pos(fn, pos)
    _need(isinstance(y, torch.Tensor) and y.dim() == 2, fn, "y must be a 2-D tensor [T*k, K]")
    K = y.shape[1]
    _arg(fn, "y", y, (T * k, K), _BF16, unit_inner=False)
    if weights is not None:
        _arg(fn, "weights", weights, (T, k), _F32, contiguous=True)
    if out is None:
        out = _rows(T, K, torch.bfloat16, y.device)
    else:
        _arg(fn, "out", out, (T, K), _BF16, contiguous=True)
    stream = _on_current(fn, y, pos, weights, out)
    y = y.contiguous()
    _check(fn, lib().moe_combine(y.data_ptr(), pos.data_ptr(), _ptr(weights), out.data_ptr(), T, k, K, stream))
    return out


def moe_combine_backward(dout, y, pos, weights, dy=None, dweights=None):
    """Gradient of moe_combine: (dy bf16 [T*k, K] with dy[pos[t, j]] =
    weights[t, j] * dout[t], other rows as they were; dweights fp32 [T, k])."""
    fn = "moe_combine_backward"
    T, k = _moe_pos(fn, pos)
    _need(isinstance(dout, torch.Tensor) and dout.dim() == 2, fn, "dout must be a 2-D tensor [T, K]")
    K = dout.shape[1]
    _arg(fn, "dout", dout, (T, K), _BF16, unit_inner=False)
    _arg(fn, "y", y, (T * k, K), _BF16, unit_inner=False)
    _arg(fn, "weights", weights, (T, k), _F32, contiguous=True)
    if dy is None:
        dy = _rows(T * k, K, torch.bfloat16, y.device)
    else:
        _arg(fn, "dy", dy, (T * k, K), _BF16, contiguous=True)
    if dweights is None:
        dweights = _rows(T, k, torch.float32, y.device)
    else:
        _arg(fn, "dweights", dweights, (T, k), _F32, contiguous=True)
    stream = _on_current(fn, dout, y, pos, weights, dy, dweights)
    dout, y = dout.contiguous(), y.contiguous()
    _check(fn, lib().moe_combine_backward(_ptr(dout), _ptr(y), _ptr(pos), _ptr(weights), _ptr(dy), _ptr(dweights),
                                          T, k, K, stream))
    return dy, dweights
