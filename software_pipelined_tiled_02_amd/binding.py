"""Thin ctypes binding of libpipegemm.so (the C ABI in include/pipegemm.h).

Argument marshalling only: every step of the GEMM runs in the HIP kernels.
The functions keep the C names; device buffers are passed as torch CUDA
tensors (their data_ptr) or plain integer addresses.  run_fp8, quantize_fp8,
rms_fp8 and rms_backward are the 8-bit operators on torch tensors; linear,
gated, gated_backward and weight_gradient those of a feed-forward block in 16
bits.  There is no fallback: if the library is missing, loading raises.
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpipegemm.so")

GEMM_I8, GEMM_F16, GEMM_BF16, GEMM_F32 = 0, 1, 2, 3
GEMM_LAYOUT_RR, GEMM_LAYOUT_RC = 0, 1
GEMM_VARIANT_REG, GEMM_VARIANT_DIRECT = 0, 1
GEMM_OK, GEMM_ERR_INVALID_ARG, GEMM_ERR_ALIGNMENT, GEMM_ERR_UNSUPPORTED, GEMM_ERR_HIP = 0, 1, 2, 3, 4
GEMM_ERR_SCRATCH = 5
GEMM_NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024
GEMM_E4M3, GEMM_E5M2 = 16, 17
GEMM_RMS_MAX_D, GEMM_RMS_MAX_ROWS = 32768, 1 << 22
GEMM_TILE_AUTO, GEMM_TILE_256x256, GEMM_TILE_128x128, GEMM_TILE_32x64, GEMM_TILE_256x256_W8 = -1, 0, 1, 2, 3

DTYPES = {"i8": GEMM_I8, "f16": GEMM_F16, "bf16": GEMM_BF16, "f32": GEMM_F32}
LAYOUTS = {"RR": GEMM_LAYOUT_RR, "RC": GEMM_LAYOUT_RC}
VARIANTS = {"reg": GEMM_VARIANT_REG, "direct": GEMM_VARIANT_DIRECT}
TILES = {"auto": GEMM_TILE_AUTO, "256x256": GEMM_TILE_256x256, "128x128": GEMM_TILE_128x128,
         "32x64": GEMM_TILE_32x64, "256x256w8": GEMM_TILE_256x256_W8}

FP8_TYPES = {"e4m3": GEMM_E4M3, "e5m2": GEMM_E5M2}
FP8_TILES = {"auto": -1, "256x256": 0, "256x128": 1, "128x128": 2, "64x64": 3, "64x64k4": 4,
             "64x32": 5, "32x32": 6, "16x32": 7, "16x16": 8}
FP8_BLOCK = 128   # values of a row that share a scale
BLOCK_ROWS = {"row": 1, "tile": FP8_BLOCK}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
LINEAR_TILES = {"auto": -1, "256x256": 0, "128x256": 1, "128x128": 2, "64x64": 3, "64x64k4": 4, "64x32": 5, "32x32": 6,
                "16x32": 7, "16x16": 8}
LINEAR_FORMS = {"linear_rc": 0, "linear_rr": 1, "gated": 2, "gated_backward": 3, "weight_gradient": 4, "linear_rc_pair": 16,
                "linear_rr_pair": 17}

# C functions exported by the library (the names include/pipegemm.h declares)
EXPORTS = ("gemm_create", "gemm_run", "gemm_destroy", "gemm_set_tile", "gemm_query",
           "gemm_run_splitk", "gemm_query_splitk", "gemm_status_string", "gemm_last_hip_error",
           "gemm_run_splitk_noalloc", "gemm_occupancy", "gemm_run_streamk", "gemm_query_streamk",
           "gemm_run_fp8", "gemm_query_fp8", "gemm_quantize_fp8", "gemm_rms_fp8", "gemm_rms_backward",
           "gemm_rms_backward_workspace", "gemm_linear", "gemm_gated", "gemm_gated_backward", "gemm_weight_gradient",
           "gemm_query_linear")


class GemmError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = "%s: %s" % (where, gemm_status_string(status))
        if status == GEMM_ERR_HIP:
            msg += " (hipError %d)" % _lib().gemm_last_hip_error()
        super().__init__(msg)


class ConfigInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "tile", "block_m", "block_n", "block_k", "waves_m", "waves_n", "threads", "lds_slots",
        "reg_sets", "tiles_in_flight", "lds_bytes", "loads_per_tile")] + [
        ("grid", ctypes.c_int64), ("k_tiles", ctypes.c_int64), ("k_tail", ctypes.c_int32),
        ("c_tiles", ctypes.c_int32), ("splits", ctypes.c_int32), ("mfma_block", ctypes.c_int32),
        ("workspace_bytes", ctypes.c_int64), ("waves_k", ctypes.c_int32), ("sk_tiles", ctypes.c_int32)]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class Occupancy(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "blocks_per_cu", "waves_per_cu", "num_regs", "lds_bytes", "scratch_bytes", "threads")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class Fp8Info(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "tile", "block_m", "block_n", "waves_k", "threads", "staged", "widened", "reserved")] + [
        ("grid", ctypes.c_int64), ("k_blocks", ctypes.c_int64), ("c_tiles", ctypes.c_int64)]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class LinearInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("tile", "block_m", "block_n", "threads", "rows16", "reserved")] + [
        ("grid", ctypes.c_int64), ("k_tiles", ctypes.c_int64)]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


_L = None


def _lib():
    global _L
    if _L is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libpipegemm.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
        lib = ctypes.CDLL(LIB_PATH)
        i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        lib.gemm_create.argtypes = [ctypes.POINTER(vp), ci]
        lib.gemm_create.restype = ci
        lib.gemm_run.argtypes = [vp, i64, i64, i64, ci, ci, ci, ci, vp, i64, vp, i64, vp, i64, vp]
        lib.gemm_run.restype = ci
        lib.gemm_destroy.argtypes = [vp]
        lib.gemm_destroy.restype = ci
        lib.gemm_set_tile.argtypes = [vp, ci]
        lib.gemm_set_tile.restype = ci
        lib.gemm_query.argtypes = [i64, i64, i64, ci, ci, ci, ci, ci, vp, i64, vp, i64, vp, i64,
                                   ctypes.POINTER(ConfigInfo)]
        lib.gemm_query.restype = ci
        lib.gemm_run_splitk.argtypes = [vp, i64, i64, i64, ci, ci, ci, ci, ci, vp, i64, vp, i64, vp, i64,
                                        vp, i64, vp]
        lib.gemm_run_splitk.restype = ci
        lib.gemm_run_streamk.argtypes = [vp, i64, i64, i64, ci, ci, ci, ci, ci, vp, i64, vp, i64, vp, i64,
                                         vp, i64, vp]
        lib.gemm_run_streamk.restype = ci
        lib.gemm_query_streamk.argtypes = [i64, i64, i64, ci, ci, ci, ci, ci, ci, vp, i64, vp, i64, vp, i64,
                                           ctypes.POINTER(ConfigInfo)]
        lib.gemm_query_streamk.restype = ci
        lib.gemm_run_splitk_noalloc.argtypes = [vp, i64, i64, i64, ci, ci, ci, ci, ci, vp, i64, vp, i64, vp,
                                                i64, vp]
        lib.gemm_run_splitk_noalloc.restype = ci
        lib.gemm_occupancy.argtypes = [vp, i64, i64, i64, ci, ci, ci, ci, ctypes.POINTER(Occupancy)]
        lib.gemm_occupancy.restype = ci
        lib.gemm_query_splitk.argtypes = [i64, i64, i64, ci, ci, ci, ci, ci, ci, vp, i64, vp, i64, vp, i64,
                                          ctypes.POINTER(ConfigInfo)]
        lib.gemm_query_splitk.restype = ci
        operand = [vp, i64, vp, i64, i64]            # matrix, leading dimension, scales, their strides
        lib.gemm_run_fp8.argtypes = [vp, i64, i64, i64] + [ci] * 6 + operand * 2 + [vp, i64, vp]
        lib.gemm_run_fp8.restype = ci
        lib.gemm_query_fp8.argtypes = [i64, i64, i64] + [ci] * 6 + operand * 2 + [vp, i64, ctypes.POINTER(Fp8Info)]
        lib.gemm_query_fp8.restype = ci
        lib.gemm_quantize_fp8.argtypes = [vp, i64, i64] + [ci] * 4 + [vp, i64] + operand * 2 + [vp]
        lib.gemm_quantize_fp8.restype = ci
        lib.gemm_rms_fp8.argtypes = ([vp, i64, i64] + [ci] * 4 + [ctypes.c_float] + [vp, i64] * 2 + [vp] +
                                     [vp, i64] * 2 + operand + [vp, vp])
        lib.gemm_rms_fp8.restype = ci
        lib.gemm_rms_backward.argtypes = [vp, i64, i64, ci, ci, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp, vp,
                                          i64, vp]
        lib.gemm_rms_backward.restype = ci
        lib.gemm_rms_backward_workspace.argtypes = [i64, i64]
        lib.gemm_rms_backward_workspace.restype = i64
        lib.gemm_linear.argtypes = [vp, i64, i64, i64] + [ci] * 5 + [vp, i64] * 4 + [vp] + [vp, i64] * 3 + [vp]
        lib.gemm_linear.restype = ci
        lib.gemm_gated.argtypes = [vp, i64, i64, i64] + [ci] * 4 + [vp, i64] * 3 + [vp, vp] + [vp, i64] * 3 + [vp]
        lib.gemm_gated.restype = ci
        lib.gemm_gated_backward.argtypes = [vp, i64, i64, i64] + [ci] * 3 + [vp, i64] * 7 + [vp]
        lib.gemm_gated_backward.restype = ci
        lib.gemm_weight_gradient.argtypes = [vp, i64, i64, i64] + [ci] * 3 + [vp, i64] * 3 + [vp, vp]
        lib.gemm_weight_gradient.restype = ci
        lib.gemm_query_linear.argtypes = [ci, i64, i64, i64] + [ci] * 3 + [ctypes.POINTER(LinearInfo)]
        lib.gemm_query_linear.restype = ci
        lib.gemm_status_string.argtypes = [ci]
        lib.gemm_status_string.restype = ctypes.c_char_p
        lib.gemm_last_hip_error.argtypes = []
        lib.gemm_last_hip_error.restype = ci
        _L = lib
    return _L


def library():
    """The loaded ctypes library (loads it on first call)."""
    return _lib()


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _enum(x, table):
    return table[x] if isinstance(x, str) else int(x)


def gemm_status_string(status):
    return _lib().gemm_status_string(int(status)).decode()


def gemm_create(device=0):
    h = ctypes.c_void_p()
    rc = _lib().gemm_create(ctypes.byref(h), int(device))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_create")
    return h


def gemm_destroy(h):
    _lib().gemm_destroy(h)


def gemm_set_tile(h, tile):
    rc = _lib().gemm_set_tile(h, _enum(tile, TILES))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_set_tile")


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def gemm_run(h, M, N, K, dtype, layout, stages, variant, A, lda, B, ldb, C, ldc, stream=None,
             check=True):
    """Enqueue C = A * B; returns the status (raises on error when check)."""
    rc = _lib().gemm_run(h, M, N, K, _enum(dtype, DTYPES), _enum(layout, LAYOUTS), int(stages),
                         _enum(variant, VARIANTS), _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc,
                         _stream(stream))
    if check and rc != GEMM_OK:
        raise GemmError(rc, "gemm_run")
    return rc


def gemm_run_splitk(h, M, N, K, dtype, layout, stages, variant, splits, A, lda, B, ldb, C, ldc,
                    workspace, workspace_bytes, stream=None, check=True):
    """Enqueue C = A * B with K split over `splits` workgroups per C tile."""
    rc = _lib().gemm_run_splitk(h, M, N, K, _enum(dtype, DTYPES), _enum(layout, LAYOUTS), int(stages),
                                _enum(variant, VARIANTS), int(splits), _ptr(A), lda, _ptr(B), ldb,
                                _ptr(C), ldc, _ptr(workspace), int(workspace_bytes), _stream(stream))
    if check and rc != GEMM_OK:
        raise GemmError(rc, "gemm_run_splitk")
    return rc


def gemm_run_streamk(h, M, N, K, dtype, layout, stages, variant, grid, A, lda, B, ldb, C, ldc,
                     workspace, workspace_bytes, stream=None, check=True):
    """Enqueue C = A * B with the tiles shared out stream-K over `grid`
    workgroups (0: one per compute unit)."""
    rc = _lib().gemm_run_streamk(h, M, N, K, _enum(dtype, DTYPES), _enum(layout, LAYOUTS), int(stages),
                                 _enum(variant, VARIANTS), int(grid), _ptr(A), lda, _ptr(B), ldb,
                                 _ptr(C), ldc, _ptr(workspace), int(workspace_bytes), _stream(stream))
    if check and rc != GEMM_OK:
        raise GemmError(rc, "gemm_run_streamk")
    return rc


def gemm_run_splitk_noalloc(h, M, N, K, dtype, layout, stages, variant, splits, A, lda, B, ldb, C, ldc,
                            stream=None, check=True):
    """Enqueue C = A * B with K split over `splits` workgroups per C tile,
    using the library's static scratch buffer (no workspace argument)."""
    rc = _lib().gemm_run_splitk_noalloc(h, M, N, K, _enum(dtype, DTYPES), _enum(layout, LAYOUTS), int(stages),
                                        _enum(variant, VARIANTS), int(splits), _ptr(A), lda, _ptr(B), ldb,
                                        _ptr(C), ldc, _stream(stream))
    if check and rc != GEMM_OK:
        raise GemmError(rc, "gemm_run_splitk_noalloc")
    return rc


def gemm_occupancy(h, M, N, K, dtype, layout, stages, variant):
    """Resources and occupancy of the instance gemm_run would launch (a dict)."""
    out = Occupancy()
    rc = _lib().gemm_occupancy(h, M, N, K, _enum(dtype, DTYPES), _enum(layout, LAYOUTS), int(stages),
                               _enum(variant, VARIANTS), ctypes.byref(out))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_occupancy")
    return out.as_dict()


def gemm_query(M, N, K, dtype, layout, stages, variant, tile="auto", A=0, lda=None, B=0,
               ldb=None, C=0, ldc=None, check=True, splits=1):
    """The configuration gemm_run (gemm_run_splitk with `splits`) would use
    (no HIP call).  Returns (status, dict)."""
    layout_v = _enum(layout, LAYOUTS)
    lda = K if lda is None else lda
    ldb = (N if layout_v == GEMM_LAYOUT_RR else K) if ldb is None else ldb
    ldc = N if ldc is None else ldc
    info = ConfigInfo()
    rc = _lib().gemm_query_splitk(M, N, K, _enum(dtype, DTYPES), layout_v, int(stages),
                                  _enum(variant, VARIANTS), _enum(tile, TILES), int(splits), A, lda, B,
                                  ldb, C, ldc, ctypes.byref(info))
    if check and rc != GEMM_OK:
        raise GemmError(rc, "gemm_query")
    return rc, info.as_dict()


def gemm_query_streamk(M, N, K, dtype, layout, stages, variant, grid=0, tile="auto", A=0, lda=None, B=0,
                       ldb=None, C=0, ldc=None, check=True):
    """The configuration gemm_run_streamk would use (no HIP call).  Returns
    (status, dict)."""
    layout_v = _enum(layout, LAYOUTS)
    lda = K if lda is None else lda
    ldb = (N if layout_v == GEMM_LAYOUT_RR else K) if ldb is None else ldb
    ldc = N if ldc is None else ldc
    info = ConfigInfo()
    rc = _lib().gemm_query_streamk(M, N, K, _enum(dtype, DTYPES), layout_v, int(stages),
                                   _enum(variant, VARIANTS), _enum(tile, TILES), int(grid), A, lda, B,
                                   ldb, C, ldc, ctypes.byref(info))
    if check and rc != GEMM_OK:
        raise GemmError(rc, "gemm_query_streamk")
    return rc, info.as_dict()


_HANDLES = {}   # device index -> Gemm, for run()


def run(a, b, *, layout="RC", stages=2, variant="direct", out=None, stream=None):
    """C = A * B on torch CUDA tensors through gemm_run.

    A is M x K row-major; B is K x N row-major for layout "RR", or its N x K
    transpose (B column-major) for "RC".  The element type is A's (int8,
    float16, bfloat16 or float32; B must match); C is int32 for int8 and A's
    type otherwise.  `out` (M x N, unit stride along the last axis) is
    written in place, else a new tensor is allocated.  The call is enqueued
    on `stream` (the current stream of A's device by default) and C is
    returned.  Argument errors raise ValueError before any HIP call."""
    import torch
    names = {torch.int8: "i8", torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32"}
    outs = {"i8": torch.int32, "f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
    if not (isinstance(a, torch.Tensor) and isinstance(b, torch.Tensor)) or a.dim() != 2 or b.dim() != 2:
        raise ValueError("A and B must be 2-D torch tensors")
    if a.dtype not in names or b.dtype != a.dtype:
        raise ValueError("A and B must share one of int8, float16, bfloat16, float32 (got %s, %s)"
                         % (a.dtype, b.dtype))
    if not (a.is_cuda and b.is_cuda) or a.device != b.device:
        raise ValueError("A and B must be CUDA tensors on one device")
    dtype = names[a.dtype]
    M, K = a.shape
    if _enum(layout, LAYOUTS) == GEMM_LAYOUT_RR:
        Kb, N = b.shape
    else:
        N, Kb = b.shape
    if Kb != K:
        raise ValueError("inner dimensions differ: A has K = %d, B has %d" % (K, Kb))
    if out is None:
        out = torch.empty((M, N), dtype=outs[dtype], device=a.device)
    elif (not isinstance(out, torch.Tensor) or out.dtype != outs[dtype] or tuple(out.shape) != (M, N)
          or out.device != a.device):
        raise ValueError("out must be an M x N %s tensor on A's device" % outs[dtype])
    dev = a.device.index if a.device.index is not None else torch.cuda.current_device()
    g = _HANDLES.get(dev)
    if g is None:
        g = _HANDLES[dev] = Gemm(dev)
    g.run(a, b, out, dtype, layout, stages, variant,
          stream if stream is not None else torch.cuda.current_stream(a.device))
    return out


# ---- 8-bit floating point with a scale for each block of 128 -----------------

def gemm_run_fp8(h, M, N, K, a_type, b_type, c_dtype, b_scale_rows, accumulate, tile, A, lda, SA, sa_row, sa_blk,
                 B, ldb, SB, sb_row, sb_blk, C, ldc, stream=None, check=True):
    """Enqueue C = A * B of 8-bit matrices with block scales; returns the
    status (raises on error when check)."""
    rc = _lib().gemm_run_fp8(h, M, N, K, _enum(a_type, FP8_TYPES), _enum(b_type, FP8_TYPES), _enum(c_dtype, DTYPES),
                             int(b_scale_rows), int(accumulate), _enum(tile, FP8_TILES), _ptr(A), lda, _ptr(SA),
                             sa_row, sa_blk, _ptr(B), ldb, _ptr(SB), sb_row, sb_blk, _ptr(C), ldc, _stream(stream))
    if check and rc != GEMM_OK:
        raise GemmError(rc, "gemm_run_fp8")
    return rc


def gemm_query_fp8(M, N, K, a_type="e4m3", b_type="e4m3", c_dtype="bf16", b_scale_rows=FP8_BLOCK, accumulate=0,
                   tile="auto", A=0, lda=None, SA=0, sa_row=1, sa_blk=None, B=0, ldb=None, SB=0, sb_row=1, sb_blk=None,
                   C=0, ldc=None, check=True):
    """The kernel gemm_run_fp8 would use (no HIP call).  Returns (status, dict)."""
    info = Fp8Info()
    n_scales = N if b_scale_rows == 1 else -(-N // FP8_BLOCK)
    rc = _lib().gemm_query_fp8(M, N, K, _enum(a_type, FP8_TYPES), _enum(b_type, FP8_TYPES), _enum(c_dtype, DTYPES),
                               int(b_scale_rows), int(accumulate), _enum(tile, FP8_TILES), A,
                               _rows16(K) if lda is None else lda, SA, sa_row, M if sa_blk is None else sa_blk, B,
                               _rows16(K) if ldb is None else ldb, SB, sb_row, n_scales if sb_blk is None else sb_blk,
                               C, N if ldc is None else ldc, ctypes.byref(info))
    if check and rc != GEMM_OK:
        raise GemmError(rc, "gemm_query_fp8")
    return rc, info.as_dict()


def gemm_quantize_fp8(h, M, K, x_dtype, fp8_type, block_rows, pow2, X, ldx, Q, ldq, S, s_row, s_blk, QT=None, ldqt=0,
                      ST=None, st_row=0, st_blk=0, stream=None, check=True):
    """Enqueue X (and its transpose) to 8 bits with block scales."""
    rc = _lib().gemm_quantize_fp8(h, M, K, _enum(x_dtype, DTYPES), _enum(fp8_type, FP8_TYPES), int(block_rows),
                                  int(pow2), _ptr(X), ldx, _ptr(Q), ldq, _ptr(S), s_row, s_blk, _ptr(QT), ldqt,
                                  _ptr(ST), st_row, st_blk, _stream(stream))
    if check and rc != GEMM_OK:
        raise GemmError(rc, "gemm_quantize_fp8")
    return rc


def gemm_rms_fp8(h, M, D, x_dtype, w_dtype, fp8_type, pow2, eps, X, ldx, R, ldr, W, H, ldh, Y, ldy, Q, ldq, S, s_row,
                 s_blk, rstd, stream=None, check=True):
    """Enqueue the norm of X + R, to 8 bits with block scales."""
    rc = _lib().gemm_rms_fp8(h, M, D, _enum(x_dtype, DTYPES), _enum(w_dtype, DTYPES), _enum(fp8_type, FP8_TYPES),
                             int(pow2), eps, _ptr(X), ldx, _ptr(R), ldr, _ptr(W), _ptr(H), ldh, _ptr(Y), ldy, _ptr(Q),
                             ldq, _ptr(S), s_row, s_blk, _ptr(rstd), _stream(stream))
    if check and rc != GEMM_OK:
        raise GemmError(rc, "gemm_rms_fp8")
    return rc


def gemm_rms_backward_workspace(M, D):
    """Bytes of workspace gemm_rms_backward needs."""
    return _lib().gemm_rms_backward_workspace(M, D)


def gemm_rms_backward(h, M, D, x_dtype, w_dtype, DY, lddy, H, ldh, W, rstd, DH, lddh, DX, lddx, DW, workspace,
                      workspace_bytes, stream=None, check=True):
    """Enqueue the norm's backward pass."""
    rc = _lib().gemm_rms_backward(h, M, D, _enum(x_dtype, DTYPES), _enum(w_dtype, DTYPES), _ptr(DY), lddy, _ptr(H),
                                  ldh, _ptr(W), _ptr(rstd), _ptr(DH), lddh, _ptr(DX), lddx, _ptr(DW),
                                  _ptr(workspace), int(workspace_bytes), _stream(stream))
    if check and rc != GEMM_OK:
        raise GemmError(rc, "gemm_rms_backward")
    return rc


def _rows16(n):
    return (n + 15) // 16 * 16


# The functions below are the operators on torch tensors.  Their checks,
# allocations and calls are compiled (csrc/torch_ops.cpp): the smallest calls
# are bound by the host.
_OPS = None
_FP8_NAMES = dict(FP8_TYPES)    # and torch's dtypes, once torch is there


def _ops():
    global _OPS
    if _OPS is None:
        import torch
        _lib()
        path = os.path.join(HERE, "_torch_ops.so")
        if not os.path.exists(path):
            raise RuntimeError("_torch_ops.so is not built (%s); run __graft_entry__.build()" % path)
        from . import _torch_ops
        _FP8_NAMES.update({torch.float8_e4m3fn: GEMM_E4M3, torch.float8_e5m2: GEMM_E5M2})
        _OPS = _torch_ops
    return _OPS


def _named(x, table, what):
    try:
        return table[x]
    except (KeyError, TypeError):
        raise ValueError("%s must be one of %s (got %r)" % (what, ", ".join(map(str, table)), x)) from None


def _on_stream(stream, t):
    """The context in which `stream` (a torch stream or a raw handle) is the
    current one: what a call allocates in it belongs to that stream."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("all tensors must be CUDA tensors")
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=t.device)
    if stream.device != t.device:
        raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, t.device))
    return torch.cuda.stream(stream)


def run_fp8(a, sa, b, sb, *, out=None, out_dtype=None, accumulate=False, tile="auto", stream=None):
    """C = A * B of 8-bit matrices with block scales, through gemm_run_fp8.

    a: M x K, float8_e4m3fn or float8_e5m2; sa: its scales, M x ceil(K / 128)
    float32.  b: B's N x K transpose; sb: ceil(N / 128) x ceil(K / 128)
    ("tile" scales) or N x ceil(K / 128) ("row" scales).  Scales may have any
    strides (expanded ones too).  C is M x N of out_dtype: bfloat16 (the
    default), float16 or float32; `out` is written in place, else a new tensor
    is allocated; accumulate=True adds to a float32 `out`.

    The call is enqueued on `stream` (a torch stream or its raw handle; the
    current stream of A's device by default).  Argument errors raise
    ValueError, or GemmError with the C status, before anything is enqueued.
    The first call on a device sets it up, which a graph capture cannot hold
    (RuntimeError).

    Rows that start on 16 bytes are the fast case, on 128 the fastest
    (quantize_fp8 and rms_fp8 lay them out so); others take twice the time
    with few rows and up to 20 times with thousands.  16-bit outputs take the
    8-bit matrix instructions' sums, float32 ones fp32's."""
    if stream is not None:
        with _on_stream(stream, a):
            return run_fp8(a, sa, b, sb, out=out, out_dtype=out_dtype, accumulate=accumulate, tile=tile)
    return (_OPS or _ops()).run_fp8(a, sa, b, sb, out, out_dtype, accumulate, _named(tile, FP8_TILES, "tile"))


def quantize_fp8(x, *, block="row", fp8="e4m3", pow2=False, rows=True, transpose=False, stream=None):
    """x (M x K; bfloat16, float16 or float32) to 8 bits with a scale for each
    block, through gemm_quantize_fp8: (q, s), or (q, s, qt, st) with
    transpose=True, or (qt, st) with rows=False as well.

    block "row": a scale for each 128 values of a row; s is M x ceil(K / 128).
    "tile": one for each 128 x 128; s is ceil(M / 128) x ceil(K / 128).
    qt (K x M) is x transposed, quantised along its own rows (by tiles: the
    same values and scales as q, transposed); st are its scales.  fp8: "e4m3"
    or "e5m2", or torch's dtype.  pow2: scales are powers of two.  Rows of q
    and qt start on 16 bytes, from 1024 columns on on 128.  Streams and errors
    as run_fp8."""
    if stream is not None:
        with _on_stream(stream, x):
            return quantize_fp8(x, block=block, fp8=fp8, pow2=pow2, rows=rows, transpose=transpose)
    ops = _OPS or _ops()
    return ops.quantize_fp8(x, _named(block, BLOCK_ROWS, "block"), _named(fp8, _FP8_NAMES, "fp8"), pow2, rows, transpose)


def rms_fp8(x, weight, *, residual=None, eps=1e-6, fp8="e4m3", pow2=False, norm=False, h_out=None, stream=None):
    """Root-mean-square norm of x + residual, to 8 bits, through gemm_rms_fp8:
    (q, s, h, rstd), or (q, s, h, rstd, y) with norm=True.

    x, residual: M x D of bfloat16, float16 or float32; weight: D values of
    x's type or float32.  h = x + residual in x's type (x itself without a
    residual), written into h_out where it is given, which may be x or
    residual; rstd: M float32, what rms_backward takes; q, s: the normalised
    rows in 8 bits, a scale for each 128 values; y: the same in x's type.
    D up to 32768.  Streams and errors as run_fp8."""
    if stream is not None:
        with _on_stream(stream, x):
            return rms_fp8(x, weight, residual=residual, eps=eps, fp8=fp8, pow2=pow2, norm=norm, h_out=h_out)
    ops = _OPS or _ops()
    return ops.rms_fp8(x, weight, residual, eps, _named(fp8, _FP8_NAMES, "fp8"), pow2, norm, h_out)


def rms_backward(dy, h, weight, rstd, *, dh=None, dx_out=None, stream=None):
    """The backward pass of rms_fp8's norm, through gemm_rms_backward: (dx, dw).

    dy: the gradient of the normalised rows; h and rstd: what the forward pass
    returned; dh: the gradient that reaches h from elsewhere (the residual
    stream); all M x D of h's type.  dx, in that type, is the gradient of x and of
    the residual; it is written into dx_out where given, which may be dy, h
    or dh.  dw is float32, its rows added in a fixed order.  Streams and errors
    as run_fp8."""
    if stream is not None:
        with _on_stream(stream, dy):
            return rms_backward(dy, h, weight, rstd, dh=dh, dx_out=dx_out)
    return (_OPS or _ops()).rms_backward(dy, h, weight, rstd, dh, dx_out)


# ---- a feed-forward block in 16 bits ---------------------------------------

def gemm_linear(h, M, N, K, dtype, layout, activation, bias_dtype, tile, A, lda, B, ldb, A2, lda2, B2, ldb2, bias, R, ldr,
                Z, ldz, C, ldc, stream=None, check=True):
    """Enqueue C = act(A B + A2 B2 + bias) + R; returns the status (raises on
    error when check)."""
    rc = _lib().gemm_linear(h, M, N, K, _enum(dtype, DTYPES), _enum(layout, LAYOUTS), _enum(activation, ACTIVATIONS),
                            _enum(bias_dtype, DTYPES), _enum(tile, LINEAR_TILES), _ptr(A), lda, _ptr(B), ldb, _ptr(A2), lda2,
                            _ptr(B2), ldb2, _ptr(bias), _ptr(R), ldr, _ptr(Z), ldz, _ptr(C), ldc, _stream(stream))
    if check and rc != GEMM_OK:
        raise GemmError(rc, "gemm_linear")
    return rc


def gemm_gated(h, M, N, K, dtype, activation, bias_dtype, tile, X, ldx, WG, ldwg, WU, ldwu, BG, BU, G, ldg, U, ldu, H, ldh,
               stream=None, check=True):
    """Enqueue H = act(X Wg + bg) * (X Wu + bu)."""
    rc = _lib().gemm_gated(h, M, N, K, _enum(dtype, DTYPES), _enum(activation, ACTIVATIONS), _enum(bias_dtype, DTYPES),
                           _enum(tile, LINEAR_TILES), _ptr(X), ldx, _ptr(WG), ldwg, _ptr(WU), ldwu, _ptr(BG), _ptr(BU),
                           _ptr(G), ldg, _ptr(U), ldu, _ptr(H), ldh, _stream(stream))
    if check and rc != GEMM_OK:
        raise GemmError(rc, "gemm_gated")
    return rc


def gemm_gated_backward(h, M, N, K, dtype, activation, tile, DY, lddy, W, ldw, G, ldg, U, ldu, DG, lddg, DU, lddu, H, ldh,
                        stream=None, check=True):
    """Enqueue the gradients of a gated layer's (or an activation's) arguments."""
    rc = _lib().gemm_gated_backward(h, M, N, K, _enum(dtype, DTYPES), _enum(activation, ACTIVATIONS),
                                    _enum(tile, LINEAR_TILES), _ptr(DY), lddy, _ptr(W), ldw, _ptr(G), ldg, _ptr(U), ldu,
                                    _ptr(DG), lddg, _ptr(DU), lddu, _ptr(H), ldh, _stream(stream))
    if check and rc != GEMM_OK:
        raise GemmError(rc, "gemm_gated_backward")
    return rc


def gemm_weight_gradient(h, M, N, K, dtype, accumulate, tile, DC, lddc, A, lda, DW, lddw, DB, stream=None, check=True):
    """Enqueue DW = DC^T A, and DB, the sums of DC's columns."""
    rc = _lib().gemm_weight_gradient(h, M, N, K, _enum(dtype, DTYPES), int(accumulate), _enum(tile, LINEAR_TILES), _ptr(DC),
                                     lddc, _ptr(A), lda, _ptr(DW), lddw, _ptr(DB), _stream(stream))
    if check and rc != GEMM_OK:
        raise GemmError(rc, "gemm_weight_gradient")
    return rc


def gemm_query_linear(form, M, N, K, dtype="bf16", rows16=True, tile="auto", check=True):
    """The kernel a call of these sizes would use (no HIP call); forms "linear_rc_pair"
    and "linear_rr_pair" are linear's with a second product.  Returns (status, dict)."""
    info = LinearInfo()
    rc = _lib().gemm_query_linear(_enum(form, LINEAR_FORMS), M, N, K, _enum(dtype, DTYPES), int(rows16),
                                  _enum(tile, LINEAR_TILES), ctypes.byref(info))
    if check and rc != GEMM_OK:
        raise GemmError(rc, "gemm_query_linear")
    return rc, info.as_dict()


def linear(a, b, *, layout="RC", bias=None, activation="none", residual=None, pair=None, keep=False, out=None, tile="auto",
           stream=None):
    """act(A B + A2 B2 + bias) + residual through gemm_linear: c, or (c, z) with
    keep=True.

    a: M x K, bfloat16 or float16; b: B's N x K transpose for layout "RC" (a
    layer's weight as it lies), K x N for "RR" (the same weight in the gradient of
    the layer's input).  pair: (a2, b2), shaped as a and b, whose product is
    added before the rounding.  bias: N values of float32 or a's type.
    activation: "none", "relu", "gelu", "gelu_tanh" or "silu".  residual: M x N,
    added behind the activation.  z: the activation's argument in a's type,
    what gated_backward takes.  c is written into out where it is given, which
    may be residual.  Sums are float32, each result is rounded once.

    The call is one kernel, enqueued on `stream` (a torch stream or its raw
    handle; the current stream of a's device by default).  Argument errors raise
    ValueError, or GemmError with the C status, before anything is enqueued.
    The first call on a device sets it up, which a graph capture cannot hold
    (RuntimeError).  Rows that start on 16 bytes are the fast case, others take a
    few percent to half longer: a matrix of an odd width is better held in padded
    rows.  out must overlap nothing else that the call reads or writes.

    Nothing is recorded for torch's autograd: results carry no gradient, also
    where an argument requires one.  The backward pass is the caller's, of
    gated_backward, linear with layout "RR" and weight_gradient, for instance in a
    torch.autograd.Function."""
    if stream is not None:
        with _on_stream(stream, a):
            return linear(a, b, layout=layout, bias=bias, activation=activation, residual=residual, pair=pair, keep=keep,
                          out=out, tile=tile)
    ops = _OPS or _ops()
    a2, b2 = _pair(pair)
    return ops.linear(a, b, _named(layout, LAYOUTS, "layout"), bias, _named(activation, ACTIVATIONS, "activation"), residual,
                      a2, b2, keep, out, _named(tile, LINEAR_TILES, "tile"))


def _pair(pair):
    if pair is None:
        return None, None
    if not isinstance(pair, (tuple, list)) or len(pair) != 2 or pair[0] is None or pair[1] is None:
        raise ValueError("pair must be two matrices")
    return pair


def gated(x, gate, up, *, gate_bias=None, up_bias=None, activation="silu", keep=False, out=None, tile="auto", stream=None):
    """act(X Wg^T + bg) * (X Wu^T + bu) through gemm_gated: h, or (h, g, u) with
    keep=True, g and u being the two factors' arguments.

    x: M x K, bfloat16 or float16; gate, up: the weights, N x K of x's type;
    gate_bias, up_bias: N values of float32 or x's type, both of one.  h is
    formed before g and u are rounded, and written into out where it is given.
    Activations, streams, errors and autograd as linear."""
    if stream is not None:
        with _on_stream(stream, x):
            return gated(x, gate, up, gate_bias=gate_bias, up_bias=up_bias, activation=activation, keep=keep, out=out,
                         tile=tile)
    return (_OPS or _ops()).gated(x, gate, up, gate_bias, up_bias, _named(activation, ACTIVATIONS, "activation"), keep, out,
                                  _named(tile, LINEAR_TILES, "tile"))


def gated_backward(dy, w, g, u=None, *, activation="silu", keep=False, tile="auto", stream=None):
    """The gradients of what a gated layer, or an activation, was taken of,
    through gemm_gated_backward: with dh = dy w,
        dg = dh u act'(g), du = dh act(g): (dg, du), or (dg, du, h) with
        keep=True, h = act(g) u again (so that it need not be kept);
        without u: dg = dh act'(g): dg, or (dg, h), h = act(g).

    dy: M x K, the gradient of the next layer's output; w: that layer's weight
    as it lies, K x N; g, u: what gated(keep=True) returned, or linear's z; all
    of one type.  dh is not rounded.  Streams, errors and autograd as linear."""
    if stream is not None:
        with _on_stream(stream, dy):
            return gated_backward(dy, w, g, u, activation=activation, keep=keep, tile=tile)
    return (_OPS or _ops()).gated_backward(dy, w, g, u, _named(activation, ACTIVATIONS, "activation"), keep,
                                           _named(tile, LINEAR_TILES, "tile"))


def weight_gradient(dc, a, *, out=None, bias=False, bias_out=None, accumulate=False, tile="auto", stream=None):
    """A layer's weight's gradient dC^T A through gemm_weight_gradient: dw (N x K,
    float32), or (dw, db) with bias=True, db being the sums of dc's columns.

    dc: M x N, the gradient of the layer's output (before its activation); a:
    M x K, its input; bfloat16 or float16.  out, bias_out: where dw and db are
    written, or with accumulate=True added.  Streams, errors and autograd as linear."""
    if stream is not None:
        with _on_stream(stream, dc):
            return weight_gradient(dc, a, out=out, bias=bias, bias_out=bias_out, accumulate=accumulate, tile=tile)
    return (_OPS or _ops()).weight_gradient(dc, a, out, bias, bias_out, accumulate, _named(tile, LINEAR_TILES, "tile"))


class Gemm:
    """Owns a handle; ``run`` takes torch CUDA tensors in the ABI's storage:
    A (M x K row-major), B (K x N row-major for RR, its N x K transpose for
    RC), C (M x N row-major)."""

    def __init__(self, device=0):
        self.h = gemm_create(device)
        self.device = device
        self.tile = "auto"
        self._ws = None   # split-K workspace: zeroed once, left zeroed by every call

    def workspace(self, nbytes):
        """A device buffer of at least nbytes for gemm_run_splitk / gemm_run_streamk (grown,
        zeroed, on demand)."""
        import torch
        if self._ws is None or self._ws.numel() < nbytes:
            self._ws = torch.zeros(max(int(nbytes), 1), dtype=torch.uint8, device="cuda:%d" % self.device)
        return self._ws

    def close(self):
        if self.h is not None:
            gemm_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_tile(self, tile):
        gemm_set_tile(self.h, tile)
        self.tile = tile

    def run(self, a, b, c, dtype, layout, stages, variant, stream=None, splits=1):
        M, K = a.shape
        N = b.shape[1] if _enum(layout, LAYOUTS) == GEMM_LAYOUT_RR else b.shape[0]
        for t in (a, b, c):
            if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
                raise ValueError("operands must be 2-D with unit stride along the last axis")
        if splits == 1:
            return gemm_run(self.h, M, N, K, dtype, layout, stages, variant,
                            a, a.stride(0), b, b.stride(0), c, c.stride(0), stream)
        return self.run_splitk(M, N, K, dtype, layout, stages, variant, splits, a, a.stride(0), b,
                               b.stride(0), c, c.stride(0), stream)

    def run_splitk(self, M, N, K, dtype, layout, stages, variant, splits, A, lda, B, ldb, C, ldc,
                   stream=None, check=True):
        """gemm_run_splitk with this handle's tile and workspace."""
        _, info = gemm_query(M, N, K, dtype, layout, stages, variant, tile=self.tile, lda=lda, ldb=ldb,
                             ldc=ldc, splits=splits, check=False)
        ws = self.workspace(info["workspace_bytes"]) if info["workspace_bytes"] > 0 else None
        return gemm_run_splitk(self.h, M, N, K, dtype, layout, stages, variant, splits, A, lda, B, ldb,
                               C, ldc, ws, ws.numel() if ws is not None else 0, stream, check)

    def run_streamk(self, M, N, K, dtype, layout, stages, variant, grid, A, lda, B, ldb, C, ldc,
                    stream=None, check=True):
        """gemm_run_streamk with this handle's tile and workspace."""
        _, info = gemm_query_streamk(M, N, K, dtype, layout, stages, variant, grid=grid, tile=self.tile,
                                     lda=lda, ldb=ldb, ldc=ldc, check=False)
        ws = self.workspace(info["workspace_bytes"]) if info["workspace_bytes"] > 0 else None
        return gemm_run_streamk(self.h, M, N, K, dtype, layout, stages, variant, grid, A, lda, B, ldb, C, ldc,
                                ws, 0 if ws is None else ws.numel(), stream, check)
