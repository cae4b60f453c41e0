"""Python binding of the gfx950 dense GEMM library (libdense_gemm.so).

The functions mirror the C ABI in include/dense_gemm.h one to one and only
marshal arguments; every step of the GEMM runs in the library's HIP kernels.
``run_tensors`` is a convenience that reads shapes, leading dimensions, device
pointers and the current stream from torch tensors (torch supplies device
memory and streams only).

Importing this package loads the library; if it has not been built the import
fails loudly (there is no fallback implementation).

One HIP runtime per process: PyTorch's ROCm wheels ship their own copy of
libamdhip64 (same soname as the system one).  Device pointers and streams
only mean something to the runtime that created them, so torch is imported
before the library is loaded; the dynamic linker then binds the library to
the runtime torch already loaded instead of loading a second one.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdense_gemm.so")

GEMM_OP_N = 0
GEMM_OP_T = 1
GEMM_DTYPE_F32 = 0
GEMM_DTYPE_BF16_F32 = 1
GEMM_DTYPE_BF16_BF16 = 2
GEMM_OK = 0
GEMM_ERR_INVALID_VALUE = 1
GEMM_ERR_NOT_SUPPORTED = 2
GEMM_ERR_HIP = 3
GEMM_ERR_ALLOC = 4
GEMM_ERR_STREAM_K = 5
# bytes of the static stream-K array gemm_run_no_alloc uses on each GPU
GEMM_NO_ALLOC_SCRATCH_BYTES = 16640 + (16 << 20)
GEMM_ACT_NONE = 0
GEMM_ACT_RELU = 1
GEMM_ACT_GELU = 2

# Every function declared in include/dense_gemm.h.
EXPORTS = ("gemm_create", "gemm_destroy", "gemm_run", "gemm_status_string",
           "gemm_variant_count", "gemm_variant_name", "gemm_variant_dtype",
           "gemm_variant_tile", "gemm_set_variant", "gemm_last_variant",
           "gemm_select_variant", "gemm_stream_k_workspace_bytes", "gemm_set_workspace",
           "gemm_set_stream_k", "gemm_last_stream_k", "gemm_run_epilogue",
           "gemm_variant_pipeline", "gemm_variant_occupancy", "gemm_stream_k_status",
           "gemm_set_stream_k_poll_limit", "gemm_run_no_alloc", "gemm_set_planning_model",
           "gemm_run_grouped", "gemm_run_grouped_wgrad", "gemm_run_lora",
           "gemm_lora_workspace_bytes", "gemm_set_group_tile", "gemm_last_group_tile",
           "gemm_set_group_tile_nth", "gemm_last_group_launch")


class GemmEpilogue(ctypes.Structure):
    """gemm_epilogue_t: bias pointer (0/None for none), activation, clamp flag
    and bounds."""
    _fields_ = [("bias", ctypes.c_void_p), ("activation", ctypes.c_int),
                ("clamp", ctypes.c_int), ("clamp_lo", ctypes.c_float),
                ("clamp_hi", ctypes.c_float)]


class GemmGroups(ctypes.Structure):
    """gemm_groups_t: device pointers to groups + 1 int32 offsets and to one
    fp32 factor per group (0/None for none)."""
    _fields_ = [("groups", ctypes.c_int), ("offsets", ctypes.c_void_p),
                ("scales", ctypes.c_void_p)]


class GemmLora(ctypes.Structure):
    """gemm_lora_t: the segments of rows and their low-rank adapters."""
    _fields_ = [("segments", ctypes.c_int), ("offsets", ctypes.c_void_p),
                ("ids", ctypes.c_void_p), ("adapters", ctypes.c_int), ("rank", ctypes.c_int),
                ("scales", ctypes.c_void_p), ("trans_down", ctypes.c_int),
                ("down", ctypes.c_void_p), ("ld_down", ctypes.c_int64),
                ("stride_down", ctypes.c_int64), ("trans_up", ctypes.c_int),
                ("up", ctypes.c_void_p), ("ld_up", ctypes.c_int64), ("stride_up", ctypes.c_int64)]


class GemmGroupLaunch(ctypes.Structure):
    """gemm_group_launch_t: what the last ragged call launched."""
    _fields_ = [(n, ctypes.c_int) for n in ("rows", "columns", "nth", "launches", "first_rows",
                                            "first_columns", "first_slices")]


class GemmError(RuntimeError):
    def __init__(self, status: int, what: str = "gemm_run"):
        self.status = status
        super().__init__(f"{what} failed: {gemm_status_string(status)}")


def hip_runtimes_loaded():
    """Distinct libamdhip64 files mapped into this process (Linux)."""
    try:
        with open("/proc/self/maps") as f:
            paths = {line.split()[-1] for line in f if "libamdhip64" in line}
    except OSError:
        return []
    return sorted({os.path.realpath(p) for p in paths})


def _load():
    try:  # bind to torch's HIP runtime when torch is present (see module docstring)
        import torch  # noqa: F401
    except ImportError:
        pass
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build the HIP library first "
            "(python dense_gemm_11_amd/build.py)")
    lib = ctypes.CDLL(LIB_PATH)
    runtimes = hip_runtimes_loaded()
    if len(runtimes) > 1:
        raise ImportError("two HIP runtimes are loaded in this process (" + ", ".join(runtimes)
                          + "); import torch before anything that loads libamdhip64")
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    lib.gemm_create.argtypes = [ctypes.POINTER(vp)]
    lib.gemm_create.restype = i32
    lib.gemm_destroy.argtypes = [vp]
    lib.gemm_destroy.restype = i32
    lib.gemm_run.argtypes = [vp, i32, i32, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64,
                             vp, i64, i32, vp]
    lib.gemm_run.restype = i32
    lib.gemm_run_no_alloc.argtypes = [vp, i32, i32, i64, i64, i64, f32, vp, i64, vp, i64, f32,
                                      vp, i64, vp, i64, i32, vp]
    lib.gemm_run_no_alloc.restype = i32
    lib.gemm_run_epilogue.argtypes = [vp, i32, i32, i64, i64, i64, f32, vp, i64, vp, i64, f32,
                                      vp, i64, vp, i64, i32, ctypes.POINTER(GemmEpilogue), vp]
    lib.gemm_run_epilogue.restype = i32
    lib.gemm_status_string.argtypes = [i32]
    lib.gemm_status_string.restype = ctypes.c_char_p
    lib.gemm_variant_count.argtypes = []
    lib.gemm_variant_count.restype = i32
    lib.gemm_variant_name.argtypes = [i32]
    lib.gemm_variant_name.restype = ctypes.c_char_p
    lib.gemm_variant_dtype.argtypes = [i32]
    lib.gemm_variant_dtype.restype = i32
    lib.gemm_variant_tile.argtypes = [i32, ctypes.POINTER(i32), ctypes.POINTER(i32),
                                      ctypes.POINTER(i32)]
    lib.gemm_variant_tile.restype = i32
    lib.gemm_variant_pipeline.argtypes = [i32, ctypes.POINTER(i32), ctypes.POINTER(i32)]
    lib.gemm_variant_pipeline.restype = i32
    lib.gemm_variant_occupancy.argtypes = [i32]
    lib.gemm_variant_occupancy.restype = i32
    lib.gemm_set_planning_model.argtypes = [i32, ctypes.POINTER(i32), i32]
    lib.gemm_set_planning_model.restype = i32
    lib.gemm_set_variant.argtypes = [vp, i32]
    lib.gemm_set_variant.restype = i32
    lib.gemm_last_variant.argtypes = [vp]
    lib.gemm_last_variant.restype = i32
    lib.gemm_select_variant.argtypes = [i32, i32, i32, i64, i64, i64]
    lib.gemm_select_variant.restype = i32
    lib.gemm_stream_k_workspace_bytes.argtypes = []
    lib.gemm_stream_k_workspace_bytes.restype = ctypes.c_size_t
    lib.gemm_set_workspace.argtypes = [vp, vp, ctypes.c_size_t, vp]
    lib.gemm_set_workspace.restype = i32
    lib.gemm_set_stream_k.argtypes = [vp, i32]
    lib.gemm_set_stream_k.restype = i32
    lib.gemm_last_stream_k.argtypes = [vp]
    lib.gemm_last_stream_k.restype = i32
    lib.gemm_stream_k_status.argtypes = [vp, vp]
    lib.gemm_stream_k_status.restype = i32
    lib.gemm_set_stream_k_poll_limit.argtypes = [vp, i32]
    lib.gemm_set_stream_k_poll_limit.restype = i32
    lib.gemm_run_grouped.argtypes = [vp, i32, i64, i64, i64, f32, vp, i64, vp, i64, i64, f32, vp,
                                     i64, vp, i64, i32, ctypes.POINTER(GemmGroups), vp]
    lib.gemm_run_grouped.restype = i32
    lib.gemm_run_grouped_wgrad.argtypes = [vp, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64,
                                           i64, vp, i64, i64, i32, ctypes.POINTER(GemmGroups), vp]
    lib.gemm_run_grouped_wgrad.restype = i32
    lib.gemm_run_lora.argtypes = [vp, i32, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, vp,
                                  i64, i32, ctypes.POINTER(GemmLora), vp, ctypes.c_size_t, vp]
    lib.gemm_run_lora.restype = i32
    lib.gemm_lora_workspace_bytes.argtypes = [i64, i32]
    lib.gemm_lora_workspace_bytes.restype = ctypes.c_size_t
    lib.gemm_set_group_tile.argtypes = [vp, i32]
    lib.gemm_set_group_tile.restype = i32
    lib.gemm_last_group_tile.argtypes = [vp]
    lib.gemm_last_group_tile.restype = i32
    lib.gemm_set_group_tile_nth.argtypes = [vp, i32, i32]
    lib.gemm_set_group_tile_nth.restype = i32
    lib.gemm_last_group_launch.argtypes = [vp, ctypes.POINTER(GemmGroupLaunch)]
    lib.gemm_last_group_launch.restype = i32
    return lib


lib = _load()


def gemm_create() -> int:
    h = ctypes.c_void_p()
    s = lib.gemm_create(ctypes.byref(h))
    if s != GEMM_OK:
        raise GemmError(s, "gemm_create")
    return h.value


def gemm_destroy(h) -> int:
    return lib.gemm_destroy(h)


def gemm_run(h, transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, D, ldd,
             dtype, stream) -> int:
    """Raw call: pointers and the stream are integers (0/None for NULL)."""
    return lib.gemm_run(h, transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                        D, ldd, dtype, stream)


def gemm_run_no_alloc(h, transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, D,
                      ldd, dtype, stream) -> int:
    """Raw call: pointers and the stream are integers (0/None for NULL)."""
    return lib.gemm_run_no_alloc(h, transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C,
                                 ldc, D, ldd, dtype, stream)


def gemm_run_epilogue(h, transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, D, ldd,
                      dtype, epilogue, stream) -> int:
    """Raw call: pointers and the stream are integers (0/None for NULL);
    epilogue is a GemmEpilogue or None."""
    ep = None if epilogue is None else ctypes.byref(epilogue)
    return lib.gemm_run_epilogue(h, transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C,
                                 ldc, D, ldd, dtype, ep, stream)


def gemm_status_string(s: int) -> str:
    return lib.gemm_status_string(s).decode()


def gemm_variant_count() -> int:
    return lib.gemm_variant_count()


def gemm_variant_name(i: int):
    n = lib.gemm_variant_name(i)
    return None if n is None else n.decode()


def gemm_variant_dtype(i: int) -> int:
    return lib.gemm_variant_dtype(i)


def gemm_variant_tile(i: int):
    bm, bn, bk = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    s = lib.gemm_variant_tile(i, ctypes.byref(bm), ctypes.byref(bn), ctypes.byref(bk))
    if s != GEMM_OK:
        raise GemmError(s, "gemm_variant_tile")
    return bm.value, bn.value, bk.value


def gemm_variant_pipeline(i: int):
    """(stages, ahead) of variant i."""
    st, ah = ctypes.c_int(), ctypes.c_int()
    s = lib.gemm_variant_pipeline(i, ctypes.byref(st), ctypes.byref(ah))
    if s != GEMM_OK:
        raise GemmError(s, "gemm_variant_pipeline")
    return st.value, ah.value


def gemm_variant_occupancy(i: int) -> int:
    return lib.gemm_variant_occupancy(i)


def gemm_set_planning_model(cus: int, occupancy=None) -> int:
    """gemm_set_planning_model: `occupancy` is a sequence of
    gemm_variant_count() workgroups-per-unit figures (0: keep the device
    query), or None (with cus = 0) to clear the model."""
    if occupancy is None:
        return lib.gemm_set_planning_model(cus, None, 0)
    arr = (ctypes.c_int32 * len(occupancy))(*occupancy)
    return lib.gemm_set_planning_model(cus, arr, len(occupancy))


def gemm_set_variant(h, i: int) -> int:
    return lib.gemm_set_variant(h, i)


def gemm_last_variant(h) -> int:
    return lib.gemm_last_variant(h)


def gemm_select_variant(dtype, transA, transB, M, N, K) -> int:
    return lib.gemm_select_variant(dtype, transA, transB, M, N, K)


def gemm_stream_k_workspace_bytes() -> int:
    return lib.gemm_stream_k_workspace_bytes()


def gemm_set_workspace(h, ws, nbytes: int, stream) -> int:
    """Raw call: ws and stream are integers (0/None for NULL)."""
    return lib.gemm_set_workspace(h, ws, nbytes, stream)


def gemm_set_stream_k(h, mode: int) -> int:
    return lib.gemm_set_stream_k(h, mode)


def gemm_last_stream_k(h) -> int:
    return lib.gemm_last_stream_k(h)


def gemm_stream_k_status(h, stream) -> int:
    """Raw call: stream is an integer (0/None for the default stream)."""
    return lib.gemm_stream_k_status(h, stream)


def gemm_set_stream_k_poll_limit(h, polls: int) -> int:
    return lib.gemm_set_stream_k_poll_limit(h, polls)


def gemm_run_grouped(h, transB, M, N, K, alpha, A, lda, B, ldb, strideB, beta, C, ldc, D, ldd,
                     dtype, groups, stream) -> int:
    """Raw call: pointers and the stream are integers (0/None for NULL); groups
    is a GemmGroups or None."""
    gr = None if groups is None else ctypes.byref(groups)
    return lib.gemm_run_grouped(h, transB, M, N, K, alpha, A, lda, B, ldb, strideB, beta, C, ldc,
                                D, ldd, dtype, gr, stream)


def gemm_run_grouped_wgrad(h, M, N, rows, alpha, A, lda, B, ldb, beta, C, ldc, strideC, D, ldd,
                           strideD, dtype, groups, stream) -> int:
    """Raw call: pointers and the stream are integers (0/None for NULL); groups
    is a GemmGroups or None."""
    gr = None if groups is None else ctypes.byref(groups)
    return lib.gemm_run_grouped_wgrad(h, M, N, rows, alpha, A, lda, B, ldb, beta, C, ldc, strideC,
                                      D, ldd, strideD, dtype, gr, stream)


def gemm_run_lora(h, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, D, ldd, dtype, lora,
                  workspace, workspace_bytes, stream) -> int:
    """Raw call: pointers and the stream are integers (0/None for NULL); lora
    is a GemmLora or None."""
    lo = None if lora is None else ctypes.byref(lora)
    return lib.gemm_run_lora(h, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, D, ldd, dtype,
                             lo, workspace, workspace_bytes, stream)


def gemm_lora_workspace_bytes(M: int, rank: int) -> int:
    return lib.gemm_lora_workspace_bytes(M, rank)


def gemm_set_group_tile(h, rows: int) -> int:
    return lib.gemm_set_group_tile(h, rows)


def gemm_last_group_tile(h) -> int:
    return lib.gemm_last_group_tile(h)


def gemm_set_group_tile_nth(h, rows: int, nth: int) -> int:
    return lib.gemm_set_group_tile_nth(h, rows, nth)


def gemm_last_group_launch(h) -> GemmGroupLaunch:
    out = GemmGroupLaunch()
    s = lib.gemm_last_group_launch(h, ctypes.byref(out))
    if s != GEMM_OK:
        raise GemmError(s, "gemm_last_group_launch")
    return out


def attach_workspace(h, nbytes=None, device=None):
    """Allocate a stream-K workspace as a torch uint8 tensor on `device` (the
    current device by default), hand it to h and return it; the caller keeps
    the tensor alive as long as h may use it."""
    import torch

    nbytes = gemm_stream_k_workspace_bytes() if nbytes is None else int(nbytes)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
    stream = torch.cuda.current_stream(ws.device).cuda_stream
    s = gemm_set_workspace(h, ws.data_ptr(), nbytes, stream)
    if s != GEMM_OK:
        raise GemmError(s, "gemm_set_workspace")
    return ws


def variants():
    """[(id, name, dtype, (bm, bn, bk))] for every kernel variant."""
    return [(i, gemm_variant_name(i), gemm_variant_dtype(i), gemm_variant_tile(i))
            for i in range(gemm_variant_count())]


def _marshal(h, A, B, D, C, transA, transB, alpha, beta, stream, bias, activation, clamp,
             no_alloc):
    """Check torch tensors and turn them into (C function, argument tuple)."""
    import torch

    def ld(t):
        if t.dim() != 2 or t.stride(1) != 1:
            raise ValueError("expected a 2-D tensor with unit column stride")
        return t.stride(0)

    if A.dtype == torch.float32 and B.dtype == torch.float32:
        dtype = GEMM_DTYPE_F32
    elif A.dtype == torch.bfloat16 and B.dtype == torch.bfloat16:
        dtype = GEMM_DTYPE_BF16_BF16 if D.dtype == torch.bfloat16 else GEMM_DTYPE_BF16_F32
    else:
        raise TypeError("A and B must both be float32 or both bfloat16")
    out = torch.bfloat16 if dtype == GEMM_DTYPE_BF16_BF16 else torch.float32
    if D.dtype != out or (C is not None and C.dtype != out):
        raise TypeError("C and D must be float32, or both bfloat16 with bfloat16 operands")
    M, K = (A.shape[0], A.shape[1]) if transA == "N" else (A.shape[1], A.shape[0])
    Kb, N = (B.shape[0], B.shape[1]) if transB == "N" else (B.shape[1], B.shape[0])
    if Kb != K or tuple(D.shape) != (M, N) or (C is not None and tuple(C.shape) != (M, N)):
        raise ValueError("inconsistent GEMM shapes")
    if bias is not None and (bias.dtype != out or bias.dim() != 1 or bias.shape[0] != N
                             or (N > 1 and bias.stride(0) != 1)):
        raise ValueError("bias must be a contiguous length-N tensor of D's dtype")
    if stream is None:
        stream = torch.cuda.current_stream(D.device).cuda_stream
    args = (h, GEMM_OP_N if transA == "N" else GEMM_OP_T,
            GEMM_OP_N if transB == "N" else GEMM_OP_T, M, N, K, float(alpha),
            A.data_ptr(), ld(A), B.data_ptr(), ld(B), float(beta),
            None if C is None else C.data_ptr(), ld(C) if C is not None else N,
            D.data_ptr(), ld(D), dtype)
    plain = bias is None and activation == GEMM_ACT_NONE and clamp is None
    if no_alloc:
        if not plain:
            raise ValueError("gemm_run_no_alloc has no fused epilogue")
        return lib.gemm_run_no_alloc, args + (stream,)
    if plain:
        return lib.gemm_run, args + (stream,)
    lo, hi = (0.0, 0.0) if clamp is None else clamp
    ep = GemmEpilogue(None if bias is None else bias.data_ptr(), int(activation),
                      int(clamp is not None), float(lo), float(hi))
    return lib.gemm_run_epilogue, args + (ctypes.byref(ep), stream)


def run_tensors(h, A, B, D, C=None, transA="N", transB="N", alpha=1.0, beta=0.0,
                stream=None, check=True, bias=None, activation=GEMM_ACT_NONE,
                clamp=None, no_alloc=False) -> int:
    """gemm_run on torch tensors (row-major 2-D views with unit column stride).

    A: op(A) is M x K (A stored M x K for "N", K x M for "T"); B likewise;
    C, D: M x N.  A and B are float32 (fp32 GEMM) or bfloat16; with bfloat16
    operands, C and D are float32 (GEMM_DTYPE_BF16_F32) or both bfloat16
    (GEMM_DTYPE_BF16_BF16).  bias (a length-N tensor of D's dtype),
    activation (GEMM_ACT_*) and clamp ((lo, hi)) select gemm_run_epilogue;
    no_alloc selects gemm_run_no_alloc.
    """
    fn, args = _marshal(h, A, B, D, C, transA, transB, alpha, beta, stream, bias, activation,
                        clamp, no_alloc)
    s = fn(*args)
    if check and s != GEMM_OK:
        raise GemmError(s)
    return s


def bind_tensors(h, A, B, D, C=None, transA="N", transB="N", alpha=1.0, beta=0.0,
                 stream=None, bias=None, activation=GEMM_ACT_NONE, clamp=None,
                 no_alloc=False):
    """run_tensors' C call with its arguments marshalled once: returns a
    function that makes the same call again and returns its status (for
    timing loops; the tensors must stay alive while it is used)."""
    fn, args = _marshal(h, A, B, D, C, transA, transB, alpha, beta, stream, bias, activation,
                        clamp, no_alloc)
    return lambda: fn(*args)


# The ragged calls are made per token by a decoding loop, where the kernels take
# a few microseconds, so their marshalling asks torch for each property once.
def _matrix(t):
    """Rows, columns and leading dimension of a 2-D tensor with unit stride in
    its last axis."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1):
        raise ValueError("expected a 2-D tensor with unit stride in its last axis")
    rows, cols = shape
    # a single row has no stride of its own; too small a stride (an expanded
    # tensor) is refused by the library
    return rows, cols, stride[0] if rows > 1 else max(cols, 1)


def _matrices(t):
    """Count, rows, columns, leading dimension and stride between the matrices of
    a 3-D tensor with unit stride in its last axis."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or (stride[2] != 1 and shape[2] > 1):
        raise ValueError("expected a 3-D tensor with unit stride in its last axis")
    count, rows, cols = shape
    return count, rows, cols, stride[1] if rows > 1 else max(cols, 1), stride[0]


def _ragged_dtype(A, B, D, C):
    """gemm_dtype_t of a ragged product's tensors."""
    import torch

    ta, td = A.dtype, D.dtype
    if ta is not B.dtype or (C is not None and C.dtype is not td):
        raise TypeError("A and B, and C and D, must have one dtype each")
    if ta is torch.bfloat16:
        if td is torch.bfloat16:
            return GEMM_DTYPE_BF16_BF16
        if td is torch.float32:
            return GEMM_DTYPE_BF16_F32
    elif ta is torch.float32 and td is torch.float32:
        return GEMM_DTYPE_F32
    raise TypeError("A and B must be float32, or bfloat16 with float32 or bfloat16 C and D")


def _device_vector(t, dtype, length, device, what):
    """Data pointer of a contiguous 1-D tensor on device index `device` (None
    stays None)."""
    if t is None:
        return None
    shape = t.shape
    if len(shape) != 1 or shape[0] != length or t.dtype is not dtype or (
            t.get_device() != device) or (length > 1 and t.stride()[0] != 1):
        raise ValueError(f"{what} must be a contiguous length-{length} {dtype} tensor on D's device")
    return t.data_ptr()


def _device_of(D, *tensors):
    """D's device index, which every tensor has to share."""
    device = D.get_device()
    if device < 0:
        raise ValueError("the tensors must be on a GPU")
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError("every tensor must be on D's device")
    return device


def _stream_on(device):
    """The current stream of a device, as an integer."""
    import torch

    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # without a Stream object
    return raw(device) if raw else torch.cuda.current_stream(device).cuda_stream


def _finish(status, check, what):
    if check and status != GEMM_OK:
        raise GemmError(status, what)
    return status


def run_grouped(h, A, B, D, offsets, C=None, transB="N", scales=None, alpha=1.0, beta=0.0,
                stream=None, check=True) -> int:
    """gemm_run_grouped on torch tensors: for each group g, with its rows
    offsets[g] .. offsets[g+1]-1,
    D[rows] = alpha * scales[g] * A[rows] @ op(B[g]) + beta * C[rows].

    A: M x K; B: groups x K x N ("N") or groups x N x K ("T"); C, D: M x N;
    offsets: int32, groups + 1, on the device; scales: float32, groups, or
    None.  Types as for run_tensors.  Rows in no group keep their values.
    """
    import torch

    dtype = _ragged_dtype(A, B, D, C)
    M, K, lda = _matrix(A)
    groups, Kb, N, ldb, stride_b = _matrices(B)
    if transB != "N":
        Kb, N = N, Kb
    Md, Nd, ldd = _matrix(D)
    c, ldc = None, N
    if C is not None:
        c = C.data_ptr()
        Mc, Nc, ldc = _matrix(C)
        if Mc != M or Nc != N:
            raise ValueError("inconsistent grouped GEMM shapes")
    if Kb != K or Md != M or Nd != N:
        raise ValueError("inconsistent grouped GEMM shapes")
    device = _device_of(D, A, B, C)
    gr = GemmGroups(groups, _device_vector(offsets, torch.int32, groups + 1, device, "offsets"),
                    _device_vector(scales, torch.float32, groups, device, "scales"))
    s = lib.gemm_run_grouped(
        h, GEMM_OP_N if transB == "N" else GEMM_OP_T, M, N, K, alpha, A.data_ptr(), lda,
        B.data_ptr(), ldb, stride_b, beta, c, ldc, D.data_ptr(), ldd, dtype, ctypes.byref(gr),
        _stream_on(device) if stream is None else stream)
    return _finish(s, check, "gemm_run_grouped")


def run_grouped_wgrad(h, A, B, D, offsets, C=None, scales=None, alpha=1.0, beta=0.0, stream=None,
                      check=True) -> int:
    """gemm_run_grouped_wgrad on torch tensors: for each group g, with its rows
    offsets[g] .. offsets[g+1]-1,
    D[g] = alpha * scales[g] * A[rows].T @ B[rows] + beta * C[g].

    A: rows x M; B: rows x N; C, D: groups x M x N; offsets and scales as for
    run_grouped.  D[g] of an empty group is beta * C[g].
    """
    import torch

    dtype = _ragged_dtype(A, B, D, C)
    rows, M, lda = _matrix(A)
    rows_b, N, ldb = _matrix(B)
    groups, Md, Nd, ldd, stride_d = _matrices(D)
    c, ldc, stride_c = None, N, 0
    if C is not None:
        if C.shape != D.shape:
            raise ValueError("inconsistent grouped GEMM shapes")
        c = C.data_ptr()
        _, _, _, ldc, stride_c = _matrices(C)
    if rows_b != rows or Md != M or Nd != N:
        raise ValueError("inconsistent grouped GEMM shapes")
    device = _device_of(D, A, B, C)
    gr = GemmGroups(groups, _device_vector(offsets, torch.int32, groups + 1, device, "offsets"),
                    _device_vector(scales, torch.float32, groups, device, "scales"))
    s = lib.gemm_run_grouped_wgrad(
        h, M, N, rows, alpha, A.data_ptr(), lda, B.data_ptr(), ldb, beta, c, ldc, stride_c,
        D.data_ptr(), ldd, stride_d, dtype, ctypes.byref(gr),
        _stream_on(device) if stream is None else stream)
    return _finish(s, check, "gemm_run_grouped_wgrad")


def lora_workspace(rows: int, rank: int, device=None):
    """A workspace for run_lora on up to `rows` rows and rank `rank`, as a torch
    uint8 tensor on `device` (the current device by default); one per
    concurrently used stream."""
    import torch

    need = gemm_lora_workspace_bytes(rows, rank)
    return torch.empty(max(need, 256), dtype=torch.uint8,
                       device="cuda" if device is None else device)


def run_lora(h, A, B, D, offsets, down, up, workspace, ids=None, scales=None, C=None, transB="N",
             transDown="T", transUp="T", alpha=1.0, beta=0.0, stream=None, check=True) -> int:
    """gemm_run_lora on torch tensors: a shared product with one low-rank
    adapter per segment of rows,
    D[rows] = alpha * (A[rows] @ op(B) + scales[a] * (A[rows] @ op(down[a])) @ op(up[a]))
              + beta * C[rows], with a = ids[segment].

    A: M x K; B: K x N ("N") or N x K ("T"); C, D: M x N; down: adapters x R x K
    ("T") or adapters x K x R ("N"); up: adapters x N x R ("T") or adapters x R
    x N ("N"); offsets: int32, segments + 1, on the device; ids: int32,
    segments (negative: no adapter), or None for adapter s in segment s;
    scales: float32, adapters, or None; workspace: from lora_workspace.
    """
    import torch

    dtype = _ragged_dtype(A, B, D, C)
    if down.dtype is not A.dtype or up.dtype is not A.dtype:
        raise TypeError("down and up must have A's dtype")
    M, K, lda = _matrix(A)
    Kb, N, ldb = _matrix(B)
    if transB != "N":
        Kb, N = N, Kb
    Md, Nd, ldd = _matrix(D)
    adapters, R, Kd, ld_down, stride_down = _matrices(down)
    if transDown == "N":
        R, Kd = Kd, R
    adapters_up, Nu, Ru, ld_up, stride_up = _matrices(up)
    if transUp == "N":
        Nu, Ru = Ru, Nu
    c, ldc = None, N
    if C is not None:
        c = C.data_ptr()
        Mc, Nc, ldc = _matrix(C)
        if Mc != M or Nc != N:
            raise ValueError("inconsistent low-rank adapter shapes")
    if Kb != K or Md != M or Nd != N or Kd != K or adapters_up != adapters or Nu != N or Ru != R:
        raise ValueError("inconsistent low-rank adapter shapes")
    device = _device_of(D, A, B, C, down, up, workspace)
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must hold segments + 1 entries")
    segments = offsets.shape[0] - 1
    lo = GemmLora(segments,
                  _device_vector(offsets, torch.int32, segments + 1, device, "offsets"),
                  _device_vector(ids, torch.int32, segments, device, "ids"), adapters, R,
                  _device_vector(scales, torch.float32, adapters, device, "scales"),
                  GEMM_OP_N if transDown == "N" else GEMM_OP_T, down.data_ptr(), ld_down,
                  stride_down, GEMM_OP_N if transUp == "N" else GEMM_OP_T, up.data_ptr(), ld_up,
                  stride_up)
    s = lib.gemm_run_lora(
        h, GEMM_OP_N if transB == "N" else GEMM_OP_T, M, N, K, alpha, A.data_ptr(), lda,
        B.data_ptr(), ldb, beta, c, ldc, D.data_ptr(), ldd, dtype, ctypes.byref(lo),
        workspace.data_ptr(), workspace.nbytes, _stream_on(device) if stream is None else stream)
    return _finish(s, check, "gemm_run_lora")
