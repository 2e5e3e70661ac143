"""ctypes binding of the lpgemm C-ABI (include/lpgemm.h).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, then their device pointers and the current HIP stream are handed
to the library.  Every step of the computation runs in the HIP kernels; there
is no fallback of any kind, and a missing library is an error.
"""
from __future__ import annotations

import collections
import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lpgemm.so")
CALLS_PATH = os.path.join(_PKG, "_tensor_calls.so")

# lpgemm_status
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_HIP, ERR_SCRATCH_LIMIT = 0, 1, 2, 3, 4
# lpgemm_kernel
KERNEL_AUTO, KERNEL_GENERAL, KERNEL_TILED, KERNEL_SKINNY = 0, 1, 2, 3
KERNEL_TILED_128, KERNEL_TILED_256, KERNEL_TILED_64, KERNEL_FP6 = 4, 5, 6, 7
KERNEL_NAMES = {KERNEL_AUTO: "auto", KERNEL_GENERAL: "general", KERNEL_TILED: "tiled",
                KERNEL_SKINNY: "skinny", KERNEL_FP6: "fp6"}
# lpgemm_variant
VARIANT_I4I4, VARIANT_W4A8 = 0, 1
# lpgemm_out_dtype
OUT_F32, OUT_BF16, OUT_F16, OUT_FP8_E4M3, OUT_FP8_E5M2 = 0, 1, 2, 3, 4
MAX_K = 131070

EXPORTS = ("lpgemm_int4_int4", "lpgemm_w4a8", "lpgemm_int4_int4_ws", "lpgemm_w4a8_ws",
           "lpgemm_int4_int4_noalloc",
           "lpgemm_workspace_size", "lpgemm_int4_int4_scaled", "lpgemm_w4a8_scaled",
           "lpgemm_int4_int4_scaled_ws", "lpgemm_int4_int4_blockscaled", "lpgemm_w4a8_blockscaled",
           "lpgemm_fp8_e4m3", "lpgemm_fp8_e5m2", "lpgemm_pack_int4",
           "lpgemm_unpack_int4", "lpgemm_status_string", "lpgemm_plan",
           "lpgemm_set_kernel_override", "lpgemm_mxfp4_quantize", "lpgemm_mxfp4_dequantize",
           "lpgemm_mxfp4", "lpgemm_mxfp4_workspace_size", "lpgemm_mxfp4_grouped", "lpgemm_mxfp4_plan",
           "lpgemm_fp8_block_quantize", "lpgemm_fp8_block_dequantize", "lpgemm_fp8_block",
           "lpgemm_fp8_block_grouped", "lpgemm_fp8_block_plan", "lpgemm_route", "lpgemm_route_workspace_size",
           "lpgemm_route_backward", "lpgemm_combine", "lpgemm_combine_backward")
SIZE_MAX = 2 ** 64 - 1
STATIC_SCRATCH_BYTES = 128 << 20  # LPGEMM_STATIC_SCRATCH_BYTES
WORKSPACE_ALIGN = 256
# microscaled 4-bit rows: units of 128 values, 64 code bytes and 4 scale bytes
MXFP4_UNIT, MXFP4_UNIT_CODES, MXFP4_UNIT_SCALES = 128, 64, 4
MXFP4_MAX_K, MXFP4_MAX_GROUPS = 1 << 20, 1024
# e4m3 rows with a scale per block of 128 values
FP8_BLOCK, FP8_BLOCK_MAX_K, FP8_BLOCK_MAX_GROUPS = 128, 1 << 20, 1024
# lpgemm_route_score, and the routing's limits
ROUTE_SCORES = {"softmax": 0, "sigmoid": 1}
ROUTE_MAX_EXPERTS, ROUTE_MAX_TOP, ROUTE_MAX_GROUPS = 1024, 32, 64
COMBINE_MAX_TOP, COMBINE_MAX_N = 1024, 1 << 24


class LpgemmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lpgemm_status_string(status)} (status {status})")


class PlanInfo(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("tile_m", ctypes.c_int32),
                ("tile_n", ctypes.c_int32), ("k_split", ctypes.c_int32),
                ("workgroups", ctypes.c_int64), ("threads", ctypes.c_int32),
                ("k_chunks", ctypes.c_int32), ("workspace_bytes", ctypes.c_int64)]

    def as_dict(self) -> dict:
        return {"kernel": KERNEL_NAMES.get(self.kernel, self.kernel), "tile_m": self.tile_m,
                "tile_n": self.tile_n, "k_split": self.k_split,
                "workgroups": self.workgroups, "threads": self.threads,
                "k_chunks": self.k_chunks, "workspace_bytes": self.workspace_bytes}


class RouteOptions(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("top", ctypes.c_int32), ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renormalise", ctypes.c_int32), ("scale", ctypes.c_float)]


# What lpgemm_route gives: experts and weights [T, top]; every expert's rows are
# offsets[e] .. offsets[e + 1] - 1, row i is token rows[i], and the token's k-th
# expert has it in row places[t, k].
Routing = collections.namedtuple("Routing", "experts weights rows offsets places")

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded HIP library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"the HIP library {LIB_PATH} is not built; run "
                          "`python -m precision_integer_gemm_amd.build` (or __graft_entry__.build())")
    # PyTorch brings its own HIP runtime: load it first, so that the library
    # binds to the same runtime as the streams and device pointers PyTorch
    # hands over (a second runtime loaded ahead of it leaves PyTorch without
    # a device).
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    L = ctypes.CDLL(LIB_PATH)
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    sz = ctypes.c_size_t
    for name in ("lpgemm_int4_int4", "lpgemm_w4a8", "lpgemm_int4_int4_noalloc"):
        f = getattr(L, name)
        f.argtypes = [p, p, p, i64, i64, i64, p]
        f.restype = ctypes.c_int
    for name in ("lpgemm_int4_int4_ws", "lpgemm_w4a8_ws"):
        f = getattr(L, name)
        f.argtypes = [p, p, p, i64, i64, i64, p, sz, p]
        f.restype = ctypes.c_int
    L.lpgemm_workspace_size.argtypes = [ctypes.c_int, i32, i64, i64, i64, i32, ctypes.POINTER(sz)]
    L.lpgemm_workspace_size.restype = ctypes.c_int
    for name in ("lpgemm_int4_int4_scaled", "lpgemm_w4a8_scaled"):
        f = getattr(L, name)
        f.argtypes = [p, p, p, p, p, ctypes.c_int, i64, i64, i64, p]
        f.restype = ctypes.c_int
    L.lpgemm_int4_int4_scaled_ws.argtypes = [p, p, p, p, p, ctypes.c_int, i64, i64, i64, p, sz, p]
    L.lpgemm_int4_int4_scaled_ws.restype = ctypes.c_int
    for name in ("lpgemm_int4_int4_blockscaled", "lpgemm_w4a8_blockscaled"):
        f = getattr(L, name)
        f.argtypes = [p, p, p, p, i64, p, ctypes.c_int, i64, i64, i64, p]
        f.restype = ctypes.c_int
    for name in ("lpgemm_fp8_e4m3", "lpgemm_fp8_e5m2"):
        getattr(L, name).argtypes = [p, p, p, ctypes.c_int, i64, i64, i64, p]
        getattr(L, name).restype = ctypes.c_int
    for name in ("lpgemm_pack_int4", "lpgemm_unpack_int4"):
        f = getattr(L, name)
        f.argtypes = [p, p, i64, i64, p]
        f.restype = ctypes.c_int
    L.lpgemm_mxfp4_quantize.argtypes = [p, ctypes.c_int, i64, p, p, i64, i64, p]
    L.lpgemm_mxfp4_dequantize.argtypes = [p, p, p, ctypes.c_int, i64, i64, p]
    L.lpgemm_mxfp4.argtypes = [p, p, p, p, p, ctypes.c_int, i64, i64, i64, p, sz, p]
    L.lpgemm_mxfp4_workspace_size.argtypes = [i64, i64, i64, i32, ctypes.POINTER(sz)]
    L.lpgemm_mxfp4_grouped.argtypes = [p, p, i64, p, p, p, i64, p, p, ctypes.c_int, i64, i64, i64, p]
    for name in ("lpgemm_mxfp4_quantize", "lpgemm_mxfp4_dequantize", "lpgemm_mxfp4",
                 "lpgemm_mxfp4_workspace_size", "lpgemm_mxfp4_grouped"):
        getattr(L, name).restype = ctypes.c_int
    L.lpgemm_fp8_block_quantize.argtypes = [p, ctypes.c_int, i64, i64, i32, p, p, i64, i64, p]
    L.lpgemm_fp8_block_dequantize.argtypes = [p, p, i64, p, ctypes.c_int, i64, i64, p]
    L.lpgemm_fp8_block.argtypes = [p, p, p, p, i64, p, ctypes.c_int, i64, i64, i64, p]
    L.lpgemm_fp8_block_grouped.argtypes = [p, p, i64, p, p, p, i64, i64, p, p, ctypes.c_int, i64, i64, i64, p]
    L.lpgemm_fp8_block_plan.argtypes = [i64, i64, i64, i64, i32, ctypes.POINTER(PlanInfo)]
    for name in ("lpgemm_fp8_block_quantize", "lpgemm_fp8_block_dequantize", "lpgemm_fp8_block",
                 "lpgemm_fp8_block_grouped", "lpgemm_fp8_block_plan"):
        getattr(L, name).restype = ctypes.c_int
    options = ctypes.POINTER(RouteOptions)
    L.lpgemm_route.argtypes = [p, ctypes.c_int, i64, p, options, p, p, p, p, p, i64, i64, p, sz, p]
    L.lpgemm_route_workspace_size.argtypes = [i64, i64, ctypes.POINTER(sz)]
    L.lpgemm_route_backward.argtypes = [p, p, ctypes.c_int, i64, p, options, p, i64, i64, p]
    L.lpgemm_combine.argtypes = [p, ctypes.c_int, i64, p, p, p, p, ctypes.c_int, i64, i64, i64, p]
    L.lpgemm_combine_backward.argtypes = [p, ctypes.c_int, p, ctypes.c_int, i64, p, p, p, p, i64, i64, i64, p]
    for name in ("lpgemm_route", "lpgemm_route_workspace_size", "lpgemm_route_backward", "lpgemm_combine", "lpgemm_combine_backward"):
        getattr(L, name).restype = ctypes.c_int
    L.lpgemm_status_string.argtypes = [ctypes.c_int]
    L.lpgemm_status_string.restype = ctypes.c_char_p
    L.lpgemm_plan.argtypes = [ctypes.c_int, p, p, p, i64, i64, i64, sz, i32, ctypes.POINTER(PlanInfo)]
    L.lpgemm_plan.restype = ctypes.c_int
    L.lpgemm_mxfp4_plan.argtypes = [i64, i64, i64, i64, i32, ctypes.POINTER(PlanInfo)]
    L.lpgemm_mxfp4_plan.restype = ctypes.c_int
    L.lpgemm_set_kernel_override.argtypes = [ctypes.c_int]
    L.lpgemm_set_kernel_override.restype = ctypes.c_int
    _lib = L
    return L


def lpgemm_status_string(status: int) -> str:
    return lib().lpgemm_status_string(int(status)).decode()


def _raise(status: int, what: str) -> None:
    if status != OK:
        raise LpgemmError(status, what)


def lpgemm_plan(variant: int, M: int, N: int, K: int, A: int = 256, B: int = 256, C: int = 256,
                cu_count: int = 0, workspace_bytes: int | None = None) -> dict:
    """Kernel and launch shape a call would use (host only; pointers are plain
    integers, inspected only for alignment).  workspace_bytes None: a call
    given all the workspace it can use; 0: a call without workspace."""
    info = PlanInfo()
    ws = SIZE_MAX if workspace_bytes is None else int(workspace_bytes)
    _raise(lib().lpgemm_plan(variant, A, B, C, M, N, K, ws, cu_count, ctypes.byref(info)),
           "lpgemm_plan")
    return info.as_dict()


def lpgemm_mxfp4_plan(R: int, N: int, K: int, E: int = 0, cu_count: int = 0) -> dict:
    """Kernel and launch shape of an mxfp4 product of R rows (E groups: of a
    grouped one with R rows of D), host only."""
    info = PlanInfo()
    _raise(lib().lpgemm_mxfp4_plan(R, N, K, E, cu_count, ctypes.byref(info)), "lpgemm_mxfp4_plan")
    return info.as_dict()


def lpgemm_workspace_size(variant: int, M: int, N: int, K: int, scaled: bool = False,
                          cu_count: int = 0) -> int:
    """Bytes of workspace a "_ws" call with these sizes can use (host only)."""
    n = ctypes.c_size_t(0)
    _raise(lib().lpgemm_workspace_size(variant, int(bool(scaled)), M, N, K, cu_count,
                                       ctypes.byref(n)), "lpgemm_workspace_size")
    return int(n.value)


def lpgemm_set_kernel_override(kernel: int) -> None:
    _raise(lib().lpgemm_set_kernel_override(int(kernel)), "lpgemm_set_kernel_override")


# ---- tensor-level calls ------------------------------------------------------
def _torch():
    import torch
    return torch


def _stream_handle(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check_dev(t, name: str, dtypes):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device, got {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _workspace(workspace, variant, M, N, K, scaled, device):
    """(pointer, bytes) of the workspace for a tensor-level call: "auto"
    allocates what the call can use through PyTorch's allocator (none when the
    call needs none), None passes none, a uint8 tensor on the device is used
    as given (aligned to 256 bytes inside it)."""
    torch = _torch()
    if workspace is None:
        return None, 0, None
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError('workspace must be "auto", None or a uint8 tensor')
        n = lpgemm_workspace_size(variant, M, N, K, scaled=scaled)
        if n == 0:
            return None, 0, None
        workspace = torch.empty(n + WORKSPACE_ALIGN, dtype=torch.uint8, device=device)
    if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 or \
            workspace.device.type != "cuda" or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 tensor on a GPU device")
    base = workspace.data_ptr()
    skip = (-base) % WORKSPACE_ALIGN
    n = max(0, workspace.numel() - skip)
    return (base + skip if n else None), n, workspace


def _out(out, M, N, device):
    torch = _torch()
    if out is None:
        return torch.empty((M, N), dtype=torch.int32, device=device)
    _check_dev(out, "out", (torch.int32,))
    if tuple(out.shape) != (M, N):
        raise ValueError(f"out must have shape ({M}, {N}), got {tuple(out.shape)}")
    return out


def lpgemm_int4_int4(A_packed, B_packed, *, out=None, workspace="auto", stream=None):
    """C[M,N] int32 = A . B^T with both operands packed int4 ([M,K/2], [N,K/2]).
    workspace: "auto" (allocated through PyTorch when the call can use one),
    None (the entry point without workspace) or a uint8 device tensor."""
    torch = _torch()
    _check_dev(A_packed, "A_packed", (torch.int8, torch.uint8))
    _check_dev(B_packed, "B_packed", (torch.int8, torch.uint8))
    M, half = A_packed.shape
    N, half_b = B_packed.shape
    if half != half_b:
        raise ValueError(f"packed K mismatch: A has {half} bytes per row, B {half_b}")
    C = _out(out, M, N, A_packed.device)
    ws, nws, _keep = _workspace(workspace, VARIANT_I4I4, M, N, 2 * half, False, A_packed.device)
    if nws:
        _raise(lib().lpgemm_int4_int4_ws(A_packed.data_ptr(), B_packed.data_ptr(), C.data_ptr(),
                                         M, N, 2 * half, ws, nws, _stream_handle(stream)),
               "lpgemm_int4_int4_ws")
    else:
        _raise(lib().lpgemm_int4_int4(A_packed.data_ptr(), B_packed.data_ptr(), C.data_ptr(),
                                      M, N, 2 * half, _stream_handle(stream)), "lpgemm_int4_int4")
    return C


def lpgemm_w4a8(A, B_packed, *, out=None, workspace="auto", stream=None):
    """C[M,N] int32 = A . B^T with A int8 [M,K] and B packed int4 [N,K/2];
    workspace as for lpgemm_int4_int4."""
    torch = _torch()
    _check_dev(A, "A", (torch.int8,))
    _check_dev(B_packed, "B_packed", (torch.uint8, torch.int8))
    M, K = A.shape
    N, half = B_packed.shape
    if K != 2 * half:
        raise ValueError(f"K mismatch: A has K={K}, B_packed holds {2 * half}")
    C = _out(out, M, N, A.device)
    ws, nws, _keep = _workspace(workspace, VARIANT_W4A8, M, N, K, False, A.device)
    if nws:
        _raise(lib().lpgemm_w4a8_ws(A.data_ptr(), B_packed.data_ptr(), C.data_ptr(), M, N, K,
                                    ws, nws, _stream_handle(stream)), "lpgemm_w4a8_ws")
    else:
        _raise(lib().lpgemm_w4a8(A.data_ptr(), B_packed.data_ptr(), C.data_ptr(), M, N, K,
                                 _stream_handle(stream)), "lpgemm_w4a8")
    return C


def _out_code(dtype):
    torch = _torch()
    codes = {torch.float32: OUT_F32, torch.bfloat16: OUT_BF16, torch.float16: OUT_F16}
    if dtype not in codes:
        raise TypeError(f"out dtype must be one of {list(codes)}, got {dtype}")
    return codes[dtype]


def _scaled_out(out, dtype, M, N, device):
    torch = _torch()
    if out is None:
        return torch.empty((M, N), dtype=dtype, device=device)
    _check_dev(out, "out", (dtype,))
    if tuple(out.shape) != (M, N):
        raise ValueError(f"out must have shape ({M}, {N}), got {tuple(out.shape)}")
    return out


def _check_scales(scale_a, scale_b, M, N):
    torch = _torch()
    for name, t, n in (("scale_a", scale_a, M), ("scale_b", scale_b, N)):
        if not isinstance(t, torch.Tensor) or t.device.type != "cuda" or t.dtype != torch.float32:
            raise TypeError(f"{name} must be a float32 tensor on a GPU device")
        if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous with shape ({n},)")


def lpgemm_int4_int4_scaled(A_packed, B_packed, scale_a, scale_b, *, dtype=None, out=None,
                            workspace="auto", stream=None):
    """D[M,N] = out(((float)C * scale_a[m]) * scale_b[n]) of the int4 x int4 product C;
    workspace as for lpgemm_int4_int4."""
    torch = _torch()
    _check_dev(A_packed, "A_packed", (torch.int8, torch.uint8))
    _check_dev(B_packed, "B_packed", (torch.int8, torch.uint8))
    M, half = A_packed.shape
    N, half_b = B_packed.shape
    if half != half_b:
        raise ValueError(f"packed K mismatch: A has {half} bytes per row, B {half_b}")
    _check_scales(scale_a, scale_b, M, N)
    dtype = dtype or (out.dtype if out is not None else torch.bfloat16)
    D = _scaled_out(out, dtype, M, N, A_packed.device)
    ws, nws, _keep = _workspace(workspace, VARIANT_I4I4, M, N, 2 * half, True, A_packed.device)
    if nws:
        _raise(lib().lpgemm_int4_int4_scaled_ws(A_packed.data_ptr(), B_packed.data_ptr(),
                                                scale_a.data_ptr(), scale_b.data_ptr(),
                                                D.data_ptr(), _out_code(dtype), M, N, 2 * half,
                                                ws, nws, _stream_handle(stream)),
               "lpgemm_int4_int4_scaled_ws")
    else:
        _raise(lib().lpgemm_int4_int4_scaled(A_packed.data_ptr(), B_packed.data_ptr(),
                                             scale_a.data_ptr(), scale_b.data_ptr(), D.data_ptr(),
                                             _out_code(dtype), M, N, 2 * half,
                                             _stream_handle(stream)),
               "lpgemm_int4_int4_scaled")
    return D


def lpgemm_w4a8_scaled(A, B_packed, scale_a, scale_b, *, dtype=None, out=None, stream=None):
    """D[M,N] = out(((float)C * scale_a[m]) * scale_b[n]) of the W4A8 product C."""
    torch = _torch()
    _check_dev(A, "A", (torch.int8,))
    _check_dev(B_packed, "B_packed", (torch.uint8, torch.int8))
    M, K = A.shape
    N, half = B_packed.shape
    if K != 2 * half:
        raise ValueError(f"K mismatch: A has K={K}, B_packed holds {2 * half}")
    _check_scales(scale_a, scale_b, M, N)
    dtype = dtype or (out.dtype if out is not None else torch.bfloat16)
    D = _scaled_out(out, dtype, M, N, A.device)
    _raise(lib().lpgemm_w4a8_scaled(A.data_ptr(), B_packed.data_ptr(), scale_a.data_ptr(),
                                    scale_b.data_ptr(), D.data_ptr(), _out_code(dtype), M, N, K,
                                    _stream_handle(stream)), "lpgemm_w4a8_scaled")
    return D


def _check_block_scales(SFA, SFB, M, N, K, g):
    torch = _torch()
    nb = -(-K // g) if g > 0 else 0
    for name, t, n in (("SFA", SFA, M), ("SFB", SFB, N)):
        if not isinstance(t, torch.Tensor) or t.device.type != "cuda" or t.dtype != torch.float32:
            raise TypeError(f"{name} must be a float32 tensor on a GPU device")
        if tuple(t.shape) != (n, nb) or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous with shape ({n}, {nb}) for K={K}, g={g}")


def lpgemm_int4_int4_blockscaled(A_packed, B_packed, SFA, SFB, g, *, dtype=None, out=None, stream=None):
    """D[M,N] = out(sum_j ((float)C_j * SFA[m,j]) * SFB[n,j]) over the K blocks
    of g (a power of two >= 32) of the int4 x int4 product, added in block order
    in binary32; SFA [M, ceil(K/g)], SFB [N, ceil(K/g)] float32."""
    torch = _torch()
    _check_dev(A_packed, "A_packed", (torch.int8, torch.uint8))
    _check_dev(B_packed, "B_packed", (torch.int8, torch.uint8))
    M, half = A_packed.shape
    N, half_b = B_packed.shape
    if half != half_b:
        raise ValueError(f"packed K mismatch: A has {half} bytes per row, B {half_b}")
    _check_block_scales(SFA, SFB, M, N, 2 * half, g)
    dtype = dtype or (out.dtype if out is not None else torch.bfloat16)
    D = _scaled_out(out, dtype, M, N, A_packed.device)
    _raise(lib().lpgemm_int4_int4_blockscaled(A_packed.data_ptr(), B_packed.data_ptr(), SFA.data_ptr(),
                                              SFB.data_ptr(), g, D.data_ptr(), _out_code(dtype), M, N,
                                              2 * half, _stream_handle(stream)),
           "lpgemm_int4_int4_blockscaled")
    return D


def lpgemm_w4a8_blockscaled(A, B_packed, SFA, SFB, g, *, dtype=None, out=None, stream=None):
    """lpgemm_int4_int4_blockscaled for int8 A [M, K] and packed int4 B."""
    torch = _torch()
    _check_dev(A, "A", (torch.int8,))
    _check_dev(B_packed, "B_packed", (torch.uint8, torch.int8))
    M, K = A.shape
    N, half = B_packed.shape
    if K != 2 * half:
        raise ValueError(f"K mismatch: A has K={K}, B_packed holds {2 * half}")
    _check_block_scales(SFA, SFB, M, N, K, g)
    dtype = dtype or (out.dtype if out is not None else torch.bfloat16)
    D = _scaled_out(out, dtype, M, N, A.device)
    _raise(lib().lpgemm_w4a8_blockscaled(A.data_ptr(), B_packed.data_ptr(), SFA.data_ptr(), SFB.data_ptr(),
                                         g, D.data_ptr(), _out_code(dtype), M, N, K, _stream_handle(stream)),
           "lpgemm_w4a8_blockscaled")
    return D


def _fp8_gemm(name, f8_name, own_code, A, B, dtype, out, stream):
    torch = _torch()
    f8 = getattr(torch, f8_name, None)
    ok = (torch.uint8,) + ((f8,) if f8 is not None else ())
    _check_dev(A, "A", ok)
    _check_dev(B, "B", ok)
    M, K = A.shape
    N, K_b = B.shape
    if K != K_b:
        raise ValueError(f"K mismatch: A has K={K}, B has {K_b}")
    dtype = dtype or (out.dtype if out is not None else torch.float32)
    if dtype == torch.float32:
        code = OUT_F32
    elif dtype in ok:
        code = own_code
    else:
        raise TypeError(f"dtype must be torch.float32, torch.uint8 or torch.{f8_name}")
    if out is None:
        C = torch.empty((M, N), dtype=dtype, device=A.device)
    else:
        _check_dev(out, "out", (dtype,))
        if tuple(out.shape) != (M, N):
            raise ValueError(f"out must have shape ({M}, {N}), got {tuple(out.shape)}")
        C = out
    _raise(getattr(lib(), name)(A.data_ptr(), B.data_ptr(), C.data_ptr(), code, M, N, K,
                                _stream_handle(stream)), name)
    return C


def lpgemm_fp8_e4m3(A, B, *, dtype=None, out=None, stream=None):
    """C[M,N] = A . B^T of e4m3 operands (uint8 codes or torch.float8_e4m3fn
    tensors [M,K] and [N,K]) with fp32 accumulation; C as float32 (default) or
    e4m3 codes (dtype=torch.uint8 or torch.float8_e4m3fn)."""
    return _fp8_gemm("lpgemm_fp8_e4m3", "float8_e4m3fn", OUT_FP8_E4M3, A, B, dtype, out, stream)


def lpgemm_fp8_e5m2(A, B, *, dtype=None, out=None, stream=None):
    """C[M,N] = A . B^T of e5m2 operands (uint8 codes or torch.float8_e5m2
    tensors [M,K] and [N,K]) with fp32 accumulation; C as float32 (default) or
    e5m2 codes (dtype=torch.uint8 or torch.float8_e5m2)."""
    return _fp8_gemm("lpgemm_fp8_e5m2", "float8_e5m2", OUT_FP8_E5M2, A, B, dtype, out, stream)


def lpgemm_pack_int4(logical, *, out=None, stream=None):
    """Logical int4 values held as int8 [rows, K] -> packed uint8 [rows, K/2]."""
    torch = _torch()
    _check_dev(logical, "logical", (torch.int8,))
    rows, K = logical.shape
    if K % 2:
        raise ValueError("the last dimension of a logical int4 tensor must be even")
    if out is None:
        out = torch.empty((rows, K // 2), dtype=torch.uint8, device=logical.device)
    else:
        _check_dev(out, "out", (torch.uint8, torch.int8))
        if tuple(out.shape) != (rows, K // 2):
            raise ValueError("out has the wrong shape")
    _raise(lib().lpgemm_pack_int4(logical.data_ptr(), out.data_ptr(), rows, K,
                                  _stream_handle(stream)), "lpgemm_pack_int4")
    return out


def lpgemm_unpack_int4(packed, *, out=None, stream=None):
    """Packed bytes [rows, K/2] -> logical int4 values as int8 [rows, K]."""
    torch = _torch()
    _check_dev(packed, "packed", (torch.uint8, torch.int8))
    rows, half = packed.shape
    if out is None:
        out = torch.empty((rows, 2 * half), dtype=torch.int8, device=packed.device)
    else:
        _check_dev(out, "out", (torch.int8,))
        if tuple(out.shape) != (rows, 2 * half):
            raise ValueError("out has the wrong shape")
    _raise(lib().lpgemm_unpack_int4(packed.data_ptr(), out.data_ptr(), rows, 2 * half,
                                    _stream_handle(stream)), "lpgemm_unpack_int4")
    return out


# ---- microscaled 4-bit floating point ------------------------------------------
# These calls take a few microseconds on the device for a token's work, so what
# the host does before a launch is kept short.
_mx = None  # torch, the library, the result types' codes and the native calls, once all are loaded


class _LongWay:
    """In the native calls' place where they are not built: every call goes through the checks here."""
    quantize = dequantize = product = grouped = staticmethod(lambda *args: None)
    block_quantize = block_dequantize = block_product = block_grouped = route = combine = quantize


def _mx_torch():
    global _mx
    if _mx is None:
        torch = _torch()
        library = lib()
        calls = _LongWay
        if os.path.exists(CALLS_PATH):  # one that does not load is an error
            from . import _tensor_calls as calls
        _mx = (torch, library, {torch.float32: OUT_F32, torch.bfloat16: OUT_BF16, torch.float16: OUT_F16}, calls)
    return _mx[0]


def _mx_launch(function, index, stream, *args):
    """Calls a library function on the tensors' device: on `stream`, or that device's current one."""
    torch = _mx[0]
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return _mx_launch(function, index, stream, *args)
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    status = function(*args, handle)
    if status != OK:
        _raise(status, function.__name__)


def _units(K: int) -> int:
    return -(-K // MXFP4_UNIT)


def _check_on(t, name: str, dtypes, dim: int, device=None):
    """A dense tensor of the library's: type, rank, device (`device`: the other operands')."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if t.dim() != dim:
        raise ValueError(f"{name} must be {dim}-D, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _mx_units(codes, scales, name: str, dim: int, device=None):
    """Units per row of an mxfp4 operand.  One expression passes what is right;
    what is not goes through the checks that say what is wrong."""
    u8 = _mx_torch().uint8
    try:
        c, s = codes.shape, scales.shape
        units = c[-1] // MXFP4_UNIT_CODES
        if (codes.dtype is u8 and scales.dtype is u8 and codes.is_cuda and len(c) == dim and c[:-1] == s[:-1]
                and units * MXFP4_UNIT_CODES == c[-1] and units * MXFP4_UNIT_SCALES == s[-1] and codes.is_contiguous()
                and scales.is_contiguous() and scales.device == (device or codes.device) and (device is None or codes.device == device)):
            return units
    except (AttributeError, IndexError):
        pass
    return _check_mx(codes, scales, name, dim, device)


def _check_mx(codes, scales, name: str, dim: int, device=None):
    torch = _torch()
    _check_on(codes, name, (torch.uint8,), dim, device)
    _check_on(scales, f"scales of {name}", (torch.uint8,), dim, codes.device)
    units, rest = divmod(codes.shape[-1], MXFP4_UNIT_CODES)
    if rest or tuple(scales.shape) != (*codes.shape[:-1], MXFP4_UNIT_SCALES * units):
        raise ValueError(f"{name} must have shape (..., {MXFP4_UNIT_CODES} U) and its scales (..., {MXFP4_UNIT_SCALES} U), "
                         f"got {tuple(codes.shape)} and {tuple(scales.shape)}")
    return units


def _mx_out(out, dtype, M, N, device):
    torch, codes = _mx[0], _mx[2]
    if out is None:
        dtype = dtype or torch.bfloat16
        code = codes.get(dtype)
        if code is None:
            raise TypeError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
        return torch.empty((M, N), dtype=dtype, device=device), code
    _check_on(out, "out", (dtype,) if dtype else tuple(codes), 2, device)
    if tuple(out.shape) != (M, N):
        raise ValueError(f"out must have shape ({M}, {N}), got {tuple(out.shape)}")
    return out, codes[out.dtype]


def lpgemm_mxfp4_quantize(x, *, codes=None, scales=None, stream=None):
    """Rows of float32, bfloat16 or float16 values [rows, K] -> (codes uint8
    [rows, 64 U], scales uint8 [rows, 4 U]) with U = ceil(K / 128): e2m1 codes
    and one e8m0 scale byte per 32 values.  Rows of x may be strided (its last
    dimension is dense)."""
    torch = _mx_torch()
    if codes is None and scales is None and stream is None:
        made = _mx[3].quantize(x)
        if made is not None:
            return made
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    code = _mx[2].get(x.dtype)
    if code is None:
        raise TypeError(f"x must be float32, bfloat16 or float16, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got shape {tuple(x.shape)}")
    if not x.is_cuda:
        raise ValueError(f"x must be on a GPU device, got {x.device}")
    rows, K = x.shape
    ldx, step = x.stride()
    if (K > 1 and step != 1) or (rows > 1 and ldx < K):
        raise ValueError(f"x must be dense along its last dimension, its rows apart: strides {x.stride()}")
    U = _units(K)
    device = x.device
    if codes is None:
        codes = torch.empty((rows, MXFP4_UNIT_CODES * U), dtype=torch.uint8, device=device)
    else:
        _check_shape(codes, "codes", (rows, MXFP4_UNIT_CODES * U), device)
    if scales is None:
        scales = torch.empty((rows, MXFP4_UNIT_SCALES * U), dtype=torch.uint8, device=device)
    else:
        _check_shape(scales, "scales", (rows, MXFP4_UNIT_SCALES * U), device)
    _mx_launch(_mx[1].lpgemm_mxfp4_quantize, device.index, stream, x.data_ptr(), code, ldx, codes.data_ptr(),
               scales.data_ptr(), rows, K)
    return codes, scales


def _check_shape(t, name: str, shape, device):
    _check_on(t, name, (_torch().uint8,), 2, device)
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")


def lpgemm_mxfp4_dequantize(codes, scales, K, *, dtype=None, out=None, stream=None):
    """The values [rows, K] that mxfp4 codes and scales stand for (bfloat16 by
    default; exact in float32 and bfloat16)."""
    _mx_torch()
    if out is None and stream is None:
        made = _mx[3].dequantize(codes, scales, K, dtype)
        if made is not None:
            return made
    units = _mx_units(codes, scales, "codes", 2)
    if K < 0 or _units(K) != units:
        raise ValueError(f"K={K} does not fit {units} units of {MXFP4_UNIT} values")
    device, rows = codes.device, codes.shape[0]
    out, code = _mx_out(out, dtype, rows, K, device)
    _mx_launch(_mx[1].lpgemm_mxfp4_dequantize, device.index, stream, codes.data_ptr(), scales.data_ptr(), out.data_ptr(),
               code, rows, K)
    return out


def lpgemm_mxfp4_workspace_size(M: int, N: int, K: int, cu_count: int = 0) -> int:
    """Bytes of workspace an lpgemm_mxfp4 call with these sizes can use (host only)."""
    n = ctypes.c_size_t(0)
    _raise(lib().lpgemm_mxfp4_workspace_size(M, N, K, cu_count, ctypes.byref(n)), "lpgemm_mxfp4_workspace_size")
    return int(n.value)


def lpgemm_mxfp4(A, SFA, B, SFB, *, dtype=None, out=None, workspace="auto", stream=None):
    """D[M,N] = A . B^T of mxfp4 operands (codes [M, 64 U] and [N, 64 U], scales
    [M, 4 U] and [N, 4 U]) with fp32 accumulation, as bfloat16 (default),
    float16 or float32.  workspace: "auto", None or a uint8 device tensor, as
    for lpgemm_int4_int4; no kernel takes scratch memory at present."""
    _mx_torch()
    if out is None and stream is None and isinstance(workspace, str) and workspace == "auto":
        made = _mx[3].product(A, SFA, B, SFB, dtype)
        if made is not None:
            return made
    units = _mx_units(A, SFA, "A", 2)
    device = A.device
    if _mx_units(B, SFB, "B", 2, device) != units:
        raise ValueError(f"K mismatch: A has {A.shape[1]} bytes per row, B {B.shape[1]}")
    M, N, K = A.shape[0], B.shape[0], MXFP4_UNIT * units
    D, code = _mx_out(out, dtype, M, N, device)
    if isinstance(workspace, str) and workspace == "auto":
        workspace = None  # no kernel takes one
    ws, nws, _keep = _workspace(workspace, None, M, N, K, True, device)
    _mx_launch(_mx[1].lpgemm_mxfp4, device.index, stream, A.data_ptr(), SFA.data_ptr(), B.data_ptr(), SFB.data_ptr(),
               D.data_ptr(), code, M, N, K, ws, nws)
    return D


def lpgemm_mxfp4_grouped(A, SFA, B, SFB, offsets, *, rows=None, dtype=None, out=None, stream=None):
    """The product of each group of rows with its own matrix: row i of the result,
    offsets[e] <= i < offsets[e + 1], is row rows[i] of A times B[e]^T (rows
    None: row i; an index outside A's rows stands for zeros).  A codes [T, 64 U],
    B codes [E, N, 64 U], offsets int32 [E + 1] and rows int32 on the device.
    Rows that no group holds are not written: without `out` they are whatever
    the new tensor's memory held."""
    _mx_torch()
    if out is None and stream is None:
        made = _mx[3].grouped(A, SFA, B, SFB, offsets, rows, dtype)
        if made is not None:
            return made
    units = _mx_units(A, SFA, "A", 2)
    device = A.device
    if _mx_units(B, SFB, "B", 3, device) != units:
        raise ValueError(f"K mismatch: A has {A.shape[1]} bytes per row, B {B.shape[2]}")
    E, N = B.shape[0], B.shape[1]
    int32 = (_mx[0].int32,)
    _check_on(offsets, "offsets", int32, 1, device)
    if offsets.shape[0] != E + 1:
        raise ValueError(f"offsets must have {E + 1} entries for {E} groups, got {offsets.shape[0]}")
    T = R = A.shape[0]
    index = None
    if rows is not None:
        _check_on(rows, "rows", int32, 1, device)
        R, index = rows.shape[0], rows.data_ptr()
    D, code = _mx_out(out, dtype, R, N, device)
    _mx_launch(_mx[1].lpgemm_mxfp4_grouped, device.index, stream, A.data_ptr(), SFA.data_ptr(), T, index, B.data_ptr(),
               SFB.data_ptr(), E, offsets.data_ptr(), D.data_ptr(), code, R, N, MXFP4_UNIT * units)
    return D


# ---- e4m3 with a scale per block of 128 ------------------------------------------
def _f8_types():
    torch = _torch()
    return (torch.float8_e4m3fn, torch.uint8)


def _check_f8(codes, scales, name: str, dim: int, device=None):
    """(units per row, rows that share a scale) of an fp8_block operand."""
    torch = _torch()
    _check_on(codes, name, _f8_types(), dim, device)
    _check_on(scales, f"scales of {name}", (torch.float32,), dim, codes.device)
    units, rest = divmod(codes.shape[-1], FP8_BLOCK)
    *lead, rows = codes.shape[:-1]
    for block_rows in (1, FP8_BLOCK):
        if not rest and tuple(scales.shape) == (*lead, -(-rows // block_rows), units):
            return units, block_rows
    raise ValueError(f"{name} must have shape (..., rows, {FP8_BLOCK} U) and its scales (..., rows or ceil(rows / {FP8_BLOCK}), U), "
                     f"got {tuple(codes.shape)} and {tuple(scales.shape)}")


def lpgemm_fp8_block_quantize(x, *, block_rows=1, power_of_two=False, codes=None, scales=None, stream=None):
    """Rows of float32, bfloat16 or float16 values [rows, K] -> (codes float8_e4m3fn
    [rows, 128 U], scales float32 [ceil(rows / block_rows), U]) with U = ceil(K /
    128): one scale for each block of 128 values of a row (block_rows 1:
    activations) or of 128 x 128 values (block_rows 128: weights), the block's
    largest magnitude / 448, or with power_of_two the power of two above that.
    Rows of x may be strided (its last dimension is dense)."""
    torch = _mx_torch()
    if codes is None and scales is None and stream is None:
        made = _mx[3].block_quantize(x, block_rows, power_of_two)
        if made is not None:
            return made
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    code = _mx[2].get(x.dtype)
    if code is None:
        raise TypeError(f"x must be float32, bfloat16 or float16, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got shape {tuple(x.shape)}")
    if block_rows not in (1, FP8_BLOCK):
        raise ValueError(f"block_rows must be 1 or {FP8_BLOCK}, got {block_rows}")
    if not x.is_cuda:
        raise ValueError(f"x must be on a GPU device, got {x.device}")
    rows, K = x.shape
    ldx, step = x.stride()
    if (K > 1 and step != 1) or (rows > 1 and ldx < K):
        raise ValueError(f"x must be dense along its last dimension, its rows apart: strides {x.stride()}")
    U, device = -(-K // FP8_BLOCK), x.device
    if codes is None:
        codes = torch.empty((rows, FP8_BLOCK * U), dtype=torch.float8_e4m3fn, device=device)
    else:
        _check_given(codes, "codes", _f8_types(), (rows, FP8_BLOCK * U), device)
    shape = (-(-rows // block_rows), U)
    if scales is None:
        scales = torch.empty(shape, dtype=torch.float32, device=device)
    else:
        _check_given(scales, "scales", (torch.float32,), shape, device)
    _mx_launch(_mx[1].lpgemm_fp8_block_quantize, device.index, stream, x.data_ptr(), code, ldx, block_rows, int(bool(power_of_two)),
               codes.data_ptr(), scales.data_ptr(), rows, K)
    return codes, scales


def _check_given(t, name: str, dtypes, shape, device):
    _check_on(t, name, dtypes, len(shape), device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def lpgemm_fp8_block_dequantize(codes, scales, K, *, dtype=None, out=None, stream=None):
    """The values [rows, K] that codes and their scales (per row or per 128 rows)
    stand for, as bfloat16 (default), float16 or float32."""
    _mx_torch()
    if out is None and stream is None:
        made = _mx[3].block_dequantize(codes, scales, K, dtype)
        if made is not None:
            return made
    units, block_rows = _check_f8(codes, scales, "codes", 2)
    if K < 0 or -(-K // FP8_BLOCK) != units:
        raise ValueError(f"K={K} does not fit {units} blocks of {FP8_BLOCK} values")
    device, rows = codes.device, codes.shape[0]
    out, code = _mx_out(out, dtype, rows, K, device)
    _mx_launch(_mx[1].lpgemm_fp8_block_dequantize, device.index, stream, codes.data_ptr(), scales.data_ptr(), block_rows, out.data_ptr(), code, rows, K)
    return out


def lpgemm_fp8_block(A, SFA, B, SFB, *, dtype=None, out=None, stream=None):
    """D[M,N] = sum over blocks of 128 k of SFA[m,j] SFB[n,j] (A_j . B_j^T): codes
    float8_e4m3fn or uint8 [M, 128 U] and [N, 128 U], scales float32 [M, U] and
    [N, U] or [ceil(N / 128), U]; D as bfloat16 (default), float16 or float32 (at
    about half the speed: sums good to binary32)."""
    _mx_torch()
    if out is None and stream is None:
        made = _mx[3].block_product(A, SFA, B, SFB, dtype)
        if made is not None:
            return made
    units, block_rows = _check_f8(A, SFA, "A", 2)
    M = A.shape[0]
    if block_rows != 1:
        raise ValueError(f"A must have a scale for every row and block: shape ({M}, {units}), got {tuple(SFA.shape)}")
    device = A.device
    units_b, block_rows = _check_f8(B, SFB, "B", 2, device)
    if units_b != units:
        raise ValueError(f"K mismatch: A has {A.shape[1]} codes per row, B {B.shape[1]}")
    N = B.shape[0]
    D, code = _mx_out(out, dtype, M, N, device)
    _mx_launch(_mx[1].lpgemm_fp8_block, device.index, stream, A.data_ptr(), SFA.data_ptr(), B.data_ptr(), SFB.data_ptr(), block_rows, D.data_ptr(),
               code, M, N, FP8_BLOCK * units)
    return D


def lpgemm_fp8_block_grouped(A, SFA, B, SFB, offsets, *, rows=None, dtype=None, out=None, stream=None):
    """lpgemm_fp8_block of each group of rows with its own matrix: row i of the
    result, offsets[e] <= i < offsets[e + 1], is row rows[i] of A times B[e]^T (rows
    None: row i; an index outside A's rows stands for zeros).  A codes [T, 128 U], B
    codes [E, N, 128 U] with scales [E, N, U] or [E, ceil(N / 128), U]; offsets int32
    [E + 1] and rows int32 on the device, as lpgemm_route gives them.  Rows that no
    group holds are not written: without `out` they are whatever the new tensor's
    memory held."""
    _mx_torch()
    if out is None and stream is None:
        made = _mx[3].block_grouped(A, SFA, B, SFB, offsets, rows, dtype)
        if made is not None:
            return made
    units, block_rows = _check_f8(A, SFA, "A", 2)
    T = R = A.shape[0]
    if block_rows != 1:
        raise ValueError(f"A must have a scale for every row and block: shape ({T}, {units}), got {tuple(SFA.shape)}")
    device = A.device
    units_b, block_rows = _check_f8(B, SFB, "B", 3, device)
    if units_b != units:
        raise ValueError(f"K mismatch: A has {A.shape[1]} codes per row, B {B.shape[2]}")
    E, N = B.shape[0], B.shape[1]
    int32 = (_mx[0].int32,)
    _check_given(offsets, "offsets", int32, (E + 1,), device)
    index = None
    if rows is not None:
        _check_on(rows, "rows", int32, 1, device)
        R, index = rows.shape[0], rows.data_ptr()
    D, code = _mx_out(out, dtype, R, N, device)
    _mx_launch(_mx[1].lpgemm_fp8_block_grouped, device.index, stream, A.data_ptr(), SFA.data_ptr(), T, index, B.data_ptr(), SFB.data_ptr(), block_rows,
               E, offsets.data_ptr(), D.data_ptr(), code, R, N, FP8_BLOCK * units)
    return D


def lpgemm_fp8_block_plan(R: int, N: int, K: int, E: int = 0, cu_count: int = 0) -> dict:
    """Kernel and launch shape of an fp8_block product of R rows (E groups: of a
    grouped one with R rows of D), host only."""
    info = PlanInfo()
    _raise(lib().lpgemm_fp8_block_plan(R, N, K, E, cu_count, ctypes.byref(info)), "lpgemm_fp8_block_plan")
    return info.as_dict()


# ---- experts: routing and the sum of a token's -----------------------------------
def _route_options(top, score, groups, top_groups, group_top, renormalise, scale):
    if score not in ROUTE_SCORES:
        raise ValueError(f"score must be one of {list(ROUTE_SCORES)}, got {score!r}")
    sizes = {"top": top, "groups": groups, "top_groups": groups if top_groups is None else top_groups, "group_top": group_top}
    for name, v in sizes.items():
        if not -2 ** 31 <= v < 2 ** 31:  # the structure's fields would keep its low bits
            raise ValueError(f"{name}={v} is out of range")
    return RouteOptions(ROUTE_SCORES[score], *sizes.values(), int(bool(renormalise)), scale)


def _route_logits(logits):
    """(type code, row stride) of [T, E] logits; their rows may be strided."""
    torch = _mx_torch()
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    code = _mx[2].get(logits.dtype)
    if code is None:
        raise TypeError(f"logits must be float32, bfloat16 or float16, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError(f"logits must be 2-D, got shape {tuple(logits.shape)}")
    if not logits.is_cuda:
        raise ValueError(f"logits must be on a GPU device, got {logits.device}")
    (T, E), (ld, step) = logits.shape, logits.stride()
    if (E > 1 and step != 1) or (T > 1 and ld < E):
        raise ValueError(f"logits must be dense along their last dimension, their rows apart: strides {logits.stride()}")
    return code, ld


def lpgemm_route_workspace_size(T: int, E: int) -> int:
    """Bytes of workspace an lpgemm_route call with these sizes needs (host only)."""
    n = ctypes.c_size_t(0)
    _raise(lib().lpgemm_route_workspace_size(T, E, ctypes.byref(n)), "lpgemm_route_workspace_size")
    return int(n.value)


def lpgemm_route(logits, top, *, score="softmax", bias=None, groups=1, top_groups=None, group_top=2, renormalise=True, scale=1.0,
                 workspace="auto", stream=None):
    """Routing of logits [T, E] (float32, bfloat16 or float16; -inf closes an expert)
    to each token's `top` experts: Routing(experts int32 [T, top], weights float32 [T,
    top], rows int32 [T * top], offsets int32 [E + 1], places int32 [T, top]).

    Scores are the softmax of a row or sigmoids; `bias` float32 [E] is added for the
    choice alone.  With `groups` of neighbouring experts, each scored by the sum of
    its `group_top` (1 or 2) best choice scores, the experts of the `top_groups`
    best stay.  Ties go to the lowest index.  A token's weights are its experts'
    scores, divided by their sum (renormalise), times `scale`.  `rows` and `offsets`
    are what the grouped products take, `places` what lpgemm_combine does; where a
    token finds no `top` open experts, the others are -1 with weight 0.  The work-
    space is allocated ("auto") or a uint8 device tensor."""
    torch = _mx_torch()
    if stream is None and isinstance(workspace, str) and workspace == "auto":
        made = _mx[3].route(logits, top, ROUTE_SCORES.get(score), bias, groups, groups if top_groups is None else top_groups, group_top, renormalise, scale)
        if made is not None:
            return tuple.__new__(Routing, made)
    code, ld = _route_logits(logits)
    T, E = logits.shape
    device = logits.device
    if bias is not None:
        _check_given(bias, "bias", (torch.float32,), (E,), device)
    options = _route_options(top, score, groups, top_groups, group_top, renormalise, scale)
    if not 1 <= top <= ROUTE_MAX_TOP:
        raise ValueError(f"top must be 1 .. {ROUTE_MAX_TOP}, got {top}")
    need = lpgemm_route_workspace_size(T, E)
    if isinstance(workspace, str) and workspace == "auto":
        workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
        if need and stream is not None:  # freed here, in use there
            workspace.record_stream(stream)
    elif workspace is not None:
        _check_on(workspace, "workspace", (torch.uint8,), 1, device)
    ints = torch.empty(3 * T * top + E + 1, dtype=torch.int32, device=device)
    experts, places, rows = ints[:T * top].view(T, top), ints[T * top:2 * T * top].view(T, top), ints[2 * T * top:3 * T * top]
    offsets = ints[3 * T * top:]
    weights = torch.empty((T, top), dtype=torch.float32, device=device)
    _mx_launch(_mx[1].lpgemm_route, device.index, stream, logits.data_ptr(), code, ld, None if bias is None else bias.data_ptr(), ctypes.byref(options),
               experts.data_ptr(), weights.data_ptr(), rows.data_ptr(), offsets.data_ptr(), places.data_ptr(), T, E,
               None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel())
    return Routing(experts, weights, rows, offsets, places)


def lpgemm_route_backward(dweights, logits, experts, *, score="softmax", renormalise=True, scale=1.0, out=None, stream=None):
    """The gradient of the logits [T, E], of their type, from that of lpgemm_route's
    weights (dweights float32 [T, top]); experts as it gave them, score, renormalise
    and scale as it took them.  The choice itself has no gradient."""
    torch = _mx_torch()
    code, ld = _route_logits(logits)
    T, E = logits.shape
    device = logits.device
    _check_on(experts, "experts", (torch.int32,), 2, device)
    top = experts.shape[1]
    if experts.shape[0] != T:
        raise ValueError(f"experts must have {T} rows, got {experts.shape[0]}")
    _check_given(dweights, "dweights", (torch.float32,), (T, top), device)
    options = _route_options(top, score, 1, 1, 1, renormalise, scale)
    if out is None:
        out = torch.empty((T, E), dtype=logits.dtype, device=device)
    else:
        _check_given(out, "out", (logits.dtype,), (T, E), device)
    _mx_launch(_mx[1].lpgemm_route_backward, device.index, stream, dweights.data_ptr(), logits.data_ptr(), code, ld, experts.data_ptr(),
               ctypes.byref(options), out.data_ptr(), T, E)
    return out


def _combine_operands(y, places, weights):
    torch = _mx_torch()
    _check_on(y, "y", tuple(_mx[2]), 2)
    device = y.device
    _check_on(places, "places", (torch.int32,), 2, device)
    if weights is not None:
        _check_given(weights, "weights", (torch.float32,), places.shape, device)
    return device, *places.shape, *y.shape


def lpgemm_combine(y, places, weights=None, *, residual=None, dtype=None, out=None, stream=None):
    """out[t] = residual[t] + sum_k weights[t, k] y[places[t, k]]: the rows of y [R, N]
    (float32, bfloat16 or float16) that belong to a token, added in float32 in order;
    places int32 [T, top] (outside y's rows: nothing is added), weights float32 [T,
    top] (None: ones), residual [T, N] of the result's type.  The result's type is
    y's unless `dtype` or `out` says otherwise."""
    _mx_torch()
    if out is None and stream is None:
        made = _mx[3].combine(y, places, weights, residual, dtype)
        if made is not None:
            return made
    device, T, top, R, N = _combine_operands(y, places, weights)
    if dtype is None and out is None:
        dtype = y.dtype
    out, code = _mx_out(out, dtype, T, N, device)
    if residual is not None:
        _check_given(residual, "residual", (out.dtype,), (T, N), device)
    _mx_launch(_mx[1].lpgemm_combine, device.index, stream, y.data_ptr(), _mx[2][y.dtype], R, places.data_ptr(),
               None if weights is None else weights.data_ptr(), None if residual is None else residual.data_ptr(), out.data_ptr(), code, T, top, N)
    return out


def lpgemm_combine_backward(dout, y, places, weights=None, *, dy=None, stream=None):
    """lpgemm_combine's gradients (dy [R, N] of y's type, dweights float32 [T, top])
    from dout [T, N]; the residual's is dout.  Rows of dy that are in no place are not
    written (without `dy` they are whatever the new tensor's memory held); no row may
    be in two."""
    device, T, top, R, N = _combine_operands(y, places, weights)
    torch = _mx[0]
    _check_given(dout, "dout", tuple(_mx[2]), (T, N), device)
    if dy is None:
        dy = torch.empty_like(y)
    else:
        _check_given(dy, "dy", (y.dtype,), (R, N), device)
    dweights = torch.empty((T, top), dtype=torch.float32, device=device)
    _mx_launch(_mx[1].lpgemm_combine_backward, device.index, stream, dout.data_ptr(), _mx[2][dout.dtype], y.data_ptr(), _mx[2][y.dtype], R,
               places.data_ptr(), None if weights is None else weights.data_ptr(), dy.data_ptr(), dweights.data_ptr(), T, top, N)
    return dy, dweights
