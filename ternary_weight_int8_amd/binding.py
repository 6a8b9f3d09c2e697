"""Python binding of libternary_gemm.so: argument marshalling only.

Every product runs in the library's HIP kernels.  There is no fallback: if the
library is missing or a call fails, these functions raise.  PyTorch supplies
device memory and the current stream; the library never allocates.  A call
launches on the current HIP device, which has to be its tensors' (one process a
GPU); the layer norm, the gated layer and the product with int8 weights refuse
tensors of another, the other calls leave that to the caller.
"""
from __future__ import annotations

import ctypes
import os
from array import array

from .build import LIB

OK = 0
ERR_NULL, ERR_DIM, ERR_PACK, ERR_BOUND, ERR_ALIAS, ERR_HIP, ERR_KIND, ERR_SCRATCH = -1, -2, -3, -4, -5, -6, -7, -8
ERR_VALUE, ERR_WORKSPACE = -9, -10
STATIC_SCRATCH_BYTES = 8 << 20   # TGEMM_STATIC_SCRATCH_BYTES
OUT_F32, OUT_BF16 = 1, 2   # output kinds of the scaled calls
IN_F32, IN_BF16 = 1, 2     # input kinds of the quantizer calls
ACTS = {"none": 0, "relu": 1, "relu2": 2, "silu": 3, "gelu_tanh": 4}   # TGEMM_ACT_*

# entry points declared in include/ternary_gemm.h
EXPORTS = (
    "ternary_gemm_s8",
    "ternary_gemm_s8_dx",
    "ternary_gemm_s8_dw",
    "ternary_gemm_status_str",
    "ternary_gemm_plan",
    "ternary_gemm_plan_on",
    "ternary_gemm_machine",
    "ternary_gemm_tile_of",
    "ternary_gemm_s8_scaled",
    "ternary_gemm_s8_dx_scaled",
    "ternary_gemm_s8_dw_scaled",
    "ternary_pack_weights",
    "ternary_quantize_rows",
    "ternary_quantize_cols",
    "ternary_gemm_s8_dx_ws",
    "ternary_gemm_s8_dx_scaled_ws",
    "ternary_gemm_dx_workspace",
    "ternary_gemm_s8_dx_noalloc",
    "ternary_rmsnorm_quantize",
    "ternary_rmsnorm_backward",
    "ternary_rmsnorm_backward_workspace",
    "ternary_gemm_s8_epilogue",
    "ternary_epilogue_backward",
    "ternary_epilogue_backward_workspace",
    "ternary_clip_grad_norm",
    "ternary_clip_grad_norm_workspace",
    "ternary_gemm_epilogue_plan",
    "ternary_layernorm_quantize",
    "ternary_layernorm_backward",
    "ternary_layernorm_backward_workspace",
    "ternary_gated_backward",
    "ternary_gated_backward_workspace",
    "ternary_gemm_s8s8_epilogue",
    "ternary_gemm_s8s8_workspace",
    "ternary_gemm_s8_gated",
    "ternary_gemm_s8_gated_workspace",
    "ternary_gemm_s8s8_plan",
    "ternary_gemm_s8_gated_plan",
)

OPS = {"fwd": 0, "dx": 1, "dw": 2}


class TgemmPlan(ctypes.Structure):
    _fields_ = [
        ("out_rows", ctypes.c_int64), ("out_cols", ctypes.c_int64), ("contraction", ctypes.c_int64),
        ("tile_rows", ctypes.c_int32), ("tile_cols", ctypes.c_int32),
        ("tiles", ctypes.c_int64),
        ("workgroups", ctypes.c_int64),
        ("tiles_per_workgroup", ctypes.c_int64),
        ("band_cols", ctypes.c_int32),
        ("threads_per_workgroup", ctypes.c_int32), ("lds_bytes", ctypes.c_int32),
        ("fast_path", ctypes.c_int32), ("kernel", ctypes.c_int32),
        ("xcds", ctypes.c_int32),
    ]


KERNEL_TILED, KERNEL_SPLIT, KERNEL_STREAM, KERNEL_SKINNY, KERNEL_RING = 0, 2, 3, 4, 5   # TgemmPlan.kernel
KERNEL_INT8, KERNEL_INT8_FEW = 6, 7


class TernaryGemmError(RuntimeError):
    def __init__(self, name, status, msg):
        super().__init__(f"{name}: status {status}: {msg}")
        self.status = status


_lib = None


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise RuntimeError(
                f"{LIB} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB)
        p, i64 = ctypes.c_void_p, ctypes.c_int64
        for name in EXPORTS[:3]:
            f = getattr(L, name)
            f.argtypes = [p, p, p, i64, i64, i64, p]
            f.restype = ctypes.c_int
        L.ternary_gemm_status_str.argtypes = [ctypes.c_int]
        L.ternary_gemm_status_str.restype = ctypes.c_char_p
        L.ternary_gemm_plan.argtypes = [ctypes.c_int, i64, i64, i64, i64, ctypes.POINTER(TgemmPlan)]
        L.ternary_gemm_plan.restype = ctypes.c_int
        L.ternary_gemm_plan_on.argtypes = [ctypes.c_int, i64, i64, i64, i64, ctypes.c_int32, ctypes.c_int32,
                                           ctypes.POINTER(TgemmPlan)]
        L.ternary_gemm_plan_on.restype = ctypes.c_int
        L.ternary_gemm_machine.argtypes = [ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]
        L.ternary_gemm_machine.restype = ctypes.c_int
        L.ternary_gemm_tile_of.argtypes = [ctypes.POINTER(TgemmPlan), i64, i64,
                                           ctypes.POINTER(i64), ctypes.POINTER(i64)]
        L.ternary_gemm_tile_of.restype = ctypes.c_int
        f32, i32 = ctypes.c_float, ctypes.c_int
        for name in ("ternary_gemm_s8_scaled", "ternary_gemm_s8_dx_scaled"):
            f = getattr(L, name)
            f.argtypes = [p, p, p, f32, p, i32, i64, i64, i64, p]
            f.restype = ctypes.c_int
        L.ternary_gemm_s8_dw_scaled.argtypes = [p, p, p, p, p, i32, i64, i64, i64, p]
        L.ternary_gemm_s8_dw_scaled.restype = ctypes.c_int
        L.ternary_pack_weights.argtypes = [p, p, i64, i64, p]
        L.ternary_pack_weights.restype = ctypes.c_int
        for name in ("ternary_quantize_rows", "ternary_quantize_cols"):
            f = getattr(L, name)
            f.argtypes = [p, i32, p, p, i64, i64, p]
            f.restype = ctypes.c_int
        L.ternary_gemm_s8_dx_ws.argtypes = [p, p, p, i64, i64, i64, p, i64, p]
        L.ternary_gemm_s8_dx_ws.restype = ctypes.c_int
        L.ternary_gemm_s8_dx_scaled_ws.argtypes = [p, p, p, f32, p, i32, i64, i64, i64, p, i64, p]
        L.ternary_gemm_s8_dx_scaled_ws.restype = ctypes.c_int
        L.ternary_gemm_s8_dx_noalloc.argtypes = [p, p, p, i64, i64, i64, p]
        L.ternary_gemm_s8_dx_noalloc.restype = ctypes.c_int
        L.ternary_gemm_dx_workspace.argtypes = [i64, i64, i64, i64, ctypes.POINTER(i64)]
        L.ternary_gemm_dx_workspace.restype = ctypes.c_int
        pi64 = ctypes.POINTER(i64)
        for name, args in (
                ("ternary_rmsnorm_quantize", [p, i32, p, p, f32, p, p, p, p, p, i64, i64, p]),
                ("ternary_rmsnorm_backward", [p, p, i32, p, p, p, p, p, i64, i64, p, i64, p]),
                ("ternary_rmsnorm_backward_workspace", [i64, i64, pi64]),
                ("ternary_gemm_s8_epilogue", [p, p, p, f32, p, i32, p, p, p, i32, i64, i64, i64, p]),
                ("ternary_epilogue_backward", [p, p, i32, i32, p, p, p, p, i64, i64, p, i64, p]),
                ("ternary_epilogue_backward_workspace", [i64, i64, pi64]),
                ("ternary_clip_grad_norm", [p, p, p, p, i64, f32, f32, p, p, i64, p]),
                ("ternary_clip_grad_norm_workspace", [p, i64, pi64]),
                ("ternary_gemm_epilogue_plan", [i64, i64, i64, i64, i32, i32, ctypes.POINTER(TgemmPlan)]),
                ("ternary_layernorm_quantize", [p, i32, p, p, p, f32, p, p, p, p, p, p, i64, i64, p]),
                ("ternary_layernorm_backward", [p, p, i32, p, p, p, p, p, p, p, i64, i64, p, i64, p]),
                ("ternary_layernorm_backward_workspace", [i64, i64, pi64]),
                ("ternary_gated_backward", [p, p, i32, i32, f32, f32, p, p, p, p, i64, i64, p, i64, p]),
                ("ternary_gated_backward_workspace", [i64, i64, pi64]),
                ("ternary_gemm_s8s8_epilogue", [p, p, p, p, p, i32, p, p, p, i32, i64, i64, i64, p, i64, p]),
                ("ternary_gemm_s8s8_workspace", [i64, i64, i64, i64, pi64]),
                ("ternary_gemm_s8_gated", [p, p, p, f32, f32, p, i32, p, p, i32, i64, i64, i64, p, i64, p]),
                ("ternary_gemm_s8_gated_workspace", [i64, i64, i64, i64, pi64]),
                ("ternary_gemm_s8s8_plan", [i64, i64, i64, i64, i32, i32, i32, i32, i32, i32, ctypes.POINTER(TgemmPlan)]),
                ("ternary_gemm_s8_gated_plan", [i64, i64, i64, i64, i32, i32, i32, i32, i32, ctypes.POINTER(TgemmPlan)])):
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        _lib = L
    return _lib


def status_str(status: int) -> str:
    return lib().ternary_gemm_status_str(int(status)).decode()


def call_raw(name: str, p0, p1, p2, M: int, N: int, K: int, stream=None) -> int:
    """Call an entry point with raw addresses (ints or None); returns its status."""
    return getattr(lib(), name)(p0, p1, p2, M, N, K, stream)


def call_raw_scaled(name: str, p0, p1, s0, s1, out, kind: int, M: int, N: int, K: int, stream=None) -> int:
    """Call a scaled entry point with raw addresses; s1 is the weight scale
    (a float) for the forward and dX, the dC column scales' address for dW."""
    return getattr(lib(), name)(p0, p1, s0, s1, out, kind, M, N, K, stream)


def ternary_gemm_dx_workspace(M: int, N: int, K: int, align: int = 256) -> int:
    """Workspace bytes the dX calls with a workspace use (0: the one-pass kernels run)."""
    b = ctypes.c_int64()
    st = lib().ternary_gemm_dx_workspace(M, N, K, align, ctypes.byref(b))
    if st != OK:
        raise TernaryGemmError("ternary_gemm_dx_workspace", st, status_str(st))
    return b.value


def machine():
    """(compute units, XCDs) of the current HIP device, as the calls plan for it."""
    cus, xcds = ctypes.c_int32(), ctypes.c_int32()
    st = lib().ternary_gemm_machine(ctypes.byref(cus), ctypes.byref(xcds))
    if st != OK:
        raise TernaryGemmError("ternary_gemm_machine", st, status_str(st))
    return cus.value, xcds.value


def plan(op: str, M: int, N: int, K: int, align: int = 256, cus: int = None, xcds: int = None):
    """The launch plan of a call, for MI355X (256 CUs, 8 XCDs) unless cus and
    xcds name another machine."""
    pl = TgemmPlan()
    if cus is None and xcds is None:
        st = lib().ternary_gemm_plan(OPS[op], M, N, K, align, ctypes.byref(pl))
    else:
        st = lib().ternary_gemm_plan_on(OPS[op], M, N, K, align, cus, xcds, ctypes.byref(pl))
    if st != OK:
        raise TernaryGemmError("ternary_gemm_plan", st, status_str(st))
    return pl


def epilogue_plan(M: int, N: int, K: int, align: int = 256, cus: int = 256, xcds: int = 8):
    """The launch plan of ternary_gemm_s8_epilogue, for MI355X unless cus and xcds name another machine."""
    pl = TgemmPlan()
    _done("ternary_gemm_epilogue_plan",
          lib().ternary_gemm_epilogue_plan(M, N, K, align, cus, xcds, ctypes.byref(pl)))
    return pl


def s8s8_plan(M: int, N: int, K: int, align: int = 256, act: str = "none", residual: bool = False, save: bool = False,
              kind: int = OUT_BF16, cus: int = 256, xcds: int = 8):
    """The launch plan of ternary_gemm_s8s8_epilogue, for MI355X unless cus and xcds name another machine."""
    pl = TgemmPlan()
    _done("ternary_gemm_s8s8_plan",
          lib().ternary_gemm_s8s8_plan(M, N, K, align, _act(act), residual, save, kind, cus, xcds, ctypes.byref(pl)))
    return pl


def gated_plan(M: int, N: int, K: int, align: int = 256, act: str = "silu", save: bool = False, kind: int = OUT_BF16,
               cus: int = 256, xcds: int = 8):
    """The launch plan of ternary_gemm_s8_gated, for MI355X unless cus and xcds name another machine."""
    pl = TgemmPlan()
    _done("ternary_gemm_s8_gated_plan",
          lib().ternary_gemm_s8_gated_plan(M, N, K, align, _act(act), save, kind, cus, xcds, ctypes.byref(pl)))
    return pl


def tile_of(pl: TgemmPlan, workgroup: int, iteration: int = 0):
    """(row0, col0) of the tile a workgroup computes in one iteration, or None if none."""
    r, c = ctypes.c_int64(), ctypes.c_int64()
    st = lib().ternary_gemm_tile_of(ctypes.byref(pl), workgroup, iteration, ctypes.byref(r),
                                    ctypes.byref(c))
    if st == ERR_DIM and 0 <= workgroup < pl.workgroups and 0 <= iteration < pl.tiles_per_workgroup:
        return None
    if st != OK:
        raise TernaryGemmError("ternary_gemm_tile_of", st, status_str(st))
    return r.value, c.value


# ---------------------------------------------------------------------------
# torch-tensor wrappers (same names as the C entry points)
# ---------------------------------------------------------------------------

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _check(t, dtype, ndim, what):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{what} must be {ndim}-D, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def _stream(stream, device):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _invoke(name, a, b, out, M, N, K, stream):
    st = getattr(lib(), name)(a.data_ptr(), b.data_ptr(), out.data_ptr(), M, N, K,
                              _stream(stream, out.device))
    if st != OK:
        raise TernaryGemmError(name, st, status_str(st))
    return out


def ternary_gemm_s8(A, Wpacked, C=None, stream=None):
    """C int32 [M][N] = A int8 [M][K] x W, W stored as uint8 [N][K/4]."""
    torch = _torch()
    _check(A, torch.int8, 2, "A")
    _check(Wpacked, torch.uint8, 2, "Wpacked")
    M, K = A.shape
    N = Wpacked.shape[0]
    if Wpacked.shape[1] * 4 != K:
        raise ValueError(f"Wpacked must be [N][K/4] = [{N}][{K // 4}], got {tuple(Wpacked.shape)}")
    if C is None:
        C = torch.empty((M, N), dtype=torch.int32, device=A.device)
    _check(C, torch.int32, 2, "C")
    if tuple(C.shape) != (M, N):
        raise ValueError(f"C must be [{M}][{N}]")
    return _invoke("ternary_gemm_s8", A, Wpacked, C, M, N, K, stream)


def ternary_gemm_s8_dx(dC, Wpacked, K, dX=None, stream=None):
    """dX int32 [M][K] = dC int8 [M][N] x W^T, same stored W as the forward."""
    torch = _torch()
    _check(dC, torch.int8, 2, "dC")
    _check(Wpacked, torch.uint8, 2, "Wpacked")
    M, N = dC.shape
    if tuple(Wpacked.shape) != (N, K // 4) or K % 4:
        raise ValueError(f"Wpacked must be [N][K/4] = [{N}][{K // 4}], got {tuple(Wpacked.shape)}")
    if dX is None:
        dX = torch.empty((M, K), dtype=torch.int32, device=dC.device)
    _check(dX, torch.int32, 2, "dX")
    if tuple(dX.shape) != (M, K):
        raise ValueError(f"dX must be [{M}][{K}]")
    return _invoke("ternary_gemm_s8_dx", dC, Wpacked, dX, M, N, K, stream)


def _lowbit(addr: int) -> int:
    return addr & -addr if addr else 1 << 20


def _workspace(workspace, M, N, K, dC, Wpacked, stream):
    """The caller's workspace (a contiguous uint8 device tensor), or a new one
    of the size the library asks for; (address, bytes)."""
    torch = _torch()
    if workspace is None:
        align = min(_lowbit(dC.data_ptr()), _lowbit(Wpacked.data_ptr()))
        nbytes = ternary_gemm_dx_workspace(M, N, K, align)
        if nbytes == 0:
            return None, 0, None
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dC.device)
        if stream is not None:
            workspace.record_stream(stream)   # freed here, in use on `stream`
    _check(workspace, torch.uint8, workspace.dim(), "workspace")
    if workspace.device != dC.device:
        raise ValueError(f"workspace must be on {dC.device}, got {workspace.device}")
    if workspace.numel() == 0:
        return None, 0, workspace
    return workspace.data_ptr(), workspace.numel(), workspace


def ternary_gemm_s8_dx_ws(dC, Wpacked, K, workspace=None, dX=None, stream=None):
    """ternary_gemm_s8_dx with a workspace (a contiguous uint8 device tensor of
    at least ternary_gemm_dx_workspace() bytes, empty for none; None: one of
    that size is allocated here)."""
    torch = _torch()
    _check(dC, torch.int8, 2, "dC")
    _check(Wpacked, torch.uint8, 2, "Wpacked")
    M, N = dC.shape
    if tuple(Wpacked.shape) != (N, K // 4) or K % 4:
        raise ValueError(f"Wpacked must be [N][K/4] = [{N}][{K // 4}], got {tuple(Wpacked.shape)}")
    dX = _output(dX, (M, K), torch.int32, dC.device, "dX")
    ws, nbytes, _keep = _workspace(workspace, M, N, K, dC, Wpacked, stream)
    st = lib().ternary_gemm_s8_dx_ws(dC.data_ptr(), Wpacked.data_ptr(), dX.data_ptr(), M, N, K, ws, nbytes,
                                     _stream(stream, dX.device))
    if st != OK:
        raise TernaryGemmError("ternary_gemm_s8_dx_ws", st, status_str(st))
    return dX


def ternary_gemm_s8_dx_noalloc(dC, Wpacked, K, dX=None, stream=None):
    """ternary_gemm_s8_dx with the library's static device scratch in place of
    a workspace (the C call allocates nothing; dX is allocated here when not
    given)."""
    torch = _torch()
    _check(dC, torch.int8, 2, "dC")
    _check(Wpacked, torch.uint8, 2, "Wpacked")
    M, N = dC.shape
    if tuple(Wpacked.shape) != (N, K // 4) or K % 4:
        raise ValueError(f"Wpacked must be [N][K/4] = [{N}][{K // 4}], got {tuple(Wpacked.shape)}")
    dX = _output(dX, (M, K), torch.int32, dC.device, "dX")
    st = lib().ternary_gemm_s8_dx_noalloc(dC.data_ptr(), Wpacked.data_ptr(), dX.data_ptr(), M, N, K,
                                          _stream(stream, dX.device))
    if st != OK:
        raise TernaryGemmError("ternary_gemm_s8_dx_noalloc", st, status_str(st))
    return dX


def ternary_gemm_s8_dw(A, dC, dW=None, stream=None):
    """dW int32 [K][N] = A^T x dC, A int8 [M][K], dC int8 [M][N]."""
    torch = _torch()
    _check(A, torch.int8, 2, "A")
    _check(dC, torch.int8, 2, "dC")
    M, K = A.shape
    if dC.shape[0] != M:
        raise ValueError("A and dC must have the same number of rows")
    N = dC.shape[1]
    if dW is None:
        dW = torch.empty((K, N), dtype=torch.int32, device=A.device)
    _check(dW, torch.int32, 2, "dW")
    if tuple(dW.shape) != (K, N):
        raise ValueError(f"dW must be [{K}][{N}]")
    return _invoke("ternary_gemm_s8_dw", A, dC, dW, M, N, K, stream)


# ---------------------------------------------------------------------------
# scaled outputs: the integer product times per-row and per-column scales,
# stored as float32 or bfloat16
# ---------------------------------------------------------------------------

def _out_kind(dtype):
    torch = _torch()
    if dtype == torch.float32:
        return OUT_F32
    if dtype == torch.bfloat16:
        return OUT_BF16
    raise TypeError(f"out_dtype must be torch.float32 or torch.bfloat16, got {dtype}")


def _scales(t, n, what):
    torch = _torch()
    _check(t, torch.float32, 1, what)
    if t.shape[0] != n:
        raise ValueError(f"{what} must have {n} entries, got {t.shape[0]}")


def _output(out, shape, dtype, device, what):
    torch = _torch()
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
    _check(out, dtype, 2, what)
    if tuple(out.shape) != shape:
        raise ValueError(f"{what} must be {list(shape)}")
    return out


def ternary_gemm_s8_scaled(A, Wpacked, a_row_scale, w_scale, out_dtype=None, Y=None, stream=None):
    """Y [M][N] = (float(A x W) * a_row_scale[m]) * w_scale, float32 or bfloat16."""
    torch = _torch()
    out_dtype = out_dtype or torch.bfloat16
    _check(A, torch.int8, 2, "A")
    _check(Wpacked, torch.uint8, 2, "Wpacked")
    M, K = A.shape
    N = Wpacked.shape[0]
    if Wpacked.shape[1] * 4 != K:
        raise ValueError(f"Wpacked must be [N][K/4] = [{N}][{K // 4}], got {tuple(Wpacked.shape)}")
    _scales(a_row_scale, M, "a_row_scale")
    Y = _output(Y, (M, N), out_dtype, A.device, "Y")
    st = lib().ternary_gemm_s8_scaled(A.data_ptr(), Wpacked.data_ptr(), a_row_scale.data_ptr(),
                                      float(w_scale), Y.data_ptr(), _out_kind(out_dtype), M, N, K,
                                      _stream(stream, Y.device))
    if st != OK:
        raise TernaryGemmError("ternary_gemm_s8_scaled", st, status_str(st))
    return Y


def ternary_gemm_s8_dx_scaled(dC, Wpacked, K, dc_row_scale, w_scale, out_dtype=None, dX=None,
                              stream=None):
    """dX [M][K] = (float(dC x W^T) * dc_row_scale[m]) * w_scale, float32 or bfloat16."""
    torch = _torch()
    out_dtype = out_dtype or torch.bfloat16
    _check(dC, torch.int8, 2, "dC")
    _check(Wpacked, torch.uint8, 2, "Wpacked")
    M, N = dC.shape
    if tuple(Wpacked.shape) != (N, K // 4) or K % 4:
        raise ValueError(f"Wpacked must be [N][K/4] = [{N}][{K // 4}], got {tuple(Wpacked.shape)}")
    _scales(dc_row_scale, M, "dc_row_scale")
    dX = _output(dX, (M, K), out_dtype, dC.device, "dX")
    st = lib().ternary_gemm_s8_dx_scaled(dC.data_ptr(), Wpacked.data_ptr(), dc_row_scale.data_ptr(),
                                         float(w_scale), dX.data_ptr(), _out_kind(out_dtype), M, N, K,
                                         _stream(stream, dX.device))
    if st != OK:
        raise TernaryGemmError("ternary_gemm_s8_dx_scaled", st, status_str(st))
    return dX


def ternary_gemm_s8_dx_scaled_ws(dC, Wpacked, K, dc_row_scale, w_scale, out_dtype=None, workspace=None,
                                 dX=None, stream=None):
    """ternary_gemm_s8_dx_scaled with a workspace, as ternary_gemm_s8_dx_ws."""
    torch = _torch()
    out_dtype = out_dtype or torch.bfloat16
    _check(dC, torch.int8, 2, "dC")
    _check(Wpacked, torch.uint8, 2, "Wpacked")
    M, N = dC.shape
    if tuple(Wpacked.shape) != (N, K // 4) or K % 4:
        raise ValueError(f"Wpacked must be [N][K/4] = [{N}][{K // 4}], got {tuple(Wpacked.shape)}")
    _scales(dc_row_scale, M, "dc_row_scale")
    dX = _output(dX, (M, K), out_dtype, dC.device, "dX")
    ws, nbytes, _keep = _workspace(workspace, M, N, K, dC, Wpacked, stream)
    st = lib().ternary_gemm_s8_dx_scaled_ws(dC.data_ptr(), Wpacked.data_ptr(), dc_row_scale.data_ptr(),
                                            float(w_scale), dX.data_ptr(), _out_kind(out_dtype), M, N, K,
                                            ws, nbytes, _stream(stream, dX.device))
    if st != OK:
        raise TernaryGemmError("ternary_gemm_s8_dx_scaled_ws", st, status_str(st))
    return dX


def ternary_gemm_s8_dw_scaled(A, dC, a_col_scale, dc_col_scale, out_dtype=None, dW=None, stream=None):
    """dW [K][N] = (float(A^T x dC) * a_col_scale[k]) * dc_col_scale[n], float32 or bfloat16."""
    torch = _torch()
    out_dtype = out_dtype or torch.bfloat16
    _check(A, torch.int8, 2, "A")
    _check(dC, torch.int8, 2, "dC")
    M, K = A.shape
    if dC.shape[0] != M:
        raise ValueError("A and dC must have the same number of rows")
    N = dC.shape[1]
    _scales(a_col_scale, K, "a_col_scale")
    _scales(dc_col_scale, N, "dc_col_scale")
    dW = _output(dW, (K, N), out_dtype, A.device, "dW")
    st = lib().ternary_gemm_s8_dw_scaled(A.data_ptr(), dC.data_ptr(), a_col_scale.data_ptr(),
                                         dc_col_scale.data_ptr(), dW.data_ptr(), _out_kind(out_dtype),
                                         M, N, K, _stream(stream, dW.device))
    if st != OK:
        raise TernaryGemmError("ternary_gemm_s8_dw_scaled", st, status_str(st))
    return dW


# ---------------------------------------------------------------------------
# the steps before the product: packing the trainer's ternary weights, and
# per-row / per-column int8 quantization of activations
# ---------------------------------------------------------------------------

def ternary_pack_weights(Wt, Wpacked=None, stream=None):
    """Wpacked uint8 [N][K/4] from int8 weights Wt [N][K] (codes by sign)."""
    torch = _torch()
    _check(Wt, torch.int8, 2, "Wt")
    N, K = Wt.shape
    Wpacked = _output(Wpacked, (N, K // 4), torch.uint8, Wt.device, "Wpacked")
    st = lib().ternary_pack_weights(Wt.data_ptr(), Wpacked.data_ptr(), N, K, _stream(stream, Wt.device))
    if st != OK:
        raise TernaryGemmError("ternary_pack_weights", st, status_str(st))
    return Wpacked


def _quantize(name, X, Q, scale, n_scale, stream):
    torch = _torch()
    if not isinstance(X, torch.Tensor) or X.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("X must be a float32 or bfloat16 torch.Tensor")
    _check(X, X.dtype, 2, "X")
    R, C = X.shape
    Q = _output(Q, (R, C), torch.int8, X.device, "Q")
    n = R if n_scale == "rows" else C
    if scale is None:
        scale = torch.empty((n,), dtype=torch.float32, device=X.device)
    _scales(scale, n, "scale")
    kind = IN_F32 if X.dtype == torch.float32 else IN_BF16
    st = getattr(lib(), name)(X.data_ptr(), kind, Q.data_ptr(), scale.data_ptr(), R, C,
                              _stream(stream, X.device))
    if st != OK:
        raise TernaryGemmError(name, st, status_str(st))
    return Q, scale


def ternary_quantize_rows(X, Q=None, scale=None, stream=None):
    """(Q int8 [R][C], scale float32 [R]): per-row symmetric int8 quantization of X [R][C]."""
    return _quantize("ternary_quantize_rows", X, Q, scale, "rows", stream)


def ternary_quantize_cols(X, Q=None, scale=None, stream=None):
    """(Q int8 [R][C], scale float32 [C]): per-column symmetric int8 quantization of X [R][C]."""
    return _quantize("ternary_quantize_cols", X, Q, scale, "cols", stream)


# ---------------------------------------------------------------------------
# the operators around the product: norm, epilogue, their backward passes, and
# the clipping of gradients
# ---------------------------------------------------------------------------

def _kind(t, what):
    """The kind of a float matrix (IN_* and OUT_* have the same values)."""
    torch = _torch()
    if isinstance(t, torch.Tensor):
        if t.dtype == torch.float32:
            return IN_F32
        if t.dtype == torch.bfloat16:
            return IN_BF16
    raise TypeError(f"{what} must be a float32 or bfloat16 torch.Tensor")


def _given(t, dtype, shape, device, what):
    """An argument that has to have this type, shape and device (a GPU's)."""
    try:
        if t.dtype == dtype and t.shape == shape and t.device == device and t.is_contiguous():
            return t
    except AttributeError:   # not a tensor: _check says so
        pass
    _check(t, dtype, len(shape), what)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what} must be on {device}, got {t.device}")
    return t


def _made(t, dtype, shape, device, what, stream):
    """The caller's output, or a new one.  A new one comes from the pool of the
    stream the kernels run on, so that no pending work of another stream still
    uses its memory."""
    if t is not None:
        return _given(t, dtype, shape, device, what)
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _like(t, x, stream, what, dtype=None):
    """The caller's output of x's shape and of dtype (x's), or a new one."""
    dtype = dtype or x.dtype
    if t is None and stream is None:
        return _torch().empty_like(x, dtype=dtype)
    return _made(t, dtype, x.shape, x.device, what, stream)


def _scratch(workspace, nbytes, device, stream):
    """The caller's workspace (a contiguous uint8 device tensor), or a new one;
    None if the call needs none."""
    torch = _torch()
    if workspace is None:
        return _made(None, torch.uint8, (nbytes,), device, "workspace", stream) if nbytes else None
    _check(workspace, torch.uint8, 1, "workspace")
    if workspace.device != device:
        raise ValueError(f"workspace must be on {device}, got {workspace.device}")
    return workspace


def _raw_stream(stream, device):
    """The handle of `stream`, or of the device's current one (the direct
    query where this torch has it: making a Stream object takes 2 us)."""
    if stream is not None:
        return stream.cuda_stream
    torch = _torch()
    query = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch.cuda.current_stream(device).cuda_stream if query is None else query(device.index)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _done(name, st):
    if st != OK:
        raise TernaryGemmError(name, st, status_str(st))


def _queried(name, *args):
    b = ctypes.c_int64()
    _done(name, getattr(lib(), name)(*args, ctypes.byref(b)))
    return b.value


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act must be one of {', '.join(ACTS)}, got {act!r}")
    return ACTS[act]


def ternary_rmsnorm_quantize(X, gain, eps=1e-6, residual=None, save=False, H=None, Y=None, rstd=None, Q=None,
                             scale=None, stream=None):
    """RMS norm of h = X + residual [R][C] (float32 or bfloat16) into the int8
    rows that the product takes: (Q int8 [R][C], scale float32 [R], H, Y, rstd).

    H is h in X's type (given as `H`, it may be X or residual; X itself without
    a residual).  With `save`, Y [R][C] in X's type holds the normed values
    h * rstd * gain and rstd float32 [R] the rows' 1 / rms, for the backward
    pass; without, both are None."""
    torch = _torch()
    kind = _kind(X, "X")
    _check(X, X.dtype, 2, "X")
    (R, C), dt, dev = X.shape, X.dtype, X.device
    _given(gain, torch.float32, (C,), dev, "gain")
    if residual is not None:
        _given(residual, dt, X.shape, dev, "residual")
        H = _like(H, X, stream, "H")
    elif H is not None and H is not X:
        raise ValueError("H is given without a residual: it would be X")
    if not save and (Y is not None or rstd is not None):
        raise ValueError("Y and rstd are outputs of save=True")
    if save:
        Y = _like(Y, X, stream, "Y")
        rstd = _made(rstd, torch.float32, (R,), dev, "rstd", stream)
    Q = _like(Q, X, stream, "Q", torch.int8)
    scale = _made(scale, torch.float32, (R,), dev, "scale", stream)
    _done("ternary_rmsnorm_quantize",
          lib().ternary_rmsnorm_quantize(X.data_ptr(), kind, _ptr(residual), gain.data_ptr(), eps,
                                         None if residual is None else H.data_ptr(), _ptr(Y), _ptr(rstd),
                                         Q.data_ptr(), scale.data_ptr(), R, C, _raw_stream(stream, dev)))
    return Q, scale, X if residual is None else H, Y, rstd


def ternary_rmsnorm_backward(dY, H, gain, rstd, dH=None, dX=None, dgain=None, workspace=None, stream=None):
    """(dX [R][C] in H's type, dgain float32 [C]) from the gradient dY of the
    normed values, the H and rstd that the norm kept and, with a residual
    stream, the gradient dH that reaches H past the norm (dX may be dH)."""
    torch = _torch()
    kind = _kind(H, "H")
    _check(H, H.dtype, 2, "H")
    (R, C), dt, dev = H.shape, H.dtype, H.device
    _given(dY, dt, (R, C), dev, "dY")
    _given(gain, torch.float32, (C,), dev, "gain")
    _given(rstd, torch.float32, (R,), dev, "rstd")
    if dH is not None:
        _given(dH, dt, (R, C), dev, "dH")
    dX = _like(dX, H, stream, "dX")
    dgain = _like(dgain, gain, stream, "dgain")
    ws = _scratch(workspace, _queried("ternary_rmsnorm_backward_workspace", R, C), dev, stream)
    _done("ternary_rmsnorm_backward",
          lib().ternary_rmsnorm_backward(dY.data_ptr(), H.data_ptr(), kind, gain.data_ptr(), rstd.data_ptr(),
                                         _ptr(dH), dX.data_ptr(), dgain.data_ptr(), R, C, _ptr(ws),
                                         0 if ws is None else ws.numel(), _raw_stream(stream, dev)))
    return dX, dgain


def ternary_gemm_s8_epilogue(A, Wpacked, a_row_scale, w_scale, bias=None, act="none", residual=None, out_dtype=None,
                             save=False, Y=None, Z=None, stream=None):
    """(Y, Z): Y [M][N] = act(z) + residual with z = (float(A x W) * a_row_scale[m])
    * w_scale + bias[n], float32 or bfloat16.  With `save`, Z holds z for the
    backward pass; without, it is None.  act: none, relu, relu2, silu or
    gelu_tanh; residual has Y's type and may be Y itself."""
    torch = _torch()
    out_dtype = out_dtype or torch.bfloat16
    _check(A, torch.int8, 2, "A")
    _check(Wpacked, torch.uint8, 2, "Wpacked")
    (M, K), dev = A.shape, A.device
    N, kb = Wpacked.shape
    if kb * 4 != K or Wpacked.device != dev:
        raise ValueError(f"Wpacked must be [N][K/4] = [{N}][{K // 4}] on {dev}, got {tuple(Wpacked.shape)} on "
                         f"{Wpacked.device}")
    _given(a_row_scale, torch.float32, (M,), dev, "a_row_scale")
    if bias is not None:
        _given(bias, torch.float32, (N,), dev, "bias")
    kind, act = _out_kind(out_dtype), _act(act)
    if residual is not None:
        _given(residual, out_dtype, (M, N), dev, "residual")
    if Z is not None and not save:
        raise ValueError("Z is an output of save=True")
    Y = _made(Y, out_dtype, (M, N), dev, "Y", stream)
    if save:
        Z = _made(Z, out_dtype, (M, N), dev, "Z", stream)
    _done("ternary_gemm_s8_epilogue",
          lib().ternary_gemm_s8_epilogue(A.data_ptr(), Wpacked.data_ptr(), a_row_scale.data_ptr(), float(w_scale),
                                         _ptr(bias), act, _ptr(residual), Y.data_ptr(), _ptr(Z), kind, M, N, K,
                                         _raw_stream(stream, dev)))
    return Y, Z


def ternary_epilogue_backward(dY, Z, act="none", bias=True, dZ=None, dbias=None, Q=None, scale=None, workspace=None,
                              stream=None):
    """(dZ, dbias, Q, scale) from Y's gradient and the saved pre-activation Z
    [R][C] of the same type: dZ = dY * act'(Z) for dW, its sums over the rows
    (float32 [C]; None with bias=False), and its int8 rows and scales for dX."""
    torch = _torch()
    kind = _kind(Z, "Z")
    _check(Z, Z.dtype, 2, "Z")
    (R, C), dt, dev = Z.shape, Z.dtype, Z.device
    _given(dY, dt, (R, C), dev, "dY")
    act = _act(act)
    dZ = _like(dZ, Z, stream, "dZ")
    ws = None
    if bias:
        dbias = _made(dbias, torch.float32, (C,), dev, "dbias", stream)
        ws = _scratch(workspace, _queried("ternary_epilogue_backward_workspace", R, C), dev, stream)
    elif dbias is not None:
        raise ValueError("dbias is an output of bias=True")
    Q = _like(Q, Z, stream, "Q", torch.int8)
    scale = _made(scale, torch.float32, (R,), dev, "scale", stream)
    _done("ternary_epilogue_backward",
          lib().ternary_epilogue_backward(dY.data_ptr(), Z.data_ptr(), kind, act, dZ.data_ptr(), _ptr(dbias),
                                          Q.data_ptr(), scale.data_ptr(), R, C, _ptr(ws),
                                          0 if ws is None else ws.numel(), _raw_stream(stream, dev)))
    return dZ, dbias, Q, scale


def _current(device):
    """The device the call launches on has to be its tensors'."""
    if device.index != _torch().cuda.current_device():
        raise ValueError(f"tensors are on {device}, and the current device is cuda:{_torch().cuda.current_device()}")


def ternary_layernorm_quantize(X, gain, beta=None, eps=1e-5, residual=None, save=False, H=None, Y=None, mean=None,
                               rstd=None, Q=None, scale=None, stream=None):
    """Layer norm of h = X + residual [R][C] (float32 or bfloat16) into the int8
    rows that the product takes: (Q int8 [R][C], scale float32 [R], H, Y, mean, rstd).

    H as in ternary_rmsnorm_quantize; beta None counts as 0.  With `save`, Y
    [R][C] in X's type holds the normed values and mean, rstd float32 [R] the
    rows' statistics, for the backward pass; without, they are None."""
    torch = _torch()
    kind = _kind(X, "X")
    _check(X, X.dtype, 2, "X")
    (R, C), dt, dev = X.shape, X.dtype, X.device
    _current(dev)
    _given(gain, torch.float32, (C,), dev, "gain")
    if beta is not None:
        _given(beta, torch.float32, (C,), dev, "beta")
    if residual is not None:
        _given(residual, dt, X.shape, dev, "residual")
        H = _like(H, X, stream, "H")
    elif H is not None and H is not X:
        raise ValueError("H is given without a residual: it would be X")
    if save:
        Y = _like(Y, X, stream, "Y")
        mean = _made(mean, torch.float32, (R,), dev, "mean", stream)
        rstd = _made(rstd, torch.float32, (R,), dev, "rstd", stream)
    elif Y is not None or mean is not None or rstd is not None:
        raise ValueError("Y, mean and rstd are outputs of save=True")
    Q = _like(Q, X, stream, "Q", torch.int8)
    scale = _made(scale, torch.float32, (R,), dev, "scale", stream)
    _done("ternary_layernorm_quantize",
          lib().ternary_layernorm_quantize(X.data_ptr(), kind, _ptr(residual), gain.data_ptr(), _ptr(beta), eps,
                                           None if residual is None else H.data_ptr(), _ptr(Y), _ptr(mean), _ptr(rstd),
                                           Q.data_ptr(), scale.data_ptr(), R, C, _raw_stream(stream, dev)))
    return Q, scale, X if residual is None else H, Y, mean, rstd


def ternary_layernorm_backward(dY, H, gain, mean, rstd, dH=None, beta=True, dX=None, dgain=None, dbeta=None,
                               workspace=None, stream=None):
    """(dX [R][C] in H's type, dgain float32 [C], dbeta float32 [C]; None with
    beta=False) from the gradient dY of the normed values, the H, mean and rstd
    that the norm kept and, with a residual stream, the gradient dH that
    reaches H past the norm (dX may be dH)."""
    torch = _torch()
    kind = _kind(H, "H")
    _check(H, H.dtype, 2, "H")
    (R, C), dt, dev = H.shape, H.dtype, H.device
    _current(dev)
    _given(dY, dt, (R, C), dev, "dY")
    _given(gain, torch.float32, (C,), dev, "gain")
    _given(mean, torch.float32, (R,), dev, "mean")
    _given(rstd, torch.float32, (R,), dev, "rstd")
    if dH is not None:
        _given(dH, dt, (R, C), dev, "dH")
    dX = _like(dX, H, stream, "dX")
    dgain = _like(dgain, gain, stream, "dgain")
    if beta:
        dbeta = _like(dbeta, gain, stream, "dbeta")
    elif dbeta is not None:
        raise ValueError("dbeta is an output of beta=True")
    ws = _scratch(workspace, _queried("ternary_layernorm_backward_workspace", R, C), dev, stream)
    _done("ternary_layernorm_backward",
          lib().ternary_layernorm_backward(dY.data_ptr(), H.data_ptr(), kind, gain.data_ptr(), mean.data_ptr(),
                                           rstd.data_ptr(), _ptr(dH), dX.data_ptr(), dgain.data_ptr(), _ptr(dbeta), R, C,
                                           _ptr(ws), 0 if ws is None else ws.numel(), _raw_stream(stream, dev)))
    return dX, dgain, dbeta


def ternary_gemm_s8s8_epilogue(A, W, a_row_scale, w_col_scale=None, bias=None, act="none", residual=None, out_dtype=None,
                               save=False, Y=None, Z=None, workspace=None, stream=None):
    """(Y, Z): Y [M][N] = act(z) + residual with z = (float(A x W^T) *
    a_row_scale[m]) * w_col_scale[n] + bias[n], of int8 rows A [M][K] and int8
    weights W [N][K]; w_col_scale None counts as 1.  The other arguments are
    ternary_gemm_s8_epilogue's."""
    torch = _torch()
    out_dtype = out_dtype or torch.bfloat16
    _check(A, torch.int8, 2, "A")
    _check(W, torch.int8, 2, "W")
    (M, K), dev = A.shape, A.device
    N = W.shape[0]
    if W.shape[1] != K or W.device != dev:
        raise ValueError(f"W must be [N][K] = [{N}][{K}] on {dev}, got {tuple(W.shape)} on {W.device}")
    _current(dev)
    _given(a_row_scale, torch.float32, (M,), dev, "a_row_scale")
    if w_col_scale is not None:
        _given(w_col_scale, torch.float32, (N,), dev, "w_col_scale")
    if bias is not None:
        _given(bias, torch.float32, (N,), dev, "bias")
    kind, act = _out_kind(out_dtype), _act(act)
    if residual is not None:
        _given(residual, out_dtype, (M, N), dev, "residual")
    if Z is not None and not save:
        raise ValueError("Z is an output of save=True")
    Y = _made(Y, out_dtype, (M, N), dev, "Y", stream)
    if save:
        Z = _made(Z, out_dtype, (M, N), dev, "Z", stream)
    a, w = A.data_ptr(), W.data_ptr()
    ws = _scratch(workspace, _queried("ternary_gemm_s8s8_workspace", M, N, K, min(_lowbit(a), _lowbit(w))), dev, stream)
    _done("ternary_gemm_s8s8_epilogue",
          lib().ternary_gemm_s8s8_epilogue(a, w, a_row_scale.data_ptr(), _ptr(w_col_scale), _ptr(bias), act,
                                           _ptr(residual), Y.data_ptr(), _ptr(Z), kind, M, N, K, _ptr(ws),
                                           0 if ws is None else ws.numel(), _raw_stream(stream, dev)))
    return Y, Z


def ternary_gemm_s8_gated(A, Wpacked, a_row_scale, gate_scale, up_scale, bias=None, act="silu", out_dtype=None,
                          save=False, Y=None, Z=None, workspace=None, stream=None):
    """(Y, Z): Y [M][N] = act(g) * u, the gated layer of int8 rows A [M][K] and
    stored ternary weights Wpacked [2N][K/4], the gate's rows before the up
    projection's: g = (float(A x Wg) * a_row_scale[m]) * gate_scale + bias[n],
    u likewise with up_scale and bias[N + n].  With `save`, Z [M][2N] holds
    (g | u) for ternary_gated_backward; without, it is None."""
    torch = _torch()
    out_dtype = out_dtype or torch.bfloat16
    _check(A, torch.int8, 2, "A")
    _check(Wpacked, torch.uint8, 2, "Wpacked")
    (M, K), dev = A.shape, A.device
    N2, kb = Wpacked.shape
    if kb * 4 != K or N2 % 2 or Wpacked.device != dev:
        raise ValueError(f"Wpacked must be [2N][K/4] with K/4 = {K // 4} on {dev}, got {tuple(Wpacked.shape)} on "
                         f"{Wpacked.device}")
    _current(dev)
    N = N2 // 2
    _given(a_row_scale, torch.float32, (M,), dev, "a_row_scale")
    if bias is not None:
        _given(bias, torch.float32, (N2,), dev, "bias")
    kind, act = _out_kind(out_dtype), _act(act)
    if Z is not None and not save:
        raise ValueError("Z is an output of save=True")
    Y = _made(Y, out_dtype, (M, N), dev, "Y", stream)
    if save:
        Z = _made(Z, out_dtype, (M, N2), dev, "Z", stream)
    a, w = A.data_ptr(), Wpacked.data_ptr()
    ws = _scratch(workspace, _queried("ternary_gemm_s8_gated_workspace", M, N, K, min(_lowbit(a), _lowbit(w))), dev, stream)
    _done("ternary_gemm_s8_gated",
          lib().ternary_gemm_s8_gated(a, w, a_row_scale.data_ptr(), float(gate_scale), float(up_scale), _ptr(bias), act,
                                      Y.data_ptr(), _ptr(Z), kind, M, N, K, _ptr(ws), 0 if ws is None else ws.numel(),
                                      _raw_stream(stream, dev)))
    return Y, Z


def ternary_gated_backward(dY, Z, gate_scale, up_scale, act="silu", bias=True, dZ=None, dbias=None, Q=None, scale=None,
                           workspace=None, stream=None):
    """(dZ [R][2C], dbias float32 [2C], Q int8 [R][2C], scale float32 [R]) from
    the gradient dY [R][C] of a gated product's output and the Z [R][2C] that
    it saved, gate first: dZ for dW, its sums over the rows (None with
    bias=False), and the int8 rows of (gate_scale dg | up_scale du) for one dX
    call with the stored weights of both matrices and a weight scale of 1."""
    torch = _torch()
    kind = _kind(Z, "Z")
    _check(Z, Z.dtype, 2, "Z")
    (R, C2), dt, dev = Z.shape, Z.dtype, Z.device
    _current(dev)
    if C2 % 2:
        raise ValueError(f"Z must have the gate's and the up projection's columns, got {C2}")
    C = C2 // 2
    _given(dY, dt, (R, C), dev, "dY")
    act = _act(act)
    dZ = _like(dZ, Z, stream, "dZ")
    ws = None
    if bias:
        dbias = _made(dbias, torch.float32, (C2,), dev, "dbias", stream)
        ws = _scratch(workspace, _queried("ternary_gated_backward_workspace", R, C), dev, stream)
    elif dbias is not None:
        raise ValueError("dbias is an output of bias=True")
    Q = _like(Q, Z, stream, "Q", torch.int8)
    scale = _made(scale, torch.float32, (R,), dev, "scale", stream)
    _done("ternary_gated_backward",
          lib().ternary_gated_backward(dY.data_ptr(), Z.data_ptr(), kind, act, float(gate_scale), float(up_scale),
                                       dZ.data_ptr(), _ptr(dbias), Q.data_ptr(), scale.data_ptr(), R, C, _ptr(ws),
                                       0 if ws is None else ws.numel(), _raw_stream(stream, dev)))
    return dZ, dbias, Q, scale

def ternary_clip_grad_norm(grads, max_norm, eps=1e-6, out=None, norm=None, workspace=None, stream=None):
    """(out, norm float32 [1]): the gradients scaled by min(1, max_norm / (norm
    + eps)), norm the root of the sum of all their squares.  grads is a list of
    contiguous float32 or bfloat16 device tensors of any shapes, on one device;
    out a list of tensors of the same types and sizes (`grads` itself: in
    place), new ones if None."""
    torch = _torch()
    grads = list(grads)
    if not grads:
        raise ValueError("grads must hold at least one tensor")
    n = len(grads)
    # many tensors, little time: one comprehension a property
    try:
        types, idx, sizes = [g.dtype for g in grads], grads[0].get_device(), [g.numel() for g in grads]
        kinds = [IN_F32 if t is torch.float32 else IN_BF16 if t is torch.bfloat16 else None for t in types]
        fits = all([g.get_device() == idx and g.is_contiguous() for g in grads])
        src = [g.data_ptr() for g in grads]
    except AttributeError:
        raise TypeError("grads must hold torch.Tensors") from None
    if None in kinds:
        raise TypeError("grads must be float32 or bfloat16 tensors")
    if idx < 0 or not fits:
        raise ValueError("grads must be contiguous tensors on one GPU device")
    dev = grads[0].device
    if out is None:
        out = [_like(None, g, stream, "out") for g in grads]
    elif len(out) != n:
        raise ValueError(f"out must hold {n} tensors, got {len(out)}")
    else:
        try:
            fits = ([o.dtype for o in out] == types and [o.numel() for o in out] == sizes
                    and all([o.get_device() == idx and o.is_contiguous() for o in out]))
        except AttributeError:
            raise TypeError("out must hold torch.Tensors") from None
        if not fits:
            raise ValueError("out must hold contiguous tensors of the types and sizes of grads, on their device")
    # the C call's four host arrays, alive until it returns
    arrays = (array("q", src), array("q", [o.data_ptr() for o in out]), array("q", sizes), array("i", kinds))
    src, dst, sizes, kinds = [a.buffer_info()[0] for a in arrays]
    norm = _made(norm, torch.float32, (1,), dev, "norm", stream)
    ws = _scratch(workspace, _queried("ternary_clip_grad_norm_workspace", sizes, n), dev, stream)
    _done("ternary_clip_grad_norm",
          lib().ternary_clip_grad_norm(src, dst, sizes, kinds, n, max_norm, eps, norm.data_ptr(), ws.data_ptr(),
                                       ws.numel(), _raw_stream(stream, dev)))
    return out, norm
