"""Thin ctypes binding of libconvrot.so (the C ABI in include/convrot.h).

Argument marshalling only: every step of the ConvRot path runs in the HIP
kernels behind the C ABI.  PyTorch provides device memory (output tensors are
allocated with ``torch.empty``) and the stream (torch's current stream).
Function names are those of the C ABI.  A non-zero status raises
``ConvRotError``; a missing library raises at load time -- there is no
fallback of any kind.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import numpy as np

from . import build as _build

LIB_PATH = _build.LIB_PATH

CONVROT_OK = 0
CONVROT_EINVAL = 1
CONVROT_EWORKSPACE = 2
CONVROT_EHIP = 3
CONVROT_EDEVICE = 4
# OR'd into a group size g: rotate with the regular Hadamard matrix
CONVROT_REGULAR_HADAMARD = 0x10000
# OR'd into a group size g: the weight image holds the INT4 codes only (0.5 bytes
# per weight); every product then runs on the INT8 matrix cores
CONVROT_INT4_IMAGE = 0x20000
_GROUP_FLAGS = CONVROT_REGULAR_HADAMARD | CONVROT_INT4_IMAGE
# workspace status word: offset, and the value a split-K wait that ran out leaves
WORKSPACE_STATUS_OFFSET = 2048
CONVROT_STATUS_SPLIT_TIMEOUT = 1
# test flag of convrot_gemm_i32_tiled
CONVROT_TEST_SPLIT_TIMEOUT = 1
CONVROT_TILE_FP6 = 0x10000  # or-ed into tile_n of the tiled hooks: the FP6 tile of that size (192 x 384)
MAX_K = 16384           # largest rotated width K_rot
MAX_ROWS = 16777216     # largest M or N


def rotated_width(K: int, g: int) -> int:
    """Codes and rotated values are K rounded up to a whole number of groups wide
    (the missing values of the last group are zero)."""
    gs = g & ~_GROUP_FLAGS
    return -(-K // gs) * gs

_lock = threading.Lock()
_lib = None


class ConvRotError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        text = _lib.convrot_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{where}: status {status} ({text})")


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_SZ = ctypes.c_size_t


_SIGNATURES = {
    "convrot_status_string": ([_I], ctypes.c_char_p),
    "convrot_version": ([], ctypes.c_char_p),
    "convrot_weight_image_bytes": ([_I64, _I64, _I, ctypes.POINTER(_SZ)], _I),
    "convrot_workspace_bytes": ([_I64, _I64, _I64, _I, ctypes.POINTER(_SZ)], _I),
    "convrot_linear_kernel_count": ([_I64, _I64, _I64, _I, ctypes.POINTER(_I)], _I),
    "convrot_linear_plan": ([_I64, _I64, _I64, _I] + [ctypes.POINTER(_I)] * 4, _I),
    "convrot_validate_weight": ([_P, _I64, _I64, _I, _P, _P], _I),
    "convrot_validate_linear": ([_P, _I64, _I64, _P, _P, _P, _I64, _I, _P, _P, _SZ], _I),
    "convrot_prepare_weight": ([_P, _I64, _I64, _I, _P, _P, _P], _I),
    "convrot_quantize_weight": ([_P, _I64, _I64, _I, _P, _P, _P], _I),
    "convrot_repack_nk_to_image": ([_P, _I64, _I64, _I, _P, _P], _I),
    "convrot_linear": ([_P, _I64, _I64, _P, _P, _P, _I64, _I, _P, _P, _SZ, _P], _I),
    "convrot_linear_noalloc": ([_P, _I64, _I64, _P, _P, _P, _I64, _I, _P, _P], _I),
    "convrot_prepare_activations": ([_P, _I64, _I64, _I, _P, _SZ, _P], _I),
    "convrot_gemm": ([_P, _SZ, _I64, _I64, _P, _P, _P, _I64, _I, _P, _P], _I),
    "convrot_prepare_rows": ([_P, _I64, _I64, _I, _P, _P, _P, _P], _I),
    "convrot_w4a16_workspace_bytes": ([_I64, _I64, _I, _P], _I),
    "convrot_validate_linear_w4a16": ([_P, _I64, _I64, _P, _P, _P, _I64, _I, _P, _P, _SZ], _I),
    "convrot_linear_w4a16": ([_P, _I64, _I64, _P, _P, _P, _I64, _I, _P, _P, _SZ, _P], _I),
    "convrot_gemm_i32": ([_P, _I64, _I64, _P, _I64, _P, _P, _SZ, _P], _I),
    "convrot_workspace_bytes_tiled": ([_I64, _I64, _I64, _I, _I, _I, ctypes.POINTER(_SZ)], _I),
    "convrot_gemm_i32_tiled": ([_P, _I64, _I64, _P, _I64, _P, _I, _I, _I, _I, _P, _SZ, _P], _I),
    "convrot_split_k_extent": ([_I64, _I64, _I64, _I, _I, _I, ctypes.POINTER(_SZ), ctypes.POINTER(_I),
                                ctypes.POINTER(_SZ)], _I),
    "convrot_matrix_core_probe_bytes": ([ctypes.POINTER(_SZ)], _I),
    "convrot_matrix_core_probe": ([_I, _I, _P, _SZ, ctypes.POINTER(_I64), _P], _I),
    "convrot_residual_norm": ([_P, _P], _I),
    "convrot_validate_residual_norm": ([_P], _I),
    "convrot_rope": ([_P, _P], _I),
    "convrot_validate_rope": ([_P], _I),
    "convrot_linear_grouped": ([_P, _P], _I),
    "convrot_validate_linear_grouped": ([_P], _I),
    "convrot_quantize_weight_grouped": ([_P, _I64, _I64, _I, _I, _P, _P, _P, _P], _I),
    "convrot_validate_quantize_weight_grouped": ([_P, _I64, _I64, _I, _I, _P, _P, _P], _I),
    "convrot_host_pack_nk": ([_P, _I64, _I64, _P], _I),
    "convrot_host_unpack_nk": ([_P, _I64, _I64, _P], _I),
    "convrot_host_nk_to_kn": ([_P, _I64, _I64, _P], _I),
    "convrot_host_kn_to_nk": ([_P, _I64, _I64, _P], _I),
    "convrot_host_nk_to_image": ([_P, _I64, _I64, _P], _I),
    "convrot_host_image_to_nk": ([_P, _I64, _I64, _P], _I),
    "convrot_host_act_image_to_codes": ([_P, _I64, _I64, _P], _I),
    "convrot_host_image_fp6_to_nk": ([_P, _I64, _I64, _P], _I),
    "convrot_host_workspace_fp6_codes": ([_P, _I64, _I64, _P], _I),
}


def load():
    """Load libconvrot.so (building it only if nothing is built).

    torch is imported first: it brings its own HIP runtime library, and the
    library's HIP dependency must resolve to that same, already loaded copy --
    loaded the other way round, the process would hold two HIP runtimes and
    torch's device pointers and streams would be foreign to the library's."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        import torch  # noqa: F401  (see above)
        if not os.path.exists(LIB_PATH):
            _build.build()
        lib = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


def _call(name, *args):
    rc = getattr(_lib or load(), name)(*args)
    if rc != CONVROT_OK:
        raise ConvRotError(rc, name)


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t, dtype, name):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


# --------------------------------------------------------------------------
# sizes and checks
# --------------------------------------------------------------------------

def convrot_version() -> str:
    return load().convrot_version().decode()


def convrot_status_string(status: int) -> str:
    return load().convrot_status_string(int(status)).decode()


def convrot_weight_image_bytes(N: int, K: int, g: int) -> int:
    out = _SZ(0)
    _call("convrot_weight_image_bytes", N, K, g, ctypes.byref(out))
    return out.value


def convrot_workspace_bytes(M: int, K: int, N: int, g: int) -> int:
    out = _SZ(0)
    _call("convrot_workspace_bytes", M, K, N, g, ctypes.byref(out))
    return out.value


def convrot_linear_kernel_count(M: int, K: int, N: int, g: int) -> int:
    out = _I(0)
    _call("convrot_linear_kernel_count", M, K, N, g, ctypes.byref(out))
    return out.value


CONVROT_MFMA_I8 = 1
CONVROT_MFMA_FP6 = 2


def convrot_linear_plan(M: int, K: int, N: int, g: int) -> dict:
    """The product plan: {"mfma": CONVROT_MFMA_I8 / CONVROT_MFMA_FP6 (0 if M or N
    is 0), "tile": (tile_m, tile_n) ((0, 0) for M <= 128), "splits": S}."""
    v = [ctypes.c_int() for _ in range(4)]
    _call("convrot_linear_plan", M, K, N, g, *[ctypes.byref(x) for x in v])
    return {"mfma": v[0].value, "tile": (v[1].value, v[2].value), "splits": v[3].value}


def convrot_validate_weight(W_ptr, N, K, g, image_ptr, sw_ptr) -> int:
    """Raw pointer values (ints); returns the status code."""
    return load().convrot_validate_weight(W_ptr, N, K, g, image_ptr, sw_ptr)


def convrot_validate_linear(X_ptr, M, K, image_ptr, sw_ptr, bias_ptr, N, g, Y_ptr, ws_ptr, ws_bytes) -> int:
    """Raw pointer values (ints); returns the status code."""
    return load().convrot_validate_linear(X_ptr, M, K, image_ptr, sw_ptr, bias_ptr, N, g, Y_ptr, ws_ptr, ws_bytes)


# --------------------------------------------------------------------------
# device entry points
# --------------------------------------------------------------------------

def convrot_prepare_weight(W, g: int, image=None, sw=None, stream=None):
    """W: bf16 [N, K] on the GPU -> (weight image uint8, sw float32 [N])."""
    import torch
    N, K = W.shape
    nbytes = convrot_weight_image_bytes(N, K, g)
    if image is None:
        image = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    if sw is None:
        sw = torch.empty(N, dtype=torch.float32, device=W.device)
    if image.numel() < nbytes:
        raise ValueError("weight image buffer too small")
    _call("convrot_prepare_weight", _dev(W, torch.bfloat16, "W"), N, K, g, _dev(image, torch.uint8, "image"),
          _dev(sw, torch.float32, "sw"), _stream(stream))
    return image, sw


def convrot_quantize_weight(W, g: int, stream=None):
    """W: bf16 [N, K] -> (N x packed-K uint8 [N, K_rot/2], sw float32 [N]), K_rot = rotated_width(K, g)."""
    import torch
    N, K = W.shape
    nk = torch.empty((N, rotated_width(K, g) // 2), dtype=torch.uint8, device=W.device)
    sw = torch.empty(N, dtype=torch.float32, device=W.device)
    _call("convrot_quantize_weight", _dev(W, torch.bfloat16, "W"), N, K, g, _dev(nk, torch.uint8, "nk"),
          _dev(sw, torch.float32, "sw"), _stream(stream))
    return nk, sw


def convrot_repack_nk_to_image(nk, N: int, K: int, g: int = 64, stream=None):
    """N x packed-K uint8 [N, K_rot/2] -> weight image (the FP6 copy too unless g has CONVROT_INT4_IMAGE)."""
    import torch
    image = torch.empty(convrot_weight_image_bytes(N, K, g), dtype=torch.uint8, device=nk.device)
    _call("convrot_repack_nk_to_image", _dev(nk, torch.uint8, "nk"), N, K, g, _dev(image, torch.uint8, "image"),
          _stream(stream))
    return image


def new_workspace(M: int, K: int, N: int, g: int, device="cuda"):
    import torch
    return torch.empty(convrot_workspace_bytes(M, K, N, g), dtype=torch.uint8, device=device)


def convrot_linear(X, image, sw, bias, N: int, g: int, Y=None, workspace=None, stream=None):
    """X: bf16 [M, K]; bias: bf16 [N] or None -> Y bf16 [M, N]."""
    import torch
    M, K = X.shape
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    if workspace is None:
        workspace = new_workspace(M, K, N, g, X.device)
    bias_p = None if bias is None else _dev(bias, torch.bfloat16, "bias")
    _call("convrot_linear", _dev(X, torch.bfloat16, "X"), M, K, _dev(image, torch.uint8, "image"),
          _dev(sw, torch.float32, "sw"), bias_p, N, g, _dev(Y, torch.bfloat16, "Y"),
          _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream))
    return Y


# the largest workspace convrot_linear_noalloc has (CONVROT_NOALLOC_MAX_WORKSPACE)
NOALLOC_MAX_WORKSPACE = 48 << 20


def convrot_linear_noalloc(X, image, sw, bias, N: int, g: int, Y, stream=None):
    """convrot_linear with the library's own device workspace (no allocation in
    the call; Y must be given).  Calls on one GPU share that workspace."""
    import torch
    M, K = X.shape
    bias_p = None if bias is None else _dev(bias, torch.bfloat16, "bias")
    _call("convrot_linear_noalloc", _dev(X, torch.bfloat16, "X"), M, K, _dev(image, torch.uint8, "image"),
          _dev(sw, torch.float32, "sw"), bias_p, N, g, _dev(Y, torch.bfloat16, "Y"), _stream(stream))
    return Y


def convrot_prepare_activations(X, g: int, workspace, stream=None):
    import torch
    M, K = X.shape
    _call("convrot_prepare_activations", _dev(X, torch.bfloat16, "X"), M, K, g,
          _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream))
    return workspace


def convrot_gemm(workspace, M: int, K: int, image, sw, bias, N: int, g: int, Y=None, stream=None):
    """The GEMM half of convrot_linear (M, K, N, g as for the linear) on a prepared workspace."""
    import torch
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=workspace.device)
    bias_p = None if bias is None else _dev(bias, torch.bfloat16, "bias")
    _call("convrot_gemm", _dev(workspace, torch.uint8, "workspace"), workspace.numel(), M, K,
          _dev(image, torch.uint8, "image"), _dev(sw, torch.float32, "sw"), bias_p, N, g,
          _dev(Y, torch.bfloat16, "Y"), _stream(stream))
    return Y


def convrot_prepare_rows(X, g: int, want_rotated: bool = False, stream=None):
    """Rotation + quantization of bf16 rows -> (codes int8 [rows, K_rot], scales f32 [rows],
    rotated f32 [rows, K_rot] or None), K_rot = rotated_width(K, g)."""
    import torch
    rows, K = X.shape
    Kr = rotated_width(K, g)
    codes = torch.empty((rows, Kr), dtype=torch.int8, device=X.device)
    scales = torch.empty(rows, dtype=torch.float32, device=X.device)
    rot = torch.empty((rows, Kr), dtype=torch.float32, device=X.device) if want_rotated else None
    _call("convrot_prepare_rows", _dev(X, torch.bfloat16, "X"), rows, K, g, _dev(codes, torch.int8, "codes"),
          _dev(scales, torch.float32, "scales"), None if rot is None else _dev(rot, torch.float32, "rotated"),
          _stream(stream))
    return codes, scales, rot


def convrot_gemm_i32(qx, image, N: int, workspace=None, stream=None):
    """qx: int8 codes [M, K] -> int32 [M, N] products against the weight image."""
    import torch
    M, K = qx.shape
    if workspace is None:
        workspace = new_workspace(M, K, N, 64, qx.device)
    acc = torch.empty((M, N), dtype=torch.int32, device=qx.device)
    _call("convrot_gemm_i32", _dev(qx, torch.int8, "qx"), M, K, _dev(image, torch.uint8, "image"), N,
          _dev(acc, torch.int32, "acc"), _dev(workspace, torch.uint8, "workspace"), workspace.numel(),
          _stream(stream))
    return acc


def convrot_workspace_bytes_tiled(M: int, K: int, N: int, tile, splits: int) -> int:
    out = _SZ(0)
    _call("convrot_workspace_bytes_tiled", M, K, N, tile[0], tile[1], splits, ctypes.byref(out))
    return out.value


def convrot_gemm_i32_tiled(qx, image, N: int, tile, splits: int, test_flags: int = 0, workspace=None, stream=None):
    """convrot_gemm_i32 with the block tile (tile_m, tile_n) and the K split given
    (tile_n | CONVROT_TILE_FP6 picks the FP6 192 x 384 tile over the INT8 one).
    Returns (acc int32 [M, N], workspace)."""
    import torch
    M, K = qx.shape
    if workspace is None:
        workspace = torch.empty(convrot_workspace_bytes_tiled(M, K, N, tile, splits), dtype=torch.uint8,
                                device=qx.device)
    acc = torch.empty((M, N), dtype=torch.int32, device=qx.device)
    _call("convrot_gemm_i32_tiled", _dev(qx, torch.int8, "qx"), M, K, _dev(image, torch.uint8, "image"), N,
          _dev(acc, torch.int32, "acc"), tile[0], tile[1], splits, test_flags,
          _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream))
    return acc, workspace


def convrot_split_k_extent(M: int, K: int, N: int, tile, splits: int) -> dict:
    """Host check of a split-K plan's footprint: one past the largest partial-area
    byte, counter word and LDS byte the exchange touches."""
    pe, cu, le = _SZ(0), _I(0), _SZ(0)
    _call("convrot_split_k_extent", M, K, N, tile[0], tile[1], splits, ctypes.byref(pe), ctypes.byref(cu),
          ctypes.byref(le))
    return {"partial_end": pe.value, "counters_used": cu.value, "lds_end": le.value}


CONVROT_PROBE_FP6 = 1
CONVROT_PROBE_INT8 = 2
PROBE_OPS_PER_MFMA = {CONVROT_PROBE_FP6: 2 * 32 * 32 * 64, CONVROT_PROBE_INT8: 2 * 32 * 32 * 32}


def convrot_matrix_core_probe(kind: int, iterations: int, out=None, stream=None):
    """Enqueue the MFMA-only rate loop; returns (MFMA instructions it runs, out).
    The caller times it on the stream."""
    import torch
    if out is None:
        nbytes = _SZ(0)
        _call("convrot_matrix_core_probe_bytes", ctypes.byref(nbytes))
        out = torch.empty(nbytes.value // 4, dtype=torch.float32, device="cuda")
    count = _I64(0)
    _call("convrot_matrix_core_probe", kind, iterations, _dev(out, torch.float32, "out"), out.numel() * 4,
          ctypes.byref(count), _stream(stream))
    return count.value, out


def workspace_status(workspace) -> int:
    """The workspace's status word after a completed call (0, or CONVROT_STATUS_SPLIT_TIMEOUT)."""
    import torch
    return int(workspace[WORKSPACE_STATUS_OFFSET:WORKSPACE_STATUS_OFFSET + 4].view(torch.int32).item())


# --------------------------------------------------------------------------
# host layout tools (numpy in, numpy out)
# --------------------------------------------------------------------------

def _np(a, dtype):
    return np.ascontiguousarray(a, dtype=dtype)


def _hp(a):
    return a.ctypes.data_as(ctypes.c_void_p)


def convrot_host_pack_nk(codes) -> np.ndarray:
    q = _np(codes, np.int8)
    N, K = q.shape
    out = np.empty((N, K // 2), np.uint8)
    _call("convrot_host_pack_nk", _hp(q), N, K, _hp(out))
    return out


def convrot_host_unpack_nk(nk, K: int) -> np.ndarray:
    p = _np(nk, np.uint8)
    N = p.shape[0]
    out = np.empty((N, K), np.int8)
    _call("convrot_host_unpack_nk", _hp(p), N, K, _hp(out))
    return out


def convrot_host_nk_to_kn(nk, N: int, K: int) -> np.ndarray:
    p = _np(nk, np.uint8)
    out = np.empty((K, N // 2), np.uint8)
    _call("convrot_host_nk_to_kn", _hp(p), N, K, _hp(out))
    return out


def convrot_host_kn_to_nk(kn, N: int, K: int) -> np.ndarray:
    p = _np(kn, np.uint8)
    out = np.empty((N, K // 2), np.uint8)
    _call("convrot_host_kn_to_nk", _hp(p), N, K, _hp(out))
    return out


def convrot_host_nk_to_image(nk, N: int, K: int) -> np.ndarray:
    p = _np(nk, np.uint8)
    out = np.empty(convrot_weight_image_bytes(N, K, 64), np.uint8)
    _call("convrot_host_nk_to_image", _hp(p), N, K, _hp(out))
    return out


def convrot_host_image_to_nk(image, N: int, K: int) -> np.ndarray:
    p = _np(image, np.uint8)
    out = np.empty((N, K // 2), np.uint8)
    _call("convrot_host_image_to_nk", _hp(p), N, K, _hp(out))
    return out


def convrot_host_image_fp6_to_nk(image, N: int, K: int) -> np.ndarray:
    """The FP6 copy of the codes in a weight image, as N x packed-K."""
    p = _np(image, np.uint8)
    out = np.empty((N, K // 2), np.uint8)
    _call("convrot_host_image_fp6_to_nk", _hp(p), N, K, _hp(out))
    return out


def convrot_host_workspace_fp6_codes(workspace, M: int, K: int) -> np.ndarray:
    """The FP6 activation codes of a workspace (M > 32), as int8 [M, K]."""
    ws = workspace.cpu().numpy() if hasattr(workspace, "cpu") else np.asarray(workspace)
    p = _np(ws, np.uint8)
    out = np.empty((M, K), np.int8)
    _call("convrot_host_workspace_fp6_codes", _hp(p), M, K, _hp(out))
    return out


# Offset of the activation-code image inside a workspace
# (CONVROT_WORKSPACE_IMAGE_OFFSET in include/convrot.h).
WORKSPACE_IMAGE_OFFSET = 4096


def workspace_act_codes(workspace, M: int, K: int) -> np.ndarray:
    """Activation codes int8 [M, K] decoded from a workspace (tensor or array); K is
    the code width (the rotated width of the prepared rows)."""
    ws = workspace.cpu().numpy() if hasattr(workspace, "cpu") else np.asarray(workspace)
    return convrot_host_act_image_to_codes(ws[WORKSPACE_IMAGE_OFFSET:], M, K)


def convrot_host_act_image_to_codes(image, M: int, K: int) -> np.ndarray:
    p = _np(image, np.uint8)
    out = np.empty((M, K), np.int8)
    _call("convrot_host_act_image_to_codes", _hp(p), M, K, _hp(out))
    return out


# --------------------------------------------------------------------------
# W4A16 variant (M <= 32)
# --------------------------------------------------------------------------

def convrot_w4a16_workspace_bytes(M: int, K: int, g: int) -> int:
    out = ctypes.c_size_t()
    _call("convrot_w4a16_workspace_bytes", M, K, g, ctypes.byref(out))
    return out.value


def convrot_validate_linear_w4a16(X_ptr, M, K, image_ptr, sw_ptr, bias_ptr, N, g, Y_ptr, ws_ptr, ws_bytes) -> int:
    """Raw pointer values (ints); returns the status code."""
    return load().convrot_validate_linear_w4a16(X_ptr, M, K, image_ptr, sw_ptr, bias_ptr, N, g, Y_ptr, ws_ptr,
                                                ws_bytes)


def convrot_linear_w4a16(X, image, sw, bias, N: int, g: int, Y=None, workspace=None, stream=None):
    """Y = X W^T + bias with INT4 weights and bf16 rotated activations (M <= 32).
    The workspace receives the bf16 rotated rows [M, K]."""
    import torch
    M, K = X.shape
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    if workspace is None:
        workspace = torch.empty(max(convrot_w4a16_workspace_bytes(M, K, g), 1), dtype=torch.uint8, device=X.device)
    bias_p = None if bias is None else _dev(bias, torch.bfloat16, "bias")
    _call("convrot_linear_w4a16", _dev(X, torch.bfloat16, "X"), M, K, _dev(image, torch.uint8, "image"),
          _dev(sw, torch.float32, "sw"), bias_p, N, g, _dev(Y, torch.bfloat16, "Y"),
          _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream))
    return Y


# --------------------------------------------------------------------------
# operators around the linears of a block
# --------------------------------------------------------------------------

CONVROT_BF16 = 1
CONVROT_F16 = 2
CONVROT_F32 = 3
CONVROT_I32 = 4
CONVROT_NORM_NONE = 0
CONVROT_NORM_LAYER = 1
CONVROT_NORM_RMS = 2
CONVROT_ROPE_INTERLEAVED = 1
CONVROT_ROPE_HALVES = 2

# The argument structs of the C calls, in their order (native alignment).
NORM_ARGS = struct.Struct("@9P10q2f4i")
ROPE_ARGS = struct.Struct("@" + 2 * "3P7q" + "i2qi" + "P2q3i2P3if0P")
GROUPED_ARGS = struct.Struct("@6P3q2i")

_NORMS = {None: CONVROT_NORM_NONE, "layer": CONVROT_NORM_LAYER, "rms": CONVROT_NORM_RMS}
_LAYOUTS = {"interleaved": CONVROT_ROPE_INTERLEAVED, "halves": CONVROT_ROPE_HALVES}
_GROUPS = (32, 64, 128)
_torch = None   # the module, its types' codes and its current device and stream, from the first call on
_forward = None   # its forward differentiation
_types = {}
_current_device = _raw_stream = None


def _use_torch():
    global _torch, _forward, _current_device, _raw_stream
    import torch
    import torch.autograd.forward_ad as _forward
    _types.update({torch.bfloat16: CONVROT_BF16, torch.float16: CONVROT_F16, torch.float32: CONVROT_F32})
    # The handles themselves: torch.cuda.current_stream builds an object around
    # one, which takes longer than a launch.
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda device: torch.cuda.current_stream(device).cuda_stream)
    _torch = torch
    return torch


def _choice(table, key, what):
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError(f"unknown {what} {key!r}") from None


def _on_gpu(t, name):
    """The index of the device of a call's first tensor."""
    if not isinstance(t, (_torch or _use_torch()).Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.get_device()


def _check_tensor(t, name, device):
    """A tensor of this call: on its device, and one that asks for no gradient here."""
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda or t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    if t.requires_grad and _torch.is_grad_enabled():
        raise RuntimeError(f"{name} requires a gradient, and this operator has none: call it under torch.no_grad()")


def _check_tangents(*tensors):
    """No tensor of this call carries a tangent of forward differentiation, which
    ``requires_grad`` does not tell; outside of any dual level there are none."""
    for t in tensors:
        if isinstance(t, _torch.Tensor) and _forward.unpack_dual(t).tangent is not None:
            raise RuntimeError("a tensor of this call has a tangent, and this operator has no derivative: "
                               "call it on the primal of torch.autograd.forward_ad.unpack_dual")


def _written(*tensors):
    """Outputs that the caller gave: autograd is told that they changed."""
    for t in tensors:
        if t is not None:
            _torch.autograd.graph.increment_version(t)


def _type_of(t, name):
    code = _types.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} has an unsupported type {t.dtype}")
    return code


def _launch(device, stream, call, tensors):
    """call(raw stream) with the device current, and with ``stream`` (or the
    device's current stream) the one that its allocations belong to.  The
    memory of the call's own ``tensors`` is kept until a ``stream`` given has run
    it, whenever they are freed; that the stream waits for what makes them, and
    others for its outputs, is the caller's to order."""
    if stream is None:
        if _current_device() == device:
            return call(_raw_stream(device))
        with _torch.cuda.device(device):
            return call(_raw_stream(device))
    if stream.device.index != device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on cuda:{device}")
    with _torch.cuda.stream(stream):
        out = call(stream.cuda_stream)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return out


def _rows(t, name, width):
    """(rows, row stride) of a tensor seen as rows of its dense last dimension."""
    shape = t.shape
    if not shape or shape[-1] != width:
        raise ValueError(f"{name} must have rows of {width} values, got shape {tuple(shape)}")
    strides = t.stride()
    if strides[-1] != 1 and width > 1:
        raise ValueError(f"{name} must be dense in its last dimension")
    if len(shape) == 2:
        return shape[0], strides[0]
    if len(shape) == 1:
        return 1, width
    if t.is_contiguous():
        return (t.numel() // width, width) if width else (0, 0)
    if t.numel() == 0:
        return 0, 0
    rows, stride = 1, 0
    for n, s in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if n == 1:
            continue
        if rows == 1:
            stride = s
        elif s != rows * stride:
            raise ValueError(f"the rows of {name} are not evenly spaced: strides {strides}")
        rows *= n
    return rows, stride


def convrot_residual_norm(x, y=None, *, gate=None, scale=None, shift=None, weight=None, post_weight=None,
                          norm="layer", post_norm=None, residual_scale: float = 1.0, eps: float = 1e-6, r=None,
                          h=None, want_r: bool = True, want_h: bool = True, stream=None):
    """r = residual_scale x + gate * P(y);  h = N(r) * weight * (1 + scale) + shift.

    x, y: bf16, f16 or f32 [..., width], rows evenly spaced and dense.  norm,
    post_norm: "layer", "rms" or None.  gate, scale, shift: of the same type or
    f32, [width] for all rows, or [..., width] with the leading dimensions of x,
    or the first of them (one vector a batch entry; ones may follow); for a
    matrix x also [V, width], one vector for every rows / V rows.  weight,
    post_weight: [width], of the vectors' type.  Returns (r, h) of x's shape; r
    or h given is written (x or y itself may be), and one not wanted is None.
    ``stream``: where to run, if not on the current stream; it has to wait for what
    makes the inputs, and their memory is kept until it is done."""
    device = _on_gpu(x, "x")
    _check_tensor(x, "x", device)
    if getattr(_forward, "_current_level", 0) >= 0:
        _check_tangents(x, y, gate, scale, shift, weight, post_weight, r, h)
    shape, dtype = x.shape, x.dtype
    width = shape[-1] if shape else 0
    code = _type_of(x, "x")
    norms = _choice(_NORMS, norm, "norm"), _choice(_NORMS, post_norm, "norm")
    rows, x_stride = _rows(x, "x", width)
    y_ptr = y_stride = 0
    if y is not None:
        _check_tensor(y, "y", device)
        if y.shape != shape or y.dtype != dtype:
            raise ValueError(f"y must have the shape and type of x, got {tuple(y.shape)} {y.dtype}")
        y_ptr, y_stride = y.data_ptr(), _rows(y, "y", width)[1]
    vec_type, vec_code, per = None, 0, 0
    vectors = []   # addresses and strides of gate, scale, shift, weight, post_weight
    for name, v in (("gate", gate), ("scale", scale), ("shift", shift), ("weight", weight),
                    ("post_weight", post_weight)):
        if v is None:
            vectors.append((0, 0))
            continue
        if not isinstance(v, _torch.Tensor) or v.get_device() != device or v.requires_grad:
            _check_tensor(v, name, device)
        if v.dtype is not vec_type:
            v_code = _type_of(v, name)
            if vec_type is not None or v_code not in (code, CONVROT_F32):
                raise TypeError("the vectors and weights must have one type, that of x or float32")
            vec_type, vec_code = v.dtype, v_code
        n, step = _rows(v, name, width)
        if n == 1:
            step = 0
        else:
            lead = v.shape[:-1]
            while lead and lead[-1] == 1:
                lead = lead[:-1]
            if "weight" in name:
                raise ValueError(f"{name} must be one vector of {width} values")
            if rows % n if len(shape) == 2 and len(lead) == 1 and n else lead != shape[:-1][:len(lead)]:
                raise ValueError(f"{name} of shape {tuple(v.shape)} does not fit x of shape {tuple(shape)}")
            if rows:
                if per not in (0, rows // n):
                    raise ValueError("gate, scale and shift must have one vector, or as many as one another")
                per = rows // n
        vectors.append((v.data_ptr(), step))
    (gate_ptr, gate_step), (scale_ptr, scale_step), (shift_ptr, shift_step), (w_ptr, _), (post_ptr, _) = vectors

    def output(out, name, wanted):
        """The output given, or a new one: it, its address and row stride."""
        if out is None:
            if not wanted:
                return None, 0, 0
            out = _torch.empty_like(x, memory_format=_torch.contiguous_format)
            return out, out.data_ptr(), width
        _check_tensor(out, name, device)
        if out.shape != shape or out.dtype != dtype:
            raise ValueError(f"{name} must have the shape and type of x")
        return out, out.data_ptr(), _rows(out, name, width)[1]

    def call(raw):
        r_out, r_ptr, r_stride = output(r, "r", want_r)
        h_out, h_ptr, h_stride = output(h, "h", want_h)
        _call("convrot_residual_norm", NORM_ARGS.pack(
            x.data_ptr(), y_ptr, gate_ptr, scale_ptr, shift_ptr, w_ptr, post_ptr, r_ptr, h_ptr, rows, width, x_stride,
            y_stride, r_stride, h_stride, gate_step, scale_step, shift_step, per or 1, residual_scale, eps, code,
            vec_code or code, *norms), raw)
        if r is not None or h is not None:
            _written(r, h)
        return r_out, h_out

    return _launch(device, stream, call, (x, y, gate, scale, shift, weight, post_weight, r, h))


def rope_frequencies(sizes, theta: float = 10000.0, shared: bool = False):
    """(freq float64 [pairs], axis int32 [pairs]) of a rotation over several axes.

    Axis a owns sizes[a] of a head's elements (an even number) and runs through
    a spectrum of its own, theta^(-2 i / sizes[a]); with ``shared`` all axes
    cut one spectrum over sum(sizes) elements into sections, in order."""
    sizes = [int(s) for s in sizes]
    if not sizes or any(s < 2 or s % 2 for s in sizes):
        raise ValueError("every axis needs an even, positive number of elements")
    axis = np.repeat(np.arange(len(sizes), dtype=np.int32), [s // 2 for s in sizes])
    if shared:
        freq = theta ** (-np.arange(len(axis)) * 2.0 / sum(sizes))
    else:
        freq = np.concatenate([theta ** (-np.arange(s // 2) * 2.0 / s) for s in sizes])
    return freq, axis


def _address(a):
    """Of a host array; ndarray.ctypes, which takes twice as long, where it must be."""
    if a.size and a.flags.writeable:
        return ctypes.addressof(ctypes.c_char.from_buffer(a))
    return a.ctypes.data


def _heads(t, out, weight, name, shape, device):
    """The fields of one convrot_heads; t and out are [batch, tokens, heads, head_dim]."""
    own = t.shape
    if len(own) != 4 or own[0] != shape[0] or own[1] != shape[1] or own[3] != shape[3]:
        raise ValueError(f"{name} must be [batch, tokens, heads, head_dim], got {tuple(own)}")
    if out.shape != own or out.dtype != t.dtype:
        raise ValueError(f"{name}_out must have the shape and type of {name}")
    tb, tt, th, td = t.stride()
    ob, ot, oh, od = out.stride()
    if shape[3] > 1 and (td != 1 or od != 1):
        raise ValueError(f"{name} and its output must be dense in their last dimension")
    w = 0
    if weight is not None:
        if not isinstance(weight, _torch.Tensor) or weight.get_device() != device or weight.requires_grad:
            _check_tensor(weight, f"{name}_weight", device)
        if weight.dtype != t.dtype or weight.shape != own[3:] or not weight.is_contiguous():
            raise ValueError(f"{name}_weight must be one dense vector of head_dim values of {name}'s type")
        w = weight.data_ptr()
    return t.data_ptr(), out.data_ptr(), w, own[2], tb, tt, th, ob, ot, oh


def convrot_rope(q, k, positions, freq, axis, *, layout: str = "interleaved", qk_norm: bool = False, q_weight=None,
                 k_weight=None, eps: float = 1e-6, q_out=None, k_out=None, stream=None):
    """Turn the pairs of every head by positions[..., axis] * freq.

    q, k: bf16, f16 or f32 [batch, tokens, heads, head_dim] of any strides but a
    dense last one (slices of a packed projection); k may be None.  positions:
    int32 or float32 [batch or 1, tokens, axes].  freq (float64), axis (int32):
    host arrays, one value a pair (``rope_frequencies``).  qk_norm: divide each
    head by its root mean square first, times q_weight / k_weight [head_dim].
    Returns (q_out, k_out); given ones are written and may be q, k themselves or
    transposed views ([batch, heads, tokens, head_dim] storage).  ``stream``: as in
    ``convrot_residual_norm``."""
    device = _on_gpu(q, "q")
    _check_tensor(q, "q", device)
    if getattr(_forward, "_current_level", 0) >= 0:
        _check_tangents(q, k, positions, q_weight, k_weight, q_out, k_out)
    shape, dtype = q.shape, q.dtype
    if len(shape) != 4:
        raise ValueError(f"q must be [batch, tokens, heads, head_dim], got {tuple(shape)}")
    code, order = _type_of(q, "q"), _choice(_LAYOUTS, layout, "layout")
    freq, axis = np.ascontiguousarray(freq, np.float64), np.ascontiguousarray(axis, np.int32)
    if freq.ndim != 1 or freq.shape != axis.shape:
        raise ValueError("freq and axis must hold one value for every pair")
    if not isinstance(positions, _torch.Tensor) or positions.get_device() != device or positions.requires_grad:
        _check_tensor(positions, "positions", device)
    if positions.dtype == _torch.int32:
        pos_code = CONVROT_I32
    elif positions.dtype == _torch.float32:
        pos_code = CONVROT_F32
    else:
        raise TypeError(f"positions must be int32 or float32, got {positions.dtype}")
    pos_shape = positions.shape
    if len(pos_shape) != 3 or pos_shape[0] not in (1, shape[0]) or pos_shape[1] != shape[1]:
        raise ValueError(f"positions must be [batch or 1, tokens, axes], got {tuple(pos_shape)}")
    pos_strides = positions.stride()
    if pos_shape[2] > 1 and pos_strides[2] != 1:
        raise ValueError("positions must be dense in their last dimension")
    if k is not None:
        _check_tensor(k, "k", device)
        if k.dtype != dtype:
            raise TypeError("k must have the type of q")
    elif k_weight is not None or k_out is not None:
        raise ValueError("k_weight and k_out need k")

    def call(raw):
        outs, fields = [], []
        for name, t, out, weight in (("q", q, q_out, q_weight), ("k", k, k_out, k_weight)):
            if t is None:
                outs.append(None)
                fields.append((0,) * 10)
                continue
            if out is None:
                out = _torch.empty_like(t, memory_format=_torch.contiguous_format)
            else:
                _check_tensor(out, name + "_out", device)
            outs.append(out)
            fields.append(_heads(t, out, weight, name, shape, device))
        _call("convrot_rope", ROPE_ARGS.pack(
            *fields[0], *fields[1], 1 if k is None else 2, shape[0], shape[1], shape[3], positions.data_ptr(),
            pos_strides[0] if pos_shape[0] > 1 else 0, pos_strides[1], pos_code, pos_shape[2], freq.shape[0],
            _address(freq), _address(axis), order, CONVROT_NORM_RMS if qk_norm else CONVROT_NORM_NONE, code,
            eps), raw)
        if q_out is not None or k_out is not None:
            _written(q_out, k_out)
        return outs[0], outs[1]

    return _launch(device, stream, call, (q, k, positions, q_weight, k_weight, q_out, k_out))


def _check_group(group, K):
    if group not in _GROUPS or K % group:
        raise ValueError(f"group must be 32, 64 or 128 and divide K = {K}, got {group}")


def convrot_quantize_weight_grouped(W, group: int, asymmetric: bool = False, stream=None):
    """W: bf16 or f16 [N, K] -> (codes uint8 [N, K/2], scales [N, K/group] of W's
    type, zeros uint8 [N, K/group], or None unless ``asymmetric``).  ``stream``:
    as in ``convrot_residual_norm``."""
    device = _on_gpu(W, "W")
    if W.dim() != 2 or not W.is_contiguous():
        raise ValueError("W must be a dense [N, K] tensor")
    code = _type_of(W, "W")
    if code == CONVROT_F32:
        raise TypeError("W must be bfloat16 or float16")
    N, K = W.shape
    _check_group(group, K)

    def call(raw):
        codes = _torch.empty((N, K // 2), dtype=_torch.uint8, device=W.device)
        scales = _torch.empty((N, K // group), dtype=W.dtype, device=W.device)
        zeros = _torch.empty((N, K // group), dtype=_torch.uint8, device=W.device) if asymmetric else None
        _call("convrot_quantize_weight_grouped", W.data_ptr(), N, K, group, code, codes.data_ptr(),
              scales.data_ptr(), None if zeros is None else zeros.data_ptr(), raw)
        return codes, scales, zeros

    return _launch(device, stream, call, (W,))


def convrot_linear_grouped(X, codes, scales, zeros, bias, group: int, Y=None, stream=None):
    """Y = X W^T + bias, W = scales * (codes - zeros) in groups of ``group``
    channels.  X: bf16 or f16 [M, K], M <= 32; codes: uint8 [N, K/2] (N x
    packed-K); scales: [N, K/group] of X's type; zeros: uint8 [N, K/group] with
    unsigned codes, None with two's complement ones; bias: [N] or None.
    ``stream``: as in ``convrot_residual_norm``."""
    device = _on_gpu(X, "X")
    if getattr(_forward, "_current_level", 0) >= 0:
        _check_tangents(X, codes, scales, zeros, bias, Y)
    dtype = X.dtype
    code = _type_of(X, "X")
    if code == CONVROT_F32:
        raise TypeError("X must be bfloat16 or float16")
    if X.dim() != 2 or not isinstance(codes, _torch.Tensor) or codes.dim() != 2:
        raise ValueError("X and codes must be matrices")
    M, K = X.shape
    N = codes.shape[0]
    _check_group(group, K)
    byte, groups = _torch.uint8, K // group

    def place(t, name, kind, *shape):
        if not isinstance(t, _torch.Tensor) or t.get_device() != device or t.requires_grad:
            _check_tensor(t, name, device)
        if t.dtype != kind or t.shape != shape:
            raise ValueError(f"{name} must be {kind} {shape}, got {t.dtype} {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    x_ptr, codes_ptr = place(X, "X", dtype, M, K), place(codes, "codes", byte, N, K // 2)
    scales_ptr = place(scales, "scales", dtype, N, groups)
    zeros_ptr = 0 if zeros is None else place(zeros, "zeros", byte, N, groups)
    bias_ptr = 0 if bias is None else place(bias, "bias", dtype, N)

    def call(raw):
        y = X.new_empty((M, N)) if Y is None else Y
        y_ptr = y.data_ptr() if Y is None else place(Y, "Y", dtype, M, N)
        _call("convrot_linear_grouped",
              GROUPED_ARGS.pack(x_ptr, codes_ptr, scales_ptr, zeros_ptr, bias_ptr, y_ptr, M, N, K, group, code), raw)
        if Y is not None:
            _written(Y)
        return y

    return _launch(device, stream, call, (X, codes, scales, zeros, bias, Y))
