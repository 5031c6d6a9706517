"""Python binding of libmq (nested r-bit weight GEMM on B200).

Argument marshalling only: every computation runs in libmq's CUDA kernels.
The function names follow the C ABI in include/mq.h (mq_pack, mq_slice,
mq_gemm, mq_unpack, ...).  PyTorch supplies device memory and streams.

If libmq.so has not been built, importing this package raises; there is no
CPU or PyTorch fallback for any step.
"""
from __future__ import annotations

import ctypes
import functools
import os

__all__ = [
    "MQError", "MqWeights", "NestedWeights", "lib", "library_path",
    "mq_plane_bytes", "mq_scale_bytes", "mq_pack", "mq_slice", "mq_gemm",
    "mq_gemm_workspace_bytes", "mq_unpack", "mq_version", "pack_parent", "gemm",
    "mq_set_gemv_variant", "mq_get_gemv_variant", "GEMV_TC", "GEMV_VIA_GEMM",
    "mq_device_status", "mq_gemm_kernel", "uses_gemv", "KERNEL_GEMV", "KERNEL_GEMM",
    "MqCall", "mq_gemm_chain", "gemm_chain", "pack_fused", "workspace_for", "mq_pack_zeros",
    "MqMx4", "Mx4Matrix", "mx4_quantize", "mx4_from_nested", "mx4_dequantize", "mx4_gemm", "mx4_gemm_bf16",
    "mq_mx4_code_bytes", "mq_mx4_scale_bytes", "mq_mx4_gemm_bf16_workspace_bytes",
    "MqChoice", "bitwidth_search", "layer_errors", "matgptq_prepare", "matgptq_quantize",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libmq.so")

MQ_OK = 0
STATUS = {0: "MQ_OK", 1: "MQ_ERR_INVALID_ARG", 2: "MQ_ERR_UNSUPPORTED",
          3: "MQ_ERR_MISALIGNED", 4: "MQ_ERR_CUDA", 5: "MQ_ERR_TIMEOUT",
          6: "MQ_ERR_WORKSPACE"}


class MQError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class MqWeights(ctypes.Structure):
    """Mirror of the C struct mq_weights (a view, owns nothing)."""
    _fields_ = [("planes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("group", ctypes.c_int32), ("r", ctypes.c_int32),
                ("zeros", ctypes.c_void_p)]                # fp16 zero points or None (symmetric)


class MqMx4(ctypes.Structure):
    """Mirror of the C struct mq_mx4 (an MXFP4 matrix, owns nothing)."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("K", ctypes.c_int64)]


class MqChoice(ctypes.Structure):
    """One candidate of mq_bitwidth_search (mq_choice in include/mq.h)."""
    _fields_ = [("r", ctypes.c_int32), ("bytes", ctypes.c_uint64), ("error", ctypes.c_double)]


class MqCall(ctypes.Structure):
    """One product of mq_gemm_chain (mq_call in include/mq.h)."""
    _fields_ = [("X", ctypes.c_void_p), ("w", ctypes.POINTER(MqWeights)),
                ("M", ctypes.c_int64), ("Y", ctypes.c_void_p)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(library_path):
        raise ImportError(
            f"{library_path} is missing: build it with "
            "`python nested_bit_weight_b200/_build.py` (nvcc, sm_100a)")
    L = ctypes.CDLL(library_path)
    P, I64, I, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    W, X4 = ctypes.POINTER(MqWeights), ctypes.POINTER(MqMx4)
    sig = {
        "mq_plane_bytes": (SZ, [I64, I64, I]),
        "mq_scale_bytes": (SZ, [I64, I64, I]),
        "mq_pack": (I, [P, P, I64, I64, I, P, P, P]),
        "mq_slice": (I, [W, I, W]),
        "mq_gemm_workspace_bytes": (SZ, [I64, I64, I64, I]),
        "mq_gemm": (I, [P, W, I64, I64, I64, P, P, SZ, P]),
        "mq_unpack": (I, [W, P, P]),
        "mq_last_error": (I, []),
        "mq_device_status": (I, []),
        "mq_last_error_string": (ctypes.c_char_p, []),
        "mq_status_string": (ctypes.c_char_p, [I]),
        "mq_version": (ctypes.c_char_p, []),
        "mq_set_gemv_variant": (I, [I]),
        "mq_get_gemv_variant": (I, []),
        "mq_gemm_kernel": (I, [I64, I64, I64, I]),
        "mq_gemm_chain": (I, [ctypes.POINTER(MqCall), I, P, SZ, P]),
        "mq_pack_zeros": (I, [P, I64, I64, I, P, P]),
        "mq_mx4_code_bytes": (SZ, [I64, I64]),
        "mq_mx4_scale_bytes": (SZ, [I64, I64]),
        "mq_mx4_quantize": (I, [P, I, I64, I64, I64, P, P, P]),
        "mq_mx4_from_nested": (I, [W, P, P, P]),
        "mq_mx4_dequantize": (I, [X4, P, I, I64, P]),
        "mq_mx4_gemm": (I, [X4, X4, P, I, I64, P]),
        "mq_mx4_gemm_bf16_workspace_bytes": (SZ, [I64, I64, I64]),
        "mq_mx4_gemm_bf16": (I, [P, I64, I64, X4, P, I, I64, P, SZ, P]),
        "mq_bitwidth_search": (I, [ctypes.POINTER(MqChoice), I, I, ctypes.c_uint64,
                                   ctypes.POINTER(I), ctypes.POINTER(ctypes.c_double)]),
        "mq_matgptq_prepare": (I, [P, I64, ctypes.c_double, P]),
        "mq_matgptq_quantize": (I, [P, I64, I64, P, P, P, I, P, I, I, P, P]),
        "mq_matgptq_quantize_asym": (I, [P, I64, I64, P, P, P, I, P, I, I, P, P, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    return L


lib = _load()


def _check(status: int) -> None:
    if status != MQ_OK:
        raise MQError(status, lib.mq_last_error_string().decode())


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


# ------------------------------------------------------------------ raw C ABI

def mq_plane_bytes(N: int, K: int, r: int) -> int:
    return lib.mq_plane_bytes(N, K, r)


def mq_scale_bytes(N: int, K: int, group: int = 128) -> int:
    return lib.mq_scale_bytes(N, K, group)


def mq_gemm_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    return lib.mq_gemm_workspace_bytes(M, N, K, r)


GEMV_TC, GEMV_VIA_GEMM = 0, 1


def mq_set_gemv_variant(variant: int) -> None:
    _check(lib.mq_set_gemv_variant(variant))


def mq_get_gemv_variant() -> int:
    return lib.mq_get_gemv_variant()


KERNEL_GEMV, KERNEL_GEMM = 1, 2


def mq_gemm_kernel(M: int, N: int, K: int, r: int) -> int:
    """KERNEL_GEMV or KERNEL_GEMM: the kernel mq_gemm would run (0: invalid)."""
    return lib.mq_gemm_kernel(M, N, K, r)


def uses_gemv(M: int, N: int, K: int, r: int) -> bool:
    return mq_gemm_kernel(M, N, K, r) == KERNEL_GEMV


def mq_device_status() -> None:
    """Synchronise the device; raise if a bounded wait in an earlier launch gave up."""
    _check(lib.mq_device_status())


def mq_version() -> str:
    return lib.mq_version().decode()


def mq_pack(codes, scales, planes_out, scales_out, stream=None) -> None:
    """codes uint8 [N, K], scales fp32 [N, K/128] -> planes_out (the 8 tiled
    planes, mq_plane_bytes(N, K, 8) bytes), scales_out (fp16 in the tiled
    block order, mq_scale_bytes(N, K) bytes); all on device."""
    N, K = codes.shape
    _check(lib.mq_pack(codes.data_ptr(), scales.data_ptr(), N, K, 128,
                       planes_out.data_ptr(), scales_out.data_ptr(), _stream(stream)))


def mq_slice(parent: MqWeights, r: int) -> MqWeights:
    out = MqWeights()
    _check(lib.mq_slice(ctypes.byref(parent), r, ctypes.byref(out)))
    return out


def mq_gemm(X, w: MqWeights, Y, workspace=None, stream=None) -> None:
    """Y[M, N] = X[M, K] . W_r^T (bf16 device tensors)."""
    M, K = X.shape
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.mq_gemm(X.data_ptr(), ctypes.byref(w), M, w.N, K, Y.data_ptr(),
                       ws_ptr, ws_bytes, _stream(stream)))


def mq_gemm_chain(calls, workspace=None, stream=None) -> None:
    """Enqueue the products [(X, w, Y), ...] back to back (X, Y bf16 device
    tensors, w an MqWeights view): a call may read the previous call's Y."""
    arr = (MqCall * len(calls))()
    keep = []
    for i, (X, w, Y) in enumerate(calls):
        wp = ctypes.pointer(w)
        keep.append(wp)
        arr[i] = MqCall(X.data_ptr(), wp, X.shape[0], Y.data_ptr())
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.mq_gemm_chain(arr, len(calls), ws_ptr, ws_bytes, _stream(stream)))


def mq_unpack(w: MqWeights, codes_out, stream=None) -> None:
    _check(lib.mq_unpack(ctypes.byref(w), codes_out.data_ptr(), _stream(stream)))


# ------------------------------------------------------------- owning helpers

class NestedWeights:
    """A packed 8-bit parent (device tensors) and its r-bit views; zeros16
    (fp16 zero points, asymmetric variant) or None."""

    def __init__(self, planes, scales16, N: int, K: int, zeros16=None):
        self.planes, self.scales16, self.N, self.K = planes, scales16, N, K
        self.zeros16 = zeros16
        self.parent = MqWeights(planes.data_ptr(), scales16.data_ptr(), N, K, 128, 8,
                                zeros16.data_ptr() if zeros16 is not None else None)

    def view(self, r: int) -> MqWeights:
        return mq_slice(self.parent, r)


def mq_pack_zeros(zeros, zeros_out, stream=None) -> None:
    """zero points fp32 [N, K/128] -> fp16 in the scales' tiled order (device)."""
    N, G = zeros.shape
    _check(lib.mq_pack_zeros(zeros.data_ptr(), N, G * 128, 128, zeros_out.data_ptr(), _stream(stream)))


def pack_parent(codes, scales, stream=None, zeros=None) -> NestedWeights:
    """Allocate the 8-plane buffer and fp16 scales with torch, then mq_pack;
    with `zeros` (fp32 [N, K/128]) the asymmetric variant."""
    import torch
    N, K = codes.shape
    planes = torch.empty(mq_plane_bytes(N, K, 8) // 4, dtype=torch.int32, device=codes.device)
    s16 = torch.empty(mq_scale_bytes(N, K, 128) // 2, dtype=torch.float16, device=codes.device)
    mq_pack(codes, scales, planes, s16, stream)
    z16 = None
    if zeros is not None:
        z16 = torch.empty(mq_scale_bytes(N, K, 128) // 2, dtype=torch.float16, device=codes.device)
        mq_pack_zeros(zeros, z16, stream)
    return NestedWeights(planes, s16, N, K, z16)


def pack_fused(codes_list, scales_list, stream=None) -> NestedWeights:
    """One parent for several layers that share X (q|k|v, gate|up): their
    rows concatenated (codes uint8 [N_i, K], scales fp32 [N_i, K/128] device
    tensors), so one launch computes all of them; Y's columns follow the same
    order (layer i at rows offsets[i] .. offsets[i] + N_i of W)."""
    import torch
    codes = torch.cat(list(codes_list), dim=0).contiguous()
    scales = torch.cat(list(scales_list), dim=0).contiguous()
    w = pack_parent(codes, scales, stream)
    offs, o = [], 0
    for c in codes_list:
        offs.append(o)
        o += c.shape[0]
    w.offsets = offs
    return w


def workspace_for(device, need: int):
    """The cached zero-initialised workspace of `device`, at least `need` bytes."""
    import torch
    key = device.index
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.zeros(max(need, 1 << 20), dtype=torch.uint8, device=device)
        _ws_cache[key] = ws
    return ws


def gemm_chain(calls, stream=None):
    """[(X, NestedWeights, r, Y or None), ...] -> the Y tensors, enqueued as
    one mq_gemm_chain (consecutive launches overlap)."""
    import torch
    views, outs, need = [], [], 0
    for X, weights, r, Y in calls:
        if Y is None:
            Y = torch.empty((X.shape[0], weights.N), dtype=torch.bfloat16, device=X.device)
        views.append((X, weights.view(r), Y))
        outs.append(Y)
        need = max(need, mq_gemm_workspace_bytes(X.shape[0], weights.N, weights.K, r))
    ws = workspace_for(calls[0][0].device, need) if need else None
    mq_gemm_chain(views, ws, stream)
    return outs


def bitwidth_search(table, budget_bytes: int):
    """table[l] = [(r, bytes, error), ...] per layer -> (index chosen per
    layer, summed error): the least summed error within the byte budget
    (mq_bitwidth_search; exact)."""
    L, C = len(table), len(table[0])
    arr = (MqChoice * (L * C))()
    for l, row in enumerate(table):
        if len(row) != C:
            raise ValueError("every layer needs the same number of candidates")
        for j, (r, nbytes, err) in enumerate(row):
            arr[l * C + j] = MqChoice(r, nbytes, err)
    out = (ctypes.c_int * L)()
    total = ctypes.c_double()
    _check(lib.mq_bitwidth_search(arr, L, C, budget_bytes, out, ctypes.byref(total)))
    return list(out), total.value


def matgptq_prepare(H, damp: float = 0.01):
    """U (K x K, fp64, upper) with U^T U = (H + damp * mean(diag H) * I)^-1
    (mq_matgptq_prepare, host)."""
    import numpy as np
    H = np.ascontiguousarray(H, np.float64)
    if H.ndim != 2 or H.shape[0] != H.shape[1]:
        raise ValueError("H must be a square matrix")
    K = H.shape[0]
    U = np.empty((K, K), np.float64)
    _check(lib.mq_matgptq_prepare(H.ctypes.data, K, float(damp), U.ctypes.data))
    return U


def matgptq_quantize(W, U, rs=(3, 4, 8), lambdas=(1.0, 1.0, 1.0),
                     alphas=(1.0, 0.95, 0.9, 0.85, 0.8), threads: int = 0, asymmetric: bool = False):
    """(codes uint8 N x K, scales fp32 N x K/128): the parent codes of the
    nested format from float weights W by the multi-precision column loop
    (mq_matgptq_quantize, host; the inputs of pack_parent).  asymmetric=True:
    (codes, scales, zeros) by mq_matgptq_quantize_asym (zeros: the input of
    pack_parent's `zeros`)."""
    import numpy as np
    W = np.ascontiguousarray(W, np.float32)
    U = np.ascontiguousarray(U, np.float64)
    if W.ndim != 2 or U.shape != (W.shape[1], W.shape[1]):
        raise ValueError("need W of N x K and U of K x K")
    if len(rs) != len(lambdas):
        raise ValueError("one lambda per bit width")
    N, K = W.shape
    rs_a = np.ascontiguousarray(rs, np.int32)
    lam_a = np.ascontiguousarray(lambdas, np.float64)
    al_a = np.ascontiguousarray(alphas, np.float64)
    codes = np.empty((N, K), np.uint8)
    scales = np.empty((N, max(K // 128, 1)), np.float32)
    args = (W.ctypes.data, N, K, U.ctypes.data, rs_a.ctypes.data, lam_a.ctypes.data, len(rs_a),
            al_a.ctypes.data, len(al_a), int(threads), codes.ctypes.data, scales.ctypes.data)
    if asymmetric:
        zeros = np.empty_like(scales)
        _check(lib.mq_matgptq_quantize_asym(*args, zeros.ctypes.data))
        return codes, scales, zeros
    _check(lib.mq_matgptq_quantize(*args))
    return codes, scales


def layer_errors(X, weights: NestedWeights, rs, stream=None):
    """{r: ||X W_r^T - X W_8^T||^2 / ||X W_8^T||^2} for one layer, the outputs
    computed by mq_gemm and reduced on the host in fp64 (the sensitivities a
    bit-width search consumes)."""
    import numpy as np
    ref = gemm(X, weights, 8, stream=stream).float().cpu().numpy().astype(np.float64)
    den = float(np.sum(ref * ref))
    out = {}
    for r in rs:
        y = gemm(X, weights, r, stream=stream).float().cpu().numpy().astype(np.float64)
        out[r] = float(np.sum((y - ref) ** 2)) / den
    return out


_ws_cache: dict = {}


def gemm(X, weights: NestedWeights, r: int, Y=None, stream=None):
    """Y = X . W_r^T with a cached, zero-initialised workspace per device."""
    import torch
    M, K = X.shape
    w = weights.view(r)
    if Y is None:
        Y = torch.empty((M, weights.N), dtype=torch.bfloat16, device=X.device)
    need = mq_gemm_workspace_bytes(M, weights.N, K, r)
    ws = workspace_for(X.device, need) if need else None
    mq_gemm(X, w, Y, ws, stream)
    return Y


# ----------------------------------------------- MXFP4 (microscaled 4-bit floats)

BF16, F16, F32 = 0, 1, 2


def mq_mx4_code_bytes(rows: int, K: int) -> int:
    return lib.mq_mx4_code_bytes(rows, K)


def mq_mx4_scale_bytes(rows: int, K: int) -> int:
    return lib.mq_mx4_scale_bytes(rows, K)


def mq_mx4_gemm_bf16_workspace_bytes(M: int, N: int, K: int) -> int:
    return lib.mq_mx4_gemm_bf16_workspace_bytes(M, N, K)


# Small calls are bound by the host, so the common case of each function below
# (tensors on the current device, its current stream) takes no detours: torch's
# names are looked up once, and no context is entered.
_torch = _u8 = _raw_stream = _get_device = None
_types: dict = {}          # torch dtype -> MQ_* code


def _init() -> None:
    global _torch, _u8, _raw_stream, _get_device
    import torch
    _types.update({torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32})
    _raw_stream, _get_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    _torch, _u8 = torch, torch.uint8


def _dtype_code(dtype) -> int:
    t = _types.get(dtype)
    if t is None:
        raise ValueError(f"dtype {dtype} is not one of bfloat16, float16, float32")
    return t


def _rows(t, what: str):
    """Check a 2-D device tensor whose rows are contiguous: rows, columns, row stride."""
    try:
        n, k = t.shape
        ld, one = t.stride()
        cuda = t.is_cuda
    except (AttributeError, TypeError, ValueError):
        raise ValueError(f"{what} must be a 2-D tensor") from None
    if not cuda:
        raise ValueError(f"{what} must be on a GPU")
    if one != 1 and k > 1:
        raise ValueError(f"{what} must have contiguous rows (stride 1 along the last axis)")
    if n <= 1:
        return n, k, k or 1
    if ld < k:
        raise ValueError(f"the rows of {what} overlap")
    return n, k, ld


def _given(t, what: str, rows: int, cols: int, dtype, device) -> int:
    """Check a tensor given for a result; its row stride."""
    n, k, ld = _rows(t, what)
    if (n, k) != (rows, cols):
        raise ValueError(f"{what} has shape {(n, k)}, expected {(rows, cols)}")
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{what} differs in dtype or device")
    return ld


class _On:
    """`device` current and `stream` current for torch's allocator, so that what
    a call allocates belongs to the stream it runs on."""

    def __init__(self, device, stream):
        torch = _torch
        if stream is None:
            stream = torch.cuda.current_stream(device)
        elif not isinstance(stream, torch.cuda.Stream):
            ptr = int(getattr(stream, "cuda_stream", stream))
            stream = torch.cuda.ExternalStream(ptr, device=device) if ptr else torch.cuda.default_stream(device)
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        self._ctx = torch.cuda.stream(stream)
        self.ptr = stream.cuda_stream

    def __enter__(self):
        self._ctx.__enter__()
        return self.ptr

    def __exit__(self, *exc):
        return self._ctx.__exit__(*exc)


class Mx4Matrix:
    """A rows x K matrix in MXFP4 (device tensors): codes uint8 [rows, K/2] and
    the scale blocks (mq_mx4 in include/mq.h)."""

    _codes = _scales = _struct = None          # made when asked for

    def __init__(self, codes, scales, rows: int, K: int):
        if _torch is None:
            _init()
        for t, n, what in ((codes, mq_mx4_code_bytes(rows, K), "codes"),
                           (scales, mq_mx4_scale_bytes(rows, K), "scales")):
            if t.dtype != _torch.uint8 or not t.is_cuda or not t.is_contiguous() or t.numel() != n:
                raise ValueError(f"{what} must be {n} contiguous uint8 on a GPU")
        if codes.device != scales.device:
            raise ValueError("codes and scales are on different devices")
        self.rows, self.K, self.device = rows, K, codes.device
        self._codes, self._scales, self._like = codes, scales, codes
        self._ptrs = codes.data_ptr(), scales.data_ptr()

    @classmethod
    def empty(cls, rows: int, K: int, device):
        """Uninitialised buffers for a rows x K matrix."""
        if _torch is None:
            _init()
        if _torch.device(device).type != "cuda":
            raise ValueError("an MXFP4 matrix lives on a GPU")
        return _new_mx4(rows, K, _torch.empty(0, device=device))

    @property
    def codes(self):
        if self._codes is None:
            self._codes = self._like[:self.rows * (self.K // 2)].view(self.rows, self.K // 2)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self._scales = self._like[self.rows * (self.K // 2):]
        return self._scales

    @property
    def struct(self) -> MqMx4:
        s = self._struct
        if s is None:
            s = self._struct = MqMx4(*self._ptrs, self.rows, self.K)
        return s


def _new_mx4(rows: int, K: int, like) -> Mx4Matrix:
    """Uninitialised buffers on the device of the tensor `like`, in one allocation:
    the codes (rows of 16-byte multiples), then the scale blocks.  (new_empty
    with the sizes as arguments takes the host 1.5 us, torch.empty 2.3.)"""
    if rows < 0 or K < 32 or K % 32:
        raise ValueError("need rows >= 0 and K a positive multiple of 32")
    m = Mx4Matrix.__new__(Mx4Matrix)
    nc = rows * (K >> 1)
    m._like = buf = like.new_empty(nc + ((rows + 127) >> 7) * ((K + 127) >> 7) * 512, dtype=_u8)
    ptr = buf.data_ptr()
    m._ptrs = ptr, ptr + nc
    m.rows, m.K, m.device = rows, K, buf.device
    return m


def _mx4_out(out, rows: int, K: int, like) -> Mx4Matrix:
    """The matrix for a result: `out`, or new buffers on the device of `like`."""
    if out is None:
        return _new_mx4(rows, K, like)
    if (out.rows, out.K) != (rows, K) or out.device != like.device:
        raise ValueError(f"out is {out.rows} x {out.K} on {out.device}, expected {rows} x {K} on {like.device}")
    return out


def _quantize(X, dt, rows, K, ld, out, st):
    out = _mx4_out(out, rows, K, X)
    codes, scales = out._ptrs
    s = lib.mq_mx4_quantize(X.data_ptr(), dt, rows, K, ld, codes, scales, st)
    if s:
        _check(s)
    return out


def mx4_quantize(X, out: Mx4Matrix | None = None, stream=None) -> Mx4Matrix:
    """Rows of X (bf16, fp16 or fp32 [rows, K], K a multiple of 32) in MXFP4;
    `out` (of the same size) receives them in place of new buffers."""
    if _torch is None:
        _init()
    rows, K, ld = _rows(X, "X")
    dt = _dtype_code(X.dtype)
    device = X.device
    if stream is None and device.index == _get_device():
        return _quantize(X, dt, rows, K, ld, out, _raw_stream(device.index))
    with _On(device, stream) as st:
        return _quantize(X, dt, rows, K, ld, out, st)


def _from_nested(weights, r, out, st):
    w = weights.view(r)
    out = _mx4_out(out, w.N, w.K, weights.planes)
    s = lib.mq_mx4_from_nested(w, *out._ptrs, st)
    if s:
        _check(s)
    return out


def mx4_from_nested(weights: NestedWeights, r: int, out: Mx4Matrix | None = None, stream=None) -> Mx4Matrix:
    """The r-bit model of a nested parent in MXFP4."""
    if _torch is None:
        _init()
    device = weights.planes.device
    if stream is None and device.index == _get_device():
        return _from_nested(weights, r, out, _raw_stream(device.index))
    with _On(device, stream) as st:
        return _from_nested(weights, r, out, st)


def _dequantize(m, dtype, dt, out, st):
    if out is None:
        ld = m.K
        out = m._like.new_empty(m.rows, ld, dtype=dtype)
    else:
        ld = _given(out, "out", m.rows, m.K, dtype, m.device)
    s = lib.mq_mx4_dequantize(m.struct, out.data_ptr(), dt, ld, st)
    if s:
        _check(s)
    return out


def mx4_dequantize(m: Mx4Matrix, dtype=None, out=None, stream=None):
    """The values m stands for, bf16 (default) or fp32; both hold them exactly
    below 2^128 (no converter here makes larger ones)."""
    if dtype is None:
        dtype = out.dtype if out is not None else _torch.bfloat16
    dt = _dtype_code(dtype)
    device = m.device
    if stream is None and device.index == _get_device():
        return _dequantize(m, dtype, dt, out, _raw_stream(device.index))
    with _On(device, stream) as st:
        return _dequantize(m, dtype, dt, out, st)


def _mx4_y(Y, M: int, w: Mx4Matrix, dtype):
    """The tensor for a product's result, its dtype's code and its row stride."""
    if Y is None:
        if dtype is None:
            dtype = _torch.bfloat16
        N = w.rows
        return w._like.new_empty(M, N, dtype=dtype), _dtype_code(dtype), N
    if dtype is None:
        dtype = Y.dtype
    dt = _dtype_code(dtype)
    return Y, dt, _given(Y, "Y", M, w.rows, dtype, w.device)


def _gemm4(X, w, Y, dtype, st):
    Y, dt, ldy = _mx4_y(Y, X.rows, w, dtype)
    s = lib.mq_mx4_gemm(X.struct, w.struct, Y.data_ptr(), dt, ldy, st)
    if s:
        _check(s)
    return Y


def mx4_gemm(X: Mx4Matrix, w: Mx4Matrix, Y=None, dtype=None, stream=None):
    """Y = X . w^T, both in MXFP4 (X: M x K, w: N x K); Y bf16 (default), fp16
    or fp32 [M, N]."""
    device = w.device
    if X.device != device:
        raise ValueError("X and w are on different devices")
    if stream is None and device.index == _get_device():
        return _gemm4(X, w, Y, dtype, _raw_stream(device.index))
    with _On(device, stream) as st:
        return _gemm4(X, w, Y, dtype, st)


@functools.lru_cache(maxsize=1024)
def _ws16(M: int, N: int, K: int) -> int:
    return lib.mq_mx4_gemm_bf16_workspace_bytes(M, N, K)


def _gemm16(X, M, ldx, w, Y, dtype, st):
    Y, dt, ldy = _mx4_y(Y, M, w, dtype)
    # the workspace is this call's own, on its stream
    need = _ws16(M, w.rows, w.K) if M > 2 else 0
    ws = w._like.new_empty(need, dtype=_u8) if need else None
    s = lib.mq_mx4_gemm_bf16(X.data_ptr(), M, ldx, w.struct, Y.data_ptr(), dt, ldy,
                             ws.data_ptr() if need else None, need, st)
    if s:
        _check(s)
    return Y


def mx4_gemm_bf16(X, w: Mx4Matrix, Y=None, dtype=None, stream=None):
    """Y = X . w^T with X in bf16 [M, K], w in MXFP4.  X is taken to within 2^-22
    of the largest value of each block of 32 (mq_mx4_gemm_bf16)."""
    M, K, ldx = _rows(X, "X")
    if K != w.K:
        raise ValueError(f"X has {K} columns, expected {w.K}")
    if X.dtype != _torch.bfloat16:
        raise ValueError("X must be bfloat16")
    device = w.device
    if X.device != device:
        raise ValueError("X and w are on different devices")
    if stream is None and device.index == _get_device():
        return _gemm16(X, M, ldx, w, Y, dtype, _raw_stream(device.index))
    with _On(device, stream) as st:
        return _gemm16(X, M, ldx, w, Y, dtype, st)
