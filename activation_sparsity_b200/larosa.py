"""Python binding of liblarosa.so: argument marshalling only.

Every function here has the name of the C entry point it calls, takes torch
tensors that live on a CUDA device, passes their data pointers, sizes and the
current CUDA stream to the library, and raises LarosaError on a nonzero
status.  All arithmetic happens in the library's CUDA kernels; there is no
CPU or PyTorch fallback, and importing this module fails if the library has
not been built.

Tensors must be contiguous.  Output tensors and the workspace may be passed
in; when omitted they are allocated with torch (the only thing PyTorch does
here besides providing the stream).
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblarosa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m activation_sparsity_b200.build_lib` "
        "(there is no fallback implementation)")

_lib = ctypes.CDLL(LIB_PATH)

_c = ctypes
_vp, _i, _sz = _c.c_void_p, _c.c_int, _c.c_size_t

_SIGNATURES = {
    "larosa_status_string": ([_i], _c.c_char_p),
    "larosa_version": ([], _i),
    "larosa_last_error_string": ([], _c.c_char_p),
    "larosa_prepare_weights": ([_vp, _vp, _vp, _i, _i, _i, _vp], _i),
    "larosa_fold_rotation": ([_vp, _vp, _vp, _i, _i, _i, _vp], _i),
    "larosa_rotate": ([_vp, _vp, _vp, _i, _i, _i, _vp], _i),
    "larosa_topk": ([_vp, _i, _i, _i, _vp, _vp, _vp, _vp], _i),
    "larosa_rotate_topk": ([_vp, _vp, _vp, _vp, _vp, _i, _i, _vp, _sz, _vp, _i, _vp], _i),
    "larosa_sparse_linear": ([_vp, _vp, _i, _i, _vp, _i, _i, _vp, _vp, _sz, _i, _vp, _vp], _i),
    "larosa_rotate_topk_linear": ([_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _sz, _vp, _i, _vp], _i),
    "larosa_topk_linear": ([_vp, _vp, _i, _i, _i, _i, _vp, _vp, _sz, _vp, _i, _vp], _i),
    "larosa_threshold": ([_vp, _i, _i, _c.c_float, _vp, _vp, _vp, _vp, _vp], _i),
    "larosa_rotate_threshold_linear": ([_vp, _vp, _vp, _i, _i, _i, _c.c_float, _vp, _vp, _sz, _vp, _i,
                                        _vp], _i),
    "larosa_dense_linear": ([_vp, _vp, _i, _i, _i, _vp, _i, _vp], _i),
    "larosa_sparse_lowrank_linear": ([_vp, _vp, _vp, _i, _i, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _sz, _i, _vp,
                                      _vp], _i),
    "larosa_lowrank_workspace_bytes": ([_i, _i, _i, _i, _i], _sz),
    "larosa_sparse_linear_noalloc": ([_vp, _vp, _i, _i, _vp, _i, _i, _vp, _i, _vp, _vp], _i),
    "larosa_sparse_linear_noalloc_bytes": ([_i, _i, _i, _i, _i], _sz),
    "larosa_mx4_quantize": ([_vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp], _i),
    "larosa_mx4_dequantize": ([_vp, _vp, _i, _i, _i, _i, _vp, _vp], _i),
    "larosa_mx4_linear": ([_vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _sz, _vp, _i, _vp], _i),
    "larosa_mx4_linear_workspace_bytes": ([_i, _i, _i], _sz),
    "larosa_mx4_sparse_linear": ([_vp, _vp, _i, _i, _vp, _vp, _i, _i, _vp, _vp, _sz, _vp, _vp], _i),
    "larosa_mx4_topk_linear": ([_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _sz, _vp, _vp], _i),
    "larosa_moe_layer": ([_vp] * 6 + [_i] * 6 + [_vp] * 4 + [_sz, _vp, _i, _vp], _i),
    "larosa_moe_workspace_bytes": ([_i, _i, _i, _i, _i], _sz),
    "larosa_workspace_sync_offset": ([_i, _i, _i, _i, _c.POINTER(_sz)], _i),
    "larosa_set_wait_limit_ns": ([_c.c_uint64, _c.POINTER(_c.c_uint64)], _i),
    "larosa_set_debug": ([_i, _c.POINTER(_i)], _i),
    "larosa_set_split_k": ([_i, _c.POINTER(_i)], _i),
    "larosa_workspace_bytes": ([_i, _i, _i, _i], _sz),
    "larosa_workspace_layout": ([_i, _i, _i, _i, _c.POINTER(_sz), _c.POINTER(_sz), _c.POINTER(_sz)], _i),
    "larosa_workspace_nnz_offset": ([_i, _i, _i, _i, _c.POINTER(_sz)], _i),
    "larosa_check": ([_vp, _vp, _c.POINTER(_i)], _i),
}
for _name, (_args, _ret) in _SIGNATURES.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _ret

LAROSA_F32 = 0
LAROSA_BF16 = 1
LAROSA_OK = 0
LAROSA_ERR_NONFINITE = 7
LAROSA_ERR_TIMEOUT = 8
LAROSA_ERR_INDEX = 9
LAROSA_ERR_LIST = 10
LAROSA_DEV_NONFINITE = 0x1
LAROSA_DEV_TIMEOUT = 0x2
LAROSA_DEV_INDEX = 0x4
LAROSA_DEV_LIST = 0x8
LAROSA_MAX_SPLIT_K = 8
LAROSA_MAX_M = 16
LAROSA_MAX_D = 32768
LAROSA_MX4_BLOCK = 32
LAROSA_MX4_MAX_M = 1048576
LAROSA_MOE_MAX_E = 512
LAROSA_MOE_MAX_K = 16
LAROSA_NOALLOC_SCRATCH_BYTES = 2 << 20


class LarosaError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = _lib.larosa_status_string(status).decode()
        detail = _lib.larosa_last_error_string().decode()
        super().__init__(f"{where}: {msg}" + (f" ({detail})" if detail and status == 5 else ""))
        self.status = status


def _check(status: int, where: str) -> None:
    if status != LAROSA_OK:
        raise LarosaError(status, where)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _as2d(t: torch.Tensor) -> torch.Tensor:
    return t if t.dim() == 2 else t.reshape(1, -1)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return LAROSA_BF16
    if t.dtype == torch.float32:
        return LAROSA_F32
    raise TypeError(f"unsupported dtype {t.dtype}: bfloat16 or float32")


def _need(t: torch.Tensor, name: str, dtype=None) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


# ------------------------------------------------------------------ workspace

_cuda_driver = None


def _capture_id(device: torch.device) -> int:
    """The number of the capture that the device's current stream takes part in, 0 outside of one."""
    global _cuda_driver
    with torch.cuda.device(device):
        if not torch.cuda.is_current_stream_capturing():
            return 0
    if _cuda_driver is None:
        _cuda_driver = ctypes.CDLL("libcuda.so.1")
    state, number = ctypes.c_int(0), ctypes.c_uint64(0)
    status = _cuda_driver.cuStreamGetCaptureInfo_v2(_stream(device), ctypes.byref(state), ctypes.byref(number),
                                                    None, None, None)
    if status != 0:
        raise RuntimeError(f"cuStreamGetCaptureInfo_v2: error {status}")
    return number.value


class Workspace:
    """A zero-initialised scratch buffer for one stream, grown on demand.

    The library leaves the counter words it uses at zero after every call, so
    the buffer is reused without clearing.  A buffer serves one stream at a
    time; calls on different streams that may overlap need their own, and so do
    graphs that may be replayed at the same time.

    A captured graph goes on using the buffer it was captured with: one that
    has been outgrown is kept (sizes at least double, so that together they are no
    larger than the last).  A buffer that had to be made inside a capture is
    zeroed by that graph, at every replay and at no other time, so nothing
    outside of that capture uses it.
    """

    def __init__(self, device=None):
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None \
            else torch.device(device)
        self.buf = torch.zeros(0, dtype=torch.uint8, device=self.device)
        self._need: dict[tuple, int] = {}  # by the name of the size query and its arguments
        self._outgrown: list[torch.Tensor] = []
        self._capture = 0  # the capture that buf was made in, 0: none

    def get(self, M: int, d_in: int, d_out: int, K: int) -> torch.Tensor:
        return self._sized(("larosa_workspace_bytes", M, d_in, d_out, K))

    def get_mx4_linear(self, M: int, d_in: int, d_out: int) -> torch.Tensor:
        """The buffer for larosa_mx4_linear of these sizes."""
        return self._sized(("larosa_mx4_linear_workspace_bytes", M, d_in, d_out))

    def get_moe(self, M: int, d: int, f: int, E: int, k: int) -> torch.Tensor:
        """The buffer for larosa_moe_layer of these sizes."""
        return self._sized(("larosa_moe_workspace_bytes", M, d, f, E, k))

    def _sized(self, query: tuple) -> torch.Tensor:
        """The buffer for a size query: the name of the library's function, then its arguments."""
        need = self._need.get(query)
        if need is None:
            with torch.cuda.device(self.device):
                need = int(getattr(_lib, query[0])(*query[1:]))
            if need == 0:
                raise LarosaError(2, query[0])
            self._need[query] = need
        if self.buf.numel() < need or self._capture:
            self._renew(need)
        return self.buf

    def _renew(self, need: int) -> None:
        """A buffer of at least `need` bytes that may be used where the caller is."""
        capture, have = _capture_id(self.device), self.buf.numel()
        if have >= need and capture == self._capture:
            return
        if have and not self._capture:  # (one made in a capture belongs to that graph's memory)
            self._outgrown.append(self.buf)
        self.buf = torch.zeros(have if have >= need else max(need, 2 * have), dtype=torch.uint8, device=self.device)
        self._capture = capture

    def reset(self) -> None:
        """Zero the buffer again, and those that graphs may still use (needed after a device-side error)."""
        for buf in (*self._outgrown, self.buf):
            buf.zero_()


_ws_lock = threading.Lock()
_ws_cache: dict[tuple[int, int], Workspace] = {}
_status_cache: dict[int, torch.Tensor] = {}


def default_workspace(device: torch.device) -> Workspace:
    key = (device.index, torch.cuda.current_stream(device).cuda_stream)
    with _ws_lock:
        ws = _ws_cache.get(key)
        if ws is None:
            ws = _ws_cache[key] = Workspace(device)
        return ws


def default_status(device: torch.device) -> torch.Tensor:
    """The per-device status word used when none is passed (see larosa_check)."""
    with _ws_lock:
        st = _status_cache.get(device.index)
        if st is None:
            st = _status_cache[device.index] = torch.zeros(1, dtype=torch.int32, device=device)
        return st


def _ws_args(ws, device, M, d_in, d_out, K):
    if ws is None:
        ws = default_workspace(device)
    buf = ws.get(M, d_in, d_out, K) if isinstance(ws, Workspace) else ws
    return ctypes.c_void_p(buf.data_ptr()), ctypes.c_size_t(buf.numel() * buf.element_size())


def _status_ptr(dev_status, device):
    return _ptr(default_status(device) if dev_status is None else dev_status)


# ------------------------------------------------------------------ entry points

def larosa_version() -> int:
    return int(_lib.larosa_version())


def larosa_workspace_bytes(M: int, d_in: int, d_out: int, K: int) -> int:
    return int(_lib.larosa_workspace_bytes(M, d_in, d_out, K))


def larosa_lowrank_workspace_bytes(M: int, d_in: int, d_out: int, K: int, r: int) -> int:
    return int(_lib.larosa_lowrank_workspace_bytes(M, d_in, d_out, K, r))


def larosa_workspace_layout(M: int, d_in: int, d_out: int, K: int) -> tuple[int, int, int]:
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(_lib.larosa_workspace_layout(M, d_in, d_out, K, ctypes.byref(a), ctypes.byref(b),
                                        ctypes.byref(c)), "larosa_workspace_layout")
    return a.value, b.value, c.value


def larosa_workspace_nnz_offset(M: int, d_in: int, d_out: int, K: int) -> int:
    a = ctypes.c_size_t()
    _check(_lib.larosa_workspace_nnz_offset(M, d_in, d_out, K, ctypes.byref(a)),
           "larosa_workspace_nnz_offset")
    return a.value


def larosa_workspace_sync_offset(M: int, d_in: int, d_out: int, K: int) -> int:
    a = ctypes.c_size_t()
    _check(_lib.larosa_workspace_sync_offset(M, d_in, d_out, K, ctypes.byref(a)),
           "larosa_workspace_sync_offset")
    return a.value


def larosa_set_wait_limit_ns(limit_ns: int) -> int:
    """Sets the in-kernel wait limit for later launches (0: the default);
    returns the previous limit."""
    prev = ctypes.c_uint64(0)
    _check(_lib.larosa_set_wait_limit_ns(int(limit_ns), ctypes.byref(prev)), "larosa_set_wait_limit_ns")
    return prev.value


def larosa_set_debug(on: bool) -> bool:
    """Turns the library's debug checks of kept lists on or off for later
    calls; returns the previous setting (see larosa_set_debug in the header)."""
    prev = ctypes.c_int(0)
    _check(_lib.larosa_set_debug(1 if on else 0, ctypes.byref(prev)), "larosa_set_debug")
    return bool(prev.value)


def larosa_set_split_k(splits: int) -> int:
    """Forces the reduction split of the tensor-core kernels of 2 to 16 tokens
    (0: chosen per shape); returns the previous setting."""
    prev = ctypes.c_int(0)
    _check(_lib.larosa_set_split_k(int(splits), ctypes.byref(prev)), "larosa_set_split_k")
    return prev.value


def larosa_sparse_linear_noalloc_bytes(M: int, d_in: int, d_out: int, K: int,
                                       dtype: torch.dtype = torch.bfloat16) -> int:
    code = LAROSA_BF16 if dtype == torch.bfloat16 else LAROSA_F32
    return int(_lib.larosa_sparse_linear_noalloc_bytes(M, d_in, d_out, K, code))


def larosa_prepare_weights(Qt: torch.Tensor, W: torch.Tensor, W_rot: torch.Tensor | None = None
                           ) -> torch.Tensor:
    """W_rot = Q^T . W = Qt . W (offline counter-rotation), same dtype as W.

    Qt is the rotation stored transposed (Qt = Q.T.contiguous() for x_rot = x @ Q).
    """
    _need(Qt, "Qt")
    _need(W, "W", Qt.dtype)
    d_in, d_out = W.shape
    if W_rot is None:
        W_rot = torch.empty_like(W)
    _need(W_rot, "W_rot", W.dtype)
    _check(_lib.larosa_prepare_weights(_ptr(Qt), _ptr(W), _ptr(W_rot), d_in, d_out, _dtype_code(W),
                                       _stream(W.device)), "larosa_prepare_weights")
    return W_rot


def larosa_fold_rotation(Qt: torch.Tensor, Wt_prev: torch.Tensor, out: torch.Tensor | None = None
                         ) -> torch.Tensor:
    """Q^T . Wt_prev: the producer's nn.Linear weight [d, d_prev] after folding the
    rotation into it, so that the producer outputs x . Q."""
    _need(Qt, "Qt")
    _need(Wt_prev, "Wt_prev", Qt.dtype)
    d, d_prev = Wt_prev.shape
    if out is None:
        out = torch.empty_like(Wt_prev)
    _need(out, "out", Wt_prev.dtype)
    _check(_lib.larosa_fold_rotation(_ptr(Qt), _ptr(Wt_prev), _ptr(out), d, d_prev, _dtype_code(Wt_prev),
                                     _stream(Wt_prev.device)), "larosa_fold_rotation")
    return out


def larosa_rotate(x: torch.Tensor, Qt: torch.Tensor, x_rot: torch.Tensor | None = None
                  ) -> torch.Tensor:
    """x_rot = x . Q with Qt = Q^T, fp32 output [M, d]."""
    _need(x, "x")
    _need(Qt, "Qt", x.dtype)
    x2 = _as2d(x)
    M, d = x2.shape
    if x_rot is None:
        x_rot = torch.empty((M, d), dtype=torch.float32, device=x.device)
    _need(x_rot, "x_rot", torch.float32)
    _check(_lib.larosa_rotate(_ptr(x2), _ptr(Qt), _ptr(x_rot), M, d, _dtype_code(x),
                              _stream(x.device)), "larosa_rotate")
    return x_rot


def larosa_topk(x_rot: torch.Tensor, K: int, idx: torch.Tensor | None = None,
                val: torch.Tensor | None = None, dev_status: torch.Tensor | None = None
                ) -> tuple[torch.Tensor, torch.Tensor]:
    """Per-row Top-K by magnitude: (idx int32 [M, K] ascending, val fp32 [M, K])."""
    _need(x_rot, "x_rot", torch.float32)
    x2 = _as2d(x_rot)
    M, d = x2.shape
    if idx is None:
        idx = torch.empty((M, K), dtype=torch.int32, device=x_rot.device)
    if val is None:
        val = torch.empty((M, K), dtype=torch.float32, device=x_rot.device)
    _need(idx, "idx", torch.int32)
    _need(val, "val", torch.float32)
    _check(_lib.larosa_topk(_ptr(x2), M, d, K, _ptr(idx), _ptr(val),
                            _status_ptr(dev_status, x_rot.device), _stream(x_rot.device)),
           "larosa_topk")
    return idx, val


def larosa_rotate_topk(x: torch.Tensor, Qt: torch.Tensor, K: int, x_rot: torch.Tensor | None = None,
                       idx: torch.Tensor | None = None, val: torch.Tensor | None = None, ws=None,
                       dev_status: torch.Tensor | None = None
                       ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """One token: x_rot = x @ Q (Qt = Q^T) and its Top-K by magnitude in one
    kernel; returns (x_rot fp32 [1, d], idx int32 [1, K] ascending, val fp32 [1, K])."""
    _need(x, "x")
    _need(Qt, "Qt", x.dtype)
    x2 = _as2d(x)
    M, d = x2.shape
    if M != 1:
        raise LarosaError(2, "larosa_rotate_topk: one token only")
    if x_rot is None:
        x_rot = torch.empty((1, d), dtype=torch.float32, device=x.device)
    if idx is None:
        idx = torch.empty((1, K), dtype=torch.int32, device=x.device)
    if val is None:
        val = torch.empty((1, K), dtype=torch.float32, device=x.device)
    _need(x_rot, "x_rot", torch.float32)
    _need(idx, "idx", torch.int32)
    _need(val, "val", torch.float32)
    p, n = _ws_args(ws, x.device, 1, d, 1, K)
    _check(_lib.larosa_rotate_topk(_ptr(x2), _ptr(Qt), _ptr(x_rot), _ptr(idx), _ptr(val), d, K, p, n,
                                   _status_ptr(dev_status, x.device), _dtype_code(x),
                                   _stream(x.device)), "larosa_rotate_topk")
    return x_rot, idx, val


def larosa_sparse_linear(idx: torch.Tensor, val: torch.Tensor, W_rot: torch.Tensor,
                         y: torch.Tensor | None = None, ws=None,
                         dev_status: torch.Tensor | None = None) -> torch.Tensor:
    """y = sum_k val[:, k] * W_rot[idx[:, k]], fp32 [M, d_out]."""
    _need(idx, "idx", torch.int32)
    _need(val, "val", torch.float32)
    _need(W_rot, "W_rot")
    i2 = _as2d(idx)
    val = _as2d(val)
    M, K = i2.shape
    d_in, d_out = W_rot.shape
    if y is None:
        y = torch.empty((M, d_out), dtype=torch.float32, device=W_rot.device)
    _need(y, "y", torch.float32)
    p, n = _ws_args(ws, W_rot.device, M, d_in, d_out, K)
    _check(_lib.larosa_sparse_linear(_ptr(i2), _ptr(val), M, K, _ptr(W_rot), d_in, d_out, _ptr(y),
                                     p, n, _dtype_code(W_rot), _status_ptr(dev_status, W_rot.device),
                                     _stream(W_rot.device)), "larosa_sparse_linear")
    return y


def larosa_sparse_linear_noalloc(idx: torch.Tensor, val: torch.Tensor, W_rot: torch.Tensor,
                                 y: torch.Tensor | None = None,
                                 dev_status: torch.Tensor | None = None) -> torch.Tensor:
    """larosa_sparse_linear with the library's fixed device scratch instead of a
    workspace (for callers that cannot allocate); calls on one device must not
    overlap."""
    _need(idx, "idx", torch.int32)
    _need(val, "val", torch.float32)
    _need(W_rot, "W_rot")
    i2 = _as2d(idx)
    val = _as2d(val)
    M, K = i2.shape
    d_in, d_out = W_rot.shape
    if y is None:
        y = torch.empty((M, d_out), dtype=torch.float32, device=W_rot.device)
    _need(y, "y", torch.float32)
    status = _lib.larosa_sparse_linear_noalloc(_ptr(i2), _ptr(val), M, K, _ptr(W_rot), d_in, d_out,
                                               _ptr(y), _dtype_code(W_rot),
                                               _status_ptr(dev_status, W_rot.device),
                                               _stream(W_rot.device))
    if status != LAROSA_OK:
        raise LarosaError(status, "larosa_sparse_linear_noalloc: "
                          + _lib.larosa_last_error_string().decode())
    return y


def larosa_rotate_topk_linear(x: torch.Tensor, Qt: torch.Tensor | None, W_rot: torch.Tensor, K: int,
                              y: torch.Tensor | None = None, ws=None,
                              dev_status: torch.Tensor | None = None) -> torch.Tensor:
    """Fused rotate -> Top-K -> sparse linear (Qt = Q^T), fp32 output [M, d_out].

    Qt = None is the identity rotation (the unrotated fixed-K mode)."""
    _need(x, "x")
    if Qt is not None:
        _need(Qt, "Qt", x.dtype)
    _need(W_rot, "W_rot", x.dtype)
    x2 = _as2d(x)
    M, d_in = x2.shape
    d_out = W_rot.shape[1]
    if y is None:
        y = torch.empty((M, d_out), dtype=torch.float32, device=x.device)
    _need(y, "y", torch.float32)
    p, n = _ws_args(ws, x.device, M, d_in, d_out, K)
    _check(_lib.larosa_rotate_topk_linear(_ptr(x2), _ptr(Qt), _ptr(W_rot), M, d_in, d_out, K, _ptr(y),
                                          p, n, _status_ptr(dev_status, x.device), _dtype_code(x),
                                          _stream(x.device)), "larosa_rotate_topk_linear")
    return y


def larosa_topk_linear(x_rot: torch.Tensor, W_rot: torch.Tensor, K: int, y: torch.Tensor | None = None,
                       ws=None, dev_status: torch.Tensor | None = None) -> torch.Tensor:
    """Top-K of an already rotated fp32 vector and the sparse linear over the kept
    rows of W_rot, fp32 output [M, d_out] (the kept list stays in the workspace)."""
    _need(x_rot, "x_rot", torch.float32)
    _need(W_rot, "W_rot")
    x2 = _as2d(x_rot)
    M, d_in = x2.shape
    d_out = W_rot.shape[1]
    if W_rot.shape[0] != d_in:
        raise ValueError("W_rot must be [d_in, d_out]")
    if y is None:
        y = torch.empty((M, d_out), dtype=torch.float32, device=x_rot.device)
    _need(y, "y", torch.float32)
    p, n = _ws_args(ws, x_rot.device, M, d_in, d_out, K)
    _check(_lib.larosa_topk_linear(_ptr(x2), _ptr(W_rot), M, d_in, d_out, K, _ptr(y), p, n,
                                   _status_ptr(dev_status, x_rot.device), _dtype_code(W_rot),
                                   _stream(x_rot.device)), "larosa_topk_linear")
    return y


def larosa_threshold(x_rot: torch.Tensor, t: float, idx: torch.Tensor | None = None,
                     val: torch.Tensor | None = None, nnz: torch.Tensor | None = None,
                     dev_status: torch.Tensor | None = None
                     ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Per-row threshold selection |x_rot| >= t: (idx int32 [M, d], val fp32 [M, d],
    nnz int32 [M]); row m's first nnz[m] entries are the kept ones, ascending."""
    _need(x_rot, "x_rot", torch.float32)
    x2 = _as2d(x_rot)
    M, d = x2.shape
    dev = x_rot.device
    if idx is None:
        idx = torch.empty((M, d), dtype=torch.int32, device=dev)
    if val is None:
        val = torch.empty((M, d), dtype=torch.float32, device=dev)
    if nnz is None:
        nnz = torch.empty((M,), dtype=torch.int32, device=dev)
    _need(idx, "idx", torch.int32)
    _need(val, "val", torch.float32)
    _need(nnz, "nnz", torch.int32)
    _check(_lib.larosa_threshold(_ptr(x2), M, d, float(t), _ptr(idx), _ptr(val), _ptr(nnz),
                                 _status_ptr(dev_status, dev), _stream(dev)), "larosa_threshold")
    return idx, val, nnz


def larosa_rotate_threshold_linear(x: torch.Tensor, Qt: torch.Tensor | None, W_rot: torch.Tensor,
                                   t: float, y: torch.Tensor | None = None, ws=None,
                                   dev_status: torch.Tensor | None = None) -> torch.Tensor:
    """Fused rotate -> threshold |x_rot| >= t -> sparse linear, fp32 output [M, d_out].

    Qt = None is the identity rotation.  The kept lists and counts stay in the
    workspace (larosa_workspace_layout / larosa_workspace_nnz_offset with K = d_in)."""
    _need(x, "x")
    if Qt is not None:
        _need(Qt, "Qt", x.dtype)
    _need(W_rot, "W_rot", x.dtype)
    x2 = _as2d(x)
    M, d_in = x2.shape
    d_out = W_rot.shape[1]
    if y is None:
        y = torch.empty((M, d_out), dtype=torch.float32, device=x.device)
    _need(y, "y", torch.float32)
    p, n = _ws_args(ws, x.device, M, d_in, d_out, d_in)
    _check(_lib.larosa_rotate_threshold_linear(_ptr(x2), _ptr(Qt), _ptr(W_rot), M, d_in, d_out, float(t),
                                               _ptr(y), p, n, _status_ptr(dev_status, x.device),
                                               _dtype_code(x), _stream(x.device)),
           "larosa_rotate_threshold_linear")
    return y


def larosa_sparse_lowrank_linear(x: torch.Tensor, idx: torch.Tensor, val: torch.Tensor, W: torch.Tensor,
                                 A_r: torch.Tensor, B_r: torch.Tensor, y: torch.Tensor | None = None,
                                 ws: torch.Tensor | None = None, dev_status: torch.Tensor | None = None
                                 ) -> torch.Tensor:
    """y = sparse(x) . W + ((x - sparse(x)) . A_r) . B_r for the kept lists idx/val of x (fp32)."""
    _need(x, "x", torch.float32)
    _need(W, "W")
    _need(A_r, "A_r", W.dtype)
    _need(B_r, "B_r", W.dtype)
    x2 = _as2d(x)
    M, d_in = x2.shape
    d_out, r = W.shape[1], A_r.shape[1]
    idx2, val2 = _as2d(idx), _as2d(val)
    K = idx2.shape[1]
    _need(idx2, "idx", torch.int32)
    _need(val2, "val", torch.float32)
    if y is None:
        y = torch.empty((M, d_out), dtype=torch.float32, device=x.device)
    _need(y, "y", torch.float32)
    nb = int(_lib.larosa_lowrank_workspace_bytes(M, d_in, d_out, K, r))
    if nb == 0:
        raise LarosaError(2, "larosa_lowrank_workspace_bytes")
    if ws is None or ws.numel() * ws.element_size() < nb:
        ws = torch.zeros(nb, dtype=torch.uint8, device=x.device)
    _check(_lib.larosa_sparse_lowrank_linear(_ptr(x2), _ptr(idx2), _ptr(val2), M, K, _ptr(W), _ptr(A_r),
                                             _ptr(B_r), d_in, d_out, r, _ptr(y), _ptr(ws),
                                             ws.numel() * ws.element_size(), _dtype_code(W),
                                             _status_ptr(dev_status, x.device), _stream(x.device)),
           "larosa_sparse_lowrank_linear")
    return y


def larosa_dense_linear(x: torch.Tensor, Wt: torch.Tensor, y: torch.Tensor | None = None
                        ) -> torch.Tensor:
    """Dense baseline y = x . W with Wt = W^T in torch.nn.Linear layout [d_out, d_in]."""
    _need(x, "x")
    _need(Wt, "Wt", x.dtype)
    x2 = _as2d(x)
    M, d_in = x2.shape
    d_out = Wt.shape[0]
    if Wt.shape[1] != d_in:
        raise ValueError("Wt must be [d_out, d_in]")
    if y is None:
        y = torch.empty((M, d_out), dtype=torch.float32, device=x.device)
    _need(y, "y", torch.float32)
    _check(_lib.larosa_dense_linear(_ptr(x2), _ptr(Wt), M, d_in, d_out, _ptr(y), _dtype_code(x),
                                    _stream(x.device)), "larosa_dense_linear")
    return y


# The calls below are short next to what Python spends around them (a one-token
# product takes 5 to 10 us on the device), so they pass plain integers to
# ctypes, compare device numbers instead of device objects, ask for the raw
# stream and enter a device context only where the tensors' device is not the
# current one.

_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _need_fast(t: torch.Tensor, name: str, dtype: torch.dtype, dev: int) -> None:
    """_need, and on the device (number) of the call's other tensors."""
    if not (isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype is dtype and t.is_contiguous()):
        _need(t, name, dtype)
        raise ValueError(f"{name} is on {t.device}, the other tensors are on cuda:{dev}")


def _need_out(t: torch.Tensor, name: str, shape: tuple, dtype: torch.dtype, dev: int) -> None:
    """A given output: type, device, size."""
    _need_fast(t, name, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _need_typed(t: torch.Tensor, name: str, shape: tuple, dtype: torch.dtype | None, dev: int) -> None:
    """A given output whose type the caller chooses, by `dtype` or (None) by the output itself."""
    _need_out(t, name, shape, getattr(t, "dtype", None) if dtype is None else dtype, dev)


def _call(where: str, dev: int, fn, args: tuple) -> None:
    """fn(*args, stream) on device `dev`, on its current stream."""
    if _current_device() == dev:
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status != LAROSA_OK:
        raise LarosaError(status, where)


def _status_word(dev_status: torch.Tensor | None, dev: int) -> int:
    if dev_status is None:
        st = _status_cache.get(dev)
        return (default_status(torch.device("cuda", dev)) if st is None else st).data_ptr()
    _need_fast(dev_status, "dev_status", torch.int32, dev)
    return dev_status.data_ptr()


def _ws_pair(ws, dev: int, query: tuple) -> tuple[int, int]:
    """(address, bytes) of a workspace for a size query (see Workspace._sized);
    ws: a Workspace, a tensor, or None for the current stream's own."""
    if ws is None:
        ws = _ws_cache.get((dev, _raw_stream(dev)))
        if ws is None:
            ws = default_workspace(torch.device("cuda", dev))
    if isinstance(ws, Workspace):
        buf = ws.buf
        n = buf.numel()  # of bytes
        need = ws._need.get(query)
        if need is None or n < need or ws._capture:
            buf = ws._sized(query)
            n = buf.numel()
    else:
        buf = ws
        n = buf.numel() * buf.element_size()
    if buf.get_device() != dev:
        raise ValueError(f"the workspace is on {buf.device}, the other tensors are on cuda:{dev}")
    return buf.data_ptr(), n


def _mx4_shapes(shape: tuple, axis: int) -> tuple[tuple, tuple, int, int]:
    """(codes shape, scales shape, rows, cols) of a matrix or a stack of them
    ([..., rows, cols]; the stacked matrices' rows follow one another)."""
    if axis != 0 and axis != 1:
        raise ValueError("axis must be 0 or 1")
    if len(shape) < 2:
        raise ValueError("expected a matrix or a stack of matrices")
    r, c = shape[-2], shape[-1]
    b = LAROSA_MX4_BLOCK
    if c % b or (axis == 0 and r % b):
        raise ValueError(f"the blocked axis and the rows must be multiples of {b}")
    if len(shape) == 2:
        return (r, c // 2), ((r, c // b) if axis == 1 else (r // b, c)), r, c
    lead = tuple(shape[:-2])
    n = 1
    for k in lead:
        n *= k
    return lead + (r, c // 2), lead + ((r, c // b) if axis == 1 else (r // b, c)), n * r, c


def larosa_mx4_quantize(src: torch.Tensor, axis: int = 1, codes: torch.Tensor | None = None,
                        scales: torch.Tensor | None = None, dev_status: torch.Tensor | None = None
                        ) -> tuple[torch.Tensor, torch.Tensor]:
    """A matrix (or a stack of matrices, [..., rows, cols]) in microscaled 4-bit
    form: (codes uint8 [..., rows, cols / 2], scales uint8).  axis 1: blocks of
    32 along a row, scales [..., rows, cols / 32]; axis 0: down a column, scales
    [..., rows / 32, cols].  A single token [d] is a row [1, d].  See
    larosa_mx4_quantize in the header."""
    _need(src, "src")
    dev, device = src.get_device(), src.device
    if src.dim() < 2:
        src = _as2d(src)
    cs, ss, rows, cols = _mx4_shapes(src.shape, axis)
    if codes is None:
        codes = torch.empty(*cs, dtype=torch.uint8, device=device)  # a third faster than with one tuple
    else:
        _need_out(codes, "codes", cs, torch.uint8, dev)
    if scales is None:
        scales = torch.empty(*ss, dtype=torch.uint8, device=device)
    else:
        _need_out(scales, "scales", ss, torch.uint8, dev)
    _call("larosa_mx4_quantize", dev, _lib.larosa_mx4_quantize,
          (src.data_ptr(), rows, cols, axis, _dtype_code(src), codes.data_ptr(), scales.data_ptr(),
           _status_word(dev_status, dev)))
    return codes, scales


def _mx4_pair(codes: torch.Tensor, scales: torch.Tensor, axis: int, what: str) -> tuple[int, int, int]:
    """Checks a (codes, scales) pair; returns its (rows, cols, device number)."""
    if not (isinstance(codes, torch.Tensor) and isinstance(scales, torch.Tensor)):
        _need(codes, what + "codes")
        _need(scales, what + "scales")
    dev = codes.get_device()
    shape = codes.shape
    if (dev >= 0 and len(shape) == 2 and codes.dtype is torch.uint8 and scales.dtype is torch.uint8
            and scales.get_device() == dev and codes.is_contiguous() and scales.is_contiguous()):
        rows, half = shape
        if axis == 1:
            if scales.shape == (rows, half // 16) and half % 16 == 0:
                return rows, 2 * half, dev
        elif scales.shape == (rows // 32, 2 * half) and rows % 32 == 0 and half % 16 == 0:
            return rows, 2 * half, dev
    # a stack of matrices, or something to refuse
    _need(codes, what + "codes", torch.uint8)
    _need_fast(scales, what + "scales", torch.uint8, dev)
    if len(shape) < 2:
        raise ValueError(f"{what}codes must be a matrix or a stack of matrices")
    _, ss, rows, cols = _mx4_shapes((*shape[:-1], 2 * shape[-1]), axis)
    if scales.shape != ss:
        raise ValueError(f"{what}scales must have shape {ss}, got {tuple(scales.shape)}")
    return rows, cols, dev


def larosa_mx4_dequantize(codes: torch.Tensor, scales: torch.Tensor, axis: int = 1,
                          dtype: torch.dtype | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values that codes and scales (larosa_mx4_quantize) stand for, in `dtype`
    (None: out's, or fp32)."""
    rows, cols, dev = _mx4_pair(codes, scales, axis, "")
    if out is None:
        out = torch.empty(*codes.shape[:-1], cols, dtype=dtype or torch.float32, device=codes.device)
    else:
        _need_typed(out, "out", (*codes.shape[:-1], cols), dtype, dev)
    _call("larosa_mx4_dequantize", dev, _lib.larosa_mx4_dequantize,
          (codes.data_ptr(), scales.data_ptr(), rows, cols, axis, _dtype_code(out), out.data_ptr()))
    return out


def larosa_mx4_linear_workspace_bytes(M: int, d_in: int, d_out: int) -> int:
    return int(_lib.larosa_mx4_linear_workspace_bytes(M, d_in, d_out))


def larosa_mx4_linear(x_codes: torch.Tensor, x_scales: torch.Tensor, Wt_codes: torch.Tensor,
                      Wt_scales: torch.Tensor, dtype: torch.dtype | None = None, y: torch.Tensor | None = None,
                      ws=None, dev_status: torch.Tensor | None = None) -> torch.Tensor:
    """y = x . W of two 4-bit matrices, [M, d_out] in `dtype` (None: y's, or fp32):
    x [M, d_in] and the weight in torch.nn.Linear layout [d_out, d_in], both of
    larosa_mx4_quantize with axis 1."""
    M, d_in, x_dev = _mx4_pair(x_codes, x_scales, 1, "x_")
    d_out, d_w, dev = _mx4_pair(Wt_codes, Wt_scales, 1, "Wt_")
    if d_w != d_in or x_codes.dim() != 2 or Wt_codes.dim() != 2:
        raise ValueError("x_codes must be [M, d_in / 2], Wt_codes [d_out, d_in / 2]")
    if x_dev != dev:
        raise ValueError(f"x_codes is on {x_codes.device}, the other tensors are on cuda:{dev}")
    if y is None:
        y = torch.empty(M, d_out, dtype=dtype or torch.float32, device=Wt_codes.device)
    else:
        _need_typed(y, "y", (M, d_out), dtype, dev)
    p, n = _ws_pair(ws, dev, ("larosa_mx4_linear_workspace_bytes", M, d_in, d_out))
    _call("larosa_mx4_linear", dev, _lib.larosa_mx4_linear,
          (x_codes.data_ptr(), x_scales.data_ptr(), Wt_codes.data_ptr(), Wt_scales.data_ptr(), M, d_in, d_out,
           y.data_ptr(), p, n, _status_word(dev_status, dev), _dtype_code(y)))
    return y


def larosa_mx4_sparse_linear(idx: torch.Tensor, val: torch.Tensor, W_codes: torch.Tensor, W_scales: torch.Tensor,
                             y: torch.Tensor | None = None, ws=None, dev_status: torch.Tensor | None = None
                             ) -> torch.Tensor:
    """y = sum_k val[:, k] * W[idx[:, k]], fp32 [M, d_out], with a 4-bit weight
    (W_codes, W_scales of larosa_mx4_quantize(W, axis=0))."""
    d_in, d_out, dev = _mx4_pair(W_codes, W_scales, 0, "W_")
    _need_fast(idx, "idx", torch.int32, dev)
    _need_fast(val, "val", torch.float32, dev)
    idx, val = _as2d(idx), _as2d(val)
    if idx.shape != val.shape or W_codes.dim() != 2:
        raise ValueError("idx and val must have one shape [M, K], W_codes [d_in, d_out / 2]")
    M, K = idx.shape
    if y is None:
        y = torch.empty(M, d_out, dtype=torch.float32, device=W_codes.device)
    else:
        _need_out(y, "y", (M, d_out), torch.float32, dev)
    p, n = _ws_pair(ws, dev, ("larosa_workspace_bytes", M, d_in, d_out, K))
    _call("larosa_mx4_sparse_linear", dev, _lib.larosa_mx4_sparse_linear,
          (idx.data_ptr(), val.data_ptr(), M, K, W_codes.data_ptr(), W_scales.data_ptr(), d_in, d_out, y.data_ptr(),
           p, n, _status_word(dev_status, dev)))
    return y


def larosa_mx4_topk_linear(x_rot: torch.Tensor, W_codes: torch.Tensor, W_scales: torch.Tensor, K: int,
                           y: torch.Tensor | None = None, ws=None, dev_status: torch.Tensor | None = None
                           ) -> torch.Tensor:
    """larosa_topk_linear with a 4-bit weight (W_codes, W_scales of
    larosa_mx4_quantize(W, axis=0)); the kept list stays in the workspace."""
    d_in, d_out, dev = _mx4_pair(W_codes, W_scales, 0, "W_")
    _need_fast(x_rot, "x_rot", torch.float32, dev)
    x_rot = _as2d(x_rot)
    M, d_x = x_rot.shape
    if d_x != d_in or W_codes.dim() != 2:
        raise ValueError("x_rot must be [M, d_in], W_codes [d_in, d_out / 2]")
    if y is None:
        y = torch.empty(M, d_out, dtype=torch.float32, device=W_codes.device)
    else:
        _need_out(y, "y", (M, d_out), torch.float32, dev)
    p, n = _ws_pair(ws, dev, ("larosa_workspace_bytes", M, d_in, d_out, K))
    _call("larosa_mx4_topk_linear", dev, _lib.larosa_mx4_topk_linear,
          (x_rot.data_ptr(), W_codes.data_ptr(), W_scales.data_ptr(), M, d_in, d_out, K, y.data_ptr(), p, n,
           _status_word(dev_status, dev)))
    return y


def larosa_moe_workspace_bytes(M: int, d: int, f: int, E: int, k: int) -> int:
    return int(_lib.larosa_moe_workspace_bytes(M, d, f, E, k))


def larosa_moe_layer(x: torch.Tensor, Wr: torch.Tensor, W_gu: torch.Tensor, W_d: torch.Tensor, k: int,
                     S_gu: torch.Tensor | None = None, S_d: torch.Tensor | None = None, renormalize: bool = True,
                     y: torch.Tensor | None = None, idx: torch.Tensor | None = None,
                     gate: torch.Tensor | None = None, ws=None, dev_status: torch.Tensor | None = None
                     ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """A mixture-of-experts layer of a few tokens in one kernel: (y fp32 [M, d],
    idx int32 [M, k], gate fp32 [M, k]).

    x [M, d], router Wr [E, d], experts W_gu [E, d, 2 f] (gate | up) and W_d
    [E, f, d] of x's type; or 4-bit experts, W_gu and W_d the codes and S_gu, S_d
    the scales of larosa_mx4_quantize(W, axis=0)."""
    _need(x, "x")
    dev, device, dt = x.get_device(), x.device, x.dtype
    x = _as2d(x)
    M, d = x.shape
    code = _dtype_code(x)
    _need_fast(Wr, "Wr", dt, dev)
    if (S_gu is None) != (S_d is None):
        raise ValueError("S_gu and S_d go together")
    gu, dn = W_gu.shape, W_d.shape
    if len(gu) != 3 or len(dn) != 3:
        raise ValueError("Wr must be [E, d], W_gu [E, d, 2 f], W_d [E, f, d]")
    E, f = dn[0], dn[1]
    if S_gu is None:
        _need_fast(W_gu, "W_gu", dt, dev)
        _need_fast(W_d, "W_d", dt, dev)
        ok = gu == (E, d, 2 * f) and dn[2] == d
        sg = sd = 0
    else:
        for t, name in ((W_gu, "W_gu"), (W_d, "W_d"), (S_gu, "S_gu"), (S_d, "S_d")):
            _need_fast(t, name, torch.uint8, dev)
        b = LAROSA_MX4_BLOCK
        ok = (gu == (E, d, f) and 2 * dn[2] == d and S_gu.shape == (E, d // b, 2 * f)
              and S_d.shape == (E, f // b, d))
        sg, sd = S_gu.data_ptr(), S_d.data_ptr()
    if not ok or Wr.shape != (E, d):
        raise ValueError("shapes of x, Wr, the experts and their scales do not agree")
    p, n = _ws_pair(ws, dev, ("larosa_moe_workspace_bytes", M, d, f, E, k))
    if y is None:
        y = torch.empty(M, d, dtype=torch.float32, device=device)
    else:
        _need_out(y, "y", (M, d), torch.float32, dev)
    if idx is None:
        idx = torch.empty(M, k, dtype=torch.int32, device=device)
    else:
        _need_out(idx, "idx", (M, k), torch.int32, dev)
    if gate is None:
        gate = torch.empty(M, k, dtype=torch.float32, device=device)
    else:
        _need_out(gate, "gate", (M, k), torch.float32, dev)
    _call("larosa_moe_layer", dev, _lib.larosa_moe_layer,
          (x.data_ptr(), Wr.data_ptr(), W_gu.data_ptr(), sg, W_d.data_ptr(), sd, M, d, f, E, k,
           1 if renormalize else 0, y.data_ptr(), idx.data_ptr(), gate.data_ptr(), p, n,
           _status_word(dev_status, dev), code))
    return y, idx, gate


def larosa_check(dev_status: torch.Tensor | None = None, device=None) -> int:
    """Synchronises the current stream and returns the raw device status bits.

    Raises LarosaError for a nonzero word (the status of its lowest bit).
    """
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    st = default_status(device) if dev_status is None else dev_status
    flags = ctypes.c_int(0)
    status = _lib.larosa_check(_ptr(st), _stream(st.device), ctypes.byref(flags))
    _check(status, "larosa_check")
    return flags.value


def raw_library() -> ctypes.CDLL:
    """The loaded ctypes library (for tests of the C ABI itself)."""
    return _lib
