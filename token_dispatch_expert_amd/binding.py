"""ctypes binding of the C ABI declared in include/moe.h.

Argument marshalling only: each function checks that it got device tensors of the expected
dtype and layout, reads the sizes off their shapes, and passes raw pointers and the current
HIP stream to the library. Every step of the layer runs in the library's HIP kernels; there is
no fallback of any kind. The library is the in-tree `libmoe.so` built by
`__graft_entry__.build()`; if it is missing, the first call raises.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import c_int, c_size_t, c_void_p

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_NAME = "libmoe.so"

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(5)
MOE_F32, MOE_BF16, MOE_FP8_E4M3FN, MOE_BF16_BLOCKED, MOE_FP8_E4M3FN_BLOCKED = 0, 1, 2, 3, 4

_DTYPE_ENUM = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16,
               torch.float8_e4m3fn: MOE_FP8_E4M3FN, torch.uint8: MOE_FP8_E4M3FN}

ENTRY_POINTS = (
    "moe_status_string", "moe_route", "moe_permute_workspace_size", "moe_permute",
    "moe_ffn_workspace_size", "moe_grouped_ffn", "moe_combine", "moe_layer_workspace_size",
    "moe_layer", "moe_expert_capacity", "moe_permute_capped", "moe_layer_capped",
    "moe_route_gemm", "moe_route_gemm_workspace_size", "moe_permute_noalloc",
    "moe_block_weights",
    "moe_grouped_gemm", "moe_grouped_gemm_dgrad", "moe_grouped_gemm_wgrad", "moe_checkpoint_pack",
    "moe_checkpoint_unpack", "moe_swiglu", "moe_swiglu_backward", "moe_combine_backward",
    "moe_permute_backward", "moe_route_backward",
)

_lib = None


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{msg} (status {status})")
        self.status = status


def library_path() -> str:
    return os.path.join(_HERE, LIB_NAME)


def load_library(path: str | None = None):
    """Load libmoe.so and declare its signatures (raises if it is not built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or library_path()
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is not built; run __graft_entry__.build() first")
    lib = ctypes.CDLL(p)
    P, I, S = c_void_p, c_int, c_size_t
    sig = {
        "moe_status_string": ([I], ctypes.c_char_p),
        "moe_route": ([P, I, I, I, P, P, P, P], I),
        "moe_permute_workspace_size": ([I, I, I], S),
        "moe_permute": ([P, I, P, I, I, I, I, P, P, P, P, P, P, S, P], I),
        "moe_ffn_workspace_size": ([I, I, I, I, I, I], S),
        "moe_grouped_ffn": ([P, I, P, I, I, I, I, P, P, P, I, P, P, P, P, P, S, P], I),
        "moe_combine": ([P, P, P, I, I, I, P, I, P], I),
        "moe_layer_workspace_size": ([I, I, I, I, I, I, I], S),
        "moe_layer": ([P, P, I, I, I, I, I, I, P, P, P, I, P, P, P,
                       P, P, P, P, P, P, P, P, P, I, P, S, P], I),
        "moe_expert_capacity": ([I, I, I, I], I),
        "moe_route_gemm": ([P, I, P, I, I, I, I, I, P, P, P, P, P, S, P], I),
        "moe_route_gemm_workspace_size": ([I, I, I], S),
        "moe_permute_capped": ([P, I, P, I, I, I, I, I, P, P, P, P, P, P, S, P], I),
        "moe_permute_noalloc": ([P, I, P, I, I, I, I, P, P, P, P, P, P], I),
        "moe_block_weights": ([P, P, I, I, I, I, P], I),
        "moe_layer_capped": ([P, P, I, I, I, I, I, I, I, P, P, P, I, P, P, P,
                              P, P, P, P, P, P, P, P, P, I, P, S, P], I),
        "moe_grouped_gemm": ([P, I, P, I, I, I, I, P, I, P, I, P], I),
        "moe_grouped_gemm_dgrad": ([P, P, I, P, I, I, I, I, P, P, I, P, I, P], I),
        "moe_grouped_gemm_wgrad": ([P, P, I, P, I, I, I, I, P, I, I, P], I),
        "moe_checkpoint_pack": ([P, I, I, I, P, P, P], I),
        "moe_checkpoint_unpack": ([P, P, I, I, I, P, P, I, P], I),
        "moe_swiglu": ([P, P, I, P, I, I, I, P, P, P, P, P, P], I),
        "moe_swiglu_backward": ([P, I, P, P, I, P, P, P, I, I, I, P, P, P, P], I),
        "moe_combine_backward": ([P, I, P, P, P, I, I, I, P, I, P, P], I),
        "moe_permute_backward": ([P, I, P, I, I, I, P, I, P], I),
        "moe_route_backward": ([P, P, P, I, I, I, P, P], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path is None:
        _lib = lib
    return lib


def _check(status: int):
    if status != MOE_OK:
        msg = load_library().moe_status_string(status).decode()
        raise MoeError(status, msg)


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return c_void_p(stream.cuda_stream)


def _need(t, dtype, shape, name):
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape and t.shape != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _dt(t, name):
    try:
        return _DTYPE_ENUM[t.dtype]
    except KeyError:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}") from None


# ----------------------------------------------------------------------------------------
# workspace
# ----------------------------------------------------------------------------------------
def moe_permute_workspace_size(T: int, E: int, k: int) -> int:
    return int(load_library().moe_permute_workspace_size(T, E, k))


def moe_ffn_workspace_size(rows: int, E: int, d: int, d_ff: int, act_dtype, w_dtype) -> int:
    return int(load_library().moe_ffn_workspace_size(rows, E, d, d_ff,
                                                     _DTYPE_ENUM[act_dtype], _DTYPE_ENUM[w_dtype]))


def moe_layer_workspace_size(T: int, E: int, k: int, d: int, d_ff: int, act_dtype, w_dtype) -> int:
    return int(load_library().moe_layer_workspace_size(T, E, k, d, d_ff, _DTYPE_ENUM[act_dtype],
                                                       _DTYPE_ENUM[w_dtype]))


class Workspace:
    """A device byte buffer (allocated by torch) handed to the library as scratch."""

    def __init__(self, nbytes: int, device="cuda"):
        self.nbytes = int(nbytes)
        self.buf = torch.empty(max(self.nbytes, 16), dtype=torch.uint8, device=device)

    @property
    def ptr(self):
        return c_void_p(self.buf.data_ptr()) if self.nbytes > 0 else None


# ----------------------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ----------------------------------------------------------------------------------------
def moe_route(logits, k: int, topk_ids, topk_gates, counts=None, stream=None):
    T, E = logits.shape
    _need(logits, torch.float32, (T, E), "logits")
    _need(topk_ids, torch.int32, (T, k), "topk_ids")
    _need(topk_gates, torch.float32, (T, k), "topk_gates")
    if counts is not None:
        _need(counts, torch.int32, (E,), "counts")
    _check(load_library().moe_route(_ptr(logits), T, E, k, _ptr(topk_ids), _ptr(topk_gates),
                                    _ptr(counts), _stream(stream)))


def moe_route_gemm_workspace_size(T: int, E: int, k: int) -> int:
    return load_library().moe_route_gemm_workspace_size(T, E, k)


def moe_route_gemm(x, w_router, k: int, topk_ids, topk_gates, counts=None, logits=None,
                   workspace: "Workspace | None" = None, stream=None):
    """Router scores x @ w_router^T (fp32) and top-k gating; logits optional. Small batches
    need a workspace of moe_route_gemm_workspace_size bytes (allocated here if not given)."""
    T, d = x.shape
    E = w_router.shape[0]
    if workspace is None:
        workspace = Workspace(moe_route_gemm_workspace_size(T, E, k), device=x.device)
    _need(w_router, x.dtype, (E, d), "w_router")
    _need(topk_ids, torch.int32, (T, k), "topk_ids")
    _need(topk_gates, torch.float32, (T, k), "topk_gates")
    if counts is not None:
        _need(counts, torch.int32, (E,), "counts")
    if logits is not None:
        _need(logits, torch.float32, (T, E), "logits")
    _check(load_library().moe_route_gemm(
        _ptr(x), _dt(x, "x"), _ptr(w_router), _dt(w_router, "w_router"), T, E, k, d,
        _ptr(logits), _ptr(topk_ids), _ptr(topk_gates), _ptr(counts), workspace.ptr,
        workspace.nbytes, _stream(stream)))


def moe_permute(x, topk_ids, E: int, counts, offsets, sorted_to_flat, flat_to_sorted, x_sorted,
                workspace: Workspace, stream=None, capacity: int | None = None):
    """capacity (optional): most kept assignments per expert (moe_permute_capped)."""
    T, d = x.shape
    k = topk_ids.shape[1]
    R = T * k
    _need(topk_ids, torch.int32, (T, k), "topk_ids")
    _need(counts, torch.int32, (E,), "counts")
    _need(offsets, torch.int32, (E + 1,), "offsets")
    _need(sorted_to_flat, torch.int32, (R,), "sorted_to_flat")
    _need(flat_to_sorted, torch.int32, (R,), "flat_to_sorted")
    _need(x_sorted, x.dtype, (R, d), "x_sorted")
    lib = load_library()
    head = (_ptr(x), _dt(x, "x"), _ptr(topk_ids), T, E, k, d)
    tail = (_ptr(counts), _ptr(offsets), _ptr(sorted_to_flat), _ptr(flat_to_sorted),
            _ptr(x_sorted), workspace.ptr, workspace.nbytes, _stream(stream))
    if capacity is None:
        _check(lib.moe_permute(*head, *tail))
    else:
        _check(lib.moe_permute_capped(*head, int(capacity), *tail))


def moe_permute_noalloc(x, topk_ids, E: int, counts, offsets, sorted_to_flat, flat_to_sorted,
                        x_sorted, stream=None):
    """moe_permute without a workspace: the library's static per-GPU scratch (no allocation)."""
    T, d = x.shape
    k = topk_ids.shape[1]
    R = T * k
    _need(topk_ids, torch.int32, (T, k), "topk_ids")
    _need(counts, torch.int32, (E,), "counts")
    _need(offsets, torch.int32, (E + 1,), "offsets")
    _need(sorted_to_flat, torch.int32, (R,), "sorted_to_flat")
    _need(flat_to_sorted, torch.int32, (R,), "flat_to_sorted")
    _need(x_sorted, x.dtype, (R, d), "x_sorted")
    _check(load_library().moe_permute_noalloc(
        _ptr(x), _dt(x, "x"), _ptr(topk_ids), T, E, k, d, _ptr(counts), _ptr(offsets),
        _ptr(sorted_to_flat), _ptr(flat_to_sorted), _ptr(x_sorted), _stream(stream)))


# bytes of the static scratch behind moe_permute_noalloc (MOE_PERMUTE_NOALLOC_SCRATCH_BYTES)
PERMUTE_NOALLOC_SCRATCH_BYTES = 4 << 20


def moe_expert_capacity(T: int, E: int, k: int, factor_percent: int) -> int:
    """ceil(C * T * k / E) for C = factor_percent / 100 (exact; -1 for invalid sizes)."""
    return load_library().moe_expert_capacity(T, E, k, int(factor_percent))


def _weights(w_gate, w_up, w_down, s_gate, s_up, s_down, blocked=False):
    """blocked: the bf16 or fp8 weights are in their blocked layout (see moe_block_weights); the
    tensors keep their [E, d_ff, d] / [E, d, d_ff] shapes."""
    E, d_ff, d = w_gate.shape
    _need(w_up, w_gate.dtype, (E, d_ff, d), "w_up")
    _need(w_down, w_gate.dtype, (E, d, d_ff), "w_down")
    w_dt = _dt(w_gate, "w_gate")
    if blocked:
        if w_dt not in (MOE_BF16, MOE_FP8_E4M3FN):
            raise TypeError("blocked weights are bfloat16 or float8_e4m3fn")
        w_dt = MOE_BF16_BLOCKED if w_dt == MOE_BF16 else MOE_FP8_E4M3FN_BLOCKED
    if w_dt == MOE_FP8_E4M3FN:
        for s, shp, n in ((s_gate, (E, -(-d_ff // 128), -(-d // 128)), "s_gate"),
                          (s_up, (E, -(-d_ff // 128), -(-d // 128)), "s_up"),
                          (s_down, (E, -(-d // 128), -(-d_ff // 128)), "s_down")):
            if s is None:
                raise ValueError(f"{n} is required for fp8 weights")
            _need(s, torch.float32, shp, n)
    return E, d, d_ff, w_dt


def moe_block_weights(src, dst, stream=None):
    """dst [E, N, K] <- src [E, N, K] (bfloat16 or float8_e4m3fn) in its blocked layout."""
    if src.dim() != 3:
        raise ValueError("src: expected [E, N, K]")
    E, N, K = src.shape
    if src.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
        raise TypeError(f"src: expected bfloat16 or float8_e4m3fn, got {src.dtype}")
    _need(src, src.dtype, (E, N, K), "src")
    _need(dst, src.dtype, (E, N, K), "dst")
    _check(load_library().moe_block_weights(_ptr(src), _ptr(dst), _dt(src, "src"), E, N, K,
                                            _stream(stream)))


def moe_grouped_ffn(x_sorted, offsets, w_gate, w_up, w_down, y_sorted, workspace: Workspace,
                    s_gate=None, s_up=None, s_down=None, stream=None, weights_blocked=False):
    rows, d_x = x_sorted.shape
    E, d, d_ff, w_dt = _weights(w_gate, w_up, w_down, s_gate, s_up, s_down, weights_blocked)
    if d_x != d:
        raise ValueError("x_sorted and weights disagree on d")
    _need(offsets, torch.int32, (E + 1,), "offsets")
    _need(y_sorted, torch.float32, (rows, d), "y_sorted")
    _check(load_library().moe_grouped_ffn(
        _ptr(x_sorted), _dt(x_sorted, "x_sorted"), _ptr(offsets), rows, E, d, d_ff, _ptr(w_gate),
        _ptr(w_up), _ptr(w_down), w_dt, _ptr(s_gate), _ptr(s_up), _ptr(s_down), _ptr(y_sorted),
        workspace.ptr, workspace.nbytes, _stream(stream)))


def _y_dt(y):
    """The combine's output format, from y's dtype: float32 or bfloat16."""
    if y.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"y: expected float32 or bfloat16, got {y.dtype}")
    return _DTYPE_ENUM[y.dtype]


def moe_combine(y_sorted, flat_to_sorted, topk_gates, y, stream=None):
    """y (float32 or bfloat16) receives the gate-weighted sums; bfloat16 is the fp32 sum
    rounded to nearest even."""
    T, k = topk_gates.shape
    R, d = y_sorted.shape
    if R != T * k:
        raise ValueError("y_sorted rows must equal T*k")
    _need(y_sorted, torch.float32, (R, d), "y_sorted")
    _need(flat_to_sorted, torch.int32, (R,), "flat_to_sorted")
    _need(topk_gates, torch.float32, (T, k), "topk_gates")
    _need(y, y.dtype, (T, d), "y")
    _check(load_library().moe_combine(_ptr(y_sorted), _ptr(flat_to_sorted), _ptr(topk_gates), T,
                                      k, d, _ptr(y), _y_dt(y), _stream(stream)))


def moe_layer(logits, x, w_gate, w_up, w_down, k: int, out: dict, workspace: Workspace,
              s_gate=None, s_up=None, s_down=None, stream=None, capacity: int | None = None,
              weights_blocked=False):
    """out holds the caller's buffers: topk_ids, topk_gates, counts, offsets, sorted_to_flat,
    flat_to_sorted, x_sorted, y_sorted, y (see `layer_buffers`; y float32 or bfloat16).
    capacity (optional): most kept assignments per expert (moe_layer_capped).
    weights_blocked: bf16 weights in the MOE_BF16_BLOCKED layout (moe_block_weights)."""
    T, E = logits.shape
    _need(logits, torch.float32, (T, E), "logits")
    Ew, d, d_ff, w_dt = _weights(w_gate, w_up, w_down, s_gate, s_up, s_down, weights_blocked)
    if Ew != E or x.shape != (T, d):
        raise ValueError("logits, x and weights disagree on T, E or d")
    R = T * k
    shapes = dict(topk_ids=(torch.int32, (T, k)), topk_gates=(torch.float32, (T, k)),
                  counts=(torch.int32, (E,)), offsets=(torch.int32, (E + 1,)),
                  sorted_to_flat=(torch.int32, (R,)), flat_to_sorted=(torch.int32, (R,)),
                  x_sorted=(x.dtype, (R, d)), y_sorted=(torch.float32, (R, d)),
                  y=(out["y"].dtype, (T, d)))
    for n, (dt, shp) in shapes.items():
        _need(out[n], dt, shp, n)
    o = out
    lib = load_library()
    head = (_ptr(logits), _ptr(x), _dt(x, "x"), T, E, k, d, d_ff)
    tail = (_ptr(w_gate), _ptr(w_up), _ptr(w_down), w_dt, _ptr(s_gate), _ptr(s_up), _ptr(s_down),
            _ptr(o["topk_ids"]), _ptr(o["topk_gates"]), _ptr(o["counts"]), _ptr(o["offsets"]),
            _ptr(o["sorted_to_flat"]), _ptr(o["flat_to_sorted"]), _ptr(o["x_sorted"]),
            _ptr(o["y_sorted"]), _ptr(o["y"]), _y_dt(o["y"]), workspace.ptr, workspace.nbytes,
            _stream(stream))
    if capacity is None:
        _check(lib.moe_layer(*head, *tail))
    else:
        _check(lib.moe_layer_capped(*head, int(capacity), *tail))


# ----------------------------------------------------------------------------------------
# training: the pieces of the layer's gradient (same names as the C ABI)
# ----------------------------------------------------------------------------------------
_Tensor = torch.Tensor
_FLOAT_DT = {t: _DTYPE_ENUM[t] for t in (torch.float32, torch.bfloat16)}
_CODE_DT = (torch.float8_e4m3fn, torch.uint8)


# A small call is bound by the host, so these checks look each property of a tensor up once.
def _call(name: str, stream, *args):
    """Enqueue lib.<name>(*args, stream), tensors among args as their addresses, on the device that
    every tensor is on, whichever is current: on `stream`, or on that device's current stream."""
    device = None
    raw = []
    for a in args:
        if isinstance(a, _Tensor):
            d = a.get_device()
            if d != device:
                if d < 0:
                    raise ValueError("expected a device tensor")
                if device is not None:
                    raise ValueError("expected every tensor on one device")
                device = d
            if not a.is_contiguous():
                raise ValueError("expected a contiguous tensor")
            a = a.data_ptr()
        raw.append(a)
    if stream is not None and stream.device.index != device:
        raise ValueError("expected a stream of the tensors' device")
    fn = getattr(_lib if _lib is not None else load_library(), name)
    # (the raw handle of the current stream: 0.2 us, against 2.7 for torch.cuda.current_stream())
    handle = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
    if device == torch._C._cuda_getDevice():  # (torch.cuda.current_device() without its set-up check)
        status = fn(*raw, handle)
    else:
        with torch.cuda.device(device):
            status = fn(*raw, handle)
    if status != MOE_OK:
        _check(status)


def _float_dt(t, name):
    dt = _FLOAT_DT.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name}: expected float32 or bfloat16, got {t.dtype}")
    return dt


def _dims(t, n, name):
    shape = t.shape
    if len(shape) != n:
        raise ValueError(f"{name}: expected {n} dimensions, got shape {tuple(shape)}")
    return shape


def _held(codes, scales, shape, name):
    """codes (float8_e4m3fn or uint8) and scales of rows held in 8 bits."""
    dt = codes.dtype
    if dt not in _CODE_DT:
        raise TypeError(f"{name}_codes: expected float8_e4m3fn or uint8, got {dt}")
    _need(codes, dt, shape, name + "_codes")
    _need(scales, torch.float32, (shape[0], -(-shape[1] // 128)), name + "_scales")


def moe_grouped_gemm(x, offsets, w, y, stream=None):
    """y[r] = W_e x[r] for the rows of each expert e. x [rows, K] and w [E, N, K] in one dtype
    (bfloat16 or float32), y [rows, N] float32 or bfloat16."""
    rows, K = _dims(x, 2, "x")
    E, N, _ = _dims(w, 3, "w")
    _need(w, x.dtype, (E, N, K), "w")
    _need(offsets, torch.int32, (E + 1,), "offsets")
    _need(y, y.dtype, (rows, N), "y")
    _call("moe_grouped_gemm", stream, x, _float_dt(x, "x"), offsets, rows, E, N, K, w,
          _float_dt(w, "w"), y, _float_dt(y, "y"))


def moe_grouped_gemm_dgrad(dy, offsets, w, dx, dy2=None, w2=None, stream=None):
    """dx[r] = W_e^T dy[r], plus W2_e^T dy2[r] with dy2 and w2. dy [rows, N] and w [E, N, K] in one
    dtype (bfloat16 or float32), dx [rows, K] float32 or bfloat16."""
    rows, N = _dims(dy, 2, "dy")
    E, _, K = _dims(w, 3, "w")
    _need(w, dy.dtype, (E, N, K), "w")
    _need(offsets, torch.int32, (E + 1,), "offsets")
    _need(dx, dx.dtype, (rows, K), "dx")
    if (dy2 is None) != (w2 is None):
        raise ValueError("dy2 and w2 come together")
    if dy2 is not None:
        _need(dy2, dy.dtype, (rows, N), "dy2")
        _need(w2, dy.dtype, (E, N, K), "w2")
    _call("moe_grouped_gemm_dgrad", stream, dy, dy2, _float_dt(dy, "dy"), offsets, rows, E, N, K, w,
          w2, _float_dt(w, "w"), dx, _float_dt(dx, "dx"))


def moe_grouped_gemm_wgrad(dy, x, offsets, dw, accumulate: bool = False, stream=None):
    """dw[e] = sum over expert e's rows of dy[r] x[r]^T, or dw[e] += with accumulate. dy [rows, N] and
    x [rows, K] in one dtype (bfloat16 or float32), dw [E, N, K] float32 or bfloat16."""
    rows, N = _dims(dy, 2, "dy")
    _, K = _dims(x, 2, "x")
    E = _dims(dw, 3, "dw")[0]
    _need(x, dy.dtype, (rows, K), "x")
    _need(offsets, torch.int32, (E + 1,), "offsets")
    _need(dw, dw.dtype, (E, N, K), "dw")
    _call("moe_grouped_gemm_wgrad", stream, dy, x, _float_dt(dy, "dy"), offsets, rows, E, N, K, dw,
          _float_dt(dw, "dw"), int(bool(accumulate)))


def moe_checkpoint_pack(x, codes, scales, stream=None):
    """Hold x [rows, d] (bfloat16 or float32) in 8 bits: codes [rows, d] (float8_e4m3fn or uint8) and
    scales [rows, ceil(d/128)] float32."""
    rows, d = _dims(x, 2, "x")
    _held(codes, scales, (rows, d), "x")
    _call("moe_checkpoint_pack", stream, x, _float_dt(x, "x"), rows, d, codes, scales)


def moe_checkpoint_unpack(codes, scales, out, flat_to_sorted=None, stream=None):
    """Held rows back as values: out [T, d], or with flat_to_sorted [T*k] out [T*k, d], where row t
    goes to each of its k sorted rows (bfloat16 or float32)."""
    T, d = _dims(codes, 2, "codes")
    _held(codes, scales, (T, d), "x")
    rows = T if flat_to_sorted is None else flat_to_sorted.numel()
    if flat_to_sorted is not None:
        _need(flat_to_sorted, torch.int32, (rows,), "flat_to_sorted")
        if (rows % T or rows < T) if T else rows:  # (k >= 1; no entries without tokens)
            raise ValueError("flat_to_sorted must have k entries for every row")
    _need(out, out.dtype, (rows, d), "out")
    _call("moe_checkpoint_unpack", stream, codes, scales, T, rows // T if T else 1, d,
          flat_to_sorted, out, _float_dt(out, "out"))


def moe_swiglu(g, u, h, g_codes=None, g_scales=None, u_codes=None, u_scales=None, offsets=None, stream=None):
    """h = silu(g) * u, all [rows, d_ff] in one dtype (bfloat16 or float32); with codes and scales, g
    and u are held in 8 bits too. offsets [E+1]: only rows below offsets[E]."""
    shape = _dims(g, 2, "g")
    _need(u, g.dtype, shape, "u")
    _need(h, g.dtype, shape, "h")
    if not (g_codes is None and g_scales is None and u_codes is None and u_scales is None):
        if g_codes is None or g_scales is None or u_codes is None or u_scales is None:
            raise ValueError("g_codes, g_scales, u_codes and u_scales come together")
        _held(g_codes, g_scales, shape, "g")
        _held(u_codes, u_scales, shape, "u")
    E = _row_offsets(offsets)
    _call("moe_swiglu", stream, g, u, _float_dt(g, "g"), offsets, E, *shape, h, g_codes, g_scales,
          u_codes, u_scales)


def _row_offsets(offsets) -> int:
    if offsets is None:
        return 0
    n, = _dims(offsets, 1, "offsets")
    _need(offsets, torch.int32, (n,), "offsets")
    if n < 2:  # (an empty tensor's address is NULL, which means all rows)
        raise ValueError("offsets: expected E + 1 entries")
    return n - 1


def moe_swiglu_backward(dh, g, u, dg, du, h=None, g_scales=None, u_scales=None, offsets=None, stream=None):
    """dg and du (and h again, if given) from dh, all [rows, d_ff] in dh's dtype; g and u in that dtype,
    or held in 8 bits (codes, with g_scales and u_scales)."""
    shape = _dims(dh, 2, "dh")
    dt = dh.dtype
    _need(dg, dt, shape, "dg")
    _need(du, dt, shape, "du")
    if h is not None:
        _need(h, dt, shape, "h")
    if g_scales is None and u_scales is None:
        _need(g, dt, shape, "g")
        _need(u, dt, shape, "u")
        gu = _float_dt(g, "g")
    elif g_scales is None or u_scales is None:
        raise ValueError("g_scales and u_scales come together")
    else:
        _held(g, g_scales, shape, "g")
        _held(u, u_scales, shape, "u")
        gu = MOE_FP8_E4M3FN
    E = _row_offsets(offsets)
    _call("moe_swiglu_backward", stream, dh, _float_dt(dh, "dh"), g, u, gu, g_scales, u_scales,
          offsets, E, *shape, dg, du, h)


def moe_combine_backward(dy, y_sorted, flat_to_sorted, topk_gates, dy_sorted, dgates, stream=None):
    """dy_sorted [T*k, d] and dgates [T, k] (float32) from dy [T, d]; dy and dy_sorted float32 or
    bfloat16. y_sorted and dgates None together: dy_sorted alone."""
    T, d = _dims(dy, 2, "dy")
    k = _dims(topk_gates, 2, "topk_gates")[1]
    _need(topk_gates, torch.float32, (T, k), "topk_gates")
    _need(flat_to_sorted, torch.int32, (T * k,), "flat_to_sorted")
    _need(dy_sorted, dy_sorted.dtype, (T * k, d), "dy_sorted")
    if (y_sorted is None) != (dgates is None):
        raise ValueError("y_sorted and dgates come together")
    if dgates is not None:
        _need(y_sorted, torch.float32, (T * k, d), "y_sorted")
        _need(dgates, torch.float32, (T, k), "dgates")
    _call("moe_combine_backward", stream, dy, _float_dt(dy, "dy"), y_sorted, flat_to_sorted,
          topk_gates, T, k, d, dy_sorted, _float_dt(dy_sorted, "dy_sorted"), dgates)


def moe_permute_backward(dx_sorted, flat_to_sorted, k: int, dx, stream=None):
    """dx[t] = sum of the k rows of dx_sorted that token t went to (float32 or bfloat16 each)."""
    T, d = _dims(dx, 2, "dx")
    _need(dx_sorted, dx_sorted.dtype, (T * k, d), "dx_sorted")
    _need(flat_to_sorted, torch.int32, (T * k,), "flat_to_sorted")
    _call("moe_permute_backward", stream, dx_sorted, _float_dt(dx_sorted, "dx_sorted"),
          flat_to_sorted, T, k, d, dx, _float_dt(dx, "dx"))


def moe_route_backward(dgates, topk_ids, topk_gates, dlogits, stream=None):
    """dlogits [T, E] (all of it) from dgates [T, k], the gradient of moe_route's gates."""
    T, k = _dims(dgates, 2, "dgates")
    E = _dims(dlogits, 2, "dlogits")[1]
    _need(dgates, torch.float32, (T, k), "dgates")
    _need(topk_ids, torch.int32, (T, k), "topk_ids")
    _need(topk_gates, torch.float32, (T, k), "topk_gates")
    _need(dlogits, torch.float32, (T, E), "dlogits")
    _call("moe_route_backward", stream, dgates, topk_ids, topk_gates, T, E, k, dlogits)


def layer_buffers(T: int, E: int, k: int, d: int, act_dtype, device="cuda",
                  y_dtype=torch.float32) -> dict:
    """Allocate (with torch) every output buffer moe_layer writes."""
    R = T * k
    z = lambda shape, dt: torch.empty(shape, dtype=dt, device=device)  # noqa: E731
    return dict(topk_ids=z((T, k), torch.int32), topk_gates=z((T, k), torch.float32),
                counts=z((E,), torch.int32), offsets=z((E + 1,), torch.int32),
                sorted_to_flat=z((R,), torch.int32), flat_to_sorted=z((R,), torch.int32),
                x_sorted=z((R, d), act_dtype), y_sorted=z((R, d), torch.float32),
                y=z((T, d), y_dtype))
