"""Python binding of libfp8q: online fine-grained E4M3 quantization and block-scaled FP8
GEMMs on AMD Instinct MI355X (gfx950).

The functions below carry the names of the C ABI (include/fp8q.h) and only marshal
arguments: PyTorch provides device memory and the current stream, every step of the
computation runs in the library's HIP kernels.  There is no fallback: if the library is
missing or no GPU is present the calls raise.

    xq, sa = fp8q_quantize_act_1x128(x)            # x: bf16 [M, K] on cuda
    wq, sb = fp8q_quantize_w_128x128(w)            # w: bf16 [G, N, K] or [N, K]
    xq, sa, wq, sb = fp8q_quantize_act_w(x, w)     # both in one launch
    c = fp8q_gemm_blockscaled(xq, sa, wq, sb)      # bf16 [M, N] (or out_dtype=torch.float32)
    c = fp8q_grouped_gemm_blockscaled(xq, sa, wq, sb, offsets)   # offsets: int32 [G+1] on cuda

Backward pass (same E4M3 format):
    wq, sb, wqt, sbt = fp8q_quantize_w_128x128_t(w)   # also W^T codes / scales
    dx = fp8q_gemm_blockscaled(dyq, sa_dy, wqt, sbt)    # dgrad dX = dY W
    xq, sa, xqt, sat = fp8q_quantize_act_dual(x)        # tiles along K and along the tokens
    dw = fp8q_gemm_rowscaled(dyqt, sat_dy, xqt, sat)    # wgrad dW = dY^T X

Training step of an MoE layer (the forward pass with values beside the codes, and back):
    xs, offsets, token_row, _ = fp8q_moe_sort(topk_ids, x, e_begin, n_experts)   # values by expert
    dys, dw = fp8q_moe_combine_backward(dy, expert_out, token_row, topk_w)
    dgu, h = fp8q_swiglu_backward(gu, dh, want_h=True)
    xq, sa, xqt, sat = fp8q_quantize_act_grouped(xs, offsets)    # rows, and token tiles per expert
    dw = fp8q_grouped_gemm_rowscaled(dguqt, sat_dgu, xqt, sat, offsets, m_tot)   # dW[g] = dgu[g]^T xs[g]
    dx = fp8q_moe_sort_backward(dxs, token_row)
    plan = fp8q_adamw_plan(params, grads, m, v)                  # states in FP32 or in E4M3
    fp8q_adamw(plan, lr=2e-4, step=1)

Around the experts:
    y, mean, rstd = fp8q_layer_norm(x, weight, bias)             # center=False: RMS norm
    dx, dweight, dbias = fp8q_layer_norm_backward(dy, x, weight, mean, rstd, want_bias=True)
    topk_ids, topk_w, counts, loss, slope = fp8q_moe_route(logits, k, bias, balance=1e-4)
    dlogits = fp8q_moe_route_backward(logits, topk_ids, topk_w, dw, slope, dloss)
    out = fp8q_orthogonalize(x)                                  # singular values near one
    fp8q_muon(param, grad, momentum, lr=2e-4)                    # the optimizer for matrices, in place

Layouts: xq uint8 [M, K]; sa float32 [K/128, M]; wq uint8 [G, N, K]; sb float32
[G, N/128, K/128]; C row-major [M, N].
"""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# FP8Q_LIBRARY may point at another build of the same library (e.g. a tuning variant).
LIB_PATH = os.environ.get("FP8Q_LIBRARY") or os.path.join(HERE, "libfp8q.so")

FP8Q_OK = 0
FP8Q_ERR_OFFSETS = -7  # grouped GEMM offsets rejected by the FP8Q_DEBUG check
FP8Q_OUT_BF16 = 0
FP8Q_OUT_F32 = 1
FP8Q_STATE_F32 = 0
FP8Q_STATE_E4M3 = 1
FP8Q_SCORE_SOFTMAX = 0
FP8Q_SCORE_SIGMOID = 1
ABI_VERSION = 9

EXPORTED = ("fp8q_quantize_act_1x128", "fp8q_quantize_w_128x128", "fp8q_gemm_blockscaled",
            "fp8q_grouped_gemm_blockscaled", "fp8q_quantize_w_128x128_t", "fp8q_quantize_act_dual",
            "fp8q_gemm_rowscaled", "fp8q_swiglu_quantize_act_1x128", "fp8q_quantize_per_tensor",
            "fp8q_quantize_act_w", "fp8q_moe_dispatch", "fp8q_moe_combine", "fp8q_moe_sort",
            "fp8q_moe_sort_backward", "fp8q_moe_combine_backward", "fp8q_swiglu_backward",
            "fp8q_quantize_act_grouped", "fp8q_grouped_gemm_rowscaled", "fp8q_adamw", "fp8q_layer_norm",
            "fp8q_layer_norm_backward", "fp8q_layer_norm_backward_workspace", "fp8q_moe_route",
            "fp8q_moe_route_workspace", "fp8q_moe_route_backward", "fp8q_orthogonalize", "fp8q_muon",
            "fp8q_muon_workspace", "fp8q_status_string", "fp8q_abi_version")


class Fp8qError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


class _AdamwTensor(ctypes.Structure):
    """fp8q_adamw_tensor of include/fp8q.h."""
    _fields_ = [(name, ctypes.c_void_p) for name in ("p", "grad", "m", "v", "m_scale", "v_scale", "p_bf16")] + [
        ("n", ctypes.c_int64)]


class _AdamwHyper(ctypes.Structure):
    """fp8q_adamw_hyper of include/fp8q.h."""
    _fields_ = [(name, ctypes.c_double) for name in ("lr", "beta1", "beta2", "eps", "weight_decay", "grad_scale")] + [
        ("step", ctypes.c_int64), ("scalars", ctypes.c_void_p)]


class _NewtonSchulz(ctypes.Structure):
    """fp8q_newton_schulz of include/fp8q.h."""
    _fields_ = [(name, ctypes.c_double) for name in "abc"] + [("steps", ctypes.c_int64)]


class _MuonHyper(ctypes.Structure):
    """fp8q_muon_hyper of include/fp8q.h."""
    _fields_ = [(name, ctypes.c_double) for name in ("lr", "beta", "weight_decay", "scale", "grad_scale")] + [
        ("ns", _NewtonSchulz), ("nesterov", ctypes.c_int64), ("device_lr", ctypes.c_void_p)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libfp8q.so (built by fp8_fine_grained_fp8q_amd.build) and declare its C ABI."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libfp8q.so not found at {path}; build it with "
                           "`python -m fp8_fine_grained_fp8q_amd.build`")
    lib = ctypes.CDLL(path)
    i64, vp, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32
    lib.fp8q_quantize_act_1x128.argtypes = [vp, i64, i64, vp, vp, vp]
    lib.fp8q_quantize_w_128x128.argtypes = [vp, i64, i64, i64, vp, vp, vp]
    lib.fp8q_gemm_blockscaled.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, i32, vp]
    lib.fp8q_grouped_gemm_blockscaled.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i32, vp]
    lib.fp8q_quantize_w_128x128_t.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp]
    lib.fp8q_quantize_act_dual.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp]
    lib.fp8q_gemm_rowscaled.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, i32, vp]
    lib.fp8q_swiglu_quantize_act_1x128.argtypes = [vp, i64, i64, vp, vp, vp]
    lib.fp8q_quantize_per_tensor.argtypes = [vp, i64, vp, vp, vp, vp]
    lib.fp8q_quantize_act_w.argtypes = [vp, i64, vp, i64, i64, i64, vp, vp, vp, vp, vp]
    lib.fp8q_moe_dispatch.argtypes = [vp, i64, i64, i64, i64, vp, vp, i64, i64, vp, vp, vp, vp, vp, vp]
    lib.fp8q_moe_combine.argtypes = [vp, i32, i64, i64, vp, vp, i64, i64, vp, i32, vp]
    lib.fp8q_moe_sort.argtypes = [vp, i64, i64, i64, i64, vp, i32, i64, i64, vp, vp, vp, vp, vp]
    lib.fp8q_moe_sort_backward.argtypes = [vp, i32, i64, i64, vp, i64, i64, vp, i32, vp]
    lib.fp8q_moe_combine_backward.argtypes = [vp, i32, vp, i32, i64, i64, vp, vp, i64, i64, vp, vp, vp]
    lib.fp8q_swiglu_backward.argtypes = [vp, vp, i32, i64, i64, vp, vp, vp]
    lib.fp8q_quantize_act_grouped.argtypes = [vp, vp, i64, i64, i64, vp, vp, vp, vp, vp]
    lib.fp8q_grouped_gemm_rowscaled.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i32, vp]
    lib.fp8q_adamw.argtypes = [ctypes.POINTER(_AdamwTensor), i64, i32, i32, ctypes.POINTER(_AdamwHyper), vp]
    f64 = ctypes.c_double
    lib.fp8q_layer_norm.argtypes = [vp, i32, vp, vp, i64, i64, f64, i32, vp, i32, vp, vp, vp]
    lib.fp8q_layer_norm_backward.argtypes = [vp, i32, vp, i32, vp, vp, vp, i64, i64, vp, i32, vp, vp, vp, vp]
    lib.fp8q_layer_norm_backward_workspace.argtypes = [i64, i64]
    lib.fp8q_moe_route.argtypes = [vp, i32, i64, i64, i64, i64, vp, vp, i32, i32, f64, f64, vp, vp, vp, vp, vp, vp, vp]
    lib.fp8q_moe_route_workspace.argtypes = [i64, i64, i64]
    lib.fp8q_moe_route_backward.argtypes = [vp, i32, i64, i64, i64, i64, vp, vp, vp, vp, vp, i32, i32, f64, vp, i32, vp]
    lib.fp8q_orthogonalize.argtypes = [vp, i32, i64, i64, i64, ctypes.POINTER(_NewtonSchulz), vp, vp, vp]
    lib.fp8q_muon.argtypes = [vp, vp, i32, vp, i64, i64, i64, ctypes.POINTER(_MuonHyper), vp, vp, vp]
    lib.fp8q_muon_workspace.argtypes = [i64, i64, i64]
    for name in EXPORTED:
        getattr(lib, name).restype = i64 if name.endswith("_workspace") else i32
    lib.fp8q_status_string.argtypes = [i32]
    lib.fp8q_status_string.restype = ctypes.c_char_p
    lib.fp8q_abi_version.argtypes = []
    lib.fp8q_abi_version.restype = i32
    if lib.fp8q_abi_version() != ABI_VERSION:
        raise RuntimeError("libfp8q ABI version mismatch; rebuild the library")
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().fp8q_status_string(int(status)).decode()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _check(status: int, what: str):
    if status != FP8Q_OK:
        raise Fp8qError(status, what)


def _need(t: torch.Tensor, dtype, name: str, shape=None):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _here(*tensors) -> int:
    """Checks that the tensors are on the current device; the current stream's handle.
    (torch.cuda.current_stream() wraps it in an object first, 3 us of a call that takes 8.)"""
    device = torch.cuda.current_device()
    for t in tensors:
        if t is not None and (not isinstance(t, torch.Tensor) or t.get_device() != device):
            raise ValueError(f"tensors must be on the current device cuda:{device}, got {getattr(t, 'device', type(t))}")
    return torch._C._cuda_getCurrentRawStream(device)


def _on(stream):
    """`stream` (a torch stream or a handle) as the current one, so that what is allocated inside
    belongs to the stream that writes it."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _out(t, dtype, name: str, shape, like: torch.Tensor):
    """The caller's output, checked, or a new one on `like`'s device.  (Of the ways to make one,
    empty_like takes 1.2 us, new_empty 1.2 to 1.5 and torch.empty 1.7.)"""
    if t is None:
        if shape == like.shape:
            return torch.empty_like(like) if dtype == like.dtype else torch.empty_like(like, dtype=dtype)
        return like.new_empty(*shape) if dtype == like.dtype else like.new_empty(*shape, dtype=dtype)
    _need(t, dtype, name, shape)
    return t


def _need_rows(t, name: str, columns: int = 8, rows=None):
    """A contiguous bf16 or float32 [rows, C] with C a multiple of `columns`."""
    if not isinstance(t, torch.Tensor) or (t.dtype != torch.bfloat16 and t.dtype != torch.float32):
        raise ValueError(f"{name} must be a bfloat16 or float32 tensor")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    shape = t.shape
    if len(shape) != 2 or shape[1] % columns or (rows is not None and shape[0] != rows):
        raise ValueError(f"{name} must be [{'rows' if rows is None else rows}, C] with C a multiple of {columns}, "
                         f"got {tuple(t.shape)}")


def fp8q_quantize_act_1x128(x: torch.Tensor, xq: torch.Tensor | None = None,
                            sa: torch.Tensor | None = None, stream=None):
    """1x128 activation tiles -> (xq uint8 [M, K], sa float32 [K/128, M])."""
    _need(x, torch.bfloat16, "x")
    M, K = x.shape
    if xq is None:
        xq = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    if sa is None:
        sa = torch.empty((K // 128, M), dtype=torch.float32, device=x.device)
    _need(xq, torch.uint8, "xq", (M, K))
    _need(sa, torch.float32, "sa", (K // 128, M))
    _check(load_library().fp8q_quantize_act_1x128(_ptr(x), M, K, _ptr(xq), _ptr(sa), _stream(stream)),
           "fp8q_quantize_act_1x128")
    return xq, sa


def fp8q_quantize_w_128x128(w: torch.Tensor, wq: torch.Tensor | None = None,
                            sb: torch.Tensor | None = None, stream=None):
    """128x128 weight blocks of w [G, N, K] (or [N, K]) -> (wq uint8, sb float32 [G, N/128, K/128])."""
    _need(w, torch.bfloat16, "w")
    squeeze = w.dim() == 2
    G, N, K = (1, *w.shape) if squeeze else w.shape
    if wq is None:
        wq = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    shape = (N // 128, K // 128) if squeeze else (G, N // 128, K // 128)
    if sb is None:
        sb = torch.empty(shape, dtype=torch.float32, device=w.device)
    _need(wq, torch.uint8, "wq", w.shape)
    _need(sb, torch.float32, "sb", shape)
    _check(load_library().fp8q_quantize_w_128x128(_ptr(w), G, N, K, _ptr(wq), _ptr(sb), _stream(stream)),
           "fp8q_quantize_w_128x128")
    return wq, sb


def fp8q_quantize_act_w(x: torch.Tensor, w: torch.Tensor, xq: torch.Tensor | None = None,
                        sa: torch.Tensor | None = None, wq: torch.Tensor | None = None,
                        sb: torch.Tensor | None = None, stream=None):
    """Both quantizers of a linear layer in one launch: x [M, K] -> (xq, sa) as
    fp8q_quantize_act_1x128 and w [G, N, K] (or [N, K]) -> (wq, sb) as fp8q_quantize_w_128x128."""
    _need(x, torch.bfloat16, "x")
    _need(w, torch.bfloat16, "w")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    M, K = x.shape
    squeeze = w.dim() == 2
    G, N, Kw = (1, *w.shape) if squeeze else w.shape
    if Kw != K:
        raise ValueError(f"x and w must share K, got {K} and {Kw}")
    if xq is None:
        xq = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    if sa is None:
        sa = torch.empty((K // 128, M), dtype=torch.float32, device=x.device)
    if wq is None:
        wq = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    sb_shape = (N // 128, K // 128) if squeeze else (G, N // 128, K // 128)
    if sb is None:
        sb = torch.empty(sb_shape, dtype=torch.float32, device=w.device)
    _need(xq, torch.uint8, "xq", (M, K))
    _need(sa, torch.float32, "sa", (K // 128, M))
    _need(wq, torch.uint8, "wq", w.shape)
    _need(sb, torch.float32, "sb", sb_shape)
    _check(load_library().fp8q_quantize_act_w(_ptr(x), M, _ptr(w), G, N, K, _ptr(xq), _ptr(sa), _ptr(wq), _ptr(sb),
                                              _stream(stream)), "fp8q_quantize_act_w")
    return xq, sa, wq, sb


def fp8q_moe_dispatch(topk_ids: torch.Tensor, xq: torch.Tensor, sa: torch.Tensor, e_begin: int, n_experts: int,
                      capacity: int | None = None, stream=None):
    """Expert-parallel dispatch of quantized tokens to the local experts [e_begin,
    e_begin + n_experts): topk_ids int32 [T, k], xq uint8 [T, K], sa float32 [K/128, T] ->
    (xq_sorted uint8 [capacity, K], sa_sorted float32 [K/128, capacity], offsets int32
    [n_experts + 1], token_row int32 [T, k], row_token int32 [capacity]); capacity defaults
    to T*k.  offsets feed fp8q_grouped_gemm_blockscaled with the sorted tensors."""
    _need(topk_ids, torch.int32, "topk_ids")
    if topk_ids.dim() != 2:
        raise ValueError("topk_ids must be 2-D [T, k]")
    T, k = topk_ids.shape
    _need(xq, torch.uint8, "xq")
    if xq.dim() != 2 or xq.shape[0] != T:
        raise ValueError(f"xq must be [T={T}, K]")
    K = xq.shape[1]
    _need(sa, torch.float32, "sa", (K // 128, T))
    cap = T * k if capacity is None else int(capacity)
    dev = xq.device
    xs = torch.empty((cap, K), dtype=torch.uint8, device=dev)
    ss = torch.empty((K // 128, cap), dtype=torch.float32, device=dev)
    offsets = torch.empty(n_experts + 1, dtype=torch.int32, device=dev)
    token_row = torch.empty((T, k), dtype=torch.int32, device=dev)
    row_token = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    _check(load_library().fp8q_moe_dispatch(_ptr(topk_ids), T, k, e_begin, n_experts, _ptr(xq), _ptr(sa), K, cap,
                                            _ptr(xs), _ptr(ss), _ptr(offsets), _ptr(token_row), _ptr(row_token),
                                            _stream(stream)), "fp8q_moe_dispatch")
    return xs, ss, offsets, token_row, row_token[:cap]


def fp8q_moe_combine(expert_out: torch.Tensor, token_row: torch.Tensor, topk_w: torch.Tensor,
                     y: torch.Tensor | None = None, out_dtype=torch.bfloat16, stream=None):
    """Expert-parallel combine: y[t] = sum over local slots of topk_w[t, s] * expert_out[token_row[t, s]]
    (expert_out bf16 or float32 [capacity, N]; token_row int32 / topk_w float32 [T, k])."""
    if expert_out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("expert_out must be bfloat16 or float32")
    _need(expert_out, expert_out.dtype, "expert_out")
    _need(token_row, torch.int32, "token_row")
    if token_row.dim() != 2 or expert_out.dim() != 2:
        raise ValueError("token_row must be [T, k] and expert_out [capacity, N]")
    T, k = token_row.shape
    cap, N = expert_out.shape
    _need(topk_w, torch.float32, "topk_w", (T, k))
    if y is None:
        y = torch.empty((T, N), dtype=out_dtype, device=expert_out.device)
    _need(y, out_dtype, "y", (T, N))
    _check(load_library().fp8q_moe_combine(_ptr(expert_out), _out_code(expert_out.dtype), cap, N, _ptr(token_row),
                                           _ptr(topk_w), T, k, _ptr(y), _out_code(out_dtype), _stream(stream)),
           "fp8q_moe_combine")
    return y


def _out_code(out_dtype) -> int:
    if out_dtype == torch.bfloat16:
        return FP8Q_OUT_BF16
    if out_dtype == torch.float32:
        return FP8Q_OUT_F32
    raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")


def fp8q_gemm_blockscaled(xq, sa, wq, sb, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
                          stream=None):
    """C = dequant(xq, sa) @ dequant(wq, sb)^T with FP32 promotion per 128-wide K block."""
    _need(xq, torch.uint8, "xq")
    _need(wq, torch.uint8, "wq")
    _need(sa, torch.float32, "sa")
    _need(sb, torch.float32, "sb")
    M, K = xq.shape
    if wq.dim() == 3 and wq.shape[0] == 1:
        wq, sb = wq[0], sb.reshape(sb.shape[-2:])
    if wq.dim() != 2:
        raise ValueError("the dense GEMM takes one weight matrix wq [N, K]; use the grouped GEMM for experts")
    N = wq.shape[0]
    _need(wq, torch.uint8, "wq", (N, K))
    _need(sa, torch.float32, "sa", (K // 128, M))
    _need(sb, torch.float32, "sb", (N // 128, K // 128))
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=xq.device)
    _need(out, out.dtype, "out", (M, N))
    _check(load_library().fp8q_gemm_blockscaled(_ptr(xq), _ptr(sa), _ptr(wq), _ptr(sb), M, N, K, _ptr(out),
                                                _out_code(out.dtype), _stream(stream)),
           "fp8q_gemm_blockscaled")
    return out


def fp8q_grouped_gemm_blockscaled(xq, sa, wq, sb, offsets, out_dtype=torch.bfloat16,
                                  out: torch.Tensor | None = None, stream=None):
    """Grouped (MoE): rows offsets[g]..offsets[g+1]-1 use expert g's weights wq[g], sb[g]."""
    _need(xq, torch.uint8, "xq")
    _need(wq, torch.uint8, "wq")
    _need(sa, torch.float32, "sa")
    _need(sb, torch.float32, "sb")
    _need(offsets, torch.int32, "offsets")
    M, K = xq.shape
    G, N, _ = wq.shape
    _need(wq, torch.uint8, "wq", (G, N, K))
    _need(sa, torch.float32, "sa", (K // 128, M))
    _need(sb, torch.float32, "sb", (G, N // 128, K // 128))
    _need(offsets, torch.int32, "offsets", (G + 1,))
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=xq.device)
    _need(out, out.dtype, "out", (M, N))
    _check(load_library().fp8q_grouped_gemm_blockscaled(
        _ptr(xq), _ptr(sa), _ptr(wq), _ptr(sb), _ptr(offsets), G, M, N, K, _ptr(out),
        _out_code(out.dtype), _stream(stream)), "fp8q_grouped_gemm_blockscaled")
    return out


def fp8q_quantize_w_128x128_t(w: torch.Tensor, wq=None, sb=None, wqt=None, sbt=None, stream=None):
    """128x128 blocks of w [G, N, K] (or [N, K]) -> (wq, sb, wqt, sbt): the codes and scales
    of w and of its transpose (wqt uint8 [G, K, N], sbt float32 [G, K/128, N/128])."""
    _need(w, torch.bfloat16, "w")
    squeeze = w.dim() == 2
    G, N, K = (1, *w.shape) if squeeze else w.shape
    lead = () if squeeze else (G,)
    dev = w.device
    wq = torch.empty(w.shape, dtype=torch.uint8, device=dev) if wq is None else wq
    sb = torch.empty(lead + (N // 128, K // 128), dtype=torch.float32, device=dev) if sb is None else sb
    wqt = torch.empty(lead + (K, N), dtype=torch.uint8, device=dev) if wqt is None else wqt
    sbt = torch.empty(lead + (K // 128, N // 128), dtype=torch.float32, device=dev) if sbt is None else sbt
    _need(wq, torch.uint8, "wq", w.shape)
    _need(sb, torch.float32, "sb", lead + (N // 128, K // 128))
    _need(wqt, torch.uint8, "wqt", lead + (K, N))
    _need(sbt, torch.float32, "sbt", lead + (K // 128, N // 128))
    _check(load_library().fp8q_quantize_w_128x128_t(_ptr(w), G, N, K, _ptr(wq), _ptr(sb), _ptr(wqt), _ptr(sbt),
                                                    _stream(stream)), "fp8q_quantize_w_128x128_t")
    return wq, sb, wqt, sbt


def fp8q_quantize_act_dual(x: torch.Tensor, xq=None, sa=None, xqt=None, sat=None, stream=None):
    """x bf16 [M, K] (M % 128 == 0) -> (xq [M, K], sa [K/128, M], xqt [K, M], sat [M/128, K]):
    1x128 tiles along K and tiles of 128 tokens along M (codes channel-major)."""
    _need(x, torch.bfloat16, "x")
    M, K = x.shape
    dev = x.device
    xq = torch.empty((M, K), dtype=torch.uint8, device=dev) if xq is None else xq
    sa = torch.empty((K // 128, M), dtype=torch.float32, device=dev) if sa is None else sa
    xqt = torch.empty((K, M), dtype=torch.uint8, device=dev) if xqt is None else xqt
    sat = torch.empty((M // 128, K), dtype=torch.float32, device=dev) if sat is None else sat
    _need(xq, torch.uint8, "xq", (M, K))
    _need(sa, torch.float32, "sa", (K // 128, M))
    _need(xqt, torch.uint8, "xqt", (K, M))
    _need(sat, torch.float32, "sat", (M // 128, K))
    _check(load_library().fp8q_quantize_act_dual(_ptr(x), M, K, _ptr(xq), _ptr(sa), _ptr(xqt), _ptr(sat),
                                                 _stream(stream)), "fp8q_quantize_act_dual")
    return xq, sa, xqt, sat


def fp8q_gemm_rowscaled(aq, sa, bq, sb, out_dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None):
    """C [P, Q] = dequant(aq, sa) @ dequant(bq, sb)^T with 1x128 row scales on both operands:
    aq [P, Kc], sa [Kc/128, P], bq [Q, Kc], sb [Kc/128, Q]."""
    _need(aq, torch.uint8, "aq")
    _need(bq, torch.uint8, "bq")
    _need(sa, torch.float32, "sa")
    _need(sb, torch.float32, "sb")
    P, Kc = aq.shape
    Q = bq.shape[0]
    _need(bq, torch.uint8, "bq", (Q, Kc))
    _need(sa, torch.float32, "sa", (Kc // 128, P))
    _need(sb, torch.float32, "sb", (Kc // 128, Q))
    if out is None:
        out = torch.empty((P, Q), dtype=out_dtype, device=aq.device)
    _need(out, out.dtype, "out", (P, Q))
    _check(load_library().fp8q_gemm_rowscaled(_ptr(aq), _ptr(sa), _ptr(bq), _ptr(sb), P, Q, Kc, _ptr(out),
                                              _out_code(out.dtype), _stream(stream)), "fp8q_gemm_rowscaled")
    return out


def fp8q_swiglu_quantize_act_1x128(gu: torch.Tensor, xq=None, sa=None, stream=None):
    """gu bf16 [M, 2I] (g | u) -> (xq uint8 [M, I], sa float32 [I/128, M]) for h = SiLU(g) * u."""
    _need(gu, torch.bfloat16, "gu")
    M, I2 = gu.shape
    I = I2 // 2
    xq = torch.empty((M, I), dtype=torch.uint8, device=gu.device) if xq is None else xq
    sa = torch.empty((I // 128, M), dtype=torch.float32, device=gu.device) if sa is None else sa
    _need(xq, torch.uint8, "xq", (M, I))
    _need(sa, torch.float32, "sa", (I // 128, M))
    _check(load_library().fp8q_swiglu_quantize_act_1x128(_ptr(gu), M, I, _ptr(xq), _ptr(sa), _stream(stream)),
           "fp8q_swiglu_quantize_act_1x128")
    return xq, sa


def fp8q_quantize_per_tensor(x: torch.Tensor, scale: torch.Tensor | None = None, q=None, stats=None, stream=None):
    """One scale for all of x (bf16, any shape, numel % 8 == 0): tensor-level scaling when
    `scale` is None, else delayed scaling with that device float32 scale.  Returns
    (q uint8 like x, stats int32 [3]: amax bits, saturated count, scale bits)."""
    _need(x, torch.bfloat16, "x")
    if scale is not None:
        _need(scale, torch.float32, "scale")
    q = torch.empty(x.shape, dtype=torch.uint8, device=x.device) if q is None else q
    stats = torch.empty(3, dtype=torch.int32, device=x.device) if stats is None else stats
    _need(q, torch.uint8, "q", x.shape)
    _need(stats, torch.int32, "stats", (3,))
    if scale is not None and scale.numel() != 1:
        raise ValueError("scale must hold one float32")
    _check(load_library().fp8q_quantize_per_tensor(_ptr(x), x.numel(), _ptr(scale), _ptr(q), _ptr(stats),
                                                   _stream(stream)), "fp8q_quantize_per_tensor")
    return q, stats


def tensor_stats(stats: torch.Tensor):
    """(amax, saturated count, scale) of a stats tensor from fp8q_quantize_per_tensor."""
    h = stats.cpu()
    return (float(h[0:1].view(torch.float32)), int(h[1]), float(h[2:3].view(torch.float32)))


def fp8q_moe_sort(topk_ids: torch.Tensor, x: torch.Tensor, e_begin: int, n_experts: int, capacity: int | None = None,
                  xs: torch.Tensor | None = None, row_token: torch.Tensor | None = None, stream=None):
    """Rows of x (bf16 or float32 [T, H]) in expert order for the local experts [e_begin, e_begin
    + n_experts): topk_ids int32 [T, k] -> (xs [capacity, H], offsets int32 [n_experts + 1],
    token_row int32 [T, k], row_token int32 [capacity]), the maps as fp8q_moe_dispatch gives
    them; capacity defaults to xs's rows, or to T*k.  Rows of xs and row_token behind the last
    routed one are left as they were."""
    if stream is not None:
        with _on(stream):
            return fp8q_moe_sort(topk_ids, x, e_begin, n_experts, capacity, xs, row_token)
    _need(topk_ids, torch.int32, "topk_ids")
    if topk_ids.dim() != 2:
        raise ValueError("topk_ids must be 2-D [T, k]")
    T, k = topk_ids.shape
    _need_rows(x, "x", rows=T)
    H = x.shape[1]
    cap = int(capacity) if capacity is not None else (xs.shape[0] if xs is not None else T * k)
    if cap < 0 or n_experts < 1:
        raise ValueError("capacity must not be negative and n_experts must be positive")
    s = _here(topk_ids, x, xs, row_token)
    xs = _out(xs, x.dtype, "xs", (cap, H), x)
    row_token = _out(row_token, torch.int32, "row_token", (cap,), x)
    offsets, token_row = topk_ids.new_empty(n_experts + 1), torch.empty_like(topk_ids)
    _check(load_library().fp8q_moe_sort(_ptr(topk_ids), T, k, e_begin, n_experts, _ptr(x), _out_code(x.dtype), H, cap,
                                        _ptr(xs), _ptr(offsets), _ptr(token_row), _ptr(row_token), s),
           "fp8q_moe_sort")
    return xs, offsets, token_row, row_token


def fp8q_moe_sort_backward(dxs: torch.Tensor, token_row: torch.Tensor, dx: torch.Tensor | None = None,
                           out_dtype=torch.bfloat16, stream=None):
    """Gradient of the sort: dx[t] = sum over the token's rows of dxs[row] (dxs bf16 or float32
    [capacity, H], token_row int32 [T, k]) -> dx [T, H] in out_dtype."""
    if stream is not None:
        with _on(stream):
            return fp8q_moe_sort_backward(dxs, token_row, dx, out_dtype)
    _need_rows(dxs, "dxs")
    _need(token_row, torch.int32, "token_row")
    if token_row.dim() != 2:
        raise ValueError("token_row must be 2-D [T, k]")
    (T, k), (cap, H) = token_row.shape, dxs.shape
    s = _here(dxs, token_row, dx)
    dx = _out(dx, out_dtype if dx is None else dx.dtype, "dx", (T, H), dxs)
    _check(load_library().fp8q_moe_sort_backward(_ptr(dxs), _out_code(dxs.dtype), cap, H, _ptr(token_row), T, k,
                                                 _ptr(dx), _out_code(dx.dtype), s), "fp8q_moe_sort_backward")
    return dx


def fp8q_moe_combine_backward(dy: torch.Tensor, expert_out: torch.Tensor, token_row: torch.Tensor,
                              topk_w: torch.Tensor, dout: torch.Tensor | None = None, dw: torch.Tensor | None = None,
                              stream=None):
    """Gradients of fp8q_moe_combine: dy [T, N] and expert_out [capacity, N] (bf16 or float32
    each), token_row int32 / topk_w float32 [T, k] -> (dout like expert_out with dout[row] =
    topk_w[t, s] * dy[t], dw float32 [T, k] with dw[t, s] = <expert_out[row], dy[t]>).  Rows of
    dout without a slot are left as they were; dw is 0 for slots without a row."""
    if stream is not None:
        with _on(stream):
            return fp8q_moe_combine_backward(dy, expert_out, token_row, topk_w, dout, dw)
    _need(token_row, torch.int32, "token_row")
    if token_row.dim() != 2:
        raise ValueError("token_row must be 2-D [T, k]")
    T, k = token_row.shape
    _need_rows(dy, "dy", rows=T)
    N = dy.shape[1]
    _need_rows(expert_out, "expert_out")
    if expert_out.shape[1] != N:
        raise ValueError(f"expert_out must be [capacity, {N}], got {tuple(expert_out.shape)}")
    _need(topk_w, torch.float32, "topk_w", (T, k))
    s = _here(dy, expert_out, token_row, topk_w, dout, dw)
    dout = _out(dout, expert_out.dtype, "dout", expert_out.shape, expert_out)
    dw = _out(dw, torch.float32, "dw", (T, k), topk_w)
    _check(load_library().fp8q_moe_combine_backward(_ptr(dy), _out_code(dy.dtype), _ptr(expert_out),
                                                    _out_code(expert_out.dtype), expert_out.shape[0], N,
                                                    _ptr(token_row), _ptr(topk_w), T, k, _ptr(dout), _ptr(dw), s),
           "fp8q_moe_combine_backward")
    return dout, dw


def fp8q_swiglu_backward(gu: torch.Tensor, dh: torch.Tensor, dgu: torch.Tensor | None = None,
                         h: torch.Tensor | None = None, want_h: bool = False, stream=None):
    """Gradient of h = SiLU(g) * u: gu bf16 [M, 2I] (g | u), dh bf16 or float32 [M, I] -> (dgu bf16
    [M, 2I], h bf16 [M, I] if want_h or a buffer for it is given, else None)."""
    if stream is not None:
        with _on(stream):
            return fp8q_swiglu_backward(gu, dh, dgu, h, want_h)
    _need(gu, torch.bfloat16, "gu")
    if gu.dim() != 2 or gu.shape[1] % 16:
        raise ValueError(f"gu must be [M, 2I] with I a multiple of 8, got {tuple(gu.shape)}")
    M, I = gu.shape[0], gu.shape[1] // 2
    _need_rows(dh, "dh", rows=M)
    if dh.shape[1] != I:
        raise ValueError(f"dh must be [{M}, {I}], got {tuple(dh.shape)}")
    s = _here(gu, dh, dgu, h)
    dgu = _out(dgu, torch.bfloat16, "dgu", (M, 2 * I), gu)
    if want_h or h is not None:
        h = _out(h, torch.bfloat16, "h", (M, I), gu)
    _check(load_library().fp8q_swiglu_backward(_ptr(gu), _ptr(dh), _out_code(dh.dtype), M, I, _ptr(dgu), _ptr(h), s),
           "fp8q_swiglu_backward")
    return dgu, h


def fp8q_quantize_act_grouped(x: torch.Tensor, offsets: torch.Tensor, rows: bool = True, xq=None, sa=None, xqt=None,
                              sat=None, stream=None):
    """x bf16 [M, K] sorted by expert, offsets int32 [G + 1] -> (xq uint8 [M, K], sa float32
    [K/128, M], xqt uint8 [B, K, 128], sat float32 [B, K]) with B = M // 128 + G: 1x128 tiles
    along K (None, None with rows=False) and tiles of 128 tokens of one expert."""
    if stream is not None:
        with _on(stream):
            return fp8q_quantize_act_grouped(x, offsets, rows, xq, sa, xqt, sat)
    _need(x, torch.bfloat16, "x")
    _need(offsets, torch.int32, "offsets")
    if x.dim() != 2 or x.shape[1] % 128 or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError(f"x must be [M, K] with K a multiple of 128 and offsets [G + 1], got {tuple(x.shape)} and "
                         f"{tuple(offsets.shape)}")
    (M, K), G = x.shape, offsets.shape[0] - 1
    tiles = M // 128 + G
    if not rows and (xq is not None or sa is not None):
        raise ValueError("xq and sa are written with rows=True only")
    s = _here(x, offsets, xq, sa, xqt, sat)
    if rows:
        xq = _out(xq, torch.uint8, "xq", (M, K), x)
        sa = _out(sa, torch.float32, "sa", (K // 128, M), x)
    xqt = _out(xqt, torch.uint8, "xqt", (tiles, K, 128), x)
    sat = _out(sat, torch.float32, "sat", (tiles, K), x)
    _check(load_library().fp8q_quantize_act_grouped(_ptr(x), _ptr(offsets), G, M, K, _ptr(xq), _ptr(sa), _ptr(xqt),
                                                    _ptr(sat), s), "fp8q_quantize_act_grouped")
    return xq, sa, xqt, sat


def fp8q_grouped_gemm_rowscaled(aq, sa, bq, sb, offsets, m_tot: int, out_dtype=torch.bfloat16,
                                out: torch.Tensor | None = None, stream=None):
    """The experts' weight gradients C [G, P, Q]: C[g] = dequant(aq, sa) @ dequant(bq, sb)^T over expert
    g's token tiles; aq [B, P, 128], sa [B, P], bq [B, Q, 128], sb [B, Q] from
    fp8q_quantize_act_grouped of tensors with m_tot rows and these offsets."""
    if stream is not None:
        with _on(stream):
            return fp8q_grouped_gemm_rowscaled(aq, sa, bq, sb, offsets, m_tot, out_dtype, out)
    _need(aq, torch.uint8, "aq")
    _need(bq, torch.uint8, "bq")
    _need(offsets, torch.int32, "offsets")
    if aq.dim() != 3 or bq.dim() != 3 or offsets.dim() != 1 or offsets.shape[0] < 2 or m_tot < 0:
        raise ValueError("aq must be [B, P, 128], bq [B, Q, 128] and offsets [G + 1]")
    P, Q, G = aq.shape[1], bq.shape[1], offsets.shape[0] - 1
    tiles = int(m_tot) // 128 + G
    _need(aq, torch.uint8, "aq", (tiles, P, 128))
    _need(bq, torch.uint8, "bq", (tiles, Q, 128))
    _need(sa, torch.float32, "sa", (tiles, P))
    _need(sb, torch.float32, "sb", (tiles, Q))
    s = _here(aq, sa, bq, sb, offsets, out)
    out = _out(out, out_dtype if out is None else out.dtype, "out", (G, P, Q), aq)
    _check(load_library().fp8q_grouped_gemm_rowscaled(_ptr(aq), _ptr(sa), _ptr(bq), _ptr(sb), _ptr(offsets), G,
                                                      int(m_tot), P, Q, _ptr(out), _out_code(out.dtype), s),
           "fp8q_grouped_gemm_rowscaled")
    return out


class AdamwPlan:
    """The tensors of an AdamW step, their types, sizes and memory checked once (fp8q_adamw_plan makes
    it).  It holds the tensors.  A step checks that each still has its memory and that a gradient
    which was its parameter's `.grad` still is, and raises ValueError otherwise: `tensor.data = ...`,
    a resized storage and zero_grad(set_to_none=True) need a new plan.  A captured step does
    not check when it is replayed."""

    def __init__(self, tensors, descriptors, grad_dtype, state_dtype, device):
        self.tensors, self.descriptors = tensors, descriptors
        self.grad_dtype, self.state_dtype, self.device = grad_dtype, state_dtype, device
        self.every = [t for each in tensors.values() for t in each]
        self.addresses = list(map(torch.Tensor.data_ptr, self.every))
        self.followed = [(p, g) for p, g in zip(tensors["params"], tensors["grads"]) if p.is_leaf and p.grad is g]

    def check(self):
        """Raises ValueError if a tensor's memory or a parameter's gradient is another one than the plan's.
        (0.04 us a tensor: 9 us for 64 parameters with FP32 states.)"""
        if list(map(torch.Tensor.data_ptr, self.every)) != self.addresses:
            raise ValueError("a tensor of the plan has other memory than when the plan was made; make a new plan")
        for p, g in self.followed:
            if p.grad is not g:
                raise ValueError("a parameter's .grad is not the plan's gradient any more; make a new plan, or keep the "
                                 "gradients (zero_grad(set_to_none=False))")


def fp8q_adamw_plan(params, grads, m, v, m_scales=None, v_scales=None, copies=None) -> AdamwPlan:
    """Lists of tensors, one entry per parameter, any shapes: params float32, grads bf16 or float32
    (one type for all), states m and v float32, or uint8 with float32 m_scales / v_scales of
    ceil(n / 128) entries each (E4M3 codes of m and of sqrt(v); zeros start a run); copies
    bf16, written with the new parameters, or None.  All memory disjoint."""
    lists = {"params": params, "grads": grads, "m": m, "v": v, "m_scales": m_scales, "v_scales": v_scales,
             "copies": copies}
    if any(lists[k] is None for k in ("params", "grads", "m", "v")):
        raise ValueError("params, grads, m and v are needed")
    lists = {k: list(x) for k, x in lists.items() if x is not None}
    count = len(lists["params"])
    if any(len(x) != count for x in lists.values()):
        raise ValueError(f"the lists must have {count} tensors each")
    e4m3 = "m_scales" in lists
    if e4m3 != ("v_scales" in lists):
        raise ValueError("m_scales and v_scales go together")
    grad = getattr(lists["grads"][0], "dtype", None) if count else torch.float32  # None: a parameter's .grad may be
    if grad not in (torch.bfloat16, torch.float32):
        raise ValueError("grads must be bfloat16 or float32 tensors")
    state = torch.uint8 if e4m3 else torch.float32
    types = {"params": torch.float32, "grads": grad, "m": state, "v": state, "m_scales": torch.float32,
             "v_scales": torch.float32, "copies": torch.bfloat16}
    table = (_AdamwTensor * max(count, 1))()
    fields = {"params": "p", "grads": "grad", "m": "m", "v": "v", "m_scales": "m_scale", "v_scales": "v_scale",
              "copies": "p_bf16"}
    spans, devices = [], set()
    for name, tensors in lists.items():
        for i, t in enumerate(tensors):
            _need(t, types[name], f"{name}[{i}]")
            n = lists["params"][i].numel()
            want = -(-n // 128) if name.endswith("scales") else n
            if t.numel() != want:
                raise ValueError(f"{name}[{i}] must have {want} elements, got {t.numel()}")
            if n and t.data_ptr() % (4 if name.endswith("scales") else 16):
                raise ValueError(f"{name}[{i}] must be {4 if name.endswith('scales') else 16}-byte aligned")
            setattr(table[i], fields[name], t.data_ptr() if n else None)
            table[i].n = n
            devices.add(t.device)
            if n:
                spans.append((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), f"{name}[{i}]"))
    spans.sort()
    for a, b in zip(spans, spans[1:]):
        if b[0] < a[1]:
            raise ValueError(f"{a[2]} and {b[2]} share memory")
    if len(devices) > 1:
        raise ValueError("all tensors must be on one device")
    return AdamwPlan(lists, table, _out_code(grad), FP8Q_STATE_E4M3 if e4m3 else FP8Q_STATE_F32,
                     devices.pop() if devices else None)


def fp8q_adamw(plan: AdamwPlan, lr: float, betas=(0.9, 0.95), eps: float = 1e-8, weight_decay: float = 0.0, step: int = 1,
               grad_scale: float = 1.0, scalars: torch.Tensor | None = None, stream=None) -> None:
    """One AdamW step over the plan's tensors, in place; ValueError if one of them has other memory or
    another gradient than when the plan was made.  `step` counts from 1.  `scalars`: a device
    float32 [4] holding {lr, 1 - beta1^step, 1 - beta2^step, grad_scale}, read by the kernels in
    place of those arguments (a captured step is replayed with new values in it)."""
    if stream is not None:
        with _on(stream):
            return fp8q_adamw(plan, lr, betas, eps, weight_decay, step, grad_scale, scalars)
    if not isinstance(plan, AdamwPlan):
        raise ValueError("plan must come from fp8q_adamw_plan")
    if scalars is not None:
        _need(scalars, torch.float32, "scalars", (4,))
    if plan.device is None:
        return
    plan.check()
    hyper = _AdamwHyper(lr, betas[0], betas[1], eps, weight_decay, grad_scale, step, _ptr(scalars) or None)
    s = _here(plan.tensors["params"][0], scalars)
    _check(load_library().fp8q_adamw(plan.descriptors, len(plan.tensors["params"]), plan.grad_dtype, plan.state_dtype,
                                     ctypes.byref(hyper), s), "fp8q_adamw")


def _workspace(size, like: torch.Tensor):
    """`size` bytes (or a status) of scratch memory on `like`'s device, of the current stream's allocator."""
    if size < 0:
        raise Fp8qError(int(size), "workspace")
    return like.new_empty(size, dtype=torch.uint8)


def fp8q_layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, eps: float = 1e-5,
                    center: bool = True, out_dtype=None, y: torch.Tensor | None = None, stream=None):
    """Layer norm, or RMS norm with center=False, of every row: x bf16 or float32 [T, H], weight and bias
    float32 [H] -> (y [T, H] in out_dtype (x's by default), mean float32 [T] or None, rstd float32 [T])."""
    if stream is not None:
        with _on(stream):
            return fp8q_layer_norm(x, weight, bias, eps, center, out_dtype, y)
    _need_rows(x, "x")
    T, H = x.shape
    _need(weight, torch.float32, "weight", (H,))
    if bias is not None:
        _need(bias, torch.float32, "bias", (H,))
    s = _here(x, weight, bias, y)
    y = _out(y, (out_dtype or x.dtype) if y is None else y.dtype, "y", x.shape, x)
    mean = weight.new_empty(T) if center else None
    rstd = weight.new_empty(T)
    _check(load_library().fp8q_layer_norm(_ptr(x), _out_code(x.dtype), _ptr(weight), _ptr(bias), T, H, eps, bool(center),
                                          _ptr(y), _out_code(y.dtype), _ptr(mean), _ptr(rstd), s), "fp8q_layer_norm")
    return y, mean, rstd


def fp8q_layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor | None,
                             rstd: torch.Tensor, want_bias: bool = False, out_dtype=None, dx: torch.Tensor | None = None,
                             stream=None):
    """Gradients of fp8q_layer_norm (mean None: RMS norm): dy and x bf16 or float32 [T, H] each, weight [H],
    mean and rstd [T] float32 -> (dx [T, H] in out_dtype (x's by default), dweight float32 [H], dbias float32
    [H] with want_bias, else None)."""
    if stream is not None:
        with _on(stream):
            return fp8q_layer_norm_backward(dy, x, weight, mean, rstd, want_bias, out_dtype, dx)
    _need_rows(x, "x")
    T, H = x.shape
    _need_rows(dy, "dy", rows=T)
    if dy.shape[1] != H:
        raise ValueError(f"dy must be [{T}, {H}], got {tuple(dy.shape)}")
    _need(weight, torch.float32, "weight", (H,))
    if mean is not None:
        _need(mean, torch.float32, "mean", (T,))
    _need(rstd, torch.float32, "rstd", (T,))
    s = _here(dy, x, weight, mean, rstd, dx)
    lib = load_library()
    dx = _out(dx, (out_dtype or x.dtype) if dx is None else dx.dtype, "dx", x.shape, x)
    dweight = torch.empty_like(weight)
    dbias = torch.empty_like(weight) if want_bias else None
    work = _workspace(lib.fp8q_layer_norm_backward_workspace(T, H), x)
    _check(lib.fp8q_layer_norm_backward(_ptr(dy), _out_code(dy.dtype), _ptr(x), _out_code(x.dtype), _ptr(weight),
                                        _ptr(mean), _ptr(rstd), T, H, _ptr(dx), _out_code(dx.dtype), _ptr(dweight),
                                        _ptr(dbias), _ptr(work), s), "fp8q_layer_norm_backward")
    return dx, dweight, dbias


_SCORES = {"softmax": FP8Q_SCORE_SOFTMAX, "sigmoid": FP8Q_SCORE_SIGMOID}


def _logits_shape(logits):
    """(B, S, E) of the router's logits [S, E] or [B, S, E]."""
    if not isinstance(logits, torch.Tensor) or (logits.dtype != torch.bfloat16 and logits.dtype != torch.float32):
        raise ValueError("logits must be a bfloat16 or float32 tensor")
    if not logits.is_cuda or not logits.is_contiguous() or logits.dim() not in (2, 3):
        raise ValueError("logits must be a contiguous CUDA tensor [S, E] or [B, S, E]")
    return (1, *logits.shape) if logits.dim() == 2 else tuple(logits.shape)


def _score_code(score):
    if score not in _SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    return _SCORES[score]


def fp8q_moe_route(logits: torch.Tensor, k: int, bias: torch.Tensor | None = None, valid: torch.Tensor | None = None,
                   score: str = "softmax", normalize: bool = True, scale: float = 1.0, balance: float = 0.0, stream=None):
    """Top-k experts of every token: logits bf16 or float32 [S, E], or [B, S, E] of B sequences -> (topk_ids int32
    [.., S, k], topk_weights float32 [.., S, k], counts int32 [.., E], loss float32 [1], slope float32
    [.., E]).  Chosen by score + bias (float32 [E]); weights scale * score, normalized over the chosen ones;
    loss = balance * the mean over the sequences of E sum_e (share of the slots)_e (mean of p_e), slope its
    derivative by each p.  Tokens with valid (bool [.., S]) False, or whose experts all have logit or bias -inf, get ids -1
    and weights 0 and do not count."""
    if stream is not None:
        with _on(stream):
            return fp8q_moe_route(logits, k, bias, valid, score, normalize, scale, balance)
    B, S, E = _logits_shape(logits)
    lead = logits.shape[:-1]
    if bias is not None:
        _need(bias, torch.float32, "bias", (E,))
    if valid is not None:
        _need(valid, torch.bool, "valid", lead)
    code = _score_code(score)
    s = _here(logits, bias, valid)
    lib = load_library()
    work = _workspace(lib.fp8q_moe_route_workspace(B, S, E), logits)
    if not 1 <= k <= min(E, 64):
        raise ValueError(f"k must be between 1 and min(E, 64), got {k}")
    ids = logits.new_empty(*lead, k, dtype=torch.int32)
    w = logits.new_empty(*lead, k, dtype=torch.float32)
    counts = logits.new_empty(*lead[:-1], E, dtype=torch.int32)
    slope = logits.new_empty(*lead[:-1], E, dtype=torch.float32)
    loss = logits.new_empty(1, dtype=torch.float32)
    _check(lib.fp8q_moe_route(_ptr(logits), _out_code(logits.dtype), B, S, E, k, _ptr(bias), _ptr(valid), code,
                              bool(normalize), scale, balance, _ptr(ids), _ptr(w), _ptr(counts), _ptr(loss), _ptr(slope),
                              _ptr(work), s), "fp8q_moe_route")
    return ids, w, counts, loss, slope


def fp8q_moe_route_backward(logits: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor, dw: torch.Tensor,
                            slope: torch.Tensor, dloss: torch.Tensor | None = None, score: str = "softmax",
                            normalize: bool = True, scale: float = 1.0, out_dtype=None,
                            dlogits: torch.Tensor | None = None, stream=None):
    """Gradient of fp8q_moe_route by the logits, from dw float32 like topk_w and dloss float32 [1] (None: 1);
    topk_ids, topk_w and slope as fp8q_moe_route gave them, score, normalize and scale as it got them ->
    dlogits like logits, in out_dtype (logits' by default).  Zeros for tokens with ids -1."""
    if stream is not None:
        with _on(stream):
            return fp8q_moe_route_backward(logits, topk_ids, topk_w, dw, slope, dloss, score, normalize, scale, out_dtype,
                                           dlogits)
    B, S, E = _logits_shape(logits)
    lead = logits.shape[:-1]
    if not isinstance(topk_ids, torch.Tensor) or topk_ids.dim() != logits.dim():
        raise ValueError("topk_ids must be [.., S, k] like the logits")
    k = topk_ids.shape[-1]
    _need(topk_ids, torch.int32, "topk_ids", (*lead, k))
    _need(topk_w, torch.float32, "topk_w", (*lead, k))
    _need(dw, torch.float32, "dw", (*lead, k))
    _need(slope, torch.float32, "slope", (*lead[:-1], E))
    if dloss is not None:
        _need(dloss, torch.float32, "dloss")
        if dloss.numel() != 1:
            raise ValueError("dloss must hold one float32")
    code = _score_code(score)
    s = _here(logits, topk_ids, topk_w, dw, slope, dloss, dlogits)
    dlogits = _out(dlogits, (out_dtype or logits.dtype) if dlogits is None else dlogits.dtype, "dlogits", logits.shape,
                   logits)
    _check(load_library().fp8q_moe_route_backward(
        _ptr(logits), _out_code(logits.dtype), B, S, E, k, _ptr(topk_ids), _ptr(topk_w), _ptr(dw), _ptr(slope),
        _ptr(dloss), code, bool(normalize), scale, _ptr(dlogits), _out_code(dlogits.dtype), s), "fp8q_moe_route_backward")
    return dlogits


def _need_matrices(t, name: str):
    """A contiguous bf16 or float32 [P, Q] or [G, P, Q]; returns (G, P, Q)."""
    if not isinstance(t, torch.Tensor) or (t.dtype != torch.bfloat16 and t.dtype != torch.float32):
        raise ValueError(f"{name} must be a bfloat16 or float32 tensor")
    if not t.is_cuda or not t.is_contiguous() or t.dim() not in (2, 3):
        raise ValueError(f"{name} must be a contiguous CUDA tensor [P, Q] or [G, P, Q]")
    return (1, *t.shape) if t.dim() == 2 else tuple(t.shape)


NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)  # a + b s^2 + c s^4 takes singular values from 0.002 to 1 near one in five steps


def fp8q_orthogonalize(x: torch.Tensor, steps: int = 5, coefficients=NEWTON_SCHULZ, out: torch.Tensor | None = None,
                       stream=None):
    """The matrices x (bf16 or float32 [P, Q] or [G, P, Q]) with their singular values brought near one, as bf16
    like x: `steps` times X = (a I + b X X^T + c (X X^T)^2) X, from X = x / |x|_F.  FP16 products: off by up to 1e-3
    of the norm with both sides of 128 and more, by more with smaller ones (include/fp8q.h)."""
    if stream is not None:
        with _on(stream):
            return fp8q_orthogonalize(x, steps, coefficients, out)
    G, P, Q = _need_matrices(x, "x")
    s = _here(x, out)
    if G == 0:
        return _out(out, torch.bfloat16, "out", x.shape, x)
    lib = load_library()
    out = _out(out, torch.bfloat16, "out", x.shape, x)
    work = _workspace(lib.fp8q_muon_workspace(G, P, Q), x)
    ns = _NewtonSchulz(*coefficients, steps)
    _check(lib.fp8q_orthogonalize(_ptr(x), _out_code(x.dtype), G, P, Q, ctypes.byref(ns), _ptr(out), _ptr(work), s),
           "fp8q_orthogonalize")
    return out


def fp8q_muon(param: torch.Tensor, grad: torch.Tensor, momentum: torch.Tensor, lr: float, beta: float = 0.95,
              nesterov: bool = True, weight_decay: float = 0.0, scale: float | None = None, steps: int = 5,
              coefficients=NEWTON_SCHULZ, grad_scale: float = 1.0, copy: torch.Tensor | None = None,
              device_lr: torch.Tensor | None = None, stream=None) -> None:
    """One Muon step in place on a matrix [P, Q] or on G of them [G, P, Q]: param and momentum float32, grad bf16 or
    float32.  param = param (1 - lr weight_decay) - lr scale O with O the momentum (Nesterov's, by default) made
    orthogonal as by fp8q_orthogonalize; scale defaults to 0.2 sqrt(max(P, Q)).  copy: bf16, written with the new
    parameters.  device_lr: a device float32 [1] read by the kernels in place of lr."""
    if stream is not None:
        with _on(stream):
            return fp8q_muon(param, grad, momentum, lr, beta, nesterov, weight_decay, scale, steps, coefficients,
                             grad_scale, copy, device_lr)
    G, P, Q = _need_matrices(grad, "grad")
    _need(param, torch.float32, "param", grad.shape)
    _need(momentum, torch.float32, "momentum", grad.shape)
    if copy is not None:
        _need(copy, torch.bfloat16, "copy", grad.shape)
    if device_lr is not None:
        _need(device_lr, torch.float32, "device_lr", (1,))
    s = _here(param, grad, momentum, copy, device_lr)
    if G == 0:
        return
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in (param, grad, momentum, copy)
                   if t is not None)
    if any(b[0] < a[1] for a, b in zip(spans, spans[1:])):
        raise ValueError("param, grad, momentum and copy must not share memory")
    lib = load_library()
    work = _workspace(lib.fp8q_muon_workspace(G, P, Q), grad)
    hyper = _MuonHyper(lr, beta, weight_decay, 0.2 * max(P, Q) ** 0.5 if scale is None else scale, grad_scale,
                       _NewtonSchulz(*coefficients, steps), bool(nesterov), _ptr(device_lr) or None)
    _check(lib.fp8q_muon(_ptr(param), _ptr(grad), _out_code(grad.dtype), _ptr(momentum), G, P, Q, ctypes.byref(hyper),
                         _ptr(copy), _ptr(work), s), "fp8q_muon")


quantize_act_1x128 = fp8q_quantize_act_1x128
quantize_w_128x128 = fp8q_quantize_w_128x128
gemm_blockscaled = fp8q_gemm_blockscaled
grouped_gemm_blockscaled = fp8q_grouped_gemm_blockscaled
quantize_w_128x128_t = fp8q_quantize_w_128x128_t
quantize_act_dual = fp8q_quantize_act_dual
gemm_rowscaled = fp8q_gemm_rowscaled
swiglu_quantize_act_1x128 = fp8q_swiglu_quantize_act_1x128
quantize_per_tensor = fp8q_quantize_per_tensor
moe_sort = fp8q_moe_sort
moe_sort_backward = fp8q_moe_sort_backward
moe_combine_backward = fp8q_moe_combine_backward
swiglu_backward = fp8q_swiglu_backward
quantize_act_grouped = fp8q_quantize_act_grouped
grouped_gemm_rowscaled = fp8q_grouped_gemm_rowscaled
adamw_plan = fp8q_adamw_plan
adamw = fp8q_adamw
layer_norm = fp8q_layer_norm
layer_norm_backward = fp8q_layer_norm_backward
moe_route = fp8q_moe_route
moe_route_backward = fp8q_moe_route_backward
orthogonalize = fp8q_orthogonalize
muon = fp8q_muon
