"""Python binding of libconvrot (ctypes).  Argument marshalling only: every step of the ConvRot
linear runs in the library's HIP kernels; torch provides device memory and the current stream.

Raises ``ConvRotError`` when the library rejects a call and ``ImportError``-style
``RuntimeError`` when the built library is missing -- there is no fallback path.

Returned tensors carry no autograd history.  The fused linears' gradients are calls of their own
(``linear_act_backward`` and so on); a training loop pairs the two in a ``torch.autograd.Function``.
"""
from __future__ import annotations

import ctypes
import os
import threading
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libconvrot.so")

CONVROT_DTYPE_F32, CONVROT_DTYPE_BF16 = 0, 1
STATUS = {0: "CONVROT_OK", 1: "CONVROT_ERR_NULL", 2: "CONVROT_ERR_SHAPE", 3: "CONVROT_ERR_GROUP",
          4: "CONVROT_ERR_ALIGN", 5: "CONVROT_ERR_DTYPE", 6: "CONVROT_ERR_BITS", 7: "CONVROT_ERR_WORKSPACE",
          8: "CONVROT_ERR_HIP", 9: "CONVROT_ERR_DEVICE", 10: "CONVROT_ERR_ACT", 11: "CONVROT_ERR_OVERLAP",
          12: "CONVROT_ERR_SCORE"}
SCORES = {"softmax": 0, "sigmoid": 1}
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

# name -> (argtypes, restype); mirrors include/convrot.h
P, I64, I, SZ, F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
SIGNATURES = {
    "convrot_prepare_weight": ([P, I, I64, I64, I, I, P, P, P], I),
    "convrot_quantize_act": ([P, I, I64, I64, I, I, P, P, P], I),
    "convrot_workspace_bytes": ([I64, I64, I64, I], SZ),
    "convrot_linear": ([P, I, P, P, I64, I64, I64, I, P, P, P, P, P, SZ, P], I),
    "convrot_linear_act": ([P, I, P, P, I64, I64, I64, I, P, P, P, I, P, P, P, P, SZ, P], I),
    "convrot_linear_gated": ([P, I, P, P, I64, I64, I64, I, P, P, P, P, P, P, I, P, P, P, SZ, P], I),
    "convrot_workspace_bytes_act": ([I64, I64, I64], SZ),
    "convrot_workspace_bytes_gated": ([I64, I64, I64], SZ),
    "convrot_ffn_gated": ([P, I, I64, I64, I64, I, I, P, P, P, P, P, P, P, P, P, I, P, P, P, P, SZ, P], I),
    "convrot_workspace_bytes_ffn": ([I64, I64, I64], SZ),
    "convrot_linear_act_backward": ([P, P, I64, I64, I64, I, P, P, I, P, P, P, P, SZ, P], I),
    "convrot_linear_gated_backward": ([P, P, I64, I64, I64, I, P, P, P, P, I, P, P, P, P, P, SZ, P], I),
    "convrot_ffn_gated_backward": ([P, P, I64, I64, I64, I, I, P, P, P, P, P, P, I, P, P, P, P, P, P, SZ, P], I),
    "convrot_workspace_bytes_backward": ([I64, I64, I64], SZ),
    "convrot_workspace_bytes_gated_backward": ([I64, I64, I64], SZ),
    "convrot_workspace_bytes_ffn_backward": ([I64, I64, I64], SZ),
    "convrot_linear_noalloc": ([P, I, P, P, I64, I64, I64, I, P, P, P, P, P], I),
    "convrot_linear_w4a4": ([P, I, P, P, I64, I64, I64, I, P, P, P, P, P, SZ, P], I),
    "convrot_pack_weight_w4a4": ([P, I64, I64, P, P], I),
    "convrot_packed_bytes_w4a4": ([I64, I64], SZ),
    "convrot_linear_w4a4_packed": ([P, I, P, P, I64, I64, I64, I, P, P, P, P, P, SZ, P], I),
    "convrot_linear_w4a8": ([P, I, P, P, I64, I64, I64, I, P, SZ, P, P, P, SZ, P], I),
    "convrot_pack_weight_w4a8": ([P, P, I64, I64, P, P], I),
    "convrot_packed_bytes_w4a8": ([I64, I64], SZ),
    "convrot_pack_weight_w4a8_group": ([P, P, I64, I64, I, P, P], I),
    "convrot_packed_bytes_w4a8_group": ([I64, I64, I], SZ),
    "convrot_workspace_bytes_w4a8": ([I64, I64, I64], SZ),
    "convrot_gemm_i8_i32": ([P, P, I64, I64, I64, P, P, SZ, P], I),
    "convrot_gemm_i4_i32": ([P, P, I64, I64, I64, P, P, SZ, P], I),
    "convrot_moe_route": ([P, I, I64, I64, I, I, I, F32, P, P, P, P], I),
    "convrot_moe_route_backward": ([P, P, I, I64, I64, I, I, I, F32, P, P, P], I),
    "convrot_linear_grouped": ([P, I, P, P, I64, I64, I64, I, P, I64, P, P, P, P, SZ, P], I),
    "convrot_workspace_bytes_grouped": ([I64, I64, I64, I64], SZ),
    "convrot_linear_grouped_backward": ([P, I64, I64, I64, I, P, I64, P, P, P, P, P, SZ, P], I),
    "convrot_workspace_bytes_grouped_backward": ([I64, I64, I64, I64], SZ),
    "convrot_moe_ffn_gated": ([P, I, P, P, I64, I, I64, I64, I64, I, I, P, P, P, P, P, P, I, P, P, P, P, P, SZ, P], I),
    "convrot_workspace_bytes_moe_ffn": ([I64, I, I64, I64, I64], SZ),
    "convrot_moe_ffn_gated_backward": ([P, P, P, P, P, I64, I, I64, I64, I64, I, I, P, P, P, P, P, P, I, P, P, P, P, SZ,
                                        P], I),
    "convrot_workspace_bytes_moe_ffn_backward": ([I64, I, I64, I64, I64], SZ),
    "convrot_dynamic_group": ([I64, I], I),
    "convrot_last_error": ([], ctypes.c_char_p),
    "convrot_status_string": ([I], ctypes.c_char_p),
}

_lock = threading.Lock()
_lib = None


class ConvRotError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


def load() -> ctypes.CDLL:
    """Load the in-tree libconvrot.so (built by ``python -m int4_quantized_linear_amd.build``)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError("libconvrot.so is not built (%s); run python -m int4_quantized_linear_amd.build"
                                   % LIB_PATH)
            lib = ctypes.CDLL(LIB_PATH)
            for name, (args, res) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.argtypes = args
                fn.restype = res
            _lib = lib
        return _lib


def _call(name: str, *args) -> int:
    lib = load()
    rc = getattr(lib, name)(*args)
    if rc != 0:
        raise ConvRotError(rc, lib.convrot_last_error().decode() or STATUS.get(rc, str(rc)))
    return rc


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _stream(dev: torch.device):
    return torch.cuda.current_stream(dev).cuda_stream


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return CONVROT_DTYPE_BF16
    if t.dtype == torch.float32:
        return CONVROT_DTYPE_F32
    raise TypeError("ConvRot inputs are bf16 or fp32, got %s" % t.dtype)


def _check_dev(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("ConvRot tensors must be on a GPU device")
            if not t.is_contiguous():
                raise ValueError("ConvRot tensors must be contiguous")


def dynamic_group(K: int, max_group: int = 256) -> int:
    """Largest power-of-two rotation group <= max_group dividing K (dynamic ConvRot mode)."""
    g = int(load().convrot_dynamic_group(K, max_group))
    if g == 0:
        raise ConvRotError(3, "CONVROT_ERR_GROUP: invalid K=%d or max_group=%d" % (K, max_group))
    return g


def workspace_bytes(M: int, N: int, K: int, bits: int = 8) -> int:
    return int(load().convrot_workspace_bytes(M, N, K, bits))


def _workspace(M: int, N: int, K: int, bits: int, dev: torch.device) -> torch.Tensor:
    return torch.empty(max(workspace_bytes(M, N, K, bits), 256), dtype=torch.uint8, device=dev)


def _quant(name: str, v: torch.Tensor, group: int, bits: int):
    _check_dev(v)
    R, K = v.shape
    if bits == 8:
        q = torch.empty((R, K), dtype=torch.int8, device=v.device)
        s = torch.empty((R,), dtype=torch.float32, device=v.device)
    else:
        q = torch.empty((R, K // 2), dtype=torch.uint8, device=v.device)
        # one fp16 scale per (group, row); an invalid group is rejected by the library before any write
        ngroups = K // group if group > 0 and K % group == 0 else 1
        s = torch.empty((ngroups, R), dtype=torch.float16, device=v.device)
    _call(name, _ptr(v), _dtype_code(v), R, K, group, bits, _ptr(q), _ptr(s), _stream(v.device))
    return q, s


def prepare_weight(w: torch.Tensor, group: int = 256, bits: int = 8):
    """Rotate + quantize a weight [N, K] -> (wq, w_scale).  bits 8: int8 [N,K], fp32 [N];
    bits 4: uint8 [N,K/2] packed, fp16 [K/group, N] (group 256 or 128)."""
    return _quant("convrot_prepare_weight", w, group, bits)


def quantize_act(x: torch.Tensor, group: int = 256, bits: int = 8):
    """Rotate + quantize activations [M, K] per token -> (xq, x_scale) (layouts as prepare_weight)."""
    return _quant("convrot_quantize_act", x, group, bits)


def linear(x: torch.Tensor | None, wq: torch.Tensor, w_scale: torch.Tensor, bias: torch.Tensor | None = None,
           group: int = 256, xq: torch.Tensor | None = None, x_scale: torch.Tensor | None = None,
           out: torch.Tensor | None = None, split_k: bool = True) -> torch.Tensor:
    """INT8 ConvRot linear: y = bf16((q(xR) . q(wR)^T) * sx * sw + bias).  Pass x (bf16/fp32 [M,K])
    or a pre-quantized (xq, x_scale) pair.  The workspace passed has room for the GEMM's split-K
    tail; split_k=False (pre-quantized x only) passes none, so the GEMM runs without it."""
    _check_dev(x, wq, w_scale, bias, xq, x_scale, out)
    N, K = wq.shape
    M = x.shape[0] if x is not None else xq.shape[0]
    dev = wq.device
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    if split_k:
        ws = _workspace(M, N, K, 8, dev)
    elif x is None:
        ws = None
    else:
        raise ValueError("split_k=False needs a pre-quantized (xq, x_scale) pair")
    _call("convrot_linear", _ptr(x), _dtype_code(x) if x is not None else 0, _ptr(xq), _ptr(x_scale), M, N, K, group,
          _ptr(wq), _ptr(w_scale), _ptr(bias), _ptr(y), _ptr(ws), ws.numel() if ws is not None else 0, _stream(dev))
    return y


def workspace_bytes_act(M: int, N: int, K: int) -> int:
    return int(load().convrot_workspace_bytes_act(M, N, K))


def _act_code(act: str) -> int:
    if act not in ACTS:
        raise ValueError("act is one of %s, got %r" % (", ".join(ACTS), act))
    return ACTS[act]


def _check(dev: torch.device, **tensors):
    """name=(tensor or None, shape, dtype or tuple of dtypes): contiguous, on dev, of that shape and type."""
    for name, (t, shape, dtype) in tensors.items():
        if t is None:
            continue
        if t.device != dev or not t.is_cuda:
            raise ValueError("%s is on %s; the call runs on the weights' GPU, %s" % (name, t.device, dev))
        if t.shape != shape:
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
        if t.dtype is not dtype and not (type(dtype) is tuple and t.dtype in dtype):
            raise TypeError("%s is %s, expected %s" % (name, t.dtype, dtype))
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)


def _call_on(dev: torch.device, name: str, *args):
    """_call with the tensors' device current (the library launches on the current device), on its
    current torch stream, which is appended as the last argument.  (The raw stream query: building a
    torch.cuda.Stream for its handle takes 4 us, a quarter of a small call's host time.)"""
    if torch.cuda.current_device() == dev.index:
        return _call(name, *args, torch._C._cuda_getCurrentRawStream(dev.index))
    with torch.cuda.device(dev):
        return _call(name, *args, torch._C._cuda_getCurrentRawStream(dev.index))


_X_DTYPES = (torch.bfloat16, torch.float32)


def _tokens(x, xq, x_scale, K: int, dev: torch.device) -> int:
    """Checks x, or the pre-quantized pair, and returns the token count."""
    if x is None and (xq is None or x_scale is None):
        raise ValueError("give x, or both xq and x_scale")
    M = x.shape[0] if x is not None else xq.shape[0]
    if x is not None:
        _check(dev, x=(x, (M, K), _X_DTYPES))
    else:
        _check(dev, xq=(xq, (M, K), torch.int8), x_scale=(x_scale, (M,), torch.float32))
    return M


def _no_history(name: str, *inputs: torch.Tensor | None):
    """Warns where autograd would take the result for a constant: inputs that require a gradient, outside
    torch.no_grad() and torch.autograd.Function (which turns recording off in its forward)."""
    for t in inputs:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            warnings.warn("%s returns a tensor without autograd history, so no gradient reaches its inputs; pair it with "
                          "%s_backward in a torch.autograd.Function, or call it under torch.no_grad()" % (name, name),
                          stacklevel=3)
            return


def linear_act(x: torch.Tensor | None, wq: torch.Tensor, w_scale: torch.Tensor, bias: torch.Tensor | None = None,
               act: str = "none", residual: torch.Tensor | None = None, group: int = 256,
               xq: torch.Tensor | None = None, x_scale: torch.Tensor | None = None, out: torch.Tensor | None = None,
               save_pre: bool = False):
    """INT8 ConvRot linear with its activation and residual in the epilogue:
    z = (q(xR) . q(wR)^T) * sx * sw + bias,  y = bf16(act(z) + residual).  x (or xq, x_scale) and the
    weight as in linear(); act one of ACTS; residual bf16 [M, N], may be ``out`` (added in place).
    save_pre=True returns (y, pre) with pre = bf16(z) [M, N] for linear_act_backward; the result itself has no
    autograd history."""
    _no_history("linear_act", x, bias, residual)
    code = _act_code(act)
    N, K = wq.shape
    dev = wq.device
    M = _tokens(x, xq, x_scale, K, dev)
    _check(dev, wq=(wq, (N, K), torch.int8), w_scale=(w_scale, (N,), torch.float32), bias=(bias, (N,), torch.float32),
           residual=(residual, (M, N), torch.bfloat16), out=(out, (M, N), torch.bfloat16))
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    pre = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if save_pre else None
    ws = torch.empty(max(workspace_bytes_act(M, N, K), 256), dtype=torch.uint8, device=dev)
    _call_on(dev, "convrot_linear_act", _ptr(x), _dtype_code(x) if x is not None else 0, _ptr(xq), _ptr(x_scale), M, N,
             K, group, _ptr(wq), _ptr(w_scale), _ptr(bias), code, _ptr(residual), _ptr(pre), _ptr(y), _ptr(ws),
             ws.numel())
    return (y, pre) if save_pre else y


def workspace_bytes_gated(M: int, N: int, K: int) -> int:
    return int(load().convrot_workspace_bytes_gated(M, N, K))


def linear_gated(x: torch.Tensor | None, wq_gate: torch.Tensor, gate_scale: torch.Tensor, wq_up: torch.Tensor,
                 up_scale: torch.Tensor, bias_gate: torch.Tensor | None = None, bias_up: torch.Tensor | None = None,
                 act: str = "silu", group: int = 256, xq: torch.Tensor | None = None,
                 x_scale: torch.Tensor | None = None, out: torch.Tensor | None = None, save_pre: bool = False):
    """Gate and up projections of one input, the activation and the product in one kernel:
    h = bf16(act(g) * u) with g and u the INT8 ConvRot linears of x.  save_pre=True returns (h, pre)
    with pre = bf16 [2, M, N], g then u, for linear_gated_backward; the result itself has no autograd history."""
    _no_history("linear_gated", x, bias_gate, bias_up)
    code = _act_code(act)
    N, K = wq_gate.shape
    dev = wq_gate.device
    M = _tokens(x, xq, x_scale, K, dev)
    f32 = torch.float32
    _check(dev, wq_gate=(wq_gate, (N, K), torch.int8), gate_scale=(gate_scale, (N,), f32),
           wq_up=(wq_up, (N, K), torch.int8), up_scale=(up_scale, (N,), f32), bias_gate=(bias_gate, (N,), f32),
           bias_up=(bias_up, (N,), f32), out=(out, (M, N), torch.bfloat16))
    h = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    pre = torch.empty((2, M, N), dtype=torch.bfloat16, device=dev) if save_pre else None
    ws = torch.empty(max(workspace_bytes_gated(M, N, K), 256), dtype=torch.uint8, device=dev)
    _call_on(dev, "convrot_linear_gated", _ptr(x), _dtype_code(x) if x is not None else 0, _ptr(xq), _ptr(x_scale), M,
             N, K, group, _ptr(wq_gate), _ptr(gate_scale), _ptr(bias_gate), _ptr(wq_up), _ptr(up_scale), _ptr(bias_up),
             code, _ptr(pre), _ptr(h), _ptr(ws), ws.numel())
    return (h, pre) if save_pre else h


def workspace_bytes_ffn(M: int, F: int, K: int) -> int:
    return int(load().convrot_workspace_bytes_ffn(M, F, K))


def ffn_gated(x: torch.Tensor, wq_gate: torch.Tensor, gate_scale: torch.Tensor, wq_up: torch.Tensor,
              up_scale: torch.Tensor, wq_down: torch.Tensor, down_scale: torch.Tensor,
              bias_gate: torch.Tensor | None = None, bias_up: torch.Tensor | None = None,
              bias_down: torch.Tensor | None = None, act: str = "silu", residual: torch.Tensor | None = None,
              group: int = 256, group_h: int = 256, out: torch.Tensor | None = None, save_pre: bool = False):
    """Gated feed-forward block on INT8 ConvRot weights: h = bf16(act(g) * u) as in linear_gated
    (gate, up [F, K], prepared with ``group``), then y = bf16(linear(h) + bias_down + residual) (down
    [K, F], prepared with ``group_h``).  residual bf16 [M, K], may be ``out``.  save_pre=True returns
    (y, pre) with pre = bf16 [2, M, F], g then u, for ffn_gated_backward; the result itself has no autograd
    history."""
    _no_history("ffn_gated", x, bias_gate, bias_up, bias_down, residual)
    code = _act_code(act)
    F, K = wq_gate.shape
    dev = wq_gate.device
    M = _tokens(x, None, None, K, dev)
    f32 = torch.float32
    _check(dev, wq_gate=(wq_gate, (F, K), torch.int8), gate_scale=(gate_scale, (F,), f32),
           wq_up=(wq_up, (F, K), torch.int8), up_scale=(up_scale, (F,), f32),
           wq_down=(wq_down, (K, F), torch.int8), down_scale=(down_scale, (K,), f32), bias_gate=(bias_gate, (F,), f32),
           bias_up=(bias_up, (F,), f32), bias_down=(bias_down, (K,), f32), residual=(residual, (M, K), torch.bfloat16),
           out=(out, (M, K), torch.bfloat16))
    y = out if out is not None else torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    pre = torch.empty((2, M, F), dtype=torch.bfloat16, device=dev) if save_pre else None
    ws = torch.empty(max(workspace_bytes_ffn(M, F, K), 256), dtype=torch.uint8, device=dev)
    _call_on(dev, "convrot_ffn_gated", _ptr(x), _dtype_code(x), M, F, K, group, group_h, _ptr(wq_gate),
             _ptr(gate_scale), _ptr(bias_gate), _ptr(wq_up), _ptr(up_scale), _ptr(bias_up), _ptr(wq_down),
             _ptr(down_scale), _ptr(bias_down), code, _ptr(residual), _ptr(pre), _ptr(y), _ptr(ws), ws.numel())
    return (y, pre) if save_pre else y


def workspace_bytes_backward(M: int, N: int, K: int) -> int:
    return int(load().convrot_workspace_bytes_backward(M, N, K))


def workspace_bytes_gated_backward(M: int, N: int, K: int) -> int:
    return int(load().convrot_workspace_bytes_gated_backward(M, N, K))


def workspace_bytes_ffn_backward(M: int, F: int, K: int) -> int:
    return int(load().convrot_workspace_bytes_ffn_backward(M, F, K))


def _backward_buffers(M: int, K: int, ws_bytes: int, out: torch.Tensor | None, dev: torch.device):
    dx = out if out is not None else torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    return dx, torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)


def linear_act_backward(dy: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor, pre: torch.Tensor | None = None,
                        act: str = "none", group: int = 256, bias_grad: bool = False,
                        dx_add: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """Input gradient of linear_act (or linear) through its frozen weight, the token quantizer taken as
    the identity: dz = dy * act'(pre), dx = bf16((sum_n bf16(dz * sw) wq) R + dx_add).  dy bf16 [M, N];
    pre as the forward saved it (not needed for act "none"); dx_add bf16 [M, K], may be ``out``.
    Returns (dx, dbias), dbias fp32 [N] with bias_grad=True, else None."""
    code = _act_code(act)
    N, K = wq.shape
    M = dy.shape[0]
    dev, bf16 = wq.device, torch.bfloat16
    _check(dev, dy=(dy, (M, N), bf16), wq=(wq, (N, K), torch.int8), w_scale=(w_scale, (N,), torch.float32),
           pre=(pre, (M, N), bf16), dx_add=(dx_add, (M, K), bf16), out=(out, (M, K), bf16))
    dx, ws = _backward_buffers(M, K, workspace_bytes_backward(M, N, K), out, dev)
    db = torch.empty((N,), dtype=torch.float32, device=dev) if bias_grad else None
    _call_on(dev, "convrot_linear_act_backward", _ptr(dy), _ptr(pre), M, N, K, group, _ptr(wq), _ptr(w_scale), code,
             _ptr(dx_add), _ptr(dx), _ptr(db), _ptr(ws), ws.numel())
    return dx, db


def linear_gated_backward(dh: torch.Tensor, pre: torch.Tensor, wq_gate: torch.Tensor, gate_scale: torch.Tensor,
                          wq_up: torch.Tensor, up_scale: torch.Tensor, act: str = "silu", group: int = 256,
                          bias_grad: bool = False, dx_add: torch.Tensor | None = None,
                          out: torch.Tensor | None = None):
    """Input gradient of linear_gated through both frozen weights: dg = dh * u * act'(g), du = dh * act(g),
    dx = bf16((dg Wg + du Wu) R + dx_add).  pre bf16 [2, M, N] as the forward saved it.  Returns dx, or
    (dx, dbias_gate, dbias_up) with bias_grad=True."""
    code = _act_code(act)
    N, K = wq_gate.shape
    M = dh.shape[0]
    dev, bf16, f32 = wq_gate.device, torch.bfloat16, torch.float32
    _check(dev, dh=(dh, (M, N), bf16), pre=(pre, (2, M, N), bf16), wq_gate=(wq_gate, (N, K), torch.int8),
           gate_scale=(gate_scale, (N,), f32), wq_up=(wq_up, (N, K), torch.int8), up_scale=(up_scale, (N,), f32),
           dx_add=(dx_add, (M, K), bf16), out=(out, (M, K), bf16))
    dx, ws = _backward_buffers(M, K, workspace_bytes_gated_backward(M, N, K), out, dev)
    db = [torch.empty((N,), dtype=f32, device=dev) if bias_grad else None for _ in range(2)]
    _call_on(dev, "convrot_linear_gated_backward", _ptr(dh), _ptr(pre), M, N, K, group, _ptr(wq_gate),
             _ptr(gate_scale), _ptr(wq_up), _ptr(up_scale), code, _ptr(dx_add), _ptr(dx), _ptr(db[0]), _ptr(db[1]),
             _ptr(ws), ws.numel())
    return (dx, *db) if bias_grad else dx


def ffn_gated_backward(dy: torch.Tensor, pre: torch.Tensor, wq_gate: torch.Tensor, gate_scale: torch.Tensor,
                       wq_up: torch.Tensor, up_scale: torch.Tensor, wq_down: torch.Tensor, down_scale: torch.Tensor,
                       act: str = "silu", group: int = 256, group_h: int = 256, bias_grad: bool = False,
                       dx_add: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """Input gradient of ffn_gated: dy bf16 [M, K] through down (rounded to bf16, h's type), the product,
    gate and up.  pre bf16 [2, M, F] as the forward saved it; dx_add = dy where the residual was x.
    Returns dx, or (dx, dbias_gate, dbias_up, dbias_down) with bias_grad=True."""
    code = _act_code(act)
    F, K = wq_gate.shape
    M = dy.shape[0]
    dev, bf16, f32, i8 = wq_gate.device, torch.bfloat16, torch.float32, torch.int8
    _check(dev, dy=(dy, (M, K), bf16), pre=(pre, (2, M, F), bf16), wq_gate=(wq_gate, (F, K), i8),
           gate_scale=(gate_scale, (F,), f32), wq_up=(wq_up, (F, K), i8), up_scale=(up_scale, (F,), f32),
           wq_down=(wq_down, (K, F), i8), down_scale=(down_scale, (K,), f32), dx_add=(dx_add, (M, K), bf16),
           out=(out, (M, K), bf16))
    dx, ws = _backward_buffers(M, K, workspace_bytes_ffn_backward(M, F, K), out, dev)
    db = [torch.empty((n,), dtype=f32, device=dev) if bias_grad else None for n in (F, F, K)]
    _call_on(dev, "convrot_ffn_gated_backward", _ptr(dy), _ptr(pre), M, F, K, group, group_h, _ptr(wq_gate),
             _ptr(gate_scale), _ptr(wq_up), _ptr(up_scale), _ptr(wq_down), _ptr(down_scale), code, _ptr(dx_add),
             _ptr(dx), _ptr(db[0]), _ptr(db[1]), _ptr(db[2]), _ptr(ws), ws.numel())
    return (dx, *db) if bias_grad else dx


def _score_code(score: str) -> int:
    if score not in SCORES:
        raise ValueError("score is one of %s, got %r" % (", ".join(SCORES), score))
    return SCORES[score]


def moe_route(logits: torch.Tensor, top: int, bias: torch.Tensor | None = None, score: str = "softmax",
              normalize: bool = True, scale: float = 1.0):
    """Router of a mixture of experts: logits [M, E] fp32 or bf16 -> (experts int32 [M, top], weights fp32
    [M, top]).  The experts are the top scores' (s = softmax or sigmoid of the logits; with bias fp32 [E] those of s +
    bias), in falling order, ties to the lowest index; the weights scale * s, divided by the chosen ones' sum with
    normalize.  A logit of -inf masks its expert; slots that find none get expert -1 and weight 0.  A NaN logit, or +inf
    under a softmax, makes its row's weights NaN, a NaN in the bias every row's.  The weights have no autograd history:
    moe_route_backward."""
    _no_history("moe_route", logits)
    code = _score_code(score)
    M, E = logits.shape
    dev = logits.device
    _check(dev, logits=(logits, (M, E), _X_DTYPES), bias=(bias, (E,), torch.float32))
    experts = torch.empty((M, top), dtype=torch.int32, device=dev)
    weights = torch.empty((M, top), dtype=torch.float32, device=dev)
    _call_on(dev, "convrot_moe_route", _ptr(logits), _dtype_code(logits), M, E, top, code, int(normalize), scale, _ptr(bias),
             _ptr(experts), _ptr(weights))
    return experts, weights


def moe_route_backward(dweights: torch.Tensor, logits: torch.Tensor, experts: torch.Tensor, score: str = "softmax",
                       normalize: bool = True, scale: float = 1.0, out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of moe_route's logits (in their type) from that of its weights, dweights fp32 [M, top], the chosen
    experts held fixed.  out may be logits itself."""
    code = _score_code(score)
    M, E = logits.shape
    top = experts.shape[1]
    dev = logits.device
    _check(dev, logits=(logits, (M, E), _X_DTYPES), dweights=(dweights, (M, top), torch.float32),
           experts=(experts, (M, top), torch.int32), out=(out, (M, E), logits.dtype))
    dlogits = out if out is not None else torch.empty_like(logits)
    _call_on(dev, "convrot_moe_route_backward", _ptr(dweights), _ptr(logits), _dtype_code(logits), M, E, top, code,
             int(normalize), scale, _ptr(experts), _ptr(dlogits))
    return dlogits


def workspace_bytes_grouped(rows: int, groups: int, N: int, K: int) -> int:
    return int(load().convrot_workspace_bytes_grouped(rows, groups, N, K))


def linear_grouped(x: torch.Tensor | None, wq: torch.Tensor, w_scale: torch.Tensor, offsets: torch.Tensor,
                   group: int = 256, xq: torch.Tensor | None = None, x_scale: torch.Tensor | None = None,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """INT8 ConvRot linear of rows sorted by group, each group through its own weight: y[r] = linear(x[r]) with
    wq[e] for offsets[e] <= r < offsets[e + 1].  x (or xq, x_scale) [rows, K] as in linear(); wq int8 [groups, N, K],
    w_scale fp32 [groups, N]; offsets int32 [groups + 1] on the GPU (the host never reads them).  Rows of no group
    are not written: pass ``out`` where they matter."""
    _no_history("linear_grouped", x)
    groups, N, K = wq.shape
    dev = wq.device
    rows = _tokens(x, xq, x_scale, K, dev)
    _check(dev, wq=(wq, (groups, N, K), torch.int8), w_scale=(w_scale, (groups, N), torch.float32),
           offsets=(offsets, (groups + 1,), torch.int32), out=(out, (rows, N), torch.bfloat16))
    y = out if out is not None else torch.empty((rows, N), dtype=torch.bfloat16, device=dev)
    ws = torch.empty(max(workspace_bytes_grouped(rows, groups, N, K), 256), dtype=torch.uint8, device=dev)
    _call_on(dev, "convrot_linear_grouped", _ptr(x), _dtype_code(x) if x is not None else 0, _ptr(xq), _ptr(x_scale), rows,
             N, K, group, _ptr(offsets), groups, _ptr(wq), _ptr(w_scale), _ptr(y), _ptr(ws), ws.numel())
    return y


def workspace_bytes_grouped_backward(rows: int, groups: int, N: int, K: int) -> int:
    return int(load().convrot_workspace_bytes_grouped_backward(rows, groups, N, K))


def linear_grouped_backward(dy: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor, offsets: torch.Tensor,
                            group: int = 256, dx_add: torch.Tensor | None = None,
                            out: torch.Tensor | None = None) -> torch.Tensor:
    """Input gradient of linear_grouped through its frozen weights, as linear_act_backward takes it: dy bf16
    [rows, N] -> dx bf16 [rows, K]; dx_add bf16 [rows, K], may be ``out``.  Rows of no group are not written."""
    groups, N, K = wq.shape
    rows = dy.shape[0]
    dev, bf16 = wq.device, torch.bfloat16
    _check(dev, dy=(dy, (rows, N), bf16), wq=(wq, (groups, N, K), torch.int8), w_scale=(w_scale, (groups, N), torch.float32),
           offsets=(offsets, (groups + 1,), torch.int32), dx_add=(dx_add, (rows, K), bf16), out=(out, (rows, K), bf16))
    dx, ws = _backward_buffers(rows, K, workspace_bytes_grouped_backward(rows, groups, N, K), out, dev)
    _call_on(dev, "convrot_linear_grouped_backward", _ptr(dy), rows, N, K, group, _ptr(offsets), groups, _ptr(wq),
             _ptr(w_scale), _ptr(dx_add), _ptr(dx), _ptr(ws), ws.numel())
    return dx


def workspace_bytes_moe_ffn(M: int, top: int, E: int, F: int, K: int) -> int:
    return int(load().convrot_workspace_bytes_moe_ffn(M, top, E, F, K))


def _check_experts(dev, M, top, E, F, K, experts, weights, wq_gate, gate_scale, wq_up, up_scale, wq_down, down_scale):
    f32, i8 = torch.float32, torch.int8
    _check(dev, experts=(experts, (M, top), torch.int32), weights=(weights, (M, top), f32),
           wq_gate=(wq_gate, (E, F, K), i8), gate_scale=(gate_scale, (E, F), f32), wq_up=(wq_up, (E, F, K), i8),
           up_scale=(up_scale, (E, F), f32), wq_down=(wq_down, (E, K, F), i8), down_scale=(down_scale, (E, K), f32))


def moe_ffn_gated(x: torch.Tensor, experts: torch.Tensor, weights: torch.Tensor, wq_gate: torch.Tensor,
                  gate_scale: torch.Tensor, wq_up: torch.Tensor, up_scale: torch.Tensor, wq_down: torch.Tensor,
                  down_scale: torch.Tensor, act: str = "silu", residual: torch.Tensor | None = None, group: int = 256,
                  group_h: int = 256, out: torch.Tensor | None = None, save: bool = False):
    """Gated expert layer on INT8 ConvRot weights: each token through the gated blocks of its experts (experts int32
    and weights fp32 [M, top], as moe_route gives them), y = bf16(sum_j weights[:, j] * block(x) + residual).
    gate, up [E, F, K] (prepared with ``group``), down [E, K, F] (with ``group_h``).  Slots with an expert outside [0, E) add
    nothing.  residual bf16 [M, K], may be ``out``.  save=True returns (y, pre, d) for moe_ffn_gated_backward: pre = bf16
    [2, M, top, F], g then u, and d = bf16 [M, top, K], the blocks' results; their rows of slots without an expert are
    not written.  The result itself has no autograd history."""
    _no_history("moe_ffn_gated", x, weights, residual)
    code = _act_code(act)
    E, F, K = wq_gate.shape
    dev, bf16 = wq_gate.device, torch.bfloat16
    M = _tokens(x, None, None, K, dev)
    top = experts.shape[1]
    _check_experts(dev, M, top, E, F, K, experts, weights, wq_gate, gate_scale, wq_up, up_scale, wq_down, down_scale)
    _check(dev, residual=(residual, (M, K), bf16), out=(out, (M, K), bf16))
    y = out if out is not None else torch.empty((M, K), dtype=bf16, device=dev)
    pre = torch.empty((2, M, top, F), dtype=bf16, device=dev) if save else None
    d = torch.empty((M, top, K), dtype=bf16, device=dev) if save else None
    ws = torch.empty(max(workspace_bytes_moe_ffn(M, top, E, F, K), 256), dtype=torch.uint8, device=dev)
    _call_on(dev, "convrot_moe_ffn_gated", _ptr(x), _dtype_code(x), _ptr(experts), _ptr(weights), M, top, E, F, K, group,
             group_h, _ptr(wq_gate), _ptr(gate_scale), _ptr(wq_up), _ptr(up_scale), _ptr(wq_down), _ptr(down_scale), code,
             _ptr(residual), _ptr(pre), _ptr(d), _ptr(y), _ptr(ws), ws.numel())
    return (y, pre, d) if save else y


def workspace_bytes_moe_ffn_backward(M: int, top: int, E: int, F: int, K: int) -> int:
    return int(load().convrot_workspace_bytes_moe_ffn_backward(M, top, E, F, K))


def moe_ffn_gated_backward(dy: torch.Tensor, pre: torch.Tensor, d: torch.Tensor | None, experts: torch.Tensor,
                           weights: torch.Tensor, wq_gate: torch.Tensor, gate_scale: torch.Tensor, wq_up: torch.Tensor,
                           up_scale: torch.Tensor, wq_down: torch.Tensor, down_scale: torch.Tensor, act: str = "silu",
                           group: int = 256, group_h: int = 256, dx_add: torch.Tensor | None = None,
                           out: torch.Tensor | None = None):
    """Gradients of moe_ffn_gated: dy bf16 [M, K] through down, the product, gate and up of each slot's expert (pre as
    the forward saved it), summed over a token's slots; dx_add = dy where the residual was x.  Returns (dx, dweights),
    dweights fp32 [M, top] = dy . d of each slot (0 without an expert), or None where d is None."""
    code = _act_code(act)
    E, F, K = wq_gate.shape
    M = dy.shape[0]
    top = experts.shape[1]
    dev, bf16 = wq_gate.device, torch.bfloat16
    _check_experts(dev, M, top, E, F, K, experts, weights, wq_gate, gate_scale, wq_up, up_scale, wq_down, down_scale)
    _check(dev, dy=(dy, (M, K), bf16), pre=(pre, (2, M, top, F), bf16), d=(d, (M, top, K), bf16), dx_add=(dx_add, (M, K), bf16),
           out=(out, (M, K), bf16))
    dx, ws = _backward_buffers(M, K, workspace_bytes_moe_ffn_backward(M, top, E, F, K), out, dev)
    dw = torch.empty((M, top), dtype=torch.float32, device=dev) if d is not None else None
    _call_on(dev, "convrot_moe_ffn_gated_backward", _ptr(dy), _ptr(pre), _ptr(d), _ptr(experts), _ptr(weights), M, top, E, F,
             K, group, group_h, _ptr(wq_gate), _ptr(gate_scale), _ptr(wq_up), _ptr(up_scale), _ptr(wq_down),
             _ptr(down_scale), code, _ptr(dx_add), _ptr(dx), _ptr(dw), _ptr(ws), ws.numel())
    return dx, dw


def linear_noalloc(x: torch.Tensor | None, wq: torch.Tensor, w_scale: torch.Tensor, bias: torch.Tensor | None = None,
                   group: int = 256, xq: torch.Tensor | None = None, x_scale: torch.Tensor | None = None,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """linear() through convrot_linear_noalloc: the library's fixed per-GPU scratch instead of a
    workspace (the output is allocated here unless ``out`` is given)."""
    _check_dev(x, wq, w_scale, bias, xq, x_scale, out)
    N, K = wq.shape
    M = x.shape[0] if x is not None else xq.shape[0]
    dev = wq.device
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    _call("convrot_linear_noalloc", _ptr(x), _dtype_code(x) if x is not None else 0, _ptr(xq), _ptr(x_scale), M, N, K,
          group, _ptr(wq), _ptr(w_scale), _ptr(bias), _ptr(y), _stream(dev))
    return y


def linear_w4a4(x: torch.Tensor | None, wq: torch.Tensor, w_scale: torch.Tensor, bias: torch.Tensor | None = None,
                group: int = 256, xq: torch.Tensor | None = None, x_scale: torch.Tensor | None = None,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """W4A4 ConvRot linear with packed int4 operands and fp16 group scales."""
    _check_dev(x, wq, w_scale, bias, xq, x_scale, out)
    N, Kh = wq.shape
    K = 2 * Kh
    M = x.shape[0] if x is not None else xq.shape[0]
    dev = wq.device
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    ws = _workspace(M, N, K, 4, dev)
    _call("convrot_linear_w4a4", _ptr(x), _dtype_code(x) if x is not None else 0, _ptr(xq), _ptr(x_scale), M, N, K,
          group, _ptr(wq), _ptr(w_scale), _ptr(bias), _ptr(y), _ptr(ws), ws.numel(), _stream(dev))
    return y


def packed_bytes_w4a4(N: int, K: int) -> int:
    return int(load().convrot_packed_bytes_w4a4(N, K))


def pack_weight_w4a4(wq: torch.Tensor) -> torch.Tensor:
    """Re-encode INT4 weights (prepare_weight(bits=4): wq uint8 [N, K/2]) once as FP6 codes in
    matrix-core order (a flat uint8 buffer) for linear_w4a4_packed; the scales are unchanged."""
    _check_dev(wq)
    N, Kh = wq.shape
    K = 2 * Kh
    out = torch.empty(max(packed_bytes_w4a4(N, K), 16), dtype=torch.uint8, device=wq.device)
    _call("convrot_pack_weight_w4a4", _ptr(wq), N, K, _ptr(out), _stream(wq.device))
    return out


def linear_w4a4_packed(x: torch.Tensor | None, w_packed: torch.Tensor, w_scale: torch.Tensor,
                       bias: torch.Tensor | None = None, group: int = 256, xq: torch.Tensor | None = None,
                       x_scale: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """linear_w4a4 with weights from pack_weight_w4a4 (N = w_scale.shape[1]); same result."""
    _check_dev(x, w_packed, w_scale, bias, xq, x_scale, out)
    N = w_scale.shape[1]
    M, K = x.shape if x is not None else (xq.shape[0], 2 * xq.shape[1])
    dev = w_packed.device
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    ws = _workspace(M, 0, K, 4, dev)
    _call("convrot_linear_w4a4_packed", _ptr(x), _dtype_code(x) if x is not None else 0, _ptr(xq), _ptr(x_scale), M,
          N, K, group, _ptr(w_packed), _ptr(w_scale), _ptr(bias), _ptr(y), _ptr(ws), ws.numel(), _stream(dev))
    return y


def workspace_bytes_w4a8(M: int, N: int, K: int) -> int:
    return int(load().convrot_workspace_bytes_w4a8(M, N, K))


def packed_bytes_w4a8(N: int, K: int, group: int = 256) -> int:
    return int(load().convrot_packed_bytes_w4a8_group(N, K, group))


def pack_weight_w4a8(wq: torch.Tensor, w_scale: torch.Tensor, group: int = 256) -> torch.Tensor:
    """Re-lay out INT4 weights (prepare_weight(bits=4): wq uint8 [N, K/2], w_scale fp16
    [K/group, N], group 256 or 128) into the W4A8 decode kernel's block layout (a flat uint8
    buffer); linear_w4a8 must then be called with the same group."""
    _check_dev(wq, w_scale)
    N, Kh = wq.shape
    K = 2 * Kh
    out = torch.empty(max(packed_bytes_w4a8(N, K, group), 16), dtype=torch.uint8, device=wq.device)
    if group == 256:
        _call("convrot_pack_weight_w4a8", _ptr(wq), _ptr(w_scale), N, K, _ptr(out), _stream(wq.device))
    else:
        _call("convrot_pack_weight_w4a8_group", _ptr(wq), _ptr(w_scale), N, K, group, _ptr(out), _stream(wq.device))
    return out


def linear_w4a8(x: torch.Tensor | None, w_packed: torch.Tensor, N: int, bias: torch.Tensor | None = None,
                group: int = 256, xq: torch.Tensor | None = None, x_scale: torch.Tensor | None = None,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """W4A8 ConvRot linear (at most 16 tokens): INT4 weights in the W4A8 block layout
    (pack_weight_w4a8) with N output channels, against int8 tokens (quantize_act(bits=8), or x
    quantized here)."""
    _check_dev(x, w_packed, bias, xq, x_scale, out)
    M, K = x.shape if x is not None else xq.shape
    dev = w_packed.device
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    # the workspace only holds the quantized tokens when x is given
    ws = None if x is None else torch.empty(max(workspace_bytes_w4a8(M, N, K), 256), dtype=torch.uint8, device=dev)
    # the library checks the packed size against this group's layout (the two groups' sizes differ)
    _call("convrot_linear_w4a8", _ptr(x), _dtype_code(x) if x is not None else 0, _ptr(xq), _ptr(x_scale), M, N, K,
          group, _ptr(w_packed), w_packed.numel() * w_packed.element_size(), _ptr(bias), _ptr(y), _ptr(ws),
          0 if ws is None else ws.numel(), _stream(dev))
    return y


def gemm_i8_i32(xq: torch.Tensor, wq: torch.Tensor) -> torch.Tensor:
    """Unscaled integer core: int32 [M, N] = xq . wq^T (same dispatch as linear)."""
    _check_dev(xq, wq)
    M, K = xq.shape
    N = wq.shape[0]
    acc = torch.empty((M, N), dtype=torch.int32, device=xq.device)
    ws = _workspace(M, N, K, 8, xq.device)
    _call("convrot_gemm_i8_i32", _ptr(xq), _ptr(wq), M, N, K, _ptr(acc), _ptr(ws), ws.numel(), _stream(xq.device))
    return acc


def gemm_i4_i32(xq: torch.Tensor, wq: torch.Tensor) -> torch.Tensor:
    """Unscaled W4A4 integer core over packed codes: int32 [M, N] = sum_k cx * cw."""
    _check_dev(xq, wq)
    M, Kh = xq.shape
    N = wq.shape[0]
    acc = torch.empty((M, N), dtype=torch.int32, device=xq.device)
    ws = _workspace(M, N, 2 * Kh, 4, xq.device)
    _call("convrot_gemm_i4_i32", _ptr(xq), _ptr(wq), M, N, 2 * Kh, _ptr(acc), _ptr(ws), ws.numel(), _stream(xq.device))
    return acc
