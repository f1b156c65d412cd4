"""int8_quantized_amd -- Python binding of libq8ta (MI355X / gfx950).

Thin ctypes marshalling over the C ABI declared in ``include/q8ta.h``: every
function here has the name of the C entry point it calls, checks that its
tensors are dense device tensors of the right dtype, and passes their data
pointers, sizes and the current HIP stream.  All arithmetic runs in the HIP
kernels of ``libq8ta.so``; there is no fallback.  If the library has not been
built, loading fails loudly (build it with ``python -m int8_quantized_amd.build``).

PyTorch is used only for device memory and streams.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libq8ta.so")

Q8TA_OK = 0
Q8TA_ERR_NULL = 1
Q8TA_ERR_SHAPE = 2
Q8TA_ERR_QPARAM = 3
Q8TA_ERR_UNSUPPORTED = 4
Q8TA_ERR_HIP = 5

STATUS_NAMES = {0: "Q8TA_OK", 1: "Q8TA_ERR_NULL", 2: "Q8TA_ERR_SHAPE", 3: "Q8TA_ERR_QPARAM",
                4: "Q8TA_ERR_UNSUPPORTED", 5: "Q8TA_ERR_HIP"}


class Q8taError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status
        self.message = message


_I = ctypes.c_int
_I64 = ctypes.c_int64
_DBL = ctypes.c_double
_P = ctypes.c_void_p
_S = ctypes.c_char_p

# argument types of every exported entry point, in declaration order
SIGNATURES = {
    "q8ta_last_error": ([], ctypes.c_char_p),
    "q8ta_select_kernel": ([_S, _S], ctypes.c_int),
    "q8ta_quantize_per_tensor": ([_P, _P, _I64, _DBL, _I64, _P], ctypes.c_int),
    "q8ta_dequantize_per_tensor": ([_P, _P, _I64, _DBL, _I64, _P], ctypes.c_int),
    "q8ta_linear": ([_P, _I64, _I64, _DBL, _I64, _P, _I64, _P, _P, _P, _DBL, _I64, _S, _P, _P],
                    ctypes.c_int),
    "q8ta_linear_gemv": ([_P, _I64, _I64, _DBL, _I64, _P, _I64, _P, _P, _P, _DBL, _I64, _S, _P,
                          _P], ctypes.c_int),
    "q8ta_conv2d_transposed": ([_P, _I64, _I64, _I64, _I64, _DBL, _I64, _P, _I64, _I64, _I64, _I64,
                                _P, _P, _P, _DBL, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _I64,
                                _I64, _I64, _S, _P, _I64, _I64, _P], ctypes.c_int),
    "q8ta_linear_dq": ([_P, _I64, _I64, _DBL, _I64, _P, _I64, _P, _P, _P, _DBL, _I64, _S, _P, _P],
                       ctypes.c_int),
    "q8ta_quantize_linear": ([_P, _I64, _I64, _DBL, _I64, _P, _I64, _P, _P, _P, _DBL, _I64, _S,
                              _P, _P], ctypes.c_int),
    "q8ta_quantize_linear_dq": ([_P, _I64, _I64, _DBL, _I64, _P, _I64, _P, _P, _P, _DBL, _I64,
                                 _S, _P, _P], ctypes.c_int),
    "q8ta_quantize_linear_noalloc": ([_P, _I64, _I64, _DBL, _I64, _P, _I64, _P, _P, _P, _DBL,
                                      _I64, _S, _P, _P], ctypes.c_int),
    "q8ta_weight_sums": ([_P, _I64, _I64, _P, _P], ctypes.c_int),
    "q8ta_linear_presummed": ([_P, _I64, _I64, _DBL, _I64, _P, _I64, _P, _P, _P, _DBL, _I64, _S,
                               _P, _P], ctypes.c_int),
    "q8ta_linear_dq_presummed": ([_P, _I64, _I64, _DBL, _I64, _P, _I64, _P, _P, _P, _DBL, _I64,
                                  _S, _P, _P], ctypes.c_int),
    "q8ta_weight_prepacked_bytes": ([_I64, _I64], ctypes.c_int64),
    "q8ta_conv2d_transposed_weight_prepacked_bytes": ([_I64, _I64, _I64, _I64], ctypes.c_int64),
    "q8ta_conv2d_transposed_weight_prepack": ([_P, _I64, _I64, _I64, _I64, _I64, _P, _P],
                                              ctypes.c_int),
    "q8ta_conv2d_transposed_prepacked": ([_P, _I64, _I64, _I64, _I64, _DBL, _I64, _P, _I64, _I64,
                                          _I64, _P, _P, _P, _DBL, _I64, _I64, _I64, _I64, _I64,
                                          _I64, _I64, _I64, _I64, _I64, _S, _P, _I64, _I64, _P],
                                         ctypes.c_int),
    "q8ta_quantize_conv2d_transposed_prepacked": ([_P, _I64, _I64, _I64, _I64, _DBL, _I64, _P, _I64,
                                                   _I64, _I64, _P, _P, _P, _DBL, _I64, _I64, _I64,
                                                   _I64, _I64, _I64, _I64, _I64, _I64, _I64, _S,
                                                   _P, _I64, _I64, _P], ctypes.c_int),
    "q8ta_weight_prepack": ([_P, _I64, _I64, _P, _P], ctypes.c_int),
    "q8ta_linear_prepacked": ([_P, _I64, _I64, _DBL, _I64, _P, _I64, _P, _P, _P, _DBL, _I64, _S,
                               _P, _P], ctypes.c_int),
    "q8ta_linear_dq_prepacked": ([_P, _I64, _I64, _DBL, _I64, _P, _I64, _P, _P, _P, _DBL, _I64,
                                  _S, _P, _P], ctypes.c_int),
    "q8ta_quantize_conv2d_transposed": ([_P, _I64, _I64, _I64, _I64, _DBL, _I64, _P, _I64, _I64,
                                         _I64, _I64, _P, _P, _P, _DBL, _I64, _I64, _I64, _I64,
                                         _I64, _I64, _I64, _I64, _I64, _I64, _S, _P, _I64, _I64,
                                         _P], ctypes.c_int),
    "q8ta_linear_acc": ([_P, _I64, _I64, _I64, _P, _I64, _P, _P], ctypes.c_int),
    "q8ta_conv2d_transposed_acc": ([_P, _I64, _I64, _I64, _I64, _I64, _P, _I64, _I64, _I64, _I64,
                                    _I64, _I64, _I64, _I64, _I64, _I64, _I64, _P, _I64, _I64, _P],
                                   ctypes.c_int),
    "q8ta_conv2d": ([_P, _I64, _I64, _I64, _I64, _DBL, _I64, _P, _I64, _I64, _I64, _I64,
                     _P, _P, _P, _DBL, _I64, _I64, _I64, _I64, _I64, _I64, _I64,
                     _I64, _S, _P, _I64, _I64, _P], ctypes.c_int),
    "q8ta_conv2d_acc": ([_P, _I64, _I64, _I64, _I64, _I64, _P, _I64, _I64, _I64, _I64,
                         _I64, _I64, _I64, _I64, _I64, _I64, _I64, _P, _I64, _I64, _P],
                        ctypes.c_int),
    "q8ta_rope_append": ([_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _I, _I64, _I64, _I64,
                          _I64, _P, _P, _P, _I64, _DBL, _I64, _P, _P, _P, _I64, _I64, _P],
                         ctypes.c_int),
    "q8ta_tree_attention": ([_P, _I64, _I64, _I64, _I, _I64, _I64, _I64, _I64, _I64, _P, _P, _I64,
                             _I64, _P, _I64, _P, _P, _P, _DBL, _P, _P, _P], ctypes.c_int),
    "q8ta_linear_lora": ([_P, _I64, _I64, _DBL, _I64, _P, _I64, _P, _P, _P, _P, _I, _I64, _I64, _P,
                          _P, _P, _S, _P, _I, _P], ctypes.c_int),
    "q8ta_sample": ([_P, _I64, _I, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "q8ta_norm_quantize": ([_P, _I64, _P, _I64, _I, _I64, _I64, _P, _P, _I64, _DBL, _P, _DBL, _P, _P,
                            _P, _P], ctypes.c_int),
    "q8ta_quantize_per_token": ([_P, _I64, _I, _I64, _I64, _P, _P, _P], ctypes.c_int),
    "q8ta_linear_per_token": ([_P, _I64, _I64, _P, _P, _I64, _P, _P, _S, _P, _I, _P], ctypes.c_int),
    "q8ta_gated_linear": ([_P, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _I64, _S, _P, _I, _P],
                          ctypes.c_int),
    "q8ta_verify_drafts": ([_P, _I64, _I64, _P, _I64, _I64, _I, _I64, _I64, _I64, _P, _P, _P, _P, _P,
                            _P, _P, _P, _P, _P], ctypes.c_int),
    "q8ta_pages_take": ([_P, _I64, _I64, _I64, _P, _P, _P, _I64, _P, _P], ctypes.c_int),
    "q8ta_pages_fork": ([_P, _I64, _I64, _I64, _P, _P, _P, _I64, _P, _I64, _P, _P, _P, _P, _P],
                        ctypes.c_int),
    "q8ta_pages_release": ([_P, _I64, _I64, _I64, _P, _P, _P, _I64, _P, _I64, _P], ctypes.c_int),
    "q8ta_pages_copy": ([_P, _P, _I64, _I64, _I64, _I64, _P, _P, _P, _I64, _P], ctypes.c_int),
    "q8ta_cache_compact": ([_P, _P, _I64, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _I64, _P, _P],
                           ctypes.c_int),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libq8ta.so with argument types set (raises if not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"libq8ta.so not found at {LIB_PATH}: build it with "
                "`python -m int8_quantized_amd.build` (there is no CPU fallback)")
        l = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(l, name)
            fn.argtypes = args
            fn.restype = res
        _lib = l
    return _lib


def q8ta_last_error() -> str:
    return lib().q8ta_last_error().decode()


def _check(status: int):
    if status != Q8TA_OK:
        raise Q8taError(status, q8ta_last_error())


def q8ta_select_kernel(op: str, kernel: str) -> None:
    """Force one kernel family of ``op`` ("linear", "conv2d_transposed",
    "conv2d") where the shape allows it; "default" restores the normal choice."""
    _check(lib().q8ta_select_kernel(op.encode(), kernel.encode()))


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dev(t, dtype, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _opt(t, dtype, name):
    return None if t is None else _dev(t, dtype, name)


def _stream(stream):
    if stream is None:
        # the handle of torch.cuda.current_stream(), without building its Python object (2.8 us)
        c = _torch()._C
        return c._cuda_getCurrentRawStream(c._cuda_getDevice())
    return getattr(stream, "cuda_stream", stream)


def _act(activation):
    return None if activation is None else activation.encode()


# ---------------------------------------------------------------------------
def q8ta_quantize_per_tensor(x, out, scale: float, zero_point: int, stream=None):
    """out (int8) = clamp(rint(x * (float)(1/scale)) + zero_point, -128, 127)."""
    torch = _torch()
    if x.numel() != out.numel():
        raise ValueError("x and out must have the same number of elements")
    _check(lib().q8ta_quantize_per_tensor(_dev(x, torch.float32, "x"), _dev(out, torch.int8, "out"),
                                          x.numel(), float(scale), int(zero_point), _stream(stream)))
    return out


def q8ta_dequantize_per_tensor(x, out, scale: float, zero_point: int, stream=None):
    """out (fp32) = (float)(x - zero_point) * (float)scale."""
    torch = _torch()
    if x.numel() != out.numel():
        raise ValueError("x and out must have the same number of elements")
    _check(lib().q8ta_dequantize_per_tensor(_dev(x, torch.int8, "x"), _dev(out, torch.float32, "out"),
                                            x.numel(), float(scale), int(zero_point), _stream(stream)))
    return out


def _linear(fn, x, input_scale, input_zero_point, weight, weight_sums, weight_scales, bias,
            output_scale, output_zero_point, activation, out, stream):
    torch = _torch()
    if x.dim() != 2 or weight.dim() != 2 or out.dim() != 2:
        raise ValueError("x [M,K], weight [N,K] and out [M,N] must be 2-D")
    M, K = x.shape
    N = weight.shape[0]
    if weight.shape[1] != K or tuple(out.shape) != (M, N):
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, weight {tuple(weight.shape)}, "
                         f"out {tuple(out.shape)}")
    _check(fn(_dev(x, torch.int8, "x"), M, K, float(input_scale), int(input_zero_point),
              _dev(weight, torch.int8, "weight"), N, _opt(weight_sums, torch.int32, "weight_sums"),
              _dev(weight_scales, torch.float32, "weight_scales"), _opt(bias, torch.float32, "bias"),
              float(output_scale), int(output_zero_point), _act(activation),
              _dev(out, torch.int8, "out"), _stream(stream)))
    return out


def q8ta_linear(x, input_scale, input_zero_point, weight, weight_sums, weight_scales, bias,
                output_scale, output_zero_point, activation, out, stream=None):
    """int8 [M,K] x int8 [N,K] -> int8 [M,N] with the per-channel epilogue."""
    return _linear(lib().q8ta_linear, x, input_scale, input_zero_point, weight, weight_sums,
                   weight_scales, bias, output_scale, output_zero_point, activation, out, stream)


def q8ta_linear_gemv(x, input_scale, input_zero_point, weight, weight_sums, weight_scales, bias,
                     output_scale, output_zero_point, activation, out, stream=None):
    """q8ta_linear for M == 1."""
    return _linear(lib().q8ta_linear_gemv, x, input_scale, input_zero_point, weight, weight_sums,
                   weight_scales, bias, output_scale, output_zero_point, activation, out, stream)


def q8ta_weight_sums(weight, sums, stream=None):
    """sums[n] = sum_k weight[n, k] (int32 [N]) for int8 weight [N, K]."""
    torch = _torch()
    if weight.dim() != 2 or tuple(sums.shape) != (weight.shape[0],):
        raise ValueError("weight [N, K] and sums [N] expected")
    _check(lib().q8ta_weight_sums(_dev(weight, torch.int8, "weight"), weight.shape[0],
                                  weight.shape[1], _dev(sums, torch.int32, "sums"),
                                  _stream(stream)))
    return sums


def q8ta_linear_presummed(x, input_scale, input_zero_point, weight, weight_sums, weight_scales,
                          bias, output_scale, output_zero_point, activation, out, stream=None):
    """q8ta_linear with the caller's (trusted) weight_sums."""
    if weight_sums is None:
        raise ValueError("weight_sums is required")
    return _linear(lib().q8ta_linear_presummed, x, input_scale, input_zero_point, weight,
                   weight_sums, weight_scales, bias, output_scale, output_zero_point, activation,
                   out, stream)


def q8ta_linear_dq_presummed(x, input_scale, input_zero_point, weight, weight_sums, weight_scales,
                             bias, output_scale, output_zero_point, activation, out, stream=None):
    """q8ta_linear_dq with the caller's (trusted) weight_sums: fp32 out [M, N]."""
    torch = _torch()
    if weight_sums is None:
        raise ValueError("weight_sums is required")
    M, K = x.shape
    N = weight.shape[0]
    if weight.shape[1] != K or tuple(out.shape) != (M, N):
        raise ValueError("weight [N, K] and out [M, N] expected")
    _check(lib().q8ta_linear_dq_presummed(
        _dev(x, torch.int8, "x"), M, K, float(input_scale), int(input_zero_point),
        _dev(weight, torch.int8, "weight"), N, _dev(weight_sums, torch.int32, "weight_sums"),
        _dev(weight_scales, torch.float32, "weight_scales"), _opt(bias, torch.float32, "bias"),
        float(output_scale), int(output_zero_point), _act(activation),
        _dev(out, torch.float32, "out"), _stream(stream)))
    return out


def q8ta_weight_prepacked_bytes(N: int, K: int) -> int:
    """Size in bytes of the prepacked layout of an int8 [N, K] weight (-1 if invalid)."""
    return int(lib().q8ta_weight_prepacked_bytes(int(N), int(K)))


def q8ta_weight_prepack(weight, packed, stream=None):
    """Rearrange int8 weight [N, K] into the matrix-core fragment layout
    (packed: int8 device tensor of q8ta_weight_prepacked_bytes(N, K) bytes)."""
    torch = _torch()
    if weight.dim() != 2:
        raise ValueError("weight [N, K] expected")
    N, K = weight.shape
    if packed.numel() != q8ta_weight_prepacked_bytes(N, K):
        raise ValueError(f"packed must hold {q8ta_weight_prepacked_bytes(N, K)} bytes")
    _check(lib().q8ta_weight_prepack(_dev(weight, torch.int8, "weight"), N, K,
                                     _dev(packed, torch.int8, "packed"), _stream(stream)))
    return packed


def _linear_pk(fn, out_dtype, x, input_scale, input_zero_point, packed, N, weight_sums,
               weight_scales, bias, output_scale, output_zero_point, activation, out, stream):
    torch = _torch()
    if weight_sums is None:
        raise ValueError("weight_sums is required")
    if x.dim() != 2 or tuple(out.shape) != (x.shape[0], N):
        raise ValueError("x [M, K] and out [M, N] expected")
    M, K = x.shape
    if packed.numel() != q8ta_weight_prepacked_bytes(N, K):
        raise ValueError("packed does not hold an [N, K] prepacked weight")
    _check(fn(_dev(x, torch.int8, "x"), M, K, float(input_scale), int(input_zero_point),
              _dev(packed, torch.int8, "packed"), int(N),
              _dev(weight_sums, torch.int32, "weight_sums"),
              _dev(weight_scales, torch.float32, "weight_scales"), _opt(bias, torch.float32, "bias"),
              float(output_scale), int(output_zero_point), _act(activation),
              _dev(out, out_dtype, "out"), _stream(stream)))
    return out


def q8ta_linear_prepacked(x, input_scale, input_zero_point, packed, N, weight_sums, weight_scales,
                          bias, output_scale, output_zero_point, activation, out, stream=None):
    """q8ta_linear_presummed on a prepacked weight of N rows: int8 out [M, N]."""
    return _linear_pk(lib().q8ta_linear_prepacked, _torch().int8, x, input_scale,
                      input_zero_point, packed, N, weight_sums, weight_scales, bias, output_scale,
                      output_zero_point, activation, out, stream)


def q8ta_linear_dq_prepacked(x, input_scale, input_zero_point, packed, N, weight_sums,
                             weight_scales, bias, output_scale, output_zero_point, activation, out,
                             stream=None):
    """q8ta_linear_dq_presummed on a prepacked weight of N rows: fp32 out [M, N]."""
    return _linear_pk(lib().q8ta_linear_dq_prepacked, _torch().float32, x, input_scale,
                      input_zero_point, packed, N, weight_sums, weight_scales, bias, output_scale,
                      output_zero_point, activation, out, stream)


def q8ta_linear_acc(x, input_zero_point, weight, acc, stream=None):
    """int32 accumulator of q8ta_linear: acc[m,n] = sum_k (x[m,k]-izp)*w[n,k]."""
    torch = _torch()
    M, K = x.shape
    N = weight.shape[0]
    if weight.shape[1] != K or tuple(acc.shape) != (M, N):
        raise ValueError("shape mismatch")
    _check(lib().q8ta_linear_acc(_dev(x, torch.int8, "x"), M, K, int(input_zero_point),
                                 _dev(weight, torch.int8, "weight"), N,
                                 _dev(acc, torch.int32, "acc"), _stream(stream)))
    return acc


def q8ta_linear_dq(x, input_scale, input_zero_point, weight, weight_sums, weight_scales, bias,
                   output_scale, output_zero_point, activation, out, stream=None):
    """q8ta_linear then dequantize_per_tensor of its output, in one call:
    fp32 out [M, N]."""
    torch = _torch()
    M, K = x.shape
    N = weight.shape[0]
    if weight.shape[1] != K or tuple(out.shape) != (M, N):
        raise ValueError("weight [N, K] and out [M, N] expected")
    _check(lib().q8ta_linear_dq(
        _dev(x, torch.int8, "x"), M, K, float(input_scale), int(input_zero_point),
        _dev(weight, torch.int8, "weight"), N, _opt(weight_sums, torch.int32, "weight_sums"),
        _dev(weight_scales, torch.float32, "weight_scales"), _opt(bias, torch.float32, "bias"),
        float(output_scale), int(output_zero_point), _act(activation),
        _dev(out, torch.float32, "out"), _stream(stream)))
    return out


def _quantize_linear(fn, out_dtype, x, input_scale, input_zero_point, weight, weight_sums,
                     weight_scales, bias, output_scale, output_zero_point, activation, out, stream):
    torch = _torch()
    if x.dim() != 2 or weight.dim() != 2 or out.dim() != 2:
        raise ValueError("x [M,K], weight [N,K] and out [M,N] must be 2-D")
    M, K = x.shape
    N = weight.shape[0]
    if weight.shape[1] != K or tuple(out.shape) != (M, N):
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, weight {tuple(weight.shape)}, "
                         f"out {tuple(out.shape)}")
    _check(fn(_dev(x, torch.float32, "x"), M, K, float(input_scale), int(input_zero_point),
              _dev(weight, torch.int8, "weight"), N, _opt(weight_sums, torch.int32, "weight_sums"),
              _dev(weight_scales, torch.float32, "weight_scales"), _opt(bias, torch.float32, "bias"),
              float(output_scale), int(output_zero_point), _act(activation),
              _dev(out, out_dtype, "out"), _stream(stream)))
    return out


def q8ta_quantize_linear(x, input_scale, input_zero_point, weight, weight_sums, weight_scales,
                         bias, output_scale, output_zero_point, activation, out, stream=None):
    """quantize_per_tensor of fp32 x [M, K] (input_scale, input_zero_point), then
    q8ta_linear, in one call: int8 out [M, N]."""
    return _quantize_linear(lib().q8ta_quantize_linear, _torch().int8, x, input_scale,
                            input_zero_point, weight, weight_sums, weight_scales, bias,
                            output_scale, output_zero_point, activation, out, stream)


def q8ta_quantize_linear_noalloc(x, input_scale, input_zero_point, weight, weight_sums,
                                 weight_scales, bias, output_scale, output_zero_point, activation,
                                 out, stream=None):
    """q8ta_quantize_linear without any device allocation (the quantized
    activations go through the library's static scratch; M * K <= 16 MiB)."""
    return _quantize_linear(lib().q8ta_quantize_linear_noalloc, _torch().int8, x, input_scale,
                            input_zero_point, weight, weight_sums, weight_scales, bias,
                            output_scale, output_zero_point, activation, out, stream)


def q8ta_quantize_linear_dq(x, input_scale, input_zero_point, weight, weight_sums, weight_scales,
                            bias, output_scale, output_zero_point, activation, out, stream=None):
    """quantize_per_tensor -> q8ta_linear -> dequantize_per_tensor of fp32 x [M, K]
    in one call: fp32 out [M, N]."""
    return _quantize_linear(lib().q8ta_quantize_linear_dq, _torch().float32, x, input_scale,
                            input_zero_point, weight, weight_sums, weight_scales, bias,
                            output_scale, output_zero_point, activation, out, stream)


def q8ta_conv2d_transposed(x, input_scale, input_zero_point, weight, Kh, Kw, weight_sums,
                           weight_scales, bias, output_scale, output_zero_point, stride, padding,
                           output_padding, dilation, groups, activation, out, stream=None):
    """int8 NCHW x int8 [OC, ldw] -> int8 NCHW out (H_out, W_out taken from out)."""
    torch = _torch()
    if x.dim() != 4 or weight.dim() != 2 or out.dim() != 4:
        raise ValueError("x [N,IC,H,W], weight [OC, ldw] and out [N,OC,H_out,W_out] expected")
    N, IC, H_in, W_in = x.shape
    OC, ldw = weight.shape
    if out.shape[0] != N or out.shape[1] != OC:
        raise ValueError("out must be [N, OC, H_out, W_out]")
    H_out, W_out = out.shape[2], out.shape[3]
    _check(lib().q8ta_conv2d_transposed(
        _dev(x, torch.int8, "x"), N, IC, H_in, W_in, float(input_scale), int(input_zero_point),
        _dev(weight, torch.int8, "weight"), OC, int(Kh), int(Kw), ldw,
        _opt(weight_sums, torch.int32, "weight_sums"),
        _dev(weight_scales, torch.float32, "weight_scales"), _opt(bias, torch.float32, "bias"),
        float(output_scale), int(output_zero_point), int(stride[0]), int(stride[1]),
        int(padding[0]), int(padding[1]), int(output_padding[0]), int(output_padding[1]),
        int(dilation[0]), int(dilation[1]), int(groups), _act(activation),
        _dev(out, torch.int8, "out"), H_out, W_out, _stream(stream)))
    return out


def q8ta_conv2d_transposed_weight_prepacked_bytes(OC: int, IC: int, Kh: int, Kw: int) -> int:
    """Size in bytes of the prepacked transposed-conv weight (-1 if unsupported)."""
    return int(lib().q8ta_conv2d_transposed_weight_prepacked_bytes(int(OC), int(IC), int(Kh),
                                                                   int(Kw)))


def q8ta_conv2d_transposed_weight_prepack(weight, IC, Kh, Kw, packed, stream=None):
    """Rearrange the int8 [OC, ldw] transposed-conv weight into its fragment
    layout (packed: int8 device tensor of the prepacked size)."""
    torch = _torch()
    if weight.dim() != 2:
        raise ValueError("weight [OC, ldw] expected")
    OC, ldw = weight.shape
    nb = q8ta_conv2d_transposed_weight_prepacked_bytes(OC, IC, Kh, Kw)
    if packed.numel() != nb:
        raise ValueError(f"packed must hold {nb} bytes")
    _check(lib().q8ta_conv2d_transposed_weight_prepack(
        _dev(weight, torch.int8, "weight"), OC, int(IC), int(Kh), int(Kw), ldw,
        _dev(packed, torch.int8, "packed"), _stream(stream)))
    return packed


def q8ta_conv2d_transposed_prepacked(x, input_scale, input_zero_point, packed, OC, Kh, Kw,
                                     weight_sums, weight_scales, bias, output_scale,
                                     output_zero_point, stride, padding, output_padding, dilation,
                                     groups, activation, out, stream=None):
    """q8ta_conv2d_transposed on a prepacked weight (H_out, W_out taken from out);
    with an fp32 x, q8ta_quantize_conv2d_transposed_prepacked."""
    torch = _torch()
    fp32 = x.dtype == torch.float32
    fn = (lib().q8ta_quantize_conv2d_transposed_prepacked if fp32
          else lib().q8ta_conv2d_transposed_prepacked)
    if x.dim() != 4 or out.dim() != 4:
        raise ValueError("x [N,IC,H,W] and out [N,OC,H_out,W_out] expected")
    N, IC, H_in, W_in = x.shape
    if out.shape[0] != N or out.shape[1] != OC:
        raise ValueError("out must be [N, OC, H_out, W_out]")
    if packed.numel() != q8ta_conv2d_transposed_weight_prepacked_bytes(OC, IC, Kh, Kw):
        raise ValueError("packed does not hold an [OC, Kh*Kw*IC] prepacked weight")
    _check(fn(
        _dev(x, torch.float32 if fp32 else torch.int8, "x"), N, IC, H_in, W_in,
        float(input_scale), int(input_zero_point),
        _dev(packed, torch.int8, "packed"), int(OC), int(Kh), int(Kw),
        _opt(weight_sums, torch.int32, "weight_sums"),
        _dev(weight_scales, torch.float32, "weight_scales"), _opt(bias, torch.float32, "bias"),
        float(output_scale), int(output_zero_point), int(stride[0]), int(stride[1]),
        int(padding[0]), int(padding[1]), int(output_padding[0]), int(output_padding[1]),
        int(dilation[0]), int(dilation[1]), int(groups), _act(activation),
        _dev(out, torch.int8, "out"), out.shape[2], out.shape[3], _stream(stream)))
    return out


def q8ta_quantize_conv2d_transposed(x, input_scale, input_zero_point, weight, Kh, Kw,
                                    weight_sums, weight_scales, bias, output_scale,
                                    output_zero_point, stride, padding, output_padding, dilation,
                                    groups, activation, out, stream=None):
    """quantize_per_tensor of the fp32 NCHW x, then q8ta_conv2d_transposed, in
    one call (H_out, W_out taken from out)."""
    torch = _torch()
    if x.dim() != 4 or weight.dim() != 2 or out.dim() != 4:
        raise ValueError("x [N,IC,H,W], weight [OC, ldw] and out [N,OC,H_out,W_out] expected")
    N, IC, H_in, W_in = x.shape
    OC, ldw = weight.shape
    if out.shape[0] != N or out.shape[1] != OC:
        raise ValueError("out must be [N, OC, H_out, W_out]")
    _check(lib().q8ta_quantize_conv2d_transposed(
        _dev(x, torch.float32, "x"), N, IC, H_in, W_in, float(input_scale),
        int(input_zero_point), _dev(weight, torch.int8, "weight"), OC, int(Kh), int(Kw), ldw,
        _opt(weight_sums, torch.int32, "weight_sums"),
        _dev(weight_scales, torch.float32, "weight_scales"), _opt(bias, torch.float32, "bias"),
        float(output_scale), int(output_zero_point), int(stride[0]), int(stride[1]),
        int(padding[0]), int(padding[1]), int(output_padding[0]), int(output_padding[1]),
        int(dilation[0]), int(dilation[1]), int(groups), _act(activation),
        _dev(out, torch.int8, "out"), out.shape[2], out.shape[3], _stream(stream)))
    return out


def q8ta_conv2d_transposed_acc(x, input_zero_point, weight, Kh, Kw, stride, padding, acc,
                               stream=None, dilation=(1, 1), groups=1):
    """int32 accumulator of q8ta_conv2d_transposed (NCHW [N, OC, H_out, W_out])."""
    torch = _torch()
    N, IC, H_in, W_in = x.shape
    OC, ldw = weight.shape
    if acc.dim() != 4 or acc.shape[0] != N or acc.shape[1] != OC:
        raise ValueError("acc must be [N, OC, H_out, W_out]")
    _check(lib().q8ta_conv2d_transposed_acc(
        _dev(x, torch.int8, "x"), N, IC, H_in, W_in, int(input_zero_point),
        _dev(weight, torch.int8, "weight"), OC, int(Kh), int(Kw), ldw, int(stride[0]),
        int(stride[1]), int(padding[0]), int(padding[1]), int(dilation[0]), int(dilation[1]),
        int(groups), _dev(acc, torch.int32, "acc"), acc.shape[2], acc.shape[3],
        _stream(stream)))
    return acc


def q8ta_conv2d(x, input_scale, input_zero_point, weight, Kh, Kw, weight_sums, weight_scales,
                bias, output_scale, output_zero_point, stride, padding, dilation, groups,
                activation, out, stream=None):
    """Forward conv: int8 NCHW x int8 [OC, ldw] -> int8 NCHW out (H_out, W_out
    taken from out)."""
    torch = _torch()
    if x.dim() != 4 or weight.dim() != 2 or out.dim() != 4:
        raise ValueError("x [N,IC,H,W], weight [OC, ldw] and out [N,OC,H_out,W_out] expected")
    N, IC, H_in, W_in = x.shape
    OC, ldw = weight.shape
    if out.shape[0] != N or out.shape[1] != OC:
        raise ValueError("out must be [N, OC, H_out, W_out]")
    _check(lib().q8ta_conv2d(
        _dev(x, torch.int8, "x"), N, IC, H_in, W_in, float(input_scale), int(input_zero_point),
        _dev(weight, torch.int8, "weight"), OC, int(Kh), int(Kw), ldw,
        _opt(weight_sums, torch.int32, "weight_sums"),
        _dev(weight_scales, torch.float32, "weight_scales"), _opt(bias, torch.float32, "bias"),
        float(output_scale), int(output_zero_point), int(stride[0]), int(stride[1]),
        int(padding[0]), int(padding[1]), int(dilation[0]), int(dilation[1]), int(groups),
        _act(activation), _dev(out, torch.int8, "out"), out.shape[2], out.shape[3],
        _stream(stream)))
    return out


def q8ta_conv2d_acc(x, input_zero_point, weight, Kh, Kw, stride, padding, dilation, acc,
                    groups=1, stream=None):
    """int32 accumulator of q8ta_conv2d (NCHW [N, OC, H_out, W_out])."""
    torch = _torch()
    N, IC, H_in, W_in = x.shape
    OC, ldw = weight.shape
    if acc.dim() != 4 or acc.shape[0] != N or acc.shape[1] != OC:
        raise ValueError("acc must be [N, OC, H_out, W_out]")
    _check(lib().q8ta_conv2d_acc(
        _dev(x, torch.int8, "x"), N, IC, H_in, W_in, int(input_zero_point),
        _dev(weight, torch.int8, "weight"), OC, int(Kh), int(Kw), ldw, int(stride[0]),
        int(stride[1]), int(padding[0]), int(padding[1]), int(dilation[0]), int(dilation[1]),
        int(groups), _dev(acc, torch.int32, "acc"), acc.shape[2], acc.shape[3],
        _stream(stream)))
    return acc


# ---------------------------------------------------------------------------
# Decode-step operators

_dtype_codes = None


def _code(t, name, allowed=("fp32", "fp16", "bf16")):
    """q8ta_dtype of a floating-point tensor."""
    global _dtype_codes
    if _dtype_codes is None:
        torch = _torch()
        _dtype_codes = {torch.float32: (0, "fp32"), torch.float16: (1, "fp16"),
                        torch.bfloat16: (2, "bf16")}
    c = _dtype_codes.get(t.dtype)
    if c is None or c[1] not in allowed:
        raise TypeError(f"{name} must be {' or '.join(allowed)} (got {t.dtype})")
    return c[0]


def _view(t, name, dim):
    """Data pointer, shape and strides of a device tensor whose last of `dim` dimensions has
    stride 1."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    shape, strides = t.shape, t.stride()
    if len(shape) != dim or (strides[-1] != 1 and shape[-1] > 1):
        raise ValueError(f"{name} must have {dim} dimensions, the last of stride 1")
    return t.data_ptr(), shape, strides


def _ptr(t, dtype, name):
    """_dev for the operators whose calls are short: the same checks, by their cheapest tests."""
    if t.dtype is dtype and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    return _dev(t, dtype, name)


def _opt_ptr(t, dtype, name):
    return None if t is None else _ptr(t, dtype, name)


def q8ta_rope_append(q, k, v, positions, slots, inv_freq, factor, interleaved, q_out, cache,
                     cache_scales, stream=None):
    """Rotary positions on q and k, and the append of k and v to the paged int8 cache.

    q [T, heads, dim], k and v [T, kv_heads, dim] (fp32, fp16 or bf16, any token and head
    strides), positions int32 [T], slots int64 [T] (negative: not stored, else each once), inv_freq fp64
    [rot / 2]; q_out like q, dense; cache int8 [pages, 2, kv_heads, page, dim] and cache_scales
    fp32 [pages, 2, kv_heads, page].  ``interleaved`` pairs neighbours, else the two halves of
    the rotated part; ``factor`` multiplies cos and sin.  Returns q_out."""
    torch = _torch()
    cs = cache.shape
    if len(cs) != 5 or cs[1] != 2 or cs[:4] != cache_scales.shape:
        raise ValueError("cache [pages, 2, kv_heads, page, dim] and cache_scales [pages, 2, "
                         "kv_heads, page] expected")
    pages, _, hk, page, d = cs
    qp, qs, qt = _view(q, "q", 3)
    kp, ks, kt = _view(k, "k", 3)
    vp, vs, vt = _view(v, "v", 3)
    T, hq, qd = qs
    if qd != d or ks != (T, hk, d) or vs != ks or q_out.shape != qs:
        raise ValueError(f"shape mismatch: q {tuple(qs)}, k {tuple(ks)}, v {tuple(vs)}, q_out "
                         f"{tuple(q_out.shape)}, cache {tuple(cs)}")
    pairs = inv_freq.shape
    if positions.shape != (T,) or slots.shape != (T,) or len(pairs) != 1:
        raise ValueError("positions [T], slots [T] and inv_freq [rot / 2] expected")
    dtype = q.dtype
    if k.dtype is not dtype or v.dtype is not dtype:
        raise TypeError("q, k and v must have one dtype")
    _check(lib().q8ta_rope_append(
        qp, qt[0], qt[1], kp, kt[0], kt[1], vp, vt[0], vt[1], _code(q, "q"), T, hq, hk, d,
        _ptr(positions, torch.int32, "positions"), _ptr(slots, torch.int64, "slots"),
        _ptr(inv_freq, torch.float64, "inv_freq"), 2 * pairs[0], factor, int(interleaved),
        _ptr(q_out, dtype, "q_out"), _ptr(cache, torch.int8, "cache"),
        _ptr(cache_scales, torch.float32, "cache_scales"), pages, page, _stream(stream)))
    return q_out


def q8ta_tree_attention(q, cache, cache_scales, table, lens, counts, mask, softmax_scale, out,
                        lse=None, stream=None):
    """Attention of each request's newest tokens (one, or a tree of drafted ones) over the paged
    int8 cache.

    q [B, T, heads, dim] (fp16 or bf16, any outer strides, T <= 64); cache and cache_scales as
    q8ta_rope_append fills them; table int32 [B, pages of a request]; lens int32 [B]: context rows
    before the T tokens' own; counts int32 [B] or None: tokens in use; mask int64 [B, T] or None:
    bit j of mask[b, i] lets token i see token j (None: a chain); out like q, dense; lse fp32
    [B, T, heads] or None.  Returns out."""
    torch = _torch()
    cs = cache.shape
    if len(cs) != 5 or cs[1] != 2 or cs[:4] != cache_scales.shape:
        raise ValueError("cache [pages, 2, kv_heads, page, dim] and cache_scales [pages, 2, "
                         "kv_heads, page] expected")
    pages, _, hk, page, d = cs
    qp, qs, qt = _view(q, "q", 4)
    B, T, hq, qd = qs
    if qd != d or out.shape != qs or (lse is not None and lse.shape != (B, T, hq)):
        raise ValueError(f"shape mismatch: q {tuple(qs)}, cache {tuple(cs)}, out "
                         f"{tuple(out.shape)}, lse {None if lse is None else tuple(lse.shape)}")
    ts = table.shape
    if (len(ts) != 2 or ts[0] != B or lens.shape != (B,) or
            (counts is not None and counts.shape != (B,)) or
            (mask is not None and mask.shape != (B, T))):
        raise ValueError("table [B, pages], lens [B], counts [B] and mask [B, T] expected")
    i32 = torch.int32
    _check(lib().q8ta_tree_attention(
        qp, qt[0], qt[1], qt[2], _code(q, "q", ("fp16", "bf16")), B, T, hq, hk, d,
        _ptr(cache, torch.int8, "cache"), _ptr(cache_scales, torch.float32, "cache_scales"), pages,
        page, _ptr(table, i32, "table"), ts[1], _ptr(lens, i32, "lens"),
        _opt_ptr(counts, i32, "counts"), _opt_ptr(mask, torch.int64, "mask"), softmax_scale,
        _ptr(out, q.dtype, "out"), _opt_ptr(lse, torch.float32, "lse"), _stream(stream)))
    return out


def q8ta_sample(logits, temperature, top_k, top_p, min_p, u, tokens, logprobs=None, stream=None):
    """One token a row by temperature, top-k, top-p and min-p from given random numbers.

    logits [B, V] (fp32, fp16 or bf16, rows may be strided); temperature, top_p, min_p and u fp32
    [B], top_k int32 [B] (top_k, top_p and min_p may be None); tokens int32 [B]; logprobs fp32 [B]
    or None: the token's log-probability among those kept.  Temperature 0 is greedy.  Returns
    tokens."""
    torch = _torch()
    lp, ls, lt = _view(logits, "logits", 2)
    B, V = ls
    rows = (B,)
    for t in (temperature, top_k, top_p, min_p, u, tokens, logprobs):
        if t is not None and t.shape != rows:
            raise ValueError(f"temperature, top_k, top_p, min_p, u, tokens and logprobs must be [{B}] "
                             f"(got {tuple(t.shape)})")
    f32, i32 = torch.float32, torch.int32
    _check(lib().q8ta_sample(
        lp, lt[0], _code(logits, "logits"), B, V, _ptr(temperature, f32, "temperature"),
        _opt_ptr(top_k, i32, "top_k"), _opt_ptr(top_p, f32, "top_p"), _opt_ptr(min_p, f32, "min_p"),
        _ptr(u, f32, "u"), _ptr(tokens, i32, "tokens"), _opt_ptr(logprobs, f32, "logprobs"),
        _stream(stream)))
    return tokens


def q8ta_linear_lora(x, input_scale, input_zero_point, weight, weight_scales, bias, lora_a, lora_b,
                     adapter_scales, ranks, adapter_ids, activation, out, stream=None):
    """q8ta_linear's projection with the low-rank adapters of many requests, floating-point out.

    x int8 [M, K], weight int8 [N, K]; lora_a [adapters, rank, K] and lora_b [adapters, N, rank]
    (fp16 or bf16); adapter_scales fp32 [adapters] or None; ranks int32 [adapters] or None (each
    adapter's own rank); adapter_ids int32 [M], negative for none; out [M, N] fp32, fp16 or bf16.
    Returns out."""
    torch = _torch()
    xs, wsh, ash = x.shape, weight.shape, lora_a.shape
    if len(xs) != 2 or len(wsh) != 2 or len(ash) != 3:
        raise ValueError("x [M, K], weight [N, K], lora_a [adapters, rank, K] and lora_b [adapters, N, "
                         "rank] expected")
    M, K = xs
    N = wsh[0]
    na, r, ak = ash
    if (wsh[1] != K or ak != K or lora_b.shape != (na, N, r) or out.shape != (M, N) or
            adapter_ids.shape != (M,)):
        raise ValueError(f"shape mismatch: x {tuple(xs)}, weight {tuple(wsh)}, lora_a {tuple(ash)}, "
                         f"lora_b {tuple(lora_b.shape)}, adapter_ids {tuple(adapter_ids.shape)}, out "
                         f"{tuple(out.shape)}")
    for name, t, n in (("weight_scales", weight_scales, N), ("bias", bias, N),
                       ("adapter_scales", adapter_scales, na), ("ranks", ranks, na)):
        if t is not None and t.numel() < n:
            raise ValueError(f"{name} must have {n} entries (got {t.numel()})")
    f32, i8, i32, ad = torch.float32, torch.int8, torch.int32, lora_a.dtype
    _check(lib().q8ta_linear_lora(
        _ptr(x, i8, "x"), M, K, input_scale, input_zero_point, _ptr(weight, i8, "weight"), N,
        _ptr(weight_scales, f32, "weight_scales"), _opt_ptr(bias, f32, "bias"),
        _ptr(lora_a, ad, "lora_a"), _ptr(lora_b, ad, "lora_b"),
        _code(lora_a, "lora_a", ("fp16", "bf16")), na, r,
        _opt_ptr(adapter_scales, f32, "adapter_scales"), _opt_ptr(ranks, i32, "ranks"),
        _ptr(adapter_ids, i32, "adapter_ids"), _act(activation), _ptr(out, out.dtype, "out"),
        _code(out, "out"), _stream(stream)))
    return out


def q8ta_norm_quantize(x, residual, post_weight, gate, residual_scale, weight, eps, residual_out, codes,
                       scales, stream=None):
    """Norms before and after a block with its gate and scaled residual, and the next projection's codes.

    x and residual [T, N] (fp32, fp16 or bf16, rows may be strided), residual may be None; post_weight
    and weight fp32 [N] or None (no norm of x, or of the sum); gate [T, N] or [1, N] or None;
    residual_out like x, dense, or None: residual_scale * residual + gate * norm(x); codes int8 [T, N]
    and scales fp32 [T]: the norm of that in int8, one scale a token.  Returns codes."""
    torch = _torch()
    xp, xs, xt = _view(x, "x", 2)
    T, N = xs
    rp = gp = None
    rt = gt = (0, 1)
    dtype = x.dtype
    if residual is not None:
        rp, rs, rt = _view(residual, "residual", 2)
        if rs != xs or residual.dtype is not dtype:
            raise ValueError(f"residual must be {dtype} {tuple(xs)} (got {residual.dtype} {tuple(rs)})")
    if gate is not None:
        gp, gs, gt = _view(gate, "gate", 2)
        if gs[1] != N or gs[0] not in (1, T) or gate.dtype is not dtype:
            raise ValueError(f"gate must be {dtype} [{T} or 1, {N}] (got {gate.dtype} {tuple(gs)})")
        if gs[0] == 1:
            gt = (0, 1)
    if (post_weight is not None and post_weight.shape != (N,)) or (weight is not None and weight.shape != (N,)):
        raise ValueError(f"post_weight and weight must be [{N}]")
    if codes.shape != xs or scales.shape != (T,) or (residual_out is not None and residual_out.shape != xs):
        raise ValueError(f"codes and residual_out must be {tuple(xs)} and scales [{T}]")
    f32 = torch.float32
    _check(lib().q8ta_norm_quantize(
        xp, xt[0], rp, rt[0], _code(x, "x"), T, N, _opt_ptr(post_weight, f32, "post_weight"), gp, gt[0],
        residual_scale, _opt_ptr(weight, f32, "weight"), eps,
        _opt_ptr(residual_out, dtype, "residual_out"), _ptr(codes, torch.int8, "codes"),
        _ptr(scales, f32, "scales"), _stream(stream)))
    return codes


def q8ta_quantize_per_token(x, codes, scales, stream=None):
    """x [T, N] (fp32, fp16 or bf16, rows may be strided) in int8 codes [T, N] with one scale a token,
    scales fp32 [T]: max |x| / 127.  Returns codes."""
    torch = _torch()
    xp, xs, xt = _view(x, "x", 2)
    T, N = xs
    if codes.shape != xs or scales.shape != (T,):
        raise ValueError(f"codes must be {tuple(xs)} and scales [{T}] (got {tuple(codes.shape)}, "
                         f"{tuple(scales.shape)})")
    _check(lib().q8ta_quantize_per_token(xp, xt[0], _code(x, "x"), T, N, _ptr(codes, torch.int8, "codes"),
                                         _ptr(scales, torch.float32, "scales"), _stream(stream)))
    return codes


def q8ta_linear_per_token(x, x_scales, weight, weight_scales, bias, activation, out, stream=None):
    """The int8 product with a scale for each token and channel, floating-point out.

    x int8 [M, K], x_scales fp32 [M], weight int8 [N, K], weight_scales fp32 [N], bias fp32 [N] or None;
    activation "none" or "relu"; out [M, N] fp32, fp16 or bf16.  Returns out."""
    torch = _torch()
    xs, wsh = x.shape, weight.shape
    if len(xs) != 2 or len(wsh) != 2 or wsh[1] != xs[1] or out.shape != (xs[0], wsh[0]):
        raise ValueError(f"x [M, K], weight [N, K] and out [M, N] expected (got {tuple(xs)}, {tuple(wsh)}, "
                         f"{tuple(out.shape)})")
    (M, K), N = xs, wsh[0]
    if x_scales.shape != (M,) or weight_scales.shape != (N,) or (bias is not None and bias.shape != (N,)):
        raise ValueError(f"x_scales must be [{M}], weight_scales and bias [{N}]")
    f32, i8 = torch.float32, torch.int8
    _check(lib().q8ta_linear_per_token(
        _ptr(x, i8, "x"), M, K, _ptr(x_scales, f32, "x_scales"), _ptr(weight, i8, "weight"), N,
        _ptr(weight_scales, f32, "weight_scales"), _opt_ptr(bias, f32, "bias"), _act(activation),
        _ptr(out, out.dtype, "out"), _code(out, "out"), _stream(stream)))
    return out


def q8ta_gated_linear(x, x_scales, gate_weight, gate_scales, gate_bias, up_weight, up_scales, up_bias,
                      activation, out, stream=None):
    """The gated feed-forward block's first half: act(x gate^T) * (x up^T) in one launch.

    x int8 [M, K], x_scales fp32 [M]; gate_weight and up_weight int8 [N, K], each with scales fp32 [N]
    and a bias fp32 [N] or None; activation "silu", "gelu", "gelu_tanh" or "relu"; out [M, N] fp32, fp16
    or bf16.  Returns out."""
    torch = _torch()
    xs, wsh = x.shape, gate_weight.shape
    if (len(xs) != 2 or len(wsh) != 2 or wsh[1] != xs[1] or up_weight.shape != wsh or
            out.shape != (xs[0], wsh[0])):
        raise ValueError(f"x [M, K], gate_weight and up_weight [N, K] and out [M, N] expected (got {tuple(xs)}, "
                         f"{tuple(wsh)}, {tuple(up_weight.shape)}, {tuple(out.shape)})")
    (M, K), N = xs, wsh[0]
    if x_scales.shape != (M,):
        raise ValueError(f"x_scales must be [{M}] (got {tuple(x_scales.shape)})")
    if (gate_scales.shape != (N,) or up_scales.shape != (N,) or
            (gate_bias is not None and gate_bias.shape != (N,)) or
            (up_bias is not None and up_bias.shape != (N,))):
        raise ValueError(f"gate_scales, gate_bias, up_scales and up_bias must be [{N}]")
    f32, i8 = torch.float32, torch.int8
    _check(lib().q8ta_gated_linear(
        _ptr(x, i8, "x"), M, K, _ptr(x_scales, f32, "x_scales"), _ptr(gate_weight, i8, "gate_weight"),
        _ptr(gate_scales, f32, "gate_scales"), _opt_ptr(gate_bias, f32, "gate_bias"),
        _ptr(up_weight, i8, "up_weight"), _ptr(up_scales, f32, "up_scales"),
        _opt_ptr(up_bias, f32, "up_bias"), N, _act(activation), _ptr(out, out.dtype, "out"),
        _code(out, "out"), _stream(stream)))
    return out


def q8ta_verify_drafts(logits, draft_logits, ids, counts, mask, temperature, draft_temperature, u, path,
                       accepted, next_ids, stream=None):
    """Which drafted tokens the target keeps, from given random numbers, and the token after them.

    logits [B, T, V] (fp32, fp16 or bf16, any outer strides): the target's after each token of a chain or
    tree, ids int32 [B, T] (token 0: the last one known), counts and mask as for q8ta_tree_attention;
    draft_logits [B, T - 1, V] or None: what the drafts of a chain were drawn from (None: they were not
    drawn); temperature and draft_temperature fp32 [B] (the second may be None: the first); u fp32 [B, T]:
    u[:, i] keeps token i, u[:, 0] draws the next one.  path int32 [B, T]: the kept tokens' places, then -1,
    accepted int32 [B]: their number, next_ids int32 [B].  Returns next_ids."""
    torch = _torch()
    lp, ls, lt = _view(logits, "logits", 3)
    B, T, V = ls
    dp, dt = None, (0, 0, 1)
    if draft_logits is not None:
        dp, ds, dt = _view(draft_logits, "draft_logits", 3)
        if ds != (B, T - 1, V) or draft_logits.dtype is not logits.dtype:
            raise ValueError(f"draft_logits must be {logits.dtype} [{B}, {T - 1}, {V}] (got "
                             f"{draft_logits.dtype} {tuple(ds)})")
        dp = dp or lp   # (no rows of a single token's chain: a pointer that is not read)
    each, one = (B, T), (B,)
    if (ids.shape != each or u.shape != each or path.shape != each or temperature.shape != one or
            accepted.shape != one or next_ids.shape != one or (counts is not None and counts.shape != one) or
            (mask is not None and mask.shape != each) or
            (draft_temperature is not None and draft_temperature.shape != one)):
        raise ValueError(f"ids, mask, u and path must be {list(each)}, counts, both temperatures, accepted and "
                         f"next_ids {list(one)}")
    f32, i32 = torch.float32, torch.int32
    _check(lib().q8ta_verify_drafts(
        lp, lt[0], lt[1], dp, dt[0], dt[1], _code(logits, "logits"), B, T, V, _ptr(ids, i32, "ids"),
        _opt_ptr(counts, i32, "counts"), _opt_ptr(mask, torch.int64, "mask"),
        _ptr(temperature, f32, "temperature"), _opt_ptr(draft_temperature, f32, "draft_temperature"),
        _ptr(u, f32, "u"), _ptr(path, i32, "path"), _ptr(accepted, i32, "accepted"),
        _ptr(next_ids, i32, "next_ids"), _stream(stream)))
    return next_ids


def _table(table, lens, refs):
    """Pointers and sizes of a block table, its requests' rows and its pages' holders."""
    torch = _torch()
    i32 = torch.int32
    ts, ps = table.shape, refs.shape
    if len(ts) != 2 or lens.shape != (ts[0],) or len(ps) != 1:
        raise ValueError("table [requests, table_pages], lens [requests] and refs [pages] expected")
    return (_ptr(table, i32, "table"), ts[0], ts[1], _ptr(lens, i32, "lens"), _ptr(refs, i32, "refs"), ps[0],
            i32)


def _each(n, **lists):
    for name, t in lists.items():
        if t is not None and t.shape != (n,):
            raise ValueError(f"{name} must be [{n}] (got {tuple(t.shape)})")


def q8ta_pages_take(table, lens, page_size, more, refs, granted, stream=None):
    """The lowest free pages for more [R] rows behind each request's lens.

    table int32 [R, table_pages], lens, more and granted int32 [R], refs int32 [pages]: how many tables
    hold each page (0: free).  granted: 1 where a request got what it asked for.  A request cut back to a row
    inside a page that others hold has to go on as a fork of itself (q8ta_pages_release).  Returns table."""
    tp, R, width, lp, rp, pages, i32 = _table(table, lens, refs)
    _each(R, more=more, granted=granted)
    _check(lib().q8ta_pages_take(tp, R, width, page_size, lp, _ptr(more, i32, "more"), rp, pages,
                                 _ptr(granted, i32, "granted"), _stream(stream)))
    return table


def q8ta_pages_fork(table, lens, page_size, src, dst, refs, granted, copy_src, copy_dst, copy_rows,
                    stream=None):
    """Request dst[i] becomes a copy of request src[i]: whole pages shared, a page of its own for the rest.

    All int32: table [R, table_pages], lens [R], refs [pages]; src, dst and the outputs granted, copy_src,
    copy_dst and copy_rows [n]: what q8ta_pages_copy has to copy in each layer's cache.  Returns table."""
    tp, R, width, lp, rp, pages, i32 = _table(table, lens, refs)
    n = src.shape[0] if src.dim() == 1 else -1
    _each(n, src=src, dst=dst, granted=granted, copy_src=copy_src, copy_dst=copy_dst, copy_rows=copy_rows)
    _check(lib().q8ta_pages_fork(tp, R, width, page_size, lp, _ptr(src, i32, "src"), _ptr(dst, i32, "dst"), n, rp,
                                 pages, _ptr(granted, i32, "granted"), _ptr(copy_src, i32, "copy_src"),
                                 _ptr(copy_dst, i32, "copy_dst"), _ptr(copy_rows, i32, "copy_rows"),
                                 _stream(stream)))
    return table


def q8ta_pages_release(table, lens, page_size, rows, keep, refs, stream=None):
    """Requests rows [n] (None: all) give up their pages behind the first keep [n] rows (None: all pages).

    All int32: table [R, table_pages], lens [R], refs [pages].  A last page in part stays, also where others
    hold it: rows behind are theirs, and the request goes on as a fork of itself into a free one.  Returns table."""
    tp, R, width, lp, rp, pages, i32 = _table(table, lens, refs)
    n = R if rows is None else (rows.shape[0] if rows.dim() == 1 else -1)
    _each(n, rows=rows, keep=keep)
    _check(lib().q8ta_pages_release(tp, R, width, page_size, lp, _opt_ptr(rows, i32, "rows"),
                                    _opt_ptr(keep, i32, "keep"), n, rp, pages, _stream(stream)))
    return table


def _cache(cache, cache_scales):
    torch = _torch()
    cs = cache.shape
    if len(cs) != 5 or cs[1] != 2 or cs[:4] != cache_scales.shape:
        raise ValueError("cache [pages, 2, kv_heads, page, dim] and cache_scales [pages, 2, "
                         "kv_heads, page] expected")
    return (_ptr(cache, torch.int8, "cache"), _ptr(cache_scales, torch.float32, "cache_scales"), cs[0], cs[3],
            cs[2], cs[4])


def q8ta_pages_copy(cache, cache_scales, src, dst, rows=None, stream=None):
    """Pages src [n] of the int8 cache are copied to pages dst [n] (int32, negative: none), of each the
    first rows [n] rows, or all.  Returns cache."""
    i32 = _torch().int32
    args = _cache(cache, cache_scales)
    n = src.shape[0] if src.dim() == 1 else -1
    _each(n, src=src, dst=dst, rows=rows)
    _check(lib().q8ta_pages_copy(*args, _ptr(src, i32, "src"), _ptr(dst, i32, "dst"), _opt_ptr(rows, i32, "rows"),
                                 n, _stream(stream)))
    return cache


def q8ta_cache_compact(cache, cache_scales, table, base, path, counts, stream=None):
    """Row base[b] + path[b, i] of request b moves to row base[b] + i, for i < counts[b].

    cache and cache_scales as q8ta_rope_append fills them, table int32 [B, table_pages], base and counts
    int32 [B], path int32 [B, n], rising (q8ta_verify_drafts' path and accepted).  Rows may move only to pages
    that no other request holds.  Returns cache."""
    i32 = _torch().int32
    args = _cache(cache, cache_scales)
    ts, ps = table.shape, path.shape
    if len(ts) != 2 or len(ps) != 2 or ps[0] != ts[0]:
        raise ValueError("table [B, table_pages] and path [B, n] expected")
    _each(ts[0], base=base, counts=counts)
    _check(lib().q8ta_cache_compact(*args, _ptr(table, i32, "table"), ts[0], ts[1], _ptr(base, i32, "base"),
                                    _ptr(path, i32, "path"), ps[1], _ptr(counts, i32, "counts"),
                                    _stream(stream)))
    return cache


__all__ = [
    "Q8taError", "lib", "q8ta_last_error", "q8ta_quantize_per_tensor", "q8ta_dequantize_per_tensor",
    "q8ta_linear", "q8ta_linear_gemv", "q8ta_linear_dq", "q8ta_linear_acc", "q8ta_conv2d_transposed",
    "q8ta_quantize_linear", "q8ta_quantize_linear_dq",
    "q8ta_weight_sums", "q8ta_linear_presummed", "q8ta_linear_dq_presummed",
    "q8ta_weight_prepacked_bytes", "q8ta_weight_prepack", "q8ta_linear_prepacked",
    "q8ta_linear_dq_prepacked",
    "q8ta_conv2d_transposed_acc", "q8ta_quantize_conv2d_transposed", "q8ta_conv2d",
    "q8ta_conv2d_acc", "q8ta_conv2d_transposed_weight_prepacked_bytes",
    "q8ta_conv2d_transposed_weight_prepack", "q8ta_conv2d_transposed_prepacked",
    "q8ta_quantize_conv2d_transposed_prepacked",
    "q8ta_linear_lora", "q8ta_rope_append", "q8ta_tree_attention", "q8ta_sample",
    "q8ta_norm_quantize", "q8ta_quantize_per_token", "q8ta_linear_per_token", "q8ta_gated_linear",
    "q8ta_verify_drafts", "q8ta_pages_take", "q8ta_pages_fork", "q8ta_pages_release", "q8ta_pages_copy",
    "q8ta_cache_compact",
]
