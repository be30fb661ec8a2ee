"""Python binding of libloco (include/loco.h): argument marshalling only.

Every function has the name of the C entry point it calls and does nothing
but turn tensors (or raw integer device addresses) into pointers and sizes,
pick the current torch CUDA stream, and raise ``LocoError`` on a non-OK
status.  All arithmetic runs in the CUDA kernels of ``libloco.so``; there is
no CPU or PyTorch fallback: if the library is missing, importing this module
fails.  The layer calls take torch's memory in one case, for aligned copies of
operands of large products (see ALIGN_WORK); everything else is the caller's.
"""
from __future__ import annotations

import ctypes
import functools
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libloco.so")

LOCO_OK, LOCO_ERR_INVALID_ARG, LOCO_ERR_UNSUPPORTED, LOCO_ERR_MISALIGNED, LOCO_ERR_CUDA = 0, 1, 2, 3, 4
LOCO_F32, LOCO_BF16 = 0, 1
LOCO_SCALE_ABSMAX, LOCO_SCALE_FIXED = 0, 1
LOCO_ACT_NONE, LOCO_ACT_RELU, LOCO_ACT_GELU, LOCO_ACT_GELU_TANH, LOCO_ACT_SILU = 0, 1, 2, 3, 4
LOCO_NORM_LAYER, LOCO_NORM_RMS = 0, 1
LOCO_CKPT_BLOCK = 32
LOCO_STATE_BLOCK = 256
LOCO_STATE_M, LOCO_STATE_V = 0, 1
LOCO_MAX_TOP = 32
LOCO_MAX_DIM = 0x7FFFFFFF
LOCO_MAX_RANKS = 16
LOCO_MAX_N = 1 << 48

EXPORTS = ("loco_num_blocks", "loco_code_bytes", "loco_compress", "loco_compress_e8", "loco_decode_reduce",
           "loco_adam_step", "loco_adam_step_bf16", "loco_sgd_step", "loco_shard_range", "loco_status_string",
           "loco_last_error", "loco_ckpt_code_bytes", "loco_ckpt_scale_bytes", "loco_ckpt_encode", "loco_ckpt_decode",
           "loco_norm_forward", "loco_norm_workspace_bytes", "loco_norm_backward", "loco_linear_align",
           "loco_matrices_overlap", "loco_linear_forward", "loco_linear_backward_input", "loco_linear_workspace_bytes",
           "loco_linear_backward_weight", "loco_linear_timeouts", "loco_join_forward", "loco_join_workspace_bytes",
           "loco_join_backward", "loco_logprob_forward", "loco_logprob_backward", "loco_adam_tensors",
           "loco_adam_state_decode")


class LocoError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        super().__init__(f"{_status_name(status)}: {message}")


class loco_config(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("block", ctypes.c_int32), ("scale_mode", ctypes.c_int32),
                ("fixed_scale", ctypes.c_float), ("beta", ctypes.c_float), ("err_scale_mult", ctypes.c_float),
                ("reset_period", ctypes.c_int64)]


class loco_adam_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("bias_correction", ctypes.c_int32), ("eps_inside_sqrt", ctypes.c_int32)]


class loco_norm_config(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("eps", ctypes.c_float), ("x_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32)]


class loco_linear_config(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("param_dtype", ctypes.c_int32)]


class loco_join_config(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("post", ctypes.c_int32), ("eps", ctypes.c_float),
                ("residual_scale", ctypes.c_float), ("block_scale", ctypes.c_float), ("x_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32)]


class loco_adam_tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_steps", ctypes.c_void_p), ("v_steps", ctypes.c_void_p), ("param_bf16", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("lr_scale", ctypes.c_float), ("decay_scale", ctypes.c_float)]


class loco_adam_tensors_config(ctypes.Structure):
    _fields_ = [("state_bits", ctypes.c_int32), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("dither", ctypes.c_uint32)]


def make_config(bits=4, block=256, beta=0.9, err_scale_mult=4.0, reset_period=0, fixed_scale=None):
    return loco_config(bits, block, LOCO_SCALE_FIXED if fixed_scale is not None else LOCO_SCALE_ABSMAX,
                       float(fixed_scale or 0.0), float(beta), float(err_scale_mult), int(reset_period))


def make_adam(lr=1e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0, bias_correction=True,
              eps_inside_sqrt=False):
    return loco_adam_hparams(lr, beta1, beta2, eps, weight_decay, int(bias_correction), int(eps_inside_sqrt))


def make_norm(kind=LOCO_NORM_LAYER, eps=1e-5):
    """A norm's kind and eps; the calls fill in the types of the tensors they are given."""
    return loco_norm_config(kind, float(eps), LOCO_F32, LOCO_F32, LOCO_F32, LOCO_F32)


def make_join(kind=LOCO_NORM_LAYER, eps=1e-5, post=True, residual_scale=1.0, block_scale=1.0):
    """A join's norms and scales; the calls fill in the types of the tensors they are given."""
    return loco_join_config(kind, int(post), float(eps), float(residual_scale), float(block_scale), LOCO_F32, LOCO_F32,
                            LOCO_F32, LOCO_F32)


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built: run bit_gradient_compression_gb300.build.build() "
                      "(nvcc, sm_103a); there is no fallback implementation")

lib = ctypes.CDLL(LIB_PATH)
_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
lib.loco_num_blocks.argtypes = [_i64, _i32]
lib.loco_num_blocks.restype = _i64
lib.loco_code_bytes.argtypes = [_i64, _i32, _i32]
lib.loco_code_bytes.restype = _i64
lib.loco_compress.argtypes = [ctypes.POINTER(loco_config), _vp, _i32, _vp, _i64, _i64, _vp, _vp, _vp]
lib.loco_compress.restype = ctypes.c_int
lib.loco_compress_e8.argtypes = [ctypes.POINTER(loco_config), _vp, _i32, _vp, _vp, _i64, _i64, _vp, _vp, _vp]
lib.loco_compress_e8.restype = ctypes.c_int
lib.loco_decode_reduce.argtypes = [ctypes.POINTER(loco_config), _vp, _vp, _i32, _i64, _vp, _vp]
lib.loco_decode_reduce.restype = ctypes.c_int
lib.loco_adam_step.argtypes = [ctypes.POINTER(loco_config), _vp, _vp, _i32, _i64, _vp, _vp, _vp,
                               ctypes.POINTER(loco_adam_hparams), _i64, _vp]
lib.loco_adam_step.restype = ctypes.c_int
lib.loco_adam_step_bf16.argtypes = [ctypes.POINTER(loco_config), _vp, _vp, _i32, _i64, _vp, _vp, _vp, _vp,
                                    ctypes.POINTER(loco_adam_hparams), _i64, _vp]
lib.loco_adam_step_bf16.restype = ctypes.c_int
lib.loco_sgd_step.argtypes = [ctypes.POINTER(loco_config), _vp, _vp, _i32, _i64, _vp, _vp, ctypes.c_float, _vp]
lib.loco_sgd_step.restype = ctypes.c_int
lib.loco_shard_range.argtypes = [_i64, _i32, _i32, _i32, ctypes.POINTER(_i64), ctypes.POINTER(_i64)]
lib.loco_shard_range.restype = ctypes.c_int
_norm, _lin = ctypes.POINTER(loco_norm_config), ctypes.POINTER(loco_linear_config)
lib.loco_ckpt_code_bytes.argtypes = [_i64, _i64]
lib.loco_ckpt_code_bytes.restype = _i64
lib.loco_ckpt_scale_bytes.argtypes = [_i64, _i64]
lib.loco_ckpt_scale_bytes.restype = _i64
lib.loco_ckpt_encode.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp]
lib.loco_ckpt_encode.restype = ctypes.c_int
lib.loco_ckpt_decode.argtypes = [_vp, _vp, _i64, _i64, _i32, _vp, _vp, _i32, _vp, _i32, _i64, _vp]
lib.loco_ckpt_decode.restype = ctypes.c_int
lib.loco_norm_forward.argtypes = [_norm, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp]
lib.loco_norm_forward.restype = ctypes.c_int
lib.loco_norm_workspace_bytes.argtypes = [_i64, _i64]
lib.loco_norm_workspace_bytes.restype = _i64
lib.loco_norm_backward.argtypes = [_norm, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp,
                                   _i64, _vp, _vp, _vp, _i64, _vp]
lib.loco_norm_backward.restype = ctypes.c_int
lib.loco_linear_align.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _vp]
lib.loco_linear_align.restype = ctypes.c_int
lib.loco_matrices_overlap.argtypes = [_vp, _i64, _i64, _i64, _i32, _vp, _i64, _i64, _i64, _i32]
lib.loco_matrices_overlap.restype = _i32
lib.loco_linear_forward.argtypes = [_lin, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp,
                                    _vp]
lib.loco_linear_forward.restype = ctypes.c_int
lib.loco_linear_backward_input.argtypes = [_lin, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp,
                                           _i64, _vp]
lib.loco_linear_backward_input.restype = ctypes.c_int
lib.loco_linear_workspace_bytes.argtypes = [_i64]
lib.loco_linear_workspace_bytes.restype = _i64
lib.loco_linear_backward_weight.argtypes = [_lin, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp,
                                            _i64, _vp, _vp, _i64, _vp]
lib.loco_linear_backward_weight.restype = ctypes.c_int
lib.loco_linear_timeouts.argtypes = [ctypes.POINTER(_i64)]
lib.loco_linear_timeouts.restype = ctypes.c_int
_join = ctypes.POINTER(loco_join_config)
lib.loco_join_forward.argtypes = [_join, _vp, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp,
                                  _i64, _vp, _vp]
lib.loco_join_forward.restype = ctypes.c_int
lib.loco_join_workspace_bytes.argtypes = [_i64, _i64]
lib.loco_join_workspace_bytes.restype = _i64
lib.loco_join_backward.argtypes = [_join, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _vp,
                                   _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp]
lib.loco_join_backward.restype = ctypes.c_int
lib.loco_logprob_forward.argtypes = [_vp, _i32, _i64, _i64, _i64, ctypes.c_float, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp]
lib.loco_logprob_forward.restype = ctypes.c_int
lib.loco_logprob_backward.argtypes = [_vp, _i32, _i64, _i64, _i64, ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp]
lib.loco_logprob_backward.restype = ctypes.c_int
lib.loco_adam_tensors.argtypes = [ctypes.POINTER(loco_adam_tensors_config), ctypes.POINTER(loco_adam_tensor), _i32,
                                  ctypes.POINTER(loco_adam_hparams), _i64, _vp, _vp]
lib.loco_adam_tensors.restype = ctypes.c_int
lib.loco_adam_state_decode.argtypes = [_i32, _vp, _vp, _i64, _vp, _i32, _vp]
lib.loco_adam_state_decode.restype = ctypes.c_int
lib.loco_status_string.argtypes = [ctypes.c_int]
lib.loco_status_string.restype = ctypes.c_char_p
lib.loco_last_error.argtypes = []
lib.loco_last_error.restype = ctypes.c_char_p


def _status_name(s: int) -> str:
    return lib.loco_status_string(s).decode()


def _check(status: int):
    if status != LOCO_OK:
        raise LocoError(status, lib.loco_last_error().decode())


def _addr(x) -> int:
    """Device address of a tensor (must be contiguous) or an integer address."""
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    if not x.is_contiguous():
        raise ValueError("tensors passed to libloco must be contiguous")
    return x.data_ptr()


_raw_stream = None  # torch's stream handle of a device, without a Stream object around it; set once CUDA is there


def _stream(stream) -> int:
    global _raw_stream
    if stream is None:
        import torch
        if _raw_stream is None:
            if not torch.cuda.is_available():
                return 0
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
                lambda device: torch.cuda.current_stream(device).cuda_stream)
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _grad_dtype(grad, grad_dtype):
    if grad_dtype is not None:
        return grad_dtype
    import torch
    if grad.dtype == torch.bfloat16:
        return LOCO_BF16
    if grad.dtype == torch.float32:
        return LOCO_F32
    raise ValueError(f"gradient dtype {grad.dtype} is not supported (float32 or bfloat16)")


def loco_num_blocks(n: int, block: int) -> int:
    return lib.loco_num_blocks(n, block)


def loco_code_bytes(n: int, bits: int, block: int) -> int:
    return lib.loco_code_bytes(n, bits, block)


def loco_compress(cfg: loco_config, grad, err, step: int, codes, scales, *, n: int | None = None,
                  grad_dtype: int | None = None, stream=None):
    """Sender step (compensate, quantise, pack, error update) on one bucket."""
    if n is None:
        n = grad.numel()
    _check(lib.loco_compress(ctypes.byref(cfg), _addr(grad), _grad_dtype(grad, grad_dtype), _addr(err),
                             n, step, _addr(codes), _addr(scales), _stream(stream)))


def loco_compress_e8(cfg: loco_config, grad, err_codes, err_steps, step: int, codes, scales, *,
                     n: int | None = None, grad_dtype: int | None = None, stream=None):
    """Sender step with the error kept as int8 codes + one step per block (updated in place)."""
    if n is None:
        n = grad.numel()
    _check(lib.loco_compress_e8(ctypes.byref(cfg), _addr(grad), _grad_dtype(grad, grad_dtype), _addr(err_codes),
                                _addr(err_steps), n, step, _addr(codes), _addr(scales), _stream(stream)))


def _rank_arrays(codes, scales):
    W = len(codes)
    if len(scales) != W:
        raise ValueError("codes and scales must list the same ranks")
    ca = (ctypes.c_void_p * max(W, 1))(*[_addr(c) for c in codes])
    sa = (ctypes.c_void_p * max(W, 1))(*[_addr(s) for s in scales])
    return W, ca, sa


def loco_decode_reduce(cfg: loco_config, codes, scales, n: int, mean, *, stream=None):
    """Average of W ranks' decoded buckets (fp32), written to mean."""
    W, ca, sa = _rank_arrays(codes, scales)
    _check(lib.loco_decode_reduce(ctypes.byref(cfg), ca, sa, W, n, _addr(mean), _stream(stream)))


def loco_adam_step(cfg: loco_config, codes, scales, n: int, param, m, v, hp: loco_adam_hparams, t: int, *,
                   stream=None):
    """Decode-reduce fused with one Adam(W) update of param, m, v (in place)."""
    W, ca, sa = _rank_arrays(codes, scales)
    _check(lib.loco_adam_step(ctypes.byref(cfg), ca, sa, W, n, _addr(param), _addr(m), _addr(v),
                              ctypes.byref(hp), t, _stream(stream)))


def loco_adam_step_bf16(cfg: loco_config, codes, scales, n: int, param, m, v, param_bf16, hp: loco_adam_hparams,
                        t: int, *, stream=None):
    """loco_adam_step that also writes bf16(param) into param_bf16."""
    W, ca, sa = _rank_arrays(codes, scales)
    _check(lib.loco_adam_step_bf16(ctypes.byref(cfg), ca, sa, W, n, _addr(param), _addr(m), _addr(v),
                                   _addr(param_bf16), ctypes.byref(hp), t, _stream(stream)))


def loco_sgd_step(cfg: loco_config, codes, scales, n: int, param, lr: float, *, param_bf16=None, stream=None):
    """Decode-reduce fused with one LoCo-SGD step (param -= lr * mean), optional bf16 copy."""
    W, ca, sa = _rank_arrays(codes, scales)
    _check(lib.loco_sgd_step(ctypes.byref(cfg), ca, sa, W, n, _addr(param), _addr(param_bf16), float(lr),
                             _stream(stream)))


def loco_shard_range(n: int, block: int, W: int, j: int) -> tuple[int, int]:
    """Element range [lo, hi) of shard j of W (the sharded receiver's split of a bucket)."""
    lo, hi = ctypes.c_int64(), ctypes.c_int64()
    _check(lib.loco_shard_range(n, block, W, j, ctypes.byref(lo), ctypes.byref(hi)))
    return lo.value, hi.value


# --------------------------------------------------------------------------
# Layers: norms, linear layers and 8-bit activation checkpoints.  Matrices are
# two-dimensional tensors whose rows are contiguous (any row pitch).
# --------------------------------------------------------------------------

# A linear layer's operand whose rows start on no 16-byte boundary is copied to aligned rows first, in memory
# of torch's allocator, in products of at least this many multiplications (a call for T, N, K = 200, 1000, 1001:
# 18.6 us as they lie, 20.6 us copied; 333, 1407, 2049: 28.0 and 24.8 us; 4095, 4097, 4099: 440 and 144 us), and
# where w is an operand in those over at least this many rows, as a copy of w costs more than reading it once
# (input gradient of 64 rows, 11007, 4097: 47 us as they lie, 61 us copied; of 129, 1407, 2049: 24.7 and 23.9 us).
ALIGN_WORK, ALIGN_ROWS = 1 << 28, 96

# The same marshalling in C (csrc/marshal.c): its functions return the status of the call they made, or
# None where an argument is not as the entry point wants it; the code below then says what is wrong.
try:
    from bit_gradient_compression_gb300 import _marshal
except ImportError:
    class _marshal:  # built without Python's headers
        init = ckpt_encode = ckpt_decode = norm_forward = norm_backward = linear_forward = staticmethod(lambda *a: None)
        linear_backward_input = linear_backward_weight = join_forward = join_backward = logprob_forward = init
        logprob_backward = adam_state_decode = adam_tensors = init

_DTYPES: dict = {}  # torch.dtype -> loco_dtype, filled on first use (torch is imported only then)


def _dtypes():
    import torch
    _DTYPES.update({torch.float32: LOCO_F32, torch.bfloat16: LOCO_BF16})
    _marshal.init(torch.float32, torch.bfloat16, torch.int8, torch.uint8, torch.int64, ALIGN_WORK, ALIGN_ROWS)
    return _DTYPES


def _dtype(t, name: str) -> int:
    d = (_DTYPES or _dtypes()).get(t.dtype)
    if d is None:
        raise ValueError(f"{name}: dtype {t.dtype} is not supported (float32 or bfloat16)")
    return d


def _one_dtype(name: str, *tensors) -> int:
    """The one dtype of the tensors that are given (LOCO_F32 where none is)."""
    first = None
    for t in tensors:
        if t is not None:
            if first is None:
                first = t
            elif t.dtype != first.dtype:
                raise ValueError(f"{name} must have one dtype (got {first.dtype} and {t.dtype})")
    return LOCO_F32 if first is None else _dtype(first, name)


def _mat(t, name: str, rows: int, cols: int):
    """(address, row pitch) of a [rows, cols] matrix; (0, 0) for None."""
    if t is None:
        return 0, 0
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be {(rows, cols)} (got {tuple(t.shape)})")
    pitch, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return t.data_ptr(), (cols if rows <= 1 and pitch < cols else pitch)


def _dims(t, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must be two-dimensional (got {t.dim()} dimensions)")
    return t.shape


def _vec(t, name: str, count: int) -> int:
    """Address of a contiguous vector of count elements; 0 for None."""
    if t is None:
        return 0
    if t.shape != (count,) or (count > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {count} (got {tuple(t.shape)})")
    return t.data_ptr()


def _f32(t, name: str, count: int) -> int:
    if t is not None and (_DTYPES or _dtypes()).get(t.dtype) != LOCO_F32:
        raise ValueError(f"{name} must be torch.float32 (got {t.dtype})")
    return _vec(t, name, count)


def _ckpt(codes, scales, rows: int, cols: int):
    """Addresses of a checkpoint of [rows, cols]: int8 codes and uint8 scales of the sizes the library states."""
    if codes is None and scales is None:
        return 0, 0
    import torch
    nb = -(-cols // LOCO_CKPT_BLOCK)
    for t, name, dtype, size in ((codes, "codes", torch.int8, rows * nb * LOCO_CKPT_BLOCK),
                                 (scales, "scales", torch.uint8, rows * nb)):
        if t is not None and (t.dtype != dtype or t.numel() != size or not t.is_contiguous()):
            raise ValueError(f"{name} must be {size} contiguous {dtype} (got {t.numel()} {t.dtype})")
    return (0 if codes is None else codes.data_ptr()), (0 if scales is None else scales.data_ptr())


def _bf16(t, name: str):
    if t is not None and (_DTYPES or _dtypes()).get(t.dtype) != LOCO_BF16:
        raise ValueError(f"{name}: dtype {t.dtype} is not supported (bfloat16)")


def _workspace(t):
    if t is None:
        return 0, 0
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


@functools.lru_cache(maxsize=256)
def _norm_ref(*fields):
    return ctypes.byref(loco_norm_config(*fields))


@functools.lru_cache(maxsize=256)
def _linear_ref(*fields):
    return ctypes.byref(loco_linear_config(*fields))


def loco_ckpt_code_bytes(rows: int, cols: int) -> int:
    return lib.loco_ckpt_code_bytes(rows, cols)


def loco_ckpt_scale_bytes(rows: int, cols: int) -> int:
    return lib.loco_ckpt_scale_bytes(rows, cols)


def loco_ckpt_encode(x, codes, scales, *, stream=None):
    """8-bit checkpoint of x [rows, cols]: int8 codes [rows, nb*32], uint8 scales [rows, nb], nb = ceil(cols/32)."""
    status = _marshal.ckpt_encode(x, codes, scales, _stream(stream))
    if status is not None:
        return _check(status) if status else None
    rows, cols = _dims(x, "x")
    px, ldx = _mat(x, "x", rows, cols)
    pc, ps = _ckpt(codes, scales, rows, cols)
    _check(lib.loco_ckpt_encode(px, _dtype(x, "x"), ldx, rows, cols, pc, ps, _stream(stream)))


def loco_ckpt_decode(codes, scales, out, *, act: int = LOCO_ACT_NONE, gamma=None, beta=None, stream=None):
    """out [rows, cols] = act(values of the checkpoint * gamma + beta)."""
    status = _marshal.ckpt_decode(codes, scales, out, act, gamma, beta, _stream(stream))
    if status is not None:
        return _check(status) if status else None
    rows, cols = _dims(out, "out")
    po, ldo = _mat(out, "out", rows, cols)
    pc, ps = _ckpt(codes, scales, rows, cols)
    _check(lib.loco_ckpt_decode(pc, ps, rows, cols, act, _vec(gamma, "gamma", cols), _vec(beta, "beta", cols),
                                _one_dtype("gamma and beta", gamma, beta), po, _dtype(out, "out"), ldo,
                                _stream(stream)))


def loco_norm_forward(cfg: loco_norm_config, x, gamma, beta, y, *, mean=None, rstd=None, codes=None, scales=None,
                      stream=None):
    """y = norm(x) * gamma + beta per row; optionally its statistics and an 8-bit checkpoint of the normalised rows."""
    status = _marshal.norm_forward(cfg.kind, cfg.eps, x, gamma, beta, y, mean, rstd, codes, scales, _stream(stream))
    if status is not None:
        return _check(status) if status else None
    rows, cols = _dims(x, "x")
    px, ldx = _mat(x, "x", rows, cols)
    py, ldy = _mat(y, "y", rows, cols)
    pc, ps = _ckpt(codes, scales, rows, cols)
    c = _norm_ref(cfg.kind, cfg.eps, _dtype(x, "x"), _dtype(y, "y"), _one_dtype("gamma and beta", gamma, beta), LOCO_F32)
    _check(lib.loco_norm_forward(c, px, ldx, rows, cols, _vec(gamma, "gamma", cols), _vec(beta, "beta", cols), py, ldy,
                                 _f32(mean, "mean", rows), _f32(rstd, "rstd", rows), pc, ps, _stream(stream)))


def loco_norm_workspace_bytes(rows: int, cols: int) -> int:
    return lib.loco_norm_workspace_bytes(rows, cols)


def loco_norm_backward(cfg: loco_norm_config, dy, gamma, rstd, dx, *, x=None, mean=None, codes=None, scales=None,
                       residual=None, dgamma=None, dbeta=None, workspace=None, stream=None):
    """Gradients of loco_norm_forward, from x or from the checkpoint of the normalised rows."""
    status = _marshal.norm_backward(cfg.kind, cfg.eps, dy, gamma, rstd, dx, x, mean, codes, scales, residual, dgamma,
                                    dbeta, workspace, _stream(stream))
    if status is not None:
        return _check(status) if status else None
    rows, cols = _dims(dy, "dy")
    pdy, lddy = _mat(dy, "dy", rows, cols)
    px, ldx = _mat(x, "x", rows, cols)
    pr, ldr = _mat(residual, "residual", rows, cols)
    pdx, lddx = _mat(dx, "dx", rows, cols)
    pc, ps = _ckpt(codes, scales, rows, cols)
    pw, nw = _workspace(workspace)
    c = _norm_ref(cfg.kind, cfg.eps, _one_dtype("x, residual and dx", x, residual, dx), _dtype(dy, "dy"),
                  _one_dtype("gamma", gamma), _one_dtype("dgamma and dbeta", dgamma, dbeta))
    _check(lib.loco_norm_backward(c, pdy, lddy, px, ldx, pc, ps, _f32(mean, "mean", rows), _f32(rstd, "rstd", rows),
                                  rows, cols, _vec(gamma, "gamma", cols), pr, ldr, pdx, lddx,
                                  _vec(dgamma, "dgamma", cols), _vec(dbeta, "dbeta", cols), pw, nw, _stream(stream)))


def loco_linear_align(src, dst, *, stream=None):
    """dst [rows, cols] = src, both bf16; the rows of dst start on 16-byte boundaries and are followed by zeros up to
    the next multiple of 8 columns."""
    rows, cols = _dims(src, "src")
    _bf16(src, "src")
    _bf16(dst, "dst")
    ps, lds = _mat(src, "src", rows, cols)
    pd, ldd = _mat(dst, "dst", rows, cols)
    _check(lib.loco_linear_align(ps, lds, rows, cols, pd, ldd, _stream(stream)))


def _scratch(nbytes: int):
    """Memory for a call on the current stream; None if there is none left."""
    import torch
    try:
        return torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    except torch.cuda.OutOfMemoryError:
        return None


def loco_matrices_overlap(a: int, lda: int, rows_a: int, cols_a: int, bytes_a: int,
                          b: int, ldb: int, rows_b: int, cols_b: int, bytes_b: int) -> bool:
    """Whether two matrices, given by their addresses, row pitches, sizes and element sizes, may share a byte."""
    return bool(lib.loco_matrices_overlap(a, lda, rows_a, cols_a, bytes_a, b, ldb, rows_b, cols_b, bytes_b))


def _output(t, p: int, ld: int, rows: int, cols: int):
    """An output as loco_matrices_overlap takes a matrix (one that is not there has address 0)."""
    return p, ld, rows, cols, 1 if t is None else t.element_size()


def _row(p: int, size: int):
    """A contiguous output of `size` bytes as a matrix of one row."""
    return p, size, 1, size, 1


def _operand(t, name: str, rows: int, cols: int, product, stream: int, outputs, least: int = 0):
    """(address, row pitch, what keeps it) of an operand of a product of T, N, K, in aligned rows where that pays.
    One that an output overlaps (each as loco_matrices_overlap takes it) stays as it lies: the call then refuses it."""
    p, ld = _mat(t, name, rows, cols)
    T, N, K = product
    if (t is None or T < least or T * N * K < ALIGN_WORK or not t.is_cuda
            or (p % 16 == 0 and (rows <= 1 or ld % 8 == 0))
            or any(loco_matrices_overlap(p, ld, rows, cols, 2, *o) for o in outputs)):
        return p, ld, None
    import torch
    pitch = -(-cols // 8) * 8
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, t.device)):  # memory comes and goes in its order
        copy = _scratch(rows * pitch * 2)
    if copy is None:
        return p, ld, None
    _check(lib.loco_linear_align(p, ld, rows, cols, copy.data_ptr(), pitch, stream))
    return copy.data_ptr(), pitch, copy


def loco_linear_forward(x, w, y, *, act: int = LOCO_ACT_NONE, bias=None, residual=None, codes=None, scales=None,
                        stream=None):
    """y = act(x w^T + bias) + residual; optionally an 8-bit checkpoint of the pre-activation.  x, w bf16."""
    status = _marshal.linear_forward(x, w, y, act, bias, residual, codes, scales, _stream(stream),
                                     _scratch if stream is None else None)
    if status is not None:
        return _check(status) if status else None
    T, K = _dims(x, "x")
    N, _ = _dims(w, "w")
    _bf16(x, "x")
    _bf16(w, "w")
    st = _stream(stream)
    pr, ldr = _mat(residual, "residual", T, N)
    py, ldy = _mat(y, "y", T, N)
    pc, ps = _ckpt(codes, scales, T, N)
    c, pb = _linear_ref(act, _one_dtype("y and residual", y, residual), _one_dtype("bias", bias)), _vec(bias, "bias", N)
    outs = (_output(y, py, ldy, T, N), _row(pc, loco_ckpt_code_bytes(T, N)), _row(ps, loco_ckpt_scale_bytes(T, N)))
    px, ldx, _x = _operand(x, "x", T, K, (T, N, K), st, outs, ALIGN_ROWS)
    pw, ldw, _w = _operand(w, "w", N, K, (T, N, K), st, outs, ALIGN_ROWS)
    _check(lib.loco_linear_forward(c, px, ldx, pw, ldw, pb, pr, ldr, T, N, K, py, ldy, pc, ps, st))


def loco_linear_backward_input(dy, w, dx, *, act: int = LOCO_ACT_NONE, codes=None, scales=None, residual=None,
                               stream=None):
    """dx = (dy w) * act'(z) + residual, z from the checkpoint of the layer below's pre-activation.  dy, w bf16."""
    status = _marshal.linear_backward_input(dy, w, dx, act, codes, scales, residual, _stream(stream),
                                            _scratch if stream is None else None)
    if status is not None:
        return _check(status) if status else None
    T, N = _dims(dy, "dy")
    _, K = _dims(w, "w")
    _bf16(dy, "dy")
    _bf16(w, "w")
    st = _stream(stream)
    pr, ldr = _mat(residual, "residual", T, K)
    pdx, lddx = _mat(dx, "dx", T, K)
    pc, ps = _ckpt(codes, scales, T, K)
    c = _linear_ref(act, _one_dtype("dx and residual", dx, residual), LOCO_F32)
    outs = (_output(dx, pdx, lddx, T, K),)
    pdy, lddy, _dy = _operand(dy, "dy", T, N, (T, N, K), st, outs, ALIGN_ROWS)
    pw, ldw, _w = _operand(w, "w", N, K, (T, N, K), st, outs, ALIGN_ROWS)
    _check(lib.loco_linear_backward_input(c, pdy, lddy, pw, ldw, pc, ps, pr, ldr, T, N, K, pdx, lddx, st))


def loco_linear_workspace_bytes(N: int) -> int:
    return lib.loco_linear_workspace_bytes(N)


def loco_linear_backward_weight(dy, dw, *, x=None, codes=None, scales=None, gamma=None, beta=None, db=None,
                                workspace=None, stream=None):
    """dw = dy^T x, db = column sums of dy; x [T, K] bf16, or gamma * (values of a checkpoint) + beta."""
    status = _marshal.linear_backward_weight(dy, dw, x, codes, scales, gamma, beta, db, workspace,
                                             _stream(stream), _scratch if stream is None else None)
    if status is not None:
        return _check(status) if status else None
    T, N = _dims(dy, "dy")
    _, K = _dims(dw, "dw")
    _bf16(dy, "dy")
    _bf16(x, "x")
    st = _stream(stream)
    pdw, lddw = _mat(dw, "dw", N, K)
    pc, ps = _ckpt(codes, scales, T, K)
    pg, pb, pdb, (pw, nw) = _vec(gamma, "gamma", K), _vec(beta, "beta", K), _vec(db, "db", N), _workspace(workspace)
    c = _linear_ref(LOCO_ACT_NONE, _one_dtype("dw and db", dw, db), _one_dtype("gamma and beta", gamma, beta))
    outs = (_output(dw, pdw, lddw, N, K), _row(pdb, N * dw.element_size()),
            _row(pw, loco_linear_workspace_bytes(N) if x is None and beta is not None else 0))
    pdy, lddy, _dy = _operand(dy, "dy", T, N, (T, N, K), st, outs)
    px, ldx, _x = _operand(x, "x", T, K, (T, N, K), st, outs)
    _check(lib.loco_linear_backward_weight(c, pdy, lddy, px, ldx, pc, ps, pg, pb, T, N, K, pdw, lddw, pdb, pw, nw, st))


def loco_linear_timeouts() -> int:
    """Waits that the linear-layer and join kernels gave up on the current device (0 unless something is wrong);
    synchronises."""
    v = ctypes.c_int64()
    _check(lib.loco_linear_timeouts(ctypes.byref(v)))
    return v.value


# --------------------------------------------------------------------------
# Joins of blocks, log probabilities of given tokens, AdamW on many tensors.
# --------------------------------------------------------------------------

@functools.lru_cache(maxsize=256)
def _join_ref(*fields):
    return ctypes.byref(loco_join_config(*fields))


def _join_cfg(cfg, x: int, y: int, param: int, grad: int):
    return _join_ref(cfg.kind, cfg.post, cfg.eps, cfg.residual_scale, cfg.block_scale, x, y, param, grad)


def _stats(t, rows: int) -> int:
    if t is None:
        return 0
    if (_DTYPES or _dtypes()).get(t.dtype) != LOCO_F32 or t.shape != (4, rows) or not t.is_contiguous():
        raise ValueError(f"stats must be contiguous torch.float32 {(4, rows)} (got {t.dtype} {tuple(t.shape)})")
    return t.data_ptr()


def loco_join_forward(cfg: loco_join_config, x, y, h, u=None, *, gamma=None, beta=None, post_gamma=None, post_beta=None,
                      gate=None, row_gate=None, stats=None, stream=None):
    """h = residual_scale x + block_scale row_gate gate norm(y), u = norm(h): both norms with their own parameters
    (without post, y itself; without u, no second norm).  stats [4, rows]: what the backward pass needs."""
    status = _marshal.join_forward(cfg.kind, cfg.post, cfg.eps, cfg.residual_scale, cfg.block_scale, x, y, h, u, gamma, beta,
                                   post_gamma, post_beta, gate, row_gate, stats, _stream(stream))
    if status is not None:
        return _check(status) if status else None
    rows, cols = _dims(x, "x")
    px, ldx = _mat(x, "x", rows, cols)
    py, ldy = _mat(y, "y", rows, cols)
    ph, ldh = _mat(h, "h", rows, cols)
    pu, ldu = _mat(u, "u", rows, cols)
    c = _join_cfg(cfg, _one_dtype("x and h", x, h), _one_dtype("y and u", y, u),
                  _one_dtype("gammas, betas and gate", gamma, beta, post_gamma, post_beta, gate), LOCO_F32)
    _check(lib.loco_join_forward(c, px, ldx, py, ldy, rows, cols, _vec(post_gamma, "post_gamma", cols),
                                 _vec(post_beta, "post_beta", cols), _vec(gate, "gate", cols),
                                 _f32(row_gate, "row_gate", rows), _vec(gamma, "gamma", cols), _vec(beta, "beta", cols),
                                 ph, ldh, pu, ldu, _stats(stats, rows), _stream(stream)))


def loco_join_workspace_bytes(rows: int, cols: int) -> int:
    return lib.loco_join_workspace_bytes(rows, cols)


def loco_join_backward(cfg: loco_join_config, dh, du, h, y, stats, dx, dy, *, gamma=None, post_gamma=None, post_beta=None,
                       gate=None, row_gate=None, dgamma=None, dbeta=None, dpost_gamma=None, dpost_beta=None, dgate=None,
                       drow_gate=None, workspace=None, stream=None):
    """Gradients of loco_join_forward: dx of the stream, dy of the block's output, and those of the parameters that
    are given.  dh or du may be None (zeros)."""
    status = _marshal.join_backward(cfg.kind, cfg.post, cfg.eps, cfg.residual_scale, cfg.block_scale, dh, du, h, y, stats,
                                    dx, dy, gamma, post_gamma, post_beta, gate, row_gate, dgamma, dbeta, dpost_gamma,
                                    dpost_beta, dgate, drow_gate, workspace, _stream(stream))
    if status is not None:
        return _check(status) if status else None
    rows, cols = _dims(dx, "dx")
    pdh, lddh = _mat(dh, "dh", rows, cols)
    pdu, lddu = _mat(du, "du", rows, cols)
    ph, ldh = _mat(h, "h", rows, cols)
    py, ldy = _mat(y, "y", rows, cols)
    pdx, lddx = _mat(dx, "dx", rows, cols)
    pdy, lddy = _mat(dy, "dy", rows, cols)
    pw, nw = _workspace(workspace)
    c = _join_cfg(cfg, _one_dtype("dh, h and dx", dh, h, dx), _one_dtype("du, y and dy", du, y, dy),
                  _one_dtype("gammas, betas and gate", gamma, post_gamma, post_beta, gate),
                  _one_dtype("the parameters' gradients", dgamma, dbeta, dpost_gamma, dpost_beta, dgate))
    _check(lib.loco_join_backward(c, pdh, lddh, pdu, lddu, ph, ldh, py, ldy, _stats(stats, rows), rows, cols,
                                  _vec(post_gamma, "post_gamma", cols), _vec(post_beta, "post_beta", cols),
                                  _vec(gate, "gate", cols), _f32(row_gate, "row_gate", rows), _vec(gamma, "gamma", cols),
                                  pdx, lddx, pdy, lddy, _vec(dpost_gamma, "dpost_gamma", cols),
                                  _vec(dpost_beta, "dpost_beta", cols), _vec(dgate, "dgate", cols),
                                  _f32(drow_gate, "drow_gate", rows), _vec(dgamma, "dgamma", cols),
                                  _vec(dbeta, "dbeta", cols), pw, nw, _stream(stream)))


def _i64_of(t, name: str, shape) -> int:
    if t is None:
        return 0
    import torch
    if t.dtype != torch.int64 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous torch.int64 {shape} (got {t.dtype} {tuple(t.shape)})")
    return t.data_ptr()


def loco_logprob_forward(logits, targets, logp, *, lse=None, entropy=None, top_ids=None, top_logp=None, scale: float = 1.0,
                         stream=None):
    """Log probabilities of the given tokens under softmax(scale * logits) [rows, vocab], with the rows' log sums, their
    entropies and, where top_ids and top_logp [rows, top] are given, the most likely tokens."""
    status = _marshal.logprob_forward(logits, targets, logp, lse, entropy, top_ids, top_logp, scale, _stream(stream))
    if status is not None:
        return _check(status) if status else None
    rows, vocab = _dims(logits, "logits")
    pz, ld = _mat(logits, "logits", rows, vocab)
    top = 0
    for t, name in ((top_ids, "top_ids"), (top_logp, "top_logp")):
        if t is not None:
            if t.dim() != 2 or t.shape[0] != rows or (top_ids is not None and t.shape != top_ids.shape):
                raise ValueError(f"{name} must be [rows, top] (got {tuple(t.shape)})")
            top = t.shape[1]
    if top_logp is not None and not top_logp.is_contiguous():
        raise ValueError("top_logp must be contiguous")
    alts = None if top_logp is None else top_logp.view(-1)
    _check(lib.loco_logprob_forward(pz, _dtype(logits, "logits"), ld, rows, vocab, scale, _i64_of(targets, "targets", (rows,)),
                                    _f32(logp, "logp", rows), _f32(lse, "lse", rows), _f32(entropy, "entropy", rows), top,
                                    _i64_of(top_ids, "top_ids", (rows, top)), _f32(alts, "top_logp", rows * top),
                                    _stream(stream)))


def loco_logprob_backward(logits, targets, lse, dlogits, *, dlogp=None, entropy=None, dentropy=None, scale: float = 1.0,
                          stream=None):
    """dlogits (may be the logits) for the gradients of logp and of the entropies; lse and entropy from the forward pass."""
    status = _marshal.logprob_backward(logits, targets, lse, dlogits, dlogp, entropy, dentropy, scale, _stream(stream))
    if status is not None:
        return _check(status) if status else None
    rows, vocab = _dims(logits, "logits")
    pz, ld = _mat(logits, "logits", rows, vocab)
    pd, ldd = _mat(dlogits, "dlogits", rows, vocab)
    _check(lib.loco_logprob_backward(pz, _one_dtype("logits and dlogits", logits, dlogits), ld, rows, vocab, scale,
                                     _i64_of(targets, "targets", (rows,)), _f32(lse, "lse", rows),
                                     _f32(entropy, "entropy", rows), _f32(dlogp, "dlogp", rows),
                                     _f32(dentropy, "dentropy", rows), pd, ldd, _stream(stream)))


class AdamTensors:
    """The tensors of loco_adam_tensors with their types: their addresses, and the tensors themselves, which it keeps."""

    def __init__(self, array, count: int, cfg: loco_adam_tensors_config, tensors):
        self.array, self.count, self.cfg, self.tensors = array, count, cfg, tensors
        self.addresses = ctypes.addressof(cfg), ctypes.addressof(array)


def make_adam_tensors(params, grads, ms, vs, *, m_steps=None, v_steps=None, params_bf16=None, lr_scales=None,
                      decay_scales=None, dither: int = 0) -> AdamTensors:
    """The tensors of an optimizer step, from lists of contiguous tensors of one length.

    params fp32 or bf16, grads fp32 or bf16; ms and vs fp32 of the params' sizes, or int8 and uint8 codes of whole blocks
    of 256 (then m_steps and v_steps hold an fp32 step for each block).  params_bf16: where the updated fp32 parameters go
    in bf16.  lr_scales, decay_scales: factors of the learning rate and of the weight decay (1 where not given).  dither:
    the seed of the rounding of 8-bit states and bf16 parameters, 0 for rounding to nearest.

    The list is made once and used for every step, as long as its tensors stay where they are.
    """
    import torch
    count, f32 = len(params), torch.float32
    eight = m_steps is not None or v_steps is not None
    lists = [("params", params, None), ("grads", grads, None), ("ms", ms, torch.int8 if eight else f32),
             ("vs", vs, torch.uint8 if eight else f32), ("m_steps", m_steps, f32), ("v_steps", v_steps, f32),
             ("params_bf16", params_bf16, torch.bfloat16)]
    if eight and (m_steps is None or v_steps is None):
        raise ValueError("m_steps and v_steps go together")
    addresses = []
    for name, tensors, dtype in lists:
        if tensors is None:
            addresses.append([None] * count)
            continue
        if len(tensors) != count:
            raise ValueError(f"{name} must list {count} tensors (got {len(tensors)})")
        for i, (t, p) in enumerate(zip(tensors, params)):
            nb = -(-p.numel() // LOCO_STATE_BLOCK)
            want = nb if name.endswith("steps") else nb * LOCO_STATE_BLOCK if eight and name in ("ms", "vs") else p.numel()
            if dtype is not None and t.dtype != dtype:
                raise ValueError(f"{name}[{i}] must be {dtype} (got {t.dtype})")
            if t.numel() != want or not t.is_contiguous():
                raise ValueError(f"{name}[{i}] must hold {want} contiguous elements (got {tuple(t.shape)})")
        addresses.append([t.data_ptr() or None for t in tensors])
    for name, values in (("lr_scales", lr_scales), ("decay_scales", decay_scales)):
        if values is not None and len(values) != count:
            raise ValueError(f"{name} must list {count} factors (got {len(values)})")
    if not 0 <= dither < 1 << 32:
        raise ValueError(f"dither = {dither} outside [0, 2^32)")
    array = (loco_adam_tensor * max(count, 1))(*(
        loco_adam_tensor(*(a[i] for a in addresses), params[i].numel(), 1.0 if lr_scales is None else float(lr_scales[i]),
                         1.0 if decay_scales is None else float(decay_scales[i])) for i in range(count)))
    cfg = loco_adam_tensors_config(8 if eight else 32, _one_dtype("params", *params), _one_dtype("grads", *grads), dither)
    return AdamTensors(array, count, cfg, [tensors for _, tensors, _ in lists])


def loco_adam_tensors(tensors: AdamTensors, hp: loco_adam_hparams, t: int, *, grad_scale=None, stream=None):
    """One Adam(W) step on every tensor of the list, in place.  grad_scale: one fp32 value on the device, the factor of
    every gradient (of clipping, of a loss scale)."""
    status = _marshal.adam_tensors(tensors.addresses[0], tensors.addresses[1], tensors.count, ctypes.addressof(hp), t,
                                   grad_scale, _stream(stream))
    if status is not None:
        return _check(status) if status else None
    _check(lib.loco_adam_tensors(ctypes.byref(tensors.cfg), tensors.array, tensors.count, ctypes.byref(hp), t,
                                 0 if grad_scale is None else _f32(grad_scale.view(-1), "grad_scale", 1), _stream(stream)))


def loco_adam_state_decode(codes, steps, out, *, stream=None):
    """out [n] (fp32 or bf16) = the values of an 8-bit state: int8 codes of a first moment, uint8 codes of a second."""
    status = _marshal.adam_state_decode(codes, steps, out, _stream(stream))
    if status is not None:
        return _check(status) if status else None
    import torch
    kind = {torch.int8: LOCO_STATE_M, torch.uint8: LOCO_STATE_V}.get(codes.dtype)
    if kind is None:
        raise ValueError(f"codes must be torch.int8 or torch.uint8 (got {codes.dtype})")
    n = out.numel()
    nb = -(-n // LOCO_STATE_BLOCK)
    if codes.numel() != nb * LOCO_STATE_BLOCK or not codes.is_contiguous():
        raise ValueError(f"codes must be {nb * LOCO_STATE_BLOCK} contiguous codes (got {tuple(codes.shape)})")
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    _check(lib.loco_adam_state_decode(kind, codes.data_ptr(), _f32(steps.view(-1), "steps", nb), n, out.data_ptr(),
                                      _dtype(out, "out"), _stream(stream)))
