"""Python binding of libqerl (C ABI in include/qerl.h): NVFP4 weight-only
linear with a LoRA branch and Adaptive Quantization Noise on GB300.

Argument marshalling only: every function hands raw device pointers, sizes
and the current CUDA stream to the C library, whose CUDA kernels do all the
work.  There is no CPU path; if libqerl.so is missing every call raises.

The functions named like the C entry points take torch tensors:

    qerl_nvfp4_quantize(W, codes, scales, tensor_scale, workspace)
    qerl_nvfp4_quantize_with_scale(W, tensor_scale, codes, scales, workspace)
    qerl_nvfp4_amax(W, amax, workspace)
    qerl_aqn_sigma(stage, num_stages, sigma_start, sigma_end)       (host)
    qerl_aqn_stage(step, total_steps, num_stages)                   (host)
    qerl_aqn_sigma_schedule(schedule, stage, num_stages, ...)       (host)
    qerl_aqn_sample(z, sigma, seed, stream_id, counter)
    qerl_nvfp4_packed_size(n, k)                                    (host)
    qerl_nvfp4_pack(codes, scales, packed)
    qerl_lora_linear(x, wpacked, tensor_scale, z, A, B, alpha, y, workspace)
    qerl_lora_linear_noalloc(x, wpacked, tensor_scale, z, A, B, alpha, y)
    qerl_lora_linear_group(x, z, [(wpacked, tensor_scale, A, B, alpha, y), ...], workspace)
    qerl_rope_append(cache, q, k, v, positions, inv_freq, q_out, k_out, workspace, seq_ids)
    qerl_decode_attention(cache, q, lengths, scale, out, lse, workspace)
    qerl_prompt_attention(q, k, v, cu_seqlens, scale, out, lse, workspace)
    qerl_read_status(workspace)

`kv_cache()` builds the descriptor of a paged key-value cache once, and
`linear_descs()` builds the descriptor array of a group once; passing it
instead of the list skips that marshalling on every call.

The functions return the qerl_status integer (QERL_OK == 0); `check()` turns a
non-zero status into an exception.  `quantize()`, `pack()`, `lora_linear()`,
`rope_append()`, `decode_attention()` and `prompt_attention()` are conveniences
that allocate the outputs with torch (the library itself never allocates).

What only the device sees (a page number outside the cache, offsets that step
back, a wait that ran out) is recorded in the call's workspace, for
`qerl_read_status(workspace)`.  A convenience makes a workspace of its own where
it is given none, and that record is lost with it: pass `ws` and read its status
wherever lengths, positions or pages may be wrong.
"""
import ctypes
import os
import threading

import torch

from . import build as _build

__all__ = [
    "QERL_OK", "QERL_F32", "QERL_BF16", "QerlError", "check", "lib", "lib_path", "status_string",
    "qerl_nvfp4_quantize", "qerl_nvfp4_quantize_with_scale", "qerl_nvfp4_amax",
    "qerl_nvfp4_quantize_workspace_size", "qerl_aqn_sigma", "qerl_aqn_stage", "qerl_aqn_sample",
    "qerl_aqn_sigma_schedule", "QERL_SCHEDULE_EXPONENTIAL", "QERL_SCHEDULE_LINEAR", "QERL_SCHEDULE_COSINE",
    "QERL_SCHEDULE_LOGARITHMIC",
    "qerl_nvfp4_packed_size", "qerl_nvfp4_pack", "pack",
    "qerl_lora_linear_workspace_size", "qerl_lora_linear", "qerl_lora_linear_noalloc", "qerl_read_status",
    "qerl_lora_linear_group", "qerl_lora_linear_group_workspace_size", "LinearDesc", "linear_descs",
    "quantize", "lora_linear", "workspace",
    "QERL_E4M3", "KvCache", "kv_cache", "qerl_rope_append", "qerl_rope_append_workspace_size",
    "qerl_decode_attention", "qerl_decode_attention_workspace_size", "rope_append", "decode_attention",
    "qerl_prompt_attention", "qerl_prompt_attention_workspace_size", "prompt_attention",
]

class LinearDesc(ctypes.Structure):
    """Mirror of qerl_linear_desc (include/qerl.h)."""
    _fields_ = [("wpacked", ctypes.c_void_p), ("tensor_scale", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("r", ctypes.c_int), ("alpha", ctypes.c_float),
                ("y", ctypes.c_void_p), ("y_dtype", ctypes.c_int), ("w_format", ctypes.c_int)]


class KvCache(ctypes.Structure):
    """Mirror of qerl_kv_cache (include/qerl.h)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("page_size", ctypes.c_int),
                ("num_pages", ctypes.c_int64), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("num_seqs", ctypes.c_int64), ("max_pages", ctypes.c_int64),
                ("ld_table", ctypes.c_int64)]
    device = None  # the device number of the memory, where kv_cache() made the descriptor


QERL_OK = 0
QERL_F32, QERL_BF16, QERL_E4M3 = 0, 1, 2
QERL_W_NVFP4, QERL_W_NF4 = 0, 1
QERL_SCHEDULE_EXPONENTIAL, QERL_SCHEDULE_LINEAR, QERL_SCHEDULE_COSINE, QERL_SCHEDULE_LOGARITHMIC = 0, 1, 2, 3
STATUS_NAMES = {0: "QERL_OK", 1: "QERL_ERR_INVALID_ARGUMENT", 2: "QERL_ERR_UNSUPPORTED_SHAPE",
                3: "QERL_ERR_MISALIGNED", 4: "QERL_ERR_CUDA", 5: "QERL_ERR_TIMEOUT", 6: "QERL_ERR_NONFINITE",
                7: "QERL_ERR_WORKSPACE", 8: "QERL_ERR_RANGE"}

_lib = None
_lock = threading.Lock()
_vp = ctypes.c_void_p
_i64 = ctypes.c_int64


class QerlError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")
        self.status = status


def lib_path() -> str:
    return _build.LIB


def lib():
    """The loaded libqerl.so.  Raises if it has not been built (no fallback)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_build.LIB):
                raise RuntimeError(f"libqerl.so not built at {_build.LIB}; run "
                                   "nvfp4_weight_quantized_03_gb300.build.build() (nvcc, sm_103a)")
            L = ctypes.CDLL(_build.LIB)
            L.qerl_status_string.restype = ctypes.c_char_p
            L.qerl_status_string.argtypes = [ctypes.c_int]
            L.qerl_version.restype = ctypes.c_int
            L.qerl_version.argtypes = []
            L.qerl_nvfp4_quantize_workspace_size.restype = ctypes.c_size_t
            L.qerl_nvfp4_quantize_workspace_size.argtypes = []
            L.qerl_nvfp4_quantize.restype = ctypes.c_int
            L.qerl_nvfp4_quantize.argtypes = [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp, _vp,
                                              ctypes.c_size_t, _vp]
            L.qerl_nvfp4_quantize_with_scale.restype = ctypes.c_int
            L.qerl_nvfp4_quantize_with_scale.argtypes = [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp, _vp,
                                                         ctypes.c_size_t, _vp]
            L.qerl_nvfp4_pack_transposed.restype = ctypes.c_int
            L.qerl_nvfp4_pack_transposed.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp]
            L.qerl_lora_linear_backward_workspace_size.restype = ctypes.c_size_t
            L.qerl_lora_linear_backward_workspace_size.argtypes = [_i64, _i64, _i64, ctypes.c_int]
            L.qerl_lora_linear_backward.restype = ctypes.c_int
            L.qerl_lora_linear_backward.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _vp,
                                                    ctypes.c_int, ctypes.c_float, _vp, ctypes.c_int, _vp, _vp, _vp,
                                                    ctypes.c_size_t, _vp]
            L.qerl_nf4_quantize.restype = ctypes.c_int
            L.qerl_nf4_quantize.argtypes = [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp, _vp,
                                            ctypes.c_size_t, _vp]
            L.qerl_mxfp4_quantize.restype = ctypes.c_int
            L.qerl_mxfp4_quantize.argtypes = [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp, ctypes.c_size_t,
                                              _vp]
            L.qerl_mxfp4_pack.restype = ctypes.c_int
            L.qerl_mxfp4_pack.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _vp, ctypes.c_size_t, _vp]
            L.qerl_nvfp4_amax.restype = ctypes.c_int
            L.qerl_nvfp4_amax.argtypes = [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, ctypes.c_size_t, _vp]
            L.qerl_aqn_sigma.restype = ctypes.c_double
            L.qerl_aqn_sigma.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_double, ctypes.c_double]
            L.qerl_aqn_sigma_schedule.restype = ctypes.c_double
            L.qerl_aqn_sigma_schedule.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_double,
                                                  ctypes.c_double]
            L.qerl_aqn_stage.restype = ctypes.c_int
            L.qerl_aqn_stage.argtypes = [_i64, _i64, ctypes.c_int]
            L.qerl_aqn_sample.restype = ctypes.c_int
            L.qerl_aqn_sample.argtypes = [_vp, _i64, ctypes.c_float, ctypes.c_uint64, ctypes.c_uint32,
                                          ctypes.c_uint64, _vp]
            L.qerl_nvfp4_packed_size.restype = ctypes.c_size_t
            L.qerl_nvfp4_packed_size.argtypes = [_i64, _i64]
            L.qerl_nvfp4_pack.restype = ctypes.c_int
            L.qerl_nvfp4_pack.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp]
            L.qerl_lora_linear_workspace_size.restype = ctypes.c_size_t
            L.qerl_lora_linear_workspace_size.argtypes = [_i64, _i64, _i64, ctypes.c_int]
            L.qerl_lora_linear.restype = ctypes.c_int
            L.qerl_lora_linear.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _vp, ctypes.c_int,
                                           ctypes.c_float, _vp, ctypes.c_int, _vp, ctypes.c_size_t, _vp]
            L.qerl_lora_linear_group_workspace_size.restype = ctypes.c_size_t
            L.qerl_lora_linear_group_workspace_size.argtypes = [_i64, _i64, ctypes.POINTER(LinearDesc), ctypes.c_int]
            L.qerl_lora_linear_group.restype = ctypes.c_int
            L.qerl_lora_linear_group.argtypes = [_vp, _i64, _i64, _i64, _vp, ctypes.POINTER(LinearDesc), ctypes.c_int,
                                                 _vp, ctypes.c_size_t, _vp]
            L.qerl_nvfp4_tensor_scale.restype = ctypes.c_int
            L.qerl_nvfp4_tensor_scale.argtypes = [_vp, _vp, _vp]
            L.qerl_lora_linear_group_rowz.restype = ctypes.c_int
            L.qerl_lora_linear_group_rowz.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, ctypes.POINTER(LinearDesc),
                                                      ctypes.c_int, _vp, ctypes.c_size_t, _vp]
            L.qerl_rmsnorm_lora_linear_group_workspace_size.restype = ctypes.c_size_t
            L.qerl_rmsnorm_lora_linear_group_workspace_size.argtypes = [_i64, _i64, ctypes.POINTER(LinearDesc),
                                                                        ctypes.c_int]
            L.qerl_rmsnorm_lora_linear_group.restype = ctypes.c_int
            L.qerl_rmsnorm_lora_linear_group.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, ctypes.c_double,
                                                         ctypes.POINTER(LinearDesc), ctypes.c_int, _vp,
                                                         ctypes.c_size_t, _vp]
            L.qerl_rmsnorm_noise.restype = ctypes.c_int
            L.qerl_rmsnorm_noise.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, ctypes.c_double, _vp, _i64, _vp]
            L.qerl_lora_linear_noalloc.restype = ctypes.c_int
            L.qerl_lora_linear_noalloc.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _vp,
                                                   ctypes.c_int, ctypes.c_float, _vp, ctypes.c_int, _vp]
            _c = ctypes.POINTER(KvCache)
            L.qerl_rope_append_workspace_size.restype = ctypes.c_size_t
            L.qerl_rope_append_workspace_size.argtypes = []
            L.qerl_rope_append.restype = ctypes.c_int
            L.qerl_rope_append.argtypes = [_c, _vp, _i64, ctypes.c_int, _vp, _i64, _vp, _i64, ctypes.c_int,
                                           ctypes.c_int, _i64, _vp, _vp, _vp, ctypes.c_int, _vp, _i64, _vp, _i64,
                                           _vp, ctypes.c_size_t, _vp]
            L.qerl_decode_attention_workspace_size.restype = ctypes.c_size_t
            L.qerl_decode_attention_workspace_size.argtypes = [_i64, ctypes.c_int, ctypes.c_int, ctypes.c_int]
            L.qerl_decode_attention.restype = ctypes.c_int
            L.qerl_decode_attention.argtypes = [_c, _vp, _i64, ctypes.c_int, _vp, ctypes.c_float, _vp, _i64, _vp,
                                                _vp, ctypes.c_size_t, _vp]
            L.qerl_prompt_attention_workspace_size.restype = ctypes.c_size_t
            L.qerl_prompt_attention_workspace_size.argtypes = [_i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, _i64]
            L.qerl_prompt_attention.restype = ctypes.c_int
            L.qerl_prompt_attention.argtypes = [_vp, _i64, _vp, _i64, _vp, _i64, _i64, ctypes.c_int, ctypes.c_int,
                                                ctypes.c_int, _vp, _i64, ctypes.c_float, _vp, _i64, _vp, _vp,
                                                ctypes.c_size_t, _vp]
            L.qerl_read_status.restype = ctypes.c_int
            L.qerl_read_status.argtypes = [_vp, _vp]
            _lib = L
    return _lib


def status_string(st: int) -> str:
    return lib().qerl_status_string(int(st)).decode()


def check(st: int, where: str = "qerl") -> None:
    if st != QERL_OK:
        raise QerlError(st, where)


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# current_stream() builds an object (3 us a call), current_device() looks whether CUDA is up each time.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream, dev=None):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_device() if dev is None else dev)
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _wdtype(W):
    if W.dtype == torch.float32:
        return QERL_F32
    if W.dtype == torch.bfloat16:
        return QERL_BF16
    raise TypeError("W must be float32 or bfloat16")


def _nbytes(t):
    return t.nbytes


# ---- C entry points ---------------------------------------------------------

def qerl_nvfp4_quantize_workspace_size() -> int:
    return lib().qerl_nvfp4_quantize_workspace_size()


def qerl_nvfp4_quantize(W, codes, scales, tensor_scale, workspace, stream=None) -> int:
    n, k = W.shape
    return lib().qerl_nvfp4_quantize(_p(W), _wdtype(W), n, k, W.stride(0), _p(codes), _p(scales),
                                     _p(tensor_scale), _p(workspace), _nbytes(workspace), _stream(stream))


def qerl_nvfp4_quantize_with_scale(W, tensor_scale, codes, scales, workspace, stream=None) -> int:
    n, k = W.shape
    return lib().qerl_nvfp4_quantize_with_scale(_p(W), _wdtype(W), n, k, W.stride(0), _p(tensor_scale),
                                                _p(codes), _p(scales), _p(workspace), _nbytes(workspace),
                                                _stream(stream))


def qerl_nvfp4_amax(W, amax, workspace, stream=None) -> int:
    n, k = W.shape
    return lib().qerl_nvfp4_amax(_p(W), _wdtype(W), n, k, W.stride(0), _p(amax), _p(workspace),
                                 _nbytes(workspace), _stream(stream))


def qerl_nvfp4_tensor_scale(amax, tensor_scale, stream=None) -> int:
    return lib().qerl_nvfp4_tensor_scale(_p(amax), _p(tensor_scale), _stream(stream))


def global_amax(amax, group=None):
    """All-reduce(max) of a shard's amax (a one-element float tensor, in place) over the
    process group: with it, qerl_nvfp4_tensor_scale and qerl_nvfp4_quantize_with_scale give
    every shard the codes and scales of the whole tensor.  Plain torch.distributed
    plumbing (any backend: gloo for CPU tensors, NCCL for device tensors)."""
    import torch.distributed as dist
    if dist.is_available() and dist.is_initialized():
        dist.all_reduce(amax, op=dist.ReduceOp.MAX, group=group)
    return amax


def qerl_aqn_sigma(stage: int, num_stages: int, sigma_start: float = 1e-2, sigma_end: float = 5e-4) -> float:
    return lib().qerl_aqn_sigma(int(stage), int(num_stages), float(sigma_start), float(sigma_end))


def qerl_aqn_sigma_schedule(schedule: int, stage: int, num_stages: int, sigma_start: float = 1e-2,
                            sigma_end: float = 5e-4) -> float:
    return lib().qerl_aqn_sigma_schedule(int(schedule), int(stage), int(num_stages), float(sigma_start),
                                         float(sigma_end))


def qerl_aqn_stage(step: int, total_steps: int, num_stages: int) -> int:
    return lib().qerl_aqn_stage(int(step), int(total_steps), int(num_stages))


def qerl_aqn_sample(z, sigma: float, seed: int, stream_id: int = 0, counter: int = 0, stream=None) -> int:
    return lib().qerl_aqn_sample(_p(z), z.numel(), float(sigma), int(seed) & (2**64 - 1),
                                 int(stream_id) & 0xFFFFFFFF, int(counter) & (2**64 - 1), _stream(stream))


def qerl_nvfp4_packed_size(n: int, k: int) -> int:
    return lib().qerl_nvfp4_packed_size(int(n), int(k))


def qerl_nvfp4_pack(codes, scales, packed, stream=None) -> int:
    """codes [n, k/2], scales [n, k/16] (uint8) -> packed (uint8, qerl_nvfp4_packed_size(n, k) bytes)."""
    n = codes.shape[0]
    k = codes.shape[1] * 2
    return lib().qerl_nvfp4_pack(_p(codes), _p(scales), n, k, _p(packed), _stream(stream))


def qerl_nvfp4_pack_transposed(codes, scales, packed_t, stream=None) -> int:
    """codes [n, k/2], scales [n, k/16] -> the transposed packed layout (qerl_nvfp4_packed_size(k, n) bytes)."""
    n = codes.shape[0]
    k = codes.shape[1] * 2
    return lib().qerl_nvfp4_pack_transposed(_p(codes), _p(scales), n, k, _p(packed_t), _stream(stream))


def qerl_lora_linear_backward_workspace_size(m: int, n: int, k: int, r: int) -> int:
    return lib().qerl_lora_linear_backward_workspace_size(int(m), int(n), int(k), int(r))


def qerl_lora_linear_backward(xt, dy, wpacked_t, tensor_scale, A, B, alpha, dxt, dA, dB, workspace,
                              stream=None) -> int:
    """xt [m, k] bf16 (the forward's x~), dy [m, n] bf16, wpacked_t from qerl_nvfp4_pack_transposed;
    dxt [m, k] bf16/fp32; dA [r, k], dB [n, r] fp32 or None."""
    m, n = dy.shape
    k = dxt.shape[1]
    r = 0 if A is None else A.shape[0]
    ddt = QERL_F32 if dxt.dtype == torch.float32 else QERL_BF16
    ldxt = xt.stride(0) if xt is not None else k
    return lib().qerl_lora_linear_backward(_p(xt), m, k, ldxt, _p(dy), n, dy.stride(0), _p(wpacked_t),
                                           _p(tensor_scale), _p(A), _p(B), r, float(alpha), _p(dxt), ddt, _p(dA),
                                           _p(dB), _p(workspace), _nbytes(workspace), _stream(stream))


def qerl_nf4_quantize(W, codes, scales, tensor_scale, workspace, stream=None) -> int:
    """W [n, k] f32/bf16 -> NF4 codes [n, k/2], E4M3 scales [n, k/16], tensor scale (the layout of
    qerl_nvfp4_quantize, so qerl_nvfp4_pack packs it; the linear takes w_format QERL_W_NF4)."""
    n, k = W.shape
    return lib().qerl_nf4_quantize(_p(W), _wdtype(W), n, k, W.stride(0), _p(codes), _p(scales), _p(tensor_scale),
                                   _p(workspace), _nbytes(workspace), _stream(stream))


def qerl_mxfp4_quantize(W, codes, scales, workspace, stream=None) -> int:
    """W [n, k] f32/bf16 -> codes [n, k/2], E8M0 scales [n, k/32] (uint8)."""
    n, k = W.shape
    return lib().qerl_mxfp4_quantize(_p(W), _wdtype(W), n, k, W.stride(0), _p(codes), _p(scales), _p(workspace),
                                     _nbytes(workspace), _stream(stream))


def qerl_mxfp4_pack(codes, scales, packed, tensor_scale, workspace, stream=None) -> int:
    """codes [n, k/2], E8M0 scales [n, k/32] -> packed (qerl_nvfp4_packed_size(n, k) bytes) and the
    power-of-two tensor scale the linear applies."""
    n = codes.shape[0]
    k = codes.shape[1] * 2
    return lib().qerl_mxfp4_pack(_p(codes), _p(scales), n, k, _p(packed), _p(tensor_scale), _p(workspace),
                                 _nbytes(workspace), _stream(stream))


def qerl_lora_linear_workspace_size(m: int, n: int, k: int, r: int) -> int:
    return lib().qerl_lora_linear_workspace_size(int(m), int(n), int(k), int(r))


def qerl_lora_linear(x, wpacked, tensor_scale, z, A, B, alpha, y, workspace, stream=None) -> int:
    """x [m, k] bf16; wpacked: the n x k weight packed by qerl_nvfp4_pack; y [m, n] (n taken from y);
    A: [r, k] bf16 (LoRA down-projection), B: [n, r] bf16 (LoRA up-projection)."""
    m, k = x.shape
    n = y.shape[1]
    r = 0 if A is None else A.shape[0]
    ydt = QERL_F32 if y.dtype == torch.float32 else QERL_BF16
    return lib().qerl_lora_linear(_p(x), m, k, x.stride(0), _p(wpacked), _p(tensor_scale), n, _p(z), _p(A), _p(B),
                                  r, float(alpha), _p(y), ydt, _p(workspace), _nbytes(workspace), _stream(stream))


def qerl_lora_linear_noalloc(x, wpacked, tensor_scale, z, A, B, alpha, y, stream=None) -> int:
    """qerl_lora_linear without a workspace, for callers that cannot allocate
    device memory at the call site; the library's own fixed scratch array is
    used (shared by all calls: keep them ordered)."""
    m, k = x.shape
    n = y.shape[1]
    r = 0 if A is None else A.shape[0]
    ydt = QERL_F32 if y.dtype == torch.float32 else QERL_BF16
    return lib().qerl_lora_linear_noalloc(_p(x), m, k, x.stride(0), _p(wpacked), _p(tensor_scale), n, _p(z),
                                          _p(A), _p(B), r, float(alpha), _p(y), ydt, _stream(stream))


def _descs(linears):
    """[(wpacked, tensor_scale, A, B, alpha, y[, w_format]), ...] -> ctypes array of LinearDesc
    (an array built before is passed through)."""
    if isinstance(linears, ctypes.Array):
        return linears
    arr = (LinearDesc * len(linears))()
    for d, item in zip(arr, linears):
        wp, ts, A, B, alpha, y = item[:6]
        d.w_format = int(item[6]) if len(item) > 6 else QERL_W_NVFP4
        d.wpacked, d.tensor_scale, d.n = _p(wp), _p(ts), y.shape[1]
        d.A, d.B, d.r = _p(A), _p(B), 0 if A is None else A.shape[0]
        d.alpha, d.y = float(alpha), _p(y)
        d.y_dtype = QERL_F32 if y.dtype == torch.float32 else QERL_BF16
    return arr


def linear_descs(linears):
    """The qerl_linear_desc array of a group, [(wpacked, tensor_scale, A, B, alpha, y), ...],
    built once: the array holds raw pointers, so the tensors must outlive it."""
    return _descs(linears)


def qerl_lora_linear_group_workspace_size(m: int, k: int, linears) -> int:
    arr = _descs(linears)
    return lib().qerl_lora_linear_group_workspace_size(int(m), int(k), arr, len(arr))


def qerl_lora_linear_group(x, z, linears, workspace, stream=None) -> int:
    """Up to four linears of one input x [m, k] (bf16) and noise z: linears is a list of
    (wpacked, tensor_scale, A, B, alpha, y) with y [m, n_i], or its linear_descs() array;
    one launch for all."""
    m, k = x.shape
    arr = _descs(linears)
    return lib().qerl_lora_linear_group(_p(x), m, k, x.stride(0), _p(z), arr, len(arr), _p(workspace),
                                        _nbytes(workspace), _stream(stream))


def qerl_lora_linear_group_rowz(x, z, linears, workspace, stream=None) -> int:
    """The grouped linear with per-row noise: z is None, a [k] vector (every row), or [m, k]
    float32 (row i of x uses z[i]; its row stride is passed)."""
    m, k = x.shape
    arr = _descs(linears)
    ldz = 0 if z is None or z.dim() == 1 else z.stride(0)
    return lib().qerl_lora_linear_group_rowz(_p(x), m, k, x.stride(0), _p(z), ldz, arr, len(arr), _p(workspace),
                                             _nbytes(workspace), _stream(stream))


def qerl_rmsnorm_lora_linear_group_workspace_size(m: int, k: int, linears) -> int:
    arr = _descs(linears)
    return lib().qerl_rmsnorm_lora_linear_group_workspace_size(int(m), int(k), arr, len(arr))


def qerl_rmsnorm_lora_linear_group(h, w_norm, Z, delta, linears, workspace, stream=None) -> int:
    """RMSNorm of h [m, k] (bf16) with the noise Z [k] (float32, or None) merged into its
    weight w_norm [k] (bf16), then the grouped linear of the result."""
    m, k = h.shape
    arr = _descs(linears)
    return lib().qerl_rmsnorm_lora_linear_group(_p(h), m, k, h.stride(0), _p(w_norm), _p(Z), float(delta), arr,
                                                len(arr), _p(workspace), _nbytes(workspace), _stream(stream))


def qerl_rmsnorm_noise(h, w_norm, Z, delta, out, stream=None) -> int:
    """The normalisation step alone: out [m, k] bf16 = bf16((w_norm + Z) * h / rms(h))."""
    m, k = h.shape
    return lib().qerl_rmsnorm_noise(_p(h), m, k, h.stride(0), _p(w_norm), _p(Z), float(delta), _p(out),
                                    out.stride(0), _stream(stream))


# ---- attention ----------------------------------------------------------------

_BF16, _I32, _F32, _F64 = torch.bfloat16, torch.int32, torch.float32, torch.float64


def _expect(name, t, dtype, dims, dev=None):
    """Raises unless t is a CUDA tensor of this type and dimension count, on device number dev (if given): a
    raw pointer of another type would be misread, one of other memory would fault."""
    if t.dtype is not dtype or not t.is_cuda or t.dim() != dims:
        raise TypeError(f"{name}: expected a {dims}-d CUDA tensor of {dtype}, got {tuple(t.shape)} {t.dtype} on "
                        f"{t.device}")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{dev}")


def _heads(name, t, shape, dev):
    """Row stride of bf16 rows of heads [rows, heads, head_dim], of this shape, whose heads lie side by side."""
    if t.dtype is not _BF16 or t.get_device() != dev:
        _expect(name, t, _BF16, 3, dev)
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    ld, s1, s2 = t.stride()
    rows, heads, dim = shape
    if s2 != 1 or s1 != dim or rows < 2:
        if (dim > 1 and s2 != 1) or (heads > 1 and s1 != dim):
            raise ValueError(f"{name}: the heads of a row must be contiguous, got strides {t.stride()}")
        ld = ld if rows > 1 else max(ld, heads * dim)
    return ld


def _vector(name, t, dtype, n, dev):
    """Raises unless t is a contiguous vector of n entries of this type on device number dev."""
    if t.dtype is not dtype or t.get_device() != dev:
        _expect(name, t, dtype, 1, dev)
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name}: expected {n} contiguous entries, got {tuple(t.shape)} with strides {t.stride()}")


def _memory(ws, cache, dev):
    """Raises unless the workspace, and the cache if there is one, are memory of device number dev."""
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"workspace: expected contiguous memory on cuda:{dev}, got strides {ws.stride()} on {ws.device}")
    if cache is not None and cache.device is not None and cache.device != dev:
        raise ValueError(f"cache: on cuda:{cache.device}, expected cuda:{dev}")


def _heads_shape(name, t):
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name}: expected [rows, heads, head_dim], got {tuple(shape)}")
    return shape


def kv_cache(k, v, page_table, k_scale=None, v_scale=None):
    """The qerl_kv_cache descriptor of pages k, v [num_pages, num_kv_heads, page_size, head_dim]
    (bfloat16 or float8_e4m3fn), page_table [num_seqs, max_pages] int32 and, for float8_e4m3fn,
    scales [num_kv_heads] float32 (or None).  It keeps the tensors alive."""
    if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
        raise TypeError("k: the cache holds bfloat16 or float8_e4m3fn")
    _expect("k", k, k.dtype, 4)
    dev = k.get_device()
    _expect("v", v, k.dtype, 4, dev)
    _expect("page_table", page_table, torch.int32, 2, dev)
    if v.shape != k.shape or not k.is_contiguous() or not v.is_contiguous():
        raise ValueError("k and v: contiguous pages of one shape")
    if page_table.shape[1] > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table: the entries of a row must be contiguous")
    c = KvCache()
    c.num_pages, c.num_kv_heads, c.page_size, c.head_dim = k.shape
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t is not None:
            _expect(name, t, torch.float32, 1, dev)
            if t.numel() != c.num_kv_heads or not t.is_contiguous():
                raise ValueError(f"{name}: one contiguous float per key-value head")
    c.k, c.v = _p(k), _p(v)
    c.dtype = QERL_E4M3 if k.dtype == torch.float8_e4m3fn else QERL_BF16
    c.k_scale, c.v_scale = _p(k_scale), _p(v_scale)
    c.page_table = _p(page_table)
    c.num_seqs, c.max_pages = page_table.shape
    c.ld_table = page_table.stride(0) if c.num_seqs > 1 else max(page_table.stride(0), c.max_pages)
    c.tensors = (k, v, page_table, k_scale, v_scale)
    c.device = dev
    return c


def qerl_rope_append_workspace_size() -> int:
    return lib().qerl_rope_append_workspace_size()


def qerl_rope_append(cache, q, k, v, positions, inv_freq, q_out, k_out, workspace, seq_ids=None, stream=None) -> int:
    """q [tokens, num_heads, head_dim] or None, k, v [tokens, num_kv_heads, head_dim] (bf16, strided rows),
    positions [tokens] int32 (negative: padding), inv_freq [rot_dim / 2] float64, seq_ids [tokens] int32 or
    None (token t is sequence t); q_out, k_out like q, k (may be them; k_out may be None with a cache).
    cache None: rotation only (v may be None)."""
    shape = _heads_shape("k", k)
    tokens, hk, d = shape
    dev = _device()  # where the launch goes
    ldk = _heads("k", k, shape, dev)
    h = ldq = ldqo = ldv = ldko = 0
    if q is not None:
        wide = _heads_shape("q", q)
        h = wide[1]
        if wide[0] != tokens or wide[2] != d:
            raise ValueError(f"q: expected k's tokens and head_dim, got {tuple(wide)}")
        ldq, ldqo = _heads("q", q, wide, dev), _heads("q_out", q_out, wide, dev)
    if v is not None:
        ldv = _heads("v", v, shape, dev)
    if k_out is not None:
        ldko = _heads("k_out", k_out, shape, dev)
    _vector("positions", positions, _I32, tokens, dev)
    half = inv_freq.numel()
    _vector("inv_freq", inv_freq, _F64, half, dev)
    if seq_ids is not None:
        _vector("seq_ids", seq_ids, _I32, tokens, dev)
    if workspace.get_device() != dev or not workspace.is_contiguous() or cache is not None and cache.device != dev:
        _memory(workspace, cache, dev)
    return (_lib or lib()).qerl_rope_append(
        cache, None if q is None else q.data_ptr(), ldq, h, k.data_ptr(), ldk, None if v is None else v.data_ptr(), ldv,
        hk, d, tokens, None if seq_ids is None else seq_ids.data_ptr(), positions.data_ptr(), inv_freq.data_ptr(),
        2 * half, None if q is None else q_out.data_ptr(), ldqo, None if k_out is None else k_out.data_ptr(), ldko,
        workspace.data_ptr(), workspace.nbytes, _stream(stream, dev))


def qerl_decode_attention_workspace_size(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return lib().qerl_decode_attention_workspace_size(int(num_seqs), int(num_heads), int(num_kv_heads), int(head_dim))


def _lse(lse, rows, heads, dev):
    if lse.dtype is not _F32 or lse.get_device() != dev:
        _expect("lse", lse, _F32, 2, dev)
    if lse.shape != (rows, heads) or not lse.is_contiguous():
        raise ValueError("lse: contiguous [rows, num_heads]")
    return lse.data_ptr()


def qerl_decode_attention(cache, q, lengths, scale, out, lse, workspace, stream=None) -> int:
    """q, out [num_seqs, num_heads, head_dim] bf16 (strided rows), lengths [num_seqs] int32, lse [num_seqs,
    num_heads] float32 or None: one new token per sequence over the cache's first lengths[s] rows."""
    shape = _heads_shape("q", q)
    n, h, d = shape
    if n != cache.num_seqs or d != cache.head_dim:
        raise ValueError("q: [num_seqs, num_heads, head_dim] of the cache")
    dev = _device()  # where the launch goes
    ldq, ldo = _heads("q", q, shape, dev), _heads("out", out, shape, dev)
    _vector("lengths", lengths, _I32, n, dev)
    lse_p = None if lse is None else _lse(lse, n, h, dev)
    if workspace.get_device() != dev or not workspace.is_contiguous() or cache.device != dev:
        _memory(workspace, cache, dev)
    return (_lib or lib()).qerl_decode_attention(cache, q.data_ptr(), ldq, h, lengths.data_ptr(), scale,
                                                 out.data_ptr(), ldo, lse_p, workspace.data_ptr(), workspace.nbytes,
                                                 _stream(stream, dev))


def qerl_prompt_attention_workspace_size(tokens: int, num_heads: int, num_kv_heads: int, head_dim: int,
                                         num_seqs: int) -> int:
    return lib().qerl_prompt_attention_workspace_size(int(tokens), int(num_heads), int(num_kv_heads), int(head_dim),
                                                      int(num_seqs))


def qerl_prompt_attention(q, k, v, cu_seqlens, scale, out, lse, workspace, stream=None) -> int:
    """q, out [tokens, num_heads, head_dim], k, v [tokens, num_kv_heads, head_dim] bf16 (strided rows),
    cu_seqlens [num_seqs + 1] int32, lse [tokens, num_heads] float32 or None: causal attention of the
    packed sequences."""
    shape = _heads_shape("q", q)
    t, h, d = shape
    hk = _heads_shape("k", k)[1]
    dev = _device()  # where the launch goes
    ldq, ldo = _heads("q", q, shape, dev), _heads("out", out, shape, dev)
    ldk, ldv = _heads("k", k, (t, hk, d), dev), _heads("v", v, (t, hk, d), dev)
    n = cu_seqlens.numel()
    _vector("cu_seqlens", cu_seqlens, _I32, n, dev)
    if n < 1:
        raise ValueError("cu_seqlens: [num_seqs + 1]")
    lse_p = None if lse is None else _lse(lse, t, h, dev)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _memory(workspace, None, dev)
    return (_lib or lib()).qerl_prompt_attention(q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, t, h, hk, d,
                                                 cu_seqlens.data_ptr(), n - 1, scale, out.data_ptr(), ldo, lse_p,
                                                 workspace.data_ptr(), workspace.nbytes, _stream(stream, dev))


def qerl_read_status(workspace, stream=None) -> int:
    return lib().qerl_read_status(_p(workspace), _stream(stream))


# ---- conveniences (allocation by torch; compute by the library) -------------

def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zero-filled, 256-byte aligned device workspace of at least nbytes."""
    return torch.zeros(max(256, (nbytes + 255) // 256 * 256), dtype=torch.uint8, device=device or "cuda")


def quantize(W: torch.Tensor, ws: torch.Tensor = None):
    """NVFP4-quantize an n x k float32/bfloat16 CUDA tensor -> (codes, scales, tensor_scale)."""
    n, k = W.shape
    codes = torch.empty((n, k // 2), dtype=torch.uint8, device=W.device)
    scales = torch.empty((n, k // 16), dtype=torch.uint8, device=W.device)
    ts = torch.empty(1, dtype=torch.float32, device=W.device)
    ws = workspace(qerl_nvfp4_quantize_workspace_size(), W.device) if ws is None else ws
    check(qerl_nvfp4_quantize(W, codes, scales, ts, ws), "qerl_nvfp4_quantize")
    return codes, scales, ts


def pack(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """Packed (kernel-native) form of quantized weights, for qerl_lora_linear."""
    n, k = codes.shape[0], codes.shape[1] * 2
    packed = torch.empty(qerl_nvfp4_packed_size(n, k), dtype=torch.uint8, device=codes.device)
    check(qerl_nvfp4_pack(codes, scales, packed), "qerl_nvfp4_pack")
    return packed


def pack_transposed(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """The transposed packed layout of quantized weights, for qerl_lora_linear_backward."""
    n, k = codes.shape[0], codes.shape[1] * 2
    packed = torch.empty(qerl_nvfp4_packed_size(k, n), dtype=torch.uint8, device=codes.device)
    check(qerl_nvfp4_pack_transposed(codes, scales, packed), "qerl_nvfp4_pack_transposed")
    return packed


def nf4_quantize(W: torch.Tensor, ws: torch.Tensor = None):
    """NF4-quantize an n x k float32/bfloat16 CUDA tensor -> (codes, scales, tensor_scale)."""
    n, k = W.shape
    codes = torch.empty((n, k // 2), dtype=torch.uint8, device=W.device)
    scales = torch.empty((n, k // 16), dtype=torch.uint8, device=W.device)
    ts = torch.empty(1, dtype=torch.float32, device=W.device)
    ws = workspace(qerl_nvfp4_quantize_workspace_size(), W.device) if ws is None else ws
    check(qerl_nf4_quantize(W, codes, scales, ts, ws), "qerl_nf4_quantize")
    return codes, scales, ts


def mxfp4_quantize(W: torch.Tensor, ws: torch.Tensor = None):
    """MXFP4-quantize an n x k float32/bfloat16 CUDA tensor -> (codes, E8M0 scales)."""
    n, k = W.shape
    codes = torch.empty((n, k // 2), dtype=torch.uint8, device=W.device)
    scales = torch.empty((n, k // 32), dtype=torch.uint8, device=W.device)
    ws = workspace(qerl_nvfp4_quantize_workspace_size(), W.device) if ws is None else ws
    check(qerl_mxfp4_quantize(W, codes, scales, ws), "qerl_mxfp4_quantize")
    return codes, scales


def mxfp4_pack(codes: torch.Tensor, scales: torch.Tensor, ws: torch.Tensor = None):
    """Packed form of an MXFP4 weight for qerl_lora_linear -> (packed, tensor_scale)."""
    n, k = codes.shape[0], codes.shape[1] * 2
    packed = torch.empty(qerl_nvfp4_packed_size(n, k), dtype=torch.uint8, device=codes.device)
    ts = torch.empty(1, dtype=torch.float32, device=codes.device)
    ws = workspace(qerl_nvfp4_quantize_workspace_size(), codes.device) if ws is None else ws
    check(qerl_mxfp4_pack(codes, scales, packed, ts, ws), "qerl_mxfp4_pack")
    return packed, ts


def lora_linear(x, wpacked, tensor_scale, n, z=None, A=None, B=None, alpha=0.0, out_dtype=torch.bfloat16,
                ws=None):
    """y = x~ . dequant(W)^T + (alpha/r) (x~ A^T) B^T, x~ = bf16(x(1+z)), for bf16 x [m, k],
    W n x k packed by pack(), A [r, k], B [n, r]."""
    m, k = x.shape
    r = 0 if A is None else A.shape[0]
    y = torch.empty((m, n), dtype=out_dtype, device=x.device)
    ws = workspace(qerl_lora_linear_workspace_size(m, n, k, r), x.device) if ws is None else ws
    check(qerl_lora_linear(x, wpacked, tensor_scale, z, A, B, alpha, y, ws), "qerl_lora_linear")
    return y


def rope_append(cache, q, k, v, positions, inv_freq, seq_ids=None, ws=None):
    """Rotated copies (q, k) of q (or None) and k, with k and v appended to the cache (see qerl_rope_append);
    rows of padding are 0.  A token outside the page table or the cache is not appended and is recorded in ws."""
    q_out = None if q is None else torch.zeros_like(q, memory_format=torch.contiguous_format)
    k_out = torch.zeros_like(k, memory_format=torch.contiguous_format)
    ws = workspace(qerl_rope_append_workspace_size(), k.device) if ws is None else ws
    check(qerl_rope_append(cache, q, k, v, positions, inv_freq, q_out, k_out, ws, seq_ids), "qerl_rope_append")
    return q_out, k_out


def decode_attention(cache, q, lengths, scale, ws=None):
    """(out, lse) of one new token per sequence over the cache (see qerl_decode_attention).  Lengths and pages
    outside the cache are recorded in ws."""
    n, h, d = q.shape
    out = torch.empty((n, h, d), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((n, h), dtype=torch.float32, device=q.device)
    ws = workspace(qerl_decode_attention_workspace_size(n, h, cache.num_kv_heads, d), q.device) if ws is None else ws
    check(qerl_decode_attention(cache, q, lengths, scale, out, lse, ws), "qerl_decode_attention")
    return out, lse


def prompt_attention(q, k, v, cu_seqlens, scale, ws=None):
    """(out, lse) of causal attention of packed sequences (see qerl_prompt_attention); rows of no sequence
    are 0 and -inf, and so is every row where the offsets step back or out, which is recorded in ws."""
    t, h, d = q.shape
    out = torch.zeros((t, h, d), dtype=torch.bfloat16, device=q.device)
    lse = torch.full((t, h), -float("inf"), dtype=torch.float32, device=q.device)
    n = cu_seqlens.numel() - 1
    ws = workspace(qerl_prompt_attention_workspace_size(t, h, k.shape[1], d, n), q.device) if ws is None else ws
    check(qerl_prompt_attention(q, k, v, cu_seqlens, scale, out, lse, ws), "qerl_prompt_attention")
    return out, lse
