"""ctypes binding of libattn.so (include/attn.h), with the same entry-point
names, plus allocating conveniences ``fwd`` / ``bwd``.

Only argument marshalling happens here: every step of the computation runs
in the library's CUDA kernels.  PyTorch supplies device memory and streams.
Loading fails loudly if the library has not been built; there is no other
implementation to fall back to.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import math
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libattn.so")

ATTN_F16, ATTN_BF16 = 0, 1
ATTN_OK = 0
ATTN_ERR_INVALID = -1
ATTN_ERR_UNSUPPORTED = -2
ATTN_ERR_ALIGN = -3
ATTN_ERR_CUDA = -4
ATTN_ERR_TIMEOUT = -5
ATTN_ERR_WORKSPACE = -6
ERROR_NAMES = {0: "ATTN_OK", -1: "ATTN_ERR_INVALID", -2: "ATTN_ERR_UNSUPPORTED",
               -3: "ATTN_ERR_ALIGN", -4: "ATTN_ERR_CUDA", -5: "ATTN_ERR_TIMEOUT",
               -6: "ATTN_ERR_WORKSPACE"}

# Kernel ids of attn_profile_end.
KERNEL_NAMES = ["attn_fwd", "attn_bwd_pre", "attn_bwd_main", "attn_dq_post",
                "attn_decode_split", "attn_decode_merge", "attn_pages_extend",
                "attn_pages_release", "attn_kv8_append", "attn_kv8_split", "attn_kv8_merge",
                "attn_varlen_merge"]


class AttnError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{ERROR_NAMES.get(code, code)}: {msg}")
        self.code = code


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is not built; run exact_tiled_attention_22_gb300.build.build() "
            "(needs nvcc).  There is no fallback implementation.")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp]
    lib.attn_fwd.restype = i
    lib.attn_bwd_workspace_size.argtypes = [i, i, i, i]
    lib.attn_bwd_workspace_size.restype = sz
    lib.attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp, sz, vp]
    lib.attn_bwd.restype = i
    lib.attn_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp]
    lib.attn_bwd_noalloc.restype = i
    lib.attn_fwd_alibi.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, i, vp]
    lib.attn_fwd_alibi.restype = i
    lib.attn_bwd_alibi.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, i, vp, sz, vp]
    lib.attn_bwd_alibi.restype = i
    lib.attn_decode_alibi.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, i, vp, sz, vp]
    lib.attn_decode_alibi.restype = i
    lib.attn_fwd_sparse.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, vp, i, vp]
    lib.attn_fwd_sparse.restype = i
    lib.attn_bwd_sparse.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, vp, i,
                                    vp, sz, vp]
    lib.attn_bwd_sparse.restype = i
    u64, u32 = ctypes.c_uint64, ctypes.c_uint32
    lib.attn_fwd_ex.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, vp, f, u64, u32, i, vp]
    lib.attn_fwd_ex.restype = i
    lib.attn_bwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, vp, f, u64,
                                u32, i, vp, sz, vp]
    lib.attn_bwd_ex.restype = i
    lib.attn_decode_workspace_size.argtypes = [i, i, i, i, i]
    lib.attn_decode_workspace_size.restype = sz
    lib.attn_decode.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, sz, vp]
    lib.attn_decode.restype = i
    lib.attn_status.argtypes = [vp]
    lib.attn_status.restype = i
    lib.attn_last_error_string.argtypes = []
    lib.attn_last_error_string.restype = ctypes.c_char_p
    lib.attn_set_wait_limit.argtypes = [ctypes.c_ulonglong, i]
    lib.attn_set_wait_limit.restype = i
    lib.attn_profile_begin.argtypes = []
    lib.attn_profile_begin.restype = i
    lib.attn_profile_end.argtypes = [ctypes.POINTER(i), ctypes.POINTER(ctypes.c_double), i]
    lib.attn_profile_end.restype = i
    lib.attn_fwd_acc.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, i, i, vp]
    lib.attn_fwd_acc.restype = i
    lib.attn_bwd_acc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, i, i, i, vp,
                                 sz, vp]
    lib.attn_bwd_acc.restype = i
    lib.attn_cast_acc.argtypes = [vp, vp, sz, f, i, vp]
    lib.attn_cast_acc.restype = i
    lib.attn_philox4x32_10.argtypes = [vp, vp, i, vp]
    lib.attn_philox4x32_10.restype = i
    ll = ctypes.c_longlong
    lib.attn_pages_extend.argtypes = [vp, vp, i, vp, i, vp, vp, i, i, ll, vp, vp, vp, vp, vp, vp]
    lib.attn_pages_extend.restype = i
    lib.attn_pages_release.argtypes = [vp, vp, i, vp, i, vp, vp, i, i, vp, vp, vp]
    lib.attn_pages_release.restype = i
    lib.attn_kv8_append.argtypes = [vp, vp, ll, ll, vp, ll, i, i, vp, vp, vp, vp, i, i, i, vp]
    lib.attn_kv8_append.restype = i
    lib.attn_kv8_decode_workspace_size.argtypes = [i, i, i, i]
    lib.attn_kv8_decode_workspace_size.restype = sz
    lib.attn_kv8_decode.argtypes = [vp] * 9 + [i] * 8 + [f, i, i, vp, sz, vp]
    lib.attn_kv8_decode.restype = i
    lib.attn_varlen_fwd_workspace_size.argtypes = [i, ll, ll, i, i, i]
    lib.attn_varlen_fwd_workspace_size.restype = sz
    lib.attn_varlen_fwd.argtypes = [vp] * 7 + [i, ll, ll, i, i, i, ll, ll, ll, f, i, i, vp, sz, vp]
    lib.attn_varlen_fwd.restype = i
    lib.attn_varlen_bwd_workspace_size.argtypes = [i, ll, i, i, i]
    lib.attn_varlen_bwd_workspace_size.restype = sz
    lib.attn_varlen_bwd.argtypes = [vp] * 11 + [i, ll, ll, i, i, i, ll, ll, ll, f, i, i, vp, sz, vp]
    lib.attn_varlen_bwd.restype = i
    return lib


lib = _load()


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


# The current stream's handle without building a torch.cuda.Stream (0.1 against
# 3.8 us on the GPU's Grace host, a third of a small call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None and torch.cuda.is_initialized():
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def dtype_code(dt) -> int:
    if dt in (torch.bfloat16, "bf16", ATTN_BF16):
        return ATTN_BF16
    if dt in (torch.float16, "fp16", ATTN_F16):
        return ATTN_F16
    raise ValueError(f"unsupported dtype {dt}")


def last_error() -> str:
    return (lib.attn_last_error_string() or b"").decode()


def attn_philox4x32_10(inp, out, n: int, stream=None) -> int:
    """Device uint32 [n, 6] (counter words, key words) -> [n, 4] outputs."""
    return lib.attn_philox4x32_10(_ptr(inp), _ptr(out), n, _stream(stream))


def check(rc: int) -> int:
    if rc != ATTN_OK:
        raise AttnError(rc, last_error())
    return rc


# ---- raw entry points (same names and argument order as include/attn.h) ----
def attn_fwd(q, k, v, o, lse, B, H, N, d, scale, causal, dtype, stream=None) -> int:
    return lib.attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                        float(scale), int(bool(causal)), dtype_code(dtype), _stream(stream))


def attn_bwd_workspace_size(B, H, N, d) -> int:
    return int(lib.attn_bwd_workspace_size(B, H, N, d))


def attn_bwd(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, scale, causal, dtype,
             workspace, workspace_bytes, stream=None) -> int:
    return lib.attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                        _ptr(dk), _ptr(dv), B, H, N, d, float(scale), int(bool(causal)),
                        dtype_code(dtype), _ptr(workspace), int(workspace_bytes),
                        _stream(stream))


# Bytes of the library-owned scratch array used by attn_bwd_noalloc.
NOALLOC_WORKSPACE_BYTES = 32 * 1024 * 1024


def attn_bwd_noalloc(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, scale, causal, dtype,
                     stream=None) -> int:
    """attn_bwd without a caller workspace (library-owned scratch array);
    for callers that cannot allocate device memory."""
    return lib.attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO),
                                _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, float(scale),
                                int(bool(causal)), dtype_code(dtype), _stream(stream))


def attn_fwd_alibi(q, k, v, o, lse, B, H, N, d, scale, causal, alibi_slopes, dtype,
                   stream=None) -> int:
    return lib.attn_fwd_alibi(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                              float(scale), int(bool(causal)), _ptr(alibi_slopes),
                              dtype_code(dtype), _stream(stream))


def attn_bwd_alibi(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, scale, causal, alibi_slopes,
                   dtype, workspace, workspace_bytes, stream=None) -> int:
    return lib.attn_bwd_alibi(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                              _ptr(dk), _ptr(dv), B, H, N, d, float(scale), int(bool(causal)),
                              _ptr(alibi_slopes), dtype_code(dtype), _ptr(workspace),
                              int(workspace_bytes), _stream(stream))


def attn_fwd_sparse(q, k, v, o, lse, B, H, N, d, scale, causal, alibi_slopes, block_mask, dtype,
                    stream=None) -> int:
    return lib.attn_fwd_sparse(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                               float(scale), int(bool(causal)), _ptr(alibi_slopes),
                               _ptr(block_mask), dtype_code(dtype), _stream(stream))


def attn_bwd_sparse(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, scale, causal, alibi_slopes,
                    block_mask, dtype, workspace, workspace_bytes, stream=None) -> int:
    return lib.attn_bwd_sparse(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                               _ptr(dk), _ptr(dv), B, H, N, d, float(scale), int(bool(causal)),
                               _ptr(alibi_slopes), _ptr(block_mask), dtype_code(dtype),
                               _ptr(workspace), int(workspace_bytes), _stream(stream))


def attn_fwd_ex(q, k, v, o, lse, B, H, N, d, scale, causal, alibi_slopes, block_mask, dropout_p,
                seed, offset, dtype, stream=None) -> int:
    return lib.attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                           float(scale), int(bool(causal)), _ptr(alibi_slopes), _ptr(block_mask),
                           float(dropout_p), int(seed), int(offset), dtype_code(dtype),
                           _stream(stream))


def attn_bwd_ex(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, scale, causal, alibi_slopes,
                block_mask, dropout_p, seed, offset, dtype, workspace, workspace_bytes,
                stream=None) -> int:
    return lib.attn_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                           _ptr(dk), _ptr(dv), B, H, N, d, float(scale), int(bool(causal)),
                           _ptr(alibi_slopes), _ptr(block_mask), float(dropout_p), int(seed),
                           int(offset), dtype_code(dtype), _ptr(workspace), int(workspace_bytes),
                           _stream(stream))


ATTN_ACC_FIRST, ATTN_ACC_LAST = 1, 2


def attn_fwd_acc(q, k, v, o_acc, lse, o, B, H, N, d, scale, causal, flags, dtype,
                 stream=None) -> int:
    return lib.attn_fwd_acc(_ptr(q), _ptr(k), _ptr(v), _ptr(o_acc), _ptr(lse), _ptr(o), B, H, N, d,
                            float(scale), int(bool(causal)), int(flags), dtype_code(dtype),
                            _stream(stream))


def attn_bwd_acc(q, k, v, o, lse, dO, dq, dk_acc, dv_acc, B, H, N, d, scale, causal, dq_flags,
                 kv_flags, dtype, workspace, workspace_bytes, stream=None) -> int:
    return lib.attn_bwd_acc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                            _ptr(dk_acc), _ptr(dv_acc), B, H, N, d, float(scale),
                            int(bool(causal)), int(dq_flags), int(kv_flags), dtype_code(dtype),
                            _ptr(workspace), int(workspace_bytes), _stream(stream))


def attn_cast_acc(acc, out, n, mul, dtype, stream=None) -> int:
    return lib.attn_cast_acc(_ptr(acc), _ptr(out), int(n), float(mul), dtype_code(dtype),
                             _stream(stream))


def attn_decode_alibi(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, alibi_slopes, dtype,
                      workspace, workspace_bytes, stream=None) -> int:
    return lib.attn_decode_alibi(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Nq, Nk, d,
                                 float(scale), int(bool(causal)), _ptr(alibi_slopes),
                                 dtype_code(dtype), _ptr(workspace), int(workspace_bytes),
                                 _stream(stream))


def attn_decode_workspace_size(B, H, Nq, Nk, d) -> int:
    return int(lib.attn_decode_workspace_size(B, H, Nq, Nk, d))


def attn_decode(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, dtype, workspace,
                workspace_bytes, stream=None) -> int:
    return lib.attn_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Nq, Nk, d,
                           float(scale), int(bool(causal)), dtype_code(dtype), _ptr(workspace),
                           int(workspace_bytes), _stream(stream))


def attn_pages_extend(lens, add, B, block_table, width, free_pages, free_count, free_cap, page, T,
                      new_lens, granted, cu_new, slots, free_left, stream=None) -> int:
    return lib.attn_pages_extend(_ptr(lens), _ptr(add), B, _ptr(block_table), width,
                                 _ptr(free_pages), _ptr(free_count), free_cap, page, T,
                                 _ptr(new_lens), _ptr(granted), _ptr(cu_new), _ptr(slots),
                                 _ptr(free_left), _stream(stream))


def attn_pages_release(lens, finished, B, block_table, width, free_pages, free_count, free_cap,
                       page, new_lens, free_left, stream=None) -> int:
    return lib.attn_pages_release(_ptr(lens), _ptr(finished), B, _ptr(block_table), width,
                                  _ptr(free_pages), _ptr(free_count), free_cap, page,
                                  _ptr(new_lens), _ptr(free_left), _stream(stream))


def attn_kv8_append(k, v, k_stride, v_stride, slots, T, H, d, k_cache, v_cache, k_scale, v_scale,
                    P, page, dtype, stream=None) -> int:
    return lib.attn_kv8_append(_ptr(k), _ptr(v), k_stride, v_stride, _ptr(slots), T, H, d,
                               _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), P, page,
                               dtype_code(dtype), _stream(stream))


def attn_kv8_decode_workspace_size(Nq, Hq, H, d) -> int:
    return int(lib.attn_kv8_decode_workspace_size(Nq, Hq, H, d))


def attn_kv8_decode(q, k_cache, v_cache, k_scale, v_scale, block_table, lens, o, lse, B, Nq, Hq, H,
                    d, P, page, width, scale, causal, dtype, workspace, workspace_bytes,
                    stream=None) -> int:
    return lib.attn_kv8_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                               _ptr(v_scale), _ptr(block_table), _ptr(lens), _ptr(o), _ptr(lse),
                               B, Nq, Hq, H, d, P, page, width, float(scale), int(bool(causal)),
                               dtype_code(dtype), _ptr(workspace), int(workspace_bytes),
                               _stream(stream))


def attn_varlen_fwd_workspace_size(B, Tq, Tk, Hq, Hkv, d) -> int:
    return int(lib.attn_varlen_fwd_workspace_size(B, Tq, Tk, Hq, Hkv, d))


def attn_varlen_fwd(q, k, v, o, lse, cu_q, cu_k, B, Tq, Tk, Hq, Hkv, d, q_stride, k_stride,
                    v_stride, scale, causal, dtype, workspace=None, workspace_bytes=0,
                    stream=None) -> int:
    return lib.attn_varlen_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_q),
                               _ptr(cu_k), B, Tq, Tk, Hq, Hkv, d, q_stride, k_stride, v_stride,
                               float(scale), int(bool(causal)), dtype_code(dtype),
                               _ptr(workspace), int(workspace_bytes), _stream(stream))


def attn_varlen_bwd_workspace_size(B, Tq, Hq, Hkv, d) -> int:
    return int(lib.attn_varlen_bwd_workspace_size(B, Tq, Hq, Hkv, d))


def attn_varlen_bwd(q, k, v, o, lse, dO, dq, dk, dv, cu_q, cu_k, B, Tq, Tk, Hq, Hkv, d, q_stride,
                    k_stride, v_stride, scale, causal, dtype, workspace, workspace_bytes,
                    stream=None) -> int:
    return lib.attn_varlen_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                               _ptr(dk), _ptr(dv), _ptr(cu_q), _ptr(cu_k), B, Tq, Tk, Hq, Hkv, d,
                               q_stride, k_stride, v_stride, float(scale), int(bool(causal)),
                               dtype_code(dtype), _ptr(workspace), int(workspace_bytes),
                               _stream(stream))


def attn_status(stream=None) -> int:
    return lib.attn_status(_stream(stream))


def attn_set_wait_limit(limit_ns: int, debug_flags: int = 0) -> int:
    return lib.attn_set_wait_limit(int(limit_ns), int(debug_flags))


def attn_profile_begin() -> int:
    return lib.attn_profile_begin()


def attn_profile_end():
    """Returns {kernel name: (launches, total ms)}."""
    n = len(KERNEL_NAMES)
    launches = (ctypes.c_int * n)()
    ms = (ctypes.c_double * n)()
    check(min(0, lib.attn_profile_end(launches, ms, n)))
    return {KERNEL_NAMES[i]: (launches[i], ms[i]) for i in range(n)}


# ---- allocating conveniences --------------------------------------------
def _shape(q):
    if q.dim() != 4 or not q.is_contiguous():
        raise ValueError("tensors must be contiguous [B, N, H, d]")
    B, N, H, d = q.shape
    return B, N, H, d


def _block_mask(block_mask, H, N):
    """None, or a contiguous uint8 CUDA tensor [H, nb, nb], nb = ceil(N / 128)."""
    if block_mask is None:
        return None
    nb = (N + 127) // 128
    if (block_mask.dtype != torch.uint8 or tuple(block_mask.shape) != (H, nb, nb)
            or not block_mask.is_contiguous() or not block_mask.is_cuda):
        raise ValueError(f"block_mask must be a contiguous uint8 CUDA tensor [{H}, {nb}, {nb}]")
    return block_mask


def fwd(q, k, v, scale=None, causal=False, stream=None, alibi=None, block_mask=None,
        dropout_p=0.0, seed=0, offset=0):
    """(o, lse) for contiguous [B, N, H, d] fp16/bf16 CUDA tensors.
    alibi: optional fp32 CUDA tensor [H] of ALiBi slopes.
    block_mask: optional uint8 CUDA tensor [H, nb, nb] over 128 x 128 blocks
    (0 removes a block).
    dropout_p, seed, offset: dropout of the probabilities (attn_fwd_ex)."""
    B, N, H, d = _shape(q)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    bm = _block_mask(block_mask, H, N)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    check(attn_fwd_ex(q, k, v, o, lse, B, H, N, d, scale, causal, alibi, bm, dropout_p, seed,
                      offset, q.dtype, stream))
    return o, lse


def workspace(B, H, N, d, device) -> torch.Tensor:
    n = attn_bwd_workspace_size(B, H, N, d)
    return torch.empty(n, dtype=torch.uint8, device=device)


def bwd(q, k, v, o, lse, do, scale=None, causal=False, ws=None, stream=None, alibi=None,
        block_mask=None, dropout_p=0.0, seed=0, offset=0):
    """(dq, dk, dv) for the forward that produced (o, lse) (same alibi,
    block_mask and dropout)."""
    B, N, H, d = _shape(q)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    bm = _block_mask(block_mask, H, N)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if ws is None:
        ws = workspace(B, H, N, d, q.device)
    check(attn_bwd_ex(q, k, v, o, lse, do, dq, dk, dv, B, H, N, d, scale, causal, alibi, bm,
                      dropout_p, seed, offset, q.dtype, ws, ws.numel(), stream))
    return dq, dk, dv


def decode(q, k, v, scale=None, causal=False, ws=None, stream=None, alibi=None):
    """(o, lse) of q [B, Nq, H, d] (the last Nq positions) against the cache
    k, v [B, Nk, H, d]."""
    B, Nq, H, d = _shape(q)
    Nk = k.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = torch.empty(attn_decode_workspace_size(B, H, Nq, Nk, d), dtype=torch.uint8,
                         device=q.device)
    check(attn_decode_alibi(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, alibi, q.dtype, ws,
                            ws.numel(), stream))
    return o, lse


# ---- serving and packed batches ---------------------------------------------
# The calls of attn_bind.so (csrc/attn_bind.cpp): they check the tensors (a
# ValueError says what is wrong), allocate outputs and workspaces on the current
# stream and call the entry points above.  Each takes stream=, the stream to run
# on instead of the current one.
# The module is loaded at the first of these calls: the dense calls need libattn.so
# only, not a torch whose C++ interface the module was built for.
@functools.cache
def _bind():
    path = os.path.join(os.path.dirname(LIB_PATH), "attn_bind.so")
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run exact_tiled_attention_22_gb300.build.build()")
    spec = importlib.util.spec_from_file_location("attn_bind", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.set_error(AttnError)
    return mod


def _on_stream(f):
    """A `stream` argument (a torch stream or a handle, of the tensors' device) is
    made the current stream for the call, so that what the call allocates belongs to it;
    tensors of other streams are marked as used there, so that freeing one after the
    call does not hand its memory on before the kernels have read it."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        given = [x for a in (*args, *kw.values()) for x in (a if isinstance(a, (tuple, list)) else (a,))
                 if isinstance(x, torch.Tensor)]
        dev = given[0].device if given else None
        if dev is None or any(x.device != dev or dev.type != "cuda" for x in given):
            return f(*args, **kw)  # refused there
        if isinstance(stream, int):
            stream = (torch.cuda.ExternalStream(stream, device=dev) if stream
                      else torch.cuda.default_stream(dev))
        if stream.device != dev:
            raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
        with torch.cuda.stream(stream):
            out = f(*args, **kw)
        for x in given:
            x.record_stream(stream)
        return out
    return call


@_on_stream
def pages_extend(lens, add, block_table, free_pages, free_count, page, max_new, new_lens=None,
                 free_left=None):
    """Pages and slots for add[b] new tokens of each request (attn_pages_extend).
    lens, add: int32 [B]; block_table: int32 [B, width], updated in place;
    free_pages: int32 [cap], a stack of free page ids, free_count: int32 [1];
    max_new: length of the slot map.  new_lens may be lens and free_left may
    be free_count.  Returns (new_lens, granted, cu_new, slots, free_left)."""
    return _bind().pages_extend(lens, add, block_table, free_pages, free_count, page, max_new,
                                new_lens, free_left)


@_on_stream
def pages_release(lens, finished, block_table, free_pages, free_count, page, new_lens=None,
                  free_left=None):
    """Pages of the requests with finished[b] != 0 (int32 [B]) go back onto the
    stack free_pages, written in place (attn_pages_release).  Returns (new_lens, free_left)."""
    return _bind().pages_release(lens, finished, block_table, free_pages, free_count, page, new_lens,
                                 free_left)


@_on_stream
def kv8_append(k, v, slots, k_cache, v_cache, k_scale, v_scale):
    """Rounds new keys and values [T, H, d] into their slots (int64 [T]) of the
    8-bit cache [P, H, page, d] with scales [P, H], in place (attn_kv8_append).
    k and v may be slices of a wider projection (any token stride that is a multiple of 8)."""
    _bind().kv8_append(k, v, slots, k_cache, v_cache, k_scale, v_scale)


@_on_stream
def kv8_decode(q, k_cache, v_cache, k_scale, v_scale, block_table, lens, scale=None, causal=True,
               ws=None):
    """(o, lse) of q [B, Nq, Hq, d], the last Nq tokens of every request, against
    the 8-bit cache (attn_kv8_decode); lens counts the Nq tokens."""
    return _bind().kv8_decode(q, k_cache, v_cache, k_scale, v_scale, block_table, lens, scale, causal,
                              ws)


@_on_stream
def varlen_fwd(q, k, v, cu_q, cu_k, scale=None, causal=False, ws=None, o=None):
    """(o, lse [Hq, Tq]) of packed sequences: q [Tq, Hq, d], k, v [Tk, Hkv, d]
    fp16/bf16 CUDA tensors (any token stride that is a multiple of d), cu_q, cu_k
    int32 [B + 1] row offsets on the device (attn_varlen_fwd).  o: an output to
    write into; rows of no sequence are left as they are there."""
    return _bind().varlen_fwd(q, k, v, cu_q, cu_k, scale, causal, ws, o)


@_on_stream
def varlen_bwd(q, k, v, o, lse, do, cu_q, cu_k, scale=None, causal=False, ws=None, grads=None):
    """(dq, dk, dv) for the varlen_fwd that produced (o, lse).  grads: three
    contiguous tensors to write into (rows of no sequence are left as they are)."""
    dq, dk, dv = (None, None, None) if grads is None else grads
    return _bind().varlen_bwd(q, k, v, o, lse, do, cu_q, cu_k, scale, causal, ws, dq, dk, dv)


# ---- autograd -------------------------------------------------------------
class _SecondDerivative(torch.autograd.Function):
    """Hands gradients on unchanged; whoever differentiates them gets an error."""

    @staticmethod
    def forward(ctx, dq, dk, dv, *sources):
        return dq.view_as(dq), dk.view_as(dk), dv.view_as(dv)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("attention can be differentiated once, not twice: its backward is a kernel "
                           "without a derivative")


def _once(backward):
    """A backward pass whose results refuse to be differentiated.  (torch's
    once_differentiable lets them pass as constants where the incoming gradient is
    one, although they depend on q, k and v.)"""
    @functools.wraps(backward)
    def call(ctx, do):
        saved = ctx.saved_tensors  # (once: a checkpointed forward hands them out only once)
        with torch.no_grad():
            grads = backward(ctx, do, *saved)
        if torch.is_grad_enabled():  # create_graph=True
            grads = (*_SecondDerivative.apply(*grads[:3], do, *saved[:3]), *grads[3:])
        return grads
    return call


class AttentionFunction(torch.autograd.Function):
    """O = attention(q, k, v) with the backward of the library (attn_bwd_ex):
    saves q, k, v, O and LSE (O(N) extra state), never P."""

    @staticmethod
    def forward(ctx, q, k, v, scale, causal, alibi, block_mask, dropout_p, seed, offset):
        o, lse = fwd(q, k, v, scale, causal, alibi=alibi, block_mask=block_mask,
                     dropout_p=dropout_p, seed=seed, offset=offset)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.opts = (scale, causal, alibi, block_mask, dropout_p, seed, offset)
        return o

    @staticmethod
    @_once
    def backward(ctx, do, q, k, v, o, lse):
        scale, causal, alibi, block_mask, dropout_p, seed, offset = ctx.opts
        dq, dk, dv = bwd(q, k, v, o, lse, do.contiguous(), scale, causal, alibi=alibi,
                         block_mask=block_mask, dropout_p=dropout_p, seed=seed, offset=offset)
        return dq, dk, dv, None, None, None, None, None, None, None


def attention(q, k, v, scale=None, causal=False, alibi=None, block_mask=None, dropout_p=0.0,
              seed=0, offset=0):
    """Differentiable attention on contiguous [B, N, H, d] fp16/bf16 CUDA
    tensors (forward and backward in the library's kernels).  The backward has no
    derivative of its own: asking for a second one raises."""
    return AttentionFunction.apply(q, k, v, scale, causal, alibi, block_mask, dropout_p, seed,
                                   offset)


class VarlenAttentionFunction(torch.autograd.Function):
    """Packed attention with the backward of the library (attn_varlen_bwd).
    Rows of no sequence (padding behind the last one) have zero output and zero
    gradients here, so that they add nothing to the parameters' gradients: o and the
    gradients are filled first, four launches and about 20 us of a 7457-token step's 331
    (16 / 4 heads, d 128) beside varlen_fwd and varlen_bwd."""

    @staticmethod
    def forward(ctx, q, k, v, cu_q, cu_k, scale, causal):
        o, lse = varlen_fwd(q, k, v, cu_q, cu_k, scale, causal,
                            o=torch.zeros(q.shape, dtype=q.dtype, device=q.device))
        ctx.save_for_backward(q, k, v, o, lse, cu_q, cu_k)
        ctx.opts = (scale, causal)
        return o

    @staticmethod
    @_once
    def backward(ctx, do, q, k, v, o, lse, cu_q, cu_k):
        grads = [torch.zeros(x.shape, dtype=x.dtype, device=x.device) for x in (q, k, v)]
        dq, dk, dv = varlen_bwd(q, k, v, o, lse, do.contiguous(), cu_q, cu_k, *ctx.opts,
                                grads=grads)
        return dq, dk, dv, None, None, None, None


def attention_varlen(q, k, v, cu_q, cu_k, scale=None, causal=False):
    """Differentiable attention on packed sequences (see varlen_fwd), once: asking
    for a second derivative raises.  A training
    step may be captured into a CUDA graph, forward and backward together; as for
    every torch operator, no autograd graph of the same leaves from before the
    capture may still be alive then (drop its loss first): torch would run their
    gradient accumulation on the stream of that graph, outside the capture."""
    return VarlenAttentionFunction.apply(q, k, v, cu_q, cu_k, scale, causal)
