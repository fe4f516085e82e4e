"""ctypes binding of libfp8mla.so with the same names as the C ABI (include/fp8mla.h).

Argument marshalling only: tensors are checked for device, dtype and layout,
their device pointers and the current CUDA stream are passed through, and a
non-zero status raises.  Every step of the computation runs in the library's
CUDA kernels; there is no CPU fallback, and a missing library or missing CUDA
device raises instead of computing anything.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

from . import build as _build

KV8_DL, KV8_DR, KV8_D, KV8_BLOCK = 512, 64, 576, 64
KV8_DECODE_AUTO, KV8_DECODE_SIMT, KV8_DECODE_TCGEN05 = 0, 1, 2
KV8_DECODE_TCGEN05_CTA, KV8_DECODE_TCGEN05_PAIR = 3, 4
STATUS = {0: "KV8_OK", -1: "KV8_EINVAL", -2: "KV8_EALIGN", -3: "KV8_EUNSUPPORTED",
          -4: "KV8_ECUDA", -5: "KV8_EBOUNDS", -6: "KV8_EWORKSPACE", -7: "KV8_ETIMEOUT",
          -8: "KV8_ESCRATCH", -9: "KV8_EIO", -10: "KV8_EFORMAT"}
KV8_PAGES_EINDEX, KV8_PAGES_ENOROOM, KV8_PAGES_ETIMEOUT = 1, 2, 4  # bits of the pages' err_word

_lock = threading.Lock()
_lib = None


class Kv8Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = lib().kv8_status_string(status).decode()
        if status in (-3, -4):
            msg += ", " + lib().kv8_last_cuda_error().decode()
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} ({msg})")


def lib() -> ctypes.CDLL:
    """Load libfp8mla.so, building it in-tree first if it is missing or stale."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not _build.up_to_date():
                _build.build()
            L = ctypes.CDLL(_build.LIB)
            P, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
            sig = {
                "kv8_quantize_rows": (i32, [P, i64, i64, P, P, P, i64, P]),
                "kv8_produce_rows": (i32, [P, i64, i64, P, ctypes.c_float, P, P, P, i64, P, P, P,
                                           i64, P, P]),
                "mla_wuv_epilogue": (i32, [P, P, i32, i32, i32, P, P]),
                "kv8_selftest_wait_timeout": (i32, [P, i64, i64, P]),
                "kv8_prefill_project": (i32, [P, P, i64, P, i64, P, i32, P, P, P, P]),
                "mla_absorb_decode_fp8_workspace_size": (i64, [i64, i32, i32]),
                "mla_absorb_decode_fp8": (i32, [P, P, P, P, i64, i32, f32, P, P, P, i64, i32, P]),
                "mla_absorb_decode_fp8_batch_workspace_size": (i64, [i32, i32, i32, i32, i32]),
                "mla_absorb_decode_fp8_batch": (i32, [P, P, P, P, P, P, i32, i32, i32, i32, i64, f32,
                                                      P, P, P, i64, i32, P]),
                "mla_absorb_decode_fp8_batch_partials": (i32, [P, P, P, P, P, P, i32, i32, i32, i32,
                                                               i64, f32, P, i64, i32, P]),
                "mla_absorb_decode_fp8_batch_combine": (i32, [P, i32, i32, i32, i32, P, P, P, i64,
                                                              i32, P]),
                "mla_absorb_decode_fp8_batch_noalloc": (i32, [P, P, P, P, P, P, i32, i32, i32, i32,
                                                              i64, f32, P, P, i32, P]),
                "mla_absorb_chunk_fp8_batch_workspace_size": (i64, [i32, i32, i64, i32]),
                "mla_absorb_chunk_fp8_batch": (i32, [P, i64, i64, P, i64, i64, P, P, P, P, P, i64, i32,
                                                     i32, i32, i32, i64, i32, f32, P, P, P, i64, P]),
                "kv8_pages_append": (i32, [P, P, P, i32, i32, i64, P, P, P, i64, P, P]),
                "kv8_pages_fork": (i32, [P, P, P, i32, i32, i64, P, P, P, i32, P, P, P, P]),
                "kv8_pages_free": (i32, [P, P, P, i32, i32, i64, P, i32, P, P]),
                "kv8_pages_compact": (i32, [P, P, P, i32, i32, i64, P, P, P, P, P]),
                "kv8_pages_copy": (i32, [P, P, i32, i64, P, P, i64, P, P]),
                "kv8_noalloc_error": (i32, [P]),
                "kv8_workspace_error": (i32, [P, P]),
                "kv8_disk_open": (i32, [ctypes.c_char_p, i64, ctypes.POINTER(P)]),
                "kv8_disk_info": (i32, [P, ctypes.POINTER(i64), ctypes.POINTER(i32)]),
                "kv8_disk_append": (i32, [P, P, P, i64, P, i64, P]),
                "kv8_disk_load": (i32, [P, i64, i64, P, P, i64, P, P]),
                "kv8_disk_close": (i32, [P]),
                "kv8_status_string": (ctypes.c_char_p, [i32]),
                "kv8_last_cuda_error": (ctypes.c_char_p, []),
                "kv8_abi_version": (i32, []),
            }
            for name, (res, args) in sig.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def library_path() -> str:
    return os.path.abspath(_build.LIB)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:  # (the handle alone: a Stream object costs 3 us a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _is_device(t) -> bool:
    """Whether a tensor lives in device memory (the one place the binding asks)."""
    return t.is_cuda


def _need(t, name, dtype, ndim=None, device=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device and not _is_device(t):
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def _need_cache(kv_codes, kv_scales):
    """The cache: codes uint8 [slots, 576] and their row scales f32 [slots, 2]."""
    _need(kv_codes, "kv_codes", torch.uint8, 2)
    _need(kv_scales, "kv_scales", torch.float32, 2)
    if kv_codes.shape[1] != KV8_D or tuple(kv_scales.shape) != (kv_codes.shape[0], 2):
        raise ValueError("kv_codes must be [slots,576] and kv_scales [slots,2]")


def _need_workspace(ws):
    """A caller's workspace: a contiguous CUDA tensor of any dtype (its size is
    checked by the library against the call's need)."""
    if not isinstance(ws, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if not _is_device(ws):
        raise ValueError("workspace must be a CUDA tensor (the library has no CPU path)")
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")


def _check(fn, status):
    if status != 0:
        raise Kv8Error(fn, status)


# ----------------------------------------------------------------- quantizer
def kv8_quantize_rows(src, kv_codes, kv_scales, dst_slot=None, stream=None):
    """Quantize f32 rows src [n, >=576] (row stride = src.stride(0)) into the cache."""
    if not (isinstance(src, torch.Tensor) and src.dtype == torch.float32 and _is_device(src)
            and src.dim() == 2 and src.stride(1) == 1
            and src.shape[1] >= KV8_D):
        raise ValueError("src must be a CUDA float32 [n, >=576] tensor with unit column stride")
    _need_cache(kv_codes, kv_scales)
    if dst_slot is not None:
        _need(dst_slot, "dst_slot", torch.int64, 1)
        if dst_slot.numel() != src.shape[0]:
            raise ValueError("dst_slot must have one entry per source row")
    st = lib().kv8_quantize_rows(_ptr(src), src.shape[0], src.stride(0), _ptr(dst_slot),
                                 _ptr(kv_codes), _ptr(kv_scales), kv_codes.shape[0],
                                 _stream(stream))
    _check("kv8_quantize_rows", st)


def kv8_produce_rows(src, norm_weight, eps, positions, rope_cos, rope_sin, kv_codes, kv_scales,
                     dst_slot=None, err_word=None, stream=None):
    """Fused producer: RMS norm (Lc) + rotary pairs (Rc) + quantize raw rows src [n, >=576]."""
    if not (isinstance(src, torch.Tensor) and src.dtype == torch.float32 and _is_device(src)
            and src.dim() == 2 and src.stride(1) == 1
            and src.shape[1] >= KV8_D):
        raise ValueError("src must be a CUDA float32 [n, >=576] tensor with unit column stride")
    _need(norm_weight, "norm_weight", torch.float32, 1)
    _need(positions, "positions", torch.int64, 1)
    _need(rope_cos, "rope_cos", torch.float32, 2)
    _need(rope_sin, "rope_sin", torch.float32, 2)
    _need_cache(kv_codes, kv_scales)
    if norm_weight.numel() != KV8_DL:
        raise ValueError("norm_weight must have 512 entries")
    if positions.numel() != src.shape[0]:
        raise ValueError("positions must have one entry per source row")
    if rope_cos.shape != rope_sin.shape or rope_cos.shape[1] != KV8_DR // 2:
        raise ValueError("rope_cos and rope_sin must both be [max_pos, 32]")
    if dst_slot is not None:
        _need(dst_slot, "dst_slot", torch.int64, 1)
        if dst_slot.numel() != src.shape[0]:
            raise ValueError("dst_slot must have one entry per source row")
    if err_word is not None and not (isinstance(err_word, torch.Tensor) and _is_device(err_word)
                                     and err_word.dtype == torch.int32 and err_word.numel() >= 1):
        raise ValueError("err_word must be a CUDA int32 tensor")
    st = lib().kv8_produce_rows(_ptr(src), src.shape[0], src.stride(0), _ptr(norm_weight),
                                float(eps), _ptr(positions), _ptr(rope_cos), _ptr(rope_sin),
                                rope_cos.shape[0], _ptr(dst_slot), _ptr(kv_codes),
                                _ptr(kv_scales), kv_codes.shape[0], _ptr(err_word),
                                _stream(stream))
    _check("kv8_produce_rows", st)


def kv8_prefill_project(kv_codes, kv_scales, w_ukv, T=None, slots=None, y=None, k_rope=None,
                        err_word=None, stream=None):
    """Y [T, N] bf16 = dequantized cached latent (slots or 0..T-1) @ W_UKV (bf16 [512, N]);
    k_rope (optional f32 [T, 64]) receives the dequantized rope keys."""
    _need_cache(kv_codes, kv_scales)
    if not (isinstance(w_ukv, torch.Tensor) and _is_device(w_ukv) and w_ukv.dim() == 2
            and w_ukv.dtype == torch.bfloat16 and w_ukv.is_contiguous() and w_ukv.shape[0] == KV8_DL):
        raise ValueError("w_ukv must be a contiguous CUDA bfloat16 [512, N] tensor")
    if slots is not None:
        _need(slots, "slots", torch.int64, 1)
        T = slots.numel()
    elif T is None:
        T = kv_codes.shape[0]
    N = w_ukv.shape[1]
    if y is None:
        y = torch.empty((T, N), dtype=torch.bfloat16, device=kv_codes.device)
    if not (y.dtype == torch.bfloat16 and _is_device(y) and y.is_contiguous() and tuple(y.shape) == (T, N)):
        raise ValueError("y must be a contiguous CUDA bfloat16 [T, N] tensor")
    if k_rope is not None and not (k_rope.dtype == torch.float32 and _is_device(k_rope)
                                   and k_rope.is_contiguous() and tuple(k_rope.shape) == (T, KV8_DR)):
        raise ValueError("k_rope must be a contiguous CUDA float32 [T, 64] tensor")
    if err_word is not None and not (isinstance(err_word, torch.Tensor) and _is_device(err_word)
                                     and err_word.dtype == torch.int32 and err_word.numel() >= 1):
        raise ValueError("err_word must be a CUDA int32 tensor")
    st = lib().kv8_prefill_project(_ptr(kv_codes), _ptr(kv_scales), kv_codes.shape[0], _ptr(slots),
                                   int(T), _ptr(w_ukv), int(N), _ptr(y), _ptr(k_rope),
                                   _ptr(err_word), _stream(stream))
    _check("kv8_prefill_project", st)
    return y


def kv8_selftest_wait_timeout(workspace, limit_us: int, stream=None):
    """Run the bounded-wait failure check; afterwards kv8_workspace_error(workspace) is -7."""
    _need(workspace, "workspace", torch.uint8, 1)
    st = lib().kv8_selftest_wait_timeout(_ptr(workspace), workspace.numel(), int(limit_us),
                                         _stream(stream))
    _check("kv8_selftest_wait_timeout", st)


def mla_wuv_epilogue(o, w_uv, y=None, stream=None):
    """Per-head value projection y[b,h,:] = o[b,h,:] @ W_UV[h]; o f32 [B,H,512], w_uv bf16 [H,512,V]."""
    _need(o, "o", torch.float32, 3)
    if not (isinstance(w_uv, torch.Tensor) and _is_device(w_uv) and w_uv.dim() == 3
            and w_uv.dtype in (torch.bfloat16, torch.int16, torch.uint16)
            and w_uv.is_contiguous()):
        raise ValueError("w_uv must be a contiguous CUDA bfloat16 [H, 512, V] tensor")
    B, H, dl = o.shape
    if dl != KV8_DL or w_uv.shape[0] != H or w_uv.shape[1] != KV8_DL:
        raise ValueError("shapes must be o [B, H, 512] and w_uv [H, 512, V]")
    V = w_uv.shape[2]
    if y is None:
        y = torch.empty((B, H, V), dtype=torch.float32, device=o.device)
    _need(y, "y", torch.float32, 3)
    if tuple(y.shape) != (B, H, V):
        raise ValueError("y must be [B, H, V]")
    st = lib().mla_wuv_epilogue(_ptr(o), _ptr(w_uv), B, H, V, _ptr(y), _stream(stream))
    _check("mla_wuv_epilogue", st)
    return y


# ----------------------------------------------------------------- decode
def mla_absorb_decode_fp8_workspace_size(T: int, H: int, variant: int = KV8_DECODE_AUTO) -> int:
    n = lib().mla_absorb_decode_fp8_workspace_size(int(T), int(H), int(variant))
    if n < 0:
        raise ValueError("invalid T, H or variant")
    return int(n)


def mla_absorb_decode_fp8_batch_workspace_size(B: int, H: int, max_blocks: int,
                                               block_size: int = KV8_BLOCK,
                                               variant: int = KV8_DECODE_AUTO) -> int:
    n = lib().mla_absorb_decode_fp8_batch_workspace_size(int(B), int(H), int(max_blocks),
                                                         int(block_size), int(variant))
    if n < 0:
        raise ValueError("invalid B, H, max_blocks, block_size or variant")
    return int(n)


def alloc_workspace(nbytes: int, device=None) -> torch.Tensor:
    # torch's caching allocator returns 512-byte aligned blocks
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


def mla_absorb_decode_fp8(q_lat, q_rope, kv_codes, kv_scales, T, sm_scale, out=None, lse=None,
                          workspace=None, variant=KV8_DECODE_AUTO, stream=None):
    """One query (q_lat [H,512], q_rope [H,64]) against kv rows 0..T-1 -> out [H,512]."""
    _need(q_lat, "q_lat", torch.float32, 2)
    _need(q_rope, "q_rope", torch.float32, 2)
    _need_cache(kv_codes, kv_scales)
    H = q_lat.shape[0]
    if q_lat.shape[1] != KV8_DL or tuple(q_rope.shape) != (H, KV8_DR):
        raise ValueError("q_lat must be [H,512] and q_rope [H,64]")
    if T > kv_codes.shape[0] or T > kv_scales.shape[0]:
        raise ValueError("T exceeds the cache rows")
    if out is None:
        out = torch.empty((H, KV8_DL), dtype=torch.float32, device=q_lat.device)
    _need(out, "out", torch.float32, 2)
    if tuple(out.shape) != (H, KV8_DL):
        raise ValueError("out must be [H,512]")
    if lse is not None:
        _need(lse, "lse", torch.float32, 1)
        if lse.shape[0] != H:
            raise ValueError("lse must be [H]")
    need = mla_absorb_decode_fp8_workspace_size(T, H, variant)
    if workspace is None:
        workspace = alloc_workspace(need, q_lat.device)
    _need_workspace(workspace)
    st = lib().mla_absorb_decode_fp8(_ptr(q_lat), _ptr(q_rope), _ptr(kv_codes), _ptr(kv_scales),
                                     int(T), H, float(sm_scale), _ptr(out), _ptr(lse),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     int(variant), _stream(stream))
    _check("mla_absorb_decode_fp8", st)
    return out


def _batch_inputs(q_lat, q_rope, kv_codes, kv_scales, block_table, seq_lens, out=None, lse=None,
                  outputs=True):
    """The checks every batched decode wrapper runs: dtypes, shapes and one row per
    sequence (and of out / lse when the call writes them); returns (B, H, out), out
    allocated if None."""
    _need(q_lat, "q_lat", torch.float32, 3)
    _need(q_rope, "q_rope", torch.float32, 3)
    _need_cache(kv_codes, kv_scales)
    _need(block_table, "block_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    B, H = q_lat.shape[:2]
    if q_lat.shape[2] != KV8_DL or tuple(q_rope.shape) != (B, H, KV8_DR):
        raise ValueError("q_lat must be [B,H,512] and q_rope [B,H,64]")
    if block_table.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_table and seq_lens need one row per sequence")
    if not outputs:
        return B, H, None
    if out is None:
        out = torch.empty((B, H, KV8_DL), dtype=torch.float32, device=q_lat.device)
    _need(out, "out", torch.float32, 3)
    if tuple(out.shape) != (B, H, KV8_DL):
        raise ValueError("out must be [B,H,512]")
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
        if tuple(lse.shape) != (B, H):
            raise ValueError("lse must be [B,H]")
    return B, H, out


def mla_absorb_decode_fp8_batch(q_lat, q_rope, kv_codes, kv_scales, block_table, seq_lens,
                                sm_scale, out=None, lse=None, workspace=None,
                                variant=KV8_DECODE_AUTO, block_size=KV8_BLOCK, stream=None):
    """B queries (q_lat [B,H,512], q_rope [B,H,64]) over a paged cache -> out [B,H,512]."""
    B, H, out = _batch_inputs(q_lat, q_rope, kv_codes, kv_scales, block_table, seq_lens, out, lse)
    max_blocks = block_table.shape[1]
    n_blocks = kv_codes.shape[0] // block_size
    need = mla_absorb_decode_fp8_batch_workspace_size(B, H, max_blocks, block_size, variant)
    if workspace is None:
        workspace = alloc_workspace(need, q_lat.device)
    _need_workspace(workspace)
    st = lib().mla_absorb_decode_fp8_batch(
        _ptr(q_lat), _ptr(q_rope), _ptr(kv_codes), _ptr(kv_scales), _ptr(block_table),
        _ptr(seq_lens), B, H, max_blocks, int(block_size), int(n_blocks), float(sm_scale),
        _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
        int(variant), _stream(stream))
    _check("mla_absorb_decode_fp8_batch", st)
    return out


def mla_absorb_decode_fp8_batch_partials(q_lat, q_rope, kv_codes, kv_scales, block_table,
                                         seq_lens, sm_scale, workspace,
                                         variant=KV8_DECODE_AUTO, block_size=KV8_BLOCK,
                                         stream=None):
    """Split phase 1: the split-T kernel only; partials stay in ``workspace``."""
    B, H, _ = _batch_inputs(q_lat, q_rope, kv_codes, kv_scales, block_table, seq_lens,
                            outputs=False)
    _need_workspace(workspace)
    st = lib().mla_absorb_decode_fp8_batch_partials(
        _ptr(q_lat), _ptr(q_rope), _ptr(kv_codes), _ptr(kv_scales), _ptr(block_table),
        _ptr(seq_lens), B, H, block_table.shape[1], int(block_size),
        int(kv_codes.shape[0] // block_size), float(sm_scale), _ptr(workspace),
        workspace.numel() * workspace.element_size(), int(variant), _stream(stream))
    _check("mla_absorb_decode_fp8_batch_partials", st)


def mla_absorb_decode_fp8_batch_combine(seq_lens, H, max_blocks, out, lse, workspace,
                                        variant=KV8_DECODE_AUTO, block_size=KV8_BLOCK,
                                        stream=None):
    """Split phase 2: merge the workspace partials into ``out`` / ``lse``."""
    _need(seq_lens, "seq_lens", torch.int32, 1)
    B = seq_lens.shape[0]
    _need(out, "out", torch.float32, 3)
    if tuple(out.shape) != (B, int(H), KV8_DL):
        raise ValueError("out must be [B,H,512], B = len(seq_lens)")
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
        if tuple(lse.shape) != (B, int(H)):
            raise ValueError("lse must be [B,H]")
    _need_workspace(workspace)
    st = lib().mla_absorb_decode_fp8_batch_combine(
        _ptr(seq_lens), seq_lens.shape[0], int(H), int(max_blocks), int(block_size), _ptr(out),
        _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(), int(variant),
        _stream(stream))
    _check("mla_absorb_decode_fp8_batch_combine", st)


def kv8_workspace_error(workspace, stream=None) -> int:
    _need_workspace(workspace)
    return int(lib().kv8_workspace_error(_ptr(workspace), _stream(stream)))


def mla_absorb_decode_fp8_batch_noalloc(q_lat, q_rope, kv_codes, kv_scales, block_table, seq_lens,
                                        sm_scale, out=None, lse=None, variant=KV8_DECODE_AUTO,
                                        block_size=KV8_BLOCK, stream=None):
    """The batched decode without a caller workspace (for callers that cannot
    allocate device memory): partials go to the library's static device scratch."""
    B, H, out = _batch_inputs(q_lat, q_rope, kv_codes, kv_scales, block_table, seq_lens, out, lse)
    st = lib().mla_absorb_decode_fp8_batch_noalloc(
        _ptr(q_lat), _ptr(q_rope), _ptr(kv_codes), _ptr(kv_scales), _ptr(block_table),
        _ptr(seq_lens), B, H, block_table.shape[1], int(block_size),
        int(kv_codes.shape[0] // block_size), float(sm_scale), _ptr(out), _ptr(lse), int(variant),
        _stream(stream))
    _check("mla_absorb_decode_fp8_batch_noalloc", st)
    return out


def _strides(t):
    """Element strides of the first two dimensions (0 for one of size 1, whose stride says nothing)."""
    a, b = t.stride()[:2]
    rows, heads = t.shape[:2]
    return a if rows > 1 else 0, b if heads > 1 else 0


_AS_IS = contextlib.nullcontext()


def _allocating(stream):
    """What a call allocates for itself, while it is to run on `stream`, is that stream's memory: what
    the current one frees may still be in use there."""
    return torch.cuda.stream(stream) if isinstance(stream, torch.cuda.Stream) else _AS_IS


def _on_device_of(first, *others):
    """The device of a call's tensors, made current for it (its launch, its default stream)."""
    d = first.get_device()
    for t in others:
        if t is not None and t.get_device() != d:
            raise ValueError("all tensors must be on the same device")
    return torch.cuda.device(d) if d >= 0 and d != torch.cuda.current_device() else _AS_IS


# ----------------------------------------------------------------- chunks of new tokens
def mla_absorb_chunk_fp8_batch_workspace_size(B: int, H: int, total_q: int, max_blocks: int) -> int:
    n = lib().mla_absorb_chunk_fp8_batch_workspace_size(int(B), int(H), int(total_q), int(max_blocks))
    if n < 0:
        raise ValueError("invalid B, H, total_q or max_blocks")
    return int(n)


def mla_absorb_chunk_fp8_batch(q_lat, q_rope, kv_codes, kv_scales, block_table, seq_lens, q_start,
                               sm_scale, causal=True, out=None, lse=None, workspace=None,
                               block_size=KV8_BLOCK, stream=None):
    """The new tokens of B sequences (bf16 q_lat [total_q,H,512], q_rope [total_q,H,64], sequence
    b's rows q_start[b]..q_start[b+1]-1) over a paged cache that holds them -> bf16 out
    [total_q,H,512].  The queries may be strided views whose last dimension is contiguous.  Bad
    table entries, lengths and query ranges, and timeouts, are told by kv8_workspace_error(workspace)
    alone: without a workspace of the caller's they are not heard of."""
    for t, name, width in ((q_lat, "q_lat", KV8_DL), (q_rope, "q_rope", KV8_DR)):
        if not (isinstance(t, torch.Tensor) and t.dtype == torch.bfloat16 and _is_device(t)
                and t.dim() == 3 and t.shape[2] == width and t.stride(2) == 1):
            raise ValueError(f"{name} must be a CUDA bfloat16 [total_q, H, {width}] tensor with unit "
                             "stride in its last dimension")
    _need_cache(kv_codes, kv_scales)
    _need(block_table, "block_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(q_start, "q_start", torch.int32, 1)
    rows, H, _ = q_lat.shape
    B, max_blocks = block_table.shape
    if q_rope.shape[0] != rows or q_rope.shape[1] != H:
        raise ValueError("q_lat must be [total_q,H,512] and q_rope [total_q,H,64]")
    if seq_lens.shape[0] != B or q_start.shape[0] != B + 1:
        raise ValueError("seq_lens needs one entry per row of block_table, and q_start one more")
    if out is None:
        with _allocating(stream):
            out = torch.empty((rows, H, KV8_DL), dtype=torch.bfloat16, device=q_lat.device)
    else:
        _need(out, "out", torch.bfloat16, 3)
        if out.shape != (rows, H, KV8_DL):
            raise ValueError("out must be [total_q,H,512]")
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
        if lse.shape != (rows, H):
            raise ValueError("lse must be [total_q,H]")
    need = mla_absorb_chunk_fp8_batch_workspace_size(B, H, rows, max_blocks)
    if workspace is None:
        with _allocating(stream):
            workspace = alloc_workspace(need, q_lat.device)
    _need_workspace(workspace)
    with _on_device_of(q_lat, q_rope, kv_codes, kv_scales, block_table, seq_lens, q_start, out, lse,
                       workspace):
        st = lib().mla_absorb_chunk_fp8_batch(
            _ptr(q_lat), *_strides(q_lat), _ptr(q_rope), *_strides(q_rope), _ptr(kv_codes),
            _ptr(kv_scales), _ptr(block_table), _ptr(seq_lens), _ptr(q_start), rows, B, H, max_blocks,
            int(block_size), int(kv_codes.shape[0] // block_size), int(bool(causal)),
            float(sm_scale), _ptr(out), _ptr(lse), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream))
    _check("mla_absorb_chunk_fp8_batch", st)
    return out


# ----------------------------------------------------------------- pages
def _page_table(block_table, seq_lens, page_refs, err_word):
    """The checks of every call on a page table; its C arguments."""
    _need(block_table, "block_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(page_refs, "page_refs", torch.int32, 1)
    if seq_lens.shape[0] != block_table.shape[0]:
        raise ValueError("seq_lens must have one entry per row of block_table")
    _need_err(err_word)
    return (_ptr(block_table), _ptr(seq_lens), _ptr(page_refs), block_table.shape[0],
            block_table.shape[1], page_refs.shape[0])


def _need_err(err_word):
    if err_word is not None and not (isinstance(err_word, torch.Tensor) and _is_device(err_word)
                                     and err_word.dtype == torch.int32 and err_word.numel() >= 1):
        raise ValueError("err_word must be a CUDA int32 tensor")


def _moves_out(moves, n_moves, room, device, stream):
    """The list a call writes its page moves to, and their count; allocated if None."""
    with _allocating(stream):
        if moves is None:
            moves = torch.empty((max(room, 1), 2), dtype=torch.int32, device=device)
        if n_moves is None:
            n_moves = torch.empty(1, dtype=torch.int32, device=device)
    _need(moves, "moves", torch.int32, 2)
    _need(n_moves, "n_moves", torch.int32, 1)
    if moves.shape[1] != 2 or moves.shape[0] < room:
        raise ValueError(f"moves must be [>= {room}, 2]")
    if n_moves.numel() < 1:
        raise ValueError("n_moves must have one entry")
    return moves, n_moves


def kv8_pages_append(block_table, seq_lens, page_refs, n_new, cap=None, q_start=None, dst_slot=None,
                     err_word=None, stream=None):
    """Room for n_new[b] more tokens of every sequence: pages taken, seq_lens raised.  Returns
    (q_start int32 [B+1], dst_slot int64 [cap]): where each sequence's new rows start, and the
    cache slots of the new tokens in that order (-1 behind the last).  Give dst_slot or cap.  An
    append that cannot be gives no token a slot (q_start all 0) and says so in err_word alone."""
    table = _page_table(block_table, seq_lens, page_refs, err_word)
    B = table[3]
    _need(n_new, "n_new", torch.int32, 1)
    if n_new.shape[0] != B:
        raise ValueError("n_new must have one entry per sequence")
    if q_start is None:
        with _allocating(stream):
            q_start = torch.empty(B + 1, dtype=torch.int32, device=n_new.device)
    _need(q_start, "q_start", torch.int32, 1)
    if q_start.shape[0] != B + 1:
        raise ValueError("q_start must have one entry more than there are sequences")
    if dst_slot is None:
        if cap is None:
            raise ValueError("dst_slot or cap must be given")
        with _allocating(stream):
            dst_slot = torch.empty(int(cap), dtype=torch.int64, device=n_new.device)
    _need(dst_slot, "dst_slot", torch.int64, 1)
    with _on_device_of(block_table, seq_lens, page_refs, n_new, q_start, dst_slot, err_word):
        st = lib().kv8_pages_append(*table, _ptr(n_new), _ptr(q_start), _ptr(dst_slot),
                                    dst_slot.shape[0], _ptr(err_word), _stream(stream))
    _check("kv8_pages_append", st)
    return q_start, dst_slot


def kv8_pages_fork(block_table, seq_lens, page_refs, src_seq, dst_seq, fork_len=None, moves=None,
                   n_moves=None, err_word=None, stream=None):
    """Sequences dst_seq become prefixes of src_seq (fork_len tokens, or all) that share their full
    pages.  Returns (moves int32 [>= n, 2], n_moves int32 [1]) for kv8_pages_copy."""
    table = _page_table(block_table, seq_lens, page_refs, err_word)
    _need(src_seq, "src_seq", torch.int32, 1)
    _need(dst_seq, "dst_seq", torch.int32, 1)
    n = src_seq.shape[0]
    if dst_seq.shape[0] != n:
        raise ValueError("dst_seq must have one entry per entry of src_seq")
    if fork_len is not None:
        _need(fork_len, "fork_len", torch.int32, 1)
        if fork_len.shape[0] != n:
            raise ValueError("fork_len must have one entry per entry of src_seq")
    moves, n_moves = _moves_out(moves, n_moves, n, block_table.device, stream)
    with _on_device_of(block_table, seq_lens, page_refs, src_seq, dst_seq, fork_len, moves, n_moves, err_word):
        st = lib().kv8_pages_fork(*table, _ptr(src_seq), _ptr(dst_seq), _ptr(fork_len), n, _ptr(moves),
                                  _ptr(n_moves), _ptr(err_word), _stream(stream))
    _check("kv8_pages_fork", st)
    return moves, n_moves


def kv8_pages_free(block_table, seq_lens, page_refs, seq, err_word=None, stream=None):
    """Empty the sequences seq: their pages lose a count, their entries become -1."""
    table = _page_table(block_table, seq_lens, page_refs, err_word)
    _need(seq, "seq", torch.int32, 1)
    with _on_device_of(block_table, seq_lens, page_refs, seq, err_word):
        st = lib().kv8_pages_free(*table, _ptr(seq), seq.shape[0], _ptr(err_word), _stream(stream))
    _check("kv8_pages_free", st)


def kv8_pages_compact(block_table, seq_lens, page_refs, moves=None, n_moves=None, n_live=None,
                      err_word=None, stream=None):
    """Pack the pages in use into the front of the pool.  Returns (moves int32 [>= n_blocks // 2, 2],
    n_moves int32 [1]) for kv8_pages_copy; n_live (int32 [1], optional) takes the pages in use."""
    table = _page_table(block_table, seq_lens, page_refs, err_word)
    moves, n_moves = _moves_out(moves, n_moves, page_refs.shape[0] // 2, block_table.device, stream)
    if n_live is not None:
        _need(n_live, "n_live", torch.int32, 1)
        if n_live.numel() < 1:
            raise ValueError("n_live must have one entry")
    with _on_device_of(block_table, seq_lens, page_refs, moves, n_moves, n_live, err_word):
        st = lib().kv8_pages_compact(*table, _ptr(moves), _ptr(n_moves), _ptr(n_live), _ptr(err_word),
                                     _stream(stream))
    _check("kv8_pages_compact", st)
    return moves, n_moves


def kv8_pages_copy(kv_codes, kv_scales, moves, n_moves=None, err_word=None, stream=None):
    """Copy page moves[i, 0] over page moves[i, 1] in a cache (kv_codes uint8 [slots, 576],
    kv_scales f32 [slots, 2]) or in every layer of a stack of them ([layers, slots, ...])."""
    if isinstance(kv_codes, torch.Tensor) and kv_codes.dim() == 3:
        _need(kv_codes, "kv_codes", torch.uint8, 3)
        _need(kv_scales, "kv_scales", torch.float32, 3)
        if kv_codes.shape[2] != KV8_D or tuple(kv_scales.shape) != (*kv_codes.shape[:2], 2):
            raise ValueError("kv_codes must be [layers,slots,576] and kv_scales [layers,slots,2]")
        if kv_codes.shape[0] == 0:
            raise ValueError("kv_codes must have at least one layer")
        layers, slots = kv_codes.shape[:2]
    else:
        _need_cache(kv_codes, kv_scales)
        layers, slots = 1, kv_codes.shape[0]
    _need(moves, "moves", torch.int32, 2)
    if moves.shape[1] != 2:
        raise ValueError("moves must be [n, 2]")
    if n_moves is not None:
        _need(n_moves, "n_moves", torch.int32, 1)
        if n_moves.numel() < 1:
            raise ValueError("n_moves must have one entry")
    _need_err(err_word)
    with _on_device_of(kv_codes, kv_scales, moves, n_moves, err_word):
        st = lib().kv8_pages_copy(_ptr(kv_codes), _ptr(kv_scales), layers, slots, _ptr(moves),
                                  _ptr(n_moves), moves.shape[0], _ptr(err_word), _stream(stream))
    _check("kv8_pages_copy", st)


# ----------------------------------------------------------------- cache file
class Kv8Disk:
    """An open cache file (the kv8_disk_* calls): save rows of a device cache to it,
    load them back.  Use as a context manager or call close()."""

    def __init__(self, path: str, staging_rows: int = 4096):
        h = ctypes.c_void_p()
        _check("kv8_disk_open", lib().kv8_disk_open(os.fsencode(path), int(staging_rows),
                                                    ctypes.byref(h)))
        self._h = h

    def info(self):
        """(committed rows, version)."""
        n, v = ctypes.c_int64(), ctypes.c_int()
        _check("kv8_disk_info", lib().kv8_disk_info(self._h, ctypes.byref(n), ctypes.byref(v)))
        return n.value, v.value

    def append(self, kv_codes, kv_scales, slots=None, n=None, stream=None):
        """Append the cache rows at device slots (int64 [n]) or slots 0..n-1."""
        _need(kv_codes, "kv_codes", torch.uint8, 2)
        _need(kv_scales, "kv_scales", torch.float32, 2)
        if slots is not None:
            _need(slots, "slots", torch.int64, 1)
            n = slots.numel()
        elif n is None:
            n = kv_codes.shape[0]
        _check("kv8_disk_append", lib().kv8_disk_append(self._h, _ptr(kv_codes), _ptr(kv_scales),
                                                        kv_codes.shape[0], _ptr(slots), int(n),
                                                        _stream(stream)))

    def load(self, kv_codes, kv_scales, first_row=0, n=None, dst_slot=None, stream=None):
        """Load committed rows [first_row, first_row + n) into the cache at device
        dst_slot (int64 [n]) or slots first_row + i."""
        _need(kv_codes, "kv_codes", torch.uint8, 2)
        _need(kv_scales, "kv_scales", torch.float32, 2)
        if dst_slot is not None:
            _need(dst_slot, "dst_slot", torch.int64, 1)
            n = dst_slot.numel()
        elif n is None:
            n = self.info()[0] - first_row
        _check("kv8_disk_load", lib().kv8_disk_load(self._h, int(first_row), int(n), _ptr(kv_codes),
                                                    _ptr(kv_scales), kv_codes.shape[0],
                                                    _ptr(dst_slot), _stream(stream)))

    def close(self):
        if self._h is not None and self._h.value is not None:
            _check("kv8_disk_close", lib().kv8_disk_close(self._h))
        self._h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
