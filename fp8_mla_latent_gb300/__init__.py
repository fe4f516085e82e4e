"""fp8 e4m3 latent-KV absorbed MLA decode for one GB300 (sm_103a).

The product is the C-ABI library ``libfp8mla.so`` (sources in ``csrc/``, calls
declared in ``include/fp8mla.h``); this package holds its in-tree build step
(``build``), a ctypes binding with the same call names (``_lib``) and the seeded
synthetic workloads (``workloads``).
"""
from ._lib import (KV8_BF16, KV8_BLOCK, KV8_D, KV8_DECODE_AUTO, KV8_DECODE_SIMT, KV8_DECODE_TCGEN05,
                   KV8_DECODE_TCGEN05_CTA, KV8_DECODE_TCGEN05_PAIR,
                   KV8_DL, KV8_DR, KV8_F16, KV8_F32, KV8_NORM_MAX_WIDTH, KV8_PAGES_EINDEX, KV8_PAGES_ENOROOM,
                   KV8_PAGES_ETIMEOUT, KV8_SHARE_ALWAYS, KV8_SHARE_AUTO, Kv8Disk, Kv8Error, alloc_workspace, kv8_norm_quantize_rows,
                   kv8_prefill_project, kv8_produce_rows, kv8_quantize_rows,
                   kv8_selftest_wait_timeout,
                   kv8_pages_append, kv8_pages_compact, kv8_pages_copy, kv8_pages_fork, kv8_pages_free,
                   kv8_workspace_error, lib, library_path, mla_absorb_chunk_fp8_batch,
                   mla_absorb_chunk_fp8_batch_workspace_size, mla_absorb_decode_fp8,
                   mla_absorb_decode_fp8_batch, mla_absorb_decode_fp8_batch_combine,
                   mla_absorb_decode_fp8_batch_noalloc, mla_absorb_decode_fp8_batch_partials,
                   mla_absorb_decode_fp8_batch_workspace_size,
                   mla_absorb_decode_fp8_workspace_size, mla_absorb_shared_fp8_batch,
                   mla_absorb_shared_fp8_batch_workspace_size, mla_absorb_window_fp8_batch,
                   mla_absorb_window_fp8_batch_workspace_size, mla_wuv_epilogue)

__all__ = [
    "KV8_BLOCK", "KV8_D", "KV8_DECODE_AUTO", "KV8_DECODE_SIMT", "KV8_DECODE_TCGEN05",
    "KV8_DECODE_TCGEN05_CTA", "KV8_DECODE_TCGEN05_PAIR", "KV8_DL",
    "KV8_DR", "Kv8Disk", "Kv8Error", "alloc_workspace", "kv8_prefill_project", "kv8_produce_rows", "kv8_quantize_rows",
    "kv8_selftest_wait_timeout", "kv8_workspace_error", "lib",
    "library_path", "mla_absorb_decode_fp8", "mla_absorb_decode_fp8_batch",
    "mla_absorb_decode_fp8_batch_combine", "mla_absorb_decode_fp8_batch_noalloc",
    "mla_absorb_decode_fp8_batch_partials",
    "mla_absorb_decode_fp8_batch_workspace_size", "mla_absorb_decode_fp8_workspace_size",
    "mla_wuv_epilogue", "mla_absorb_chunk_fp8_batch", "mla_absorb_chunk_fp8_batch_workspace_size",
    "kv8_pages_append", "kv8_pages_compact", "kv8_pages_copy", "kv8_pages_fork", "kv8_pages_free",
    "mla_absorb_window_fp8_batch", "mla_absorb_window_fp8_batch_workspace_size",
    "mla_absorb_shared_fp8_batch", "mla_absorb_shared_fp8_batch_workspace_size",
    "kv8_norm_quantize_rows", "KV8_BF16", "KV8_F16", "KV8_F32", "KV8_NORM_MAX_WIDTH",
    "KV8_SHARE_AUTO", "KV8_SHARE_ALWAYS",
    "KV8_PAGES_EINDEX", "KV8_PAGES_ENOROOM", "KV8_PAGES_ETIMEOUT",
]
