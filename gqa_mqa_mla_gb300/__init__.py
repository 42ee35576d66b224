"""libdecattn: GB300-native attention over a paged KV cache, for decoding and for
the serving step around it.

MHA / GQA / MQA decode (``gqa_decode``, ``gqa_decode_fp8kv`` over an 8-bit e4m3 KV
cache, their sliding-window forms ``gqa_decode_window`` /
``gqa_decode_fp8kv_window``, and those with the first tokens kept,
``gqa_decode_sinks`` / ``gqa_decode_fp8kv_sinks``) and absorbed MLA
(``mla_decode``), the decode step's cache write (``gqa_kv_append``,
``gqa_kv_append_fp8kv``, ``mla_kv_append``) and MLA's absorption GEMMs
(``mla_absorb_q``, ``mla_unabsorb_out``).  For steps with any number of new tokens
per request: ``paged_plan`` (block tables, slots and positions from lengths),
``gqa_rope_append`` / ``gqa_rope_append_fp8kv`` (rotary positions and the cache
write by slot) and ``gqa_prefill`` / ``gqa_prefill_fp8kv`` (attention of chunks over
the cache).  Hand-written CUDA kernels for sm_103a behind a C ABI
(include/decattn.h); this package is the thin Python binding, ``synth`` draws
seeded synthetic inputs.
"""
from .binding import (  # noqa: F401
    DecAttnError,
    FLAG_BAD_BLOCK,
    FLAG_BAD_SEQ_LEN,
    FLAG_NO_ROOM,
    FLAG_TIMEOUT,
    PagedPlan,
    RopeTable,
    gqa_decode,
    gqa_decode_fp8kv,
    gqa_decode_fp8kv_sinks,
    gqa_decode_fp8kv_window,
    gqa_decode_sinks,
    gqa_decode_window,
    gqa_fp8_plan_splits,
    gqa_kv_append,
    gqa_kv_append_fp8kv,
    gqa_plan_splits,
    gqa_prefill,
    gqa_prefill_fp8kv,
    gqa_prefill_plan_splits,
    gqa_prefill_workspace_size,
    gqa_rope_append,
    gqa_rope_append_fp8kv,
    gqa_sinks_plan_splits,
    gqa_window_plan_splits,
    gqa_workspace_size,
    kv_bytes_per_token,
    lib,
    library_path,
    mla_bytes_per_token,
    mla_absorb_q,
    mla_decode,
    mla_kv_append,
    mla_plan_splits,
    mla_unabsorb_out,
    mla_workspace_size,
    paged_plan,
    rope_table,
    status_string,
)

__version__ = "0.1.0"
