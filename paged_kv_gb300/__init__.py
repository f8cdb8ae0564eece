"""GB300-native decode-step tail: batched per-request sampling with fused
token write-back, paged-KV page allocation / page-table fill, the 8-bit paged
KV cache with its attention, and logit penalties, biases and masks.

The work runs in the CUDA library ``libpkv.so`` (C ABI in ``include/pkv.h``);
``paged_kv_gb300.pkv`` is its thin Python binding and
``paged_kv_gb300.workloads`` draws seeded synthetic inputs.
``paged_kv_gb300.serve`` is an example: a small decoder served through them all.
"""

__all__ = ["pkv", "serve", "workloads"]
