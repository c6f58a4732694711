"""GB300-native batched speculative-sampling verify step.

The hot path is one CUDA library (``_build/libspecverify.so``, sources in ``csrc/``, C ABI in
``include/spec_verify.h``); ``api`` is its thin torch binding and ``workloads`` makes the seeded
synthetic inputs. ``kvcache`` binds the paged key/value cache around the verify step
(``include/spec_kv.h``).
"""
from .api import (device_error, draft_sample, hbm_read_probe, lmhead_stats, residual_topf,
                  spec_verify, to_device_logits, verify, verify_hidden, verify_host)
from .kvcache import (block_tables, kv4_append, kv4_attention, kv4_cache, kv4_page_bytes,
                      kv8_append, kv8_attention, kv8_cache, kv8_page_bytes, prompt_attention,
                      qk_norm_rope)

__all__ = ["spec_verify", "verify", "verify_host", "draft_sample", "residual_topf",
           "lmhead_stats", "verify_hidden", "device_error", "hbm_read_probe",
           "to_device_logits", "block_tables", "qk_norm_rope", "kv4_append", "kv4_attention",
           "kv4_cache", "kv4_page_bytes", "kv8_append", "kv8_attention", "kv8_cache",
           "kv8_page_bytes", "prompt_attention"]
