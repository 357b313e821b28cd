"""GB300 (sm_103a) ragged GQA attention with its full vector-Jacobian product.

The computation lives in ``libattn_varlen.so`` (hand-written CUDA: a device
tile scheduler, a tcgen05/TMA forward, the D = rowsum(dO * O) preprocess, and
an atomic-free backward with separate dk/dv and dq passes).  This package is
its thin binding; ``cache`` holds the calls that take a model from training to
generation (rotary positions, a paged K/V cache, attention over it, key weights,
eviction); ``workloads`` draws seeded synthetic inputs.
"""
from .cache import (attention_varlen_cache_append, attention_varlen_cache_evict,
                    attention_varlen_cache_fwd, attention_varlen_cache_weights,
                    attention_varlen_rotary)
from .binding import (AttnError, attention_varlen_feature_full_vjp, attention_varlen_fvjp,
                      device_status, launch_count, load, workspace_size)

__all__ = ["AttnError", "attention_varlen_cache_append", "attention_varlen_cache_evict",
           "attention_varlen_cache_fwd", "attention_varlen_cache_weights",
           "attention_varlen_feature_full_vjp", "attention_varlen_fvjp", "attention_varlen_rotary",
           "device_status", "launch_count", "load", "workspace_size"]
