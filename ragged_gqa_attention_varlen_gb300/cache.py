"""Generation: rotary positions, the paged K/V cache, attention over it, key
weights and eviction (argument marshalling only, by a native module).

A cache is two tensors of pages ``[num_pages, page_size, Hkv, d]`` (K and V;
``page_size`` a power of two from 16 to 1024), a table ``[B, width]`` (int32)
with the pages of each sequence, and its lengths ``lens`` ``[B]`` (int32), all
on the device.  One generation step, with the tokens' ``positions`` ``[T]``, the
keys' ``key_pos`` and accumulated ``scores`` ``[B, Hkv, slots]``, and ``next_pos``
``[B]``, the position that each sequence's next token will have:

    q, _ = attention_varlen_rotary(q, None, positions, inv_freq)
    attention_varlen_cache_append(k, v, k_cache, v_cache, table, lens, cu_q, positions=positions,
                                  inv_freq=inv_freq, key_pos=key_pos, scores=scores, lens_out=new_lens)
    out, lse = attention_varlen_cache_fwd(q, k_cache, v_cache, table, new_lens, cu_q,
                                          q_pos=positions, key_pos=key_pos, causal=True)
    attention_varlen_cache_weights(q, k_cache, table, new_lens, cu_q, lse, scores,
                                   q_pos=positions, key_pos=key_pos, causal=True)
    attention_varlen_cache_evict(k_cache, v_cache, table, new_lens, scores, key_pos, next_pos, budget)

An eviction leaves the slots in another order: from then on the positions say
which key is which, and the next step's ``lens`` are ``new_lens``, which the
eviction has shortened.

Every call is asynchronous on ``stream`` (default: the current stream of the
tensors' device).  Problems that only the device can see (lengths beyond the
table, page numbers outside of the pool, inconsistent cu arrays) set bits of
``status``, an int32 CUDA tensor the caller zeroes and reads when it likes;
the calls never read or write out of range because of them.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import AttnError

DEV_BAD_CACHE = 0x40

# in the order in which the native module takes their addresses
EXPORTS = ("attn_varlen_rotary", "attn_varlen_cache_append", "attn_varlen_cache_fwd",
           "attn_varlen_cache_fwd_workspace_size", "attn_varlen_cache_weights",
           "attn_varlen_cache_weights_workspace_size", "attn_varlen_cache_evict",
           "attn_varlen_cache_evict_workspace_size")

_native = None


def load():
    """The native entry points, bound to the library (once).  Raises if they
    have not been built."""
    global _native
    if _native is None:
        lib = binding.load()
        try:
            from . import _native as native
        except ImportError as e:
            raise RuntimeError("native entry points not built: _native.so is missing "
                               "(run __graft_entry__.build() or "
                               "ragged_gqa_attention_varlen_gb300/_build.py)") from e
        native.bind(AttnError, *(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                                 for name in EXPORTS + ("attn_status_string",)))
        _native = native
    return _native


def _run(name, stream, first, args):
    """The native call `name` on `stream` (default: the current stream of the
    device of the call's first tensor); what it allocates belongs to that stream."""
    call = getattr(_native or load(), name)
    if stream is None:
        return call(*args)
    if stream.device != first.device:
        raise ValueError("stream belongs to another device than the tensors")
    with torch.cuda.stream(stream):
        return call(*args)


def attention_varlen_rotary(q, k, positions, inv_freq, pair_axis=None, interleaved=False,
                            inverse=False, q_out=None, k_out=None, stream=None):
    """Turn packed q ``[T, Hq, d]`` and k ``[T, Hkv, d]`` (or None) by rotary
    positions with one or several axes; returns (q_out, k_out).

    ``positions`` is int32 ``[axes, T]`` (or ``[T]``), ``inv_freq`` float64
    ``[pairs]`` with 2 * pairs <= d (features beyond are copied) and
    ``pair_axis`` int32 ``[pairs]``: which axis turns a pair (None: the first).
    Pairs are features (i, i + pairs), or (2i, 2i + 1) with ``interleaved``.
    ``inverse`` turns back, which is the vector-Jacobian product: it takes the
    gradients of the turned q, k to those of the unturned ones.  ``q_out = q``
    and ``k_out = k`` turn in place."""
    return _run("rotary", stream, q, (q, k, positions, inv_freq, pair_axis, interleaved, inverse, q_out,
                                      k_out))


def attention_varlen_cache_append(k, v, k_cache, v_cache, table, lens, cu_new, positions=None,
                                  inv_freq=None, pair_axis=None, interleaved=False, key_pos=None,
                                  scores=None, lens_out=None, status=None, stream=None):
    """Write packed new tokens k, v ``[T, Hkv, d]`` into the cache: token
    ``cu_new[b] + i`` becomes slot ``lens[b] + i`` of sequence b (its pages are
    in the table already).  With ``inv_freq`` the K rows are turned on the way
    (see attention_varlen_rotary).  ``key_pos`` ``[B, Hkv, slots]`` receives the
    tokens' ``positions[0]`` (or slot numbers), ``scores`` zeros, ``lens_out``
    the new lengths (not ``lens`` itself).  A sequence whose tokens do not all fit
    its table takes none and keeps its length; with an inconsistent ``cu_new``
    nothing is appended."""
    _run("append", stream, k, (k, v, k_cache, v_cache, table, lens, cu_new, positions, inv_freq, pair_axis,
                               interleaved, key_pos, scores, lens_out, status))


def attention_varlen_cache_fwd(q, k_cache, v_cache, table, lens, cu_q, alibi_slopes=None,
                               prefix_table=None, prefix_lens=None, cu_prefix=None, q_pos=None,
                               key_pos=None, prefix_key_pos=None, causal=False, window_left=-1,
                               window_right=-1, softcap=3.0, scale_multiplier=0.75, out=None,
                               lse=None, workspace=None, status=None, stream=None):
    """Attention of packed queries q ``[T, Hq, d]`` over the cache; returns
    (out, lse) as attention_varlen_fwd does, with its options.

    Sequence b's tokens ``cu_q[b] .. cu_q[b+1]`` attend to its ``lens[b]``
    slots and before them, when ``cu_prefix[p] <= b < cu_prefix[p+1]``, to the
    ``prefix_lens[p]`` slots of the shared prefix p (pages in
    ``prefix_table[p]``), whose keys are read once for all its sequences.  With
    Lk slots in all, query i of Lq stands at position Lk - Lq + i and slot j at
    position j; ``q_pos`` ``[T]`` and ``key_pos`` ``[B, Hkv, slots]`` (after an
    eviction) say otherwise.  Tokens behind cu_q[B] are left as they are."""
    return _run("fwd", stream, q, (
        q, k_cache, table, lens, cu_q, alibi_slopes, prefix_table, prefix_lens, cu_prefix, q_pos, key_pos,
        prefix_key_pos, causal, window_left, window_right, softcap, scale_multiplier, v_cache, out, lse,
        workspace, status))


def attention_varlen_cache_weights(q, k_cache, table, lens, cu_q, lse, scores=None,
                                   alibi_slopes=None, scores_out=None, prefix_table=None,
                                   prefix_lens=None, cu_prefix=None, prefix_scores=None,
                                   prefix_scores_out=None, q_pos=None, key_pos=None,
                                   prefix_key_pos=None, causal=False, window_left=-1,
                                   window_right=-1, softcap=3.0, scale_multiplier=0.75,
                                   workspace=None, status=None, stream=None):
    """Add to ``scores`` ``[B, Hkv, slots]`` (fp32) the attention weight that
    each cached key receives from these queries, summed over their tokens and
    the heads of its K/V head; ``lse`` is what attention_varlen_cache_fwd
    returned for the same arguments.  Writes to ``scores_out`` (default:
    ``scores``, in place; with ``scores`` None the sums start at 0), for the
    slots below the lengths only.  Keys of shared prefixes are counted in
    ``prefix_scores`` ``[P, Hkv, slots]`` likewise, over all sequences of the
    prefix, if it or ``prefix_scores_out`` is given.  Returns (scores_out,
    prefix_scores_out)."""
    return _run("weights", stream, q, (
        q, k_cache, table, lens, cu_q, alibi_slopes, prefix_table, prefix_lens, cu_prefix, q_pos, key_pos,
        prefix_key_pos, causal, window_left, window_right, softcap, scale_multiplier, lse, scores,
        scores_out, prefix_scores, prefix_scores_out, workspace, status))


def attention_varlen_cache_evict(k_cache, v_cache, table, lens, scores, key_pos, next_pos, budget,
                                 recent=0, scores_out=None, key_pos_out=None, lens_out=None,
                                 workspace=None, status=None, stream=None):
    """Evict down to ``budget`` slots a sequence.  Each K/V head keeps the
    slots with ``key_pos >= next_pos[b] - recent`` (0 <= recent <= budget) and
    of the others those with the highest ``scores`` (equal ones: the lowest
    slot).  Kept rows behind the new end move, in the K and V pages, into the
    evicted slots before it; scores, positions and lengths follow into
    ``scores_out``, ``key_pos_out`` and ``lens_out`` (default: in place).
    Returns (lens_out, scores_out, key_pos_out).  The rows may as well be shared
    prefixes, with their own table."""
    return _run("evict", stream, k_cache, (
        k_cache, v_cache, table, lens, scores, key_pos, next_pos, budget, recent, scores_out, key_pos_out,
        lens_out, workspace, status))
