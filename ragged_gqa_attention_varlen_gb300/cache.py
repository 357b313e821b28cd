"""Generation: rotary positions, the paged K/V cache, attention over it, key
weights and eviction (ctypes marshalling of the library's calls only).

A cache is two tensors of pages ``[num_pages, page_size, Hkv, d]`` (K and V;
``page_size`` a power of two from 16 to 1024), a table ``[B, width]`` (int32)
with the pages of each sequence, and its lengths ``lens`` ``[B]`` (int32), all
on the device.  One generation step:

    q, k = attention_varlen_rotary(q, k, positions, inv_freq)
    attention_varlen_cache_append(k, v, k_cache, v_cache, table, lens, cu_q, lens_out=new_lens)
    out, lse = attention_varlen_cache_fwd(q, k_cache, v_cache, table, new_lens, cu_q)
    attention_varlen_cache_weights(q, k_cache, table, new_lens, cu_q, lse, scores)
    attention_varlen_cache_evict(k_cache, v_cache, table, new_lens, scores, key_pos, next_pos, budget)

Every call is asynchronous on ``stream`` (default: the current stream of the
tensors' device).  Problems that only the device can see (lengths beyond the
table, page numbers outside of the pool, inconsistent cu arrays) set bits of
``status``, an int32 CUDA tensor the caller zeroes and reads when it likes;
the calls never read or write out of range because of them.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import binding
from .binding import ATTN_BF16, ATTN_F16, HEAD_DIMS, AttnError

DEV_BAD_CACHE = 0x40

EXPORTS = ("attn_varlen_rotary", "attn_varlen_cache_append", "attn_varlen_cache_fwd",
           "attn_varlen_cache_fwd_workspace_size", "attn_varlen_cache_weights",
           "attn_varlen_cache_weights_workspace_size", "attn_varlen_cache_evict",
           "attn_varlen_cache_evict_workspace_size")

_lib = None
_NOSTRIDE = (0, 0)


def load():
    """The library with the signatures of this module's calls."""
    global _lib
    if _lib is not None:
        return _lib
    lib = binding.load()
    P, I, L, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    x, pages, rows = [P, L, L], [P, L, L, L], [P, L, L]
    table = [P, L, I, P]
    rotary = [P, L, I, P, P, I, I]
    read = ([I, I] + table + table + [P, P, P] + rows + rows + [P, L, I, I, I, F, F])
    sig = {
        "attn_varlen_rotary": [I, L, I, I, I] + x + x + rotary + [I] + x + x + [P],
        "attn_varlen_cache_append": ([I, I, I, I, L] + x + x + pages + pages + [I, I] + table +
                                     [P] + rotary + rows + rows + [P, P, P]),
        "attn_varlen_cache_fwd": ([I, I, I, I, I, I, L] + x + pages + pages + read + x +
                                  [P, P, Z, P, P]),
        "attn_varlen_cache_weights": ([I, I, I, I, I, I, L] + x + pages + read + [P] + rows * 4 +
                                      [P, Z, P, P]),
        "attn_varlen_cache_evict": ([I, I, I] + pages + pages + [I, I] + table + rows + rows +
                                    [P, I, I] + rows + rows + [P, P, Z, P, P]),
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, I
    for name, n in (("fwd", [I, I, I, I, I, L]), ("weights", []),
                    ("evict", [I, I, I, I, I])):
        f = getattr(lib, f"attn_varlen_cache_{name}_workspace_size")
        f.argtypes, f.restype = n, Z
    _lib = lib
    return lib


def _raise(code):
    raise AttnError(code, load().attn_status_string(code).decode())


_HERE = contextlib.nullcontext()


def _on(t, stream):
    """(stream handle, context): within it t's device is current, and what the
    call allocates belongs to the stream it runs on."""
    if not t.is_cuda:
        raise ValueError("the tensors of a call must be CUDA tensors")
    dev = t.device
    if stream is not None:
        if stream.device != dev:
            raise ValueError("stream belongs to another device than the tensors")
        return stream.cuda_stream, torch.cuda.stream(stream)
    handle = torch.cuda.current_stream(dev).cuda_stream
    return handle, (_HERE if torch.cuda.current_device() == dev.index else torch.cuda.device(dev))


def _rows16(name, t, dtype, heads, d, tokens):
    """(pointer, token stride, head stride) of a packed 16-bit tensor."""
    if not t.is_cuda or t.dtype != dtype or t.dim() != 3:
        raise ValueError(f"{name} must be a {dtype} CUDA tensor [tokens, heads, d]")
    shape, stride = t.shape, t.stride()
    if shape[0] != tokens or shape[1] != heads or shape[2] != d or stride[2] != 1:
        raise ValueError(f"{name} must be [{tokens}, {heads}, {d}] with a contiguous feature axis")
    return t.data_ptr(), _stride(stride[0], tokens, heads * d), _stride(stride[1], heads, d)


def _stride(s, size, dense):
    """A stride that no index uses (an axis of one) may be anything."""
    return s if size > 1 else dense


def _pages(name, t, dtype):
    if not t.is_cuda or t.dtype != dtype or t.dim() != 4 or t.stride(3) != 1:
        raise ValueError(f"{name} must be a {dtype} CUDA tensor [num_pages, page_size, Hkv, d] "
                         "with a contiguous feature axis")
    n, ps, h, d = t.shape
    s = t.stride()
    return (t.data_ptr(), _stride(s[0], n, ps * h * d), _stride(s[1], ps, h * d), _stride(s[2], h, d))


def _i32(name, t, n):
    if not t.is_cuda or t.dtype != torch.int32 or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 CUDA vector of {n}")
    return t.data_ptr()


def _table(name, table, lens, rows):
    if (not table.is_cuda or table.dtype != torch.int32 or table.dim() != 2 or
            table.shape[0] != rows or table.shape[1] < 1 or
            (table.shape[1] > 1 and table.stride(1) != 1)):
        raise ValueError(f"{name} must be an int32 CUDA tensor [{rows}, width] with contiguous rows")
    return (table.data_ptr(), _stride(table.stride(0), rows, table.shape[1]), table.shape[1],
            _i32(f"{name}'s lengths", lens, rows))


def _slots(name, t, dtype, rows, heads, slots):
    """(pointer, row stride, head stride) of an array with a value per slot."""
    if t is None:
        return 0, 0, 0
    if not t.is_cuda or t.dtype != dtype or t.dim() != 3:
        raise ValueError(f"{name} must be a {dtype} CUDA tensor [rows, Hkv, slots]")
    if t.shape[0] != rows or t.shape[1] != heads or t.shape[2] < slots or t.stride(2) != 1:
        raise ValueError(f"{name} must be [{rows}, {heads}, at least {slots}], slots contiguous")
    return t.data_ptr(), t.stride(0), t.stride(1)


def _same_device(first, *others):
    for t in others:
        if t is not None and t.device != first.device:
            raise ValueError("every tensor of a call must be on the same device")


def _dtype(t):
    if t.dtype == torch.bfloat16:
        return ATTN_BF16
    if t.dtype == torch.float16:
        return ATTN_F16
    raise ValueError("q, k, v and the cache must be fp16 or bf16")


def _status(status):
    return 0 if status is None else _i32("status", status, status.numel())


def _workspace(workspace, need, device):
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    elif not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA buffer")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _rotary(positions, inv_freq, pair_axis, d, tokens):
    """The rotary arguments of a call, (positions pointer ... pairs)."""
    if positions.dim() == 1:
        positions = positions.unsqueeze(0)
    if (not positions.is_cuda or positions.dtype != torch.int32 or positions.dim() != 2 or
            positions.shape[0] < 1 or positions.shape[1] != tokens or
            (tokens > 1 and positions.stride(1) != 1)):
        raise ValueError(f"positions must be an int32 CUDA tensor [axes, {tokens}], rows contiguous")
    if inv_freq is None:
        return positions.data_ptr(), positions.stride(0), positions.shape[0], 0, 0, 0
    if (not inv_freq.is_cuda or inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or
            not inv_freq.is_contiguous()):
        raise ValueError("inv_freq must be a contiguous float64 CUDA vector")
    pairs = inv_freq.numel()
    if pairs < 1 or 2 * pairs > d:
        raise ValueError(f"{pairs} pairs do not fit {d} features")
    axis = 0 if pair_axis is None else _i32("pair_axis", pair_axis, pairs)
    return positions.data_ptr(), positions.stride(0), positions.shape[0], inv_freq.data_ptr(), axis, pairs


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
    lib = load()
    handle, guard = _on(q, stream)
    with guard:
        dt = _dtype(q)
        if q.dim() != 3 or q.shape[2] not in HEAD_DIMS:
            raise ValueError(f"q must be [tokens, heads, d] with d in {HEAD_DIMS}")
        T, Hq, d = q.shape
        Hkv = 0 if k is None else k.shape[1]
        _same_device(q, k, positions, inv_freq, pair_axis, q_out, k_out)
        q_out = torch.empty((T, Hq, d), dtype=q.dtype, device=q.device) if q_out is None else q_out
        if k is not None and k_out is None:
            k_out = torch.empty((T, Hkv, d), dtype=k.dtype, device=k.device)
        if T == 0:
            return q_out, k_out
        pos, axis_stride, axes, freq, axis, pairs = _rotary(positions, inv_freq, pair_axis, d, T)
        none = (0, 0, 0)
        code = lib.attn_varlen_rotary(
            dt, T, Hq, Hkv, d, *_rows16("q", q, q.dtype, Hq, d, T),
            *(none if k is None else _rows16("k", k, q.dtype, Hkv, d, T)),
            pos, axis_stride, axes, freq, axis, pairs, bool(interleaved), bool(inverse),
            *_rows16("q_out", q_out, q.dtype, Hq, d, T),
            *(none if k is None else _rows16("k_out", k_out, q.dtype, Hkv, d, T)), handle)
        if code:
            _raise(code)
        return q_out, k_out


def attention_varlen_cache_append(k, v, k_cache, v_cache, table, lens, cu_new, positions=None,
                                  inv_freq=None, pair_axis=None, interleaved=False, key_pos=None,
                                  scores=None, lens_out=None, status=None, stream=None):
    """Write packed new tokens k, v ``[T, Hkv, d]`` into the cache: token
    ``cu_new[b] + i`` becomes slot ``lens[b] + i`` of sequence b (its pages are
    in the table already).  With ``inv_freq`` the K rows are turned on the way
    (see attention_varlen_rotary).  ``key_pos`` ``[B, Hkv, slots]`` receives the
    tokens' ``positions[0]`` (or slot numbers), ``scores`` zeros, ``lens_out``
    the new lengths (not ``lens`` itself)."""
    lib = load()
    handle, guard = _on(k, stream)
    with guard:
        dt = _dtype(k)
        if k.dim() != 3 or k.shape[2] not in HEAD_DIMS:
            raise ValueError(f"k must be [tokens, heads, d] with d in {HEAD_DIMS}")
        T, Hkv, d = k.shape
        B = lens.numel()
        _same_device(k, v, k_cache, v_cache, table, lens, cu_new, positions, inv_freq, pair_axis,
                     key_pos, scores, lens_out, status)
        kc, vc = _pages("k_cache", k_cache, k.dtype), _pages("v_cache", v_cache, k.dtype)
        if k_cache.shape != v_cache.shape or k_cache.shape[2:] != (Hkv, d):
            raise ValueError(f"k_cache and v_cache must both be [num_pages, page_size, {Hkv}, {d}]")
        slots = table.shape[-1] * k_cache.shape[1]
        if inv_freq is not None and positions is None:
            raise ValueError("rotary positions are missing")
        rot = (0, 0, 0, 0, 0, 0) if positions is None else _rotary(positions, inv_freq, pair_axis, d, T)
        if lens_out is not None and lens_out.data_ptr() == lens.data_ptr() and B:
            raise ValueError("lens_out must not be lens")
        code = lib.attn_varlen_cache_append(
            dt, B, Hkv, d, T, *_rows16("k", k, k.dtype, Hkv, d, T), *_rows16("v", v, k.dtype, Hkv, d, T),
            *kc, *vc, k_cache.shape[0], k_cache.shape[1], *_table("table", table, lens, B),
            _i32("cu_new", cu_new, B + 1), *rot, bool(interleaved),
            *_slots("key_pos", key_pos, torch.int32, B, Hkv, slots),
            *_slots("scores", scores, torch.float32, B, Hkv, slots),
            0 if lens_out is None else _i32("lens_out", lens_out, B), _status(status), handle)
        if code:
            _raise(code)


def _read(q, k_cache, table, lens, cu_q, alibi_slopes, prefix_table, prefix_lens, cu_prefix, q_pos,
          key_pos, prefix_key_pos, causal, window_left, window_right, softcap, scale_multiplier):
    """The arguments that attention and the key weights share: (dtype code and
    sizes, arguments from num_pages on)."""
    if q.dim() != 3 or q.shape[2] not in HEAD_DIMS:
        raise ValueError(f"q must be [tokens, heads, d] with d in {HEAD_DIMS}")
    T, Hq, d = q.shape
    pages, page, Hkv, dc = k_cache.shape
    if Hkv < 1 or Hq % Hkv or dc != d:
        raise ValueError(f"q's {Hq} heads of {d} do not fit the cache's {Hkv} heads of {dc}")
    B = lens.numel()
    slots = table.shape[-1] * page
    _same_device(q, k_cache, table, lens, cu_q, alibi_slopes, prefix_table, prefix_lens, cu_prefix,
                 q_pos, key_pos, prefix_key_pos)
    P, pslots, prefix, cup = 0, 0, (0, 0, 0, 0), 0
    if prefix_table is not None:
        if prefix_lens is None or cu_prefix is None:
            raise ValueError("prefixes need prefix_table, prefix_lens and cu_prefix")
        P = prefix_lens.numel()
        if P:
            pslots = prefix_table.shape[-1] * page
            prefix = _table("prefix_table", prefix_table, prefix_lens, P)
            cup = _i32("cu_prefix", cu_prefix, P + 1)
    elif prefix_lens is not None or cu_prefix is not None or prefix_key_pos is not None:
        raise ValueError("prefixes need prefix_table, prefix_lens and cu_prefix")
    if (key_pos is not None or prefix_key_pos is not None) and q_pos is None:
        raise ValueError("key positions need q_pos")
    slope, slope_stride = 0, 0
    if alibi_slopes is not None:
        if (not alibi_slopes.is_cuda or alibi_slopes.dtype != torch.float32 or
                alibi_slopes.shape != (B, Hq) or (Hq > 1 and alibi_slopes.stride(1) != 1)):
            raise ValueError("alibi_slopes must be fp32 [B, Hq] on the device, head stride 1")
        slope, slope_stride = alibi_slopes.data_ptr(), alibi_slopes.stride(0)
    args = (pages, page, *_table("table", table, lens, B), *prefix, cup, _i32("cu_q", cu_q, B + 1),
            0 if q_pos is None else _i32("q_pos", q_pos, T),
            *_slots("key_pos", key_pos, torch.int32, B, Hkv, slots),
            *_slots("prefix_key_pos", prefix_key_pos if P else None, torch.int32, P, Hkv, pslots),
            slope, slope_stride, bool(causal), window_left, window_right, softcap, scale_multiplier)
    return (_dtype(q), B, P, Hq, Hkv, d, T), args, slots, pslots


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
    lib = load()
    handle, guard = _on(q, stream)
    with guard:
        head, args, _, _ = _read(q, k_cache, table, lens, cu_q, alibi_slopes, prefix_table,
                                         prefix_lens, cu_prefix, q_pos, key_pos, prefix_key_pos, causal,
                                         window_left, window_right, softcap, scale_multiplier)
        _, B, P, Hq, Hkv, d, T = head
        kc, vc = _pages("k_cache", k_cache, q.dtype), _pages("v_cache", v_cache, q.dtype)
        if v_cache.shape != k_cache.shape:
            raise ValueError("k_cache and v_cache must have the same shape")
        _same_device(q, v_cache, out, lse, status)
        if out is None:
            out = torch.empty((T, Hq, d), dtype=q.dtype, device=q.device)
        if lse is None:
            lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
        binding._check_lse(lse, T, Hq)
        ws, ws_bytes = _workspace(workspace, lib.attn_varlen_cache_fwd_workspace_size(*head[1:]), q.device)
        code = lib.attn_varlen_cache_fwd(
            *head, *_rows16("q", q, q.dtype, Hq, d, T), *kc, *vc, *args,
            *_rows16("out", out, q.dtype, Hq, d, T), lse.data_ptr(), ws, ws_bytes, _status(status),
            handle)
        if code:
            _raise(code)
        return out, lse


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
    lib = load()
    handle, guard = _on(q, stream)
    with guard:
        head, args, slots, pslots = _read(
            q, k_cache, table, lens, cu_q, alibi_slopes, prefix_table, prefix_lens, cu_prefix, q_pos,
            key_pos, prefix_key_pos, causal, window_left, window_right, softcap, scale_multiplier)
        _, B, P, Hq, Hkv, d, T = head
        if scores_out is None:
            scores_out = scores if scores is not None else torch.zeros(
                (B, Hkv, slots), dtype=torch.float32, device=q.device)
        if prefix_scores_out is None:
            prefix_scores_out = prefix_scores
        if prefix_scores_out is not None and not P:
            raise ValueError("prefix_scores without prefixes")
        _same_device(q, lse, scores, scores_out, prefix_scores, prefix_scores_out, status)
        binding._check_lse(lse, T, Hq)
        f32 = torch.float32
        ws, ws_bytes = _workspace(
            workspace, lib.attn_varlen_cache_weights_workspace_size(),
            q.device)
        code = lib.attn_varlen_cache_weights(
            *head, *_rows16("q", q, q.dtype, Hq, d, T), *_pages("k_cache", k_cache, q.dtype), *args,
            lse.data_ptr(), *_slots("scores", scores, f32, B, Hkv, slots),
            *_slots("scores_out", scores_out, f32, B, Hkv, slots),
            *_slots("prefix_scores", prefix_scores, f32, P, Hkv, pslots),
            *_slots("prefix_scores_out", prefix_scores_out, f32, P, Hkv, pslots), ws, ws_bytes,
            _status(status), handle)
        if code:
            _raise(code)
        return scores_out, prefix_scores_out


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
    lib = load()
    handle, guard = _on(k_cache, stream)
    with guard:
        dt = k_cache.dtype
        _dtype(k_cache)
        kc, vc = _pages("k_cache", k_cache, dt), _pages("v_cache", v_cache, dt)
        if v_cache.shape != k_cache.shape or k_cache.shape[3] not in HEAD_DIMS:
            raise ValueError(f"k_cache and v_cache must have the same shape, with d in {HEAD_DIMS}")
        pages, page, Hkv, d = k_cache.shape
        B = lens.numel()
        scores_out = scores if scores_out is None else scores_out
        key_pos_out = key_pos if key_pos_out is None else key_pos_out
        lens_out = lens if lens_out is None else lens_out
        _same_device(k_cache, v_cache, table, lens, scores, key_pos, next_pos, scores_out, key_pos_out,
                     lens_out, status)
        tab = _table("table", table, lens, B)
        slots = table.shape[1] * page
        ws, ws_bytes = _workspace(
            workspace, lib.attn_varlen_cache_evict_workspace_size(B, Hkv, table.shape[1], page, budget),
            k_cache.device)
        code = lib.attn_varlen_cache_evict(
            B, Hkv, d, *kc, *vc, pages, page, *tab,
            *_slots("scores", scores, torch.float32, B, Hkv, slots),
            *_slots("key_pos", key_pos, torch.int32, B, Hkv, slots), _i32("next_pos", next_pos, B),
            budget, recent, *_slots("scores_out", scores_out, torch.float32, B, Hkv, slots),
            *_slots("key_pos_out", key_pos_out, torch.int32, B, Hkv, slots),
            _i32("lens_out", lens_out, B), ws, ws_bytes, _status(status), handle)
        if code:
            _raise(code)
        return lens_out, scores_out, key_pos_out
