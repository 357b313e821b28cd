"""Cases of the operators that take attention from packed training batches to generation:
rotary positions with several axes, the paged K/V cache that new tokens are appended to,
attention over it with prefixes that sequences share, the attention weight that each cached
key has received, and eviction by it.

``own`` selects who computes: the plain torch form (fp32, rounded once at the end) or the
framework's entry points.  ``exact`` computes the same from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user's next token: the smallest attention call, where latency counts
        dict(name="attend_one_user", op="attend", B=1, lo=700, hi=700, prefixes=0, plen=0, Lq=1, Hq=96, Hkv=1, d=160,
             page=64, dtype="bf16", cap=3.0, alibi=True, causal=True, window=-1, evicted=False, std=2.0),
        # a serving batch of unrelated requests of very different lengths, small pages
        dict(name="attend_ragged_batch", op="attend", B=64, lo=64, hi=32000, prefixes=0, plen=0, Lq=1, Hq=80, Hkv=1, d=160,
             page=16, dtype="fp16", cap=3.0, alibi=True, causal=True, window=-1, evicted=False, std=2.0),
        # many users behind one long system prompt, grouped heads without a cap
        dict(name="attend_shared_prefix", op="attend", B=128, lo=32, hi=1024, prefixes=1, plen=8200, Lq=1, Hq=32, Hkv=8,
             d=128, page=64, dtype="bf16", cap=0.0, alibi=False, causal=True, window=-1, evicted=False, std=2.0),
        # several prompts, each sampled several times, checking up to eight drafted tokens at once
        dict(name="attend_drafts", op="attend", B=32, lo=100, hi=2000, prefixes=2, plen=12001, Lq=8, Hq=96, Hkv=1, d=160,
             page=128, dtype="bf16", cap=3.0, alibi=True, causal=True, window=-1, evicted=False, std=2.0),
        # the weights that one decode step adds to a batch's keys, in a cache that was evicted from before
        dict(name="weights_step", op="weights", B=64, lo=512, hi=16000, prefixes=0, plen=0, Lq=1, Hq=64, Hkv=1, d=160,
             page=32, dtype="bf16", cap=3.0, alibi=True, causal=True, window=-1, evicted=True, std=2.0),
        # the weights of whole prompts behind a shared prefix, before the first eviction
        dict(name="weights_prompt", op="weights", B=5, lo=200, hi=1500, prefixes=1, plen=1000, Lq=1500, Hq=32, Hkv=8, d=64,
             page=64, dtype="fp16", cap=0.0, alibi=False, causal=True, window=-1, evicted=False, std=2.0),
        # every step one key leaves each full cache
        dict(name="evict_step", op="evict", B=32, lo=1025, hi=1025, Hkv=1, d=160, page=64, dtype="bf16", budget=1024, recent=256),
        # long prompts cut down to a budget once, each K/V head keeping its own keys
        dict(name="evict_prompts", op="evict", B=12, lo=2000, hi=20000, Hkv=8, d=128, page=64, dtype="fp16", budget=4096,
             recent=512),
        # the new tokens of one decode step, rotated on the way into their pages
        dict(name="append_step", op="append", B=64, lo=1, hi=1, held=5000, Hkv=8, d=128, page=64, dtype="bf16",
             rot=128, axes=3, pairs_of="halves"),
        # packed prompts
        dict(name="append_prompts", op="append", B=9, lo=100, hi=12000, held=300, Hkv=1, d=160, page=128, dtype="fp16",
             rot=160, axes=1, pairs_of="neighbours"),
        # a training batch's q and k, forward
        dict(name="rotary_forward", op="rotary", T=16000, Hq=96, Hkv=1, d=160, dtype="bf16", rot=160, axes=3,
             pairs_of="halves", inverse=False, far=40000),
        # the gradients of q and k, with part of the features rotated, at odd lengths and far positions
        dict(name="rotary_backward", op="rotary", T=4999, Hq=32, Hkv=8, d=128, dtype="fp16", rot=96, axes=2,
             pairs_of="neighbours", inverse=True, far=1000000),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "weights", "evict", "append", "rotary"])
    heads = rng.choice([(96, 1, 160), (80, 1, 160), (64, 1, 160), (48, 1, 160), (32, 8, 128), (32, 8, 64), (12, 3, 128), (5, 5, 64)])
    Hq, Hkv, d = heads
    page, dtype = rng.choice([16, 32, 64, 128]), rng.choice(["fp16", "bf16"])
    if op in ("attend", "weights"):
        hi = _spread(rng, 20, 8000)
        prefixes = rng.choice([0, 1, 2])
        c = dict(op=op, B=_spread(rng, max(1, prefixes), 40), lo=_spread(rng, 1, hi), hi=hi, prefixes=prefixes,
                 plen=_spread(rng, 1, 6000) if prefixes else 0, Lq=rng.choice([1, 1, 1, 3, 8, 40]), Hq=Hq, Hkv=Hkv, d=d, page=page,
                 dtype=dtype, cap=rng.choice([0.0, 3.0, 30.0]), alibi=rng.random() < 0.5, causal=rng.random() < 0.8,
                 window=rng.choice([-1, -1, _spread(rng, 1, 4000)]), evicted=rng.random() < 0.3, std=2.0)
        while work(c)["flops"] > 1.5e10:  # below the largest listed cases
            c["B"], c["Lq"], c["hi"] = max(c["prefixes"], 1, c["B"] // 2), (c["Lq"] + 1) // 2, (c["hi"] + 1) // 2
            c["lo"] = min(c["lo"], c["hi"])
        return c
    if op == "evict":
        budget = _spread(rng, 16, 4096)
        hi = _spread(rng, budget + 1, 20000)
        return dict(op=op, B=_spread(rng, 1, 32 if Hkv == 1 else 12), lo=_spread(rng, max(1, budget // 2), hi), hi=hi, Hkv=Hkv, d=d, page=page,
                    dtype=dtype, budget=budget, recent=rng.randrange(0, budget + 1))
    rot = rng.choice([d, d, d // 2])
    axes, pairs_of = rng.choice([1, 2, 3]), rng.choice(["halves", "neighbours"])
    if op == "append":
        return dict(op=op, B=_spread(rng, 1, 64), lo=1, hi=_spread(rng, 1, 1000), held=_spread(rng, 1, 5000), Hkv=Hkv, d=d, page=page,
                    dtype=dtype, rot=rot, axes=axes, pairs_of=pairs_of)
    return dict(op=op, T=_spread(rng, 1, 16000), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, rot=rot, axes=axes, pairs_of=pairs_of,
                inverse=rng.random() < 0.5, far=_spread(rng, 1000, 1000000))


def _lengths(c):
    """The lengths of the case's sequences: spread over their logarithm, the longest one always there."""
    r = random.Random(7)
    n = [_spread(r, c["lo"], c["hi"]) for _ in range(c["B"])]
    n[len(n) // 2] = c["hi"]
    return n


def _plan(c):
    """(queries, own keys, prefix of each sequence or -1) of an attention case, as host lists."""
    r = random.Random(8)
    B, P = c["B"], c["prefixes"]
    keys = _lengths(c)
    if c["Lq"] > 100:  # prompts: every own key is also a query
        queries = [min(n, c["Lq"]) for n in keys]
    else:
        queries = [r.randint(1, c["Lq"]) for _ in keys]
        queries[0] = c["Lq"]
    group = [b * P // B if P else -1 for b in range(B)]
    return queries, keys, group


def work(c):
    e = 2  # bytes of an element
    if c["op"] in ("attend", "weights"):
        queries, keys, group = _plan(c)
        pairs = 0
        for q, n in zip(queries, keys):
            total = n + c["plen"]
            if c["evicted"]:
                pairs += q * total
                continue
            for i in range(q):
                k0 = i + total - q
                hi = min(total, k0 + 1) if c["causal"] else total
                lo = max(0, k0 - c["window"]) if c["window"] >= 0 else 0
                pairs += max(0, hi - lo)
        T, held = sum(queries), sum(keys) + c["prefixes"] * c["plen"]
        if c["op"] == "attend":
            nbytes = 2 * T * c["Hq"] * c["d"] * e + 4 * T * c["Hq"] + 2 * held * c["Hkv"] * c["d"] * e
            return {"bytes": nbytes, "flops": 4 * c["d"] * c["Hq"] * pairs}
        nbytes = T * c["Hq"] * c["d"] * e + 4 * T * c["Hq"] + held * c["Hkv"] * (c["d"] * e + 4)
        return {"bytes": nbytes, "flops": 2 * c["d"] * c["Hq"] * pairs}
    if c["op"] == "evict":
        nbytes = 0
        for n in _lengths(c):
            kept = min(n, c["budget"])
            moved = kept * (n - kept) / n  # of the kept keys, those that lie behind the new end
            nbytes += c["Hkv"] * (8 * n + 8 * kept + 2 * 2 * moved * c["d"] * e)
        return {"bytes": nbytes, "flops": 0}
    if c["op"] == "append":
        T = sum(_lengths(c))
        return {"bytes": T * c["Hkv"] * (4 * c["d"] * e + 4) + T * c["axes"] * 4, "flops": 3 * T * c["Hkv"] * c["rot"]}
    rows = c["T"] * (c["Hq"] + c["Hkv"])
    return {"bytes": 2 * rows * c["d"] * e + 4 * c["T"] * c["axes"], "flops": 3 * rows * c["rot"]}


# ------------------------------------------------------------------ inputs

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(lengths):
    return torch.cat([torch.zeros(1, dtype=torch.int32), torch.tensor(lengths).cumsum(0).int()]).cuda()


def _tables(seed, page, *groups):
    """A page table for each list of lengths, over one pool of pages in random order, and the pool's size."""
    width = [max(1, max((-(-n // page) for n in g), default=1)) for g in groups]
    need = sum(w * len(g) for w, g in zip(width, groups))
    pages = need + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))[:need].int().cuda()
    tables, at = [], 0
    for w, g in zip(width, groups):
        tables.append(order[at:at + w * len(g)].view(len(g), w))
        at += w * len(g)
    return tables, pages


def _rotary_parts(c):
    """inv_freq of each pair (base 10000) and the axis that turns it: consecutive runs of pairs, one an axis."""
    pairs = c["rot"] // 2
    inv_freq = [10000.0 ** (-i / pairs) for i in range(pairs)]
    axis = [min(c["axes"] - 1, i * c["axes"] // pairs) for i in range(pairs)]
    return inv_freq, axis


def _rotary(c):
    inv_freq, axis = _rotary_parts(c)
    return dict(inv_freq=torch.tensor(inv_freq, dtype=torch.float64, device="cuda"), pair_axis=_ints(axis),
                neighbours=c["pairs_of"] == "neighbours")


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dt)

    s = dict(c)
    if c["op"] in ("attend", "weights"):
        queries, keys, group = _plan(c)
        P = c["prefixes"]
        tables, pages = _tables(seed, c["page"], keys, [c["plen"]] * P)
        T = sum(queries)
        s.update(q=normal(T, c["Hq"], c["d"], std=c["std"]), table=tables[0], lens=_ints(keys), cu_q=_cu(queries),
                 k_cache=normal(pages, c["page"], c["Hkv"], c["d"]), v_cache=normal(pages, c["page"], c["Hkv"], c["d"]),
                 slopes=None, max_q=max(queries), max_k=max(keys), q_pos=None, key_pos=None)
        s["token_seq"] = torch.repeat_interleave(torch.arange(c["B"]), torch.tensor(queries)).cuda()
        s["group"] = torch.tensor(group, device="cuda")
        s["prefix_table"], s["prefix_lens"], s["cu_prefix"] = None, None, None
        if P:
            s.update(prefix_table=tables[1], prefix_lens=_ints([c["plen"]] * P), cu_prefix=_cu([group.count(p) for p in range(P)]))
        if c["alibi"]:
            h = torch.arange(1, c["Hq"] + 1, device="cuda", dtype=torch.float32)
            s["slopes"] = torch.exp2(-8 * h / c["Hq"]).expand(c["B"], -1).contiguous()
        if c["evicted"]:  # the cached keys are a subset of a history twice as long, in no order
            cap = tables[0].shape[1] * c["page"]
            at = torch.rand(c["B"], c["Hkv"], 2 * cap, generator=g, device="cuda")
            n = _ints(keys).view(-1, 1, 1)
            at[torch.arange(2 * cap, device="cuda").expand_as(at) >= 2 * n] = 2.0
            s["key_pos"] = (c["plen"] + at.argsort(-1)[..., :cap]).int()
            first = torch.tensor([c["plen"] + 2 * k - q for q, k in zip(queries, keys)], device="cuda")
            s["q_pos"] = (first[s["token_seq"]] + torch.arange(T, device="cuda") - s["cu_q"][s["token_seq"]]).int()
        if c["op"] == "weights":
            s["lse"] = _plain_attend(s)[1]  # what the attention call of the same step returned
            s["scores"] = torch.rand(c["B"], c["Hkv"], tables[0].shape[1] * c["page"], generator=g, device="cuda")
            s["scores_out"] = torch.zeros_like(s["scores"])
            s["prefix_scores"] = s["prefix_scores_out"] = None
            if P:
                s["prefix_scores"] = torch.rand(P, c["Hkv"], tables[1].shape[1] * c["page"], generator=g, device="cuda")
                s["prefix_scores_out"] = torch.zeros_like(s["prefix_scores"])
    elif c["op"] == "evict":
        keys = _lengths(c)
        (table,), pages = _tables(seed, c["page"], keys)
        cap = table.shape[1] * c["page"]
        n = torch.tensor(keys, device="cuda")
        at = torch.rand(c["B"], c["Hkv"], cap, generator=g, device="cuda")
        at[torch.arange(cap, device="cuda").expand_as(at) >= n.view(-1, 1, 1)] = 2.0
        s.update(k_cache=normal(pages, c["page"], c["Hkv"], c["d"]), v_cache=normal(pages, c["page"], c["Hkv"], c["d"]),
                 table=table, lens=n.int(), key_pos=at.argsort(-1).int(), next_pos=n.int(),
                 # accumulated weights: few keys carry most of it; equal ones occur
                 scores=(torch.rand(c["B"], c["Hkv"], cap, generator=g, device="cuda").pow(8) * 65536).round() / 1024)
        s.update(scores_out=torch.zeros_like(s["scores"]), key_pos_out=torch.zeros_like(s["key_pos"]), lens_out=torch.zeros_like(s["lens"]))
    elif c["op"] == "append":
        new = _lengths(c)
        r = random.Random(9)
        held = [r.randint(0, c["held"]) for _ in new]
        (table,), pages = _tables(seed, c["page"], [a + b for a, b in zip(new, held)])
        T, cap = sum(new), table.shape[1] * c["page"]
        lens, cu = _ints(held), _cu(new)
        seq = torch.repeat_interleave(torch.arange(c["B"]), torch.tensor(new)).cuda()
        slot = lens[seq] + torch.arange(T, device="cuda", dtype=torch.int32) - cu[seq]
        step = torch.randint(0, 7, (c["axes"], T), generator=g, device="cuda", dtype=torch.int32)
        step[0] = 0  # the first axis counts tokens; the others are a picture's rows and columns
        s.update(k=normal(T, c["Hkv"], c["d"]), v=normal(T, c["Hkv"], c["d"]), table=table, lens=lens, cu_new=cu,
                 positions=slot[None] + step, token_seq=seq, **_rotary(c),
                 k_cache=torch.zeros(pages, c["page"], c["Hkv"], c["d"], dtype=dt, device="cuda"),
                 v_cache=torch.zeros(pages, c["page"], c["Hkv"], c["d"], dtype=dt, device="cuda"),
                 key_pos=torch.zeros(c["B"], c["Hkv"], cap, dtype=torch.int32, device="cuda"),
                 scores=torch.ones(c["B"], c["Hkv"], cap, device="cuda"), lens_out=torch.zeros_like(lens))
    else:
        T = c["T"]
        s.update(q=normal(T, c["Hq"], c["d"]), k=normal(T, c["Hkv"], c["d"]), **_rotary(c),
                 positions=torch.randint(0, c["far"], (c["axes"], T), generator=g, device="cuda", dtype=torch.int32))
    return s


# ------------------------------------------------------------------ the plain form

def _slots(table, page, n):
    """The cache row of each of the first n slots of every table row."""
    j = torch.arange(n, device=table.device)
    return table[:, j // page].long() * page + j % page


def _context(s):
    """Keys of every sequence, prefix first, as rows of the cache [B, N], with their positions [B, Hkv, N] and which exist."""
    plen, page, Hkv = s["plen"], s["page"], s["Hkv"]
    n = min(s["max_k"], s["table"].shape[1] * page)
    rows = _slots(s["table"], page, n)
    there = torch.arange(n, device=rows.device) < s["lens"][:, None]
    pos = s["key_pos"][..., :n].long() if s["key_pos"] is not None else (plen + torch.arange(n, device=rows.device)).expand(len(rows), Hkv, -1)
    if plen:
        pre = _slots(s["prefix_table"], page, plen)[s["group"]]
        rows = torch.cat([pre, rows], 1)
        there = torch.cat([torch.ones_like(pre, dtype=torch.bool), there], 1)
        pos = torch.cat([torch.arange(plen, device=rows.device).expand(len(rows), Hkv, -1), pos], 2)
    return rows, pos, there


def _logits(s):
    """Masked logits [B, Hkv, Lq * group, N] of the padded queries, and how to get rows back."""
    B, Hq, Hkv, d, L = s["B"], s["Hq"], s["Hkv"], s["d"], s["max_q"]
    rows, pos, there = _context(s)
    counts = s["cu_q"][1:] - s["cu_q"][:-1]
    i = torch.arange(L, device=rows.device)
    token = (s["cu_q"][:-1, None] + i).clamp(max=len(s["q"]) - 1).long()
    q = s["q"][token].float().view(B, L, Hkv, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d)
    k = s["k_cache"].view(-1, Hkv, d)[rows].float().permute(0, 2, 3, 1)
    x = (q @ k) * (0.75 / math.sqrt(d))
    if s["cap"] > 0:
        x = s["cap"] * torch.tanh(x / s["cap"])
    x = x.view(B, Hkv, L, Hq // Hkv, -1)
    if s["q_pos"] is not None:
        qpos = s["q_pos"][token].long()
    else:
        qpos = i + (s["plen"] + s["lens"] - counts)[:, None].long()
    off = qpos[:, None, :, None] - pos[:, :, None, :]  # [B, Hkv, L, N]
    if s["slopes"] is not None:
        x = x - s["slopes"].view(B, Hkv, 1, -1, 1) * off[:, :, :, None].abs().float()
    ok = there[:, None, None, :] & (i < counts[:, None])[:, None, :, None]
    if s["causal"]:
        ok = ok & (off >= 0)
    if s["window"] >= 0:
        ok = ok & (off <= s["window"])
    x = x.masked_fill(~ok[:, :, :, None], -math.inf)
    return x.reshape(B, Hkv, -1, x.shape[-1]), rows, i


def _back(s, x):
    """[B, Hkv, Lq * group, ...] -> packed [T, Hq, ...]."""
    B, Hq, Hkv, L = s["B"], s["Hq"], s["Hkv"], s["max_q"]
    x = x.reshape(B, Hkv, L, Hq // Hkv, -1).transpose(1, 2).reshape(B * L, Hq, -1)
    at = torch.arange(len(s["q"]), device=x.device) - s["cu_q"][s["token_seq"]]
    return x[s["token_seq"] * L + at]


def _plain_attend(s):
    x, rows, _ = _logits(s)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    v = s["v_cache"].view(-1, s["Hkv"], s["d"])[rows].float().transpose(1, 2)
    out = (p @ v) / torch.where(total > 0, total, 1.0)
    return _back(s, out).to(s["q"].dtype), _back(s, top + torch.log(total))[..., 0]


def _plain_weights(s):
    x, rows, i = _logits(s)
    B, Hkv, L = s["B"], s["Hkv"], s["max_q"]
    token = (s["cu_q"][:-1, None] + i).clamp(max=len(s["q"]) - 1).long()
    lse = s["lse"][token].view(B, L, Hkv, -1).transpose(1, 2).reshape(B, Hkv, -1, 1)
    w = torch.exp(x - torch.where(lse > -math.inf, lse, 0.0)).sum(2)  # [B, Hkv, N]
    n = s["lens"][:, None, None]
    mine = w[..., s["plen"]:]
    keep = torch.arange(mine.shape[-1], device=w.device) < n
    out = s["scores_out"]
    out[..., :mine.shape[-1]] = torch.where(keep, s["scores"][..., :mine.shape[-1]] + mine, out[..., :mine.shape[-1]])
    if not s["plen"]:
        return out
    pre = s["prefix_scores_out"]
    pre[..., :s["plen"]] = s["prefix_scores"][..., :s["plen"]].index_add(0, s["group"], w[..., :s["plen"]])
    return out, pre


def _plain_evict(s):
    B, Hkv, cap = s["scores"].shape
    slot = torch.arange(cap, device="cuda")
    n = s["lens"].long()[:, None, None]
    kept_n = n.clamp(max=s["budget"])
    safe = s["key_pos"] >= (s["next_pos"] - s["recent"])[:, None, None]
    rank = torch.where(safe, math.inf, s["scores"]).masked_fill(slot >= n, -math.inf)
    order = rank.sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(rank, dtype=torch.bool).scatter_(-1, order, (slot < kept_n).expand_as(order))
    hole, mover = ~kept & (slot < kept_n), kept & (slot >= kept_n)
    # the i-th hole and the i-th mover of a head are at the same place of these two lists
    b, h, dst = hole.nonzero(as_tuple=True)
    src = mover.nonzero(as_tuple=True)[2]
    page = s["page"]
    for cache in (s["k_cache"], s["v_cache"]):
        cache[s["table"][b, dst // page].long(), dst % page, h] = cache[s["table"][b, src // page].long(), src % page, h]
    for x, out in ((s["scores"], s["scores_out"]), (s["key_pos"], s["key_pos_out"])):
        x = x.clone()
        x[b, h, dst] = x[b, h, src]
        out.copy_(torch.where(slot < kept_n, x, out))
    s["lens_out"].copy_(kept_n[:, 0, 0])
    return s["k_cache"], s["v_cache"], s["scores_out"], s["key_pos_out"], s["lens_out"]


def _plain_rotate(s, x, inverse):
    angle = s["positions"][s["pair_axis"].long()].double() * s["inv_freq"][:, None]  # [pairs, T]
    cos, sin = (f(angle).float().t()[:, None] for f in (torch.cos, torch.sin))
    sin = -sin if inverse else sin
    head, rest = x[..., :s["rot"]].float(), x[..., s["rot"]:]
    a, b = (head[..., 0::2], head[..., 1::2]) if s["neighbours"] else head.chunk(2, -1)
    a, b = a * cos - b * sin, b * cos + a * sin
    head = torch.stack([a, b], -1).flatten(-2) if s["neighbours"] else torch.cat([a, b], -1)
    return torch.cat([head.to(x.dtype), rest], -1)


def _plain_append(s):
    seq, page = s["token_seq"], s["page"]
    slot = (s["lens"][seq] + torch.arange(len(seq), device="cuda") - s["cu_new"][seq]).long()
    at = s["table"][seq, slot // page].long(), slot % page
    s["k_cache"][at] = _plain_rotate(s, s["k"], False)
    s["v_cache"][at] = s["v"]
    s["key_pos"][seq, :, slot] = s["positions"][0][:, None]
    s["scores"][seq, :, slot] = 0.0
    s["lens_out"].copy_(s["lens"] + s["cu_new"][1:] - s["cu_new"][:-1])
    return s["k_cache"], s["v_cache"], s["key_pos"], s["scores"], s["lens_out"]


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _own(s)
    if s["op"] == "attend":
        return _plain_attend(s)
    if s["op"] == "weights":
        return _plain_weights(s)
    if s["op"] == "evict":
        return _plain_evict(s)
    if s["op"] == "append":
        return _plain_append(s)
    return _plain_rotate(s, s["q"], s["inverse"]), _plain_rotate(s, s["k"], s["inverse"])


def _own(s):
    from ragged_gqa_attention_varlen_gb300 import cache
    if s["op"] == "attend":
        return cache.attention_varlen_cache_fwd(
            s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu_q"], s["slopes"], prefix_table=s["prefix_table"],
            prefix_lens=s["prefix_lens"], cu_prefix=s["cu_prefix"], q_pos=s["q_pos"], key_pos=s["key_pos"], causal=s["causal"],
            window_left=s["window"], softcap=s["cap"])
    if s["op"] == "weights":
        out = cache.attention_varlen_cache_weights(
            s["q"], s["k_cache"], s["table"], s["lens"], s["cu_q"], s["lse"], s["scores"], s["slopes"], scores_out=s["scores_out"],
            prefix_table=s["prefix_table"], prefix_lens=s["prefix_lens"], cu_prefix=s["cu_prefix"], prefix_scores=s["prefix_scores"],
            prefix_scores_out=s["prefix_scores_out"], q_pos=s["q_pos"], key_pos=s["key_pos"], causal=s["causal"],
            window_left=s["window"], softcap=s["cap"])
        return out if s["plen"] else out[0]
    if s["op"] == "evict":
        cache.attention_varlen_cache_evict(
            s["k_cache"], s["v_cache"], s["table"], s["lens"], s["scores"], s["key_pos"], s["next_pos"], s["budget"], s["recent"],
            scores_out=s["scores_out"], key_pos_out=s["key_pos_out"], lens_out=s["lens_out"])
        return s["k_cache"], s["v_cache"], s["scores_out"], s["key_pos_out"], s["lens_out"]
    if s["op"] == "append":
        cache.attention_varlen_cache_append(
            s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu_new"], positions=s["positions"],
            inv_freq=s["inv_freq"],
            pair_axis=s["pair_axis"], interleaved=s["neighbours"], key_pos=s["key_pos"], scores=s["scores"], lens_out=s["lens_out"])
        return s["k_cache"], s["v_cache"], s["key_pos"], s["scores"], s["lens_out"]
    return cache.attention_varlen_rotary(s["q"], s["k"], s["positions"], s["inv_freq"], s["pair_axis"], interleaved=s["neighbours"],
                                         inverse=s["inverse"])


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(c, seed):
    """Sequence by sequence and head by head from the definitions; None where only copies and whole numbers come back."""
    if c["op"] == "evict":
        return None
    s = prepare(c, seed)
    if c["op"] in ("append", "rotary"):
        inv_freq, axis = _rotary_parts(c)
        pos = s["positions"].double().cpu()
        turn = torch.polar(torch.ones(pos.shape[1], len(axis), dtype=torch.float64),
                           torch.stack([pos[a] * f for a, f in zip(axis, inv_freq)], 1)).cuda()
        if c["op"] == "rotary" and c["inverse"]:
            turn = turn.conj()

        def rotated(x):
            y = x.double()
            half, near = c["rot"] // 2, c["pairs_of"] == "neighbours"
            ia = torch.arange(half, device="cuda") * 2 if near else torch.arange(half, device="cuda")
            ib = ia + 1 if near else ia + half
            z = torch.complex(y[..., ia], y[..., ib]) * turn[:, None]
            y[..., ia], y[..., ib] = z.real, z.imag
            return y

        if c["op"] == "rotary":
            return rotated(s["q"]), rotated(s["k"])
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        k, cu, lens, table = rotated(s["k"]), s["cu_new"].tolist(), s["lens"].tolist(), s["table"].long()
        for b in range(c["B"]):
            j = torch.arange(cu[b + 1] - cu[b], device="cuda") + lens[b]
            kc[table[b, j // c["page"]], j % c["page"]] = k[cu[b]:cu[b + 1]]
            vc[table[b, j // c["page"]], j % c["page"]] = s["v"][cu[b]:cu[b + 1]].double()
        return kc, vc, None, None, None

    queries, keys, group = _plan(c)
    R, page, plen, cu = c["Hq"] // c["Hkv"], c["page"], c["plen"], s["cu_q"].tolist()
    out = torch.zeros(sum(queries), c["Hq"], c["d"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(queries), c["Hq"], dtype=torch.float64, device="cuda")
    if c["op"] == "weights":
        own_w, pre_w = s["scores_out"].double(), None if not plen else s["prefix_scores_out"].double()
        for b, n in enumerate(keys):
            own_w[b, :, :n] = s["scores"][b, :, :n].double()
        if plen:
            pre_w[..., :plen] = s["prefix_scores"][..., :plen].double()
    for b, (nq, n) in enumerate(zip(queries, keys)):
        def gather(cache):
            own_rows = cache[s["table"][b].long()].flatten(0, 1)[:n]
            if not plen:
                return own_rows.double()
            return torch.cat([cache[s["prefix_table"][group[b]].long()].flatten(0, 1)[:plen], own_rows]).double()
        keys_b, q = gather(s["k_cache"]), s["q"][cu[b]:cu[b + 1]].double()
        values_b = gather(s["v_cache"]) if c["op"] == "attend" else None
        for g in range(c["Hkv"]):
            x = torch.einsum("ihf,jf->hij", q[:, g * R:(g + 1) * R], keys_b[:, g]) * (0.75 / math.sqrt(c["d"]))
            if c["cap"] > 0:
                x = c["cap"] * torch.tanh(x / c["cap"])
            if c["evicted"]:
                qp = s["q_pos"][cu[b]:cu[b + 1]].double()
                kp = torch.cat([torch.arange(plen, device="cuda"), s["key_pos"][b, g, :n]]).double()
            else:
                qp = torch.arange(n + plen - nq, n + plen, device="cuda").double()
                kp = torch.arange(n + plen, device="cuda").double()
            gap = qp[:, None] - kp[None]
            if c["alibi"]:
                x -= s["slopes"][b, g * R:(g + 1) * R].double()[:, None, None] * gap.abs()
            if c["causal"]:
                x[:, gap < 0] = -math.inf
            if c["window"] >= 0:
                x[:, gap > c["window"]] = -math.inf
            if c["op"] == "attend":
                total = torch.logsumexp(x, -1)
                p = torch.exp(x - total[..., None]).nan_to_num(0.0)
                lse[cu[b]:cu[b + 1], g * R:(g + 1) * R] = total.t()
                out[cu[b]:cu[b + 1], g * R:(g + 1) * R] = torch.einsum("hij,jf->ihf", p, values_b[:, g])
            else:
                given = s["lse"][cu[b]:cu[b + 1], g * R:(g + 1) * R].double().t()
                w = torch.exp(x - given[..., None]).nan_to_num(0.0).sum((0, 1))
                own_w[b, g, :n] += w[plen:]
                if plen:
                    pre_w[group[b], g] += torch.nn.functional.pad(w[:plen], (0, pre_w.shape[-1] - plen))
    if c["op"] == "attend":
        return out, lse
    return own_w if not plen else (own_w, pre_w)
