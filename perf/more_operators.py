"""Cases of the operators that take the paged K/V cache further: attention over a cache held in 8 bits
with a scale for each block of tokens and head, the append that quantises, norms of queries and keys
with the rotation in the same pass (and their gradients), and forking and compacting the cache's pages.

``own`` selects who computes: the plain torch form (fp32, rounded once at the end) or the
framework's entry points.  ``exact`` computes the same from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn  # largest value 448
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user's next token over an 8-bit cache: the smallest attention call, where latency counts
        dict(name="attend8_one_user", op="attend8", B=1, lo=700, hi=700, prefixes=0, plen=0, Lq=1, Hq=96, Hkv=1, d=160,
             page=64, block=64, dtype="bf16", cap=3.0, alibi=True, causal=True, window=-1),
        # a serving batch of unrelated requests of very different lengths, small pages
        dict(name="attend8_ragged_batch", op="attend8", B=64, lo=64, hi=32000, prefixes=0, plen=0, Lq=1, Hq=80, Hkv=1, d=160,
             page=16, block=16, dtype="fp16", cap=3.0, alibi=True, causal=True, window=-1),
        # a large batch of grouped heads without a cap: few query rows a key, so the cache's bytes count
        dict(name="attend8_grouped_batch", op="attend8", B=96, lo=500, hi=8000, prefixes=0, plen=0, Lq=1, Hq=32, Hkv=8, d=128,
             page=64, block=32, dtype="bf16", cap=0.0, alibi=False, causal=True, window=-1),
        # several prompts, each sampled several times, checking up to eight drafted tokens at once
        dict(name="attend8_drafts", op="attend8", B=32, lo=100, hi=2000, prefixes=2, plen=12001, Lq=8, Hq=96, Hkv=1, d=160,
             page=128, block=128, dtype="bf16", cap=3.0, alibi=True, causal=True, window=-1),
        # the new tokens of one decode step, normed, rotated and quantised on the way into their pages
        dict(name="append8_step", op="append8", B=64, lo=1, hi=1, held=5000, Hkv=8, d=128, page=64, block=32, dtype="bf16",
             rot=128, axes=3, pairs_of="halves", norm=True),
        # packed prompts, rotated and quantised
        dict(name="append8_prompts", op="append8", B=9, lo=100, hi=12000, held=300, Hkv=1, d=160, page=128, block=16, dtype="fp16",
             rot=160, axes=1, pairs_of="neighbours", norm=False),
        # q and k of one decode step
        dict(name="norm_rotary_step", op="norm", T=64, Hq=80, Hkv=1, d=160, dtype="fp16", rot=160, axes=1, pairs_of="halves",
             backward=False, far=32000),
        # a training batch's q and k, forward
        dict(name="norm_rotary_forward", op="norm", T=16000, Hq=96, Hkv=1, d=160, dtype="bf16", rot=160, axes=3,
             pairs_of="halves", backward=False, far=40000),
        # the gradients of q, k and both weights, with part of the features rotated, at odd lengths and far positions
        dict(name="norm_rotary_backward", op="norm", T=9999, Hq=32, Hkv=8, d=128, dtype="bf16", rot=96, axes=2,
             pairs_of="neighbours", backward=True, far=1000000),
        # beam search over a few layers' cache: every step beams are continued, doubled or dropped
        dict(name="fork_beams", op="fork", R=32, hi=3000, layers=4, Hkv=1, d=160, page=64, dtype="bf16", room=1, kept=0.5),
        # prompts that are sampled many times at once, large pages
        dict(name="fork_samples", op="fork", R=256, hi=1500, layers=6, Hkv=8, d=128, page=128, dtype="fp16", room=200, kept=0.1),
        # a pool with holes after many requests have ended, packed so that its end can be given back
        dict(name="compact_pool", op="compact", R=96, hi=6000, layers=2, Hkv=8, d=128, page=128, dtype="bf16", holes=0.3),
    ]


HEADS = [(96, 1, 160), (80, 1, 160), (64, 1, 160), (48, 1, 160), (32, 8, 128), (32, 8, 64), (12, 3, 128), (5, 5, 64)]


def _spread(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["attend8", "attend8", "append8", "norm", "fork", "compact"])
    Hq, Hkv, d = rng.choice(HEADS)
    page, dtype = rng.choice([16, 32, 64, 128]), rng.choice(["fp16", "bf16"])
    block = rng.choice([b for b in (16, 32, 64, 128) if b <= page])
    if op == "attend8":
        hi = _spread(rng, 20, 8000)
        prefixes = rng.choice([0, 1, 2])
        c = dict(op=op, B=_spread(rng, max(1, prefixes), 90), lo=_spread(rng, 1, hi), hi=hi, prefixes=prefixes,
                 plen=_spread(rng, 1, 6000) if prefixes else 0, Lq=rng.choice([1, 1, 1, 3, 8, 40]), Hq=Hq, Hkv=Hkv, d=d, page=page,
                 block=block, dtype=dtype, cap=rng.choice([0.0, 3.0, 30.0]), alibi=rng.random() < 0.5, causal=rng.random() < 0.8,
                 window=rng.choice([-1, -1, _spread(rng, 1, 4000)]))
        while work(c)["flops"] > 1.5e10 or work(c)["bytes"] > 4e8:  # below the largest listed cases
            c["B"], c["Lq"], c["hi"] = max(c["prefixes"], 1, c["B"] // 2), (c["Lq"] + 1) // 2, (c["hi"] + 1) // 2
            c["lo"] = min(c["lo"], c["hi"])
        return c
    if op in ("fork", "compact"):
        hi = _spread(rng, 1, 3000)
        c = dict(op=op, R=_spread(rng, 1, 200), hi=hi, layers=rng.randint(1, 4), Hkv=Hkv, d=d, page=page, dtype=dtype)
        if op == "fork":
            return dict(c, room=rng.choice([0, 1, _spread(rng, 1, 300)]), kept=rng.choice([0.1, 0.5, 0.9]))
        return dict(c, holes=rng.choice([0.05, 0.3, 0.6]))
    rot = rng.choice([d, d, d // 2])
    axes, pairs_of = rng.choice([1, 2, 3]), rng.choice(["halves", "neighbours"])
    if op == "append8":
        return dict(op=op, B=_spread(rng, 1, 64), lo=1, hi=_spread(rng, 1, 1000), held=_spread(rng, 1, 5000), Hkv=Hkv, d=d, page=page,
                    block=block, dtype=dtype, rot=rot, axes=axes, pairs_of=pairs_of, norm=rng.random() < 0.5)
    return dict(op=op, T=_spread(rng, 1, 9000), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, rot=rot, axes=axes, pairs_of=pairs_of,
                backward=rng.random() < 0.5, far=_spread(rng, 1000, 1000000))


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
    queries = [r.randint(1, c["Lq"]) for _ in keys]
    queries[0] = c["Lq"]
    return queries, keys, [b * P // B if P else -1 for b in range(B)]


def _held(c):
    """The tokens that each sequence of an append holds already."""
    r = random.Random(9)
    return [r.randint(0, c["held"]) for _ in range(c["B"])]


def _fork_plan(c):
    """(lengths, parents) of a fork: the rows that go on, each continued about as often as the others."""
    r = random.Random(10)
    lens = [r.randint(1, c["hi"]) for _ in range(c["R"])]
    going = sorted(r.sample(range(c["R"]), max(1, round(c["R"] * c["kept"]))))
    return lens, [r.choice(going) if r.random() < 0.97 else -1 for _ in range(c["R"])]


def _compact_plan(c):
    """(pages of each row, whether it has ended) of a compaction."""
    r = random.Random(11)
    pages = [-(-r.randint(1, c["hi"]) // c["page"]) for _ in range(c["R"])]
    return pages, [r.random() < c["holes"] for _ in range(c["R"])]


def work(c):
    e = 2  # bytes of an element
    if c["op"] == "attend8":
        queries, keys, group = _plan(c)
        pairs = 0
        for q, n in zip(queries, keys):
            total = n + c["plen"]
            for i in range(q):
                k0 = i + total - q
                hi = min(total, k0 + 1) if c["causal"] else total
                lo = max(0, k0 - c["window"]) if c["window"] >= 0 else 0
                pairs += max(0, hi - lo)
        T, held = sum(queries), sum(keys) + c["prefixes"] * c["plen"]
        nbytes = 2 * T * c["Hq"] * c["d"] * e + 4 * T * c["Hq"] + 2 * held * c["Hkv"] * (c["d"] + 4 / c["block"])
        return {"bytes": nbytes, "flops": 4 * c["d"] * c["Hq"] * pairs}
    if c["op"] == "append8":
        T = sum(_lengths(c))
        blocks = sum((a + n - 1) // c["block"] - a // c["block"] + 1 for n, a in zip(_lengths(c), _held(c)))
        return {"bytes": T * c["Hkv"] * (2 * c["d"] * (e + 1) + 4) + 2 * blocks * c["Hkv"] * 8 + T * c["axes"] * 4,
                "flops": T * c["Hkv"] * (3 * c["rot"] + 6 * c["d"])}
    if c["op"] == "norm":
        rows = c["T"] * (c["Hq"] + c["Hkv"])
        times = 3 if c["backward"] else 2
        return {"bytes": times * rows * c["d"] * e + 4 * c["T"] * c["axes"] + 4 * (2 + 2 * c["backward"]) * c["d"],
                "flops": rows * (3 * c["rot"] + (12 if c["backward"] else 5) * c["d"])}
    row = c["Hkv"] * c["d"] * e * 2 * c["layers"]  # of a token in all pools
    if c["op"] == "fork":
        lens, parents = _fork_plan(c)
        seen, copied, held = set(), 0, 0
        for p in parents:
            if p < 0:
                continue
            if p in seen:
                copied += lens[p] % c["page"]
            seen.add(p)
            held += -(-(lens[p] + c["room"]) // c["page"])
        before = sum(-(-n // c["page"]) for n in lens)
        return {"bytes": 2 * copied * row + 4 * (before + held) + 4 * before * 2, "flops": 0}
    pages, ended = _compact_plan(c)
    pool, live = sum(pages), sum(n for n, x in zip(pages, ended) if not x)
    moved = live * (pool - live) / pool  # of the live pages, those that lie behind the new end
    return {"bytes": 2 * moved * c["page"] * row + 4 * (2 * pool + 2 * live), "flops": 0}


# ------------------------------------------------------------------ inputs

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(lengths):
    return torch.cat([torch.zeros(1, dtype=torch.int32), torch.tensor(lengths).cumsum(0).int()]).cuda()


def _tables(seed, page, *groups):
    """A page table for each list of lengths, over one pool of pages in random order, and the pool's size."""
    width = [max(1, max((-(-n // page) for n in g), default=1)) for g in groups]
    counts = [[-(-n // page) for n in g] for g in groups]
    pages = sum(map(sum, counts)) + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int()
    tables, at = [], 0
    for w, g in zip(width, counts):
        t = torch.zeros(len(g), w, dtype=torch.int32)
        for row, n in zip(t, g):
            row[:n] = order[at:at + n]
            at += n
        tables.append(t.cuda())
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


def _pow2_scale(top):
    """The smallest power of two s with top <= 448 s; 0 for 0."""
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(top > 0, ((e + 127) << 23).view(torch.float32), 0.0)


def _quantised(pool, block):
    """fp32 pages [pages, page, Hkv, d] -> (e4m3 values, scales [pages, page / block, Hkv])."""
    x = pool.view(pool.shape[0], -1, block, *pool.shape[2:])
    scale = _pow2_scale(x.abs().amax((2, 4)))
    inv = torch.where(scale > 0, 1 / scale, 0.0)
    return (x * inv[:, :, None, :, None]).view(pool.shape).to(F8), scale


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dt)

    def cached(pages):  # keys have features that are larger than others, tokens that are larger than others
        x = torch.randn(pages, c["page"], c["Hkv"], c["d"], generator=g, device="cuda")
        x.mul_(torch.rand(c["d"], generator=g, device="cuda").add_(0.5)).mul_(torch.rand(pages, c["page"], 1, 1, generator=g, device="cuda").add_(0.5))
        return _quantised(x, c["block"])

    s = dict(c)
    if c["op"] == "attend8":
        queries, keys, group = _plan(c)
        P = c["prefixes"]
        tables, pages = _tables(seed, c["page"], keys, [c["plen"]] * P)
        T = sum(queries)
        s.update(q=normal(T, c["Hq"], c["d"], std=2.0), table=tables[0], lens=_ints(keys), cu_q=_cu(queries), slopes=None,
                 max_q=max(queries), max_k=max(keys))
        s["k_cache"], s["k_scale"] = cached(pages)
        s["v_cache"], s["v_scale"] = cached(pages)
        s["token_seq"] = torch.repeat_interleave(torch.arange(c["B"]), torch.tensor(queries)).cuda()
        s["group"] = torch.tensor(group, device="cuda")
        s["prefix_table"], s["prefix_lens"], s["cu_prefix"] = None, None, None
        if P:
            s.update(prefix_table=tables[1], prefix_lens=_ints([c["plen"]] * P), cu_prefix=_cu([group.count(p) for p in range(P)]))
        if c["alibi"]:
            h = torch.arange(1, c["Hq"] + 1, device="cuda", dtype=torch.float32)
            s["slopes"] = torch.exp2(-8 * h / c["Hq"]).expand(c["B"], -1).contiguous()
    elif c["op"] == "append8":
        new, held = _lengths(c), _held(c)
        (table,), pages = _tables(seed, c["page"], [a + b for a, b in zip(new, held)])
        T = sum(new)
        lens, cu = _ints(held), _cu(new)
        seq = torch.repeat_interleave(torch.arange(c["B"]), torch.tensor(new)).cuda()
        slot = lens[seq] + torch.arange(T, device="cuda", dtype=torch.int32) - cu[seq]
        step = torch.randint(0, 7, (c["axes"], T), generator=g, device="cuda", dtype=torch.int32)
        step[0] = 0  # the first axis counts tokens; the others are a picture's rows and columns
        s.update(k=normal(T, c["Hkv"], c["d"], std=1.5), v=normal(T, c["Hkv"], c["d"], std=1.5), table=table, lens=lens, cu_new=cu,
                 positions=slot[None] + step, token_seq=seq, lens_out=torch.zeros_like(lens), k_weight=None,
                 key_pos=torch.zeros(c["B"], c["Hkv"], table.shape[1] * c["page"], dtype=torch.int32, device="cuda"), **_rotary(c))
        s["k_cache"], s["k_scale"] = cached(pages)
        s["v_cache"], s["v_scale"] = cached(pages)
        if c["norm"]:
            s["k_weight"] = torch.rand(c["d"], generator=g, device="cuda").add_(0.5)
    elif c["op"] == "norm":
        T = c["T"]
        s.update(q=normal(T, c["Hq"], c["d"], std=3.0), k=normal(T, c["Hkv"], c["d"], std=3.0), **_rotary(c),
                 q_weight=torch.rand(c["d"], generator=g, device="cuda").add_(0.5),
                 k_weight=torch.rand(c["d"], generator=g, device="cuda").add_(0.5),
                 positions=torch.randint(0, c["far"], (c["axes"], T), generator=g, device="cuda", dtype=torch.int32))
        if c["backward"]:
            s.update(dq=normal(T, c["Hq"], c["d"]), dk=normal(T, c["Hkv"], c["d"]))
    else:
        if c["op"] == "fork":
            lens, parents = _fork_plan(c)
            counts = [-(-n // c["page"]) for n in lens]
            width = max(counts) + -(-c["room"] // c["page"]) + 1
            pages = sum(counts) + c["R"] * (2 + -(-c["room"] // c["page"]))
            s.update(lens=_ints(lens), parents=_ints(parents), room=_ints([c["room"]] * c["R"]),
                     lens_out=_ints([0] * c["R"]), held_out=_ints([0] * c["R"]))
        else:
            counts, ended = _compact_plan(c)
            width, pages = max(counts), sum(counts)
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int()
        table, refs, at = torch.zeros(c["R"], width, dtype=torch.int32), torch.zeros(pages, dtype=torch.int32), 0
        for r, n in enumerate(counts):
            if c["op"] == "fork" or not ended[r]:
                table[r, :n] = order[at:at + n]
                refs[order[at:at + n].long()] = 1
            else:
                counts[r] = 0
            at += n
        s.update(table=table.cuda(), refs=refs.cuda(), held=_ints(counts), table_out=torch.zeros_like(table).cuda(),
                 refs_out=torch.zeros_like(refs).cuda(), live=_ints([0]),
                 pools=[normal(pages, c["page"], c["Hkv"], c["d"]) for _ in range(2 * c["layers"])])
    return s


# ------------------------------------------------------------------ the plain form

def _slots(table, page, n):
    """The cache row of each of the first n slots of every table row."""
    j = torch.arange(n, device=table.device)
    return table[:, j // page].long() * page + j % page


def _values(s, name, rows):
    """fp32 values of the cache rows [B, N] -> [B, N, Hkv, d]."""
    x = s[name + "_cache"].view(torch.uint8).view(-1, s["Hkv"], s["d"])[rows].view(F8).float()
    return x * s[name + "_scale"].view(-1, s["Hkv"])[rows // s["block"]][..., None]


def _plain_attend(s):
    B, Hq, Hkv, d, L, page, plen = s["B"], s["Hq"], s["Hkv"], s["d"], s["max_q"], s["page"], s["plen"]
    rows = _slots(s["table"], page, s["max_k"])
    there = torch.arange(s["max_k"], device=rows.device) < s["lens"][:, None]
    if plen:
        pre = _slots(s["prefix_table"], page, plen)[s["group"]]
        rows = torch.cat([pre, rows], 1)
        there = torch.cat([torch.ones_like(pre, dtype=torch.bool), there], 1)
    counts = s["cu_q"][1:] - s["cu_q"][:-1]
    i = torch.arange(L, device=rows.device)
    token = (s["cu_q"][:-1, None] + i).clamp(max=len(s["q"]) - 1).long()
    q = s["q"][token].float().view(B, L, Hkv, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d)
    x = (q @ _values(s, "k", rows).permute(0, 2, 3, 1)) * (0.75 / math.sqrt(d))
    if s["cap"] > 0:
        x = s["cap"] * torch.tanh(x / s["cap"])
    x = x.view(B, Hkv, L, Hq // Hkv, -1)
    qpos = i + (plen + s["lens"] - counts)[:, None].long()
    off = (qpos[:, :, None] - torch.arange(rows.shape[1], device=rows.device))[:, None]  # [B, 1, L, N]
    if s["slopes"] is not None:
        x = x - s["slopes"].view(B, Hkv, 1, -1, 1) * off[:, :, :, None].abs().float()
    ok = there[:, None, None, :] & (i < counts[:, None])[:, None, :, None]
    if s["causal"]:
        ok = ok & (off >= 0)
    if s["window"] >= 0:
        ok = ok & (off <= s["window"])
    x = x.masked_fill(~ok[:, :, :, None], -math.inf).view(B, Hkv, -1, rows.shape[1])
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    out = (p @ _values(s, "v", rows).transpose(1, 2)) / torch.where(total > 0, total, 1.0)
    at = s["token_seq"] * L + torch.arange(len(s["q"]), device=x.device) - s["cu_q"][s["token_seq"]]

    def back(y):  # [B, Hkv, Lq * group, ...] -> packed [T, Hq, ...]
        return y.reshape(B, Hkv, L, Hq // Hkv, -1).transpose(1, 2).reshape(B * L, Hq, -1)[at]
    return back(out).to(s["q"].dtype), back(top + torch.log(total))[..., 0]


def _plain_turn(s, x, inverse=False):
    """fp32 rows [T, H, d] turned."""
    angle = s["positions"][s["pair_axis"].long()].double() * s["inv_freq"][:, None]  # [pairs, T]
    cos, sin = (f(angle).float().t()[:, None] for f in (torch.cos, torch.sin))
    sin = -sin if inverse else sin
    head, rest = x[..., :s["rot"]], x[..., s["rot"]:]
    a, b = (head[..., 0::2], head[..., 1::2]) if s["neighbours"] else head.chunk(2, -1)
    a, b = a * cos - b * sin, b * cos + a * sin
    head = torch.stack([a, b], -1).flatten(-2) if s["neighbours"] else torch.cat([a, b], -1)
    return torch.cat([head, rest], -1)


def _plain_norm(x, weight):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight


def _plain_norm_bwd(s, dy, x, weight):
    g, x32 = _plain_turn(s, dy.float(), inverse=True), x.float()
    r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS)
    xhat, h = x32 * r, g * weight
    dx = r * (h - xhat * (h * xhat).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * xhat).sum((0, 1), dtype=torch.float64).float()


def _plain_append(s):
    seq, page, block = s["token_seq"], s["page"], s["block"]
    slot = (s["lens"][seq] + torch.arange(len(seq), device="cuda") - s["cu_new"][seq]).long()
    row = s["table"][seq, slot // page].long() * page + slot % page
    k = s["k"].float() if s["k_weight"] is None else _plain_norm(s["k"], s["k_weight"])
    held = (s["lens"][seq] - slot // block * block).clamp(min=0)  # slots of the token's block that hold one already
    lead = s["cu_new"][:-1].long()  # the only tokens whose block may hold some: the first of each sequence
    for name, x in (("k", _plain_turn(s, k)), ("v", s["v"].float())):
        cache, scale = s[name + "_cache"].view(torch.uint8).view(-1, block, s["Hkv"], s["d"]), s[name + "_scale"].view(-1, s["Hkv"])
        blocks = row // block
        top = torch.zeros_like(scale).index_reduce_(0, blocks, x.abs().amax(-1), "amax")[blocks]
        was = torch.where(held[:, None] > 0, scale[blocks], 0.0)
        now = torch.where(top <= 448 * was, was, _pow2_scale(top))
        # the held values of blocks whose scale grew, once more under the new one
        again = cache[blocks[lead]].view(F8).float() * torch.where(now > 0, was / now, 0.0)[lead, None, :, None]
        there = (torch.arange(block, device="cuda") < held[lead, None])[..., None, None]
        cache[blocks[lead]] = torch.where(there, again.to(F8).view(torch.uint8), cache[blocks[lead]])
        inv = torch.where(now > 0, 1 / now, 0.0)
        cache.view(-1, s["Hkv"], s["d"])[row] = (x * inv[..., None]).to(F8).view(torch.uint8)
        scale[blocks] = now
    s["key_pos"][seq, :, slot] = s["positions"][0][:, None]
    s["lens_out"].copy_(s["lens"] + s["cu_new"][1:] - s["cu_new"][:-1])
    return _appended(s)


def _appended(s):
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["key_pos"], s["lens_out"]


def _plain_fork(s):
    page, R, W = s["page"], *s["table"].shape
    table, held, parents, row = s["table"].long(), s["held"].long(), s["parents"].long(), torch.arange(s["R"], device="cuda")
    goes, p = parents >= 0, parents.clamp(min=0)
    length = torch.where(goes, s["lens"][p].long(), 0)
    full = length // page
    lowest = torch.full_like(row, R).scatter_reduce_(0, p, torch.where(goes, row, R), "amin")
    first = goes & (lowest[p] == row)
    had = torch.where(first, held[p], full)
    want = torch.where(goes, torch.maximum(had, (length + s["room"] + page - 1) // page), 0)
    # every old row's pages: the full ones go to all that continue it, the others to the first of them
    times, col = torch.zeros_like(row).index_add_(0, p, goes.long()), torch.arange(W, device="cuda")
    change = torch.where(col < (s["lens"] // page)[:, None], times[:, None] - 1, torch.where(times > 0, 0, -1)[:, None])
    change = torch.where(col < held[:, None], change, 0).int()
    refs = s["refs"].index_add(0, table.flatten(), change.flatten())
    free = (refs == 0).nonzero()[:, 0]
    new = torch.where(goes, want - had, 0)
    at = (new.cumsum(0) - new - had)[:, None] + col
    fresh = (col >= had[:, None]) & (col < want[:, None])
    out = torch.where(fresh, free[at.clamp(0, len(free) - 1)], table[p])
    s["table_out"].copy_(torch.where(col < want[:, None], out.int(), s["table_out"]))
    s["refs_out"].copy_(refs.index_fill(0, out[fresh], 1))
    s["lens_out"].copy_(length)
    s["held_out"].copy_(want)
    copies = (goes & ~first & (length % page > 0)).nonzero()[:, 0]
    src, dst = table[p[copies], full[copies]], out[copies, full[copies]]
    used = (torch.arange(page, device="cuda") < (length % page)[copies, None])[..., None, None]
    for pool in s["pools"]:
        pool[dst] = torch.where(used, pool[src], pool[dst])
    return s["table_out"], s["lens_out"], s["held_out"], s["refs_out"], s["pools"]


def _plain_compact(s):
    live = s["refs"] > 0
    n = live.sum()
    index = torch.arange(len(live), device="cuda")
    holes, movers = (~live & (index < n)).nonzero()[:, 0], (live & (index >= n)).nonzero()[:, 0]
    to = index.index_copy(0, movers, holes)
    col = torch.arange(s["table"].shape[1], device="cuda")
    s["table_out"].copy_(torch.where(col < s["held"][:, None], to[s["table"].long()].int(), s["table_out"]))
    s["refs_out"].copy_(s["refs"].index_copy(0, holes, s["refs"][movers]).index_fill(0, movers, 0))
    s["live"].copy_(n)
    for pool in s["pools"]:
        pool[holes] = pool[movers]
    return s["table_out"], s["refs_out"], s["live"], s["pools"]


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _own(s)
    if s["op"] == "attend8":
        return _plain_attend(s)
    if s["op"] == "append8":
        return _plain_append(s)
    if s["op"] == "fork":
        return _plain_fork(s)
    if s["op"] == "compact":
        return _plain_compact(s)
    if s["backward"]:
        (dq, dqw), (dk, dkw) = _plain_norm_bwd(s, s["dq"], s["q"], s["q_weight"]), _plain_norm_bwd(s, s["dk"], s["k"], s["k_weight"])
        return dq, dk, dqw, dkw
    return tuple(_plain_turn(s, _plain_norm(s[x], s[x + "_weight"])).to(s[x].dtype) for x in "qk")


def _own(s):
    from ragged_gqa_attention_varlen_gb300 import cache
    if s["op"] == "attend8":
        return cache.attention_varlen_cache8_fwd(
            s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lens"], s["cu_q"], s["slopes"],
            prefix_table=s["prefix_table"], prefix_lens=s["prefix_lens"], cu_prefix=s["cu_prefix"], causal=s["causal"],
            window_left=s["window"], softcap=s["cap"])
    if s["op"] == "append8":
        cache.attention_varlen_cache8_append(
            s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lens"], s["cu_new"],
            positions=s["positions"], inv_freq=s["inv_freq"], pair_axis=s["pair_axis"], interleaved=s["neighbours"],
            k_weight=s["k_weight"], eps=EPS, key_pos=s["key_pos"], lens_out=s["lens_out"])
        return _appended(s)
    if s["op"] == "fork":
        cache.attention_varlen_cache_fork(s["pools"], s["table"], s["lens"], s["held"], s["refs"], s["parents"], s["room"],
                                          table_out=s["table_out"], lens_out=s["lens_out"], held_out=s["held_out"],
                                          refs_out=s["refs_out"])
        return s["table_out"], s["lens_out"], s["held_out"], s["refs_out"], s["pools"]
    if s["op"] == "compact":
        cache.attention_varlen_cache_compact(s["pools"], s["table"], s["held"], s["refs"], table_out=s["table_out"],
                                             refs_out=s["refs_out"], live=s["live"])
        return s["table_out"], s["refs_out"], s["live"], s["pools"]
    turn = dict(positions=s["positions"], inv_freq=s["inv_freq"], pair_axis=s["pair_axis"], interleaved=s["neighbours"], eps=EPS)
    if s["backward"]:
        return cache.attention_varlen_norm_rotary_bwd(s["dq"], s["dk"], s["q"], s["k"], s["q_weight"], s["k_weight"], **turn)
    return cache.attention_varlen_norm_rotary(s["q"], s["k"], s["q_weight"], s["k_weight"], **turn)


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_turns(c, s):
    """e^(i angle) [T, 1, pairs] of every token and pair, and the features of the pairs."""
    inv_freq, axis = _rotary_parts(c)
    pos = s["positions"].double().cpu()
    turn = torch.polar(torch.ones(pos.shape[1], len(axis), dtype=torch.float64),
                       torch.stack([pos[a] * f for a, f in zip(axis, inv_freq)], 1)).cuda()
    half = torch.arange(c["rot"] // 2, device="cuda")
    return turn[:, None], (2 * half, 2 * half + 1) if c["pairs_of"] == "neighbours" else (half, half + c["rot"] // 2)


def _exact_turned(x, turn, pairs):
    x = x.clone()
    z = torch.complex(x[..., pairs[0]], x[..., pairs[1]]) * turn
    x[..., pairs[0]], x[..., pairs[1]] = z.real, z.imag
    return x


def _exact_e4m3(x):
    """The nearest value of four bits' exponent and three bits' fraction, ties to even, 448 at most."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(c, seed):
    """Sequence by sequence and head by head from the definitions; None where only copies and whole numbers come back."""
    if c["op"] in ("fork", "compact"):
        return None
    s = prepare(c, seed)
    if c["op"] == "norm":
        turn, pairs = _exact_turns(c, s)
        outs, grads = [], []
        for name in "qk":
            x, w = s[name].double(), s[name + "_weight"].double()
            root = ((x * x).sum(-1, keepdim=True) / c["d"] + EPS).sqrt()
            if not c["backward"]:
                outs.append(_exact_turned(x / root * w, turn, pairs))
                continue
            g = _exact_turned(s["d" + name].double(), turn.conj(), pairs)
            grads.append(torch.einsum("thf,thf->f", g, x / root))
            along = torch.einsum("thf,thf->th", g * w, x)[..., None] / c["d"]
            outs.append(g * w / root - x * along / root ** 3)
        return (*outs, *grads)
    if c["op"] == "append8":
        turn, pairs = _exact_turns(c, s)
        k = s["k"].double()
        if c["norm"]:
            k = k / ((k * k).sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * s["k_weight"].double()
        new = {"k": _exact_turned(k, turn, pairs), "v": s["v"].double()}
        cu, lens, table = s["cu_new"].tolist(), s["lens"].tolist(), s["table"].tolist()
        got = []
        for name in "kv":
            cache, scale = s[name + "_cache"].double(), s[name + "_scale"].double()
            for b in range(c["B"]):
                at, end = lens[b], lens[b] + cu[b + 1] - cu[b]
                for first in range(at // c["block"] * c["block"], end, c["block"]):
                    page, in_page = table[b][first // c["page"]], first % c["page"]
                    lo, hi = max(at, first), min(end, first + c["block"])
                    x = new[name][cu[b] + lo - at:cu[b] + hi - at]
                    top = x.abs().amax((0, 2))
                    need = torch.exp2(torch.ceil(torch.log2(top / 448)))
                    old = scale[page, in_page // c["block"]].clone()
                    if first >= at:
                        old = torch.zeros_like(old)
                    now = torch.where(top <= 448 * old, old, need)
                    held = cache[page, in_page:in_page + lo - first]
                    held.copy_(_exact_e4m3(held * (old / now).nan_to_num(0.0)[:, None]))
                    cache[page, in_page + lo - first:in_page + hi - first] = _exact_e4m3((x / now[:, None]).nan_to_num(0.0))
                    scale[page, in_page // c["block"]] = now
            got.append((cache, scale))
        return got[0][0], got[1][0], got[0][1], got[1][1], None, None

    queries, keys, group = _plan(c)
    R, plen, cu = c["Hq"] // c["Hkv"], c["plen"], s["cu_q"].tolist()
    out = torch.zeros(sum(queries), c["Hq"], c["d"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(queries), c["Hq"], dtype=torch.float64, device="cuda")
    for b, (nq, n) in enumerate(zip(queries, keys)):
        def gather(name):
            parts = []
            for table, length in ([(s["prefix_table"][group[b]], plen)] if plen else []) + [(s["table"][b], n)]:
                used = table[:-(-length // c["page"])].long()
                x = s[name + "_cache"].view(torch.uint8)[used].view(F8).double() * s[name + "_scale"][used].double().repeat_interleave(c["block"], 1)[..., None]
                parts.append(x.flatten(0, 1)[:length])
            return torch.cat(parts)
        keys_b, values_b, q = gather("k"), gather("v"), s["q"][cu[b]:cu[b + 1]].double()
        gap = torch.arange(n + plen - nq, n + plen, device="cuda").double()[:, None] - torch.arange(n + plen, device="cuda").double()
        for h in range(c["Hkv"]):
            heads = slice(h * R, (h + 1) * R)
            x = torch.einsum("ihf,jf->hij", q[:, heads], keys_b[:, h]) * (0.75 / math.sqrt(c["d"]))
            if c["cap"] > 0:
                x = c["cap"] * torch.tanh(x / c["cap"])
            if c["alibi"]:
                x -= s["slopes"][b, heads].double()[:, None, None] * gap.abs()
            if c["causal"]:
                x[:, gap < 0] = -math.inf
            if c["window"] >= 0:
                x[:, gap > c["window"]] = -math.inf
            total = torch.logsumexp(x, -1)
            lse[cu[b]:cu[b + 1], heads] = total.t()
            out[cu[b]:cu[b + 1], heads] = torch.einsum("hij,jf->ihf", torch.exp(x - total[..., None]).nan_to_num(0.0), values_b[:, h])
    return out, lse
