"""Plain 64-bit forms of the generation calls, and the caches their tests run on."""
import math
import random

import torch

# half a step of a type's rounding, relative to the value
UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
NAN = math.nan


class Cache:
    """A pool of pages in random order with tables for sequences of the given
    lengths and, first, for shared prefixes.  Everything that no slot uses
    holds NaN, and table entries of unused pages are numbers out of the pool."""

    def __init__(self, lens, plens=(), Hkv=1, d=160, page=16, dtype=torch.bfloat16, seed=0,
                 strided=False, extra_width=1, device="cuda", poison=True):
        g = torch.Generator().manual_seed(seed)
        self.lens_l, self.plens_l, self.Hkv, self.d, self.page = list(lens), list(plens), Hkv, d, page
        rows = list(lens) + list(plens)
        used = sum(-(-n // page) for n in rows)
        pages = used + 2
        order = torch.randperm(pages, generator=g)[:used].tolist()
        pad_h, pad_f = (1, 8) if strided else (0, 0)
        shape = (pages, page, Hkv + pad_h, d + pad_f)

        def pool(std):
            x = torch.full(shape, NAN) if poison else torch.zeros(shape)
            view = x[:, :, :Hkv, :d]
            at = 0
            for n in rows:
                for j0 in range(0, n, page):
                    m = min(page, n - j0)
                    view[order[at], :m] = torch.randn(m, Hkv, d, generator=g) * std
                    at += 1
            return x.to(dtype).to(device)[:, :, :Hkv, :d]

        self.k, self.v = pool(1.0), pool(1.0)

        def table(lengths, at):
            width = max([1] + [-(-n // page) for n in lengths]) + extra_width
            t = torch.full((max(1, len(lengths)), width), -7 if poison else 0, dtype=torch.int32)
            for r, n in enumerate(lengths):
                c = -(-n // page)
                t[r, :c] = torch.tensor(order[at:at + c], dtype=torch.int32)
                if poison:
                    t[r, c:] = pages + 1000 if r % 2 else -7
                at += c
            return t[:len(lengths)].to(device), at

        self.table, at = table(lens, 0)
        self.ptable, _ = table(plens, at)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=device)
        self.plens = torch.tensor(plens, dtype=torch.int32, device=device)
        self.num_pages = pages

    def rows(self, pool, table, r, n):
        """The first n slots of a table row, fp64 on the CPU [n, Hkv, d]."""
        t = table[r].cpu().long()
        c = -(-n // self.page)
        return pool.cpu().double()[t[:c]].reshape(-1, self.Hkv, self.d)[:n]


def cu(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def contexts(c, group):
    """Of every sequence: K, V (fp64), default positions, prefix length."""
    got = []
    for b, n in enumerate(c.lens_l):
        p = group[b] if group else -1
        pl = c.plens_l[p] if p >= 0 else 0
        k, v = c.rows(c.k, c.table, b, n), c.rows(c.v, c.table, b, n)
        if pl:
            k = torch.cat([c.rows(c.k, c.ptable, p, pl), k])
            v = torch.cat([c.rows(c.v, c.ptable, p, pl), v])
        got.append((k, v, pl))
    return got


def logits(q, k, g, R, qpos, kpos, slopes, causal, wl, wr, cap, mult):
    """Masked fp64 logits [R, Lq, Lk] of one K/V head, and a bound on their fp32 error."""
    d = q.shape[-1]
    sigma = mult / math.sqrt(d)
    qg, kg = q[:, g * R:(g + 1) * R].double(), k[:, g]
    s = torch.einsum("ihf,jf->hij", qg, kg) * sigma
    mag = torch.einsum("ihf,jf->hij", qg.abs(), kg.abs()) * abs(sigma)
    # d products summed in fp32, each addition off by at most a whole step (2^-23)
    # of the partial sum's bound; the scale and the cap add a few steps of the value
    err = mag * d * 2.0 ** -23
    z = cap * torch.tanh(s / cap) if cap > 0 else s
    err = err + z.abs() * 2.0 ** -20 + (abs(cap) * 2.0 ** -20 if cap > 0 else 0.0)
    gap = (qpos[:, None] - kpos[None, :]).double()
    if slopes is not None:
        bias = slopes[g * R:(g + 1) * R, None, None].double() * gap.abs()[None]
        z = z - bias
        err = err + bias.abs() * 2.0 ** -22
    w_r = 0 if causal else wr
    bad = torch.zeros_like(gap, dtype=torch.bool)
    if wl >= 0:
        bad |= gap > wl
    if w_r >= 0:
        bad |= -gap > w_r
    z = z.masked_fill(bad[None], -math.inf)
    return z, err.masked_fill(bad[None], 0.0)


def attention(q, c, counts, group=None, slopes=None, causal=False, wl=-1, wr=-1, cap=3.0, mult=0.75,
              q_pos=None, key_pos=None, pkey_pos=None):
    """out, lse (fp64), and the bounds on a 16-bit kernel's error in each."""
    T, Hq, d = q.shape
    R, u, qc, at = Hq // c.Hkv, UNIT[q.dtype], q.cpu(), cu(counts)
    out = torch.zeros(T, Hq, d, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    for b, (k, v, pl) in enumerate(contexts(c, group)):
        n, Lq, Lk = c.lens_l[b], counts[b], len(k)
        if Lq == 0 or Lk == 0:
            continue
        qp = torch.arange(Lk - Lq, Lk) if q_pos is None else q_pos.cpu()[at[b]:at[b + 1]].long()
        for g in range(c.Hkv):
            own = torch.arange(pl, Lk) if key_pos is None else key_pos.cpu()[b, g, :n].long()
            pre = torch.arange(pl) if pkey_pos is None or not pl else pkey_pos.cpu()[group[b], g, :pl].long()
            sl = None if slopes is None else slopes.cpu()[b]
            z, e = logits(qc[at[b]:at[b + 1]], k, g, R, qp, torch.cat([pre, own]), sl, causal, wl, wr, cap, mult)
            total = torch.logsumexp(z, -1)
            w = torch.exp(z - total[..., None]).nan_to_num(0.0)
            worst = e.amax(-1)
            hs = slice(g * R, (g + 1) * R)
            lse[at[b]:at[b + 1], hs] = total.t()
            # the sum of Lk fp32 terms, the exponentials and the final logarithm
            lse_tol[at[b]:at[b + 1], hs] = (worst + 2.0 ** -19 + total.abs().nan_to_num(0, 0, 0) * 2.0 ** -22).t()
            o = torch.einsum("hij,jf->ihf", w, v[:, g])
            mag = torch.einsum("hij,jf->ihf", w, v[:, g].abs())
            out[at[b]:at[b + 1], hs] = o
            # a weight is rounded to 16 bits as a numerator and (or) in the sum that divides
            # it (2 u of the weighted magnitudes), off by its logit's error twice, and the
            # result is rounded once
            out_tol[at[b]:at[b + 1], hs] = (2 * u + 2.0 ** -18 + 2 * worst.t()[..., None]) * mag + u * o.abs() + 2.0 ** -24
    return out, lse, out_tol, lse_tol


def weights(q, c, counts, lse, group=None, slopes=None, causal=False, wl=-1, wr=-1, cap=3.0, mult=0.75,
            q_pos=None, key_pos=None, pkey_pos=None):
    """Sums of exp(z - lse) per own key [B][Hkv, n] and prefix key [P][Hkv, n], and their bounds."""
    Hq = q.shape[1]
    R, qc, at = Hq // c.Hkv, q.cpu(), cu(counts)
    own = [torch.zeros(c.Hkv, n, dtype=torch.float64) for n in c.lens_l]
    pre = [torch.zeros(c.Hkv, n, dtype=torch.float64) for n in c.plens_l]
    own_t, pre_t = [torch.zeros_like(x) for x in own], [torch.zeros_like(x) for x in pre]
    for b, (k, _, pl) in enumerate(contexts(c, group)):
        n, Lq, Lk = c.lens_l[b], counts[b], len(k)
        if Lq == 0 or Lk == 0:
            continue
        qp = torch.arange(Lk - Lq, Lk) if q_pos is None else q_pos.cpu()[at[b]:at[b + 1]].long()
        for g in range(c.Hkv):
            kp = torch.arange(pl, Lk) if key_pos is None else key_pos.cpu()[b, g, :n].long()
            pp = torch.arange(pl) if pkey_pos is None or not pl else pkey_pos.cpu()[group[b], g, :pl].long()
            sl = None if slopes is None else slopes.cpu()[b]
            z, e = logits(qc[at[b]:at[b + 1]], k, g, R, qp, torch.cat([pp, kp]), sl, causal, wl, wr, cap, mult)
            L = lse.cpu()[at[b]:at[b + 1], g * R:(g + 1) * R].double().t()[..., None]
            w = torch.exp(z - L).nan_to_num(0.0)
            # the exponent's absolute error is the logit's plus a few steps of its size
            t = w * (e + 2.0 ** -18 + (z.abs().nan_to_num(0, 0, 0) + L.abs().nan_to_num(0, 0, 0)) * 2.0 ** -22)
            w, t = w.sum((0, 1)), t.sum((0, 1))
            own[b][g] += w[pl:]
            own_t[b][g] += t[pl:]
            if pl:
                pre[group[b]][g] += w[:pl]
                pre_t[group[b]][g] += t[:pl]
    return own, pre, own_t, pre_t


def evicted(n, scores, key_pos, next_pos, budget, recent):
    """(new length, [(dst, src)]) of one row and K/V head, by sorting."""
    k = min(n, budget)

    def order(j):
        s = float(scores[j])
        return (int(key_pos[j]) < next_pos - recent,
                0.0 if int(key_pos[j]) >= next_pos - recent else (math.inf if math.isnan(s) else -s),
                math.isnan(s) and int(key_pos[j]) < next_pos - recent, j)

    kept = set(sorted(range(n), key=order)[:k])
    holes = [j for j in range(k) if j not in kept]
    movers = [j for j in range(k, n) if j in kept]
    assert len(holes) == len(movers)
    return k, list(zip(holes, movers))


def rotated(x, positions, inv_freq, pair_axis, interleaved, inverse=False):
    """fp64 rotation of x [T, H, d] and a bound on a 16-bit kernel's error."""
    y = x.cpu().double()
    n = len(inv_freq)
    pos = positions.cpu().double()
    axis = pair_axis.cpu().long() if pair_axis is not None else torch.zeros(n, dtype=torch.long)
    ang = pos[axis].t() * inv_freq.cpu().double()[None]
    if inverse:
        ang = -ang
    cos, sin = ang.cos()[:, None], ang.sin()[:, None]
    i = torch.arange(n)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    a, b = y[..., ia].clone(), y[..., ib].clone()
    out, tol = y.clone(), torch.zeros_like(y)
    out[..., ia], out[..., ib] = a * cos - b * sin, b * cos + a * sin
    # one rounding of the result, and sine and cosine off by a few steps of 2^-24
    for ix in (ia, ib):
        tol[..., ix] = UNIT[x.dtype] * out[..., ix].abs() + (a.abs() + b.abs()) * 2.0 ** -20 + 2.0 ** -26
    return out, tol


def spread(seed, count, lo, hi):
    r = random.Random(seed)
    return [max(lo, min(hi, round(math.exp(r.uniform(math.log(max(lo, 1)), math.log(hi)))))) for _ in range(count)]
