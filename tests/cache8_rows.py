"""The plain 64-bit form of attention over a cache held in 8 bits with bounds from each row's own
weights: what a value adds to the bound is its own size times its own weight."""
import math

import torch

import cache_ref as ref


def contexts(c, group, keep=None):
    """Of every sequence: K, V (fp64), V's factor of each key and head, positions, prefix length, and
    which keys there are (`keep`: a function of (sequence, prefix row or -1, keys of either))."""
    got = []
    per_slot = c.v_scale.cpu().double().repeat_interleave(c.block, 1)[..., None].expand(*c.v.shape[:3], c.d)
    for b, n in enumerate(c.lens_l):
        p = group[b] if group else -1
        pl = c.plens_l[p] if p >= 0 else 0
        parts = [(c.ptable, p, pl)] * (pl > 0) + [(c.table, b, n)]
        k, v, s = (torch.cat([c.rows(x, t, r, m) for t, r, m in parts]) for x in (c.k, c.v, per_slot))
        there = torch.ones(pl + n, dtype=torch.bool) if keep is None else keep(b, p, pl, n)
        got.append((k, v, s[..., 0].nan_to_num(0.0), pl, there))
    return got


def attention(q, c, counts, group=None, slopes=None, causal=False, wl=-1, wr=-1, cap=3.0, mult=0.75, q_pos=None,
              key_pos=None, pkey_pos=None, keep=None):
    """out, lse and their bounds.  The kernels' roundings, each relative to what it rounds:
    - q enters as pieces of e4m3 that leave at most 2^-17 of the row's largest value of an element;
    - a weight is rounded to fp16 where it multiplies V and where it divides (2^-11 each);
    - sums of n weighted values: products of 16 keys are added at a time, by half a step of 2^-22;
    - fp16's smallest step (2^-24): half of it for each key, where the row's largest weight is at least
      2^7 (a cap c up to 9.5 at known positions: 2^(15 - 2c log2 e) if that is less), and where a
      factor far below the largest is left with the weights, down to 2^18 s / top of them (the kernel
      for few rows: 2^-12);
    - the result is rounded once."""
    T, Hq, d = q.shape
    R, u, qc, at = Hq // c.Hkv, ref.UNIT[q.dtype], q.cpu(), ref.cu(counts)
    out = torch.zeros(T, Hq, d, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    largest = min(2.0 ** 7, 2.0 ** (15 - 2 * cap / math.log(2))) if 0 < cap <= 9.5 and key_pos is None else 2.0 ** 7
    for b, (k, v, s, pl, there) in enumerate(contexts(c, group, keep)):
        n, Lq, Lk = c.lens_l[b], counts[b], len(k)
        if Lq == 0 or not there.any():
            continue
        rows = slice(at[b], at[b + 1])
        qp = torch.arange(Lk - Lq, Lk) if q_pos is None else q_pos.cpu()[rows].long()
        for g in range(c.Hkv):
            own = torch.arange(pl, Lk) if key_pos is None else key_pos.cpu()[b, g, :n].long()
            pre = torch.arange(pl) if pkey_pos is None or not pl else pkey_pos.cpu()[group[b], g, :pl].long()
            sl = None if slopes is None else slopes.cpu()[b]
            kpos = torch.cat([pre, own])[there]
            z, e = ref.logits(qc[rows], k[there], g, R, qp, kpos, sl, causal, wl, wr, cap, mult)
            hs = slice(g * R, (g + 1) * R)
            piece = qc[rows, hs].double().abs().amax(-1).t()[..., None] * k[there][:, g].abs().sum(-1) * abs(mult) / math.sqrt(d) * 2.0 ** -17
            worst = (e + piece).masked_fill(torch.isinf(z), 0.0).amax(-1)
            total = torch.logsumexp(z, -1)
            w = torch.exp(z - total[..., None]).nan_to_num(0.0)
            vg, sg = v[there][:, g], s[there][:, g]
            least = (sg / s[:, g].max().clamp(min=1e-300)).clamp(min=2.0 ** -100)
            rest = torch.minimum((least * 2.0 ** 18).clamp(max=1.0), torch.where(least < 0.5, 2.0 ** -12, 1.0).double())
            lost = torch.einsum("hij,jf->ihf", (w > 0).double(), vg.abs() / rest[:, None]) * 2.0 ** -25 / largest
            o, mag = torch.einsum("hij,jf->ihf", w, vg), torch.einsum("hij,jf->ihf", w, vg.abs())
            some = torch.isfinite(total)
            lse[rows, hs] = total.t()
            lse_tol[rows, hs] = (worst + 2.0 ** -19 + total.abs().nan_to_num(0, 0, 0) * 2.0 ** -22).t()
            out[rows, hs] = o
            off = 2 * 2.0 ** -11 + 2.0 ** -18 + (Lk / 16 + 60) * 2.0 ** -22
            out_tol[rows, hs] = (off + 2 * worst.t()[..., None]) * mag + u * o.abs() + lost + (2.0 ** -25 if q.dtype == torch.float16 else 0.0)
            assert not w[~some].any()
    return out, lse, out_tol, lse_tol
