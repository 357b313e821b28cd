"""Plain 64-bit forms of the calls over a cache held in 8 bits, of norms with rotation
and of the calls that move pages, and the caches their tests run on."""
import math

import torch

import cache_ref as ref

F8 = torch.float8_e4m3fn
NAN8 = 0x7f


def e4m3(x):
    """The nearest e4m3 value (ties to even, at most 448) of fp64 values."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def pow2_scale(top):
    """The smallest power of two s >= 2^-126 with top <= 448 s; 0 for 0 (fp64)."""
    m, e = torch.frexp(top.double())
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    return torch.where(top > 0, torch.exp2(e.double()), torch.zeros_like(m))


class Cache8(ref.Cache):
    """ref.Cache with its pools in 8 bits.  What no slot uses holds NaN bytes, and so
    do the scales of blocks without slots.  `scale_of(rows, blocks, heads)` gives the
    scales (default: what the values need)."""

    def __init__(self, lens, plens=(), Hkv=1, d=160, page=16, block=16, seed=0, strided=False, scales=None, device="cuda"):
        super().__init__(lens, plens, Hkv, d, page, torch.float32, seed, False, device="cpu")
        self.block = block
        self.k8, self.k_scale = self._quantised(self.k, strided, scales, device, seed)
        self.v8, self.v_scale = self._quantised(self.v, strided, scales, device, seed + 1)
        # the values the pools stand for, for the plain forms
        self.k = self._values(self.k8, self.k_scale)
        self.v = self._values(self.v8, self.v_scale)
        for name in ("table", "ptable", "lens", "plens"):
            setattr(self, name, getattr(self, name).to(device))

    def _quantised(self, pool, strided, scales, device, seed):
        pages, page, Hkv, d = pool.shape
        x = pool.double().view(pages, page // self.block, self.block, Hkv, d)
        used = ~torch.isnan(x)
        top = torch.where(used, x, 0.0).abs().amax((2, 4))
        scale = pow2_scale(top) if scales is None else scales(top, torch.Generator().manual_seed(seed + 7)).double()
        q = e4m3(torch.where(used, x, 0.0) / scale.clamp(min=1e-300)[:, :, None, :, None])
        bits = q.float().to(F8).view(torch.uint8)
        bits[~used] = NAN8
        bits = bits.view(pages, page, Hkv, d)
        scale = torch.where(used.any(4).any(2), scale, math.nan).float()
        if strided:
            wide = torch.full((pages + 1, page, Hkv + 1, d + 16), NAN8, dtype=torch.uint8)
            wide[:pages, :, :Hkv, :d] = bits
            swide = torch.full((pages, page // self.block + 1, Hkv + 2), math.nan)
            swide[:, :page // self.block, 1:Hkv + 1] = scale
            return wide.to(device).view(F8)[:pages, :, :Hkv, :d], swide.to(device)[:, :page // self.block, 1:Hkv + 1]
        return bits.to(device).view(F8), scale.to(device)

    def _values(self, pool, scale):
        x = pool.cpu().float().double()
        return x * scale.cpu().double().repeat_interleave(self.block, 1)[..., None]


def attention(q, c, counts, **opt):
    """ref.attention with the bounds of the 8-bit kernel: a row of q enters as pieces of
    e4m3, which leaves at most 2^-17 of its largest value of each element; weights and V
    times its scale are rounded to fp16 (2^-11 each, V's twice where a scale is no power
    of two)."""
    out, lse, out_tol, lse_tol = ref.attention(q, c, counts, **opt)
    Hq, d = q.shape[1], q.shape[2]
    R, qc, at = Hq // c.Hkv, q.cpu().double(), ref.cu(counts)
    sigma = opt.get("mult", 0.75) / math.sqrt(d)
    u = ref.UNIT[q.dtype]
    for b, (k, v, pl) in enumerate(ref.contexts(c, opt.get("group"))):
        if counts[b] == 0 or len(k) == 0:
            continue
        rows = slice(at[b], at[b + 1])
        for g in range(c.Hkv):
            hs = slice(g * R, (g + 1) * R)
            piece = qc[rows, hs].abs().amax(-1) * float(k[:, g].abs().sum(-1).max()) * abs(sigma) * 2.0 ** -17
            vmax = v[:, g].abs().amax()
            lse_tol[rows, hs] += piece
            # weights far below the row's largest end at fp16's smallest step: 2^-31 of it each
            out_tol[rows, hs] += 2 * piece[..., None] * vmax + 3 * 2.0 ** -11 * vmax + len(k) * 2.0 ** -31 * vmax
    return out, lse, out_tol, lse_tol


def normed(x, w, eps):
    """fp64 norm of rows, and r."""
    y = x.cpu().double()
    r = 1 / (y.square().mean(-1, keepdim=True) + eps).sqrt()
    return y * r * (1.0 if w is None else w.cpu().double()), r


def turned(y, positions, inv_freq, pair_axis, interleaved, inverse=False):
    """fp64 rotation of fp64 rows, and the sum of magnitudes that meet in each feature."""
    if inv_freq is None:
        return y, y.abs()
    n = len(inv_freq)
    pos = positions.cpu().double()
    pos = pos[None] if pos.dim() == 1 else pos
    axis = pair_axis.cpu().long() if pair_axis is not None else torch.zeros(n, dtype=torch.long)
    ang = pos[axis].t() * inv_freq.cpu().double()[None] * (-1 if inverse else 1)
    cos, sin = ang.cos()[:, None], ang.sin()[:, None]
    i = torch.arange(n)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    a, b = y[..., ia], y[..., ib]
    out, mag = y.clone(), y.abs()
    out[..., ia], out[..., ib] = a * cos - b * sin, b * cos + a * sin
    mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return out, mag


def forked(page, N, W, table, lens, held, refs, parents, room):
    """(table rows, lens, held, refs, copies (src, dst, used)) by the definition, in lists; None if pages lack."""
    R = len(lens)
    refs = list(refs)
    first = {}
    for r, p in enumerate(parents):
        if p >= 0:
            first.setdefault(p, r)
    for p in range(R):
        times = parents.count(p)
        for c in range(held[p]):
            refs[table[p][c]] += times - 1 if c < lens[p] // page else (0 if times else -1)
    rows, new_lens, new_held, copies = [], [], [], []
    free = [i for i in range(N) if refs[i] == 0]
    for r, p in enumerate(parents):
        if p < 0:
            rows.append([])
            new_lens.append(0)
            new_held.append(0)
            continue
        full = lens[p] // page
        mine = list(table[p][:held[p] if first[p] == r else full])
        want = -(-(lens[p] + room[r]) // page)
        if want > W:
            return None
        while len(mine) < want:
            if not free:
                return None
            mine.append(free.pop(0))
            refs[mine[-1]] = 1
        if first[p] != r and lens[p] % page:
            copies.append((table[p][full], mine[full], lens[p] % page))
        rows.append(mine)
        new_lens.append(lens[p])
        new_held.append(len(mine))
    return rows, new_lens, new_held, refs, copies


def compacted(refs):
    """(live, moves (src, dst)) by the definition."""
    live = sum(x > 0 for x in refs)
    holes = [i for i in range(live) if refs[i] <= 0]
    movers = [i for i in range(live, len(refs)) if refs[i] > 0]
    return live, list(zip(movers, holes))
