"""The generation calls on the GPU at their edges: exact means of equal V rows, metadata
that does not fit, pages out of the pool, expanded inputs, calls without tokens."""
import math

import pytest
import torch

import cache_ref as ref
from ragged_gqa_attention_varlen_gb300 import cache as C
from test_cache_gpu import BF, HF, i32, normal, status, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from ragged_gqa_attention_varlen_gb300 import _build

    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return C.load()


# ---------------------------------------------------------------- sums of the weights

@pytest.mark.parametrize("cap", [0.0, 3.0, 9.0, 30.0])
@pytest.mark.parametrize("lens,plens,counts,Hq,Hkv,d,page,dtype", [
    ([1, 2, 3, 5], (), [20] * 4, 16, 1, 160, 16, BF), ([2, 4, 130], (), [30, 10, 40], 8, 2, 128, 32, BF),
    ([3, 9, 200], (), [10, 20, 10], 8, 1, 64, 16, HF), ([2, 1, 4], [3], [10, 10, 20], 16, 1, 160, 16, BF),
    ([5000], (), [1], 8, 1, 160, 64, BF)])
def test_equal_values_come_out_exactly(lens, plens, counts, Hq, Hkv, d, page, dtype, cap):
    """out is a weighted mean of V rows: where they are all the same row it is that row, whatever
    the weights' roundings, as the weights that multiply V are those whose sum divides.  Sums of
    at most 5000 terms in fp32 are off by 5000 / 16 additions of 2^-22 (a product of 16 keys is
    added at a time) and the row sum, halves and reciprocal by less than 1000 * 2^-24: 1.4e-4
    together, below half a step of either type (bf16 2^-9, fp16 2^-12 of the value)."""
    group = [0] * len(lens) if plens else None
    kc = ref.Cache(lens, plens, Hkv, d, page, dtype)
    # half of the features as large as their exponent has them: half a step is least there
    row = normal(7, Hkv, d, dtype=dtype)
    row[:, ::2] = torch.where(row[:, ::2] > 0, 2.0, -2.0) * (1 - torch.finfo(dtype).eps / 2)
    kc.v.copy_(row)
    q = normal(8, sum(counts), Hq, d, dtype=dtype, std=3.0)
    call = {}
    if plens:
        call = dict(prefix_table=kc.ptable, prefix_lens=kc.plens, cu_prefix=i32([0, len(lens)]))
    out, _ = C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, kc.lens, i32(ref.cu(counts)), softcap=cap, **call)
    want = row.repeat_interleave(Hq // Hkv, 0).expand_as(out)
    assert torch.equal(out, want), (out != want).float().mean()


# ---------------------------------------------------------------- key weights of many Q tiles

# Q tiles that a CTA streams, at least 12 of them, so that they go round the ring several times
STREAMS = [
    dict(lens=[700], counts=[600], Hq=96, Hkv=1, d=160, dtype=BF, cap=3.0, causal=False),
    dict(lens=[1000], counts=[800], Hq=96, Hkv=1, d=160, dtype=HF, cap=0.0, causal=True, alibi=True),
    dict(lens=[400] * 16, counts=[40] * 16, Hq=96, Hkv=1, d=160, dtype=BF, cap=3.0, causal=True, alibi=True),
    dict(lens=[20] * 64, counts=[1] * 64, plens=[5000], Hq=96, Hkv=1, d=160, dtype=BF, cap=3.0, causal=True),
    dict(lens=[30, 900, 5, 300], counts=[1, 500, 1, 300], plens=[300], Hq=48, Hkv=1, d=160, dtype=HF, cap=30.0, causal=False),
    dict(lens=[1500], counts=[1500], Hq=32, Hkv=8, d=128, dtype=HF, cap=0.0, causal=True),
    dict(lens=[900, 2, 1300], counts=[900, 1, 1300], plens=[], Hq=32, Hkv=4, d=128, dtype=BF, cap=3.0, causal=True,
         alibi=True),
    dict(lens=[64] * 128, counts=[1] * 128, plens=[4000], Hq=64, Hkv=2, d=128, dtype=HF, cap=0.0, causal=False),
    dict(lens=[1200], counts=[1200], Hq=32, Hkv=4, d=64, dtype=HF, cap=3.0, causal=True, alibi=True)]


@pytest.mark.parametrize("c", STREAMS, ids=lambda c: f"d{c['d']}-{c['Hq']}-{len(c['lens'])}-{max(c['counts'])}-{c['cap']:g}")
def test_key_weights_of_many_tiles(c):
    plens, d, Hq, Hkv, dt = c.get("plens", []), c["d"], c["Hq"], c["Hkv"], c["dtype"]
    B, T = len(c["lens"]), sum(c["counts"])
    kc = ref.Cache(c["lens"], plens, Hkv, d, 64, dt)
    q = normal(3, T, Hq, d, dtype=dt, std=2.0)
    opt = dict(causal=c["causal"], cap=c["cap"], group=[0] * B if plens else None)
    call = dict(causal=c["causal"], softcap=c["cap"])
    if c.get("alibi"):
        opt["slopes"] = torch.rand(B, Hq, generator=torch.Generator().manual_seed(2)) * 0.05
        call["alibi_slopes"] = opt["slopes"].cuda()
    pre0 = None
    if plens:
        call.update(prefix_table=kc.ptable, prefix_lens=kc.plens, cu_prefix=i32([0, B]))
        pre0 = torch.zeros(1, Hkv, kc.ptable.shape[1] * 64, device="cuda")
    st, cu_q = status(), i32(ref.cu(c["counts"]))
    _, lse = C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, kc.lens, cu_q, status=st, **call)

    def weights():
        own, pre = C.attention_varlen_cache_weights(q, kc.k, kc.table, kc.lens, cu_q, lse, status=st,
                                                    prefix_scores=None if pre0 is None else pre0.clone(), **call)
        torch.cuda.synchronize()
        assert int(st) == 0
        return own, pre

    own, pre = weights()
    want, pwant, tol, ptol = ref.weights(q, kc, c["counts"], lse, **opt)
    for b, n in enumerate(c["lens"]):
        within(f"own {b}", own[b, :, :n], want[b], tol[b] + want[b] * 2.0 ** -22)
    for b, n in enumerate(plens):
        within(f"prefix {b}", pre[b, :, :n], pwant[b], ptol[b] + pwant[b] * 2.0 ** -22)
    for _ in range(3):
        again, pagain = weights()
        assert torch.equal(again, own) and (pre is None or torch.equal(pagain, pre))


# ---------------------------------------------------------------- append: metadata that does not fit

@pytest.mark.parametrize("cu,lens,written", [
    ([2, 3, 6], [20, 9], []),             # does not start at 0
    ([0, 4, 2], [20, 9], []),             # decreases
    ([0, -1, 6], [20, 9], []),
    ([0, 3, 7], [20, 9], []),             # more tokens than there are
    ([0, 3, 6], [-2, 9], [1]),            # a negative length: the other sequence's tokens are taken
    ([0, 3, 6], [20, 10 ** 6], [0]),
    ([0, 3, 6], [46, 9], [1]),            # two of three tokens would fit: none is taken
    ([0, 3, 6], [20, 2 ** 31 - 1], [0])])
@pytest.mark.parametrize("rot", [False, True])
def test_append_leaves_out_what_does_not_fit(cu, lens, written, rot):
    kc = ref.Cache([48, 48], page=16, extra_width=0, poison=False)
    k0, v0 = kc.k.clone(), kc.v.clone()
    k, v = normal(1, 6, 1, 160), normal(2, 6, 1, 160)
    kp = torch.full((2, 1, 48), -5, dtype=torch.int32, device="cuda")
    sc, out, st = torch.full((2, 1, 48), 3.0, device="cuda"), i32([-7, -7]), status()
    kw = {}
    if rot:
        kw = dict(positions=i32([9] * 6), inv_freq=torch.zeros(80, dtype=torch.float64, device="cuda"))  # angle 0
    C.attention_varlen_cache_append(k, v, kc.k, kc.v, kc.table, i32(lens), i32(cu), key_pos=kp, scores=sc, lens_out=out,
                                    status=st, **kw)
    torch.cuda.synchronize()
    bad_cu = not written
    assert int(st) == (1 if bad_cu else C.DEV_BAD_CACHE)
    wl, wk, wv, wp, ws = list(lens), k0.clone(), v0.clone(), torch.full_like(kp, -5), torch.full_like(sc, 3.0)
    for b in written:
        n = cu[b + 1] - cu[b]
        wl[b] += n
        for i in range(n):
            j = lens[b] + i
            pg = int(kc.table[b, j // 16])
            wk[pg, j % 16], wv[pg, j % 16] = k[cu[b] + i], v[cu[b] + i]
            wp[b, :, j], ws[b, :, j] = 9 if rot else j, 0.0
    assert out.tolist() == wl
    assert torch.equal(kc.k, wk) and torch.equal(kc.v, wv) and torch.equal(kp, wp) and torch.equal(sc, ws)


# ---------------------------------------------------------------- calls without tokens

def test_no_tokens_with_key_positions():
    """After an eviction (key positions) a step without query tokens is as good as one before it."""
    kc = ref.Cache([20, 9], [30], page=16, Hkv=2, d=128)
    none = torch.empty(0, 8, 128, dtype=BF, device="cuda")
    kp = torch.zeros(2, 2, kc.table.shape[1] * 16, dtype=torch.int32, device="cuda")
    call = dict(key_pos=kp, prefix_table=kc.ptable, prefix_lens=kc.plens, cu_prefix=i32([0, 2]),
                prefix_key_pos=torch.zeros(1, 2, kc.ptable.shape[1] * 16, dtype=torch.int32, device="cuda"), causal=True)
    for qp in (None, torch.empty(0, dtype=torch.int32, device="cuda")):
        st = status()
        out, lse = C.attention_varlen_cache_fwd(none, kc.k, kc.v, kc.table, kc.lens, i32([0, 0, 0]), q_pos=qp, status=st,
                                                **call)
        assert out.shape == (0, 8, 128) and lse.shape == (0, 8)
        sc = torch.rand(2, 2, kc.table.shape[1] * 16, device="cuda")
        got, _ = C.attention_varlen_cache_weights(none, kc.k, kc.table, kc.lens, i32([0, 0, 0]), lse, sc, q_pos=qp,
                                                  scores_out=torch.full_like(sc, 5.0), status=st, **call)
        torch.cuda.synchronize()
        assert int(st) == 0
        for b, n in enumerate([20, 9]):
            assert torch.equal(got[b, :, :n], sc[b, :, :n]) and (got[b, :, n:] == 5).all()


# ---------------------------------------------------------------- pages out of the pool, lengths beyond the table

class Without:
    """A cache as its calls are to read it: slots of pages out of the pool do not exist."""

    def __init__(self, kc, lens, plens, own_gone, pre_gone):
        self.Hkv, self.d, self.k, self.v, self.kc = kc.Hkv, kc.d, kc.k, kc.v, kc
        self.table, self.ptable = "own", "prefix"
        self.keep = {"own": [[j for j in range(n) if (b, j // kc.page) not in own_gone] for b, n in enumerate(lens)],
                     "prefix": [[j for j in range(n) if (b, j // kc.page) not in pre_gone] for b, n in enumerate(plens)]}
        self.lens_l, self.plens_l = ([len(x) for x in self.keep[t]] for t in ("own", "prefix"))

    def rows(self, pool, table, r, n):
        keep = self.keep[table][r]
        whole = self.kc.rows(pool, self.kc.table if table == "own" else self.kc.ptable, r, max(keep, default=-1) + 1)
        return whole[torch.tensor(keep, dtype=torch.long)] if keep else whole[:0]

    def positions(self, table, offset):
        width = max([1] + [len(x) for x in self.keep[table]])
        kp = torch.zeros(len(self.keep[table]), self.Hkv, width, dtype=torch.int32)
        for b, x in enumerate(self.keep[table]):
            kp[b, :, :len(x)] = torch.tensor([offset + j for j in x], dtype=torch.int32)
        return kp


@pytest.mark.parametrize("cap,alibi,causal,moved", [(3.0, True, True, False), (0.0, False, False, False),
                                                    (30.0, True, True, False), (3.0, True, True, True),
                                                    (0.0, False, True, True)])
@pytest.mark.parametrize("lens,plens,counts,Hq,Hkv,d,page,own_gone,pre_gone", [
    ([70, 40, 200], (), [1, 3, 2], 16, 1, 160, 16, [(0, 1), (2, 0), (2, 12)], []),
    ([300, 129], (), [1, 40], 8, 2, 128, 64, [(0, 0), (0, 4), (1, 1)], []),
    ([2000, 700], (), [1, 1], 8, 1, 64, 256, [(0, 3), (0, 7)], []),
    ([40, 90], [500], [2, 1], 48, 1, 160, 32, [(1, 2)], [(0, 0), (0, 9), (0, 10)]),
    ([33], (), [2], 8, 1, 64, 64, [(0, 0)], [])])  # nothing is left
def test_pages_out_of_the_pool_are_left_out(lens, plens, counts, Hq, Hkv, d, page, own_gone, pre_gone, cap, alibi, causal,
                                           moved):
    kc = ref.Cache(lens, plens, Hkv, d, page, HF)
    bad, pbad = kc.table.clone(), kc.ptable.clone()
    for i, (b, j) in enumerate(own_gone):
        bad[b, j] = -1 if i % 2 else kc.num_pages
    for i, (b, j) in enumerate(pre_gone):
        pbad[b, j] = 2 ** 31 - 1 if i % 2 else -2 ** 31
    left = Without(kc, lens, plens, own_gone, pre_gone)
    B, P, T = len(lens), len(plens), sum(counts)
    plen = plens[0] if P else 0
    group = [0] * B if P else None
    qp = [plen + n - c + i for n, c in zip(lens, counts) for i in range(c)]
    slopes = torch.rand(B, Hq, generator=torch.Generator().manual_seed(3)) * 0.05 if alibi else None
    q = normal(5, T, Hq, d, dtype=HF, std=2.0)
    opt = dict(group=group, slopes=slopes, causal=causal, cap=cap, q_pos=torch.tensor(qp),
               key_pos=left.positions("own", plen), pkey_pos=left.positions("prefix", 0) if P else None)
    call = dict(causal=causal, softcap=cap)
    if alibi:
        call["alibi_slopes"] = slopes.cuda()
    if P:
        call.update(prefix_table=pbad, prefix_lens=kc.plens, cu_prefix=i32([0, B]))
    if moved:  # the same positions, given explicitly
        call["q_pos"] = i32(qp)
        call["key_pos"] = (plen + torch.arange(bad.shape[1] * page, dtype=torch.int32, device="cuda")).expand(B, Hkv, -1)
    st, cu_q = status(), i32(ref.cu(counts))
    want, wl, otol, ltol = ref.attention(q, left, counts, **opt)
    out, lse = C.attention_varlen_cache_fwd(q, kc.k, kc.v, bad, kc.lens, cu_q, status=st, **call)
    torch.cuda.synchronize()
    assert int(st) == C.DEV_BAD_CACHE
    within("lse", lse, wl, ltol)
    within("out", out, want, otol)
    start = torch.rand(B, Hkv, bad.shape[1] * page, device="cuda")
    pstart = torch.rand(P, Hkv, pbad.shape[1] * page, device="cuda") if P else None
    st = status()
    own, pre, wtol, ptol = ref.weights(q, left, counts, lse, **opt)
    sc, psc = C.attention_varlen_cache_weights(q, kc.k, bad, kc.lens, cu_q, lse, start.clone(), status=st,
                                               prefix_scores=None if pstart is None else pstart.clone(), **call)
    torch.cuda.synchronize()
    assert int(st) == C.DEV_BAD_CACHE
    for got, x0, w, tol, table in ((sc, start, own, wtol, "own"), (psc, pstart, pre, ptol, "prefix")):
        for b, keep in enumerate(left.keep[table] if got is not None else []):
            j = torch.tensor(keep, dtype=torch.long)
            target = x0[b].cpu().double()[:, j] + w[b]
            within(f"{table} {b}", got[b][:, j.cuda()], target, tol[b] + target.abs() * 2.0 ** -22)
            gone = torch.ones(got.shape[2], dtype=torch.bool)
            gone[j] = False
            assert torch.equal(got[b][:, gone.cuda()], x0[b][:, gone.cuda()])  # keep what they had


def test_a_bad_length_concerns_its_keys_only():
    """The other sequences' results are what they are without it; the sequence itself has its
    prefix left, or nothing."""
    lens, counts = [300, 40, 90, 20], [1, 2, 1, 1]
    kc = ref.Cache(lens, [50], page=16)
    q, cu_q = normal(3, 5, 8, 160), i32(ref.cu(counts))
    group = dict(prefix_table=kc.ptable, prefix_lens=kc.plens, cu_prefix=i32([2, 4]))
    sc0 = torch.rand(4, 1, kc.table.shape[1] * 16, device="cuda")
    for bad in (-1, 10 ** 6, -2 ** 31):
        for at in (1, 2):
            ln, st = list(lens), status()
            ln[at] = bad
            out, lse = C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, i32(ln), cu_q, status=st, softcap=3.0, **group)
            torch.cuda.synchronize()
            assert int(st) == C.DEV_BAD_CACHE
            left = Without(kc, [0 if b == at else n for b, n in enumerate(lens)], [50], [], [])
            want, wl, otol, ltol = ref.attention(q, left, counts, group=[-1, -1, 0, 0])
            within("lse", lse, wl, ltol)
            within("out", out, want, otol)
            st = status()
            sc, _ = C.attention_varlen_cache_weights(q, kc.k, kc.table, i32(ln), cu_q, lse, sc0.clone(), status=st, **group)
            torch.cuda.synchronize()
            assert int(st) == C.DEV_BAD_CACHE and torch.equal(sc[at], sc0[at])
            own, _, wtol, _ = ref.weights(q, left, counts, lse, group=[-1, -1, 0, 0])
            for b, n in enumerate(left.lens_l):
                target = sc0[b, :, :n].cpu().double() + own[b]
                within("w", sc[b, :, :n], target, wtol[b] + target.abs() * 2.0 ** -22)
                assert torch.equal(sc[b, :, n:], sc0[b, :, n:])
    st = status()
    out, lse = C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, kc.lens, cu_q, status=st,
                                            **{**group, "prefix_lens": i32([10 ** 6])})
    torch.cuda.synchronize()
    assert int(st) == C.DEV_BAD_CACHE
    want, wl, otol, ltol = ref.attention(q, kc, counts)
    within("out", out, want, otol)


def test_evict_keeps_rows_scores_and_positions_together():
    """Where a move's page is out of the pool nothing of it moves: the slot keeps its key, score
    and position."""
    kc = ref.Cache([64], page=16, extra_width=0, dtype=HF, poison=False)
    k0, v0, table = kc.k.clone(), kc.v.clone(), kc.table.clone()
    table[0, 3] = 1000  # sources 48 .. 63
    sc = torch.arange(64, dtype=torch.float32, device="cuda").view(1, 1, 64)
    kp = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 1, 64)
    for in_place in (True, False):
        s, p, lens, st = sc.clone(), kp.clone(), i32([64]), status()
        kc.k.copy_(k0), kc.v.copy_(v0)
        kw = {} if in_place else dict(scores_out=torch.full_like(sc, -1.0), key_pos_out=torch.full_like(kp, -1))
        _, so, po = C.attention_varlen_cache_evict(kc.k, kc.v, table, lens, s, p, i32([64]), 20, 0, status=st, **kw)
        torch.cuda.synchronize()
        assert int(st) == C.DEV_BAD_CACHE and lens.tolist() == [20]
        # kept: scores 44 .. 63; the movers 44 .. 47 go into the first evicted slots, 0 .. 3
        want = [44, 45, 46, 47] + list(range(4, 20))
        assert po[0, 0, :20].tolist() == want and so[0, 0, :20].tolist() == [float(x) for x in want]
        t = kc.table[0].tolist()
        for slot, src in enumerate(want):
            for x, x0 in ((kc.k, k0), (kc.v, v0)):
                assert torch.equal(x[t[slot // 16], slot % 16], x0[t[src // 16], src % 16]), (slot, src)


# ---------------------------------------------------------------- arguments

def test_read_only_arrays_may_be_expanded():
    """One page table for several readers of the same keys, one row of q for several tokens."""
    kc = ref.Cache([100], [40], page=16, Hkv=2, d=128)
    B = 3
    q = normal(1, 1, 8, 128).expand(B, 8, 128)
    cu_q, lens, plens = i32([0, 1, 2, 3]), i32([100, 7, 64]), i32([40, 33])
    one = dict(prefix_table=kc.ptable.expand(2, -1), prefix_lens=plens, cu_prefix=i32([0, 1, 3]))
    each = dict(one, prefix_table=kc.ptable.repeat(2, 1))
    st = status()
    a, la = C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table.expand(B, -1), lens, cu_q, status=st, **one)
    b, lb = C.attention_varlen_cache_fwd(q.contiguous(), kc.k, kc.v, kc.table.repeat(B, 1), lens, cu_q, status=st, **each)
    assert torch.equal(a, b) and torch.equal(la, lb)
    w, _ = C.attention_varlen_cache_weights(q, kc.k, kc.table.expand(B, -1), lens, cu_q, la, status=st, **one)
    x, _ = C.attention_varlen_cache_weights(q.contiguous(), kc.k, kc.table.repeat(B, 1), lens, cu_q, la, status=st, **each)
    assert torch.equal(w, x)
    k = normal(2, 3, 1, 128).expand(3, 2, 128)  # one K row for both heads
    inv = torch.ones(64, dtype=torch.float64, device="cuda")
    u = C.attention_varlen_rotary(q, k, i32([1, 2, 3]), inv)
    v = C.attention_varlen_rotary(q.contiguous(), k.contiguous(), i32([1, 2, 3]), inv)
    assert torch.equal(u[0], v[0]) and torch.equal(u[1], v[1])
    big = ref.Cache([20, 20, 20], page=16, Hkv=2, d=128, poison=False)
    k0 = big.k.clone()
    C.attention_varlen_cache_append(k, k, big.k, big.v, big.table, i32([3, 4, 5]), cu_q, status=st)
    for b in range(B):
        pg = int(big.table[b, 0])
        assert torch.equal(big.k[pg, 3 + b], k[b]) and torch.equal(big.v[pg, 3 + b], k[b])
        k0[pg, 3 + b] = k[b]
    assert torch.equal(big.k, k0) and int(st) == 0
    with pytest.raises(C.AttnError):  # one page written by several sequences
        C.attention_varlen_cache_append(k, k, big.k, big.v, big.table[:1].expand(3, -1), i32([3, 4, 5]), cu_q)


def test_an_option_without_a_truth_value_is_refused():
    class Neither:
        def __bool__(self):
            raise KeyError("neither")

    kc = ref.Cache([20, 9], page=16, Hkv=2, d=128)
    q, cu_q = normal(1, 2, 8, 128), i32([0, 1, 2])
    out = torch.full_like(q, 5.0)
    with pytest.raises(KeyError, match="neither"):
        C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, kc.lens, cu_q, out=out, causal=Neither())
    with pytest.raises(KeyError, match="neither"):
        C.attention_varlen_rotary(q, None, i32([0, 1]), torch.ones(4, dtype=torch.float64, device="cuda"),
                                  inverse=Neither(), q_out=out)
    torch.cuda.synchronize()
    assert (out == 5).all()


# ---------------------------------------------------------------- the documented step

def documented_steps():
    """The lines of code of a generation step in the module's docstring and in the readme."""
    import os
    import re

    from conftest import ROOT

    doc = re.search(r"One generation step(?:.|\n)*?:\n\n((?:    .*\n)+)\n", C.__doc__).group(1)
    block = next(x for x in re.findall(r"```python\n(.*?)```", open(os.path.join(ROOT, "README.md")).read(), re.S)
                 if "cache_evict" in x)
    return re.sub(r"(?m)^    ", "", doc), block


@pytest.mark.parametrize("which", [0, 1], ids=["docstring", "readme"])
def test_the_documented_step(which):
    """Steps as the documents write them, over evictions: every new token's key has its position
    and its weight, and attention is that over the keys that are left."""
    code = documented_steps()[which]
    B, Hq, d, page, width, budget = 2, 8, 64, 16, 4, 20
    kc = ref.Cache([width * page] * B, (), 1, d, page, HF, extra_width=0)
    lens, cu_q = i32([0, 0]), i32([0, 1, 2])
    key_pos = torch.full((B, 1, width * page), -1, dtype=torch.int32, device="cuda")
    scores = torch.full((B, 1, width * page), math.nan, device="cuda")
    inv_freq = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).cuda()
    slopes = torch.zeros(B, Hq, device="cuda")
    for t in range(30):
        q, k, v = (normal(3 * t + i, B, h, d, dtype=HF, std=2.0) for i, h in ((0, Hq), (1, 1), (2, 1)))
        new = torch.zeros_like(lens)
        before = {}

        def evict(*a, **kw):  # what stood before the eviction
            before.update(key_pos=key_pos.clone(), scores=scores.clone(), lens=new.tolist(), k=kc.k.clone(), v=kc.v.clone())
            return C.attention_varlen_cache_evict(*a, **kw)

        space = {x: getattr(C, x) for x in dir(C) if x.startswith("attention_varlen")}
        space.update(q=q, k=k, v=v, k_cache=kc.k, v_cache=kc.v, table=kc.table, lens=lens, new_lens=new, lens1=new, cu_q=cu_q,
                     positions=i32([t] * B), inv_freq=inv_freq, key_pos=key_pos, scores=scores, slopes=slopes,
                     next_pos=i32([t + 1] * B), budget=budget, attention_varlen_cache_evict=evict)
        fake = type("module", (), {x: staticmethod(f) for x, f in space.items() if x.startswith("attention_varlen")})
        exec(code.replace("from ragged_gqa_attention_varlen_gb300 import cache as C\n", ""), {**space, "C": fake}, space)
        n = min(t, budget) + 1
        assert before["lens"] == [n, n] and new.tolist() == [min(t + 1, budget)] * B
        kc.lens_l = [n, n]
        after = kc.k.clone(), kc.v.clone()
        kc.k.copy_(before["k"]), kc.v.copy_(before["v"])
        want, wl, tol, ltol = ref.attention(space["q"], kc, [1, 1], causal=True, q_pos=torch.tensor([t, t]),
                                            key_pos=before["key_pos"])
        kc.k.copy_(after[0]), kc.v.copy_(after[1])
        within("out", space["out"], want, tol)
        for b in range(B):
            assert t in key_pos[b, 0, :new.tolist()[b]].tolist() or n > budget
            assert t in before["key_pos"][b, 0, :n].tolist()
            # each of the 8 rows has spread a weight of 1 over the keys in every step so far, and what
            # an evicted key had is gone with it: no more than 8 (t + 1), and finite
            total = float(before["scores"][b, 0, :n].double().sum())
            assert 8 * (1 - 2 ** -10) <= total <= 8 * (t + 1) * (1 + 2 ** -10)
        lens = new


# ---------------------------------------------------------------- rows far from their keys

@pytest.mark.parametrize("cap", [0.0, 3.0, 30.0])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("far", [1000, 1 << 20, (1 << 24) + 1, (1 << 30) - 700])
def test_alibi_of_rows_far_from_their_keys(far, dtype, cap):
    """ALiBi's weights depend on how the keys' distances differ: a row at any distance behind its
    keys gives what it gives next to them, and lse is less by slope times the way between."""
    lens, counts, Hq = [300, 40, 5000], [1, 20, 2], 16
    kc = ref.Cache(lens, [260], d=160, page=64, dtype=dtype)
    q = normal(2, sum(counts), Hq, 160, dtype=dtype)
    g = torch.Generator().manual_seed(4)
    slopes = torch.rand(3, Hq, generator=g) + 0.01
    slopes[:, ::4] = 0.0
    group = [0, -1, -1]
    end = [260 + 300, 40, 5000]
    near = [end[b] + i for b, n in enumerate(counts) for i in range(n)]
    call = dict(softcap=cap, alibi_slopes=slopes.cuda(), prefix_table=kc.ptable, prefix_lens=kc.plens,
                cu_prefix=i32([0, 1]), causal=True)
    want, wl, otol, ltol = ref.attention(q, kc, counts, group=group, slopes=slopes, causal=True, cap=cap,
                                         q_pos=torch.tensor(near))
    st = status()
    out, lse = C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, kc.lens, i32(ref.cu(counts)), status=st,
                                            q_pos=i32([x + far for x in near]), **call)
    torch.cuda.synchronize()
    assert int(st) == 0
    less = far * torch.repeat_interleave(slopes.double(), torch.tensor(counts), 0)
    within("lse", lse, wl - less, ltol + less * 2.0 ** -22)
    flat = slopes[0] == 0  # without ALiBi every row is what it was
    within("out", out[:, flat.cuda()], want[:, flat], otol[:, flat])
    within("out", out[1:], want[1:], otol[1:])
    # the first sequence's prefix and own keys are weighed against one another by two terms, each off by
    # half a step: 2^-24 of twice its size
    within("out", out[:1], want[:1], otol[:1] + torch.expm1((4 * less[:1, :, None] * 2.0 ** -24).clamp(max=20)) * 4)
