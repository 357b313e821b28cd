"""The cache held in 8 bits on the GPU: the append that quantises and attention over it,
against plain 64-bit forms (cache8_ref)."""
import math

import pytest
import torch

import cache8_ref as ref8
import cache_ref as ref
from ragged_gqa_attention_varlen_gb300 import cache as C
from test_cache_gpu import BF, CASES, HF, case, i32, lib, normal, status, within  # noqa: F401

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------- attention

# calls whose sequences have few rows a K/V head, which have a kernel of their own: many
# pieces for each CTA, stages that wrap, rows of several tokens, tiles that 8 rows cut
FEW = [
    case("few_many_pieces", ref.spread(21, 60, 1, 1500), [1] * 60, Hq=32, Hkv=8, d=128, page=64, cap=0.0),
    case("few_long", [20000, 9000, 1], [1, 1, 1], Hq=8, Hkv=2, d=128, page=16, cap=0.0, alibi=True, dtype=HF),
    case("few_wide_head", ref.spread(22, 20, 1, 900), [1] * 20, Hq=10, Hkv=5, d=160, page=32, alibi=True),
    case("few_wide_head_small_pages", [4000, 33, 64, 65], [1] * 4, Hq=8, Hkv=8, d=160, page=16, cap=30.0, dtype=HF),
    case("few_narrow_head", ref.spread(23, 70, 1, 700), [1] * 70, Hq=5, Hkv=5, d=64, page=128, cap=0.0, wl=100),
    case("few_tokens", [300, 20, 513, 64], [2, 3, 1, 1], Hq=6, Hkv=3, d=128, page=64, alibi=True, dtype=HF),
    case("few_but_one_prompt", [300] + [40] * 30, [60] + [1] * 30, Hq=4, Hkv=2, d=64, page=16, cap=3.0),
    case("few_uncausal_window", [700, 31], [2, 2], Hq=4, Hkv=2, d=128, page=16, causal=False, wl=90, wr=0, cap=0.0),
    case("few_shuffled", [400, 33], [1, 2], Hq=4, Hkv=2, d=160, page=64, alibi=True, shuffled=True, cap=0.0),
    case("few_without_keys", [0, 5, 0], [1, 0, 2], Hq=4, Hkv=2, d=64, cap=0.0),
    case("few_peaked", [600, 100], [1, 1], Hq=8, Hkv=4, d=128, cap=0.0, std=12.0, dtype=HF),
    case("few_in_two_tiles", ref.spread(24, 30, 1, 1200), [1] * 30, Hq=32, Hkv=2, d=128, page=64, cap=0.0),
    case("few_in_tiles_of_eight_and_four", [900, 65, 1, 31], [1] * 4, Hq=24, Hkv=2, d=160, page=32, alibi=True, dtype=HF),
    case("few_strided", [200, 31], [1, 2], Hq=6, Hkv=2, d=160, page=32, strided=True),
]


def odd_scales(top, g):
    """Scales that are no powers of two, four times apart, some larger than needed."""
    return top.clamp(min=1e-3) / 448 * (1 + 3 * torch.rand(top.shape, generator=g))


def steep_scales(top, g):
    """Scales that lie up to 2^40 apart: V's reference has to move, small blocks vanish."""
    return ref8.pow2_scale(top) * torch.exp2(torch.randint(-20, 21, top.shape, generator=g).double())


def build(c, block, seed=1, scales=None, std=None):
    kc = ref8.Cache8(c["lens"], c["plens"], c["Hkv"], c["d"], c["page"], block, seed, c["strided"], scales)
    T, std = sum(c["counts"]), std or c["std"]
    q = normal(seed, T, c["Hq"] + 1, c["d"] + 16, dtype=c["dtype"], std=std)[:, :c["Hq"], :c["d"]] if c["strided"] else \
        normal(seed, T, c["Hq"], c["d"], dtype=c["dtype"], std=std)
    opt = dict(causal=c["causal"], wl=c["wl"], wr=c["wr"], cap=c["cap"], mult=0.75, group=c["group"])
    call = dict(causal=c["causal"], window_left=c["wl"], window_right=c["wr"], softcap=c["cap"])
    B, P = len(c["lens"]), len(c["plens"])
    if c["alibi"]:
        opt["slopes"] = torch.rand(B, c["Hq"], generator=torch.Generator().manual_seed(seed + 1)) * 0.1
        call["alibi_slopes"] = opt["slopes"].cuda()
    if P:
        first = [next((b for b, g in enumerate(c["group"]) if g == p), 0) for p in range(P)]
        members = [sum(g == p for g in c["group"]) for p in range(P)]
        call.update(prefix_table=kc.ptable, prefix_lens=kc.plens, cu_prefix=i32(first + [first[-1] + members[-1]]))
    if c["shuffled"]:
        g = torch.Generator().manual_seed(seed + 2)

        def positions(table, lens, base):
            kp = torch.full((len(lens), c["Hkv"], table.shape[1] * c["page"] + 3), 1 << 29, dtype=torch.int32)
            for b, n in enumerate(lens):
                for h in range(c["Hkv"]):
                    kp[b, h, :n] = base + torch.randperm(2 * n + 1, generator=g)[:n].int()
            return kp.cuda()

        base = max(c["plens"], default=0) * 2 + 1
        opt["key_pos"] = call["key_pos"] = positions(kc.table, c["lens"], base)
        if P:
            opt["pkey_pos"] = call["prefix_key_pos"] = positions(kc.ptable, c["plens"], 0)
        opt["q_pos"] = call["q_pos"] = i32([base + 2 * c["lens"][b] - n + i for b, n in enumerate(c["counts"]) for i in range(n)])
    return kc, q, i32(ref.cu(c["counts"])), opt, call


def attend(q, kc, cu_q, call, **more):
    return C.attention_varlen_cache8_fwd(q, kc.k8, kc.v8, kc.k_scale, kc.v_scale, kc.table, kc.lens, cu_q, **call, **more)


@pytest.mark.parametrize("c", CASES + FEW)
def test_attention(c):
    block = min(c["page"], (16, 32, 64, 128)[len(c["lens"]) % 4])
    kc, q, cu_q, opt, call = build(c, block)
    st = status()
    want, lse, out_tol, lse_tol = ref8.attention(q, kc, c["counts"], **opt)
    out = torch.full((len(q), c["Hq"] + 1, c["d"] + 8), 7.0, dtype=q.dtype, device="cuda")
    got, got_lse = attend(q, kc, cu_q, call, status=st, out=out[:, :c["Hq"], :c["d"]])
    torch.cuda.synchronize()
    assert int(st) == 0
    within("lse", got_lse, lse, lse_tol)
    within("out", got, want, out_tol)
    assert (out[:, c["Hq"]:] == 7).all() and (out[:, :, c["d"]:] == 7).all()
    again, lse2 = attend(q, kc, cu_q, call)
    assert torch.equal(again, got) and torch.equal(lse2, got_lse)


PICKED = [x for x in CASES if x.id in ("wide_group", "long_split", "three_groups", "drafts", "window_both", "prefixes_some_without",
                                       "shuffled_prefix", "odd_heads", "prompt", "peaked_fp16", "saturated_fp16")] + FEW


@pytest.mark.parametrize("scales", [odd_scales, steep_scales])
@pytest.mark.parametrize("c", PICKED)
def test_attention_of_any_scales(c, scales):
    """Scales of another quantiser: no powers of two, and far apart."""
    kc, q, cu_q, opt, call = build(c, 16, seed=9, scales=scales, std=0.05 if scales is steep_scales else None)
    st = status()
    want, lse, out_tol, lse_tol = ref8.attention(q, kc, c["counts"], **opt)
    got, got_lse = attend(q, kc, cu_q, call, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    within("lse", got_lse, lse, lse_tol)
    within("out", got, want, out_tol)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128, 160])
def test_rows_of_q_far_apart(d, dtype):
    """Rows and elements of q that lie many binades apart, rows of zeros: each row has
    its own factor, and lse keeps fp32's accuracy."""
    kc = ref8.Cache8([300, 40], Hkv=1, d=d, page=32, block=32)
    g = torch.Generator().manual_seed(4)
    q = torch.randn(2, 40, d, generator=g) * torch.exp2(torch.randint(-12, 5, (2, 40, d), generator=g).float())
    q[:, ::3] *= 2.0 ** -8
    q[0, 5] = 0
    q[1, 7, 1:] = 0
    q = q.to(dtype).cuda()
    want, lse, tol, ltol = ref8.attention(q, kc, [1, 1], cap=0.0)
    got, got_lse = C.attention_varlen_cache8_fwd(q, kc.k8, kc.v8, kc.k_scale, kc.v_scale, kc.table, kc.lens, i32([0, 1, 2]), softcap=0.0)
    within("lse", got_lse, lse, ltol)
    within("out", got, want, tol)


def test_blocks_of_zeros_and_huge_pools():
    """Blocks with a scale of 0 are zero keys and values, and pages may lie beyond 2^32 bytes."""
    kc = ref8.Cache8([200], Hkv=2, d=128, page=64, block=16, scales=lambda top, g: torch.where(
        torch.rand(top.shape, generator=g) < 0.5, 0.0, ref8.pow2_scale(top)))
    q = normal(2, 1, 8, 128, dtype=HF)
    want, lse, tol, ltol = ref8.attention(q, kc, [1], cap=0.0)
    got, got_lse = C.attention_varlen_cache8_fwd(q, kc.k8, kc.v8, kc.k_scale, kc.v_scale, kc.table, kc.lens, i32([0, 1]), softcap=0.0)
    within("lse", got_lse, lse, ltol)
    within("out", got, want, tol)
    # the same pages at the end of a pool of 5 GB
    far = (5 << 30) // (64 * 2 * 128)
    n = kc.k8.shape[0]
    pools = []
    for x, s in ((kc.k8, kc.k_scale), (kc.v8, kc.v_scale)):
        big = torch.empty(far + n, 64, 2, 128, dtype=torch.uint8, device="cuda")
        big[far:] = x.view(torch.uint8)
        scale = torch.full((far + n, 4, 2), math.nan, device="cuda")
        scale[far:] = s
        pools.append((big.view(F8), scale))
    got2, lse2 = C.attention_varlen_cache8_fwd(q, pools[0][0], pools[1][0], pools[0][1], pools[1][1], (kc.table + far).int(), kc.lens,
                                               i32([0, 1]), softcap=0.0)
    assert torch.equal(got, got2) and torch.equal(got_lse, lse2)


def test_padded_batch_leaves_rows_behind_the_last_sequence():
    kc = ref8.Cache8([40, 20, 0, 0], page=16, Hkv=1)
    q = normal(3, 9, 8, 160)
    q[3:] = math.nan
    out, lse, st = torch.full_like(q, 5.0), torch.full((9, 8), 5.0, device="cuda"), status()
    attend(q, kc, i32([0, 1, 3, 3, 3]), dict(causal=True), out=out, lse=lse, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0 and (out[3:] == 5).all() and (lse[3:] == 5).all()
    want, wlse, tol, ltol = ref8.attention(q[:3], kc, [1, 2, 0, 0], causal=True)
    within("out", out[:3], want, tol)
    within("lse", lse[:3], wlse, ltol)


def test_pages_out_of_the_pool_count_for_nothing():
    """As if their slots were not there; bad lengths and cu arrays are reported and harmless."""
    kc = ref8.Cache8([100, 20], page=16, Hkv=1)
    q = normal(3, 2, 8, 160)
    table = kc.table.clone()
    table[0, 2], table[0, 4] = 10 ** 6, -3
    st = status()
    got, lse = C.attention_varlen_cache8_fwd(q, kc.k8, kc.v8, kc.k_scale, kc.v_scale, table, kc.lens, i32([0, 1, 2]), status=st)
    torch.cuda.synchronize()
    assert int(st) & C.DEV_BAD_CACHE
    keep = [j for j in range(100) if j // 16 not in (2, 4)]
    k, v = (kc.rows(x, kc.table, 0, 100)[keep] for x in (kc.k, kc.v))
    z = 3 * torch.tanh(torch.einsum("hf,jf->hj", q[0].cpu().double(), k[:, 0]) * 0.75 / math.sqrt(160) / 3)
    assert float((torch.logsumexp(z, -1) - lse[0].cpu().double()).abs().max()) < 1e-4
    assert float((torch.softmax(z, -1) @ v[:, 0] - got[0].cpu().double()).abs().max()) < 0.02
    for lens, cu_q, bit in (([10 ** 6, 5], [0, 1, 2], C.DEV_BAD_CACHE), ([-1, 5], [0, 1, 2], C.DEV_BAD_CACHE),
                            ([100, 20], [0, 2, 1], 1), ([100, 20], [0, 1, 900], 1)):
        st = status()
        C.attention_varlen_cache8_fwd(q, kc.k8, kc.v8, kc.k_scale, kc.v_scale, kc.table, i32(lens), i32(cu_q), status=st)
        torch.cuda.synchronize()
        assert int(st) & bit


@pytest.mark.parametrize("Hq", [48, 6])
def test_captured_and_on_two_streams(Hq):
    kc = ref8.Cache8([700, 90], page=64, block=64, Hkv=1)
    q = normal(3, 2, Hq, 160)
    cu_q = i32([0, 1, 2])
    want = attend(q, kc, cu_q, dict(causal=True))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a, b = attend(q, kc, cu_q, dict(causal=True), stream=s1), attend(q, kc, cu_q, dict(causal=True), stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for r in (a, b) for x, y in zip(r, want))
    out, lse, ws = torch.empty_like(q), torch.empty(2, Hq, device="cuda"), torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attend(q, kc, cu_q, dict(causal=True), out=out, lse=lse, workspace=ws)
    for _ in range(2):
        out.zero_()
        g.replay()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_the_same_call_many_times():
    """One answer, whatever the order in which the CTAs' loads land."""
    kc = ref8.Cache8(ref.spread(31, 90, 100, 1500), Hkv=4, d=128, page=64, block=32)
    q, cu_q = normal(3, 90, 8, 128), i32(range(91))
    want = attend(q, kc, cu_q, dict(causal=True, softcap=0.0))
    for _ in range(300):
        got = attend(q, kc, cu_q, dict(causal=True, softcap=0.0))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---------------------------------------------------------------- append

APPENDS = [pytest.param(*x, id=f"{len(x[0])}_sequences-{x[2]}x{x[3]}-page{x[4]}-block{x[5]}-{x[6]}-{x[7]}_pairs") for x in [
    # new, held, Hkv, d, page, block, dtype, pairs (0: no turn), interleaved, norm
    ([1], [0], 1, 160, 16, 16, "bf16", 80, False, False), ([1, 1, 1, 1], [15, 16, 17, 500], 8, 128, 64, 32, "bf16", 64, False, True),
    ([0, 3, 0, 1], [5, 0, 9, 31], 3, 64, 32, 16, "fp16", 0, False, True), ([300, 1, 47], [7, 130, 0], 1, 160, 128, 128, "fp16", 80, True, False),
    ([129, 200], [127, 1], 2, 128, 128, 64, "bf16", 48, True, True), ([70, 65, 64], [1, 63, 64], 5, 64, 64, 64, "fp16", 31, False, True),
    ([1000], [3], 1, 128, 1024, 128, "bf16", 63, True, False), ([33] * 40, list(range(40)), 1, 160, 16, 16, "bf16", 7, False, True),
    ([2] * 300, list(range(0, 600, 2)), 1, 64, 16, 16, "fp16", 32, True, False)]]


def append_case(new, held, Hkv, d, page, block, dtype, pairs, seed=3):
    dt = BF if dtype == "bf16" else HF
    kc = ref8.Cache8([a + b for a, b in zip(new, held)], Hkv=Hkv, d=d, page=page, block=block, seed=seed)
    T = sum(new)
    k, v = normal(seed, T, Hkv + 1, d + 8, dtype=dt, std=2.0)[:, :Hkv, :d], normal(seed + 1, T, Hkv, d, dtype=dt)
    g = torch.Generator().manual_seed(seed + 2)
    # tokens of very different sizes: some grow their block's scale, some do not; a few are zeros
    size = torch.exp2(torch.randint(-9, 6, (T, 1, 1), generator=g).float()).to(dt).cuda()
    k, v = k * size, v * size.flip(0)
    if T > 2:
        v[1] = 0
    pos = torch.randint(0, 1 << 20, (2, max(T, 1)), generator=g, dtype=torch.int32)[:, :T].contiguous().cuda()
    inv = axis = None
    if pairs:
        inv = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).cuda()
        axis = torch.randint(0, 2, (pairs,), generator=g, dtype=torch.int32).cuda()
    return kc, k, v, pos, inv, axis, g


@pytest.mark.parametrize("new,held,Hkv,d,page,block,dtype,pairs,interleaved,norm", APPENDS)
def test_append(new, held, Hkv, d, page, block, dtype, pairs, interleaved, norm):
    kc, k, v, pos, inv, axis, g = append_case(new, held, Hkv, d, page, block, dtype, pairs)
    w = (torch.rand(d, generator=g) + 0.5).cuda() if norm else None
    lens, cu, st, lens_out = i32(held), i32(ref.cu(new)), status(), torch.zeros(len(new), dtype=torch.int32, device="cuda")
    before = {n: (getattr(kc, n + "8").view(torch.uint8).clone(), getattr(kc, n + "_scale").clone()) for n in "kv"}
    key_pos = torch.full((len(new), Hkv, kc.table.shape[1] * page), -5, dtype=torch.int32, device="cuda")
    C.attention_varlen_cache8_append(k, v, kc.k8, kc.v8, kc.k_scale, kc.v_scale, kc.table, lens, cu, positions=pos, inv_freq=inv,
                                     pair_axis=axis, interleaved=interleaved, k_weight=w, key_pos=key_pos, lens_out=lens_out, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0 and lens_out.tolist() == [a + b for a, b in zip(new, held)]
    kd, mag = k.cpu().double(), None
    if norm:
        kd, _ = ref8.normed(k, w, 1e-6)
    kd, mag = ref8.turned(kd, pos, inv, axis, interleaved)
    table, at = kc.table.cpu(), ref.cu(new)
    for name, x, m in (("k", kd, mag), ("v", v.cpu().double(), v.cpu().double().abs())):
        bits, scales = getattr(kc, name + "8").view(torch.uint8).cpu(), getattr(kc, name + "_scale").cpu()
        got = bits.view(F8).float()
        old_bits, old_scale = (y.cpu() for y in before[name])
        old = old_bits.view(F8).float()
        touched = torch.zeros(bits.shape[:2], dtype=torch.bool)
        # fp32 arithmetic: the norm, sine and cosine are off by a few steps of 2^-20; V is exact
        slack = 2.0 ** -19 if name == "k" and (norm or inv is not None) else 0.0
        for b, n in enumerate(new):
            for first in range(held[b] // block * block, held[b] + n, block):
                lo, hi = max(held[b], first), min(held[b] + n, first + block)
                if lo >= hi:
                    continue
                page_at, s0 = int(table[b, first // page]), first % page
                rows, mr = x[at[b] + lo - held[b]:at[b] + hi - held[b]], m[at[b] + lo - held[b]:at[b] + hi - held[b]]
                top, off = rows.abs().amax((0, 2)), mr.amax((0, 2)) * slack
                was = old_scale[page_at, s0 // block].double() if held[b] > first else torch.zeros(Hkv, dtype=torch.float64)
                now = scales[page_at, s0 // block].double()
                lowest = torch.where(top - off <= 448 * was, was, ref8.pow2_scale((top - off).clamp(min=0)))
                highest = torch.where(top + off <= 448 * was, was, ref8.pow2_scale(top + off))
                assert ((now == lowest) | (now == highest)).all(), (name, b, first)
                q = got[page_at, s0 + lo - first:s0 + hi - first].double()
                want = rows / now.clamp(min=2.0 ** -140)[:, None]
                step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
                assert ((q - want).abs() <= step / 2 + mr / now.clamp(min=2.0 ** -140)[:, None] * slack + step * 2.0 ** -20).all(), (name, b, first)
                if slack == 0.0:
                    assert torch.equal(q, ref8.e4m3(want)), (name, b, first)
                if held[b] > first:
                    kept = ref8.e4m3(old[page_at, s0:s0 + lo - first].double() * (was / now.clamp(min=2.0 ** -140))[:, None])
                    assert torch.equal(got[page_at, s0:s0 + lo - first].double(), kept), (name, b, first)
                touched[page_at, s0:s0 + hi - first] = True
        assert torch.equal(bits[~touched], old_bits[~touched])
    for b, n in enumerate(new):
        for h in range(Hkv):
            row = key_pos[b, h].cpu()
            assert torch.equal(row[held[b]:held[b] + n], pos[0, at[b]:at[b + 1]].cpu())
            assert (row[:held[b]] == -5).all() and (row[held[b] + n:] == -5).all()


def test_append_keeps_what_it_may_not_touch():
    """Sequences that do not fit, pages out of the pool, padded batches, inconsistent cu_new."""
    def state():
        kc = ref8.Cache8([20, 40, 33], Hkv=2, d=64, page=16, block=16, seed=5)
        return kc, [x.clone() for x in (kc.k8.view(torch.uint8), kc.v8.view(torch.uint8), kc.k_scale, kc.v_scale)]

    def same(kc, old, rows=None):
        for x, y in zip((kc.k8.view(torch.uint8), kc.v8.view(torch.uint8), kc.k_scale, kc.v_scale), old):
            a, b = (x, y) if rows is None else (x[rows], y[rows])
            assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))

    k, v = normal(1, 6, 2, 64), normal(2, 6, 2, 64)
    kc, old = state()
    st, lens_out = status(), i32([9, 9, 9])
    C.attention_varlen_cache8_append(k, v, kc.k8, kc.v8, kc.k_scale, kc.v_scale, kc.table, i32([18, 38, 31]), i32([0, 2, 1, 6]), status=st, lens_out=lens_out)
    torch.cuda.synchronize()
    assert int(st) & 1 and lens_out.tolist() == [18, 38, 31]
    same(kc, old)
    # the first does not fit its table, the third has a negative length; rows behind cu_new[B] are left out
    kc, old = state()
    st = status()
    k[5] = v[5] = math.nan
    full = kc.table.shape[1] * 16
    C.attention_varlen_cache8_append(k, v, kc.k8, kc.v8, kc.k_scale, kc.v_scale, kc.table, i32([full - 1, 38, -1]), i32([0, 2, 4, 5]), status=st, lens_out=lens_out)
    torch.cuda.synchronize()
    assert int(st) & C.DEV_BAD_CACHE and lens_out.tolist() == [full - 1, 40, -1]
    mine = int(kc.table[1, 2])
    others = [p for p in range(kc.num_pages) if p != mine]
    same(kc, old, others)
    assert torch.isfinite(kc.k8[mine, 6:8].float()).all()
    # a page out of the pool
    kc, old = state()
    st, table = status(), kc.table.clone()
    table[1, 2] = 10 ** 7
    C.attention_varlen_cache8_append(k, v, kc.k8, kc.v8, kc.k_scale, kc.v_scale, table, i32([18, 38, 31]), i32([0, 0, 2, 2]), status=st)
    torch.cuda.synchronize()
    assert int(st) & C.DEV_BAD_CACHE
    same(kc, old)


def test_append_at_the_ends_of_the_range():
    """Tiny and huge values, zeros: scales stay powers of two in [2^-126, 2^120] or 0."""
    kc = ref8.Cache8([4] * 5, Hkv=1, d=64, page=16, block=16)
    k = torch.zeros(5, 1, 64)
    k[0, 0, 3], k[1, 0, 0], k[2], k[3, 0, 9] = 1e-39, 3.3e38, 0.0, 448.0
    k[4, 0, 1] = 448.0 * 1.0078125
    k = k.to(BF).cuda()
    C.attention_varlen_cache8_append(k, k, kc.k8, kc.v8, kc.k_scale, kc.v_scale, kc.table, i32([0] * 5), i32(range(6)))
    for s, x in ((kc.k_scale, kc.k8), (kc.v_scale, kc.v8)):
        got = [float(s[int(kc.table[b, 0]), 0, 0]) for b in range(5)]
        assert got == [2.0 ** -126, 2.0 ** 120, 0.0, 1.0, 2.0], got
        assert float(x[int(kc.table[3, 0]), 0, 0, 9].float()) == 448.0


# ---------------------------------------------------------------- together

def test_steps_of_generation():
    """Norm and turn q, append (normed, turned, quantised) and attend, token by token behind a
    prompt: against the 64-bit attention over the values that the cache holds."""
    B, Hq, Hkv, d, page, block = 3, 12, 3, 128, 32, 16
    g = torch.Generator().manual_seed(8)
    kc = ref8.Cache8([60] * B, Hkv=Hkv, d=d, page=page, block=block)
    qw, kw = (torch.rand(d, generator=g) + 0.5).cuda(), (torch.rand(d, generator=g) + 0.5).cuda()
    inv = (10000.0 ** (-torch.arange(48, dtype=torch.float64) / 48)).cuda()
    lens, st = i32([0] * B), status()
    for step, counts in enumerate(([40, 17, 31], [1, 1, 1], [1, 3, 1], [2, 1, 1])):
        T = sum(counts)
        q, k, v = (normal(step * 3 + i, T, h, d, dtype=BF, std=2.0) for i, h in enumerate((Hq, Hkv, Hkv)))
        cu, new = i32(ref.cu(counts)), torch.zeros_like(lens)
        pos = i32([int(n) + i for n, c in zip(lens.tolist(), counts) for i in range(c)])
        qn, kn = C.attention_varlen_norm_rotary(q, k, qw, kw, pos, inv)
        C.attention_varlen_cache8_append(k, v, kc.k8, kc.v8, kc.k_scale, kc.v_scale, kc.table, lens, cu, positions=pos, inv_freq=inv,
                                         k_weight=kw, lens_out=new, status=st)
        out, lse = C.attention_varlen_cache8_fwd(qn, kc.k8, kc.v8, kc.k_scale, kc.v_scale, kc.table, new, cu, causal=True, status=st)
        torch.cuda.synchronize()
        assert int(st) == 0
        lens = new
        kc.lens_l = lens.tolist()
        kc.k, kc.v = kc._values(kc.k8, kc.k_scale), kc._values(kc.v8, kc.v_scale)
        want, wlse, tol, ltol = ref8.attention(qn, kc, counts, causal=True)
        within("out", out, want, tol)
        within("lse", lse, wlse, ltol)
        # the cache holds what the norm's own call gives, to e4m3's half step and the block's smallest step
        at = ref.cu(counts)
        for b, c in enumerate(counts):
            held = kc.rows(kc.k, kc.table, b, kc.lens_l[b])[-c:]
            mine = kn[at[b]:at[b + 1]].cpu().double()
            scale = max(float(s) for s in kc.k_scale[kc.table[b, :2].long()].nan_to_num(0).flatten())
            assert ((held - mine).abs() <= mine.abs() * (2.0 ** -4 + 2.0 ** -7) + scale * 2.0 ** -9).all()


def test_a_captured_step_is_the_step():
    """Norm, fork, append and attend in a graph, replayed: the same bits as the calls one by one,
    with lengths and tables that move on the device."""
    R, Hq, Hkv, d, page, block, N = 6, 8, 2, 64, 16, 16, 40
    inv = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).cuda()
    q, k, v = (normal(50 + i, R, h, d, dtype=BF, std=2.0) for i, h in enumerate((Hq, Hkv, Hkv)))
    cu, parents, room, pos = i32(range(R + 1)), i32([0, 0, 2, 2, 5, 4]), i32([1] * R), i32([9] * R)
    kw = torch.full((d,), 1.5, device="cuda")

    def state():
        pools = [torch.zeros(N, page, Hkv, d, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2)]
        pools += [torch.zeros(N, page // block, Hkv, device="cuda") for _ in range(2)]
        table, lens, held = torch.full((R, 5), -1, dtype=torch.int32, device="cuda"), i32([0] * R), i32([0] * R)
        return pools, table, lens, held, torch.zeros(N, dtype=torch.int32, device="cuda"), torch.zeros_like(lens), status(), \
            torch.empty_like(q), torch.empty(R, Hq, device="cuda")

    def step(pools, table, lens, held, refs, new, st, out, lse):
        C.attention_varlen_cache_fork(pools, table, lens, held, refs, parents, room, status=st)
        qn, _ = C.attention_varlen_norm_rotary(q, None, kw, None, pos, inv)
        C.attention_varlen_cache8_append(k, v, *pools, table, lens, cu, positions=pos, inv_freq=inv, k_weight=kw, lens_out=new,
                                         status=st)
        C.attention_varlen_cache8_fwd(qn, *pools, table, new, cu, causal=True, out=out, lse=lse, status=st)
        lens.copy_(new)

    one, two = state(), state()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(*two)
    for n in range(40):
        step(*one)
        g.replay()
        torch.cuda.synchronize()
        flat = lambda x: [t.view(torch.uint8) for t in (*x[0], *x[1:])]
        assert all(torch.equal(a, b) for a, b in zip(flat(one), flat(two))), n
    assert int(one[6]) == 0 and one[2].tolist() == [40] * R
