"""The generation calls on the GPU against plain 64-bit forms (cache_ref), with
tolerances derived there from the roundings of the types."""
import math

import pytest
import torch

import cache_ref as ref
from ragged_gqa_attention_varlen_gb300 import cache as C

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def lib():
    from ragged_gqa_attention_varlen_gb300 import _build

    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return C.load()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def normal(seed, *shape, dtype=BF, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).cuda()


def within(name, x, want, tol):
    x = x.detach().cpu().double()
    assert x.shape == want.shape, (name, x.shape, want.shape)
    fin = torch.isfinite(want)
    assert torch.equal(x[~fin], want[~fin]), f"{name}: infinite values differ"
    assert torch.isfinite(x[fin]).all(), f"{name}: not finite"
    over = ((x - want).abs() - tol)[fin]
    if over.numel():
        assert float(over.max()) <= 0, f"{name}: {int((over > 0).sum())} values off, worst by {float(over.max()):.3e}"


# ---------------------------------------------------------------- attention and key weights

def case(name, lens, counts, plens=(), group=None, Hq=16, Hkv=1, d=160, page=16, dtype=BF, cap=3.0,
         alibi=False, causal=True, wl=-1, wr=-1, shuffled=False, strided=False, std=2.0):
    return pytest.param(dict(lens=lens, counts=counts, plens=plens, group=group, Hq=Hq, Hkv=Hkv, d=d,
                             page=page, dtype=dtype, cap=cap, alibi=alibi, causal=causal, wl=wl, wr=wr,
                             shuffled=shuffled, strided=strided, std=std), id=name)


CASES = [
    case("one_token_one_key", [1], [1]),
    case("one_head", [5, 130], [1, 1], Hq=1),
    case("wide_group", [700], [1], Hq=96, page=64, alibi=True),
    case("lengths_around_a_tile", [127, 128, 129, 255, 256, 257, 1, 64], [1] * 8, Hq=8, page=16),
    case("no_keys_and_no_queries", [0, 33, 0, 17], [1, 0, 0, 2], Hq=4, page=32),
    case("long_split", [5000, 3], [1, 1], Hq=48, page=128, alibi=True),
    case("many_short", ref.spread(3, 200, 1, 60), [1] * 200, Hq=8, page=16, dtype=HF),
    case("odd_heads", [77, 300], [1, 3], Hq=5, Hkv=5, d=64, page=16, cap=0.0, dtype=HF),
    case("three_groups", [200, 90], [2, 1], Hq=12, Hkv=3, d=128, page=32, cap=30.0),
    case("grouped_fp16", ref.spread(4, 12, 3, 900), [1] * 12, Hq=32, Hkv=8, d=128, page=64, dtype=HF, cap=0.0),
    case("drafts", [300, 20, 513], [8, 3, 5], Hq=48, page=64, alibi=True, dtype=HF),
    case("prompt", [400, 129], [400, 129], Hq=16, Hkv=4, d=64, page=64, cap=0.0),
    case("prompt_uncausal", [150], [70], Hq=6, causal=False),
    case("window_left", [1000, 40], [1, 2], Hq=8, page=32, wl=37),
    case("window_both", [300], [60], Hq=8, causal=False, wl=20, wr=5, alibi=True),
    case("window_leaves_nothing", [12], [40], Hq=8, causal=True, wl=3),
    case("more_queries_than_keys", [5, 0], [9, 4], Hq=8, causal=True),
    case("prefix", [20, 300, 1, 64], [1] * 4, plens=[500], group=[0] * 4, Hq=48, page=64, alibi=True),
    case("prefix_many_rows", ref.spread(5, 30, 1, 200), [1, 2] * 15, plens=[777], group=[0] * 30, Hq=32, Hkv=8,
         d=128, page=16, cap=0.0),
    case("prefixes_some_without", [10, 20, 30, 40, 50], [1, 2, 1, 0, 3], plens=[100, 257], group=[-1, 0, 0, 1, -1],
         Hq=16, page=32, alibi=True, dtype=HF),
    case("prefix_empty", [9, 8], [1, 1], plens=[0], group=[0, 0], Hq=8),
    case("prefix_alone", [0, 0], [1, 2], plens=[200], group=[0, 0], Hq=8, causal=False),
    case("prefix_window", [30, 300, 6], [2, 1, 4], plens=[150], group=[0, 0, 0], Hq=8, wl=100),
    case("prefix_window_both", [30, 300, 6], [2, 1, 9], plens=[150], group=[0, 0, 0], Hq=8, wl=64, wr=3, causal=False),
    case("shuffled_alibi", [400, 33], [1, 2], Hq=16, page=64, alibi=True, shuffled=True),
    case("shuffled_heads_window", [130, 257], [3, 1], Hq=8, Hkv=4, d=64, page=16, cap=0.0, wl=90, shuffled=True,
         dtype=HF),
    case("shuffled_prefix", [50, 60], [1, 1], plens=[300], group=[0, 0], Hq=16, Hkv=2, d=128, page=32, alibi=True,
         shuffled=True),
    case("strided", [200, 31], [1, 2], plens=[70], group=[0, 0], Hq=16, Hkv=2, d=128, page=32, strided=True),
    case("strided_160", [200, 31], [1, 2], Hq=16, strided=True, dtype=HF),
    case("steep", [600], [2], Hq=8, alibi=True, cap=0.0, std=6.0),
    case("peaked_fp16", [600, 100], [2, 1], Hq=8, cap=0.0, std=12.0, dtype=HF),
    case("big_cap", [600], [2], Hq=8, cap=50.0, std=12.0),
    # logits at both ends of the cap, and rows that nothing of the nearest tile is left for
    case("saturated_fp16", [300, 260], [150, 200], Hq=8, dtype=HF, cap=9.0, std=30.0),
    case("saturated_small_cap_fp16", [300, 260], [150, 200], Hq=8, dtype=HF, cap=3.0, std=30.0, alibi=True),
    case("saturated_window_fp16", [700], [300], Hq=8, dtype=HF, cap=9.4, std=30.0, wl=200),
    case("saturated_uncausal", [700], [3], Hq=16, dtype=HF, cap=9.5, std=30.0, causal=False),
    case("huge_page", [2000, 1500], [1, 1], Hq=8, page=1024),
    case("heads_beyond_a_tile", [200], [3], Hq=200, page=16, alibi=True),
    case("more_sequences_than_threads", ref.spread(9, 700, 1, 30), [1] * 700, Hq=4, d=64, page=16, cap=0.0),
    case("many_prefixes", ref.spread(10, 60, 1, 40), [1, 0, 2] * 20, plens=ref.spread(11, 20, 1, 300),
         group=[b // 3 for b in range(60)], Hq=6, Hkv=2, d=64, page=32, cap=0.0, alibi=True),
    case("parts_beyond_a_warp", [20000], [1], Hq=8, d=64, page=256, cap=0.0),
    case("prompt_over_many_parts", [700, 2], [300, 2], Hq=12, Hkv=4, d=64, page=64, cap=30.0, alibi=True, dtype=HF),
    case("prompt_window_behind_prefix", [500, 90], [260, 90], plens=[150], group=[0, 0], Hq=8, Hkv=2, d=64, page=32,
         cap=0.0, wl=70),
]


def build(c, seed=1):
    kc = ref.Cache(c["lens"], c["plens"], c["Hkv"], c["d"], c["page"], c["dtype"], seed, c["strided"])
    T = sum(c["counts"])
    if c["strided"]:
        q = normal(seed, T, c["Hq"] + 1, c["d"] + 16, dtype=c["dtype"], std=c["std"])[:, :c["Hq"], :c["d"]]
    else:
        q = normal(seed, T, c["Hq"], c["d"], dtype=c["dtype"], std=c["std"])
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
        qp = []
        for b, n in enumerate(c["counts"]):
            qp += [base + 2 * c["lens"][b] - n + i for i in range(n)]
        opt["q_pos"] = call["q_pos"] = i32(qp)
    return kc, q, i32(ref.cu(c["counts"])), opt, call


@pytest.mark.parametrize("c", CASES)
def test_attention(c):
    kc, q, cu_q, opt, call = build(c)
    st = status()
    want, lse, out_tol, lse_tol = ref.attention(q, kc, c["counts"], **opt)
    T = len(q)
    # an output with rows behind the last sequence and gaps between its rows: left alone
    out = torch.full((T, c["Hq"] + 1, c["d"] + 8), 7.0, dtype=q.dtype, device="cuda")
    got, got_lse = C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, kc.lens, cu_q, status=st,
                                                out=out[:, :c["Hq"], :c["d"]], **call)
    torch.cuda.synchronize()
    assert int(st) == 0
    within("lse", got_lse, lse, lse_tol)
    within("out", got, want, out_tol)
    assert (out[:, c["Hq"]:] == 7).all() and (out[:, :, c["d"]:] == 7).all()
    again, lse2 = C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, kc.lens, cu_q, **call)
    assert torch.equal(again, got) and torch.equal(lse2, got_lse)


@pytest.mark.parametrize("c", CASES)
def test_key_weights(c):
    kc, q, cu_q, opt, call = build(c, seed=5)
    st = status()
    lse = ref.attention(q, kc, c["counts"], **opt)[1].float().cuda()
    own, pre, own_tol, pre_tol = ref.weights(q, kc, c["counts"], lse, **opt)
    B, P, slots = len(c["lens"]), len(c["plens"]), kc.table.shape[1] * c["page"]
    start = torch.rand(B, c["Hkv"], slots + 5, device="cuda")
    scores = start.clone()
    pstart = torch.rand(P, c["Hkv"], kc.ptable.shape[1] * c["page"], device="cuda") if P else None
    pscores = None if pstart is None else pstart.clone()
    got, pgot = C.attention_varlen_cache_weights(q, kc.k, kc.table, kc.lens, cu_q, lse, scores, status=st,
                                                 prefix_scores=pscores, **call)
    torch.cuda.synchronize()
    assert int(st) == 0 and got is scores and pgot is pscores
    for x, x0, w, tol, lens, name in ((got, start, own, own_tol, c["lens"], "own"),
                                      (pgot, pstart, pre, pre_tol, c["plens"], "prefix")):
        for b, n in enumerate(lens):
            base = x0[b, :, :n].cpu().double()
            want = base + w[b]
            within(f"{name} {b}", x[b, :, :n], want, tol[b] + want.abs() * 2.0 ** -22)
            assert torch.equal(x[b, :, n:], x0[b, :, n:])
    # into another array, from zero: the same sums; and twice the same bits
    fresh = torch.full_like(scores, -1.0)
    a, _ = C.attention_varlen_cache_weights(q, kc.k, kc.table, kc.lens, cu_q, lse, None, scores_out=fresh, **call)
    b2, _ = C.attention_varlen_cache_weights(q, kc.k, kc.table, kc.lens, cu_q, lse, None,
                                             scores_out=torch.full_like(scores, -1.0), **call)
    assert torch.equal(a, b2)
    for b, n in enumerate(c["lens"]):
        within(f"fresh {b}", a[b, :, :n], own[b], own_tol[b] + own[b].abs() * 2.0 ** -22)
        assert (a[b, :, n:] == -1).all()


def test_weights_of_a_row_sum_to_one():
    """Every non-empty row spreads a weight of 1 over its keys."""
    c = dict(next(x for x in CASES if x.id == "prefix").values[0])
    kc, q, cu_q, _, call = build(c)
    out, lse = C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, kc.lens, cu_q, **call)
    z = torch.zeros(1, c["Hkv"], kc.ptable.shape[1] * c["page"], device="cuda")
    own, pre = C.attention_varlen_cache_weights(q, kc.k, kc.table, kc.lens, cu_q, lse, prefix_scores=z, **call)
    rows = len(q) * c["Hq"]
    total = float(own.double().sum() + pre.double().sum())
    # lse and every exponent are good to 2^-16 here
    assert abs(total - rows) <= rows * 2.0 ** -15


def test_padded_batch_leaves_rows_behind_the_last_sequence():
    kc = ref.Cache([40, 20, 0, 0], page=16, Hkv=1)
    q = normal(3, 9, 8, 160)
    q[3:] = math.nan
    out = torch.full_like(q, 5.0)
    lse = torch.full((9, 8), 5.0, device="cuda")
    st = status()
    C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, kc.lens, i32([0, 1, 3, 3, 3]), out=out, lse=lse, status=st,
                                 causal=True)
    scores = torch.zeros(4, 1, kc.table.shape[1] * 16, device="cuda")
    C.attention_varlen_cache_weights(q, kc.k, kc.table, kc.lens, i32([0, 1, 3, 3, 3]), lse, scores, status=st, causal=True)
    torch.cuda.synchronize()
    assert int(st) == 0
    assert (out[3:] == 5).all() and (lse[3:] == 5).all() and torch.isfinite(out[:3]).all()
    want, wlse, tol, ltol = ref.attention(q[:3], kc, [1, 2, 0, 0], causal=True)
    within("out", out[:3], want, tol)
    assert torch.isfinite(scores).all() and (scores[2:] == 0).all()


def test_matches_the_packed_forward():
    """A cache of whole prompts gives what attention_varlen_fwd gives for the same packed keys."""
    from ragged_gqa_attention_varlen_gb300 import binding
    lens = [130, 257, 64]
    kc = ref.Cache(lens, page=64, Hkv=1, dtype=HF)
    q = normal(4, sum(lens), 16, 160, dtype=HF)
    k = torch.cat([kc.rows(kc.k, kc.table, b, n) for b, n in enumerate(lens)]).to(HF).cuda()
    v = torch.cat([kc.rows(kc.v, kc.table, b, n) for b, n in enumerate(lens)]).to(HF).cuda()
    cu_q = i32(ref.cu(lens))
    slopes = torch.rand(3, 16, device="cuda") * 0.2
    a, la = binding.attention_varlen_fwd(q, k, v, cu_q, cu_q, slopes, causal=True)
    b, lb = C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, kc.lens, cu_q, slopes, causal=True)
    want, lse, tol, ltol = ref.attention(q, kc, lens, slopes=slopes, causal=True)
    within("out", b, want, tol)
    within("lse", lb, lse, ltol)
    assert float((la.double() - lb.double()).abs().max()) <= 2e-3  # the packed forward's lse is good to 1e-3


def test_bad_metadata_is_reported_and_harmless():
    """Lengths beyond the table, page numbers out of the pool and cu arrays that do not
    fit: a status bit, and nothing written out of range."""
    kc = ref.Cache([40, 20], page=16)
    q = normal(3, 2, 8, 160)
    table = kc.table.clone()
    table[0, 1] = 10 ** 6
    st = status()
    C.attention_varlen_cache_fwd(q, kc.k, kc.v, table, kc.lens, i32([0, 1, 2]), status=st)
    torch.cuda.synchronize()
    assert int(st) & C.DEV_BAD_CACHE
    for lens, cu_q, bit in (([10 ** 6, 5], [0, 1, 2], C.DEV_BAD_CACHE), ([-1, 5], [0, 1, 2], C.DEV_BAD_CACHE),
                            ([40, 20], [0, 2, 1], 1), ([40, 20], [0, 1, 900], 1)):
        st = status()
        lse = torch.zeros(2, 8, device="cuda")
        scores = torch.zeros(2, 1, kc.table.shape[1] * 16, device="cuda")
        C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, i32(lens), i32(cu_q), lse=lse, status=st)
        C.attention_varlen_cache_weights(q, kc.k, kc.table, i32(lens), i32(cu_q), lse, scores, status=st)
        torch.cuda.synchronize()
        assert int(st) & bit, (lens, cu_q, int(st))


# ---------------------------------------------------------------- rotary

ROT = [pytest.param(*x, id="-".join(map(str, x))) for x in [
    # T, Hq, Hkv, d, pairs, axes, interleaved, dtype, far
    (1, 1, 0, 64, 32, 1, False, "bf16", 100), (3, 96, 1, 160, 80, 3, False, "bf16", 1 << 20),
    (77, 5, 5, 64, 16, 2, False, "fp16", 5000), (130, 32, 8, 128, 48, 2, True, "fp16", 1 << 29),
    (33, 12, 3, 128, 63, 3, False, "bf16", 4000), (33, 12, 3, 128, 63, 3, True, "fp16", 4000),
    (50, 7, 1, 160, 1, 1, False, "fp16", 90), (2000, 0, 1, 160, 80, 3, True, "bf16", 1 << 20),
    (9, 300, 2, 64, 30, 1, True, "bf16", 70000)]]


@pytest.mark.parametrize("T,Hq,Hkv,d,pairs,axes,interleaved,dtype,far", ROT)
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary(T, Hq, Hkv, d, pairs, axes, interleaved, dtype, far, inverse):
    dt = BF if dtype == "bf16" else HF
    Hq, Hkv = (Hkv, 0) if Hq == 0 else (Hq, Hkv)
    q = normal(1, T, Hq + 1, d + 8, dtype=dt)[:, :Hq, :d]
    k = normal(2, T, Hkv, d, dtype=dt) if Hkv else None
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(0, far, (axes, T), generator=g, dtype=torch.int32).cuda()
    inv = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).cuda()
    axis = None if axes == 1 else torch.randint(0, axes, (pairs,), generator=g, dtype=torch.int32).cuda()
    got = C.attention_varlen_rotary(q, k, pos, inv, axis, interleaved, inverse)
    for x, y in ((q, got[0]), (k, got[1])):
        if x is not None:
            within("turned", y, *ref.rotated(x, pos, inv, axis, interleaved, inverse))
    whole = q.clone()
    C.attention_varlen_rotary(whole, k, pos, inv, axis, interleaved, inverse, q_out=whole,
                              k_out=None if k is None else k)
    assert torch.equal(whole, got[0]) and (k is None or torch.equal(k, got[1]))


def test_rotary_inverse_is_the_gradient():
    """<turn(x), y> = <x, turn_back(y)>, and differences of the 64-bit form give it too."""
    T, H, d, n = 20, 3, 128, 40
    x, y = normal(1, T, H, d, dtype=HF), normal(2, T, H, d, dtype=HF)
    pos = torch.randint(0, 9999, (2, T), dtype=torch.int32, device="cuda")
    inv = (10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)).cuda()
    axis = (torch.arange(n, device="cuda") % 2).int()
    grad = C.attention_varlen_rotary(y, None, pos, inv, axis, inverse=True)[0]
    xd, yd = x.cpu().double(), y.cpu().double()

    def f(z):  # the definition on fp64 values
        a = pos.cpu().double()[axis.cpu().long()].t() * inv.cpu()[None]
        cs, sn = a.cos()[:, None], a.sin()[:, None]
        p, q, r = z[..., :n], z[..., n:2 * n], z[..., 2 * n:]
        return float((torch.cat([p * cs - q * sn, q * cs + p * sn, r], -1) * yd).sum())

    r = torch.Generator().manual_seed(5)
    for _ in range(8):
        v = torch.randn(T, H, d, generator=r, dtype=torch.float64)
        diff = (f(xd + v) - f(xd - v)) / 2  # the map is linear: no truncation error
        tol = float((v.abs() * (yd.abs() * 2.0 ** -11 * 2 + 2.0 ** -18)).sum())
        assert abs(diff - float((grad.cpu().double() * v).sum())) <= tol


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("Hkv,d,page,dtype,new,held,rot", [
    (1, 160, 16, BF, [1, 1, 1], [0, 15, 16], 80), (8, 128, 64, HF, [5, 0, 200], [3, 7, 60], 64),
    (3, 64, 32, BF, [1], [31], 0), (2, 128, 128, HF, [300, 1], [0, 500], 33), (5, 64, 16, BF, [40] * 30, [9] * 30, 0)])
@pytest.mark.parametrize("strided", [False, True])
def test_append(Hkv, d, page, dtype, new, held, rot, strided):
    total = [a + b for a, b in zip(new, held)]
    kc = ref.Cache(total, (), Hkv, d, page, dtype, strided=strided)
    k0, v0 = kc.k.clone(), kc.v.clone()
    T, B = sum(new), len(new)
    k, v = normal(1, T + 2, Hkv, d, dtype=dtype), normal(2, T + 2, Hkv, d, dtype=dtype)  # two rows of padding
    kw, pos, inv = {}, None, None
    if rot:
        pos = torch.randint(0, 5000, (2, T + 2), dtype=torch.int32, device="cuda")
        inv = (10000.0 ** (-torch.arange(rot, dtype=torch.float64) / rot)).cuda()
        kw = dict(positions=pos, inv_freq=inv, pair_axis=(torch.arange(rot, device="cuda") % 2).int())
    kp = torch.full((B, Hkv, kc.table.shape[1] * page), -1, dtype=torch.int32, device="cuda")
    sc = torch.full(kp.shape, 3.0, device="cuda")
    out, st, lens = torch.zeros(B, dtype=torch.int32, device="cuda"), status(), i32(held)
    C.attention_varlen_cache_append(k, v, kc.k, kc.v, kc.table, lens, i32(ref.cu(new)), key_pos=kp, scores=sc,
                                    lens_out=out, status=st, **kw)
    torch.cuda.synchronize()
    assert int(st) == 0 and out.tolist() == total
    want_k, tol = ((k.cpu().double(), torch.zeros_like(k.cpu().double())) if not rot
                   else ref.rotated(k, pos, inv, kw["pair_axis"], False))
    want, bound = k0.cpu().double(), torch.zeros(k0.shape, dtype=torch.float64)
    wv, at = v0.clone(), ref.cu(new)
    for b in range(B):
        for i in range(new[b]):
            j = held[b] + i
            pg, o = int(kc.table[b, j // page]), j % page
            want[pg, o], bound[pg, o], wv[pg, o] = want_k[at[b] + i], tol[at[b] + i], v[at[b] + i]
            assert kp[b, :, j].tolist() == [int(pos[0, at[b] + i]) if rot else j] * Hkv
    got = kc.k.cpu().double()
    same = torch.isnan(want)
    assert torch.equal(torch.isnan(got), same) and torch.equal(torch.isnan(kc.v), torch.isnan(wv))
    assert ((got - want).abs()[~same] <= bound[~same]).all()
    assert torch.equal(kc.v.nan_to_num(9), wv.nan_to_num(9))
    n = sum(new)
    assert int((kp >= 0).sum()) == n * Hkv and int((sc == 0).sum()) == n * Hkv


def test_append_skips_what_has_no_page():
    kc = ref.Cache([16, 16], page=16, extra_width=0)
    k0, v0 = kc.k.clone(), kc.v.clone()
    k = normal(1, 3, 1, 160)
    table = kc.table.clone()
    table[1, 0] = 999
    st = status()
    # sequence 0 is full (slot 16 is behind the table), sequence 1's page is out of the pool
    C.attention_varlen_cache_append(k, k, kc.k, kc.v, table, i32([16, 3]), i32([0, 1, 3]), status=st)
    torch.cuda.synchronize()
    assert int(st) == C.DEV_BAD_CACHE
    assert torch.equal(kc.k.view(torch.int16), k0.view(torch.int16))
    assert torch.equal(kc.v.view(torch.int16), v0.view(torch.int16))


# ---------------------------------------------------------------- eviction

EV = [pytest.param(*x, id="-".join(map(str, x[:6])) + f"-{i}") for i, x in enumerate([
    # lens, Hkv, d, page, budget, recent, kind of scores
    ([65, 64, 3, 0], 1, 160, 16, 64, 8, "spread"), ([300, 1000, 40], 8, 128, 64, 100, 0, "spread"),
    ([500], 3, 64, 32, 77, 77, "spread"), ([400, 399], 2, 64, 16, 200, 50, "equal"),
    ([2500, 1025], 1, 128, 128, 1024, 100, "few"), ([5000], 2, 64, 1024, 1, 0, "spread"),
    ([700], 1, 160, 16, 300, 10, "odd"), ([60000, 50000], 1, 64, 64, 20000, 512, "spread"),
    ([33, 34, 35], 2, 64, 16, 32, 1, "negative"), ([201, 201, 201, 201], 3, 64, 16, 200, 20, "few"),
    ([301], 4, 64, 32, 300, 0, "odd"), ([5001, 5001], 2, 64, 64, 5000, 5000, "equal"),
    ([2, 2, 2], 1, 128, 16, 1, 0, "negative"), ([1030, 1030], 2, 64, 16, 1029, 1000, "spread")])]


@pytest.mark.parametrize("lens,Hkv,d,page,budget,recent,kind", EV)
@pytest.mark.parametrize("in_place", [True, False])
def test_evict(lens, Hkv, d, page, budget, recent, kind, in_place):
    g = torch.Generator().manual_seed(4)
    kc = ref.Cache(lens, (), Hkv, d, page, HF, strided=True)
    k0, v0 = kc.k.clone(), kc.v.clone()
    B, slots = len(lens), kc.table.shape[1] * page
    shape = (B, Hkv, slots + 1)
    sc = {"spread": lambda: torch.rand(shape, generator=g) ** 6, "equal": lambda: torch.ones(shape),
          "few": lambda: torch.randint(0, 3, shape, generator=g).float(),
          "negative": lambda: torch.randn(shape, generator=g),
          "odd": lambda: torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-42, -1e-42, 3e38])[
              torch.randint(0, 8, shape, generator=g)]}[kind]().cuda()
    kp = torch.full(shape, 1 << 29, dtype=torch.int32)
    for b, n in enumerate(lens):
        for h in range(Hkv):
            kp[b, h, :n] = torch.randperm(n + 5, generator=g)[:n].int()
    kp = kp.cuda()
    nxt, st = i32([n + 5 for n in lens]), status()
    so, po, lo = ((None, None, None) if in_place else
                  (torch.full_like(sc, -9.0), torch.full_like(kp, -9), torch.zeros_like(kc.lens)))
    s0, p0, lens_in = sc.clone(), kp.clone(), kc.lens.clone()
    lens_got, s_got, p_got = C.attention_varlen_cache_evict(
        kc.k, kc.v, kc.table, lens_in, sc, kp, nxt, budget, recent, scores_out=so, key_pos_out=po, lens_out=lo, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    wk, wv = k0.clone(), v0.clone()
    ws, wp = (s0.clone(), p0.clone()) if in_place else (so.new_full(shape, -9.0), po.new_full(shape, -9))
    table, news = kc.table.cpu(), []
    sl, pl = s0.cpu(), p0.cpu()
    for b, n in enumerate(lens):
        for h in range(Hkv):
            m, moves = ref.evicted(n, sl[b, h, :n].tolist(), pl[b, h, :n].tolist(), n + 5, budget, recent)
            if not in_place:
                ws[b, h, :m], wp[b, h, :m] = s0[b, h, :m], p0[b, h, :m]
            if moves:
                dst, src = (torch.tensor(x) for x in zip(*moves))
                row = table[b].long()
                dp, do, sp, s_o = row[dst // page].cuda(), (dst % page).cuda(), row[src // page].cuda(), (src % page).cuda()
                wk[dp, do, h], wv[dp, do, h] = k0[sp, s_o, h], v0[sp, s_o, h]
                ws[b, h, dst.cuda()], wp[b, h, dst.cuda()] = s0[b, h, src.cuda()], p0[b, h, src.cuda()]
        news.append(m)
    assert lens_got.tolist() == news
    eq = lambda a, b: torch.equal(a.nan_to_num(12345.0), b.nan_to_num(12345.0))  # noqa: E731
    assert eq(kc.k, wk) and eq(kc.v, wv)
    assert torch.equal(p_got, wp)
    assert torch.equal(torch.isnan(s_got), torch.isnan(ws)) and eq(s_got, ws)
    if not in_place:
        assert eq(sc, s0) and torch.equal(kp, p0) and torch.equal(lens_in, kc.lens)


def test_evict_bad_lengths():
    kc = ref.Cache([40, 20], page=16)
    k0 = kc.k.clone()
    sc = torch.rand(2, 1, kc.table.shape[1] * 16, device="cuda")
    kp = torch.zeros(sc.shape, dtype=torch.int32, device="cuda")
    st, lens = status(), i32([10 ** 6, -4])
    C.attention_varlen_cache_evict(kc.k, kc.v, kc.table, lens, sc, kp, i32([0, 0]), 4, 2, status=st)
    torch.cuda.synchronize()
    assert int(st) == C.DEV_BAD_CACHE and lens.tolist() == [10 ** 6, -4]
    assert torch.equal(kc.k.nan_to_num(1), k0.nan_to_num(1))


# ---------------------------------------------------------------- as they are used together

@pytest.mark.parametrize("Hq,Hkv,d,dtype,alibi", [(16, 1, 160, BF, True), (8, 4, 64, HF, False)])
def test_generation_steps(Hq, Hkv, d, dtype, alibi):
    """Prompts, then steps of rotary, append, attention, weights and eviction, every step's
    attention and weights against the 64-bit form on the cache as it stands."""
    page, budget, recent, B, plen = 16, 48, 12, 3, 40
    new = [50, 30, 47]
    width = 8
    g = torch.Generator().manual_seed(0)
    kc = ref.Cache([width * page] * B, [plen], Hkv, d, page, dtype, extra_width=0)
    kc.lens_l, lens = [0] * B, i32([0] * B)
    slots = width * page
    kp = torch.zeros(B, Hkv, slots, dtype=torch.int32, device="cuda")
    sc = torch.full((B, Hkv, slots), 77.0, device="cuda")
    pairs = d // 2
    inv = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).cuda()
    slopes = (torch.rand(B, Hq, generator=g) * 0.05) if alibi else None
    nxt, st = [plen] * B, status()
    for step in range(6):
        counts = new if step == 0 else [1, 2, 1]
        T = sum(counts)
        pos = i32([nxt[b] + i for b in range(B) for i in range(counts[b])]).view(1, T)
        q, k, v = (normal(10 * step + i, T, h, d, dtype=dtype) for i, h in ((1, Hq), (2, Hkv), (3, Hkv)))
        cu_q = i32(ref.cu(counts))
        q, _ = C.attention_varlen_rotary(q, None, pos, inv)
        longer = torch.empty_like(lens)
        C.attention_varlen_cache_append(k, v, kc.k, kc.v, kc.table, lens, cu_q, positions=pos, inv_freq=inv,
                                        key_pos=kp, scores=sc, lens_out=longer, status=st)
        lens, kc.lens_l = longer, longer.tolist()
        nxt = [a + b for a, b in zip(nxt, counts)]
        call = dict(prefix_table=kc.ptable, prefix_lens=kc.plens, cu_prefix=i32([0, B]), q_pos=pos[0], key_pos=kp,
                    causal=True, softcap=0.0)
        if alibi:
            call["alibi_slopes"] = slopes.cuda()
        opt = dict(group=[0] * B, slopes=slopes, causal=True, cap=0.0, q_pos=pos[0], key_pos=kp)
        out, lse = C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, lens, cu_q, status=st, **call)
        want, wl, otol, ltol = ref.attention(q, kc, counts, **opt)
        within("out", out, want, otol)
        within("lse", lse, wl, ltol)
        before = sc.clone()
        C.attention_varlen_cache_weights(q, kc.k, kc.table, lens, cu_q, lse, sc, status=st, **call)
        own, _, wtol, _ = ref.weights(q, kc, counts, lse, **opt)
        for b, n in enumerate(kc.lens_l):
            target = before[b, :, :n].cpu().double() + own[b]
            within("scores", sc[b, :, :n], target, wtol[b] + target.abs() * 2.0 ** -22)
        C.attention_varlen_cache_evict(kc.k, kc.v, kc.table, lens, sc, kp, i32(nxt), budget, recent, status=st)
        kc.lens_l = lens.tolist()
        assert max(kc.lens_l) <= budget
        for b in range(B):  # the recent tokens stay
            for h in range(Hkv):
                have = set(kp[b, h, :kc.lens_l[b]].tolist())
                assert set(range(max(plen, nxt[b] - recent), nxt[b])) <= have and len(have) == kc.lens_l[b]
    assert int(st) == 0


def test_captured_step_replays_on_new_inputs():
    """One step captured into a CUDA graph: replays follow lengths and tokens that change between them."""
    kc = ref.Cache([70, 90], page=16, extra_width=2, poison=False)
    full = kc.table.clone()
    free = [i for i in range(kc.num_pages) if i not in set(full[:, :6].flatten().tolist())]
    full[:, 6:] = free[0]
    B, Hq, d = 2, 16, 160
    q, k, v = normal(1, B, Hq, d), normal(2, B, 1, d), normal(3, B, 1, d)
    lens, longer = i32([70, 90]), i32([0, 0])
    cu_q = i32([0, 1, 2])
    out, lse = torch.empty_like(q), torch.empty(B, Hq, device="cuda")
    sc = torch.zeros(B, 1, full.shape[1] * 16, device="cuda")

    def step():
        C.attention_varlen_cache_append(k, v, kc.k, kc.v, full, lens, cu_q, lens_out=longer)
        C.attention_varlen_cache_fwd(q, kc.k, kc.v, full, longer, cu_q, out=out, lse=lse)
        C.attention_varlen_cache_weights(q, kc.k, full, longer, cu_q, lse, None, scores_out=sc)
        lens.copy_(longer)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        q.copy_(normal(20 + i, B, Hq, d))
        k.copy_(normal(30 + i, B, 1, d))
        graph.replay()
        torch.cuda.synchronize()
        kc.table, kc.lens_l = full, longer.tolist()
        assert kc.lens_l == [72 + i, 92 + i]
        want, wl, tol, ltol = ref.attention(q, kc, [1, 1])
        within("out", out, want, tol)
        within("lse", lse, wl, ltol)
        own, _, wt, _ = ref.weights(q, kc, [1, 1], lse)
        for b, n in enumerate(kc.lens_l):
            within("w", sc[b, :, :n], own[b], wt[b] + own[b] * 2.0 ** -22)


def test_other_stream():
    """On a stream of its own: what the call allocates belongs to that stream."""
    kc = ref.Cache([3000, 200], page=64)
    q = normal(1, 2, 48, 160)
    want, wl, tol, ltol = ref.attention(q, kc, [1, 1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, kc.lens, i32([0, 1, 2]), stream=s)
    s.synchronize()
    within("out", out, want, tol)
    within("lse", lse, wl, ltol)


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with what it allocates."""
    caches = [ref.Cache([4000, 100], page=64, seed=i) for i in range(2)]
    qs = [normal(i, 2, 48, 160) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            got[i] = C.attention_varlen_cache_fwd(qs[i], caches[i].k, caches[i].v, caches[i].table, caches[i].lens,
                                                  i32([0, 1, 2]), stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        want, wl, tol, ltol = ref.attention(qs[i], caches[i], [1, 1])
        within("out", got[i][0], want, tol)
        within("lse", got[i][1], wl, ltol)


def test_offsets_beyond_32_bits():
    """Pages behind 2^32 elements: append, attention, weights and eviction."""
    pages, page, H, d = 70000, 64, 8, 128  # 4.6e9 elements, 9.2 GB, K and V in one pool
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    k = torch.empty(pages, page, H, d, dtype=HF, device="cuda")
    v = torch.empty(pages, page, H, d, dtype=HF, device="cuda")
    far = [pages - 1, pages - 3, pages - 5]
    table = i32([far])
    new = normal(1, 150, H, d, dtype=HF)
    val = normal(2, 150, H, d, dtype=HF)
    lens, st = i32([0]), status()
    C.attention_varlen_cache_append(new, val, k, v, table, lens, i32([0, 150]), lens_out=(n := i32([0])), status=st)
    assert n.tolist() == [150]
    for x, src in ((k, new), (v, val)):
        got = torch.cat([x[p] for p in far])[:150]
        assert torch.equal(got, src)
    q = normal(3, 1, 32, d, dtype=HF, std=2.0)

    class Small:  # the same keys in a small pool
        lens_l, plens_l, Hkv, page_ = [150], [], H, page

        @staticmethod
        def rows(pool, t, r, m):
            return pool.cpu().double()[:m]

        table = ptable = None

    Small.k, Small.v, Small.d = new, val, d
    want, wl, tol, ltol = ref.attention(q, Small, [1], cap=0.0)
    out, lse = C.attention_varlen_cache_fwd(q, k, v, table, n, i32([0, 1]), softcap=0.0, status=st)
    within("out", out, want, tol)
    within("lse", lse, wl, ltol)
    sc, _ = C.attention_varlen_cache_weights(q, k, table, n, i32([0, 1]), lse, softcap=0.0, status=st)
    own, _, wt, _ = ref.weights(q, Small, [1], lse, cap=0.0)
    within("weights", sc[0, :, :150], own[0], wt[0] + own[0] * 2.0 ** -22)
    kp = torch.arange(192, dtype=torch.int32, device="cuda").expand(1, H, -1).contiguous()
    before = sc.clone()
    C.attention_varlen_cache_evict(k, v, table, n, sc, kp, i32([150]), 70, 8, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0 and n.tolist() == [70]
    flat_k = torch.cat([k[p] for p in far])
    for h in range(H):
        m, moves = ref.evicted(150, before[0, h, :150].tolist(), list(range(150)), 150, 70, 8)
        for dst, src in moves:
            assert torch.equal(flat_k[dst, h], new[src, h]) and int(kp[0, h, dst]) == src


def test_captured_eviction_step():
    """Weights and eviction captured into a graph: every replay takes one key from each full cache."""
    kc = ref.Cache([80, 80], page=16, Hkv=2, d=64, dtype=HF, poison=False)
    q, lens, budget = normal(1, 2, 8, 64, dtype=HF), i32([80, 80]), i32([0])
    sc = torch.rand(2, 2, kc.table.shape[1] * 16, device="cuda")
    kp = torch.arange(sc.shape[2], dtype=torch.int32, device="cuda").expand(2, 2, -1).contiguous()
    nxt, cu_q = i32([80, 80]), i32([0, 1, 2])
    qp = i32([79, 79])

    def step():
        out, lse = C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, lens, cu_q, q_pos=qp, key_pos=kp, causal=True)
        C.attention_varlen_cache_weights(q, kc.k, kc.table, lens, cu_q, lse, sc, q_pos=qp, key_pos=kp, causal=True)
        C.attention_varlen_cache_evict(kc.k, kc.v, kc.table, lens, sc, kp, nxt, 60, 10)
        return out, lse

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    saved = [x.clone() for x in (kc.k, kc.v, sc, kp, lens)]
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    for a, b in zip((kc.k, kc.v, sc, kp, lens), saved):
        a.copy_(b)
    kc.lens_l = [80, 80]
    for i in range(2):
        kc.lens_l = lens.tolist()
        want, wl, tol, ltol = ref.attention(q, kc, [1, 1], causal=True, q_pos=qp, key_pos=kp)
        graph.replay()
        torch.cuda.synchronize()
        within("out", out, want, tol)
        assert lens.tolist() == [60, 60]
        for b in range(2):
            for h in range(2):
                assert set(range(70, 80)) <= set(kp[b, h, :60].tolist())


def test_python_refusals():
    kc = ref.Cache([20, 9], page=16, Hkv=2, d=128)
    q, cu_q = normal(1, 2, 8, 128), i32([0, 1, 2])
    ok = dict(q=q, k_cache=kc.k, v_cache=kc.v, table=kc.table, lens=kc.lens, cu_q=cu_q)
    C.attention_varlen_cache_fwd(**ok)
    for change in (dict(q=q.half()), dict(q=q[:, :7]), dict(q=q.transpose(1, 2)), dict(v_cache=kc.v[:-1]),
                   dict(table=kc.table.long()), dict(table=kc.table.t()), dict(lens=kc.lens.float()),
                   dict(lens=kc.lens[:1]), dict(cu_q=cu_q[:2]), dict(cu_q=cu_q.cpu()), dict(q=q.cpu()),
                   dict(alibi_slopes=torch.zeros(2, 7, device="cuda")), dict(prefix_lens=kc.lens),
                   dict(prefix_table=kc.table), dict(key_pos=torch.zeros(2, 2, 64, dtype=torch.int32, device="cuda")),
                   dict(q_pos=i32([1]),), dict(out=torch.empty(2, 8, 64, dtype=BF, device="cuda")),
                   dict(lse=torch.empty(2, 9, device="cuda")), dict(k_cache=kc.k.transpose(2, 3)),
                   dict(status=torch.zeros(1, device="cuda")), dict(causal="x", window_left="y")):
        with pytest.raises(ValueError):
            C.attention_varlen_cache_fwd(**{**ok, **change})
    with pytest.raises(C.AttnError) as e:
        C.attention_varlen_cache_fwd(**ok, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -4
    with pytest.raises(C.AttnError) as e:
        C.attention_varlen_cache_fwd(**{**ok, "softcap": math.nan})
    assert e.value.code == -1
    with pytest.raises(ValueError):
        C.attention_varlen_rotary(q, None, i32([0, 1]), torch.ones(65, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError):
        C.attention_varlen_rotary(q, None, i32([0, 1, 2]), torch.ones(4, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError):
        C.attention_varlen_rotary(q, None, i32([0, 1]), torch.ones(4, device="cuda"))
    k = normal(2, 2, 2, 128)
    with pytest.raises(ValueError):
        C.attention_varlen_cache_append(k, k, kc.k, kc.v, kc.table, kc.lens, cu_q, lens_out=kc.lens)
    with pytest.raises(ValueError):
        C.attention_varlen_cache_append(k, k, kc.k, kc.v, kc.table, kc.lens, cu_q,
                                        inv_freq=torch.ones(4, dtype=torch.float64, device="cuda"))


def test_empty_calls():
    kc = ref.Cache([20, 9], page=16, Hkv=2, d=128)
    none = torch.empty(0, 8, 128, dtype=BF, device="cuda")
    out, lse = C.attention_varlen_cache_fwd(none, kc.k, kc.v, kc.table, kc.lens, i32([0, 0, 0]))
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)
    sc = torch.rand(2, 2, kc.table.shape[1] * 16, device="cuda")
    got, _ = C.attention_varlen_cache_weights(none, kc.k, kc.table, kc.lens, i32([0, 0, 0]), lse, sc,
                                              scores_out=torch.full_like(sc, 5.0))
    assert torch.equal(got[0, :, :20], sc[0, :, :20]) and (got[0, :, 20:] == 5).all()
    a, b = C.attention_varlen_rotary(none, None, torch.empty(1, 0, dtype=torch.int32, device="cuda"),
                                     torch.ones(4, dtype=torch.float64, device="cuda"))
    assert a.shape == none.shape and b is None
    lo = torch.zeros(2, dtype=torch.int32, device="cuda")
    C.attention_varlen_cache_append(none[:, :2], none[:, :2], kc.k, kc.v, kc.table, kc.lens, i32([0, 0, 0]), lens_out=lo)
    assert lo.tolist() == [20, 9]
    assert torch.isfinite(kc.k[kc.table[0, 0].long()]).all()


def test_expanded_outputs_are_refused():
    """One row of positions or scores for all heads may be read, not written."""
    kc = ref.Cache([40, 20], page=16, Hkv=2, d=64, dtype=HF)
    n, nxt = kc.table.shape[1] * 16, i32([40, 20])
    sc = torch.rand(2, 2, n, device="cuda")
    kp = torch.arange(n, dtype=torch.int32, device="cuda").expand(2, 2, n)
    with pytest.raises(C.AttnError):
        C.attention_varlen_cache_evict(kc.k, kc.v, kc.table, kc.lens, sc, kp, nxt, 8)
    po, lo = torch.empty(2, 2, n, dtype=torch.int32, device="cuda"), torch.empty_like(kc.lens)
    C.attention_varlen_cache_evict(kc.k, kc.v, kc.table, kc.lens, sc, kp, nxt, 8, key_pos_out=po, lens_out=lo)
    assert lo.tolist() == [8, 8]
    q, cu = normal(3, 2, 8, 64, dtype=HF), i32([0, 1, 2])
    out = torch.empty(1, 8, 64, dtype=HF, device="cuda").expand(2, 8, 64)
    with pytest.raises(C.AttnError):
        C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, lo, cu, out=out)
    lse = C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, lo, cu)[1]
    with pytest.raises(C.AttnError):
        C.attention_varlen_cache_weights(q, kc.k, kc.table, lo, cu, lse, sc[:, :1].expand(2, 2, n))
    with pytest.raises(C.AttnError):
        C.attention_varlen_rotary(q, None, nxt, torch.ones(32, dtype=torch.float64, device="cuda"), q_out=out)
