"""The cache held in 8 bits at its edges, for both of its attention kernels: exact means, rows bounded by
their own weights, factors far apart, missing pages, rows far from their keys; and the append's
smallest factors."""
import math

import pytest
import torch

import cache8_ref as ref8
import cache8_rows as rows8
import cache_ref as ref
from ragged_gqa_attention_varlen_gb300 import cache as C
from test_cache8_gpu import F8, PICKED, attend, build, odd_scales, steep_scales
from test_cache_gpu import BF, HF, case, i32, lib, normal, status, within  # noqa: F401

pytestmark = pytest.mark.gpu


def run(q, kc, counts, call, want_status=0, **more):
    st = status()
    got = attend(q, kc, i32(ref.cu(counts)), call, status=st, **more)
    torch.cuda.synchronize()
    assert int(st) == want_status
    return got


def check(got, want, where=slice(None)):
    within("lse", got[1][where], want[1][where], want[3][where])
    within("out", got[0][where], want[0][where], want[2][where])


# ---------------------------------------------------------------- sums of the weights

@pytest.mark.parametrize("cap,std", [(0.0, 3.0), (3.0, 3.0), (30.0, 3.0), (0.0, 12.0)])
@pytest.mark.parametrize("scale", [0.25, 2.0 - 2.0 ** -10])
@pytest.mark.parametrize("lens,plens,counts,Hq,Hkv,d,page", [
    ([1, 2, 3, 5], (), [20] * 4, 16, 1, 160, 16), ([2, 4, 130], (), [30, 10, 40], 8, 2, 128, 32), ([2, 1, 4], [3], [10, 10, 20], 16, 1, 160, 16),
    ([3, 9, 200], (), [10, 20, 10], 8, 1, 64, 16), ([2, 3, 4, 5, 700], (), [1] * 5, 96, 1, 160, 64),
    ([2, 3, 5, 40] * 20, (), [1] * 80, 32, 8, 128, 16), ([1500, 600, 900] * 10, (), [1] * 30, 32, 8, 64, 64),
    ([1500, 600], (), [2, 3], 96, 1, 128, 64), ([2, 3, 7, 300] * 10, (), [1] * 40, 16, 1, 160, 64), ([2, 3, 4] * 20, (), [1] * 60, 8, 2, 64, 16)])
def test_equal_values_come_out_exactly(lens, plens, counts, Hq, Hkv, d, page, scale, cap, std):
    """As over the 16-bit cache: where all V rows are the same, out is that row, whatever the weights'
    roundings, and whatever the factor.  The sums' errors (below 300 additions of 2^-22, the reciprocal and
    products less than 60 * 2^-24) stay below half a step of fp16 (2^-12 of the value)."""
    kc = ref8.Cache8(lens, plens, Hkv=Hkv, d=d, page=page, block=16)
    bits = torch.tensor([-1.0, 1.0, 0.5, -2.0] if scale > 1 else [1.875, -1.875, 0.9375, 1.0, -1.125])
    row = bits[torch.randint(0, len(bits), (Hkv, d), generator=torch.Generator().manual_seed(3))].cuda()
    kc.v8.view(torch.uint8).copy_(row.to(F8).view(torch.uint8))
    kc.v_scale.fill_(scale)
    q = normal(8, sum(counts), Hq, d, dtype=HF, std=std)
    call = dict(prefix_table=kc.ptable, prefix_lens=kc.plens, cu_prefix=i32([0, len(lens)])) if plens else {}
    out, _ = run(q, kc, counts, dict(softcap=cap, **call))
    want = (row * scale).to(HF).repeat_interleave(Hq // Hkv, 0).expand_as(out)
    assert torch.equal(out, want), (out != want).float().mean()


# ---------------------------------------------------------------- each row by its own size

# single tokens, a few and prompts in one batch, on both sides of the rule for few rows; keys enough to be cut
MIXED = [
    case("mixed_one_prompt", [900] + ref.spread(41, 60, 1, 900), [130] + [1] * 60, Hq=4, Hkv=2, d=64, page=32, cap=0.0),
    case("mixed_prompt_in_the_middle", ref.spread(42, 30, 1, 600) + [1500] + [40] * 30, [1] * 30 + [60] + [0, 2] * 15, Hq=4, Hkv=1, d=160, page=64, alibi=True),
    case("mixed_long", [9000, 7000, 33, 2500], [1, 5, 1, 1], Hq=16, Hkv=2, d=128, page=64, cap=0.0, dtype=HF, alibi=True),
    case("mixed_window", ref.spread(43, 20, 1, 900), [1, 3] * 10, Hq=16, Hkv=2, d=128, page=16, wl=100, cap=30.0),
    case("mixed_at_the_border", [300, 301, 302, 303] * 5, [1, 2, 3, 1] * 5, Hq=16, Hkv=2, d=64, page=16, cap=9.0, dtype=HF),
    case("mixed_shuffled", [400, 33, 250, 600], [1, 30, 2, 1], Hq=2, Hkv=1, d=160, page=64, alibi=True, shuffled=True),
    case("mixed_no_keys", [0, 5, 0, 400], [30, 0, 1, 1], Hq=2, Hkv=2, d=64, cap=0.0),
    case("fewer_tokens_than_sequences", [700, 20, 30, 500, 5, 6, 7, 8] * 8, ([40] + [0] * 7) + [0, 0, 0, 1, 0, 0, 0, 0] * 7, Hq=8, Hkv=2, d=128, page=64, cap=0.0),
]


@pytest.mark.parametrize("scales", [None, odd_scales, steep_scales])
@pytest.mark.parametrize("c", PICKED + MIXED)
def test_rows_by_their_own_size(c, scales):
    kc, q, cu_q, opt, call = build(c, 16, seed=5, scales=scales, std=0.05 if scales is steep_scales else None)
    got = run(q, kc, c["counts"], call)
    check(got, rows8.attention(q, kc, c["counts"], **opt))
    again = run(q, kc, c["counts"], call)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


@pytest.mark.parametrize("c", MIXED[:3])
def test_both_kernels_captured_and_on_two_streams(c):
    """Where both kernels work, the tiles start beside the other's last CTAs: the same bits captured,
    replayed between other calls, and on two streams at once."""
    kc, q, cu_q, opt, call = build(c, 16, seed=5)
    want = attend(q, kc, cu_q, call)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    pairs = [attend(q, kc, cu_q, call, stream=s) for _ in range(5) for s in (s1, s2)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for r in pairs for x, y in zip(r, want))
    out, lse, ws = torch.empty_like(q).contiguous(), torch.empty(q.shape[:2], device="cuda"), torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            attend(q, kc, cu_q, call, out=out, lse=lse, workspace=ws)
    for _ in range(3):
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("apart", [20, 30, 40])
@pytest.mark.parametrize("Hq,cap", [(8, 0.0), (48, 0.0), (48, 3.0)])
def test_small_blocks_beside_huge_ones(Hq, cap, apart, odd):
    """The window holds blocks 2^20 to 2^40 below the others of its key tiles, which no row reads."""
    kc = ref8.Cache8([300, 1000], Hkv=1, d=160, page=64, block=16, scales=odd_scales if odd else None)
    for b, n in enumerate(kc.lens_l):
        for first in range(0, (n - 51) // 16 * 16, 16):
            kc.v_scale[int(kc.table[b, first // 64]), first % 64 // 16] *= 2.0 ** apart
    kc.v = kc._values(kc.v8, kc.v_scale)
    q = normal(4, 2, Hq, 160, dtype=HF)
    got = run(q, kc, [1, 1], dict(causal=True, window_left=50, softcap=cap))
    check(got, rows8.attention(q, kc, [1, 1], causal=True, wl=50, cap=cap))


# ---------------------------------------------------------------- what the pages hold

@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("cap", [0.0, 3.0, 30.0])
@pytest.mark.parametrize("Hq", [8, 48])
def test_missing_pages_in_both_kernels(Hq, cap, alibi):
    """As if their slots were not there: single pages, a whole key tile, the nearest and the farthest."""
    kc = ref8.Cache8([300, 700, 40], Hkv=1, page=16, block=16)
    gone = {0: [2, 4, 18], 1: list(range(8, 16)) + [0, 43], 2: [0, 1, 2]}
    good = kc.table.clone()
    for b, pages in gone.items():
        for i, p in enumerate(pages):
            kc.table[b, p] = 10 ** 6 if i % 2 else -3
    q = normal(3, 3, Hq, 160)
    slopes = torch.rand(3, Hq, generator=torch.Generator().manual_seed(2)) * 0.2
    slopes[:, 1::3] *= -1
    call = dict(causal=True, softcap=cap, **(dict(alibi_slopes=slopes.cuda()) if alibi else {}))
    got = run(q, kc, [1] * 3, call, C.DEV_BAD_CACHE)
    kc.table = good
    keep = lambda b, p, pl, n: torch.tensor([j // 16 not in gone[b] for j in range(n)])
    want = rows8.attention(q, kc, [1] * 3, causal=True, cap=cap, slopes=slopes if alibi else None, keep=keep)
    check(got, want)
    assert (got[0][2] == 0).all()


@pytest.mark.parametrize("cap", [0.0, 3.0])
def test_missing_page_of_a_prefix(cap):
    kc = ref8.Cache8([30, 1, 200], [400], Hkv=2, d=128, page=64, block=32)
    good = kc.ptable.clone()
    kc.ptable[0, 3] = -1
    q = normal(3, 4, 8, 128)
    call = dict(causal=True, softcap=cap, prefix_table=kc.ptable, prefix_lens=kc.plens, cu_prefix=i32([0, 3]))
    got = run(q, kc, [1, 2, 1], call, C.DEV_BAD_CACHE)
    kc.ptable = good
    keep = lambda b, p, pl, n: torch.tensor([not 192 <= j < 256 for j in range(pl)] + [True] * n)
    check(got, rows8.attention(q, kc, [1, 2, 1], causal=True, cap=cap, group=[0, 0, 0], keep=keep))


@pytest.mark.parametrize("cap", [0.0, 3.0])
@pytest.mark.parametrize("Hq", [8, 96])
def test_zero_factors_in_both_kernels(Hq, cap):
    """Blocks of zeros among others, and all the keys that are met first."""
    kc = ref8.Cache8([700, 400], Hkv=2, d=128, page=64, block=16, scales=lambda top, g: torch.where(
        torch.rand(top.shape, generator=g) < 0.5, 0.0, ref8.pow2_scale(top)))
    for p in kc.table[0, 4:11].tolist():
        kc.v_scale[p] = torch.where(torch.isnan(kc.v_scale[p]), math.nan, 0.0)
    kc.v = kc._values(kc.v8, kc.v_scale)
    q = normal(2, 2, Hq, 128, dtype=HF)
    check(run(q, kc, [1, 1], dict(softcap=cap)), rows8.attention(q, kc, [1, 1], cap=cap))


def test_pages_beyond_4_gb_in_the_tiles():
    kc = ref8.Cache8([200, 700], Hkv=1, d=128, page=64, block=16)
    q = normal(2, 2, 48, 128, dtype=HF)
    want = run(q, kc, [1, 1], dict(softcap=0.0))
    far = (5 << 30) // (64 * 128)
    n = kc.k8.shape[0]
    for x in ("k", "v"):
        big = torch.empty(far + n, 64, 1, 128, dtype=torch.uint8, device="cuda")
        big[far:] = getattr(kc, x + "8").view(torch.uint8)
        scale = torch.full((far + n, 4, 1), math.nan, device="cuda")
        scale[far:] = getattr(kc, x + "_scale")
        setattr(kc, x + "8", big.view(F8))
        setattr(kc, x + "_scale", scale)
    kc.table = (kc.table + far).int()
    got = run(q, kc, [1, 1], dict(softcap=0.0))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("counts", [[1, 1, 0, 0], [1, 2, 0, 0], [20, 1, 0, 0]])
def test_padded_batch_of_few_rows(counts):
    kc = ref8.Cache8([40, 20, 0, 0], page=16, Hkv=1)
    T = sum(counts)
    q = normal(3, T + 5, 2, 160)
    q[T:] = math.nan
    out, lse = torch.full_like(q, 5.0), torch.full((T + 5, 2), 5.0, device="cuda")
    run(q, kc, counts, dict(causal=True), out=out, lse=lse)
    assert (out[T:] == 5).all() and (lse[T:] == 5).all()
    check((out[:T], lse[:T]), rows8.attention(q[:T], kc, counts, causal=True))


# ---------------------------------------------------------------- rows far from their keys

@pytest.mark.parametrize("cap", [0.0, 3.0, 30.0])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("far", [1000, 1 << 20, (1 << 24) + 1, (1 << 30) - 6000])
@pytest.mark.parametrize("Hq", [4, 32])
def test_alibi_of_rows_far_from_their_keys(Hq, far, dtype, cap):
    """A row at any distance behind its keys weighs them as one next to them does; lse is less by
    slope times the way between."""
    lens, counts = [300, 40, 5000], [1, 2, 1]
    kc = ref8.Cache8(lens, Hkv=2, d=160, page=64, block=32)
    q = normal(2, sum(counts), Hq, 160, dtype=dtype)
    slopes = torch.rand(3, Hq, generator=torch.Generator().manual_seed(4)) + 0.01
    slopes[:, ::4] = 0.0
    near = [lens[b] + i for b, n in enumerate(counts) for i in range(n)]
    want = rows8.attention(q, kc, counts, slopes=slopes, causal=True, cap=cap, q_pos=torch.tensor(near))
    out, lse = run(q, kc, counts, dict(softcap=cap, alibi_slopes=slopes.cuda(), causal=True, q_pos=i32([x + far for x in near])))
    less = far * torch.repeat_interleave(slopes.double(), torch.tensor(counts), 0)
    within("lse", lse, want[1] - less, want[3] + less * 2.0 ** -22)
    within("out", out, want[0], want[2])


# ---------------------------------------------------------------- append

def test_append_to_blocks_with_the_smallest_factors():
    """Factors below 2^-126 (another quantiser's) are factors all the same: zeros stay zeros beside
    them, and small values are value / factor."""
    kc = ref8.Cache8([16] * 4, Hkv=1, d=64, page=16, block=16)
    tiny = [2.0 ** -127, 2.0 ** -130, 3 * 2.0 ** -149, 2.0 ** -128]
    k = torch.zeros(4, 1, 64)
    k[1, 0, :3] = torch.tensor([2.0 ** -126, -(2.0 ** -128), 2.0 ** -133])
    k[3, 0, 5] = 1.0
    k = k.to(BF).cuda()
    pages = [int(p) for p in kc.table[:, 0]]
    for p, s in zip(pages, tiny):
        kc.k_scale[p] = kc.v_scale[p] = s
    held = [x.view(torch.uint8).clone() for x in (kc.k8, kc.v8)]
    C.attention_varlen_cache8_append(k, k, kc.k8, kc.v8, kc.k_scale, kc.v_scale, kc.table, i32([8] * 4), i32(range(5)))
    for x, s, old in ((kc.k8, kc.k_scale, held[0]), (kc.v8, kc.v_scale, held[1])):
        assert [float(s[p, 0, 0]) for p in pages] == tiny[:3] + [2.0 ** -8]
        for b in (0, 1, 2):
            got = x[pages[b], 8, 0].float().cpu().double()
            assert torch.equal(got, ref8.e4m3(k[b, 0].cpu().double() / tiny[b])), b
            assert torch.equal(x[pages[b], :8].view(torch.uint8), old[pages[b], :8])
        assert float(x[pages[3], 8, 0, 5].float()) == 256.0


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("d,pairs,interleaved", [(160, 80, True), (160, 40, False), (128, 64, False), (64, 20, True)])
def test_append_rounds_keys_as_64_bits_would(d, pairs, interleaved, norm):
    """No K value falls to the other side of an e4m3 border, unless it lies there within what is left of
    the arithmetic's error: sine and cosine are off by 2^-27; with a norm, the fp32 sum of squares by
    20 additions' half steps (2^-25 each, half of it in the root) and the normed values by a step."""
    T, dt = 40000, HF
    pages = T // 64
    k = normal(3, T, 1, d, dtype=dt, std=1.5)
    pools = [torch.zeros(pages, 64, 1, d, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2)]
    scales = [torch.zeros(pages, 4, 1, device="cuda") for _ in range(2)]
    g = torch.Generator().manual_seed(2)
    pos = torch.randint(0, 100000, (T,), generator=g, dtype=torch.int32).cuda()
    inv = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).cuda()
    w = (torch.rand(d, generator=g) + 0.5).cuda() if norm else None
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    C.attention_varlen_cache8_append(k, k, *pools, *scales, table, i32([0]), i32([0, T]), positions=pos, inv_freq=inv, interleaved=interleaved,
                                     k_weight=w)
    x = k[:, 0].double()
    if norm:
        x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
    ang = pos.double()[:, None] * inv[None]
    i = torch.arange(pairs, device="cuda")
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    a, b = x[:, ia].clone(), x[:, ib].clone()
    mag = x.abs()
    x[:, ia], x[:, ib] = a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()
    mag[:, ia] = mag[:, ib] = a.abs() + b.abs()
    now = scales[0].view(T // 16, 1, 1).double()
    assert torch.equal(now.flatten(), ref8.pow2_scale(x.view(T // 16, -1).abs().amax(1).cpu()).cuda())
    x, mag, got = x.view(T // 16, 16, d) / now, mag.view(T // 16, 16, d) / now, pools[0].view(T // 16, 16, d).double()
    off = mag * (2.0 ** -21 if norm else 2.0 ** -26)
    wrong = (got != ref8.e4m3(x)) & (ref8.e4m3(x - off) == ref8.e4m3(x + off))
    assert not wrong.any(), (int(wrong.sum()), wrong.numel())
    # values lie anywhere between two borders, a step apart: the share of them that is within `off` of one
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    assert float((got != ref8.e4m3(x)).double().mean()) <= float((2 * off / step).mean())
