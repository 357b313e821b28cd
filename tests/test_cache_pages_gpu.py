"""Forking, freeing, reserving, packing and copying pages on the GPU, against the definitions in lists."""
import random

import pytest
import torch

import cache8_ref as ref8
from ragged_gqa_attention_varlen_gb300 import cache as C
from test_cache_gpu import BF, i32, lib, status  # noqa: F401

pytestmark = pytest.mark.gpu


def world(seed, R, page, hi, spare, layers=2, Hkv=2, d=64, shared=True, width=None, free_share=0.1):
    """Rows over a pool, some sharing full pages, pools of 16-bit and 8-bit pages and scales."""
    r = random.Random(seed)
    lens = [r.choice([0, 1, page - 1, page, page + 1, r.randint(0, hi)]) for _ in range(R)]
    held = [-(-n // page) + (r.random() < 0.3) for n in lens]
    W = width or max(held) + 3
    N = sum(held) + spare
    order = r.sample(range(N), N)
    refs, table = [0] * N, []
    for n, h in zip(lens, held):
        row = []
        for c in range(h):
            full_donors = [t for t, m in zip(table, lens) if c < min(m // page, len(t))]
            if shared and c < n // page and full_donors and r.random() < 0.4 and c == len(row):
                row.append(r.choice(full_donors)[c])
            else:
                row.append(order.pop())
            refs[row[-1]] += 1
        table.append(row)
    for _ in range(spare // 4):  # pages that others hold
        refs[order.pop()] = r.randint(1, 3)
    t = torch.full((R, W), -9, dtype=torch.int32)
    for row, x in zip(t, table):
        row[:len(x)] = torch.tensor(x, dtype=torch.int32)
    g = torch.Generator().manual_seed(seed)
    pools = []
    for _ in range(layers):
        pools.append(torch.randn(N, page, Hkv, d, generator=g).to(BF).cuda())
        pools.append(torch.randint(0, 256, (N, page, Hkv, d), generator=g, dtype=torch.uint8).cuda().view(torch.float8_e4m3fn))
        pools.append(torch.rand(N, page // 16, Hkv, generator=g).cuda())
    wide = torch.randn(N, page, Hkv + 1, d + 8, generator=g).cuda()
    pools.append(wide[:, :, :Hkv, :d])  # fp32, with gaps
    return dict(N=N, W=W, page=page, lens=lens, held=held, refs=refs, table=table, t=t.cuda(), pools=pools, r=r, wide=wide)


def bits(pools):
    return [p.view(torch.uint8) if p.dtype == torch.float8_e4m3fn else p.clone() for p in pools]


def moved(old, page, copies):
    want = [x.clone() for x in old]
    for x in want:
        for s, d, used in copies:
            rows = -(-used * x.shape[1] // page)
            x[d, :rows] = x[s, :rows]
    return want


@pytest.mark.parametrize("seed,R,page,hi,kind", [(1, 1, 16, 40, "keep"), (2, 6, 16, 70, "beams"), (3, 40, 32, 300, "beams"), (4, 40, 64, 900, "free"),
                                                 (5, 300, 16, 400, "beams"), (6, 7, 128, 1000, "reserve"), (7, 900, 16, 300, "reserve"),
                                                 (8, 33, 1024, 3000, "beams"), (9, 12, 16, 50, "none")])
@pytest.mark.parametrize("inplace", [False, True])
def test_fork(seed, R, page, hi, kind, inplace):
    w = world(seed, R, page, hi, spare=R * 6 + 8)
    r = w["r"]
    if kind == "beams":
        parents = [r.randrange(-1, R) if r.random() < 0.9 else r.randrange(R) for _ in range(R)]
    elif kind == "free":
        parents = [i if r.random() < 0.5 else -1 for i in range(R)]
    elif kind == "none":
        parents = [-1] * R
    else:
        parents = list(range(R))
    room = [r.choice([0, 0, 1, page, 2 * page - 1]) if kind != "keep" else 0 for _ in range(R)]
    want = ref8.forked(page, w["N"], w["W"], w["table"], w["lens"], w["held"], w["refs"], parents, room)
    assert want is not None
    rows, lens, held, refs, copies = want
    old = [x.clone() for x in bits(w["pools"])]
    st = status()
    args = [i32(w["lens"]), i32(w["held"]), i32(w["refs"])]
    outs = {} if inplace else dict(table_out=torch.full_like(w["t"], -4), lens_out=torch.zeros_like(args[0]), held_out=torch.zeros_like(args[1]),
                                   refs_out=torch.zeros_like(args[2]))
    before = w["t"].clone() if inplace else torch.full_like(w["t"], -4)
    got = C.attention_varlen_cache_fork(w["pools"], w["t"], *args, i32(parents), i32(room) if kind != "keep" else None, status=st, **outs)
    torch.cuda.synchronize()
    assert int(st) == 0
    assert got[1].tolist() == lens and got[2].tolist() == held and got[3].tolist() == refs
    t, before = got[0].cpu(), before.cpu()
    for i, x in enumerate(rows):
        assert t[i, :len(x)].tolist() == x
        assert torch.equal(t[i, len(x):], before[i, len(x):])
    for x, y in zip(bits(w["pools"]), moved(old, page, copies)):
        assert torch.equal(x, y)
    if not inplace:
        assert args[0].tolist() == w["lens"] and args[2].tolist() == w["refs"]


@pytest.mark.parametrize("what", ["pages", "width", "parent", "room", "length", "held", "held_wide", "entry", "entry_negative"])
@pytest.mark.parametrize("inplace", [False, True])
def test_fork_does_nothing_when_something_does_not_fit(what, inplace):
    w = world(11, 9, 16, 120, spare=8, width=14)
    lens, held, refs, parents, room = list(w["lens"]), list(w["held"]), list(w["refs"]), list(range(9)), [0] * 9
    t = w["t"].clone()
    row = max(range(9), key=lambda i: held[i])
    bit = C.DEV_BAD_CACHE
    if what == "pages":
        room, bit = [100] * 9, C.DEV_NO_PAGES
    elif what == "width":
        room[row], bit = 16 * 14 - lens[row] + 1, C.DEV_NO_PAGES
    elif what == "parent":
        parents[3] = 9
    elif what == "room":
        room[2] = -1
    elif what == "length":
        lens[row] = held[row] * 16 + 1
    elif what == "held":
        held[row] = -1
    elif what == "held_wide":
        held[row] = 15
    elif what == "entry":
        t[row, 1] = w["N"]
    else:
        t[row, 0] = -1
    a, b, c = i32(lens), i32(held), i32(refs)
    old, t0 = [x.clone() for x in bits(w["pools"])], t.clone()
    outs = {} if inplace else dict(table_out=torch.full_like(t, -4), lens_out=torch.zeros_like(a), held_out=torch.zeros_like(b), refs_out=torch.zeros_like(c))
    st = status()
    got = C.attention_varlen_cache_fork(w["pools"], t, a, b, c, i32(parents), i32(room), status=st, **outs)
    torch.cuda.synchronize()
    assert int(st) & bit
    assert torch.equal(got[0], t0) and got[1].tolist() == lens and got[2].tolist() == held and got[3].tolist() == refs
    assert all(torch.equal(x, y) for x, y in zip(bits(w["pools"]), old))


def test_fork_of_a_large_table():
    """More cells and pages than one block takes, no pools: the metadata alone."""
    w = world(21, 2000, 16, 600, spare=20000, layers=1, Hkv=1)
    parents = [w["r"].randrange(2000) for _ in range(2000)]
    room = [w["r"].randrange(40) for _ in range(2000)]
    rows, lens, held, refs, _ = ref8.forked(16, w["N"], w["W"], w["table"], w["lens"], w["held"], w["refs"], parents, room)
    got = C.attention_varlen_cache_fork([], w["t"], i32(w["lens"]), i32(w["held"]), i32(w["refs"]), i32(parents), i32(room), page_size=16)
    assert got[1].tolist() == lens and got[2].tolist() == held and got[3].tolist() == refs
    t = got[0].tolist()
    assert all(t[i][:len(x)] == x for i, x in enumerate(rows))


@pytest.mark.parametrize("seed,R,page,hi,prefix", [(1, 1, 16, 40, False), (2, 12, 16, 200, True), (3, 90, 64, 700, False), (4, 600, 16, 500, True)])
@pytest.mark.parametrize("inplace", [False, True])
def test_compact(seed, R, page, hi, prefix, inplace):
    w = world(seed, R, page, hi, spare=R * 3 + 20)
    refs = list(w["refs"])
    keep = [i for i in range(R) if w["r"].random() < 0.6]
    t, held, table = w["t"][keep].contiguous(), [w["held"][i] for i in keep], [w["table"][i] for i in keep]
    for i in set(range(R)) - set(keep):
        for p in w["table"][i]:
            refs[p] -= 1
    pt, pheld = (t[1:3].clone(), held[1:3]) if prefix else (None, None)
    live, moves = ref8.compacted(refs)
    to = {s: d for s, d in moves}
    old = [x.clone() for x in bits(w["pools"])]
    before = t.clone() if inplace else torch.full_like(t, -4)
    a, st = i32(refs), status()
    outs = {} if inplace else dict(table_out=torch.full_like(t, -4), refs_out=torch.zeros_like(a), prefix_table_out=None if pt is None else torch.full_like(pt, -4))
    n, t2, refs2, pt2 = C.attention_varlen_cache_compact(w["pools"], t, i32(held), a, prefix_table=pt, prefix_held=None if pt is None else i32(pheld), status=st, **outs)
    torch.cuda.synchronize()
    assert int(st) == 0 and int(n) == live
    new = [refs[i] if i < live and refs[i] > 0 else 0 for i in range(len(refs))]
    for s, d in moves:
        new[d] = refs[s]
    assert refs2.tolist() == new
    for i, x in enumerate(table):
        assert t2[i, :held[i]].tolist() == [to.get(p, p) for p in x]
        assert torch.equal(t2[i, held[i]:], before[i, held[i]:])
    if prefix:
        for i in range(len(pheld)):
            assert pt2[i, :pheld[i]].tolist() == [to.get(p, p) for p in table[1 + i]]
    for x, y in zip(bits(w["pools"]), moved(old, page, [(s, d, page) for s, d in moves])):
        assert torch.equal(x, y)


def test_compact_of_bad_tables_and_of_nothing():
    """Entries out of the pool or of free pages are left as they are and reported; an empty and a full pool."""
    page, N = 16, 6
    pool = torch.randn(N, page, 1, 64, device="cuda")
    old = pool.clone()
    st = status()
    t = i32([[5, 77, 1], [-2, 5, 9]])
    n, t2, refs, _ = C.attention_varlen_cache_compact([pool], t, i32([3, 1]), i32([0, 0, 1, 0, 0, 2]), status=st)
    torch.cuda.synchronize()
    assert int(st) == C.DEV_BAD_CACHE and int(n) == 2
    # the first free page (0) takes the first live one at or above 2, which is 2; 5 goes to 1
    assert t2.tolist() == [[1, 77, 1], [-2, 5, 9]] and refs.tolist() == [1, 2, 0, 0, 0, 0]
    assert torch.equal(pool[0], old[2]) and torch.equal(pool[1], old[5])
    for refs in ([0] * N, [1] * N):
        old = pool.clone()
        n, _, out, _ = C.attention_varlen_cache_compact([pool], i32([[0]]), i32([0]), i32(refs))
        assert int(n) == sum(refs) and out.tolist() == refs and torch.equal(pool, old)


def test_copy():
    w = world(31, 20, 32, 300, spare=30)
    N = w["N"]
    src, dst = w["r"].sample(range(N), 20), None
    dst = w["r"].sample([i for i in range(N) if i not in src], 20)
    old = [x.clone() for x in bits(w["pools"])]
    st = status()
    C.attention_varlen_cache_copy(w["pools"], i32(src), i32(dst), status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    for x, y in zip(bits(w["pools"]), moved(old, 32, [(s, d, 32) for s, d in zip(src, dst)])):
        assert torch.equal(x, y)
    # into other pools, of another size and other strides; pairs out of range are left out
    other = [torch.zeros(8, 32, 3, 72, dtype=BF, device="cuda")[:, :, :2, :64], torch.zeros(8, 2, 5, device="cuda")[:, :, 1:3]]
    C.attention_varlen_cache_copy([w["pools"][0], w["pools"][2]], i32([3, 1, N, -1, 2]), i32([7, 0, 1, 2, 8]), other, status=st)
    torch.cuda.synchronize()
    assert int(st) == C.DEV_BAD_CACHE
    for x, y in zip((w["pools"][0], w["pools"][2]), other):
        assert torch.equal(y[7], x[3]) and torch.equal(y[0], x[1]) and (y[1:7] == 0).all()


def test_many_pools_and_a_graph():
    """More pools than one launch takes, as one call and replayed from a graph."""
    N, page = 12, 16
    pools = [torch.randn(N, page, 1, 64, device="cuda") for _ in range(70)]
    old = [p.clone() for p in pools]
    t, lens, held, refs = i32([[4, 7, 0], [9, 0, 0]]), i32([20, 5]), i32([2, 1]), [0] * N
    for p in (4, 7, 9):
        refs[p] = 1
    outs = dict(table_out=torch.zeros_like(t), lens_out=torch.zeros_like(lens), held_out=torch.zeros_like(held), refs_out=i32([0] * N),
                workspace=torch.empty(1 << 16, dtype=torch.uint8, device="cuda"))
    refs_t, parents = i32(refs), i32([0, 0])
    graph = torch.cuda.CUDAGraph()
    C.attention_varlen_cache_fork(pools, t, lens, held, refs_t, parents, **outs)
    with torch.cuda.graph(graph):
        C.attention_varlen_cache_fork(pools, t, lens, held, refs_t, parents, **outs)
    for p, x in zip(pools, old):
        p.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    # row 1 shares page 4 and takes page 0 for the four tokens behind it; its own page 9 is free again
    assert outs["table_out"][:, :2].tolist() == [[4, 7], [4, 0]] and outs["lens_out"].tolist() == [20, 20]
    want = [0] * N
    want[4], want[7], want[0] = 2, 1, 1
    assert outs["refs_out"].tolist() == want
    for p, x in zip(pools, old):
        assert torch.equal(p[0, :4], x[7, :4]) and torch.equal(p[0, 4:], x[0, 4:]) and torch.equal(p[1:], x[1:])


def test_beams_over_a_growing_cache():
    """Fork, append to the children, attend: each row reads its own history (against rows kept apart)."""
    page, Hkv, d, Hq, N = 16, 1, 64, 8, 64
    kc, vc = (torch.zeros(N, page, Hkv, d, dtype=BF, device="cuda") for _ in range(2))
    R, W = 4, 8
    t, lens, held, refs = torch.zeros(R, W, dtype=torch.int32, device="cuda"), i32([0] * R), i32([0] * R), i32([0] * N)
    history = [[] for _ in range(R)]
    r, st = random.Random(3), status()
    g = torch.Generator(device="cuda").manual_seed(3)
    for step in range(30):
        parents = list(range(R)) if step == 0 else [r.randrange(R) for _ in range(R)]
        counts = [r.randint(1, 5) for _ in range(R)]
        C.attention_varlen_cache_fork([kc, vc], t, lens, held, refs, i32(parents), i32(counts), status=st)
        cu = i32([0] + [sum(counts[:i + 1]) for i in range(R)])
        k, v = (torch.randn(sum(counts), Hkv, d, device="cuda", generator=g).to(BF) for _ in range(2))
        q = torch.randn(R, Hq, d, device="cuda", generator=g).to(BF)
        new = torch.zeros_like(lens)
        C.attention_varlen_cache_append(k, v, kc, vc, t, lens, cu, lens_out=new, status=st)
        lens.copy_(new)
        out, _ = C.attention_varlen_cache_fwd(q, kc, vc, t, lens, i32(range(R + 1)), softcap=0.0, status=st)
        at = [sum(counts[:i]) for i in range(R)]
        history = [history[p] + [(k[at[i] + j], v[at[i] + j]) for j in range(counts[i])] for i, p in enumerate(parents)]
        if any(len(h) > W * page - 6 for h in history):
            break
        for i, h in enumerate(history):
            kk, vv = (torch.stack([x[n][0] for x in h]).double() for n in (0, 1))
            w = torch.softmax(q[i].double() @ kk.t() * 0.75 / 8, -1)
            assert float((w @ vv - out[i].double()).abs().max()) < 0.03
    assert int(st) == 0 and int((refs > 0).sum()) <= sum(held.tolist())
