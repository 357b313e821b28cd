"""Forks of tables whose pages are counted wrongly, on the GPU: nothing changes."""
import pytest
import torch

from ragged_gqa_attention_varlen_gb300 import cache as C
from test_cache_gpu import i32, lib, status  # noqa: F401
from test_cache_pages_gpu import bits, world

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", ["held_but_free", "dropped_but_free", "two_holders_one_counted", "two_holders_one_dropped"])
@pytest.mark.parametrize("R,inplace", [(9, False), (9, True), (900, True)])
def test_fork_refuses_pages_with_more_holders_than_counts(what, R, inplace):
    """A page that a row holds must not be given to another, nor its count pass below 0."""
    w = world(11, R, 16, 120, spare=4 * R, width=14, shared=False)
    lens, held, refs, parents, room = list(w["lens"]), list(w["held"]), list(w["refs"]), list(range(R)), [20] * R
    t = w["t"].clone()
    row = max(range(R), key=lambda i: min(lens[i] // 16, held[i]))
    other = next(i for i in range(R) if i != row and lens[i] >= 16)
    if what.startswith("two_holders"):
        t[other, 0] = t[row, 0]  # (its count stays 1)
    else:
        refs[w["table"][row][0]] = 0
    if what.startswith("dropped") or what.endswith("dropped"):
        parents[row] = -1
    a, b, c = i32(lens), i32(held), i32(refs)
    old, t0 = [x.clone() for x in bits(w["pools"])], t.clone()
    outs = {} if inplace else dict(table_out=torch.full_like(t, -4), lens_out=torch.zeros_like(a), held_out=torch.zeros_like(b), refs_out=torch.zeros_like(c))
    st = status()
    got = C.attention_varlen_cache_fork(w["pools"], t, a, b, c, i32(parents), i32(room), status=st, **outs)
    torch.cuda.synchronize()
    assert int(st) == C.DEV_BAD_CACHE
    assert torch.equal(got[0], t0) and got[1].tolist() == lens and got[2].tolist() == held and got[3].tolist() == refs
    assert all(torch.equal(x, y) for x, y in zip(bits(w["pools"]), old))


def test_fork_of_pages_that_others_hold_too():
    """More counts than holders in the table (prefix tables) are as before: such pages are not given away."""
    N, page = 6, 16
    pool = torch.randn(N, page, 1, 64, device="cuda")
    st = status()
    t, lens, held, refs = i32([[3, 0], [5, 0]]), i32([16, 16]), i32([1, 1]), i32([2, 0, 0, 3, 0, 1])
    C.attention_varlen_cache_fork([pool], t, lens, held, refs, i32([-1, 1]), i32([0, 16]), status=st)
    torch.cuda.synchronize()
    assert int(st) == 0 and refs.tolist() == [2, 1, 0, 2, 0, 1] and t[1].tolist() == [5, 1] and held.tolist() == [0, 2]


def test_beams_with_key_positions():
    """Children of a row whose slots stand in another order read their parent's positions once the
    caller has taken them along, as the documentation says."""
    page, Hkv, d, Hq, N = 16, 1, 64, 4, 12
    g = torch.Generator(device="cuda").manual_seed(5)
    kc, vc = (torch.randn(N, page, Hkv, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    t, lens, held = i32([[3, 7, 0], [9, 0, 0], [4, 0, 0]]), i32([20, 5, 9]), i32([2, 1, 1])
    refs = i32([0, 0, 0, 1, 1, 0, 0, 1, 0, 1, 0, 0])
    key_pos = torch.stack([torch.randperm(48, device="cuda", generator=g) for _ in range(3)]).int()[:, None].contiguous()
    q = torch.randn(3, Hq, d, device="cuda", generator=g).to(torch.bfloat16)
    slopes = torch.full((3, Hq), 0.3, device="cuda")

    def attend(positions):
        return C.attention_varlen_cache_fwd(q[:1].expand(3, Hq, d).contiguous(), kc, vc, t, lens, i32([0, 1, 2, 3]), slopes, key_pos=positions,
                                            q_pos=i32([30] * 3), window_left=25, window_right=0)[0]

    want = attend(key_pos)[:1].clone()
    parents = i32([0, 0, 0])
    C.attention_varlen_cache_fork([kc, vc], t, lens, held, refs, parents)
    got = attend(key_pos[parents.long()].contiguous())
    assert all(torch.equal(got[r:r + 1], want) for r in range(3))
    assert not torch.equal(attend(key_pos)[1:2], want)  # (left behind, they are the old row's)
