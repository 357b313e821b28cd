"""CPU checks of the generation calls: what their C entry points and the Python
module refuse before anything reaches a device."""
import ctypes

import pytest
import torch

FAKE = 0x10000  # aligned, never touched: every case here fails its checks


@pytest.fixture(scope="module")
def lib():
    from ragged_gqa_attention_varlen_gb300 import _build, binding, cache

    _build.build()
    cache.load()
    return binding.load()


P, I, L, F, D, Z = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_size_t)


def call(lib, name, types, args):
    f = getattr(lib, name)
    f.restype = I
    return f(*(t(a) for t, a in zip(types, args, strict=True)))


def rotary(lib, **over):
    a = dict(dtype=(I, 1), total=(L, 4), Hq=(I, 8), Hkv=(I, 1), d=(I, 160), q=(P, FAKE), qts=(L, 1280), qhs=(L, 160),
             k=(P, FAKE), kts=(L, 160), khs=(L, 160), pos=(P, FAKE), axs=(L, 4), axes=(I, 1), freq=(P, FAKE),
             axis=(P, None), pairs=(I, 80), inter=(I, 0), inv=(I, 0), qo=(P, 0x10008), qots=(L, 1280), qohs=(L, 160),
             ko=(P, FAKE), kots=(L, 160), kohs=(L, 160), stream=(P, None))
    for k, v in over.items():
        a[k] = (a[k][0], v)
    return call(lib, "attn_varlen_rotary", [t for t, _ in a.values()], [v for _, v in a.values()])


def test_rotary_refusals(lib):
    assert rotary(lib) == -3                      # q_out not 16-byte aligned: the last check
    assert rotary(lib, dtype=5) == -1
    assert rotary(lib, d=96) == -2
    assert rotary(lib, pairs=81) == -1 and rotary(lib, pairs=0) == -1
    assert rotary(lib, axes=0) == -1
    assert rotary(lib, pos=None) == -1 and rotary(lib, freq=None) == -1
    assert rotary(lib, q=None) == -1 and rotary(lib, k=None) == -1
    assert rotary(lib, total=-1) == -1 and rotary(lib, total=1 << 31) == -1
    assert rotary(lib, qhs=164) == -3 and rotary(lib, khs=164) == -3
    assert rotary(lib, total=0) == 0              # nothing to do


PAGES = [("ps", L, 16 * 160), ("ss", L, 160), ("hs", L, 160)]


def append(lib, **over):
    a = dict(dtype=(I, 0), B=(I, 2), Hkv=(I, 1), d=(I, 160), total=(L, 3), k=(P, FAKE), kts=(L, 160), khs=(L, 160),
             v=(P, FAKE), vts=(L, 160), vhs=(L, 160))
    for c in ("kc", "vc"):
        a[c] = (P, FAKE)
        a.update({c + n: (t, v) for n, t, v in PAGES})
    a.update(pages=(I, 5), page=(I, 16), table=(P, FAKE), trs=(L, 2), width=(I, 2), lens=(P, FAKE), cu=(P, FAKE),
             pos=(P, FAKE), axs=(L, 3), axes=(I, 1), freq=(P, FAKE), axis=(P, None), pairs=(I, 80), inter=(I, 0),
             kp=(P, None), kprs=(L, 0), kphs=(L, 0), sc=(P, None), scrs=(L, 0), schs=(L, 0), lo=(P, 0x20000),
             st=(P, None), stream=(P, None))
    for k, v in over.items():
        a[k] = (a[k][0], v)
    return call(lib, "attn_varlen_cache_append", [t for t, _ in a.values()], [v for _, v in a.values()])


def test_append_refusals(lib):
    assert append(lib, khs=164) == -3
    assert append(lib, kc=FAKE + 8) == -3 and append(lib, vcss=162) == -3
    for page in (0, 8, 24, 2048):
        assert append(lib, page=page) == -2
    assert append(lib, pages=0) == -2
    assert append(lib, lo=FAKE) == -1             # lens_out is lens
    assert append(lib, table=None) == -1 and append(lib, cu=None) == -1 and append(lib, lens=None) == -1
    assert append(lib, width=0) == -1 and append(lib, trs=1) == -1
    assert append(lib, pairs=200) == -1 and append(lib, pos=None) == -1
    assert append(lib, B=20000) == -2 and append(lib, Hkv=5000) == -2
    assert append(lib, B=0) == -1 and append(lib, B=0, total=0) == 0


def read(lib, name, extra, **over):
    a = dict(dtype=(I, 0), B=(I, 2), P=(I, 0), Hq=(I, 16), Hkv=(I, 1), d=(I, 160), total=(L, 3), q=(P, FAKE),
             qts=(L, 2560), qhs=(L, 160), kc=(P, FAKE))
    a.update({"kc" + n: (t, v) for n, t, v in PAGES})
    if name == "attn_varlen_cache_fwd":
        a["vc"] = (P, FAKE)
        a.update({"vc" + n: (t, v) for n, t, v in PAGES})
    a.update(pages=(I, 5), page=(I, 16), table=(P, FAKE), trs=(L, 2), width=(I, 2), lens=(P, FAKE), pt=(P, None),
             prs=(L, 0), pw=(I, 0), pl=(P, None), cup=(P, None), cuq=(P, FAKE), qpos=(P, None), kp=(P, None),
             kprs=(L, 0), kphs=(L, 0), pkp=(P, None), pkprs=(L, 0), pkphs=(L, 0), slopes=(P, None), sbs=(L, 0),
             causal=(I, 0), wl=(I, -1), wr=(I, -1), cap=(F, 3.0), mult=(F, 0.75))
    a.update(extra)
    for k, v in over.items():
        a[k] = (a[k][0], v)
    return call(lib, name, [t for t, _ in a.values()], [v for _, v in a.values()])


def fwd(lib, **over):
    extra = dict(out=(P, FAKE), ots=(L, 2560), ohs=(L, 160), lse=(P, FAKE), ws=(P, FAKE), wsb=(Z, 0), st=(P, None),
                 stream=(P, None))
    return read(lib, "attn_varlen_cache_fwd", extra, **over)


def weights(lib, **over):
    extra = dict(lse=(P, FAKE), si=(P, None), sirs=(L, 0), sihs=(L, 0), so=(P, FAKE), sors=(L, 32), sohs=(L, 32),
                 psi=(P, None), psirs=(L, 0), psihs=(L, 0), pso=(P, None), psors=(L, 0), psohs=(L, 0), ws=(P, FAKE),
                 wsb=(Z, 0), st=(P, None), stream=(P, None))
    return read(lib, "attn_varlen_cache_weights", extra, **over)


@pytest.mark.parametrize("f", [fwd, weights])
def test_reading_refusals(lib, f):
    assert f(lib) == -4                            # all is well but the workspace
    assert f(lib, dtype=9) == -1 and f(lib, Hkv=3) == -1 and f(lib, Hkv=0) == -1
    assert f(lib, d=96) == -2 and f(lib, B=20000) == -2 and f(lib, P=20000) == -2
    assert f(lib, d=128) == -4 and f(lib, d=64) == -4
    assert f(lib, page=48) == -2 and f(lib, pages=0) == -2
    assert f(lib, q=None) == -1 and f(lib, kc=None) == -1 and f(lib, cuq=None) == -1 and f(lib, lse=None) == -1
    assert f(lib, kchs=4) == -3 and f(lib, q=FAKE + 2) == -3 and f(lib, qts=2564) == -3
    assert f(lib, P=1) == -1                       # a prefix without its table
    assert f(lib, kp=FAKE) == -1                   # key positions without the queries'
    assert f(lib, kp=FAKE, qpos=FAKE) == -4
    assert f(lib, slopes=FAKE, sbs=3) == -1 and f(lib, slopes=FAKE, sbs=0) == -4
    assert f(lib, cap=float("nan")) == -1 and f(lib, cap=float("inf")) == -1 and f(lib, mult=float("nan")) == -1
    assert f(lib, total=1 << 30) == -2
    assert f(lib, B=0) == -1 and f(lib, B=0, total=0) == 0
    assert f(lib, ws=FAKE + 64, wsb=1 << 40) == -4


def test_reading_refusals_of_outputs(lib):
    assert fwd(lib, out=None) == -1 and fwd(lib, ohs=12) == -3 and fwd(lib, vc=None) == -1
    assert fwd(lib, total=0) == 0
    assert weights(lib, so=None) == -1


def evict(lib, **over):
    a = dict(S=(I, 2), Hkv=(I, 1), d=(I, 160))
    for c in ("kc", "vc"):
        a[c] = (P, FAKE)
        a.update({c + n: (t, v) for n, t, v in PAGES})
    a.update(pages=(I, 5), page=(I, 16), table=(P, FAKE), trs=(L, 2), width=(I, 2), lens=(P, FAKE), sc=(P, FAKE),
             scrs=(L, 32), schs=(L, 32), kp=(P, FAKE), kprs=(L, 32), kphs=(L, 32), nxt=(P, FAKE), budget=(I, 8),
             recent=(I, 2), so=(P, FAKE), sors=(L, 32), sohs=(L, 32), po=(P, FAKE), pors=(L, 32), pohs=(L, 32),
             lo=(P, FAKE), ws=(P, FAKE), wsb=(Z, 0), st=(P, None), stream=(P, None))
    for k, v in over.items():
        a[k] = (a[k][0], v)
    return call(lib, "attn_varlen_cache_evict", [t for t, _ in a.values()], [v for _, v in a.values()])


def test_evict_refusals(lib):
    assert evict(lib) == -4
    assert evict(lib, budget=0) == -1 and evict(lib, recent=-1) == -1 and evict(lib, recent=9) == -1
    assert evict(lib, recent=8) == -4
    assert evict(lib, d=32) == -2 and evict(lib, page=17) == -2 and evict(lib, S=20000) == -2
    assert evict(lib, sc=None) == -1 and evict(lib, nxt=None) == -1 and evict(lib, lo=None) == -1
    assert evict(lib, sors=40) == -1               # in place means the same elements
    assert evict(lib, so=0x30000, sors=40) == -4
    assert evict(lib, kcss=12) == -3
    assert evict(lib, S=0) == 0


def test_outputs_with_shared_elements_are_refused(lib):
    """An expanded or overlapping output would keep whichever row came last."""
    # rotary (its last check is not reached): heads over one another, a token's rows reaching into the next, in place with other strides
    ok = dict(qo=0x40000, ko=0x80000, kots=160, kohs=160)
    assert rotary(lib, **ok, qots=1280, qohs=152) == -1 and rotary(lib, **ok, qots=1272) == -1
    assert rotary(lib, qo=0x40000, ko=0x80000, kots=152) == -1
    assert rotary(lib, qo=FAKE, qots=2560) == -1 and rotary(lib, qo=0x40000, kots=320) == -1
    # key positions or scores of several heads in one row, as of an expanded tensor
    two = dict(Hkv=2, kcss=320, kcps=16 * 320, vcss=320, vcps=16 * 320)
    assert append(lib, **two, kp=FAKE, kprs=32, kphs=0) == -1
    assert append(lib, **two, sc=FAKE, scrs=32, schs=32) == -1
    assert append(lib, **two, sc=FAKE, scrs=0, schs=32) == -1
    assert append(lib, Hkv=2) == -1                # a head's rows are the next slot's
    assert evict(lib, **two, scrs=64, sors=64, kprs=32, kphs=0, pors=32, pohs=0) == -1
    assert evict(lib, **two, scrs=64, sors=64, kprs=64, pors=64) == -4
    assert evict(lib, **two, scrs=32, schs=64, sors=32, sohs=64, kprs=64, pors=64) == -4   # [Hkv, S, slots]
    assert evict(lib, Hkv=2, scrs=64, sors=64, kprs=64, pors=64) == -1
    # key positions that are only read may be expanded
    assert evict(lib, **two, scrs=64, sors=64, kprs=32, kphs=0, po=0x30000, pors=64) == -4
    assert fwd(lib, ohs=152) == -1 and fwd(lib, ots=2552) == -1 and fwd(lib, ots=160, ohs=480) == -4
    assert weights(lib, Hkv=2, sors=32, sohs=0) == -1 and weights(lib, Hkv=2, sors=64) == -4
    assert weights(lib, si=FAKE, sirs=64) == -1 and weights(lib, si=0x30000, sirs=64) == -4
    prefix = dict(P=2, pt=FAKE, prs=1, pw=1, pl=FAKE, cup=FAKE, pso=FAKE, Hkv=2, sors=64)
    assert weights(lib, **prefix, psors=16, psohs=0) == -1 and weights(lib, **prefix, psors=32, psohs=16) == -4


def test_workspace_sizes(lib):
    f = lib.attn_varlen_cache_fwd_workspace_size
    f.argtypes, f.restype = [I, I, I, I, I, L], Z
    a, b = f(4, 0, 96, 1, 160, 4), f(4, 1, 96, 1, 160, 4)
    assert 0 < a < b and a % 256 == 0 and f(4, 0, 96, 1, 96, 4) == 0 and f(4, 0, 5, 2, 160, 4) == 0
    # every row may wait for its prefix: one fp32 row each for its own keys and the prefix's
    assert f(4, 1, 96, 1, 160, 1004) - b >= 1000 * 96 * 2 * 160 * 4
    e = lib.attn_varlen_cache_evict_workspace_size
    e.argtypes, e.restype = [I, I, I, I, I], Z
    assert e(4, 2, 10, 16, 20) > 0 and e(4, 2, 10, 16, 0) == 0 and e(4, 2, 10, 17, 5) == 0
    assert lib.attn_varlen_cache_weights_workspace_size() > 0


def test_python_calls_refuse_host_tensors(lib):
    """No CPU fallback: a call on host tensors raises before it looks further."""
    from ragged_gqa_attention_varlen_gb300 import cache as C
    x, pool = torch.zeros(2, 4, 64, dtype=torch.half), torch.zeros(3, 16, 1, 64, dtype=torch.half)
    i = torch.zeros(2, dtype=torch.int32)
    t, s = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1, 16)
    with pytest.raises(ValueError, match="CUDA"):
        C.attention_varlen_rotary(x, None, i, i.double())
    with pytest.raises(ValueError, match="CUDA"):
        C.attention_varlen_cache_append(x, x, pool, pool, t, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        C.attention_varlen_cache_fwd(x, pool, pool, t, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        C.attention_varlen_cache_weights(x, pool, t, i, i, x)
    with pytest.raises(ValueError, match="CUDA"):
        C.attention_varlen_cache_evict(pool, pool, t, i, s, s.int(), i, 4)
    with pytest.raises(ValueError, match="tensor"):
        C.attention_varlen_cache_fwd(None, pool, pool, t, i, i)


@pytest.mark.parametrize("f", [fwd, weights])
def test_key_positions_without_tokens(lib, f):
    """Without query tokens there are no positions of theirs to give."""
    prefix = dict(P=1, pt=FAKE, prs=1, pw=1, pl=FAKE, cup=FAKE)
    assert f(lib, kp=FAKE) == -1 and f(lib, **prefix, pkp=FAKE) == -1
    nothing = 0 if f is fwd else -4                # attention has nothing to do, weights has scores to copy
    assert f(lib, kp=FAKE, total=0, q=None) == nothing and f(lib, **prefix, pkp=FAKE, total=0) == nothing


def test_expanded_inputs_are_taken(lib):
    """Strides of 0 where rows are only read: q, k, v, and the tables of calls that read the pages."""
    for f in (fwd, weights):
        assert f(lib, trs=0) == -4 and f(lib, qts=0, qhs=0) == -4 and f(lib, trs=-1) == -1 and f(lib, qts=-8) == -3
        assert f(lib, P=2, pt=FAKE, prs=0, pw=4, pl=FAKE, cup=FAKE) == -4
        assert f(lib, kcss=0) == -3                # (a pool has its rows)
    shared = dict(qts=0, khs=0, qo=0x40000, ko=0x80000)
    assert rotary(lib, **shared, kots=152) == -1 and rotary(lib, **shared, qohs=0) == -3
    assert append(lib, trs=0) == -1 and evict(lib, trs=0) == -1   # pages that are written belong to one row
    assert append(lib, kts=0, vhs=0, sc=FAKE, scrs=0, schs=0) == -1 and append(lib, kts=-160) == -3
