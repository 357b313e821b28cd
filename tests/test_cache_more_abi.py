"""CPU checks of norms with rotation, the 8-bit cache and the calls that move pages: what
their C entry points and the Python module refuse before anything reaches a device."""
import ctypes

import pytest
import torch

from test_cache_abi import FAKE, D, F, I, L, P, Z, call, lib  # noqa: F401


class Pool(ctypes.Structure):
    _fields_ = [("base", P), ("page", L), ("row", L), ("piece", L), ("rows", ctypes.c_int32), ("pieces", ctypes.c_int32), ("bytes", ctypes.c_int32)]


def run(lib, name, a, over):
    for k, v in over.items():
        a[k] = (a[k][0], v)
    return call(lib, name, [t for t, _ in a.values()], [v for _, v in a.values()])


ROTARY = dict(pos=(P, FAKE), axs=(L, 4), axes=(I, 1), freq=(P, FAKE), axis=(P, None), pairs=(I, 80), inter=(I, 0))


def norm(lib, **over):
    a = dict(dtype=(I, 1), total=(L, 4), Hq=(I, 8), Hkv=(I, 1), d=(I, 160), q=(P, FAKE), qts=(L, 1280), qhs=(L, 160), k=(P, FAKE),
             kts=(L, 160), khs=(L, 160), qw=(P, FAKE), kw=(P, FAKE), eps=(F, 1e-6), **ROTARY, qo=(P, 0x10008), qots=(L, 1280), qohs=(L, 160),
             ko=(P, 0x40000), kots=(L, 160), kohs=(L, 160), stream=(P, None))
    return run(lib, "attn_varlen_norm_rotary", a, over)


def norm_bwd(lib, **over):
    a = dict(dtype=(I, 1), total=(L, 4), Hq=(I, 8), Hkv=(I, 1), d=(I, 160))
    for n in ("dqo", "dko", "q", "k"):
        s = 1280 if "q" in n else 160
        a.update({n: (P, FAKE), n + "ts": (L, s), n + "hs": (L, 160)})
    a.update(qw=(P, FAKE), kw=(P, FAKE), eps=(F, 1e-6), **ROTARY)
    for n in ("dq", "dk"):
        s = 1280 if "q" in n else 160
        a.update({n: (P, 0x40000), n + "ts": (L, s), n + "hs": (L, 160)})
    a.update(dqw=(P, 0x50000), dkw=(P, 0x60000), ws=(P, FAKE), wsb=(Z, 0), stream=(P, None))
    return run(lib, "attn_varlen_norm_rotary_bwd", a, over)


def test_norm_refusals(lib):
    assert norm(lib) == -3                      # q_out not 16-byte aligned: the last check
    for f, good in ((norm, -3), (norm_bwd, -4)):
        assert f(lib) == good
        assert f(lib, dtype=5) == -1 and f(lib, d=96) == -2 and f(lib, Hq=0) == -1 and f(lib, Hkv=-1) == -1
        assert f(lib, total=-1) == -1 and f(lib, total=1 << 31) == -1 and f(lib, Hq=65535) == -2
        assert f(lib, eps=-1.0) == -1 and f(lib, eps=float("nan")) == -1 and f(lib, eps=float("inf")) == -1
        assert f(lib, pairs=81) == -1 and f(lib, pairs=0) == -1 and f(lib, axes=0) == -1 and f(lib, pos=None) == -1
        assert f(lib, freq=None, pos=None, pairs=0, axes=0) == good      # no turn: its arguments are not looked at
        assert f(lib, q=None) == -1 and f(lib, qhs=164) == -3 and f(lib, qw=FAKE + 2, **({"qo": 0x40000} if f is norm else {})) == -3
    assert norm(lib, qo=0x40000, k=None) == -1 and norm(lib, qo=0x40000, khs=164) == -3
    assert norm(lib, qo=0x40000, qots=0) == -3 and norm(lib, qo=0x40000, qohs=0) == -3 and norm(lib, qo=0x40000, qots=640) == -1
    assert norm(lib, total=0) == 0
    assert norm_bwd(lib, total=0, dqw=None, dkw=None) == 0 and norm_bwd(lib, total=0) == -4
    assert norm_bwd(lib, dq=None) == -1 and norm_bwd(lib, dqo=None) == -1 and norm_bwd(lib, dqw=0x60000) == -1
    assert norm_bwd(lib, Hkv=0) == -1           # the gradient of a weight without rows
    assert norm_bwd(lib, dq=FAKE, dqts=1288) == -1  # in place with other strides
    lib.attn_varlen_norm_rotary_bwd_workspace_size.restype = Z
    size = lib.attn_varlen_norm_rotary_bwd_workspace_size
    assert size(L(0), I(1), I(0), I(64)) >= 256 and size(L(-1), I(1), I(0), I(64)) == 0 and size(L(4), I(1), I(0), I(96)) == 0


PAGES8 = [("ps", 16 * 160), ("ss", 160), ("hs", 160)]
SCALES = [("ps", 1), ("bs", 1), ("hs", 1)]


def append8(lib, **over):
    a = dict(dtype=(I, 0), B=(I, 2), Hkv=(I, 1), d=(I, 160), total=(L, 3), k=(P, FAKE), kts=(L, 160), khs=(L, 160), v=(P, FAKE), vts=(L, 160),
             vhs=(L, 160))
    for i, c in enumerate(("kc", "vc")):
        a[c] = (P, FAKE + 0x1000 * i)
        a.update({c + n: (L, v) for n, v in PAGES8})
    for i, c in enumerate(("ks", "vs")):
        a[c] = (P, FAKE + 0x1000 * i)
        a.update({c + n: (L, v) for n, v in SCALES})
    a.update(pages=(I, 5), page=(I, 16), block=(I, 16), table=(P, FAKE), trs=(L, 2), width=(I, 2), lens=(P, FAKE), cu=(P, FAKE), **ROTARY,
             norm=(I, 1), kw=(P, FAKE), eps=(F, 1e-6), kp=(P, None), kprs=(L, 0), kphs=(L, 0), lo=(P, 0x20000), st=(P, None), stream=(P, None))
    return run(lib, "attn_varlen_cache8_append", a, over)


def test_append8_refusals(lib):
    assert append8(lib, khs=164) == -3
    assert append8(lib, kcss=168) == -3 and append8(lib, kc=FAKE + 8) == -3    # 16 elements, not 8
    for page in (0, 8, 24, 2048):
        assert append8(lib, page=page) == -2
    for block in (0, 8, 24, 32, 256):
        assert append8(lib, block=block) == -2
    assert append8(lib, page=256, block=256) == -2
    assert append8(lib, ks=None) == -1 and append8(lib, vs=None) == -1 and append8(lib, ks=FAKE + 2) == -3 and append8(lib, ksps=-1) == -3
    assert append8(lib, ksps=0) == -1 and append8(lib, kcps=160) == -1         # shared by pages
    assert append8(lib, vc=FAKE) == -1 and append8(lib, vs=FAKE) == -1         # K's own pool
    assert append8(lib, eps=-1.0) == -1 and append8(lib, eps=-1.0, norm=0, khs=164) == -3
    assert append8(lib, lo=FAKE) == -1 and append8(lib, table=None) == -1 and append8(lib, cu=None) == -1 and append8(lib, trs=1) == -1
    assert append8(lib, pairs=200) == -1 and append8(lib, B=20000) == -2 and append8(lib, Hkv=5000) == -2
    assert append8(lib, kp=FAKE, kprs=3, kphs=3) == -1
    assert append8(lib, B=0) == -1 and append8(lib, B=0, total=0) == 0


def fwd8(lib, **over):
    a = dict(dtype=(I, 0), B=(I, 2), P=(I, 0), Hq=(I, 16), Hkv=(I, 1), d=(I, 160), total=(L, 3), q=(P, FAKE), qts=(L, 2560), qhs=(L, 160))
    for c in ("kc", "vc"):
        a[c] = (P, FAKE)
        a.update({c + n: (L, v) for n, v in PAGES8})
    for c in ("ks", "vs"):
        a[c] = (P, FAKE)
        a.update({c + n: (L, v) for n, v in SCALES})
    a.update(pages=(I, 5), page=(I, 16), block=(I, 16), table=(P, FAKE), trs=(L, 2), width=(I, 2), lens=(P, FAKE), pt=(P, None), prs=(L, 0),
             pw=(I, 0), pl=(P, None), cup=(P, None), cuq=(P, FAKE), qpos=(P, None), kp=(P, None), kprs=(L, 0), kphs=(L, 0), pkp=(P, None),
             pkprs=(L, 0), pkphs=(L, 0), slopes=(P, None), sbs=(L, 0), causal=(I, 0), wl=(I, -1), wr=(I, -1), cap=(F, 3.0), mult=(F, 0.75),
             out=(P, FAKE), ots=(L, 2560), ohs=(L, 160), lse=(P, FAKE), ws=(P, FAKE), wsb=(Z, 0), st=(P, None), stream=(P, None))
    return run(lib, "attn_varlen_cache8_fwd", a, over)


def test_fwd8_refusals(lib):
    assert fwd8(lib) == -4                         # all is well but the workspace
    assert fwd8(lib, dtype=9) == -1 and fwd8(lib, Hkv=3) == -1 and fwd8(lib, d=96) == -2 and fwd8(lib, B=20000) == -2
    assert fwd8(lib, page=48) == -2 and fwd8(lib, pages=0) == -2 and fwd8(lib, block=32) == -2 and fwd8(lib, block=8) == -2
    assert fwd8(lib, kcss=168) == -3 and fwd8(lib, vc=FAKE + 8) == -3 and fwd8(lib, qhs=164) == -3
    assert fwd8(lib, ks=None) == -1 and fwd8(lib, vs=None) == -1 and fwd8(lib, ks=FAKE + 1) == -3 and fwd8(lib, vsbs=-1) == -3
    assert fwd8(lib, ksps=0) == -4                 # scales that pages share may be read
    assert fwd8(lib, P=1) == -1 and fwd8(lib, kp=FAKE) == -1 and fwd8(lib, kp=FAKE, qpos=FAKE) == -4
    assert fwd8(lib, cap=float("nan")) == -1 and fwd8(lib, total=1 << 30) == -2
    assert fwd8(lib, out=None) == -1 and fwd8(lib, ohs=12) == -3 and fwd8(lib, total=0) == 0
    assert fwd8(lib, B=0) == -1 and fwd8(lib, B=0, total=0) == 0


def pool(**over):
    a = dict(base=FAKE, page=16 * 128, row=128, piece=128, rows=16, pieces=1, bytes=128)
    a.update(over)
    return Pool(**a)


def fork(lib, pools=None, **over):
    pools = [pool()] if pools is None else pools
    arr = (Pool * max(1, len(pools)))(*pools)
    a = dict(rows=(I, 3), pages=(I, 9), page=(I, 16), pools=(P, ctypes.addressof(arr)), n=(I, len(pools)), table=(P, 0x10000), trs=(L, 4), W=(I, 4),
             lens=(P, 0x11000), held=(P, 0x12000), refs=(P, 0x13000), parents=(P, 0x14000), room=(P, 0x15000), to=(P, 0x10000), tors=(L, 4),
             lo=(P, 0x11000), ho=(P, 0x12000), ro=(P, 0x13000), ws=(P, 0x20000), wsb=(Z, 0), st=(P, None), stream=(P, None))
    return run(lib, "attn_varlen_cache_fork", a, over)


def test_fork_refusals(lib):
    assert fork(lib) == -4 and fork(lib, pools=[], page=16) == -4
    assert fork(lib, rows=-1) == -1 and fork(lib, pages=0) == -1 and fork(lib, W=0) == -1
    assert fork(lib, rows=20000) == -2 and fork(lib, page=24) == -2 and fork(lib, W=1 << 27, trs=1 << 27, tors=1 << 27) == -2
    for name in ("table", "lens", "held", "refs", "parents", "to", "lo", "ho", "ro"):
        assert fork(lib, **{name: None}) == -1, name
    assert fork(lib, trs=3) == -1 and fork(lib, tors=3) == -1 and fork(lib, tors=5) == -1 and fork(lib, to=0x40000, tors=5) == -4
    assert fork(lib, lo=0x12000) == -1 and fork(lib, ho=0x14000) == -1 and fork(lib, room=0x11000) == -1 and fork(lib, room=None) == -4
    for bad, want in ((dict(base=None), -1), (dict(rows=0), -1), (dict(rows=32), -1), (dict(rows=3), -1), (dict(bytes=0), -1), (dict(bytes=126), -3),
                      (dict(base=FAKE + 2), -3), (dict(row=130), -3), (dict(page=-2048), -3), (dict(page=128), -1), (dict(row=0), -1),
                      (dict(bytes=1 << 30, row=1 << 30, page=1 << 40), -2), (dict(rows=1, bytes=4, page=4, row=4, piece=4), -4)):
        assert fork(lib, pools=[pool(), pool(**bad)]) == want, bad
    assert fork(lib, n=-1) == -1 and fork(lib, n=1, pools=[pool()], ws=0x20010, wsb=1 << 30) == -4
    lib.attn_varlen_cache_fork_workspace_size.restype = Z
    size = lib.attn_varlen_cache_fork_workspace_size
    assert size(I(3), I(4), I(9)) > 0 and size(I(-1), I(4), I(9)) == 0 and size(I(16384), I(1 << 20), I(9)) == 0


def test_fork_refuses_outputs_that_meet_other_arrays(lib):
    for out, at in (("ro", 0x14000), ("ro", 0x15000), ("ro", 0x11000 - 4), ("lo", 0x14000 + 8), ("ho", 0x15000), ("to", 0x14000),
                    ("lo", 0x13000 + 32), ("to", 0x10004), ("to", 0x12000 - 44), ("ho", 0x11000 + 8)):
        assert fork(lib, **{out: at}) == -1, (out, hex(at))
    for out, at in (("ro", 0x14000 + 12), ("ro", 0x14000 - 36), ("to", 0x12000 - 48), ("lo", 0x13000 + 36), ("to", 0x70000)):
        assert fork(lib, **{out: at}) == -4, (out, hex(at))      # side by side


def compact(lib, pools=None, **over):
    pools = [pool()] if pools is None else pools
    arr = (Pool * max(1, len(pools)))(*pools)
    a = dict(pages=(I, 9), page=(I, 16), pools=(P, ctypes.addressof(arr)), n=(I, len(pools)), rows=(I, 3), table=(P, 0x10000), trs=(L, 4), W=(I, 4),
             held=(P, 0x12000), to=(P, 0x10000), tors=(L, 4), prows=(I, 2), ptable=(P, 0x30000), prs=(L, 4), pW=(I, 4), pheld=(P, 0x31000),
             pto=(P, 0x30000), ptors=(L, 4), refs=(P, 0x13000), ro=(P, 0x13000), live=(P, 0x14000), ws=(P, 0x20000), wsb=(Z, 0), st=(P, None),
             stream=(P, None))
    return run(lib, "attn_varlen_cache_compact", a, over)


def test_compact_and_copy_refusals(lib):
    assert compact(lib) == -4 and compact(lib, prows=0, ptable=None) == -4 and compact(lib, rows=0, table=None) == -4
    assert compact(lib, pages=0) == -1 and compact(lib, page=12) == -2 and compact(lib, rows=-1) == -1 and compact(lib, rows=20000) == -2
    for name in ("table", "held", "to", "ptable", "pheld", "pto", "refs", "ro", "live"):
        assert compact(lib, **{name: None}) == -1, name
    assert compact(lib, trs=3) == -1 and compact(lib, tors=6) == -1 and compact(lib, ptors=3) == -1
    assert compact(lib, pools=[pool(row=0)]) == -1
    for out, at in (("pto", 0x10000), ("to", 0x30000), ("ro", 0x12000), ("live", 0x13000 + 32), ("live", 0x12000), ("ro", 0x31000 - 8),
                    ("to", 0x13000), ("live", 0x10000 + 44)):
        assert compact(lib, **{out: at}) == -1, (out, hex(at))
    assert compact(lib, live=0x13000 + 36) == -4 and compact(lib, pto=0x30000 + 32) == -4
    assert compact(lib, ptable=0x10000, pto=0x50000, to=0x60000) == -4      # one table twice, read

    def copy(src=None, dst=None, **over):
        src, dst = (Pool * 1)(src or pool()), (Pool * 1)(dst or pool(base=0x50000))
        a = dict(count=(I, 2), s=(P, FAKE), d=(P, FAKE), sp=(I, 9), dp=(I, 4), page=(I, 16), src=(P, ctypes.addressof(src)), dst=(P, ctypes.addressof(dst)),
                 n=(I, 1), st=(P, None), stream=(P, None))
        return run(lib, "attn_varlen_cache_copy", a, over)

    assert copy(count=0) == 0 and copy(n=0) == 0 and copy(count=-1) == -1 and copy(s=None) == -1 and copy(sp=0) == -1 and copy(page=20) == -2
    assert copy(dst=pool(base=0x50000, bytes=64)) == -1 and copy(dst=pool(base=0x50000, rows=8)) == -1
    assert copy(dst=pool(base=0x50000, row=64)) == -1                        # rows that overlap where they are written
    assert copy(dst=pool(row=256, page=4096)) == -1                          # one base, other strides


def test_python_refusals(lib):
    """Tensors on the CPU never reach the library."""
    from ragged_gqa_attention_varlen_gb300 import cache as C
    q, w, i = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(64), torch.zeros(2, dtype=torch.int32)
    k8 = torch.zeros(3, 16, 4, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.zeros(3, 1, 4)
    with pytest.raises(ValueError, match="CUDA"):
        C.attention_varlen_norm_rotary(q, None, w)
    with pytest.raises(ValueError, match="CUDA"):
        C.attention_varlen_norm_rotary_bwd(q, None, q, None, w)
    with pytest.raises(ValueError, match="CUDA"):
        C.attention_varlen_cache8_fwd(q, k8, k8, s, s, i[None], i[:1], i)
    with pytest.raises(ValueError, match="CUDA"):
        C.attention_varlen_cache8_append(q, q, k8, k8, s, s, i[None], i[:1], i)
    with pytest.raises(ValueError, match="CUDA"):
        C.attention_varlen_cache_fork([q[None]], i[None], i[:1], i[:1], i, i[:1])
    with pytest.raises(ValueError, match="CUDA"):
        C.attention_varlen_cache_compact([q[None]], i[None], i[:1], i)
    with pytest.raises(ValueError, match="CUDA"):
        C.attention_varlen_cache_copy([q[None]], i, i)
    with pytest.raises(ValueError, match="tensor"):
        C.attention_varlen_norm_rotary(None, None)
