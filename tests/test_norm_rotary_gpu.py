"""Norms of queries and keys with rotation, and their gradients, on the GPU against plain
64-bit forms (cache8_ref), with tolerances from the roundings."""
import pytest
import torch

import cache8_ref as ref8
import cache_ref as ref
from ragged_gqa_attention_varlen_gb300 import cache as C
from test_cache_gpu import BF, HF, lib, normal, within  # noqa: F401

pytestmark = pytest.mark.gpu

FORMS = [pytest.param(*x, id="-".join(map(str, x))) for x in [
    # T, Hq, Hkv, d, pairs (0: no turn), axes, interleaved, dtype, far
    (1, 1, 0, 64, 32, 1, False, "bf16", 100), (3, 96, 1, 160, 80, 3, False, "bf16", 1 << 20), (77, 5, 5, 64, 16, 2, False, "fp16", 5000),
    (130, 32, 8, 128, 48, 2, True, "fp16", 1 << 29), (33, 12, 3, 128, 63, 3, False, "bf16", 4000), (33, 12, 3, 128, 63, 3, True, "fp16", 4000),
    (50, 7, 1, 160, 1, 1, False, "fp16", 90), (2000, 3, 1, 160, 79, 3, True, "bf16", 1 << 20), (9, 300, 2, 64, 30, 1, True, "bf16", 70000),
    (700, 80, 1, 160, 80, 1, True, "fp16", 4000), (41, 2, 9, 128, 0, 1, False, "bf16", 1), (300, 48, 1, 64, 0, 1, False, "fp16", 1),
    (5, 1000, 1, 64, 32, 1, False, "bf16", 900)]]


def make(T, Hq, Hkv, d, pairs, axes, dtype, far):
    dt = BF if dtype == "bf16" else HF
    g = torch.Generator().manual_seed(3)
    q = normal(1, T, Hq + 1, d + 8, dtype=dt, std=3.0)[:, :Hq, :d]
    k = normal(2, T, Hkv, d, dtype=dt, std=0.2) if Hkv else None
    qw, kw = (torch.randn(d, generator=g).cuda(), (torch.rand(d, generator=g) + 0.5).cuda() if Hkv else None)
    pos = torch.randint(0, far, (axes, T), generator=g, dtype=torch.int32).cuda()
    inv = axis = None
    if pairs:
        inv = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).cuda()
        axis = None if axes == 1 else torch.randint(0, axes, (pairs,), generator=g, dtype=torch.int32).cuda()
    return dt, q, k, qw, kw, pos if pairs else None, inv, axis


@pytest.mark.parametrize("T,Hq,Hkv,d,pairs,axes,interleaved,dtype,far", FORMS)
def test_forward(T, Hq, Hkv, d, pairs, axes, interleaved, dtype, far):
    dt, q, k, qw, kw, pos, inv, axis = make(T, Hq, Hkv, d, pairs, axes, dtype, far)
    eps = 1e-5
    got = C.attention_varlen_norm_rotary(q, k, qw, kw, pos, inv, axis, interleaved, eps)
    for x, w, y in ((q, qw, got[0]), (k, kw, got[1])):
        if x is None:
            assert y is None
            continue
        n, _ = ref8.normed(x, w, eps)
        want, mag = ref8.turned(n, pos, inv, axis, interleaved)
        # one rounding of the result, and fp32 arithmetic: the sum of d squares and the norm a few
        # steps of 2^-23, sine and cosine 2^-21
        within("normed", y, want, ref.UNIT[dt] * want.abs() + mag * 2.0 ** -19 + 2.0 ** -25)
    a, b = q.clone(), None if k is None else k.clone()
    C.attention_varlen_norm_rotary(a, b, qw, kw, pos, inv, axis, interleaved, eps, q_out=a, k_out=b)
    assert torch.equal(a, got[0]) and (b is None or torch.equal(b, got[1]))
    # without weights they are ones
    plain = C.attention_varlen_norm_rotary(q, None, None, None, pos, inv, axis, interleaved, eps)[0]
    ones = C.attention_varlen_norm_rotary(q, None, torch.ones(d, device="cuda"), None, pos, inv, axis, interleaved, eps)[0]
    assert torch.equal(plain, ones)


@pytest.mark.parametrize("T,Hq,Hkv,d,pairs,axes,interleaved,dtype,far", FORMS)
def test_backward(T, Hq, Hkv, d, pairs, axes, interleaved, dtype, far):
    dt, q, k, qw, kw, pos, inv, axis = make(T, Hq, Hkv, d, pairs, axes, dtype, far)
    eps = 1e-5
    dq, dk = normal(7, T, Hq, d + 8, dtype=dt)[..., :d], normal(8, T, Hkv, d, dtype=dt) if Hkv else None
    got = C.attention_varlen_norm_rotary_bwd(dq, dk, q, k, qw, kw, pos, inv, axis, interleaved, eps)
    for x, w, dy, dx, dw in ((q, qw, dq, got[0], got[2]), (k, kw, dk, got[1], got[3])):
        if x is None:
            assert dx is None and dw is None
            continue
        wd, xd = w.cpu().double(), x.cpu().double()
        g, mag = ref8.turned(dy.cpu().double(), pos, inv, axis, interleaved, inverse=True)
        _, r = ref8.normed(x, None, eps)
        xhat = xd * r
        h = g * wd
        mean = (h * xhat).mean(-1, keepdim=True)
        want = r * (h - xhat * mean)
        # fp32: g is off by mag 2^-20, everything else by a few steps of its magnitudes
        slack = r * (mag * wd.abs() + xhat.abs() * (mag * wd.abs() * xhat.abs()).mean(-1, keepdim=True)) * 2.0 ** -19
        within("dx", dx, want, ref.UNIT[dt] * want.abs() + slack + 2.0 ** -25)
        terms = mag * xhat.abs()
        # a sum of n terms in parts: each part's additions are off by half a step of what it holds, at
        # most n / 600 + 60 additions in a row (the lanes' rows, then lanes, warps and blocks)
        rows = T * x.shape[1]
        within("dw", dw, (g * xhat).sum((0, 1)), terms.sum((0, 1)) * (2.0 ** -19 + (rows / 600 + 60) * 2.0 ** -24) + 2.0 ** -25)
    again = C.attention_varlen_norm_rotary_bwd(dq, dk, q, k, qw, kw, pos, inv, axis, interleaved, eps)
    assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(got, again))
    a, b = dq.clone(), None if dk is None else dk.clone()
    C.attention_varlen_norm_rotary_bwd(a, b, q, k, qw, kw, pos, inv, axis, interleaved, eps, dq=a, dk=b)
    assert torch.equal(a, got[0]) and (b is None or torch.equal(b, got[1]))
    assert C.attention_varlen_norm_rotary_bwd(dq, dk, q, k, None, None, pos, inv, axis, interleaved, eps)[2:] == (None, None)


def test_backward_is_the_gradient():
    """Against central differences of the 64-bit form, in directions of x and of the weights."""
    T, H, d, n, eps = 6, 3, 128, 40, 1e-2
    x, y = normal(1, T, H, d, dtype=HF), normal(2, T, H, d, dtype=HF)
    w = (torch.rand(d, generator=torch.Generator().manual_seed(1)) + 0.5).cuda()
    pos = torch.randint(0, 9999, (2, T), dtype=torch.int32, device="cuda")
    inv = (10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)).cuda()
    axis = (torch.arange(n, device="cuda") % 2).int()
    dx, _, dw, _ = C.attention_varlen_norm_rotary_bwd(y, None, x, None, w, None, pos, inv, axis, eps=eps)
    yd = y.cpu().double()

    def f(xx, ww):
        return float((ref8.turned(ref8.normed(xx, ww, eps)[0], pos, inv, axis, False)[0] * yd).sum())

    r = torch.Generator().manual_seed(5)
    x64, w64, step = x.cpu().double(), w.cpu().double(), 1e-4
    for _ in range(6):
        v, u = torch.randn(T, H, d, generator=r, dtype=torch.float64), torch.randn(d, generator=r, dtype=torch.float64)
        # the second-order difference's error is step^2 times a third derivative of order the values' own sum
        diff = (f(x64 + step * v, w64) - f(x64 - step * v, w64)) / (2 * step)
        tol = float((v.abs() * (dx.cpu().double().abs() * 2.0 ** -11 + 2.0 ** -18)).sum()) + 1e-4
        assert abs(diff - float((dx.cpu().double() * v).sum())) <= tol
        diff = (f(x64, w64 + step * u) - f(x64, w64 - step * u)) / (2 * step)
        assert abs(diff - float((dw.cpu().double() * u).sum())) <= 1e-3


def test_rows_of_zeros_and_no_rows():
    """A row of zeros stays zero and has a finite gradient; no rows: the weights' gradients are zeros."""
    q = torch.zeros(3, 2, 64, dtype=BF, device="cuda")
    q[1] = 1.0
    out, _ = C.attention_varlen_norm_rotary(q, None, eps=1e-6)
    assert (out[0] == 0).all() and (out[1] == 1).all()
    w = torch.ones(64, device="cuda")
    dq, _, dw, _ = C.attention_varlen_norm_rotary_bwd(torch.ones_like(q), None, q, None, w, None, eps=1e-6)
    assert torch.isfinite(dq).all() and float((dq[0].float() - 1000.0).abs().max()) <= 4
    none = q[:0]
    dq, dk, dw, dkw = C.attention_varlen_norm_rotary_bwd(none, none, none, none, w, w, dq_weight=torch.full_like(w, 3.0))
    assert dq.shape == none.shape and (dw == 0).all() and (dkw == 0).all()


def test_captured_on_other_streams_and_in_a_graph():
    dt, q, k, qw, kw, pos, inv, axis = make(300, 32, 8, 128, 64, 1, "bf16", 5000)
    dq, dk = torch.randn_like(q), torch.randn_like(k)
    want = C.attention_varlen_norm_rotary_bwd(dq, dk, q, k, qw, kw, pos, inv, axis)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = C.attention_varlen_norm_rotary_bwd(dq, dk, q, k, qw, kw, pos, inv, axis, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [torch.empty_like(x) for x in want]
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        C.attention_varlen_norm_rotary_bwd(dq, dk, q, k, qw, kw, pos, inv, axis, dq=outs[0], dk=outs[1], dq_weight=outs[2], dk_weight=outs[3], workspace=ws)
    for _ in range(2):
        for o in outs:
            o.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_expanded_inputs():
    """Rows that share memory (a gradient of a sum) are read as they are."""
    q = normal(1, 1, 1, 128).expand(70, 6, 128)
    dy = normal(2, 1, 6, 128).expand(70, 6, 128)
    w = torch.ones(128, device="cuda")
    a = C.attention_varlen_norm_rotary_bwd(dy, None, q, None, w, None)
    b = C.attention_varlen_norm_rotary_bwd(dy.contiguous(), None, q.contiguous(), None, w, None)
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
    with pytest.raises(C.AttnError):
        C.attention_varlen_norm_rotary(q, None, q_out=torch.empty(1, 6, 128, dtype=BF, device="cuda").expand(70, 6, 128))


def test_heads_far_apart():
    """Head-major rows more than 2^32 elements apart, in place: the bits of packed ones."""
    T, H, d, far = 70, 2, 64, 2 ** 32 + 64
    pos, inv = torch.arange(T, dtype=torch.int32, device="cuda") * 37, (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).cuda()
    q, dy = (torch.randn(T, H, d, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda() for i in (1, 2))
    w = torch.linspace(0.5, 1.5, d, device="cuda")
    want, _ = C.attention_varlen_norm_rotary(q, None, w, None, pos, inv)
    dq, _, dw, _ = C.attention_varlen_norm_rotary_bwd(dy, None, q, None, w, None, pos, inv)
    store = torch.empty(far + T * d, dtype=torch.bfloat16, device="cuda")
    x = store.as_strided((T, H, d), (d, far, 1))
    x.copy_(q)
    C.attention_varlen_norm_rotary(x, None, w, None, pos, inv, q_out=x)
    assert torch.equal(x, want)
    x.copy_(dy)
    got, _, gw, _ = C.attention_varlen_norm_rotary_bwd(x, None, q, None, w, None, pos, inv, dq=x)
    assert torch.equal(got, dq) and torch.equal(gw, dw)
