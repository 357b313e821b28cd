"""Gradients of the norms at the ends of what eps and the rows may be, on the GPU against
plain 64-bit forms."""
import pytest
import torch

import cache8_ref as ref8
import cache_ref as ref
from ragged_gqa_attention_varlen_gb300 import cache as C
from test_cache_gpu import BF, HF, lib, normal, within  # noqa: F401

pytestmark = pytest.mark.gpu


def turns(T, pairs):
    if not pairs:
        return None, None
    pos = torch.randint(0, 4000, (1, T), generator=torch.Generator().manual_seed(6), dtype=torch.int32).cuda()
    return pos, (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).cuda()


def check_gradients(x, w, dy, pos, inv, eps, dx, dw):
    """The tolerances count the roundings: g (sine and cosine, a product and a sum) is off by 2^-20 of
    the magnitudes that meet in it, r and the two means by a few steps of 2^-23 of theirs, dx is
    rounded once.  dw sums n terms in parts: each addition is off by half a step of what its part
    holds, at most n / 600 + 60 additions one after another (a lane's rows, then lanes, warps, blocks)."""
    g, mag = ref8.turned(dy.cpu().double(), pos, inv, None, False, inverse=True)
    xd, wd = x.cpu().double(), w.cpu().double()
    r = 1 / (xd.square().mean(-1, keepdim=True) + eps).sqrt()
    xhat = xd * r
    want = r * (g * wd - xhat * (g * wd * xhat).mean(-1, keepdim=True))
    slack = r * (mag * wd.abs() + xhat.abs() * (mag * wd.abs() * xhat.abs()).mean(-1, keepdim=True)) * 2.0 ** -19
    within("dx", dx, want, ref.UNIT[x.dtype] * want.abs() + slack + 2.0 ** -25)
    rows = x.shape[0] * x.shape[1]
    within("dw", dw, (g * xhat).sum((0, 1)), (mag * xhat.abs()).sum((0, 1)) * (2.0 ** -19 + (rows / 600 + 60) * 2.0 ** -24) + 2.0 ** -25)


# rows that do and do not fill the last pass of a warp (3, 4, 8 rows) and of a block
SHAPES = [(1, 1, 64, 0, BF), (1, 8, 64, 32, HF), (3, 3, 128, 0, BF), (5, 1, 128, 64, BF), (1, 1, 160, 80, HF), (7, 5, 160, 79, BF), (33, 12, 128, 63, HF),
          (24, 1, 160, 0, BF), (2000, 3, 160, 80, BF)]


@pytest.mark.parametrize("eps", [0.0, 1e-60])
@pytest.mark.parametrize("T,H,d,pairs,dtype", SHAPES)
def test_gradients_without_eps(T, H, d, pairs, dtype, eps):
    """eps = 0, or one that fp32 rounds to 0: lanes behind the last row of a run add nothing to the
    weights' gradients."""
    q, dy = normal(1, T, H, d, dtype=dtype, std=2.0), normal(2, T, H, d, dtype=dtype)
    k, dk = normal(3, T, 2, d, dtype=dtype), normal(4, T, 2, d, dtype=dtype)
    qw, kw = normal(5, d, dtype=torch.float32), normal(6, d, dtype=torch.float32)
    pos, inv = turns(T, pairs)
    dx, dkx, dw, dkw = C.attention_varlen_norm_rotary_bwd(dy, dk, q, k, qw, kw, pos, inv, eps=eps)
    check_gradients(q, qw, dy, pos, inv, 0.0, dx, dw)
    check_gradients(k, kw, dk, pos, inv, 0.0, dkx, dkw)


@pytest.mark.parametrize("T,H,d,pairs", [(40, 3, 64, 32), (40, 3, 128, 0), (40, 3, 160, 33)])
def test_gradients_of_small_rows(T, H, d, pairs):
    """Rows down to 2^-60 with eps = 0: the cube of 1 / their size passes fp32's range, their
    gradient (2^60 and less) does not."""
    x, dy = normal(1, T, H, d), normal(2, T, H, d)
    x = (x.float() * torch.exp2(torch.randint(-60, 3, (T, H, 1), generator=torch.Generator().manual_seed(3)).float()).cuda()).to(BF)
    w = normal(5, d, dtype=torch.float32)
    pos, inv = turns(T, pairs)
    dx, _, dw, _ = C.attention_varlen_norm_rotary_bwd(dy, None, x, None, w, None, pos, inv, eps=0.0)
    check_gradients(x, w, dy, pos, inv, 0.0, dx, dw)
