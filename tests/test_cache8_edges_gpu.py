"""The cache held in 8 bits at its edges, for both of its attention kernels: exact means."""
import pytest
import torch

import cache8_ref as ref8
import cache_ref as ref
from ragged_gqa_attention_varlen_gb300 import cache as C
from test_cache8_gpu import F8, attend
from test_cache_gpu import HF, i32, lib, normal, status  # noqa: F401

pytestmark = pytest.mark.gpu


def run(q, kc, counts, call, want_status=0, **more):
    st = status()
    got = attend(q, kc, i32(ref.cu(counts)), call, status=st, **more)
    torch.cuda.synchronize()
    assert int(st) == want_status
    return got


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
