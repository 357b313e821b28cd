"""The generation calls on the GPU at their edges: exact means of equal V rows, metadata
that does not fit, pages out of the pool, expanded inputs, calls without tokens."""
import math

import pytest
import torch

import cache_ref as ref
from ragged_gqa_attention_varlen_gb300 import cache as C
from test_cache_gpu import BF, HF, i32, normal, status, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from ragged_gqa_attention_varlen_gb300 import _build

    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return C.load()


# ---------------------------------------------------------------- sums of the weights

@pytest.mark.parametrize("cap", [0.0, 3.0, 9.0, 30.0])
@pytest.mark.parametrize("lens,plens,counts,Hq,Hkv,d,page,dtype", [
    ([1, 2, 3, 5], (), [20] * 4, 16, 1, 160, 16, BF), ([2, 4, 130], (), [30, 10, 40], 8, 2, 128, 32, BF),
    ([3, 9, 200], (), [10, 20, 10], 8, 1, 64, 16, HF), ([2, 1, 4], [3], [10, 10, 20], 16, 1, 160, 16, BF),
    ([5000], (), [1], 8, 1, 160, 64, BF)])
def test_equal_values_come_out_exactly(lens, plens, counts, Hq, Hkv, d, page, dtype, cap):
    """out is a weighted mean of V rows: where they are all the same row it is that row, whatever
    the weights' roundings, as the weights that multiply V are those whose sum divides.  Sums of
    at most 5000 terms in fp32 are off by 5000 / 16 additions of 2^-22 (a product of 16 keys is
    added at a time) and the row sum, halves and reciprocal by less than 1000 * 2^-24: 1.4e-4
    together, below half a step of either type (bf16 2^-9, fp16 2^-12 of the value)."""
    group = [0] * len(lens) if plens else None
    kc = ref.Cache(lens, plens, Hkv, d, page, dtype)
    # half of the features as large as their exponent has them: half a step is least there
    row = normal(7, Hkv, d, dtype=dtype)
    row[:, ::2] = torch.where(row[:, ::2] > 0, 2.0, -2.0) * (1 - torch.finfo(dtype).eps / 2)
    kc.v.copy_(row)
    q = normal(8, sum(counts), Hq, d, dtype=dtype, std=3.0)
    call = {}
    if plens:
        call = dict(prefix_table=kc.ptable, prefix_lens=kc.plens, cu_prefix=i32([0, len(lens)]))
    out, _ = C.attention_varlen_cache_fwd(q, kc.k, kc.v, kc.table, kc.lens, i32(ref.cu(counts)), softcap=cap, **call)
    want = row.repeat_interleave(Hq // Hkv, 0).expand_as(out)
    assert torch.equal(out, want), (out != want).float().mean()
