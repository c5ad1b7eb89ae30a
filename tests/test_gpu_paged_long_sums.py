"""mita_paged_attn over so many keys a warp that a sum which is cut at every step, instead of rounded,
leans visibly towards zero."""
import pytest
import torch

from test_gpu_paged import M

pytestmark = pytest.mark.gpu


def test_values_do_not_lean_towards_zero():
    """One sequence an SM, all of them over the same four pages: 15.4 million keys each, 1.9 million a
    warp, in 60 thousand tiles of 32.  All scores are equal, so that weights are 1 and their sum is
    exact; values are positive and spread over twelve binades, so that hardly a sum of them is.  A
    tile's sum, added to the running one in fp32, is off by at most U of that: 60000 U in all, and
    half a step for the result.  (Cut four times a tile by half a step on average, the sums come out
    1 % short.)"""
    mita = M()
    S, page, d, tiles = torch.cuda.get_device_properties(0).multi_processor_count, 1024, 64, 60000
    length = tiles * 32 * 8 // page * page
    g = torch.Generator().manual_seed(0)
    size = torch.rand(4, 1, page, d, generator=g) + 1
    size = size * 2.0 ** -torch.randint(0, 12, size.shape, generator=g).float()
    v = size.bfloat16()
    k = torch.zeros_like(v).cuda()
    table = (torch.arange(length // page) % 4).to(torch.int32).expand(S, -1).contiguous().cuda()
    lengths = torch.full((S,), length, dtype=torch.int32).cuda()
    q = torch.randn(S, 1, d, generator=g).bfloat16().cuda()
    out, lse = mita.mita_paged_attn(q, k, v.cuda(), table, lengths, return_lse=True)
    want = torch.zeros(d, dtype=torch.float64)
    for p in range(4):                         # the pages come in turn: each equally often, or once more
        want += v[p].double().sum((0, 1)) * ((length // page + 3 - p) // 4)
    want /= length
    off = (out[:, 0].cpu().double() - want) / want
    assert float(off.abs().max()) <= tiles * 2.0 ** -24 + 2.0 ** -9
    assert bool((lse.cpu().double() - torch.tensor(float(length)).double().log()).abs().max() <= 1e-5)
    assert mita.get_last_device_error() == 0
