"""The counters in mita_paged_attn's workspace: zero after every call, whatever was in them before."""
import pytest
import torch

import decode_util as R

pytestmark = pytest.mark.gpu


def M():
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    return mita


def lens(*n):
    return torch.tensor(n, dtype=torch.int32).cuda()


def arguments(lengths, Hq, Hkv, d, dt):
    cache = R.Cache(lengths, Hkv, 16, d, dt)
    q = torch.randn(len(lengths), Hq, d, generator=torch.Generator().manual_seed(1)).to(dt)
    return q.cuda(), cache.k.cuda(), cache.v.cuda(), cache.table.cuda(), lens(*lengths)


def counters(mita):
    """The counters of the current stream's workspace."""
    ws = mita._paged_workspaces[0, torch.cuda.current_stream().cuda_stream]
    return ws[:mita._PAGED_COUNTERS].view(torch.int32)


SHAPES = [((1,), 1, 1, 64), ((0, 0), 4, 2, 32), ((300,), 8, 2, 128), ((20000, 5, 0, 700), 4, 2, 64),
          ((9000,), 16, 1, 128), (tuple(i * 29 % 90 for i in range(400)), 4, 1, 32)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{max(s[0])}-{s[1:]}")
def test_zero_after_every_call(shape, dt):
    mita = M()
    args = arguments(*shape, dt)
    for _ in range(3):
        mita.mita_paged_attn(*args)
        assert int(counters(mita).abs().sum()) == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES[2:5], ids=lambda s: f"{len(s[0])}x{max(s[0])}-{s[1:]}")
def test_what_a_disturbed_call_leaves_is_gone_after_the_next(shape, dt):
    """Counts left above zero, as a call would leave them whose lengths changed while it ran: they
    spoil the call that finds them (it joins parts too early: every place is in the workspace),
    and no other."""
    mita = M()
    args = arguments(*shape, dt)
    want = mita.mita_paged_attn(*args, return_lse=True)
    for left in (1, 2, 7):
        counters(mita)[:-1] = left
        mita.mita_paged_attn(*args)
        assert int(counters(mita).abs().sum()) == 0
        got = mita.mita_paged_attn(*args, return_lse=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
