"""The counters in mita_paged_attn's workspace: 255 words that hold the number of the call that counted
last (from bit 16 on) and its count, then the word that numbers the calls, 256 a call."""
import pytest
import torch

import decode_util as R

pytestmark = pytest.mark.gpu

STEP, BITS = 256, 16


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
    """The counters of the current stream's workspace, the calls' number last."""
    ws = mita._paged_workspaces[0, torch.cuda.current_stream().cuda_stream]
    return ws[:mita._PAGED_COUNTERS].view(torch.int64)


SHAPES = [((1,), 1, 1, 64), ((0, 0), 4, 2, 32), ((300,), 8, 2, 128), ((20000, 5, 0, 700), 4, 2, 64),
          ((9000,), 16, 1, 128), (tuple(i * 29 % 90 for i in range(400)), 4, 1, 32)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_calls_are_numbered_whatever_their_shapes(dt):
    mita = M()
    calls = [arguments(*shape, dt) for shape in SHAPES]
    want = []
    for args in calls:
        mita.workspace_release()
        want.append(mita.mita_paged_attn(*args))
    mita.workspace_release()
    mita.mita_paged_attn(*max(calls, key=lambda a: a[1].numel()))     # as large as it gets
    for _ in range(3):
        for args, out in zip(calls, want):
            before = counters(mita).clone()
            assert torch.equal(mita.mita_paged_attn(*args), out)
            after = counters(mita)
            if int(before[-1]) <= int(after[-1]):                     # the same workspace, not a larger one
                assert int(after[-1]) - int(before[-1]) == STEP
            number = int(after[-1]) // STEP - 1
            assert int(after[-1]) % STEP == 0
            assert int((after[:-1] >> BITS).max()) <= number
            assert int((after[:-1] & ((1 << BITS) - 1)).max()) <= STEP


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES[2:5], ids=lambda s: f"{len(s[0])}x{max(s[0])}-{s[1:]}")
def test_what_a_disturbed_call_leaves_does_not_count(shape, dt):
    """Counts as a call would leave them whose lengths changed while it ran: any number up to two of
    each CTA, under that call's number.  The next call, and a call after a very great many, is
    right."""
    mita = M()
    args = arguments(*shape, dt)
    want = mita.mita_paged_attn(*args, return_lse=True)
    for number in (None, 1 << 20, (1 << 40) + 5):
        for left in (1, 2, 7, 510):
            w = counters(mita)
            if number is not None:
                w[-1] = (number + left) * STEP
            last = int(w[-1]) // STEP - 1
            w[:-1] = (last << BITS) + left
            for _ in range(2):
                got = mita.mita_paged_attn(*args, return_lse=True)
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    mita.workspace_release()


def test_graphs_replayed_out_of_order():
    """Two captured calls of different grids on workspaces of their graphs, replayed in any order and
    between eager calls: each is right every time."""
    mita = M()
    runs = []
    for shape in (SHAPES[3], SHAPES[4]):
        args = arguments(*shape, torch.bfloat16)
        want = mita.mita_paged_attn(*args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = [mita.mita_paged_attn(*args) for _ in range(3)]
        runs.append((args, want, graph, out))
    for i in (0, 1, 1, 0, 0, 0, 1, 0, 1, 1):
        args, want, graph, out = runs[i]
        graph.replay()
        assert torch.equal(mita.mita_paged_attn(*args), want)
        assert all(torch.equal(o, want) for o in out)
