"""Calls of the q / k preparation and the paged cache at the edges of what is allowed: far
strides, chains of launches on the same memory, empty tables, bad indices, many heads, a first
call inside a capture."""
import subprocess
import sys

import pytest
import torch

import decode_util as R
from conftest import ROOT

pytestmark = pytest.mark.gpu


def M():
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    return mita


def lens(*n):
    return torch.tensor(n, dtype=torch.int32).cuda()


def test_in_place_chain():
    """Twenty launches back to back, each rotating what the one before left in the same memory (the
    next kernel's blocks are launched early): the same bits as with a buffer for each."""
    mita = M()
    g = torch.Generator().manual_seed(0)
    x = torch.randn(1, 24, 4001, 64, generator=g).bfloat16().cuda()
    w, freq = (1 + 0.1 * torch.randn(64, generator=g)).cuda(), R.inv_freq(64).cuda()
    want = [x]
    for _ in range(20):
        want.append(mita.mita_qk_norm_rope(want[-1], None, freq, w)[0])
    got = x.clone()
    for _ in range(20):
        mita.mita_qk_norm_rope(got, None, freq, w, q_out=got)
    assert torch.equal(got, want[-1])
    for _ in range(20):
        mita.mita_qk_norm_rope_backward(x, None, got, None, freq, w, dq=got)
    ref = want[-1]
    for _ in range(20):
        ref = mita.mita_qk_norm_rope_backward(x, None, ref, None, freq, w)[0]
    assert torch.equal(got, ref)


def test_append_then_attend_chain():
    """Steps back to back with nothing waited for, lengths, tables and queries made on the device
    just before each step: the same bits as with a synchronisation after every call."""
    mita = M()
    S, Hq, Hkv, d, page, steps = 5, 8, 2, 64, 16, 60
    g = torch.Generator().manual_seed(1)
    x = torch.randn(steps, S, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda()
    freq = R.inv_freq(d).cuda()
    table0 = torch.randperm(S * 8, generator=g).to(torch.int32).view(S, 8).cuda()

    def decode(wait):
        kc = torch.zeros(S * 8, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
        vc, n, outs = torch.zeros_like(kc), torch.zeros(S, dtype=torch.int32, device="cuda"), []
        table = torch.full_like(table0, -1)
        for t in range(steps):
            n += 1
            if t % page == 0:
                table[:, t // page] = table0[:, t // page]
            tok = x[t] * 1.0
            q = mita.mita_cache_append(tok[:, Hq:Hq + Hkv], tok[:, Hq + Hkv:], kc, vc, table, n,
                                       q=tok[:, :Hq], inv_freq=freq)
            if wait:
                torch.cuda.synchronize()
            outs.append(mita.mita_paged_attn(q, kc, vc, table, n))
            if wait:
                torch.cuda.synchronize()
        return torch.stack(outs), kc, vc

    for a, b in zip(decode(False), decode(True)):
        assert torch.equal(a, b)
    assert mita.get_last_device_error() == 0


def test_far_strides():
    """Rows more than 2^31 elements (2^32 bytes) apart, in inputs and outputs."""
    mita = M()
    far = 2_300_000_000                                     # a multiple of 8
    base = torch.zeros(far + 4096, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(base)
    x = base.as_strided((2, 2, 3, 64), (far, 192, 64, 1))
    y = out.as_strided((2, 2, 3, 64), (far, 192, 64, 1))
    g = torch.Generator().manual_seed(0)
    v = torch.randn(2, 2, 3, 64, generator=g).bfloat16().cuda()
    x.copy_(v)
    freq = R.inv_freq(64).cuda()
    want = mita.mita_qk_norm_rope(v, None, freq)[0]
    mita.mita_qk_norm_rope(x, None, freq, q_out=y)
    assert torch.equal(y, want)
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    vc, table = torch.zeros_like(kc), lens(1, 0).view(2, 1)
    tok = x[:, :, 0]
    mita.mita_cache_append(tok, tok, kc, vc, table, lens(1, 1), q=tok, inv_freq=freq,
                           q_out=y[:, :, 1])
    assert torch.equal(vc[[1, 0], :, 0], v[:, :, 0])
    got = mita.mita_paged_attn(tok, kc, vc, table, lens(1, 1))
    assert torch.equal(got, v[:, :, 0])                     # one key: its value


def test_tables_without_room():
    mita = M()
    q = torch.randn(2, 4, 64, device="cuda")
    kc = torch.zeros(3, 2, 16, 64, device="cuda")
    none = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    out, lse = mita.mita_paged_attn(q, kc, kc, none, lens(0, 0), return_lse=True)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    assert mita.get_last_device_error() == 0
    assert bool((mita.mita_paged_attn(q, kc, kc, none, lens(0, 5)) == 0).all())
    assert mita.get_last_device_error() == 1
    mita.mita_cache_append(q[:, :2], q[:, :2], kc, kc.clone(), none, lens(1, 0))
    assert mita.get_last_device_error() == 1 and bool((kc == 0).all())
    empty = kc[:0]                                          # a cache of no pages
    out = mita.mita_paged_attn(q, empty, empty, lens(0, 0).view(2, 1), lens(3, 0))
    assert mita.get_last_device_error() == 1 and bool((out == 0).all())


def test_bad_seq_start_writes_nothing_it_should_not():
    """Descending, negative and far too large row starts: tokens that then have no valid place are
    flagged or left out; every write lands in the cache rows of the table."""
    mita = M()
    big = 2 ** 31 - 1
    for starts in ((5, 0, 9), (-(2 ** 31), 4, big), (0, big, 3), (9, 9, 9), (-7, -3, -1),
                   (0, 8, 4)):
        kc = torch.zeros(6, 1, 4, 32, device="cuda")
        vc, out = torch.zeros_like(kc), torch.full((8, 2, 32), 9.0, device="cuda")
        x = torch.randn(8, 4, 32, device="cuda")
        mita.mita_cache_append(x[:, 2:3], x[:, 3:], kc, vc, lens(0, 1, 2, 3).view(2, 2),
                               lens(8, 6), seq_start=lens(*starts), q=x[:, :2], q_out=out)
        assert mita.get_last_device_error() in (0, 1)
        assert bool((kc[4:] == 0).all()) and bool((vc[4:] == 0).all())


def test_many_heads_and_many_sequences():
    mita = M()
    g = torch.Generator().manual_seed(3)
    x = torch.randn(1, 301, 70, 16, generator=g).cuda()
    freq = R.inv_freq(16)
    q, k = x[:, :, :69].transpose(1, 2), x[:, :, 69:].transpose(1, 2)
    got = mita.mita_qk_norm_rope(q, k, freq.cuda())
    for a, b in ((q, got[0]), (k, got[1])):
        want, bound = R.norm_rope(a.cpu(), None, torch.arange(301).expand(a.shape[:3]), freq, 1e-6,
                                  False)
        R.assert_close(b, want, bound, "rows")
    # 5000 sequences, most of them idle: 40 distinct caches, each shared by many sequences
    lengths = [(i * 7) % 41 if i % 3 == 0 else 0 for i in range(5000)]
    cache = R.Cache(range(41), 1, 8, 32, torch.bfloat16)
    cache.table = cache.table[torch.tensor(lengths)]
    cache.lengths = lengths
    q = torch.randn(5000, 2, 32, generator=g).bfloat16()
    out = mita.mita_paged_attn(q.cuda(), cache.k.cuda(), cache.v.cuda(), cache.table.cuda(),
                               lens(*lengths))
    want, bound, _, _ = R.paged_attn(q, cache, lengths)
    R.assert_close(out, want, bound, "out")
    assert mita.get_last_device_error() == 0


def test_window_of_any_size_and_float_scales():
    mita = M()
    cache = R.Cache((70,), 1, 16, 32, torch.float32)
    q = torch.randn(1, 2, 32, generator=torch.Generator().manual_seed(0))
    args = (q.cuda(), cache.k.cuda(), cache.v.cuda(), cache.table.cuda(), lens(70))
    want = mita.mita_paged_attn(*args)
    for window in (70, 71, 2 ** 31 - 1, 2 ** 40):
        assert torch.equal(mita.mita_paged_attn(*args, window=window), want)


def test_autograd_of_queries_alone_and_of_a_used_half():
    mita = M()
    freq = R.inv_freq(32).cuda()
    q = torch.randn(1, 2, 5, 32, device="cuda", requires_grad=True)
    w = torch.ones(32, device="cuda", requires_grad=True)
    out, none = mita.QKNormRopeFunction.apply(q, None, freq, w)
    assert none is None
    dy = torch.randn(1, 2, 5, 32, device="cuda")
    out.backward(dy)
    want = mita.mita_qk_norm_rope_backward(q.detach(), None, dy, None, freq, w.detach())
    assert torch.equal(q.grad, want[0]) and torch.equal(w.grad, want[2])
    # only k is used: q's upstream gradient is made of zeros
    k = torch.randn(1, 1, 5, 32, device="cuda", requires_grad=True)
    q.grad = None
    _, ko = mita.QKNormRopeFunction.apply(q, k, freq, w, w)
    ko.sum().backward()
    assert bool((q.grad == 0).all()) and bool((k.grad != 0).any())


FIRST_CALL = """
import torch
from sparse_top_landmark_gb300 import mita
q = torch.randn(1, 2, 8, 64, device="cuda")
torch.cuda.synchronize()
out = torch.empty_like(q)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    q2 = q + 1
    try:
        mita.mita_qk_norm_rope(q, q_out=out)
        raise SystemExit("not refused")
    except mita.MitaError as e:
        assert e.status == 2 and "captured" in str(e), e
graph.replay()
torch.cuda.synchronize()
assert torch.equal(q2, q + 1)
want = mita.mita_qk_norm_rope(q)[0]
with torch.cuda.graph(graph := torch.cuda.CUDAGraph()):
    mita.mita_qk_norm_rope(q, q_out=out)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(out, want)
print("fine")
"""


def test_first_call_inside_a_capture_is_refused_and_leaves_the_capture_whole():
    M()
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


def test_workspaces_are_shared_grown_released_and_left_clean():
    """Attention and gradients of growing and shrinking shapes in turn on one stream's workspace,
    and after its release: the same bits as from a workspace that nothing else has used."""
    mita = M()
    shapes = [((3000, 40), 4, 1, 128), ((700,), 16, 2, 64), ((9000, 5, 2000), 8, 2, 128), ((50,), 1, 1, 16)]
    calls = []
    for lengths, Hq, Hkv, d in shapes:
        cache = R.Cache(lengths, Hkv, 16, d, torch.bfloat16)
        q = torch.randn(len(lengths), Hq, d, generator=torch.Generator().manual_seed(1)).bfloat16()
        x = torch.randn(1, Hq, 300, d, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
        w = torch.ones(d, device="cuda")
        calls.append((lambda a: mita.mita_paged_attn(*a),
                      (q.cuda(), cache.k.cuda(), cache.v.cuda(), cache.table.cuda(), lens(*lengths))))
        calls.append((lambda a: mita.mita_qk_norm_rope_backward(*a)[2], (x, None, x, None, None, w)))
    want = []
    for f, a in calls:
        mita.workspace_release()
        want.append(f(a))
    for _ in range(3):
        for i in (0, 1, 2, 3, 4, 5, 6, 7, 4, 3, 0, 2, 1, 6):
            assert torch.equal(calls[i][0](calls[i][1]), want[i])


def test_two_threads_on_one_stream():
    """Gradients and attention from two host threads at once, on the same stream."""
    import threading
    mita = M()
    cache = R.Cache((5000, 300), 2, 16, 64, torch.bfloat16)
    g = torch.Generator().manual_seed(1)
    work = []
    for i in range(2):
        q = torch.randn(2, 8, 64, generator=g).bfloat16().cuda()
        x = torch.randn(1, 8, 400, 64, generator=g).bfloat16().cuda()
        a = (q, cache.k.cuda(), cache.v.cuda(), cache.table.cuda(), lens(5000, 300))
        b = (x, None, x, None, None, torch.ones(64, device="cuda"))
        work.append((a, b, mita.mita_paged_attn(*a), mita.mita_qk_norm_rope_backward(*b)[2]))
    torch.cuda.synchronize()
    got = [[], []]

    def run(i):
        with torch.cuda.stream(torch.cuda.default_stream()):
            for _ in range(50):
                got[i].append((mita.mita_paged_attn(*work[i][0]),
                               mita.mita_qk_norm_rope_backward(*work[i][1])[2]))
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 50
        assert all(torch.equal(o, work[i][2]) and torch.equal(w, work[i][3]) for o, w in got[i])


def test_inputs_dropped_right_after_a_call_on_another_stream():
    """The caller lets go of the inputs as soon as the call on a busy side stream is made, and
    allocates and fills as much again on its own: the call still reads what it was given."""
    mita = M()
    g = torch.Generator().manual_seed(2)
    x = torch.randn(1, 8, 20000, 64, generator=g).bfloat16()
    freq = R.inv_freq(64).cuda()
    want = mita.mita_qk_norm_rope(x.cuda(), None, freq)[0]
    side, busy = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(4):
        q = x.cuda()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                busy @ busy
        got = mita.mita_qk_norm_rope(q, None, freq, stream=side)[0]
        del q
        junk = [torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del junk


NEW_SHAPES_IN_A_CAPTURE = """
import sys
sys.path.insert(0, "tests")
import torch
import decode_util as R
from sparse_top_landmark_gb300 import mita
dt = getattr(torch, sys.argv[1])
lengths = (70, 0, 1300)
n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
cache = R.Cache(lengths, 2, 16, 64, dt)
kc, vc, table = cache.k.cuda(), cache.v.cuda(), cache.table.cuda()
g = torch.Generator().manual_seed(3)
q, k, v = (torch.randn(3, h, 64, generator=g).to(dt).cuda() for h in (6, 2, 2))
x = torch.randn(1, 6, 40, 64, generator=g).to(dt).cuda()
freq, w = R.inv_freq(64).cuda(), torch.ones(64, device="cuda")

def step():
    rotated = mita.mita_cache_append(k, v, kc, vc, table, n, q=q, inv_freq=freq, q_weight=w, k_weight=w)
    y = mita.mita_qk_norm_rope(x, None, freq, w)[0]
    return (rotated, mita.mita_paged_attn(rotated, kc, vc, table, n), y,
            *mita.mita_qk_norm_rope_backward(x, None, y, None, freq, w)[::2])

mita.mita_qk_norm_rope(torch.ones(1, 1, 1, 16, device="cuda"))     # the library's first call
torch.cuda.synchronize()
with torch.cuda.graph(graph := torch.cuda.CUDAGraph()):
    got = step()
graph.replay()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
want = step()
seen = torch.tensor([0, 2], device="cuda")
for i, (a, b) in enumerate(zip(got, want)):
    if i < 2:
        a, b = a[seen], b[seen]            # the idle slot's rows are not written
    assert torch.equal(a, b), i
print("fine")
"""


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_shapes_never_run_before_inside_a_capture(dt):
    """Each entry point's kernel is launched for the first time while a graph is captured."""
    M()
    r = subprocess.run([sys.executable, "-c", NEW_SHAPES_IN_A_CAPTURE, dt], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("n", [31, 32, 33, 127, 128, 129, 257, 513])
@pytest.mark.parametrize("dt,d", [("bfloat16", 32), ("float32", 16)])
def test_numbers_of_sequences(n, dt, d):
    """Batches around the sizes in which sequences are counted, idle slots and long ones among them,
    a long one first or last, or nothing but idle slots before the last."""
    mita = M()
    dt = getattr(torch, dt)
    for lengths in ([i * 53 % 70 for i in range(n - 1)] + [1500], [1500] + [i % 3 for i in range(n - 1)],
                    [0] * (n - 1) + [700]):
        cache = R.Cache(lengths, 2, 16, d, dt)
        q = torch.randn(n, 4, d, generator=torch.Generator().manual_seed(n)).to(dt)
        got = mita.mita_paged_attn(q.cuda(), cache.k.cuda(), cache.v.cuda(), cache.table.cuda(),
                                   lens(*lengths))
        want, bound = R.paged_attn(q, cache, lengths)[:2]
        R.assert_close(got, want, bound, "out")
        assert bool((got.cpu()[torch.tensor(lengths) == 0] == 0).all())
    assert mita.get_last_device_error() == 0
