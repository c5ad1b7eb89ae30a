"""mita_qk_norm_rope and its gradient on the GPU against plain fp64 restatements, with bounds
counted from the kernels' roundings (decode_util.py), and the gradient against differences."""
import pytest
import torch

import decode_util as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def M():
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    return mita


def make(B, Hq, Hkv, N, d, dt, seed=0, fused=True):
    """q, k as transposed views of one projection's output (or dense), on the CPU."""
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(B, N, Hq + 2 * Hkv, d, generator=g) * 1.5).to(DT[dt])
    q, k = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
    w = [1 + 0.3 * torch.randn(d, generator=g) for _ in range(2)]
    return (q, k, *w) if fused else (q.contiguous(), k.contiguous(), *w)


def cuda_views(q, k):
    """The same views on the GPU: strides kept."""
    def up(t):
        base = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
        return base.copy_(t)
    return up(q), up(k)


CASES = [
    # B, Hq, Hkv, N, d, dtype, rot, interleaved, norms (q, k), positions, fused
    (1, 1, 1, 1, 64, "bf16", 64, False, (1, 1), None, True),
    (2, 6, 6, 196, 64, "bf16", 64, False, (1, 1), None, False),
    (1, 8, 2, 77, 128, "bf16", 128, False, (1, 1), "shared", True),
    (3, 4, 1, 33, 32, "f32", 32, True, (1, 1), "own", True),
    (2, 3, 1, 50, 16, "f32", 16, False, (1, 1), "far", True),
    (1, 5, 3, 301, 16, "bf16", 8, True, (1, 1), "own", False),
    (2, 8, 4, 129, 128, "bf16", 64, False, (1, 1), "negative", True),
    (1, 2, 2, 63, 128, "f32", 24, False, (1, 1), None, True),
    (1, 4, 2, 40, 64, "bf16", 0, False, (1, 1), None, True),
    (1, 4, 2, 41, 64, "bf16", 64, True, (0, 0), "own", True),
    (2, 7, 2, 43, 32, "f32", 16, False, (1, 0), None, True),
    (2, 7, 2, 43, 32, "bf16", 16, False, (0, 1), None, True),
    # enough tokens for several heads in a run, and for blocks that loop
    (1, 10, 5, 20011, 128, "bf16", 128, False, (1, 1), None, True),
    (2, 2, 2, 40000, 64, "bf16", 64, False, (1, 1), "far", False),
]


def positions(kind, B, N):
    g = torch.Generator().manual_seed(3)
    if kind == "own":
        return torch.randint(0, 5000, (B, N), generator=g, dtype=torch.int32)
    if kind == "shared":
        return torch.randint(0, 5000, (N,), generator=g, dtype=torch.int32)
    if kind == "far":
        p = torch.randint(0, 2 ** 31 - 1, (B, N), generator=g, dtype=torch.int64)
        p[:, :2] = torch.tensor([2 ** 31 - 1, 2 ** 20])[:min(2, N)]
        return p.to(torch.int32)
    if kind == "negative":
        return torch.randint(-100000, 100, (B, N), generator=g, dtype=torch.int32)
    return None


def up(t):
    return None if t is None else t.cuda()


def setup(case):
    B, Hq, Hkv, N, d, dt, rot, pairs, norms, pos, fused = case
    q, k, wq, wk = make(B, Hq, Hkv, N, d, dt, fused=fused)
    wq, wk = wq if norms[0] else None, wk if norms[1] else None
    freq = R.inv_freq(rot) if rot else None
    p = positions(pos, B, N)
    at = torch.arange(N).expand(B, N) if p is None else p.expand(B, N)
    return q, k, wq, wk, freq, p, at[:, None, :], pairs


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward(case):
    mita = M()
    q, k, wq, wk, freq, pos, at, pairs = setup(case)
    gq, gk = cuda_views(q, k)
    got = mita.mita_qk_norm_rope(gq, gk, up(freq), up(wq), up(wk), up(pos), 1e-5, pairs)
    for x, w, y, n in ((q, wq, got[0], "q"), (k, wk, got[1], "k")):
        want, bound = R.norm_rope(x, w, at.expand(x.shape[:3]), freq, 1e-5, pairs)
        assert y.is_contiguous() and y.dtype == x.dtype
        R.assert_close(y, want, bound, n)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_backward(case):
    mita = M()
    q, k, wq, wk, freq, pos, at, pairs = setup(case)
    g = torch.Generator().manual_seed(9)
    dyq, dyk = (torch.randn(x.shape, generator=g).to(x.dtype) for x in (q, k))
    gq, gk = cuda_views(q, k)
    args = (gq, gk, dyq.cuda(), dyk.cuda(), up(freq), up(wq), up(wk), up(pos), 1e-5, pairs)
    got = mita.mita_qk_norm_rope_backward(*args)
    for x, dy, w, dx, dw, n in ((q, dyq, wq, got[0], got[2], "q"), (k, dyk, wk, got[1], got[3], "k")):
        want, bound, dwant, dbound = R.norm_rope_grad(x, dy, w, at.expand(x.shape[:3]), freq, 1e-5,
                                                      pairs)
        R.assert_close(dx, want, bound, "d" + n)
        assert (dw is None) == (w is None)
        if w is not None:
            R.assert_close(dw, dwant, dbound, "dw" + n)
    again = mita.mita_qk_norm_rope_backward(*args)
    for a, b in zip(got, again):          # summed in a fixed order: the same bits
        assert a is None or torch.equal(a, b)


def test_gradient_against_differences():
    """The kernels' gradients, fp32, against central differences of the fp64 forward along random
    directions.  Rounding of the fp32 gradient, dotted with the direction, is below
    64 u * sqrt(n) of the terms' sizes; the difference's own error is O(h^2) of the third
    derivative, 1e-8 of the sizes here with h = 1e-4."""
    mita = M()
    B, Hq, Hkv, N, d = 2, 3, 1, 5, 32
    q, k, wq, wk = make(B, Hq, Hkv, N, d, "f32")
    freq, at = R.inv_freq(d), torch.arange(N).expand(B, 1, N)
    g = torch.Generator().manual_seed(5)
    dy = [torch.randn(x.shape, generator=g) for x in (q, k)]
    got = mita.mita_qk_norm_rope_backward(*cuda_views(q, k), dy[0].cuda(), dy[1].cuda(),
                                          freq.cuda(), wq.cuda(), wk.cuda(), None, 1e-6)

    def loss(q_, k_, wq_, wk_):
        total = 0.0
        for x, w, y in ((q_, wq_, dy[0]), (k_, wk_, dy[1])):
            u = R.norm(x, w, 1e-6)
            total += float((R.rotate(u, at.expand(x.shape[:3]), freq, False) * y.double()).sum())
        return total

    at0 = [t.double() for t in (q, k, wq, wk)]
    for i, grad in enumerate(got):
        v = torch.randn(at0[i].shape, generator=g).double()
        h = 1e-4
        hi, lo = list(at0), list(at0)
        hi[i], lo[i] = at0[i] + h * v, at0[i] - h * v
        slope = (loss(*hi) - loss(*lo)) / (2 * h)
        terms = (grad.cpu().double() * v).abs().sum().item()
        assert abs(slope - (grad.cpu().double() * v).sum().item()) <= 1e-5 * terms, i


def test_autograd_function_and_broadcast_inputs():
    """Leaves behind views, a key head shared by expansion, an upstream gradient that is itself a
    broadcast: every gradient against autograd through the fp64 restatement."""
    mita = M()
    B, H, N, d = 2, 4, 9, 64
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(B, N, H + 1, d, generator=g)
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g) for _ in range(2))
    freq = R.inv_freq(d)

    def parts(t):
        return t[:, :, :H].transpose(1, 2), t[:, :, H:].transpose(1, 2).expand(B, H, N, d)

    leaf = [t.cuda().requires_grad_() for t in (qkv, wq, wk)]
    q, k = parts(leaf[0])
    qo, ko = mita.QKNormRopeFunction.apply(q, k, freq.cuda(), leaf[1], leaf[2])
    (qo.sum() + (ko * ko).sum()).backward()

    ref = [t.double().requires_grad_() for t in (qkv, wq, wk)]
    q, k = parts(ref[0])
    at = torch.arange(N).expand(B, H, N)

    def full(x, w):
        u = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        a, b = u[..., :d // 2], u[..., d // 2:]
        ang = at.double()[..., None] * freq
        return torch.cat((a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()), -1)
    (full(q, ref[1]).sum() + (full(k, ref[2]) ** 2).sum()).backward()
    for a, b in zip(leaf, ref):
        # fp32 roundings of some hundred terms of the gradient's size
        assert (a.grad.cpu().double() - b.grad).abs().max() <= 512 * R.U * b.grad.abs().max()


def test_in_place_out_strides_and_q_alone():
    mita = M()
    q, k, wq, wk = make(2, 4, 2, 37, 64, "bf16")
    freq = R.inv_freq(64).cuda()
    gq, gk = cuda_views(q, k)
    want = mita.mita_qk_norm_rope(gq, gk, freq, wq.cuda(), wk.cuda())
    alone, none = mita.mita_qk_norm_rope(gq, None, freq, wq.cuda())
    assert none is None and torch.equal(alone, want[0])
    # into a token-major buffer with room around it, the rest left as it was
    buf = torch.full((2, 37, 9, 64), 7.0, dtype=q.dtype, device="cuda")
    o = mita.mita_qk_norm_rope(gq, gk, freq, wq.cuda(), wk.cuda(),
                               q_out=buf[:, :, 1:5].transpose(1, 2),
                               k_out=buf[:, :, 6:8].transpose(1, 2))
    assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])
    for h in (0, 5, 8):
        assert bool((buf[:, :, h] == 7.0).all())
    dy = torch.randn(want[0].shape, device="cuda").to(q.dtype)
    dk = torch.randn(want[1].shape, device="cuda").to(q.dtype)
    grads = mita.mita_qk_norm_rope_backward(gq, gk, dy, dk, freq, wq.cuda(), wk.cuda())
    assert grads[0].transpose(1, 2).is_contiguous()      # token-major like the projection
    mita.mita_qk_norm_rope_backward(gq, gk, dy, dk, freq, wq.cuda(), wk.cuda(), dq=dy, dk=dk)
    assert torch.equal(dy, grads[0]) and torch.equal(dk, grads[1])
    # and the forward in place
    mita.mita_qk_norm_rope(gq, gk, freq, wq.cuda(), wk.cuda(), q_out=gq, k_out=gk)
    assert torch.equal(gq, want[0]) and torch.equal(gk, want[1])


def test_empty_calls():
    mita = M()
    n0 = mita.kernel_launches()
    q = torch.empty(2, 4, 0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    assert mita.mita_qk_norm_rope(q, q, None, w, w)[0].shape == q.shape
    grads = mita.mita_qk_norm_rope_backward(q, q, q, q, None, w, w)
    assert grads[0].shape == q.shape and float(grads[2].abs().sum() + grads[3].abs().sum()) == 0
    assert mita.kernel_launches() == n0


def test_rows_with_infinities_stay_alone():
    """A NaN or infinite row gives NaN in itself and leaves its neighbours' values alone."""
    mita = M()
    q, k, wq, wk = make(1, 2, 2, 70, 32, "f32", fused=False)
    freq = R.inv_freq(32).cuda()
    want = mita.mita_qk_norm_rope(q.cuda(), k.cuda(), freq, wq.cuda(), wk.cuda())
    q[0, 1, 5, 3], q[0, 0, 8, 0], k[0, 1, 33, 31] = float("nan"), float("inf"), -float("inf")
    got = mita.mita_qk_norm_rope(q.cuda(), k.cuda(), freq, wq.cuda(), wk.cuda())
    bad = [torch.zeros(1, 2, 70, dtype=torch.bool) for _ in range(2)]
    bad[0][0, 1, 5] = bad[0][0, 0, 8] = bad[1][0, 1, 33] = True
    for y, x, b in zip(got, want, bad):
        assert torch.equal(y.cpu()[~b], x.cpu()[~b])
        assert bool(torch.isnan(y.cpu()[b]).any(-1).all())


def test_streams_and_graphs():
    """A side stream; a captured forward and backward replayed on new inputs; two graphs of the
    gradient, which share nothing."""
    mita = M()
    q, k, wq, wk = make(1, 4, 2, 500, 64, "bf16")
    freq, wq, wk = R.inv_freq(64).cuda(), wq.cuda(), wk.cuda()
    gq, gk = cuda_views(q, k)
    dq, dk = torch.randn(gq.shape, device="cuda").to(q.dtype), torch.randn(gk.shape, device="cuda").to(q.dtype)
    want = mita.mita_qk_norm_rope(gq, gk, freq, wq, wk)
    gwant = mita.mita_qk_norm_rope_backward(gq, gk, dq, dk, freq, wq, wk)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = mita.mita_qk_norm_rope(gq, gk, freq, wq, wk, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graphs = []
    for i in range(2):
        sq, sk, sdq, sdk = (torch.zeros_like(t) for t in (gq, gk, dq, dk))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = mita.mita_qk_norm_rope(sq, sk, freq, wq, wk)
            grads = mita.mita_qk_norm_rope_backward(sq, sk, sdq, sdk, freq, wq, wk)
        graphs.append((graph, (sq, sk, sdq, sdk), out, grads))
    for i, (graph, ins, out, grads) in enumerate(graphs):
        for t, x in zip(ins, (gq, gk, dq, dk)):
            t.copy_(x if i == 0 else -x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for (graph, *_), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for i, (_, _, out, grads) in enumerate(graphs):
        sign = 1 if i == 0 else -1
        assert torch.equal(out[0], sign * want[0]) and torch.equal(out[1], sign * want[1])
        for a, b, s in zip(grads, gwant, (sign, sign, 1, 1)):
            assert torch.equal(a, s * b)
