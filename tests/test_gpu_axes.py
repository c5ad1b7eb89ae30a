"""Norm and rotation by positions of several axes on the GPU: mita_qk_norm_rope_axes, its gradient and its
autograd function, against plain fp64 (decode_util.py, an axis at a time)."""
import pytest
import torch

import decode_util as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def M():
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    return mita


def gen(seed):
    return torch.Generator().manual_seed(seed)


def grid(*shape, lead=0):
    """Positions [axes, N] of a grid behind `lead` tokens that stand at the same place on every axis."""
    at = torch.stack(torch.meshgrid(*(torch.arange(n) for n in shape), indexing="ij")).flatten(1)
    first = torch.arange(lead).expand(len(shape), lead)
    return torch.cat((first, at + lead), 1).to(torch.int32)


def axis_of(kind, half, A):
    i = torch.arange(half)
    if kind == "sections":
        a = i * A // half
    elif kind == "turns":
        a = i % A
    else:                                   # any order
        a = torch.randint(0, A, (half,), generator=gen(half))
    return a.to(torch.int32)


def turn(x, positions, axis, freq, interleaved, back=False):
    """x [B, H, N, d] fp64 turned by positions [A, B or 1, N]: pairs of different axes do not meet, so one
    axis after the other, the other axes' frequencies zero."""
    for a in range(positions.shape[0]):
        x = R.rotate(x, positions[a][:, None], freq * (axis == a), interleaved, back)
    return x


def forward(x, w, positions, axis, freq, eps, interleaved):
    u = R.norm(x.double(), w, eps)
    y = turn(u, positions, axis, freq, interleaved) if freq is not None else u
    far = float(positions.abs().max()) * 2.0 ** -51
    return y, (R.half_step(x.dtype) * y.abs()
               + (32 * R.U + far) * R.pair_size(u, freq, interleaved))       # as decode_util.norm_rope


def gradient(x, dy, w, positions, axis, freq, eps, interleaved):
    """(dx, bound, dw, bound), as decode_util.norm_rope_grad."""
    xd = x.double()
    g = turn(dy.double(), positions, axis, freq, interleaved, back=True)
    size = R.pair_size(dy.double(), freq, interleaved)
    if w is None:
        return g, R.half_step(x.dtype) * g.abs() + 32 * R.U * size, None, None
    wd = w.double()
    r = 1 / torch.sqrt((xd * xd).mean(-1, keepdim=True) + eps)
    dx = r * wd * g - xd * r ** 3 * (wd * g * xd).mean(-1, keepdim=True)
    terms = r * wd.abs() * size + xd.abs() * r ** 3 * (wd.abs() * size * xd.abs()).mean(-1, True)
    rows = x[..., 0].numel()
    return (dx, R.half_step(x.dtype) * dx.abs() + 64 * R.U * terms, (g * xd * r).sum((0, 1, 2)),
            (32 + rows) * R.U * (size * xd.abs() * r).sum((0, 1, 2)))


CASES = [
    # B, shape, lead, Hq, Hkv, d, rot, kind, dtype, interleaved, norm, batch positions
    (1, (14, 14), 0, 6, 6, 64, 64, "sections", "bf16", False, True, False),
    (2, (3, 5, 7), 4, 4, 2, 128, 128, "sections", "bf16", False, True, True),
    (2, (3, 5, 7), 1, 4, 1, 64, 32, "turns", "f32", True, True, True),
    (1, (1, 1), 0, 1, 1, 32, 32, "turns", "f32", False, True, False),
    (3, (9, 11), 0, 3, 3, 16, 16, "any", "f32", False, True, False),
    (3, (9, 11), 0, 3, 3, 16, 8, "any", "bf16", True, False, False),
    (1, (2, 2, 2, 2, 3), 0, 2, 1, 128, 64, "any", "bf16", False, True, False),
    (1, (513,), 0, 2, 2, 64, 64, "sections", "f32", False, False, False),
    (2, (40, 41), 1, 12, 12, 64, 64, "sections", "bf16", False, True, False),
]
IDS = ["x".join(map(str, c[1])) + "-" + "-".join(map(str, c[3:11])) for c in CASES]


def made(case):
    B, shape, lead, Hq, Hkv, d, rot, kind, dt, inter, norm, each = case
    g = gen(1)
    N = lead + torch.Size(shape).numel()
    x = torch.randn(B, N, Hq + 2 * Hkv, d, generator=g).to(DT[dt])
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2)
    pos = grid(*shape, lead=lead)
    if each:
        pos = (pos[:, None] + torch.randint(-50, 2000, (1, B, 1), generator=g, dtype=torch.int32)).contiguous()
    wq, wk = (1 + 0.3 * torch.randn(2, d, generator=g)) if norm else (None, None)
    return (x, q, k, pos, pos if each else pos[:, None], axis_of(kind, rot // 2, len(shape)),
            R.inv_freq(rot), wq, wk)


def up(*ts):
    return [None if t is None else t.cuda() for t in ts]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    mita = M()
    x, q, k, pos, pos3, axis, freq, wq, wk = made(case)
    Hq, Hkv, inter = case[3], case[4], case[9]
    xc = x.cuda()
    qc, kc = xc[:, :, :Hq].transpose(1, 2), xc[:, :, Hq:Hq + Hkv].transpose(1, 2)
    dev = up(freq, axis, pos, wq, wk)
    qo, ko = mita.mita_qk_norm_rope_axes(qc, kc, *dev, interleaved=inter)
    assert mita.get_last_device_error() == 0
    for got, t, w in ((qo, q, wq), (ko, k, wk)):
        want, bound = forward(t, w, pos3, axis, freq, 1e-6, inter)
        R.assert_close(got, want, bound, "out")
    # in place, into token-major memory, and without k
    out = torch.empty_like(xc)[:, :, :Hq].transpose(1, 2)
    got, none = mita.mita_qk_norm_rope_axes(qc, None, *dev, interleaved=inter, q_out=out)
    assert got is out and none is None and torch.equal(out, qo)
    mita.mita_qk_norm_rope_axes(qc, kc, *dev, interleaved=inter, q_out=qc, k_out=kc)
    assert torch.equal(qc, qo) and torch.equal(kc, ko) and torch.equal(xc[:, :, Hq + Hkv:], x.cuda()[:, :, Hq + Hkv:])


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_gradient(case):
    mita = M()
    x, q, k, pos, pos3, axis, freq, wq, wk = made(case)
    Hq, Hkv, inter = case[3], case[4], case[9]
    g = gen(9)
    dq, dk = (torch.randn(t.shape, generator=g).to(t.dtype) for t in (q, k))
    xc = x.cuda()
    qc, kc = xc[:, :, :Hq].transpose(1, 2), xc[:, :, Hq:Hq + Hkv].transpose(1, 2)
    dev = up(freq, axis, pos, wq, wk)
    got = mita.mita_qk_norm_rope_axes_backward(qc, kc, dq.cuda(), dk.cuda(), *dev, interleaved=inter)
    again = mita.mita_qk_norm_rope_axes_backward(qc, kc, dq.cuda(), dk.cuda(), *dev, interleaved=inter)
    assert mita.get_last_device_error() == 0
    for i, (t, dy, w) in enumerate(((q, dq, wq), (k, dk, wk))):
        dx, bx, dw, bw = gradient(t, dy, w, pos3, axis, freq, 1e-6, inter)
        R.assert_close(got[i], dx, bx, "dx")
        assert torch.equal(got[i], again[i])
        if w is None:
            assert got[2 + i] is None
        else:
            R.assert_close(got[2 + i], dw, bw, "dw")
            assert torch.equal(got[2 + i], again[2 + i])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_equal_positions_are_the_single_axis(dt):
    """Text: the same position on every axis gives mita_qk_norm_rope's bits, forward and back."""
    mita = M()
    g = gen(3)
    q, k = (torch.randn(2, h, 300, 128, generator=g).to(DT[dt]).cuda() for h in (4, 2))
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (300,), generator=g).to(torch.int32).cuda()
    freq, axis = R.inv_freq(96).cuda(), axis_of("any", 48, 3).cuda()
    w = torch.rand(128, generator=g).cuda()
    same = pos.expand(3, 300)
    one = mita.mita_qk_norm_rope(q, k, freq, w, w, positions=pos)
    many = mita.mita_qk_norm_rope_axes(q, k, freq, axis, same, w, w)
    assert all(torch.equal(a, b) for a, b in zip(one, many))
    one = mita.mita_qk_norm_rope_backward(q, k, q, k, freq, w, w, positions=pos)
    many = mita.mita_qk_norm_rope_axes_backward(q, k, q, k, freq, axis, same, w, w)
    assert all(torch.equal(a, b) for a, b in zip(one, many))


def test_position_strides():
    """Positions as views: one axis of a wider array, batches shared or apart."""
    mita = M()
    g = gen(4)
    q = torch.randn(2, 2, 50, 32, generator=g).cuda()
    wide = torch.randint(0, 900, (5, 2, 77), generator=g).to(torch.int32).cuda()
    freq, axis = R.inv_freq(32).cuda(), axis_of("turns", 16, 2).cuda()
    pos = wide[1:4:2, :, :50]
    want = mita.mita_qk_norm_rope_axes(q, None, freq, axis, pos.contiguous())[0]
    assert torch.equal(mita.mita_qk_norm_rope_axes(q, None, freq, axis, pos)[0], want)
    shared = wide[1:4:2, 0, :50]
    want = mita.mita_qk_norm_rope_axes(q, None, freq, axis, shared[:, None].expand(2, 2, 50).contiguous())[0]
    assert torch.equal(mita.mita_qk_norm_rope_axes(q, None, freq, axis, shared)[0], want)
    assert torch.equal(mita.mita_qk_norm_rope_axes(q, None, freq, axis, shared[:, None].expand(2, 2, 50))[0], want)


def test_an_axis_out_of_range_is_flagged_and_counts_as_the_first():
    mita = M()
    q = torch.randn(1, 2, 40, 64, generator=gen(4)).cuda()
    pos = torch.stack((torch.arange(40), torch.arange(40) * 3)).to(torch.int32).cuda()
    freq, axis = R.inv_freq(64).cuda(), axis_of("turns", 32, 2).cuda()
    bad = axis.clone()
    bad[5], bad[6], bad[9] = 2, -1, 2 ** 31 - 1
    fine = axis.clone()
    fine[5] = fine[6] = fine[9] = 0
    got = mita.mita_qk_norm_rope_axes(q, None, freq, bad, pos)[0]
    assert mita.get_last_device_error() == 1
    assert torch.equal(got, mita.mita_qk_norm_rope_axes(q, None, freq, fine, pos)[0])
    assert mita.get_last_device_error() == 0


def test_empty_and_unrotated():
    mita = M()
    pos = torch.zeros(2, 5, dtype=torch.int32, device="cuda")
    w = torch.rand(64, device="cuda")
    q = torch.randn(1, 2, 5, 64, device="cuda")
    none = mita.mita_qk_norm_rope_axes(q, None, None, None, pos, w)[0]
    assert torch.equal(none, mita.mita_qk_norm_rope(q, None, None, w)[0])
    freq, axis = R.inv_freq(64).cuda(), torch.zeros(32, dtype=torch.int32, device="cuda")
    z = q[:, :, :0]
    assert mita.mita_qk_norm_rope_axes(z, z, freq, axis, pos[:, :0], w, w)[0].shape == (1, 2, 0, 64)
    grads = mita.mita_qk_norm_rope_axes_backward(z, z, z, z, freq, axis, pos[:, :0], w, w)
    assert bool((grads[2] == 0).all()) and bool((grads[3] == 0).all())


def test_autograd_against_differences():
    """The autograd function's gradients of a scalar, against central differences of the fp64 formula, and
    every layout of the upstream gradient."""
    mita = M()
    g = gen(6)
    B, Hq, Hkv, N, d = 1, 2, 1, 15, 32
    q, k = (torch.randn(B, h, N, d, generator=g) for h in (Hq, Hkv))
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g) for _ in range(2))
    pos, freq, axis = grid(3, 5), R.inv_freq(d), axis_of("any", d // 2, 2)
    cq, ck = torch.randn(B, Hq, N, d, generator=g), torch.randn(B, Hkv, N, d, generator=g)

    def value(q, k, wq, wk):
        yq = turn(R.norm(q, wq, 1e-6), pos[:, None], axis, freq, False)
        yk = turn(R.norm(k, wk, 1e-6), pos[:, None], axis, freq, False)
        return float((yq * cq.double()).sum() + (yk * ck.double()).sum())

    leaves = [t.cuda().requires_grad_() for t in (q, k, wq, wk)]
    yq, yk = mita.QKNormRopeAxesFunction.apply(leaves[0], leaves[1], freq.cuda(), axis.cuda(), pos.cuda(),
                                               leaves[2], leaves[3])
    grads = torch.autograd.grad(((yq * cq.cuda()).sum() + (yk * ck.cuda()).sum()), leaves,
                                retain_graph=True)
    base = [t.double() for t in (q, k, wq, wk)]
    h = 1e-5
    for i, (t, got) in enumerate(zip(base, grads)):
        for at in (0, t.numel() // 3, t.numel() - 1):
            near = []
            for sign in (1, -1):
                moved = [x.clone() for x in base]
                moved[i].view(-1)[at] += sign * h
                near.append(value(*moved))
            slope = (near[0] - near[1]) / (2 * h)
            # fp32 gradients of terms of size 1 to 10 (64 roundings); differences to h^2 and 2^-50 / h
            assert abs(float(got.flatten()[at]) - slope) <= 64 * R.U * 100 + 1e-8
    turned = cq.transpose(1, 2).contiguous().transpose(1, 2).cuda()
    off = torch.zeros(cq.numel() + 1, device="cuda")[1:].view(cq.shape).copy_(cq)
    want = torch.autograd.grad(yq, leaves[0], cq.cuda(), retain_graph=True)[0]
    for up_grad in (turned, off):
        assert torch.equal(torch.autograd.grad(yq, leaves[0], up_grad, retain_graph=True)[0], want)


def test_captured_and_on_another_stream():
    mita = M()
    g = gen(7)
    q = torch.randn(1, 2, 60, 64, generator=g).bfloat16().cuda()
    pos, axis, freq = grid(3, 4, 5).cuda(), axis_of("sections", 32, 3).cuda(), R.inv_freq(64).cuda()
    w = torch.rand(64, generator=g).cuda()
    want = mita.mita_qk_norm_rope_axes(q, None, freq, axis, pos, w)[0]
    dwant = mita.mita_qk_norm_rope_axes_backward(q, None, q, None, freq, axis, pos, w)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = mita.mita_qk_norm_rope_axes(q, None, freq, axis, pos, w)[0]
        grads = mita.mita_qk_norm_rope_axes_backward(q, None, q, None, freq, axis, pos, w)
    gr.replay()
    assert torch.equal(out, want) and torch.equal(grads[0], dwant[0]) and torch.equal(grads[2], dwant[2])
    pos += 11
    gr.replay()
    assert torch.equal(out, mita.mita_qk_norm_rope_axes(q, None, freq, axis, pos, w)[0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = mita.mita_qk_norm_rope_axes(q, None, freq, axis, pos, w, stream=side)[0]
    torch.cuda.synchronize()
    assert torch.equal(out, got)


def test_python_refusals():
    mita = M()
    q = torch.zeros(2, 2, 6, 64, device="cuda")
    f = torch.ones(32, dtype=torch.float64, device="cuda")
    a = torch.zeros(32, dtype=torch.int32, device="cuda")
    p = torch.zeros(2, 6, dtype=torch.int32, device="cuda")
    mita.mita_qk_norm_rope_axes(q, q, f, a, p)
    n0 = mita.kernel_launches()
    for bad, err in (
            (lambda: mita.mita_qk_norm_rope_axes(q, q, f, a[:16], p), ValueError),
            (lambda: mita.mita_qk_norm_rope_axes(q, q, f, a.long(), p), TypeError),
            (lambda: mita.mita_qk_norm_rope_axes(q, q, f, a, p.long()), TypeError),
            (lambda: mita.mita_qk_norm_rope_axes(q, q, f, a, p[:, :5]), ValueError),
            (lambda: mita.mita_qk_norm_rope_axes(q, q, f, a, p[:, None]), ValueError),
            (lambda: mita.mita_qk_norm_rope_axes(q, q, f, a, p[:0]), mita.MitaError),
            (lambda: mita.mita_qk_norm_rope_axes(q, q, f, a, p.t().contiguous().t()), ValueError),
            (lambda: mita.mita_qk_norm_rope_axes(q, q, f, a.cpu(), p), ValueError),
            (lambda: mita.mita_qk_norm_rope_axes_backward(q, q, q, None, f, a, p), ValueError)):
        with pytest.raises(err):
            bad()
    assert mita.kernel_launches() == n0
