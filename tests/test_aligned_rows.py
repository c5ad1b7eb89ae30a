"""What the autograd function hands to the gradient kernel: rows that start on 16-byte boundaries,
whatever the upstream gradient looks like."""
import pytest
import torch

from sparse_top_landmark_gb300 import mita


def views(dt):
    """Gradients of shape [2, 3, 4, 16] with the same values, laid out in every way."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(2, 3, 4, 16, generator=g).to(dt)

    def put(base, view):
        view(base).copy_(x)
        return view(base)
    yield "dense", x
    for off in (1, 2, 3, 5, 8):
        flat = torch.zeros(x.numel() + 16, dtype=dt)
        yield f"dense, {off} values on", put(flat, lambda b: b[off:off + x.numel()].view(x.shape))
    yield "token-major", put(torch.zeros(2, 4, 3, 16, dtype=dt), lambda b: b.transpose(1, 2))
    yield "rows apart", put(torch.zeros(2, 3, 4, 24, dtype=dt), lambda b: b[..., 8:])
    yield "rows off", put(torch.zeros(2, 3, 4, 19, dtype=dt), lambda b: b[..., 3:])
    yield "columns apart", put(torch.zeros(2, 3, 4, 32, dtype=dt), lambda b: b[..., ::2])
    yield "transposed", put(torch.zeros(2, 3, 16, 4, dtype=dt), lambda b: b.transpose(2, 3))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rows_are_aligned_and_the_same(dt):
    step = 128 // torch.finfo(dt).bits
    x = next(views(dt))[1]
    for name, t in views(dt):
        assert torch.equal(t, x), name
        got = mita._aligned_rows(t)
        assert torch.equal(got, x), name
        assert got.data_ptr() % 16 == 0 and got.stride(-1) == 1, name
        assert all(s % step == 0 for s in got.stride()[:-1]), name
    broadcast = x[:, :1].expand(2, 3, 4, 16)
    assert mita._aligned_rows(broadcast) is broadcast


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_gradient_that_starts_off_a_boundary(dt):
    """The upstream gradient is a slice of a flat one, an odd number of values from its start."""
    from sparse_top_landmark_gb300 import build
    build.build()
    g = torch.Generator().manual_seed(1)
    q, k = (torch.randn(2, h, 5, 32, generator=g).to(dt).cuda().requires_grad_() for h in (4, 2))
    w = torch.ones(32, device="cuda", requires_grad=True)
    freq = (10000.0 ** (-torch.arange(0, 32, 2, dtype=torch.float64) / 32)).cuda()
    up = torch.randn(1 + (4 + 2) * 2 * 5 * 32, generator=g).to(dt).cuda()
    qo, ko = mita.QKNormRopeFunction.apply(q, k, freq, w, w)
    torch.cat((up[:1], qo.flatten(), ko.flatten())).backward(up)
    n = qo.numel()
    want = mita.mita_qk_norm_rope_backward(q.detach(), k.detach(), up[1:1 + n].clone().view(qo.shape),
                                           up[1 + n:].clone().view(ko.shape), freq, w.detach(),
                                           w.detach())
    assert torch.equal(q.grad, want[0]) and torch.equal(k.grad, want[1])
    assert torch.equal(w.grad, want[2] + want[3])
