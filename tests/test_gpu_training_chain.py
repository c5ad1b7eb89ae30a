"""The training path: queries and keys through QKNormRopeFunction into MiTAFunction, gradients back to
the projection's output and the norm weights."""
import pytest
import torch

import decode_util as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_norm_rope_into_mita(dt):
    """Autograd through both against the library's own gradient calls one after the other.  Those of
    MiTA are added by atomics, in another order each time: sums of at most N terms in fp32, of
    which each is at most 16 times the largest gradient here, are off by N * U * 16 of it; a bf16 cast
    of them by one step more, and each passes through the norm's gradient's two products."""
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    B, H, N, d, m, topk = 2, 2, 96, 64, 8, 12
    g = torch.Generator().manual_seed(0)
    x = torch.randn(B, N, 3 * H, d, generator=g).to(dt).cuda()
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g).cuda() for _ in range(2))
    up = torch.randn(B, H, N, d, generator=g).to(dt).cuda()
    freq = R.inv_freq(d).cuda()

    def parts(t):
        return (t[:, :, i * H:(i + 1) * H].transpose(1, 2) for i in range(3))
    leaf, lq, lk = (t.clone().requires_grad_() for t in (x, wq, wk))
    q, k, v = parts(leaf)
    qr, kr = mita.QKNormRopeFunction.apply(q, k, freq, lq, lk)
    out = mita.MiTAFunction.apply(qr, kr, v, 1, N, m, topk)
    out.backward(up)

    q, k, v = parts(x)
    qr, kr = mita.mita_qk_norm_rope(q, k, freq, wq, wk)
    want_out = mita.mita_forward(qr, kr, v.contiguous(), 1, N, m, topk)
    assert torch.equal(out, want_out)
    dqr, dkr, dv = (t.to(dt) for t in mita.mita_backward(qr, kr, v.contiguous(), up, 1, N, m, topk))
    dq, dk, dwq, dwk = mita.mita_qk_norm_rope_backward(q, k, dqr, dkr, freq, wq, wk)
    step = 16 * N * R.U + (2 * R.half_step(dt) if dt != torch.float32 else 0.0)
    for got, want in zip(parts(leaf.grad), (dq, dk, dv)):
        assert bool(torch.isfinite(got.float()).all()) and bool((got != 0).any())
        size = want.double().abs().max()
        assert bool((got.double() - want.double()).abs().max() <= 4 * step * size)
    for got, want, each in ((lq.grad, dwq, dqr), (lk.grad, dwk, dkr)):
        # B * H * N rows of the size of `each`, of which every one may be a step off
        size = each.double().abs().sum((0, 1, 2)).max()
        assert bool((got.double() - want.double()).abs().max() <= 8 * step * size)
