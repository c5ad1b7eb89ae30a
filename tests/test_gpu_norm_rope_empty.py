"""mita_qk_norm_rope_backward where one part has no rows: its weight's gradient is zero, not
whatever the memory held."""
import pytest
import torch

import decode_util as R

pytestmark = pytest.mark.gpu


def M():
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    return mita


def dirty(mita, d):
    """Leaves NaN in the memory that the next small allocations get."""
    junk = [torch.full((d,), float("nan"), device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    del junk


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("q_weighted", [True, False])
def test_no_key_heads_but_a_key_weight(dt, q_weighted):
    mita = M()
    d = 64
    g = torch.Generator().manual_seed(0)
    q, dy = (torch.randn(2, 3, 7, d, generator=g).to(dt).cuda() for _ in range(2))
    none = torch.empty(2, 0, 7, d, dtype=dt, device="cuda")
    w, freq = torch.ones(d, device="cuda"), R.inv_freq(d).cuda()
    qw = w if q_weighted else None
    want = mita.mita_qk_norm_rope_backward(q, None, dy, None, freq, qw)
    dirty(mita, d)
    got = mita.mita_qk_norm_rope_backward(q, none, dy, none, freq, qw, w)
    assert torch.equal(got[0], want[0]) and got[1].shape == none.shape
    assert bool((got[3] == 0).all())
    if q_weighted:
        assert torch.equal(got[2], want[2])
    else:
        assert got[2] is None


def test_no_key_heads_through_autograd():
    mita = M()
    d = 32
    q = torch.randn(1, 2, 5, d, device="cuda", requires_grad=True)
    k = torch.empty(1, 0, 5, d, device="cuda", requires_grad=True)
    wq, wk = (torch.ones(d, device="cuda", requires_grad=True) for _ in range(2))
    dirty(mita, d)
    qo, ko = mita.QKNormRopeFunction.apply(q, k, R.inv_freq(d).cuda(), wq, wk)
    (qo.sum() + ko.sum()).backward()
    assert bool((wk.grad == 0).all()) and bool((wq.grad != 0).any()) and k.grad.shape == k.shape
