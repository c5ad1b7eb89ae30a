"""What the norm-and-rotation gradients leave allocated: their results, and nothing besides, whichever thread and
stream they ran on."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def M():
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    return mita


def inputs(d):
    g = torch.Generator().manual_seed(d)
    x = torch.randn(1, 3, 200, d, generator=g).bfloat16().cuda()
    freq = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).cuda()
    axis = (torch.arange(d // 2, dtype=torch.int32) % 2).cuda()
    at = torch.arange(200, dtype=torch.int32).cuda()
    return x, freq, axis, torch.stack((at // 14, at % 14)), torch.ones(d, device="cuda")


def held():
    torch.cuda.synchronize()
    return torch.cuda.memory_allocated()


def test_gradients_keep_no_memory():
    mita = M()
    x, freq, axis, at, w = inputs(64)
    mita.mita_qk_norm_rope_backward(x, None, x, None, freq, w)         # what the first call loads
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()

    def calls():
        for s in streams:
            mita.mita_qk_norm_rope_backward(x, None, x, None, freq, w, stream=s)
            mita.mita_qk_norm_rope_axes_backward(x, None, x, None, freq, axis, at, w, stream=s)

    before = held()
    calls()
    assert held() == before
    thread = threading.Thread(target=calls)
    thread.start()
    thread.join()
    assert held() == before


def test_backward_passes_keep_no_memory():
    """The autograd engine runs them on a thread of its own."""
    mita = M()
    x, freq, axis, at, w = inputs(32)

    def step():
        q, weight = x.clone().requires_grad_(), w.clone().requires_grad_()
        y, _ = mita.QKNormRopeAxesFunction.apply(q, None, freq, axis, at, weight)
        z, _ = mita.QKNormRopeFunction.apply(y, None, freq, weight)
        z.float().square().sum().backward()
        return q.grad is not None and weight.grad is not None

    mita.mita_qk_norm_rope_backward(x, None, x, None, freq, w)         # what the first call loads
    mita.workspace_release()
    before = held()
    assert step()
    mita.workspace_release()
    assert held() == before
