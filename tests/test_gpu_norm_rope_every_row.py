"""The weight gradients of mita_qk_norm_rope_backward: every row counts exactly once, and their sums
are as good as fp32 sums in short chains are."""
import pytest
import torch

import decode_util as R

pytestmark = pytest.mark.gpu


def M():
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    return mita


SHAPES = [
    # B, Hq, Hkv, N, d, dtype
    (1, 10, 5, 20011, 128, torch.bfloat16),
    (2, 2, 2, 40000, 64, torch.bfloat16),
    (3, 4, 1, 777, 32, torch.float32),
    (1, 3, 2, 30001, 16, torch.float32),
    (1, 33, 7, 2500, 64, torch.float32),
]


def inputs(shape):
    B, Hq, Hkv, N, d, dt = shape
    g = torch.Generator(device="cuda").manual_seed(0)
    x = [torch.randn(B, h, N, d, generator=g, device="cuda").to(dt) for h in (Hq, Hkv)]
    dy = [torch.randn(t.shape, generator=g, device="cuda").to(dt) for t in x]
    return x, dy, torch.ones(d, device="cuda")


def terms(x, dy, eps):
    """What each row adds to the gradient, fp64 (no rotation)."""
    x = x.double()
    return dy.double() * x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_every_row_counts_once(shape):
    """The upstream gradient is zero but for one row in each column: at the ends of the batch and
    around multiples of 8 to 4096 tokens, where slots, warps, blocks and their strides meet."""
    mita = M()
    B, Hq, Hkv, N, d, dt = shape
    x, _, w = inputs(shape)
    rows = {0, 1, N - 1, N - 2, N // 2}
    for step in (8, 16, 32, 64, 128, 304 * 16, 304 * 32, 152 * 16, 4096):
        for i in (1, 2, 3, max(1, N // step - 1), N // step):
            rows |= {i * step - 1, i * step, i * step + 1}
    rows = sorted(r for r in rows if 0 <= r < N)
    places = [(b, h, r) for r in rows for b in range(B) for h in {0, 1, -1}]
    for part, heads in ((0, Hq), (1, Hkv)):
        at = [(b, h % heads, r) for b, h, r in places]
        for i in range(0, len(at), d):
            some = torch.tensor(at[i:i + d], device="cuda")
            c = torch.arange(len(some), device="cuda")
            dy = [torch.zeros_like(t) for t in x]
            dy[part][some[:, 0], some[:, 1], some[:, 2], c] = 1.0
            got = mita.mita_qk_norm_rope_backward(x[0], x[1], dy[0], dy[1], None, w, w)[2 + part]
            want = terms(x[part], dy[part], 1e-6).sum((0, 1, 2))
            # one term: the row's square sum, root and product (20 u), and sums with zero
            assert bool(((got.double() - want).abs() <= 32 * R.U * want.abs()).all())


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_sums_in_short_chains(shape):
    """A lane adds at most a few hundred rows one after the other, the rest is added in pairs.  A sum
    of n terms in a chain of L is off by at most L u of their sizes: here that is far below what
    one block's rows add, so that none can be missing."""
    mita = M()
    B, Hq, Hkv, N, d, dt = shape
    x, dy, w = inputs(shape)
    got = mita.mita_qk_norm_rope_backward(x[0], x[1], dy[0], dy[1], None, w, w)
    for t, g, dw in ((x[0], dy[0], got[2]), (x[1], dy[1], got[3])):
        each = terms(t, g, 1e-6).reshape(-1, d)
        want, size = each.sum(0), each.abs().sum(0)
        chain = -(-each.shape[0] // (152 * 16)) + 64       # no fewer slots than 16 an SM
        bound = (chain + 32) * R.U * size
        assert bool(bound.max() < 0.02 * want.abs().max())
        R.assert_close(dw, want.cpu(), bound.cpu(), "dw")


def test_error_of_a_sum_in_pairs():
    """3 x 777 tokens, heads of 32, fp32: the root mean square of the columns' errors.  Added in pairs,
    a level of the tree adds a rounding, at most U / sqrt(3) in the root mean square, of sums
    whose squares add up to those of all terms; there are 16 levels (a lane's rows, eight slots, a
    block's groups, the lanes of a warp, warps), and a term's own four roundings: together
    sqrt(16 + 4) U / sqrt(3) = 2.6 U of the terms' root sum of squares.  (A chain of a block's 64 slots
    alone has sqrt(64 / 2) U / sqrt(3) = 3.3 U.)"""
    mita = M()
    x, dy, w = inputs((3, 4, 1, 777, 32, torch.float32))
    got = mita.mita_qk_norm_rope_backward(x[0], x[1], dy[0], dy[1], None, w, w)[2]
    each = terms(x[0], dy[0], 1e-6).reshape(-1, 32)
    off = ((got.double() - each.sum(0)) ** 2).mean().sqrt()
    assert bool(off <= 2.6 * R.U * (each ** 2).sum(0).mean().sqrt())
