"""mita_paged_attn in fp32: what its products keep of a factor's 24 bits, one key at a time, so that
nothing else is lost."""
import pytest
import torch

import decode_util as R
from test_gpu_paged import M

pytestmark = pytest.mark.gpu

MOST = torch.finfo(torch.float32).max


def one_key(q, k, v):
    """(out, lse) of sequences of one key each: q, k, v [S, 1, d]."""
    mita = M()
    S, _, d = q.shape
    kc, vc = torch.zeros(S, 1, 16, d, device="cuda"), torch.zeros(S, 1, 16, d, device="cuda")
    kc[:, :, 0], vc[:, :, 0] = k, v
    table = torch.arange(S, dtype=torch.int32, device="cuda").view(S, 1)
    n = torch.ones(S, dtype=torch.int32, device="cuda")
    out, lse = mita.mita_paged_attn(q, kc, vc, table, n, scale=1.0, return_lse=True)
    assert mita.get_last_device_error() == 0
    return out, lse[:, 0]


def numbers(*shape):
    """Of all mantissas, in (0.5, 4), either sign."""
    g = torch.Generator().manual_seed(0)
    x = (1 + torch.rand(shape, generator=g)) * 2.0 ** torch.randint(-1, 2, shape, generator=g)
    return (x * (torch.randint(0, 2, shape, generator=g) * 2 - 1)).cuda()


@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_a_value_comes_out_to_2_of_its_last_places_and_unbiased(d):
    S = 512
    v = numbers(S, 1, d)
    q, k = torch.zeros(S, 1, d, device="cuda"), torch.zeros(S, 1, d, device="cuda")
    out, _ = one_key(q, k, v)                  # the weight is 1, its sum 1: nothing else is rounded
    off = (out.double() - v.double()) / v.double().abs()
    assert float(off.abs().max()) <= 4 * R.U   # two units of 2^-23 of the power of two below
    # 11 of 13 bits, cut: 0.9 units short on average, 1.2 U of the value; rounded, 0.1 units
    assert abs(float((off * v.sign()).mean())) <= 0.5 * R.U
    eight = v.bfloat16().float()               # what fits in two halves stays bit for bit
    assert torch.equal(one_key(q, k, eight)[0], eight)


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("turned", [False, True])
def test_a_score_is_as_near_and_unbiased(d, turned):
    """One value of the query is 1 and the key's any number (or the other way round): the logarithm of
    the sum is that number."""
    S = 4096
    x = numbers(S)
    one, k = torch.zeros(S, 1, d, device="cuda"), torch.zeros(S, 1, d, device="cuda")
    one[:, 0, 3], k[:, 0, 3] = 1.0, x
    q, k = (k, one) if turned else (one, k)
    _, lse = one_key(q, k, torch.zeros_like(k))
    off = (lse.double() - x.double()) / x.double().abs()
    # the factor's 4 U (a key's are 2), to log2 units and back: a constant's and a product's each
    assert float(off.abs().max()) <= (4 + 4) * R.U
    assert abs(float((off * x.sign()).mean())) <= 0.7 * R.U


def test_the_largest_numbers():
    """Keys up to the largest number against queries so small that the score is a few; values up to a
    2^-21 below it."""
    d, S = 64, 8
    big = torch.tensor([MOST, -MOST, MOST * (1 - 2.0 ** -13), -MOST * (1 - 2.0 ** -12), MOST / 2, 1e38,
                        -3e38, 3.40e38]).cuda()
    q, k, v = (torch.zeros(S, 1, d, device="cuda") for _ in range(3))
    q[:, 0, 7], k[:, 0, 7] = 2.0 ** -125, big
    v[:, 0, 0] = big * (1 - 2.0 ** -21)
    out, lse = one_key(q, k, v)
    want = big.double() * 2.0 ** -125
    assert float(((lse.double() - want) / want).abs().max()) <= 8 * R.U
    assert float(((out[:, 0, 0].double() - v[:, 0, 0].double()) / big.double()).abs().max()) <= 4 * R.U
