"""mita_paged_attn's cap, softcap * tanh(z / softcap), from the smallest caps to the largest numbers,
against fp64 with a bound that is relative to the score, not to the cap."""
import math

import pytest
import torch

import decode_util as R

pytestmark = pytest.mark.gpu

CAPS = [1e-44, 1e-30, 0.5, 2.0, 10.0, 50.0, 1e3, 1e4, 1e6, 1e9, 1e20, 1e38, 3.4e38]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [0.02, 3.0, 40.0])
@pytest.mark.parametrize("bias", [False, True])
def test_caps(dt, size, bias):
    """Queries and keys have one value that is not zero, keys' of 8 bits: a dot product is one
    product, exact in either type, so that the cap's own roundings are all there is."""
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    S, Hq, d, page, N = 2, 3, 32, 32, 1024
    g = torch.Generator().manual_seed(0)
    k = torch.zeros(S, N, d)
    k[..., 5] = torch.randn(S, N, generator=g) * size
    k[:, ::7, 5] *= 0.01
    v = torch.randn(S, N, d, generator=g)
    k, v = k.bfloat16().to(dt), v.bfloat16().to(dt)
    q = torch.zeros(S, Hq, d, dtype=dt)
    q[..., 5] = torch.tensor([1.0, -0.5, 2.0])
    slopes = torch.tensor([0.0, 0.25, -0.125]) if bias else None
    kc, vc = (t.view(-1, 1, page, d).cuda() for t in (k, v))
    table = torch.arange(S * N // page, dtype=torch.int32).view(S, -1).cuda()
    lengths = torch.full((S,), N, dtype=torch.int32).cuda()
    dot = q[..., 5].double()[..., None] * k[..., 5].double()[:, None]
    for cap in CAPS:
        for scale in (1.0, -0.75):
            cap32, z = torch.tensor(cap).double(), dot * scale      # the cap as a float
            z = cap32 * torch.tanh(z / cap32)
            # x = dot * (scale / cap): 2 roundings, of which tanh passes on no more; below 0.4 the
            # series 4 (its sum is in [0.9, 1]) and 2 products; above it tanh's 2^-20 = 16 and 3
            err = 24 * R.U * z.abs()
            if bias:
                z = z + slopes.double()[:, None] * torch.arange(1 - N, 1).double()
                err = err + 4 * R.U * z.abs()      # slope, product, sum
            # log2 units and the running maximum: a rounding each of the largest score; the
            # exponential's 2^-22 and its difference's rounding
            err = (err + 2 * R.U * z.abs()).amax(-1) + 2 * R.U * z.abs().amax(-1) + 2.0 ** -22
            p = torch.softmax(z, -1)
            want, lse = p @ v.double(), torch.logsumexp(z, -1)
            # sums: at most N / 8 keys to a lane or chain, then the warps' and parts'
            rel = 2 * err + 2 * (N // 8 + 64) * R.U + 2.0 ** -16 * (dt != torch.float32)
            bound = rel[..., None] * (p @ v.double().abs()) + R.half_step(dt) * want.abs()
            got, got_lse = mita.mita_paged_attn(
                q.cuda(), kc, vc, table, lengths, scale=scale, softcap=cap, return_lse=True,
                alibi_slopes=None if slopes is None else slopes.cuda())
            what = f"cap {cap} scale {scale}"
            R.assert_close(got, want, bound, what)
            R.assert_close(got_lse, lse, err + (N // 8 + 64) * R.U + 4 * R.U * lse.abs(), what + " lse")
            if cap == 3.4e38:                      # as without a cap, to fp32's own accuracy
                plain = mita.mita_paged_attn(
                    q.cuda(), kc, vc, table, lengths, scale=scale,
                    alibi_slopes=None if slopes is None else slopes.cuda(), return_lse=True)[1]
                assert bool((plain.cpu().double() - got_lse.cpu().double()).abs().le(
                    2 * err + 4 * R.U * lse.abs()).all())
    assert mita.get_last_device_error() == 0
    assert math.isfinite(float(got.float().sum()))
