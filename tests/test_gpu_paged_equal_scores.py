"""mita_paged_attn where all scores are the same number, of any size: every weight is exactly 1 / n."""
import pytest
import torch

import decode_util as R

pytestmark = pytest.mark.gpu

U = R.U
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def M():
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    return mita


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("size", [-1e30, -1e9, -7e6, -1e3, 1e6, 3e6, 7e6, 1.5e7, 3e7, 1e9, 1e12, 1e30])
def test_equal_scores_of_any_size(dt, d, size):
    mita = M()
    for Hq, lengths in ((5, (3, 200, 2500)), (12, (64, 1000))):
        S, page, width = len(lengths), 16, -(-max(lengths) // 16)
        g = torch.Generator().manual_seed(5)
        k = torch.full((S * width, 1, page, d), 7.0, dtype=DT[dt])
        v = torch.randn(S * width, 1, page, d, generator=g).to(DT[dt])
        table = torch.arange(S * width, dtype=torch.int32).view(S, width)
        q = torch.full((S, Hq, d), 1.0 / d, dtype=DT[dt])                      # q k is 7, exactly
        out, lse = mita.mita_paged_attn(q.cuda(), k.cuda(), v.cuda(), table.cuda(),
                                        torch.tensor(lengths, dtype=torch.int32).cuda(), scale=size,
                                        return_lse=True)
        for s, n in enumerate(lengths):
            rows = v[s * width:(s + 1) * width].reshape(-1, d)[:n].double()
            want = rows.mean(0)
            # the weights are alike: what is left are the parts that a weight is given as (2^-16 of it in two bf16
            # values, 2^-21 in tf32 ones, and of a value in these) and the sums
            rel = (2.0 ** -16 if dt == "bf16" else 2.0 ** -20) + 2 * n * U
            bound = rel * rows.abs().mean(0) + R.half_step(DT[dt]) * want.abs()
            R.assert_close(out[s], want.expand(Hq, d), bound.expand(Hq, d), f"{n} keys")
            z = 7 * float(torch.tensor(size)) + float(torch.log(torch.tensor(float(n), dtype=torch.float64)))
            assert float((lse[s].cpu().double() - z).abs().max()) <= 4 * 2 * U * abs(z) + 2 * n * U + 2.0 ** -20
