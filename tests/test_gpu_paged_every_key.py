"""mita_paged_attn: every key counts exactly once, wherever it lies in a tile, a warp's part of one,
a CTA's share or a page.

With queries of zero all keys weigh the same: 1 / n of them.  Values are zero but for one key in each
column, so that a key left out, or taken twice, changes its column by all of it, where a sum over
tens of thousands of keys of one size would hide it among its roundings."""
import math

import pytest
import torch

import decode_util as R

pytestmark = pytest.mark.gpu

CASES = [
    # lengths, Hq, Hkv, d, page, dtype, window
    ((40000,), 4, 1, 64, 64, torch.bfloat16, 0),            # cut over every SM
    ((9001, 5, 0, 7777, 1), 4, 2, 128, 16, torch.bfloat16, 0),
    ((20011, 33), 16, 1, 128, 32, torch.bfloat16, 0),       # 16 query rows in a CTA
    ((15000,), 20, 1, 64, 8, torch.bfloat16, 0),            # two blocks of query rows
    ((12345, 100), 2, 2, 32, 128, torch.bfloat16, 0),
    ((9999,), 3, 1, 16, 16, torch.bfloat16, 7000),
    (tuple(1 + i * 37 % 300 for i in range(130)), 2, 1, 64, 16, torch.bfloat16, 0),
    ((16001, 5), 4, 1, 64, 16, torch.float32, 0),
    ((9001, 64, 3), 3, 1, 128, 4, torch.float32, 0),
    ((12000,), 10, 1, 32, 64, torch.float32, 0),
    ((8000,), 1, 1, 16, 256, torch.float32, 5003),
    (tuple(i * 29 % 90 for i in range(200)), 4, 1, 32, 8, torch.float32, 0),
]


@pytest.mark.parametrize("case", CASES,
                         ids=lambda c: f"{len(c[0])}x{max(c[0])}-" + "-".join(map(str, c[1:])))
def test_every_key_counts_once(case):
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    lengths, Hq, Hkv, d, page, dt, window = case
    cache = R.Cache(lengths, Hkv, page, d, dt, fill=False)
    S = len(lengths)
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    seen = (n.clamp(max=window) if window else n).double()
    first = (n - window).clamp(min=0) if window else torch.zeros_like(n)
    table, kc = cache.table.cuda(), torch.zeros_like(cache.k).cuda()
    vc, q = torch.zeros_like(kc), torch.zeros(S, Hq, d, dtype=dt, device="cuda")
    seq, col = torch.arange(S, device="cuda")[:, None], torch.arange(d, device="cuda")[None]
    # fp32 sums of ones are exact; then a division, a product and the result's own rounding
    off = R.half_step(dt) + 4 * R.U
    bad = torch.zeros((), dtype=torch.bool, device="cuda")
    for at in range(0, max(lengths), d):
        key = at + col.expand(S, d)
        there = key < n[:, None]
        s, c = (seq.expand(S, d)[there], col.expand(S, d)[there])
        pages, rows = table[s, key[there] // page].long(), key[there] % page
        vc[pages, :, rows, c] = 1.0
        out, lse = mita.mita_paged_attn(q, kc, vc, table, n, window=window, return_lse=True)
        vc[pages, :, rows, c] = 0.0
        want = (there & (key >= first[:, None])).double()[:, None]
        got = out.double() * seen.clamp(min=1)[:, None, None]
        bad |= ((got - want).abs() > off * want).any()
        if at == 0:
            some = n > 0
            assert bool(((lse.double() - seen.log()[:, None]).abs()[some] <= 4 * R.U * (
                1 + seen.log()[some, None])).all())
            assert bool((lse[~some] == -math.inf).all())
    assert not bool(bad)
    assert mita.get_last_device_error() == 0
