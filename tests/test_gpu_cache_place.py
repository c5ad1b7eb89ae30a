"""mita_cache_append with row starts and lengths at the ends of 32 bits: which rows are written,
which outputs stay as they were, and what the status word says, for each of them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

LO, HI = -2 ** 31, 2 ** 31 - 1

# (row starts, lengths, flagged); two sequences of a table of two pages of eight tokens each
CASES = [
    ((0, 3, 8), (3, 13), False),
    ((2, 5, 7), (3, 13), False),               # rows 0, 1 and 7 are nobody's
    ((-7, 3, 5), (12, 2), False),              # the first sequence's new tokens begin before the rows
    ((0, 3, HI), (3, 16), True),               # more new tokens than the sequence has
    ((LO + 10, HI, HI), (-4, 1), True),        # both differences leave 32 bits
    ((LO, 4, HI), (16, 16), True),
    ((LO, LO + 1, HI), (1, LO), True),
    ((0, 4, 8), (HI, 4), True),                # beyond the table
    ((0, 4, 8), (17, 4), True),
    ((0, 4, 8), (16, -1), True),
    ((0, 4, 8), (0, 4), False),                # an idle slot with rows
    ((9, 9, 9), (4, 4), False),
    ((-7, -3, -1), (4, 4), False),
    ((8, 8, 8), (LO, HI), False),              # rows of nobody: lengths are not looked at
]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("starts,lengths,flagged", CASES)
def test_rows_and_status(starts, lengths, flagged, dt):
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    T, page, d = 8, 8, 32
    g = torch.Generator().manual_seed(0)
    x = torch.randn(T, 4, d, generator=g).to(dt)
    table = torch.tensor([[4, 1], [0, 5]], dtype=torch.int32)
    k, v = torch.zeros(7, 1, page, d, dtype=dt), torch.zeros(7, 1, page, d, dtype=dt)
    q = torch.full((T, 2, d), 9.0, dtype=dt)
    bad = False
    for s in (0, 1):
        begin, end, n = starts[s], starts[s + 1], lengths[s]
        for t in range(max(begin, 0), min(end, T)):
            if n == 0:
                continue
            if n < 0 or n > 2 * page or end - begin > n:
                bad = True
                continue
            pos = n - (end - t)
            at = int(table[s, pos // page])
            k[at, 0, pos % page], v[at, 0, pos % page], q[t] = x[t, 2], x[t, 3], x[t, :2]
    assert bad == flagged
    gx = x.cuda()
    kc, vc, out = torch.zeros_like(k).cuda(), torch.zeros_like(v).cuda(), torch.full_like(q, 9.0).cuda()
    mita.mita_cache_append(gx[:, 2:3], gx[:, 3:], kc, vc, table.cuda(),
                           torch.tensor(lengths, dtype=torch.int32).cuda(),
                           seq_start=torch.tensor(starts, dtype=torch.int32).cuda(), q=gx[:, :2],
                           q_out=out)                  # neither normalised nor turned: bit for bit
    assert mita.get_last_device_error() == int(flagged)
    for got, want in ((kc, k), (vc, v), (out, q)):
        assert torch.equal(got.cpu(), want)
