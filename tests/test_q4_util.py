"""The restatement of the 4-bit codes, against the format's definition."""
import numpy as np
import pytest
import torch

import q4_util as Q


def test_scale_bytes_are_half_bits():
    assert Q.SCALES[0] == 0 and Q.SCALES[8] == 2.0 ** -14 and Q.SCALES[247] == 61440
    assert Q.SCALES[1] == 2.0 ** -17 and Q.SCALES == sorted(Q.SCALES)
    assert np.isnan(Q.scale_of_byte(255))


@pytest.mark.parametrize("a,want", [(0.0, 0.0), (7.0, 1.0), (7 * 61440.0, 61440.0), (1e30, 61440.0),
                                    (7 * 1.0625, 1.0), (7 * 1.1875, 1.25), (7 * 2.0 ** -17, 2.0 ** -17),
                                    (7 * 0.4 * 2.0 ** -17, 0.0)])
def test_scales_are_rounded_to_the_nearest(a, want):
    assert Q.scale_of_byte(Q.scale_byte(a)) == want


@pytest.mark.parametrize("d", [32, 64, 128])
def test_rows_come_back(d):
    x = torch.randn(5, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    code, byte, value = Q.quantise(x)
    page = torch.zeros(16 * 17 * d // 32, dtype=torch.uint8)
    for r in range(5):
        page = Q.put_row(page, code[r], byte[r], 3 * r, 16, d)
    for r in range(5):
        c, b = Q.read_row(page, 3 * r, 16, d)
        assert torch.equal(c, code[r]) and torch.equal(b, byte[r])
    # every value within half a step, and every one a bf16 number
    s = torch.tensor([Q.scale_of_byte(int(t)) for t in byte.flatten()]).repeat_interleave(32).view(5, d)
    assert bool(((value - x.float()).abs() <= s * (0.5 + 2.0 ** -19)).all())
    assert torch.equal(value.bfloat16().float(), value)


def test_halves_go_towards_zero():
    x = torch.zeros(32)
    x[0] = 7.0                                   # scale 1
    x[1:15] = torch.tensor([n + 0.5 for n in range(-7, 7)])
    want = torch.tensor([float(np.sign(n + 0.5) * np.ceil(abs(n + 0.5) - 0.5)) for n in range(-7, 7)])
    assert torch.equal(Q.quantise(x[None])[2][0, 1:15], want)


def test_every_bf16_quotient_keeps_off_the_halves():
    """x / s for bf16 x (8 bits) and a scale of 4 bits is n + 1/2 exactly or further off it than the factor
    1 - 2^-20 reaches, so that codes are those of exact arithmetic."""
    m, s = np.arange(128, 256, dtype=np.float64)[:, None], np.arange(8, 16, dtype=np.float64)[None]
    for e in range(-3, 4):
        y = m / 128 * 2.0 ** e / (s / 8)
        off = np.abs(y - np.floor(y) - 0.5)
        y, off = y[(off > 0) & (y < 8)], off[(off > 0) & (y < 8)]
        assert (off > y * 2.0 ** -19).all()


def test_plan_of_one_step():
    # page of 4; three sequences: 4 held (+1: a page), 2 held (+1: none), done (its page comes back)
    got = Q.plan([1, 1, -1], [4, 2, 3], [[5, -1], [6, -1], [7, -1]], [1, 2, 0, 0, 0, 0, 0, 0], 2, 3, 4)
    assert got["table"] == [[5, 7], [6, -1], [7, -1]] and got["count"] == 2
    assert got["slots"] == [28, 26, -1] and got["positions"] == [4, 2, 0]
    assert got["new_lengths"] == [5, 3, 0] and got["seq_start"] == [0, 1, 2, 2]
