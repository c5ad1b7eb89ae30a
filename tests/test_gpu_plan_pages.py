"""Page numbers that come back to the pool of mita_cache_plan, and lengths beyond their row of the table."""
import pytest
import torch

import q4_util as Q

pytestmark = pytest.mark.gpu


def M():
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    return mita


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def plan(new, lengths, table, free, count, tokens, page):
    """What the call leaves, held to the restatement; the device's error bits."""
    mita = M()
    want = Q.plan(new, lengths, table, free, count, tokens, page)
    state = i32(lengths), i32(table), i32(free), i32([count])
    got = mita.mita_cache_plan(i32(new), *state, tokens, page)
    error = mita.get_last_device_error()
    assert [t.tolist() for t in got] == [want[k] for k in ("seq_start", "positions", "slots", "granted")]
    assert [t.tolist() for t in state] == [want["new_lengths"], want["table"], want["free"], [want["count"]]]
    return error


@pytest.mark.parametrize("bad", [-1, 6, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("at", [0, 2])
def test_page_numbers_that_come_back_are_looked_at(bad, at):
    """No row stands on the page: it is the push that tells."""
    row = [0, 1, 2]
    assert plan([-1, 0], [40, 3], [row, [5, -1, -1]], [4, 3, -1, -1, -1, -1], 2, 0, 16) == 0
    row[at] = bad
    assert plan([-1, 0], [40, 3], [row, [5, -1, -1]], [4, 3, -1, -1, -1, -1], 2, 0, 16) == 1
    # entries behind the pages that it held are not looked at
    assert plan([-1, 0], [32, 3], [[0, 1, bad], [5, -1, -1]], [4, 3, -1, -1, -1, -1], 2, 0, 16) == 0


def test_a_done_sequence_that_is_too_long_is_cut_to_its_row():
    """Its row comes back as it is, and the flag says so; one of a negative length gives back nothing."""
    assert plan([-1], [200], [[4, 5]], [0, -1, -1, -1, -1, -1], 1, 0, 16) == 1
    assert plan([-1], [33], [[4, -1]], [0, -1, -1, -1, -1, -1], 1, 0, 16) == 1
    assert plan([-1], [-2 ** 31], [[4, 5]], [0, -1, -1, -1, -1, -1], 1, 0, 16) == 1
    assert plan([-1], [2 ** 31 - 1], [[4, 5]], [0, -1, -1, -1, -1, -1], 1, 0, 16) == 1
    assert plan([-1], [32], [[4, 5]], [0, -1, -1, -1, -1, -1], 1, 0, 16) == 0
