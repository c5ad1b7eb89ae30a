"""The pages of a serving step on the GPU: mita_cache_plan against a plain restatement (q4_util.py)."""
import random

import pytest
import torch

import q4_util as Q

pytestmark = pytest.mark.gpu


def M():
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    return mita


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def check(new, lengths, table, free, count, tokens, page, in_place=False, error=0):
    mita = M()
    want = Q.plan(new, lengths, table, free, count, tokens, page)
    S, width = len(new), len(table[0]) if table else 0
    n, tb, st, ct = ints(lengths), ints(table).view(S, width), ints(free), ints([count])
    after, ct2 = (n, ct) if in_place else (torch.full_like(n, -77), torch.full_like(ct, -77))
    got = mita.mita_cache_plan(ints(new), n, tb, st, ct, tokens, page,
                               new_lengths=None if in_place else after,
                               new_free_count=None if in_place else ct2)
    assert mita.get_last_device_error() == error
    for name, t in zip(("seq_start", "positions", "slots", "granted"), got):
        assert t.tolist() == want[name], name
    assert got[2].dtype == torch.int64 and got[1].dtype == torch.int32
    assert after.tolist() == want["new_lengths"]
    assert tb.tolist() == want["table"]
    assert st.tolist() == want["free"]
    assert ct2.tolist() == [want["count"]]
    if not in_place:
        assert n.tolist() == list(lengths) and ct.tolist() == [count]
    return want


def random_step(rng, S, most, page, width, spare, done=0.1, prompts=0.3, padded=0):
    """Sequences with pages of their own, and a pool with `spare` more free pages than are needed."""
    lengths, new = [], []
    for _ in range(S):
        lengths.append(rng.randrange(0, most + 1))
        r = rng.random()
        new.append(-1 if r < done else rng.randrange(0, most + 1) if r < done + prompts else
                   rng.choice([0, 1, 1, 1]))
    held = [-(-n // page) for n in lengths]
    need = sum(-(-(n + max(x, 0)) // page) - h for n, x, h in zip(lengths, new, held))
    free = max(0, need + spare)
    pool = list(range(sum(held) + free))
    rng.shuffle(pool)
    table, at = [], free
    for h in held:
        table.append(pool[at:at + h] + [-1] * (width - h))
        at += h
    stack = pool[:free] + [-1] * (len(pool) - free)
    return new, lengths, table, stack, free, sum(max(x, 0) for x in new) + padded, page


@pytest.mark.parametrize("S,most,page,spare,padded", [
    (1, 5, 16, 0, 0), (3, 40, 16, 2, 3), (17, 100, 4, 0, 1), (200, 300, 16, 10, 8), (60, 2000, 64, 0, 5),
    (1023, 20, 16, 0, 0), (1024, 30, 8, 5, 2), (1025, 30, 8, 5, 2), (3000, 10, 1, 7, 0), (5, 30000, 16, 0, 9),
    (40, 200, 16, -20, 4), (300, 50, 8, -200, 0), (2000, 40, 4, -900, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(S, most, page, spare, padded, in_place):
    rng = random.Random(S * 31 + most)
    width = -(-2 * most // page) + 1
    check(*random_step(rng, S, most, page, width, spare, padded=padded), in_place=in_place)


def test_no_sequences_and_no_rows():
    check([], [], [], [3, 4], 2, 5, 16)
    check([0, 0], [3, 0], [[1], [0]], [2, -1, -1], 1, 0, 16)
    check([-1, -1], [33, 0], [[1, 2, 0], [9, 9, 9]], [3, -1, -1, -1], 1, 0, 16)


def test_first_come_first_served():
    """Three free pages: the second sequence would need two more than are left, those behind it that need a
    page get none, those that need none go on."""
    want = check([20, 40, 1, 1, 5], [0, 0, 16, 3, 10], [[-1, -1, -1], [-1, -1, -1], [4, -1, -1], [5, -1, -1],
                                                        [6, -1, -1]],
                 [0, 1, 2, -1, -1, -1, -1], 3, 67, 16)
    assert want["granted"] == [20, 0, 0, 1, 5]


@pytest.mark.parametrize("spare", [-60, 0, 5])
def test_every_page_is_free_or_held_once(spare):
    """Also where sequences that need no page go on behind one that is refused: what the refused ones would
    have needed stays on the stack."""
    for seed in range(7):
        new, lengths, table, stack, count, tokens, page = random_step(random.Random(seed), 50, 60, 16, 9, spare)
        state = ints(lengths), ints(table), ints(stack), ints([count])
        granted = M().mita_cache_plan(ints(new), *state, tokens, page)[3].tolist()
        n, rows, free, left = (x.tolist() for x in state)
        if spare < 0:
            assert any(x > 0 and g == 0 for x, g in zip(new, granted))
        held = [p for s, row in enumerate(rows) for p in row[:-(-n[s] // page)]]
        assert sorted(held + free[:left[0]]) == list(range(len(stack)))


def test_pages_that_come_back_are_handed_out_again():
    want = check([-1, 30, -1], [20, 0, 1], [[3, 4], [-1, -1], [5, -1]], [0, -1, -1, -1, -1, -1], 1, 30, 16)
    assert want["table"][1] == [5, 4] and want["count"] == 2


def test_rows_and_table_that_are_too_short():
    # the second sequence's rows end behind the step's, the third's begin there
    check([10, 10, 1], [0, 0, 0], [[-1], [-1], [-1]], [0, 1, 2], 3, 15, 16)
    # one page a sequence: 17 tokens do not fit, 16 do
    check([17, 16, 1], [0, 0, 16], [[-1], [-1], [0]], [1, 2, 3, 0], 3, 40, 16)


def test_bad_numbers_are_flagged_and_get_nothing():
    check([-5, 1, 1, -1], [3, -4, 99, 200], [[0, -1], [1, -1], [2, 3], [4, 5]], [6, 7, 0, 0, 0, 0, 0, 0], 2,
          4, 16, error=1)
    # a page number outside the pool under a row: no place
    check([1, 1, 20], [3, 5, 0], [[99, -1], [-3, -1], [-1, -1]], [0, 1, 55, -1], 3, 22, 16, error=1)
    # a count outside the stack
    check([1], [0], [[-1]], [0, 1], 7, 1, 16, error=1)
    check([1], [0], [[-1]], [0, 1], -2, 1, 16, error=1)
    # more pages come back than the stack holds
    check([-1, -1], [40, 40], [[0, 1, 2], [3, 4, 5]], [7, 6, 9, 9], 2, 0, 16, error=1)


def test_two_plans_at_once():
    """Two pools' plans on two streams, many times over, next to each other: each is right."""
    mita = M()
    steps = [random_step(random.Random(i), 700 + 400 * i, 60, 16, 12, 4, padded=3) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        state = [(ints(new), ints(lengths), ints(table), ints(free), ints([count]), tokens, page)
                 for new, lengths, table, free, count, tokens, page in steps]
        torch.cuda.synchronize()
        outs = [mita.mita_cache_plan(*args, stream=st) for args, st in zip(state, streams)]
        torch.cuda.synchronize()
        for step, args, got in zip(steps, state, outs):
            want = Q.plan(*step)
            assert got[2].tolist() == want["slots"] and args[1].tolist() == want["new_lengths"]
            assert args[2].tolist() == want["table"] and args[4].tolist() == [want["count"]]


def test_most_sequences():
    """2^14 sequences, of which most get one token."""
    rng = random.Random(3)
    check(*random_step(rng, 1 << 14, 20, 16, 4, 0, prompts=0.01, padded=7))


def test_given_outputs_and_another_stream():
    mita = M()
    args = random_step(random.Random(5), 50, 100, 16, 20, 4, padded=3)
    new, lengths, table, free, count, tokens, page = args
    want = Q.plan(*args)
    side = torch.cuda.Stream()
    S = len(new)
    outs = dict(seq_start=ints([0] * (S + 1)), positions=ints([7] * tokens),
                slots=ints([7] * tokens, torch.int64), granted=ints([7] * S))
    ins = (ints(new), ints(lengths), ints(table), ints(free), ints([count]))
    torch.cuda.synchronize()
    got = mita.mita_cache_plan(*ins, tokens, page, stream=side, **outs)
    torch.cuda.synchronize()
    for (name, t), g in zip(outs.items(), got):
        assert g is t and t.tolist() == want[name], name
    assert ins[1].tolist() == want["new_lengths"] and ins[4].tolist() == [want["count"]]


def test_captured_plan_goes_on_from_step_to_step():
    """A decoding step's plan in a graph, in place, until the pool is empty, against the restatement."""
    mita = M()
    S, page, width, pool = 6, 4, 8, 20
    new, lengths = [1] * S, [0, 1, 3, 4, 7, 0]
    held = [-(-n // page) for n in lengths]
    rest = list(range(pool))
    table = []
    for h in held:
        table.append(rest[:h] + [-1] * (width - h))
        rest = rest[h:]
    count = len(rest)
    free = rest + [-1] * (pool - count)
    t_new, t_len, t_table, t_free, t_count = (ints(new), ints(lengths), ints(table), ints(free),
                                              ints([count]))
    mita.mita_cache_plan(t_new, t_len.clone(), t_table.clone(), t_free.clone(), t_count.clone(), S, page)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = mita.mita_cache_plan(t_new, t_len, t_table, t_free, t_count, S, page)
    for step in range(24):
        if step == 15:
            new[2] = -1
        if step == 16:
            new[2] = 1
        t_new.copy_(torch.tensor(new, dtype=torch.int32))
        want = Q.plan(new, lengths, table, free, count, S, page)
        g.replay()
        assert [t.tolist() for t in outs] == [want[k] for k in ("seq_start", "positions", "slots",
                                                                "granted")]
        lengths, table, free, count = want["new_lengths"], want["table"], want["free"], want["count"]
        assert t_len.tolist() == lengths and t_table.tolist() == table and t_count.tolist() == [count]
        assert t_free.tolist() == free
    assert 0 in want["granted"] and mita.get_last_device_error() == 0


def test_python_refusals():
    mita = M()
    good = dict(new_tokens=ints([1, 1]), lengths=ints([0, 0]), page_table=ints([[0], [0]]),
                free_pages=ints([0, 1]), free_count=ints([2]), tokens=2, page_size=16)
    mita.mita_cache_plan(**good)
    n0 = mita.kernel_launches()
    for change, err in ((dict(new_tokens=ints([1])), ValueError), (dict(lengths=ints([0, 0]).long()), TypeError),
                        (dict(page_table=ints([0, 0])), ValueError), (dict(free_count=ints([2, 2])), ValueError),
                        (dict(slots=ints([0, 0])), TypeError), (dict(positions=ints([0])), ValueError),
                        (dict(page_size=12), mita.MitaError), (dict(seq_start=ints([0, 0])), ValueError),
                        (dict(lengths=torch.zeros(2, dtype=torch.int32)), ValueError),
                        (dict(page_table=ints([[0, 1], [2, 3]])[:, :1]), ValueError)):
        with pytest.raises(err):
            mita.mita_cache_plan(**{**good, **change})
    assert mita.kernel_launches() == n0
