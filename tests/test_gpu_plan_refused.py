"""Steps of which some sequences get no page, into the bf16 cache: what a refused sequence holds stays."""
import pytest
import torch

import decode_util as R

pytestmark = pytest.mark.gpu


def M():
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    return mita


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("captured", [False, True])
def test_refused_sequences_keep_their_tokens(captured):
    """Two sequences in a pool of three pages of 4 tokens.  The second has a page full when the pool is empty, and
    offers its next token step after step, until the first one is done and its pages come back."""
    mita = M()
    S, Hq, Hkv, d, page, pool = 2, 2, 1, 32, 4, 3
    g = torch.Generator().manual_seed(1)
    x = torch.randn(20, S, Hq + 2 * Hkv, d, generator=g).bfloat16()
    freq = R.inv_freq(d).cuda()
    lengths, table = i32([0, 0]), torch.full((S, 3), -1, dtype=torch.int32, device="cuda")
    free, count, new = i32([0, 1, 2]), i32([pool]), i32([1, 1])
    kc, vc = (torch.zeros(pool, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rows = torch.zeros(S, Hq + 2 * Hkv, d, dtype=torch.bfloat16, device="cuda")

    def step():
        q, k, v = rows.split((Hq, Hkv, Hkv), 1)
        start, _, _, granted = mita.mita_cache_plan(new, lengths, table, free, count, S, page)
        q = mita.mita_cache_append(k, v, kc, vc, table, lengths, start, q, freq, granted=granted)
        return granted, mita.mita_paged_attn(q, kc, vc, table, lengths)

    if captured:
        state = [t.clone() for t in (lengths, table, free, count, kc, vc)]
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        for t, was in zip((lengths, table, free, count, kc, vc), state):
            t.copy_(was)
    held = [[], []]                     # the value rows that each sequence should hold
    refused = 0
    for t in range(12):
        ask = [1, 1] if t < 8 else [-1, 1] if t == 8 else [0, 1]
        new.copy_(torch.tensor(ask, dtype=torch.int32))
        # packed rows: those of sequences with a new token, one behind the other
        live = [s for s in range(S) if ask[s] == 1]
        rows.zero_()
        for i, s in enumerate(live):
            rows[i] = x[t, s]
        if captured:
            graph.replay()
            granted = outs[0].tolist()
        else:
            granted = step()[0].tolist()
        for s in range(S):
            if ask[s] == -1:
                held[s] = []
            elif granted[s]:
                held[s].append(x[t, s, Hq + Hkv:])
            else:
                refused += ask[s]
        assert lengths.tolist() == [len(h) for h in held]
        for s in range(S):
            for p, want in enumerate(held[s]):
                assert torch.equal(vc[int(table[s, p // page]), :, p % page].cpu(), want), (t, s, p)
    assert refused == 4 and mita.get_last_device_error() == 0


def test_granted_is_checked():
    mita = M()
    k = torch.zeros(2, 1, 32, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(2, 1, 4, 32, dtype=torch.bfloat16, device="cuda")
    args = (k, k, c, c.clone(), i32([[0], [1]]), i32([1, 1]))
    for bad, err in ((i32([1]), ValueError), (i32([1, 1]).long(), TypeError),
                     (torch.ones(2, dtype=torch.int32), ValueError)):
        with pytest.raises(err):
            mita.mita_cache_append(*args, granted=bad)


def test_granted_on_another_stream():
    mita = M()
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(2, 1, 32, generator=g).bfloat16().cuda() for _ in range(2))
    kc, vc = (torch.zeros(2, 1, 4, 32, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, n, granted = i32([[0], [1]]), i32([1, 1]), i32([0, 1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mita.mita_cache_append(k, v, kc, vc, table, n, granted=granted, stream=side)
    torch.cuda.synchronize()
    assert bool((vc[0] == 0).all()) and torch.equal(vc[1, :, 0], v[1]) and n.tolist() == [1, 1]
