"""The paged cache on the GPU: mita_cache_append and mita_paged_attn against plain fp64
restatements (decode_util.py), and a run of all of them as a decoder uses them."""
import math

import pytest
import torch

import decode_util as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def M():
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    return mita


def up(t):
    return None if t is None else t.cuda()


def lens(*n):
    return torch.tensor(n, dtype=torch.int32)


# --------------------------------------------------------------------------------------------
# attention
# --------------------------------------------------------------------------------------------
EDGES = (0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 0, 700)
ATTN = [
    # lengths, Hq, Hkv, d, page, dtype, options
    ((1,), 1, 1, 64, 16, "bf16", {}),
    (EDGES, 4, 2, 64, 16, "bf16", {}),
    (EDGES, 8, 1, 128, 64, "bf16", {}),
    (EDGES, 3, 3, 32, 1, "bf16", {}),
    (EDGES, 6, 2, 16, 8, "bf16", {}),
    (EDGES, 4, 2, 64, 16, "f32", {}),
    (EDGES, 8, 1, 128, 2, "f32", {}),
    (EDGES, 3, 3, 32, 32, "f32", {}),
    (EDGES, 10, 2, 16, 256, "f32", {}),
    # groups of odd size, of a whole tile of rows, and of more than one
    (EDGES, 7, 1, 64, 32, "bf16", {}),
    (EDGES, 15, 3, 128, 32, "bf16", {}),
    (EDGES, 32, 2, 128, 128, "bf16", {}),
    ((300, 0, 129), 17, 1, 128, 64, "bf16", {}),
    ((300, 0, 129), 40, 1, 64, 64, "bf16", {}),
    ((300, 0, 129), 40, 2, 32, 16, "f32", {}),
    ((300, 0, 129), 17, 1, 128, 16, "f32", {}),
    # options
    (EDGES, 4, 2, 64, 16, "bf16", {"softcap": 2.0}),
    (EDGES, 4, 2, 64, 16, "f32", {"softcap": 2.0}),
    (EDGES, 4, 2, 64, 16, "bf16", {"slopes": True}),
    (EDGES, 4, 2, 64, 16, "f32", {"slopes": True, "softcap": 5.0}),
    (EDGES, 4, 2, 64, 16, "bf16", {"window": 1}),
    (EDGES, 4, 2, 64, 16, "bf16", {"window": 100}),
    (EDGES, 4, 2, 128, 32, "f32", {"window": 130, "slopes": True}),
    (EDGES, 4, 2, 64, 16, "bf16", {"window": 5000, "scale": 0.5}),
    (EDGES, 4, 2, 64, 16, "bf16", {"scale": -1.0}),
    (EDGES, 4, 2, 64, 16, "bf16", {"scale": 0.0}),
    # cut over every SM, and joined
    ((40000,), 4, 1, 64, 64, "bf16", {}),
    ((33333, 5, 20001, 0, 1), 4, 2, 128, 16, "bf16", {"slopes": True}),
    ((30000, 3), 3, 1, 32, 128, "f32", {}),
    ((21111,), 6, 1, 128, 16, "f32", {"window": 20000}),
    # many short sequences: several segments to a CTA
    (tuple(1 + i * 37 % 300 for i in range(130)), 2, 2, 64, 16, "bf16", {}),
    (tuple(i * 29 % 90 for i in range(400)), 4, 1, 32, 8, "f32", {}),
]


def make_slopes(on, Hq):
    return 2.0 ** (-8.0 * torch.arange(1, Hq + 1, dtype=torch.float32) / Hq) if on else None


@pytest.mark.parametrize("case", ATTN, ids=lambda c: f"{len(c[0])}x{max(c[0])}-" + "-".join(
    map(str, c[1:6])) + "".join(f"-{k}{v}" for k, v in c[6].items()))
def test_attention(case):
    mita = M()
    lengths, Hq, Hkv, d, page, dt, opt = case
    opt = dict(opt)
    slopes = make_slopes(opt.pop("slopes", False), Hq)
    cache = R.Cache(lengths, Hkv, page, d, DT[dt], slack=len(lengths) % 3)
    q = torch.randn(len(lengths), Hq, d, generator=torch.Generator().manual_seed(2)).to(DT[dt])
    args = (q.cuda(), cache.k.cuda(), cache.v.cuda(), cache.table.cuda(), lens(*lengths).cuda())
    out, lse = mita.mita_paged_attn(*args, alibi_slopes=up(slopes), return_lse=True, **opt)
    assert mita.get_last_device_error() == 0
    want, bound, lwant, lbound = R.paged_attn(q, cache, lengths, slopes=slopes, **opt)
    R.assert_close(out, want, bound, "out")
    empty = torch.tensor([n == 0 for n in lengths])
    assert bool((lse.cpu()[empty] == -math.inf).all()) and bool((out.cpu()[empty] == 0).all())
    R.assert_close(lse[~empty.cuda()], lwant[~empty], lbound[~empty], "lse")
    again = mita.mita_paged_attn(*args, alibi_slopes=up(slopes), **opt)
    assert torch.equal(again, out)


def test_attention_matches_dense_attention():
    """A full cache, each sequence's last query: the row that dense attention gives it.  Both are
    bf16 kernels; each is within its own bound of the fp64 value, dense attention's weights
    being bf16 (half a step each)."""
    mita = M()
    B, H, N, d, page = 2, 2, 512, 64, 64
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(B, H, N, d, generator=g).bfloat16().cuda() for _ in range(3))
    dense = mita.mita_dense_attn(q, k, v)[:, :, -1]
    pages = lambda t: t.view(B, H, N // page, page, d).transpose(1, 2).reshape(-1, H, page, d).contiguous()  # noqa: E731
    table = torch.arange(B * N // page, dtype=torch.int32, device="cuda").view(B, -1)
    out = mita.mita_paged_attn(q[:, :, -1], pages(k), pages(v), table, lens(N, N).cuda())
    size = v.float().abs().max().item()
    assert (out.float() - dense.float()).abs().max().item() <= 4 * 2.0 ** -8 * size


def test_bad_pages_are_left_out_and_flagged():
    mita = M()
    for dt in ("bf16", "f32"):
        lengths = (300, 40, 16, 200)
        cache = R.Cache(lengths, 2, 16, 64, DT[dt])
        cache.table[0, 3], cache.table[0, 7], cache.table[3, 12] = -1, cache.num, 2 ** 30
        cache.table[2, 0] = -5                     # nothing is left of sequence 2
        q = torch.randn(4, 4, 64, generator=torch.Generator().manual_seed(2)).to(DT[dt])
        out, lse = mita.mita_paged_attn(q.cuda(), cache.k.cuda(), cache.v.cuda(),
                                        cache.table.cuda(), lens(*lengths).cuda(), return_lse=True)
        assert mita.get_last_device_error() == 1
        want, bound, lwant, lbound = R.paged_attn(q, cache, lengths, skip_bad=True)
        R.assert_close(out, want, bound, "out")
        assert bool((lse[2].cpu() == -math.inf).all()) and bool((out[2] == 0).all())
        live = [0, 1, 3]
        R.assert_close(lse[live], lwant[live], lbound[live], "lse")


def test_bad_lengths_are_cut_and_flagged():
    mita = M()
    lengths = (64, 48)
    cache = R.Cache(lengths, 1, 16, 32, torch.float32)     # 4 pages a row of the table
    q = torch.randn(2, 2, 32, generator=torch.Generator().manual_seed(2))
    told = lens(1000, -3).cuda()
    out = mita.mita_paged_attn(q.cuda(), cache.k.cuda(), cache.v.cuda(), cache.table.cuda(), told)
    assert mita.get_last_device_error() == 1
    want, bound, _, _ = R.paged_attn(q, cache, (64, 0))
    R.assert_close(out, want, bound, "out")


def test_extreme_scores():
    """Scores far outside exp's range, keys whose score is -inf, and a key that is NaN."""
    mita = M()
    for dt in ("bf16", "f32"):
        cache = R.Cache((200, 200, 30, 150), 1, 16, 64, DT[dt])
        q = torch.randn(4, 2, 64, generator=torch.Generator().manual_seed(2)).to(DT[dt])
        q[0] *= 100                                        # scores in the hundreds
        q[1:3, :, 0] = 1.0
        for p in (0, 3, 17, 199):                          # some keys at -inf
            cache.k[cache.table[1, p // 16], 0, p % 16, 0] = -math.inf
        for p in range(30):                                # all of them
            cache.k[cache.table[2, p // 16], 0, p % 16, 0] = -math.inf
        cache.v[cache.table[3, 5], 0, 3, 7] = math.nan     # one value: its column alone
        out, lse = mita.mita_paged_attn(q.cuda(), cache.k.cuda(), cache.v.cuda(),
                                        cache.table.cuda(), lens(200, 200, 30, 150).cuda(),
                                        return_lse=True)
        assert mita.get_last_device_error() == 0
        want, bound, lwant, lbound = R.paged_attn(q, cache, (200, 0, 0, 0))
        R.assert_close(out[:1], want[:1], bound[:1], "large scores")
        seen = [p for p in range(200) if p not in (0, 3, 17, 199)]
        page = cache.table[1, torch.tensor(seen) // 16].long()
        k, v = (t[page, 0, torch.tensor(seen) % 16].double() for t in (cache.k, cache.v))
        p = torch.softmax(q[1].double() @ k.T / 8, -1)
        off = (out[1].cpu().double() - p @ v).abs()
        assert bool((off <= R.half_step(DT[dt]) * (p @ v).abs() + 2.0 ** -13 * (p @ v.abs())).all())
        assert bool((out[2] == 0).all()) and bool((lse[2] == -math.inf).all())
        nan = torch.isnan(out[3].cpu())
        assert bool(nan[:, 7].all()) and int(nan.sum()) == 2


def test_strided_queries_out_and_table_views():
    mita = M()
    lengths = (100, 33)
    cache = R.Cache(lengths, 2, 16, 64, torch.bfloat16)
    qkv = torch.randn(2, 10, 64, generator=torch.Generator().manual_seed(2)).bfloat16()
    q = qkv[:, 1:7]
    want, bound, _, _ = R.paged_attn(q, cache, lengths)
    gq = qkv.cuda()[:, 1:7]
    out = torch.full((4, 6, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    got = mita.mita_paged_attn(gq, cache.k.cuda(), cache.v.cuda(), cache.table.cuda(),
                               lens(*lengths).cuda(), out=out[1:3])
    R.assert_close(got, want, bound, "out")
    assert bool((out[0] == 5).all()) and bool((out[3] == 5).all())
    one = q[:, :1].expand(2, 6, 64)                        # one query for all heads
    want, bound, _, _ = R.paged_attn(one, cache, lengths)
    got = mita.mita_paged_attn(gq[:, :1].expand(2, 6, 64), cache.k.cuda(), cache.v.cuda(),
                               cache.table.cuda(), lens(*lengths).cuda())
    R.assert_close(got, want, bound, "broadcast query")


def test_no_sequences():
    mita = M()
    n0 = mita.kernel_launches()
    kc = torch.zeros(3, 2, 16, 64, device="cuda")
    table, n = torch.zeros(0, 4, dtype=torch.int32, device="cuda"), lens().cuda()
    q = torch.zeros(0, 4, 64, device="cuda")
    assert mita.mita_paged_attn(q, kc, kc, table, n).shape == (0, 4, 64)
    assert mita.mita_cache_append(q[:, :2], q[:, :2], kc, kc, table, n, q=q).shape == (0, 4, 64)
    assert mita.kernel_launches() == n0


# --------------------------------------------------------------------------------------------
# append
# --------------------------------------------------------------------------------------------
APPEND = [
    # (cached before, new) of each sequence, Hq, Hkv, d, page, dtype, rot, interleaved, norms, step
    (((0, 1),), 1, 1, 64, 16, "bf16", 64, False, True, True),
    (((5, 1), (0, 1), (15, 1), (16, 1), (31, 1)), 8, 2, 128, 16, "bf16", 128, False, True, True),
    (((5, 1), (None, 1), (15, 1), (None, 1)), 4, 2, 64, 8, "f32", 64, True, True, True),
    (((0, 40), (7, 0), (3, 1), (20, 33)), 4, 2, 32, 16, "bf16", 16, True, True, False),
    (((0, 0), (0, 0), (1, 50)), 6, 3, 16, 1, "f32", 8, False, True, False),
    (((100, 3), (0, 129)), 0, 2, 128, 64, "f32", 128, False, True, False),
    (((100, 3), (0, 129)), 0, 2, 128, 64, "bf16", 0, False, False, False),
    (((1000000, 2), (0, 9)), 2, 1, 64, 256, "bf16", 64, False, False, False),
    (((0, 3000), (17, 4100)), 10, 5, 128, 32, "bf16", 64, False, True, False),
]


def append_reference(case, seed=0):
    plan, Hq, Hkv, d, page, dt, rot, pairs, norms, step = case
    g = torch.Generator().manual_seed(seed)
    lengths = [0 if old is None else old + n for old, n in plan]
    # the cache is not filled: most of a long sequence's pages may be shared
    cache = R.Cache([min(n, 20000) for n in lengths], Hkv, page, d, DT[dt], fill=False, junk=3.0)
    if max(lengths) > 20000:
        wide = torch.zeros(len(lengths), -(-max(lengths) // page), dtype=torch.int32)
        for s, n in enumerate(lengths):
            need = -(-n // page)
            wide[s, :need] = torch.arange(need) % (cache.num - 1) if n > 20000 else cache.num - 1
        cache.table = wide
    T = sum(n for _, n in plan)
    x = torch.randn(T + (0 if step else 4), Hq + 2 * Hkv, d, generator=g).to(DT[dt])
    w = [1 + 0.3 * torch.randn(d, generator=g) for _ in range(2)] if norms else [None, None]
    freq = R.inv_freq(rot) if rot else None
    starts = [0]
    for _, n in plan:
        starts.append(starts[-1] + n)
    k, v, q = (cache.k.double(), cache.v.double(), torch.full((x.shape[0], Hq, d), 9.0).double())
    kb, qb = torch.zeros_like(k), torch.zeros_like(q)
    for s, (old, n) in enumerate(plan):
        if old is None or n == 0:
            continue
        pos = torch.arange(old, old + n)
        rows = x[starts[s]:starts[s + 1]]
        at = pos[:, None]
        if Hq:
            q[starts[s]:starts[s + 1]], qb[starts[s]:starts[s + 1]] = R.norm_rope(
                rows[:, :Hq], w[0], at.expand(n, Hq), freq, 1e-6, pairs)
        y, b = R.norm_rope(rows[:, Hq:Hq + Hkv], w[1], at.expand(n, Hkv), freq, 1e-6, pairs)
        page_of, off = cache.table[s, pos // page].long(), pos % page
        k[page_of, :, off], kb[page_of, :, off] = y, b
        v[page_of, :, off] = rows[:, Hq + Hkv:].double()
    return cache, x, w, freq, lengths, None if step else starts, (q, qb, k, kb, v)


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(map(str, c[1:])))
def test_append(case):
    mita = M()
    plan, Hq, Hkv, d, page, dt, rot, pairs, norms, step = case
    cache, x, w, freq, lengths, starts, (q, qb, k, kb, v) = append_reference(case)
    gx, kc, vc = x.cuda(), cache.k.cuda(), cache.v.cuda()
    q_out = torch.full((x.shape[0], Hq, d), 9.0, dtype=x.dtype, device="cuda")
    got = mita.mita_cache_append(
        gx[:, Hq:Hq + Hkv], gx[:, Hq + Hkv:], kc, vc, cache.table.cuda(), lens(*lengths).cuda(),
        seq_start=None if starts is None else lens(*starts).cuda(),
        q=gx[:, :Hq] if Hq else None, inv_freq=up(freq), q_weight=up(w[0]), k_weight=up(w[1]),
        interleaved=pairs, q_out=q_out if Hq else None)
    assert mita.get_last_device_error() == 0
    R.assert_close(kc, k, kb, "k_cache")
    assert torch.equal(vc.cpu().double(), v)               # untouched rows among them
    if Hq:
        assert got is q_out
        R.assert_close(got, q, qb, "q_out")
    else:
        assert got is None


def test_append_refuses_bad_places():
    """A page outside the cache, a length beyond the table, one below the number of new tokens, a
    negative one: flagged, nothing of those tokens written, the others' written."""
    mita = M()
    d, page = 64, 16
    for plan, told, table_at in (
            (((20, 4), (3, 2)), (24, 5), (0, 1, -1)),
            (((20, 4), (3, 2)), (24, 5), (0, 1, 99)),
            (((20, 4), (3, 2)), (500, 5), None),
            (((20, 4), (3, 2)), (3, 5), None),
            (((20, 4), (3, 2)), (-4, 5), None)):
        case = (plan, 2, 1, d, page, "f32", 64, False, True, False)
        cache, x, w, freq, lengths, starts, (q, qb, k, kb, v) = append_reference(case)
        table = cache.table.clone()
        if table_at:
            table[table_at[0], table_at[1]] = table_at[2]
        kc, vc, gx = cache.k.cuda(), cache.v.cuda(), x.cuda()
        q_out = torch.full((x.shape[0], 2, d), 9.0, device="cuda")
        mita.mita_cache_append(gx[:, 2:3], gx[:, 3:], kc, vc, table.cuda(), lens(*told).cuda(),
                               seq_start=lens(*starts).cuda(), q=gx[:, :2], inv_freq=freq.cuda(),
                               q_weight=w[0].cuda(), k_weight=w[1].cuda(), q_out=q_out)
        assert mita.get_last_device_error() == 1
        own = cache.table[1, 0].item()                     # sequence 1 went through
        others = [p for p in range(cache.num) if p != own]
        assert torch.equal(kc.cpu()[others], cache.k[others])
        assert torch.equal(vc.cpu()[others], cache.v[others])
        R.assert_close(kc[own], k[own], kb[own], "k_cache")
        assert torch.equal(vc[own].cpu().double(), v[own])
        R.assert_close(q_out[4:], q[4:], qb[4:], "q_out")
        assert bool((q_out[:4] == 9).all())


def test_offsets_past_32_bits():
    """A cache of more than 2^32 values: rows far behind that offset are written and read."""
    mita = M()
    pages, Hkv, page, d = 17000, 8, 256, 128               # 4.46e9 values each, 8.9 GB
    kc = torch.zeros(pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    g = torch.Generator().manual_seed(0)
    x = torch.randn(300, Hkv * 3, d, generator=g).bfloat16().cuda()
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    n = lens(300).cuda()
    mita.mita_cache_append(x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:], kc, vc, table, n,
                           seq_start=lens(0, 300).cuda())
    assert torch.equal(kc[pages - 1], x[:256, Hkv:2 * Hkv].transpose(0, 1))
    assert torch.equal(vc[pages - 2][:, :44], x[256:, 2 * Hkv:].transpose(0, 1))
    assert float(kc[:pages - 2].abs().sum(dtype=torch.float32)) == 0
    got = mita.mita_paged_attn(x[299:, :Hkv], kc, vc, table, n)
    small = R.Cache((300,), Hkv, page, d, torch.bfloat16, fill=False, spare=0)
    small.k, small.v = kc[[pages - 1, pages - 2]].cpu(), vc[[pages - 1, pages - 2]].cpu()
    small.table = lens(0, 1)[None]
    want, bound, _, _ = R.paged_attn(x[299:, :Hkv].cpu(), small, (300,))
    R.assert_close(got, want, bound, "out")
    assert mita.get_last_device_error() == 0


# --------------------------------------------------------------------------------------------
# together
# --------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_prompt_then_decode(dt):
    """A prompt through norm + rotation and the MiTA forward, its keys into the cache, then tokens
    one by one through append and attention: each against the fp64 restatement of the cache's
    own contents; the cache against the keys that the whole sequence would have had."""
    mita = M()
    B, H, N, d, page, steps = 2, 4, 96, 64, 16, 40
    g = torch.Generator().manual_seed(8)
    total = N + steps
    x = torch.randn(B, total, 3 * H, d, generator=g).to(DT[dt]).cuda()
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g).cuda() for _ in range(2))
    freq = R.inv_freq(d).cuda()
    q, k, v = (x[:, :N, i * H:(i + 1) * H].transpose(1, 2) for i in range(3))
    qn, kn = mita.mita_qk_norm_rope(q, k, freq, wq, wk)
    out = mita.mita_forward(qn, kn, v.contiguous(), 1, N, 8, 12)
    assert bool(torch.isfinite(out.float()).all())
    cache = R.Cache((total,) * B, H, page, d, DT[dt], fill=False)
    kc, vc, table = cache.k.cuda(), cache.v.cuda(), cache.table.cuda()
    n = lens(*(N,) * B).cuda()
    # the prompt's keys are rotated already: appended as they are
    mita.mita_cache_append(kn.transpose(1, 2).reshape(B * N, H, d), v.transpose(1, 2).reshape(B * N, H, d),
                           kc, vc, table, n, seq_start=lens(*range(0, B * N + 1, N)).cuda())
    whole = mita.mita_qk_norm_rope(x[:, :, :H].transpose(1, 2), x[:, :, H:2 * H].transpose(1, 2),
                                   freq, wq, wk)
    for t in range(steps):
        n += 1
        tok = x[:, N + t]
        qr = mita.mita_cache_append(tok[:, H:2 * H], tok[:, 2 * H:], kc, vc, table, n,
                                    q=tok[:, :H], inv_freq=freq, q_weight=wq, k_weight=wk)
        assert torch.equal(qr, whole[0][:, :, N + t])      # the same arithmetic, bit for bit
        out = mita.mita_paged_attn(qr, kc, vc, table, n)
        if t % 13 == 0 or t == steps - 1:
            cache.k, cache.v = kc.cpu(), vc.cpu()
            want, bound, _, _ = R.paged_attn(qr.cpu(), cache, n.tolist())
            R.assert_close(out, want, bound, f"token {t}")
    for b in range(B):
        keys, values, _ = cache.rows(b, 0, total)
        assert torch.equal(keys, whole[1][b].cpu().double())
        assert torch.equal(values, x[b, :, 2 * H:].transpose(0, 1).cpu().double())
    assert mita.get_last_device_error() == 0


def test_decode_step_in_graphs():
    """One step of append and attention captured twice (two batches, one of them with an idle
    slot), replayed on two streams at once with lengths that grow on the device."""
    mita = M()
    Hq, Hkv, d, page, steps = 8, 2, 128, 16, 6
    freq = R.inv_freq(d).cuda()
    runs = []
    g = torch.Generator().manual_seed(0)
    for seed, lengths in ((1, (500, 3, 77)), (2, (2000, 0))):
        S = len(lengths)
        cache = R.Cache([n + steps if n else 0 for n in lengths], Hkv, page, d, torch.bfloat16, seed=seed)
        live = torch.tensor([int(n > 0) for n in lengths], dtype=torch.int32).cuda()
        tokens = torch.randn(steps, S, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda()
        state = dict(S=S, cache=cache, kc=cache.k.cuda(), vc=cache.v.cuda(),
                     table=cache.table.cuda(), n=lens(*lengths).cuda(), live=live, tokens=tokens,
                     x=torch.zeros_like(tokens[0]))

        def step(s=state):
            x = s["x"]
            s["n"] += s["live"]
            qr = mita.mita_cache_append(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], s["kc"], s["vc"],
                                        s["table"], s["n"], q=x[:, :Hq], inv_freq=freq)
            return qr, mita.mita_paged_attn(qr, s["kc"], s["vc"], s["table"], s["n"])
        before = s_n = state["n"].clone()
        keep = state["kc"].clone(), state["vc"].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            state["out"] = step()
        state["n"].copy_(before)
        state["kc"].copy_(keep[0])
        state["vc"].copy_(keep[1])
        state.update(graph=graph, stream=torch.cuda.Stream(), lengths=list(lengths))
        runs.append(state)
    torch.cuda.synchronize()
    for t in range(steps):
        for s in runs:
            with torch.cuda.stream(s["stream"]):
                s["x"].copy_(s["tokens"][t])
                s["graph"].replay()
        torch.cuda.synchronize()
        for s in runs:
            s["lengths"] = [n + 1 if n else 0 for n in s["lengths"]]
            assert s["n"].tolist() == s["lengths"]
            s["cache"].k, s["cache"].v = s["kc"].cpu(), s["vc"].cpu()
            qr, out = s["out"]
            want, bound, _, _ = R.paged_attn(qr.cpu(), s["cache"], s["lengths"])
            R.assert_close(out, want, bound, f"step {t}")
            q, qb = R.norm_rope(s["tokens"][t, :, :Hq].cpu(), None,
                                torch.tensor(s["lengths"])[:, None].expand(-1, Hq) - 1,
                                freq.cpu(), 1e-6, False)
            on = torch.tensor(s["lengths"]) > 0
            R.assert_close(qr[on.cuda()], q[on], qb[on], "q")
    assert mita.get_last_device_error() == 0


def test_side_stream_and_two_calls_at_once():
    mita = M()
    lengths = (5000, 300, 1)
    cache = R.Cache(lengths, 2, 32, 64, torch.bfloat16)
    q = torch.randn(3, 8, 64, generator=torch.Generator().manual_seed(2)).bfloat16()
    args = (q.cuda(), cache.k.cuda(), cache.v.cuda(), cache.table.cuda(), lens(*lengths).cuda())
    want = mita.mita_paged_attn(*args)
    other = mita.mita_paged_attn(-args[0], *args[1:])
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    neg = -args[0]
    torch.cuda.synchronize()
    for _ in range(20):
        got[0].append(mita.mita_paged_attn(*args, stream=sides[0]))
        got[1].append(mita.mita_paged_attn(neg, *args[1:], stream=sides[1]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got[0]) and all(torch.equal(o, other) for o in got[1])
