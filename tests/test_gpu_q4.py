"""The 4-bit cache on the GPU: mita_cache_append_q4 and mita_paged_attn_q4 against plain
restatements (q4_util.py)."""
import math

import pytest
import torch

import decode_util as R
import q4_util as Q

pytestmark = pytest.mark.gpu

U = R.U
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def M():
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    return mita


def up(t):
    return None if t is None else t.cuda()


def lens(*n):
    return torch.tensor(n, dtype=torch.int32)


def gen(seed):
    return torch.Generator().manual_seed(seed)


# --------------------------------------------------------------------------------------------
# append
# --------------------------------------------------------------------------------------------
def rows_of(kind, T, Hkv, d, dtype):
    g = gen(7)
    x = torch.randn(T, Hkv, d, generator=g)
    if kind == "spread":          # every size, the smallest scales and the largest ones among them
        x = x * torch.exp2(torch.randint(-26, 24, (T, Hkv, 1), generator=g).float())
    elif kind == "ties":          # halves of scales, zeros, blocks of zeros
        x = torch.randint(-14, 15, (T, Hkv, d), generator=g) / 2.0
        x[..., 0] = 7.0 * torch.randint(1, 15, (T, Hkv), generator=g)
        x[::3] = 0
    elif kind == "odd":           # infinities and NaN: their block becomes NaN, its neighbours do not
        x[0, 0, 3], x[1, 0, d - 1], x[2, 0, 0] = math.inf, math.nan, -math.inf
    return x.to(dtype)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d,page,Hkv,T,kind", [
    (64, 16, 2, 1, "plain"), (128, 64, 3, 70, "plain"), (32, 16, 1, 131, "plain"),
    (128, 16, 2, 33, "spread"), (64, 32, 1, 40, "spread"), (32, 256, 2, 50, "spread"),
    (64, 16, 1, 64, "ties"), (128, 32, 1, 64, "ties"), (128, 16, 1, 20, "odd"), (32, 16, 3, 20, "odd"),
    (128, 16, 5, 700, "plain"), (64, 16, 4, 2500, "spread")])
def test_append(dt, d, page, Hkv, T, kind):
    """Codes and scales bit for bit, in their places; every other byte, and rows passed over, as they were."""
    mita = M()
    dtype = DT[dt]
    pages = -(-T // page) + 3
    k, v = rows_of(kind, T, Hkv, d, dtype), rows_of("plain", T, Hkv, d, dtype) * 0.3
    g = gen(3)
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[::5] = -1
    kc, vc = (torch.randint(0, 256, mita.cache_q4_shape(pages, Hkv, page, d), generator=g).to(torch.uint8)
              for _ in range(2))
    ko, vo = (torch.full((T, Hkv, d), -9.0, dtype=dtype) for _ in range(2))
    dk, dv, dko, dvo = (t.cuda() for t in (kc, vc, ko, vo))
    mita.mita_cache_append_q4(k.cuda(), v.cuda(), dk, dv, slots.cuda(), k_out=dko, v_out=dvo)
    assert mita.get_last_device_error() == 0
    for x, cache, got, out, had in ((k, kc, dk, dko, ko), (v, vc, dv, dvo, vo)):
        code, byte, value = Q.quantise(x)
        nan = (byte == 255).repeat_interleave(32, -1)
        want = cache.clone()
        for t in range(T):
            s = int(slots[t])
            if s >= 0:
                for h in range(Hkv):
                    want[s // page, h] = Q.put_row(want[s // page, h], code[t, h], byte[t, h], s % page,
                                                   page, d)
        assert torch.equal(got.cpu(), want)
        live = (slots >= 0)[:, None, None]
        assert torch.equal(out.cpu()[live.expand(nan.shape) & ~nan].float(),
                           value[live.expand(nan.shape) & ~nan])
        assert bool(out.cpu()[live.expand(nan.shape) & nan].isnan().all())
        assert torch.equal(out.cpu()[slots < 0], had[slots < 0])


def test_append_takes_views_and_needs_no_outputs():
    mita = M()
    T, Hkv, d, page = 37, 2, 64, 16
    x = torch.randn(T, 3 * Hkv, d, generator=gen(1)).bfloat16().cuda()
    q, k, v = x.split(Hkv, 1)
    slots = torch.arange(T, dtype=torch.int64, device="cuda") + 5
    shape = mita.cache_q4_shape(4, Hkv, page, d)
    a = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
    b = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
    mita.mita_cache_append_q4(k, v, *a, slots)
    wide = torch.zeros(T, 2 * Hkv, d, dtype=x.dtype, device="cuda")
    mita.mita_cache_append_q4(k.contiguous(), v.contiguous(), *b, slots, k_out=wide[:, Hkv:])
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    assert bool((wide[:, :Hkv] == 0).all()) and bool((wide[:, Hkv:] != 0).any())
    # heads before tokens
    c = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
    turned = k.transpose(0, 1).contiguous().transpose(0, 1)
    mita.mita_cache_append_q4(turned, v, *c, slots)
    assert torch.equal(a[0], c[0])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_append_rounds_in_place(dt):
    """k_out and v_out may be k and v: a row's block is read before its values are written."""
    mita = M()
    T, Hkv, d, page = 300, 3, 128, 16
    x = torch.randn(T, 2 * Hkv, d, generator=gen(2)).to(DT[dt]).cuda()
    slots = torch.arange(T, device="cuda")
    shape = mita.cache_q4_shape(T // page + 1, Hkv, page, d)
    a, b = ([torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)] for _ in range(2))
    out = [torch.empty(T, Hkv, d, dtype=x.dtype, device="cuda") for _ in range(2)]
    mita.mita_cache_append_q4(*x.split(Hkv, 1), *a, slots, *out)
    mita.mita_cache_append_q4(*x.split(Hkv, 1), *b, slots, *x.split(Hkv, 1))
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    assert torch.equal(x, torch.cat(out, 1))


def test_append_nothing_and_bad_slots():
    mita = M()
    Hkv, d, page, pages = 1, 32, 16, 2
    shape = mita.cache_q4_shape(pages, Hkv, page, d)
    kc, vc = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    empty = torch.zeros(0, Hkv, d, device="cuda")
    mita.mita_cache_append_q4(empty, empty, kc, vc, torch.zeros(0, dtype=torch.int64, device="cuda"))
    x = torch.ones(6, Hkv, d, device="cuda")
    out = torch.full_like(x, 5.0)
    slots = torch.tensor([-1, 32, -2, 2 ** 40, -2 ** 62, 31], device="cuda")
    mita.mita_cache_append_q4(x, x, kc, vc, slots, k_out=out)
    assert mita.get_last_device_error() == 1
    assert bool((out[:5] == 5).all()) and bool((out[5] != 5).all())
    code, byte = Q.read_row(kc[1, 0].cpu(), 15, page, d)
    assert bool((code == 15).all()) and Q.scale_of_byte(int(byte[0])) * 7 == pytest.approx(1, rel=0.07)
    assert int((kc[0] != 0).sum()) == 0
    none = torch.zeros(mita.cache_q4_shape(0, Hkv, page, d), dtype=torch.uint8, device="cuda")
    mita.mita_cache_append_q4(x, x, none, none, torch.full((6,), -1, dtype=torch.int64, device="cuda"))
    assert mita.get_last_device_error() == 0


# --------------------------------------------------------------------------------------------
# attention
# --------------------------------------------------------------------------------------------
EDGES = (0, 1, 2, 15, 16, 17, 31, 32, 33, 65, 129, 255, 256, 257, 0, 513)
MANY = tuple(430 if i % 19 == 7 else i * 53 % 60 for i in range(120))
ATTN = [
    # lengths, Hq, Hkv, d, page, dtype, options
    ((1,), 1, 1, 64, 16, "bf16", {}),
    (EDGES, 4, 2, 64, 16, "bf16", {}),
    (EDGES, 8, 1, 128, 64, "bf16", {}),
    (EDGES, 3, 3, 32, 32, "bf16", {}),
    (EDGES, 4, 2, 64, 16, "f32", {}),
    (EDGES, 8, 1, 128, 32, "f32", {}),
    (EDGES, 3, 3, 32, 16, "f32", {}),
    # groups of odd size, of a whole tile of rows, and of more than one
    (EDGES, 7, 1, 64, 32, "bf16", {}),
    (EDGES, 15, 3, 128, 16, "bf16", {}),
    (EDGES, 32, 2, 128, 128, "bf16", {}),
    (EDGES, 24, 2, 32, 16, "bf16", {}),
    ((300, 0, 129), 17, 1, 128, 64, "bf16", {}),
    ((300, 0, 129), 40, 1, 64, 64, "bf16", {}),
    ((300, 0, 129), 40, 2, 32, 16, "f32", {}),
    ((300, 0, 129), 17, 1, 128, 16, "f32", {}),
    # options
    (EDGES, 4, 2, 64, 16, "bf16", {"softcap": 2.0}),
    (EDGES, 4, 2, 64, 16, "f32", {"softcap": 2.0}),
    (EDGES, 4, 2, 128, 16, "bf16", {"slopes": True}),
    (EDGES, 4, 2, 64, 16, "f32", {"slopes": True, "softcap": 5.0}),
    (EDGES, 4, 2, 64, 16, "bf16", {"window": 1}),
    (EDGES, 4, 2, 64, 16, "bf16", {"window": 100}),
    (EDGES, 4, 2, 128, 32, "f32", {"window": 130, "slopes": True}),
    (EDGES, 4, 2, 32, 16, "bf16", {"window": 37}),
    (EDGES, 4, 2, 64, 16, "bf16", {"window": 5000, "scale": 0.5}),
    (EDGES, 4, 2, 64, 16, "bf16", {"scale": -1.0}),
    (EDGES, 4, 2, 64, 16, "f32", {"scale": 0.0}),
    # cut over every SM, and joined
    ((9000,), 4, 1, 64, 64, "bf16", {}),
    ((5333, 5, 4001, 0, 1), 4, 2, 128, 16, "bf16", {"slopes": True}),
    ((7000, 3), 3, 1, 32, 128, "f32", {}),
    ((4111,), 6, 1, 128, 16, "f32", {"window": 3000}),
    # many short sequences: several segments to a CTA
    (tuple(1 + i * 37 % 100 for i in range(130)), 2, 2, 64, 16, "bf16", {}),
    (tuple(i * 29 % 40 for i in range(400)), 4, 1, 32, 16, "f32", {}),
    # so many that a CTA has four shares
    (MANY, 12, 4, 128, 16, "bf16", {"window": 333, "softcap": 5.0, "slopes": True}),
    (MANY, 4, 4, 128, 16, "f32", {"window": 200}),
    (MANY, 8, 4, 128, 16, "bf16", {}),
    (MANY, 36, 4, 64, 32, "f32", {"slopes": True}),
    (tuple(i * 29 % 90 for i in range(480)), 5, 1, 32, 16, "bf16", {"softcap": 2.0}),
]
_caches = {}


def cache_of(lengths, Hkv, page, d, **how):
    """A cache, made once for cases that agree on it (bytes are written in plain Python)."""
    key = (lengths, Hkv, page, d, tuple(sorted(how.items())))
    if key not in _caches:
        _caches[key] = Q.Cache4(lengths, Hkv, page, d, slack=len(lengths) % 3, **how)
    return _caches[key]


def make_slopes(on, Hq):
    return 2.0 ** (-8.0 * torch.arange(1, Hq + 1, dtype=torch.float32) / Hq) if on else None


@pytest.mark.parametrize("case", ATTN, ids=lambda c: f"{len(c[0])}x{max(c[0])}-" + "-".join(
    map(str, c[1:6])) + "".join(f"-{k}{v}" for k, v in c[6].items()))
def test_attention(case):
    mita = M()
    lengths, Hq, Hkv, d, page, dt, opt = case
    opt = dict(opt)
    slopes = make_slopes(opt.pop("slopes", False), Hq)
    cache = cache_of(lengths, Hkv, page, d)
    q = torch.randn(len(lengths), Hq, d, generator=gen(2)).to(DT[dt])
    args = (q.cuda(), cache.k8.cuda(), cache.v8.cuda(), cache.table.cuda(), lens(*lengths).cuda())
    out, lse = mita.mita_paged_attn_q4(*args, alibi_slopes=up(slopes), return_lse=True, **opt)
    assert mita.get_last_device_error() == 0
    want, bound, lwant, lbound = Q.paged_attn(q, cache, lengths, slopes=slopes, **opt)
    R.assert_close(out, want, bound, "out")
    empty = torch.tensor([n == 0 for n in lengths])
    assert bool((lse.cpu()[empty] == -math.inf).all()) and bool((out.cpu()[empty] == 0).all())
    R.assert_close(lse[~empty.cuda()], lwant[~empty], lbound[~empty], "lse")
    again = mita.mita_paged_attn_q4(*args, alibi_slopes=up(slopes), **opt)
    assert torch.equal(again, out)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("spread", [2.0 ** -16, 2.0 ** -12, 3.0, 30.0, 3000.0, 2.0e4, 1e5])
def test_scales_of_every_size(dt, d, spread):
    """Values (and keys, the scores kept in range by `scale`) whose scales are subnormal, above 2, and near the
    format's end."""
    mita = M()
    lengths = (300, 33)
    cache = cache_of(lengths, 1, 16, d, spread=spread)
    q = torch.randn(2, 3, d, generator=gen(2)).to(DT[dt])
    how = dict(scale=1.0 / (spread * d ** 0.5))
    out, lse = mita.mita_paged_attn_q4(q.cuda(), cache.k8.cuda(), cache.v8.cuda(), cache.table.cuda(),
                                       lens(*lengths).cuda(), return_lse=True, **how)
    want, bound, lwant, lbound = Q.paged_attn(q, cache, lengths, **how)
    R.assert_close(out, want, bound, "out")
    R.assert_close(lse, lwant, lbound, "lse")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_one_large_row_among_small_ones(dt):
    """A value row two hundred times its neighbours, under a small weight and under a large one."""
    mita = M()
    n, d = 200, 64
    k, v = (torch.randn(1, 1, n, d, generator=gen(i)) for i in (1, 2))
    v = v * 0.1
    v[0, 0, 77] *= 200
    for sign in (-1.0, 1.0):
        q = (sign * k[0, :, 77] * 0.5)[None].to(DT[dt])
        cache = Q.Cache4((n,), 1, 16, d, k=k, v=v)
        out = mita.mita_paged_attn_q4(q.cuda(), cache.k8.cuda(), cache.v8.cuda(), cache.table.cuda(),
                                      lens(n).cuda())
        want, bound, _, _ = Q.paged_attn(q, cache, (n,))
        R.assert_close(out, want, bound, f"sign {sign}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e6, 1e20])
def test_queries_of_every_size(dt, size):
    """Rows of one call that differ in size, scores kept in range by `scale`."""
    mita = M()
    n, d = 100, 64
    cache = cache_of((n,), 1, 16, d)
    q = (torch.randn(1, 4, d, generator=gen(2)) * size)
    q[0, 1] = 0
    q[0, 2] *= 2.0 ** -3
    q = q.to(DT[dt])
    how = dict(scale=1.0 / (size * 8))
    out, lse = mita.mita_paged_attn_q4(q.cuda(), cache.k8.cuda(), cache.v8.cuda(), cache.table.cuda(),
                                       lens(n).cuda(), return_lse=True, **how)
    want, bound, lwant, lbound = Q.paged_attn(q, cache, (n,), **how)
    R.assert_close(out, want, bound, "out")
    R.assert_close(lse, lwant, lbound, "lse")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nan_blocks(dt):
    """A NaN among a seen key's scales makes its sequence NaN, among a value's its block; unseen ones
    nothing."""
    mita = M()
    n, d, page = 50, 128, 16
    lengths = (n, n, n)
    cache = Q.Cache4(lengths, 1, page, d)
    for s, c, pos in ((0, cache.k8, 17), (1, cache.v8, 33), (2, cache.v8, 3)):
        at, row = cache.place(s, pos)
        c[at, 0, page * d // 2 + row * 4 + 2] = 255
    q = torch.randn(3, 2, d, generator=gen(5)).to(DT[dt])
    args = (q.cuda(), cache.k8.cuda(), cache.v8.cuda(), cache.table.cuda(), lens(*lengths).cuda())
    out = mita.mita_paged_attn_q4(*args, window=40).cpu()       # position 3 is not seen
    want, bound, _, _ = Q.paged_attn(q, cache, lengths, window=40)
    assert bool(out[0].isnan().all())
    assert bool(out[1, :, 64:96].isnan().all()) and not bool(out[1, :, :64].isnan().any())
    R.assert_close(out[2], want[2], bound[2], "unseen")
    keep = [i for i in range(d) if not 64 <= i < 96]
    R.assert_close(out[1][:, keep], want[1][:, keep], bound[1][:, keep], "other blocks")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_masked_rows_hold_anything(dt):
    """Every byte behind a length, before a window and on free pages 0xff: NaN scales reach nothing."""
    mita = M()
    for window in (0, 19):
        lengths = (1, 5, 16, 30, 47, 100)
        cache = Q.Cache4(lengths, 2, 16, 64, junk=255)
        if window:
            for s, n in enumerate(lengths):
                for p in range(max(0, n - window)):
                    at, row = cache.place(s, p)
                    for c in (cache.k8, cache.v8):
                        c[at, :, row * 32:row * 32 + 32] = 255
                        c[at, :, 16 * 32 + row * 2:16 * 32 + row * 2 + 2] = 255
        q = torch.randn(6, 4, 64, generator=gen(5)).to(DT[dt])
        out = mita.mita_paged_attn_q4(q.cuda(), cache.k8.cuda(), cache.v8.cuda(), cache.table.cuda(),
                                      lens(*lengths).cuda(), window=window)
        want, bound, _, _ = Q.paged_attn(q, cache, lengths, window=window)
        R.assert_close(out, want, bound, "out")


def test_bad_pages_are_left_out_and_flagged():
    mita = M()
    for dt in ("bf16", "f32"):
        lengths = (300, 40, 16, 200)
        cache = Q.Cache4(lengths, 2, 16, 64)
        cache.table[0, 3], cache.table[0, 7], cache.table[3, 12] = -1, cache.num, 2 ** 30
        cache.table[2, 0] = -5
        q = torch.randn(4, 4, 64, generator=gen(5)).to(DT[dt])
        out, lse = mita.mita_paged_attn_q4(q.cuda(), cache.k8.cuda(), cache.v8.cuda(),
                                           cache.table.cuda(), lens(*lengths).cuda(), return_lse=True)
        assert mita.get_last_device_error() == 1
        want, bound, lwant, lbound = Q.paged_attn(q, cache, lengths, skip_bad=True)
        R.assert_close(out, want, bound, "out")
        R.assert_close(lse[[0, 1, 3]], lwant[[0, 1, 3]], lbound[[0, 1, 3]], "lse")
        assert bool((out[2] == 0).all()) and bool((lse[2] == -math.inf).all())


def test_lengths_out_of_range_are_cut_and_flagged():
    mita = M()
    cache = Q.Cache4((64, 64, 64), 1, 16, 64)
    q = torch.randn(3, 2, 64, generator=gen(5))
    out = mita.mita_paged_attn_q4(q.cuda(), cache.k8.cuda(), cache.v8.cuda(), cache.table.cuda(),
                                  lens(64, 2 ** 31 - 1, -3).cuda())
    assert mita.get_last_device_error() == 1
    want, bound, _, _ = Q.paged_attn(q, cache, (64, 64, 0))
    R.assert_close(out, want, bound, "out")


def test_strided_queries_and_given_output():
    mita = M()
    lengths = (70, 20)
    cache = cache_of(lengths, 2, 16, 64)
    x = torch.randn(2, 8, 64, generator=gen(5)).bfloat16()
    args = (cache.k8.cuda(), cache.v8.cuda(), cache.table.cuda(), lens(*lengths).cuda())
    want = mita.mita_paged_attn_q4(x[:, ::2].contiguous().cuda(), *args)
    out = torch.empty_like(want)
    got = mita.mita_paged_attn_q4(x.cuda()[:, ::2], *args, out=out)
    assert got is out and torch.equal(out, want)


def test_a_long_context_of_equal_values():
    """Values of one size under equal weights, over 300 thousand keys of a page that repeats."""
    mita = M()
    d, page = 128, 16
    for dt in ("bf16", "f32"):
        cache = Q.Cache4((page,), 1, page, d, k=[torch.zeros(1, page, d)], v=[torch.full((1, page, d), 0.7)])
        reps = 300_000 // page
        table = torch.full((1, reps), int(cache.table[0, 0]), dtype=torch.int32, device="cuda")
        q = torch.randn(1, 2, d, generator=gen(1)).to(DT[dt])
        out = mita.mita_paged_attn_q4(q.cuda(), cache.k8.cuda(), cache.v8.cuda(), table,
                                      lens(reps * page).cuda())
        want = cache.kv[0][1][0][0, 0]
        # Sums are rounded to nearest but for a product's own, which a tile cuts (two or four times in a
        # chain, at 2^-23 each).  fp32: some 250 keys a warp (its SM's share, dealt to 8 warps or more)
        # are at most 16 tiles added up, the warps' sums 16 more, the 152 parts' a few for each: under
        # 64 roundings, and the weight's two, its exponential cancelling.
        tol = 2.0 ** -8 if dt == "bf16" else 4 * 2.0 ** -23 + 64 * U
        assert float(((out.cpu().double() - want) / want).abs().max()) <= tol


def test_every_key_counts_once():
    """A value row that stands out, at each key in turn: the output moves by its weight and no more."""
    mita = M()
    n, d = 97, 32
    v = torch.zeros(n, 1, n, d)
    for i in range(n):
        v[i, 0, i] = 7.0                     # scale 1, exactly
    cache = Q.Cache4((n,) * n, 1, 16, d, k=torch.zeros(n, 1, n, d), v=v)
    q = torch.randn(n, 1, d, generator=gen(1))
    out = mita.mita_paged_attn_q4(q.cuda(), cache.k8.cuda(), cache.v8.cuda(), cache.table.cuda(),
                                  torch.full((n,), n, dtype=torch.int32, device="cuda"))
    assert float((out.cpu().double() - 7.0 / n).abs().max()) <= 7.0 / n * 2.0 ** -18


# --------------------------------------------------------------------------------------------
# streams, graphs
# --------------------------------------------------------------------------------------------
def test_on_another_stream():
    mita = M()
    cache = cache_of((300, 40), 2, 16, 64)
    q = torch.randn(2, 4, 64, generator=gen(5)).bfloat16().cuda()
    args = (cache.k8.cuda(), cache.v8.cuda(), cache.table.cuda(), lens(300, 40).cuda())
    want = mita.mita_paged_attn_q4(q, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mita.mita_paged_attn_q4(q, *args, stream=side)
    x = torch.randn(3, 2, 64, generator=gen(6)).bfloat16().cuda()
    slots = torch.tensor([0, 1, 2], device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    a = [torch.zeros_like(args[0]) for _ in range(2)]
    b = [torch.zeros_like(args[0]) for _ in range(2)]
    torch.cuda.synchronize()
    mita.mita_cache_append_q4(x, x, *a, slots, stream=side)
    mita.mita_cache_append_q4(x, x, *b, slots)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_step_replays_with_new_tokens():
    """Append and attention in one graph, replayed as the sequences grow; two graphs alive at once."""
    mita = M()
    S, Hq, Hkv, d, page, N = 2, 4, 2, 64, 16, 40
    g = gen(8)
    x = torch.randn(N, S, Hq + 2 * Hkv, d, generator=g).bfloat16()
    k = [x[:, s, Hq:Hq + Hkv].transpose(0, 1) for s in range(S)]
    v = [x[:, s, Hq + Hkv:].transpose(0, 1) for s in range(S)]
    cache = Q.Cache4((N,) * S, Hkv, page, d, k=k, v=v)
    kc, vc = (torch.full_like(cache.k8, 255).cuda() for _ in range(2))
    table, n = cache.table.cuda(), torch.zeros(S, dtype=torch.int32, device="cuda")
    step, slots = torch.zeros(S, Hq + 2 * Hkv, d, dtype=torch.bfloat16, device="cuda"), torch.full(
        (S,), -1, dtype=torch.int64, device="cuda")

    def one():
        mita.mita_cache_append_q4(step[:, Hq:Hq + Hkv], step[:, Hq + Hkv:], kc, vc, slots)
        return mita.mita_paged_attn_q4(step[:, :Hq], kc, vc, table, n)

    one()
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(one())
        graphs.append(gr)
    for t in range(N):
        step.copy_(x[t])
        n.fill_(t + 1)
        slots.copy_(torch.tensor([at * page + row for at, row in (cache.place(s, t) for s in range(S))]))
        graphs[t % 2].replay()
        if t in (0, 1, 15, 16, 17, 38, 39):
            want, bound, _, _ = Q.paged_attn(x[t, :, :Hq], cache, (t + 1,) * S)
            R.assert_close(outs[t % 2], want, bound, f"step {t}")
    assert mita.get_last_device_error() == 0


def test_one_workspace_serves_both_caches():
    """Calls over the two kinds of cache, of different shapes, one after the other on one stream."""
    mita = M()
    a = R.Cache((3000, 7), 2, 16, 64, torch.bfloat16)
    b = cache_of((1500, 40), 1, 16, 128)
    qa = torch.randn(2, 4, 64, generator=gen(1)).bfloat16()
    qb = torch.randn(2, 11, 128, generator=gen(2)).bfloat16()
    wa, ba, _, _ = R.paged_attn(qa, a, (3000, 7))
    wb, bb, _, _ = Q.paged_attn(qb, b, (1500, 40))
    ta = (qa.cuda(), a.k.cuda(), a.v.cuda(), a.table.cuda(), lens(3000, 7).cuda())
    tb = (qb.cuda(), b.k8.cuda(), b.v8.cuda(), b.table.cuda(), lens(1500, 40).cuda())
    for _ in range(5):
        x, y = mita.mita_paged_attn(*ta), mita.mita_paged_attn_q4(*tb)
    R.assert_close(x, wa, ba, "bf16 cache")
    R.assert_close(y, wb, bb, "4-bit cache")


def test_python_refusals():
    mita = M()
    t = torch.zeros(3, 2, 64, device="cuda")
    q = torch.zeros(3, 4, 64, device="cuda")
    c = torch.zeros(mita.cache_q4_shape(5, 2, 16, 64), dtype=torch.uint8, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    table = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    n = torch.ones(3, dtype=torch.int32, device="cuda")
    mita.mita_cache_append_q4(t, t, c, c.clone(), slots)
    mita.mita_paged_attn_q4(q, c, c, table, n)
    n0 = mita.kernel_launches()
    for bad, err in (
            (lambda: mita.mita_cache_append_q4(t, t[:2], c, c, slots), ValueError),
            (lambda: mita.mita_cache_append_q4(t[:, :1], t[:, :1], c, c, slots), ValueError),
            (lambda: mita.mita_cache_append_q4(t, t, c, c, slots.int()), TypeError),
            (lambda: mita.mita_cache_append_q4(t, t, c, c, slots[:2]), ValueError),
            (lambda: mita.mita_cache_append_q4(t, t, c.int(), c, slots), TypeError),
            (lambda: mita.mita_cache_append_q4(t, t, c, c[:4], slots), ValueError),
            (lambda: mita.mita_cache_append_q4(t, t, c[..., :300], c[..., :300], slots), ValueError),
            (lambda: mita.mita_cache_append_q4(t.half(), t.half(), c, c, slots), TypeError),
            (lambda: mita.mita_cache_append_q4(t, t, c, c, slots, k_out=t[:, :1].expand(3, 2, 64)), ValueError),
            (lambda: mita.mita_cache_append_q4(t, t, c, c, slots, v_out=t.bfloat16()), TypeError),
            (lambda: mita.mita_cache_append_q4(t[..., :16], t[..., :16], c, c, slots), ValueError),
            (lambda: mita.mita_cache_append_q4(t, t, c[..., :272].contiguous(), c[..., :272].contiguous(),
                                               slots), mita.MitaError),          # pages of 8
            (lambda: mita.mita_paged_attn_q4(q[:, :3], c, c, table, n), mita.MitaError),
            (lambda: mita.mita_paged_attn_q4(q[:2], c, c, table, n), ValueError),
            (lambda: mita.mita_paged_attn_q4(q, c.cpu(), c, table, n), ValueError),
            (lambda: mita.mita_paged_attn_q4(q, c.view(5, 2, 16, 34), c, table, n), ValueError),
            (lambda: mita.mita_paged_attn_q4(q, c, c, table[:, ::2], n), ValueError),
            (lambda: mita.mita_paged_attn_q4(q, c, c, table, n, softcap=-1.0), mita.MitaError),
            (lambda: mita.mita_paged_attn_q4(q, c, c, table, n, out=q.bfloat16()), TypeError)):
        with pytest.raises(err):
            bad()
    assert mita.kernel_launches() == n0
