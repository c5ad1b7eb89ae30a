"""mita_paged_attn_q4 where most of the weight is on keys whose values are small or zero: what the other keys
add is held to a bound relative to itself, whatever the size of weights and scales."""
import pytest
import torch

import decode_util as R
import q4_util as Q

pytestmark = pytest.mark.gpu

U = R.U
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GAPS, SIZES = (6.0, 9.0, 12.0, 15.0, 40.0), (1.0, 2.0 ** -4, 2.0 ** -7, 2.0 ** -10, 2.0 ** -14)


def M():
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    return mita


def reference(q, cache, lengths, scale):
    """(out, bound) fp64: the bound of an element is relative to its terms, sum of p |v|; and in bf16 besides to
    the largest term of its row and to the scales of its block, far below a rounding of either."""
    S, Hq, d = q.shape
    f32 = q.dtype == torch.float32
    out, bound = (torch.zeros(S, Hq, d, dtype=torch.float64) for _ in range(2))
    for s, n in enumerate(lengths):
        k, ks, v, vs, _ = cache.rows(s, 0, n)
        if k is None:
            continue
        qs = q[s].double().view(cache.Hkv, -1, d)
        z = torch.einsum("hgd,hjd->hgj", qs, k) * scale
        p = torch.softmax(z, -1)
        out[s] = torch.einsum("hgj,hjd->hgd", p, v).reshape(Hq, d)
        # scores as q4_util.paged_attn derives it
        terms = torch.einsum("hgd,hjd->hgj", qs.abs(), k.abs() + (0 if f32 else 8) * ks)
        err = (d * 4 * U * (2 if f32 else 1) + (2.0 ** -22 if f32 else 0)) * scale * terms + 8 * U * z.abs()
        # A weight is off by its score's error, and its sum's by as much; its exponential 2^-20; what is left of
        # it as a sum of three bf16 values, half a step each, 2^-8; in bf16 its rounding to fp16 and its
        # product's with a scale, 2^-11 each.  The sums are cut or rounded at 2^-23 a key at most.
        rel = 2 * err.amax(-1) + 2.0 ** -20 + (2.0 ** -24 if f32 else 2.0 ** -10) + 2 * n * U
        size = torch.einsum("hgj,hjd->hgd", p, v.abs()).reshape(Hq, d)
        bound[s] = rel.view(Hq, 1) * size + R.half_step(q.dtype) * out[s].abs()
        if not f32:
            # A weight stands with the power of two w of its row's largest scale s (2 w <= s < 4 w; below 2^-14,
            # where fp16's powers end, w = 2^-15), and the largest such is 2^10 or more when they are
            # rounded.  Below fp16's normal numbers a weight is off by 2^-25, which the scale (s / w < 4) makes
            # 2^-23, and the product by 2^-25: five times that, times 8 for the code, of s p's 2^11.
            top = vs.amax(-1)[:, None]
            tiny = n * 8 * 5 * 2.0 ** -36 * (p * top.clamp(min=2.0 ** -14)).amax(-1)
            # and a scale s / w, where its block is a millionth of its row, by 2^-25 of 2
            tiny = tiny + 8 * 2.0 ** -26 * (p * top).sum(-1)
            bound[s] += tiny.view(Hq, 1)
            # Of two values that share a byte the upper one's sum is a sixteenth of what is left of
            # the byte's without the lower one's: both are cut twice at 2^-23, and added up, of up to 8 scales.
            bound[s] += ((2.0 ** -22 + 2 * n * U) * torch.einsum("hgj,hjd->hgd", p, vs)).reshape(Hq, d)
    return out, bound


def run(q, cache, lengths, scale):
    mita = M()
    out = mita.mita_paged_attn_q4(q.cuda(), cache.k8.cuda(), cache.v8.cuda(), cache.table.cuda(),
                                  torch.tensor(lengths, dtype=torch.int32).cuda(), scale=scale)
    assert mita.get_last_device_error() == 0
    return out


def sinks(lengths, Hkv, G, d, seed=0, zeros=slice(None)):
    """q and a cache in which one key of every sequence stands `gap` above the others and has zeros in its value
    row; gaps and sizes of the other values go through all pairs."""
    g = torch.Generator().manual_seed(seed)
    q0 = torch.randn(len(lengths), Hkv, 1, d, generator=g)
    q = q0 * (1 + 0.05 * torch.randn(len(lengths), Hkv, G, 1, generator=g))
    k, v = [], []
    for s, n in enumerate(lengths):
        gap, size = GAPS[s % 5], SIZES[s // 5 % 5]
        ks, vs = (torch.randn(Hkv, n, d, generator=g) for _ in range(2))
        vs = vs * size
        if n:
            at = s * 37 % n
            ks[:, at] = q0[s, :, 0] * gap * d ** 0.5 / (q0[s, :, 0] ** 2).sum(-1, keepdim=True)
            vs[:, at, zeros] = 0
        k.append(ks)
        v.append(vs)
    return q.reshape(len(lengths), Hkv * G, d), k, v


_made = {}


def case(lengths, Hkv, G, d, make):
    key = (lengths, Hkv, G, d, make)
    if key not in _made:
        q, k, v = make(lengths, Hkv, G, d)
        _made[key] = q, Q.Cache4(lengths, Hkv, 16, d, k=k, v=v)
    return _made[key]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,Hkv,G,d", [
    (tuple(50 + 9 * i for i in range(25)), 1, 3, 32), (tuple(50 + 9 * i for i in range(25)), 1, 3, 64),
    (tuple(50 + 9 * i for i in range(25)), 1, 3, 128),
    # 16 query rows, several warps and CTAs to a sequence, four shares to a CTA
    (tuple(50 + 9 * i for i in range(25)), 1, 12, 128), ((2, 1, 0) * 8 + (2500,), 1, 12, 64),
    (tuple(2 + i % 7 for i in range(475)), 1, 4, 32)])
def test_a_key_without_values_above_all_others(dt, lengths, Hkv, G, d):
    q, cache = case(lengths, Hkv, G, d, sinks)
    q = q.to(DT[dt])
    want, bound = reference(q, cache, lengths, d ** -0.5)
    R.assert_close(run(q, cache, lengths, d ** -0.5), want, bound, "out")


def half_sinks(lengths, Hkv, G, d):
    return sinks(lengths, Hkv, G, d, 1, slice(1, None, 2))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_zeros_beside_values_of_a_key_above_all_others(dt, d):
    lengths = tuple(40 + 7 * i for i in range(25))
    q, cache = case(lengths, 1, 4, d, half_sinks)
    q = q.to(DT[dt])
    want, bound = reference(q, cache, lengths, d ** -0.5)
    R.assert_close(run(q, cache, lengths, d ** -0.5), want, bound, "out")


def all_sizes(lengths, Hkv, G, d, seed=3):
    """Scores of a wide range, and value blocks from 2^-17 to 2^14 side by side."""
    g = torch.Generator().manual_seed(seed)
    k = [4 * torch.randn(Hkv, n, d, generator=g) for n in lengths]
    v = []
    for n in lengths:
        size = torch.exp2(torch.randint(-14, 15, (Hkv, n, d // 32, 1), generator=g).float())
        v.append((torch.randn(Hkv, n, d // 32, 32, generator=g) * size).flatten(2))
    return torch.randn(len(lengths), Hkv * G, d, generator=g), k, v


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,Hkv,G,d", [((1, 63, 64, 65, 300), 2, 2, 32), ((1, 63, 64, 65, 300), 1, 9, 64),
                                             ((1, 63, 64, 65, 900), 1, 4, 128)])
def test_values_of_every_size_side_by_side(dt, lengths, Hkv, G, d):
    q, cache = case(lengths, Hkv, G, d, all_sizes)
    q = q.to(DT[dt])
    want, bound = reference(q, cache, lengths, d ** -0.5)
    R.assert_close(run(q, cache, lengths, d ** -0.5), want, bound, "out")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", [-1e30, -1e9, -1.5e7, -7e6, -1e6, -1e3, 1e6, 3e6, 7e6, 1.5e7, 3e7, 1e9, 1e12, 1e30])
def test_equal_scores_of_any_size(dt, size):
    """Scores that are the same number for all keys, so that every weight is exactly 1 / n, over some keys and over
    many; rows of zeros among the values, or not."""
    mita = M()
    d = 64
    lengths = (3, 200, 2500)
    for zeros in (False, True):
        g = torch.Generator().manual_seed(5)
        k = [torch.full((1, n, d), 7.0) for n in lengths]
        v = [torch.randn(1, n, d, generator=g) for n in lengths]
        if zeros:
            for x in v:
                x[:, ::3] = 0
        cache = Q.Cache4(lengths, 1, 16, d, k=k, v=v)
        q = torch.full((3, 5, d), 1 / 64.0).to(DT[dt])              # q k is 7, exactly
        out, lse = mita.mita_paged_attn_q4(q.cuda(), cache.k8.cuda(), cache.v8.cuda(), cache.table.cuda(),
                                           torch.tensor(lengths, dtype=torch.int32).cuda(), scale=size,
                                           return_lse=True)
        for s, n in enumerate(lengths):
            value, scale = cache.kv[s][1]
            want, size_of = value.mean(1), value.abs().mean(1)
            # the weights are alike: what is left are a product's rounding (2^-11 twice in bf16), the sums, and what
            # `reference` says of bytes and of weights far below the largest (rows are alike here, within 2^6)
            rel = (2.0 ** -10 if dt == "bf16" else 2.0 ** -24) + 2 * n * U
            bound = rel * size_of + R.half_step(DT[dt]) * want.abs() + 2.0 ** -20 * scale.mean(1)
            R.assert_close(out[s], want.expand(5, d), bound.expand(5, d), f"{n} keys")
            z = 7 * float(torch.tensor(size)) + float(torch.log(torch.tensor(float(n), dtype=torch.float64)))
            assert float((lse[s].cpu().double() - z).abs().max()) <= 4 * 2 * U * abs(z) + 2 * n * U + 2.0 ** -20


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -15, 2.0 ** -6, 1.0, 2.0 ** 13])
def test_the_logarithm_of_the_sum_does_not_depend_on_values(dt, size):
    """Sums near one, of a few keys each: what is left of the logarithm is its own rounding."""
    mita = M()
    S, d = 600, 32
    lengths = tuple(1 + i % 3 for i in range(S))
    g = torch.Generator().manual_seed(9)
    k = [torch.randn(1, n, d, generator=g) for n in lengths]
    v = [torch.randn(1, n, d, generator=g) * size for n in lengths]
    cache = Q.Cache4(lengths, 1, 16, d, k=k, v=v)
    q = torch.zeros(S, 8, d, dtype=DT[dt])                # scores are the slopes'
    slopes = torch.rand(8, generator=g) * 0.1
    _, lse = mita.mita_paged_attn_q4(q.cuda(), cache.k8.cuda(), cache.v8.cuda(), cache.table.cuda(),
                                     torch.tensor(lengths, dtype=torch.int32).cuda(), return_lse=True,
                                     alibi_slopes=slopes.cuda())
    _, _, want, bound = Q.paged_attn(q, cache, lengths, slopes=slopes)
    R.assert_close(lse, want, bound, "lse")
