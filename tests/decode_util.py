"""Plain fp64 restatements (CPU, loops) of the head norm with rotation, the paged cache and the
single-token attention over it, with the error bounds that the GPU tests hold the kernels to.

Half a step of a type, relative to the value, is finfo(t).eps / 2; u = 2^-24 is fp32's.
"""
import math

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def inv_freq(rot, theta=10000.0):
    return theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def _pairs(d, rot, interleaved):
    """[(first, second, frequency)] of the rotated values."""
    if interleaved:
        return [(2 * i, 2 * i + 1, i) for i in range(rot // 2)]
    return [(i, i + rot // 2, i) for i in range(rot // 2)]


def rotate(x, pos, freq, interleaved, back=False):
    """x [..., d] fp64 turned (or turned back) by positions pos [...]."""
    y = x.clone()
    if freq is None:
        return y
    for a, b, i in _pairs(x.shape[-1], 2 * len(freq), interleaved):
        angle = pos.double() * freq[i].item()
        c, s = torch.cos(angle), torch.sin(angle) * (-1 if back else 1)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def pair_size(x, freq, interleaved):
    """For each value the size of its pair (what a rotation's error is relative to)."""
    y = x.abs()
    if freq is not None:
        for a, b, _ in _pairs(x.shape[-1], 2 * len(freq), interleaved):
            y[..., a] = y[..., b] = torch.hypot(x[..., a], x[..., b])
    return y


def norm(x, weight, eps):
    if weight is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()


def norm_rope(x, weight, pos, freq, eps, interleaved):
    """(y, bound): y fp64 for x of any type; bound: what a kernel's value may be off by."""
    u = norm(x.double(), weight, eps)
    y = rotate(u, pos, freq, interleaved)
    # fp32 roundings, each at most u of the pair's size: the row's sum of squares (at most 16
    # in a chain, halved by the root), the root (2), scale and weight (2), the angle (pi u),
    # sine and cosine (2 each), products and sum (3): below 32 in all; then the result's own.
    # An angle's fp64 frequency is off by 2^-53 of itself, its product by position times that.
    far = float(pos.abs().max()) * 2.0 ** -51 if freq is not None and pos.numel() else 0.0
    bound = half_step(x.dtype) * y.abs() + (32 * U + far) * pair_size(u, freq, interleaved)
    return y, bound


def norm_rope_grad(x, dy, weight, pos, freq, eps, interleaved):
    """Gradients (dx, dx bound, dw, dw bound) of one part [B, H, N, d]."""
    xd, dyd = x.double(), dy.double()
    g = rotate(dyd, pos, freq, interleaved, back=True)
    size = pair_size(dyd, freq, interleaved)
    if weight is None:
        return g, half_step(x.dtype) * g.abs() + 32 * U * size, None, None
    w, d = weight.double(), x.shape[-1]
    r = 1 / torch.sqrt((xd * xd).mean(-1, keepdim=True) + eps)
    dx = r * w * g - xd * r ** 3 * (w * g * xd).mean(-1, keepdim=True)
    # the roundings of norm_rope and as many again for the dot product, of each term's size
    terms = r * w.abs() * size + xd.abs() * r ** 3 * (w.abs() * size * xd.abs()).mean(-1, True)
    dw = (g * xd * r).sum((0, 1, 2))
    rows = x[..., 0].numel()
    # a sum of `rows` terms in fp32, whatever its order, is off by at most rows * u of their sizes
    return (dx, half_step(x.dtype) * dx.abs() + 64 * U * terms, dw,
            (32 + rows) * U * (size * xd.abs() * r).sum((0, 1, 2)))


def assert_close(got, want, bound, what):
    off = (got.double().cpu() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (
        f"{what}: {int(bad.sum())} of {bad.numel()} values are off, the first at "
        f"{bad.nonzero()[0].tolist()}: {got.cpu()[tuple(bad.nonzero()[0])].item()} for "
        f"{want[tuple(bad.nonzero()[0])].item()}, worst {float((off / bound.clamp(min=1e-300)).max()):.3g} "
        "of the bound")


class Cache:
    """A paged cache on the CPU: random pages, the free rows full of `junk`."""

    def __init__(self, lengths, Hkv, page, d, dtype, seed=0, spare=3, junk=float("nan"),
                 fill=True, slack=0):
        g = torch.Generator().manual_seed(seed)
        self.page, self.lengths = page, list(lengths)
        pages = [-(-n // page) for n in lengths]
        self.num = sum(pages) + spare
        self.width = max([1] + pages) + slack
        order = torch.randperm(self.num, generator=g).tolist()
        self.table = torch.full((len(lengths), self.width), -7, dtype=torch.int32)
        self.k = torch.full((self.num, Hkv, page, d), junk, dtype=dtype)
        self.v = torch.full((self.num, Hkv, page, d), junk, dtype=dtype)
        for s, n in enumerate(pages):
            self.table[s, :n] = torch.tensor(order[:n], dtype=torch.int32)
            order = order[n:]
        if fill:
            for s, n in enumerate(lengths):
                for p in range(n):
                    at = int(self.table[s, p // page])
                    self.k[at, :, p % page] = torch.randn(Hkv, d, generator=g).to(dtype)
                    self.v[at, :, p % page] = torch.randn(Hkv, d, generator=g).to(dtype)

    def rows(self, s, first, last, ok=None):
        """Keys and values [Hkv, n, d] of sequence s, fp64, and their positions."""
        at = [p for p in range(first, last)
              if ok is None or 0 <= int(self.table[s, p // self.page]) < self.num]
        if not at:
            return None, None, None
        page = self.table[s, torch.tensor(at) // self.page].long()
        off = torch.tensor(at) % self.page
        return (self.k[page, :, off].transpose(0, 1).double(),
                self.v[page, :, off].transpose(0, 1).double(), torch.tensor(at))


def paged_attn(q, cache, lengths, scale=None, softcap=0.0, window=0, slopes=None, skip_bad=False):
    """(out, out bound, lse, lse bound) fp64 for q [S, Hq, d]."""
    S, Hq, d = q.shape
    Hkv = cache.k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out, ob = torch.zeros(S, Hq, d, dtype=torch.float64), torch.zeros(S, Hq, d, dtype=torch.float64)
    lse = torch.full((S, Hq), -math.inf, dtype=torch.float64)
    lb = torch.zeros(S, Hq, dtype=torch.float64)
    room = cache.table.shape[1] * cache.page
    # one rounding a product (fp32) or, on the tensor cores, sums cut at twice that
    gamma = d * (U if q.dtype == torch.float32 else 4 * U)
    for s in range(S):
        n = min(max(int(lengths[s]), 0), room)
        first = max(0, n - window) if window else 0
        k, v, at = cache.rows(s, first, n, ok=True if skip_bad else None)
        if k is None:
            continue
        qs = q[s].double().view(Hkv, Hq // Hkv, d)
        raw = torch.einsum("hgd,hjd->hgj", qs, k)
        z = raw * scale
        if softcap:
            z = softcap * torch.tanh(z / softcap)
        if slopes is not None:
            z = z + slopes.double().view(Hkv, -1, 1) * (at - (int(lengths[s]) - 1)).double()
        p = torch.softmax(z, -1)
        out[s] = torch.einsum("hgj,hjd->hgd", p, v).reshape(Hq, d)
        lse[s] = torch.logsumexp(z, -1).flatten()
        # a score is off by its dot product's roundings, and by 8 u of its size and of the
        # cap's (scale, tanh, bias and the running maximum); a weight by as much, relatively,
        # by its exponential (2^-21) and, bf16, by the 2^-16 that its two halves leave; then the
        # sums over the keys: u each.
        err = gamma * abs(scale) * torch.einsum("hgd,hjd->hgj", qs.abs(), k.abs())
        size = torch.maximum((raw * scale).abs().clamp(max=softcap or math.inf), z.abs())
        err = (err + 8 * U * (size + softcap)).amax(-1)
        rel = 2 * err + 2.0 ** -20 + 2.0 ** -15 * (q.dtype != torch.float32) + 2 * len(at) * U
        size = torch.einsum("hgj,hjd->hgd", p, v.abs()).reshape(Hq, d)
        ob[s] = rel.view(Hq, 1) * size + half_step(q.dtype) * out[s].abs()
        lb[s] = (rel + 4 * U * lse[s].view(Hkv, -1).abs()).flatten()
    return out, ob, lse, lb
