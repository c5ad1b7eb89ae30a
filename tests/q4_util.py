"""Plain restatements (CPU) of the 4-bit cache and of the page plan, and the error bounds that the GPU tests
hold the attention over that cache to.

Half a step of a type, relative to the value, is finfo(t).eps / 2; u = 2^-24 is fp32's, 2^-11 fp16's.
"""
import math

import numpy as np
import torch

import decode_util as R

U = R.U
BLOCK = 32
CODE = 8


def scale_of_byte(b):
    """What a scale byte stands for: bits 7 to 14 of an fp16 number."""
    return float(np.array([b << 7], dtype=np.uint16).view(np.float16)[0])


SCALES = [scale_of_byte(b) for b in range(248)]


def scale_byte(a):
    """The byte of the scale nearest to a / 7 (ties to the even byte), at most the largest finite one."""
    t = float(np.float32(a) / np.float32(7))
    if not math.isfinite(t):
        return 255
    at = int(np.searchsorted(SCALES, t))
    if at >= 248:
        return 247
    if at == 0 or SCALES[at] == t:
        return at
    lo, hi = t - SCALES[at - 1], SCALES[at] - t
    return at if hi < lo or (hi == lo and at % 2 == 0) else at - 1


def quantise(rows):
    """(codes [..., d], scale bytes [..., d / 32], values [..., d] fp32) of rows [..., d]; fp32
    arithmetic as the header says."""
    x = rows.float().numpy().reshape(-1, BLOCK)
    a = np.abs(x).max(-1)
    byte = np.array([scale_byte(v) for v in a], dtype=np.int64)
    s = np.array([scale_of_byte(b) for b in byte], dtype=np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.where(s > 0, (np.float32(1) / s) * np.float32(1 - 2.0 ** -20), np.float32(0))
        n = np.rint(np.clip(x * r[:, None].astype(np.float32), -7, 7))
    n = np.where(np.isfinite(a)[:, None] & (s > 0)[:, None], n, 0)
    value = (n * s[:, None]).astype(np.float32)
    shape = rows.shape
    return (torch.from_numpy(n.astype(np.int64) + CODE).view(shape),
            torch.from_numpy(byte).view(shape[:-1] + (shape[-1] // BLOCK,)),
            torch.from_numpy(value).view(shape))


def chunk_place(c, row, d):
    return c ^ ({128: row >> 1 & 3, 64: row >> 2 & 1, 32: 0}[d])


class Cache4:
    """A 4-bit paged cache on the CPU: random pages; free rows full of `junk` bytes (255: codes 15 and
    scales NaN)."""

    def __init__(self, lengths, Hkv, page, d, seed=0, spare=3, junk=255, slack=0, k=None, v=None,
                 spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.page, self.lengths, self.d, self.Hkv = page, list(lengths), d, Hkv
        pages = [-(-n // page) for n in lengths]
        self.num = sum(pages) + spare
        self.width = max([1] + pages) + slack
        order = torch.randperm(self.num, generator=g).tolist()
        self.table = torch.full((len(lengths), self.width), -7, dtype=torch.int32)
        self.row_bytes = 17 * d // 32
        self.k8, self.v8 = (torch.full((self.num, Hkv, page * self.row_bytes), junk, dtype=torch.uint8)
                            for _ in range(2))
        for s, n in enumerate(pages):
            self.table[s, :n] = torch.tensor(order[:n], dtype=torch.int32)
            order = order[n:]
        self.kv = []             # per sequence: values [Hkv, n, d] and value scales, of k and v
        for s, n in enumerate(lengths):
            rows = []
            for given, cache in ((k, self.k8), (v, self.v8)):
                x = (torch.randn(Hkv, n, d, generator=g) * spread if given is None
                     else given[s].float())
                rows.append(self.put(cache, s, x))
            self.kv.append(rows)

    def place(self, s, p):
        return int(self.table[s, p // self.page]), p % self.page

    def put(self, cache, s, x):
        """Rows [Hkv, n, d] of sequence s from position 0 on; their values and scales, fp64."""
        Hkv, n, d = x.shape
        code, byte, value = quantise(x)
        for p in range(n):
            at, row = self.place(s, p)
            for h in range(Hkv):
                cache[at, h] = put_row(cache[at, h], code[h, p], byte[h, p], row, self.page, d)
        scale = torch.tensor([scale_of_byte(int(b)) for b in byte.flatten()],
                             dtype=torch.float64).view(Hkv, n, d // BLOCK)
        return value.double(), scale.repeat_interleave(BLOCK, -1)

    def rows(self, s, first, last, ok=None):
        at = [p for p in range(first, last)
              if ok is None or 0 <= int(self.table[s, p // self.page]) < self.num]
        if not at:
            return None, None, None, None, None
        (k, ks), (v, vs) = self.kv[s]
        t = torch.tensor(at)
        return k[:, t], ks[:, t], v[:, t], vs[:, t], t


def put_row(page_bytes, code, byte, row, page, d):
    """One head's page with a row written."""
    out = page_bytes.clone()
    pairs = (code[0::2] | code[1::2] << 4).to(torch.uint8)
    for c in range(d // 32):
        to = row * d // 2 + 16 * chunk_place(c, row, d)
        out[to:to + 16] = pairs[16 * c:16 * c + 16]
    at = page * d // 2 + row * (d // 32)
    out[at:at + d // 32] = byte.to(torch.uint8)
    return out


def read_row(page_bytes, row, page, d):
    """(codes [d], scale bytes [d / 32]) of a row of one head's page."""
    b = page_bytes.to(torch.int64)
    parts = []
    for c in range(d // 32):
        at = row * d // 2 + 16 * chunk_place(c, row, d)
        x = b[at:at + 16]
        parts.append(torch.stack((x & 15, x >> 4), -1).flatten())
    at = page * d // 2 + row * (d // 32)
    return torch.cat(parts), b[at:at + d // 32]


def paged_attn(q, cache, lengths, scale=None, softcap=0.0, window=0, slopes=None, skip_bad=False):
    """(out, out bound, lse, lse bound) fp64 for q [S, Hq, d] over a Cache4."""
    S, Hq, d = q.shape
    Hkv = cache.Hkv
    scale = d ** -0.5 if scale is None else scale
    f32 = q.dtype == torch.float32
    out, ob = torch.zeros(S, Hq, d, dtype=torch.float64), torch.zeros(S, Hq, d, dtype=torch.float64)
    lse = torch.full((S, Hq), -math.inf, dtype=torch.float64)
    lb = torch.zeros(S, Hq, dtype=torch.float64)
    room = cache.table.shape[1] * cache.page
    for s in range(S):
        n = min(max(int(lengths[s]), 0), room)
        first = max(0, n - window) if window else 0
        k, ks, v, vs, at = cache.rows(s, first, n, ok=True if skip_bad else None)
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
        # A score's sums are cut, a term at twice a rounding, twice over where a query is two values (whose
        # halves leave 2^-22 of it); bf16 takes code n as n q - 8 q, so that a term is up to 8 scales
        # larger than its value.  Then 8 u of its size and of the cap's.
        terms = torch.einsum("hgd,hjd->hgj", qs.abs(), k.abs() + (0 if f32 else 8) * ks)
        err = (d * 4 * U * (2 if f32 else 1) + (2.0 ** -22 if f32 else 0)) * abs(scale) * terms
        size = torch.maximum((raw * scale).abs().clamp(max=softcap or math.inf), z.abs())
        err = (err + 8 * U * (size + softcap)).amax(-1)
        # a weight is off by as much, relatively, by its exponential (2^-21), and by its roundings: two to
        # fp16 (bf16), or what two fp16 values leave of its product with the scale (2^-22); below fp16's
        # normal numbers, where the largest weight is 2^10 to 2^15 and its scale at most 2, by 2^-25 once
        # or twice, which is 2^-34 of the largest weight times seven scales a key.
        rel = (2 * err + 2.0 ** -20 + (2.0 ** -21 if f32 else 2.0 ** -10) + 2 * len(at) * U)
        size = torch.einsum("hgj,hjd->hgd", p, v.abs()).reshape(Hq, d)
        tiny = 7 * len(at) * 2.0 ** -34 * (1 + vs.amax()) * p.amax()
        ob[s] = rel.view(Hq, 1) * size + tiny + R.half_step(q.dtype) * out[s].abs()
        # the logarithm's sum is of weights before their rounding
        rel = 2 * err + 2.0 ** -20 + 2 * len(at) * U
        lb[s] = (rel + 4 * U * lse[s].view(Hkv, -1).abs()).flatten()
    return out, ob, lse, lb


def plan(new, lengths, table, free, count, tokens, page):
    """A step's plan in plain Python; lists.  Returns what the call gives and changes, as a dict."""
    S, width, pages = len(new), len(table[0]) if table else 0, len(free)
    table, free = [list(r) for r in table], list(free)
    ceil = lambda n: -(-n // page)  # noqa: E731
    lengths = list(lengths)
    count = min(max(count, 0), pages)
    for s in range(S):
        if new[s] == -1:
            held = min(ceil(max(lengths[s], 0)), width)
            for p in table[s][:held]:
                if count < pages:
                    free[count] = p
                    count += 1
    top, wanted, taken, row = count, 0, 0, 0
    starts, granted, positions, slots = [], [], [0] * tokens, [-1] * tokens
    after = list(lengths)
    old = [list(r) for r in table]
    for s in range(S):
        n = max(new[s], 0)
        starts.append(min(row, tokens))
        fits = (n > 0 and 0 <= lengths[s] and lengths[s] + n <= width * page and row + n <= tokens)
        need = ceil(lengths[s] + n) - ceil(lengths[s]) if fits else 0
        first = wanted
        wanted += need
        ok = fits and (need == 0 or wanted <= top)
        granted.append(n if ok else 0)
        if new[s] == -1:
            after[s] = 0
        if ok:
            taken = max(taken, wanted if need else 0)
            held = ceil(lengths[s])
            for i in range(need):
                table[s][held + i] = free[top - 1 - first - i]
            after[s] = lengths[s] + n
            for j in range(n):
                pos = lengths[s] + j
                at = (table if pos // page >= held else old)[s][pos // page]
                positions[row + j] = pos
                slots[row + j] = at * page + pos % page if 0 <= at < pages else -1
        row += n
    starts.append(min(row, tokens))
    return dict(seq_start=starts, positions=positions, slots=slots, granted=granted, new_lengths=after,
                table=table, free=free, count=top - taken)
