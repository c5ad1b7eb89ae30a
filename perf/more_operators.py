"""Measured cases of the operators for images and video, and of serving from a cache held in 4 bits.

Five kinds of pass:

* ``axes``        q and k of a fused projection, RMS-normed per head and rotated by positions of
                  several axes (rows and columns of an image, time in a video);
* ``axes_grad``   the gradients of that (inputs and norm weights);
* ``plan``        a serving step's pages: the pages of requests that are done go back to the pool,
                  new tokens get theirs, and every row of the step's packed tokens its position and
                  its place in the cache;
* ``append``      new tokens' keys and values into a paged cache of 4-bit codes;
* ``decode``      attention of one new token per sequence over that cache.

``run`` computes a pass in its plain form (elementary torch operations in fp32, angles in fp64), or,
where ``own`` is set, by this library's operators.  ``exact`` restates each definition in fp64.

The 4-bit cache holds a page's rows of a head one behind the other, d / 2 bytes each, value 2b in the
low half of byte b, and behind them their scales, one byte for each 32 values.  A value is
(code - 8) * scale; a scale byte holds the upper bits of an fp16 number without its sign (5 of
exponent, 3 of mantissa).  The 16-byte chunks of row r stand in the order c ^ ((r >> 1) & 3) for
d = 128 and c ^ ((r >> 2) & 1) for d = 64.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 32               # values of a scale


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------
def _axes(op, B, shape, Hq, Hkv, d, dtype="bf16", rot=None, interleaved=False, norm=True, lead=0,
          mixed=False, own_positions=False):
    """shape: "time x height x width" or "height x width"; lead: tokens before the grid's (a class
    token, a prompt's text); mixed: frequencies dealt to the axes in turn, not in sections."""
    return {"op": op, "B": B, "shape": shape, "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": dtype,
            "rot": d if rot is None else rot, "interleaved": interleaved, "norm": norm,
            "lead": lead, "mixed": mixed, "own_positions": own_positions}


def _plan(S, most, page, prompts, done=0, spare=8, padded=0):
    """A step: each sequence has up to ``most`` tokens and gets one more, or, with prompts, up to as
    many as that; ``done`` of them are done; ``spare``: free pages behind (or, negative, short of) those
    that the step needs; ``padded``: rows behind the last token."""
    return {"op": "plan", "S": S, "most": most, "page": page, "prompts": prompts, "done": done,
            "spare": spare, "padded": padded}


def _append(S, most, Hkv, d, page, dtype="bf16", step=True, padded=0):
    return {"op": "append", "S": S, "most": most, "Hkv": Hkv, "d": d, "page": page, "dtype": dtype,
            "step": step, "padded": padded}


def _decode(S, most, Hq, Hkv, d, page, dtype="bf16", ragged=True, padded=0, softcap=0.0, window=0,
            alibi=False, lse=False):
    return {"op": "decode", "S": S, "most": most, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page,
            "dtype": dtype, "ragged": ragged, "padded": padded, "softcap": softcap,
            "window": window, "alibi": alibi, "lse": lse}


def listed():
    named = [
        # one image of the library's 14 x 14 token grid with its 6 heads of 64: launch latency
        ("axes_grid_196", _axes("axes", 1, "14x14", 6, 6, 64)),
        # a video's latent grid behind a text prompt of odd length, grouped heads, three axes
        ("axes_video_66k", _axes("axes", 1, "16x64x64", 16, 4, 128, lead=777, own_positions=True)),
        # the gradient of a training batch of images, a class token before each
        ("axes_grad_images", _axes("axes_grad", 16, "32x32", 12, 12, 64, lead=1)),
        # fp32, neighbouring pairs, half of each head rotated, axes in turn: a small video step
        ("axes_grad_f32", _axes("axes_grad", 2, "5x13x11", 4, 1, 64, dtype="f32", rot=32,
                                interleaved=True, mixed=True, own_positions=True)),
        # one step of a served batch: most sequences stay within their last page; latency
        ("plan_step_200", _plan(200, 2500, 64, False, done=3, padded=8)),
        # prompts of a served batch, small pages, requests that are done among them
        ("plan_prompts", _plan(48, 4096, 16, True, done=6, padded=5)),
        # one step of a served batch, some rows padding: latency
        ("append_step_200", _append(200, 2500, 8, 128, 64, padded=8)),
        # prompts of a served batch entering the cache, ragged, small pages
        ("append_prompts", _append(24, 4096, 8, 128, 16, step=False, padded=5)),
        # one user's next token over a short cache: latency
        ("decode_one", _decode(1, 333, 32, 8, 128, 64, ragged=False)),
        # a served batch of ragged lengths, 4 query heads to a key head, idle slots among them
        ("decode_batch", _decode(128, 8192, 32, 8, 128, 64, padded=3)),
        # one cache of a million tokens, the library's longest sequence
        ("decode_long_1m", _decode(1, 1048575, 8, 2, 64, 256, ragged=False)),
        # fp32 with capped scores, a distance bias, a window and groups of 3
        ("decode_f32_capped", _decode(17, 2500, 9, 3, 64, 32, dtype="f32", softcap=20.0,
                                      window=1000, alibi=True, lse=True)),
    ]
    return [dict(case, name=name) for name, case in named]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ranges: sizes spread over their logarithm, cut to the largest listed
    case's traffic."""
    op = rng.choice(["axes", "axes_grad", "plan", "append", "append", "decode", "decode", "decode"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    es = 2 if dtype == "bf16" else 4
    d = rng.choice([32, 64, 64, 128, 128])
    Hkv = rng.choice([1, 2, 3, 4, 6, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    if op in ("axes", "axes_grad"):
        B = rng.choice([1, 1, 2, 3, 4, 16])
        most = max(4, int(3.0e8 / (B * (Hq + Hkv) * d * es)))
        n = _log(rng, 1, min(most, 1 << 17))
        h = max(1, int(round(n ** 0.5 * rng.uniform(0.5, 1.0))))
        t = rng.choice([0, 0, 1, 3, 8])
        w = max(1, n // (h * max(1, t)))
        shape = ("%dx" % t if t else "") + "%dx%d" % (h, w)
        return _axes(op, B, shape, Hq, Hkv, d, dtype, rng.choice([d, d, d // 2]),
                     rng.random() < 0.3, rng.random() < 0.8, rng.choice([0, 0, 1, 77]),
                     rng.random() < 0.3, rng.random() < 0.5)
    if op == "plan":
        prompts = rng.random() < 0.5
        S = _log(rng, 1, 256 if prompts else 2000)
        most = _log(rng, 1, 4096)
        while prompts and S * most > 400000:
            most = max(1, most // 2)
        return _plan(S, most, page, prompts, rng.randrange(0, max(1, S // 4) + 1),
                     rng.choice([0, 8, 500, -3]), rng.choice([0, 0, 1, 40]))
    if op == "append":
        step = rng.random() < 0.5
        S = _log(rng, 1, 256 if step else 24)
        most = _log(rng, 1, 4096)
        while S * most * Hkv * d * es > 2.2e8:
            most = max(1, most // 2)
        return _append(S, most, Hkv, d, page, dtype, step, rng.choice([0, 0, 1, 5]))
    S = _log(rng, 1, 256)
    most = _log(rng, 1, 65536)
    while S * most * Hkv * d > 6.0e8 or S * most * Hq > 4.0e7:
        most = max(1, most // 2)
    return _decode(S, most, Hq, Hkv, d, page, dtype, rng.random() < 0.8, rng.choice([0, 0, 2]),
                   rng.choice([0.0, 0.0, 30.0]), rng.choice([0, 0, 0, max(1, most // 3)]),
                   rng.random() < 0.3, rng.random() < 0.3)


def _grid(c):
    return [int(n) for n in c["shape"].split("x")]


def _tokens(c):
    return c["lead"] + math.prod(_grid(c))


def _lengths(c):
    """Keys of each sequence: ``most`` or, ragged, from one to ``most`` with the first at ``most``;
    idle slots (length 0) at the end."""
    S, most = c["S"], c["most"]
    ragged = c.get("ragged", True)
    live = max(1, S - c["padded"]) if c["op"] == "decode" else S
    got = []
    for i in range(S):
        if i >= live:
            got.append(0)
        elif i == 0 or not ragged:
            got.append(most)
        else:
            got.append(1 + (most - 1) * ((i * 7919 + 13) % 1009) // 1009)
    return got


def _step(c):
    """(tokens before the step, new tokens; -1: done) of each sequence in a plan."""
    before = _lengths(c)
    if c["prompts"]:
        # every third one continues a prompt, the others begin
        new, before = before, [n // 2 if i % 3 == 2 else 0 for i, n in enumerate(before)]
    else:
        new = [1] * c["S"]
    gone = {(i * 37 + 5) % c["S"] for i in range(c["done"])}
    before = [max(n, 1) if i in gone else n for i, n in enumerate(before)]
    return before, [-1 if i in gone else n for i, n in enumerate(new)]


def work(c):
    es = 2 if c.get("dtype") == "bf16" else 4
    if c["op"] in ("axes", "axes_grad"):
        d, A, N = c["d"], len(_grid(c)), _tokens(c)
        values = c["B"] * N * (c["Hq"] + c["Hkv"]) * d
        positions = 4 * A * N * (c["B"] if c["own_positions"] else 1)
        if c["op"] == "axes":
            return {"bytes": 2 * values * es + positions, "flops": 7 * values}
        return {"bytes": 3 * values * es + positions + (4 * 2 * d if c["norm"] else 0),
                "flops": 16 * values}
    if c["op"] == "plan":
        before, new = _step(c)
        rows = sum(max(0, n) for n in new) + c["padded"]
        pages = sum(-(-(b + max(0, n)) // c["page"]) for b, n in zip(before, new))
        # lengths and new tokens in, lengths, grants and row starts out; a row's position (4 bytes) and
        # place (8); page numbers
        return {"bytes": 20 * c["S"] + 12 * rows + 8 * pages, "flops": 4 * rows}
    d = c["d"]
    if c["op"] == "append":
        values = (c["S"] if c["step"] else sum(_lengths(c))) * c["Hkv"] * d
        # k and v read; their codes, scales and rounded values written
        return {"bytes": 2 * values * es * 2 + 2 * values * 17 // 32, "flops": 8 * values}
    keys = sum(min(n, c["window"]) if c["window"] else n for n in _lengths(c))
    rows = c["S"] * c["Hq"] * d
    return {"bytes": 2 * keys * c["Hkv"] * d * 17 // 32 + 2 * es * rows + 4 * -(-keys // c["page"]),
            "flops": 4 * keys * c["Hq"] * d}


# --------------------------------------------------------------------------------------------
# the 4-bit cache
# --------------------------------------------------------------------------------------------
def _scales_of(x):
    """The scale of each block [..., n, 32] fp32: a seventh of its largest size, rounded to 4 bits of
    an fp16 number's range; NaN for a block that holds an infinity or NaN."""
    t = x.abs().amax(-1)
    t = t / torch.full_like(t, 7.0)      # (a number as divisor would be a product with its inverse)
    power = (t.view(torch.int32) & 0x7f800000).view(torch.float32)        # the one at or below t
    quantum = power.clamp(min=2.0 ** -14) * 0.125
    s = (torch.round(t / quantum) * quantum).clamp(max=61440.0)
    return torch.where(torch.isfinite(t), s, math.nan)


def _quantise(x):
    """(whole numbers -7..7, scales) of rows [..., d] fp32; halves go towards zero."""
    blocks = x.unflatten(-1, (-1, BLOCK))
    s = _scales_of(blocks)
    r = torch.where(s > 0, (1.0 / s) * (1.0 - 2.0 ** -20), 0.0)[..., None]
    n = torch.round((blocks * r).clamp(-7.0, 7.0))
    return torch.where(torch.isfinite(s)[..., None], n, 0.0), s


def _chunk_order(rows, d):
    """For each row of a page the order in which its chunks of 16 bytes stand."""
    c = torch.arange(d // 32, device=rows.device)
    turn = (rows >> 1) & 3 if d == 128 else (rows >> 2) & 1 if d == 64 else rows * 0
    return c ^ turn[..., None]


def _bytes_of(n, s, rows):
    """(code bytes [..., d / 2], scale bytes [..., d / 32]) of rows that stand at `rows` [...] of
    their pages."""
    d = n.shape[-2] * BLOCK
    code = (n + 8.0).to(torch.uint8)
    chunks = code[..., 0::2] | (code[..., 1::2] << 4)             # [..., d / 32, 16]
    order = _chunk_order(rows, d)[..., None].expand(chunks.shape)
    chunks = torch.gather(chunks, -2, order)
    scale = (s.half().view(torch.int16) >> 7).to(torch.uint8)
    return chunks.flatten(-2), torch.where(torch.isnan(s), 255, scale)


def _parts(cache, page, d):
    """A cache [pages, Hkv, bytes] as its codes [pages, Hkv, page, d / 2] and scales
    [pages, Hkv, page, d / 32]."""
    codes, scales = cache.split((page * d // 2, page * d // 32), -1)
    return codes.unflatten(-1, (page, d // 2)), scales.unflatten(-1, (page, d // 32))


def _values_of(codes, scales, rows, d, dtype):
    """The values [..., d] that rows of a cache stand for."""
    chunks = codes.unflatten(-1, (-1, 16))
    order = _chunk_order(rows, d)[..., None].expand(chunks.shape)
    chunks = torch.gather(chunks, -2, order)
    n = torch.stack((chunks & 15, chunks >> 4), -1).flatten(-2).to(dtype) - 8
    s = (scales.to(torch.int16) << 7).view(torch.float16).to(dtype)
    return (n * s[..., None]).flatten(-2)


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------
def _table(pages, order, device):
    """Pages handed out in an order; entries behind a sequence's last one are -1."""
    table = torch.full((len(pages), max([1] + pages)), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return table.to(device)


def _prepare_axes(c, g, randn, dev):
    A, B, d, Hq, Hkv = len(_grid(c)), c["B"], c["d"], c["Hq"], c["Hkv"]
    half, N = c["rot"] // 2, _tokens(c)
    s = {"eps": 1e-6}
    s["inv_freq"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
    i = torch.arange(half, device=dev)
    s["freq_axis"] = (i % A if c["mixed"] else i * A // half).to(torch.int32)
    # a lead token stands at the same place on every axis, the grid behind it
    at = torch.arange(N - c["lead"], device=dev)
    places, rest = [], at
    for n in reversed(_grid(c)):
        places.insert(0, rest % n)
        rest = rest // n
    lead = torch.arange(c["lead"], device=dev)
    positions = torch.stack([torch.cat((lead, c["lead"] + p)) for p in places]).to(torch.int32)
    if c["own_positions"]:       # each of the batch at a place of its own
        shift = torch.randint(0, 100, (1, B, 1), generator=g, device=dev, dtype=torch.int32)
        positions = positions[:, None] + shift
    s["positions"] = positions.contiguous()
    weight = lambda: 1 + 0.2 * torch.randn(d, generator=g, device=dev)  # noqa: E731
    s["wq"], s["wk"] = (weight(), weight()) if c["norm"] else (None, None)
    # the projection's output: q, k and v heads of a token next to each other
    s["qkv"] = randn(B, N, Hq + 2 * Hkv, d)
    if c["op"] == "axes_grad":
        s["dq"], s["dk"] = randn(B, Hq, N, d), randn(B, Hkv, N, d)
    return s


def _prepare_plan(c, g, dev):
    before, new = _step(c)
    page = c["page"]
    held = [-(-n // page) for n in before]
    wanted = [-(-(b + max(0, n)) // page) for b, n in zip(before, new)]
    need = sum(w - h for w, h in zip(wanted, held))
    back = sum(h for h, n in zip(held, new) if n < 0)
    free = max(0, need - back + c["spare"])
    pool = sum(held) + free
    order = torch.randperm(pool, generator=g, device=dev).tolist()
    table = _table(held, order[free:], "cpu")
    wide = torch.full((c["S"], max(wanted) + 1), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    stack = torch.full((max(1, pool),), -1, dtype=torch.int32)
    stack[:free] = torch.tensor(order[:free], dtype=torch.int32)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    return {"new": ints(new), "lengths": ints(before), "table": wide.to(dev),
            "free": stack.to(dev), "count": ints([free]), "new_lengths": ints([0] * c["S"]),
            "new_count": ints([0]), "tokens": sum(max(0, n) for n in new) + c["padded"]}


def prepare(case, seed):
    c = dict(case)
    dev = "cuda"
    dt = DTYPES[c.get("dtype", "f32")]
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    if c["op"] in ("axes", "axes_grad"):
        return dict(_prepare_axes(c, g, randn, dev), case=c)
    if c["op"] == "plan":
        return dict(_prepare_plan(c, g, dev), case=c)
    Hkv, d, page, lengths = c["Hkv"], c["d"], c["page"], _lengths(c)
    s = {"case": c}
    pages = [-(-n // page) for n in lengths]
    used = sum(pages)
    pool = used + 7                      # the rest of the pool is other users'
    order = torch.randperm(pool, generator=g, device=dev)[:used].tolist()
    s["table"] = _table(pages, order, dev)
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=dev)

    def cache(scale):
        """A pool full of rows of normal values, some channels larger than others."""
        channel = scale * torch.exp(0.3 * torch.randn(Hkv, 1, d, generator=g, device=dev))
        out = torch.empty(pool, Hkv, page * d * 17 // 32, dtype=torch.uint8, device=dev)
        rows = torch.arange(page, device=dev).expand(Hkv, page)
        each = max(1, (1 << 26) // (Hkv * page * d))
        for p in range(0, pool, each):
            n = min(each, pool - p)
            x = torch.randn(n, Hkv, page, d, generator=g, device=dev) * channel
            codes, scales = _bytes_of(*_quantise(x), rows.expand(n, Hkv, page))
            out[p:p + n] = torch.cat((codes.flatten(2), scales.flatten(2)), -1)
        return out

    s["k_cache"], s["v_cache"] = cache(1.0), cache(0.5)
    if c["op"] == "append":
        seq = torch.arange(c["S"], device=dev)
        n = s["lengths"].long()
        if c["step"]:
            pos = n - 1
        else:
            seq = torch.repeat_interleave(seq, n)
            pos = torch.arange(len(seq), device=dev) - (torch.cumsum(n, 0) - n)[seq]
        slots = s["table"][seq, pos // page].long() * page + pos % page
        # rows that belong to nobody are spread among the others
        T = len(slots) + c["padded"]
        s["slots"] = torch.full((T,), -1, dtype=torch.int64, device=dev)
        s["slots"][torch.randperm(T, generator=g, device=dev)[:len(slots)].sort()[0]] = slots
        # the projection's output: k and v heads of a token next to each other
        s["kv"] = randn(T, 2 * Hkv, d)
        s["k_out"], s["v_out"] = (torch.zeros(T, Hkv, d, dtype=dt, device=dev) for _ in range(2))
        return s
    s["q"] = randn(c["S"], c["Hq"], d)
    s["slopes"] = None
    if c["alibi"]:
        i = torch.arange(1, c["Hq"] + 1, device=dev, dtype=torch.float32)
        s["slopes"] = 2.0 ** (-8.0 * i / c["Hq"])
    return s


# --------------------------------------------------------------------------------------------
# the plain form
# --------------------------------------------------------------------------------------------
def _rotate(x, cos, sin, rot, interleaved):
    """x [..., d] fp32, its first ``rot`` values turned by cos, sin [..., rot / 2]."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _turns(s):
    """cos and sin of every token's angles, [B or 1, 1, N, rot / 2]."""
    p = s["positions"] if s["positions"].dim() == 3 else s["positions"][:, None]
    angle = p[s["freq_axis"].long()].double() * s["inv_freq"][:, None, None]
    angle = angle.permute(1, 2, 0)[:, None]
    return angle.cos().float(), angle.sin().float()


def _heads(qkv, c):
    """q [B, Hq, N, d] and k [B, Hkv, N, d] in a fused projection's output."""
    q = qkv[:, :, :c["Hq"]].transpose(1, 2)
    k = qkv[:, :, c["Hq"]:c["Hq"] + c["Hkv"]].transpose(1, 2)
    return q, k


def _plain_axes(s, c):
    cos, sin = _turns(s)
    rot, inter, eps = c["rot"], c["interleaved"], s["eps"]

    def forward(x, w):
        u = x.float()
        if w is not None:
            u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + eps) * w
        return _rotate(u, cos, sin, rot, inter).to(x.dtype)

    def gradient(x, dy, w):
        g = _rotate(dy.float(), cos, -sin, rot, inter)
        if w is None:
            return g.to(x.dtype), None
        u = x.float()
        r = torch.rsqrt((u * u).mean(-1, keepdim=True) + eps)
        dw = (g * u * r).sum((0, 1, 2))
        gw = g * w
        dx = r * gw - u * (r * r * r) * (gw * u).mean(-1, keepdim=True)
        return dx.to(x.dtype), dw

    q, k = _heads(s["qkv"], c)
    if c["op"] == "axes":
        return [forward(q, s["wq"]), forward(k, s["wk"])]
    dq, dwq = gradient(q, s["dq"], s["wq"])
    dk, dwk = gradient(k, s["dk"], s["wk"])
    return [dq, dk, dwq, dwk] if c["norm"] else [dq, dk]


def _plain_plan(s, c):
    page, T, table, stack = c["page"], s["tokens"], s["table"], s["free"]
    S, width = table.shape
    n, new = s["lengths"].long(), s["new"].long()
    fresh = new.clamp(min=0)
    ends = torch.cumsum(fresh, 0)
    held = (n + page - 1) // page
    fits = (fresh > 0) & (n + fresh <= width * page) & (ends <= T)
    need = torch.where(fits, (n + fresh + page - 1) // page - held, 0)
    # pages of sequences that are done, in order, onto the stack
    col = torch.arange(width, device=n.device)
    back = ((new < 0)[:, None] & (col < held[:, None])).flatten()
    count = s["count"].long()
    at = torch.cumsum(back, 0) - 1 + count
    merged = torch.cat((stack, stack.new_zeros(1)))
    merged[torch.where(back, at, len(stack))] = table.flatten()
    avail = count + back.sum()
    # pages for new tokens, from its top, first come first served
    through = torch.cumsum(need, 0)
    granted = fits & ((need == 0) | (through <= avail))
    taken = torch.where(granted, through, 0).amax()
    j = col - held[:, None]
    mine = granted[:, None] & (j >= 0) & (j < need[:, None])
    top = (avail - 1 - (through - need)[:, None] - j).clamp(0, len(stack) - 1)
    table.copy_(torch.where(mine, merged[top], table))
    stack.copy_(merged[:-1])
    s["new_lengths"].copy_(torch.where(new < 0, 0, n + torch.where(granted, fresh, 0)))
    s["new_count"].copy_(avail - taken)
    # every row's sequence, position and place
    t = torch.arange(T, device=n.device)
    seq = torch.searchsorted(ends, t, right=True).clamp(max=S - 1)
    live = (t < ends[-1]) & granted[seq]
    pos = torch.where(live, n[seq] + t - (ends - fresh)[seq], 0)
    slot = table[seq, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    starts = torch.cat((ends.new_zeros(1), ends)).clamp(max=T)
    return [starts.int(), pos.int(), torch.where(live, slot, -1),
            torch.where(granted, fresh, 0).int(), s["new_lengths"], table, stack, s["new_count"]]


def _plain_append(s, c):
    Hkv, d, page = c["Hkv"], c["d"], c["page"]
    row = torch.nonzero(s["slots"] >= 0)[:, 0]
    slot = s["slots"][row]
    at, off = slot // page, slot % page
    for x, cache, out in ((s["kv"][:, :Hkv], s["k_cache"], s["k_out"]),
                          (s["kv"][:, Hkv:], s["v_cache"], s["v_out"])):
        n, scale = _quantise(x[row].float())
        codes, scales = _parts(cache, page, d)
        codes[at, :, off], scales[at, :, off] = _bytes_of(n, scale, off[:, None].expand(-1, Hkv))
        out[row] = (n * scale[..., None]).flatten(-2).to(out.dtype)
    return [s["k_out"], s["v_out"], s["k_cache"], s["v_cache"]]


def _plain_decode(s, c):
    S, Hq, Hkv, d, page = c["S"], c["Hq"], c["Hkv"], c["d"], c["page"]
    table, lengths = s["table"], s["lengths"]
    keys = table.shape[1] * page
    pages = table.clamp(min=0).long()
    j = torch.arange(keys, device=table.device)
    seen = j[None] < lengths[:, None]
    if c["window"]:
        seen = seen & (j[None] >= lengths[:, None] - c["window"])

    def rows(cache):
        codes, scales = _parts(cache, page, d)
        at = torch.arange(page, device=table.device).expand(pages.shape + (Hkv, page))
        x = _values_of(codes[pages], scales[pages], at, d, torch.float32)
        return x.transpose(1, 2).reshape(S, Hkv, keys, d)

    k = rows(s["k_cache"])
    score = torch.matmul(s["q"].float().view(S, Hkv, Hq // Hkv, d), k.transpose(2, 3))
    del k
    score = score * (1 / math.sqrt(d))
    if c["softcap"]:
        score = c["softcap"] * torch.tanh(score / c["softcap"])
    if s["slopes"] is not None:
        back = (j[None] - (lengths[:, None] - 1)).float()
        score = score + s["slopes"].view(1, Hkv, Hq // Hkv, 1) * back[:, None, None]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = rows(s["v_cache"]).masked_fill(~seen[:, None, :, None], 0.0)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    out = out.view(S, Hq, d).to(s["q"].dtype)
    return [out, (top + torch.log(total)).view(S, Hq)] if c["lse"] else [out]


# --------------------------------------------------------------------------------------------
# the library's operators
# --------------------------------------------------------------------------------------------
def _own(s, c):
    from sparse_top_landmark_gb300 import mita
    if c["op"] in ("axes", "axes_grad"):
        q, k = _heads(s["qkv"], c)
        how = dict(inv_freq=s["inv_freq"], freq_axis=s["freq_axis"], positions=s["positions"],
                   q_weight=s["wq"], k_weight=s["wk"], eps=s["eps"],
                   interleaved=c["interleaved"])
        if c["op"] == "axes":
            return list(mita.mita_qk_norm_rope_axes(q, k, **how))
        grads = mita.mita_qk_norm_rope_axes_backward(q, k, s["dq"], s["dk"], **how)
        return list(grads) if c["norm"] else list(grads[:2])
    if c["op"] == "plan":
        got = mita.mita_cache_plan(s["new"], s["lengths"], s["table"], s["free"], s["count"],
                                   tokens=s["tokens"], page_size=c["page"],
                                   new_lengths=s["new_lengths"], new_free_count=s["new_count"])
        return list(got) + [s["new_lengths"], s["table"], s["free"], s["new_count"]]
    if c["op"] == "append":
        k, v = s["kv"][:, :c["Hkv"]], s["kv"][:, c["Hkv"]:]
        mita.mita_cache_append_q4(k, v, s["k_cache"], s["v_cache"], s["slots"], k_out=s["k_out"],
                                  v_out=s["v_out"])
        return [s["k_out"], s["v_out"], s["k_cache"], s["v_cache"]]
    got = mita.mita_paged_attn_q4(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"],
                                  softcap=c["softcap"], window=c["window"],
                                  alibi_slopes=s["slopes"], return_lse=c["lse"])
    return list(got) if c["lse"] else [got]


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    if c["op"] in ("axes", "axes_grad"):
        return _plain_axes(state, c)
    if c["op"] == "plan":
        return _plain_plan(state, c)
    return _plain_append(state, c) if c["op"] == "append" else _plain_decode(state, c)


# --------------------------------------------------------------------------------------------
# the definitions in fp64
# --------------------------------------------------------------------------------------------
def _exact_axes(s, c):
    d, rot, N = c["d"], c["rot"], _tokens(c)
    i = torch.arange(d, device="cuda")
    half = rot // 2
    if c["interleaved"]:
        partner, first, f = torch.where(i < rot, i ^ 1, i), i % 2 == 0, i // 2
    else:
        partner = torch.where(i < half, i + half, torch.where(i < rot, i - half, i))
        first, f = i < half, i % half
    f = f.clamp(max=half - 1)
    freq = torch.exp(-math.log(10000.0) * f.double() / half) * (i < rot)
    A = len(_grid(c))
    axis = f % A if c["mixed"] else f * A // half
    sign = torch.where(first, -1.0, 1.0).double()
    outs, sums = [], []
    for name, at, heads in (("q", 0, c["Hq"]), ("k", c["Hq"], c["Hkv"])):
        w = s["w" + name]
        out = torch.empty(c["B"], heads, N, d, dtype=torch.float64, device="cuda")
        total = torch.zeros(d, dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            p = s["positions"][:, b] if c["own_positions"] else s["positions"]
            angle = torch.stack([p[a] for a in axis.tolist()], -1).double() * freq
            same, other = torch.cos(angle), torch.sin(angle) * sign * (i < rot)
            for h in range(heads):
                x = s["qkv"][b, :, at + h].double()
                norm = torch.sqrt((x ** 2).sum(-1, keepdim=True) / d + s["eps"])
                if c["op"] == "axes":
                    u = x if w is None else x / norm * w.double()
                    out[b, h] = u * same + u[:, partner] * other
                    continue
                dy = s["d" + name][b, h].double()
                # value i is reached from i (same) and from its partner
                g = dy * same + (dy * other)[:, partner]
                if w is None:
                    out[b, h] = g
                    continue
                unit = x / norm
                total += (g * unit).sum(0)
                gw = g * w.double()
                out[b, h] = (gw - unit * (gw * unit).sum(-1, keepdim=True) / d) / norm
        outs.append(out)
        sums.append(total)
    return outs + sums if c["op"] == "axes_grad" and c["norm"] else outs


def _exact_rows(x, d):
    """Values [T, H, d] as the cache keeps them."""
    b = x.double().unflatten(-1, (-1, BLOCK))
    t = b.abs().amax(-1, keepdim=True) / 7
    _, exponent = torch.frexp(t)
    powers = torch.tensor([2.0 ** (e - 4) for e in range(-13, 18)], dtype=torch.float64, device="cuda")
    step = powers[(exponent + 13).clamp(0, 30)]
    s = (torch.round(t / step) * step).clamp(max=61440.0)
    n = torch.ceil(b.abs() / torch.where(s > 0, s, 1.0) - 0.5).clamp(0, 7)
    return (torch.sign(b) * n * s).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] in ("axes", "axes_grad"):
        return _exact_axes(s, c)
    if c["op"] == "plan":
        return None                      # whole numbers throughout
    Hkv, d, page = c["Hkv"], c["d"], c["page"]
    if c["op"] == "append":
        outs = []
        for x, out in ((s["kv"][:, :Hkv], s["k_out"]), (s["kv"][:, Hkv:], s["v_out"])):
            outs.append(torch.where((s["slots"] < 0)[:, None, None], out.double(),
                                    _exact_rows(x, d)))
        return outs + [None, None]
    Hq, lengths, table = c["Hq"], _lengths(c), s["table"].tolist()
    out = torch.zeros(c["S"], Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((c["S"], Hq), -math.inf, dtype=torch.float64, device="cuda")
    codes = torch.arange(256, device="cuda")
    pairs = torch.stack((codes % 16 - 8, codes // 16 - 8), -1).double()      # of a code byte
    scale_of = torch.tensor([b * 2.0 ** -17 if b < 8 else (8 + b % 8) * 2.0 ** (b // 8 - 18)
                             for b in range(256)], dtype=torch.float64, device="cuda")
    row = torch.arange(page, device="cuda")
    turn = {128: (row // 2) % 4, 64: (row // 4) % 2, 32: row * 0}[d]

    def values(cache, used):
        raw = cache[used].long()                                             # [n, Hkv, bytes]
        byte = raw[..., :page * d // 2].reshape(len(used), Hkv, page, d // 32, 16)
        byte = torch.stack([byte[:, :, r, turn[r] ^ torch.arange(d // 32, device="cuda")]
                            for r in range(page)], 2)
        x = pairs[byte].flatten(-2)
        x = x * scale_of[raw[..., page * d // 2:]].reshape(x.shape[:-1] + (1,))
        return x.flatten(-2).permute(1, 0, 2, 3).flatten(1, 2)               # [Hkv, keys, d]

    for i, n in enumerate(lengths):
        if n == 0:
            continue
        first = max(0, n - c["window"]) if c["window"] else 0
        used = torch.tensor(table[i][:-(-n // page)], device="cuda", dtype=torch.int64)
        k, v = (values(x, used)[:, first:n] for x in (s["k_cache"], s["v_cache"]))
        q = s["q"][i].double().view(Hkv, Hq // Hkv, d)
        z = torch.einsum("hgd,hjd->hgj", q, k) / d ** 0.5
        if c["softcap"]:
            z = torch.tanh(z / c["softcap"]) * c["softcap"]
        if s["slopes"] is not None:
            away = torch.arange(first - (n - 1), 1, device="cuda", dtype=torch.float64)
            z = z + s["slopes"].double().view(Hkv, Hq // Hkv, 1) * away
        lse[i] = torch.logsumexp(z, -1).flatten()
        out[i] = torch.einsum("hgj,hjd->hgd", torch.softmax(z, -1), v).reshape(Hq, d)
    return [out, lse] if c["lse"] else [out]
