"""Measured cases of the language-model operators around the attention of this library.

Four kinds of pass:

* ``norm_rope``       q and k of a fused projection, RMS-normed per head and rotated by position;
* ``norm_rope_grad``  the gradients of that (inputs and norm weights);
* ``append``          new tokens: q normed and rotated, k normed, rotated and written with v into a
                      paged key-value cache;
* ``decode``          attention of one new token per sequence over the paged cache.

``run`` computes a pass in its plain form (elementary torch operations in fp32, angles in fp64), or,
where ``own`` is set, by this library's operators.  ``exact`` restates each definition in fp64.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------
def _rope(op, B, N, Hq, Hkv, d, dtype="bf16", rot=None, interleaved=False, norm=True):
    return {"op": op, "B": B, "N": N, "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": dtype,
            "rot": d if rot is None else rot, "interleaved": interleaved, "norm": norm}


def _append(S, most, Hq, Hkv, d, page, dtype="bf16", step=True, ragged=True, padded=0, rot=None,
            interleaved=False, norm=True):
    return {"op": "append", "S": S, "most": most, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page,
            "dtype": dtype, "step": step, "ragged": ragged, "padded": padded,
            "rot": d if rot is None else rot, "interleaved": interleaved, "norm": norm}


def _decode(S, most, Hq, Hkv, d, page, dtype="bf16", ragged=True, padded=0, softcap=0.0, window=0,
            alibi=False, lse=False):
    return {"op": "decode", "S": S, "most": most, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page,
            "dtype": dtype, "ragged": ragged, "padded": padded, "softcap": softcap,
            "window": window, "alibi": alibi, "lse": lse}


def listed():
    named = [
        # one image of the library's 14 x 14 token grid with its 6 heads of 64: launch latency
        ("rope_grid_196", _rope("norm_rope", 1, 196, 6, 6, 64)),
        # the library's longest sequence (2 heads of 64): positions up to a million
        ("rope_long_1m", _rope("norm_rope", 1, 1048576, 2, 2, 64)),
        # grouped heads, half of each head rotated, an odd length: a training batch's forward
        ("rope_gqa_8k", _rope("norm_rope", 2, 8191, 32, 8, 128, rot=64)),
        # the gradient of such a training batch
        ("rope_grad_gqa_4k", _rope("norm_rope_grad", 2, 4096, 32, 8, 128)),
        # fp32, neighbouring pairs, one shared key head, ragged: a small training step
        ("rope_grad_f32", _rope("norm_rope_grad", 3, 777, 4, 1, 32, dtype="f32", interleaved=True)),
        # one user's next token: latency
        ("append_one", _append(1, 900, 32, 8, 128, 64)),
        # one step of a served batch, 200 slots of which 8 are idle
        ("append_step_200", _append(200, 2500, 32, 8, 128, 64, padded=8)),
        # prompts of a served batch entering the cache, ragged, small pages
        ("append_prompts", _append(24, 4096, 32, 8, 128, 16, step=False)),
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
    op = rng.choice(["norm_rope", "norm_rope_grad", "append", "append", "decode", "decode",
                     "decode"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([32, 64, 64, 128, 128])
    Hkv = rng.choice([1, 2, 3, 4, 6, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    rot = rng.choice([d, d, d // 2])
    pairs = rng.random() < 0.3
    norm = rng.random() < 0.8
    es = 2 if dtype == "bf16" else 4
    if op in ("norm_rope", "norm_rope_grad"):
        B = rng.choice([1, 1, 2, 3, 4])
        most = int(3.0e8 / (B * (Hq + Hkv) * d * es))
        N = _log(rng, 1, max(2, min(most, 1 << 18)))
        return _rope(op, B, N, Hq, Hkv, d, dtype, rot, pairs, norm)
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        step = rng.random() < 0.5
        S = _log(rng, 1, 256 if step else 24)
        most = _log(rng, 1, 2500)
        while S * most * Hkv * d * es > 2.0e8:
            most = max(1, most // 2)
        return _append(S, most, Hq, Hkv, d, page, dtype, step, rng.random() < 0.8,
                       rng.choice([0, 0, 1, 5]) if step else 0, rot, pairs, norm)
    S = _log(rng, 1, 256)
    most = _log(rng, 1, 65536)
    while S * most * Hkv * d * es > 4.0e8 or S * most * Hq > 4.0e7:
        most = max(1, most // 2)
    return _decode(S, most, Hq, Hkv, d, page, dtype, rng.random() < 0.8, rng.choice([0, 0, 2]),
                   rng.choice([0.0, 0.0, 30.0]), rng.choice([0, 0, 0, max(1, most // 3)]),
                   rng.random() < 0.3, rng.random() < 0.3)


def _lengths(c):
    """Keys of each sequence after the call: ``most`` or, ragged, from one to ``most`` with the
    first at ``most``; idle slots (length 0) at the end."""
    S, most = c["S"], c["most"]
    live = max(1, S - c["padded"])
    got = []
    for i in range(S):
        if i >= live:
            got.append(0)
        elif i == 0 or not c["ragged"]:
            got.append(most)
        else:
            got.append(1 + (most - 1) * ((i * 7919 + 13) % 1009) // 1009)
    return got


def _new_tokens(c):
    """New tokens of each sequence in this append: 1 in a step, all of them in a prompt."""
    lengths = _lengths(c)
    return [1] * c["S"] if c["step"] else lengths


def work(c):
    es = 2 if c["dtype"] == "bf16" else 4
    d = c["d"]
    if c["op"] in ("norm_rope", "norm_rope_grad"):
        values = c["B"] * c["N"] * (c["Hq"] + c["Hkv"]) * d
        if c["op"] == "norm_rope":
            return {"bytes": 2 * values * es, "flops": 7 * values}
        return {"bytes": 3 * values * es + (4 * 2 * d if c["norm"] else 0), "flops": 16 * values}
    if c["op"] == "append":
        tokens = sum(n for n, keys in zip(_new_tokens(c), _lengths(c)) if keys)
        values = tokens * (c["Hq"] + c["Hkv"]) * d
        return {"bytes": 2 * es * (values + tokens * c["Hkv"] * d), "flops": 7 * values}
    keys = sum(min(n, c["window"]) if c["window"] else n for n in _lengths(c))
    rows = c["S"] * c["Hq"] * d
    return {"bytes": es * (2 * keys * c["Hkv"] * d + 2 * rows) + 4 * -(-keys // c["page"]),
            "flops": 4 * keys * c["Hq"] * d}


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------
def _inv_freq(rot, device):
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)


def prepare(case, seed):
    c = dict(case)
    dev = "cuda"
    dt = DTYPES[c["dtype"]]
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    def weight():
        return 1 + 0.2 * torch.randn(d, generator=g, device=dev)

    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    s = {"case": c, "eps": 1e-6}
    if c["op"] != "decode":
        s["inv_freq"] = _inv_freq(c["rot"], dev)
        s["wq"], s["wk"] = (weight(), weight()) if c["norm"] else (None, None)
    if c["op"] in ("norm_rope", "norm_rope_grad"):
        # the projection's output: q, k and v heads of a token next to each other
        s["qkv"] = randn(c["B"], c["N"], Hq + 2 * Hkv, d)
        if c["op"] == "norm_rope_grad":
            s["dq"] = randn(c["B"], Hq, c["N"], d)
            s["dk"] = randn(c["B"], Hkv, c["N"], d)
        return s
    # the cache: pages handed out in a random order, the rest of the pool other users'
    lengths = _lengths(c)
    page = c["page"]
    pages = [-(-n // page) for n in lengths]
    width, used = max(1, max(pages)), sum(pages)
    pool = used + 7
    order = torch.randperm(pool, generator=g, device=dev)[:used].tolist()
    table = torch.full((c["S"], width), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    s["table"] = table.to(dev)
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=dev)
    s["k_cache"] = randn(pool, Hkv, page, d)
    s["v_cache"] = randn(pool, Hkv, page, d)
    if c["op"] == "append":
        counts = _new_tokens(c)
        T = sum(counts)
        # prompts come in a buffer that is longer than they are
        s["qkv"] = randn(T if c["step"] else T + 5, Hq + 2 * Hkv, d)
        s["q_out"] = torch.zeros(s["qkv"].shape[0], Hq, d, device=dev, dtype=dt)
        starts = [0]
        for n in counts:
            starts.append(starts[-1] + n)
        s["starts"] = None if c["step"] else torch.tensor(starts, dtype=torch.int32, device=dev)
        # the plain form's row of every new token: sequence, position and row of the buffer
        row = [(i, lengths[i] - n + j, starts[i] + j) for i, n in enumerate(counts)
               for j in range(n) if lengths[i]]
        s["rows"] = torch.tensor(row, dtype=torch.int64, device=dev)
        return s
    s["q"] = randn(c["S"], Hq, d)
    s["slopes"] = None
    if c["alibi"]:
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device=dev, dtype=torch.float32) / Hq)
    return s


# --------------------------------------------------------------------------------------------
# the plain form
# --------------------------------------------------------------------------------------------
def _angles(positions, inv_freq):
    turn = positions.double()[..., None] * inv_freq
    return turn.cos().float(), turn.sin().float()


def _rotate(x, cos, sin, rot, interleaved):
    """x [..., d] fp32, its first ``rot`` values turned by cos, sin [..., rot / 2]."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _norm(x, weight, eps):
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight


def _norm_rope(x, weight, eps, cos, sin, rot, interleaved):
    return _rotate(_norm(x.float(), weight, eps), cos, sin, rot, interleaved).to(x.dtype)


def _norm_rope_grad(x, dy, weight, eps, cos, sin, rot, interleaved):
    xf = x.float()
    gy = _rotate(dy.float(), cos, -sin, rot, interleaved)
    if weight is None:
        return gy.to(x.dtype), None
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + eps)
    dw = (gy * xf * r).sum((0, 1, 2))
    gw = gy * weight
    dx = r * gw - xf * (r * r * r) * (gw * xf).mean(-1, keepdim=True)
    return dx.to(x.dtype), dw


def _heads(qkv, c):
    """q [B, Hq, N, d] and k [B, Hkv, N, d] in a fused projection's output."""
    q = qkv[:, :, :c["Hq"]].transpose(1, 2)
    k = qkv[:, :, c["Hq"]:c["Hq"] + c["Hkv"]].transpose(1, 2)
    return q, k


def _token_heads(qkv, c):
    """q [T, Hq, d], k and v [T, Hkv, d] in a fused projection's output."""
    a, b = c["Hq"], c["Hq"] + c["Hkv"]
    return qkv[:, :a], qkv[:, a:b], qkv[:, b:]


def _plain_rope(s, c):
    q, k = _heads(s["qkv"], c)
    cos, sin = _angles(torch.arange(c["N"], device=q.device), s["inv_freq"])
    how = (s["eps"], cos, sin, c["rot"], c["interleaved"])
    if c["op"] == "norm_rope":
        return [_norm_rope(q, s["wq"], *how), _norm_rope(k, s["wk"], *how)]
    dq, dwq = _norm_rope_grad(q, s["dq"], s["wq"], *how)
    dk, dwk = _norm_rope_grad(k, s["dk"], s["wk"], *how)
    return [dq, dk, dwq, dwk] if c["norm"] else [dq, dk]


def _plain_append(s, c):
    seq, pos, row = s["rows"].unbind(1)
    q, k, v = _token_heads(s["qkv"], c)
    cos, sin = _angles(pos, s["inv_freq"])
    how = (s["eps"], cos[:, None], sin[:, None], c["rot"], c["interleaved"])
    s["q_out"][row] = _norm_rope(q[row], s["wq"], *how)
    page = s["table"][seq, pos // c["page"]].long()
    s["k_cache"][page, :, pos % c["page"]] = _norm_rope(k[row], s["wk"], *how)
    s["v_cache"][page, :, pos % c["page"]] = v[row]
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _plain_decode(s, c):
    S, Hq, Hkv, d = c["S"], c["Hq"], c["Hkv"], c["d"]
    table, lengths = s["table"], s["lengths"]
    keys = table.shape[1] * c["page"]
    pages = table.clamp(min=0).long()
    j = torch.arange(keys, device=table.device)
    seen = j[None] < lengths[:, None]
    if c["window"]:
        seen = seen & (j[None] >= lengths[:, None] - c["window"])
    k = s["k_cache"][pages].transpose(1, 2).reshape(S, Hkv, keys, d).float()
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
    v = s["v_cache"][pages].transpose(1, 2).reshape(S, Hkv, keys, d).float()
    v = v.masked_fill(~seen[:, None, :, None], 0.0)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    out = out.view(S, Hq, d).to(s["q"].dtype)
    return [out, (top + torch.log(total)).view(S, Hq)] if c["lse"] else [out]


# --------------------------------------------------------------------------------------------
# the library's operators
# --------------------------------------------------------------------------------------------
def _own(s, c):
    from sparse_top_landmark_gb300 import mita
    if c["op"] in ("norm_rope", "norm_rope_grad"):
        q, k = _heads(s["qkv"], c)
        how = dict(inv_freq=s["inv_freq"], q_weight=s["wq"], k_weight=s["wk"], eps=s["eps"],
                   interleaved=c["interleaved"])
        if c["op"] == "norm_rope":
            return list(mita.mita_qk_norm_rope(q, k, **how))
        grads = mita.mita_qk_norm_rope_backward(q, k, s["dq"], s["dk"], **how)
        return list(grads) if c["norm"] else list(grads[:2])
    if c["op"] == "append":
        q, k, v = _token_heads(s["qkv"], c)
        mita.mita_cache_append(k, v, s["k_cache"], s["v_cache"], s["table"], s["lengths"],
                               seq_start=s["starts"], q=q, inv_freq=s["inv_freq"],
                               q_weight=s["wq"], k_weight=s["wk"], eps=s["eps"],
                               interleaved=c["interleaved"], q_out=s["q_out"])
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    got = mita.mita_paged_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"],
                               softcap=c["softcap"], window=c["window"],
                               alibi_slopes=s["slopes"], return_lse=c["lse"])
    return list(got) if c["lse"] else [got]


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    if c["op"] in ("norm_rope", "norm_rope_grad"):
        return _plain_rope(state, c)
    return _plain_append(state, c) if c["op"] == "append" else _plain_decode(state, c)


# --------------------------------------------------------------------------------------------
# the definitions in fp64
# --------------------------------------------------------------------------------------------
def _turn_matrix(positions, rot, d, interleaved, device):
    """For each position the partner of every value and the two factors of the rotation:
    y = x * same + x[partner] * other."""
    i = torch.arange(d, device=device)
    half = rot // 2
    if interleaved:
        partner = torch.where(i < rot, i ^ 1, i)
        first, f = i % 2 == 0, i // 2
    else:
        partner = torch.where(i < half, i + half, torch.where(i < rot, i - half, i))
        first, f = i < half, i % max(1, half)
    freq = torch.exp(-math.log(10000.0) * 2.0 * f.double() / rot)
    angle = positions.double()[:, None] * freq
    in_rot = (i < rot).double()
    same = torch.cos(angle) * in_rot + (1 - in_rot)
    other = torch.sin(angle) * in_rot * torch.where(first, -1.0, 1.0).double()
    return partner, same, other


def _exact_forward(x, weight, eps, turn):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + eps) * weight.double()
    partner, same, other = turn
    return x * same + x[..., partner] * other


def _exact_gradient(x, dy, weight, eps, turn):
    """One head [N, d] at a time: (dx, dw)."""
    x, dy = x.double(), dy.double()
    partner, same, other = turn
    # the transpose of the rotation: value i is reached from i (same) and from its partner
    g = dy * same + (dy * other)[..., partner]
    g = torch.where((partner == torch.arange(x.shape[-1], device=x.device)), dy, g)
    if weight is None:
        return g, None
    norm = torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + eps)
    unit = x / norm
    dw = (g * unit).sum(0)
    h = g * weight.double()
    return (h - unit * (h * unit).sum(-1, keepdim=True) / x.shape[-1]) / norm, dw


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    if c["op"] in ("norm_rope", "norm_rope_grad"):
        turn = _turn_matrix(torch.arange(c["N"], device="cuda"), c["rot"], d, c["interleaved"],
                            "cuda")
        outs, sums = [], []
        for first, heads, w, dy in ((0, Hq, s["wq"], s.get("dq")), (Hq, Hkv, s["wk"], s.get("dk"))):
            out = torch.empty(c["B"], heads, c["N"], d, dtype=torch.float64, device="cuda")
            total = torch.zeros(d, dtype=torch.float64, device="cuda")
            for b in range(c["B"]):
                for h in range(heads):
                    x = s["qkv"][b, :, first + h]
                    if c["op"] == "norm_rope":
                        out[b, h] = _exact_forward(x, w, s["eps"], turn)
                    else:
                        out[b, h], dw = _exact_gradient(x, dy[b, h], w, s["eps"], turn)
                        total = total if dw is None else total + dw
            outs.append(out)
            sums.append(total)
        return outs + sums if c["op"] == "norm_rope_grad" and c["norm"] else outs
    lengths, table, page = _lengths(c), s["table"].tolist(), c["page"]
    if c["op"] == "append":
        q_out, k_cache, v_cache = (s[n].double() for n in ("q_out", "k_cache", "v_cache"))
        row = 0
        for i, n in enumerate(_new_tokens(c)):
            if lengths[i]:
                pos = torch.arange(lengths[i] - n, lengths[i], device="cuda")
                turn = _turn_matrix(pos, c["rot"], d, c["interleaved"], "cuda")
                turn = (turn[0], turn[1][:, None], turn[2][:, None])
                x = s["qkv"][row:row + n]
                q_out[row:row + n] = _exact_forward(x[:, :Hq], s["wq"], s["eps"], turn)
                k = _exact_forward(x[:, Hq:Hq + Hkv], s["wk"], s["eps"], turn)
                at = torch.tensor([table[i][p // page] for p in pos.tolist()], device="cuda")
                k_cache[at, :, pos % page] = k
                v_cache[at, :, pos % page] = x[:, Hq + Hkv:].double()
            row += n
        return [q_out, k_cache, v_cache]
    out = torch.zeros(c["S"], Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((c["S"], Hq), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(lengths):
        if n == 0:
            continue
        first = max(0, n - c["window"]) if c["window"] else 0
        used = torch.tensor(table[i][:-(-n // page)], device="cuda", dtype=torch.int64)
        k = s["k_cache"][used].permute(1, 0, 2, 3).flatten(1, 2)[:, first:n].double()
        v = s["v_cache"][used].permute(1, 0, 2, 3).flatten(1, 2)[:, first:n].double()
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
