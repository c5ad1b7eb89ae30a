"""A serving engine's steps as they would be run: pages from mita_cache_plan, keys and queries rotated by
positions of several axes (an image in each prompt), keys and values into the cache of 4-bit codes, attention
of each new token over it; against plain fp64."""
import pytest
import torch

import decode_util as R
import q4_util as Q
from test_gpu_axes import axis_of, forward, grid

pytestmark = pytest.mark.gpu


def M():
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    return mita


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_prompts_then_steps(dt):
    mita = M()
    S, Hq, Hkv, d, page, pool = 3, 4, 2, 64, 16, 16
    prompts, steps = [33, 0, 52], 18
    g = torch.Generator().manual_seed(1)
    most = max(prompts) + steps
    x = torch.randn(S, most, Hq + 2 * Hkv, d, generator=g).to(dt)
    w = 1 + 0.2 * torch.randn(2, d, generator=g)
    freq, axis = R.inv_freq(d), axis_of("sections", d // 2, 3)
    # a prompt: 3 x 3 x 3 patches behind three tokens of text, then text, whose place on every axis goes on
    pos = torch.arange(most).expand(3, most).clone().to(torch.int32)
    pos[:, :30] = grid(3, 3, 3, lead=3)

    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    lengths, table = i32([0] * S), torch.full((S, 6), -1, dtype=torch.int32, device="cuda")
    free, count = torch.arange(pool, dtype=torch.int32, device="cuda"), i32([pool])
    kc, vc = (torch.full(mita.cache_q4_shape(pool, Hkv, page, d), 255, dtype=torch.uint8, device="cuda")
              for _ in range(2))
    how = dict(inv_freq=freq.cuda(), freq_axis=axis.cuda(), q_weight=w[0].cuda(), k_weight=w[1].cuda())
    pos_dev = pos.cuda()

    def run(rows, new, places):
        """A step over packed rows [T, heads, d]; returns rotated q and the keys' rounded values."""
        start, at, slots, granted = mita.mita_cache_plan(i32(new), lengths, table, free, count,
                                                         rows.shape[0], page)
        q, k, v = rows.split((Hq, Hkv, Hkv), 1)
        # packed rows are one batch; their places on the axes go by the plan's positions
        qr, kr = mita.mita_qk_norm_rope_axes(q.transpose(0, 1)[None], k.transpose(0, 1)[None],
                                             positions=places[:, at.long()], **how)
        mita.mita_cache_append_q4(kr[0].transpose(0, 1), v, kc, vc, slots)
        return qr[0].transpose(0, 1), kr[0].transpose(0, 1), granted

    packed = torch.cat([x[s, :n] for s, n in enumerate(prompts)] + [x[0, :2]]).cuda()   # two rows nobody's
    _, kr, granted = run(packed, prompts, pos_dev)
    assert granted.tolist() == prompts and lengths.tolist() == prompts
    keys = [[] for _ in range(S)]
    first = 0
    for s, n in enumerate(prompts):
        keys[s] += list(kr[first:first + n].cpu())
        first += n
    tokens = list(prompts)
    for step in range(steps):
        new = [1] * S
        if step == 7:
            new[0] = -1                     # done: its pages go back, and are handed out again
        if 7 < step < 10:
            new[0] = 0
        if step == 10:
            new[0], tokens[0], keys[0] = 1, 0, []
        rows = torch.stack([x[s, tokens[s]] for s in range(S) if new[s] == 1]).cuda()
        qr, kr, granted = run(rows, new, pos_dev)
        live = [s for s in range(S) if new[s] == 1]
        assert granted.tolist() == [max(n, 0) for n in new]
        for i, s in enumerate(live):
            keys[s].append(kr[i].cpu())
            tokens[s] += 1
        n = [tokens[s] if new[s] == 1 else 0 for s in range(S)]
        assert lengths.tolist() == n
        q_all = torch.zeros(S, Hq, d, dtype=dt, device="cuda")
        q_all[live] = qr
        out = mita.mita_paged_attn_q4(q_all, kc, vc, table, lengths)
        if step in (0, 6, 7, 9, 10, steps - 1):
            assert mita.get_last_device_error() == 0
            # the rotation, of this step's rows
            for i, s in enumerate(live):
                raw = rows[i, :Hq].cpu()[None, :, None]
                at = pos[:, tokens[s] - 1][:, None, None]
                want, bound = forward(raw, w[0], at, axis, freq, 1e-6, False)
                R.assert_close(qr[i][None, :, None], want, bound, "q")
            # the attention, over what the cache holds of the keys that went in
            k = [torch.stack(keys[s], 1) if n[s] else torch.zeros(Hkv, 0, d) for s in range(S)]
            v = [x[s, :n[s], Hq + Hkv:].transpose(0, 1) for s in range(S)]
            cache = Q.Cache4(n, Hkv, page, d, k=k, v=v)
            want, bound, _, _ = Q.paged_attn(q_all.cpu(), cache, n)
            R.assert_close(out, want, bound, f"step {step}")


def test_prompts_into_the_bf16_cache():
    """The plan in front of mita_cache_append and mita_paged_attn, whose tables and row starts it gives."""
    mita = M()
    S, Hq, Hkv, d, page, pool = 2, 2, 1, 32, 8, 16
    prompts = [19, 30]
    g = torch.Generator().manual_seed(2)
    x = torch.randn(sum(prompts) + 3, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    lengths, table = i32([0] * S), torch.full((S, 5), -1, dtype=torch.int32, device="cuda")
    free, count = torch.arange(pool, dtype=torch.int32, device="cuda"), i32([pool])
    kc, vc = (torch.zeros(pool, Hkv, page, d, dtype=x.dtype, device="cuda") for _ in range(2))
    start, pos, slots, granted = mita.mita_cache_plan(i32(prompts), lengths, table, free, count,
                                                      x.shape[0], page)
    q, k, v = x.split((Hq, Hkv, Hkv), 1)
    freq = R.inv_freq(d).cuda()
    mita.mita_cache_append(k, v, kc, vc, table, lengths, seq_start=start, inv_freq=freq)
    kr = mita.mita_qk_norm_rope(k.transpose(0, 1)[None], None, freq, positions=pos)[0][0].transpose(0, 1)
    assert mita.get_last_device_error() == 0 and granted.tolist() == prompts
    for t in range(sum(prompts)):
        at, row = divmod(int(slots[t]), page)
        assert torch.equal(kc[at, :, row], kr[t]) and torch.equal(vc[at, :, row], v[t])
    assert slots[sum(prompts):].tolist() == [-1] * 3
