"""The counters in the workspace of mita_paged_attn_q4: as in mita_paged_attn's (test_gpu_paged_counters.py),
255 words under the number of the call that counted last, each for the two or four shares of a CTA."""
import pytest
import torch

import q4_util as Q

pytestmark = pytest.mark.gpu

STEP, BITS = 256, 16


def M():
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    return mita


def arguments(lengths, Hq, Hkv, d, dt, page=16):
    """Random codes: a cache of any bytes but scales that are NaN, infinite or beyond 8."""
    g = torch.Generator().manual_seed(1)
    pages = [-(-n // page) for n in lengths]
    num = sum(pages) + 1
    caches = []
    for _ in range(2):
        codes = torch.randint(0, 256, (num, Hkv, page * d // 2), generator=g)
        scales = torch.randint(90, 144, (num, Hkv, page * d // 32), generator=g)
        caches.append(torch.cat((codes, scales), -1).to(torch.uint8).cuda())
    table = torch.full((len(lengths), max(pages + [1])), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = torch.arange(at, at + n)
        at += n
    q = torch.randn(len(lengths), Hq, d, generator=g).to(dt)
    return q.cuda(), *caches, table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda()


def counters(mita):
    ws = mita._paged_workspaces[0, torch.cuda.current_stream().cuda_stream]
    return ws[:mita._PAGED_COUNTERS].view(torch.int64)


# one share's segments, segments of two shares and of many, cut at every place
SHAPES = [((1,), 1, 1, 64), ((0, 0), 4, 2, 32), ((3000,), 8, 2, 128), ((200000, 5, 0, 7000), 4, 2, 64),
          ((90000,), 16, 1, 128), (tuple(200 + i * 29 % 900 for i in range(400)), 4, 1, 32),
          (tuple(384 * (1 + i % 3) for i in range(211)), 4, 1, 128),
          # as many segments as make four shares to a CTA, of one part, of two to six, of a hundred
          (tuple(1 + i * 37 % 400 for i in range(470)), 4, 1, 128), ((20000,) + (1,) * 480, 8, 1, 128),
          (tuple(200 * (1 + i % 7) for i in range(310)), 14, 2, 64), ((24000, 3, 24000) + (180,) * 454, 2, 1, 32),
          ((33000,) + (1,) * 500, 3, 1, 64)]          # a table too wide for four


def scale_of_values():
    return torch.tensor([Q.scale_of_byte(b) for b in range(256)], dtype=torch.float64)


def reference(args, page=16):
    """fp64 on the GPU, sequence by sequence."""
    q, kc, vc, table, n = args
    S, Hq, d = q.shape
    Hkv = kc.shape[1]
    scales = scale_of_values().cuda()
    row = torch.arange(page, device="cuda")
    turn = {128: row >> 1 & 3, 64: row >> 2 & 1, 32: row * 0}[d]
    order = turn[:, None] ^ torch.arange(d // 32, device="cuda")

    def values(cache, used):
        b = cache[used].long()
        code = b[..., :page * d // 2].view(len(used), Hkv, page, d // 32, 16)
        code = torch.gather(code, 3, order[None, None, :, :, None].expand_as(code))
        x = torch.stack((code & 15, code >> 4), -1).flatten(-2).double() - 8
        x = x * scales[b[..., page * d // 2:]].view(x.shape[:-1] + (1,))
        return x.flatten(-2).permute(1, 0, 2, 3).flatten(1, 2)

    out = torch.zeros(S, Hq, d, dtype=torch.float64, device="cuda")
    for s in range(S):
        length = int(n[s])
        if length:
            used = table[s, :-(-length // page)].long()
            k, v = (values(c, used)[:, :length] for c in (kc, vc))
            z = torch.einsum("hgd,hjd->hgj", q[s].double().view(Hkv, -1, d), k) / d ** 0.5
            out[s] = torch.einsum("hgj,hjd->hgd", torch.softmax(z, -1), v).reshape(Hq, d)
    return out


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES[2:], ids=lambda s: f"{len(s[0])}x{max(s[0])}-{s[1:]}")
def test_segments_cut_between_two_shares_and_many(shape, dt):
    mita = M()
    args = arguments(*shape, dt)
    out = mita.mita_paged_attn_q4(*args)
    assert mita.get_last_device_error() == 0
    want = reference(args)
    # relative to each row's size: bf16's and fp16's half steps of the terms, or fp32's sums
    tol = 2.0 ** -8 + 2.0 ** -10 if dt == torch.bfloat16 else 2.0 ** -15
    off = (out.double() - want).norm(dim=-1) / want.norm(dim=-1).clamp(min=1e-30)
    assert float(off.max()) <= tol


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_calls_are_numbered_whatever_their_shapes(dt):
    mita = M()
    calls = [arguments(*shape, dt) for shape in SHAPES]
    want = []
    for args in calls:
        mita.workspace_release()
        want.append(mita.mita_paged_attn_q4(*args))
    mita.workspace_release()
    for args in calls:                                                # the workspace as large as it gets
        mita.mita_paged_attn_q4(*args)
    for _ in range(3):
        for args, out in zip(calls, want):
            before = counters(mita).clone()
            assert torch.equal(mita.mita_paged_attn_q4(*args), out)
            after = counters(mita)
            assert int(after[-1]) - int(before[-1]) == STEP and int(after[-1]) % STEP == 0
            number = int(after[-1]) // STEP - 1
            assert int((after[:-1] >> BITS).max()) <= number
            # two shares: two parts of 1, and 4 for each of at most 510; four: up to four parts of 1, 8 and 64,
            # and 512 for each of at most 127
            assert int((after[:-1] & ((1 << BITS) - 1)).max()) <= 512 * 127 + 4 * (64 + 8 + 1)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES[2:5] + SHAPES[6:9], ids=lambda s: f"{len(s[0])}x{max(s[0])}-{s[1:]}")
def test_what_a_disturbed_call_leaves_does_not_count(shape, dt):
    """Counts as a call would leave them whose lengths changed while it ran, under that call's number: the
    next call, and a call after a very great many, is right."""
    mita = M()
    args = arguments(*shape, dt)
    want = mita.mita_paged_attn_q4(*args, return_lse=True)
    for number in (None, 1 << 20, (1 << 40) + 5):
        for left in (1, 2, 7, 4080):
            w = counters(mita)
            if number is not None:
                w[-1] = (number + left) * STEP
            last = int(w[-1]) // STEP - 1
            w[:-1] = (last << BITS) + left
            for _ in range(2):
                got = mita.mita_paged_attn_q4(*args, return_lse=True)
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    mita.workspace_release()
