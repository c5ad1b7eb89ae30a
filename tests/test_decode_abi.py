"""Refusals of the q / k preparation and paged-cache entry points: every call below fails its
validation on the host (nothing is launched, no GPU is needed), in C and in Python; and the
binding's packed arguments against the header's structs."""
import re

import pytest
import torch

from sparse_top_landmark_gb300 import build as B
from sparse_top_landmark_gb300 import mita

OK = 1 << 20          # aligned, never dereferenced
ODD = OK + 2


@pytest.fixture(scope="module")
def lib():
    B.build()
    return mita.load()


def msg(lib):
    return lib.mita_last_error_message().decode()


def call(lib, name, layout, base, change):
    values = []
    for v in {**base, **change}.values():
        values += v if isinstance(v, (tuple, list)) else [v]
    return getattr(lib, name)(layout.pack(*values), None)


ROPE = dict(q=OK, k=OK, qw=OK, kw=OK, pos=0, freq=OK, qo=OK, ko=OK, qs=(2048, 512, 64),
            ks=(1024, 512, 64), qos=(2048, 512, 64), kos=(1024, 512, 64), ps=0, B=1, Hq=4, Hkv=2, N=8,
            d=64, rot=64, il=0, eps=1e-6)
BAD_ROPE = [
    (dict(d=48), 2, "head dim"), (dict(rot=4), 1, "rot"), (dict(rot=72), 1, "rot"),
    (dict(rot=-8), 1, "rot"), (dict(freq=0), 1, "inv_freq"), (dict(freq=OK + 4), 1, "inv_freq"),
    (dict(eps=-1.0), 1, "eps"), (dict(eps=float("nan")), 1, "eps"), (dict(q=0), 1, "q is NULL"),
    (dict(q=ODD), 1, "aligned"), (dict(ko=ODD), 1, "k_out"), (dict(qw=ODD), 1, "q_weight"),
    (dict(B=-1), 1, "B, N"), (dict(Hq=0), 1, "Hq"), (dict(Hkv=-1), 1, "Hkv"),
    (dict(N=1 << 30, B=4), 2, "2^31"), (dict(qs=(0, 512, 62)), 1, "q: stride"),
    (dict(kos=(0, -64, 64)), 1, "k_out: stride"), (dict(pos=OK + 1), 1, "positions"),
    (dict(pos=OK, ps=-1), 1, "positions"),
]


@pytest.mark.parametrize("suffix", ["", "_f32"])
@pytest.mark.parametrize("change,code,text", BAD_ROPE)
def test_norm_rope_refusals(lib, suffix, change, code, text):
    assert call(lib, "mita_qk_norm_rope" + suffix, mita._NORM_ROPE, ROPE, change) == code, msg(lib)
    assert text in msg(lib)


BACKWARD = dict(q=OK, k=OK, dqo=OK, dko=OK, qw=OK, kw=OK, pos=0, freq=OK, dq=OK, dk=OK, dwq=OK, dwk=OK,
                ws=OK, wb=1 << 30, qs=(2048, 512, 64), ks=(1024, 512, 64), dqos=(2048, 512, 64),
                dkos=(1024, 512, 64), dqs=(2048, 512, 64), dks=(1024, 512, 64), ps=0, B=1, Hq=4,
                Hkv=2, N=8, d=64, rot=64, il=0, eps=1e-6)


@pytest.mark.parametrize("suffix", ["", "_f32"])
@pytest.mark.parametrize("change,text", [
    (dict(wb=100), "workspace"), (dict(ws=0), "workspace"), (dict(dwq=0), "dq_weight"),
    (dict(kw=0), "dk_weight given"), (dict(q=0), "q is NULL"), (dict(dqo=0), "dq_out"),
    (dict(dk=ODD), "dk is not"), (dict(rot=12), "rot"), (dict(dqs=(4096, 64, 2)), "dq: stride"),
    (dict(pos=OK, ps=-8), "positions")])
def test_norm_rope_backward_refusals(lib, suffix, change, text):
    assert lib.mita_qk_norm_rope_backward_workspace_bytes(64) > 100
    assert lib.mita_qk_norm_rope_backward_workspace_bytes(48) == 0
    name = "mita_qk_norm_rope_backward" + suffix
    assert call(lib, name, mita._NORM_ROPE_BACKWARD, BACKWARD, change) == 1, msg(lib)
    assert text in msg(lib)


APPEND = dict(q=OK, k=OK, v=OK, qw=0, kw=0, freq=OK, table=OK, n=OK, start=OK, qo=OK, kc=OK, vc=OK,
              qs=(256, 64), ks=(128, 64), vs=(128, 64), qos=(256, 64), T=10, S=3, Hq=4, Hkv=2, d=64,
              pages=8, page=16, width=4, rot=64, il=0, eps=1e-6)
BAD_APPEND = [
    (dict(page=24), 2, "page_size"), (dict(page=0), 2, "page_size"), (dict(d=80), 2, "head dim"),
    (dict(page=1 << 21), 2, "page_size"), (dict(width=1 << 27), 2, "table_width"),
    (dict(S=-1), 1, "S, num_pages"), (dict(Hkv=0), 1, "Hkv"), (dict(T=-1), 1, "tokens"),
    (dict(start=0), 1, "without seq_start"), (dict(rot=20), 1, "rot"),
    (dict(freq=0), 1, "inv_freq"), (dict(kc=0), 1, "k_cache"), (dict(vc=ODD), 1, "v_cache"),
    (dict(table=0), 1, "page_table"), (dict(n=0), 1, "lengths"), (dict(v=0), 1, "v is"),
    (dict(ks=(130, 64)), 1, "k: stride"), (dict(qo=0), 1, "q_out"), (dict(qw=ODD), 1, "q_weight"),
    (dict(T=1 << 29), 2, "2^31"), (dict(Hkv=1 << 30), 2, "2^31"),
]


@pytest.mark.parametrize("suffix", ["", "_f32"])
@pytest.mark.parametrize("change,code,text", BAD_APPEND)
def test_append_refusals(lib, suffix, change, code, text):
    got = call(lib, "mita_cache_append" + suffix, mita._CACHE_APPEND, APPEND, change)
    assert got == code, msg(lib)
    assert text in msg(lib)


ATTN = dict(q=OK, kc=OK, vc=OK, table=OK, n=OK, slopes=0, ws=OK, out=OK, lse=0, wb=1 << 30,
            qs=(256, 64), S=3, Hq=4, Hkv=2, d=64, pages=8, page=16, width=4, window=0, scale=0.125,
            cap=0.0)
BAD_ATTN = [
    (dict(Hq=5), 1, "multiple"), (dict(Hq=0), 1, "multiple"), (dict(page=3), 2, "page_size"),
    (dict(d=256), 2, "head dim"), (dict(scale=float("inf")), 1, "scale"),
    (dict(cap=-1.0), 1, "softcap"), (dict(cap=float("nan")), 1, "softcap"),
    (dict(cap=float("inf")), 1, "softcap"), (dict(window=-1), 1, "window"),
    (dict(out=0), 1, "out"), (dict(kc=0), 1, "k_cache"), (dict(vc=ODD), 1, "v_cache"),
    (dict(n=0), 1, "lengths"), (dict(table=0), 1, "page_table"), (dict(lse=OK + 2), 1, "lse"),
    (dict(qs=(258, 64)), 1, "q: stride"), (dict(S=1 << 30, Hq=4), 2, "S*Hq"),
    (dict(width=-1), 1, "table_width"), (dict(wb=64), 1, "workspace"), (dict(ws=0), 1, "workspace"),
    (dict(slopes=OK + 1), 1, "alibi_slopes"),
]


@pytest.mark.parametrize("suffix", ["", "_f32"])
@pytest.mark.parametrize("change,code,text", BAD_ATTN)
def test_paged_attn_refusals(lib, suffix, change, code, text):
    got = call(lib, "mita_paged_attn" + suffix, mita._PAGED_ATTN, ATTN, change)
    assert got == code, msg(lib)
    assert text in msg(lib)


def test_paged_attn_workspace_query(lib):
    f = lib.mita_paged_attn_workspace_bytes
    assert f(4, 8, 2, 64, 16, 100, 0) > 0
    assert f(4, 8, 3, 64, 16, 100, 0) == 0 and f(4, 8, 2, 64, 17, 100, 0) == 0
    assert f(4, 8, 2, 48, 16, 100, 1) == 0


def test_counter_bytes_are_the_headers():
    with open(mita.HEADER_PATH) as f:
        want = re.search(r"MITA_PAGED_COUNTERS = (\d+)", f.read()).group(1)
    assert mita._PAGED_COUNTERS == int(want)


def test_null_params(lib):
    for name in ("mita_qk_norm_rope", "mita_qk_norm_rope_backward", "mita_cache_append",
                 "mita_paged_attn"):
        for suffix in ("", "_f32"):
            assert getattr(lib, name + suffix)(None, None) == 1
            assert "params" in msg(lib)


@pytest.mark.parametrize("name,layout", [
    ("mita_qk_norm_rope", mita._NORM_ROPE), ("mita_qk_norm_rope_backward", mita._NORM_ROPE_BACKWARD),
    ("mita_cache_append", mita._CACHE_APPEND), ("mita_paged_attn", mita._PAGED_ATTN)])
def test_packed_layout_is_the_headers(name, layout):
    """The binding's format string against the header's struct, field by field."""
    with open(mita.HEADER_PATH) as f:
        body = re.search(r"typedef struct %s_params \{(.*?)\}" % name, f.read(), re.S).group(1)
    want = ""
    for line in body.replace("\n", " ").split(";"):
        m = re.match(r"\s*(?:const )?(void|float|double|int32_t|int64_t|uint64_t)(.*)", line)
        if not m:
            continue
        for field in m.group(2).split(","):
            n = re.search(r"\[(\d+)\]", field)
            code = "P" if "*" in field else {"float": "f", "int32_t": "i", "int64_t": "q",
                                            "uint64_t": "Q"}[m.group(1)]
            want += code * (int(n.group(1)) if n else 1)
    got = re.sub(r"(\d+)([a-zA-Z])", lambda m: m.group(2) * int(m.group(1)), layout.format)
    assert got.rstrip("x") == want


def test_python_refuses_host_tensors():
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        mita.mita_qk_norm_rope(q, q)
    with pytest.raises(ValueError, match="CUDA"):
        mita.mita_qk_norm_rope_backward(q, q, q, q)
    t = torch.zeros(1, 2, 64)
    c = torch.zeros(2, 2, 16, 64)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        mita.mita_cache_append(t, t, c, c, n[None], n)
    with pytest.raises(ValueError, match="CUDA"):
        mita.mita_paged_attn(t, c, c, n[None], n)


@pytest.mark.parametrize("suffix", ["", "_f32"])
def test_sizes_at_the_ends_of_32_bits(lib, suffix):
    """A table that a tile behind its last token would lead past 2^31 - 1, and heads whose values
    have no 32-bit count."""
    end = dict(width=(1 << 27) - 1)               # 2^31 - 16 tokens
    attn, append = "mita_paged_attn" + suffix, "mita_cache_append" + suffix
    assert call(lib, attn, mita._PAGED_ATTN, ATTN, end) == 2, msg(lib)
    assert "table_width" in msg(lib)
    assert call(lib, append, mita._CACHE_APPEND, APPEND, end) == 2, msg(lib)
    assert "table_width" in msg(lib)
    assert call(lib, attn, mita._PAGED_ATTN, ATTN, dict(S=1, Hq=1 << 25)) == 2, msg(lib)
    assert "Hq*d" in msg(lib)
    f = lib.mita_paged_attn_workspace_bytes
    most = (1 << 27) - (1 << 12)
    assert f(1, 4, 2, 64, 16, most, suffix != "") > 0 and f(1, 4, 2, 64, 16, most + 1, suffix != "") == 0
