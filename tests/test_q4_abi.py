"""Refusals of the calls with positions of several axes, of the page plan and of the 4-bit cache: each
fails its validation on the host (nothing is launched, no GPU is needed), in C and in Python; and the
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


AXES = dict(q=OK, k=OK, qw=OK, kw=OK, pos=OK, axis=OK, freq=OK, qo=OK, ko=OK, qs=(2048, 512, 64),
            ks=(1024, 512, 64), qos=(2048, 512, 64), kos=(1024, 512, 64), ps=0, pa=8, B=1, Hq=4, Hkv=2,
            N=8, d=64, rot=64, il=0, A=2, eps=1e-6)


@pytest.mark.parametrize("suffix", ["", "_f32"])
@pytest.mark.parametrize("change,code,text", [
    (dict(A=0), 1, "axes"), (dict(A=-1), 1, "axes"), (dict(pos=0), 1, "positions"),
    (dict(axis=0), 1, "freq_axis"), (dict(axis=ODD), 1, "freq_axis"), (dict(pos=ODD), 1, "positions"),
    (dict(pa=-1), 1, "axis_stride"), (dict(ps=-1), 1, "positions"), (dict(freq=0), 1, "inv_freq"),
    (dict(d=48), 2, "head dim"), (dict(rot=72), 1, "rot"), (dict(q=0), 1, "q is NULL"),
    (dict(N=1 << 30, B=4), 2, "2^31"), (dict(eps=-1.0), 1, "eps"), (dict(qs=(0, 512, 62)), 1, "q: stride")])
def test_axes_refusals(lib, suffix, change, code, text):
    got = call(lib, "mita_qk_norm_rope_axes" + suffix, mita._NORM_ROPE_AXES, AXES, change)
    assert got == code, msg(lib)
    assert text in msg(lib)


AXES_BACKWARD = dict(q=OK, k=OK, dqo=OK, dko=OK, qw=OK, kw=OK, pos=OK, axis=OK, freq=OK, dq=OK, dk=OK,
                     dwq=OK, dwk=OK, ws=OK, wb=1 << 30, qs=(2048, 512, 64), ks=(1024, 512, 64),
                     dqos=(2048, 512, 64), dkos=(1024, 512, 64), dqs=(2048, 512, 64),
                     dks=(1024, 512, 64), ps=0, pa=8, B=1, Hq=4, Hkv=2, N=8, d=64, rot=64, il=0, A=3,
                     eps=1e-6)


@pytest.mark.parametrize("suffix", ["", "_f32"])
@pytest.mark.parametrize("change,text", [
    (dict(A=0), "axes"), (dict(pos=0), "positions"), (dict(axis=0), "freq_axis"), (dict(wb=100), "workspace"),
    (dict(ws=0), "workspace"), (dict(dwq=0), "dq_weight"), (dict(kw=0), "dk_weight given"),
    (dict(pa=-4), "axis_stride"), (dict(dqo=0), "dq_out"), (dict(rot=12), "rot")])
def test_axes_backward_refusals(lib, suffix, change, text):
    name = "mita_qk_norm_rope_axes_backward" + suffix
    assert call(lib, name, mita._NORM_ROPE_AXES_BACKWARD, AXES_BACKWARD, change) == 1, msg(lib)
    assert text in msg(lib)


PLAN = dict(new=OK, n=OK, after=OK, table=OK, free=OK, count=OK, count2=OK, start=OK, pos=OK, slots=OK,
            granted=OK, S=4, T=10, pages=8, page=16, width=4)


@pytest.mark.parametrize("change,code,text", [
    (dict(S=-1), 1, "S, num_pages"), (dict(T=-1), 1, "tokens"), (dict(pages=-1), 1, "num_pages"),
    (dict(width=-1), 1, "table_width"), (dict(page=24), 2, "page_size"), (dict(page=0), 2, "page_size"),
    (dict(width=1 << 27), 2, "table_width"), (dict(S=(1 << 14) + 1), 2, "sequences"),
    (dict(T=(1 << 30) + 1), 2, "tokens"), (dict(T=(1 << 31) - 1), 2, "tokens"),
    (dict(new=0), 1, "new_tokens"), (dict(n=ODD), 1, "lengths"), (dict(after=0), 1, "new_lengths"),
    (dict(table=0), 1, "page_table"), (dict(free=0), 1, "free_pages"), (dict(count=0), 1, "free_count"),
    (dict(count2=ODD), 1, "new_free_count"), (dict(start=0), 1, "seq_start"),
    (dict(pos=0), 1, "positions"), (dict(slots=OK + 4), 1, "slots"), (dict(granted=0), 1, "granted")])
def test_plan_refusals(lib, change, code, text):
    assert call(lib, "mita_cache_plan", mita._CACHE_PLAN, PLAN, change) == code, msg(lib)
    assert text in msg(lib)


APPEND = dict(k=OK, v=OK, slots=OK, kc=OK, vc=OK, ko=OK, vo=OK, ks=(128, 64), vs=(128, 64), kos=(128, 64),
              vos=(128, 64), T=10, Hkv=2, d=64, pages=8, page=16)


@pytest.mark.parametrize("suffix", ["", "_f32"])
@pytest.mark.parametrize("change,code,text", [
    (dict(d=16), 2, "4-bit"), (dict(d=80), 2, "head dim"), (dict(page=8), 2, "at least 16"),
    (dict(page=48), 2, "page_size"), (dict(page=1 << 21), 2, "page_size"), (dict(T=-1), 1, "tokens"),
    (dict(Hkv=0), 1, "Hkv"), (dict(Hkv=1 << 30), 2, "2^31"), (dict(T=1 << 30), 2, "2^31"),
    (dict(k=0), 1, "k is"), (dict(v=ODD), 1, "v is"), (dict(ko=ODD), 1, "k_out"),
    (dict(vos=(-128, 64)), 1, "v_out: stride"), (dict(ks=(130, 66)), 1, "k: stride"),
    (dict(kc=0), 1, "k_cache"), (dict(vc=ODD), 1, "v_cache"), (dict(slots=0), 1, "slots"),
    (dict(slots=OK + 4), 1, "slots"), (dict(pages=-1), 1, "num_pages")])
def test_append_refusals(lib, suffix, change, code, text):
    got = call(lib, "mita_cache_append_q4" + suffix, mita._CACHE_APPEND_Q4, APPEND, change)
    assert got == code, msg(lib)
    assert text in msg(lib)


ATTN = dict(q=OK, kc=OK, vc=OK, table=OK, n=OK, slopes=0, ws=OK, out=OK, lse=0, wb=1 << 30,
            qs=(256, 64), S=3, Hq=4, Hkv=2, d=64, pages=8, page=16, width=4, window=0, scale=0.125,
            cap=0.0)


@pytest.mark.parametrize("suffix", ["", "_f32"])
@pytest.mark.parametrize("change,code,text", [
    (dict(d=16), 2, "4-bit"), (dict(d=256), 2, "head dim"), (dict(page=8), 2, "at least 16"),
    (dict(page=3), 2, "page_size"), (dict(Hq=5), 1, "multiple"), (dict(scale=float("inf")), 1, "scale"),
    (dict(cap=-1.0), 1, "softcap"), (dict(window=-1), 1, "window"), (dict(out=0), 1, "out"),
    (dict(kc=0), 1, "k_cache"), (dict(vc=ODD), 1, "v_cache"), (dict(n=0), 1, "lengths"),
    (dict(table=0), 1, "page_table"), (dict(lse=OK + 2), 1, "lse"), (dict(qs=(258, 64)), 1, "q: stride"),
    (dict(S=1 << 30, Hq=4), 2, "S*Hq"), (dict(wb=64), 1, "workspace"), (dict(ws=0), 1, "workspace"),
    (dict(width=(1 << 27) - 1), 2, "table_width")])
def test_paged_attn_refusals(lib, suffix, change, code, text):
    got = call(lib, "mita_paged_attn_q4" + suffix, mita._PAGED_ATTN, ATTN, change)
    assert got == code, msg(lib)
    assert text in msg(lib)


def test_workspace_query(lib):
    f = lib.mita_paged_attn_q4_workspace_bytes
    assert f(4, 8, 2, 64, 16, 100, 0) > 0 and f(4, 8, 2, 128, 16, 100, 1) > 0
    assert f(4, 8, 3, 64, 16, 100, 0) == 0 and f(4, 8, 2, 64, 8, 100, 0) == 0
    assert f(4, 8, 2, 16, 16, 100, 0) == 0


@pytest.mark.parametrize("name", ["mita_qk_norm_rope_axes", "mita_qk_norm_rope_axes_backward",
                                  "mita_cache_append_q4", "mita_paged_attn_q4"])
def test_null_params(lib, name):
    for suffix in ("", "_f32"):
        assert getattr(lib, name + suffix)(None, None) == 1
        assert "params" in msg(lib)
    assert lib.mita_cache_plan(None, None) == 1


@pytest.mark.parametrize("name,layout", [
    ("mita_qk_norm_rope_axes", mita._NORM_ROPE_AXES),
    ("mita_qk_norm_rope_axes_backward", mita._NORM_ROPE_AXES_BACKWARD),
    ("mita_cache_plan", mita._CACHE_PLAN), ("mita_cache_append_q4", mita._CACHE_APPEND_Q4)])
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
    i = torch.zeros(2, 4, dtype=torch.int32)
    f = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        mita.mita_qk_norm_rope_axes(q, q, f, i[0], i)
    with pytest.raises(ValueError, match="positions"):
        mita.mita_qk_norm_rope_axes(q, q, f, i[0], None)
    with pytest.raises(ValueError, match="freq_axis"):
        mita.mita_qk_norm_rope_axes_backward(q, q, q, q, f, None, i)
    t = torch.zeros(1, 2, 64)
    c = torch.zeros(mita.cache_q4_shape(2, 2, 16, 64), dtype=torch.uint8)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        mita.mita_cache_append_q4(t, t, c, c, n.long())
    with pytest.raises(ValueError, match="CUDA"):
        mita.mita_paged_attn_q4(t, c, c, n[None], n)
    with pytest.raises(ValueError, match="CUDA"):
        mita.mita_cache_plan(n, n, n[None], n, n, 1, 16)


def test_cache_shape():
    assert mita.cache_q4_shape(7, 2, 16, 128) == (7, 2, 16 * 68)
    assert mita.cache_q4_shape(7, 2, 64, 32) == (7, 2, 64 * 17)
