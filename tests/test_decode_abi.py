"""Refusals of the q / k preparation and paged-cache entry points: every call below fails its
validation on the host (nothing is launched, no GPU is needed), in C and in Python."""
import ctypes

import pytest
import torch

from sparse_top_landmark_gb300 import build as B
from sparse_top_landmark_gb300 import mita

OK = ctypes.c_void_p(1 << 20)          # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return mita.load()


def msg(lib):
    return lib.mita_last_error_message().decode()


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


ROPE = dict(q=OK, k=OK, qw=OK, kw=OK, pos=None, ps=0, freq=OK, B=1, Hq=4, Hkv=2, N=8, d=64, rot=64,
            il=0, eps=1e-6, qs=None, ks=None, qos=None, kos=None, qo=OK, ko=OK)
BAD_ROPE = [
    (dict(d=48), 2, "head dim"), (dict(rot=4), 1, "rot"), (dict(rot=72), 1, "rot"),
    (dict(rot=-8), 1, "rot"), (dict(freq=None), 1, "inv_freq"), (dict(eps=-1.0), 1, "eps"),
    (dict(eps=float("nan")), 1, "eps"), (dict(q=None), 1, "q is NULL"),
    (dict(q=ODD), 1, "aligned"), (dict(ko=ODD), 1, "k_out"), (dict(qw=ODD), 1, "q_weight"),
    (dict(B=-1), 1, "B, N"), (dict(Hq=0), 1, "Hq"), (dict(Hkv=-1), 1, "Hkv"),
    (dict(N=1 << 30, B=4), 2, "2^31"), (dict(qs=i64(4096, 64, 60)), 1, "q: stride"),
    (dict(kos=i64(4096, -64, 64)), 1, "k_out: stride"), (dict(pos=ctypes.c_void_p((1 << 20) + 1)), 1, "positions"), (dict(pos=OK, ps=-1), 1, "positions"),
]


@pytest.mark.parametrize("suffix", ["", "_f32"])
@pytest.mark.parametrize("change,code,text", BAD_ROPE)
def test_norm_rope_refusals(lib, suffix, change, code, text):
    a = {**ROPE, **change}
    if suffix and "qs" in change:
        a["qs"] = i64(4096, 64, 62)
    assert getattr(lib, "mita_qk_norm_rope" + suffix)(*a.values(), None) == code, msg(lib)
    assert text in msg(lib)


def test_norm_rope_backward_refusals(lib):
    need = lib.mita_qk_norm_rope_backward_workspace_bytes(64)
    assert need > 0 and lib.mita_qk_norm_rope_backward_workspace_bytes(48) == 0
    base = dict(q=OK, k=OK, dqo=OK, dko=OK, qw=OK, kw=OK, pos=None, ps=0, freq=OK, B=1, Hq=4,
                Hkv=2, N=8, d=64, rot=64, il=0, eps=1e-6, qs=None, ks=None, dqos=None, dkos=None,
                dqs=None, dks=None, ws=OK, wb=need, dq=OK, dk=OK, dwq=OK, dwk=OK)
    for change, text in ((dict(wb=need - 1), "workspace"), (dict(ws=None), "workspace"),
                         (dict(dwq=None), "dq_weight"), (dict(kw=None), "dk_weight given"),
                         (dict(q=None), "q is NULL"), (dict(dqo=None), "dq_out"),
                         (dict(dk=ODD), "dk is not"), (dict(rot=12), "rot"),
                         (dict(dqs=i64(4096, 64, 2)), "dq: stride"),
                         (dict(pos=OK, ps=-8), "positions")):
        a = {**base, **change}
        for f in (lib.mita_qk_norm_rope_backward, lib.mita_qk_norm_rope_backward_f32):
            assert f(*a.values(), None) == 1, (change, msg(lib))
            assert text in msg(lib)


APPEND = dict(q=OK, k=OK, v=OK, qw=None, kw=None, freq=OK, table=OK, n=OK, start=OK, T=10, S=3, Hq=4,
              Hkv=2, d=64, pages=8, page=16, width=4, rot=64, il=0, eps=1e-6, qs=None, ks=None,
              vs=None, qos=None, qo=OK, kc=OK, vc=OK)
BAD_APPEND = [
    (dict(page=24), 2, "page_size"), (dict(page=0), 2, "page_size"), (dict(d=80), 2, "head dim"),
    (dict(page=1 << 21), 2, "page_size"), (dict(width=1 << 27), 2, "table_width"),
    (dict(S=-1), 1, "S, num_pages"), (dict(Hkv=0), 1, "Hkv"), (dict(T=-1), 1, "tokens"),
    (dict(start=None), 1, "without seq_start"), (dict(rot=20), 1, "rot"),
    (dict(freq=None), 1, "inv_freq"), (dict(kc=None), 1, "k_cache"), (dict(vc=ODD), 1, "v_cache"),
    (dict(table=None), 1, "page_table"), (dict(n=None), 1, "lengths"), (dict(v=None), 1, "v is"),
    (dict(ks=i64(8, 4)), 1, "k: stride"), (dict(qo=None), 1, "q_out"), (dict(qw=ODD), 1, "q_weight"),
    (dict(T=1 << 29), 2, "2^31"),
]


@pytest.mark.parametrize("suffix", ["", "_f32"])
@pytest.mark.parametrize("change,code,text", BAD_APPEND)
def test_append_refusals(lib, suffix, change, code, text):
    a = {**APPEND, **change}
    if suffix and "ks" in change:
        a["ks"] = i64(8, 2)
    assert getattr(lib, "mita_cache_append" + suffix)(*a.values(), None) == code, msg(lib)
    assert text in msg(lib)


ATTN = dict(q=OK, kc=OK, vc=OK, table=OK, n=OK, slopes=None, S=3, Hq=4, Hkv=2, d=64, pages=8, page=16,
            width=4, qs=None, scale=0.125, cap=0.0, window=0, ws=OK, wb=1 << 30, out=OK, lse=None)
BAD_ATTN = [
    (dict(Hq=5), 1, "multiple"), (dict(Hq=0), 1, "multiple"), (dict(page=3), 2, "page_size"),
    (dict(d=256), 2, "head dim"), (dict(scale=float("inf")), 1, "scale"),
    (dict(cap=-1.0), 1, "softcap"), (dict(cap=float("nan")), 1, "softcap"),
    (dict(cap=float("inf")), 1, "softcap"), (dict(window=-1), 1, "window"),
    (dict(out=None), 1, "out"), (dict(kc=None), 1, "k_cache"), (dict(vc=ODD), 1, "v_cache"),
    (dict(n=None), 1, "lengths"), (dict(table=None), 1, "page_table"),
    (dict(qs=i64(256, 4)), 1, "q: stride"), (dict(S=1 << 30, Hq=4), 2, "S*Hq"),
    (dict(width=-1), 1, "table_width"),
]


@pytest.mark.parametrize("change,code,text", BAD_ATTN)
def test_paged_attn_refusals(lib, change, code, text):
    a = {**ATTN, **change}
    assert lib.mita_paged_attn(*a.values(), None) == code, msg(lib)
    assert text in msg(lib)


def test_paged_attn_workspace_query(lib):
    f = lib.mita_paged_attn_workspace_bytes
    assert f(4, 8, 2, 64, 16, 100, 0) > 0
    assert f(4, 8, 3, 64, 16, 100, 0) == 0 and f(4, 8, 2, 64, 17, 100, 0) == 0
    assert f(4, 8, 2, 48, 16, 100, 1) == 0


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
