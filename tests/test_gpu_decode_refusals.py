"""What the Python entry points refuse of GPU tensors, before anything is launched."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def M():
    from sparse_top_landmark_gb300 import build, mita
    build.build()
    return mita


def test_norm_rope_refusals():
    mita = M()
    q = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16, device="cuda")
    k = q[:, :2]
    f = torch.zeros(32, dtype=torch.float64, device="cuda")
    w = torch.ones(64, device="cuda")
    mita.mita_qk_norm_rope(q, k, f, w, w)
    n0 = mita.kernel_launches()
    for bad, err in (
            (lambda: mita.mita_qk_norm_rope(q.half(), k.half()), TypeError),
            (lambda: mita.mita_qk_norm_rope(q, k.float()), TypeError),
            (lambda: mita.mita_qk_norm_rope(q, k.cpu()), ValueError),
            (lambda: mita.mita_qk_norm_rope(q, k[:1]), ValueError),
            (lambda: mita.mita_qk_norm_rope(q[..., ::2], k[..., ::2]), ValueError),
            (lambda: mita.mita_qk_norm_rope(q, k, f.float()), TypeError),
            (lambda: mita.mita_qk_norm_rope(q, k, f.view(2, 16)), ValueError),
            (lambda: mita.mita_qk_norm_rope(q, k, torch.cat((f, f))), mita.MitaError),   # rot > d
            (lambda: mita.mita_qk_norm_rope(q, k, f[:3]), mita.MitaError),               # rot = 6
            (lambda: mita.mita_qk_norm_rope(q, k, f, w.bfloat16()), TypeError),
            (lambda: mita.mita_qk_norm_rope(q, k, f, w[:32]), ValueError),
            (lambda: mita.mita_qk_norm_rope(q, k, f, positions=torch.zeros(8, device="cuda")), TypeError),
            (lambda: mita.mita_qk_norm_rope(q, k, f, positions=torch.zeros(
                3, 8, dtype=torch.int32, device="cuda")), ValueError),
            (lambda: mita.mita_qk_norm_rope(q, k, q_out=q[:, :1].expand(2, 4, 8, 64)), ValueError),
            (lambda: mita.mita_qk_norm_rope(torch.zeros(2, 4, 8, 48, device="cuda")), mita.MitaError),
            # rows off 16-byte boundaries: by their start, and by a stride
            (lambda: mita.mita_qk_norm_rope(torch.zeros(66, device="cuda")[2:].view(1, 1, 1, 64)),
             mita.MitaError),
            (lambda: mita.mita_qk_norm_rope(torch.zeros(1, 1, 4, 66, device="cuda")[..., :64]),
             mita.MitaError),
            (lambda: mita.mita_qk_norm_rope_backward(q, k, q, None), ValueError),
            (lambda: mita.mita_qk_norm_rope_backward(q, k, q, k.float()), TypeError),
            (lambda: mita.mita_qk_norm_rope_backward(q, k, q[:, :1], k), ValueError)):
        with pytest.raises(err):
            bad()
    assert mita.kernel_launches() == n0


def test_paged_refusals():
    mita = M()
    t = torch.zeros(3, 2, 64, device="cuda")
    q = torch.zeros(3, 4, 64, device="cuda")
    c = torch.zeros(5, 2, 16, 64, device="cuda")
    table = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    n = torch.ones(3, dtype=torch.int32, device="cuda")
    mita.mita_cache_append(t, t, c, c.clone(), table, n, q=q)
    mita.mita_paged_attn(q, c, c, table, n)
    n0 = mita.kernel_launches()
    for bad, err in (
            (lambda: mita.mita_cache_append(t, t[:2], c, c, table, n), ValueError),
            (lambda: mita.mita_cache_append(t[:2], t[:2], c, c, table, n), mita.MitaError),
            (lambda: mita.mita_cache_append(t, t, c.bfloat16(), c, table, n), TypeError),
            (lambda: mita.mita_cache_append(t, t, c, c[:4], table, n), ValueError),
            (lambda: mita.mita_cache_append(t, t, c.transpose(1, 2), c.transpose(1, 2), table, n), ValueError),
            (lambda: mita.mita_cache_append(t, t, c, c, table.long(), n), TypeError),
            (lambda: mita.mita_cache_append(t, t, c, c, table, n[:2]), ValueError),
            (lambda: mita.mita_cache_append(t, t, c, c, table, n, seq_start=n), ValueError),
            (lambda: mita.mita_cache_append(t, t, c, c, table, n, q=q[:2]), ValueError),
            (lambda: mita.mita_cache_append(t, t, c[:, :, :3].contiguous(), c[:, :, :3].contiguous(),
                                            table, n), mita.MitaError),
            (lambda: mita.mita_paged_attn(q[:, :3], c, c, table, n), mita.MitaError),
            (lambda: mita.mita_paged_attn(q[:2], c, c, table, n), ValueError),
            (lambda: mita.mita_paged_attn(q, c.cpu(), c, table, n), ValueError),
            (lambda: mita.mita_paged_attn(q, c, c, table[:, ::2], n), ValueError),
            (lambda: mita.mita_paged_attn(q, c, c, table, n, softcap=-1.0), mita.MitaError),
            (lambda: mita.mita_paged_attn(q, c, c, table, n, window=-1), mita.MitaError),
            (lambda: mita.mita_paged_attn(q, c, c, table, n, scale=float("nan")), mita.MitaError),
            (lambda: mita.mita_paged_attn(q, c, c, table, n, alibi_slopes=n.float()), ValueError),
            (lambda: mita.mita_paged_attn(q, c, c, table, n, out=q.bfloat16()), TypeError),
            (lambda: mita.mita_paged_attn(q, c, c, table, n, out=q[:, :1].expand(3, 4, 64)), ValueError)):
        with pytest.raises(err):
            bad()
    assert mita.kernel_launches() == n0
