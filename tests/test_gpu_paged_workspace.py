"""Workspaces that a caller passes: contiguous memory only.  An expanded tensor or a slice with gaps counts more bytes, or others,
than lie behind its address."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    from _lib import load_fa
    m = load_fa()
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu-marked tests")
    return m


def _bad(n):
    return (torch.empty(1, dtype=torch.uint8, device="cuda").expand(n), torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2],
            torch.empty(2, n, dtype=torch.uint8, device="cuda").t(), torch.empty(n, dtype=torch.uint8))


def test_decode_workspace(fa):
    B, H, d, page, most = 2, 4, 64, 64, 40960
    kc, vc = (torch.zeros(4, H, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(B, H, d, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(B, 4, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), 70, dtype=torch.int32, device="cuda")
    need = fa.fa_decode_paged_workspace_bytes(B, 1, H, H, most, d)
    assert need > 0
    for ws in _bad(need):
        with pytest.raises(ValueError, match="workspace"):
            fa.attention_decode_paged(q, kc, vc, table, lens, max_seqlen_k=most, workspace=ws)
    ws = torch.full((need + 64,), 7, dtype=torch.uint8, device="cuda")
    o, lse = fa.attention_decode_paged(q, kc, vc, table, lens, max_seqlen_k=most, workspace=ws[:need])
    want = fa.attention_decode_paged(q, kc, vc, table, lens, max_seqlen_k=most)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and bool((ws[need:] == 7).all())
    with pytest.raises(fa.FAError):
        fa.attention_decode_paged(q, kc, vc, table, lens, max_seqlen_k=most, workspace=ws[:need - 1])
    assert fa.fa_check_device_status(torch.cuda.current_stream().cuda_stream) == fa.FA_OK


def test_gradient_workspace(fa):
    T, H, d = 40, 2, 64
    g = torch.Generator().manual_seed(3)
    q, k, dq, dk = (torch.randn(T, H, d, generator=g).bfloat16().cuda() for _ in range(4))
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    cos, sin = fa.attention_rope_table(T, d)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    kw = dict(q=q, k=k, wq=w, wk=w)
    need = fa.fa_qk_norm_rope_bwd_workspace_bytes(d)
    for ws in _bad(need):
        with pytest.raises(ValueError, match="workspace"):
            fa.attention_qk_norm_rope_backward(dq, dk, cos, sin, pos, workspace=ws, **kw)
    ws = torch.full((need + 64,), 7, dtype=torch.uint8, device="cuda")
    got = fa.attention_qk_norm_rope_backward(dq, dk, cos, sin, pos, workspace=ws[:need], **kw)
    want = fa.attention_qk_norm_rope_backward(dq, dk, cos, sin, pos, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool((ws[need:] == 7).all())
    with pytest.raises(fa.FAError):
        fa.attention_qk_norm_rope_backward(dq, dk, cos, sin, pos, workspace=ws[:need - 1], **kw)
    assert fa.fa_check_device_status(torch.cuda.current_stream().cuda_stream) == fa.FA_OK
