"""Host-side checks of the query/key preparation and the paged cache: every bad argument the host can see is refused before
anything is launched, so these run without a GPU (the addresses are never read)."""

import ctypes

import pytest

P16 = 1 << 20


@pytest.fixture(scope="module")
def fa():
    from _lib import load_fa
    return load_fa()


def _check(fn, good, cases, status):
    for bad in cases:
        assert set(bad) <= set(good), bad
        assert fn(**dict(good, **bad)) == status, bad


def ints(*v):
    a = (ctypes.c_int * len(v))(*v)
    return ctypes.addressof(a), a


def test_rope_table_refusals(fa):
    good = dict(cos_t=P16, sin_t=P16, table_rows=8, rot_dim=64, base=1e4, stream=None)
    _check(fa.fa_rope_table, good, [dict(cos_t=0), dict(sin_t=P16 + 4), dict(table_rows=0), dict(rot_dim=8), dict(rot_dim=72),
                                    dict(rot_dim=144), dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")),
                                    dict(base=-3.0)], fa.FA_ERR_INVALID_ARG)


QK = dict(q=P16, k=P16, q_out=P16, k_out=P16, wq=P16, wk=P16, cos_t=P16, sin_t=P16, positions=P16, T=4, Hq=2, Hk=1, d=64,
          q_stride=128, k_stride=64, q_out_stride=128, k_out_stride=64, rot_dim=64, table_rows=16, axes=1, sections=None,
          interleaved=0, eps=1e-6, dtype=0, stream=None)

ROPE_BAD = [dict(cos_t=0), dict(sin_t=P16 + 8), dict(positions=P16 + 2), dict(rot_dim=0), dict(rot_dim=24), dict(rot_dim=80),
            dict(table_rows=0), dict(axes=0), dict(axes=5), dict(axes=2), dict(interleaved=2)]


def test_qk_norm_rope_refusals(fa):
    keep = [ints(16, 12), ints(14, 18), ints(0, 32), ints(-4, 36), ints(8, 8, 16)]
    _check(fa.fa_qk_norm_rope, QK, [
        dict(q=0), dict(k=P16 + 8), dict(q_out=0), dict(k_out=P16 + 2), dict(wq=None), dict(wk=None), dict(wq=P16 + 8),
        dict(T=0), dict(Hq=0), dict(Hk=0), dict(d=96), dict(dtype=2), dict(q_stride=120), dict(q_stride=132), dict(k_stride=0),
        dict(q_out_stride=64), dict(k_out_stride=65), dict(eps=0.0), dict(eps=float("nan")), dict(positions=None)]
        + ROPE_BAD + [dict(axes=2, sections=p) for p, _ in keep[:4]], fa.FA_ERR_INVALID_ARG)


def test_qk_norm_rope_backward_refusals(fa):
    ws = fa.fa_qk_norm_rope_bwd_workspace_bytes(64)
    assert ws > 0 and fa.fa_qk_norm_rope_bwd_workspace_bytes(96) == 0
    good = dict(dq_out=P16, dk_out=P16, q=P16, k=P16, wq=P16, wk=P16, cos_t=P16, sin_t=P16, positions=P16, dq=P16, dk=P16,
                dwq=P16, dwk=P16, T=4, Hq=2, Hk=1, d=64, dq_out_stride=128, dk_out_stride=64, q_stride=128, k_stride=64,
                dq_stride=128, dk_stride=64, rot_dim=64, table_rows=16, axes=1, sections=None, interleaved=0, eps=1e-6, dtype=0,
                workspace=P16, workspace_bytes=ws, stream=None)
    _check(fa.fa_qk_norm_rope_bwd, good, [
        dict(dq_out=0), dict(dk_out=P16 + 8), dict(q=0), dict(k=P16 + 4), dict(wq=None), dict(wk=None), dict(dq=P16 + 8),
        dict(dk=0), dict(dwq=0), dict(dwk=P16 + 1), dict(T=0), dict(Hq=-1), dict(d=32), dict(dtype=-1), dict(dq_out_stride=127),
        dict(k_stride=63), dict(dk_stride=60), dict(eps=-1.0), dict(workspace=0), dict(workspace=P16 + 64),
        dict(workspace_bytes=ws - 1), dict(positions=None)] + ROPE_BAD, fa.FA_ERR_INVALID_ARG)


APPEND = dict(q=P16, k=P16, v=P16, q_out=P16, k_cache=P16, v_cache=P16, wq=P16, wk=P16, cos_t=P16, sin_t=P16, positions=None,
              page_table=P16, seqlens_k=P16, cu_seqlens=None, B=2, T=4, Hq=2, Hk=1, d=64, q_stride=128, k_stride=64, v_stride=64,
              q_out_stride=128, page_size=16, num_pages=3, max_pages=2, rot_dim=64, table_rows=16, axes=1, sections=None,
              interleaved=0, eps=1e-6, dtype=0, cache_format=0, stream=None)
CACHE_BAD = [dict(k_cache=0), dict(v_cache=P16 + 8), dict(page_table=0), dict(page_table=P16 + 2), dict(B=0), dict(Hk=0),
             dict(d=80), dict(page_size=0), dict(num_pages=0), dict(max_pages=0), dict(dtype=3), dict(cache_format=2),
             dict(cache_format=-1)]
CACHE_UNSUPPORTED = [dict(page_size=8), dict(page_size=24), dict(page_size=1 << 21), dict(max_pages=1 << 27), dict(Hk=70000)]


def test_cache_append_refusals(fa):
    _check(fa.fa_cache_append, APPEND, CACHE_BAD + [
        dict(k=0), dict(v=P16 + 2), dict(T=0), dict(T=5), dict(q=None), dict(q_out=None), dict(Hq=0), dict(seqlens_k=0),
        dict(seqlens_k=P16 + 1), dict(cu_seqlens=P16 + 2), dict(wq=None), dict(wk=None), dict(wk=P16 + 8), dict(k_stride=56),
        dict(v_stride=66), dict(q_stride=64), dict(q_out_stride=1), dict(eps=0.0), dict(cos_t=None), dict(sin_t=None),
        dict(cos_t=None, sin_t=None, positions=P16), dict(rot_dim=40), dict(table_rows=0), dict(axes=2), dict(interleaved=-1)],
        fa.FA_ERR_INVALID_ARG)
    _check(fa.fa_cache_append, APPEND, CACHE_UNSUPPORTED, fa.FA_ERR_UNSUPPORTED)


def test_cache_gather_refusals(fa):
    good = dict(k_cache=P16, v_cache=P16, k=P16, v=P16, page_table=P16, cu_seqlens_k=P16, starts=None, B=2, total_keys=8, Hk=1,
                d=64, page_size=16, num_pages=3, max_pages=2, dtype=0, cache_format=1, stream=None)
    _check(fa.fa_cache_gather, good, CACHE_BAD + [dict(k=0), dict(v=P16 + 8), dict(total_keys=0), dict(cu_seqlens_k=P16 + 2),
                                                  dict(cu_seqlens_k=None, total_keys=7), dict(starts=P16 + 3)],
           fa.FA_ERR_INVALID_ARG)
    _check(fa.fa_cache_gather, good, CACHE_UNSUPPORTED, fa.FA_ERR_UNSUPPORTED)


def test_decode_paged_refusals(fa):
    ws = fa.fa_decode_paged_workspace_bytes(2, 1, 4, 2, 40960, 64)
    good = dict(q=P16, k_cache=P16, v_cache=P16, o=P16, lse=P16, page_table=P16, seqlens_k=P16, B=2, Nq=1, H=4, Hk=2, Nk=40960, d=64,
                scale=0.125, page_size=16, num_pages=3, max_pages=2, dtype=0, cache_format=0, workspace=P16, workspace_bytes=ws,
                stream=None)
    _check(fa.fa_decode_paged, good, CACHE_BAD + [
        dict(q=0), dict(o=P16 + 8), dict(lse=P16 + 2), dict(seqlens_k=0), dict(Nq=0), dict(H=0), dict(H=3), dict(Nk=0),
        dict(scale=0.0), dict(scale=float("inf")), dict(workspace=0), dict(workspace=P16 + 128),
        dict(workspace_bytes=ws - 1)], fa.FA_ERR_INVALID_ARG)
    _check(fa.fa_decode_paged, good, CACHE_UNSUPPORTED[:4] + [dict(B=70000), dict(Nk=(1 << 30) + 1), dict(Nq=1 << 21), dict(H=1 << 20, Hk=1, Nq=2)],
           fa.FA_ERR_UNSUPPORTED)


def test_sizes(fa):
    assert fa.fa_cache_bytes(3, 16, 2, 128, fa.FA_CACHE_16BIT) == 3 * 16 * 2 * 256
    assert fa.fa_cache_bytes(3, 16, 2, 128, fa.FA_CACHE_INT4) == 3 * 16 * 2 * 80
    assert fa.fa_cache_bytes(1 << 20, 64, 128, 128, fa.FA_CACHE_16BIT) == (1 << 20) * 64 * 128 * 256  # past 32 bits
    assert fa.fa_cache_bytes(3, 16, 2, 96, 0) == 0 and fa.fa_cache_bytes(0, 16, 2, 64, 0) == 0
    assert fa.fa_cache_bytes(3, 16, 2, 64, 2) == 0
    assert fa.fa_decode_paged_workspace_bytes(1, 1, 4, 3, 64, 64) == 0
    assert fa.fa_decode_paged_workspace_bytes(1, 1, 4, 2, 0, 64) == 0
    # two parts of each block at most, whatever the length; small calls need none
    for nk in (1, 100, 8192):
        assert fa.fa_decode_paged_workspace_bytes(1, 1, 8, 8, nk, 128) == 0
    for nk in (8193, 10000, 131072, 1 << 30):
        assert 0 < fa.fa_decode_paged_workspace_bytes(1, 1, 8, 8, nk, 128) < 1 << 25
    assert fa.fa_decode_paged_workspace_bytes(64, 1, 8, 8, 2049, 128) > 0


def test_wrapper_refusals(fa):
    """The torch wrappers refuse CPU tensors, wrong shapes and wrong dtypes before they reach the library."""
    import torch
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cos = torch.zeros(4, 32)
    pos = torch.zeros(4, dtype=torch.int32)
    cache = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(4, 2, dtype=torch.int32)
    lens = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: fa.attention_qk_norm_rope(q, q, cos, cos, pos),
                 lambda: fa.attention_qk_norm_rope_backward(q, q, cos, cos, pos),
                 lambda: fa.attention_cache_append(q, q, cache, cache, table, lens),
                 lambda: fa.attention_cache_gather(cache, cache, table, None, 4),
                 lambda: fa.attention_decode_paged(q, cache, cache, table, lens)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(AttributeError):
        fa.attention_no_such_thing


def test_missing_binding_fails_loudly(fa, tmp_path):
    """No fallback: without the binding the wrappers cannot be had, while the library itself still loads."""
    import os
    import shutil
    import subprocess
    import sys
    pkg = os.path.dirname(fa.__file__)
    dst = tmp_path / os.path.basename(pkg)
    os.makedirs(dst)
    for f in ("__init__.py", "paged.py", "libfa_b200.so"):
        shutil.copy(os.path.join(pkg, f), dst / f)
    code = (f"import {dst.name} as fa\nprint(fa.fa_version())\n"
            "try:\n    fa.attention_cache_append\nexcept ImportError as e:\n    print('refused:', e)\n")
    out = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-500:]
    assert "sm_100a" in out.stdout and "refused: the torch binding is missing" in out.stdout


@pytest.mark.parametrize("torch_found", [True, False])
def test_star_import_without_the_binding(fa, tmp_path, torch_found):
    """The raw ABI needs neither the binding nor torch, by `import *` either."""
    import os
    import shutil
    import subprocess
    import sys
    pkg = os.path.dirname(fa.__file__)
    dst = tmp_path / os.path.basename(pkg)
    os.makedirs(dst)
    for f in ("__init__.py", "paged.py", "libfa_b200.so"):
        shutil.copy(os.path.join(pkg, f), dst / f)
    code = (("" if torch_found else "import sys\nsys.modules['torch'] = None\n")
            + f"from {dst.name} import *\nprint(fa_version(), attention_forward.__name__, 'attention_decode_paged' in globals())\n")
    out = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-500:]
    assert "sm_100a" in out.stdout and out.stdout.split()[-2:] == ["attention_forward", "False"]


def test_star_import_brings_the_wrappers(fa):
    names = {}
    exec("from exact_io_aware_90_b200 import *", names)
    for n in ("attention_rope_table", "attention_qk_norm_rope", "attention_qk_norm_rope_backward", "attention_cache_append",
              "attention_cache_gather", "attention_decode_paged", "attention_forward", "fa_fwd"):
        assert names[n] is getattr(fa, n) and n in dir(fa)


def test_decode_workspace_of_sizes_that_are_refused(fa):
    """No size for what fa_decode_paged refuses; with 2^31 - 2 rows the row tiles passed 32 bits and gave 5.7 TB."""
    good = dict(q=P16, k_cache=P16, v_cache=P16, o=P16, lse=P16, page_table=P16, seqlens_k=P16, num_pages=3, max_pages=2, scale=0.125,
                page_size=16, dtype=0, cache_format=0, workspace=P16, workspace_bytes=1 << 50, stream=None)
    for B, Nq, H, Hk in ((1, 3906, 549791, 1), (65536, 1, 1, 1), (1, 1 << 20, 1 << 10, 1), (1, 1, 1 << 17, 1 << 17), (1, 1 << 20, 16, 16)):
        assert fa.fa_decode_paged_workspace_bytes(B, Nq, H, Hk, 100000, 64) == 0
        assert fa.fa_decode_paged(**dict(good, B=B, Nq=Nq, H=H, Hk=Hk, Nk=100000, d=64)) == fa.FA_ERR_UNSUPPORTED
    assert fa.fa_decode_paged_workspace_bytes(65535, 1, 16, 16, 100000, 64) > 0
