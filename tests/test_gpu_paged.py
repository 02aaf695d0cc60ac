"""GPU parity of the paged key/value cache (append, gather) and the decode over it, in 16 and 4 bits, against the fp64 oracle.

Tolerances, derived before the first run (u = finfo(dtype).eps / 2, half a step of the output):
* rotated rows as in test_gpu_rope: u·|y| + 2^-17·(|a cos| + |b sin|); values and rows without norm and rotation are copied:
  equal bits.  4-bit rows of given 16-bit rows: equal bytes (every operation of the rule is correctly rounded on both sides).
  Read back, a 4-bit row is rounded once: 2^-8 relative in bf16, whose step is 2^-7 at 1 (finfo.eps), so half of it is 2^-8.
* decode, 16 bits: a score's error is at most ds = 2^-18·scale·Σ_c |q_c k_c| (d <= 128 fp32 additions) + 2^-22·|s|, and a
  probability's relative error 2·max ds + 2^-16 (two 16-bit parts: 2^-18; ex2, sums: under 2^-18 each), so
  |o − ref| <= Σ_j p_j |v_j|·(2·max ds + 2^-16) + u·|o| (+ 2^-25 in fp16), |lse − ref| <= max ds + 2^-20·(1 + |lse|).
* decode, 4 bits: the magnitudes that enter a score are those of n·scale and min apart, Σ_c |q_c|(n·scale + |min|); P times the
  value's scale is one fp16 number: 2^-11 relative on the n·scale part, and numbers under 2^-14 of a range whose top is at least
  2^6 are rounded to 2^-25: N·15·2^-31 of the largest p_j·scale_j.
"""

import math

import numpy as np
import pytest
import torch

import oracle
from _gpu import f64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def fa():
    from _lib import load_fa
    m = load_fa()
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu-marked tests")
    return m


def _status(fa):
    return fa.fa_check_device_status(torch.cuda.current_stream().cuda_stream)


def _table(lens, page, g, extra=2):
    need = [-(-n // page) for n in lens]
    total = sum(need) + extra
    perm = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, total


def _pack(x, value):
    """uint8 cache [pages, hk, page, 5d/8] of 16-bit rows."""
    n, sc, mn = oracle.four_bit_rows(f64(x))
    pages, hk, page, d = x.shape
    return torch.from_numpy(oracle.four_bit_pack(n, sc, mn, value)).reshape(pages, hk, page, d * 5 // 8)


def _cache(lens, hk, d, page, dtype, bits, seed, spread=1.0):
    """(table, k_cache, v_cache) on the CPU; rows that no sequence owns hold NaN (16 bits) or bytes of NaN scales (4 bits)."""
    g = torch.Generator().manual_seed(seed)
    table, total = _table(lens, page, g)
    out = []
    for value in (False, True):
        x = torch.randn(total, hk, page, d, generator=g)
        x = (x * torch.exp(spread * 0.5 * torch.randn(total, hk, page, 1, generator=g)) if value else x).to(DT[dtype])
        owned = torch.zeros(total, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(n):
                owned[table[b, j // page], j % page] = True
        if bits == 16:
            x = torch.where(owned[:, None, :, None], x, torch.full_like(x, float("nan")))
        else:
            x = _pack(x, value).reshape(total, hk, -1)
            pairs = x[..., page * d // 2:].reshape(total, hk, page, -1)
            x[..., page * d // 2:] = torch.where(owned[:, None, :, None], pairs, torch.full_like(pairs, 255)).reshape(total, hk, -1)
            x = x.reshape(total, hk, page, d * 5 // 8)
        out.append(x)
    return table, out[0], out[1]


def _check_decode(fa, lens, nq, H, hk, d, page, dtype, bits, seed=0, scale=None, spread=1.0):
    """With the bound that the table gives (small calls: a cluster of blocks per key head) and with a wide one (the keys dealt
    out over all blocks)."""
    for max_len in (None, 100000):
        _check_decode_bounded(fa, lens, nq, H, hk, d, page, dtype, bits, seed, scale, max_len, spread)


def _check_decode_bounded(fa, lens, nq, H, hk, d, page, dtype, bits, seed, scale, max_len, spread):
    table, kc, vc = _cache(lens, hk, d, page, dtype, bits, seed, spread)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(len(lens), nq, H, d, generator=g).to(DT[dtype])
    scale = scale or 1 / math.sqrt(d)
    o, lse = fa.attention_decode_paged(q.cuda() if nq > 1 else q[:, 0].contiguous().cuda(), kc.cuda(), vc.cuda(), table.cuda(),
                                       torch.tensor(lens, dtype=torch.int32).cuda(), max_seqlen_k=max_len, scale=scale)
    assert _status(fa) == fa.FA_OK
    o, lse = f64(o).reshape(len(lens), nq, H, d), f64(lse).reshape(len(lens), nq, H)
    u = torch.finfo(DT[dtype]).eps / 2
    for b, n in enumerate(lens):
        k, ka, km, _ = oracle.cache_rows(kc, table.numpy(), b, np.arange(n), d, False)
        v, va, vm, vs = oracle.cache_rows(vc, table.numpy(), b, np.arange(n), d, True)
        ref, rl = oracle.decode_paged(f64(q[b]), k, v, scale)
        for i in range(nq):
            m = n - nq + i + 1
            if m <= 0:
                assert np.all(o[b, i] == 0) and np.all(np.isneginf(lse[b, i]))
                continue
            for h in range(H):
                e = h // (H // hk)
                qh = f64(q[b, i, h])
                s = scale * (k[:m, e] @ qh)
                mag = scale * ((np.abs(ka[:m, e]) + np.abs(km[:m, e])) @ np.abs(qh))
                ds = (2.0 ** -18 * mag + 2.0 ** -22 * np.abs(s)).max()
                p = np.exp(s - rl[i, h])
                if bits == 16:
                    bound = (p @ np.abs(v[:m, e])) * (2 * ds + 2.0 ** -16)
                else:
                    bound = ((p @ np.abs(va[:m, e])) * (2.0 ** -11 + 2 * ds + 2.0 ** -16) + (p @ np.abs(vm[:m, e])) * (2 * ds + 2.0 ** -16)
                             + m * 15 * 2.0 ** -31 * (p[:, None] * vs[:m, e]).max())
                bound = bound + u * np.abs(ref[i, h]) * (1 + 2.0 ** -7) + 2.0 ** -25
                fin = np.isfinite(ref[i, h])  # a value that passed fp16's largest makes its feature infinite or NaN
                assert np.array_equal(fin, np.isfinite(o[b, i, h]))
                err, bound = np.abs(o[b, i, h] - ref[i, h])[fin], bound[fin]
                assert np.all(err <= bound), (b, i, h, (err / bound).max())
                assert abs(lse[b, i, h] - rl[i, h]) <= ds + 2.0 ** -20 * (1 + abs(rl[i, h])), (b, i, h)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 63, 64, 65, 129, 700])
def test_decode_lengths(fa, n, dtype, d, bits):
    _check_decode(fa, [n], 1, 2, 1, d, 16, dtype, bits, seed=n)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (8, 1), (9, 1), (12, 4), (40, 2), (32, 1)])
def test_decode_heads_and_pages(fa, heads, page, bits):
    _check_decode(fa, [131, 0, 1, 300, 16], 1, heads[0], heads[1], 64 if heads[0] % 2 else 128, page, "bf16", bits, seed=page + heads[0])


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("nq", [2, 5, 8, 17])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_several_tokens(fa, d, nq, bits):
    """Lengths under the number of tokens leave the first rows without a key."""
    _check_decode(fa, [nq, nq - 1, 1, 0, 16, 33, 200], nq, 4, 2, d, 32, "fp16", bits, seed=nq)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("n", [64, 127, 128, 129, 256, 257, 512, 513, 900, 1024, 1025, 4096, 4097, 8192, 8193])
def test_decode_cluster_borders(fa, n, bits):
    """One block, two, four, all eight of a cluster, blocks without keys, and one key past the largest cluster call."""
    _check_decode(fa, [n], 1, 4, 2, 64, 64, "bf16", bits, seed=n)
    _check_decode(fa, [1, n, 0], 3, 4, 1, 128, 16, "fp16", bits, seed=n + 1)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("seqs,hk,most", [(20, 8, 300), (40, 4, 130), (80, 8, 90)])
def test_decode_many_units(fa, seqs, hk, most, bits):
    """More units than clusters of eight have room for, and than blocks fit the GPU; dealt out, more than there are blocks."""
    lens = np.random.default_rng(seqs).integers(0, most + 1, seqs).tolist()
    _check_decode(fa, lens, 1, hk, hk, 64 if seqs == 40 else 128, 16, "bf16", bits, seed=seqs)


@pytest.mark.parametrize("bits", [16, 4])
def test_decode_many_chunks_and_a_wide_bound(fa, bits):
    _check_decode(fa, [5000], 1, 4, 4, 128, 64, "bf16", bits, seed=3)
    _check_decode(fa, [4097, 3, 0, 777], 2, 8, 2, 64, 64, "fp16", bits, seed=4)
    # the bound far above the lengths, as a captured graph has it
    lens, g = [40, 0, 7], torch.Generator().manual_seed(1)
    table, kc, vc = _cache(lens, 2, 64, 16, "bf16", bits, 5)
    wide = torch.full((3, 4096), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    q = torch.randn(3, 4, 64, generator=g).bfloat16().cuda()
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    a = fa.attention_decode_paged(q, kc.cuda(), vc.cuda(), wide.cuda(), ln)
    b = fa.attention_decode_paged(q, kc.cuda(), vc.cuda(), table.cuda(), ln, max_seqlen_k=70000)  # past the table is no harm
    assert _status(fa) == fa.FA_OK
    assert np.allclose(f64(a[0]), f64(b[0]), atol=2.0 ** -7) and bool((a[0][1] == 0).all()) and bool(torch.isneginf(a[1][1]).all())


@pytest.mark.parametrize("bits", [16, 4])
def test_decode_large_scores_and_unlike_scales(fa, bits):
    _check_decode(fa, [900], 1, 4, 2, 128, 64, "bf16", bits, seed=6, scale=2.0)
    _check_decode(fa, [900], 1, 4, 2, 64, 64, "fp16", bits, seed=7, spread=6.0)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("at", [0, 900, 2999])
def test_decode_one_key_far_above_the_rest(fa, at, dtype, d, bits):
    """One key whose value is 0 scores 18 above all others, which are 2^-26 of it each: the output is theirs alone.  What a
    16-bit P adds to the module's bound: each key is off by 2^-25 beside a largest of at least 2^7, 2^-32 of it."""
    n, page = 3000, 64
    g = torch.Generator().manual_seed(30)
    table, total = _table([n], page, g)
    k = torch.zeros(total, 1, page, d)
    v = torch.rand(total, 1, page, d, generator=g) + 1.0
    k[int(table[0, at // page]), 0, at % page, 0] = 18.0
    v[int(table[0, at // page]), 0, at % page] = 0.0
    k, v = k.to(DT[dtype]), v.to(DT[dtype])
    kc, vc = (k, v) if bits == 16 else (_pack(k, False), _pack(v, True))
    q = torch.zeros(1, 1, d)
    q[..., 0] = 1.0
    kr, ka, km, _ = oracle.cache_rows(kc, table.numpy(), 0, np.arange(n), d, False)
    vr, va, vm, vs = oracle.cache_rows(vc, table.numpy(), 0, np.arange(n), d, True)
    ref, rl = oracle.decode_paged(f64(q), kr, vr, 1.0)
    p = np.exp(kr[:, 0, 0] - rl[0, 0])
    ds = 2.0 ** -18 * 18 + 2.0 ** -22 * 18
    bound = (p @ np.abs(vr[:, 0])) * (2 * ds + 2.0 ** -16) + torch.finfo(DT[dtype]).eps / 2 * np.abs(ref[0, 0]) * (1 + 2.0 ** -7)
    bound = bound + 2.0 ** -25 + 2.0 ** -32 * p.max() * np.abs(vr[:, 0]).sum(0)
    if bits == 4:  # P times the scale is rounded too
        bound = bound + (p @ np.abs(va[:, 0])) * 2.0 ** -11 + n * 15 * 2.0 ** -31 * (p.max() * vs.max())
    assert np.abs(ref).min() > 4 * bound.max() if bits == 16 else True  # the bound tells the output from 0
    for most in (None, 100000):
        o, lse = fa.attention_decode_paged(q.to(DT[dtype]).cuda(), kc.cuda(), vc.cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                                           max_seqlen_k=most, scale=1.0)
        err = np.abs(f64(o)[0, 0] - ref[0, 0])
        assert np.all(err <= bound), (err / bound).max()
        assert abs(f64(lse)[0, 0] - rl[0, 0]) <= ds + 2.0 ** -20 * (1 + abs(rl[0, 0]))
    assert _status(fa) == fa.FA_OK


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_decode_q4_constant_and_tiny_rows(fa, dtype):
    """Groups without spread (scale 0), values near fp16's smallest and queries of unlike sizes."""
    lens, hk, d, page = [70], 1, 64, 16
    g = torch.Generator().manual_seed(8)
    table, total = _table(lens, page, g)
    k = torch.randn(total, hk, page, d, generator=g)
    v = torch.randn(total, hk, page, d, generator=g) * 1e-4
    v[:, :, 3] = 1.5
    k[:, :, 5] = -0.25
    v[:, :, 7] = 0.0
    kc, vc = _pack(k.to(DT[dtype]), False), _pack(v.to(DT[dtype]), True)
    for size in (1.0, 1e-3, 300.0, 0.0):
        q = (size * torch.randn(1, 2, d, generator=g)).to(DT[dtype])
        q[0, 0, ::7] *= 1e-3
        o, lse = fa.attention_decode_paged(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                           scale=0.1)
        kr, ka, km, _ = oracle.cache_rows(kc, table.numpy(), 0, np.arange(70), d, False)
        vr, va, vm, vs = oracle.cache_rows(vc, table.numpy(), 0, np.arange(70), d, True)
        ref, rl = oracle.decode_paged(f64(q), kr, vr, 0.1)
        for h in range(2):
            s = 0.1 * (kr[:, 0] @ f64(q[0, h]))
            mag = 0.1 * ((np.abs(ka[:, 0]) + np.abs(km[:, 0])) @ np.abs(f64(q[0, h])))
            ds = (2.0 ** -18 * mag + 2.0 ** -22 * np.abs(s)).max()
            p = np.exp(s - rl[0, h])
            bound = ((p @ va[:, 0]) * (2.0 ** -11 + 2 * ds + 2.0 ** -16) + (p @ np.abs(vm[:, 0])) * (2 * ds + 2.0 ** -16)
                     + 70 * 15 * 2.0 ** -31 * (p[:, None] * vs[:, 0]).max() + torch.finfo(DT[dtype]).eps / 2 * np.abs(ref[0, h]) * 1.01
                     + 2.0 ** -25)
            assert np.all(np.abs(f64(o)[0, h] - ref[0, h]) <= bound)
            assert abs(f64(lse)[0, h] - rl[0, h]) <= ds + 2.0 ** -20 * (1 + abs(rl[0, h]))
    assert _status(fa) == fa.FA_OK


def test_decode_nan_and_infinity(fa):
    """What is masked never shows, whatever it holds; what is seen does."""
    lens, page, d = [20], 16, 64
    table, kc, vc = _cache(lens, 1, d, page, "bf16", 16, 9)
    q = torch.randn(1, 3, 1, d, generator=torch.Generator().manual_seed(2)).bfloat16()
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    clean = fa.attention_decode_paged(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), ln)
    for bad in (float("nan"), float("inf"), -float("inf")):
        k2, v2 = kc.clone(), vc.clone()
        k2[table[0, 1], :, 3], v2[table[0, 1], :, 3] = bad, bad  # position 19: only the last token sees it
        o, lse = fa.attention_decode_paged(q.cuda(), k2.cuda(), v2.cuda(), table.cuda(), ln)
        assert torch.equal(o[0, :2], clean[0][0, :2]) and torch.equal(lse[0, :2], clean[1][0, :2])
        assert bool(torch.isnan(o[0, 2]).all())
        assert _status(fa) == fa.FA_OK
    q2 = q.clone()
    q2[0, 1] = float("nan")  # a row of NaN stays its own
    o, lse = fa.attention_decode_paged(q2.cuda(), kc.cuda(), vc.cuda(), table.cuda(), ln)
    assert bool(torch.isnan(o[0, 1]).all()) and bool(torch.isnan(lse[0, 1]).all())
    assert torch.equal(o[0, 0], clean[0][0, 0]) and torch.equal(o[0, 2], clean[0][0, 2])
    k3 = kc.clone()
    k3[table[0].long()] = torch.where(torch.isnan(k3[table[0].long()]), k3[table[0].long()], torch.full_like(k3[table[0].long()], -3e38))
    o, lse = fa.attention_decode_paged(torch.ones_like(q).cuda(), k3.cuda(), vc.cuda(), table.cuda(), ln)  # every score −inf
    assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("bits", [16, 4])
def test_decode_bad_lengths_and_pages_are_skipped(fa, bits):
    lens = [40, 50, 33]
    table, kc, vc = (t.cuda() for t in _cache(lens, 2, 64, 16, "bf16", bits, 10))
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    ref = fa.attention_decode_paged(q, kc, vc, table, ln)
    for bad in (-1, table.shape[1] * 16 + 1, 2 ** 31 - 1):
        l2 = ln.clone()
        l2[1] = bad
        out, lse = torch.full_like(q, 5.0), torch.full((3, 4), 5.0, device="cuda")
        fa.attention_decode_paged(q, kc, vc, table, l2, out=out, lse=lse)
        assert _status(fa) == fa.FA_ERR_INVALID_ARG
        assert bool((out[1] == 5).all()) and bool((lse[1] == 5).all())
        assert torch.equal(out[0], ref[0][0]) and torch.equal(out[2], ref[0][2])
    for bad in (-1, kc.shape[0], 2 ** 31 - 1, -2 ** 31):
        t2 = table.clone()
        t2[2, 1] = bad  # its keys are left out
        out, lse = fa.attention_decode_paged(q, kc, vc, t2, ln)
        assert _status(fa) == fa.FA_ERR_INVALID_ARG
        assert torch.equal(out[:2], ref[0][:2]) and bool(torch.isfinite(out[2]).all())
    assert _status(fa) == fa.FA_OK


# ------------------------------------------------------------------------------------------------ append and gather

def _append_inputs(T, hq, hk, d, dtype, seed, rot, rows):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, hq + 2 * hk, d, generator=g).to(DT[dtype])
    cos, sin = (torch.from_numpy(x).float() for x in oracle.rope_table(rows, rot, 10000.0))
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).to(DT[dtype]) for _ in range(2))
    return qkv, cos, sin, wq, wk


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,hq,hk,page,rot,inter", [(64, 4, 2, 16, 64, False), (128, 5, 5, 48, 48, True), (128, 9, 1, 64, 128, False),
                                                    (64, 3, 3, 32, 16, False)])
def test_append(fa, d, hq, hk, page, rot, inter, dtype, bits):
    """Ragged new tokens (none, one, many, over page borders) behind what the pages already hold; nothing else is touched."""
    lens, new = [5, 70, 33, 20, 1], [5, 37, 0, 1, 1]
    T = sum(new) + 3  # three rows behind the last sequence
    qkv, cos, sin, wq, wk = _append_inputs(T, hq, hk, d, dtype, 11, rot, 128)
    q, k, v = qkv.split([hq, hk, hk], 1)
    table, kc, vc = _cache(lens, hk, d, page, dtype, bits, 12)
    cu = np.concatenate([[0], np.cumsum(new)])
    kg, vg = kc.clone().cuda(), vc.clone().cuda()
    dev = qkv.cuda()
    qo = torch.full((T, hq, d), 9.0, dtype=DT[dtype], device="cuda")
    got = fa.attention_cache_append(dev[:, hq:hq + hk], dev[:, hq + hk:], kg, vg, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                    cos=cos.cuda(), sin=sin.cuda(), q=dev[:, :hq], wq=wq.cuda(), wk=wk.cuda(), eps=1e-5,
                                    interleaved=inter, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), q_out=qo)
    assert _status(fa) == fa.FA_OK and got is qo and bool((qo[sum(new):] == 9).all())
    at = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)])
    seq = np.repeat(np.arange(len(lens)), new)
    # the rows as the operator that norms and rotates gives them
    c = dev[:sum(new)]
    pos = torch.tensor(at, dtype=torch.int32).cuda()
    yq, yk = fa.attention_qk_norm_rope(c[:, :hq], c[:, hq:hq + hk], cos.cuda(), sin.cuda(), pos, wq=wq.cuda(), wk=wk.cuda(), eps=1e-5,
                                       interleaved=inter)
    assert torch.equal(qo[:sum(new)], yq)
    ref = oracle.qk_norm_rope(f64(k[:sum(new)]), f64(wk), cos.double().numpy(), sin.double().numpy(), at, 1e-5, inter)
    amp = np.abs(f64(k[:sum(new)])) / np.sqrt((f64(k[:sum(new)]) ** 2).mean(-1, keepdims=True)) * np.abs(f64(wk))
    assert np.all(np.abs(f64(yk) - ref) <= torch.finfo(DT[dtype]).eps / 2 * np.abs(ref) + 2.0 ** -17 * (amp.max(-1, keepdims=True) * 2) + 2.0 ** -25)
    page_of, slot = table[torch.from_numpy(seq), torch.from_numpy(at // page)].long(), torch.from_numpy(at % page)
    for cache, before, rows, value in ((kg, kc, yk.cpu(), False), (vg, vc, v[:sum(new)], True)):
        want = before.clone()
        if bits == 16:
            want[page_of, :, slot] = rows
            assert torch.equal(cache.cpu().view(torch.int16), want.view(torch.int16))
        else:
            n, sc, mn = oracle.four_bit_unpack(want.reshape(want.shape[0], hk, -1).numpy(), page, d, value)
            n2, sc2, mn2 = oracle.four_bit_rows(f64(rows))
            n[page_of.numpy(), :, slot.numpy()], sc[page_of.numpy(), :, slot.numpy()], mn[page_of.numpy(), :, slot.numpy()] = n2, sc2, mn2
            g, gs, gm = oracle.four_bit_unpack(cache.cpu().reshape(want.shape[0], hk, -1).numpy(), page, d, value)
            assert np.array_equal(g, n) and np.array_equal(gs, sc, equal_nan=True) and np.array_equal(gm, mn, equal_nan=True)


@pytest.mark.parametrize("bits", [16, 4])
def test_append_plain_and_by_axes(fa, bits):
    """Without rotation the rows are copied; with axes the rotation's positions are the caller's; equal counts need no offsets."""
    lens, hk, d, page = [18, 40], 2, 64, 16
    qkv, cos, sin, _, wk = _append_inputs(6, 0, hk, d, "bf16", 13, 64, 64)
    k, v = qkv.cuda().split([hk, hk], 1)
    table, kc, vc = _cache(lens, hk, d, page, "bf16", bits, 14)
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    starts = ln - 3
    kg, vg = kc.cuda(), vc.cuda()
    assert fa.attention_cache_append(k, v, kg, vg, table.cuda(), ln) is None
    gk, gv = fa.attention_cache_gather(kg, vg, table.cuda(), None, 6, starts=starts, dtype=torch.bfloat16)
    if bits == 16:
        assert torch.equal(gk, k) and torch.equal(gv, v)
    else:
        for got, x in ((gk, k), (gv, v)):
            n, sc, mn = oracle.four_bit_rows(f64(x))
            val = n * np.repeat(sc, 32, -1) + np.repeat(mn, 32, -1)
            assert np.all(np.abs(f64(got) - val) <= 2.0 ** -8 * np.abs(val) + 2.0 ** -22 * (np.abs(np.repeat(mn, 32, -1)) + 15 * np.repeat(sc, 32, -1)))
    pos = torch.randint(0, 64, (3, 6), generator=torch.Generator().manual_seed(4), dtype=torch.int32).cuda()
    fa.attention_cache_append(k, v, kg, vg, table.cuda(), ln, cos=cos.cuda(), sin=sin.cuda(), positions=pos, wk=wk.cuda(), sections=(8, 12, 12))
    _, yk = fa.attention_qk_norm_rope(k, k, cos.cuda(), sin.cuda(), pos, wq=wk.cuda(), wk=wk.cuda(), sections=(8, 12, 12))
    gk2, gv2 = fa.attention_cache_gather(kg, vg, table.cuda(), None, 6, starts=starts, dtype=torch.bfloat16)
    assert torch.equal(gv2, gv)
    if bits == 16:
        assert torch.equal(gk2, yk)
    else:
        n, sc, mn = oracle.four_bit_rows(f64(yk))
        val = n * np.repeat(sc, 32, -1) + np.repeat(mn, 32, -1)
        assert np.all(np.abs(f64(gk2) - val) <= 2.0 ** -8 * np.abs(val) + 2.0 ** -22 * (np.abs(np.repeat(mn, 32, -1)) + 15 * np.repeat(sc, 32, -1)))
    assert _status(fa) == fa.FA_OK


def test_append_extreme_values(fa):
    """Constant groups, zeros, fp16's and bf16's largest, and a group with an infinity: the scale and minimum stay finite."""
    x = torch.zeros(4, 1, 64)
    x[0, 0, :32] = 65504.0
    x[0, 0, 32:] = -65504.0
    x[1, 0, 0], x[1, 0, 31], x[1, 0, 40] = 3e38, -3e38, float("inf")
    x[2, 0] = torch.linspace(-1e-7, 1e-7, 64)
    x = x.bfloat16().cuda()
    cache = torch.zeros(1, 1, 16, 40, dtype=torch.uint8, device="cuda")
    v = cache.clone()
    fa.attention_cache_append(x, x, cache, v, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([4], dtype=torch.int32, device="cuda"))
    n, sc, mn = oracle.four_bit_unpack(cache.cpu().reshape(1, 1, -1).numpy(), 16, 64, False)
    assert np.isfinite(sc).all() and np.isfinite(mn).all()
    rn, rs, rm = oracle.four_bit_rows(f64(x)[[0, 2, 3]])
    assert np.array_equal(n[0, 0, [0, 2, 3]], rn[:, 0]) and np.array_equal(sc[0, 0, [0, 2, 3]], rs[:, 0]) and np.array_equal(mn[0, 0, [0, 2, 3]], rm[:, 0])
    assert _status(fa) == fa.FA_OK


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_append_q4_rows_are_finite(fa, value):
    """An infinity becomes the largest or least number of its group, a NaN the least; the other groups are as without it."""
    g = torch.Generator().manual_seed(31)
    x = torch.randn(16, 2, 128, generator=g).bfloat16()
    clean = x.clone()
    at = torch.randint(32, (16, 2), generator=g)
    for t in range(16):
        for h in range(2):
            x[t, h, 32 + int(at[t, h])] = value
            # in the oracle's row the place holds the least value of the rest
            clean[t, h, 32 + int(at[t, h])] = torch.cat([clean[t, h, 32:32 + int(at[t, h])], clean[t, h, 33 + int(at[t, h]):64]]).min()
    n, sc, mn = oracle.four_bit_rows(f64(clean))
    caches = [torch.zeros(1, 2, 16, 80, dtype=torch.uint8, device="cuda") for _ in range(2)]
    fa.attention_cache_append(x.cuda(), x.cuda(), *caches, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                              torch.tensor([16], dtype=torch.int32, device="cuda"))
    for c, is_value in zip(caches, (False, True)):
        gn, gs, gm = (y[0].swapaxes(0, 1) for y in oracle.four_bit_unpack(c.cpu().reshape(1, 2, -1).numpy(), 16, 128, is_value))
        assert np.isfinite(gs).all() and np.isfinite(gm).all()
        same = [0, 2, 3] if not math.isnan(value) else [0, 1, 2, 3]
        assert np.array_equal(gs[..., same], sc[..., same]) and np.array_equal(gm[..., same], mn[..., same])
        feat = np.concatenate([np.arange(32 * w, 32 * w + 32) for w in same])
        assert np.array_equal(gn[..., feat], n[..., feat])
        bad = np.take_along_axis(gn, 32 + at.numpy()[..., None], -1)
        assert np.all(bad == (15 if value == math.inf else 0))
    assert _status(fa) == fa.FA_OK


@pytest.mark.parametrize("bits", [16, 4])
def test_append_bad_offsets_are_skipped(fa, bits):
    lens, hk, d, page = [18, 40], 1, 64, 16
    k, v = torch.randn(5, 2, d, generator=torch.Generator().manual_seed(5)).bfloat16().cuda().split(1, 1)
    table, kc, vc = (t.cuda() for t in _cache(lens, hk, d, page, "bf16", bits, 15))
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    cu = torch.tensor([0, 2, 5], dtype=torch.int32).cuda()

    def run(ln=ln, table=table, cu=cu):
        a, b = kc.clone(), vc.clone()
        fa.attention_cache_append(k, v, a, b, table, ln, cu_seqlens=cu)
        return a.view(torch.uint8), b.view(torch.uint8), _status(fa)
    good = run()
    assert good[2] == fa.FA_OK
    same = lambda x: torch.equal(x[0], kc.view(torch.uint8)) and torch.equal(x[1], vc.view(torch.uint8))  # noqa: E731
    t = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    for bad in (dict(ln=t(1, 2)), dict(ln=t(-5, -1)), dict(ln=t(10 ** 9, 2 ** 31 - 1)), dict(table=torch.full_like(table, kc.shape[0])),
                dict(table=torch.full_like(table, -7)), dict(cu=t(0, 9, 9))):
        x = run(**bad)
        assert x[2] == fa.FA_ERR_INVALID_ARG and same(x), bad
    x = run(cu=t(5, 5, 5))  # no sequence owns a row
    assert x[2] == fa.FA_OK and same(x)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("d,hk,page", [(64, 3, 16), (128, 2, 48), (128, 16, 64)])
def test_gather(fa, d, hk, page, bits):
    lens = [0, 50, 16, 1, 0, 131, 0]
    table, kc, vc = _cache(lens, hk, d, page, "fp16", bits, 16)
    starts = [0, 7, 0, 0, 3, 100, 0]
    take = [0, 43, 16, 1, 0, 20, 0]
    cu = torch.tensor(np.concatenate([[2], 2 + np.cumsum(take)]), dtype=torch.int32)  # two rows in front, three behind
    total = int(cu[-1]) + 3
    k, v = (torch.full((total, hk, d), 4.0, dtype=torch.float16, device="cuda") for _ in range(2))
    gk, gv = fa.attention_cache_gather(kc.cuda(), vc.cuda(), table.cuda(), cu.cuda(), total, starts=torch.tensor(starts, dtype=torch.int32).cuda(),
                                       k=k, v=v)
    assert _status(fa) == fa.FA_OK and gk is k and gv is v
    for got, cache, value in ((k, kc, False), (v, vc, True)):
        assert bool((got[:2] == 4).all()) and bool((got[total - 3:] == 4).all())
        for b, (s, n) in enumerate(zip(starts, take)):
            if n:
                val, a, m, _ = oracle.cache_rows(cache, table.numpy(), b, np.arange(s, s + n), d, value)
                x = f64(got[int(cu[b]):int(cu[b + 1])])
                if bits == 16:
                    assert np.array_equal(x, val)
                else:
                    assert np.all(np.abs(x - val) <= 2.0 ** -11 * np.abs(val) + 2.0 ** -23 * (np.abs(a) + np.abs(m)) + 2.0 ** -25)
    for bad in (dict(starts=torch.tensor([0, 7, -1, 0, 3, 2 ** 31 - 1, 0], dtype=torch.int32).cuda()),
                dict(cu=torch.tensor([2, 1, 50, 90, 200, 300, 400, 500], dtype=torch.int32).cuda())):
        k2 = torch.full_like(k, 4.0)
        fa.attention_cache_gather(kc.cuda(), vc.cuda(), table.cuda(), bad.get("cu", cu.cuda()), total, starts=bad.get("starts"), k=k2, v=k2.clone())
        assert _status(fa) == fa.FA_ERR_INVALID_ARG and bool((k2[total - 3:] == 4).all() or "cu" in bad)


def test_gather_finds_sequences_among_many(fa):
    """More sequences than one step of the search looks at, many of them empty."""
    rng = np.random.default_rng(17)
    for B in (31, 32, 33, 1024, 1025, 5000):
        lens = [int(x) for x in rng.integers(0, 3, B)]
        lens[-1] = 2
        cu = np.concatenate([[0], np.cumsum(lens)])
        cache = torch.arange(B * 16, dtype=torch.float32).remainder(2048).reshape(B, 1, 16, 1).expand(B, 1, 16, 64).half().contiguous().cuda()
        table = torch.arange(B, dtype=torch.int32).reshape(B, 1).cuda()
        k, _ = fa.attention_cache_gather(cache, cache, table, torch.tensor(cu, dtype=torch.int32).cuda(), int(cu[-1]))
        want = np.concatenate([np.arange(n) + 16 * b for b, n in enumerate(lens)]) % 2048
        assert np.array_equal(f64(k)[:, 0, 0], want) and _status(fa) == fa.FA_OK


# ------------------------------------------------------------------------------------------------ together

@pytest.mark.parametrize("bits", [16, 4])
def test_prompt_then_decoding_equals_causal_attention(fa, bits):
    """A prompt goes through the norm, rotation and attention_forward and into the pages; the following tokens are appended and
    decoded one at a time, in one captured graph.  In 16 bits every row is that of causal attention over the whole text."""
    B, N, steps, H, d, page = 2, 37, 12, 4, 64, 16
    total = N + steps
    g = torch.Generator().manual_seed(18)
    qkv = torch.randn(B, total, 3 * H, d, generator=g).bfloat16().cuda()
    wq, wk = ((1 + 0.1 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in range(2))
    cos, sin = fa.attention_rope_table(total, d)
    table = torch.randperm(2 * 5, generator=g).to(torch.int32).reshape(2, 5).cuda()
    shape = (10, H, page, d) if bits == 16 else (10, H, page, d * 5 // 8)
    kc, vc = (torch.zeros(shape, dtype=torch.bfloat16 if bits == 16 else torch.uint8, device="cuda") for _ in range(2))
    lens = torch.full((B,), N, dtype=torch.int32, device="cuda")
    # the prompt
    p = qkv[:, :N].reshape(B * N, 3 * H, d)
    q, k, v = p.split(H, 1)
    qr = fa.attention_cache_append(k, v, kc, vc, table, lens, cos=cos, sin=sin, q=q, wq=wq, wk=wk)
    kr, vr = fa.attention_cache_gather(kc, vc, table, None, B * N, dtype=torch.bfloat16)
    o, _ = fa.attention_forward(qr, kr, vr, causal=True, batch=B)
    outs = [o.reshape(B, N, H, d)]
    # the steps, from one graph
    step = torch.empty(B, 3 * H, d, dtype=torch.bfloat16, device="cuda")

    def one():
        a, b, c = step.split(H, 1)
        x = fa.attention_cache_append(b, c, kc, vc, table, lens, cos=cos, sin=sin, q=a, wq=wq, wk=wk)
        return fa.attention_decode_paged(x, kc, vc, table, lens)[0]
    step.copy_(qkv[:, N])
    lens.add_(1)
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        one()
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = one()
    lens.sub_(1)
    for i in range(steps):
        step.copy_(qkv[:, N + i])
        lens.add_(1)
        graph.replay()
        outs.append(out.clone()[:, None])
    got = torch.cat(outs, 1)
    assert _status(fa) == fa.FA_OK
    # the whole text at once
    whole = qkv.reshape(B * total, 3 * H, d)
    pos = torch.arange(total, dtype=torch.int32).repeat(B).cuda()
    qa, ka = fa.attention_qk_norm_rope(whole[:, :H], whole[:, H:2 * H], cos, sin, pos, wq=wq, wk=wk)
    va = whole[:, 2 * H:].contiguous()
    if bits == 4:
        full = [(total + page - 1) // page * b for b in range(B)]
        assert full[0] == 0
        ka, va = fa.attention_cache_gather(kc, vc, table, None, B * total, dtype=torch.bfloat16)
    ref = oracle.attention_forward(f64(qa), f64(ka), f64(va), 1 / math.sqrt(d), True, B=B, N=total)[0].reshape(B, total, H, d)
    # attention_forward rounds P to bf16 (2^-9 of Σ p|v|, |v| < 5): its own bound is 1e-2; in 4 bits the gathered rows are
    # rounded to bf16 once more than the decoded ones (2^-9 of |k| and |v|)
    assert np.abs(f64(got) - ref).max() <= (1e-2 if bits == 16 else 4e-2)


def test_training_step_of_norm_rotation_and_attention(fa):
    """qk_norm_rope → attention_forward → attention_backward → qk_norm_rope_backward against the oracle's chain."""
    B, N, H, d = 2, 70, 2, 64
    g = torch.Generator().manual_seed(19)
    qkv = torch.randn(B * N, 3 * H, d, generator=g).bfloat16()
    do = torch.randn(B * N, H, d, generator=g).bfloat16()
    wq, wk = ((1 + 0.1 * torch.randn(d, generator=g)).bfloat16() for _ in range(2))
    cos, sin = fa.attention_rope_table(N, d)
    pos = torch.arange(N, dtype=torch.int32).repeat(B)
    c = qkv.cuda()
    q, k, v = c[:, :H], c[:, H:2 * H], c[:, 2 * H:].contiguous()
    kw = dict(wq=wq.cuda(), wk=wk.cuda())
    qr, kr = fa.attention_qk_norm_rope(q, k, cos, sin, pos.cuda(), **kw)
    o, lse = fa.attention_forward(qr, kr, v, causal=True, batch=B)
    dqr, dkr, dv = fa.attention_backward(qr, kr, v, o, lse, do.cuda(), causal=True, batch=B)
    dq, dk, dwq, dwk = fa.attention_qk_norm_rope_backward(dqr, dkr, cos, sin, pos.cuda(), q=q, k=k, **kw)
    assert _status(fa) == fa.FA_OK
    C, S, P, scale = f64(cos), f64(sin), pos.numpy(), 1 / math.sqrt(d)
    x = f64(qkv)
    Q, K = (oracle.qk_norm_rope(x[:, i * H:(i + 1) * H], f64(w), C, S, P) for i, w in ((0, wq), (1, wk)))
    gQ, gK, gV = oracle.attention_backward(Q, K, x[:, 2 * H:], f64(do), scale, True, B=B)
    rq, rwq = oracle.qk_norm_rope_backward(gQ, x[:, :H], f64(wq), C, S, P)
    rk, rwk = oracle.qk_norm_rope_backward(gK, x[:, H:2 * H], f64(wk), C, S, P)
    rel = lambda a, b: np.linalg.norm(f64(a) - b) / np.linalg.norm(b)  # noqa: E731
    # the attention's own gradient bound, 2e-2 relative; the roundings of q, k and their gradients add 2^-9 each
    for a, b in ((dq, rq), (dk, rk), (dv, gV), (dwq, rwq), (dwk, rwk)):
        assert rel(a, b) <= 2.5e-2


def test_decode_matches_the_contiguous_decode(fa):
    """The paged decode and attention_decode over the gathered rows give the same numbers up to rounding."""
    lens, H, d = [100, 513, 1], 4, 128
    table, kc, vc = (t.cuda() for t in _cache(lens, H, d, 64, "bf16", 16, 20))
    q = torch.randn(3, H, d, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    k, v = fa.attention_cache_gather(kc, vc, table, cu, sum(lens))
    a, la = fa.attention_decode(q, k, v, cu_seqlens_k=cu, max_seqlen_k=513)
    b, lb = fa.attention_decode_paged(q, kc, vc, table, torch.tensor(lens, dtype=torch.int32).cuda())
    assert np.abs(f64(a) - f64(b)).max() <= 2.0 ** -8 * max(1.0, np.abs(f64(a)).max()) and np.abs(f64(la) - f64(lb)).max() <= 1e-5


def test_decode_repeats_captured_shared_workspace_and_streams(fa):
    lens = [600, 5000, 1]
    table, kc, vc = (t.cuda() for t in _cache(lens, 2, 128, 64, "bf16", 4, 21))
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    q = torch.randn(3, 8, 128, generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    ref = fa.attention_decode_paged(q, kc, vc, table, ln, max_seqlen_k=20000)
    again = fa.attention_decode_paged(q, kc, vc, table, ln, max_seqlen_k=20000)
    assert torch.equal(ref[0], again[0]) and torch.equal(ref[1], again[1])
    ws = torch.empty(fa.fa_decode_paged_workspace_bytes(3, 1, 8, 2, 20000, 128), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    ws.fill_(255)
    graphs, outs, q2 = [], [], -q
    for x in (q, q2):  # two graphs that share a workspace, replayed in turn
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(fa.attention_decode_paged(x, kc, vc, table, ln, max_seqlen_k=20000, workspace=ws))
    for _ in range(2):
        for gr in graphs:
            gr.replay()
    want = fa.attention_decode_paged(q2, kc, vc, table, ln, max_seqlen_k=20000)
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], ref[0]) and torch.equal(outs[1][0], want[0]) and torch.equal(outs[1][1], want[1])
    sides = [torch.cuda.Stream() for _ in range(2)]  # two calls at once, each with memory of its own
    got = [fa.attention_decode_paged(x, kc, vc, table, ln, max_seqlen_k=20000, stream=s.cuda_stream) for x, s in zip((q, q2), sides)]
    torch.cuda.synchronize()
    assert torch.equal(got[0][0], ref[0]) and torch.equal(got[1][0], want[0])
    assert _status(fa) == fa.FA_OK


def test_offsets_past_32_bits(fa):
    """A cache of over 2^32 bytes: the last page is written, read and decoded like any other."""
    page, hk, d = 64, 8, 128
    pages = (1 << 32) // (hk * page * d * 2) + 5
    kc, vc = (torch.zeros(pages, hk, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(8)
    k, v = (torch.randn(70, hk, d, generator=g).bfloat16().cuda() for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32).cuda()
    ln = torch.tensor([70], dtype=torch.int32).cuda()
    fa.attention_cache_append(k, v, kc, vc, table, ln)
    gk, gv = fa.attention_cache_gather(kc, vc, table, None, 70)
    assert torch.equal(gk, k) and torch.equal(gv, v) and torch.equal(kc[pages - 1].transpose(0, 1), k[:64])
    assert float(kc[:pages - 3].abs().max()) == 0.0
    q = torch.randn(1, hk, d, generator=g).bfloat16()
    o, lse = fa.attention_decode_paged(q.cuda(), kc, vc, table, ln)
    ref, rl = oracle.decode_paged(f64(q), f64(k), f64(v), 1 / math.sqrt(d))
    assert np.abs(f64(o) - ref).max() <= 2.0 ** -8 * 5 and np.abs(f64(lse) - rl).max() <= 1e-4 and _status(fa) == fa.FA_OK


def test_refusals(fa):
    table, kc, vc = (t.cuda() for t in _cache([20, 5], 2, 64, 16, "bf16", 16, 22))
    ln = torch.tensor([20, 5], dtype=torch.int32).cuda()
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: fa.attention_decode_paged(q.half(), kc, vc, table, ln), lambda: fa.attention_decode_paged(q[:1], kc, vc, table, ln),
                 lambda: fa.attention_decode_paged(q, kc, vc[:1], table, ln), lambda: fa.attention_decode_paged(q, kc, vc, table.long(), ln),
                 lambda: fa.attention_decode_paged(q, kc, vc, table, ln.cpu()), lambda: fa.attention_decode_paged(q, kc, vc, table, ln[:1]),
                 lambda: fa.attention_decode_paged(q, kc[..., :40].contiguous(), vc, table, ln),
                 lambda: fa.attention_decode_paged(q, kc, vc, table, ln, out=q[:1]),
                 lambda: fa.attention_cache_append(k, k, kc.half(), vc.half(), table, ln),
                 lambda: fa.attention_cache_append(k, k[:, :1], kc, vc, table, ln),
                 lambda: fa.attention_cache_append(k, k, kc, vc, table, ln, wq=q[0, 0]),
                 lambda: fa.attention_cache_append(k, k, kc, vc, table, ln, positions=ln),
                 lambda: fa.attention_cache_gather(kc, vc, table, None, 4, dtype=torch.float16),
                 lambda: fa.attention_cache_gather(kc, vc, table, ln, 4)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fa.attention_decode_paged(q[:, :3].contiguous(), kc, vc, table, ln),          # 3 heads over 2
                 lambda: fa.attention_decode_paged(q, kc, vc, table, ln, max_seqlen_k=0),
                 lambda: fa.attention_decode_paged(q, kc, vc, table, ln, scale=float("nan")),
                 lambda: fa.attention_decode_paged(q, kc[:, :, :8].contiguous(), vc[:, :, :8].contiguous(), table, ln),
                 lambda: fa.attention_cache_append(torch.cat([k, k[:1]]), torch.cat([k, k[:1]]), kc, vc, table, ln),
                 lambda: fa.attention_cache_gather(kc, vc, table, None, 0)):
        with pytest.raises(fa.FAError):
            call()
    assert _status(fa) == fa.FA_OK
