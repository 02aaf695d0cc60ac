"""Append and gather of thousands of tokens: the variants that load two row groups together (from 2368 tokens on), at head
counts that leave parts of a row group, against the fp64 oracle and byte for byte.

Tolerances as in test_gpu_paged.py: rotated keys u·|y| + 2^-17·(|a cos| + |b sin|) (+ 2^-25 in fp16), what is written to the
cache equal bytes; rows read from 4 bits u·|value| + 2^-22·(n·scale + |min|) (one product and sum in fp32, two numbers that
enter it at most 2^-24 each) (+ 2^-25 in fp16).
"""

import numpy as np
import pytest
import torch

import oracle
from _gpu import f64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-5


@pytest.fixture(scope="module")
def fa():
    from _lib import load_fa
    m = load_fa()
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu-marked tests")
    return m


def _status(fa):
    return fa.fa_check_device_status(torch.cuda.current_stream().cuda_stream)


def _ragged(total, seqs, rng):
    """Counts of `seqs` sequences that add up to `total`, some of them 0 and 1."""
    cut = np.sort(rng.integers(0, total + 1, seqs - 3))
    counts = np.diff(np.concatenate([[0], cut, [total]]))
    return np.concatenate([[0], counts[:-1], [0], counts[-1:]]).astype(int)


def _pages(lens, page, rng):
    need = -(-lens // page)
    total = int(need.sum()) + 2
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((len(lens), max(1, int(need.max()))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, total


@pytest.mark.parametrize("tokens", [2367, 2601])
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,hq,hk,page,rot,norm", [(64, 9, 1, 16, 64, True), (128, 5, 5, 48, 96, True), (128, 17, 3, 64, 128, True),
                                                   (64, 0, 17, 32, 48, True), (128, 0, 9, 64, 128, False), (64, 3, 5, 16, 0, False),
                                                   (128, 16, 16, 32, 0, True)])
def test_append(fa, d, hq, hk, page, rot, norm, inter, dtype, bits, tokens):
    rng = np.random.default_rng(tokens + hq + 31 * hk + d)
    new = _ragged(tokens - 3, 23, rng)                   # three rows behind the last sequence
    lens = new + rng.integers(0, 40, len(new))
    table, pages = _pages(lens, page, rng)
    g = torch.Generator().manual_seed(tokens + hq)
    qkv = torch.randn(tokens, hq + 2 * hk, d, generator=g).to(DT[dtype]).cuda()
    q, k, v = qkv.split([hq, hk, hk], 1)
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).to(DT[dtype]).cuda() for _ in range(2))
    cos, sin = fa.attention_rope_table(int(lens.max()), max(rot, 16))
    row = d if bits == 16 else d * 5 // 8
    before = [torch.randint(0, 256, (pages, hk, page, row * (2 if bits == 16 else 1)), dtype=torch.uint8, generator=g) for _ in range(2)]
    kc, vc = (x.cuda() if bits == 4 else x.cuda().view(DT[dtype]) for x in before)
    qo = torch.full((tokens, hq, d), 9.0, dtype=DT[dtype], device="cuda") if hq else None
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
    turn = dict(interleaved=inter, **(dict(cos=cos, sin=sin) if rot else {}))
    weights = dict(wq=wq if hq else None, wk=wk) if norm else {}
    got = fa.attention_cache_append(k, v, kc, vc, torch.from_numpy(table).cuda(), torch.from_numpy(lens.astype(np.int32)).cuda(), q=q if hq else None,
                                    eps=EPS, cu_seqlens=cu, q_out=qo, **turn, **weights)
    assert _status(fa) == fa.FA_OK and got is qo
    n = tokens - 3
    at = np.concatenate([np.arange(a - m, a) for a, m in zip(lens, new)])
    seq = np.repeat(np.arange(len(lens)), new)
    c64, s64 = (f64(x) for x in (cos, sin))
    if not rot:
        c64, s64 = np.ones((int(lens.max()), 8)), np.zeros((int(lens.max()), 8))
    u = torch.finfo(DT[dtype]).eps / 2
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0
    outs = []
    for x, w, y in ((q, wq, qo), (k, wk, None)):
        if x.shape[1] == 0:
            outs.append(None)
            continue
        x64, w64 = f64(x[:n]), f64(w) if norm else None
        ref = oracle.qk_norm_rope(x64, w64, c64, s64, at, EPS, inter and rot > 0)
        amp = sum(np.abs(oracle.qk_norm_rope(np.abs(x64), None if w64 is None else np.abs(w64), np.abs(c64), sign * np.abs(s64), at, EPS, inter and rot > 0))
                  for sign in (1, -1))
        outs.append((ref, u * np.abs(ref) + 2.0 ** -17 * amp + tiny))
    if hq:
        assert np.all(np.abs(f64(qo[:n]) - outs[0][0]) <= outs[0][1])
        assert bool((qo[n:] == 9).all())
    # the rows that were written, and all that were not
    p, slot = table[seq, at // page], at % page
    for cache, old, is_value in ((kc, before[0], False), (vc, before[1], True)):
        cache = cache.cpu()
        if bits == 16:
            rows, want = cache[p, :, slot], old.view(DT[dtype]).clone()
            if is_value:
                assert torch.equal(rows.view(torch.int16), v[:n].cpu().view(torch.int16))
            else:
                assert np.all(np.abs(f64(rows) - outs[1][0]) <= outs[1][1])
            want[p, :, slot] = rows
            assert torch.equal(cache.view(torch.uint8), want.view(torch.uint8))
            continue
        if is_value:
            rows = f64(v[:n])
        else:  # the 16-bit rows that the 4-bit ones are made from, by a 16-bit cache of the same call
            k16, v16 = (torch.zeros(pages, hk, page, d, dtype=DT[dtype], device="cuda") for _ in range(2))
            fa.attention_cache_append(k, v, k16, v16, torch.from_numpy(table).cuda(), torch.from_numpy(lens.astype(np.int32)).cuda(), q=q if hq else None,
                                      eps=EPS, cu_seqlens=cu, **turn, **weights)
            rows = f64(k16)[p, :, slot]
            assert np.all(np.abs(rows - outs[1][0]) <= outs[1][1])
        num, sc, mn = (x.copy() for x in oracle.four_bit_unpack(old.reshape(pages, hk, -1).numpy(), page, d, is_value))
        n2, s2, m2 = oracle.four_bit_rows(rows)
        num[p, :, slot], sc[p, :, slot], mn[p, :, slot] = n2, s2, m2
        gn, gs, gm = oracle.four_bit_unpack(cache.reshape(pages, hk, -1).numpy(), page, d, is_value)
        assert np.array_equal(gn, num) and np.array_equal(gs, sc, equal_nan=True) and np.array_equal(gm, mn, equal_nan=True)


@pytest.mark.parametrize("tokens", [2367, 3001])
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,hk,page", [(64, 5, 16), (64, 17, 48), (128, 5, 64), (128, 9, 32), (64, 8, 64), (128, 1, 16)])
def test_gather(fa, d, hk, page, dtype, bits, tokens):
    rng = np.random.default_rng(tokens + hk)
    take = _ragged(tokens - 5, 19, rng)                  # two rows in front, three behind
    starts = rng.integers(0, 30, len(take))
    lens = take + starts
    table, pages = _pages(lens, page, rng)
    g = torch.Generator().manual_seed(tokens)
    x = [torch.randn(pages, hk, page, d, generator=g).to(DT[dtype]) for _ in range(2)]
    caches = x
    if bits == 4:
        caches = [torch.from_numpy(oracle.four_bit_pack(*oracle.four_bit_rows(f64(y)), i == 1)).reshape(pages, hk, page, d * 5 // 8)
                  for i, y in enumerate(x)]
    cu = torch.from_numpy(np.concatenate([[2], 2 + np.cumsum(take)]).astype(np.int32)).cuda()
    into = [torch.full((tokens, hk, d), 4.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    fa.attention_cache_gather(caches[0].cuda(), caches[1].cuda(), torch.from_numpy(table).cuda(), cu, tokens,
                              starts=torch.from_numpy(starts.astype(np.int32)).cuda(), k=into[0], v=into[1])
    assert _status(fa) == fa.FA_OK
    at = np.concatenate([np.arange(s, s + m) for s, m in zip(starts, take)])
    seq = np.repeat(np.arange(len(take)), take)
    p, slot = table[seq, at // page], at % page
    for got, cache, is_value in zip(into, caches, (False, True)):
        assert bool((got[:2] == 4).all()) and bool((got[tokens - 3:] == 4).all())
        got = got[2:tokens - 3]
        if bits == 16:
            assert torch.equal(got.cpu(), cache[p, :, slot])
            continue
        n, sc, mn = oracle.four_bit_unpack(cache.reshape(pages, hk, -1).numpy(), page, d, is_value)
        a, m = n[p, :, slot] * np.repeat(sc[p, :, slot], 32, -1), np.repeat(mn[p, :, slot], 32, -1)
        u = torch.finfo(DT[dtype]).eps / 2
        assert np.all(np.abs(f64(got) - (a + m)) <= u * np.abs(a + m) + 2.0 ** -22 * (a + np.abs(m)) + (2.0 ** -25 if dtype == "fp16" else 0.0))
