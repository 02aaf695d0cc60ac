"""Decode over a 4-bit paged cache where keys of unlike weight hold values of unlike size, against the fp64 oracle.

Tolerance, derived before the first run (u = finfo(dtype).eps / 2).  Key j of weight p_j (Σ p = 1) holds n_j·scale_j + min_j:
* its probability is rounded to fp16 once, 2^-11 of |value|, and for bf16 outputs the product with the scale once more, 2^-11 of
  scale·|n − 8| <= 8·scale; scores and sums: 2·max ds + 2^-16 of n·scale + |min|, ds = 2^-18·Σ|q k| + 2^-22·|s| as in
  test_gpu_paged.py;
* numbers under fp16's normal range are rounded to 2^-25 where the largest p_j·2^e_j is held at 2^6 or more, 2^e_j being at
  most twice the largest of |min| and scale of key j, and at least 2^-14: a key adds at most 2^-31·max_j(p_j·2^e_j) times 16
  for n·scale + min and 8 for scale·|n − 8|;
* the output's own rounding, u·|o| (+ 2^-25 in fp16).
"""

import numpy as np
import pytest
import torch

import oracle
from _gpu import f64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
PAGE = 64


@pytest.fixture(scope="module")
def fa():
    from _lib import load_fa
    m = load_fa()
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu-marked tests")
    return m


def _check(fa, scores, values, dtype, heads, most):
    """600 sequences that share the pages of one: a block takes a whole sequence, a quarter of its keys a warp.  Key j scores
    scores[j] (feature 0 of the key; the queries are 1 there and 0 elsewhere)."""
    n, d = values.shape
    k = np.zeros((n, d))
    k[:, 0] = scores
    pages = n // PAGE
    table = np.random.default_rng(n).permutation(pages).astype(np.int32)[None]
    caches = []
    for x, is_value in ((k, False), (values, True)):
        x = f64(torch.from_numpy(x).to(DT[dtype]))
        paged = np.zeros((pages, 1, PAGE, d))
        paged[table[0], 0] = x.reshape(pages, PAGE, d)
        caches.append(oracle.four_bit_pack(*oracle.four_bit_rows(paged), is_value).reshape(pages, 1, PAGE, d * 5 // 8))
    kr, ka, km, _ = oracle.cache_rows(caches[0], table, 0, np.arange(n), d, False)
    vr, va, vm, vs = oracle.cache_rows(caches[1], table, 0, np.arange(n), d, True)
    q = np.zeros((1, heads, d))
    q[..., 0] = 1.0
    ref, rl = oracle.decode_paged(q, kr, vr, 1.0)
    s = kr[:, 0, 0]
    p = np.exp(s - rl[0, 0])
    ds = (2.0 ** -18 * (np.abs(ka[:, 0, 0]) + np.abs(km[:, 0, 0])) + 2.0 ** -22 * np.abs(s)).max()
    vr, va, vm, vs = vr[:, 0], va[:, 0], vm[:, 0], vs[:, 0]
    size = np.maximum(2.0 ** -14, 2 * np.maximum(np.abs(vm), vs).max(1))
    u = torch.finfo(DT[dtype]).eps / 2
    bound = (p @ np.abs(vr)) * 2.0 ** -11 + (p @ (np.abs(va) + np.abs(vm))) * (2 * ds + 2.0 ** -16)
    if dtype == "bf16":
        bound = bound + (p @ (8 * vs)) * 2.0 ** -11
    bound = bound + n * 24 * 2.0 ** -31 * (p * size).max() + u * np.abs(ref[0, 0]) * (1 + 2.0 ** -7) + 2.0 ** -25
    assert np.abs(ref[0, 0]).max() > 50 * bound.max()  # the bound tells the output from 0
    B = 600
    o, lse = fa.attention_decode_paged(torch.from_numpy(q).to(DT[dtype]).expand(B, heads, d).contiguous().cuda(),
                                       torch.from_numpy(caches[0]).cuda(), torch.from_numpy(caches[1]).cuda(),
                                       torch.from_numpy(table).expand(B, pages).contiguous().cuda(),
                                       torch.full((B,), n, dtype=torch.int32).cuda(), max_seqlen_k=most, scale=1.0)
    assert fa.fa_check_device_status(torch.cuda.current_stream().cuda_stream) == fa.FA_OK
    err = np.abs(f64(o) - ref)
    assert np.all(err <= bound), ((err / bound).max(), f64(o)[0, 0, :4], ref[0, 0, :4])
    assert np.all(np.abs(f64(lse) - rl) <= ds + 2.0 ** -20 * (1 + np.abs(rl)))


@pytest.mark.parametrize("most", [None, 100000])
@pytest.mark.parametrize("heads", [1, 12])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("octaves", [18, 20, 22])
def test_small_values_beside_a_key_that_outweighs_them(fa, octaves, dtype, d, heads, most):
    """The key that weighs 2^octaves of any other holds 0, the others the same row of values, of which the largest is 0.005 and
    (so that fp16 outputs are normal numbers) 8 in the last case."""
    n = 2048
    for top in (0.005, 8.0):
        if dtype == "fp16" and top < 1 and octaves > 18:
            continue  # outputs under 2^-14, which fp16 itself holds with few bits
        scores = np.zeros(n)
        scores[70] = octaves * np.log(2.0)
        values = np.tile(np.linspace(-1, 1, d) * top, (n, 1))
        values[70] = 0.0
        _check(fa, scores, values, dtype, heads, most)


@pytest.mark.parametrize("most", [None, 100000])
@pytest.mark.parametrize("heads", [1, 12])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("size", [2.0 ** 5, 2.0 ** 8, 2.0 ** 10, 2.0 ** 12])
@pytest.mark.parametrize("at,first", [(66, 70), (1866, 70), (66, 1094), (3, 70)])
def test_one_large_value_without_weight(fa, at, first, size, dtype, heads, most):
    """A row of values with a large scale and no weight beside the key that outweighs the others by e^13.5: in the same tile of
    the same warp (a warp has keys 64 … 95 of every 128), after it, before it, and in another warp."""
    n, d = 2048, 64
    scores = np.full(n, 40.5)
    scores[first], scores[at] = 54.0, 0.0
    values = np.full((n, d), 1.5)
    values[first] = 0.0
    values[at] = np.linspace(-7.5, 7.5, d) * size
    _check(fa, scores, values, dtype, heads, most)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("scale", [1e-25, 1e-37])
def test_queries_and_scales_near_zero(fa, scale, dtype):
    """Scores that are 0 to every digit: the mean of the values that a row sees, whatever the tile's places behind the sequence
    hold.  Errors as above: 2^-11 of each value and, for bf16 outputs, of 8·scale, 2^-16 of n·scale + |min|, the output's own."""
    n, d = 37, 64
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(1, 1, PAGE, d, generator=g).to(DT[dtype]) for _ in range(2))
    caches = [torch.from_numpy(oracle.four_bit_pack(*oracle.four_bit_rows(f64(x)), i == 1)).reshape(1, 1, PAGE, d * 5 // 8)
              for i, x in enumerate((k, v))]
    table = np.zeros((1, 1), np.int32)
    vr, va, vm, vs = (x[:, 0] for x in oracle.cache_rows(caches[1], table, 0, np.arange(n), d, True))
    q = torch.zeros(1, 2, 3, d, dtype=DT[dtype])
    q[0, :, 1] = 1.0
    q[0, :, 2, 0] = 2.0 ** -20
    for most in (None, 100000):
        o, lse = fa.attention_decode_paged(q.cuda(), *(x.cuda() for x in caches), torch.from_numpy(table).cuda(),
                                           torch.tensor([n], dtype=torch.int32).cuda(), max_seqlen_k=most, scale=scale)
        assert fa.fa_check_device_status(torch.cuda.current_stream().cuda_stream) == fa.FA_OK
        u = torch.finfo(DT[dtype]).eps / 2
        for i, m in enumerate((n - 1, n)):
            ref = vr[:m].mean(0)
            bound = (np.abs(vr) * 2.0 ** -11 + 8 * vs * (2.0 ** -11 if dtype == "bf16" else 0) + (np.abs(va) + np.abs(vm)) * 2.0 ** -16)[:m].mean(0)
            bound = bound + u * np.abs(ref) * (1 + 2.0 ** -7) + 2.0 ** -25
            assert np.all(np.abs(f64(o)[0, i] - ref) <= bound) and np.all(np.abs(f64(lse)[0, i] - np.log(m)) <= 2.0 ** -18)
