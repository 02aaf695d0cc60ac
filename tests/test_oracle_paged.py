"""CPU pins of the oracle for the query/key preparation and the paged cache (oracle/paged.py)."""

import math

import numpy as np
import pytest

import oracle


def _table(rows, rot, base=10000.0):
    return oracle.rope_table(rows, rot, base)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_closed_forms(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 64))
    cos, sin = _table(50, 32)
    y = oracle.qk_norm_rope(x, None, cos, sin, [0, 7, 49], interleaved=interleaved)
    assert np.array_equal(y[0], x[0])                      # position 0 turns nothing
    assert np.array_equal(y[..., 32:], x[..., 32:])        # features behind rot_dim pass
    assert np.allclose((y[..., :32] ** 2).sum(-1), (x[..., :32] ** 2).sum(-1))
    a = slice(0, 32, 2) if interleaved else slice(0, 16)
    b = slice(1, 32, 2) if interleaved else slice(16, 32)
    freq = 10000.0 ** (-np.arange(16) / 16)
    for t, p in enumerate([0, 7, 49]):                     # a pair is a complex number times e^{i·angle}
        z = (x[t, :, a] + 1j * x[t, :, b]) * np.exp(1j * p * freq)
        assert np.allclose(y[t, :, a], z.real) and np.allclose(y[t, :, b], z.imag)
    # scores after rotation depend on the distance alone
    q = oracle.qk_norm_rope(x[:1], None, cos, sin, [30], interleaved=interleaved)
    k = oracle.qk_norm_rope(x[1:2], None, cos, sin, [25], interleaved=interleaved)
    q2 = oracle.qk_norm_rope(x[:1], None, cos, sin, [12], interleaved=interleaved)
    k2 = oracle.qk_norm_rope(x[1:2], None, cos, sin, [7], interleaved=interleaved)
    assert np.allclose((q * k).sum(-1), (q2 * k2).sum(-1))


def test_rotation_by_axes():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((4, 1, 64))
    cos, sin = _table(20, 64)
    pos = np.array([[1, 2, 3, 4], [5, 6, 7, 8], [9, 10, 11, 19]])
    y = oracle.qk_norm_rope(x, None, cos, sin, pos, sections=(8, 12, 12))
    for a, (lo, hi) in enumerate([(0, 8), (8, 20), (20, 32)]):
        one = oracle.qk_norm_rope(x, None, cos, sin, pos[a])
        assert np.array_equal(y[..., lo:hi], one[..., lo:hi]) and np.array_equal(y[..., 32 + lo:32 + hi], one[..., 32 + lo:32 + hi])


def test_norm():
    rng = np.random.default_rng(3)
    x = 5 * rng.standard_normal((6, 3, 128))
    cos, sin = _table(2, 128)
    y = oracle.qk_norm_rope(x, np.ones(128), cos, sin, np.zeros(6, int), eps=1e-12)
    assert np.allclose((y * y).mean(-1), 1.0)
    w = rng.standard_normal(128)
    assert np.allclose(oracle.qk_norm_rope(x, w, cos, sin, np.zeros(6, int), eps=1e-12), y * w)


@pytest.mark.parametrize("interleaved,sections", [(False, None), (True, None), (False, (4, 4, 8))])
def test_backward_by_differences(interleaved, sections):
    rng = np.random.default_rng(4)
    x, dy, w = rng.standard_normal((2, 2, 64)), rng.standard_normal((2, 2, 64)), 1 + 0.3 * rng.standard_normal(64)
    cos, sin = _table(30, 32)
    pos = np.array([3, 17]) if sections is None else np.array([[3, 17], [5, 2], [29, 1]])
    kw = dict(eps=1e-3, interleaved=interleaved, sections=sections)
    f = lambda x, w: (oracle.qk_norm_rope(x, w, cos, sin, pos, **kw) * dy).sum()  # noqa: E731
    dx, dw = oracle.qk_norm_rope_backward(dy, x, w, cos, sin, pos, **kw)
    h = 1e-6
    for i in [(0, 0, 0), (0, 1, 17), (1, 0, 31), (1, 1, 63)]:
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    for i in [0, 5, 40]:
        e = np.zeros(64)
        e[i] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-7
    g, none = oracle.qk_norm_rope_backward(dy, None, None, cos, sin, pos, interleaved=interleaved, sections=sections)
    assert none is None
    f0 = lambda x: (oracle.qk_norm_rope(x, None, cos, sin, pos, interleaved=interleaved, sections=sections) * dy).sum()  # noqa: E731
    assert abs(f0(x) - (g * x).sum()) < 1e-10  # linear: its own gradient


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [False, True])
def test_four_bit_layout(d, value):
    """Each number lies at the nibble the format's text names, and pairs behind the rows."""
    rng = np.random.default_rng(5)
    page, words = 16, d // 32
    x = rng.standard_normal((2, page, d)).astype(np.float16)
    n, sc, mn = oracle.four_bit_rows(x)
    blk = oracle.four_bit_pack(n, sc, mn, value)
    assert blk.shape == (2, page * d * 5 // 8)
    for head, r, f in [(0, 0, 0), (0, 3, 5), (1, 15, d - 1), (1, 7, 37), (0, 9, 63)]:
        w, rest = divmod(f, 32)
        row = blk[head, r * d // 2:(r + 1) * d // 2]
        if value:
            g, i = divmod(rest, 4)
            got = (row.view(np.uint16)[g * words + w] >> (4 * i)) & 15
        else:
            t, i = divmod(rest, 8)
            got = (row.view(np.uint32)[t * words + w] >> (4 * i)) & 15
        assert got == n[head, r, f]
        pair = blk[head, page * d // 2:].view(np.float16).reshape(page, words, 2)[r, w]
        assert float(pair[0]) == sc[head, r, w] and float(pair[1]) == mn[head, r, w]
    back = oracle.four_bit_unpack(blk, page, d, value)
    assert all(np.array_equal(a, b) for a, b in zip(back, (n, sc, mn)))


def test_four_bit_error():
    rng = np.random.default_rng(6)
    x = (rng.standard_normal((50, 64)) * np.exp(rng.standard_normal((50, 1)) * 3)).astype(np.float16).astype(np.float64)
    n, sc, mn = oracle.four_bit_rows(x)
    s, m = np.repeat(sc, 32, -1), np.repeat(mn, 32, -1)
    # half a step, and what the rounding of scale (15 steps of it) and minimum leaves outside the range
    assert np.all(np.abs(n * s + m - x) <= s * (0.5 + 15 * 2.0 ** -11) + np.abs(m) * 2.0 ** -11 + 2.0 ** -24)
    const = np.full((1, 64), 3.25)
    n, sc, mn = oracle.four_bit_rows(const)
    assert np.all(n == 0) and np.all(sc == 0) and np.all(mn == 3.25)


def test_decode_against_pinned_attention():
    rng = np.random.default_rng(7)
    q, k, v = rng.standard_normal((3, 4, 64)), rng.standard_normal((9, 4, 64)), rng.standard_normal((9, 4, 64))
    o, lse = oracle.decode_paged(q[-1:], k, v, 0.2)
    O, L = oracle.decode_forward(q[-1:], k, v, 0.2, B=1, Nk=9)
    assert np.allclose(o, O) and np.allclose(lse, L)
    full = np.concatenate([rng.standard_normal((6, 4, 64)), q])  # the last rows of causal self-attention
    O, L = oracle.attention_forward(full, k, v, 0.2, True)
    o, lse = oracle.decode_paged(q, k, v, 0.2)
    assert np.allclose(o, O[-3:]) and np.allclose(lse, L[-3:])
    o, lse = oracle.decode_paged(q, k[:2], v[:2], 0.2)      # more queries than keys: the first sees none
    assert np.all(o[0] == 0) and np.all(np.isneginf(lse[0])) and np.allclose(o[1], v[0])
    # shared heads: query heads 2h, 2h + 1 read key head h
    o2, _ = oracle.decode_paged(q, k[:, :2], v[:, :2], 0.2)
    o4, _ = oracle.decode_paged(q, np.repeat(k[:, :2], 2, 1), np.repeat(v[:, :2], 2, 1), 0.2)
    assert np.allclose(o2, o4)


def test_cache_rows():
    rng = np.random.default_rng(8)
    x = rng.standard_normal((5, 2, 16, 64)).astype(np.float16)
    table = np.array([[3, 0, -1], [4, 1, 2]])
    rows = oracle.cache_rows(x, table, 1, np.arange(40), 64, False)[0]
    assert np.array_equal(rows[37], x[2, :, 5].astype(np.float64))
    n, sc, mn = oracle.four_bit_rows(x)
    blk = oracle.four_bit_pack(n, sc, mn, True).reshape(5, 2, 16, 40)
    rows = oracle.cache_rows(blk, table, 0, np.arange(20), 64, True)[0]
    want = n[0, :, 3] * np.repeat(sc[0, :, 3], 32, -1) + np.repeat(mn[0, :, 3], 32, -1)
    assert np.array_equal(rows[19], want) and math.isfinite(rows.sum())
