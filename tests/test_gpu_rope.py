"""GPU parity of the query/key norm and rotation and its gradient against the fp64 oracle.

Tolerances, derived before the first run.  u = half a step of the output type relative to the value (finfo.eps / 2:
bf16 2^-8, fp16 2^-11), E = 2^-17: a bound for the fp32 arithmetic in front of the rounding, relative to the sum of the magnitudes that
enter (the sum of squares and the mean of d <= 128 terms go through chains of at most 16 + 3 additions, rsqrt, a product with
the weight and two products of the rotation add at most 2^-22 each: 30 roundings of 2^-24 < 2^-19; E leaves a factor 4).
fp16 results under 2^-14 are rounded to multiples of 2^-24.
"""

import numpy as np
import pytest
import torch

import oracle
from _gpu import f64

pytestmark = pytest.mark.gpu

E = 2.0 ** -17
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


def _inputs(T, hq, hk, d, rot, dtype, norm=True, axes=1, rows=97, seed=0):
    g = torch.Generator().manual_seed(1000 + seed)
    r = lambda *s: torch.randn(*s, generator=g).to(DT[dtype])  # noqa: E731
    cos, sin = (torch.from_numpy(x).float() for x in oracle.rope_table(rows, rot, 10000.0))
    x = dict(qkv=r(T, hq + 2 * hk, d), gq=r(T, hq, d), gk=r(T, hk, d), cos=cos, sin=sin,
             pos=torch.randint(0, rows, (axes, T), generator=g, dtype=torch.int32))
    x["wq"], x["wk"] = ((1 + 0.2 * torch.randn(d, generator=g)).to(DT[dtype]) for _ in range(2)) if norm else (None, None)
    n = rot // 2
    x["sections"] = None if axes == 1 else {2: (4, n - 4), 3: (4, 4, n - 8), 4: (n - 12, 4, 4, 4)}[axes]
    return x


def _cuda(x):
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in x.items()}


def _amplitude(x, w, x_in, eps, interleaved, sections):
    """Σ of the magnitudes that enter each output: |a cos| + |b sin| of the normed row."""
    cos, sin = x["cos"].double().abs().numpy(), -x["sin"].double().abs().numpy()
    y = oracle.qk_norm_rope(np.abs(f64(x_in)), None if w is None else np.abs(f64(w)), cos, sin, x["pos"].numpy(), eps, interleaved, sections)
    # the second partner is b·cos + a·sin: with −|sin| it comes out as |b cos| − |a sin|, so take both signs
    z = oracle.qk_norm_rope(np.abs(f64(x_in)), None if w is None else np.abs(f64(w)), cos, -sin, x["pos"].numpy(), eps, interleaved, sections)
    return np.maximum(np.abs(y), np.abs(z))


def _bound(ref, amp, dt):
    return torch.finfo(dt).eps / 2 * np.abs(ref) + E * amp + (2.0 ** -25 if dt == torch.float16 else 0.0)


SHAPES = [  # T, hq, hk, d, rot, interleaved, axes
    (1, 1, 1, 64, 64, False, 1), (1, 5, 1, 128, 128, False, 1), (2, 4, 2, 64, 16, True, 1), (7, 3, 3, 128, 48, False, 2),
    (8, 16, 16, 128, 128, False, 1), (9, 17, 2, 64, 64, False, 3), (33, 8, 8, 128, 96, True, 3), (301, 12, 4, 64, 48, True, 4),
    (129, 1, 9, 128, 16, False, 1), (2500, 4, 4, 128, 128, False, 1),
    # few heads: several tokens in a warp, the last warp not full
    (301, 2, 1, 64, 32, False, 1), (5, 3, 2, 64, 64, True, 1), (6001, 1, 2, 128, 128, False, 1), (4003, 12, 1, 64, 64, True, 3),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(fa, shape, norm, dtype):
    T, hq, hk, d, rot, inter, axes = shape
    if rot // 2 < 4 * axes:
        axes = 1
    x = _inputs(T, hq, hk, d, rot, dtype, norm, axes, seed=T)
    c = _cuda(x)
    q, k = c["qkv"][:, :hq], c["qkv"][:, hq:hq + hk]
    before = c["qkv"].clone()
    yq, yk = fa.attention_qk_norm_rope(q, k, c["cos"], c["sin"], c["pos"], wq=c["wq"], wk=c["wk"], eps=1e-5, interleaved=inter,
                                       sections=x["sections"])
    assert _status(fa) == fa.FA_OK
    assert torch.equal(c["qkv"], before)
    for y, xin, w in ((yq, x["qkv"][:, :hq], x["wq"]), (yk, x["qkv"][:, hq:hq + hk], x["wk"])):
        ref = oracle.qk_norm_rope(f64(xin), None if w is None else f64(w), x["cos"].double().numpy(), x["sin"].double().numpy(),
                                  x["pos"].numpy(), 1e-5, inter, x["sections"])
        err = np.abs(f64(y) - ref)
        assert np.all(err <= _bound(ref, _amplitude(x, w, xin, 1e-5, inter, x["sections"]), DT[dtype])), err.max()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(fa, shape, norm, dtype):
    T, hq, hk, d, rot, inter, axes = shape
    if rot // 2 < 4 * axes:
        axes = 1
    x = _inputs(T, hq, hk, d, rot, dtype, norm, axes, seed=T + 1)
    c = _cuda(x)
    kw = dict(q=c["qkv"][:, :hq], k=c["qkv"][:, hq:hq + hk], wq=c["wq"], wk=c["wk"]) if norm else {}
    dq, dk, dwq, dwk = fa.attention_qk_norm_rope_backward(c["gq"], c["gk"], c["cos"], c["sin"], c["pos"], eps=1e-5, interleaved=inter,
                                                          sections=x["sections"], **kw)
    assert _status(fa) == fa.FA_OK
    assert (dwq is None) == (not norm) and (dwk is None) == (not norm)
    cos, sin = x["cos"].double().numpy(), x["sin"].double().numpy()
    for dx, dw, g, xin, w in ((dq, dwq, x["gq"], x["qkv"][:, :hq], x["wq"]), (dk, dwk, x["gk"], x["qkv"][:, hq:hq + hk], x["wk"])):
        ref, refw = oracle.qk_norm_rope_backward(f64(g), f64(xin), None if w is None else f64(w), cos, sin, x["pos"].numpy(), 1e-5,
                                                 inter, x["sections"])
        G = _amplitude(x, None, g, 1e-5, inter, x["sections"])  # magnitudes that enter the turned gradient
        if not norm:
            assert np.all(np.abs(f64(dx) - ref) <= _bound(ref, G, DT[dtype]))
            continue
        xf, wf = f64(xin), np.abs(f64(w))
        r = 1 / np.sqrt((xf * xf).mean(-1, keepdims=True) + 1e-5)
        n = np.abs(xf) * r
        amp = r * (G * wf + n * (G * wf * n).mean(-1, keepdims=True))
        err = np.abs(f64(dx) - ref)
        assert np.all(err <= _bound(ref, amp, DT[dtype])), err.max()
        errw = np.abs(f64(dw) - refw)
        # at most 64 additions in a row before the tree: their roundings stay within E of the sum of magnitudes
        assert np.all(errw <= 2 * E * (G * n).sum((0, 1))), (errw / (G * n).sum((0, 1))).max()


def test_gradient_by_differences(fa):
    """⟨y, g⟩ moves with x and w as dx and dw say (fp16 inputs; differences of the oracle's value over steps the type holds)."""
    x = _inputs(2, 2, 1, 64, 64, "fp16", seed=5)
    c = _cuda(x)
    dq, dk, dwq, dwk = fa.attention_qk_norm_rope_backward(c["gq"], c["gk"], c["cos"], c["sin"], c["pos"], q=c["qkv"][:, :2],
                                                          k=c["qkv"][:, 2:3], wq=c["wq"], wk=c["wk"], eps=1e-5)
    cos, sin, pos = x["cos"].double().numpy(), x["sin"].double().numpy(), x["pos"].numpy()
    f = lambda a, w: (oracle.qk_norm_rope(a, w, cos, sin, pos, 1e-5) * f64(x["gq"])).sum()  # noqa: E731
    a, w, h = f64(x["qkv"][:, :2]), f64(x["wq"]), 1e-5
    for i in [(0, 0, 0), (1, 1, 33), (0, 1, 63)]:
        e = np.zeros_like(a)
        e[i] = h
        diff = (f(a + e, w) - f(a - e, w)) / (2 * h)
        # half a step of fp16 on dx, the fp32 bound and the difference's own curvature (h², under 1e-6 here)
        assert abs(f64(dq)[i] - diff) <= 2.0 ** -11 * abs(diff) + 1e-4
    for i in [0, 31, 63]:
        e = np.zeros(64)
        e[i] = h
        assert abs(f64(dwq)[i] - (f(a, w + e) - f(a, w - e)) / (2 * h)) <= 1e-4


def test_in_place_and_strided_outputs(fa):
    x = _cuda(_inputs(37, 6, 2, 128, 128, "bf16", seed=6))
    q, k = x["qkv"][:, :6], x["qkv"][:, 6:8]
    kw = dict(wq=x["wq"], wk=x["wk"])
    yq, yk = fa.attention_qk_norm_rope(q, k, x["cos"], x["sin"], x["pos"], **kw)
    into = x["qkv"].clone()
    v = into[:, 8:].clone()
    a, b = fa.attention_qk_norm_rope(into[:, :6], into[:, 6:8], x["cos"], x["sin"], x["pos"], q_out=into[:, :6], k_out=into[:, 6:8], **kw)
    assert torch.equal(a, yq) and torch.equal(b, yk) and torch.equal(into[:, 8:], v)
    dq, dk, dwq, dwk = fa.attention_qk_norm_rope_backward(x["gq"], x["gk"], x["cos"], x["sin"], x["pos"], q=q, k=k, **kw)
    gq, gk = x["gq"].clone(), x["gk"].clone()
    again = fa.attention_qk_norm_rope_backward(gq, gk, x["cos"], x["sin"], x["pos"], q=q, k=k, dq=gq, dk=gk, **kw)
    assert all(torch.equal(s, t) for s, t in zip(again, (dq, dk, dwq, dwk)))  # dw too: its order of sums is fixed
    grad = torch.full_like(x["qkv"], 7.0)
    fa.attention_qk_norm_rope_backward(x["gq"], x["gk"], x["cos"], x["sin"], x["pos"], q=q, k=k, dq=grad[:, :6], dk=grad[:, 6:8], **kw)
    assert torch.equal(grad[:, :6], dq) and torch.equal(grad[:, 6:8], dk) and bool((grad[:, 8:] == 7).all())


@pytest.mark.parametrize("bad", [-1, 97, 2 ** 31 - 1, -2 ** 31])
def test_positions_out_of_range_are_skipped(fa, bad):
    x = _cuda(_inputs(20, 3, 2, 64, 64, "bf16", seed=7))
    q, k = x["qkv"][:, :3], x["qkv"][:, 3:5]
    args = (x["cos"], x["sin"])
    yq, yk = fa.attention_qk_norm_rope(q, k, *args, x["pos"], wq=x["wq"], wk=x["wk"])
    pos = x["pos"].clone()
    pos[0, 11] = bad
    oq, ok = torch.full_like(yq, 3.0), torch.full_like(yk, 3.0)
    fa.attention_qk_norm_rope(q, k, *args, pos, wq=x["wq"], wk=x["wk"], q_out=oq, k_out=ok)
    assert _status(fa) == fa.FA_ERR_INVALID_ARG
    assert bool((oq[11] == 3).all()) and bool((ok[11] == 3).all())
    yq[11], yk[11] = 3.0, 3.0
    assert torch.equal(oq, yq) and torch.equal(ok, yk)
    # the gradient of a skipped token adds nothing to dw
    zq, zk = x["gq"].clone(), x["gk"].clone()
    dq, dk = torch.full_like(zq, 3.0), torch.full_like(zk, 3.0)
    _, _, dwq, dwk = fa.attention_qk_norm_rope_backward(zq, zk, *args, pos, q=q, k=k, wq=x["wq"], wk=x["wk"], dq=dq, dk=dk)
    assert _status(fa) == fa.FA_ERR_INVALID_ARG
    zq[11], zk[11] = 0.0, 0.0
    eq, ek, ewq, ewk = fa.attention_qk_norm_rope_backward(zq, zk, *args, x["pos"], q=q, k=k, wq=x["wq"], wk=x["wk"])
    eq[11], ek[11] = 3.0, 3.0  # nor is it written; the others are
    assert torch.equal(dq, eq) and torch.equal(dk, ek)
    assert torch.equal(dwq, ewq) and torch.equal(dwk, ewk) and _status(fa) == fa.FA_OK


def test_zero_rows_infinities_and_nan(fa):
    x = _inputs(6, 2, 2, 64, 64, "bf16", seed=8)
    x["qkv"][0] = 0.0
    x["qkv"][1, 0, 5] = float("inf")
    x["qkv"][2, 1, 7] = float("nan")
    c = _cuda(x)
    yq, yk = fa.attention_qk_norm_rope(c["qkv"][:, :2], c["qkv"][:, 2:4], c["cos"], c["sin"], c["pos"], wq=c["wq"], wk=c["wk"])
    assert bool((yq[0] == 0).all()) and bool((yk[0] == 0).all())
    assert bool(torch.isnan(yq[1, 0]).any()) and bool(torch.isnan(yq[2, 1]).all())
    assert bool(torch.isfinite(yq[1, 1]).all()) and bool(torch.isfinite(yq[2, 0]).all()) and bool(torch.isfinite(yk).all())
    assert bool(torch.isfinite(yq[3:]).all())


@pytest.mark.parametrize("rows,rot,base", [(1, 16, 10000.0), (4097, 128, 10000.0), (1 << 20, 16, 500000.0)])
def test_table(fa, rows, rot, base):
    cos, sin = fa.attention_rope_table(rows, rot, base)
    at = np.unique(np.concatenate([np.arange(min(rows, 300)), np.linspace(0, rows - 1, 200).astype(int)]))
    i = np.arange(rot // 2)
    ang = at[:, None] * np.power(base, -2.0 * i / rot)
    # 64-bit angles up to 2^20 carry 2^-33·few; half a step of fp32 on the result
    for got, ref in ((cos, np.cos(ang)), (sin, np.sin(ang))):
        assert np.all(np.abs(f64(got[torch.from_numpy(at)]) - ref) <= 2.0 ** -25 + 2.0 ** -29)


def test_captured_and_on_another_stream(fa):
    x = _cuda(_inputs(64, 4, 4, 128, 128, "bf16", seed=9))
    q, k = x["qkv"][:, :4], x["qkv"][:, 4:8]
    kw = dict(wq=x["wq"], wk=x["wk"])
    ref = fa.attention_qk_norm_rope(q, k, x["cos"], x["sin"], x["pos"], **kw)
    refb = fa.attention_qk_norm_rope_backward(x["gq"], x["gk"], x["cos"], x["sin"], x["pos"], q=q, k=k, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = fa.attention_qk_norm_rope(q, k, x["cos"], x["sin"], x["pos"], stream=side.cuda_stream, **kw)
    gotb = fa.attention_qk_norm_rope_backward(x["gq"], x["gk"], x["cos"], x["sin"], x["pos"], q=q, k=k, stream=side.cuda_stream, **kw)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got + gotb, ref + refb))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = fa.attention_qk_norm_rope(q, k, x["cos"], x["sin"], x["pos"], **kw)
        z = fa.attention_qk_norm_rope_backward(x["gq"], x["gk"], x["cos"], x["sin"], x["pos"], q=q, k=k, **kw)
    for flip in (1, -1):
        x["qkv"].mul_(flip)
        graph.replay()
    torch.cuda.synchronize()
    want = fa.attention_qk_norm_rope(q, k, x["cos"], x["sin"], x["pos"], **kw)
    wantb = fa.attention_qk_norm_rope_backward(x["gq"], x["gk"], x["cos"], x["sin"], x["pos"], q=q, k=k, **kw)
    assert all(torch.equal(a, b) for a, b in zip(y + z, want + wantb))


def test_refusals(fa):
    x = _cuda(_inputs(8, 4, 2, 64, 64, "bf16"))
    q, k, args = x["qkv"][:, :4], x["qkv"][:, 4:6], (x["cos"], x["sin"], x["pos"])
    for call in (lambda: fa.attention_qk_norm_rope(q.transpose(0, 1), k, *args),
                 lambda: fa.attention_qk_norm_rope(q, k.half(), *args),
                 lambda: fa.attention_qk_norm_rope(q, k[:4], *args),
                 lambda: fa.attention_qk_norm_rope(q, k, x["cos"].double(), x["sin"].double(), x["pos"]),
                 lambda: fa.attention_qk_norm_rope(q, k, x["cos"], x["sin"], x["pos"].long()),
                 lambda: fa.attention_qk_norm_rope(q, k, x["cos"], x["sin"], x["pos"][:, :4]),
                 lambda: fa.attention_qk_norm_rope(q, k, *args, wq=x["wq"]),
                 lambda: fa.attention_qk_norm_rope(q, k, *args, wq=x["wq"][:32], wk=x["wk"]),
                 lambda: fa.attention_qk_norm_rope(q, k, *args, sections=(16, 8)),
                 lambda: fa.attention_qk_norm_rope(q, k, *args, q_out=torch.empty(8, 3, 64, dtype=q.dtype, device="cuda")),
                 lambda: fa.attention_qk_norm_rope_backward(x["gq"], x["gk"], *args, wq=x["wq"], wk=x["wk"])):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(fa.FAError):  # rows of one token that overlap the next one's
        fa.attention_qk_norm_rope(torch.zeros(4 * 64, dtype=q.dtype, device="cuda").expand(8, -1).reshape(8, 4, 64)[:1].expand(8, 4, 64),
                                  k, *args)
    with pytest.raises(TypeError):
        fa.attention_qk_norm_rope(q.float(), k.float(), *args)
    assert _status(fa) == fa.FA_OK
