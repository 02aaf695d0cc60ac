"""Kernels that may be scheduled while the one before them ends wait for all that they read: work on other streams joined by
events, copies in front of a call, and graphs captured from streams that fork and join."""

import math

import numpy as np
import pytest
import torch

import oracle
from _gpu import f64

pytestmark = pytest.mark.gpu

B, H, HK, D, PAGE, MOST = 3, 4, 2, 128, 64, 8


@pytest.fixture(scope="module")
def fa():
    from _lib import load_fa
    m = load_fa()
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu-marked tests")
    return m


class Step:
    """A decoding step whose inputs are made late: by a chain of large products on one stream and a copy on another."""

    def __init__(self, fa, bits):
        g = torch.Generator().manual_seed(bits)
        self.fa = fa
        self.source = torch.randn(B, H + 2 * HK, D, generator=g).bfloat16()
        self.pinned = self.source.pin_memory()
        self.qkv = torch.zeros(B, H + 2 * HK, D, dtype=torch.bfloat16, device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.cos, self.sin = fa.attention_rope_table(MOST * PAGE, D)
        self.table = torch.arange(B * MOST, dtype=torch.int32, device="cuda").reshape(B, MOST)
        shape = (B * MOST, HK, PAGE, D if bits == 16 else D * 5 // 8)
        dtype = torch.bfloat16 if bits == 16 else torch.uint8
        self.caches = [torch.zeros(shape, dtype=dtype, device="cuda") for _ in range(2)]
        self.busy = torch.eye(2048, device="cuda")
        self.counts = torch.tensor([1.0, 70.0, 300.0], device="cuda")
        self.side = torch.cuda.Stream()

    def late(self):
        """What a device needs a millisecond for, and then the lengths, which come out of it: 1, 70
        and 300 keys, of which all but the new are 0."""
        x = self.busy
        for _ in range(8):
            x = x @ self.busy
        self.lens.copy_((x[0, 0] * self.counts).to(torch.int32))

    def calls(self):
        fa, q, k, v = self.fa, *self.qkv.split([H, HK, HK], 1)
        main = torch.cuda.current_stream()
        self.side.wait_stream(main)
        with torch.cuda.stream(self.side):
            self.late()
        self.qkv.copy_(self.pinned, non_blocking=True)     # a copy in front of the join
        main.wait_stream(self.side)
        qr = fa.attention_cache_append(k, v, *self.caches, self.table, self.lens, cos=self.cos, sin=self.sin, q=q)
        # the other stream reads what this one wrote
        self.side.wait_stream(main)
        with torch.cuda.stream(self.side):
            o1, l1 = fa.attention_decode_paged(qr, *self.caches, self.table, self.lens)
            rows = fa.attention_cache_gather(*self.caches, self.table, None, B, starts=self.lens - 1, dtype=torch.bfloat16)
        o2, l2 = fa.attention_decode_paged(qr, *self.caches, self.table, self.lens, max_seqlen_k=100000)
        main.wait_stream(self.side)
        return qr, o1, l1, o2, l2, rows[0], rows[1]

    def check(self, got, bits):
        qr, o1, l1, o2, l2, kr, vr = (f64(x) for x in got)
        lens = np.array([1, 70, 300])
        x = f64(self.source)
        q, k = (oracle.qk_norm_rope(y, None, f64(self.cos), f64(self.sin), lens - 1) for y in (x[:, :H], x[:, H:H + HK]))
        assert np.all(np.abs(qr - q) <= 2.0 ** -8 * np.abs(q) + 2.0 ** -15 * np.abs(x).max())
        if bits == 16:
            assert np.all(np.abs(kr - k) <= 2.0 ** -8 * np.abs(k) + 2.0 ** -15 * np.abs(x).max()) and np.array_equal(vr, x[:, H + HK:])
        for b, n in enumerate(lens):
            keys, values = np.zeros((n, HK, D)), np.zeros((n, HK, D))
            keys[-1], values[-1] = kr[b], vr[b]
            ref, lse = oracle.decode_paged(qr[b:b + 1], keys, values, 1 / math.sqrt(D))
            # the gathered rows of a 4-bit cache are rounded to bf16: 2^-8 of each key and value, in the scores too
            score = np.abs(lse).max() + np.log(n) + 1
            tol = 2.0 ** -7 * (1 + 2 * score) * np.abs(values).max() if bits == 4 else 2.0 ** -7 * np.abs(values).max()
            for o in (o1[b], o2[b]):
                assert np.abs(o - ref[0]).max() <= tol
        assert self.fa.fa_check_device_status(torch.cuda.current_stream().cuda_stream) == self.fa.FA_OK


@pytest.mark.parametrize("bits", [16, 4])
def test_streams_joined_by_events(fa, bits):
    s = Step(fa, bits)
    for _ in range(3):
        for c in s.caches:
            c.zero_()
        s.lens.zero_()
        s.qkv.zero_()
        got = s.calls()
        torch.cuda.synchronize()
        s.check(got, bits)


@pytest.mark.parametrize("bits", [16, 4])
def test_graph_captured_from_streams_that_fork_and_join(fa, bits):
    s = Step(fa, bits)
    s.calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.calls()
    for _ in range(3):
        for c in s.caches:
            c.zero_()
        s.lens.zero_()
        s.qkv.zero_()
        graph.replay()
        torch.cuda.synchronize()
        s.check(got, bits)
