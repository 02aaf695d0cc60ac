"""The operators around the attention that are measured: what each case is, its inputs, one pass in the plain form
(elementary torch operations) and through the package's entry points, the bytes and operations it cannot do without, and
its results in 64 bits.

Operators (the case's "op"):
  qk_fwd   per-head RMS norm of queries and keys and their position rotation, one pass
  qk_bwd   its gradients: the inputs' and the norm weights'
  append   new keys (normed, rotated) and values into a paged cache of 16-bit or 4-bit rows, the queries rotated along
  gather   rows of a paged cache back into packed [T, heads, d] arrays
  decode   attention of one or a few new queries per sequence over a paged cache, 16-bit or 4-bit

Paged cache: k and v are [pages, Hk, page_size, d] of the 16-bit type, or uint8 [pages, Hk, page_size, 5d/8].  A 4-bit block
of one page and head holds page_size rows of d/2 bytes of 4-bit numbers, then page_size rows of d/32 (scale, min) pairs of
fp16, one pair for each 32 features; a number n stands for n·scale + min.  With W = d/32, feature 32w + 8t + n (t < 4,
n < 8) of a key is nibble n of the row's 32-bit word t·W + w, and feature 32w + 4g + n (g < 8, n < 4) of a value is nibble n
of its 16-bit word g·W + w.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


def listed():
    return [
        # training: the queries and keys of the benchmark's causal step (4 x 8192 tokens, 16 heads), normed and rotated
        dict(name="qk_fwd_causal_n8k", op="qk_fwd", tokens=32768, hq=16, hk=16, d=128, dtype="bf16", norm=True, rot=128,
             interleaved=False, axes=1, seqs=4),
        # one prompt of an image and text: odd token count, shared key heads, time/height/width positions, slices of a
        # fused projection
        dict(name="qk_fwd_image_d64", op="qk_fwd", tokens=1171, hq=16, hk=4, d=64, dtype="fp16", norm=True, rot=64,
             interleaved=False, axes=3, seqs=1),
        # the same training step's backward
        dict(name="qk_bwd_causal_n8k", op="qk_bwd", tokens=32768, hq=16, hk=16, d=128, dtype="bf16", norm=True, rot=128,
             interleaved=False, axes=1, seqs=4),
        # a short fine-tuning batch: d = 64, half of each head rotated in neighbouring pairs
        dict(name="qk_bwd_partial_d64", op="qk_bwd", tokens=2051, hq=16, hk=8, d=64, dtype="fp16", norm=True, rot=32,
             interleaved=True, axes=1, seqs=3),
        # one decoding step of 16 sequences: a token each into 16-bit pages
        dict(name="append_step_b16", op="append", seqs=16, new=1, lmin=512, lmax=2048, hq=16, hk=16, d=128, dtype="bf16",
             bits=16, page=64, norm=True, rot=128, interleaved=False, axes=1),
        # ragged prompts of 128 to 4096 tokens into 4-bit pages
        dict(name="append_prompts_q4", op="append", seqs=16, new=0, lmin=128, lmax=4096, hq=32, hk=8, d=128, dtype="bf16",
             bits=4, page=64, norm=True, rot=128, interleaved=False, axes=1),
        # a cached prefix read back for a prompt that continues it
        dict(name="gather_prefix_16", op="gather", seqs=3, lmin=300, lmax=1500, hk=16, d=64, dtype="fp16", bits=16, page=16),
        # a whole 4-bit cache of 16 x 8192 keys read back
        dict(name="gather_b16_kv8k_q4", op="gather", seqs=16, lmin=8192, lmax=8192, hk=8, d=128, dtype="bf16", bits=4, page=64),
        # the smallest decoding call: one sequence, under a thousand keys
        dict(name="decode_one_short", op="decode", seqs=1, lmin=777, lmax=777, q=1, hq=16, hk=16, d=128, dtype="bf16", bits=16,
             page=64),
        # the benchmark's decoding batch, over pages
        dict(name="decode_b16_kv8k", op="decode", seqs=16, lmin=8192, lmax=8192, q=1, hq=16, hk=16, d=128, dtype="bf16", bits=16,
             page=64),
        # ragged batch over 4-bit pages with four query heads to a key head
        dict(name="decode_varlen_q4", op="decode", seqs=64, lmin=512, lmax=16384, q=1, hq=32, hk=8, d=128, dtype="bf16", bits=4,
             page=64),
        # one long sequence in 4 bits, four drafted tokens checked at once
        dict(name="decode_long_q4", op="decode", seqs=1, lmin=131071, lmax=131071, q=4, hq=32, hk=8, d=128, dtype="fp16", bits=4,
             page=128),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["qk_fwd", "qk_bwd", "append", "gather", "decode", "decode"])
    d = rng.choice([64, 128])
    c = dict(op=op, d=d, dtype=rng.choice(["bf16", "fp16"]))
    hk = rng.choice([1, 2, 3, 4, 8, 16])
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 8, 12) if g * hk <= 32])
    c.update(hk=hk)
    if op != "gather":
        c.update(hq=hk * group)
    if op in ("qk_fwd", "qk_bwd", "append"):
        c.update(norm=rng.random() < 0.7, rot=rng.choice([r for r in (32, 48, 64, 96, 128) if r <= d]),
                 interleaved=rng.random() < 0.4, axes=rng.choice([1, 1, 2, 3]))
    if op in ("qk_fwd", "qk_bwd"):
        c.update(tokens=log_int(1, 16384), seqs=1)
        return c
    c.update(bits=rng.choice([16, 4]), page=rng.choice([16, 32, 48, 64, 128, 256]))
    if op == "append":
        new = rng.choice([0, 1, 1, 3])
        c.update(seqs=rng.randint(1, 24), new=new, lmin=1, lmax=log_int(16, 1500))
    elif op == "gather":
        c.update(seqs=rng.randint(1, 16), lmin=0, lmax=log_int(16, 4096))
    else:
        lmax = log_int(16, 60000)
        most = max(1, 2_000_000 // (lmax * hk))
        c.update(seqs=rng.randint(1, min(40, most)), lmin=rng.choice([0, 1, lmax // 2]), lmax=lmax, q=rng.choice([1, 1, 2, 5]))
    return c


# ------------------------------------------------------------------------------------------------ inputs

def _sections(case):
    """How many of the rot/2 frequencies go by each axis' position, in multiples of 4; None for one axis."""
    n, a = case["rot"] // 2, case["axes"]
    if a == 1:
        return None
    if a == 2:
        first = (n // 2 + 3) // 4 * 4
        return (first, n - first)
    first = max(4, n // 16 * 4)
    second = max(4, (n - first) // 8 * 4)
    return (first, second, n - first - second)


def _lengths(case, seed=None):
    """The sequences' lengths: the same ones for every seed (so that outputs have one shape), in an order of its own."""
    lens = np.random.default_rng(1007).integers(case["lmin"], case["lmax"] + 1, size=case["seqs"])
    if seed is not None:
        np.random.default_rng(seed).shuffle(lens)
    return [max(int(x), case.get("new", 0)) for x in lens]


def _table(rows, rot):
    """cos and sin of position times frequency, in fp32, from 64-bit angles."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    ang = torch.arange(rows, dtype=torch.float64, device=DEV)[:, None] * freq
    return ang.cos().float(), ang.sin().float()


def _positions(case, T, g):
    """[axes, T] int32: places in the sequence, or for several axes text followed by the cells of an image."""
    t = torch.arange(T, device=DEV)
    if case["axes"] == 1:
        return (t % max(1, -(-T // case["seqs"]))).to(torch.int32)[None].contiguous()
    side = max(1, int(math.sqrt(max(1, T // 2))))
    cell = (t - T // 3).clamp(min=0)
    image = (t >= T // 3) & (cell < side * side)
    rows = [torch.where(image, torch.full_like(t, T // 3), t), torch.where(image, T // 3 + cell // side, t),
            torch.where(image, T // 3 + cell % side, t)]
    return torch.stack(rows[: case["axes"]] if case["axes"] == 3 else rows[1:]).to(torch.int32)


def _pages(case, lens, g):
    """A shuffled page table [B, most] (-1 behind each sequence's last page) and the number of pages."""
    ps = case["page"]
    need = torch.tensor([-(-x // ps) for x in lens])
    most, total = max(1, int(need.max())), int(need.sum()) + 3
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), most), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need.tolist()):
        table[b, :n] = perm[at: at + n]
        at += n
    return table, total


def _pack_numbers(n, value):
    """4-bit numbers [..., d] (uint8) as rows [..., d/2] of bytes in the cache's order."""
    d = n.shape[-1]
    lead, w = n.shape[:-1], d // 32
    inner = (8, 4) if value else (4, 8)
    n = n.reshape(*lead, w, *inner).transpose(-3, -2).reshape(*lead, d // 2, 2)
    return n[..., 0] | (n[..., 1] << 4)


def _quantise(x):
    """The numbers (uint8), fp16 scales and fp16 minima of 16-bit rows x [..., d], a pair for each 32 features."""
    v = x.float().reshape(*x.shape[:-1], -1, 32)
    lo, hi = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
    mn = lo.clamp(-65504.0, 65504.0).half()
    sc = ((hi - lo) / 15.0).clamp(max=65504.0).half()
    s = sc.float()
    n = torch.where(s > 0, ((v - mn.float()) / torch.where(s > 0, s, torch.ones_like(s))).round().clamp(0, 15), torch.zeros_like(v))
    return n.to(torch.uint8).reshape(x.shape), sc.squeeze(-1), mn.squeeze(-1)


def _cache(case, pages, g, value):
    """A cache full of keys (features of unlike sizes, as keys have) or values."""
    shape = (pages, case["hk"], case["page"], case["d"])
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    if not value:
        x *= torch.exp(0.5 * torch.randn(case["hk"], 1, case["d"], generator=g, device=DEV))
    x = x.to(TYPES[case["dtype"]])
    if case["bits"] == 16:
        return x
    n, sc, mn = _quantise(x)
    rows = _pack_numbers(n, value).reshape(pages, case["hk"], -1)
    pairs = torch.stack([sc, mn], -1).reshape(pages, case["hk"], -1).view(torch.uint8)
    return torch.cat([rows, pairs], -1).reshape(pages, case["hk"], case["page"], case["d"] * 5 // 8).contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt, d, op = TYPES[case["dtype"]], case["d"], case["op"]

    def rand(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dt)

    s = {"case": case, "op": op}
    if op in ("qk_fwd", "qk_bwd", "append"):
        s["wq"], s["wk"] = ((1 + 0.1 * rand(d).float()).to(dt) for _ in range(2)) if case["norm"] else (None, None)
    if op in ("qk_fwd", "qk_bwd"):
        T, hq, hk = case["tokens"], case["hq"], case["hk"]
        qkv = rand(T, hq + 2 * hk, d)  # one projection's output: q, k and v side by side
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["positions"] = _positions(case, T, g)
        s["cos"], s["sin"] = _table(int(s["positions"].max()) + 1, case["rot"])
        if op == "qk_bwd":
            s["dq"], s["dk"] = rand(T, hq, d), rand(T, hk, d)
        return s
    lens = _lengths(case, seed)
    if op == "append":
        new = [case["new"] or x for x in lens]
        T = sum(new)
        qkv = rand(T, case["hq"] + 2 * case["hk"], d)
        s["q"], s["k"], s["v"] = qkv.split([case["hq"], case["hk"], case["hk"]], 1)
        s["cu"] = None if case["new"] else torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
        s["positions"] = None if case["axes"] == 1 else _positions(dict(case, seqs=1), T, g)
        s["cos"], s["sin"] = _table(max(max(lens), T) + 1, case["rot"])
        if case["bits"] == 4:  # to read the new rows back
            s["starts"] = torch.tensor([x - n for x, n in zip(lens, new)], dtype=torch.int32, device=DEV)
            s["cu_read"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
    elif op == "gather":
        s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
        s["total"] = max(1, sum(lens))
        s["into"] = [torch.zeros(s["total"], case["hk"], d, dtype=dt, device=DEV) for _ in range(2)]
    else:
        s["q"] = rand(case["seqs"], case["q"], case["hq"], d)
        s["most"] = case["lmax"]
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["table"], pages = _pages(case, lens, g)
    s["k_cache"], s["v_cache"] = _cache(case, pages, g, False), _cache(case, pages, g, True)
    return s


# ------------------------------------------------------------------------------------------------ the plain form

def _angles(s, positions):
    """fp32 cos and sin [T, 1, rot/2] of each token: frequency i goes by the position of its section's axis."""
    sec = _sections(s["case"])
    if sec is None:
        at = positions[0].long()
        return s["cos"][at][:, None], s["sin"][at][:, None]
    axis = torch.repeat_interleave(torch.arange(len(sec), device=DEV), torch.tensor(sec, device=DEV))
    at, i = positions[axis].long().t(), torch.arange(axis.numel(), device=DEV)
    return s["cos"][at, i][:, None], s["sin"][at, i][:, None]


def _pairs(x, case):
    """The two partners of each rotated pair, and what is not rotated."""
    r = case["rot"]
    if case["interleaved"]:
        return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    return x[..., : r // 2], x[..., r // 2: r], x[..., r:]


def _join(a, b, rest, case):
    if case["interleaved"]:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _norm_rotate(x, w, cos, sin, case):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    a, b, rest = _pairs(x, case)
    return _join(a * cos - b * sin, b * cos + a * sin, rest, case)


def _norm_rotate_grad(dy, x, w, cos, sin, case):
    a, b, rest = _pairs(dy.float(), case)
    g = _join(a * cos + b * sin, b * cos - a * sin, rest, case)
    if w is None:
        return g, None
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n, gw = x * r, g * w.float()
    return r * (gw - n * (gw * n).mean(-1, keepdim=True)), (g * n).sum((0, 1))


def _numbers(rows, value):
    """fp32 numbers [..., d] of 4-bit rows [..., d/2] in the cache's order."""
    lead, d = rows.shape[:-1], rows.shape[-1] * 2
    inner = (8, d // 32, 4) if value else (4, d // 32, 8)
    n = torch.stack([rows & 15, rows >> 4], -1).reshape(*lead, *inner)
    return n.transpose(-3, -2).reshape(*lead, d).float()


def _values(blocks, page, d, value):
    """fp32 [..., Hk, page, d] of cache blocks [..., Hk, page, row]."""
    if blocks.dtype != torch.uint8:
        return blocks.float()
    flat = blocks.flatten(-2)
    rows = flat[..., : page * d // 2].unflatten(-1, (page, d // 2))
    pairs = flat[..., page * d // 2:].contiguous().view(torch.float16).unflatten(-1, (page, d // 32, 2)).float()
    n = _numbers(rows, value).unflatten(-1, (d // 32, 32))
    return (n * pairs[..., :1] + pairs[..., 1:]).flatten(-2)


def _plain_append(s):
    case, lens = s["case"], s["lens"].long()
    T, B, ps, d = s["k"].shape[0], case["seqs"], case["page"], case["d"]
    t = torch.arange(T, device=DEV)
    if s["cu"] is None:
        seq, n, i = t // (T // B), torch.full_like(t, T // B), t % (T // B)
    else:
        cu = s["cu"].long()
        seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
        n, i = (cu[1:] - cu[:-1])[seq], t - cu[seq]
    at = lens[seq] - n + i
    cos, sin = _angles(s, at[None] if s["positions"] is None else s["positions"])
    dt = s["q"].dtype
    q = _norm_rotate(s["q"], s["wq"], cos, sin, case).to(dt)
    k = _norm_rotate(s["k"], s["wk"], cos, sin, case).to(dt)
    page, slot = s["table"][seq, at // ps].long(), at % ps
    if case["bits"] == 16:
        s["k_cache"][page, :, slot] = k
        s["v_cache"][page, :, slot] = s["v"]
        return q, s["k_cache"], s["v_cache"]
    out, head = [q], torch.arange(case["hk"], device=DEV)[None, :, None]
    for cache, x, value in ((s["k_cache"], k, False), (s["v_cache"], s["v"], True)):
        n, sc, mn = _quantise(x)
        flat = cache.view(cache.shape[0], cache.shape[1], -1)
        first = (slot * (d // 2))[:, None, None] + torch.arange(d // 2, device=DEV)
        flat[page[:, None, None], head, first] = _pack_numbers(n, value)
        pairs = torch.stack([sc, mn], -1).flatten(-2).view(torch.uint8)
        second = (ps * (d // 2) + slot * (d // 8))[:, None, None] + torch.arange(d // 8, device=DEV)
        flat[page[:, None, None], head, second] = pairs
        v = n.float().unflatten(-1, (-1, 32)) * sc.float()[..., None] + mn.float()[..., None]
        out.append(v.flatten(-2).to(dt))
    return tuple(out)


def _plain_gather(s):
    case, cu = s["case"], s["cu"].long()
    ps, d, dt = case["page"], case["d"], TYPES[case["dtype"]]
    t = torch.arange(s["total"], device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=case["seqs"] - 1)
    at, owned = t - cu[seq], t < cu[-1]
    page = s["table"][seq, (at // ps).clamp(max=s["table"].shape[1] - 1)].long().clamp(min=0)
    for cache, into, value in ((s["k_cache"], s["into"][0], False), (s["v_cache"], s["into"][1], True)):
        if case["bits"] == 16:
            rows = cache[page, :, at % ps]
        else:
            head = torch.arange(case["hk"], device=DEV)[None, :, None]
            flat = cache.view(cache.shape[0], cache.shape[1], -1)
            slot = (at % ps)[:, None, None]
            numbers = _numbers(flat[page[:, None, None], head, slot * (d // 2) + torch.arange(d // 2, device=DEV)], value)
            pairs = flat[page[:, None, None], head, ps * (d // 2) + slot * (d // 8) + torch.arange(d // 8, device=DEV)]
            pairs = pairs.view(torch.float16).unflatten(-1, (d // 32, 2)).float()
            rows = (numbers.unflatten(-1, (d // 32, 32)) * pairs[..., :1] + pairs[..., 1:]).flatten(-2).to(dt)
        into.copy_(torch.where(owned[:, None, None], rows, into))
    return tuple(s["into"])


def _plain_decode(s):
    case, q = s["case"], s["q"]
    B, nq, hq, d = q.shape
    hk, ps = case["hk"], case["page"]
    group, most = hq // hk, s["table"].shape[1] * ps
    pages = s["table"].long().clamp(min=0)
    k = _values(s["k_cache"][pages], ps, d, False).transpose(1, 2).reshape(B, hk, most, d)
    v = _values(s["v_cache"][pages], ps, d, True).transpose(1, 2).reshape(B, hk, most, d)
    x = q.float().reshape(B, nq, hk, group, d).permute(0, 2, 1, 3, 4).reshape(B, hk, nq * group, d)
    sc = torch.matmul(x, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    # query i of a sequence, the last nq of its tokens, sees the keys up to its own place
    last = s["lens"].long()[:, None] - nq + torch.arange(nq, device=DEV)
    seen = torch.arange(most, device=DEV) <= last[..., None]
    sc = sc.masked_fill(~seen.repeat_interleave(group, 1)[:, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (m + torch.log(total)).squeeze(-1)
    o = o.reshape(B, hk, nq, group, d).permute(0, 2, 1, 3, 4).reshape(B, nq, hq, d).to(q.dtype)
    return o, lse.reshape(B, hk, nq, group).permute(0, 2, 1, 3).reshape(B, nq, hq).contiguous()


def _plain(s):
    case = s["case"]
    if s["op"] == "qk_fwd":
        cos, sin = _angles(s, s["positions"])
        return tuple(_norm_rotate(x, w, cos, sin, case).to(x.dtype) for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])))
    if s["op"] == "qk_bwd":
        cos, sin = _angles(s, s["positions"])
        dq, dwq = _norm_rotate_grad(s["dq"], s["q"], s["wq"], cos, sin, case)
        dk, dwk = _norm_rotate_grad(s["dk"], s["k"], s["wk"], cos, sin, case)
        return (dq.to(s["q"].dtype), dk.to(s["k"].dtype)) + ((dwq, dwk) if case["norm"] else ())
    return {"append": _plain_append, "gather": _plain_gather, "decode": _plain_decode}[s["op"]](s)


# ------------------------------------------------------------------------------------------------ the package's calls

def _own(s):
    import exact_io_aware_90_b200 as fa
    case = s["case"]
    if s["op"] == "qk_fwd":
        return fa.attention_qk_norm_rope(s["q"], s["k"], s["cos"], s["sin"], s["positions"], wq=s["wq"], wk=s["wk"], eps=EPS,
                                         interleaved=case["interleaved"], sections=_sections(case))
    if s["op"] == "qk_bwd":
        norm = dict(q=s["q"], k=s["k"], wq=s["wq"], wk=s["wk"], eps=EPS) if case["norm"] else {}
        got = fa.attention_qk_norm_rope_backward(s["dq"], s["dk"], s["cos"], s["sin"], s["positions"],
                                                 interleaved=case["interleaved"], sections=_sections(case), **norm)
        return got if case["norm"] else got[:2]
    if s["op"] == "append":
        q = fa.attention_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], cos=s["cos"],
                                      sin=s["sin"], positions=s["positions"], q=s["q"], wq=s["wq"], wk=s["wk"], eps=EPS,
                                      interleaved=case["interleaved"], sections=_sections(case), cu_seqlens=s["cu"])
        if case["bits"] == 16:
            return q, s["k_cache"], s["v_cache"]
        return (q, *fa.attention_cache_gather(s["k_cache"], s["v_cache"], s["table"], s["cu_read"], s["k"].shape[0],
                                              starts=s["starts"], dtype=q.dtype))
    if s["op"] == "gather":
        return fa.attention_cache_gather(s["k_cache"], s["v_cache"], s["table"], s["cu"], s["total"], dtype=TYPES[case["dtype"]],
                                         k=s["into"][0], v=s["into"][1])
    q = s["q"]
    return fa.attention_decode_paged(q, s["k_cache"], s["v_cache"], s["table"], s["lens"], max_seqlen_k=s["most"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------ work and 64 bits

def work(case):
    d, op = case["d"], case["op"]
    if op in ("qk_fwd", "qk_bwd"):
        T, h = case["tokens"], case["hq"] + case["hk"]
        arrays = 2 if op == "qk_fwd" or not case["norm"] else 3
        return {"bytes": T * h * d * 2 * arrays + T * 4 * case["axes"] + T // case["seqs"] * case["rot"] * 4,
                "flops": T * h * d * (8 if op == "qk_fwd" else 16)}
    row = d * 2 if case["bits"] == 16 else d * 5 // 8
    keys = sum(_lengths(case))
    if op == "append":
        T = case["seqs"] * case["new"] or keys
        back = 0 if case["bits"] == 16 else 2 * case["hk"] * (row + 2 * d)  # the new rows are read back
        return {"bytes": T * (2 * d * (2 * case["hq"] + 2 * case["hk"]) + 2 * case["hk"] * row + back),
                "flops": T * (case["hq"] + 2 * case["hk"]) * d * 8}
    if op == "gather":
        return {"bytes": keys * case["hk"] * 2 * (row + 2 * d) + 4 * case["seqs"], "flops": keys * case["hk"] * 2 * d * 2}
    return {"bytes": keys * case["hk"] * 2 * row + case["seqs"] * case["q"] * case["hq"] * (4 * d + 4),
            "flops": 4 * keys * case["hq"] * case["q"] * d}


def _exact_rotated(x, w, turn, case):
    """64-bit norm and rotation of x [T, H, d]; turn: complex [T, rot/2] of cos + i sin."""
    y = x.double()
    if w is not None:
        y = y / (y.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    r = case["rot"]
    z = y[..., :r].unflatten(-1, (r // 2, 2)) if case["interleaved"] else y[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn[:, None])
    z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, y[..., r:]], -1)


def _turn(s, positions):
    case, cols = s["case"], []
    sec, first = _sections(case) or (case["rot"] // 2,), 0
    for a, n in enumerate(sec):
        p = positions[a].long()
        cols.append(torch.complex(s["cos"][p, first:first + n].double(), s["sin"][p, first:first + n].double()))
        first += n
    return torch.cat(cols, 1)


def _exact_rows(cache, page, slot, case, value):
    """64-bit rows [n, Hk, d] of a cache at (page, slot): feature by feature through the layout's formula."""
    d, ps = case["d"], case["page"]
    if case["bits"] == 16:
        return cache[page, :, slot].double()
    f = np.arange(d)
    w, rest, words = f // 32, f % 32, d // 32
    nib = ((rest // 4) * words + w) * 4 + rest % 4 if value else ((rest // 8) * words + w) * 8 + rest % 8
    flat = cache.reshape(cache.shape[0], cache.shape[1], -1)
    nib = torch.from_numpy(nib).to(DEV)
    h = torch.arange(case["hk"], device=DEV)[None, :, None]
    p, q = page[:, None, None], slot[:, None, None]
    n = (flat[p, h, q * (d // 2) + nib // 2].long() >> (nib % 2 * 4)) & 15
    half = flat[:, :, ps * (d // 2):].contiguous().view(torch.float16)
    g = 2 * torch.from_numpy(w).to(DEV)
    return n.double() * half[p, h, q * (d // 16) + g].double() + half[p, h, q * (d // 16) + g + 1].double()


def _exact_four_bits(x):
    """64-bit values that 16-bit rows stand for once they are held in 4 bits."""
    v = x.double().unflatten(-1, (-1, 32))
    lo, hi = v.min(-1, keepdim=True).values, v.max(-1, keepdim=True).values
    mn = lo.clamp(-65504, 65504).half().double()
    sc = ((hi - lo) / 15).clamp(max=65504).half().double()
    n = torch.round((v - mn) / sc).nan_to_num(0, 0, 0).clamp(0, 15)
    return (n * sc + mn).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    dt = TYPES[case["dtype"]]
    if case["op"] == "qk_fwd":
        turn = _turn(s, s["positions"])
        return tuple(_exact_rotated(s[n], s["w" + n], turn, case) for n in "qk")
    if case["op"] == "qk_bwd":
        turn, grads, weights = _turn(s, s["positions"]).conj(), [], []
        for n in "qk":
            g, w = _exact_rotated(s["d" + n], None, turn, case), s["w" + n]
            if w is None:
                grads.append(g)
                continue
            # dx_j = sum_i g_i w_i d(x_i / rms)/dx_j = (g_j w_j - x_j sum_i(g_i w_i x_i) / (d rms^2)) / rms
            x = s[n].double()
            ms = x.pow(2).mean(-1, keepdim=True) + EPS
            weights.append((g * x / ms.sqrt()).flatten(0, 1).sum(0))
            g = g * w.double()
            grads.append((g - x * (g * x).sum(-1, keepdim=True) / (case["d"] * ms)) / ms.sqrt())
        return (*grads, *weights)
    lens = s["lens"].tolist()
    table, ps = s["table"].long(), case["page"]
    if case["op"] == "append":
        T, B = s["k"].shape[0], case["seqs"]
        cu = [T // B * b for b in range(B + 1)] if s["cu"] is None else s["cu"].tolist()
        at = torch.cat([torch.arange(lens[b] - cu[b + 1] + cu[b], lens[b], device=DEV) for b in range(B)])
        seq = torch.cat([torch.full((cu[b + 1] - cu[b],), b, device=DEV) for b in range(B)])
        turn = _turn(s, at[None] if s["positions"] is None else s["positions"])
        q, k = (_exact_rotated(s[n], s["w" + n], turn, case) for n in "qk")
        if case["bits"] == 4:  # a row is rounded to 16 bits before it is held in 4
            return q, _exact_four_bits(k.to(dt)), _exact_four_bits(s["v"])
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        kc[table[seq, at // ps], :, at % ps] = k
        vc[table[seq, at // ps], :, at % ps] = s["v"].double()
        return q, kc, vc
    if case["op"] == "gather":
        out = [torch.zeros(s["total"], case["hk"], case["d"], dtype=torch.float64, device=DEV) for _ in range(2)]
        first = 0
        for b, n in enumerate(lens):
            t = torch.arange(n, device=DEV)
            for x, cache, value in zip(out, (s["k_cache"], s["v_cache"]), (False, True)):
                x[first:first + n] = _exact_rows(cache, table[b, t // ps], t % ps, case, value)
            first += n
        return tuple(out)
    B, nq, hq, d = s["q"].shape
    hk = case["hk"]
    o = torch.zeros(B, nq, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((B, nq, hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        t = torch.arange(n, device=DEV)
        k, v = (_exact_rows(c, table[b, t // ps], t % ps, case, w).repeat_interleave(hq // hk, 1)
                for c, w in ((s["k_cache"], False), (s["v_cache"], True)))
        for i in range(nq):
            m = n - nq + i + 1
            if m > 0:
                a = torch.einsum("hd,nhd->hn", s["q"][b, i].double(), k[:m]) / math.sqrt(d)
                lse[b, i] = torch.logsumexp(a, -1)
                o[b, i] = torch.einsum("hn,nhd->hd", torch.softmax(a, -1), v[:m])
    return o, lse
