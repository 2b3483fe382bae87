"""Shared helpers of the paged-cache tests: caches in use, and plain 64-bit
implementations written from the formulas (per sequence, per head, no paging).

Tolerances (derived, not fitted):
- Cached values are code * scale, exact in 64 bits, so both sides read the same
  keys and values.
- Attention with bf16 activations: probabilities enter the second product as
  f16 (relative error 2^-11 each, and below 2^-14 of the largest at most 2^-25
  of it), everything else is fp32 (scores to ~1e-5), so |error| <= 2^-9 sum_j
  p_j |v_j|, plus half a bf16 ulp of the result, at most 2^-8 of it.
- With fp32 activations queries and probabilities are f16 pairs (22 bits), sums
  fp32: |error| <= (2^-18 + 2^-20 S) sum_j p_j |v_j| with S the largest
  scale sum_i |q_i k_i| of the row (a score's error moves every p_j by it).
"""
from __future__ import annotations

import math
import random

import torch

import gated_deltanet_linear_mixer_gb300 as gdn

QMAX = {"int8": 127.0, "e4m3": 448.0}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def cu_of(counts):
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    host = torch.tensor(cu, dtype=torch.int32)
    return host.cuda(), host


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make_cache(d, kv_lens, seed, spare=3, poison=True):
    """Pages in random order holding random codes for kv_lens tokens of each sequence; rows past a
    sequence's end, unused pages and their scales hold NaN patterns (0x7F, 0xFF codes)."""
    g = gen(seed)
    b = d.page_size
    need = [-(-n // b) for n in kv_lens]
    n_pages = sum(need) + spare
    order = torch.randperm(n_pages, generator=g, device="cuda").tolist()
    table = torch.full((len(kv_lens), max(need + [1])), -1, dtype=torch.int32)
    at = 0
    used = {}
    for i, n in enumerate(need):
        for j in range(n):
            table[i, j] = order[at]
            used[order[at]] = min(b, kv_lens[i] - j * b)
            at += 1
    shape = (n_pages, d.n_kv_heads, b, d.head_dim)

    def codes():
        x = torch.randn(shape, generator=g, device="cuda") * (QMAX[d.cache] / 4)
        x = x.clamp(-QMAX[d.cache], QMAX[d.cache])
        x = x.round().to(torch.int8) if d.cache == "int8" else x.to(CODE["e4m3"])
        if poison:
            raw = x.view(torch.int8)
            rows = torch.tensor([used.get(p, 0) for p in range(n_pages)], device="cuda")
            dead = torch.arange(b, device="cuda")[None] >= rows[:, None]
            raw.masked_fill_(dead[:, None, :, None], 0x7F)
            raw[:, :, :, ::2].masked_fill_(dead[:, None, :, None], -1)
        return x.contiguous()

    def scales(centre):
        x = torch.randn(shape[:2], generator=g, device="cuda").mul(0.3).exp()
        x = x * (4 * centre / QMAX[d.cache])
        if poison:
            dead = [p for p in range(n_pages) if p not in used]
            x[dead] = float("nan")
        return x.contiguous()

    cache = gdn.KVCache(d, codes(), codes(), scales(1.0), scales(0.5))
    return cache, table.cuda()


def line(d, cache, table, name, i, length):
    """Sequence i's first `length` cached values in 64 bits, [length, Hkv, D]."""
    b = d.page_size
    pages = table[i, : -(-length // b)].long()
    x = getattr(cache, name)[pages].double()
    x = x * getattr(cache, name + "_scale")[pages].double()[:, :, None, None]
    return x.transpose(1, 2).reshape(-1, d.n_kv_heads, d.head_dim)[:length]


def attention_ref(d, cache, table, counts, kv_lens, q):
    """(out, sum_j p_j |v_j|, S) in 64 bits; out is zero for rows that see nothing."""
    outs, sizes, ss, begin = [], [], [], 0
    g = d.n_q_heads // d.n_kv_heads
    scale = d.head_dim ** -0.5 if d.scale is None else d.scale
    for i, (c, kv) in enumerate(zip(counts, kv_lens)):
        qi = q[begin:begin + c].double()
        begin += c
        if c == 0:
            continue
        n = max(kv, 0)
        k = line(d, cache, table, "k", i, n).repeat_interleave(g, 1)
        v = line(d, cache, table, "v", i, n).repeat_interleave(g, 1)
        pos = torch.arange(kv - c, kv, device="cuda")
        j = torch.arange(n, device="cuda")
        see = j[None] <= pos[:, None]
        if d.window:
            see &= j[None] > pos[:, None] - d.window
        x = torch.einsum("qhd,khd->hqk", qi, k) * scale
        x = x.masked_fill(~see, -math.inf)
        top = x.amax(-1, keepdim=True) if n else torch.zeros(d.n_q_heads, c, 1, device="cuda").double()
        top = torch.where(torch.isfinite(top), top, 0.0)
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True)
        p = torch.where(total > 0, p / total.clamp(min=1e-300), 0.0)
        outs.append(torch.einsum("hqk,khd->qhd", p, v))
        sizes.append(torch.einsum("hqk,khd->qhd", p, v.abs()))
        s = torch.einsum("qhd,khd->hqk", qi.abs(), k.abs()) * scale
        s = s.amax(-1) if n else torch.zeros(d.n_q_heads, c, device="cuda").double()
        ss.append(s.t()[..., None])
    return torch.cat(outs), torch.cat(sizes), torch.cat(ss)


def attention_excess(d, got, ref, size, s):
    """How many tolerances the worst element is off."""
    got = got.double()
    if d.dtype == torch.bfloat16:
        tol = 2.0 ** -9 * size + 2.0 ** -8 * got.abs()
    else:
        tol = (2.0 ** -18 + 2.0 ** -20 * s) * size
    bad = (got - ref).abs()
    assert torch.isfinite(got).all()
    return float((bad / tol.clamp(min=1e-30)).max()) if bad.numel() else 0.0


def lengths(seed, n, q_hi, ctx_hi, q_lo=1):
    r = random.Random(seed)
    qs = [r.randint(q_lo, q_hi) for _ in range(n)]
    return qs, [q + r.randint(0, ctx_hi) for q in qs]


def rope_table(rows, dim):
    inv = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * inv[None]
    return torch.cat([ang.cos(), ang.sin()], -1).float().cuda()


def turn(x, rows, style):
    """x [T, H, D] rotated by rows [T, r] (cosines | sines), in x's precision."""
    r = rows.shape[1]
    c, s = (t[:, None].to(x.dtype) for t in rows.chunk(2, -1))
    y = x.clone()
    if style == "half":
        a, b = x[..., : r // 2], x[..., r // 2: r]
        y[..., : r // 2], y[..., r // 2: r] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * s, b * c + a * s
    return y
