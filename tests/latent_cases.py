"""Shared helpers of the latent attention tests: caches in use, and plain 64-bit
implementations written from the formulas (per sequence, no paging).

Tolerances (derived, not fitted), both forms of the attention.  With u = 2^-8,
bf16's largest relative rounding error:
- Weights enter the second product rounded to bf16.  Where the sum takes the
  rounded ones, sum_j p_j (1 + e_j) v_j / sum_j p_j (1 + e_j) with |e_j| <= u is
  off by at most u (sum_j p_j |v_j| + |o|) / (1 - u); where it takes the
  unrounded ones, by u sum_j p_j |v_j|, which is less.
- The result's own rounding: u |o| (of the computed one: times 1 + 2 u).
- Scores: at most 53 additions of exact products one after another in fp32 (36
  steps of the tensor core and 16 products within one, each possibly truncated:
  2^-23), so a score is off by d = 2^-17 S, S = scale sum_i |q_i k_i| at its
  largest; exponentials and the arithmetic around them add 2^-20 (2 + max|s|).
  That moves every weight by as much, and the result by at most twice that
  times sum_j p_j |v_j|.
- Sums over n keys: (n / 16 + 64) additions in fp32, 2^-23 each, twice.
"""
from __future__ import annotations

import math

import torch

import gated_deltanet_linear_mixer_gb300 as gdn

U = 2.0 ** -8


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


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make_cache(d, kv_lens, seed, spare=3, first_page=0):
    """Pages in random order holding random rows for kv_lens tokens of each sequence; rows past a
    sequence's end and unused pages are NaN.  first_page: pages before it are not used."""
    g = gen(seed)
    b = d.page_size
    need = [-(-max(n, 0) // b) for n in kv_lens]
    n_pages = first_page + sum(need) + spare
    order = (torch.randperm(sum(need) + spare, generator=g, device="cuda") + first_page).tolist()
    table = torch.full((len(kv_lens), max(need + [1])), -1, dtype=torch.int32)
    rows = torch.full((n_pages, b, d.latent_dim + d.rope_dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    at = 0
    for i, n in enumerate(need):
        for j in range(n):
            p = order[at]
            at += 1
            table[i, j] = p
            k = min(b, kv_lens[i] - j * b)
            rows[p, :k] = torch.randn(k, rows.shape[2], generator=g, device="cuda").bfloat16()
    return gdn.LatentCache(d, rows), table.cuda()


def line(cache, table, i, n):
    """Sequence i's first n rows in 64 bits, and which of them are mapped."""
    b = cache.rows.shape[1]
    pages = table[i, : -(-n // b)].long()
    ok = (pages >= 0) & (pages < cache.n_pages)
    x = cache.rows[pages.clamp(0, cache.n_pages - 1)].flatten(0, 1)[:n].double()
    return x, ok.repeat_interleave(b)[:n]


def attend(q, k, v, scale, start, mapped=None):
    """Causal attention in 64 bits of queries at positions start.. : q [c, h, d], k [n, h, d], v [n, h,
    e].  Returns the result [c, h, e] and its tolerance."""
    c, n = q.shape[0], k.shape[0]
    if n == 0:
        z = q.new_zeros(c, q.shape[1], v.shape[2])
        return z, z
    hide = torch.arange(n, device="cuda") > torch.arange(start, start + c, device="cuda")[:, None]
    if mapped is not None:
        hide = hide | ~mapped
    k, v = torch.where(torch.isfinite(k), k, 0.0), torch.where(torch.isfinite(v), v, 0.0)
    s = torch.einsum("qhd,khd->hqk", q, k) * scale
    size = torch.einsum("qhd,khd->hqk", q.abs(), k.abs()) * scale
    p = torch.softmax(s.masked_fill(hide, -math.inf), -1)
    p = torch.where(hide.all(-1)[:, None], 0.0, p)
    o = torch.einsum("hqk,khe->qhe", p, v)
    weight = torch.einsum("hqk,khe->qhe", p, v.abs())
    seen = ~hide
    most = torch.where(seen, size, 0.0).amax(-1).transpose(0, 1)[..., None]
    high = torch.where(seen, s.abs(), 0.0).amax(-1).transpose(0, 1)[..., None]
    rel = 2 * (2.0 ** -17 * most + 2.0 ** -20 * (2 + high)) + 2 * (n / 16 + 64) * 2.0 ** -23
    return o, U * (weight + o.abs()) / (1 - U) + U * (1 + 2 * U) * o.abs() + rel * weight


def absorbed(d, cache, counts, kv_lens, table, q):
    """The absorbed form in 64 bits, and its tolerance."""
    outs, tols, at = [], [], 0
    scale = d.c().scale
    for i, (c, n) in enumerate(zip(counts, kv_lens)):
        x, ok = line(cache, table, i, min(max(n, 0), table.shape[1] * d.page_size))
        x = x[:, None].expand(-1, q.shape[1], -1)
        o, t = attend(q[at:at + c].double(), x, x[..., :d.latent_dim], scale, n - c, ok)
        outs.append(o)
        tols.append(t)
        at += c
    return torch.cat(outs), torch.cat(tols)


def expanded(d, counts, kv_lens, q, k, k_rope, v):
    """The expanded form in 64 bits, and its tolerance."""
    outs, tols, a, b = [], [], 0, 0
    for c, n in zip(counts, kv_lens):
        kk = torch.cat([k[b:b + n].double(), k_rope[b:b + n, None].double().expand(-1, k.shape[1], -1)], -1)
        o, t = attend(q[a:a + c].double(), kk, v[b:b + n].double(), d.c().scale, n - c)
        outs.append(o)
        tols.append(t)
        a, b = a + c, b + n
    return torch.cat(outs), torch.cat(tols)


def check(got, want, tol):
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (
        f"{int(bad.sum())} of {bad.numel()} off, the worst {float((off / tol.clamp(min=1e-300)).nan_to_num(1e9).max()):.2f} x its "
        f"tolerance, first at {bad.nonzero()[0].tolist()}: {float(got[tuple(bad.nonzero()[0])])} for "
        f"{float(want[tuple(bad.nonzero()[0])])}")


def rope_table(n, style=None):
    inv = 10000.0 ** (-torch.arange(0, 64, 2, device="cuda", dtype=torch.float64) / 64)
    ang = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], -1).float().contiguous()


def turn(x, table, style):
    """x [T, h, 64] turned by table's rows [T, 64], in 64 bits; and what a result's terms amount to."""
    x = x.double()
    c, s = table.double()[:, None].chunk(2, -1)
    a, b = x.chunk(2, -1) if style == "half" else (x[..., 0::2], x[..., 1::2])
    parts, sizes = (a * c - b * s, b * c + a * s), ((a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs())
    if style == "half":
        return torch.cat(parts, -1), torch.cat(sizes, -1)
    return torch.stack(parts, -1).flatten(-2), torch.stack(sizes, -1).flatten(-2)
