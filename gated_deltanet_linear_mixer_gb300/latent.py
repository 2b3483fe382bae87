"""Latent attention over a paged cache of latents, in both its forms, and copies of cache pages.

A layer of this kind keeps one vector a token: a normalised latent that the keys
and values of all heads are projections of, and a position key that all heads
share.  Like the rest of the binding this only marshals arguments
(``csrc/gdn_bind.cpp`` checks them); ``include/gdn.h`` states layouts, formulas
and errors.  Outputs share no memory with inputs, but for latent_append's two in-place forms
(``q_out`` is ``q_rope``, ``rows_out`` is a contiguous ``c``): else ``ValueError`` or ``GDNError``.

A step of single tokens or drafts, in the absorbed form (``w_uk`` [H, nope,
latent] and ``w_uv`` [H, latent, v] are the halves of the up projection)::

    d = LatentDims(32, 512)
    cache = LatentCache.empty(d, n_pages)
    ql = torch.empty(T, 32, 576)                 # queries in latent space | position part
    latent_append(d, cache, cu_seqlens, kv_lens, block_table, c, norm_w=w, rope=rope,
                  q_rope=q[..., 128:], q_out=ql[..., 512:])
    ql[..., :512] = torch.einsum("thn,hnc->thc", q[..., :128], w_uk)
    o = latent_attention(d, cache, cu_seqlens, kv_lens, block_table, ql)
    o = torch.einsum("thc,hcv->thv", o, w_uv)

A prompt, in the expanded form (behind a cached prefix, ``rows`` are those of the
whole sequences, from ``latent_read``)::

    rows = torch.empty(T, 576)
    latent_append(..., q_rope=q[..., 128:], q_out=q[..., 128:], rows_out=rows)
    kv = (rows[:, :512] @ w_ukv).view(T, 32, 256)
    o = expanded_attention(d, cu_seqlens, cu_seqlens, q, kv[..., :128], rows[:, 512:], kv[..., 128:])
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _check, _LatentDims, _t, load
from . import paged
from .paged import ROPE_STYLES, KVCache, _pair


@dataclass(frozen=True)
class LatentDims:
    """Geometry of one latent attention layer and its cache: heads, latent and position-key
    channels, tokens per page, rotation, a head's channels in the expanded form, softmax scale
    (None: (nope_dim + rope_dim)^-1/2, which both forms share), the norm's eps."""
    n_heads: int
    latent_dim: int = 512
    rope_dim: int = 64
    page_size: int = 64
    rope_style: str = "half"
    nope_dim: int = 128
    v_dim: int = 128
    scale: float | None = None
    norm_eps: float = 1e-6

    def c(self) -> _LatentDims:
        got = self.__dict__.get("_c")
        if got is None:
            if self.rope_style not in ROPE_STYLES:
                raise ValueError("rope_style must be 'half' or 'interleaved'")
            scale = (self.nope_dim + self.rope_dim) ** -0.5 if self.scale is None else self.scale
            got = _LatentDims(self.n_heads, self.latent_dim, self.rope_dim, self.page_size,
                              ROPE_STYLES[self.rope_style], self.nope_dim, self.v_dim, scale, self.norm_eps)
            object.__setattr__(self, "_c", got)
        return got

    def address(self) -> int:
        """Where the C struct of these dimensions lies, for as long as they do."""
        return ctypes.addressof(self.c())

    def __getstate__(self):
        """Copies and pickles hold the fields alone: the C struct belongs to one object."""
        return {name: getattr(self, name) for name in self.__dataclass_fields__}


class LatentCache:
    """The pages of one layer: rows [n_pages, page_size, latent_dim + rope_dim] bf16.  Holds the
    tensor it is given; a call takes the one that it holds then."""

    def __init__(self, d: LatentDims, rows):
        d.c()
        if not isinstance(rows, torch.Tensor):
            raise TypeError("rows must be a torch.Tensor")
        n = int(rows.shape[0]) if rows.dim() else 0
        _t(rows, "rows", torch.bfloat16, (n, d.page_size, d.latent_dim + d.rope_dim))
        self.rows = rows

    @property
    def n_pages(self) -> int:
        return int(self.rows.shape[0])

    @classmethod
    def empty(cls, d: LatentDims, n_pages: int, device="cuda") -> "LatentCache":
        """Unwritten pages; a page's contents count only once tokens were appended to it."""
        return cls(d, torch.empty((n_pages, d.page_size, d.latent_dim + d.rope_dim), dtype=torch.bfloat16,
                                  device=device))


def latent_append(d: LatentDims, cache: LatentCache, cu_seqlens, kv_lens, block_table, c, *, norm_w=None,
                  q_rope=None, q_out=None, rope=None, positions=None, rows_out=None):
    """gdn_latent_append: c [T, latent + rope] (token stride free) into the cache, its latent part
    normalised with norm_w [latent] (None: kept), its position part and q_rope [T, H, rope] (strides
    free) rotated by rope [rows, rope_dim] (cosines | sines; None: kept); positions [T] int32 where
    they are not the cache positions.  rows_out [T, latent + rope]: the rows as stored.  Returns the
    rotated q (q_out, or a new tensor; None without q_rope)."""
    cu_d, cu_h = _pair(cu_seqlens, c)
    return (paged._native or paged._bind()).latent_append(d.address(), cache.rows, cu_d, cu_h, kv_lens, block_table, c,
                                                          norm_w, q_rope, q_out, rope, positions, rows_out)


def latent_read(d: LatentDims, cache: LatentCache, cu_seqlens, starts, block_table, *, out=None):
    """gdn_latent_read: rows of cu_seqlens[i+1] - cu_seqlens[i] cached tokens of each sequence from
    position starts[i] on, packed.  Returns [R, latent + rope] bf16."""
    cu_d, cu_h = _pair(cu_seqlens, block_table)
    return (paged._native or paged._bind()).latent_read(d.address(), cache.rows, cu_d, cu_h, starts, block_table, out)


def latent_attention_workspace_size(d: LatentDims, cu_seqlens) -> int:
    """Bytes of workspace latent_attention needs for these sequences."""
    lib = load()
    if isinstance(cu_seqlens, tuple):
        cu_seqlens = cu_seqlens[1]
    if isinstance(cu_seqlens, torch.Tensor):
        host = cu_seqlens.detach().to("cpu", torch.int32).contiguous()
    else:
        host = torch.tensor(list(cu_seqlens), dtype=torch.int32)
    out = ctypes.c_size_t(0)
    dd = d.c()
    _check("gdn_latent_attention_workspace_size", lib.gdn_latent_attention_workspace_size(
        ctypes.byref(dd), host.numel() - 1, host.data_ptr(), ctypes.byref(out)))
    return int(out.value)


def latent_attention(d: LatentDims, cache: LatentCache, cu_seqlens, kv_lens, block_table, q, *, out=None,
                     workspace=None):
    """gdn_latent_attention, the absorbed form: q [T, H, latent + rope] (strides free) against the
    cache.  Returns out [T, H, latent].  workspace (None: allocated): of one call at a time."""
    cu_d, cu_h = _pair(cu_seqlens, q)
    return (paged._native or paged._bind()).latent_attention(d.address(), cache.rows, cu_d, cu_h, kv_lens, block_table,
                                                             q, out, workspace)


def expanded_attention(d: LatentDims, cu_q, cu_kv, q, k, k_rope, v, *, out=None):
    """gdn_expanded_attention: q [Tq, H, nope + rope] against k [Tk, H, nope], k_rope [Tk, rope] and
    v [Tk, H, v] (strides free), causal, sequence i's queries being its last positions.  Returns out
    [Tq, H, v]."""
    cq_d, cq_h = _pair(cu_q, q)
    ck_d, ck_h = _pair(cu_kv, q)
    return (paged._native or paged._bind()).expanded_attention(d.address(), cq_d, cq_h, ck_d, ck_h, q, k, k_rope, v, out)


def copy_pages(caches, src, dst) -> None:
    """gdn_copy_pages: page src[i] to page dst[i] in a cache (KVCache or LatentCache), or in each of a
    list of them (the layers of a stack, which share a block table).  src, dst: lists of ints, or
    1-d int32 tensors on the host; no page may be written twice, or both read and written, and no
    cache given twice."""
    tensors = []
    for c in caches if isinstance(caches, (list, tuple)) else (caches,):
        if isinstance(c, KVCache):
            tensors += [c.k, c.v, c.k_scale, c.v_scale]
        elif isinstance(c, LatentCache):
            tensors.append(c.rows)
        else:
            raise TypeError("caches must be KVCache or LatentCache objects")
    (paged._native or paged._bind()).copy_pages(tuple(tensors), src, dst)
