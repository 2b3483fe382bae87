"""Full attention over a paged 8-bit cache, and verification of drafted tokens.

Like the rest of the binding this only marshals arguments: shapes, dtypes,
devices and strides are checked, raw pointers and the current stream go to the
C ABI of ``include/gdn.h``, which states layouts, formulas and errors.  The
checks of a call's tensors are native code (``csrc/gdn_bind.cpp``): from Python
they take longer than a single token's kernels.

One step of a full-attention layer over its cache (``kv_lens`` counts the
step's own tokens)::

    d = KVDims(16, 2, 256, page_size=64, rope_dim=64)
    cache = KVCache.empty(d, n_pages, device="cuda")
    q = kv_append(d, cache, cu_seqlens, kv_lens, block_table, k, v, q=q, rope=rope)
    o = kv_attention(d, cache, cu_seqlens, kv_lens, block_table, q)

and the end of a speculative step::

    accepted, tokens = accept_drafts(drafts, logits, draft_logits, uniforms, noise,
                                     form="logits", temperature=temperature)
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from dataclasses import dataclass

import torch

from . import DTYPE_BF16, DTYPE_F32, _PKG, GDNError, _check, _cu_pair, _KVDims, _t, load

KV_FORMATS = {"int8": (0, torch.int8), "e4m3": (1, torch.float8_e4m3fn)}
ROPE_STYLES = {"half": 0, "interleaved": 1}
DIST_FORMS = {"probs": 0, "logits": 1}
_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}

_native = None


def _fail(fn: str, status: int):
    raise GDNError(fn, status, load().gdn_last_error().decode(errors="replace"))


def _bind():
    """The native marshalling module (loaded once).  Raises if it has not been built."""
    global _native
    if _native is None:
        load()
        path = os.path.join(_PKG, "_gdn_bind.so")
        if not os.path.exists(path):
            raise RuntimeError(f"_gdn_bind.so not found at {path}; build it first "
                               "(gated_deltanet_linear_mixer_gb300._build.build())")
        spec = importlib.util.spec_from_file_location("_gdn_bind", path)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        mod.on_failure(_fail)
        _native = mod
    return _native


@dataclass(frozen=True)
class KVDims:
    """Geometry of one full-attention layer and its cache: heads, head width, tokens per page
    (and per scale), activation dtype, codes, rotation, sliding window (0: none), softmax scale
    (None: head_dim^-1/2)."""
    n_q_heads: int
    n_kv_heads: int
    head_dim: int
    page_size: int = 64
    dtype: torch.dtype = torch.bfloat16
    cache: str = "int8"
    rope_dim: int = 0
    rope_style: str = "half"
    window: int = 0
    scale: float | None = None

    def c(self) -> _KVDims:
        got = self.__dict__.get("_c")
        if got is None:
            if self.dtype not in _DTYPES:
                raise ValueError("activation dtype must be torch.float32 or torch.bfloat16")
            if self.cache not in KV_FORMATS:
                raise ValueError("cache must be 'int8' or 'e4m3'")
            if self.rope_style not in ROPE_STYLES:
                raise ValueError("rope_style must be 'half' or 'interleaved'")
            scale = self.head_dim ** -0.5 if self.scale is None else self.scale
            got = _KVDims(self.n_q_heads, self.n_kv_heads, self.head_dim, self.page_size,
                          _DTYPES[self.dtype], KV_FORMATS[self.cache][0], self.rope_dim,
                          ROPE_STYLES[self.rope_style], self.window, scale)
            object.__setattr__(self, "_c", got)
        return got

    def address(self) -> int:
        """Where the C struct of these dimensions lies, for as long as they do."""
        return ctypes.addressof(self.c())

    def __getstate__(self):
        """Copies and pickles hold the fields alone: the C struct belongs to one object."""
        return {name: getattr(self, name) for name in self.__dataclass_fields__}


class KVCache:
    """The pages of one layer: codes k, v [n_pages, Hkv, page_size, head_dim] and one fp32 scale
    per page and head, k_scale, v_scale [n_pages, Hkv].  Holds the tensors it is given; a call takes
    those that it holds then, so that they may be replaced (by larger ones, by a copy's own)."""

    def __init__(self, d: KVDims, k, v, k_scale, v_scale):
        d.c()
        n = int(k.shape[0])
        code = KV_FORMATS[d.cache][1]
        shape = (n, d.n_kv_heads, d.page_size, d.head_dim)
        _t(k, "k", code, shape)
        _t(v, "v", code, shape)
        _t(k_scale, "k_scale", torch.float32, shape[:2])
        _t(v_scale, "v_scale", torch.float32, shape[:2])
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale

    @property
    def n_pages(self) -> int:
        return int(self.k.shape[0])

    @classmethod
    def empty(cls, d: KVDims, n_pages: int, device="cuda") -> "KVCache":
        """Unwritten pages; a page's contents count only once tokens were appended to it."""
        if d.cache not in KV_FORMATS:
            raise ValueError("cache must be 'int8' or 'e4m3'")
        shape = (n_pages, d.n_kv_heads, d.page_size, d.head_dim)
        codes = [torch.empty(shape, dtype=KV_FORMATS[d.cache][1], device=device) for _ in "kv"]
        scales = [torch.empty(shape[:2], device=device) for _ in "kv"]
        return cls(d, *codes, *scales)


def _pair(cu_seqlens, like):
    return cu_seqlens if type(cu_seqlens) is tuple else _cu_pair(cu_seqlens, like.device)


def kv_append(d: KVDims, cache: KVCache, cu_seqlens, kv_lens, block_table, k, v, *, q=None,
              rope=None, positions=None, q_out=None):
    """gdn_kv_append: k, v [T, Hkv, D] (token and head strides free) into the cache, rotated by
    rope [rows, rope_dim] (cosines | sines) on the way; positions [T] int32 where they are not the
    cache positions.  Returns the rotated q [T, Hq, D] (None without q)."""
    cu_d, cu_h = _pair(cu_seqlens, k)
    return (_native or _bind()).kv_append(d.address(), cache.k, cache.v, cache.k_scale, cache.v_scale, cu_d, cu_h,
                                          kv_lens, block_table, k, v, q, rope, positions, q_out)


def kv_read(d: KVDims, cache: KVCache, cu_seqlens, starts, block_table, *, dtype=None, k_out=None,
            v_out=None):
    """gdn_kv_read: values of cu_seqlens[i+1] - cu_seqlens[i] cached tokens of each sequence from
    position starts[i] on.  Returns (k, v) [R, Hkv, D] in dtype (None: the activation dtype)."""
    cu_d, cu_h = _pair(cu_seqlens, block_table)
    dtype = d.dtype if dtype is None else dtype
    if dtype not in _DTYPES:
        raise ValueError("dtype must be torch.float32 or torch.bfloat16")
    return (_native or _bind()).kv_read(d.address(), cache.k, cache.v, cache.k_scale, cache.v_scale, cu_d, cu_h,
                                        starts, block_table, _DTYPES[dtype], k_out, v_out)


def kv_attention_workspace_size(d: KVDims, cu_seqlens, max_kv_len: int) -> int:
    """Bytes of workspace kv_attention needs for these sequences and longest length."""
    lib = load()
    if isinstance(cu_seqlens, tuple):
        host = cu_seqlens[1]
    elif isinstance(cu_seqlens, torch.Tensor):
        host = cu_seqlens.detach().to("cpu", torch.int32).contiguous()
    else:
        host = torch.tensor(list(cu_seqlens), dtype=torch.int32)
    out = ctypes.c_size_t(0)
    dd = d.c()
    _check("gdn_kv_attention_workspace_size", lib.gdn_kv_attention_workspace_size(
        ctypes.byref(dd), host.numel() - 1, host.data_ptr(), max_kv_len, ctypes.byref(out)))
    return int(out.value)


def kv_attention(d: KVDims, cache: KVCache, cu_seqlens, kv_lens, block_table, q, *, max_kv_len=None,
                 out=None, workspace=None):
    """gdn_kv_attention: q [T, Hq, D] against the cache.  max_kv_len (None: what block_table can
    hold) bounds kv_lens on the host.  Returns out [T, Hq, D]."""
    cu_d, cu_h = _pair(cu_seqlens, q)
    return (_native or _bind()).kv_attention(d.address(), cache.k, cache.v, cache.k_scale, cache.v_scale, cu_d, cu_h,
                                             kv_lens, block_table, q, max_kv_len, out, workspace)


def accept_drafts(drafts, target, draft, uniforms, noise, *, form="probs", temperature=None,
                  accepted=None, tokens=None):
    """gdn_accept_drafts: drafts [n, T] int32 (-1: no draft), target [n, T + 1, vocab] and draft
    [n, T, vocab] (None: the drafts were certain) as fp32 probabilities or fp32 / bf16 logits,
    uniforms [n, T] ~ U[0, 1), noise [n, vocab] ~ Exp(1), temperature [n] (logits; None: 1).
    Returns accepted [n] and tokens [n, T + 1], int32."""
    if form not in DIST_FORMS:
        raise ValueError("form must be 'probs' or 'logits'")
    return (_native or _bind()).accept_drafts(drafts, target, draft, uniforms, noise, DIST_FORMS[form],
                                              temperature, accepted, tokens)
