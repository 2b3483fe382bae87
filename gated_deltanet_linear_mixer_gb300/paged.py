"""Full attention over a paged 8-bit cache, and verification of drafted tokens.

Like the rest of the binding this only marshals arguments: shapes, dtypes,
devices and strides are checked, raw pointers and the current stream go to the
C ABI of ``include/gdn.h``, which states layouts, formulas and errors.

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
from dataclasses import dataclass

import torch

from . import (DTYPE_BF16, DTYPE_F32, _check, _cu_pair, _KVBatch, _KVCache, _KVDims, _Rows, _stream,
               _t, load)

KV_FORMATS = {"int8": (0, torch.int8), "e4m3": (1, torch.float8_e4m3fn)}
ROPE_STYLES = {"half": 0, "interleaved": 1}
DIST_FORMS = {"probs": 0, "logits": 1}
_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}


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


class KVCache:
    """The pages of one layer: codes k, v [n_pages, Hkv, page_size, head_dim] and one fp32 scale
    per page and head, k_scale, v_scale [n_pages, Hkv].  Holds the tensors it is given."""

    def __init__(self, d: KVDims, k, v, k_scale, v_scale):
        d.c()
        n = int(k.shape[0])
        code = KV_FORMATS[d.cache][1]
        shape = (n, d.n_kv_heads, d.page_size, d.head_dim)
        _t(k, "k", code, shape)
        _t(v, "v", code, shape)
        _t(k_scale, "k_scale", torch.float32, shape[:2])
        _t(v_scale, "v_scale", torch.float32, shape[:2])
        self.k, self.v, self.k_scale, self.v_scale, self.n_pages = k, v, k_scale, v_scale, n
        self._c = _KVCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), n)
        self._of = (d.n_kv_heads, d.page_size, d.head_dim, d.cache)

    @classmethod
    def empty(cls, d: KVDims, n_pages: int, device="cuda") -> "KVCache":
        """Unwritten pages; a page's contents count only once tokens were appended to it."""
        if d.cache not in KV_FORMATS:
            raise ValueError("cache must be 'int8' or 'e4m3'")
        shape = (n_pages, d.n_kv_heads, d.page_size, d.head_dim)
        codes = [torch.empty(shape, dtype=KV_FORMATS[d.cache][1], device=device) for _ in "kv"]
        scales = [torch.empty(shape[:2], device=device) for _ in "kv"]
        return cls(d, *codes, *scales)

    def c(self, d: KVDims) -> _KVCache:
        if self._of != (d.n_kv_heads, d.page_size, d.head_dim, d.cache):
            raise ValueError("the cache was made for other dimensions or codes")
        return self._c


def _batch(cu_d, cu_h, lens, block_table, name):
    n = cu_h.numel() - 1
    _t(lens, name, torch.int32, (n,))
    _t(block_table, "block_table", torch.int32)
    if block_table.dim() != 2 or block_table.shape[0] != n:
        raise ValueError(f"block_table must have shape ({n}, pages per sequence), got "
                         f"{tuple(block_table.shape)}")
    return _KVBatch(n, block_table.shape[1], cu_d.data_ptr(), cu_h.data_ptr(), block_table.data_ptr())


def _rows(x, name, dtype, shape):
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if x.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(x.shape)}")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    st, sh, sd = x.stride()
    if sd != 1:
        raise ValueError(f"{name}: a head's channels must be contiguous")
    return _Rows(x.data_ptr(), st, sh)


def _tokens(cu_h):
    return int(cu_h[-1]) if cu_h.numel() > 1 else 0


def kv_append(d: KVDims, cache: KVCache, cu_seqlens, kv_lens, block_table, k, v, *, q=None,
              rope=None, positions=None, q_out=None):
    """gdn_kv_append: k, v [T, Hkv, D] (token and head strides free) into the cache, rotated by
    rope [rows, rope_dim] (cosines | sines) on the way; positions [T] int32 where they are not the
    cache positions.  Returns the rotated q [T, Hq, D] (None without q)."""
    lib = load()
    dev = k.device
    cu_d, cu_h = _cu_pair(cu_seqlens, dev)
    t = _tokens(cu_h)
    dd, cc = d.c(), cache.c(d)
    batch = _batch(cu_d, cu_h, kv_lens, block_table, "kv_lens")
    kr = _rows(k, "k", d.dtype, (t, d.n_kv_heads, d.head_dim))
    vr = _rows(v, "v", d.dtype, (t, d.n_kv_heads, d.head_dim))
    qr = None
    if q is not None:
        qr = _rows(q, "q", d.dtype, (t, d.n_q_heads, d.head_dim))
        if q_out is None:
            q_out = torch.empty((t, d.n_q_heads, d.head_dim), dtype=d.dtype, device=dev)
        else:
            _t(q_out, "q_out", d.dtype, (t, d.n_q_heads, d.head_dim))
    rows = 0
    if rope is not None:
        _t(rope, "rope", torch.float32)
        if rope.dim() != 2 or rope.shape[1] != d.rope_dim:
            raise ValueError(f"rope must have shape (rows, {d.rope_dim}), got {tuple(rope.shape)}")
        rows = rope.shape[0]
    if positions is not None:
        _t(positions, "positions", torch.int32, (t,))
    _check("gdn_kv_append", lib.gdn_kv_append(
        ctypes.byref(dd), ctypes.byref(cc), ctypes.byref(batch), kv_lens.data_ptr(),
        None if qr is None else ctypes.byref(qr), ctypes.byref(kr), ctypes.byref(vr),
        None if rope is None else rope.data_ptr(), rows,
        None if positions is None else positions.data_ptr(),
        None if q is None else q_out.data_ptr(), _stream(dev)))
    return None if q is None else q_out


def kv_read(d: KVDims, cache: KVCache, cu_seqlens, starts, block_table, *, dtype=None, k_out=None,
            v_out=None):
    """gdn_kv_read: values of cu_seqlens[i+1] - cu_seqlens[i] cached tokens of each sequence from
    position starts[i] on.  Returns (k, v) [R, Hkv, D] in dtype (None: the activation dtype)."""
    lib = load()
    dev = block_table.device
    cu_d, cu_h = _cu_pair(cu_seqlens, dev)
    dtype = d.dtype if dtype is None else dtype
    if dtype not in _DTYPES:
        raise ValueError("dtype must be torch.float32 or torch.bfloat16")
    shape = (_tokens(cu_h), d.n_kv_heads, d.head_dim)
    dd, cc = d.c(), cache.c(d)
    batch = _batch(cu_d, cu_h, starts, block_table, "starts")
    k_out = torch.empty(shape, dtype=dtype, device=dev) if k_out is None else _t(k_out, "k_out", dtype, shape)
    v_out = torch.empty(shape, dtype=dtype, device=dev) if v_out is None else _t(v_out, "v_out", dtype, shape)
    _check("gdn_kv_read", lib.gdn_kv_read(
        ctypes.byref(dd), ctypes.byref(cc), ctypes.byref(batch), starts.data_ptr(), _DTYPES[dtype],
        k_out.data_ptr(), v_out.data_ptr(), _stream(dev)))
    return k_out, v_out


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
    lib = load()
    dev = q.device
    cu_d, cu_h = _cu_pair(cu_seqlens, dev)
    shape = (_tokens(cu_h), d.n_q_heads, d.head_dim)
    dd, cc = d.c(), cache.c(d)
    batch = _batch(cu_d, cu_h, kv_lens, block_table, "kv_lens")
    qr = _rows(q, "q", d.dtype, shape)
    if max_kv_len is None:
        max_kv_len = min(block_table.shape[1] * d.page_size, 0x7fffffff)
    out = torch.empty(shape, dtype=d.dtype, device=dev) if out is None else _t(out, "out", d.dtype, shape)
    if workspace is None:
        need = kv_attention_workspace_size(d, (cu_d, cu_h), max_kv_len)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    ws = (None, 0) if workspace is None else (workspace.data_ptr(),
                                              workspace.numel() * workspace.element_size())
    _check("gdn_kv_attention", lib.gdn_kv_attention(
        ctypes.byref(dd), ctypes.byref(cc), ctypes.byref(batch), kv_lens.data_ptr(), max_kv_len,
        ctypes.byref(qr), out.data_ptr(), *ws, _stream(dev)))
    return out


def _dist(x, name, dtype, shape):
    """Rows of distributions: [n, rows, vocab], vocab contiguous, rows one stride apart throughout."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if x.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(x.shape)}")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    n, rows, vocab = shape
    sn, sr, sv = x.stride()
    if rows == 1:
        sr = sn if n > 1 else vocab
    if (sv != 1 and vocab > 1) or (n > 1 and sn != rows * sr):
        raise ValueError(f"{name}: rows must be contiguous and evenly spaced")
    return sr


def accept_drafts(drafts, target, draft, uniforms, noise, *, form="probs", temperature=None,
                  accepted=None, tokens=None):
    """gdn_accept_drafts: drafts [n, T] int32 (-1: no draft), target [n, T + 1, vocab] and draft
    [n, T, vocab] (None: the drafts were certain) as fp32 probabilities or fp32 / bf16 logits,
    uniforms [n, T] ~ U[0, 1), noise [n, vocab] ~ Exp(1), temperature [n] (logits; None: 1).
    Returns accepted [n] and tokens [n, T + 1], int32."""
    lib = load()
    dev = target.device
    if form not in DIST_FORMS:
        raise ValueError("form must be 'probs' or 'logits'")
    if target.dtype not in _DTYPES:
        raise TypeError("target must be torch.float32 or torch.bfloat16")
    _t(drafts, "drafts", torch.int32)
    if drafts.dim() != 2 or target.dim() != 3:
        raise ValueError("drafts must be [n, T] and target [n, T + 1, vocab]")
    n, t = drafts.shape
    vocab = target.shape[2]
    ts = _dist(target, "target", target.dtype, (n, t + 1, vocab))
    ds = vocab
    if draft is not None and t > 0:
        ds = _dist(draft, "draft", target.dtype, (n, t, vocab))
    _t(uniforms, "uniforms", torch.float32, (n, t))
    ns = _dist(noise.unsqueeze(1), "noise", torch.float32, (n, 1, vocab))
    if temperature is not None:
        _t(temperature, "temperature", torch.float32, (n,))
    if accepted is None:
        accepted = torch.empty(n, dtype=torch.int32, device=dev)
    else:
        _t(accepted, "accepted", torch.int32, (n,))
    if tokens is None:
        tokens = torch.empty((n, t + 1), dtype=torch.int32, device=dev)
    else:
        _t(tokens, "tokens", torch.int32, (n, t + 1))
    _check("gdn_accept_drafts", lib.gdn_accept_drafts(
        n, t, vocab, DIST_FORMS[form], _DTYPES[target.dtype], drafts.data_ptr(), target.data_ptr(), ts,
        None if draft is None else draft.data_ptr(), ds,
        None if temperature is None else temperature.data_ptr(), uniforms.data_ptr(),
        noise.data_ptr(), ns, accepted.data_ptr(), tokens.data_ptr(), _stream(dev)))
    return accepted, tokens
