"""CPU checks of the paged-cache and draft-verification entry points: what they
refuse, and with which message, before any CUDA call (no GPU is needed)."""
import ctypes

import pytest
import torch

import gated_deltanet_linear_mixer_gb300 as gdn
from gated_deltanet_linear_mixer_gb300 import _build

P = 0x10000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gdn.load()


def _dims(**kw):
    base = dict(n_q_heads=16, n_kv_heads=2, head_dim=256, page_size=64, dtype=1, format=0, rope_dim=64,
                rope_style=0, window=0, scale=0.0625)
    base.update(kw)
    return gdn._KVDims(**base)


def _batch(cu=(0, 4), table=P, **kw):
    host = (ctypes.c_int32 * len(cu))(*cu)
    base = dict(n_seq=len(cu) - 1, pages_per_seq=4, cu_seqlens=P, block_table=table)
    base.update(kw)
    b = gdn._KVBatch(base["n_seq"], base["pages_per_seq"], base["cu_seqlens"],
                     ctypes.cast(host, ctypes.c_void_p).value if len(cu) else None, base["block_table"])
    b.keep = host
    return b


def _cache(**kw):
    base = dict(k=P, v=P, k_scale=P, v_scale=P, n_pages=8)
    base.update(kw)
    return gdn._KVCache(*(base[k] for k in ("k", "v", "k_scale", "v_scale", "n_pages")))


def _r(data=P, token=4096, head=256):
    return ctypes.byref(gdn._Rows(data, token, head))


def _append(lib, d=None, c=None, b=None, lens=P, q=None, k=None, v=None, rope=P, rows=10, out=P):
    d, c, b = d or _dims(), c or _cache(), b or _batch()
    return lib.gdn_kv_append(ctypes.byref(d), ctypes.byref(c), ctypes.byref(b), lens, q or _r(), k or _r(),
                             v or _r(), rope, rows, None, out, None)


def _attend(lib, d=None, c=None, b=None, lens=P, longest=100, q=None, out=P, ws=P, size=1 << 40):
    d, c, b = d or _dims(), c or _cache(), b or _batch()
    return lib.gdn_kv_attention(ctypes.byref(d), ctypes.byref(c), ctypes.byref(b), lens, longest, q or _r(), out, ws,
                                size, None)


def _read(lib, d=None, c=None, b=None, starts=P, dtype=1, k=P, v=P):
    d, c, b = d or _dims(), c or _cache(), b or _batch()
    return lib.gdn_kv_read(ctypes.byref(d), ctypes.byref(c), ctypes.byref(b), starts, dtype, k, v, None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(n_q_heads=0), 1, "head counts"),
    (dict(n_q_heads=15), 2, "multiple of n_kv_heads"),
    (dict(n_q_heads=65, n_kv_heads=1), 2, "at most 64"),
    (dict(head_dim=96), 2, "head_dim"),
    (dict(page_size=48), 2, "page_size"),
    (dict(page_size=0), 2, "page_size"),
    (dict(dtype=2), 1, "gdn_dtype"),
    (dict(format=2), 1, "gdn_kv_format"),
    (dict(rope_dim=272), 2, "rope_dim"),
    (dict(rope_dim=24), 2, "rope_dim"),
    (dict(rope_dim=-16), 2, "rope_dim"),
    (dict(rope_style=5), 1, "gdn_rope_style"),
    (dict(window=-1), 1, "window"),
    (dict(scale=0.0), 1, "scale"),
    (dict(scale=float("inf")), 1, "scale"),
    (dict(scale=float("nan")), 1, "scale"),
])
def test_bad_geometry_is_refused(lib, kw, status, msg):
    for call in (_append, _attend, _read):
        assert call(lib, d=_dims(**kw)) == status
        assert msg in lib.gdn_last_error().decode()
    n, cu = ctypes.c_size_t(0), (ctypes.c_int32 * 2)(0, 4)
    assert lib.gdn_kv_attention_workspace_size(ctypes.byref(_dims(**kw)), 1, ctypes.cast(cu, ctypes.c_void_p), 10,
                                               ctypes.byref(n)) == status


@pytest.mark.parametrize("kw,msg", [
    (dict(k=None), "cache pointer"), (dict(v_scale=None), "cache pointer"), (dict(n_pages=-1), "n_pages"),
    (dict(k=P + 8), "aligned"),
])
def test_bad_caches_are_refused(lib, kw, msg):
    for call in (_append, _attend, _read):
        assert call(lib, c=_cache(**kw)) == 1
        assert msg in lib.gdn_last_error().decode()


def test_bad_batches_are_refused(lib):
    for call in (_append, _attend, _read):
        for b, status, msg in ((_batch((1, 4)), 1, "cu_seqlens[0]"), (_batch((0, 4, 3)), 1, "decreases"),
                               (_batch(n_seq=-1), 1, "n_seq"), (_batch(pages_per_seq=-2), 1, "pages_per_seq"),
                               (_batch(table=None), 1, "block_table"), (_batch(cu_seqlens=None), 1, "NULL"),
                               (_batch(tuple(range(65537))), 2, "GDN_MAX_SEQUENCES")):
            assert call(lib, b=b) == status, msg
            assert msg in lib.gdn_last_error().decode()
    assert _append(lib, lens=None) == 1 and _attend(lib, lens=None) == 1 and _read(lib, starts=None) == 1
    assert "lengths" in lib.gdn_last_error().decode()


def test_empty_batches_are_no_ops(lib):
    for call in (_append, _attend, _read):
        assert call(lib, b=_batch((0,))) == 0
        assert call(lib, b=_batch((0, 0, 0))) == 0


@pytest.mark.parametrize("kw,msg", [
    (dict(data=None), "NULL"), (dict(data=P + 2), "16 bytes"), (dict(token=4097), "16 bytes"),
    (dict(head=260), "16 bytes"), (dict(token=-8), "negative"),
])
def test_bad_rows_are_refused(lib, kw, msg):
    for call in (lambda r: _append(lib, q=r), lambda r: _append(lib, k=r), lambda r: _append(lib, v=r),
                 lambda r: _attend(lib, q=r)):
        assert call(_r(**kw)) == 1
        assert msg in lib.gdn_last_error().decode()


def test_append_refusals(lib):
    assert _append(lib, rope=None) == 1 and "rope" in lib.gdn_last_error().decode()
    assert _append(lib, rows=0) == 1 and "rope" in lib.gdn_last_error().decode()
    assert _append(lib, rope=P + 4) == 1 and "aligned" in lib.gdn_last_error().decode()
    assert _append(lib, out=None) == 1 and "q_out" in lib.gdn_last_error().decode()
    assert _append(lib, out=P + 8) == 1 and "q_out" in lib.gdn_last_error().decode()


def test_read_refusals(lib):
    assert _read(lib, dtype=3) == 1 and "out_dtype" in lib.gdn_last_error().decode()
    assert _read(lib, k=None) == 1 and "k_out" in lib.gdn_last_error().decode()
    assert _read(lib, v=P + 4) == 1 and "aligned" in lib.gdn_last_error().decode()


def test_attention_refusals(lib):
    assert _attend(lib, longest=-1) == 1 and "max_kv_len" in lib.gdn_last_error().decode()
    assert _attend(lib, out=None) == 1 and "out" in lib.gdn_last_error().decode()
    assert _attend(lib, out=P + 2) == 1 and "aligned" in lib.gdn_last_error().decode()


def _accept(lib, n=2, t=3, vocab=10, form=0, dtype=0, drafts=P, target=P, ts=10, draft=P, ds=10, temp=None, u=P,
            noise=P, ns=10, accepted=P, tokens=P):
    return lib.gdn_accept_drafts(n, t, vocab, form, dtype, drafts, target, ts, draft, ds, temp, u, noise, ns, accepted,
                                 tokens, None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(n=-1), 1, "n_seq"), (dict(n=65536), 1, "GDN_MAX_SEQUENCES"), (dict(t=17), 1, "T must be"),
    (dict(t=-1), 1, "T must be"), (dict(vocab=0), 1, "vocab"), (dict(form=2), 1, "gdn_dist_form"),
    (dict(dtype=2), 1, "gdn_dtype"), (dict(dtype=1), 2, "fp32"), (dict(temp=P), 1, "temperature"),
    (dict(ts=9), 1, "stride"), (dict(ds=9), 1, "stride"), (dict(ns=9), 1, "stride"), (dict(target=None), 1, "NULL"),
    (dict(noise=None), 1, "NULL"), (dict(drafts=None), 1, "NULL"), (dict(u=None), 1, "NULL"),
    (dict(accepted=None), 1, "NULL"), (dict(tokens=None), 1, "NULL"), (dict(target=P + 2), 1, "aligned"),
    (dict(noise=P + 2), 1, "aligned"), (dict(draft=P + 1), 1, "aligned"),
])
def test_accept_refusals(lib, kw, status, msg):
    assert _accept(lib, **kw) == status
    assert msg in lib.gdn_last_error().decode()


def test_accept_of_no_sequences(lib):
    assert _accept(lib, n=0, target=None) == 0


@pytest.mark.parametrize("site,call", [("kv_append", _append), ("kv_attention", _attend), ("kv_read", _read),
                                       ("accept", _accept)])
def test_injected_faults(lib, monkeypatch, site, call):
    monkeypatch.setenv("GDN_FAULT", f"decode,{site}")
    assert call(lib) == gdn.GDN_ERR_INJECTED
    assert site in lib.gdn_last_error().decode()


def test_workspace_query(lib):
    n, cu = ctypes.c_size_t(1), (ctypes.c_int32 * 2)(0, 1)
    host = ctypes.cast(cu, ctypes.c_void_p)
    assert lib.gdn_kv_attention_workspace_size(ctypes.byref(_dims()), 1, host, 131072, ctypes.byref(n)) == 0
    assert n.value % 256 == 0
    if n.value:
        assert _attend(lib, b=_batch((0, 1)), longest=131072, ws=None, size=0) == 4
        assert _attend(lib, b=_batch((0, 1)), longest=131072, size=n.value - 1) == 4
        assert "workspace" in lib.gdn_last_error().decode()
        assert _attend(lib, b=_batch((0, 1)), longest=131072, ws=P + 16, size=n.value) == 4
        assert "256-byte" in lib.gdn_last_error().decode()
    assert lib.gdn_kv_attention_workspace_size(ctypes.byref(_dims()), 1, host, -1, ctypes.byref(n)) == 1
    assert lib.gdn_kv_attention_workspace_size(ctypes.byref(_dims()), 1, host, 5, None) == 1


# ----------------------------------------------------- the binding's checks
D = gdn.KVDims(4, 2, 64, page_size=16)


def _tensors(n_pages=3):
    k = torch.zeros(n_pages, 2, 16, 64, dtype=torch.int8)
    return k, k.clone(), torch.zeros(n_pages, 2), torch.zeros(n_pages, 2)


@pytest.mark.parametrize("kw", [dict(dtype=torch.float16), dict(cache="int4"), dict(rope_style="spiral")])
def test_kvdims_options_are_checked(kw):
    with pytest.raises(ValueError):
        gdn.KVDims(4, 2, 64, **kw).c()


def test_cache_tensors_are_checked():
    k, v, ks, vs = _tensors()
    with pytest.raises(ValueError, match="CUDA"):
        gdn.KVCache(D, k, v, ks, vs)
    with pytest.raises(TypeError, match="k must be"):
        gdn.KVCache(D, k.float(), v, ks, vs)
    with pytest.raises(ValueError, match="shape"):
        gdn.KVCache(D, k[:, :1], v, ks, vs)
    with pytest.raises(ValueError, match="cache must be"):
        gdn.KVCache.empty(gdn.KVDims(4, 2, 64, cache="fp4"), 3)


def test_kvdims_default_scale_and_equality():
    assert D.c().scale == pytest.approx(64 ** -0.5)
    assert gdn.KVDims(4, 2, 64, scale=0.5).c().scale == 0.5
    assert D == gdn.KVDims(4, 2, 64, page_size=16) and hash(D) == hash(gdn.KVDims(4, 2, 64, page_size=16))


def test_accept_tensors_are_checked(lib):
    x = torch.zeros(2, 3, dtype=torch.int32)
    p = torch.zeros(2, 4, 10)
    with pytest.raises(ValueError, match="form"):
        gdn.accept_drafts(x, p, None, p[:, :3, 0], p[:, 0], form="odds")
    with pytest.raises(ValueError, match="CUDA"):
        gdn.accept_drafts(x, p, None, p[:, :3, 0], p[:, 0])
    with pytest.raises(TypeError, match="drafts"):
        gdn.accept_drafts(x.long(), p, None, p[:, :3, 0], p[:, 0])
