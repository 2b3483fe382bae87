"""CPU checks of the latent attention and page copy entry points: what they refuse, and with which
message, before any CUDA call (no GPU is needed)."""
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
    base = dict(n_heads=16, latent_dim=512, rope_dim=64, page_size=64, rope_style=0, nope_dim=128, v_dim=128,
                scale=0.07, norm_eps=1e-6)
    base.update(kw)
    return gdn._LatentDims(**base)


def _cu(cu):
    return (ctypes.c_int32 * len(cu))(*cu)


def _batch(cu=(0, 4), table=P, **kw):
    host = _cu(cu)
    base = dict(n_seq=len(cu) - 1, pages_per_seq=4, cu_seqlens=P)
    base.update(kw)
    b = gdn._KVBatch(base["n_seq"], base["pages_per_seq"], base["cu_seqlens"],
                     ctypes.cast(host, ctypes.c_void_p).value, table)
    b.keep = host
    return b


def _r(data=P, token=9216, head=576):
    return ctypes.byref(gdn._Rows(data, token, head))


def _cache(rows=P, n=8):
    return gdn._LatentCache(rows, n)


def _append(lib, d=None, c=None, b=None, lens=P, rows=None, norm=None, q=None, q_out=None, rope=P, n_rope=10, packed=None):
    d, c, b = d or _dims(), c or _cache(), b or _batch()
    return lib.gdn_latent_append(ctypes.byref(d), ctypes.byref(c), ctypes.byref(b), lens, rows or _r(), norm, q or _r(),
                                 q_out or _r(), rope, n_rope, None, packed, None)


def _read(lib, d=None, c=None, b=None, lens=P, out=P):
    d, c, b = d or _dims(), c or _cache(), b or _batch()
    return lib.gdn_latent_read(ctypes.byref(d), ctypes.byref(c), ctypes.byref(b), lens, out, None)


def _attend(lib, d=None, c=None, b=None, lens=P, q=None, out=P, ws=P, size=1 << 40):
    d, c, b = d or _dims(), c or _cache(), b or _batch()
    return lib.gdn_latent_attention(ctypes.byref(d), ctypes.byref(c), ctypes.byref(b), lens, q or _r(), out, ws, size, None)


def _expand(lib, d=None, cu=(0, 4), ck=(0, 9), q=None, k=None, r=None, v=None, out=P, cu_dev=P, ck_dev=P, n=None):
    d = d or _dims()
    hq, hk = _cu(cu), _cu(ck)
    return lib.gdn_expanded_attention(ctypes.byref(d), len(cu) - 1 if n is None else n, cu_dev,
                                      ctypes.cast(hq, ctypes.c_void_p), ck_dev, ctypes.cast(hk, ctypes.c_void_p), q or _r(),
                                      k or _r(), r or _r(), v or _r(), out, None)


def _message(lib):
    return lib.gdn_last_error().decode()


@pytest.mark.parametrize("kw,status,msg", [
    (dict(n_heads=0), 1, "n_heads"), (dict(n_heads=1025), 2, "n_heads"), (dict(latent_dim=384), 2, "latent_dim"),
    (dict(rope_dim=32), 2, "rope_dim"), (dict(rope_dim=0), 2, "rope_dim"), (dict(page_size=48), 2, "page_size"),
    (dict(rope_style=2), 1, "rope_style"), (dict(nope_dim=96), 2, "nope_dim"), (dict(v_dim=256), 2, "v_dim"),
    (dict(scale=0.0), 1, "scale"), (dict(scale=float("nan")), 1, "scale"), (dict(norm_eps=-1.0), 1, "norm_eps"),
    (dict(norm_eps=float("inf")), 1, "norm_eps"),
])
def test_bad_geometry_is_refused(lib, kw, status, msg):
    for call in (_append, _read, _attend, _expand):
        assert call(lib, d=_dims(**kw)) == status
        assert msg in _message(lib)
    n, cu = ctypes.c_size_t(0), _cu((0, 4))
    assert lib.gdn_latent_attention_workspace_size(ctypes.byref(_dims(**kw)), 1, ctypes.cast(cu, ctypes.c_void_p),
                                                   ctypes.byref(n)) == status


def test_bad_caches_and_batches_are_refused(lib):
    for call in (_append, _read, _attend):
        for c, msg in ((_cache(None), "NULL"), (_cache(P, -1), "n_pages"), (_cache(P + 8), "aligned")):
            assert call(lib, c=c) == 1 and msg in _message(lib)
        for b, status, msg in ((_batch((1, 4)), 1, "cu_seqlens[0]"), (_batch((0, 4, 3)), 1, "decreases"),
                               (_batch(n_seq=-1), 1, "n_seq"), (_batch(pages_per_seq=-2), 1, "pages_per_seq"),
                               (_batch(table=None), 1, "block_table"), (_batch(cu_seqlens=None), 1, "NULL"),
                               (_batch(tuple(range(65537))), 2, "GDN_MAX_SEQUENCES")):
            assert call(lib, b=b) == status, msg
            assert msg in _message(lib)
        assert call(lib, lens=None) == 1 and "lengths" in _message(lib)
        assert call(lib, b=_batch((0,))) == 0 and call(lib, b=_batch((0, 0, 0))) == 0


@pytest.mark.parametrize("bad", [dict(data=None), dict(data=P + 2), dict(token=9217), dict(token=-8), dict(head=-8), dict(head=4)])
def test_bad_rows_are_refused(lib, bad):
    r = _r(**bad)
    assert _attend(lib, q=r) == 1 and "q" in _message(lib)
    for name in ("rows", "q", "q_out"):
        if name == "rows" and "head" in bad:
            continue
        assert _append(lib, **{name: r}) == 1
    for name in ("q", "k", "r", "v"):
        if name == "r" and "head" in bad:
            continue
        assert _expand(lib, **{name: r}) == 1


def test_append_refusals(lib):
    assert _append(lib, q_out=_r(token=32)) == 1 and "overlap" in _message(lib)
    assert _append(lib, q_out=_r(head=32)) == 1 and "overlap" in _message(lib)
    assert _append(lib, n_rope=0) == 1 and "rope" in _message(lib)
    assert _append(lib, rope=P + 4) == 1 and "rope" in _message(lib)
    assert _append(lib, norm=P + 4) == 1 and "norm_w" in _message(lib)
    assert _append(lib, packed=P + 8) == 1 and "rows_out" in _message(lib)


def test_outputs_and_workspaces_are_refused(lib):
    assert _read(lib, out=None) == 1 and _read(lib, out=P + 8) == 1
    assert _attend(lib, out=None) == 1 and _attend(lib, out=P + 8) == 1 and "out" in _message(lib)
    assert _expand(lib, out=None) == 1 and _expand(lib, out=P + 2) == 1 and "out" in _message(lib)
    d, cu, n = _dims(), _cu((0, 4)), ctypes.c_size_t(0)
    assert lib.gdn_latent_attention_workspace_size(ctypes.byref(d), 1, ctypes.cast(cu, ctypes.c_void_p), ctypes.byref(n)) == 0
    assert lib.gdn_latent_attention_workspace_size(ctypes.byref(d), 1, ctypes.cast(cu, ctypes.c_void_p), None) == 1
    if n.value:
        assert _attend(lib, size=n.value - 1) == 4 and "workspace" in _message(lib)
        assert _attend(lib, ws=None) == 4 and _attend(lib, ws=P + 128) == 4


def test_expanded_refusals(lib):
    assert _expand(lib, cu=(1, 4)) == 1 and "cu_q" in _message(lib)
    assert _expand(lib, ck=(0, -4)) == 1 and "cu_kv" in _message(lib)
    assert _expand(lib, n=-1) == 1 and "n_seq" in _message(lib)
    assert _expand(lib, cu_dev=None) == 1 and _expand(lib, ck_dev=None) == 1
    for name in ("q", "k", "r", "v"):
        assert _expand(lib, **{name: _r(token=0)}) == 1 and "stride" in _message(lib)
        assert _expand(lib, **{name: _r(token=1 << 36)}) == 1 and "stride" in _message(lib)
    assert _expand(lib, cu=(0, 0)) == 0 and _expand(lib, cu=(0,), ck=(0,)) == 0


def _copy(lib, src, dst, n_pages=10, bases=(P,), sizes=(64,)):
    b, z = (ctypes.c_void_p * len(bases))(*bases), (ctypes.c_size_t * len(sizes))(*sizes)
    s, t = _cu(src), _cu(dst)
    return lib.gdn_copy_pages(len(bases), b, z, n_pages, len(src), s, t, None)


@pytest.mark.parametrize("src,dst,msg", [
    ([0], [10], "not in"), ([10], [0], "not in"), ([-1], [0], "not in"), ([0], [-1], "not in"),
    ([0, 1], [5, 5], "written twice"), ([0, 5], [5, 6], "read and written"), ([3], [3], "read and written"),
    ([9, 8, 7], [6, 5, 9], "read and written"),
])
def test_page_lists_that_overlap_or_leave_the_pool_are_refused(lib, src, dst, msg):
    assert _copy(lib, src, dst) == 1 and msg in _message(lib)


def test_copy_refusals(lib):
    assert _copy(lib, [0], [1], bases=(None,)) == 1 and _copy(lib, [0], [1], bases=(P + 2,)) == 1
    assert _copy(lib, [0], [1], sizes=(0,)) == 1 and _copy(lib, [0], [1], sizes=(6,)) == 1
    assert _copy(lib, [0], [1], sizes=((1 << 30) + 4,)) == 2
    assert _copy(lib, [0], [1], n_pages=-1) == 1 and _copy(lib, [0], [1], n_pages=0) == 1
    assert _copy(lib, [], []) == 0 and _copy(lib, [0], [1], bases=(), sizes=()) == 0
    assert lib.gdn_copy_pages(1, None, None, 10, 1, None, None, None) == 1


@pytest.mark.parametrize("site,call", [("latent_append", _append), ("latent_read", _read), ("latent_attention", _attend),
                                       ("expanded_attention", _expand), ("copy_pages", lambda lib: _copy(lib, [0], [1]))])
def test_injected_failures(lib, monkeypatch, site, call):
    """Valid calls end in the injected failure, before any CUDA call."""
    for value in (site, "all", f"conv,{site}"):
        monkeypatch.setenv("GDN_FAULT", value)
        assert call(lib) == gdn.GDN_ERR_INJECTED
        assert site in _message(lib)


def test_python_types_are_checked():
    with pytest.raises(ValueError, match="rope_style"):
        gdn.LatentDims(4, rope_style="full").c()
    d = gdn.LatentDims(4, 256, page_size=16)
    with pytest.raises(TypeError, match="rows"):
        gdn.LatentCache(d, None)
    with pytest.raises(TypeError, match="rows"):
        gdn.LatentCache(d, torch.zeros(2, 16, 320))
    with pytest.raises(ValueError, match="shape"):
        gdn.LatentCache(d, torch.zeros(2, 16, 256, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.LatentCache(d, torch.zeros(2, 16, 320, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="KVCache or LatentCache"):
        gdn.copy_pages([3], [0], [1])
    for src, dst, error in (([0], [1, 2], ValueError), ([0.5], [1], TypeError), (3, [1], TypeError),
                            ([2 ** 40], [1], ValueError), (torch.zeros(1), [1], TypeError)):
        with pytest.raises(error):
            gdn.copy_pages([], src, dst)
    assert gdn.copy_pages([], [], []) is None


def test_copied_dims_have_a_struct_of_their_own():
    import copy
    import pickle
    d = gdn.LatentDims(12, 256, page_size=32, scale=0.5)
    d.address()
    for e in (copy.deepcopy(d), pickle.loads(pickle.dumps(d)), copy.copy(d)):
        assert e == d and e.address() == ctypes.addressof(e.c())
    assert copy.deepcopy(d).address() != d.address()


@pytest.mark.parametrize("heads,token,head,overlap", [
    (8, 512, 64, False), (8, 504, 64, True), (8, 64, 256, False), (8, 64, 248, True), (8, 64, 64, True),
    (8, 128, 128, True), (8, 0, 64, True), (8, 512, 0, True), (1, 64, 0, False), (1, 56, 512, True),
])
def test_outputs_whose_rows_overlap_are_refused(lib, monkeypatch, heads, token, head, overlap):
    """4 tokens of 64 channels a head; accepted calls end in the injected failure."""
    monkeypatch.setenv("GDN_FAULT", "latent_append")
    got = _append(lib, d=_dims(n_heads=heads), q_out=_r(token=token, head=head))
    assert got == (1 if overlap else gdn.GDN_ERR_INJECTED)
    assert ("overlap" in _message(lib)) == overlap


@pytest.mark.parametrize("bases,sizes,overlap", [
    ((P, P + 640), (64, 64), False), ((P, P + 636), (64, 64), True), ((P, P), (64, 64), True),
    ((P + 640, P), (64, 64), False), ((P + 640, P, P + 320), (64, 32, 32), False), ((P + 640, P, P + 316), (64, 32, 32), True),
])
def test_arrays_that_overlap_are_refused(lib, monkeypatch, bases, sizes, overlap):
    monkeypatch.setenv("GDN_FAULT", "copy_pages")
    assert _copy(lib, [0], [1], bases=bases, sizes=sizes) == (1 if overlap else gdn.GDN_ERR_INJECTED)
    assert ("overlap" in _message(lib)) == overlap


def _calls(make):
    """The latent cache's calls as functions of their tensors."""
    d = gdn.LatentDims(2, 256, page_size=16)
    b, i, f = torch.bfloat16, torch.int32, torch.float32
    batch = {"cu": make((2,), i), "lens": make((1,), i), "table": make((1, 2), i)}
    rows = {"rows": make((3, 16, 320), b)}
    host = torch.tensor([0, 4], dtype=i)

    def cache(t):
        return gdn.LatentCache(d, t["rows"])

    def append(t):
        gdn.latent_append(d, cache(t), (t["cu"], host), t["lens"], t["table"], t["c"], norm_w=t["norm_w"], q_rope=t["q_rope"],
                          q_out=t["q_out"], rope=t["rope"], positions=t["positions"], rows_out=t["rows_out"])

    def read(t):
        gdn.latent_read(d, cache(t), (t["cu"], host), t["lens"], t["table"], out=t["out"])

    def attend(t):
        gdn.latent_attention(d, cache(t), (t["cu"], host), t["lens"], t["table"], t["q"], out=t["out"], workspace=t["ws"])

    def expand(t):
        gdn.expanded_attention(d, (t["cu"], host), (t["ck"], host), t["q"], t["k"], t["k_rope"], t["v"], out=t["out"])

    def copy(t):
        gdn.copy_pages([cache(t), gdn.LatentCache(d, t["more"])], [0], [1])

    return {
        "append": (append, {**batch, **rows, "c": make((4, 320), b), "norm_w": make((256,), f), "q_rope": make((4, 2, 64), b),
                            "q_out": make((4, 2, 64), b), "rope": make((9, 64), f), "positions": make((4,), i),
                            "rows_out": make((4, 320), b)}),
        "read": (read, {**batch, **rows, "out": make((4, 320), b)}),
        "attend": (attend, {**batch, **rows, "q": make((4, 2, 320), b), "out": make((4, 2, 256), b),
                            "ws": make((1 << 20,), torch.uint8)}),
        "expand": (expand, {"cu": make((2,), i), "ck": make((2,), i), "q": make((4, 2, 192), b), "k": make((4, 2, 128), b),
                            "k_rope": make((4, 64), b), "v": make((4, 2, 128), b), "out": make((4, 2, 128), b)}),
        "copy": (copy, {**rows, "more": make((3, 16, 320), b)}),
    }


@pytest.mark.parametrize("name", ["append", "read", "attend", "expand", "copy"])
@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_tensors_of_two_devices_are_refused(name):
    """Each tensor in turn on another device than the rest."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    mode = FakeTensorMode(allow_non_fake_inputs=True)

    def on(device):
        def make(shape, dtype):
            with mode:
                return torch.empty(shape, dtype=dtype, device=device)
        return make

    call, args = _calls(on("cuda:0"))[name]
    _, others = _calls(on("cuda:1"))[name]
    for moved in args:
        with pytest.raises(ValueError, match="device"):
            call({**args, moved: others[moved]})


def test_page_lists_may_change_while_they_are_read():
    """A list whose items' __index__ shortens it is read to its end as it is then."""
    src = []

    class Page:
        def __index__(self):
            del src[1:]
            return 3

    src += [Page(), Page(), Page()]
    with pytest.raises(ValueError, match=r"\(1, 3\)"):
        gdn.copy_pages([], src, [0, 1, 2])


def test_pieces_of_too_many_queries_are_refused(lib, monkeypatch):
    monkeypatch.setenv("GDN_FAULT", "expanded_attention")
    assert _expand(lib, cu=(0, 1 << 24), ck=(0, 1 << 24)) == gdn.GDN_ERR_INJECTED
    assert _expand(lib, cu=(0, 3, (1 << 24) + 4), ck=(0, 3, 9)) == 2 and "2^24" in _message(lib)
    assert _expand(lib, cu=(0, 3), ck=(0, 1 << 30)) == gdn.GDN_ERR_INJECTED
    assert _expand(lib, cu=(0, 3), ck=(0, (1 << 30) + 1)) == 2 and "2^30" in _message(lib)


def test_more_rows_than_32_bits_are_refused(lib, monkeypatch):
    monkeypatch.setenv("GDN_FAULT", "latent_attention,latent_append")
    d = _dims(n_heads=1024)
    for call in (_attend, _append):
        assert call(lib, d=d, b=_batch((0, (1 << 21) - 1)), **({"q_out": _r(token=1 << 16, head=64)} if call is _append else {})) == \
            gdn.GDN_ERR_INJECTED
        assert call(lib, d=d, b=_batch((0, 1 << 21))) == 2 and "rows" in _message(lib)


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_an_output_without_its_input_is_refused():
    from torch._subclasses.fake_tensor import FakeTensorMode
    mode = FakeTensorMode(allow_non_fake_inputs=True)

    def make(shape, dtype):
        with mode:
            return torch.empty(shape, dtype=dtype, device="cuda:0")

    call, args = _calls(make)["append"]
    with pytest.raises(ValueError, match="q_out without q_rope"):
        call({**args, "q_rope": None})


def test_workspace_sizes_of_any_form_of_lengths(lib):
    d = gdn.LatentDims(32, 512)
    want = gdn.latent_attention_workspace_size(d, [0, 1, 5])
    assert want > 0 and want == gdn.latent_attention_workspace_size(d, torch.tensor([0, 1, 5]))
    assert want == gdn.latent_attention_workspace_size(d, (None, torch.tensor([0, 1, 5], dtype=torch.int64)))
    assert gdn.latent_attention_workspace_size(d, [0]) == 0 and gdn.latent_attention_workspace_size(d, [0, 0, 0]) == 0
