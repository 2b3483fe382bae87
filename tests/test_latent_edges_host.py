"""CPU checks of the latent operators at their edges: what the sources may not hold, and refusals."""
import ctypes
import pathlib
import random
import re

import pytest
import torch

import gated_deltanet_linear_mixer_gb300 as gdn
from gated_deltanet_linear_mixer_gb300 import _build

P = 1 << 20  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gdn.load()


def _append(lib, heads, tokens, c, q=None, q_out=None, packed=None, rows=1 << 40):
    """c (base, token stride), q and q_out (base, token stride, head stride), strides in channels."""
    d = gdn._LatentDims(heads, 256, 64, 16, 0, 128, 128, 0.07, 1e-6)
    host = (ctypes.c_int32 * 2)(0, tokens)
    b = gdn._KVBatch(1, 1, P, ctypes.cast(host, ctypes.c_void_p).value, P)
    refs = [ctypes.byref(gdn._Rows(*r)) if r else None for r in ((*c, 0), q, q_out)]
    cache = gdn._LatentCache(rows, 3)
    return lib.gdn_latent_append(ctypes.byref(d), ctypes.byref(cache), ctypes.byref(b), P, refs[0], None, refs[1], refs[2], None, 0,
                                 None, packed, None)


def test_no_load_is_multicast():
    """One library serves single processes and replicas of several GPUs: no thread block's bulk load
    writes into another's shared memory."""
    files = [p for p in pathlib.Path(_build.CSRC).iterdir() if p.suffix in (".cu", ".cuh", ".h", ".cpp")]
    assert len(files) > 20
    for p in files:
        text = re.sub(r'"\s*"', "", p.read_text())  # literals side by side are one
        assert not re.search(r"cp\.async\.bulk[\w.:]*multicast", text), p.name


def test_a_q_out_without_q_rope_is_refused(lib, monkeypatch):
    monkeypatch.setenv("GDN_FAULT", "latent_append")
    c = (P, 320)
    assert _append(lib, 2, 4, c) == gdn.GDN_ERR_INJECTED
    assert _append(lib, 2, 4, c, q_out=(2 * P, 128, 64)) == 1 and b"q_out is given without q_rope" in lib.gdn_last_error()
    assert _append(lib, 2, 4, c, q=(3 * P, 128, 64), q_out=(2 * P, 128, 64)) == gdn.GDN_ERR_INJECTED


def _bytes(base, tokens, heads, token, head, channels):
    return {base + 2 * (t * token + h * head) + x for t in range(tokens) for h in range(heads) for x in range(0, 2 * channels, 16)}


def _apart(tokens, heads, token, head, width=64):
    """Whether the rows of an output are taken as not overlapping."""
    ts, hs = token if tokens > 1 else 1 << 60, head if heads > 1 else 1 << 60
    if ts < width or hs < width:
        return False
    return tokens == 1 or heads == 1 or (heads - 1) * hs + width <= ts or (tokens - 1) * ts + width <= hs


def test_outputs_in_the_queries_memory(lib, monkeypatch):
    """q_out in q_rope's memory at random strides, against the sets of their bytes: q_rope itself, or apart."""
    monkeypatch.setenv("GDN_FAULT", "latent_append")
    r = random.Random(5)
    seen = {True: 0, False: 0}
    while min(seen.values()) < 300:
        tokens, heads = r.randint(1, 5), r.randint(1, 4)
        first = r.random() < 0.7  # heads within a token
        head = 64 * r.randint(1, 5) if first else 0
        token = r.choice([0, 8, 64]) + heads * head if first else 64 * r.randint(1, 3)
        if not first:
            head = tokens * token + r.choice([0, 8, 64])
        q = (P, token, head)
        out_head = r.choice([head, head, head + 8, 64])
        out = (P + 16 * r.randint(-100, 100) * r.choice([0, 1, 1]), token, out_head)
        if not _apart(tokens, heads, token, out_head):
            continue
        alike = out[0] == q[0] and (heads == 1 or out_head == head)
        meet = not alike and bool(_bytes(P, tokens, heads, token, head, 64) & _bytes(out[0], tokens, heads, token, out_head, 64))
        got = _append(lib, heads, tokens, (1 << 30, 320), q, out)
        assert got == (1 if meet else gdn.GDN_ERR_INJECTED), (tokens, heads, q, out)
        assert (b"q_out shares memory with q_rope" in lib.gdn_last_error()) == meet
        seen[meet] += 1


def test_packed_rows_in_the_inputs_memory(lib, monkeypatch):
    """rows_out in the memory of c, of q or of the cache: c itself where that is contiguous, or apart."""
    monkeypatch.setenv("GDN_FAULT", "latent_append")
    r = random.Random(6)
    seen = {True: 0, False: 0}
    while min(seen.values()) < 200:
        tokens, token = r.randint(1, 4), 320 + r.choice([0, 8, 320, 2000])
        out = P + 16 * r.randint(-90, 250) * r.choice([0, 1, 1])
        alike = out == P and (tokens == 1 or token == 320)
        meet = not alike and bool(_bytes(P, tokens, 1, token, 0, 320) & _bytes(out, tokens, 1, 320, 0, 320))
        assert _append(lib, 1, tokens, (P, token), packed=out) == (1 if meet else gdn.GDN_ERR_INJECTED), (tokens, token, out - P)
        seen[meet] += 1
    c, q, to = (P, 320), (2 * P, 128, 64), (3 * P, 128, 64)
    size = 4 * 320 * 2
    for base, end in ((2 * P, 2 * P + 4 * 256), (3 * P, 3 * P + 4 * 256), (1 << 40, (1 << 40) + 3 * 16 * 640)):
        for out, bad in ((base, True), (base - size + 16, True), (end - 16, True), (base - size, False), (end, False)):
            assert _append(lib, 2, 4, c, q, to, packed=out) == (1 if bad else gdn.GDN_ERR_INJECTED)


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_caches_may_change_while_page_lists_are_read():
    """The caches are looked at as they are once both lists are read."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    d = gdn.LatentDims(1, 256, page_size=16)
    with FakeTensorMode():
        cache = gdn.LatentCache(d, torch.empty(4, 16, 320, dtype=torch.bfloat16, device="cuda:0"))

    class Page:
        def __index__(self):
            cache.rows.resize_(7)
            return 3

    with pytest.raises(ValueError, match="contiguous"):
        gdn.copy_pages(cache, [0], [Page()])


@pytest.mark.parametrize("scale,ok", [(2.3e38, True), (2.4e38, False), (3.4e38, False), (1e-45, True)])
def test_scales_that_leave_fp32_in_powers_of_two_are_refused(lib, scale, ok):
    d, n, host = gdn._LatentDims(2, 256, 64, 16, 0, 128, 128, scale, 1e-6), ctypes.c_size_t(0), (ctypes.c_int32 * 2)(0, 4)
    got = lib.gdn_latent_attention_workspace_size(ctypes.byref(d), 1, ctypes.cast(host, ctypes.c_void_p), ctypes.byref(n))
    assert got == (0 if ok else 1) and (ok or b"scale" in lib.gdn_last_error())
