"""Attention of prompts over the paged 8-bit cache: calls with enough 128-row
tiles for the tensor-memory kernel, against 64 bits (bounds: paged_cases.py).

Weights are single f16 numbers there: a weight below 2^-31 of its row's largest
is dropped, at most 2^-31 of the largest |value| a key, which the comparisons
of this file add to the bound (for rows of up to 2^11 keys 2^-20 of it)."""
import pytest
import torch

import gated_deltanet_linear_mixer_gb300 as gdn
from paged_cases import attention_ref, cu_of, gen, make_cache

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_deltanet_linear_mixer_gb300 import _build
    _build.build()
    gdn.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.fixture(autouse=True)
def _no_device_error():
    gdn.device_error(reset=True)
    yield
    assert gdn.device_error(reset=True) == 0


def _call(d, cache, table, counts, kv, q, **kw):
    """One call, which the tensor-memory kernel must have served."""
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    gdn.timing_enable(True)
    out = gdn.kv_attention(d, cache, cu_of(counts), lens, table, q, **kw)
    report = gdn.timing_report()
    gdn.timing_enable(False)
    assert set(report) == {"kv_prompt"}, report
    return out


def _excess(out, ref, size, top):
    got = out.double()
    assert torch.isfinite(got).all()
    tol = 2.0 ** -9 * size + 2.0 ** -8 * got.abs() + 2.0 ** -20 * top
    return float(((got - ref).abs() / tol.clamp(min=1e-30)).max())


def _check(d, counts, kv, seed, mags=(1.0,), edit=None):
    cache, table = make_cache(d, [max(n, 0) for n in kv], seed)
    if edit:
        edit(cache, table)
    q = torch.randn(sum(counts), d.n_q_heads, d.head_dim, generator=gen(seed + 1), device="cuda")
    mag = torch.tensor(mags, device="cuda")
    q = (q * mag[torch.arange(q.shape[0], device="cuda") % len(mags)][:, None, None]).to(BF)
    out = _call(d, cache, table, counts, kv, q)
    ref, size, _ = attention_ref(d, cache, table, counts, kv, q)
    top = float((cache.v.float().nan_to_num().abs().amax((2, 3)) * cache.v_scale.nan_to_num()).max())
    assert _excess(out, ref, size, top) <= 1.0
    return out


CASES = {
    # name: (Hq, Hkv, D, page, codes, window, counts, kv_lens)
    "d256_int8": (16, 2, 256, 64, "int8", 0, [700], [700]),
    "d256_e4m3_context": (16, 2, 256, 128, "e4m3", 0, [400, 333], [1000, 333]),
    "d256_page16_G4": (16, 4, 256, 16, "int8", 0, [130, 500, 64, 1], [129 + 130, 500, 65, 40]),
    "d128_int8": (32, 8, 128, 32, "int8", 0, [200], [200]),
    "d128_e4m3_ragged": (32, 8, 128, 16, "e4m3", 0, [1, 129, 0, 40, 333], [40, 129, 7, 1040, 400]),
    "d128_G1": (16, 16, 128, 64, "int8", 0, [150, 127, 128], [150, 300, 128]),
    "d128_G7": (28, 4, 128, 64, "e4m3", 0, [301], [555]),
    "d128_G64": (64, 1, 128, 128, "int8", 0, [90], [120]),
    "d64_int8": (8, 8, 64, 16, "int8", 0, [300, 20], [300, 520]),
    "d64_G3_e4m3": (24, 8, 64, 128, "e4m3", 0, [250], [777]),
    "window_d256": (16, 2, 256, 64, "int8", 150, [600], [1200]),
    "window_d128_ragged": (32, 8, 128, 16, "e4m3", 33, [100, 250, 5], [300, 250, 2000]),
    "window_1": (32, 8, 64, 16, "int8", 1, [200], [200]),
    "verify_many": (16, 2, 256, 64, "int8", 0, [8] * 24, [100 + 17 * i for i in range(24)]),
    "one_key_tiles": (64, 8, 128, 32, "int8", 0, [5] * 10, [5] * 10),
    "many_pages": (16, 4, 128, 16, "int8", 0, [700, 700], [1900, 700]),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_matches_64_bits(name):
    hq, hkv, dim, page, fmt, window, counts, kv = CASES[name]
    d = gdn.KVDims(hq, hkv, dim, page_size=page, cache=fmt, window=window)
    _check(d, counts, kv, len(name))


@pytest.mark.parametrize("dim,fmt", [(64, "e4m3"), (128, "int8"), (256, "int8"), (256, "e4m3")])
def test_large_and_tiny_queries(dim, fmt):
    """Scores far apart and alike in one tile; rows whose reference moves often."""
    d = gdn.KVDims(32, 8, dim, page_size=32, cache=fmt)
    _check(d, [300, 100], [300, 600], 5, mags=(1e-6, 0.0, 30.0, 1.0, 5.0))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scores_that_grow_along_the_keys(dim):
    """The reference moves at every tile: later keys score higher and higher."""
    d = gdn.KVDims(16, 8, dim, page_size=64)

    def edit(cache, table):
        for i, lens in enumerate((640, 900)):
            for lp in range(-(-lens // 64)):
                cache.k_scale[table[i, lp].long()] = 0.02 * (lp + 1)

    _check(d, [640, 500], [640, 900], 6, mags=(3.0,), edit=edit)


@pytest.mark.parametrize("dim", [128, 256])
def test_zero_scales_and_mixed_magnitudes(dim):
    d = gdn.KVDims(32, 8, dim, page_size=16)
    for low in (0.0, 2.0 ** -60):
        def edit(cache, table):
            cache.v_scale[::2] *= low
            cache.k_scale[::3] = 0.0
        _check(d, [200, 90], [333, 400], 7, edit=edit)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_that_see_nothing_are_zero(dim):
    """Sequences without cached tokens, and more queries than positions."""
    d = gdn.KVDims(32, 8, dim, page_size=16)
    counts, kv = [150, 200, 100], [0, 20, 100]
    out = _check(d, counts, kv, 8)
    assert not out[:150].any() and not out[150:330].any()


@pytest.mark.parametrize("dim", [128, 256])
def test_unmapped_pages(dim):
    """Keys of unmapped pages are not seen, and reported; windowed out they are not missed."""
    d = gdn.KVDims(16, 4, dim, page_size=32)
    counts, kv = [300, 200], [400, 200]
    cache, table = make_cache(d, kv, 9)
    q = torch.randn(500, 16, dim, generator=gen(10), device="cuda").to(BF)
    whole = _call(d, cache, table, counts, kv, q)
    holed = table.clone()
    holed[0, 5] = -1                       # positions 160..191 of sequence 0
    holed[1, 0] = cache.n_pages            # 0..31 of sequence 1
    out = _call(d, cache, holed, counts, kv, q)
    with pytest.raises(gdn.GDNError, match="code 40"):
        gdn.sync_status()
    assert torch.equal(out[: 160 - 100], whole[: 160 - 100])
    assert not out[300:332].any() and out[332:].any()
    # the hole's keys removed: the same attention as with K codes that score -inf there
    from paged_cases import line
    k, v = (line(d, cache, table, x, 0, 400).repeat_interleave(4, 1) for x in ("k", "v"))
    see = torch.ones(400, dtype=torch.bool, device="cuda")
    see[160:192] = False
    for t in (100, 250, 299):
        keys = see & (torch.arange(400, device="cuda") <= 100 + t)
        p = torch.softmax(torch.einsum("hd,khd->hk", q[t].double(), k[keys]) * dim ** -0.5, -1)
        ref, size = torch.einsum("hk,khd->hd", p, v[keys]), torch.einsum("hk,khd->hd", p, v[keys].abs())
        assert _excess(out[t], ref, size, float(v.abs().max())) <= 1.0
    w = gdn.KVDims(16, 4, dim, page_size=32, window=64)
    freed = table.clone()
    freed[0, :1] = -1                      # every query of sequence 0 is at 100 or later
    assert torch.equal(_call(w, cache, freed, [300, 200], kv, q), _call(w, cache, table, [300, 200], kv, q))


@pytest.mark.parametrize("dim", [128, 256])
def test_strides_streams_and_repeats(dim):
    d = gdn.KVDims(16, 4, dim, page_size=64)
    counts, kv = [300, 333], [300, 700]
    cache, table = make_cache(d, kv, 11)
    fused = torch.randn(633, 24, dim, generator=gen(12), device="cuda").to(BF)
    gated = torch.randn(633, 16, 2 * dim, generator=gen(13), device="cuda").to(BF)
    for q in (fused[:, 4:20], gated[..., dim:]):
        a = _call(d, cache, table, counts, kv, q)
        b = _call(d, cache, table, counts, kv, q.contiguous())
        assert torch.equal(a, b)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
            late = q + 0
            lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
            out = gdn.kv_attention(d, cache, cu_of(counts), lens, table, late)
            assert torch.equal(out, a)


def test_agrees_with_the_kernel_for_few_rows():
    """The same rows one call at a time (the other kernel) and together."""
    d = gdn.KVDims(16, 2, 256, page_size=64)
    counts, kv = [200, 150], [800, 150]
    cache, table = make_cache(d, kv, 14)
    q = torch.randn(350, 16, 256, generator=gen(15), device="cuda").to(BF)
    out = _call(d, cache, table, counts, kv, q)
    for t in (0, 77, 199):
        one = gdn.kv_attention(d, cache, cu_of([1]), torch.tensor([601 + t], dtype=torch.int32, device="cuda"),
                               table[:1], q[t:t + 1])
        assert (one[0].float() - out[t].float()).abs().max() <= 2.0 ** -6 * one.float().abs().max()
