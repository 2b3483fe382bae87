"""Edges of the paged-cache operators on the GPU: value scales of zero, subnormal and far apart,
pages that a window has left behind, windows near 2^31.

References and bounds are those of paged_cases.py; calls of many rows add the weights that f16
drops, 2^-31 of the reference a key (2^-20 of the largest |value| for up to 2^11 keys)."""
import copy

import pytest
import torch

import gated_deltanet_linear_mixer_gb300 as gdn
from paged_cases import attention_excess, attention_ref, cu_of, gen, make_cache

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


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


FORMS = {
    # name: (Hq, Hkv, D, dtype, queries, kernels of a call that ends at position 1600)
    "few": (16, 2, 128, BF, [1], {"kv_attn", "kv_attn_join"}),
    "few_f32": (16, 2, 256, F32, [3], {"kv_attn", "kv_attn_join"}),
    "prompt": (32, 8, 128, BF, [600], {"kv_prompt"}),
    "prompt_d256": (32, 8, 256, BF, [300], {"kv_prompt"}),
    "split": (16, 2, 128, BF, [40], {"kv_prompt", "kv_attn_join"}),
    "split_d256": (16, 2, 256, BF, [40], {"kv_prompt", "kv_attn_join"}),
}


def _call(d, cache, table, counts, kv, q, kernels):
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    gdn.timing_enable(True)
    out = gdn.kv_attention(d, cache, cu_of(counts), lens, table, q)
    report = gdn.timing_report()
    gdn.timing_enable(False)
    assert set(report) == kernels, report
    return out


def _excess(d, cache, table, counts, kv, q, out):
    ref, size, s = attention_ref(d, cache, table, counts, kv, q)
    if d.dtype == F32:
        return attention_excess(d, out, ref, size, s)
    got = out.double()
    assert torch.isfinite(got).all()
    values = torch.stack([cache.v[p].float().abs().amax((1, 2)) * cache.v_scale[p] for p in table[0].tolist() if p >= 0])
    tol = 2.0 ** -9 * size + 2.0 ** -8 * got.abs() + 2.0 ** -20 * float(values.max())
    return float(((got - ref).abs() / tol.clamp(min=1e-36)).max())


@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("power", [-20, -40, -80, 0, 60])
def test_values_after_many_keys_of_zeros(form, power):
    """1280 keys whose values are all zero, then values of scale 2^power: the zeros count in the
    softmax's sum and leave the others' weights their precision."""
    hq, hkv, dim, dtype, counts, kernels = FORMS[form]
    d = gdn.KVDims(hq, hkv, dim, page_size=64, dtype=dtype)
    kv = [1600]
    cache, table = make_cache(d, kv, 81)
    pages = table[0].long()
    cache.v_scale[pages[:20]] = 0.0
    cache.v_scale[pages[20:]] *= 2.0 ** power
    q = (torch.randn(sum(counts), hq, dim, generator=gen(82), device="cuda") * 0.3).to(dtype)
    out = _call(d, cache, table, counts, kv, q, kernels)
    assert out.any()
    assert _excess(d, cache, table, counts, kv, q, out) <= 1.0


@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("tiny", [1e-39, 1e-45, 2.0 ** -100])
def test_pages_of_tiny_values_beside_ordinary_ones(form, tiny):
    """Value scales whose reciprocal is no fp32 number, as appended values near the smallest normal
    numbers have them, among scales of ordinary size and of zero."""
    hq, hkv, dim, dtype, counts, kernels = FORMS[form]
    d = gdn.KVDims(hq, hkv, dim, page_size=64, dtype=dtype)
    kv = [1600]
    for zeros in (False, True):
        cache, table = make_cache(d, kv, 83)
        pages = table[0].long()
        cache.v_scale[pages[3]] = tiny
        cache.v_scale[pages[22]] = tiny
        if zeros:
            cache.v_scale[pages[4]] = 0.0
        q = (torch.randn(sum(counts), hq, dim, generator=gen(84), device="cuda") * 0.3).to(dtype)
        out = _call(d, cache, table, counts, kv, q, kernels)
        assert _excess(d, cache, table, counts, kv, q, out) <= 1.0


@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("fmt,page", [("e4m3", 16), ("int8", 32)])
def test_pages_left_behind_by_the_window_may_hold_anything(form, fmt, page):
    """Pages before every query's window may have been given to other sequences: what their entries
    point to (unwritten pages with scales and codes that are no numbers) does not reach a result."""
    hq, hkv, dim, dtype, counts, _ = FORMS[form]
    kv = [1600]
    for window in (600, 601, 657):
        d = gdn.KVDims(hq, hkv, dim, page_size=page, dtype=dtype, cache=fmt, window=window)
        cache, table = make_cache(d, kv, 85)
        q = torch.randn(sum(counts), hq, dim, generator=gen(86), device="cuda").to(dtype)
        lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
        hints = (None, 64)  # 64: the keys in one range, as in a call of many sequences
        clean = [gdn.kv_attention(d, cache, cu_of(counts), lens, table, q, max_kv_len=n) for n in hints]
        assert all(_excess(d, cache, table, counts, kv, q, x) <= 1.0 for x in clean)
        gone = max(0, kv[0] - counts[0] - window + 1) // page
        old = table[0, :gone].long()
        for x in (cache.k, cache.v):
            x.view(torch.int8)[old] = 0x7F
        for x in (cache.k_scale, cache.v_scale):
            x[old] = float("nan")
        for n, x in zip(hints, clean):
            assert torch.equal(gdn.kv_attention(d, cache, cu_of(counts), lens, table, q, max_kv_len=n), x)


@pytest.mark.parametrize("counts", [[5], [300]])
@pytest.mark.parametrize("dim", [128, 256])
def test_the_widest_window_is_none(dim, counts):
    """A window of 2^31 - 1 leaves nothing out, of sequences with more queries than positions either."""
    kv = [counts[0] - 2]
    d = gdn.KVDims(16, 8, dim, page_size=64)
    wide = gdn.KVDims(16, 8, dim, page_size=64, window=2 ** 31 - 1)
    cache, table = make_cache(d, kv, 87)
    q = torch.randn(sum(counts), 16, dim, generator=gen(88), device="cuda").to(BF)
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    a = gdn.kv_attention(d, cache, cu_of(counts), lens, table, q)
    b = gdn.kv_attention(wide, cache, cu_of(counts), lens, table, q)
    assert a[2:].any() and torch.equal(a, b)


def test_a_cache_s_tensors_may_be_replaced():
    """A call takes the tensors that the cache holds then: a cache that grew is written to and read
    where it is now."""
    d = gdn.KVDims(4, 2, 64, page_size=16)
    cache, table = make_cache(d, [16], 89, poison=False)
    old = (cache.k, cache.v, cache.k_scale, cache.v_scale)
    before = [x.clone() for x in old]
    for name, x in zip(("k", "v", "k_scale", "v_scale"), old):
        setattr(cache, name, torch.cat([x, torch.zeros_like(x)]))
    new = torch.randn(16, 2, 64, generator=gen(90), device="cuda").to(BF)
    lens = torch.tensor([16], dtype=torch.int32, device="cuda")
    entry = torch.full_like(table, cache.k.shape[0] - 1)  # a page that only the grown cache has
    gdn.kv_append(d, cache, cu_of([16]), lens, entry, new, new)
    k, _ = gdn.kv_read(d, cache, cu_of([16]), lens * 0, entry, dtype=F32)
    assert (k - new.float()).abs().max() < 0.03
    assert all(torch.equal(x, y) for x, y in zip(old, before))


def test_a_copied_cache_is_its_own():
    d = gdn.KVDims(4, 2, 64, page_size=16)
    cache, table = make_cache(d, [16], 92, poison=False)
    twin = copy.deepcopy(cache)
    new = torch.randn(16, 2, 64, generator=gen(93), device="cuda").to(BF)
    lens = torch.tensor([16], dtype=torch.int32, device="cuda")
    gdn.kv_append(d, twin, cu_of([16]), lens, table, new, new)
    k, _ = gdn.kv_read(d, twin, cu_of([16]), lens * 0, table, dtype=F32)
    assert (k - new.float()).abs().max() < 0.03
    fresh, _ = make_cache(d, [16], 92, poison=False)
    assert torch.equal(cache.k, fresh.k) and torch.equal(cache.k_scale, fresh.k_scale)
