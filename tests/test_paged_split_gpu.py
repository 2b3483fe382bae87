"""Attention of many rows whose keys are split over thread blocks and joined,
against 64 bits (bounds: paged_cases.py).

Weights are single f16 numbers: one below 2^-31 of its own range's reference is
dropped, which is at most 2^-31 of the row's largest |value| a key, so 2^-17 of
it over up to 2^14 keys, 2^-15 over 2^16; the join is fp32."""
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
    """One call, whose keys must have been split by the tensor-memory kernel."""
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    gdn.timing_enable(True)
    out = gdn.kv_attention(d, cache, cu_of(counts), lens, table, q, **kw)
    report = gdn.timing_report()
    gdn.timing_enable(False)
    assert set(report) == {"kv_prompt", "kv_attn_join"}, report
    return out


def _case(d, counts, kv, seed, mag=1.0):
    cache, table = make_cache(d, kv, seed)
    q = torch.randn(sum(counts), d.n_q_heads, d.head_dim, generator=gen(seed + 1), device="cuda") * mag
    return cache, table, q.to(BF)


def _excess(d, cache, table, counts, kv, q, out):
    ref, size, _ = attention_ref(d, cache, table, counts, kv, q)
    top = float((cache.v.float().nan_to_num().abs().amax((2, 3)) * cache.v_scale.nan_to_num()).max())
    got = out.double()
    assert torch.isfinite(got).all()
    drop = 2.0 ** -17 if max(kv) <= 1 << 14 else 2.0 ** -15
    tol = 2.0 ** -9 * size + 2.0 ** -8 * got.abs() + drop * top
    return float(((got - ref).abs() / tol.clamp(min=1e-30)).max())


CASES = {
    # name: (Hq, Hkv, D, page, codes, window, counts, kv_lens)
    "d256_long": (16, 2, 256, 64, "int8", 0, [64], [8064]),
    "d256_e4m3_odd": (8, 1, 256, 128, "e4m3", 0, [70], [3333]),
    "d256_three_rows_of_G8": (16, 2, 256, 16, "int8", 0, [3], [9001]),  # too little work: the other kernel's
    "d256_three_rows_longer": (16, 2, 256, 16, "int8", 0, [3], [12001]),
    "d128_ragged": (32, 8, 128, 16, "e4m3", 0, [40, 1, 0, 33], [4100, 1, 0, 900]),
    "d128_int8_two_tiles": (16, 2, 128, 64, "int8", 0, [50], [2050]),
    "d128_G7": (28, 4, 128, 32, "int8", 0, [61], [5000]),
    "d64_G1": (8, 8, 64, 128, "int8", 0, [130], [4130]),
    "d64_e4m3": (16, 2, 64, 16, "e4m3", 0, [17], [6017]),
    "one_block_wide_join": (4, 1, 128, 64, "int8", 0, [32], [20000]),
    "window": (16, 2, 256, 64, "int8", 2000, [40], [6000]),
    "window_ragged": (32, 8, 128, 32, "e4m3", 1500, [90, 10], [1600, 5000]),
    "prompt_from_empty": (8, 1, 128, 64, "int8", 0, [1500], [1500]),
    "verify_many": (16, 2, 256, 64, "int8", 0, [8] * 12, [2500 - 200 * i for i in range(12)]),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_matches_64_bits(name):
    hq, hkv, dim, page, fmt, window, counts, kv = CASES[name]
    d = gdn.KVDims(hq, hkv, dim, page_size=page, cache=fmt, window=window)
    cache, table, q = _case(d, counts, kv, len(name))
    if name == "d256_three_rows_of_G8":
        out = gdn.kv_attention(d, cache, cu_of(counts), torch.tensor(kv, dtype=torch.int32, device="cuda"), table, q)
    else:
        out = _call(d, cache, table, counts, kv, q)
    assert _excess(d, cache, table, counts, kv, q, out) <= 1.0


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_references_far_apart_between_ranges(dim):
    """Scores that dwarf one another: most ranges count for nothing, another each row."""
    d = gdn.KVDims(16, 2, dim, page_size=64)
    counts, kv = [64], [4096]
    cache, table, q = _case(d, counts, kv, 21, mag=40.0)
    out = _call(d, cache, table, counts, kv, q)
    assert _excess(d, cache, table, counts, kv, q, out) <= 1.0


@pytest.mark.parametrize("dim", [128, 256])
def test_rows_and_ranges_that_see_nothing(dim):
    """A sequence without cached tokens and one with more queries than positions, beside a long one."""
    d = gdn.KVDims(16, 2, dim, page_size=32)
    counts, kv = [40, 50, 30], [0, 20, 5000]
    cache, table, q = _case(d, counts, kv, 22)
    out = _call(d, cache, table, counts, kv, q)
    assert not out[:70].any()
    assert _excess(d, cache, table, counts, kv, q, out) <= 1.0


@pytest.mark.parametrize("bound", [2000, 4064, 60000])
def test_any_bound_on_the_lengths(bound):
    """max_kv_len only sets the ranges: too small a one leaves the rest to the last."""
    d = gdn.KVDims(16, 2, 256, page_size=64)
    counts, kv = [64, 20], [4064, 700]
    cache, table, q = _case(d, counts, kv, 23)
    out = _call(d, cache, table, counts, kv, q, max_kv_len=bound)
    assert _excess(d, cache, table, counts, kv, q, out) <= 1.0


def test_workspace_is_asked_for_and_checked():
    d = gdn.KVDims(16, 2, 256, page_size=64)
    counts, kv = [64], [4096]
    cache, table, q = _case(d, counts, kv, 24)
    need = gdn.kv_attention_workspace_size(d, [0, 64], 4096)
    assert need > 0
    a = _call(d, cache, table, counts, kv, q, max_kv_len=4096)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns: nothing unwritten is read
    assert torch.equal(a, _call(d, cache, table, counts, kv, q, max_kv_len=4096, workspace=ws))
    with pytest.raises((gdn.GDNError, ValueError)):
        gdn.kv_attention(d, cache, cu_of(counts), torch.tensor(kv, dtype=torch.int32, device="cuda"), table, q,
                         max_kv_len=4096, workspace=ws[:need - 256])


def test_unmapped_pages():
    d = gdn.KVDims(16, 2, 128, page_size=64)
    counts, kv = [64], [4096]
    cache, table, q = _case(d, counts, kv, 25)
    holed = table.clone()
    holed[0, 10:40] = -1  # whole ranges among them
    out = _call(d, cache, holed, counts, kv, q)
    with pytest.raises(gdn.GDNError, match="code 40"):
        gdn.sync_status()
    kept = torch.cat([table[0, :10], table[0, 40:]])[None].contiguous()
    ref = _call(d, cache, kept, counts, [4096 - 30 * 64], q)
    # the same keys either way, each side within its bound of 2^-9 and half a unit of bf16
    assert (out.float() - ref.float()).abs().max() <= 2.0 ** -6 * ref.float().abs().max()


def test_repeats_bit_for_bit_and_in_a_graph():
    d = gdn.KVDims(16, 2, 256, page_size=64)
    counts, kv = [64], [8064]
    cache, table, q = _case(d, counts, kv, 26)
    a = _call(d, cache, table, counts, kv, q)
    assert torch.equal(a, _call(d, cache, table, counts, kv, q))
    lens, cu = torch.tensor(kv, dtype=torch.int32, device="cuda"), cu_of(counts)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gdn.kv_attention(d, cache, cu, lens, table, q)
    out.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, out)
