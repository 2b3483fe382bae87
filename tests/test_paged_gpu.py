"""The paged 8-bit cache on the GPU: appending with rotation, attention over it
and reading it back, against plain 64-bit implementations (paged_cases.py)."""
import pytest
import torch

import gated_deltanet_linear_mixer_gb300 as gdn
from paged_cases import (QMAX, attention_excess, attention_ref, cu_of, gen, lengths, line, make_cache,
                         rope_table, turn)

pytestmark = pytest.mark.gpu


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


# ---------------------------------------------------------------- attention
def _attend(d, counts, kv_lens, seed, q=None, **kw):
    cache, table = make_cache(d, [max(n, 0) for n in kv_lens], seed)
    if q is None:
        q = torch.randn(sum(counts), d.n_q_heads, d.head_dim, generator=gen(seed + 1), device="cuda")
        q = q.to(d.dtype)
    lens = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
    out = gdn.kv_attention(d, cache, cu_of(counts), lens, table, q, **kw)
    ref = attention_ref(d, cache, table, counts, kv_lens, q)
    return out, ref, (cache, table, lens, q)


BF, F32 = torch.bfloat16, torch.float32
ATTN = {
    # name: (Hq, Hkv, D, page, dtype, codes, window, counts, kv_lens)
    "one_token_one_key": (4, 2, 64, 16, BF, "int8", 0, [1], [1]),
    "decode_G8_d256": (16, 2, 256, 64, BF, "int8", 0, [1] * 5, [1, 63, 64, 65, 1000]),
    "decode_G1_d64": (3, 3, 64, 16, BF, "e4m3", 0, [1] * 4, [5, 16, 17, 333]),
    "decode_G3_d128": (6, 2, 128, 32, BF, "int8", 0, [1] * 3, [31, 129, 700]),
    "decode_G7_d256": (14, 2, 256, 16, BF, "e4m3", 0, [1, 1], [40, 257]),
    "decode_G64_d128": (64, 1, 128, 128, BF, "int8", 0, [1, 1], [127, 300]),
    "decode_long": (16, 2, 256, 64, BF, "int8", 0, [1], [20011]),
    "decode_long_e4m3": (8, 8, 128, 128, BF, "e4m3", 0, [1, 1], [9001, 77]),
    "verify_T4": (16, 4, 128, 16, BF, "int8", 0, [4] * 4, [4, 5, 130, 999]),
    "verify_T16_G8": (16, 2, 256, 64, BF, "e4m3", 0, [16, 16], [16, 500]),
    "verify_ragged": (8, 2, 64, 32, BF, "int8", 0, [3, 0, 1, 9], [50, 70, 1, 9]),
    "prompt": (4, 2, 128, 64, BF, "int8", 0, [300], [300]),
    "prompt_d256": (8, 1, 256, 64, BF, "int8", 0, [257], [257]),
    "prompt_d256_e4m3_ctx": (4, 2, 256, 128, BF, "e4m3", 0, [130, 64], [1000, 65]),
    "prompt_d64_G5": (5, 1, 64, 16, BF, "e4m3", 0, [200, 1, 77], [200, 512, 90]),
    "prompts_ragged": (16, 4, 128, 32, BF, "int8", 0, [1, 129, 0, 40, 333], [40, 129, 7, 1040, 400]),
    "window_decode": (16, 2, 256, 64, BF, "int8", 100, [1] * 3, [50, 100, 1000]),
    "window_1": (4, 2, 64, 16, BF, "int8", 1, [5, 1], [20, 300]),
    "window_prompt": (8, 2, 128, 16, BF, "e4m3", 33, [200, 30], [300, 31]),
    "window_prompt_d256": (8, 2, 256, 64, BF, "int8", 150, [300], [900]),
    "f32_decode": (16, 2, 256, 64, F32, "int8", 0, [1] * 3, [1, 65, 1500]),
    "f32_verify_e4m3": (6, 2, 128, 32, F32, "e4m3", 0, [5, 2], [5, 300]),
    "f32_prompt": (4, 4, 64, 16, F32, "int8", 0, [150], [170]),
    "f32_prompt_d256_window": (8, 2, 256, 16, F32, "e4m3", 40, [70, 3], [100, 200]),
    "f32_decode_long": (8, 2, 128, 64, F32, "int8", 0, [1, 1], [7001, 3]),
}


@pytest.mark.parametrize("name", sorted(ATTN))
def test_attention_matches_64_bits(name):
    hq, hkv, dim, page, dtype, fmt, window, counts, kv = ATTN[name]
    d = gdn.KVDims(hq, hkv, dim, page_size=page, dtype=dtype, cache=fmt, window=window)
    out, ref, _ = _attend(d, counts, kv, seed=len(name))
    assert attention_excess(d, out, *ref) <= 1.0


@pytest.mark.parametrize("seed", range(12))
def test_attention_random_shapes(seed):
    import random
    r = random.Random(100 + seed)
    hkv, g = r.choice([1, 2, 4]), r.choice([1, 2, 5, 8, 16])
    d = gdn.KVDims(hkv * g, hkv, r.choice([64, 128, 256]), page_size=r.choice([16, 32, 64, 128]),
                   dtype=r.choice([BF, BF, F32]), cache=r.choice(["int8", "e4m3"]),
                   window=r.choice([0, 0, r.randint(1, 300)]))
    q_hi = r.choice([1, 8, 40, 300])
    counts, kv = lengths(seed, r.randint(1, 6), q_hi, r.choice([0, 50, 2000]), q_lo=0)
    if not sum(counts):
        counts[0], kv[0] = 1, kv[0] + 1
    out, ref, _ = _attend(d, counts, kv, seed)
    assert attention_excess(d, out, *ref) <= 1.0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("counts", [[1, 1, 1], [40, 200, 1], [0, 3, 2]])
def test_rows_that_see_nothing_are_zero(dtype, counts):
    """Lengths of zero, and more queries than positions: queries before position 0 see no key."""
    d = gdn.KVDims(8, 2, 128, page_size=16, dtype=dtype)
    kv = [0, 2, counts[2]]
    cache, table = make_cache(d, kv, 3)
    q = torch.randn(sum(counts), 8, 128, generator=gen(4), device="cuda").to(dtype)
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    out = gdn.kv_attention(d, cache, cu_of(counts), lens, table, q)
    ref = attention_ref(d, cache, table, counts, kv, q)
    assert attention_excess(d, out, *ref) <= 1.0
    blind = max(0, counts[1] - 2)
    assert not out[: counts[0]].any() and not out[counts[0]: counts[0] + blind].any()


@pytest.mark.parametrize("name", ["decode_G8_d256", "verify_T16_G8", "prompt_d256_e4m3_ctx", "f32_decode"])
def test_large_and_tiny_queries(name):
    """Scores far apart (one key takes all) and scores all alike; queries above f16's range."""
    hq, hkv, dim, page, dtype, fmt, window, counts, kv = ATTN[name]
    d = gdn.KVDims(hq, hkv, dim, page_size=page, dtype=dtype, cache=fmt, window=window)
    q = torch.randn(sum(counts), hq, dim, generator=gen(9), device="cuda")
    mag = torch.tensor([1e-6, 0.0, 30.0, 1.0], device="cuda")
    q *= mag[torch.arange(q.shape[0], device="cuda") % 4][:, None, None]
    out, ref, _ = _attend(d, counts, kv, 17, q=q.to(dtype))
    if dtype == BF:
        assert attention_excess(d, out, *ref) <= 1.0
    else:
        assert attention_excess(d, out, *ref) <= 1.0
    # one row scaled by 2^20: a score scale of 2^-20 gives the same attention
    d2 = gdn.KVDims(hq, hkv, dim, page_size=page, dtype=dtype, cache=fmt, scale=dim ** -0.5 * 2.0 ** -20)
    q1 = torch.randn(sum(counts), hq, dim, generator=gen(10), device="cuda").to(dtype)
    cache, table = make_cache(d, kv, 18)
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    one = gdn.kv_attention(d, cache, cu_of(counts), lens, table, q1)
    two = gdn.kv_attention(d2, cache, cu_of(counts), lens, table, q1 * 2.0 ** 20)
    assert torch.equal(one, two)


def test_zero_scales_and_mixed_magnitudes():
    """Blocks of zeros (scale 0) and value scales 2^60 apart."""
    d = gdn.KVDims(16, 2, 128, page_size=16)
    counts, kv = [1, 2, 150], [100, 333, 400]
    for mags in ([0.0, 1.0], [2.0 ** -60, 1.0], [0.0, 0.0]):
        cache, table = make_cache(d, kv, 5)
        cache.v_scale[::2] *= mags[0]
        cache.v_scale[1::2] *= mags[1]
        cache.k_scale[::3] = 0.0
        q = torch.randn(sum(counts), 16, 128, generator=gen(6), device="cuda").to(BF)
        lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
        out = gdn.kv_attention(d, cache, cu_of(counts), lens, table, q)
        assert attention_excess(d, out, *attention_ref(d, cache, table, counts, kv, q)) <= 1.0


@pytest.mark.parametrize("name", ["decode_long", "verify_T4", "prompts_ragged", "f32_decode_long"])
def test_attention_is_deterministic_and_reads_no_stale_workspace(name):
    hq, hkv, dim, page, dtype, fmt, window, counts, kv = ATTN[name]
    d = gdn.KVDims(hq, hkv, dim, page_size=page, dtype=dtype, cache=fmt, window=window)
    out, _, (cache, table, lens, q) = _attend(d, counts, kv, 21)
    size = gdn.kv_attention_workspace_size(d, cu_of(counts), max(kv))
    for byte in (0xFF, 0x00):
        ws = torch.full((max(size, 256),), byte, dtype=torch.uint8, device="cuda")
        again = gdn.kv_attention(d, cache, cu_of(counts), lens, table, q, max_kv_len=max(kv), workspace=ws)
        wide = gdn.kv_attention(d, cache, cu_of(counts), lens, table, q)
        assert torch.equal(again, gdn.kv_attention(d, cache, cu_of(counts), lens, table, q, max_kv_len=max(kv)))
        assert torch.equal(wide, out)


@pytest.mark.parametrize("counts,kv", [([1, 1], [3000, 40]), ([150], [700])])
def test_max_kv_len_below_the_lengths_still_attends_in_full(counts, kv):
    d = gdn.KVDims(8, 2, 128, page_size=32)
    cache, table = make_cache(d, kv, 8)
    q = torch.randn(sum(counts), 8, 128, generator=gen(9), device="cuda").to(BF)
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    ref = attention_ref(d, cache, table, counts, kv, q)
    for hint in (0, 1, 500):
        out = gdn.kv_attention(d, cache, cu_of(counts), lens, table, q, max_kv_len=hint)
        assert attention_excess(d, out, *ref) <= 1.0


@pytest.mark.parametrize("counts", [[1] * 3, [70, 9, 200]])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_strided_queries(counts, dtype):
    """q as a slice of a fused projection, and interleaved per head with a gate."""
    kv = [c + 100 for c in counts]
    d = gdn.KVDims(8, 2, 128, page_size=32, dtype=dtype)
    cache, table = make_cache(d, kv, 31)
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    fused = torch.randn(sum(counts), 12, 128, generator=gen(32), device="cuda").to(dtype)
    gated = torch.randn(sum(counts), 8, 256, generator=gen(33), device="cuda").to(dtype)
    for q in (fused[:, 2:10], gated[..., :128], gated[..., 128:]):
        a = gdn.kv_attention(d, cache, cu_of(counts), lens, table, q)
        b = gdn.kv_attention(d, cache, cu_of(counts), lens, table, q.contiguous())
        assert torch.equal(a, b)


def test_offsets_past_2_31():
    """Pages at the far end of a cache of more than 2^31 codes: decode, prompt, append, read."""
    d = gdn.KVDims(16, 2, 256, page_size=64, rope_dim=64)
    n_pages = 70000
    cache = gdn.KVCache(d, *(torch.zeros(n_pages, 2, 64, 256, dtype=torch.int8, device="cuda") for _ in "kv"),
                        *(torch.zeros(n_pages, 2, device="cuda") for _ in "kv"))
    counts, kv = [1, 70], [200, 270]
    table = torch.stack([torch.arange(n_pages - 5, n_pages), torch.arange(n_pages - 10, n_pages - 5)])
    table = table.to(torch.int32).cuda()
    g = gen(41)
    for name in ("k", "v"):
        getattr(cache, name)[-10:] = torch.randint(-127, 128, (10, 2, 64, 256), generator=g, device="cuda").to(torch.int8)
        getattr(cache, name + "_scale")[-10:] = 0.01
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    rope = rope_table(300, 64)
    q = torch.randn(71, 16, 256, generator=g, device="cuda").to(BF)
    kn, vn = (torch.randn(71, 2, 256, generator=g, device="cuda").to(BF) for _ in "kv")
    gdn.kv_append(d, cache, cu_of(counts), lens, table, kn, vn, rope=rope)
    k, v = gdn.kv_read(d, cache, cu_of(counts), lens - torch.tensor(counts, dtype=torch.int32).cuda(), table,
                       dtype=torch.float32)
    assert (v - vn.float()).abs().max() < 0.04 and v[1:].std() > 0.5
    out = gdn.kv_attention(d, cache, cu_of(counts), lens, table, q)
    assert attention_excess(d, out, *attention_ref(d, cache, table, counts, kv, q)) <= 1.0
    assert not cache.k_scale[:-10].any()
    del cache
    torch.cuda.empty_cache()


@pytest.mark.parametrize("counts", [[1, 1], [150, 2]])
def test_unmapped_pages_are_not_seen_and_reported(counts):
    kv = [300, 200]
    d = gdn.KVDims(4, 2, 128, page_size=32)
    cache, table = make_cache(d, kv, 51)
    table[0, 2], table[1, 1] = -1, cache.n_pages
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    q = torch.randn(sum(counts), 4, 128, generator=gen(52), device="cuda").to(BF)
    out = gdn.kv_attention(d, cache, cu_of(counts), lens, table, q)
    with pytest.raises(gdn.GDNError) as e:
        gdn.sync_status()
    assert e.value.status == 1 and "code 40" in str(e.value)
    # the same without those keys, one query at a time in 64 bits
    begin = 0
    for i, (c, n) in enumerate(zip(counts, kv)):
        hole = range(64, 96) if i == 0 else range(32, 64)
        t2 = table.clone()
        t2[t2 < 0], t2[t2 >= cache.n_pages] = 0, 0
        k, v = (line(d, cache, t2, x, i, n).repeat_interleave(2, 1) for x in ("k", "v"))
        for t in range(c):
            see = [j for j in range(n - c + t + 1) if j not in hole]
            x = torch.einsum("hd,khd->hk", q[begin + t].double(), k[see]) * 128 ** -0.5
            ref = torch.einsum("hk,khd->hd", torch.softmax(x, -1), v[see])
            size = torch.einsum("hk,khd->hd", torch.softmax(x, -1), v[see].abs())
            got = out[begin + t].double()
            assert ((got - ref).abs() <= 2.0 ** -9 * size + 2.0 ** -8 * got.abs()).all()
        begin += c


def test_windowed_out_pages_may_be_unmapped():
    d = gdn.KVDims(4, 2, 128, page_size=32, window=64)
    for counts, kv in (([1], [300]), ([20], [300])):
        cache, table = make_cache(d, kv, 53)
        lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
        q = torch.randn(sum(counts), 4, 128, generator=gen(54), device="cuda").to(BF)
        ref = attention_ref(d, cache, table, counts, kv, q)
        first = (kv[0] - counts[0] + 1 - 64) // 32
        table[0, :first] = -1
        out = gdn.kv_attention(d, cache, cu_of(counts), lens, table, q)
        assert attention_excess(d, out, *ref) <= 1.0


def test_a_length_beyond_the_block_table_is_reported():
    d = gdn.KVDims(4, 2, 64, page_size=16)
    cache, table = make_cache(d, [64], 55)
    q = torch.randn(1, 4, 64, generator=gen(56), device="cuda").to(BF)
    lens = torch.tensor([100], dtype=torch.int32, device="cuda")
    out = gdn.kv_attention(d, cache, cu_of([1]), lens, table, q, max_kv_len=64)
    with pytest.raises(gdn.GDNError, match="code 40"):
        gdn.sync_status()
    ref = gdn.kv_attention(d, cache, cu_of([1]), torch.tensor([64], dtype=torch.int32, device="cuda"), table, q)
    assert torch.allclose(out.float(), ref.float(), atol=1e-2)


def test_another_stream():
    """The call runs on the current stream: its inputs are made there, and its output is read there."""
    d = gdn.KVDims(16, 2, 256, page_size=64, rope_dim=64)
    counts, kv = [1] * 8, [900] * 8
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        cache, table = make_cache(d, kv, 61)
        lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
        cu = cu_of(counts)
        g = gen(62)
        q, k, v = (torch.randn(8, h, 256, generator=g, device="cuda").to(BF) for h in (16, 2, 2))
        torch.cuda._sleep(20_000_000)
        q2 = gdn.kv_append(d, cache, cu, lens, table, k, v, q=q, rope=rope_table(1000, 64))
        out = gdn.kv_attention(d, cache, cu, lens, table, q2)
        ref = attention_ref(d, cache, table, counts, kv, q2)
        assert attention_excess(d, out, *ref) <= 1.0


def test_attention_in_a_cuda_graph():
    d = gdn.KVDims(8, 2, 128, page_size=64)
    counts, kv = [1] * 4, [700, 3, 65, 2000]
    out, _, (cache, table, lens, q) = _attend(d, counts, kv, 71)
    cu = cu_of(counts)
    ws = torch.empty(max(256, gdn.kv_attention_workspace_size(d, cu, 2048)), dtype=torch.uint8, device="cuda")
    buf = torch.empty_like(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.kv_attention(d, cache, cu, lens, table, q, max_kv_len=2048, out=buf, workspace=ws)
    for step in range(3):
        lens.copy_(torch.tensor([700 - step, 3, 64 + step, 1999], dtype=torch.int32))
        buf.fill_(7.0)
        graph.replay()
        ref = attention_ref(d, cache, table, counts, lens.tolist(), q)
        assert attention_excess(d, buf, *ref) <= 1.0


# ------------------------------------------------------------------- append
def _append_ref32(d, cache, table, counts, kv_lens, rope_rows, k, v):
    """The rule in fp32, operation by operation, on copies of the cache: (k, v, k_scale, v_scale)."""
    got = {}
    top = QMAX[d.cache]
    inv = torch.tensor(1.0 / top, dtype=torch.float32)

    def code(y):
        y = torch.nan_to_num(y, nan=0.0, posinf=top, neginf=-top)
        if d.cache == "int8":
            return y.round().clamp(-top, top).to(torch.int8)
        return y.clamp(-top, top).to(torch.float8_e4m3fn).view(torch.int8)

    for name, x in (("k", k), ("v", v)):
        codes, scales = getattr(cache, name).view(torch.int8).cpu().clone(), getattr(cache, name + "_scale").cpu().clone()
        x = x.float().cpu()
        if name == "k" and d.rope_dim:
            x = turn(x, rope_rows.cpu(), d.rope_style)
        begin = 0
        for i, (c, n) in enumerate(zip(counts, kv_lens)):
            for lp in range((n - c) // d.page_size, (n - 1) // d.page_size + 1 if c else 0):
                page = int(table[i, lp])
                a, z = max(n - c, lp * d.page_size), min(n, (lp + 1) * d.page_size)
                new = x[begin + a - (n - c): begin + z - (n - c)]
                kept = a - lp * d.page_size
                fin = torch.where(torch.isfinite(new), new.abs(), 0.0)
                for h in range(d.n_kv_heads):
                    old = scales[page, h] if kept else torch.tensor(0.0)
                    s = torch.maximum(old, fin[:, h].max() * inv)
                    if kept and s > old:
                        c8 = codes[page, h, :kept]
                        val = c8.float() if d.cache == "int8" else c8.view(torch.float8_e4m3fn).float()
                        codes[page, h, :kept] = code(val * (old / s))
                    y = new[:, h] / s if s > 0 else torch.zeros_like(new[:, h])
                    codes[page, h, kept: kept + z - a] = code(y)
                    scales[page, h] = s
            begin += c
        got[name] = (codes, scales)
    return got


APPEND = {
    # name: (Hq, Hkv, D, page, dtype, codes, rope, style, counts, kv_lens)
    "decode": (16, 2, 256, 64, BF, "int8", 64, "half", [1] * 5, [1, 2, 64, 65, 200]),
    "decode_e4m3": (8, 4, 128, 16, BF, "e4m3", 128, "interleaved", [1] * 4, [1, 16, 17, 31]),
    "verify_T4": (4, 2, 64, 32, BF, "int8", 16, "half", [4] * 4, [4, 33, 34, 64]),
    "prompt": (4, 2, 128, 64, BF, "int8", 64, "half", [300], [300]),
    "prompt_page128_d256": (2, 1, 256, 128, BF, "e4m3", 256, "half", [260], [300]),
    "prompts_ragged": (4, 2, 128, 32, BF, "e4m3", 32, "interleaved", [1, 0, 70, 33], [33, 9, 100, 33]),
    "no_rope": (4, 2, 64, 16, BF, "int8", 0, "half", [20, 3], [25, 3]),
    "f32": (4, 2, 128, 16, F32, "int8", 128, "half", [20, 1], [25, 16]),
    "f32_page128_d256": (2, 1, 256, 128, F32, "e4m3", 64, "interleaved", [129, 1], [257, 100]),
}


def _append_inputs(name, seed=7):
    hq, hkv, dim, page, dtype, fmt, rope, style, counts, kv = APPEND[name]
    d = gdn.KVDims(hq, hkv, dim, page_size=page, dtype=dtype, cache=fmt, rope_dim=rope, rope_style=style)
    cache, table = make_cache(d, kv, seed)
    g = gen(seed + 1)
    t = sum(counts)
    q, k, v = (torch.randn(t, h, dim, generator=g, device="cuda").mul(1.5).to(dtype) for h in (hq, hkv, hkv))
    pos = [p for c, n in zip(counts, kv) for p in range(n - c, n)]
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    return d, cache, table, counts, kv, lens, q, k, v, rope_table(400, rope) if rope else None, pos


@pytest.mark.parametrize("name", sorted(APPEND))
def test_append_codes_are_the_rule_s(name):
    """Bit for bit the rule's codes and scales; every other byte of the cache as it was."""
    d, cache, table, counts, kv, lens, q, k, v, rope, pos = _append_inputs(name)
    rows = rope[pos] if rope is not None else None
    ref = _append_ref32(d, cache, table, counts, kv, rows, k, v)
    q2 = gdn.kv_append(d, cache, cu_of(counts), lens, table, k, v, q=q, rope=rope)
    for x in ("k", "v"):
        assert torch.equal(getattr(cache, x).view(torch.int8).cpu(), ref[x][0])
        assert torch.equal(getattr(cache, x + "_scale").cpu().nan_to_num(-1.0), ref[x][1].nan_to_num(-1.0))
    want = q.float() if rope is None else turn(q.float(), rows, d.rope_style)
    assert torch.equal(q2, want.to(d.dtype))


@pytest.mark.parametrize("name", sorted(APPEND))
def test_append_values_against_64_bits(name):
    """Stored values within half a code step of the rotated ones (the earlier tokens of a page, of
    their previous values); rotation in 64 bits."""
    d, cache, table, counts, kv, lens, q, k, v, rope, pos = _append_inputs(name, seed=9)
    before = [{x: line(d, cache, table, x, i, n - c) for x in ("k", "v")} for i, (c, n) in enumerate(zip(counts, kv))]
    kept = [{x: getattr(cache, x + "_scale")[table[i, : -(-n // d.page_size)].long()].clone() for x in ("k", "v")}
            for i, n in enumerate(kv)]
    q2 = gdn.kv_append(d, cache, cu_of(counts), lens, table, k, v, q=q, rope=rope)
    rows = rope[pos].double() if rope is not None else None
    want = {"k": turn(k.double(), rows, d.rope_style) if rope is not None else k.double(), "v": v.double()}
    qw = turn(q.double(), rows, d.rope_style) if rope is not None else q.double()
    assert ((q2.double() - qw).abs() <= 2.0 ** (-8 if d.dtype == BF else -22) * q.double().abs().amax()).all()
    begin = 0
    for i, (c, n) in enumerate(zip(counts, kv)):
        for x in ("k", "v"):
            now = line(d, cache, table, x, i, n)
            pages = table[i, : -(-n // d.page_size)].long()
            s = getattr(cache, x + "_scale")[pages].double().repeat_interleave(d.page_size, 0)[:n, :, None]
            target = torch.cat([before[i][x], want[x][begin:begin + c]])
            step = s if d.cache == "int8" else torch.maximum(target.abs() / 8, s * 2.0 ** -9)
            grew = (getattr(cache, x + "_scale")[pages] != kept[i][x]).repeat_interleave(d.page_size, 0)[:n, :, None]
            new = torch.arange(n, device="cuda")[:, None, None] >= n - c
            assert ((now - target).abs() <= torch.where(new | grew, 0.501 * step, 0.0)).all()
        begin += c


def test_append_scale_grows_only_when_it_must():
    d = gdn.KVDims(2, 1, 64, page_size=16)
    cache, table = make_cache(d, [16], 3)
    cu = cu_of([1])
    one = torch.ones(1, 1, 64, device="cuda", dtype=BF)
    scales, first = [], None
    for t in range(16):
        lens = torch.tensor([t + 1], dtype=torch.int32, device="cuda")
        mag = 2.0 if t == 5 else 1.0 / (1 + t % 3)
        gdn.kv_append(d, cache, cu, lens, table, one * mag, one * mag)
        scales.append(float(cache.k_scale[table[0, 0], 0]))
        codes = cache.k[table[0, 0].long(), 0, : t + 1, 0].tolist()
        first = codes if t == 4 else first
    assert scales[0] == pytest.approx(1 / 127) and scales[4] == scales[0]
    assert scales[5] == pytest.approx(2 / 127) and scales[15] == scales[5]
    assert codes[0] == 64 and codes[5] == 127 and first[0] == 127


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_of_zeros_infinities_and_nan(fmt):
    d = gdn.KVDims(2, 1, 64, page_size=16, cache=fmt)
    cache, table = make_cache(d, [16, 16, 16], 3)
    k = torch.zeros(3 * 16, 1, 64, device="cuda")
    k[16:32] = torch.randn(16, 1, 64, generator=gen(1), device="cuda")
    k[17, 0, 3], k[18, 0, 4], k[19, 0, 5] = float("nan"), float("inf"), -float("inf")
    k[33] = float("inf")
    k = k.to(BF)
    lens = torch.tensor([16] * 3, dtype=torch.int32, device="cuda")
    gdn.kv_append(d, cache, cu_of([16] * 3), lens, table, k, k)
    got, _ = gdn.kv_read(d, cache, cu_of([16] * 3), lens * 0, table, dtype=F32)
    assert not got[:16].any() and not got[32:].any() and torch.isfinite(got).all()
    fin = torch.isfinite(k[16:32])
    top = k[16:32][fin].float().abs().max()
    assert got[17, 0, 3] == 0 and float(got[18, 0, 4]) == pytest.approx(float(top), rel=1e-6)
    assert float(got[19, 0, 5]) == pytest.approx(-float(top), rel=1e-6)
    err = (got[16:32] - k[16:32].float())[fin].abs()
    assert err.max() <= (top / 127 * 0.501 if fmt == "int8" else top / 16 * 1.001)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_strides_aliases_and_positions(dtype):
    """A fused projection's slices, q rotated in place, and explicit rotation rows."""
    counts, kv = [5, 1], [20, 40]
    d = gdn.KVDims(4, 2, 128, page_size=16, dtype=dtype, rope_dim=64)
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    fused = torch.randn(6, 8, 128, generator=gen(2), device="cuda").to(dtype)
    q, k, v = fused[:, :4], fused[:, 4:6], fused[:, 6:]
    rope = rope_table(500, 64)
    results = []
    for strided in (True, False):
        cache, table = make_cache(d, kv, 4)
        qq, kk, vv = (q, k, v) if strided else (q.contiguous(), k.contiguous(), v.contiguous())
        pos = torch.tensor([400, 3, 17, 0, 499, 250], dtype=torch.int32, device="cuda")
        if strided:
            out = gdn.kv_append(d, cache, cu_of(counts), lens, table, kk, vv, q=qq, rope=rope, positions=pos)
        else:
            out = gdn.kv_append(d, cache, cu_of(counts), lens, table, kk, vv, q=qq, rope=rope, positions=pos, q_out=qq)
            assert out.data_ptr() == qq.data_ptr()
        results.append((out, cache.k.clone(), cache.v.clone(), cache.k_scale.nan_to_num(-1), cache.v_scale.nan_to_num(-1)))
        assert torch.equal(out, turn(q.float(), rope[pos.long()], "half").to(dtype))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(*results))


def test_append_out_of_range_is_reported_and_stays_inside():
    d = gdn.KVDims(4, 2, 64, page_size=16, rope_dim=16)
    cache, table = make_cache(d, [32, 32], 5)
    k = torch.randn(4, 2, 64, generator=gen(6), device="cuda").to(BF)
    rope = rope_table(32, 16)
    cu = cu_of([2, 2])
    table[1, 1] = -1
    gdn.kv_append(d, cache, cu, torch.tensor([32, 32], dtype=torch.int32, device="cuda"), table, k, k, rope=rope)
    with pytest.raises(gdn.GDNError, match="code 40"):
        gdn.sync_status()
    got, _ = gdn.kv_read(d, cache, cu_of([2]), torch.tensor([30], dtype=torch.int32, device="cuda"), table[:1], dtype=F32)
    assert (got - turn(k[:2].float(), rope[30:32], "half")).abs().max() < 0.05
    for lens in ([33, 32], [1, 32]):  # past the table; a first position of -1
        table[1, 1] = 0 if table[0, 1] != 0 else 1
        gdn.kv_append(d, cache, cu, torch.tensor(lens, dtype=torch.int32, device="cuda"), table, k, k,
                      rope=rope_table(64, 16))
        with pytest.raises(gdn.GDNError, match="code 40"):
            gdn.sync_status()
    gdn.kv_append(d, cache, cu_of([2, 0]), torch.tensor([32, 0], dtype=torch.int32, device="cuda"), table, k[:2], k[:2],
                  rope=rope[:31])
    with pytest.raises(gdn.GDNError, match="code 41"):
        gdn.sync_status()


# --------------------------------------------------------------------- read
@pytest.mark.parametrize("hkv,dim,page,fmt", [(2, 256, 64, "int8"), (4, 128, 16, "e4m3"), (1, 64, 128, "int8")])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_read_values(hkv, dim, page, fmt, dtype):
    d = gdn.KVDims(hkv, hkv, dim, page_size=page, cache=fmt, dtype=BF)
    kv, starts, counts = [300, 5, 70, 129], [7, 0, 70, 128], [290, 5, 0, 1]
    cache, table = make_cache(d, kv, 11)
    at = torch.tensor(starts, dtype=torch.int32, device="cuda")
    k, v = gdn.kv_read(d, cache, cu_of(counts), at, table, dtype=dtype)
    for x, got in (("k", k), ("v", v)):
        want = torch.cat([line(d, cache, table, x, i, s + c)[s:] for i, (s, c) in enumerate(zip(starts, counts))])
        # one product: exact in 64 bits, rounded to fp32, then to the output's type
        assert torch.equal(got, want.float().to(dtype))


def test_read_of_unmapped_pages_is_zero_and_reported():
    d = gdn.KVDims(2, 2, 64, page_size=16)
    cache, table = make_cache(d, [48], 12)
    table[0, 1] = cache.n_pages + 5
    k, v = gdn.kv_read(d, cache, cu_of([60]), torch.tensor([0], dtype=torch.int32, device="cuda"), table)
    with pytest.raises(gdn.GDNError, match="code 40"):
        gdn.sync_status()
    assert not k[16:32].any() and not v[48:].any() and k[:16].any() and v[32:48].any()


# ------------------------------------------------------- empty, no sequences
def test_empty_calls():
    d = gdn.KVDims(4, 2, 64, page_size=16)
    cache, table = make_cache(d, [16], 13)
    none = torch.zeros(0, 2, 64, dtype=BF, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert gdn.kv_attention(d, cache, [0, 0], zero, table, torch.zeros(0, 4, 64, dtype=BF, device="cuda")).shape == (0, 4, 64)
    gdn.kv_append(d, cache, [0, 0], zero, table, none, none)
    k, v = gdn.kv_read(d, cache, [0], zero[:0], table[:0])
    assert k.shape == v.shape == (0, 2, 64)
