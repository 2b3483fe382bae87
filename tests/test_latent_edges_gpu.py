"""Latent attention on the GPU at its edges: waits that give up, few rows and short rings, very large
scores and lengths, memory shared between arguments."""
import time

import pytest
import torch

import gated_deltanet_linear_mixer_gb300 as gdn
from latent_cases import U, absorbed, check, cu_of, expanded, gen, ints, make_cache

pytestmark = pytest.mark.gpu


def _queries(t, heads, width, seed):
    return torch.randn(t, heads, width, generator=gen(seed), device="cuda").bfloat16()


def _timeout():
    with pytest.raises(gdn.GDNError) as e:
        gdn.sync_status()
    assert e.value.status == gdn.GDN_ERR_TIMEOUT
    gdn.sync_status()  # read and cleared


@pytest.mark.parametrize("heads,dc", [(16, 512), (32, 512), (64, 256), (128, 256)])
def test_waits_that_give_up_in_the_first_of_many_rounds(monkeypatch, heads, dc):
    """Spans of many sequences, laid out a few at a time: a wait that gives up while the first ones are
    walked ends the call, by all warps alike, in the time of those; the next call is right."""
    d = gdn.LatentDims(heads, dc, page_size=16)
    n = 7600  # 50 a span
    counts, lens = [1] * n, [1 + i % 70 for i in range(n)]
    cache, table = make_cache(d, [70], 301)
    table = table.expand(n, -1).contiguous()  # all read the same pages
    q = _queries(n, heads, dc + 64, 302)
    cu = cu_of(counts)
    monkeypatch.setenv("GDN_FAULT", "stall_latent")
    torch.cuda.synchronize()
    start = time.monotonic()
    gdn.latent_attention(d, cache, cu, ints(lens), table, q)
    _timeout()
    assert time.monotonic() - start < 20.0  # waits of about 2 s one after the other, in one round of four
    monkeypatch.delenv("GDN_FAULT")
    got = gdn.latent_attention(d, cache, cu, ints(lens), table, q)
    gdn.sync_status()
    some = list(range(0, n, 97)) + [n - 1]
    check(got[some], *absorbed(d, cache, [1] * len(some), [lens[i] for i in some], table[some], q[some]))


@pytest.mark.parametrize("heads", [1, 2, 16, 20, 32])
@pytest.mark.parametrize("dc", [256, 512])
def test_few_rows_and_many_short_ragged_sequences(heads, dc):
    """Up to 32 rows a sequence, so that some softmax warps have none, over tiles that end early, one
    after the other: several calls, all alike and right."""
    d = gdn.LatentDims(heads, dc, page_size=64)
    n = 2000
    counts, lens = [1] * n, [1 + (i * 37) % 200 for i in range(n)]
    cache, table = make_cache(d, lens, 311)
    q, cu = _queries(n, heads, dc + 64, 312), cu_of(counts)
    want = absorbed(d, cache, counts, lens, table, q)
    outs = [gdn.latent_attention(d, cache, cu, ints(lens), table, q) for _ in range(5)]
    gdn.sync_status()
    check(outs[0], *want)
    assert all(torch.equal(outs[0], o) for o in outs)


@pytest.mark.parametrize("heads,dc,counts,lens", [(16, 512, [1, 1], [5000, 900]), (32, 256, [1] * 400, [400] * 400),
                                                  (32, 512, [4, 1], [3000, 200]), (128, 256, [2] * 90, [700] * 90)])
def test_latent_attention_gives_up_with_loads_in_flight(monkeypatch, heads, dc, counts, lens):
    """Products that are never issued: full rings, whose loads are waited for at the end."""
    d = gdn.LatentDims(heads, dc, page_size=32)
    cache, table = make_cache(d, lens, 321)
    q, cu = _queries(sum(counts), heads, dc + 64, 322), cu_of(counts)
    monkeypatch.setenv("GDN_FAULT", "stall_latent_products")
    torch.cuda.synchronize()
    start = time.monotonic()
    gdn.latent_attention(d, cache, cu, ints(lens), table, q)
    _timeout()
    assert time.monotonic() - start < 20.0
    monkeypatch.delenv("GDN_FAULT")
    got = gdn.latent_attention(d, cache, cu, ints(lens), table, q)
    gdn.sync_status()
    check(got, *absorbed(d, cache, counts, lens, table, q))


@pytest.mark.parametrize("nope,vd", [(128, 128), (64, 64)])
def test_expanded_attention_gives_up_with_loads_in_flight(monkeypatch, nope, vd):
    d = gdn.LatentDims(24, nope_dim=nope, v_dim=vd)
    counts, lens = [300, 5, 130, 256] * 3, [2300, 400, 131, 700] * 3
    g = gen(331)
    kv = torch.randn(sum(lens), 24, nope + vd, generator=g, device="cuda").bfloat16()
    r = torch.randn(sum(lens), 64, generator=g, device="cuda").bfloat16()
    q = _queries(sum(counts), 24, nope + 64, 332)
    args = (d, cu_of(counts), cu_of(lens), q, kv[..., :nope], r, kv[..., nope:])
    monkeypatch.setenv("GDN_FAULT", "stall_expanded_products")
    torch.cuda.synchronize()
    start = time.monotonic()
    gdn.expanded_attention(*args)
    _timeout()
    assert time.monotonic() - start < 20.0
    monkeypatch.delenv("GDN_FAULT")
    got = gdn.expanded_attention(*args)
    gdn.sync_status()
    check(got, *expanded(d, counts, lens, *args[3:]))


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("exponent", [16, 31, 40, 90])
def test_very_large_scores_pick_one_key(sign, exponent):
    """Scores n 2^exponent, n a whole number of its own for each key: exact in fp32, and far enough apart
    (192^-1/2 2^16 = 4730) that all weights but the largest are 0: the result is that key's value, to the
    rounding of its weight (at most U; the sum takes it unrounded) and of the result (at most U more)."""
    d = gdn.LatentDims(2)
    counts, lens = [300, 5, 130], [300, 700, 1000]
    g = gen(341)
    q = torch.zeros(sum(counts), 2, 192, dtype=torch.bfloat16, device="cuda")
    q[..., 5:7] = sign * 2.0 ** (exponent // 2)
    k = torch.zeros(sum(lens), 2, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.randn(sum(lens), 2, 128, generator=g, device="cuda").bfloat16()
    r = torch.zeros(sum(lens), 64, dtype=torch.bfloat16, device="cuda")
    want, b = [], 0
    for c, n in zip(counts, lens):
        picks = []
        for h in range(2):
            rank = torch.randperm(n, generator=g, device="cuda") + 1
            k[b:b + n, h, 5] = (rank // 32 * 32 * 2.0 ** (exponent - exponent // 2)).bfloat16()
            k[b:b + n, h, 6] = (rank % 32 * 2.0 ** (exponent - exponent // 2)).bfloat16()
            best = (sign * rank).cummax(0).indices[n - c:]  # of the keys up to each query's position
            picks.append(v[b + best, h])
        want.append(torch.stack(picks, 1))
        b += n
    got = gdn.expanded_attention(d, cu_of(counts), cu_of(lens), q, k, r, v)
    gdn.sync_status()
    want = torch.cat(want).double()
    check(got, want, want.abs() * (2 * U + U * U))


def test_outputs_in_the_inputs_memory_are_refused():
    """Every output in every input's memory in turn; next to it is right."""
    d = gdn.LatentDims(2, 256, page_size=16, nope_dim=64, v_dim=64)
    cache, table = make_cache(d, [40], 351)
    cu, lens = cu_of([4]), ints([40])
    big = torch.randn(1 << 16, generator=gen(352), device="cuda").bfloat16()

    def rows(at, *shape):
        n = 1
        for x in shape:
            n *= x
        return big[at:at + n].view(shape)

    q, k, v, r, qe = rows(0, 4, 2, 320), rows(8192, 9, 2, 64), rows(16384, 9, 2, 64), rows(24576, 9, 64), rows(32768, 4, 2, 128)
    want = gdn.latent_attention(d, cache, cu, lens, table, q)
    for at, bad in ((0, True), (2560 - 8, True), (2560, False)):
        out = rows(at, 4, 2, 256)
        if bad:
            with pytest.raises(ValueError, match="out shares memory with q"):
                gdn.latent_attention(d, cache, cu, lens, table, q, out=out)
        else:
            assert torch.equal(gdn.latent_attention(d, cache, cu, lens, table, q, out=out), want)
    flat = cache.rows.view(-1)
    with pytest.raises(ValueError, match="out shares memory with cache.rows"):
        gdn.latent_attention(d, cache, cu, lens, table, q, out=flat[320:320 + 2048].view(4, 2, 256))
    size = gdn.latent_attention_workspace_size(d, cu)
    space = torch.empty(size + 4096, dtype=torch.uint8, device="cuda")
    out = space[size:size + 4096].view(torch.bfloat16).view(4, 2, 256)
    assert torch.equal(gdn.latent_attention(d, cache, cu, lens, table, q, out=out, workspace=space[:size]), want)
    with pytest.raises(ValueError, match="workspace shares memory with out"):
        gdn.latent_attention(d, cache, cu, lens, table, q, out=out, workspace=space)
    with pytest.raises(ValueError, match="out shares memory with cache.rows"):
        gdn.latent_read(d, cache, cu, ints([0]), table, out=flat[-1280:].view(4, 320))
    ck = cu_of([9])
    want = gdn.expanded_attention(d, cu, ck, qe, k, r, v)
    for x, name in ((qe, "q"), (k, "k"), (r, "k_rope"), (v, "v")):
        at = (x.data_ptr() - big.data_ptr()) // 2 + x.numel()
        with pytest.raises(ValueError, match=f"out shares memory with {name}$"):
            gdn.expanded_attention(d, cu, ck, qe, k, r, v, out=rows(at - 8, 4, 2, 64))
        assert torch.equal(gdn.expanded_attention(d, cu, ck, qe, k, r, v, out=rows(at, 4, 2, 64)), want)
    c, q_rope = rows(40960, 4, 320), rows(49152, 4, 2, 64)
    for q_out, other in ((c.view(-1)[:512], "c"), (flat[:512], "cache.rows")):
        with pytest.raises(ValueError, match=f"q_out shares memory with {other}"):
            gdn.latent_append(d, cache, cu, lens, table, c, q_rope=q_rope, q_out=q_out.view(4, 2, 64))
    for at, other in ((49152 + 64, 128), (49152 + 256, 256)):  # shifted by a head; at another token stride
        with pytest.raises(ValueError, match="q_out shares memory with q_rope"):
            gdn.latent_append(d, cache, cu, lens, table, c, q_rope=q_rope, q_out=rows(at, 4, other // 64, 64)[:, :2])
    for outs in ({"rows_out": rows(40960 + 8, 4, 320)}, {"rows_out": rows(49152, 4, 320)}):
        with pytest.raises(gdn.GDNError, match="shares memory"):
            gdn.latent_append(d, cache, cu, lens, table, c, q_rope=q_rope, **outs)
    gdn.sync_status()
    # no tokens share nothing
    none = cu_of([0])
    assert gdn.latent_append(d, cache, none, lens, table, c[:0], q_rope=q_rope[:0], q_out=q_rope[:0], rows_out=c[:0]).shape == (0, 2, 64)
    assert gdn.latent_append(d, cache, none, lens, table, c[:0], q_rope=q_rope[:0]).shape == (0, 2, 64)
    assert gdn.latent_attention(d, cache, none, lens, table, q[:0], out=q[:0, :, :256]).shape == (0, 2, 256)
    assert gdn.expanded_attention(d, none, none, qe[:0], k[:0], r[:0], v[:0], out=v[:0]).shape == (0, 2, 64)
    # a projection's output that holds c and the queries side by side, turned in place
    side = torch.randn(4, 2 * 128 + 320, generator=gen(353), device="cuda").bfloat16()
    turned = gdn.latent_append(d, cache, cu, lens, table, side[:, 256:], q_rope=side[:, :256].view(4, 2, 128)[..., 64:],
                               q_out=side[:, :256].view(4, 2, 128)[..., :64])
    assert torch.equal(turned, side[:, :256].view(4, 2, 128)[..., 64:])
    gdn.sync_status()


@pytest.mark.parametrize("short", [1, 64, 65])
def test_lengths_next_to_the_largest_32_bit_number(short):
    """One page a sequence over and over, its keys alike, then the last one: its last key, which the last
    query alone sees, has a score far above the others'.  All sums are whole numbers below 2^24."""
    d = gdn.LatentDims(16, 256, page_size=128)
    n = 2 ** 31 - short
    pages = (n + 127) // 128
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    rows = torch.zeros(2, 128, 320, dtype=torch.bfloat16, device="cuda")
    rows[..., :256] = 1.0
    last = (n - 1) % 128
    rows[1, last, :256], rows[1, last, 256], rows[1, last + 1:] = 3.0, 64.0, float("nan")
    q = torch.zeros(2, 16, 320, dtype=torch.bfloat16, device="cuda")
    q[..., 256] = 64.0
    got = gdn.latent_attention(d, gdn.LatentCache(d, rows), cu_of([2]), ints([n]), table, q)
    gdn.sync_status()
    assert bool((got[0] == 1.0).all()) and bool((got[1] == 3.0).all())


@pytest.mark.parametrize("dc", [256, 512])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
def test_rows_of_all_sizes_are_normalised(dc, eps):
    """From numbers without normal bits to the largest: squares leave fp32 on both sides.  24 additions and 4
    ulp as for rows of ordinary size (2^-19); half a step of the result, or of the smallest number."""
    d = gdn.LatentDims(1, dc, page_size=128, norm_eps=eps)
    exponents = [125, 118, 70, 64, 63, 59, 58, 57, 40, 0, -14, -30, -44, -46, -60, -75, -100, -120, -128, -132]
    t = len(exponents)
    c = torch.randn(t, dc + 64, generator=gen(361), device="cuda").clamp(-3, 3)
    c = (c.double() * torch.tensor(exponents, device="cuda").double().exp2()[:, None]).bfloat16()
    c[-1, 5] = 2.0 ** -133
    w = torch.randn(dc, generator=gen(362), device="cuda").mul(0.2).add(1.0)
    cache, table = make_cache(d, [t], 363)
    packed = torch.empty_like(c)
    gdn.latent_append(d, cache, [0, t], ints([t]), table, c, norm_w=w, rows_out=packed)
    gdn.sync_status()
    x = c[:, :dc].double()
    want = x / torch.sqrt(x.square().mean(-1, keepdim=True) + d.c().norm_eps) * w.double()
    check(packed[:, :dc], want, want.abs() * (2.0 ** -19 + U * (1 + 2.0 ** -19)) + 2.0 ** -134)
    assert torch.equal(packed[:, dc:], c[:, dc:])
    # a row of zeros has none but zeros, one with an infinity as well, beside large numbers too
    c = torch.zeros(3, dc + 64, dtype=torch.bfloat16, device="cuda")
    c[1, 7], c[1, 9], c[2, 7], c[2, 9] = float("inf"), 2.0 ** 100, float("nan"), 2.0 ** 100
    gdn.latent_append(d, cache, [0, 3], ints([3]), table, c, norm_w=w, rows_out=packed[:3])
    gdn.sync_status()
    assert bool((packed[:3, :dc] == 0).all())


@pytest.mark.parametrize("heads,dc,counts,lens", [
    (32, 512, [5] * 4, [700, 5, 64, 1000]),                    # three row tiles each
    (32, 256, [1] * 40 + [3], [130] * 40 + [2000]),            # single tokens beside a piece
    (16, 512, [40] + [1] * 30, [1500] + [77] * 30),
    (20, 512, [1, 7, 0, 2, 33, 4], [300, 7, 20, 2, 40, 129]),
    (65, 256, [1, 1, 1], [500, 64, 1]),
    (192, 512, [1, 3], [3000, 90]),
])
def test_more_rows_than_a_tile_beside_odd_numbers_of_tiles(heads, dc, counts, lens):
    """Row tiles one to a group: several groups a sequence, or one among short ones; twice alike."""
    d = gdn.LatentDims(heads, dc, page_size=32)
    cache, table = make_cache(d, lens, 371)
    q, cu = _queries(sum(counts), heads, dc + 64, 372), cu_of(counts)
    got = gdn.latent_attention(d, cache, cu, ints(lens), table, q)
    gdn.sync_status()
    check(got, *absorbed(d, cache, counts, lens, table, q))
    assert torch.equal(got, gdn.latent_attention(d, cache, cu, ints(lens), table, q))
