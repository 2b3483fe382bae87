"""Latent attention on the GPU against plain 64-bit implementations: append, read, both forms of the
attention, page copies, and a run of them together."""
import math

import pytest
import torch

import gated_deltanet_linear_mixer_gb300 as gdn
from latent_cases import U, absorbed, check, cu_of, expanded, gen, ints, line, make_cache, rope_table, turn

pytestmark = pytest.mark.gpu


def _status_ok():
    gdn.sync_status()


def _status_bad(code_text):
    with pytest.raises(gdn.GDNError) as e:
        gdn.sync_status()
    assert e.value.status == 1 and code_text in str(e.value)
    gdn.sync_status()  # read and cleared


# ----------------------------------------------------------------- append
def _append_ref(d, c, w, table_rows):
    """What is stored, in 64 bits (before rounding), and its tolerance."""
    lat, key = c[:, :d.latent_dim].double(), c[:, d.latent_dim:].double()
    lat_tol = torch.zeros_like(lat)
    if w is not None:
        lat = lat / torch.sqrt(lat.square().mean(-1, keepdim=True) + d.c().norm_eps) * w.double()
        # the sum of squares, its root and two products in fp32: 24 additions, each 2^-24, and 4 ulp
        lat_tol = lat.abs() * 2.0 ** -19
    if table_rows is None:
        size = torch.zeros_like(key)
    else:
        key, size = (x[:, 0] for x in turn(key[:, None], table_rows, d.rope_style))
    tol = torch.cat([lat_tol, size * 2.0 ** -22], -1)
    want = torch.cat([lat, key], -1)
    return want, tol + U * (want.abs() + tol)


@pytest.mark.parametrize("dc,page,heads,style,norm,rope,counts,lens", [
    (512, 64, 32, "half", True, True, [1, 1, 1, 1], [128, 1, 77, 65]),
    (512, 16, 32, "interleaved", True, True, [1, 37, 0, 130], [900, 37, 5, 201]),
    (256, 32, 5, "half", False, True, [3, 64, 2], [3, 96, 33]),
    (256, 128, 17, "interleaved", True, False, [129, 4], [257, 131]),
    (512, 64, 128, "half", False, False, [9], [64]),
    (512, 64, 1, "half", True, True, [700], [1400]),
])
def test_append_stores_normed_and_rotated_rows(dc, page, heads, style, norm, rope, counts, lens):
    d = gdn.LatentDims(heads, dc, page_size=page, rope_style=style, norm_eps=1e-5)
    g = gen(11)
    t = sum(counts)
    cache, table = make_cache(d, lens, 5)
    before = cache.rows.clone()
    wide = torch.randn(t, dc + 64 + 128, generator=g, device="cuda").mul(1.5).bfloat16()
    c = wide[:, 64:64 + dc + 64]                       # a slice of a wider projection
    w = torch.randn(dc, generator=g, device="cuda").mul(0.2).add(1.0) if norm else None
    q = torch.randn(t, heads, 192, generator=g, device="cuda").bfloat16()
    ql = torch.full((t, heads, dc + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    tab = rope_table(max(lens)) if rope else None
    packed = torch.empty(t, dc + 64, dtype=torch.bfloat16, device="cuda")
    got = gdn.latent_append(d, cache, cu_of(counts), ints(lens), table, c, norm_w=w, q_rope=q[..., 128:],
                            q_out=ql[..., dc:], rope=tab, rows_out=packed)
    _status_ok()
    assert got.data_ptr() == ql[..., dc:].data_ptr()
    pos = torch.cat([torch.arange(n - k, n, device="cuda") for k, n in zip(counts, lens)])
    want, tol = _append_ref(d, c, w, tab[pos] if rope else None)
    check(packed, want, tol)
    qw, size = turn(q[..., 128:], tab[pos], style) if rope else (q[..., 128:].double(), torch.zeros(1, device="cuda"))
    check(got, qw, size * 2.0 ** -22 + U * (qw.abs() + size * 2.0 ** -22))
    assert bool((ql[..., :dc] == 7.0).all())
    # the pages hold the same rows; nothing else moved
    at = 0
    for i, (k, n) in enumerate(zip(counts, lens)):
        for j in range(n - k, n):
            p = int(table[i, j // page])
            assert torch.equal(cache.rows[p, j % page], packed[at])
            before[p, j % page] = packed[at]
            at += 1
    assert torch.equal(cache.rows.view(torch.int16), before.view(torch.int16))


def test_append_without_queries_in_place_and_by_given_positions():
    d = gdn.LatentDims(8, 256, page_size=16)
    g = gen(3)
    cache, table = make_cache(d, [40], 5)
    c = torch.randn(20, 320, generator=g, device="cuda").bfloat16()
    tab = rope_table(100)
    pos = torch.randint(0, 100, (20,), generator=g, device="cuda", dtype=torch.int32)
    packed = torch.empty_like(c)
    assert gdn.latent_append(d, cache, [0, 20], ints([40]), table, c, rope=tab, positions=pos, rows_out=packed) is None
    want, tol = _append_ref(d, c, None, tab[pos.long()])
    check(packed, want, tol)
    q = torch.randn(20, 8, 192, generator=g, device="cuda").bfloat16()
    qw, size = turn(q[..., 128:], tab[pos.long()], "half")
    head = q[..., :128].clone()
    gdn.latent_append(d, cache, [0, 20], ints([40]), table, c, rope=tab, positions=pos, q_rope=q[..., 128:],
                      q_out=q[..., 128:])
    _status_ok()
    check(q[..., 128:], qw, size * 2.0 ** -22 + U * (qw.abs() + size * 2.0 ** -22))
    assert torch.equal(q[..., :128], head)


def test_append_stores_finite_rows():
    d = gdn.LatentDims(1, 256, page_size=16)
    cache, table = make_cache(d, [6], 5)
    c = torch.ones(6, 320, device="cuda")
    c[0, 3], c[1, 5], c[2, 7], c[3, 300], c[4, 301] = math.nan, math.inf, -math.inf, math.inf, math.nan
    c[5, 260] = 3.38e38
    c = c.bfloat16()
    packed = torch.empty_like(c)
    gdn.latent_append(d, cache, [0, 6], ints([6]), table, c, rows_out=packed)
    top = torch.finfo(torch.bfloat16).max
    want = torch.nan_to_num(c, nan=0.0, posinf=top, neginf=-top)
    assert torch.equal(packed, want) and torch.equal(cache.rows[int(table[0, 0]), :6], want)
    # through the norm: a row with an infinity has no norm but zeros
    gdn.latent_append(d, cache, [0, 6], ints([6]), table, c, norm_w=torch.ones(256, device="cuda"), rows_out=packed)
    assert bool(torch.isfinite(packed).all()) and bool((packed[:3, :256] == 0).all())
    _status_ok()


def test_append_leaves_out_unmapped_pages_and_bad_positions():
    d = gdn.LatentDims(2, 256, page_size=16)
    g = gen(4)
    c = torch.randn(40, 320, generator=g, device="cuda").bfloat16()
    packed = torch.empty_like(c)
    for bad in (-1, 10 ** 6):
        cache, table = make_cache(d, [40], 5)
        table[0, 1] = bad
        before = cache.rows.clone()
        gdn.latent_append(d, cache, [0, 40], ints([40]), table, c, rows_out=packed)
        _status_bad("block table")
        assert torch.equal(packed, c)
        for j in (0, 2):
            k = min(16, 40 - 16 * j)
            before[int(table[0, j]), :k] = c[16 * j:16 * j + k]
        assert torch.equal(cache.rows.view(torch.int16), before.view(torch.int16))
    cache, table = make_cache(d, [40], 5)
    before = cache.rows.clone()
    for n in (39, 400):  # a first position before 0; a length beyond the table
        gdn.latent_append(d, cache, [0, 40], ints([n]), table, c)
        _status_bad("block table")
    gdn.latent_append(d, cache, [0, 40], ints([40]), table, c, rope=rope_table(39))
    _status_bad("rotation position")
    assert before.shape == cache.rows.shape


# ------------------------------------------------------------------- read
@pytest.mark.parametrize("dc,page,counts,starts", [(512, 16, [1], [0]), (512, 64, [5, 0, 130], [60, 3, 0]),
                                                   (256, 128, [257, 3], [1, 126]), (256, 32, [7] * 40, list(range(40)))])
def test_read_gives_the_rows_back(dc, page, counts, starts):
    d = gdn.LatentDims(4, dc, page_size=page)
    lens = [a + k for a, k in zip(starts, counts)]
    cache, table = make_cache(d, lens, 8)
    got = gdn.latent_read(d, cache, cu_of(counts), ints(starts), table)
    _status_ok()
    want = torch.cat([line(cache, table, i, n)[0][a:] for i, (a, n) in enumerate(zip(starts, lens))])
    assert torch.equal(got.double(), want)
    out = torch.empty_like(got)
    assert gdn.latent_read(d, cache, cu_of(counts), ints(starts), table, out=out) is out or torch.equal(out, got)


def test_read_of_unmapped_pages_gives_zeros():
    d = gdn.LatentDims(4, 256, page_size=16)
    cache, table = make_cache(d, [64], 8)
    table[0, 2] = -1
    got = gdn.latent_read(d, cache, [0, 64], ints([0]), table)
    _status_bad("block table")
    assert bool((got[32:48] == 0).all()) and bool((got[:32] != 0).any())
    got = gdn.latent_read(d, cache, [0, 64], ints([-60]), table)
    _status_bad("block table")
    assert bool((got[:60] == 0).all())


# ----------------------------------------------------------- absorbed form
def _queries(t, heads, width, seed, strided=False):
    g = gen(seed)
    x = torch.randn(t, heads, width + (64 if strided else 0), generator=g, device="cuda")
    x = (x * torch.randn(heads, 1, generator=g, device="cuda").mul(0.5).exp()).bfloat16()
    return x[..., 64:] if strided else x


@pytest.mark.parametrize("heads,dc,page,counts,lens", [
    (32, 512, 64, [1], [1]),
    (32, 512, 64, [1], [64]),
    (32, 512, 64, [1, 1, 1, 1], [63, 65, 1000, 128]),
    (16, 512, 16, [1] * 5, [17, 1, 333, 48, 200]),
    (1, 512, 64, [1, 1], [130, 7]),
    (3, 256, 32, [2, 5, 1], [70, 5, 31]),
    (128, 512, 128, [1, 1, 1], [300, 64, 129]),
    (128, 256, 64, [3, 1], [200, 66]),
    (20, 512, 16, [4, 0, 7, 1], [100, 50, 7, 90]),
    (20, 256, 64, [100], [100]),
    (32, 512, 64, [77, 1, 30], [177, 200, 30]),
    (64, 512, 32, [8] * 3, [2000, 8, 64]),
    (48, 512, 64, [1] * 9, [500, 64, 1, 2, 3, 640, 63, 65, 127]),
    (1024, 512, 64, [2], [150]),
])
def test_absorbed_attention(heads, dc, page, counts, lens):
    d = gdn.LatentDims(heads, dc, page_size=page)
    cache, table = make_cache(d, lens, 21)
    q = _queries(sum(counts), heads, dc + 64, 22, strided=heads % 2 == 0)
    got = gdn.latent_attention(d, cache, cu_of(counts), ints(lens), table, q)
    _status_ok()
    check(got, *absorbed(d, cache, counts, lens, table, q))


def test_absorbed_attention_of_many_and_long_sequences():
    d = gdn.LatentDims(16, 512)
    for counts, lens in (([1], [70_001]), ([1] * 300, [(37 * i) % 900 + 1 for i in range(300)]),
                         ([1] * 40 + [3], [5] * 40 + [20_000])):
        cache, table = make_cache(d, lens, 31)
        q = _queries(sum(counts), 16, 576, 32)
        got = gdn.latent_attention(d, cache, cu_of(counts), ints(lens), table, q)
        _status_ok()
        check(got, *absorbed(d, cache, counts, lens, table, q))


def test_absorbed_attention_beyond_32_bit_offsets():
    d = gdn.LatentDims(16, 512)
    first = 2 ** 32 // (64 * 576) + 1  # rows whose first element is past 2^32
    cache, table = make_cache(d, [200, 1000], 41, first_page=first)
    q = _queries(2, 16, 576, 42)
    got = gdn.latent_attention(d, cache, cu_of([1, 1]), ints([200, 1000]), table, q)
    _status_ok()
    check(got, *absorbed(d, cache, [1, 1], [200, 1000], table, q))
    assert torch.equal(gdn.latent_read(d, cache, cu_of([200, 1000]), ints([0, 0]), table).double(),
                       torch.cat([line(cache, table, i, n)[0] for i, n in enumerate((200, 1000))]))
    c = q.new_zeros(2, 576) + 0.5
    gdn.latent_append(d, cache, cu_of([1, 1]), ints([200, 1000]), table, c)
    _status_ok()
    assert bool((line(cache, table, 1, 1000)[0][999] == 0.5).all())


@pytest.mark.parametrize("heads,n", [(16, 1), (32, 4), (40, 3)])
def test_queries_that_see_nothing_give_zeros(heads, n):
    """Lengths shorter than the call's tokens, and no mapped page at all."""
    d = gdn.LatentDims(heads, 512, page_size=16)
    cache, table = make_cache(d, [50, 2, 20], 51)
    table[2] = -1
    counts, lens = [n, 5, n], [50, 2, 20]
    q = _queries(sum(counts), heads, 576, 52)
    out = torch.full((sum(counts), heads, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    got = gdn.latent_attention(d, cache, cu_of(counts), ints(lens), table, q, out=out)
    _status_bad("block table")
    want, tol = absorbed(d, cache, counts, lens, table, q)
    check(got, want, tol)
    assert bool((got[n:n + 3] == 0).all()) and bool((got[n + 5:] == 0).all())


def test_absorbed_attention_with_pages_missing_or_too_few():
    d = gdn.LatentDims(32, 512, page_size=16)
    cache, table = make_cache(d, [200, 90], 61)
    table[0, 3], table[0, 5], table[1, 0] = -1, 10 ** 7, -5
    q = _queries(4, 32, 576, 62)
    got = gdn.latent_attention(d, cache, cu_of([3, 1]), ints([200, 90]), table, q)
    _status_bad("block table")
    check(got, *absorbed(d, cache, [3, 1], [200, 90], table, q))
    # a length beyond the table: the keys that the table holds count
    cache, table = make_cache(d, [64], 63)
    got = gdn.latent_attention(d, cache, cu_of([1]), ints([100]), table, q[:1])
    _status_bad("block table")
    check(got, *absorbed(d, cache, [1], [100], table, q[:1]))


def test_scores_that_rise_and_values_of_all_sizes():
    """The reference moves at every tile; rows far apart in size."""
    d = gdn.LatentDims(32, 512)
    cache, table = make_cache(d, [1000], 71)
    size = torch.linspace(0.05, 3.0, 1000, device="cuda")
    for j in range(16):
        k = min(64, 1000 - 64 * j)
        cache.rows[int(table[0, j]), :k] *= size[64 * j:64 * j + k, None].bfloat16()
    q = _queries(1, 32, 576, 72) * 4
    got = gdn.latent_attention(d, cache, cu_of([1]), ints([1000]), table, q)
    check(got, *absorbed(d, cache, [1], [1000], table, q))
    cache.rows.mul_(1e-30)
    got = gdn.latent_attention(d, cache, cu_of([1]), ints([1000]), table, q)
    check(got, *absorbed(d, cache, [1], [1000], table, q))
    _status_ok()


def test_a_query_that_is_not_a_number_is_alone():
    d = gdn.LatentDims(32, 512)
    cache, table = make_cache(d, [300], 81)
    q = _queries(4, 32, 576, 82)
    q[1, 7, 100], q[2, 9, 3] = math.nan, math.inf
    got = gdn.latent_attention(d, cache, cu_of([4]), ints([300]), table, q)
    assert bool(got[1, 7].isnan().all()) and bool(got[2, 9].isnan().all())
    want, tol = absorbed(d, cache, [4], [300], table, q.nan_to_num(0, 0, 0))
    keep = torch.ones(4, 32, dtype=torch.bool, device="cuda")
    keep[1, 7] = keep[2, 9] = False
    check(got[keep], want[keep], tol[keep])


def test_results_depend_on_nothing_left_in_the_workspace_and_repeat():
    d = gdn.LatentDims(32, 512)
    lens = [3000, 17, 800]
    cache, table = make_cache(d, lens, 91)
    q = _queries(3, 32, 576, 92)
    cu = cu_of([1, 1, 1])
    ws = torch.empty(max(1, gdn.latent_attention_workspace_size(d, cu)), dtype=torch.uint8, device="cuda")
    outs = []
    for fill in (0, 255, 0x7F):
        ws.fill_(fill)
        outs.append(gdn.latent_attention(d, cache, cu, ints(lens), table, q, workspace=ws))
    check(outs[0], *absorbed(d, cache, [1, 1, 1], lens, table, q))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_absorbed_attention_in_a_graph_and_on_another_stream():
    """A captured call takes the lengths, the pages and the queries of each replay."""
    d = gdn.LatentDims(32, 512, page_size=32)
    cache, table = make_cache(d, [900, 900], 101)
    q = _queries(2, 32, 576, 102)
    cu, lens = cu_of([1, 1]), ints([900, 900])
    ws = torch.empty(max(1, gdn.latent_attention_workspace_size(d, cu)), dtype=torch.uint8, device="cuda")
    out = torch.empty(2, 32, 512, dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        gdn.latent_attention(d, cache, cu, lens, table, q, out=out, workspace=ws)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            gdn.latent_attention(d, cache, cu, lens, table, q, out=out, workspace=ws)
        for now in ([900, 900], [1, 640], [31, 33]):
            lens.copy_(ints(now))
            q.copy_(_queries(2, 32, 576, sum(now)))
            graph.replay()
            check(out, *absorbed(d, cache, [1, 1], now, table, q))
    _status_ok()


# ----------------------------------------------------------- expanded form
def _kv(counts_kv, heads, nope, vd, seed, fused, shared=False):
    g = gen(seed)
    t = sum(counts_kv)
    if fused:
        kv = torch.randn(t, heads, nope + vd, generator=g, device="cuda").bfloat16()
        k, v = kv[..., :nope], kv[..., nope:]
    else:
        k = torch.randn(t, 1 if shared else heads, nope, generator=g, device="cuda").bfloat16()
        v = torch.randn(t, 1 if shared else heads, vd, generator=g, device="cuda").bfloat16()
        if shared:
            k, v = k.expand(-1, heads, -1), v.expand(-1, heads, -1)
    rows = torch.randn(t, 576, generator=g, device="cuda").bfloat16()
    return k, rows[:, 512:], v


@pytest.mark.parametrize("heads,nope,vd,fused,counts,lens", [
    (1, 128, 128, False, [1], [1]),
    (4, 128, 128, True, [130], [130]),
    (4, 64, 64, True, [200, 1, 70], [200, 300, 70]),
    (3, 64, 128, False, [128, 129, 127], [128, 129, 127]),
    (2, 128, 64, True, [5, 0, 260, 64], [400, 70, 261, 64]),
    (20, 128, 128, True, [33], [1000]),
    (2, 128, 128, False, [600], [600]),
    (2, 128, 128, True, [257, 300], [513, 300]),
    (3, 64, 128, True, [300, 0, 513, 70], [300, 5, 700, 1000]),
    (1, 128, 128, False, [1030], [1030]),
    (40, 128, 128, True, [3, 300, 1, 17, 128, 5] * 4, [3, 301, 77, 400, 128, 64] * 4),   # many items a thread block
    (33, 64, 64, True, [9, 130, 1] * 9, [9, 131, 129] * 9),
    (1, 128, 64, True, [1] * 1100, [(i * 37) % 200 for i in range(1100)]),               # more blocks than are listed
    (1, 128, 128, True, [1] * 1100 + [300], [(i * 37) % 200 for i in range(1100)] + [310]),
    (2, 128, 128, True, [512, 256, 1], [640, 320, 64]),
    (16, 128, 128, True, [1] * 12, [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700]),
])
def test_expanded_attention(heads, nope, vd, fused, counts, lens):
    d = gdn.LatentDims(heads, nope_dim=nope, v_dim=vd)
    q = _queries(sum(counts), heads, nope + 64, 111, strided=True)
    k, r, v = _kv(lens, heads, nope, vd, 112, fused)
    got = gdn.expanded_attention(d, cu_of(counts), cu_of(lens), q, k, r, v)
    _status_ok()
    check(got, *expanded(d, counts, lens, q, k, r, v))


def test_expanded_attention_of_one_shared_head():
    d = gdn.LatentDims(6)
    k, r, v = _kv([150], 6, 128, 128, 121, False, shared=True)
    q = _queries(100, 6, 192, 122)
    got = gdn.expanded_attention(d, [0, 100], [0, 150], q, k, r, v)
    check(got, *expanded(d, [100], [150], q, k, r, v))


@pytest.mark.parametrize("more", [0, 400])
def test_expanded_queries_that_see_nothing_and_sequences_side_by_side(more):
    """More queries than keys; a neighbour's values that are no numbers do not come over."""
    d = gdn.LatentDims(4)
    counts, lens = [10, 140, 3, 5 + more], [4, 130, 0, 200 + more]
    k, r, v = _kv(lens, 4, 128, 128, 131, True)
    q = _queries(sum(counts), 4, 192, 132)
    want, tol = expanded(d, counts, lens, q, k, r, v)
    for bad in (math.nan, math.inf):
        k[134:], v[134:] = bad, bad       # the last sequence's
        got = gdn.expanded_attention(d, cu_of(counts), cu_of(lens), q, k, r, v)
        check(got[:153], want[:153], tol[:153])
        assert bool((got[:6] == 0).all()) and bool((got[10:20] == 0).all()) and bool((got[150:153] == 0).all())
    k[:134], v[:134] = math.nan, math.nan  # now the ones before it
    kv2 = _kv(lens, 4, 128, 128, 131, True)
    k[134:], v[134:] = kv2[0][134:], kv2[2][134:]
    got = gdn.expanded_attention(d, cu_of(counts), cu_of(lens), q, k, r, v)
    check(got[153:], want[153:], tol[153:])
    _status_ok()


def test_expanded_attention_without_any_key():
    d = gdn.LatentDims(4)
    e = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    got = gdn.expanded_attention(d, [0, 3], [0, 0], _queries(3, 4, 192, 1), e, e.new_empty(0, 64), e)
    assert bool((got == 0).all())
    got = gdn.expanded_attention(d, [0, 0], [0, 0], _queries(0, 4, 192, 1), e, e.new_empty(0, 64), e)
    assert got.shape == (0, 4, 128)


def test_expanded_attention_in_a_graph_on_another_stream():
    d = gdn.LatentDims(4)
    cu, ck = cu_of([100, 40]), cu_of([164, 300])
    q = _queries(140, 4, 192, 142)
    k, r, v = _kv([164, 300], 4, 128, 128, 141, True)
    out = torch.empty(140, 4, 128, dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        gdn.expanded_attention(d, cu, ck, q, k, r, v, out=out)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            gdn.expanded_attention(d, cu, ck, q, k, r, v, out=out)
        for seed in (1, 2):
            q.copy_(_queries(140, 4, 192, seed))
            graph.replay()
            check(out, *expanded(d, [100, 40], [164, 300], q, k, r, v))
    _status_ok()


@pytest.mark.parametrize("nope,vd", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("rise", [False, True])
def test_expanded_pieces_of_one_query_tile(nope, vd, rise):
    """Up to 128 queries, also at the end of longer pieces, behind contexts of one to many key tiles; with
    scores that rise along the keys, or fall."""
    d = gdn.LatentDims(7, nope_dim=nope, v_dim=vd)
    counts = [1, 128, 100, 1, 1, 257, 384, 5, 60, 127]
    lens = [1000, 128, 129, 128, 129, 257, 1500, 4, 385, 2600]
    k, r, v = _kv(lens, 7, nope, vd, 181, True)
    if rise:
        grow = torch.cat([torch.linspace(0.1, 4.0, n, device="cuda") for n in lens])[:, None, None]
        grow = torch.cat([grow.expand(-1, 4, 1), grow.flip(0).expand(-1, 3, 1)], 1)
        k, r = (k * grow).bfloat16(), r * 0.25
    q = _queries(sum(counts), 7, nope + 64, 182)
    check(gdn.expanded_attention(d, cu_of(counts), cu_of(lens), q, k, r, v), *expanded(d, counts, lens, q, k, r, v))
    _status_ok()


@pytest.mark.parametrize("n", [129, 200, 257, 300, 500, 640])
def test_expanded_pieces_keep_a_neighbours_values_out(n):
    """Tiles that end within the next sequence's rows, by either half of the thread block."""
    d = gdn.LatentDims(3)
    counts, lens = [7, 3], [n, 400]
    k, r, v = _kv(lens, 3, 128, 128, 191, False)
    q = _queries(10, 3, 192, 192)
    want, tol = expanded(d, counts, lens, q, k, r, v)
    k[n:], v[n:] = math.nan, math.nan
    got = gdn.expanded_attention(d, cu_of(counts), cu_of(lens), q, k, r, v)
    check(got[:7], want[:7], tol[:7])
    assert bool(got[7:].isnan().all())
    _status_ok()


def test_expanded_results_repeat():
    """Which thread block takes an item does not matter."""
    d = gdn.LatentDims(16)
    counts = [300, 1, 77, 600, 130, 256, 40, 511] * 2
    lens = [c + 137 * i for i, c in enumerate(counts)]
    k, r, v = _kv(lens, 16, 128, 128, 193, True)
    q, cu, ck = _queries(sum(counts), 16, 192, 194), cu_of(counts), cu_of(lens)
    first = gdn.expanded_attention(d, cu, ck, q, k, r, v)
    for _ in range(20):
        assert torch.equal(gdn.expanded_attention(d, cu, ck, q, k, r, v), first)
    check(first, *expanded(d, counts, lens, q, k, r, v))
    _status_ok()


# ------------------------------------------------------------------ copies
def _filled(d, n, seed):
    c = gdn.KVCache.empty(d, n) if isinstance(d, gdn.KVDims) else gdn.LatentCache.empty(d, n)
    g = gen(seed)
    for t in (c.k, c.v, c.k_scale, c.v_scale) if isinstance(d, gdn.KVDims) else (c.rows,):
        raw = t.view(torch.uint8)
        raw.copy_(torch.randint(0, 256, raw.shape, generator=g, device="cuda", dtype=torch.uint8))
    return c


def _tensors(c):
    ts = (c.k, c.v, c.k_scale, c.v_scale) if isinstance(c, gdn.KVCache) else (c.rows,)
    return [t.view(torch.uint8) for t in ts]


@pytest.mark.parametrize("make,n_pages,pairs", [
    (lambda: gdn.LatentDims(4, 512, page_size=64), 40, 7),
    (lambda: gdn.LatentDims(4, 256, page_size=16), 1300, 600),
    (lambda: gdn.KVDims(4, 1, 64, page_size=16), 20, 10),
    (lambda: gdn.KVDims(8, 3, 128, page_size=32, cache="e4m3"), 30, 9),
    (lambda: gdn.KVDims(16, 4, 256, page_size=128), 11, 5),
])
@pytest.mark.parametrize("layers", [1, 3])
def test_pages_are_copied_in_every_cache(make, n_pages, pairs, layers):
    caches = [_filled(make(), n_pages, 7 + i) for i in range(layers)]
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(3)).to(torch.int32)
    src, dst = order[:pairs].contiguous(), order[pairs:2 * pairs].contiguous()
    src[pairs // 2] = src[0]  # one page to two places: a fork
    want = [[t.clone() for t in _tensors(c)] for c in caches]
    for c in want:
        for t in c:
            t[dst.long().cuda()] = t[src.long().cuda()]
    gdn.copy_pages(caches if layers > 1 else caches[0], src, dst)
    for c, ts in zip(caches, want):
        assert all(torch.equal(a, b) for a, b in zip(_tensors(c), ts))
    gdn.copy_pages(caches, [], [])


def test_copies_of_many_layers_and_beyond_32_bits():
    d = gdn.LatentDims(1, 512)
    n = 2 ** 32 // (64 * 576 * 2) + 3
    cache = gdn.LatentCache.empty(d, n)
    cache.rows[n - 1], cache.rows[0] = 3.0, 1.0
    gdn.copy_pages(cache, [n - 1, 0], [1, n - 2])
    assert bool((cache.rows[1] == 3.0).all()) and bool((cache.rows[n - 2] == 1.0).all())
    small = gdn.KVDims(2, 1, 64, page_size=16)
    caches = [_filled(small, 6, i) for i in range(50)]
    want = [[t.clone() for t in _tensors(c)] for c in caches]
    gdn.copy_pages(caches, [0, 5], [3, 1])
    for c, ts in zip(caches, want):
        for a, b in zip(_tensors(c), ts):
            b[3], b[1] = b[0].clone(), b[5].clone()
            assert torch.equal(a, b)


def test_a_captured_copy_keeps_its_pairs():
    cache = _filled(gdn.LatentDims(1, 256, page_size=16), 10, 1)
    src, dst = [1, 2], [5, 6]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            gdn.copy_pages(cache, src, dst)
        src[0] = dst[0] = 9
        for fill in (0.5, 2.0):
            cache.rows[1], cache.rows[2] = fill, -fill
            graph.replay()
            assert bool((cache.rows[5] == fill).all()) and bool((cache.rows[6] == -fill).all())


# ---------------------------------------------------------------- together
def test_prompt_then_drafts_of_a_forked_sequence():
    """A prompt in the expanded form, its continuation behind the cached prefix in both forms, and a
    fork of the sequence whose last page was copied: all one attention."""
    heads, page = 8, 16
    d = gdn.LatentDims(heads, 512, page_size=page, rope_style="interleaved")
    g = gen(151)
    w_uk = (torch.randn(heads, 128, 512, generator=g, device="cuda") / 512 ** 0.5).bfloat16()
    w_uv = (torch.randn(heads, 512, 128, generator=g, device="cuda") / 512 ** 0.5).bfloat16()
    norm = torch.ones(512, device="cuda")
    n0, n1 = 100, 5
    c = torch.randn(n0 + n1, 576, generator=g, device="cuda").bfloat16()
    q = torch.randn(n0 + n1, heads, 192, generator=g, device="cuda").bfloat16()
    tab = rope_table(200)
    cache = gdn.LatentCache.empty(d, 20)
    table = torch.randperm(20, generator=g, device="cuda").to(torch.int32)[:16].view(2, 8)

    def expand(rows):
        lat = rows[:, :512].float()
        return (torch.einsum("tc,hnc->thn", lat, w_uk.float()).bfloat16(),
                torch.einsum("tc,hcv->thv", lat, w_uv.float()).bfloat16())

    def reference(rows, qs, start):
        """In 64 bits from the stored rows and the rotated queries."""
        r = rows.double()
        k = torch.cat([torch.einsum("tc,hnc->thn", r[:, :512], w_uk.double()),
                       r[:, None, 512:].expand(-1, heads, -1)], -1)
        v = torch.einsum("tc,hcv->thv", r[:, :512], w_uv.double())
        s = torch.einsum("qhd,khd->hqk", qs.double(), k) * 192 ** -0.5
        hide = torch.arange(len(r), device="cuda") > torch.arange(start, start + len(qs), device="cuda")[:, None]
        p = torch.softmax(s.masked_fill(hide, -math.inf), -1)
        return torch.einsum("hqk,khv->qhv", p, v), torch.einsum("hqk,khv->qhv", p, v.abs()), float(
            (torch.einsum("qhd,khd->hqk", qs.double().abs(), k.abs()) * 192 ** -0.5).max())

    def close(got, ref):
        """Keys, values (or queries and outputs in latent space) rounded to bf16 on the way: a score is
        off by at most u S, each weight and value by u, the result by u once or twice more."""
        o, weight, size = ref
        check(got.double(), o, (2 * U * size + 6 * U) * weight + 4 * U)

    rows = torch.empty(n0, 576, dtype=torch.bfloat16, device="cuda")
    qp = q[:n0].clone()
    gdn.latent_append(d, cache, [0, n0], ints([n0]), table[:1], c[:n0], norm_w=norm, rope=tab, q_rope=qp[..., 128:],
                      q_out=qp[..., 128:], rows_out=rows)
    k, v = expand(rows)
    close(gdn.expanded_attention(d, [0, n0], [0, n0], qp, k, rows[:, 512:], v), reference(rows, qp, 0))

    # fork: the full pages are shared, the last one, partly filled, is copied
    full = n0 // page
    table[1, :full] = table[0, :full]
    own = int(table[1, full])
    gdn.copy_pages(cache, [int(table[0, full])], [own])
    # both continue, the fork with other tokens
    cc = torch.cat([c[n0:], c[n0:].flip(0)])
    qq = torch.cat([q[n0:], q[n0:].flip(0)])
    lens = ints([n0 + n1, n0 + n1])
    ql = torch.empty(2 * n1, heads, 576, dtype=torch.bfloat16, device="cuda")
    gdn.latent_append(d, cache, [0, n1, 2 * n1], lens, table, cc, norm_w=norm, rope=tab, q_rope=qq[..., 128:],
                      q_out=ql[..., 512:])
    ql[..., :512] = torch.einsum("thn,hnc->thc", qq[..., :128].float(), w_uk.float()).bfloat16()
    o = gdn.latent_attention(d, cache, [0, n1, 2 * n1], lens, table, ql)
    o = torch.einsum("thc,hcv->thv", o.float(), w_uv.float())
    back = gdn.latent_read(d, cache, [0, n0 + n1, 2 * (n0 + n1)], lens - lens, table)
    assert torch.equal(back[:n0], rows) and torch.equal(back[n0 + n1:2 * n0 + n1], rows)
    qr = torch.cat([qq[..., :128], ql[..., 512:]], -1)
    k, v = expand(back)
    e = gdn.expanded_attention(d, [0, n1, 2 * n1], [0, n0 + n1, 2 * (n0 + n1)], qr, k, back[:, 512:], v)
    for i in range(2):
        part, whole = slice(i * n1, (i + 1) * n1), slice(i * (n0 + n1), (i + 1) * (n0 + n1))
        ref = reference(back[whole], qr[part], n0)
        close(o[part], ref)
        close(e[part], ref)
    _status_ok()


# ------------------------------------------------------ waits that run out
@pytest.mark.parametrize("heads,counts,lens,strided", [(16, [1, 1], [700, 80], False), (32, [1], [3000], True), (32, [4], [500], False)])
def test_latent_attention_reports_a_wait_that_runs_out(monkeypatch, heads, counts, lens, strided):
    """Loads that are never started (GDN_FAULT=stall_latent): every role gives up after 2 s, the status
    says so, and the next call is right.  By one thread block a span, and by pairs."""
    d = gdn.LatentDims(heads, 512)
    cache, table = make_cache(d, lens, 161)
    q = _queries(sum(counts), heads, 576, 162, strided=strided)
    monkeypatch.setenv("GDN_FAULT", "stall_latent")
    gdn.latent_attention(d, cache, cu_of(counts), ints(lens), table, q)
    with pytest.raises(gdn.GDNError) as e:
        gdn.sync_status()
    assert e.value.status == gdn.GDN_ERR_TIMEOUT
    _status_ok()
    monkeypatch.delenv("GDN_FAULT")
    got = gdn.latent_attention(d, cache, cu_of(counts), ints(lens), table, q)
    _status_ok()
    check(got, *absorbed(d, cache, counts, lens, table, q))


def test_expanded_attention_reports_a_wait_that_runs_out(monkeypatch):
    d = gdn.LatentDims(4)
    counts, lens = [300, 5], [300, 400]
    k, r, v = _kv(lens, 4, 128, 128, 171, True)
    q = _queries(305, 4, 192, 172)
    monkeypatch.setenv("GDN_FAULT", "stall_expanded")
    gdn.expanded_attention(d, cu_of(counts), cu_of(lens), q, k, r, v)
    with pytest.raises(gdn.GDNError) as e:
        gdn.sync_status()
    assert e.value.status == gdn.GDN_ERR_TIMEOUT
    _status_ok()
    monkeypatch.delenv("GDN_FAULT")
    got = gdn.expanded_attention(d, cu_of(counts), cu_of(lens), q, k, r, v)
    _status_ok()
    check(got, *expanded(d, counts, lens, q, k, r, v))


# ------------------------------------------------- strides, streams, graphs
@pytest.mark.parametrize("heads,counts,lens", [(16, [1, 1, 1], [70, 300, 1]), (8, [9, 40], [500, 41])])
@pytest.mark.parametrize("form", ["head_stride_0", "token_stride_0", "heads_first", "wide"])
def test_absorbed_queries_with_any_strides(heads, counts, lens, form):
    d = gdn.LatentDims(heads, 256, page_size=32)
    t, g = sum(counts), gen(161)
    cache, table = make_cache(d, lens, 162)
    if form == "head_stride_0":
        q = torch.randn(t, 1, 320, generator=g, device="cuda").bfloat16().expand(t, heads, 320)
    elif form == "token_stride_0":
        q = torch.randn(1, heads, 320, generator=g, device="cuda").bfloat16().expand(t, heads, 320)
    elif form == "heads_first":
        q = torch.randn(heads, t, 320, generator=g, device="cuda").bfloat16().transpose(0, 1)
    else:
        q = torch.randn(t, heads + 1, 384, generator=g, device="cuda").bfloat16()[:, 1:, 40:360]
    got = gdn.latent_attention(d, cache, cu_of(counts), ints(lens), table, q)
    check(got, *absorbed(d, cache, counts, lens, table, q))
    _status_ok()


@pytest.mark.parametrize("form", ["heads_first", "head_stride_0"])
def test_expanded_rows_with_any_strides(form):
    d = gdn.LatentDims(5, nope_dim=64, v_dim=128)
    g = gen(163)

    def make(t, width):
        if form == "heads_first":
            return torch.randn(5, t, width, generator=g, device="cuda").bfloat16().transpose(0, 1)
        return torch.randn(t, 1, width, generator=g, device="cuda").bfloat16().expand(t, 5, width)

    counts, lens = [3, 150], [200, 150]
    q, k, v = make(153, 128), make(350, 64), make(350, 128)
    r = torch.randn(350, 192, generator=g, device="cuda").bfloat16()[:, 64:128]
    check(gdn.expanded_attention(d, cu_of(counts), cu_of(lens), q, k, r, v), *expanded(d, counts, lens, q, k, r, v))
    _status_ok()


def test_rows_are_packed_into_the_appended_ones():
    """rows_out may be c itself."""
    d = gdn.LatentDims(2, 512, page_size=16, rope_style="interleaved")
    g = gen(164)
    cache, table = make_cache(d, [300], 165)
    c = torch.randn(300, 576, generator=g, device="cuda").bfloat16()
    w, tab = torch.rand(512, generator=g, device="cuda") + 0.5, rope_table(300)
    packed = torch.empty_like(c)
    gdn.latent_append(d, cache, [0, 300], ints([300]), table, c, norm_w=w, rope=tab, rows_out=packed)
    gdn.latent_append(d, cache, [0, 300], ints([300]), table, c, norm_w=w, rope=tab, rows_out=c)
    assert torch.equal(c, packed)
    assert torch.equal(gdn.latent_read(d, cache, [0, 300], ints([0]), table), packed)
    _status_ok()


def test_calls_on_two_streams_and_graphs_at_once():
    """Two captured calls with a workspace each, replayed on streams of their own."""
    d = gdn.LatentDims(32, 512)
    runs = []
    for i, (counts, lens) in enumerate([([1, 1, 1], [5000, 3, 900]), ([4], [3000])]):
        cache, table = make_cache(d, lens, 170 + i)
        q = _queries(sum(counts), 32, 576, 172 + i)
        cu, n, ws = cu_of(counts), ints(lens), None
        ws = torch.empty(gdn.latent_attention_workspace_size(d, cu), dtype=torch.uint8, device="cuda")
        out = torch.empty(sum(counts), 32, 512, dtype=torch.bfloat16, device="cuda")
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            gdn.latent_attention(d, cache, cu, n, table, q, out=out, workspace=ws)
        runs.append((graph, stream, out, absorbed(d, cache, counts, lens, table, q), (cache, table, q, cu, n, ws)))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, out, want, _ in runs:
        check(out, *want)
    _status_ok()


def test_copies_of_thousands_of_pairs():
    cache = _filled(gdn.LatentDims(1, 256, page_size=16), 9001, 3)
    order = torch.randperm(9001, generator=torch.Generator().manual_seed(5)).to(torch.int32)
    src, dst = order[:4500].contiguous(), order[4500:9000].contiguous()
    want = cache.rows.clone()
    want[dst.long().cuda()] = want[src.long().cuda()]
    gdn.copy_pages(cache, src.tolist(), dst)
    assert torch.equal(cache.rows.view(torch.int16), want.view(torch.int16))


def test_first_calls_of_a_process_may_be_captured():
    """Nothing is set up by an eager call that a captured one needs."""
    import subprocess
    import sys
    code = """
import torch, gated_deltanet_linear_mixer_gb300 as gdn
d = gdn.LatentDims(4, 256, page_size=16)
i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
rows = torch.ones(4, 16, 320, device="cuda").bfloat16()
cache, table, lens, starts = gdn.LatentCache(d, rows), i([[2, 0]]), i([20]), i([0])
cu = (i([0, 20]), torch.tensor([0, 20], dtype=torch.int32))
c = torch.full((20, 320), 2.0, device="cuda").bfloat16()
q, qe = torch.ones(20, 4, 320, device="cuda").bfloat16(), torch.ones(20, 4, 192, device="cuda").bfloat16()
k, v = torch.ones(20, 4, 128, device="cuda").bfloat16(), torch.full((20, 4, 128), 3.0, device="cuda").bfloat16()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    gdn.latent_append(d, cache, cu, lens, table, c)
    o = gdn.latent_attention(d, cache, cu, lens, table, q)
    e = gdn.expanded_attention(d, cu, cu, qe, k, c[:, 256:], v)
    gdn.copy_pages(cache, [2], [3])
    r = gdn.latent_read(d, cache, cu, starts, table)
assert bool((rows == 1).all())
g.replay()
torch.cuda.synchronize()
gdn.sync_status()
assert bool((o == 2).all()) and bool((e == 3).all()) and bool((r == 2).all()) and bool((rows[3] == 2).all())
assert bool((rows[0, :4] == 2).all()) and bool((rows[0, 4:] == 1).all())
"""
    import pathlib
    got = subprocess.run([sys.executable, "-c", code], cwd=pathlib.Path(__file__).parents[1], capture_output=True, text=True,
                         timeout=300)
    assert got.returncode == 0, got.stderr[-2000:]


def test_expanded_calls_on_two_streams_at_once():
    """Thread blocks take over items of their own call only; calls of several launches too."""
    runs = []
    for i, (heads, counts, lens) in enumerate([(16, [700, 90, 300], [900, 500, 301]), (8, [600, 1, 64], [600, 700, 64]),
                                               (1, [1] * 1030 + [300], [9] * 1030 + [310])]):
        d = gdn.LatentDims(heads)
        q, (k, r, v) = _queries(sum(counts), heads, 192, 200 + i), _kv(lens, heads, 128, 128, 210 + i, True)
        out = torch.empty(sum(counts), heads, 128, dtype=torch.bfloat16, device="cuda")
        args = (d, cu_of(counts), cu_of(lens), q, k, r, v)
        runs.append((args, out, torch.cuda.Stream(), expanded(d, counts, lens, q, k, r, v)))
    torch.cuda.synchronize()
    for _ in range(20):
        for args, out, stream, _ in runs:
            with torch.cuda.stream(stream):
                gdn.expanded_attention(*args, out=out)
    torch.cuda.synchronize()
    for _, out, _, want in runs:
        check(out, *want)
    _status_ok()


def test_rows_beyond_32_bit_offsets_are_appended_and_read():
    d = gdn.LatentDims(2, 512)
    first = 2 ** 32 // (64 * 576) + 1  # its first element's index passes 32 bits
    rows = torch.empty(first + 4, 64, 576, dtype=torch.bfloat16, device="cuda")
    cache, table = gdn.LatentCache(d, rows), ints([[first + 2, first]])
    c = torch.randn(100, 576, generator=gen(220), device="cuda").bfloat16()
    gdn.latent_append(d, cache, [0, 100], ints([100]), table, c)
    assert torch.equal(rows[first + 2], c[:64]) and torch.equal(rows[first, :36], c[64:])
    assert torch.equal(gdn.latent_read(d, cache, [0, 90], ints([10]), table), c[10:])
    _status_ok()


@pytest.mark.parametrize("far", ["keys", "results"])
def test_expanded_attention_beyond_32_bit_offsets(far):
    """A short sequence behind one of 600,000 keys without queries, or as many queries without keys."""
    d, n = gdn.LatentDims(32), 600_000
    counts, lens = ([0, 5], [n, 300]) if far == "keys" else ([n, 5], [0, 300])
    g = gen(221)
    k = torch.zeros(sum(lens), 32, 256, dtype=torch.bfloat16, device="cuda")
    k[-300:] = torch.randn(300, 32, 256, generator=g, device="cuda").bfloat16()
    r = torch.zeros(sum(lens), 64, dtype=torch.bfloat16, device="cuda")
    r[-300:] = torch.randn(300, 64, generator=g, device="cuda").bfloat16()
    q = torch.zeros(sum(counts), 32, 192, dtype=torch.bfloat16, device="cuda")
    q[-5:] = _queries(5, 32, 192, 222)
    got = gdn.expanded_attention(d, cu_of(counts), cu_of(lens), q, k[..., :128], r, k[..., 128:])
    _status_ok()
    check(got[-5:], *expanded(d, [5], [300], q[-5:], k[-300:, :, :128], r[-300:], k[-300:, :, 128:]))
    assert not got[:-5].any()


def test_expanded_attention_that_waits_in_vain_takes_no_other_blocks_time(monkeypatch):
    """Many more thread blocks than run at once: those that gave up keep the others from starting to
    wait as long, and the next call takes all of its blocks."""
    import time
    d = gdn.LatentDims(40)
    counts, lens = [300, 5, 130, 256] * 6, [300, 400, 131, 700] * 6
    k, r, v = _kv(lens, 40, 128, 128, 231, True)
    q = _queries(sum(counts), 40, 192, 232)
    monkeypatch.setenv("GDN_FAULT", "stall_expanded")
    torch.cuda.synchronize()
    start = time.monotonic()
    gdn.expanded_attention(d, cu_of(counts), cu_of(lens), q, k, r, v)
    with pytest.raises(gdn.GDNError) as e:
        gdn.sync_status()
    assert e.value.status == gdn.GDN_ERR_TIMEOUT
    assert time.monotonic() - start < 9.0  # waits of 2 s: of one wave of blocks, not of eight
    monkeypatch.delenv("GDN_FAULT")
    got = gdn.expanded_attention(d, cu_of(counts), cu_of(lens), q, k, r, v)
    _status_ok()
    check(got, *expanded(d, counts, lens, q, k, r, v))
