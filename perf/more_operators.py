"""Measured cases of the latent cache's operators, of expanded attention and of page copies.

A stack that interleaves per-channel-decay mixers with latent attention keeps one
vector a token in its cache: a normalised latent of C channels and a position
key of R channels that all heads share.  Five operators: appending tokens
(norm, rotation, store), reading rows back, attention over the cache in the
absorbed form (queries in latent space, values are the latents), attention in
the expanded form (keys and values of each head, made from the latents by a
projection), and copying pages for forked sequences and compacted pools.  `run`
computes them in their plain form (elementary torch operations in 32 bits), or,
where `own` is true, through this package's entry points.

The cache: rows [pages, page, C + R] bf16; block_table [n, pages per sequence];
kv_lens counts a call's own tokens, so sequence i's q_i tokens sit at
kv_lens[i] - q_i onwards.
"""
import math
import random

import torch

own = False

R = 64  # channels of the position key


def _latent(name, n, q, ragged, ctx_lo, ctx_hi, heads, dc, page, lens=1):
    return dict(name=name, op="latent", n=n, q=q, ragged=ragged, ctx_lo=ctx_lo, ctx_hi=ctx_hi,
                heads=heads, dc=dc, page=page, lens=lens)


def _expanded(name, n, q, ragged, ctx_lo, ctx_hi, heads, nope, vd, fused, lens=1):
    return dict(name=name, op="expanded", n=n, q=q, ragged=ragged, ctx_lo=ctx_lo, ctx_hi=ctx_hi,
                heads=heads, nope=nope, vd=vd, fused=fused, lens=lens)


def _append(name, n, q, ragged, ctx_lo, ctx_hi, heads, dc, page, norm, rope, style, lens=1):
    return dict(name=name, op="append", n=n, q=q, ragged=ragged, ctx_lo=ctx_lo, ctx_hi=ctx_hi,
                heads=heads, dc=dc, page=page, norm=norm, rope=rope, style=style, lens=lens)


def listed():
    return [
        # one user's chat turn: the latency of a single token's attention
        _latent("latent_1x1_ctx1000", 1, 1, False, 1000, 1000, 32, 512, 64),
        # a long document open in one session: few rows, a long axis to split
        _latent("latent_1x1_ctx131000", 1, 1, False, 131000, 131000, 16, 512, 64),
        # the decode batch of a server: 256 ragged contexts
        _latent("latent_256x1", 256, 1, False, 127, 8191, 32, 512, 64, lens=2),
        # speculative verify: four drafts of each of 64 sequences, small pages; at 128 rows a
        # sequence the products weigh as much as the cache's bytes
        _latent("latent_64x4", 64, 4, False, 500, 6000, 32, 512, 16, lens=3),
        # a prompt of 4096 tokens from an empty cache
        _expanded("expanded_prompt_4096", 1, 4096, False, 0, 0, 32, 128, 128, True),
        # ragged prompt pieces behind cached prefixes that were read back and expanded
        _expanded("expanded_16_prompts", 16, 1100, True, 0, 3000, 16, 128, 128, False, lens=4),
        # the decode batch's append: one token each, pages partly filled
        _append("append_256x1", 256, 1, False, 127, 2047, 32, 512, 64, True, True, "half", lens=2),
        # sixteen ragged prompts appended behind cached prefixes
        _append("append_16_prompts", 16, 1100, True, 0, 3000, 32, 512, 32, True, True,
                "interleaved", lens=4),
        # cached prefixes taken out of the pages to be expanded: four sequences
        dict(name="read_4x4000", op="read", n=4, rows_lo=3500, rows_hi=4500, dc=512, page=16, lens=5),
        # one short sequence's rows, for inspection
        dict(name="read_1x300", op="read", n=1, rows_lo=300, rows_hi=300, dc=256, page=64, lens=6),
        # 64 sequences forked: the last, partly filled page of each, in the caches of 4 layers
        dict(name="copy_64_pages_4_layers", op="copy", layers=4, pages=300, pairs=64, dc=512, page=64),
        # a pool compacted: a third of its pages moved, one layer
        dict(name="copy_2000_pages", op="copy", layers=1, pages=6000, pairs=2000, dc=512, page=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["latent", "latent", "latent", "expanded", "expanded", "append", "append", "read",
                     "copy"])
    page = rng.choice([16, 32, 64, 128])
    dc = rng.choice([256, 512, 512])
    lens = rng.randrange(1 << 20)
    if op == "copy":
        pages = _log_int(rng, 8, 200_000 // page)
        layers = rng.choice([1, 2, 4, 7])
        pages = max(8, pages // layers)
        return dict(op=op, layers=layers, pages=pages, pairs=_log_int(rng, 1, pages // 3), dc=dc,
                    page=page)
    if op == "read":
        hi = _log_int(rng, 1, 8000)
        n = _log_int(rng, 1, max(1, min(64, 32000 // hi)))
        return dict(op=op, n=n, rows_lo=max(1, hi // 2), rows_hi=hi, dc=dc, page=page, lens=lens)
    heads = rng.choice([8, 16, 20, 32, 64, 128]) if op == "latent" else rng.choice([4, 8, 16, 20, 32])
    kind = rng.choice(["decode", "verify", "prompt"]) if op != "expanded" else "prompt"
    if kind == "prompt":
        q = _log_int(rng, 17, 256 if op == "latent" else 2500)
        n = _log_int(rng, 1, max(1, (512 if op == "latent" else 5000) // q))
        ctx = rng.choice([0, _log_int(rng, 1, 2000)])
    else:
        q = 1 if kind == "decode" else rng.randint(2, 8)
        ctx = _log_int(rng, 1, 32000)
        n = _log_int(rng, 1, max(1, min(256, 400_000 // (ctx * max(1, heads * q // 64)))))
    base = dict(op=op, n=n, q=q, ragged=kind != "decode" and rng.random() < 0.5, ctx_lo=ctx // 2,
                ctx_hi=ctx, heads=heads, lens=lens)
    if op == "expanded":
        base.update(nope=rng.choice([64, 128, 128]), vd=rng.choice([64, 128, 128]),
                    fused=rng.random() < 0.5)
        return base
    base.update(dc=dc, page=page)
    if op == "append":
        base.update(norm=rng.random() < 0.7, rope=rng.random() < 0.8,
                    style=rng.choice(["half", "interleaved"]))
    return base


def _lengths(case):
    """Host lists of new tokens and of lengths after them (read: rows and lengths)."""
    r = random.Random(case["lens"])
    if case["op"] == "read":
        rows = [r.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["n"])]
        return rows, [k + r.randint(0, 40) for k in rows]
    qs = [r.randint(1, case["q"]) if case["ragged"] else case["q"] for _ in range(case["n"])]
    return qs, [q + r.randint(case["ctx_lo"], case["ctx_hi"]) for q in qs]


def work(case):
    if case["op"] == "copy":
        return {"bytes": 4 * case["layers"] * case["pairs"] * case["page"] * (case["dc"] + R), "flops": 0}
    qs, kvs = _lengths(case)
    t = sum(qs)
    if case["op"] == "read":
        return {"bytes": 4 * t * (case["dc"] + R), "flops": 0}
    h = case["heads"]
    if case["op"] == "append":  # the token's row read, and written to its page and packed; q both ways
        d = case["dc"] + R
        return {"bytes": 6 * t * d + 4 * t * h * R, "flops": 5 * t * d + 3 * t * h * R}
    pairs = sum(q * (kv - q) + q * (q + 1) // 2 for q, kv in zip(qs, kvs))
    if case["op"] == "latent":
        d = case["dc"] + R
        return {"bytes": 2 * sum(kvs) * d + 2 * t * h * (d + case["dc"]),
                "flops": 2 * pairs * h * (d + case["dc"])}
    n, v = case["nope"], case["vd"]
    return {"bytes": 2 * sum(kvs) * (h * (n + v) + R) + 2 * t * h * (n + R + v),
            "flops": 2 * pairs * h * (n + R + v)}


# ------------------------------------------------------------------- inputs
def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _rows(starts, counts):
    """(sequence, position) of counts[i] consecutive positions from starts[i], all sequences."""
    c = _ints(counts, torch.int64)
    seq = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), c)
    first = torch.cumsum(c, 0) - c
    pos = torch.arange(sum(counts), device="cuda") - first[seq] + _ints(starts, torch.int64)[seq]
    return seq, pos


def _cu(counts):
    total, cu = 0, [0]
    for c in counts:
        total += c
        cu.append(total)
    host = torch.tensor(cu, dtype=torch.int32)
    return host.cuda(), host


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "copy":
        # the pairs are on the host, where a server keeps its pages' bookkeeping
        order = random.Random(seed).sample(range(case["pages"]), 2 * case["pairs"])
        s["src"], s["dst"] = order[: case["pairs"]], order[case["pairs"]:]
        shape = (case["pages"], case["page"], case["dc"] + R)
        s["pools"] = [normal(*shape).bfloat16() for _ in range(case["layers"])]
        return s
    s["counts"], s["kvs"] = counts, kvs = _lengths(case)
    s["cu"], s["kv_lens"], s["max_kv"], s["max_q"] = _cu(counts), _ints(kvs), max(kvs), max(counts)
    s["q_lens"] = _ints(counts, torch.int64)
    t = sum(counts)
    s["seq"], s["pos"] = _rows([kv - q for q, kv in zip(counts, kvs)], counts)
    if case["op"] == "expanded":
        h, n, v = case["heads"], case["nope"], case["vd"]
        # heads look at different distances: some flat, some peaked
        s["q"] = (normal(t, h, n + R) * normal(h, 1).mul_(0.4).exp_()).bfloat16()
        s["cu_kv"] = _cu(kvs)
        if case["fused"]:  # one projection's output: keys | values of a head side by side
            kv = normal(sum(kvs), h, n + v).bfloat16()
            s["k"], s["v"] = kv[..., :n], kv[..., n:]
        else:
            s["k"], s["v"] = normal(sum(kvs), h, n).bfloat16(), normal(sum(kvs), h, v).bfloat16()
        s["k_rope"] = normal(sum(kvs), R).bfloat16()
        return s
    # a cache in use: pages in no order
    dc, page = case["dc"], case["page"]
    need = [-(-kv // page) for kv in kvs]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    s["table"] = torch.zeros(len(kvs), max(need), dtype=torch.int32, device="cuda")
    seq, at = _rows([0] * len(kvs), need)
    s["table"][seq, at] = order[: sum(need)]
    s["rows"] = normal(pages, page, dc + R).bfloat16()
    if case["op"] == "read":
        s["starts"] = _ints([0] * len(counts))
        s["pos"] = _rows([0] * len(counts), counts)[1]
        return s
    h = case["heads"]
    if case["op"] == "latent":
        s["q"] = (normal(t, h, dc + R) * normal(h, 1).mul_(0.4).exp_()).bfloat16()
        return s
    # the down projection's output: latent | position key of a token side by side
    s["c"] = normal(t, dc + R).mul_(1.7).bfloat16()
    s["w"] = 1.0 + 0.1 * normal(dc) if case["norm"] else None
    # queries as the expanded form has them: the position part behind 128 channels of a head
    s["q"] = normal(t, h, 128 + R).bfloat16()
    s["table_rope"] = None
    if case["rope"]:
        inv = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
        ang = torch.arange(max(kvs), device="cuda", dtype=torch.float64)[:, None] * inv[None]
        s["table_rope"] = torch.cat([ang.cos(), ang.sin()], -1).float().contiguous()
    return s


# -------------------------------------------------------------- plain forms
def _turned(s, x):
    """x [T, heads, R] turned by its token's position, in 32 bits."""
    x = x.float()
    if s["table_rope"] is None:
        return x
    c, sn = s["table_rope"][s["pos"]][:, None].chunk(2, -1)
    out = torch.empty_like(x)
    if s["style"] == "half":
        a, b = x.chunk(2, -1)
        out[..., : R // 2], out[..., R // 2:] = a * c - b * sn, b * c + a * sn
    else:
        a, b = x[..., 0::2], x[..., 1::2]
        out[..., 0::2], out[..., 1::2] = a * c - b * sn, b * c + a * sn
    return out


def _plain_append(s):
    dc = s["dc"]
    c = s["c"][:, :dc].float()
    if s["norm"]:
        c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + 1e-6) * s["w"]
    k = _turned(s, s["c"][:, None, dc:])[:, 0]
    packed = torch.cat([c, k], -1).bfloat16()
    page = s["table"][s["seq"], s["pos"] // s["page"]].long()
    s["rows"][page, s["pos"] % s["page"]] = packed
    return {"q": _turned(s, s["q"][..., 128:]).bfloat16(), "packed": packed, "rows": s["rows"]}


def _places(s):
    """The place of each token of the call in a padded batch, and what each place sees."""
    line = s["pos"] - (s["kv_lens"].long() - s["q_lens"])[s["seq"]]
    place = (s["kv_lens"].long() - s["q_lens"])[:, None] + torch.arange(s["max_q"], device="cuda")
    see = torch.arange(s["max_kv"], device="cuda")[None, None] <= place[..., None]
    return line, see


def _plain_latent(s):
    n, h, dc = s["n"], s["heads"], s["dc"]
    at = torch.arange(s["max_kv"], device="cuda")
    rows = s["rows"][s["table"][:, at // s["page"]].long(), at % s["page"]].float()
    line, see = _places(s)
    q = torch.zeros(n, s["max_q"], h, dc + R, device="cuda")
    q[s["seq"], line] = s["q"].float()
    x = q.view(n, s["max_q"] * h, dc + R) @ rows.transpose(1, 2) * (128 + R) ** -0.5
    x = x.view(n, s["max_q"], h, -1).masked_fill_(~see[:, :, None], -math.inf)
    x = (x - x.amax(-1, keepdim=True)).exp_()
    x /= x.sum(-1, keepdim=True)
    o = x.view(n, s["max_q"] * h, -1) @ rows[..., :dc]
    return o.view(n, s["max_q"], h, dc)[s["seq"], line].bfloat16()


def _plain_expanded(s):
    outs, begin, kv_begin = [], 0, 0
    for c, kv in zip(s["counts"], s["kvs"]):
        q = s["q"][begin:begin + c].float().transpose(0, 1)
        keys = slice(kv_begin, kv_begin + kv)
        k, v = s["k"][keys].float().permute(1, 2, 0), s["v"][keys].float().transpose(0, 1)
        x = q[..., : s["nope"]] @ k
        x += q[..., s["nope"]:] @ s["k_rope"][keys].float().T
        x *= (s["nope"] + R) ** -0.5
        see = torch.arange(kv, device="cuda") <= torch.arange(kv - c, kv, device="cuda")[:, None]
        x.masked_fill_(~see, -math.inf)
        x = x.sub_(x.amax(-1, keepdim=True)).exp_()
        outs.append(((x @ v) / x.sum(-1, keepdim=True)).transpose(0, 1).bfloat16())
        begin, kv_begin = begin + c, kv_begin + kv
    return torch.cat(outs)


def _plan(s):
    """What a program sets up once: the layer's geometry, the cache's handle, scratch memory."""
    import gated_deltanet_linear_mixer_gb300 as gdn
    if s["op"] == "copy":
        d = gdn.LatentDims(16, s["dc"], page_size=s["page"])
        return [gdn.LatentCache(d, p) for p in s["pools"]]
    if s["op"] == "expanded":
        return gdn.LatentDims(s["heads"], nope_dim=s["nope"], v_dim=s["vd"])
    d = gdn.LatentDims(s.get("heads", 1), s["dc"], page_size=s["page"], rope_style=s.get("style", "half"))
    if s["op"] == "latent":
        size = gdn.latent_attention_workspace_size(d, s["cu"])
        s["scratch"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return d, gdn.LatentCache(d, s["rows"])


def _own(s):
    import gated_deltanet_linear_mixer_gb300 as gdn
    if "plan" not in s:
        s["plan"] = _plan(s)
    if s["op"] == "copy":
        gdn.copy_pages(s["plan"], s["src"], s["dst"])
        return s["pools"]
    if s["op"] == "expanded":
        return gdn.expanded_attention(s["plan"], s["cu"], s["cu_kv"], s["q"], s["k"], s["k_rope"], s["v"])
    d, cache = s["plan"]
    if s["op"] == "latent":
        return gdn.latent_attention(d, cache, s["cu"], s["kv_lens"], s["table"], s["q"],
                                    workspace=s["scratch"])
    if s["op"] == "read":
        return gdn.latent_read(d, cache, s["cu"], s["starts"], s["table"])
    packed = torch.empty_like(s["c"])
    q = gdn.latent_append(d, cache, s["cu"], s["kv_lens"], s["table"], s["c"], norm_w=s["w"],
                          q_rope=s["q"][..., 128:], rope=s["table_rope"], rows_out=packed)
    return {"q": q, "packed": packed, "rows": s["rows"]}


def run(state):
    if own:
        return _own(state)
    if state["op"] == "copy":
        src, dst = _ints(state["src"], torch.int64), _ints(state["dst"], torch.int64)
        for pool in state["pools"]:
            pool[dst] = pool[src]
        return state["pools"]
    if state["op"] == "read":
        page = state["table"][state["seq"], state["pos"] // state["page"]].long()
        return state["rows"][page, state["pos"] % state["page"]]
    return {"latent": _plain_latent, "expanded": _plain_expanded, "append": _plain_append}[state["op"]](state)


# ------------------------------------------------------------------ 64 bits
def _line(s, i, length):
    """Sequence i's first `length` cached rows, one page after the other."""
    pages = s["table"][i, : -(-length // s["page"])].long()
    return s["rows"][pages].flatten(0, 1)[:length].double()


def _attend(q, k, v, scale):
    """Causal attention of the last len(q) positions; q [c, d], k [kv, d], v [kv, e]."""
    c, kv = len(q), len(k)
    late = torch.ones(c, kv, dtype=torch.bool, device="cuda").triu(kv - c + 1)
    return torch.softmax((torch.mm(q, k.T) * scale).masked_fill(late, -math.inf), -1) @ v


def _exact_latent(s, counts, kvs):
    outs, begin, h = [], 0, s["heads"]
    for i, (c, kv) in enumerate(zip(counts, kvs)):
        rows = _line(s, i, kv)
        q = s["q"][begin:begin + c].double()
        begin += c
        step = max(1, 200_000_000 // (c * kv))
        late = torch.ones(c, kv, dtype=torch.bool, device="cuda").triu(kv - c + 1)
        parts = []
        for a in range(0, h, step):
            x = torch.einsum("qhd,kd->hqk", q[:, a:a + step], rows) / math.sqrt(128 + R)
            w = torch.softmax(x.masked_fill(late, -math.inf), -1)
            parts.append(torch.einsum("hqk,kd->qhd", w, rows[:, : s["dc"]]))
        outs.append(torch.cat(parts, 1))
    return torch.cat(outs)


def _exact_expanded(s, counts, kvs):
    outs, a, b = [], 0, 0
    for c, kv in zip(counts, kvs):
        q, shared = s["q"][a:a + c].double(), s["k_rope"][b:b + kv].double()
        heads = []
        for h in range(s["heads"]):
            k = torch.cat([s["k"][b:b + kv, h].double(), shared], 1)
            heads.append(_attend(q[:, h], k, s["v"][b:b + kv, h].double(), 1 / math.sqrt(s["nope"] + R)))
        outs.append(torch.stack(heads, 1))
        a, b = a + c, b + kv
    return torch.cat(outs)


def _turn64(s, x):
    if s["table_rope"] is None:
        return x
    z = torch.complex(*s["table_rope"][s["pos"]].double().chunk(2, -1))[:, None]
    if s["style"] == "half":
        y = torch.complex(*(p.contiguous() for p in x.chunk(2, -1))) * z
        return torch.cat([y.real, y.imag], -1)
    y = torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous()) * z
    return torch.view_as_real(y).flatten(-2)


def _exact_append(s):
    c, k = s["c"].double().split([s["dc"], R], -1)
    if s["norm"]:
        c = c / torch.sqrt(c.square().sum(-1, keepdim=True) / s["dc"] + 1e-6) * s["w"].double()
    packed = torch.cat([c, _turn64(s, k[:, None])[:, 0]], -1)
    rows = s["rows"].double().flatten(0, 1)
    at = s["table"][s["seq"], torch.div(s["pos"], s["page"], rounding_mode="floor")].long() * s["page"]
    rows.index_copy_(0, at + torch.remainder(s["pos"], s["page"]), packed)
    return {"q": _turn64(s, s["q"][..., 128:].double()), "packed": packed, "rows": rows.view(s["rows"].shape)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "copy":
        outs = []
        for pool in s["pools"]:
            full = pool.double()
            for a, b in zip(s["src"], s["dst"]):
                full[b].copy_(pool[a])
            outs.append(full)
        return outs
    counts, kvs = _lengths(case)
    if case["op"] == "latent":
        return _exact_latent(s, counts, kvs)
    if case["op"] == "expanded":
        return _exact_expanded(s, counts, kvs)
    if case["op"] == "append":
        return _exact_append(s)
    return torch.cat([_line(s, i, counts[i]) for i in range(case["n"])])
