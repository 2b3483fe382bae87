"""Measured cases of the attention-cache operators and of draft verification.

Four operators of one step of a hybrid stack (recurrent mixers interleaved with
full attention): appending rotated keys and values to a paged 8-bit cache,
causal attention over that cache, reading cached values back, and deciding
which drafted tokens stand.  `run` computes them in their plain form (elementary
torch operations in 32 bits), or, where `own` is true, through this package's
entry points.

The cache: codes k, v [pages, kv heads, page, head dim] (int8 or e4m3), one f32
scale per page and head; block_table [n, pages per sequence]; kv_lens counts a
call's own tokens, so sequence i's q_i tokens sit at kv_lens[i] - q_i onwards.
"""
import math
import random

import torch

own = False

QMAX = {"int8": 127.0, "e4m3": 448.0}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
ACT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _attn(name, n, q, ragged, ctx_lo, ctx_hi, hq, hkv, d, page, act, fmt, window=0, lens=1):
    return dict(name=name, op="attention", n=n, q=q, ragged=ragged, ctx_lo=ctx_lo, ctx_hi=ctx_hi,
                hq=hq, hkv=hkv, d=d, page=page, act=act, fmt=fmt, window=window, lens=lens)


def _append(name, n, q, ragged, ctx_lo, ctx_hi, hq, hkv, d, page, act, fmt, rope, style, packed,
            lens=1):
    return dict(name=name, op="append", n=n, q=q, ragged=ragged, ctx_lo=ctx_lo, ctx_hi=ctx_hi,
                hq=hq, hkv=hkv, d=d, page=page, act=act, fmt=fmt, rope=rope, style=style,
                packed=packed, lens=lens)


def _accept(name, n, t, vocab, form, dtype, short, greedy):
    return dict(name=name, op="accept", n=n, t=t, vocab=vocab, form=form, dtype=dtype, short=short,
                greedy=greedy)


def listed():
    return [
        # one user's chat turn: the latency of a single token's attention
        _attn("attention_1x1_ctx1000", 1, 1, False, 1000, 1000, 16, 2, 256, 64, "bf16", "int8"),
        # a long document open in one session: few rows, a long axis to split
        _attn("attention_1x1_ctx131000", 1, 1, False, 131000, 131000, 16, 2, 256, 64, "bf16",
              "int8"),
        # the decode batch of a server: 256 ragged contexts
        _attn("attention_256x1", 256, 1, False, 127, 8191, 16, 2, 256, 64, "bf16", "int8", lens=2),
        # speculative verify: four drafts of each of 64 sequences, e4m3, small pages
        _attn("attention_64x4_e4m3", 64, 4, False, 500, 6000, 32, 8, 128, 16, "bf16", "e4m3",
              lens=3),
        # a prompt of 4096 tokens from an empty cache
        _attn("attention_prompt_4096", 1, 4096, False, 0, 0, 16, 2, 256, 64, "bf16", "int8"),
        # ragged prompt pieces behind cached prefixes, sliding window
        _attn("attention_16_prompts_window", 16, 1100, True, 0, 3000, 32, 8, 128, 32, "bf16",
              "e4m3", window=2048, lens=4),
        # the decode batch's append: one token each, pages partly filled
        _append("append_256x1", 256, 1, False, 127, 8191, 16, 2, 256, 64, "bf16", "int8", 64,
                "half", True, lens=2),
        # sixteen ragged prompts appended behind cached prefixes
        _append("append_16_prompts_e4m3", 16, 1100, True, 0, 3000, 32, 8, 128, 32, "bf16", "e4m3",
                128, "interleaved", False, lens=4),
        # a cached prefix taken out of the pages: four sequences
        dict(name="read_4x4000", op="read", n=4, rows_lo=3500, rows_hi=4500, hkv=8, d=128, page=16,
             fmt="e4m3", act="bf16", lens=5),
        # one short sequence's values, for inspection
        dict(name="read_1x300", op="read", n=1, rows_lo=300, rows_hi=300, hkv=2, d=256, page=64,
             fmt="int8", act="f32", lens=6),
        # four drafts of each of 64 sequences against given distributions
        _accept("accept_64x4_probs", 64, 4, 131072, "probs", "f32", True, False),
        # the same from the model's bf16 logits, odd vocabulary, some sequences greedy
        _accept("accept_48x3_logits", 48, 3, 32003, "logits", "bf16", False, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "append", "read", "accept",
                     "accept"])
    fmt = rng.choice(["int8", "e4m3"])
    page = rng.choice([16, 32, 64, 128])
    lens = rng.randrange(1 << 20)
    if op == "accept":
        form = rng.choice(["probs", "logits"])
        vocab = _log_int(rng, 1000, 131072)
        t = rng.randint(1, 8)
        n = _log_int(rng, 1, max(1, min(256, 32_000_000 // (vocab * (2 * t + 2)))))
        return dict(op=op, n=n, t=t, vocab=vocab, form=form,
                    dtype="f32" if form == "probs" else rng.choice(["bf16", "f32"]),
                    short=rng.random() < 0.5, greedy=form == "logits" and rng.random() < 0.5)
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8]) if d < 256 else rng.choice([1, 2, 4])
    if op == "read":
        hi = _log_int(rng, 1, 8000)
        n = _log_int(rng, 1, max(1, min(64, 16000 // hi)))
        return dict(op=op, n=n, rows_lo=max(1, hi // 2), rows_hi=hi, hkv=hkv, d=d, page=page, fmt=fmt,
                    act=rng.choice(["bf16", "f32"]), lens=lens)
    hq = hkv * rng.choice([1, 3, 4, 8])
    act = rng.choice(["bf16", "bf16", "bf16", "f32"])
    kind = rng.choice(["decode", "verify", "prompt"])
    if kind == "prompt":
        q = _log_int(rng, 17, 2000)
        n = _log_int(rng, 1, max(1, 4000 // q))
        ctx = rng.choice([0, _log_int(rng, 1, 2000)])
    else:
        q = 1 if kind == "decode" else rng.randint(2, 16)
        ctx = _log_int(rng, 1, 32000)
        n = _log_int(rng, 1, max(1, min(256, 400_000 // ctx)))
    base = dict(op=op, n=n, q=q, ragged=kind != "decode" and rng.random() < 0.5, ctx_lo=ctx // 2,
                ctx_hi=ctx, hq=hq, hkv=hkv, d=d, page=page, act=act, fmt=fmt, lens=lens)
    if op == "attention":
        base["window"] = rng.choice([0, 0, _log_int(rng, 16, 4096)])
    else:
        base["rope"] = rng.choice([d, d // 2, d // 4, 0])
        base["style"] = rng.choice(["half", "interleaved"])
        base["packed"] = rng.random() < 0.5
    return base


def _lengths(case):
    """Host lists of new tokens and of lengths after them (read: rows and lengths)."""
    r = random.Random(case["lens"])
    if case["op"] == "read":
        rows = [r.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["n"])]
        return rows, [k + r.randint(0, 40) for k in rows]
    qs = [r.randint(1, case["q"]) if case["ragged"] else case["q"] for _ in range(case["n"])]
    return qs, [q + r.randint(case["ctx_lo"], case["ctx_hi"]) for q in qs]


def _visible(q, kv, window):
    """Key and query pairs that q queries ending at kv see."""
    return sum(min(p + 1, window) if window else p + 1 for p in range(kv - q, kv))


def work(case):
    if case["op"] == "accept":
        n, t, v = case["n"], case["t"], case["vocab"]
        if case["form"] == "probs":  # per sequence: two numbers a draft, one row each of p, q, e
            return {"bytes": n * (12 * v + 16 * t), "flops": 3 * n * v}
        # rows are read up to the first draft that falls; about three in four drafts stand
        rows = sum(0.75 ** i for i in range(t)) * 2 + 0.75 ** t
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * v * (rows * e + 4), "flops": n * v * (4 * rows + 4)}
    qs, kvs = _lengths(case)
    h, d = case["hkv"], case["d"]
    e = 2 if case["act"] == "bf16" else 4
    if case["op"] == "read":
        return {"bytes": 2 * sum(qs) * h * d * (1 + e), "flops": 2 * sum(qs) * h * d}
    if case["op"] == "append":
        t = sum(qs)
        back = sum(kv - (kv - q) // case["page"] * case["page"] for q, kv in zip(qs, kvs))
        return {"bytes": 2 * t * h * d * (e + 1) + 2 * t * case["hq"] * d * e + 2 * back * h * d * 5,
                "flops": 12 * t * (h + case["hq"]) * d}
    w = case["window"]
    keys = sum(min(kv, w + q - 1) if w else kv for q, kv in zip(qs, kvs))
    pairs = sum(_visible(q, kv, w) for q, kv in zip(qs, kvs))
    return {"bytes": 2 * keys * h * d + 2 * sum(qs) * case["hq"] * d * e,
            "flops": 4 * pairs * case["hq"] * d}


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


def _cache(case, kvs, g, s):
    """A cache in use: pages in no order, codes and scales as quantised activations have them."""
    per = -(-max(kvs) // case["page"])
    pages = sum(-(-kv // case["page"]) for kv in kvs) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(kvs), per, dtype=torch.int32, device="cuda")
    need = [-(-kv // case["page"]) for kv in kvs]
    seq, at = _rows([0] * len(kvs), need)
    table[seq, at] = order[: sum(need)]
    shape = (pages, case["hkv"], case["page"], case["d"])

    def codes():
        x = torch.randn(shape, generator=g, device="cuda").mul_(QMAX[case["fmt"]] / 4)
        x.clamp_(-QMAX[case["fmt"]], QMAX[case["fmt"]])
        return x.round_().to(torch.int8) if case["fmt"] == "int8" else x.to(CODE["e4m3"])

    def scales(centre):
        x = torch.randn(shape[:2], generator=g, device="cuda").mul_(0.2).exp_()
        return x.mul_(4 * centre / QMAX[case["fmt"]])

    s.update(table=table, k=codes(), v=codes(), k_scale=scales(1.0), v_scale=scales(0.5),
             kv_lens=_ints(kvs))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "accept":
        n, t, v = case["n"], case["t"], case["vocab"]
        target = torch.randn(n, t + 1, v, generator=g, device="cuda").mul_(3.0)
        draft = target[:, :t] + torch.randn(n, t, v, generator=g, device="cuda").mul_(0.4)
        temp = torch.full((n,), 0.8, device="cuda")
        if case["greedy"]:
            temp[::3] = 0.0
        scale = 1.0 if case["form"] == "probs" else 1.0 / 0.8
        race = torch.empty(n, t, v, device="cuda").exponential_(generator=g)
        tokens = (torch.softmax(draft * scale, -1) / race).argmax(-1).to(torch.int32)
        if case["short"]:  # every fourth sequence has one draft fewer
            tokens[::4, t - 1] = -1
        del race
        if case["form"] == "probs":
            target, draft = torch.softmax(target, -1), torch.softmax(draft, -1)
        else:
            target, draft = target.to(ACT[case["dtype"]]), draft.to(ACT[case["dtype"]])
        s.update(target=target, draft=draft, drafts=tokens, temp=temp,
                 u=torch.rand(n, t, generator=g, device="cuda"),
                 e=torch.empty(n, v, device="cuda").exponential_(generator=g))
        return s
    counts, kvs = _lengths(case)
    _cache(case, kvs, g, s)
    s["cu"] = _cu(counts)
    t, h, hq, d = sum(counts), case["hkv"], case.get("hq", 0), case["d"]
    s["max_kv"] = max(kvs)
    if case["op"] == "read":
        s["starts"] = _ints([0] * len(counts))
        s["seq"], s["pos"] = _rows([0] * len(counts), counts)
        return s
    s["seq"], s["pos"] = _rows([kv - q for q, kv in zip(counts, kvs)], counts)
    act = ACT[case["act"]]
    if case["op"] == "attention":
        s["max_q"] = max(counts)
        s["q_lens"] = _ints(counts, torch.int64)
        s["new"] = torch.randn(t, hq, d, generator=g, device="cuda").to(act)
        return s
    if case["packed"]:  # one projection's output: q | k | v of a token side by side
        qkv = torch.randn(t, hq + 2 * h, d, generator=g, device="cuda").to(act)
        s["new"], s["nk"], s["nv"] = qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:]
    else:
        s["new"] = torch.randn(t, hq, d, generator=g, device="cuda").to(act)
        s["nk"] = torch.randn(t, h, d, generator=g, device="cuda").to(act)
        s["nv"] = torch.randn(t, h, d, generator=g, device="cuda").to(act)
    if case["rope"]:
        inv = 10000.0 ** (-torch.arange(0, case["rope"], 2, device="cuda") / case["rope"])
        ang = torch.arange(max(kvs), device="cuda")[:, None] * inv[None]
        s["rope_table"] = torch.cat([ang.cos(), ang.sin()], -1).contiguous()
    # the pages a call writes to: of each, the sequence, the place and the tokens it keeps
    first = [(kv - q) // case["page"] for q, kv in zip(counts, kvs)]
    span = [(kv - 1) // case["page"] - f + 1 for f, kv in zip(first, kvs)]
    s["touch_seq"], s["touch_at"] = _rows(first, span)
    begin = _ints([kv - q for q, kv in zip(counts, kvs)], torch.int64)
    s["kept"] = (begin[s["touch_seq"]] - s["touch_at"] * case["page"]).clamp(0, case["page"])
    starts = [f * case["page"] for f in first]
    back = [kv - a for kv, a in zip(kvs, starts)]
    s["starts"], s["back_cu"] = _ints(starts), _cu(back)
    s["back_seq"], s["back_pos"] = _rows(starts, back)
    return s


# -------------------------------------------------------------- plain forms
def _values(s, name, seq, pos):
    page = s["table"][seq, pos // s["page"]].long()
    scale = s[name + "_scale"][page]
    return s[name][page, :, pos % s["page"]].float() * scale[..., None]


def _rotate(s, x):
    x = x.float()
    r = s["rope"]
    if not r:
        return x
    row = s["rope_table"][s["pos"]][:, None]
    c, sn = row[..., : r // 2], row[..., r // 2:]
    out = x.clone()
    if s["style"] == "half":
        a, b = x[..., : r // 2], x[..., r // 2: r]
        out[..., : r // 2], out[..., r // 2: r] = a * c - b * sn, b * c + a * sn
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        out[..., 0:r:2], out[..., 1:r:2] = a * c - b * sn, b * c + a * sn
    return out


def _code(s, x):
    top = QMAX[s["fmt"]]
    if s["fmt"] == "int8":
        return x.round().clamp(-top, top).to(torch.int8)
    return x.clamp(-top, top).to(CODE["e4m3"])


def _plain_store(s, name, x):
    b = s["page"]
    page = s["table"][s["seq"], s["pos"] // b].long()
    touched = s["table"][s["touch_seq"], s["touch_at"]].long()
    scale = s[name + "_scale"]
    most = torch.zeros_like(scale)
    most.scatter_reduce_(0, page[:, None].expand(-1, scale.shape[1]), x.abs().amax(-1), "amax")
    old = torch.where(s["kept"][:, None] > 0, scale[touched], 0.0)
    new = torch.maximum(old, most[touched] / QMAX[s["fmt"]])
    ratio = torch.where(new > 0, old / new, 0.0)
    codes = s[name][touched]
    again = _code(s, codes.float() * ratio[..., None, None])
    keep = torch.arange(b, device="cuda")[None] < s["kept"][:, None]
    raw = torch.where(keep[:, None, :, None], again.view(torch.int8), codes.view(torch.int8))
    s[name].view(torch.int8)[touched] = raw
    scale[touched] = new
    mine = scale[page][..., None]
    y = torch.where(mine > 0, x / mine, 0.0)
    s[name].view(torch.int8)[page, :, s["pos"] % b] = _code(s, y).view(torch.int8)


def _plain_append(s):
    q = _rotate(s, s["new"]).to(s["new"].dtype)
    _plain_store(s, "k", _rotate(s, s["nk"]))
    _plain_store(s, "v", s["nv"].float())
    return {"q": q, "k": _values(s, "k", s["back_seq"], s["back_pos"]),
            "v": _values(s, "v", s["back_seq"], s["back_pos"])}


def _plain_attention(s):
    n, h, d, b = s["n"], s["hkv"], s["d"], s["page"]
    g = s["hq"] // h
    at = torch.arange(s["max_kv"], device="cuda")
    page = s["table"][:, at // b].long()
    k = s["k"][page, :, at % b].float() * s["k_scale"][page][..., None]
    v = s["v"][page, :, at % b].float() * s["v_scale"][page][..., None]
    line = s["pos"] - (s["kv_lens"].long() - s["q_lens"])[s["seq"]]
    q = torch.zeros(n, s["max_q"], s["hq"], d, device="cuda")
    q[s["seq"], line] = s["new"].float()
    q = q.view(n, s["max_q"], h, g, d).permute(0, 2, 3, 1, 4).reshape(n, h, g * s["max_q"], d)
    x = q @ k.permute(0, 2, 3, 1) * d ** -0.5
    place = (s["kv_lens"].long() - s["q_lens"])[:, None] + torch.arange(s["max_q"], device="cuda")
    see = at[None, None] <= place[..., None]
    if s["window"]:
        see &= at[None, None] > place[..., None] - s["window"]
    x = x.view(n, h, g, s["max_q"], -1).masked_fill_(~see[:, None, None], -math.inf)
    x = (x - x.amax(-1, keepdim=True)).exp_()
    x /= x.sum(-1, keepdim=True)
    o = x.view(n, h, g * s["max_q"], -1) @ v.permute(0, 2, 1, 3)
    o = o.view(n, h, g, s["max_q"], d).permute(0, 3, 1, 2, 4).reshape(n, s["max_q"], s["hq"], d)
    return o[s["seq"], line].to(s["new"].dtype)


def _plain_accept(s):
    n, t, v = s["n"], s["t"], s["vocab"]
    iota = torch.arange(v, device="cuda")
    p, q = s["target"].float(), s["draft"].float()
    if s["form"] == "logits":
        temp = s["temp"][:, None, None]
        top = torch.where(p == p.amax(-1, keepdim=True), iota, v).amin(-1, keepdim=True)
        over = torch.where(temp > 0, temp, 1.0)
        p, q = p / over, q / over
        p = (p - p.amax(-1, keepdim=True)).exp()
        q = (q - q.amax(-1, keepdim=True)).exp()
        p, q = p / p.sum(-1, keepdim=True), q / q.sum(-1, keepdim=True)
        p = torch.where(temp > 0, p, (iota == top).float())
    x = s["drafts"].long()
    there = (x >= 0) & (x < v)
    at = x.clamp(0, v - 1)[..., None]
    stands = there & (s["u"] * q.gather(-1, at)[..., 0] < p[:, :t].gather(-1, at)[..., 0])
    accepted = stands.long().cumprod(1).sum(1)
    line = torch.arange(n, device="cuda")
    last = p[line, accepted]
    low = accepted.clamp(max=t - 1)
    r = (last - q[line, low]).clamp(min=0)
    r = torch.where(((accepted < t) & there[line, low])[:, None], r, last)
    r = torch.where((r > 0).any(-1, keepdim=True), r, last)
    score = torch.where(r > 0, r / s["e"], -1.0)
    best = score.amax(-1, keepdim=True)
    token = torch.where((score == best) & (best > 0), iota, v).amin(-1)
    token = torch.where(token < v, token, -1)
    place = torch.arange(t + 1, device="cuda")[None]
    more = torch.cat([x, x[:, :1]], 1)
    tokens = torch.where(place < accepted[:, None], more, -1)
    tokens = torch.where(place == accepted[:, None], token[:, None], tokens)
    return {"accepted": accepted.to(torch.int32), "tokens": tokens.to(torch.int32)}


# ------------------------------------------------------------ the framework
def _plan(s):
    """What a program sets up once: the layer's geometry, the cache's handle, scratch memory."""
    import gated_deltanet_linear_mixer_gb300 as gdn
    d = gdn.KVDims(s.get("hq", s["hkv"]), s["hkv"], s["d"], page_size=s["page"],
                   dtype=ACT[s["act"]], cache=s["fmt"], rope_dim=s.get("rope", 0),
                   rope_style=s.get("style", "half"), window=s.get("window", 0))
    s["plan"] = d, gdn.KVCache(d, s["k"], s["v"], s["k_scale"], s["v_scale"])
    if s["op"] == "attention":
        size = gdn.kv_attention_workspace_size(d, s["cu"], s["max_kv"])
        s["scratch"] = torch.empty(size, dtype=torch.uint8, device="cuda")


def _own(s):
    import gated_deltanet_linear_mixer_gb300 as gdn
    if s["op"] == "accept":
        accepted, tokens = gdn.accept_drafts(
            s["drafts"], s["target"], s["draft"], s["u"], s["e"], form=s["form"],
            temperature=s["temp"] if s["form"] == "logits" else None)
        return {"accepted": accepted, "tokens": tokens}
    if "plan" not in s:
        _plan(s)
    d, cache = s["plan"]
    if s["op"] == "attention":
        return gdn.kv_attention(d, cache, s["cu"], s["kv_lens"], s["table"], s["new"],
                                max_kv_len=s["max_kv"], workspace=s["scratch"])
    if s["op"] == "read":
        k, v = gdn.kv_read(d, cache, s["cu"], s["starts"], s["table"])
        return {"k": k, "v": v}
    q = gdn.kv_append(d, cache, s["cu"], s["kv_lens"], s["table"], s["nk"], s["nv"], q=s["new"],
                      rope=s.get("rope_table"))
    k, v = gdn.kv_read(d, cache, s["back_cu"], s["starts"], s["table"], dtype=torch.float32)
    return {"q": q, "k": k, "v": v}


def run(state):
    if own:
        return _own(state)
    if state["op"] == "accept":
        return _plain_accept(state)
    if state["op"] == "attention":
        return _plain_attention(state)
    if state["op"] == "append":
        return _plain_append(state)
    act = ACT[state["act"]]
    return {"k": _values(state, "k", state["seq"], state["pos"]).to(act),
            "v": _values(state, "v", state["seq"], state["pos"]).to(act)}


# ------------------------------------------------------------------ 64 bits
def _line(s, name, i, length):
    """Sequence i's first `length` cached values, one page after the other."""
    pages = s["table"][i, : -(-length // s["page"])].long()
    x = s[name][pages].double() * s[name + "_scale"][pages].double()[:, :, None, None]
    return x.transpose(1, 2).reshape(-1, s["hkv"], s["d"])[:length]


def _exact_attention(s, counts, kvs):
    outs, begin = [], 0
    g = s["hq"] // s["hkv"]
    for i, (c, kv) in enumerate(zip(counts, kvs)):
        k, v = _line(s, "k", i, kv), _line(s, "v", i, kv)
        q = s["new"][begin:begin + c].double()
        begin += c
        gap = torch.arange(kv - c, kv, device="cuda")[:, None] - torch.arange(kv, device="cuda")
        hide = (gap < 0) | (gap >= s["window"]) if s["window"] else gap < 0
        heads = []
        for h in range(s["hkv"]):
            x = torch.einsum("qgd,kd->gqk", q[:, h * g:(h + 1) * g], k[:, h]) / math.sqrt(s["d"])
            w = torch.softmax(x.masked_fill(hide, -math.inf), -1)
            heads.append(torch.einsum("gqk,kd->qgd", w, v[:, h]))
        outs.append(torch.cat(heads, 1))
    return torch.cat(outs)


def _round8(x, fmt):
    if fmt == "int8":
        return torch.round(x).clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _turn(x, table, style, r):
    if not r:
        return x
    z = torch.complex(*table.double().chunk(2, -1))[:, None]
    head, rest = x[..., :r], x[..., r:]
    if style == "half":
        y = torch.complex(*head.chunk(2, -1)) * z
        return torch.cat([y.real, y.imag, rest], -1)
    y = torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous()) * z
    return torch.cat([torch.view_as_real(y).flatten(-2), rest], -1)


def _exact_append(s, counts, kvs):
    got = {"q": [], "k": [], "v": []}
    begin, b, top = 0, s["page"], QMAX[s["fmt"]]
    for i, (c, kv) in enumerate(zip(counts, kvs)):
        a, z = kv - c, begin + c
        table = s["rope_table"][a:kv] if s["rope"] else None
        got["q"].append(_turn(s["new"][begin:z].double(), table, s["style"], s["rope"]))
        first = a // b * b
        for name, x in (("k", s["nk"]), ("v", s["nv"])):
            x = x[begin:z].double()
            x = _turn(x, table, s["style"], s["rope"]) if name == "k" else x
            old = _line(s, name, i, a)[first:]
            y = torch.cat([old, x])
            fill = -len(y) % b
            y = torch.cat([y, y.new_zeros(fill, *y.shape[1:])]).unflatten(0, (-1, b))
            new = torch.zeros_like(y)
            new[:, :] = y
            new[0, : len(old)] = 0
            scale = new.abs().amax((1, 3)) / top
            if len(old):
                before = s[name + "_scale"][s["table"][i, first // b].long()].double()
                scale[0] = torch.maximum(scale[0], before)
            scale = scale[:, None, :, None]
            done = _round8(torch.where(scale > 0, y / scale, 0.0), s["fmt"]) * scale
            got[name].append(done.flatten(0, 1)[: kv - first])
        begin = z
    return {k: torch.cat(v) for k, v in got.items()}


def _exact_accept(s):
    accepted, tokens = [], []
    t, v = s["t"], s["vocab"]
    for i in range(s["n"]):
        p, q = s["target"][i].double(), s["draft"][i].double()
        temp = float(s["temp"][i])
        if s["form"] == "logits":
            if temp > 0:
                p, q = torch.softmax(p / temp, -1), torch.softmax(q / temp, -1)
            else:
                first = [int((row == row.max()).nonzero()[0]) for row in p]
                p = torch.zeros_like(p)
                p[torch.arange(t + 1), first] = 1.0
                q = torch.softmax(q, -1)
        x, u = s["drafts"][i].tolist(), s["u"][i].double().tolist()
        k = 0
        while k < t and 0 <= x[k] < v and u[k] * float(q[k, x[k]]) < float(p[k, x[k]]):
            k += 1
        r = p[k]
        if k < t and 0 <= x[k] < v:
            less = (p[k] - q[k]).clamp(min=0)
            r = less if bool((less > 0).any()) else r
        score = r / s["e"][i].double()
        best = score.max()
        token = int((score == best).nonzero()[0]) if float(best) > 0 else -1
        accepted.append(k)
        tokens.append(x[:k] + [token] + [-1] * (t - k))
    return {"accepted": _ints(accepted), "tokens": _ints(tokens)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "accept":
        return _exact_accept(s)
    counts, kvs = _lengths(case)
    if case["op"] == "attention":
        return _exact_attention(s, counts, kvs)
    if case["op"] == "append":
        return _exact_append(s, counts, kvs)
    ends = list(range(case["n"]))
    return {name: torch.cat([_line(s, name, i, counts[i]) for i in ends]) for name in ("k", "v")}
