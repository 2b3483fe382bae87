"""Verification of drafted tokens against a plain 64-bit implementation.

Decisions are whole numbers: they must be equal wherever the 64-bit margins
(u q against p; the race's best against its second) exceed 1e-4 relative, well
above what fp32 exponentials and sums can move them (about 1e-5 for logits up
to 60 in magnitude), and the inputs are drawn so that closer calls are rare.
"""
import math

import pytest
import torch

import gated_deltanet_linear_mixer_gb300 as gdn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_deltanet_linear_mixer_gb300 import _build
    _build.build()
    gdn.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _inputs(n, t, vocab, form, dtype, seed, temps=(1.0,), spread=3.0, noise_between=0.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    target = torch.randn(n, t + 1, vocab, generator=g, device="cuda") * spread
    draft = target[:, :t] + torch.randn(n, t, vocab, generator=g, device="cuda") * noise_between
    race = torch.empty(n, t, vocab, device="cuda").exponential_(generator=g)
    x = (torch.softmax(draft, -1) / race).argmax(-1).to(torch.int32)
    if form == "probs":
        target, draft = torch.softmax(target, -1), torch.softmax(draft, -1)
    u = torch.rand(n, t, generator=g, device="cuda")
    e = torch.empty(n, vocab, device="cuda").exponential_(generator=g)
    temp = torch.tensor([temps[i % len(temps)] for i in range(n)], device="cuda") if form == "logits" else None
    return x.contiguous(), target.to(dtype), draft.to(dtype), u, e, temp


def _ref(x, target, draft, u, e, form, temp):
    """[(accepted, tokens, sure)] in 64 bits."""
    n, t = x.shape
    got = []
    for i in range(n):
        tau = 1.0 if temp is None else float(temp[i])

        def dist(row):
            row = row.double()
            if form == "probs":
                return row
            if tau == 0:
                p = torch.zeros_like(row)
                if row.max() > -math.inf:
                    p[int((row == row.max()).nonzero()[0])] = 1.0
                return p
            p = torch.softmax(row / tau, -1)
            return torch.nan_to_num(p, nan=0.0)

        k, sure = 0, True
        while k < t and 0 <= int(x[i, k]) < target.shape[2]:
            xi = int(x[i, k])
            p, q = float(dist(target[i, k])[xi]), 1.0
            if draft is not None:
                q = float(dist(draft[i, k])[xi])
            a = float(u[i, k]) * q
            sure &= abs(a - p) > 1e-4 * max(a, p) or tau == 0
            if tau == 0:
                if p != 1.0:
                    break
            elif not a < p:
                break
            k += 1
        p = dist(target[i, k])
        r = p
        if k < t and 0 <= int(x[i, k]) < target.shape[2] and tau != 0:
            if draft is None:
                q = torch.zeros_like(p)
                q[int(x[i, k])] = 1.0
            else:
                q = dist(draft[i, k])
            less = (p - q).clamp(min=0)
            r = less if bool((less > 0).any()) else p
        score = torch.where(r > 0, r / e[i].double(), 0.0)
        top = score.topk(min(2, len(score))).values
        if tau != 0 and len(top) > 1 and float(top[0]) > 0:
            # r = p - q of nearly equal p, q carries p's rounding: the winner's share counts
            w = int(score.argmax())
            sure &= float(top[1]) < float(top[0]) * (1 - 1e-4 * max(1.0, float(p[w] / r[w])))
        token = int((score == score.max()).nonzero()[0]) if float(score.max()) > 0 else -1
        got.append((k, x[i, :k].tolist() + [token] + [-1] * (t - k), sure))
    return got


def _check(x, target, draft, u, e, form, temp, least=0.9):
    accepted, tokens = gdn.accept_drafts(x, target, draft, u, e, form=form, temperature=temp)
    ref = _ref(x, target, draft, u, e, form, temp)
    assert sum(s for _, _, s in ref) >= int(least * len(ref))  # few calls too close to hold to
    for i, (k, want, sure) in enumerate(ref):
        if sure:
            assert (int(accepted[i]), tokens[i].tolist()) == (k, want), i
    return accepted, tokens


CASES = {
    "probs": (24, 4, 1000, "probs", F32, (1.0,)),
    "probs_odd_vocab": (7, 3, 32003, "probs", F32, (1.0,)),
    "logits_f32": (24, 4, 777, "logits", F32, (1.0, 0.7)),
    "logits_bf16": (16, 5, 5001, "logits", BF, (0.8, 0.0, 1.3)),
    "greedy_bf16": (16, 4, 2000, "logits", BF, (0.0,)),
    "one_draft_one_sequence": (1, 1, 50, "probs", F32, (1.0,)),
    "sixteen_drafts": (5, 16, 300, "logits", F32, (1.0,)),
    "vocab_1": (3, 2, 1, "logits", F32, (1.0,)),
    "vocab_2": (40, 2, 2, "probs", F32, (1.0,)),
    "large_vocab": (3, 2, 200001, "logits", BF, (1.0,)),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_matches_64_bits(name):
    n, t, vocab, form, dtype, temps = CASES[name]
    _check(*_args(_inputs(n, t, vocab, form, dtype, len(name), temps), form))


def _args(inp, form):
    x, target, draft, u, e, temp = inp
    return x, target, draft, u, e, form, temp


@pytest.mark.parametrize("form,dtype", [("probs", F32), ("logits", F32), ("logits", BF)])
def test_certain_drafts(form, dtype):
    x, target, _, u, e, temp = _inputs(20, 3, 400, form, dtype, 5, spread=1.0)
    x = target[:, :3].float().argmax(-1).to(torch.int32)
    _check(x, target, None, u, e, form, temp)


@pytest.mark.parametrize("form", ["probs", "logits"])
def test_no_drafts_draws_from_the_target(form):
    x, target, draft, u, e, temp = _inputs(9, 0, 500, form, F32, 6)
    accepted, tokens = _check(x, target, draft, u, e, form, temp)
    assert not accepted.any() and tokens.shape == (9, 1)


@pytest.mark.parametrize("form", ["probs", "logits"])
def test_drafts_that_end_early(form):
    """-1, and an index past the vocabulary, end a sequence's drafts: no residual is taken there."""
    x, target, draft, u, e, temp = _inputs(12, 4, 300, form, F32, 7, noise_between=0.01)
    x[::2, 2] = -1
    x[1::4, 1] = 300
    x[3, 0] = -1
    accepted, _ = _check(x, target, draft, u, e, form, temp)
    assert (accepted[::2] <= 2).all() and int(accepted[3]) == 0 and (accepted[1::4] <= 1).all()


def test_equal_distributions_accept_everything():
    x, target, _, u, e, _ = _inputs(30, 4, 200, "probs", F32, 8)
    draft = target[:, :4].contiguous()
    x = (draft / torch.empty_like(draft).exponential_()).argmax(-1).to(torch.int32)
    accepted, _ = gdn.accept_drafts(x, target, draft, u, e)
    assert (accepted == 4).all()


def test_masked_logits_and_empty_rows():
    """-inf and the type's lowest value in masked places; a row that leaves nothing gives -1."""
    for dtype in (F32, BF):
        x, target, draft, u, e, temp = _inputs(12, 3, 500, "logits", dtype, 9, temps=(1.0, 0.0))
        target[:, :, 100:400] = -math.inf
        target[::3, :, 400:450] = torch.finfo(dtype).min
        draft[:, :, 250:400] = -math.inf
        x[0, 0], x[1, 0] = 150, 300
        target[4, 1], target[5, 0], target[6, 3], target[7] = -math.inf, -math.inf, -math.inf, -math.inf
        accepted, tokens = _check(x, target, draft, u, e, "logits", temp, least=0.7)
        assert int(accepted[0]) == 0 and int(accepted[1]) == 0
        assert int(accepted[5]) == 0 and int(tokens[5, 0]) == -1 and int(tokens[7, 0]) == -1


def test_probabilities_of_zero():
    """A draft the target rules out never stands; p = q there falls back to the target."""
    p = torch.tensor([[[0.5, 0.5, 0.0, 0.0], [0.0, 0.0, 0.0, 0.0]], [[0.0, 1.0, 0.0, 0.0], [0.25, 0.25, 0.25, 0.25]],
                      [[0.5, 0.5, 0.0, 0.0], [1.0, 0.0, 0.0, 0.0]]], device="cuda")
    q = torch.tensor([[[0.0, 0.0, 1.0, 0.0]], [[0.0, 0.0, 0.0, 1.0]], [[0.5, 0.5, 0.0, 0.0]]], device="cuda")
    x = torch.tensor([[2], [1], [0]], dtype=torch.int32, device="cuda")
    u = torch.tensor([[0.0], [0.999], [1.0]], device="cuda")
    e = torch.tensor([[1.0, 0.5, 0.1, 0.1]] * 3, device="cuda")
    accepted, tokens = gdn.accept_drafts(x, p, q, u, e)
    assert accepted.tolist() == [0, 1, 0]
    assert tokens.tolist() == [[1, -1], [1, 2], [1, -1]]


def test_ties_take_the_lowest_index():
    n, vocab = 6, 5000
    logits = torch.zeros(n, 2, vocab, device="cuda", dtype=BF)
    for i in range(n):
        logits[i, :, [4321 - i, 17 * i + 3, 2500]] = 5.0
    x = torch.tensor([[17 * i + 3 if i % 2 else 2500] for i in range(n)], dtype=torch.int32, device="cuda")
    u = torch.full((n, 1), 0.5, device="cuda")
    e = torch.ones(n, vocab, device="cuda")
    for temp in (0.0, 1.0):
        accepted, tokens = gdn.accept_drafts(x, logits, None, u, e, form="logits",
                                             temperature=torch.full((n,), temp, device="cuda"))
        for i in range(n):
            if temp == 0.0:
                assert int(accepted[i]) == i % 2
                assert int(tokens[i, i % 2]) == 17 * i + 3
            else:
                assert int(accepted[i]) == 0 and int(tokens[i, 0]) == (2500 if i % 2 else 17 * i + 3)


@pytest.mark.parametrize("pad", [1, 8, 13])
def test_padded_rows(pad):
    """Row strides above the vocabulary (a padded output projection), odd ones among them."""
    for form, dtype in (("probs", F32), ("logits", BF)):
        x, target, draft, u, e, temp = _inputs(10, 3, 1001, form, dtype, 12)
        a = gdn.accept_drafts(x, target, draft, u, e, form=form, temperature=temp)

        def padded(v):
            w = torch.full((*v.shape[:-1], v.shape[-1] + pad), 99.0, dtype=v.dtype, device="cuda")
            w[..., : v.shape[-1]] = v
            return w[..., : v.shape[-1]]

        b = gdn.accept_drafts(x, padded(target), padded(draft), u, padded(e), form=form, temperature=temp)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("form", ["probs", "logits"])
def test_tokens_follow_the_target(form):
    """Whatever the draft, the first token is distributed as the target's: 40000 sequences, a
    vocabulary of 8, each frequency within 5 standard deviations."""
    n, vocab = 40000, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    tl = torch.randn(1, 2, vocab, generator=g, device="cuda").expand(n, 2, vocab).contiguous()
    dl = torch.randn(1, 1, vocab, generator=g, device="cuda").expand(n, 1, vocab).contiguous()
    p, q = torch.softmax(tl, -1), torch.softmax(dl, -1)
    x = (q / torch.empty_like(q).exponential_(generator=g)).argmax(-1).to(torch.int32)
    u = torch.rand(n, 1, generator=g, device="cuda")
    e = torch.empty(n, vocab, device="cuda").exponential_(generator=g)
    a, tokens = gdn.accept_drafts(x, p if form == "probs" else tl, q if form == "probs" else dl, u, e, form=form)
    share = torch.bincount(tokens[:, 0].long(), minlength=vocab).double() / n
    want = p[0, 0].double()
    assert ((share - want).abs() <= 5 * (want * (1 - want) / n).sqrt()).all()
    rate = float(torch.minimum(want, q[0, 0].double()).sum())
    assert abs(float(a.double().mean()) - rate) <= 5 * math.sqrt(rate * (1 - rate) / n)


def test_many_sequences_and_another_stream():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        inp = _inputs(700, 2, 60, "logits", F32, 14, temps=(1.0, 0.0, 0.5))
        x, target, draft, u, e, temp = inp
        accepted, tokens = gdn.accept_drafts(x, target, draft, u, e, form="logits", temperature=temp)
        ref = _ref(x[:60], target[:60], draft[:60], u[:60], e[:60], "logits", temp[:60])
        for i, (k, want, sure) in enumerate(ref):
            if sure:
                assert (int(accepted[i]), tokens[i].tolist()) == (k, want)


def test_offsets_past_2_31():
    """Rows that start beyond 2^31 elements."""
    n, t, vocab = 2400, 3, 250007
    if torch.cuda.get_device_properties(0).total_memory < 60 << 30:
        pytest.skip("needs 16 GB")
    target = torch.zeros(n, t + 1, vocab, dtype=BF, device="cuda")
    draft = torch.zeros(n, t, vocab, dtype=BF, device="cuda")
    x = torch.arange(n * t, device="cuda", dtype=torch.int32).view(n, t) % vocab
    target.scatter_(2, torch.cat([x, x[:, :1] + 1], 1).long()[..., None], 40.0)
    draft.scatter_(2, x.long()[..., None], 40.0)
    u = torch.full((n, t), 0.5, device="cuda")
    e = torch.ones(1, vocab, device="cuda").expand(n, vocab).contiguous()
    accepted, tokens = gdn.accept_drafts(x, target, draft, u, e, form="logits")
    assert (accepted == t).all()
    assert torch.equal(tokens, torch.cat([x, x[:, :1] + 1], 1))
    del target, draft, e
    torch.cuda.empty_cache()


def test_feeds_decode_commit():
    """accepted is what gdn.decode_commit takes: the states kept are those of the accepted tokens."""
    n, t, hv, dk, dv = 6, 4, 2, 32, 32
    d = gdn.Dims(2, hv, dk, dv, dtype=F32)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, target, draft, u, e, temp = _inputs(n, t, 100, "probs", F32, 15)
    accepted, _ = gdn.accept_drafts(x, target, draft, u, e)
    inter = torch.randn(n, t, hv, dk, dv, generator=g, device="cuda")
    state = torch.randn(n, hv, dk, dv, generator=g, device="cuda")
    want = [state[i].clone() if int(a) == 0 else inter[i, int(a) - 1].clone() for i, a in enumerate(accepted)]
    xin = torch.randn(n, t, d.conv_dim, generator=g, device="cuda")
    gdn.decode_commit(d, accepted, xin, inter, state)
    assert torch.equal(state, torch.stack(want))
