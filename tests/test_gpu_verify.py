"""Verification of drafted tokens on the GPU against the 64-bit oracle."""

import numpy as np
import pytest
import torch

import _verify_checks as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


COUNTS = [[1], [0], [4], [0, 3, 1, 0, 7, 2], [33, 0, 70], [2] * 40]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("vocab", [1, 2, 7, 129, 1000, 4099])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_drafts_with_distributions(g, counts, vocab, dtype):
    c = C.make(counts, vocab, dtype, seed=vocab + len(counts))
    C.settle(c)
    C.check(C.call(g, c), C.want(c))


@pytest.mark.parametrize("vocab", [2, 1000, 32003])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_drafts_without_distributions(g, vocab, dtype):
    c = C.make([0, 3, 1, 0, 7, 2], vocab, dtype, seed=5, drafted=False, temperature=0.7)
    C.settle(c, 0.7)
    C.check(C.call(g, c, 0.7), C.want(c, 0.7))


@pytest.mark.parametrize("vocab,dtype", [(32000, "f32"), (50021, "bf16"), (131072, "bf16"), (131073, "f32"),
                                         (300007, "f32"), (600011, "bf16")])
def test_long_rows(g, vocab, dtype):
    c = C.make([3, 0, 2], vocab, dtype, seed=3, ruled=0.05)
    C.settle(c)
    C.check(C.call(g, c), C.want(c))


@pytest.mark.parametrize("seqs", [120, 400])
def test_many_sequences(g, seqs):
    rng = np.random.default_rng(seqs)
    c = C.make(rng.integers(0, 5, seqs).tolist(), 500, "bf16", seed=9, blur=0.5)
    C.settle(c)
    C.check(C.call(g, c), C.want(c))


@pytest.mark.parametrize("vocab", [1, 5, 1000, 50021])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_greedy(g, vocab, dtype):
    c = C.make([0, 3, 1, 0, 7, 2], vocab, dtype, seed=8, drafted=False, spread=1.0)
    if vocab > 5:  # equal largest logits in every row: the first of them counts
        c["target"][:, [3, 4, vocab - 1]] = 9.0
        c["drafts"][:9] = 3
    C.check(C.call(g, c, mode="greedy"), C.want(c, greedy=True))


@pytest.mark.parametrize("target,draft", [("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("pads", [(0, 0), (1, 3), (8, 5), (13, 16)])
def test_strides_and_types(g, target, draft, pads):
    """Rows further apart than the vocabulary, target and draft at different alignments and of different types."""
    c = C.make([3, 2, 0, 5], 1001, target, seed=4, draft_dtype=draft)
    C.settle(c, 0.9, 1.1)
    expected = C.want(c, 0.9, draft_temperature=1.1)
    d = dict(c)
    for k, pad in zip(("target", "draft_logits"), pads):
        wide = torch.full((c[k].shape[0], c[k].shape[1] + pad + 2), float("nan"), dtype=c[k].dtype)
        wide[:, 1:1 + c[k].shape[1]] = c[k]
        d[k] = wide.cuda()[:, 1:1 + c[k].shape[1]]
    C.check(C.call(g, d, 0.9, draft_temperature=1.1), expected)


def test_borders_between_equal_tokens(g):
    """Equal logits: running sums are whole numbers times one weight, and u a whole number of shares; the border
    belongs to the token behind it."""
    vocab, rows = 1 << 17, 64
    target = torch.full((rows, vocab), -3.0e38)
    target[::2] = 1.25
    u = torch.arange(rows) * 2039 / vocab  # exact
    for dtype in (torch.float32, torch.bfloat16):
        accepted, tokens, logp = g.ar_verify_drafts(
            target.to(dtype).cuda(), torch.zeros(0, dtype=torch.int64, device="cuda"), u.cuda(),
            torch.zeros(rows + 1, dtype=torch.int64, device="cuda"))
        assert tokens.tolist() == [i * 2039 for i in range(rows)] and accepted.tolist() == [0] * rows
        assert (logp.cpu() + np.log(vocab)).abs().max() < 2.0 ** -20 * 12
    # behind a looked-up draft that falls, its token has no share
    tokens = g.ar_verify_drafts(target[:2].cuda(), torch.tensor([5], device="cuda"), torch.tensor([0.5, 5 / vocab]).cuda())[1]
    assert tokens.tolist() == [4, -1]  # 5 (vocab - 1) / vocab < 5: the five shares of tokens 0 to 4 pass it
    tokens = g.ar_verify_drafts(target[:2].cuda(), torch.tensor([5], device="cuda"), torch.tensor([0.5, 7 / vocab]).cuda())[1]
    assert tokens.tolist() == [7, -1]  # just below 7 shares: of tokens 0 to 4, 6 and 7


def test_tokens_have_the_targets_distribution(g):
    """200000 drafts of q verified against p: every token's share is p's, within 5 standard deviations."""
    n, vocab = 200000, 9
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, y = torch.randn(2, vocab, generator=gen, device="cuda")
    p, q = x.double().softmax(0), y.double().softmax(0)
    drafts = torch.multinomial(q, n, replacement=True, generator=gen)
    u = torch.rand(2 * n, generator=gen, device="cuda")
    start = torch.arange(n + 1, device="cuda")
    accepted, tokens, _ = g.ar_verify_drafts(x.expand(2 * n, vocab).contiguous(), drafts, u, start,
                                             draft_logits=y.expand(n, vocab).contiguous())
    first = tokens[0::2]
    share = torch.bincount(first, minlength=vocab).double() / n
    assert ((share - p).abs() <= 5 * (p * (1 - p) / n).sqrt()).all()
    rate = torch.minimum(p, q).sum()
    assert abs(accepted.double().mean() - rate) <= 5 * (rate * (1 - rate) / n).sqrt()
    # the token behind a draft that stands is drawn from the target
    second = tokens[1::2][accepted == 1]
    share = torch.bincount(second, minlength=vocab).double() / second.numel()
    assert ((share - p).abs() <= 5 * (p * (1 - p) / second.numel()).sqrt()).all()


def test_rows_that_are_no_distribution(g):
    """A NaN, +inf or nothing but -inf in the target or the draft: no draft stands there, and no token is drawn."""
    inf, nan = float("inf"), float("nan")
    for where in ("target", "draft"):
        for bad in (nan, inf, -inf):
            for dtype in (torch.float32, torch.bfloat16):
                target, draft = torch.zeros(4, 700, dtype=dtype), torch.zeros(3, 700, dtype=dtype)
                row = (target if where == "target" else draft)[1]
                row[:] = -inf if bad == -inf else 0.0
                row[651] = bad
                u = torch.tensor([0.5, 0.0, 0.0, 0.5])
                accepted, tokens, logp = g.ar_verify_drafts(target.cuda(), torch.tensor([7, 8, 9]).cuda(), u.cuda(),
                                                            draft_logits=draft.cuda())
                assert accepted.tolist() == [1] and tokens.tolist() == [7, -1, -1, -1], (where, bad, dtype)
                assert logp[1].isnan() and logp[2:].tolist() == [0.0, 0.0]
    x = torch.zeros(2, 10)
    x[1] = nan
    accepted, tokens, logp = g.ar_verify_drafts(x.cuda(), torch.tensor([3]).cuda(), mode="greedy")
    assert (accepted.tolist(), tokens.tolist()) == ([0], [0, -1])  # row 0's largest is token 0
    accepted, tokens, logp = g.ar_verify_drafts(x.cuda(), torch.tensor([0]).cuda(), mode="greedy")
    assert (accepted.tolist(), tokens.tolist()) == ([1], [0, -1]) and logp[1].isnan()


def test_lowest_values_and_ruled_out_drafts(g):
    low = torch.finfo(torch.float32).min
    x = torch.full((3, 64), low).cuda()  # of the lowest value alone: uniform
    drafts, u = torch.tensor([5, 6]).cuda(), torch.tensor([0.9 / 64, 0.5, 0.5]).cuda()
    accepted, tokens, _ = g.ar_verify_drafts(x, drafts, u)
    assert accepted.tolist() == [1] and tokens.tolist() == [5, 32, -1]  # half of 63 shares: 31.5, token 6 has none
    y = torch.zeros(3, 64).cuda()
    y[:, 5] = -float("inf")  # ruled out by the target: never stands, even with u = 0
    accepted, tokens, _ = g.ar_verify_drafts(y, drafts, torch.tensor([0.0, 0.0, 0.0]).cuda())
    assert accepted.tolist() == [0] and tokens.tolist() == [0, -1, -1]
    # probability 0 under the draft, some under the target: stands whatever u; token 6 does not (0.999 > 63 / 64), and
    # behind it only token 5 has a residue: 1 / 64, where the others' 1 / 64 - 1 / 63 is none
    q = torch.zeros(2, 64).cuda()
    q[:, 5] = -float("inf")
    accepted, tokens, _ = g.ar_verify_drafts(x, drafts, torch.tensor([0.999, 0.999, 0.0]).cuda(), draft_logits=q)
    assert accepted.tolist() == [1] and tokens.tolist() == [5, 5, -1]


def test_drafts_outside_the_vocabulary_and_odd_uniforms(g):
    x = torch.zeros(4, 64).cuda()
    for token in (-1, 64, 1 << 40, -(1 << 62)):
        accepted, tokens, _ = g.ar_verify_drafts(x, torch.tensor([token, 0, 0]).cuda(), torch.zeros(4).cuda())
        assert accepted.tolist() == [0] and tokens.tolist() == [0, -1, -1, -1]
        accepted, tokens, _ = g.ar_verify_drafts(x, torch.tensor([token, 0, 0]).cuda(), mode="greedy")
        assert accepted.tolist() == [0] and tokens.tolist() == [0, -1, -1, -1]
    nan = float("nan")
    for u, token in ((-1.0, 0), (1.0, 63), (7.0, 63), (nan, 0), (float("inf"), 63)):
        tokens = g.ar_verify_drafts(x[:1], torch.zeros(0, dtype=torch.int64).cuda(), torch.tensor([u]).cuda())[1]
        assert tokens.tolist() == [token], u
    accepted, tokens, _ = g.ar_verify_drafts(x[:2], torch.tensor([9]).cuda(), torch.tensor([nan, 0.0]).cuda())
    assert accepted.tolist() == [0] and tokens.tolist() == [0, -1]


def test_equal_distributions_keep_every_draft(g):
    """p = q: the ratio is 1 but for rounding, and every uniform number below 1 - 2^-18 accepts."""
    c = C.make([50, 50], 3001, "bf16", seed=6)
    c["draft_logits"] = c["target"][torch.cat([torch.arange(50), torch.arange(51, 101)])].clone()
    c["uniforms"] = torch.linspace(0, 1 - 2.0 ** -17, 102)
    assert C.call(g, c)[0].tolist() == [50, 50]
    c["uniforms"][3] = float("nan")  # a draft that falls although nothing is left: the token comes from p
    c["uniforms"][50] = 0.5
    accepted, tokens, _ = C.call(g, c)
    p = c["target"][3].double().softmax(0).cumsum(0)
    assert accepted.tolist() == [3, 50] and tokens[3].item() == int((p <= 0.5 * p[-1]).sum())


def test_rows_outside_every_sequence_stay(g):
    """A padded batch: rows before the first and behind the last sequence are neither read nor written."""
    c = C.make([2, 3], 300, seed=1)
    C.settle(c)
    expected = C.want(c)
    n, extra = 5, 4
    target = torch.full((n + 2 + extra, 300), float("nan"))
    target[2:9] = c["target"]
    draft = torch.full((n + extra, 300), float("nan"))
    draft[2:7] = c["draft_logits"]
    drafts = torch.full((n + extra,), 7)
    drafts[2:7] = c["drafts"]
    u = torch.full((n + 2 + extra,), float("nan"))
    u[2:9] = c["uniforms"]
    tokens, logp = torch.full((n + 2 + extra,), -77).cuda(), torch.full((n + 2 + extra,), 77.0).cuda()
    got = g.ar_verify_drafts(target.cuda(), drafts.cuda(), u.cuda(), (c["draft_start"] + 2).cuda(), draft_logits=draft.cuda(),
                             tokens=tokens, logp=logp)
    C.check((got[0], tokens[2:9], logp[2:9]), expected)
    assert (tokens[:2] == -77).all() and (tokens[9:] == -77).all()
    assert (logp[:2] == 77).all() and (logp[9:] == 77).all()


def test_offsets_that_are_none(g):
    """Offsets beyond the drafts or descending are clamped: no fault, and sound sequences have their result."""
    c = C.make([2, 3], 300, seed=1)
    C.settle(c)
    expected = C.want(c)
    for start in ([-9, 2, 1 << 50], [0, 2, 5]):
        c["draft_start"] = torch.tensor(start)
        C.check(C.call(g, c), expected)
    for start in ([5, 2, 0], [0, 9, 3], [7, 7, 7]):
        c["draft_start"] = torch.tensor(start)
        accepted, tokens, _ = C.call(g, c, tokens=torch.zeros(7, dtype=torch.int64, device="cuda"))
        assert ((tokens >= -1) & (tokens < 300)).all() and ((accepted >= 0) & (accepted <= 5)).all()


def test_repeats_bit_for_bit_in_a_graph_and_on_another_stream(g):
    c = C.make([4, 0, 3] * 5, 5003, "bf16", seed=12)
    C.settle(c)
    expected = C.want(c)
    d = {k: v.cuda() for k, v in c.items()}
    one = g.ar_verify_drafts(**d)
    C.check(one, expected)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    two = g.ar_verify_drafts(**d, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        three = g.ar_verify_drafts(**d)
    graph.replay()
    for got in (two, three):
        for a, b in zip(one, got):
            assert torch.equal(a, b)
    # replayed on other inputs
    e = C.make([4, 0, 3] * 5, 5003, "bf16", seed=13)
    C.settle(e)
    for k in d:
        d[k].copy_(e[k])
    graph.replay()
    C.check(three, C.want(e))
    assert g.ar_device_status() == g.AR_OK


def test_logp_is_what_token_logp_gives(g):
    """Behind the verification, the tokens are labels: their log-probabilities are the policy loss's."""
    c = C.make([3, 2], 32000, "bf16", seed=2)
    C.settle(c, 0.8)
    accepted, tokens, logp = C.call(g, c, 0.8)
    again = g.ar_token_logp(c["target"].cuda(), tokens, temperature=0.8)
    assert (again - logp).abs().max() < 2.0 ** -18  # two fp32 sums of the same row
    assert torch.equal(tokens < 0, logp == 0)


@pytest.mark.parametrize("temperature", [1e-6, 1e-3, 0.1, 30.0])
@pytest.mark.parametrize("shift", [0.0, 1e4, -3e30])
def test_temperatures_and_far_scores(g, temperature, shift):
    """Scores over the temperature so large that their product with log2 e has no fraction: the maximum is taken off first.
    (A shift that fp32 can hold beside the scores' differences; one that cannot leaves equal scores.)"""
    c = C.make([3, 0, 2], 2011, "f32", seed=17, drafted=False, temperature=max(temperature, 0.1), spread=2.0)
    c["target"] = (c["target"] + shift).contiguous()
    C.settle(c, temperature)
    C.check(C.call(g, c, temperature), C.want(c, temperature))
    C.check(C.call(g, c, temperature, mode="greedy"), C.want(c, temperature, greedy=True))


def test_far_scores_of_both_policies(g):
    """Distances beyond fp32's range, scores masked with the lowest value, another temperature for the draft."""
    c = C.make([4, 1], 1500, "f32", seed=23)
    c["target"] *= 1e30
    c["draft_logits"][:, 100:] = torch.finfo(torch.float32).min
    c["target"][:, 700:] = torch.finfo(torch.float32).min
    c["drafts"][:] = torch.tensor([3, 99, 0, 7, 50])
    for t, q in ((1.0, 1.0), (1e30, 0.5), (3e29, 1e31)):
        C.settle(c, t, q)
        C.check(C.call(g, c, t, draft_temperature=q), C.want(c, t, draft_temperature=q))


def test_a_sequence_of_many_drafts(g):
    """Hundreds of drafts that stand, and one that falls between them."""
    n, vocab = 700, 64
    x = torch.zeros(n + 1, vocab)
    drafts = torch.arange(n) % vocab
    x[torch.arange(n), drafts] = 12.0
    u = torch.full((n + 1,), 0.5)
    for fall in (n, 0, 7, 8, 333, n - 1):
        v = u.clone()
        if fall < n:
            v[fall] = 0.9999  # p = 1 / (1 + 63 e^-12) = 0.99961
        accepted, tokens, _ = g.ar_verify_drafts(x.cuda(), drafts.cuda(), v.cuda())
        assert accepted.tolist() == [fall]
        assert torch.equal(tokens[:fall].cpu(), drafts[:fall]) and (tokens[fall + 1:] == -1).all()
        # half of the 63 others, or of all 64 equal scores behind the last draft
        rest = [t for t in range(vocab) if fall == n or t != int(drafts[fall])]
        assert tokens[fall].item() == rest[len(rest) // 2]


def test_many_sequences_of_many_rows_are_skipped_alike(g):
    """More rows than run at once: whichever are skipped, the result is that of each sequence alone."""
    rng = np.random.default_rng(5)
    c = C.make(rng.integers(0, 9, 300).tolist(), 3000, "f32", seed=30, blur=0.7)
    C.settle(c)
    expected = C.want(c)
    for _ in range(5):
        C.check(C.call(g, c), expected)
    d = C.make([6] * 260, 2500, "bf16", seed=31, drafted=False, spread=4.0)
    C.settle(d)
    C.check(C.call(g, d), C.want(d))
    d["drafts"][::2] = d["target"].double().argmax(1)[torch.arange(260 * 6) + torch.arange(260).repeat_interleave(6)][::2]
    C.check(C.call(g, d, mode="greedy"), C.want(d, greedy=True))


def test_workspaces_that_hold_anything(g):
    """One workspace for calls of many shapes, one after the other, filled with ones, zeros, infinities or what the last
    call left: the results do not depend on it."""
    cases = []
    for i, (counts, vocab, dtype, drafted) in enumerate([([3, 0, 2], 5000, "f32", True), ([5] * 150, 9000, "bf16", True),
                                                         ([2, 9], 300, "bf16", False), ([0], 40000, "f32", False),
                                                         ([4] * 300, 2000, "f32", False)]):
        c = C.make(counts, vocab, dtype, seed=40 + i, drafted=drafted)
        C.settle(c)
        cases.append((c, C.want(c)))
    room = max(g.ar_verify_workspace(len(c["drafts"]), len(c["draft_start"]) - 1, c["target"].shape[1]) for c, _ in cases)
    ws = torch.empty(room // 4, device="cuda")
    for fill in (float("nan"), 0.0, float("inf"), -float("inf"), 1.0, None, None):
        for c, expected in cases:
            if fill is not None:
                ws.fill_(fill)
            C.check(C.call(g, c, workspace=ws), expected, fill)


def test_calls_side_by_side(g):
    """Calls on streams of their own, each with its workspace, give what they give alone."""
    cases = []
    for i, counts in enumerate([[4] * 200, [6, 0, 1], [1] * 90]):
        c = C.make(counts, 4001, "bf16", seed=50 + i)
        C.settle(c)
        cases.append(({k: v.cuda() for k, v in c.items()}, C.want(c)))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[g.ar_verify_drafts(**d, stream=s) for (d, _), s in zip(cases, streams)] for _ in range(8)]
    torch.cuda.synchronize()
    for round_ in got:
        for out, (_, expected) in zip(round_, cases):
            C.check(out, expected)


def test_two_graphs_of_one_workspace_replayed_in_turn(g):
    c, d = C.make([3, 1, 4], 3000, seed=60), C.make([2, 2], 7001, "bf16", seed=61, drafted=False)
    room = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    graphs = []
    for x in (c, d):
        C.settle(x)
        inputs = {k: None if v is None else v.cuda() for k, v in x.items()}
        g.ar_verify_drafts(**inputs, workspace=room)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = g.ar_verify_drafts(**inputs, workspace=room)
        graphs.append((graph, out, C.want(x), inputs))
    for _ in range(3):
        for graph, out, expected, _ in graphs:
            for t in out:
                t.fill_(7)
            graph.replay()
            C.check(out, expected)
