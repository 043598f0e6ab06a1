"""Calls of so much to read that rows behind a fall are skipped: against 64 bits, whatever runs first."""

import numpy as np
import pytest
import torch

import _verify_checks as C

pytestmark = pytest.mark.gpu
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def make(counts, vocab, target="bf16", draft=None, seed=0, shift=0, odd=False, stand=0.7):
    """Device tensors as in _verify_checks.make, from the device: too many logits for the host. `odd`: rows far from
    zero, rows with a NaN and rows of nothing among them. Drafts without distributions are the likeliest tokens, or
    any, `stand` of the former."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    counts = torch.as_tensor(counts)
    start = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    n, rows = int(start[-1]), int(start[-1]) + len(counts)
    x = (3.0 * torch.randn(rows, vocab + shift, generator=gen, device="cuda")).to(KINDS[target])[:, shift:]
    at = (torch.arange(n) + torch.repeat_interleave(torch.arange(len(counts)), counts)).cuda()
    y, chosen = None, x
    if draft is not None:
        y = torch.empty(n, vocab, dtype=KINDS[draft], device="cuda")
        for lo in range(0, n, 256):
            part = x[at[lo:lo + 256]].float()
            y[lo:lo + 256] = part + 0.8 * torch.randn(part.shape, generator=gen, device="cuda")
    drafts = torch.empty(n, dtype=torch.int64, device="cuda")
    for lo in range(0, n, 256):
        p = (x[at[lo:lo + 256]] if y is None else y[lo:lo + 256]).float()
        any_ = torch.multinomial(p.softmax(1), 1, generator=gen)[:, 0]
        likely = torch.rand(any_.shape, generator=gen, device="cuda") < stand
        drafts[lo:lo + 256] = any_ if y is not None else torch.where(likely, p.argmax(1), any_)
    if odd:
        x[3::31] += 1e7 if target == "f32" else 0.0
        x[5::37, vocab // 3] = float("nan")
        x[11::41] = -float("inf")
    return dict(target=x, drafts=drafts, uniforms=torch.rand(rows, generator=gen, device="cuda"),
                draft_start=start.cuda(), draft_logits=y)


def softmax(row):
    """In 64 bits; None where the row is no distribution."""
    row = row.double()
    top = row.max()
    if not torch.isfinite(top):
        return None
    return (row - top).softmax(0)


def want(c, greedy=False):
    """As oracle.verify.verify, row by row on the device, where the rows are."""
    start, drafts = c["draft_start"].tolist(), c["drafts"].tolist()
    u = c["uniforms"].double().tolist()
    rows = c["target"].shape[0]
    tokens, logp, margins, accepted = np.full(rows, -1), np.zeros(rows), np.full(rows, np.inf), []
    for s in range(len(start) - 1):
        first, count = start[s], start[s + 1] - start[s]
        for j in range(count + 1):
            row, x = first + s + j, drafts[first + j] if j < count else -1
            p, q, qx = softmax(c["target"][row]), None, 1.0
            if j < count and c["draft_logits"] is not None:
                q = softmax(c["draft_logits"][first + j])
                qx = float(q[x])
            if p is None:
                logp[row] = np.nan
                accepted.append(j)
                break
            if greedy:
                top = c["target"][row]
                token = int((top == top.max()).nonzero()[0])
                stands = token == x
            else:
                ratio = float(p[x]) / qx if x >= 0 else 0.0
                stands = u[row] < ratio
                if x >= 0:
                    margins[row] = abs(u[row] - ratio) / ratio
                if not stands:
                    w = p
                    if j < count and q is not None:
                        w = (p - q).clamp(min=0)
                    elif j < count:
                        w = p.clone()
                        w[x] = 0.0
                    upto = w.cumsum(0)
                    last = first + count + s
                    border = u[last] * upto[-1]
                    token = int(torch.searchsorted(upto, border.reshape(1), right=True))
                    margins[last] = min(margins[last], float(upto[token] - border), float(border - upto[token] + w[token]))
            token = x if stands else token
            tokens[row], logp[row] = token, float(p[token].log())
            if not stands:
                accepted.append(j)
                break
    return np.array(accepted), tokens, logp, margins


def settle(c):
    """As _verify_checks.settle. Returns what is wanted then."""
    start = c["draft_start"].tolist()
    finals = np.zeros(c["target"].shape[0], bool)
    finals[[start[s + 1] + s for s in range(len(start) - 1)]] = True
    for _ in range(8):
        expected = want(c)
        bad = expected[3] < np.where(finals, C.SUM, C.RATIO)
        if not bad.any():
            return expected
        at = torch.from_numpy(np.nonzero(bad)[0]).cuda()
        c["uniforms"][at] = c["uniforms"][at] * 0.983 + 0.004
    raise AssertionError("inputs without room")


def call(g, c, **kw):
    if kw.get("mode") == "greedy":
        return g.ar_verify_drafts(c["target"], c["drafts"], None, c["draft_start"], **kw)
    return g.ar_verify_drafts(c["target"], c["drafts"], c["uniforms"], c["draft_start"], draft_logits=c["draft_logits"], **kw)


def room(g, c):
    return torch.empty(g.ar_verify_workspace(c["drafts"].numel(), c["draft_start"].numel() - 1, c["target"].shape[1]),
                       dtype=torch.uint8, device="cuda")


def check_skips(g, c, expected, **kw):
    """Whatever the workspace holds, equal bits, and those wanted. That rows are skipped shows in the workspace's last
    part, where the place of every sequence's first fall is kept."""
    ws, first = room(g, c), None
    seqs = c["draft_start"].numel() - 1
    places = ws[ws.numel() - (4 * seqs + 255) // 256 * 256:][:4 * seqs].view(torch.int32)
    for fill in (0x77, 0, 255, None, None):
        if fill is not None:
            ws.fill_(fill)
        got = call(g, c, workspace=ws, **kw)
        fell = places.clone()
        assert (fell != 0x77777777).all() and (fell >= 0).all()
        C.check(got, expected, fill)
        # a draft that fell is where its sequence stopped (of rows far from zero, the drawing kernel alone knows)
        known = fell < 2 ** 31 - 1
        assert known.any() and (got[0][known] <= fell[known]).all()
        first = first or got
        assert all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) for a, b in zip(got, first))


CASES = {
    "drafted": dict(counts="0-8", seqs=200, vocab=65536, draft="bf16"),
    "drafted, odd vocabulary": dict(counts="0-8", seqs=260, vocab=50021, draft="bf16", shift=3),
    "drafted, two types": dict(counts="2-6", seqs=150, vocab=32003, target="f32", draft="bf16", odd=True),
    "drafted, fp32": dict(counts="8", seqs=40, vocab=60001, target="f32", draft="f32"),
    "looked up": dict(counts="0-12", seqs=300, vocab=32003),
    "looked up, fp32": dict(counts="0-5", seqs=500, vocab=20011, target="f32", odd=True),
    "uneven": dict(counts="uneven", seqs=64, vocab=100003),
    "few long rows": dict(counts="3", seqs=30, vocab=600011, draft="bf16"),
}


def case(name, seed=0):
    k = dict(CASES[name])
    seqs, counts = k.pop("seqs"), k.pop("counts")
    rng = np.random.default_rng(len(name) + seed)
    lo, _, hi = counts.partition("-")
    if counts == "uneven":  # nearly all drafts in two sequences
        n = rng.integers(0, 3, seqs)
        n[[7, 40]] = 300
    else:
        n = rng.integers(int(lo), int(hi or lo) + 1, seqs)
    return make(n, seed=seed, **k)


@pytest.mark.parametrize("name", CASES)
def test_rows_behind_a_fall(g, name):
    c = case(name)
    check_skips(g, c, settle(c))


@pytest.mark.parametrize("vocab,target", [(50021, "bf16"), (32000, "f32")])
def test_greedy(g, vocab, target):
    c = make(np.random.default_rng(1).integers(0, 11, 300), vocab, target, seed=4, odd=True, stand=0.9)
    check_skips(g, c, want(c, greedy=True), mode="greedy")


def test_as_each_sequence_alone(g):
    """A call for one sequence skips nothing."""
    c = case("drafted", 1)
    settle(c)
    accepted, tokens, logp = call(g, c)
    start = c["draft_start"].tolist()
    for s in range(0, 200, 7):
        d, r = slice(start[s], start[s + 1]), slice(start[s] + s, start[s + 1] + s + 1)
        one = g.ar_verify_drafts(c["target"][r], c["drafts"][d], c["uniforms"][r], draft_logits=c["draft_logits"][d])
        assert one[0][0] == accepted[s] and torch.equal(one[1], tokens[r])
        # (rows are cut into other parts: two sums of the same terms)
        assert (one[2] - logp[r]).abs().max() <= 2.0 ** -19


def test_side_by_side(g):
    cases = [case("drafted", 2), case("looked up", 3)]
    expected = [settle(c) for c in cases]
    streams, rooms = [torch.cuda.Stream() for _ in cases], [room(g, c) for c in cases]
    torch.cuda.synchronize()
    got = [[call(g, c, stream=s, workspace=w) for c, s, w in zip(cases, streams, rooms)] for _ in range(6)]
    torch.cuda.synchronize()
    for outs in got:
        for out, e in zip(outs, expected):
            C.check(out, e)


def test_replayed_on_other_inputs(g):
    c, e = case("looked up", 4), case("looked up", 4)
    ws = room(g, c)
    call(g, c, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(g, c, workspace=ws)
    for flip in (False, True):
        if flip:  # other drafts and numbers on the same rows
            c["drafts"].copy_(e["drafts"].roll(1))
            c["uniforms"].copy_(e["uniforms"].flip(0))
        expected = settle(c)
        for _ in range(2):
            graph.replay()
            C.check(out, expected)
    assert g.ar_device_status() == g.AR_OK
