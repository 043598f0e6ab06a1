"""Refusals of the gradient calls and of the verification of drafted tokens, without a GPU: every bad
argument is answered before any device work is enqueued; and what the binding takes from tensors."""

import ctypes

import pytest
import torch

from test_binding_tensors import Device

A = 1 << 24  # a stand-in device address: the calls below return before it is used
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def tensors(g, *specs):
    arr = (g._lib.ArTensor * max(1, len(specs)))()
    for i, (data, count, dtype) in enumerate(specs):
        arr[i].data, arr[i].count, arr[i].dtype = data, count, dtype
    return arr


def norm(g, specs=None, outs=None, clip=False, n=None, **kw):
    a = dict(kind=0, max_norm=1.0, eps=1e-6, scale=1.0, stats=8 * A, norms=9 * A, ws=10 * A)
    a.update(kw)
    specs = [(A, 100, 0), (2 * A, 7, 1)] if specs is None else specs
    t = tensors(g, *specs)
    n = len(specs) if n is None else n
    d = g._lib.ArNormDesc(a["kind"], a["max_norm"], a["eps"], a["scale"])
    lib = g._lib.load()
    if clip:
        o = None if outs is None else tensors(g, *outs)
        return lib.ar_grad_clip(t, n, o, d, a["stats"], a["norms"], a["ws"], None)
    return lib.ar_grad_norm(t, n, d, a["stats"], a["norms"], a["ws"], None)


BAD_NORM = [dict(kind=2), dict(kind=-1), dict(max_norm=0.0), dict(max_norm=-1.0), dict(max_norm=NAN), dict(eps=-1.0),
            dict(eps=NAN), dict(eps=INF), dict(scale=NAN), dict(scale=INF), dict(stats=0), dict(stats=8 * A + 2),
            dict(norms=9 * A + 1), dict(ws=0), dict(ws=10 * A + 8), dict(n=0), dict(n=-3),
            dict(specs=[(0, 5, 0)]), dict(specs=[(A + 2, 5, 0)]), dict(specs=[(A + 1, 5, 1)]), dict(specs=[(A, -1, 0)]),
            dict(specs=[(A, 5, 2)]), dict(specs=[(A, (1 << 40) + 1, 0)]),
            dict(stats=A + 4), dict(norms=2 * A), dict(ws=A), dict(stats=9 * A + 4), dict(stats=10 * A + 64),
            dict(specs=[(A, 100, 0), (10 * A + (1 << 14), 3, 0)])]


@pytest.mark.parametrize("bad", BAD_NORM)
@pytest.mark.parametrize("clip", [False, True])
def test_bad_norms(g, bad, clip):
    assert norm(g, clip=clip, **bad) == g.AR_EINVAL


@pytest.mark.parametrize("outs", [[(A, 99, 0), (2 * A, 7, 1)], [(A, 100, 1), (2 * A, 7, 1)], [(0, 100, 0), (2 * A, 7, 1)],
                                  [(A + 4, 100, 0), (2 * A, 7, 1)], [(3 * A, 100, 0), (3 * A + 398, 7, 1)],
                                  [(2 * A, 100, 0), (3 * A, 7, 1)], [(8 * A, 100, 0), (2 * A, 7, 1)]])
def test_bad_clip_outputs(g, outs):
    """Other counts or types, missing, overlapping one another, a gradient or the statistics."""
    assert norm(g, clip=True, outs=outs) == g.AR_EINVAL


def test_more_norm_refusals(g):
    assert norm(g, n=g.AR_MAX_TENSORS + 1) == g.AR_EUNSUPPORTED
    # a tensor named twice: two outputs in one place
    assert norm(g, clip=True, specs=[(A, 100, 0), (A, 100, 0)]) == g.AR_EINVAL
    lib, b = g._lib.load(), ctypes.c_size_t()
    assert lib.ar_grad_norm(None, 1, g._lib.ArNormDesc(0, 1.0, 0.0, 1.0), 8 * A, 0, 10 * A, None) == g.AR_EINVAL
    assert lib.ar_grad_norm(tensors(g, (A, 1, 0)), 1, None, 8 * A, 0, 10 * A, None) == g.AR_EINVAL
    assert lib.ar_grad_workspace(0, b) == g.AR_EINVAL and lib.ar_grad_workspace(1, None) == g.AR_EINVAL
    assert lib.ar_grad_workspace(g.AR_MAX_TENSORS + 1, b) == g.AR_EUNSUPPORTED
    assert lib.ar_grad_workspace(g.AR_MAX_TENSORS, b) == g.AR_OK and b.value % 16 == 0


LISTS = ("params", "grads", "exp_avgs", "exp_avg_sqs", "masters", "params_out", "exp_avgs_out", "exp_avg_sqs_out",
         "masters_out")


def adam(g, n=None, clip=0, **kw):
    d = dict(lr=0.1, beta1=0.9, beta2=0.99, eps=1e-8, decay=0.0, scale=1.0, step=1, device=0, rate=0)
    lists = {k: [((i + 1) * A, 10, 0), ((i + 1) * A + 4096, 7, 0)] for i, k in enumerate(LISTS)}
    d.update({k: v for k, v in kw.items() if k in d})
    lists.update({k: v for k, v in kw.items() if k in lists})
    desc = g._lib.ArAdamwDesc(*d.values())
    c = [None if lists[k] is None else tensors(g, *lists[k]) for k in LISTS]
    return g._lib.load().ar_adamw_step(desc, 2 if n is None else n, *c, clip, None)


BAD_ADAM = [dict(lr=NAN), dict(lr=INF), dict(beta1=-0.1), dict(beta1=1.0), dict(beta2=1.0), dict(beta2=NAN), dict(eps=-1.0),
            dict(eps=INF), dict(decay=NAN), dict(scale=INF), dict(step=0), dict(step=-4), dict(device=12 * A + 4),
            dict(rate=12 * A + 2), dict(rate=7 * A), dict(clip=12 * A + 2), dict(n=0), dict(masters=None),
            *[{k: [(20 * A, 10, 0), (21 * A, 8, 0)]} for k in LISTS],      # another count
            *[{k: [(20 * A, 10, 0), (0, 7, 0)]} for k in LISTS],           # missing
            *[{k: [(20 * A + 2, 10, 0), (21 * A, 7, 0)]} for k in LISTS],  # misaligned
            *[{k: [(20 * A, 10, 5), (21 * A, 7, 0)]} for k in LISTS],      # no type
            *[{k: None} for k in LISTS[:4]],
            *[{k: [(20 * A, 10, 1), (21 * A, 7, 0)]} for k in LISTS if k not in ("params", "grads", "params_out")],
            dict(params_out=[(20 * A, 10, 1), (21 * A, 7, 0)]),            # not the parameter's type
            *[{k: [(20 * A, 10, 0), (20 * A + 36, 7, 0)]} for k in LISTS if k.endswith("_out")],  # overlapping itself
            *[{k: [(2 * A + 4, 10, 0), (21 * A, 7, 0)]} for k in LISTS if k.endswith("_out")],    # the gradients
            dict(exp_avgs_out=[(4 * A, 10, 0), (21 * A, 7, 0)]), dict(clip=7 * A), dict(device=8 * A)]


@pytest.mark.parametrize("bad", BAD_ADAM)
def test_bad_adamw_steps(g, bad):
    assert adam(g, **bad) == g.AR_EINVAL


def test_more_adamw_refusals(g):
    assert adam(g, n=g.AR_MAX_TENSORS + 1) == g.AR_EUNSUPPORTED
    # two parameters in one place, in place
    same = [(A, 10, 0), (A, 10, 0)]
    assert adam(g, params=same, params_out=None, masters=None, masters_out=None) == g.AR_EINVAL


def verify(g, n_drafts=3, n_seq=2, vocab=10, mode=0, **kw):
    rows = n_drafts + n_seq
    x = dict(data=A, rows=rows, ld=vocab, dtype=0, temperature=1.0)
    y = dict(data=2 * A, rows=n_drafts, ld=vocab, dtype=0, temperature=1.0)
    a = dict(drafts=3 * A, uniforms=4 * A, start=5 * A, accepted=6 * A, tokens=7 * A, logp=8 * A, ws=9 * A)
    for k, v in kw.items():
        if k.startswith("x_"):
            x[k[2:]] = v
        elif k.startswith("y_"):
            y[k[2:]] = v
        else:
            a[k] = v
    d = g._lib.ArVerifyDesc(g._lib.ArScoreRows(*x.values()), g._lib.ArScoreRows(*y.values()), vocab, a["drafts"],
                            a["uniforms"], a["start"], n_drafts, n_seq, mode)
    return g._lib.load().ar_verify_drafts(d, a["accepted"], a["tokens"], a["logp"], a["ws"], None)


BAD_VERIFY = [dict(n_drafts=-1, x_rows=1, y_rows=-1), dict(n_seq=0), dict(vocab=0), dict(mode=2), dict(mode=-1),
              dict(mode=1),  # greedy with draft logits
              *[{f"{r}_{k}": v} for r in "xy" for k, v in (("rows", 4), ("ld", 9), ("dtype", 2), ("temperature", 0.0),
                                                            ("temperature", -1.0), ("temperature", NAN),
                                                            ("temperature", INF), ("temperature", 1e-45))],
              dict(x_data=0), dict(x_data=A + 2), dict(y_data=2 * A + 1), dict(x_ld=1 << 61), dict(drafts=0),
              dict(drafts=3 * A + 4), dict(uniforms=0), dict(uniforms=4 * A + 2), dict(start=0), dict(start=5 * A + 4),
              *[{k: v} for k, v in (("accepted", 0), ("tokens", 0), ("logp", 0), ("ws", 0), ("accepted", 6 * A + 4),
                                    ("tokens", 7 * A + 4), ("logp", 8 * A + 2), ("ws", 9 * A + 8))],
              *[{k: v} for k in ("accepted", "tokens", "logp", "ws") for v in (A, 2 * A, 3 * A, 4 * A, 5 * A)],
              dict(tokens=6 * A), dict(logp=7 * A + 8), dict(ws=8 * A)]


@pytest.mark.parametrize("bad", BAD_VERIFY)
def test_bad_verifications(g, bad):
    assert verify(g, **bad) == g.AR_EINVAL


def test_more_verify_refusals(g):
    big = 1 << 31
    assert verify(g, n_drafts=big, x_rows=big + 2, y_rows=big) == g.AR_EUNSUPPORTED
    assert verify(g, n_drafts=big - 2, x_rows=big, y_rows=big - 2) == g.AR_EUNSUPPORTED
    assert verify(g, n_seq=big, x_rows=big + 3) == g.AR_EUNSUPPORTED
    assert verify(g, vocab=(1 << 30) + 1) == g.AR_EUNSUPPORTED
    lib, b = g._lib.load(), ctypes.c_size_t()
    assert lib.ar_verify_drafts(None, 6 * A, 7 * A, 8 * A, 9 * A, None) == g.AR_EINVAL
    assert lib.ar_verify_workspace(3, 2, 10, None) == g.AR_EINVAL
    assert lib.ar_verify_workspace(-1, 2, 10, b) == g.AR_EINVAL and lib.ar_verify_workspace(0, 0, 10, b) == g.AR_EINVAL
    assert lib.ar_verify_workspace(3, 2, 0, b) == g.AR_EINVAL
    assert lib.ar_verify_workspace(big, 2, 10, b) == g.AR_EUNSUPPORTED
    assert lib.ar_verify_workspace(0, 1, 10, b) == g.AR_OK and b.value % 16 == 0


# ---------------------------------------------------------------- the binding


def test_lists_that_do_not_match(g):
    a, b = Device(torch.zeros(4, 3)), Device(torch.zeros(5))
    good = [a, b]
    for bad in ([], [a], [a, b, b], [b, a], [a, None], [a, Device(torch.zeros(3, 4).t())]):
        for name in ("grads", "exp_avgs", "exp_avg_sqs", "params_out", "exp_avgs_out", "exp_avg_sqs_out"):
            lists = {k: good for k in ("params", "grads", "exp_avgs", "exp_avg_sqs")}
            with pytest.raises(ValueError, match=name):
                g.ar_adamw_step(**{**lists, name: bad}, lr=0.1, step=1)
        with pytest.raises(ValueError, match="outs"):
            g.ar_grad_clip(good, 1.0, outs=bad, stats=Device(torch.zeros(4)), norms=Device(torch.zeros(2)),
                           workspace=Device(torch.zeros(1 << 17, dtype=torch.uint8)))
    with pytest.raises(ValueError, match="masters"):
        g.ar_adamw_step(good, good, good, good, 0.1, 1, masters=[None])
    for bad in ([], [None], [torch.zeros(3)], [Device(torch.zeros(8)[::2])], [Device(torch.zeros(1).expand(4))]):
        with pytest.raises(ValueError, match="grads|at least one"):
            g.ar_grad_norm(bad)
    with pytest.raises(TypeError):
        g.ar_grad_norm([Device(torch.zeros(3, dtype=torch.float16))])


def test_elements_one_behind_the_other(g):
    t = torch.zeros(2, 3, 4)
    assert all(g._dense(v) for v in (t, t.permute(2, 0, 1), t.transpose(0, 1), t[:1], t[0], torch.zeros(0, 3), torch.zeros(())))
    assert not any(g._dense(v) for v in (t[:, :2], t[..., ::2], t[:, :1], torch.zeros(3, 1).expand(3, 2)))
    lists = g.TensorList([Device(t), Device(t.permute(2, 0, 1))])
    assert lists.counts == [24, 24] and lists.layouts[0] is None and lists.layouts[1] is not None and len(lists) == 2


def test_verify_tensors(g):
    x, drafts, u = Device(torch.zeros(5, 8)), Device(torch.zeros(3, dtype=torch.int64)), Device(torch.zeros(5))
    start = Device(torch.tensor([0, 1, 3]))
    ok = dict(target=x, drafts=drafts, uniforms=u, draft_start=start)
    for name, bad in (("drafts", Device(torch.zeros(5, dtype=torch.int64))), ("drafts", Device(torch.zeros(3))),
                      ("drafts", Device(torch.zeros(3, 1, dtype=torch.int64))), ("uniforms", None),
                      ("uniforms", Device(torch.zeros(4))), ("uniforms", Device(torch.zeros(5, dtype=torch.float64))),
                      ("draft_start", Device(torch.tensor([0, 3]))), ("draft_start", Device(torch.tensor([0, 1, 3]).int())),
                      ("target", Device(torch.zeros(8).expand(5, 8))), ("draft_logits", Device(torch.zeros(3, 9))),
                      ("draft_logits", Device(torch.zeros(2, 8))), ("draft_logits", Device(torch.zeros(8).expand(3, 8))),
                      ("tokens", Device(torch.zeros(5))), ("accepted", Device(torch.zeros(5, dtype=torch.int64))),
                      ("logp", Device(torch.zeros(4))), ("workspace", Device(torch.zeros(8, dtype=torch.uint8)))):
        with pytest.raises(ValueError, match=name):
            g.ar_verify_drafts(**{**ok, name: bad})


def test_clip_of_the_orthogonalised_step(g):
    plan = g.ar_ortho_plan([(4, 8)])
    lib, d = g._lib.load(), g._lib.ArMuonDesc(0.1, 0.9, 0.0, 1, 0, 1.0)

    def call(clip, ws=9 * A, plan=plan.handle, n=3):
        m = [(g._lib.ArMatrix * 1)(g._lib.ArMatrix((i + 1) * A, 8)) for i in range(3)]
        return lib.ar_muon_step_clipped(plan, d, *m, None, None, clip, ws, None)

    assert call(5 * A + 2) == g.AR_EINVAL                   # misaligned
    for at in (A, 3 * A + 4, 9 * A + 64):                   # weights, momentum, workspace
        assert call(at) == g.AR_EINVAL
    assert call(5 * A, ws=0) == g.AR_EINVAL and call(5 * A, plan=None) == g.AR_EINVAL
    x = [Device(torch.zeros(4, 8))]
    with pytest.raises(ValueError, match="clip"):
        g.ar_muon_step(plan, x, x, x, lr=0.1, clip=Device(torch.zeros(3)),
                       workspace=Device(torch.zeros(1 << 22, dtype=torch.uint8)), stream=0)
