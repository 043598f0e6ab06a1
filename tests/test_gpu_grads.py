"""Gradient norm, clipping and AdamW on the GPU against the 64-bit oracle."""

import numpy as np
import pytest
import torch

from oracle import grads as G

pytestmark = pytest.mark.gpu
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}

# A batch of up to 64 squares is summed in fp32, in chains of at most 16 and two levels of joins: its sum is off by
# 2^-24 * 18 < 2^-19.8 of itself at most, all else is in 64 bits; the root halves that.
NORM = 2.0 ** -20


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def tensors(shapes, dtype, seed=0, std=1.0, shift=0):
    """Tensors in one buffer, one behind the other, the first `shift` elements in."""
    gen = torch.Generator().manual_seed(seed)
    kinds = [KINDS[dtype] if dtype != "mixed" else (torch.float32, torch.bfloat16)[i % 2] for i in range(len(shapes))]
    flat = {k: torch.zeros(shift + sum(int(np.prod(s)) for s, q in zip(shapes, kinds) if q == k) + 64, dtype=k, device="cuda")
            for k in set(kinds)}
    at, out = {k: shift for k in flat}, []
    for s, k in zip(shapes, kinds):
        n = int(np.prod(s))
        v = flat[k][at[k]:at[k] + n].view(s)
        v.copy_(torch.randn(s, generator=gen) * std)
        at[k] += n
        out.append(v)
    return out


def wide(ts):
    return [t.detach().double().cpu().numpy() for t in ts]


LISTS = {
    "one": [(1,)],
    "empty": [(0,), (3,), (0, 5)],
    "short": [(7,), (8,), (9,), (15,), (16,), (17,), (31,), (33,)],
    "odd": [(129, 33), (1,), (0,), (2049,), (77, 131)],
    "long": [(1 << 20,), (3,), (1000, 1003)],
    "many": [(5 + i % 700,) for i in range(2000)],
    "hundred": [(513,)] * 100,
}


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("shift", [0, 1, 5])
@pytest.mark.parametrize("kind", ["l2", "max"])
def test_norm(g, name, dtype, shift, kind):
    ts = tensors(LISTS[name], dtype, shift=shift)
    stats, norms = g.ar_grad_norm(ts, 2.0, kind=kind, grad_scale=0.3)
    want, each = G.norm(wide(ts), 2.0, kind, grad_scale=float(np.float32(0.3)))
    room = NORM if kind == "l2" else 2.0 ** -23  # a maximum is exact but for the product
    assert np.allclose(norms.cpu().numpy(), each, rtol=room, atol=0)
    assert np.allclose(stats.cpu().numpy(), want, rtol=2 * room, atol=0), (stats, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e-43, 3e-39, 1e-30, 1e-20, 1e18, 1e30, 3e38])
def test_norm_over_all_of_fp32s_range(g, dtype, size):
    for mixed in (False, True):
        ts = tensors([(300,), (41, 77)], "f32", seed=3)
        for t in ts:
            t.clamp_(-1, 1).mul_(size)
            if mixed:  # beside ordinary numbers
                t.view(-1)[::7] = 1.0
        ts = [t.to(KINDS[dtype]) for t in ts]
        stats, norms = g.ar_grad_norm(ts, 1.0)
        want, each = G.norm(wide(ts), 1.0)
        # (results below fp32's normal numbers are whole multiples of 2^-149, above its range infinite)
        with np.errstate(over="ignore"):
            each, want = each.astype(np.float32).astype(np.float64), want.astype(np.float32).astype(np.float64)
        assert np.allclose(norms.cpu().numpy(), each, rtol=NORM + 2.0 ** -23, atol=2.0 ** -149)
        assert np.allclose(stats.cpu().numpy(), want, rtol=2 * NORM, atol=2.0 ** -149)
        assert stats[3] == 1.0


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("place", [0, 1, 4000, 9999])
def test_not_finite(g, kind, dtype, place):
    """Found wherever it is; a NaN makes the norm NaN, an infinity infinite; the gradients come out as zeros."""
    for bad in (float("nan"), float("inf"), -float("inf")):
        ts = tensors([(9,), (100, 100), (5,)], dtype)
        ts[1].view(-1)[place] = bad
        outs = [torch.ones_like(t) for t in ts]
        stats, norms, _ = g.ar_grad_clip(ts, 1.0, outs=outs, kind=kind)
        assert stats[1:].tolist() == [0.0, 1.0, 0.0]
        assert (stats[0].isnan() if bad != bad else stats[0] == float("inf"))
        assert norms[0].isfinite() and norms[2].isfinite() and not norms[1].isfinite()
        assert all((o == 0).all() for o in outs)
    ts[1].view(-1)[(place + 5000) % 10000] = float("nan")  # both: NaN
    assert g.ar_grad_norm(ts, 1.0, kind=kind)[0][0].isnan()
    zero = [torch.zeros_like(t) for t in ts]
    assert g.ar_grad_norm(zero, 1.0, kind=kind)[0].tolist() == [0.0, 1.0, 0.0, 1.0]


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("shifts", [(0, 0), (1, 1), (3, 8), (2, 5)])
def test_clip(g, name, dtype, shifts):
    ts = tensors(LISTS[name], dtype, shift=shifts[0])
    outs = tensors(LISTS[name], dtype, seed=1, shift=shifts[1])
    keep = [t.clone() for t in ts]
    stats, norms, got = g.ar_grad_clip(ts, 0.25, outs=outs, grad_scale=0.5)
    want, _ = G.norm(wide(ts), 0.25, grad_scale=0.5)
    assert np.allclose(stats.cpu().numpy(), want, rtol=2 * NORM, atol=0)
    factor = stats[1] * 0.5
    for t, o, k in zip(ts, outs, keep):
        assert torch.equal(t, k)
        assert torch.equal(o, (t.float() * factor).to(t.dtype))  # one product, rounded once to fp32, then to its type
    # in place, the same bits
    _, _, same = g.ar_grad_clip(ts, 0.25, grad_scale=0.5)
    assert all(a is b for a, b in zip(same, ts))
    for t, o in zip(ts, outs):
        assert torch.equal(t, o)


def test_clip_leaves_what_needs_no_clipping(g):
    ts = tensors([(100, 33), (7,)], "bf16")
    keep = [t.clone() for t in ts]
    stats, _, _ = g.ar_grad_clip(ts, 1e6)
    assert stats[1:].tolist() == [1.0, 0.0, 1.0] and all(torch.equal(a, b) for a, b in zip(ts, keep))
    outs = [torch.zeros_like(t) for t in ts]
    g.ar_grad_clip(ts, float("inf"), outs=outs)
    assert all(torch.equal(a, b) for a, b in zip(outs, keep))
    # some out of place, some in place
    outs = [ts[0], torch.zeros_like(ts[1])]
    g.ar_grad_clip(ts, 0.5, outs=outs)
    assert not torch.equal(ts[0], keep[0]) and torch.equal(ts[1], keep[1]) and (outs[1] != 0).any()


def test_transposed_gradients(g):
    """Elements in another order of the dimensions: the same norm, clipped in their own order."""
    t = torch.randn(33, 65, device="cuda")
    a, b = g.ar_grad_norm([t.t()], 1.0)[0], g.ar_grad_norm([t], 1.0)[0]
    assert torch.equal(a, b)
    out = torch.empty(33, 65, device="cuda").t()
    g.ar_grad_clip([t.t()], 1.0, outs=[out])
    assert torch.equal(out, t.t() * a[1])
    with pytest.raises(ValueError, match="outs"):
        g.ar_grad_clip([t.t()], 1.0, outs=[torch.empty(65, 33, device="cuda")])


def test_equal_calls_give_equal_bits(g):
    ts = tensors(LISTS["long"], "f32")
    a, b = g.ar_grad_norm(ts, 1.0)
    for _ in range(5):
        c, d = g.ar_grad_norm(g.TensorList(ts), 1.0, workspace=torch.full((1 << 17,), 255, dtype=torch.uint8, device="cuda"))
        assert torch.equal(a, c) and torch.equal(b, d)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,shift", [(1, 0), (1, 3), (9, 7), (4097, 1), (12289, 6), (40000, 0)])
def test_nothing_outside_is_read_or_written(g, dtype, n, shift):
    """NaN on both sides of every buffer: none reaches the norm or an output, none changes."""
    def guarded(kind):
        mem = torch.full((n + 600,), float("nan"), dtype=kind, device="cuda")
        return mem, mem[256 + shift:256 + shift + n]

    def untouched(mem):
        return mem[:256 + shift].isnan().all() and mem[256 + shift + n:].isnan().all()

    kind = KINDS[dtype]
    (gm, gr), (om, o) = guarded(kind), guarded(kind)
    gr.copy_(torch.randn(n))
    stats, _, _ = g.ar_grad_clip([gr], 0.1, outs=[o])
    assert stats.isfinite().all() and torch.equal(o, (gr.float() * stats[1]).to(kind))
    mems = {k: guarded(f) for k, f in dict(p=kind, w=torch.float32, m=torch.float32, v=torch.float32).items()}
    for _, t in mems.values():
        t.fill_(0.5)
    g.ar_adamw_step([mems["p"][1]], [gr], [mems["m"][1]], [mems["v"][1]], 0.1, 1, masters=[mems["w"][1]])
    for mem, t in [*mems.values(), (gm, gr), (om, o)]:
        assert untouched(mem) and t.isfinite().all()


# ---------------------------------------------------------------- AdamW


def adam_state(shapes, grad, param, master, shift=0, seed=0):
    gs = tensors(shapes, grad, seed, 1e-2, shift)
    ps = tensors(shapes, param, seed + 1, 0.1, shift)
    ms, vs = tensors(shapes, "f32", seed + 2, 1e-3, shift), tensors(shapes, "f32", seed + 3, 1e-2, shift)
    for v in vs:
        v.square_()
    ws = None
    if master:  # some with a master, some without
        ws = tensors(shapes, "f32", seed + 4, 0.1, shift)
        ws = [None if i % 3 == 2 else w for i, w in enumerate(ws)]
    return ps, gs, ms, vs, ws


def check_adam(before, after, masters, t, lr, betas, eps, decay, scale, on_device=False):
    """Every output against the formula, each fp32 operation counted at 2^-24 of its result. on_device: the rates are
    worked out there in fp32: an expm1f (2) and a quotient with lr's rounding (2); half of an expm1f, a root and
    a quotient (3); 1 - lr decay (2)."""
    u = 2.0 ** -24
    (ps, gs, ms, vs, ws), (po, mo, vo, wo) = before, after
    for i in range(len(ps)):
        w = ps[i] if ws is None or ws[i] is None else ws[i]
        args = [x.double().cpu().numpy() for x in (w, gs[i], ms[i], vs[i])]
        want_w, want_m, want_v = G.adamw(*args, t, lr, betas, eps, decay, scale)
        w0, g0, m0, v0 = args
        g0 = np.abs(g0 * scale)
        # G: factor and product; M' and V': their coefficients, products and one fused sum
        room_m = u * (2 * np.abs(betas[0] * m0) + 5 * (1 - betas[0]) * g0) + 2.0 ** -148
        room_v = u * (2 * betas[1] * v0 + 8 * (1 - betas[1]) * g0 * g0) + 2.0 ** -148
        assert (np.abs(mo[i].double().cpu().numpy() - want_m) <= room_m).all()
        assert (np.abs(vo[i].double().cpu().numpy() - want_v) <= room_v).all()
        # the update: M' and V' as above (the root halves V's), then rate, product, root, quotient and sum
        c1, c2 = 1 - betas[0] ** t, 1 - betas[1] ** t
        root = np.sqrt(want_v / c2) + eps
        step = lr / c1 * np.abs(want_m) / root
        with np.errstate(invalid="ignore", divide="ignore"):
            spread = np.where(want_v > 0, room_v / (2 * want_v), 0.0)
        more = 7 if on_device else 0
        room = lr / c1 * room_m / root + step * (spread + (8 + more) * u) + (3 + more) * u * np.abs(w0) + u * np.abs(want_w)
        new = (po if wo is None or wo[i] is None else wo)[i]
        half = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}
        assert (np.abs(new.double().cpu().numpy() - want_w) <= room + half[new.dtype] * (np.abs(want_w) + room)).all()
        if wo is not None and wo[i] is not None:
            assert torch.equal(po[i], wo[i].to(po[i].dtype))


@pytest.mark.parametrize("name", ["one", "empty", "short", "odd", "hundred", "many"])
@pytest.mark.parametrize("grad,param,master", [("f32", "f32", False), ("bf16", "bf16", False), ("bf16", "bf16", True),
                                               ("f32", "bf16", True), ("bf16", "f32", False), ("mixed", "mixed", True)])
@pytest.mark.parametrize("shift", [0, 3])
def test_adamw(g, name, grad, param, master, shift):
    before = adam_state(LISTS[name], grad, param, master, shift)
    ps, gs, ms, vs, ws = before
    new = [[torch.full_like(t, float("nan")) for t in x] for x in (ps, ms, vs)]
    wo = None if ws is None else [None if w is None else torch.full_like(w, float("nan")) for w in ws]
    copies = [[None if t is None else t.clone() for t in x] if x is not None else None for x in before]
    t, lr, betas, eps, decay = 7, 0.01, (0.9, 0.95), 1e-8, 0.1
    g.ar_adamw_step(ps, gs, ms, vs, lr, t, betas, eps, decay, grad_scale=0.5, masters=ws, params_out=new[0],
                    exp_avgs_out=new[1], exp_avg_sqs_out=new[2], masters_out=wo)
    check_adam(before, (*new, wo), ws, t, lr, betas, eps, decay, 0.5)
    for x, c in zip(before, copies):
        assert x is None or all(a is None or torch.equal(a, b) for a, b in zip(x, c))
    # in place, the same bits
    g.ar_adamw_step(ps, gs, ms, vs, lr, t, betas, eps, decay, grad_scale=0.5, masters=ws)
    for x, y in zip((ps, ms, vs, ws), (*new, wo)):
        assert x is None or all(a is None or torch.equal(a, b) for a, b in zip(x, y))


def test_adamw_alignments_that_differ(g):
    """Arrays that do not agree modulo 8 elements give the same bits as arrays that do."""
    n = 9001
    ps, gs, ms, vs, _ = adam_state([(n,)], "bf16", "bf16", False)
    ref = [x[0].clone() for x in (ps, ms, vs)]
    g.ar_adamw_step([ref[0]], gs, [ref[1]], [ref[2]], 0.01, 3)
    for shifts in ((1, 0, 0, 0), (0, 2, 0, 0), (0, 0, 1, 0), (0, 0, 0, 4), (4, 4, 4, 0), (3, 3, 7, 7)):
        moved = []
        for x, shift in zip((ps, gs, ms, vs), shifts):
            mem = torch.zeros(n + 8, dtype=x[0].dtype, device="cuda")
            mem[shift:shift + n] = x[0]
            moved.append([mem[shift:shift + n]])
        g.ar_adamw_step(*moved, 0.01, 3)
        for a, b in zip(ref, (moved[0], moved[2], moved[3])):
            assert torch.equal(a, b[0])


@pytest.mark.parametrize("t", [1, 2, 1000, 10 ** 9])
@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.0, 0.0), (0.0, 0.95), (0.99, 0.0)])
def test_adamw_steps_and_betas(g, t, betas):
    before = adam_state([(300,)], "f32", "f32", False)
    ps, gs, ms, vs, _ = before
    new = [[torch.empty_like(x[0])] for x in (ps, ms, vs)]
    g.ar_adamw_step(ps, gs, ms, vs, 0.1, t, betas, params_out=new[0], exp_avgs_out=new[1], exp_avg_sqs_out=new[2])
    check_adam(before, (*new, None), None, t, 0.1, betas, 1e-8, 0.0, 1.0)
    # a step number that the device holds
    dev = [[torch.empty_like(x[0])] for x in (ps, ms, vs)]
    g.ar_adamw_step(ps, gs, ms, vs, 0.1, torch.tensor([t], device="cuda"), betas, params_out=dev[0], exp_avgs_out=dev[1],
                    exp_avg_sqs_out=dev[2])
    check_adam(before, (*dev, None), None, t, 0.1, betas, 1e-8, 0.0, 1.0, on_device=True)


def test_adamw_rates_on_the_device(g):
    """A captured step whose number and learning rate change between replays: each is that of the formula."""
    ps, gs, ms, vs, _ = adam_state([(500,), (33,)], "f32", "f32", False)
    lr, t = torch.empty(1, device="cuda"), torch.empty((), dtype=torch.int64, device="cuda")
    new = [[torch.empty_like(a) for a in x] for x in (ps, ms, vs)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.ar_adamw_step(ps, gs, ms, vs, lr, t, (0.9, 0.99), weight_decay=0.2, params_out=new[0], exp_avgs_out=new[1],
                        exp_avg_sqs_out=new[2])
    for rate, step in ((0.1, 1), (0.003, 40), (1e-5, 7)):
        lr.fill_(rate)
        t.fill_(step)
        graph.replay()
        check_adam((ps, gs, ms, vs, None), (*new, None), None, step, float(np.float32(rate)), (0.9, 0.99), 1e-8, 0.2, 1.0,
                   on_device=True)
    # the rate alone
    g.ar_adamw_step(ps, gs, ms, vs, lr, 7, (0.9, 0.99), weight_decay=0.2, params_out=new[0], exp_avgs_out=new[1],
                    exp_avg_sqs_out=new[2])
    check_adam((ps, gs, ms, vs, None), (*new, None), None, 7, float(np.float32(1e-5)), (0.9, 0.99), 1e-8, 0.2, 1.0,
               on_device=True)


def test_adamw_skips_a_step_that_is_not_finite(g):
    for master in (False, True):
        ps, gs, ms, vs, ws = adam_state([(100,), (4097,), (33,)], "bf16", "bf16", master)
        if master:
            for p, w in zip(ps, ws):
                if w is not None:
                    p.copy_(w)
        gs[1][5] = float("nan")
        stats, _ = g.ar_grad_norm(gs, 1.0)
        keep = [[None if t is None else t.clone() for t in x] for x in (ps, ms, vs, ws or [None] * 3)]
        g.ar_adamw_step(ps, gs, ms, vs, 0.1, 1, weight_decay=0.1, clip=stats, masters=ws)
        new = [[torch.zeros_like(t) for t in x] for x in (ps, ms, vs)]
        wo = None if ws is None else [None if w is None else torch.zeros_like(w) for w in ws]
        g.ar_adamw_step(ps, gs, ms, vs, 0.1, 1, weight_decay=0.1, clip=stats, masters=ws, params_out=new[0],
                        exp_avgs_out=new[1], exp_avg_sqs_out=new[2], masters_out=wo)
        for x, y, k in zip((ps, ms, vs, ws or []), (*new, wo or []), keep):
            for a, b, c in zip(x, y, k):
                assert a is None or (torch.equal(a, c) and torch.equal(b, c))


def test_norm_and_step_together(g):
    """As a training step uses them: the coefficient read by the step is the one that clipping applies, in eager calls,
    on another stream and in a captured graph that advances its own step number."""
    ps, gs, ms, vs, _ = adam_state(LISTS["odd"], "f32", "f32", False)
    ref = [[t.clone() for t in x] for x in (ps, gs, ms, vs)]
    start = [[t.clone() for t in x] for x in (ps, ms, vs)]
    for t in range(1, 4):
        _, _, clipped = g.ar_grad_clip(ref[1], 0.05, grad_scale=0.5, outs=[torch.empty_like(x) for x in gs])
        g.ar_adamw_step(ref[0], clipped, ref[2], ref[3], 0.01, torch.tensor([t], device="cuda"))
        stats, _ = g.ar_grad_norm(gs, 0.05, grad_scale=0.5)
        g.ar_adamw_step(ps, gs, ms, vs, 0.01, torch.tensor([t], device="cuda"), grad_scale=0.5, clip=stats)
        for x, y in zip((ps, ms, vs), (ref[0], ref[2], ref[3])):
            assert all(torch.equal(a, b) for a, b in zip(x, y))
    for x, y in zip((ps, ms, vs), start):
        for a, b in zip(x, y):
            a.copy_(b)
    step, one = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.ones(1, dtype=torch.int64, device="cuda")
    lists = [g.TensorList(x) for x in (ps, gs, ms, vs)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(one)
        stats, _ = g.ar_grad_norm(lists[1], 0.05, grad_scale=0.5)
        g.ar_adamw_step(*lists, 0.01, step, grad_scale=0.5, clip=stats)
    for _ in range(3):
        graph.replay()
    for x, y in zip((ps, ms, vs), (ref[0], ref[2], ref[3])):
        assert all(torch.equal(a, b) for a, b in zip(x, y))
    assert g.ar_device_status() == g.AR_OK


def test_two_streams_with_workspaces_of_their_own(g):
    lists = [tensors(LISTS["long"], "f32", seed=s) for s in range(2)]
    want = [g.ar_grad_norm(ts, 1.0) for ts in lists]
    streams = [torch.cuda.Stream() for _ in lists]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got.append([g.ar_grad_norm(ts, 1.0, stream=s) for ts, s in zip(lists, streams)])
    torch.cuda.synchronize()
    for pair in got:
        for (a, b), (c, d) in zip(want, pair):
            assert torch.equal(a, c) and torch.equal(b, d)


def test_gradients_of_more_than_2_to_the_31_elements(g):
    t = torch.zeros((1 << 31) + 5, dtype=torch.bfloat16, device="cuda")
    t[-1] = 3.0
    t[7] = 4.0
    stats, _, _ = g.ar_grad_clip([t], 1.0, eps=0.0)
    assert stats[0].item() == 5.0 and abs(t[-1].item() - 0.6) < 0.6 * 2.0 ** -8 and t[-2].item() == 0.0
    del t
    torch.cuda.empty_cache()


def test_coefficients(g):
    """max_norm / (norm + eps), rounded once: against the quotient in 64 bits, over magnitudes and scales."""
    for size in (1e-35, 1e-12, 1.0, 3e15, 1e36):
        for scale in (1.0, 1e-3, -3.0):
            for kind in ("l2", "max"):
                t = torch.tensor([3.0, 4.0], device="cuda") * size
                for max_norm, eps in ((size, 0.0), (0.3 * size, size), (1e3 * size * abs(scale), 0.0), (float("inf"), 0.0)):
                    got = g.ar_grad_norm([t], max_norm, kind=kind, eps=eps, grad_scale=scale)[0].tolist()
                    want = G.norm([t.double().cpu().numpy()], max_norm, kind, eps, float(np.float32(scale)))[0]
                    # the quotient of pairs is off by some 2^-44, its rounding by 2^-24; the norm by its scale's too
                    assert abs(got[1] - want[1]) <= want[1] * 2.0 ** -23 and abs(got[0] - want[0]) <= want[0] * 2.0 ** -22
                    assert got[2:] == want[2:].tolist()
    zero = torch.zeros(5, device="cuda")
    assert g.ar_grad_norm([zero], 1.0, eps=0.0)[0].tolist() == [0.0, 1.0, 0.0, 1.0]
    big = torch.full((4,), 3e38, device="cuda")  # the scaled norm leaves fp32's range: finite elements all the same
    for kind in ("l2", "max"):
        stats = g.ar_grad_norm([big], 1.0, kind=kind, grad_scale=100.0)[0].tolist()
        assert stats[0] == float("inf") and stats[1] < 1e-38 and stats[2:] == [1.0, 1.0]


def test_a_tensor_named_twice_counts_twice(g):
    t = torch.tensor([3.0, 4.0], device="cuda")
    assert g.ar_grad_norm([t, t[:1]], 1.0)[0][0].item() == pytest.approx(34 ** 0.5, rel=2.0 ** -22)
    with pytest.raises(g.ArError):
        g.ar_grad_clip([t, t[:1]], 1.0)


def test_workspaces_that_hold_anything(g):
    lists = {name: tensors(LISTS[name], "mixed", shift=1) for name in LISTS}
    want = {name: [x.clone() for x in g.ar_grad_norm(ts, 1.0)] for name, ts in lists.items()}
    ws = torch.empty(g.ar_grad_workspace(1) // 4, device="cuda")
    for fill in (float("nan"), float("inf"), 0.0, None):
        for name, ts in lists.items():
            if fill is not None:
                ws.fill_(fill)
            for a, b in zip(g.ar_grad_norm(ts, 1.0, workspace=ws), want[name]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("n", [40, 41, 48, 49, 360, 361, 768, 769])
def test_lists_as_long_as_the_tables(g, n):
    """Lists at the lengths where launches change, with empty tensors among them: every tensor is seen once."""
    ts = tensors([(0,) if i % 5 == 3 else (100 + 7 * (i % 11),) for i in range(n)], "bf16", seed=n)
    stats, norms, outs = g.ar_grad_clip(ts, 0.5, outs=[torch.zeros_like(t) for t in ts])
    want, each = G.norm(wide(ts), 0.5)
    assert np.allclose(norms.cpu().numpy(), each, rtol=NORM, atol=0)
    assert np.allclose(stats.cpu().numpy(), want, rtol=2 * NORM, atol=0)
    for t, o in zip(ts, outs):
        assert torch.equal(o, (t.float() * stats[1]).to(t.dtype))
    ps, ms, vs = ([torch.ones_like(t, dtype=torch.float32) for t in ts] for _ in range(3))
    g.ar_adamw_step(ps, ts, ms, vs, 0.1, 1, betas=(0.5, 0.5))
    for p, t, m in zip(ps, ts, ms):
        # (a gradient of -1 leaves the first moment, and so the weight, where it was; any other bf16 moves it by 1e-4 or more)
        assert torch.equal(m, 0.5 + 0.5 * t.float()) and torch.equal(p != 1.0, m != 0.0)


def test_short_lists_of_every_size(g):
    """Around the sizes where a cluster grows, and where one launch becomes three."""
    for granules in (1, 31, 32, 33, 2047, 2049, 8191, 8193, 16385, 130000, 131072, 131073, 140000):
        t = torch.randn(granules * 8, device="cuda").bfloat16()
        for cut in (0, 3):
            x = t[cut:t.numel() - cut]
            out = torch.empty(x.numel() + 8, dtype=torch.bfloat16, device="cuda")[cut:cut + x.numel()]
            stats, norms, _ = g.ar_grad_clip([x], 1e-3, outs=[out])
            want = torch.linalg.vector_norm(x.double()).item()
            assert abs(stats[0].item() - want) <= want * NORM and torch.equal(norms, stats[:1])
            assert torch.equal(out, (x.float() * stats[1]).bfloat16())
