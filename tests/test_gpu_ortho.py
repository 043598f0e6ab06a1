"""The orthogonalised update on a GB300 against its oracle in 64 bits.

Bounds. HALF: a step computes B X from operands rounded to fp16 (u = 2^-11 at
most, u / sqrt(3) in the mean square, two operands), with |B| <= 2.9 and
|X|_F <= 1.2 sqrt(m); and B from A rounded once, with |b + 2 c lambda| <= 4.8
over |A|_F <= 1.45 sqrt(m): at most
(2.9 * 1.2 * 2 + 4.8 * 1.45 / 2) * 2^-12 / sqrt(3) * sqrt(m) < 1.5e-3 sqrt(m).
Errors of early steps sit in directions that later ones carry towards 1 with a
slope of at most 1 by the end; four such steps' worth bounds the sum: 6e-3.
SPLIT: operands to 2^-22 and fp32 sums of up to 8192 / 16 terms: 3e-5.
Both relative to sqrt(m), the norm of an orthogonal m x n matrix; single
elements within 12 times the mean square. bf16 results add half an ulp: their
spacing is 2^-7 of the power of two below, so half of it is at most 2^-8 of the
value.
"""

import numpy as np
import pytest
import torch

from oracle import ortho

pytestmark = pytest.mark.gpu

HALF, SPLIT = 6e-3, 3e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def host(t):
    return t.double().cpu().numpy()


def check(got, want, precision, rounded=0.0, factor=1.0):
    """`got` against `want`, errors measured against factor * sqrt(m) for an m x n matrix."""
    r, c = want.shape
    tol = (HALF if precision == "half" else SPLIT) * factor
    err = host(got) - want
    room = rounded * np.abs(want)
    over = np.maximum(np.abs(err) - room, 0)
    assert np.sqrt((over**2).sum()) <= tol * min(r, c) ** 0.5, np.sqrt((over**2).sum()) / min(r, c) ** 0.5
    assert over.max() <= 12 * tol / max(r, c) ** 0.5, over.max() * max(r, c) ** 0.5


def matrix(rng, r, c, dtype, kind="noise"):
    u = rng.normal(size=(r, c))
    if kind == "decay":  # a spectrum falling like 1 / k
        k = min(r, c)
        q1, q2 = np.linalg.qr(rng.normal(size=(r, k)))[0], np.linalg.qr(rng.normal(size=(c, k)))[0]
        u = (q1 / np.arange(1, k + 1)) @ q2.T
    return torch.tensor(u * 1e-3, dtype=TYPES[dtype], device="cuda")


SHAPES = [[(1, 1)], [(1, 300)], [(300, 1)], [(7, 5)], [(64, 64)], [(128, 128)], [(129, 127)], [(130, 700)],
          [(700, 130)], [(255, 257)], [(256, 256)], [(400, 1000)], [(513, 385)], [(17, 4099)], [(640, 640)],
          [(33, 65), (300, 200), (128, 512), (1, 2), (200, 300)]]


@pytest.mark.parametrize("shapes", SHAPES)
@pytest.mark.parametrize("precision,src,dst", [("half", "bf16", "bf16"), ("half", "f32", "f32"), ("split", "f32", "f32"),
                                               ("split", "bf16", "bf16")])
def test_shapes(g, shapes, precision, src, dst):
    rng = np.random.default_rng(len(shapes) * 1000 + shapes[0][0])
    mats = [matrix(rng, r, c, src) for r, c in shapes]
    plan = g.ar_ortho_plan(shapes, src, dst, precision=precision)
    for m, o in zip(mats, g.ar_orthogonalize(plan, mats)):
        assert o.dtype == TYPES[dst]
        check(o, ortho.newton_schulz(host(m)), precision, 2.0**-8 if dst == "bf16" else 0)
    assert g.ar_device_status() == g.AR_OK


def test_auto_precision_and_decaying_spectrum(g):
    rng = np.random.default_rng(3)
    for dst, precision in (("f32", "split"), ("bf16", "half")):
        m = matrix(rng, 300, 420, "f32", "decay")
        out = g.ar_orthogonalize(g.ar_ortho_plan([(300, 420)], "f32", dst), [m])[0]
        check(out, ortho.newton_schulz(host(m)), precision, 2.0**-8 if dst == "bf16" else 0)


@pytest.mark.parametrize("steps", [1, 2, 3, 7])
def test_steps_and_coefficients(g, steps):
    rng = np.random.default_rng(steps)
    m = matrix(rng, 200, 333, "f32")
    coef = [(1.875, -1.25, 0.375), (3.4445, -4.7750, 2.0315), (2.0, -1.5, 0.5)]
    coef = [coef[k % 3] for k in range(steps)]
    plan = g.ar_ortho_plan([(200, 333)], steps=steps, coefficients=coef, eps=1e-3)
    want = ortho.newton_schulz(host(m), steps=steps, coefficients=np.float32(coef).astype(np.float64), eps=np.float32(1e-3))
    check(g.ar_orthogonalize(plan, [m])[0], want, "split")


def test_scale_of_the_input_does_not_matter(g):
    """Power-of-two factors change neither the fp16 halves nor, at eps = 0, the result's bits."""
    rng = np.random.default_rng(5)
    m = matrix(rng, 150, 260, "f32")
    plan = g.ar_ortho_plan([(150, 260)], eps=0.0)
    a = g.ar_orthogonalize(plan, [m])[0]
    for f in (2.0**-40, 2.0**40):
        assert torch.equal(a, g.ar_orthogonalize(plan, [m * f])[0])


@pytest.mark.parametrize("shape", [(130, 200), (200, 130)])
def test_strided_views_and_in_place(g, shape):
    r, c = shape
    rng = np.random.default_rng(8)
    joint = torch.tensor(rng.normal(size=(r, 2 * c + 5)), dtype=torch.float32, device="cuda")
    keep = joint.clone()
    views = [joint[:, 1:1 + c], joint[:, c + 3:2 * c + 3]]  # two projections in one matrix
    plan = g.ar_ortho_plan([shape, shape])
    apart = g.ar_orthogonalize(plan, [v.contiguous() for v in views])
    outs = g.ar_orthogonalize(plan, views, outs=views)
    for v, a in zip(outs, apart):
        assert torch.equal(v, a)
    for cols in (slice(0, 1), slice(1 + c, c + 3), slice(2 * c + 3, None)):
        assert torch.equal(joint[:, cols], keep[:, cols])


def test_zero_and_not_finite(g):
    shapes = [(140, 150)] * 4
    mats = [torch.zeros(140, 150, device="cuda") for _ in shapes]
    for m in mats[1:]:
        m.normal_()
    mats[2][3, 7] = float("nan")
    mats[3][0, 0] = float("inf")
    out = g.ar_orthogonalize(g.ar_ortho_plan(shapes), mats)
    assert not out[0].any()
    check(out[1], ortho.newton_schulz(host(mats[1])), "split")
    assert torch.isnan(out[2]).all() and torch.isnan(out[3]).all()


@pytest.mark.parametrize("src,dst", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("nesterov,adjust", [(True, "shape"), (False, "rms"), (True, "none")])
def test_muon_step(g, src, dst, nesterov, adjust):
    shapes = [(300, 100), (100, 300), (129, 257), (64, 2000)]
    rng = np.random.default_rng(12)
    grads = [matrix(rng, r, c, src) for r, c in shapes]
    params = [torch.tensor(rng.normal(size=s) * 0.02, dtype=TYPES[dst], device="cuda") for s in shapes]
    momenta = [torch.tensor(rng.normal(size=s) * 2e-3, dtype=torch.float32, device="cuda") for s in shapes]
    kw = dict(lr=0.02, momentum=0.9, weight_decay=0.1, nesterov=nesterov, adjust=adjust, grad_scale=0.125)
    want = [ortho.muon_step(host(p), host(q), host(m), **kw) for p, q, m in zip(params, grads, momenta)]
    plan = g.ar_ortho_plan(shapes, src, dst)
    po, mo = [torch.empty_like(p) for p in params], [torch.empty_like(m) for m in momenta]
    g.ar_muon_step(plan, params, grads, momenta, params_out=po, momenta_out=mo, **kw)
    for s, p, m, (w, m64), p0 in zip(shapes, po, mo, want, params):
        assert np.abs(host(m) - m64).max() <= 2.0**-22 * np.abs(m64).max()
        factor = 0.02 * ortho.adjust_factor(*s, adjust)
        # the weights' own rounding: 2^-24 of the weight and of the decayed one, or half a bf16 ulp
        check(p, w, "half" if dst == "bf16" else "split", 2.0**-8 if dst == "bf16" else 2.0**-22, factor)
    # in place
    g.ar_muon_step(plan, params, grads, momenta, **kw)
    assert all(torch.equal(a, b) for a, b in zip(params + momenta, po + mo))


def test_many_matrices(g):
    """More matrices than the short launch table holds, all sizes apart."""
    rng = np.random.default_rng(4)
    shapes = [(int(rng.integers(1, 300)), int(rng.integers(1, 300))) for _ in range(40)]
    mats = [matrix(rng, r, c, "f32") for r, c in shapes]
    for m, o in zip(mats, g.ar_orthogonalize(g.ar_ortho_plan(shapes), mats)):
        check(o, ortho.newton_schulz(host(m)), "split")


@pytest.mark.parametrize("precision,dst", [("half", "bf16"), ("split", "f32")])
def test_large(g, precision, dst):
    """Several tiles a CTA, all of the pipelines' phases; the oracle on the device, in 64 bits."""
    shapes = [(2048, 2048), (1024, 4096), (3000, 1100), (2900, 1290), (100, 4500)]
    gen = torch.Generator(device="cuda").manual_seed(1)
    mats = [torch.randn(s, generator=gen, device="cuda") for s in shapes]
    outs = g.ar_orthogonalize(g.ar_ortho_plan(shapes, "f32", dst, precision=precision), mats)
    for m, o in zip(mats, outs):
        x = m.double() / (m.double().norm() + 1e-7)
        x = x.T if x.shape[0] > x.shape[1] else x
        for _ in range(5):
            a = x @ x.T
            x = 3.4445 * x + (-4.7750 * a + 2.0315 * a @ a) @ x
        x = x.T if m.shape[0] > m.shape[1] else x
        check(o, x.cpu().numpy(), precision, 2.0**-8 if dst == "bf16" else 0)


def test_repeatable_streams_and_graph(g):
    rng = np.random.default_rng(6)
    shapes = [(400, 500), (96, 1000)]
    mats = [matrix(rng, r, c, "bf16") for r, c in shapes]
    plan = g.ar_ortho_plan(shapes, "bf16", "bf16")
    want = g.ar_orthogonalize(plan, mats)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = [g.ar_orthogonalize(plan, mats) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(s)
    for outs in again:
        assert all(torch.equal(a, b) for a, b in zip(want, outs))
    ws = torch.empty(g.ar_ortho_workspace(plan), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(o) for o in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.ar_orthogonalize(plan, mats, outs=outs, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_refuses_while_a_timeout_is_recorded(g):
    plan = g.ar_ortho_plan([(8, 8)])
    m = [torch.ones(8, 8, device="cuda")]
    assert g.ar_device_status() == g.AR_OK
    g.ar_selftest_wait_timeout(polls=1000)
    torch.cuda.synchronize()
    with pytest.raises(g.ArError) as e:
        g.ar_orthogonalize(plan, m)
    assert e.value.status == g.AR_ETIMEOUT and g.ar_device_status() == g.AR_ETIMEOUT
    g.ar_orthogonalize(plan, m)
    torch.cuda.synchronize()
    assert g.ar_device_status() == g.AR_OK
