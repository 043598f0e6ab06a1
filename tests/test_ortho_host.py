"""Plans and refusals of the orthogonalised update, without a GPU."""

import ctypes

import pytest

A = 1 << 30  # a stand-in device address: the calls below return before it is used


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def refused(g, code, *args, **kw):
    with pytest.raises(g.ArError) as e:
        g.ar_ortho_plan(*args, **kw)
    assert e.value.status == code


@pytest.mark.parametrize("kw", [dict(shapes=[]), dict(shapes=[(0, 3)]), dict(shapes=[(3, 0)]),
                                dict(shapes=[(2, (1 << 20) + 1)]), dict(in_dtype=5), dict(out_dtype=-1),
                                dict(steps=0), dict(steps=17), dict(eps=-1.0), dict(eps=float("nan")),
                                dict(precision=3), dict(steps=1, coefficients=[(float("inf"), 0, 0)])])
def test_bad_plans(g, kw):
    refused(g, g.AR_EINVAL, **{"shapes": [(4, 4)], **kw})


def test_unsupported_plans(g):
    refused(g, g.AR_EUNSUPPORTED, [(4, 4)] * (g.AR_MAX_MATRICES + 1))
    refused(g, g.AR_EUNSUPPORTED, [(4, 4)], steps=3, coefficients=[(4.0, 0.0, 0.0)] * 3)  # 64 times
    refused(g, g.AR_EUNSUPPORTED, [(4, 4)], steps=1, coefficients=[(20.0, -40.0, 20.5)])  # eigenvalues to -20
    g.ar_ortho_plan([(4, 4)] * g.AR_MAX_MATRICES, steps=16)
    g.ar_ortho_plan([(4, 4)], steps=2, coefficients=[(1.875, -1.25, 0.375)] * 2)


def test_null_arguments(g):
    lib, b = g._lib.load(), ctypes.c_size_t()
    plan = g.ar_ortho_plan([(4, 4)])
    assert lib.ar_ortho_plan(None, ctypes.c_void_p()) == g.AR_EINVAL
    assert lib.ar_ortho_workspace(None, b) == g.AR_EINVAL
    assert lib.ar_ortho_workspace(plan.handle, None) == g.AR_EINVAL
    lib.ar_ortho_plan_destroy(None)


def test_workspace_sizes(g):
    small, split = (g.ar_ortho_plan([(100, 200)], out_dtype=t) for t in ("bf16", "f32"))
    # X in 1 x 4 blocks of 16 KB, four of them; A and B in 1 x 2 blocks, once or twice each; one partial sum
    assert g.ar_ortho_workspace(small) == 16 * 4 * 4 * 1024 + 2 * 2 * 16384 + 256
    assert g.ar_ortho_workspace(split) == 16 * 4 * 4 * 1024 + 4 * 2 * 16384 + 256
    assert g.ar_ortho_workspace(g.ar_ortho_plan([(200, 100)], out_dtype="bf16")) == g.ar_ortho_workspace(small)


def arrays(g, specs):
    arr = (g._lib.ArMatrix * len(specs))()
    for i, (p, ld) in enumerate(specs):
        arr[i].data, arr[i].ld = p, ld
    return arr


@pytest.mark.parametrize("ins,outs,ws", [
    ([(A, 8)], [(0, 8)], 9 * A), ([(0, 8)], [(2 * A, 8)], 9 * A), ([(A + 2, 8)], [(2 * A, 8)], 9 * A),
    ([(A, 7)], [(2 * A, 8)], 9 * A), ([(A, 8)], [(2 * A, 3)], 9 * A), ([(A, 8)], [(2 * A, 8)], 0),
    ([(A, 8)], [(2 * A, 8)], 9 * A + 8), ([(A, 8)], [(A + 16, 8)], 9 * A), ([(A, 8)], [(2 * A, 8)], A),
    ([(A, 9)], [(A, 8)], 9 * A)])
def test_orthogonalize_refusals(g, ins, outs, ws):
    plan = g.ar_ortho_plan([(4, 8)])
    got = g._lib.load().ar_orthogonalize(plan.handle, arrays(g, ins), arrays(g, outs), ws, None)
    assert got == g.AR_EINVAL


def test_outputs_must_not_share_memory(g):
    plan = g.ar_ortho_plan([(4, 8), (4, 8)])
    ins = arrays(g, [(A, 16), (A + 32, 16)])  # side by side in one matrix: apart
    lib = g._lib.load()
    assert lib.ar_orthogonalize(plan.handle, ins, arrays(g, [(2 * A, 8), (2 * A + 64, 8)]), 9 * A, None) == g.AR_EINVAL
    side = arrays(g, [(2 * A, 16), (2 * A + 28, 16)])  # one column in common
    assert lib.ar_orthogonalize(plan.handle, ins, side, 9 * A, None) == g.AR_EINVAL


def muon(g, plan, desc=None, **kw):
    a = dict(params=[(A, 8)], grads=[(2 * A, 8)], momenta=[(3 * A, 8)], po=None, mo=None, ws=9 * A)
    a.update(kw)
    d = dict(lr=0.1, momentum=0.9, weight_decay=0.0, nesterov=1, adjust=1, grad_scale=1.0)
    d.update(desc or {})
    m = {k: arrays(g, v) if v else None for k, v in a.items() if k != "ws"}
    return g._lib.load().ar_muon_step(plan.handle, g._lib.ArMuonDesc(*d.values()), m["params"], m["grads"],
                                      m["momenta"], m["po"], m["mo"], a["ws"], None)


@pytest.mark.parametrize("kw", [dict(params=None), dict(grads=None), dict(momenta=None), dict(grads=[(A, 8)]),
                                dict(momenta=[(A + 64, 8)]), dict(momenta=[(3 * A + 2, 8)]), dict(mo=[(2 * A, 8)]),
                                dict(po=[(3 * A, 8)]), dict(po=[(A, 9)]), dict(mo=[(0, 8)]), dict(ws=0),
                                dict(ws=3 * A)])
def test_muon_refusals(g, kw):
    assert muon(g, g.ar_ortho_plan([(4, 8)]), **kw) == g.AR_EINVAL


@pytest.mark.parametrize("bad", [dict(lr=float("nan")), dict(momentum=float("inf")), dict(weight_decay=float("nan")),
                                 dict(adjust=3), dict(grad_scale=float("inf"))])
def test_muon_descriptor_refusals(g, bad):
    assert muon(g, g.ar_ortho_plan([(4, 8)]), desc=bad) == g.AR_EINVAL


def test_binding_refuses_other_tensors(g):
    import torch

    plan = g.ar_ortho_plan([(4, 8)])
    with pytest.raises(ValueError):
        g.ar_orthogonalize(plan, [torch.zeros(4, 8)] * 2, outs=[torch.zeros(4, 8)] * 2)
    with pytest.raises(ValueError):
        g.ar_orthogonalize(plan, [torch.zeros(4, 8)], outs=[torch.zeros(4, 8)])  # not on a GPU
    with pytest.raises(ValueError):
        g.ar_ortho_plan([(4, 8)], steps=2, coefficients=[(1, 1, 1)])
