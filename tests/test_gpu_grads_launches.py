"""Norm and clipping at the sizes where one launch becomes several."""

import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def test_lists_around_the_sizes_where_launches_change(g):
    """Lists of up to 98304 granules of 16 bytes for a norm, 32768 for clipping, a tensor counting as 512 more, take one
    launch, which leaves the workspace as it is."""
    ws = torch.empty(g.ar_grad_workspace(1), dtype=torch.uint8, device="cuda")
    for most, clip in ((98304, False), (32768, True)):
        for tensors in (1, 3):
            for more in (-1, 0, 1, 40):
                granules = most - 512 * tensors + more
                for kind, per in ((torch.bfloat16, 8), (torch.float32, 4)):
                    sizes = [granules // tensors] * (tensors - 1)
                    sizes.append(granules - sum(sizes))
                    for cut in (0, 3):
                        ts = [torch.randn(n * per, device="cuda").to(kind)[cut:n * per - cut] for n in sizes]
                        outs = [torch.empty(n * per, device="cuda", dtype=kind)[cut:n * per - cut] for n in sizes]
                        ws.fill_(0x77)
                        if clip:
                            stats, norms, _ = g.ar_grad_clip(ts, 1e-3, outs=outs, workspace=ws)
                        else:
                            stats, norms = g.ar_grad_norm(ts, 1e-3, workspace=ws)
                        assert (ws == 0x77).all().item() == (more <= 0), (most, tensors, more, kind, cut)
                        each = torch.stack([torch.linalg.vector_norm(t.double()) for t in ts])
                        # (batches of 64 squares in fp32: 2^-20 of a root)
                        assert ((norms.double() - each).abs() <= each * 2.0 ** -20).all()
                        assert abs(stats[0].item() - each.norm().item()) <= each.norm().item() * 2.0 ** -20
                        for t, o in zip(ts, outs if clip else []):
                            assert torch.equal(o, (t.float() * stats[1]).to(kind))


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("where", ["elsewhere", "in place", "some in place", "another alignment"])
@pytest.mark.parametrize("tensors", [3, 900])
def test_clipping_of_lists_larger_than_the_l2(g, kind, shift, where, tensors):
    """Lists whose parts are kept in the L2 or not between norm and scaling, one launch or two: clipped, not clipped, and
    with a gradient that is not finite."""
    n = (200 << 20) // kind.itemsize // tensors
    flat = [torch.empty(tensors * n + 16, dtype=kind, device="cuda") for _ in range(2)]
    flat[0].normal_(generator=torch.Generator(device="cuda").manual_seed(tensors))
    ts = [flat[0][shift + i * n:shift + (i + 1) * n] for i in range(tensors)]
    more = 1 if where == "another alignment" else 0
    other = [flat[1][shift + more + i * n:shift + more + (i + 1) * n] for i in range(tensors)]
    keep = flat[0].clone()
    for bound, bad in ((1e-3, False), (float("inf"), False), (1.0, True)):
        if bad:
            ts[tensors // 2][n // 3] = float("nan")
            keep.copy_(flat[0])
        flat[1].fill_(7.0)
        outs = {"in place": ts, "some in place": [t if i % 2 else o for i, (t, o) in enumerate(zip(ts, other))]}.get(where, other)
        stats, _, _ = g.ar_grad_clip(ts, bound, outs=None if where == "in place" else outs)
        assert stats[3].item() == (0.0 if bad else 1.0) and stats[2].item() == float(bound != float("inf"))
        want = (keep.float() * stats[1]).to(kind) if not bad else torch.zeros_like(keep)
        for i, o in enumerate(outs):
            assert torch.equal(o, want[shift + i * n:shift + (i + 1) * n])
        if outs is other:
            assert torch.equal(flat[0].view(torch.uint8), keep.view(torch.uint8))
            # nothing beside the outputs
            lo, hi = shift + more, shift + more + tensors * n
            assert (flat[1][:lo] == 7.0).all() and (flat[1][hi:] == 7.0).all()
        flat[0].copy_(keep)


BEHIND = """
import torch
import gradient_sync_gb300 as g

ts = g.TensorList([torch.randn(1 << 24, device="cuda") for _ in range(4)])
outs = g.TensorList([torch.empty_like(t) for t in ts.tensors])
x = torch.ones(20 << 20, device="cuda")


def behind(call):
    times = []
    for _ in range(30):
        call()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(6):
            x.mul_(1.0)
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    return sorted(times)[len(times) // 2]


print(behind(lambda: g.ar_grad_norm(ts, 1.0)))
print(behind(lambda: g.ar_grad_clip(ts, float("inf"))))
for bad in (False, True):
    if bad:
        ts.tensors[1][5] = float("nan")
    g.ar_grad_clip(ts, 1.0, outs=outs)
    print(behind(lambda: g.ar_grad_norm(ts, 1.0)))
"""


def test_what_runs_behind_a_clip_has_the_l2(g):
    """Passes over 80 MB, of which the L2 holds most, take as long behind clips that scale nothing, or behind norms after a clip,
    as before any clip: in a process of its own, in which there has been none. (Lines left with a priority in the L2 make
    them 1.2 times as long.)"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(g.__file__)))
    run = subprocess.run([sys.executable, "-c", BEHIND], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr
    alone, *rest = (float(v) for v in run.stdout.split())
    assert len(rest) == 3 and max(rest) < 1.12 * alone, (alone, rest)
