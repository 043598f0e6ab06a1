"""Norm and clipping at the sizes where one launch becomes several."""

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
