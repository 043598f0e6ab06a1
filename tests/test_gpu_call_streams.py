"""Calls on a stream that is not the current one, with the workspaces and outputs that the binding makes."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def flat(outs):
    return [t for o in outs for t in (flat(o) if isinstance(o, (list, tuple)) else [o])]


@pytest.mark.parametrize("raw", [False, True])
def test_memory_of_a_call_is_not_handed_out_while_it_runs(g, raw):
    """The call waits on its stream while the current one asks for memory of the same sizes and fills it."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    rows, vocab, shape = 40, 500, (96, 120)
    x = torch.randn(rows, vocab, generator=gen, device="cuda")
    labels = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    lp = g.ar_token_logp(x, labels)
    ref = lp + 0.1
    start = torch.tensor([0, 9, 20, 33, rows], device="cuda")
    m = torch.randn(shape, generator=gen, device="cuda")
    plan = g.ar_ortho_plan([shape])
    params, momenta = torch.zeros_like(m), torch.zeros_like(m)

    def calls(stream):
        at = dict(params_out=[torch.empty_like(m)], momenta_out=[torch.empty_like(m)])
        outs = [g.ar_token_logp(x, labels, stream=stream),
                g.ar_policy_loss(x, labels, lp, lp, start, stream=stream),
                g.ar_preference_loss(x, labels, ref, start, stream=stream),
                g.ar_orthogonalize(plan, [m], stream=stream)]
        g.ar_muon_step(plan, [params], [m], [momenta], lr=0.1, stream=stream, **at)
        return flat(outs) + at["params_out"] + at["momenta_out"]

    want = calls(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(10_000_000)  # some milliseconds
        got = calls(side.cuda_stream if raw else side)
        sizes = {t.numel() * t.element_size() for t in want}
        sizes |= {g.ar_loss_workspace(rows, 1), g.ar_loss_workspace(rows, 4), g.ar_ortho_workspace(plan)}
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(6)]
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del junk, got
    assert g.ar_device_status() == g.AR_OK
