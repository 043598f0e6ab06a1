"""What the binding of the losses and of the optimiser takes from tensors, without a GPU: host
tensors stand in for device ones, and the library's calls are recorded in place of being made."""

import pytest
import torch


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


class Device:
    """A host tensor that calls itself a device tensor."""

    def __init__(self, t):
        self.t = t

    is_cuda = True
    device = torch.device("cpu")  # where tensors made beside it go

    def __getattr__(self, name):
        return getattr(self.t, name)


def overlapping(which):
    """2 x 8 tensors whose rows share memory: one row twice, rows one apart, rows that share one element."""
    flat = torch.zeros(16)
    return flat[:8].expand(2, 8) if which == 0 else flat.as_strided((2, 8), (1 if which == 1 else 7, 1))


@pytest.mark.parametrize("which", [0, 1, 2])
def test_rows_that_share_memory_are_refused(g, which):
    """A row stride below the width is no row stride that a kernel could use, on inputs and outputs alike."""
    x = Device(overlapping(which))
    good = Device(torch.zeros(2, 8))
    labels = Device(torch.zeros(2, dtype=torch.int64))
    row, start = Device(torch.zeros(2)), Device(torch.tensor([0, 1, 2]))
    with pytest.raises(ValueError, match="logits"):
        g.ar_token_logp(x, labels)
    with pytest.raises(ValueError, match="dlogits"):
        g.ar_policy_loss(good, labels, row, row, dlogits=x)
    with pytest.raises(ValueError, match="dlogits"):
        g.ar_preference_loss(good, labels, row, start, dlogits=x)
    plan = g.ar_ortho_plan([(2, 8)])
    with pytest.raises(ValueError, match="matrices"):
        g.ar_orthogonalize(plan, [x], outs=[good])
    with pytest.raises(ValueError, match="outs"):
        g.ar_orthogonalize(plan, [good], outs=[x])
    for bad in ("params", "grads", "momenta", "params_out", "momenta_out"):
        with pytest.raises(ValueError, match=bad):
            g.ar_muon_step(plan, **{**{k: [good] for k in ("params", "grads", "momenta")}, bad: [x]}, lr=0.1)


def test_strides_that_no_row_uses(g):
    """Of a single row, or none, the stride may be anything; rows of one element may be adjacent or
    apart."""
    flat = torch.zeros(64)
    for t, ld in ((flat.as_strided((1, 8), (0, 1)), 8), (flat.as_strided((1, 8), (3, 1)), 8),
                  (flat.as_strided((0, 8), (0, 1)), 8), (flat.as_strided((4, 1), (1, 7)), 1),
                  (flat.as_strided((4, 1), (9, 0)), 9), (flat.as_strided((4, 8), (11, 1)), 11)):
        assert g._row_major(Device(t), "x") == ld
    with pytest.raises(ValueError):
        g._row_major(Device(flat[:1].expand(4, 1)), "x")


def test_workspaces_that_the_kernels_could_not_use(g):
    """A workspace in host memory, one with gaps (whose size is not its extent), and one that is too small."""
    x, labels, row = (Device(t) for t in (torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64), torch.zeros(2)))
    start = Device(torch.tensor([0, 1, 2]))
    plan = g.ar_ortho_plan([(2, 8)])
    forward = dict(grad=False)
    calls = [(g.ar_loss_workspace(2, 1), lambda w: g.ar_policy_loss(x, labels, row, row, workspace=w, **forward)),
             (g.ar_loss_workspace(2, 2), lambda w: g.ar_preference_loss(x, labels, row, start, workspace=w, **forward)),
             (g.ar_ortho_workspace(plan), lambda w: g.ar_orthogonalize(plan, [x], outs=[x], workspace=w)),
             (g.ar_ortho_workspace(plan), lambda w: g.ar_muon_step(plan, [x], [x], [x], lr=0.1, workspace=w))]
    for need, call in calls:
        room = torch.zeros(2 * need, dtype=torch.uint8)
        for bad in (room, Device(room[:need].expand(4, need)), Device(room[::2]), Device(room[:need - 1])):
            with pytest.raises(ValueError, match="workspace"):
                call(bad)


class Made(Device):
    """A tensor that the binding has made: under which current stream, and which other streams it was told of."""

    def __init__(self, t, stream):
        super().__init__(t)
        self.stream, self.told = stream, []

    def record_stream(self, stream):
        self.told.append(stream.cuda_stream)


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


@pytest.mark.parametrize("stream,owner", [(None, 64), (64, 64), (32, 32), (0, 0), (1, 0), (2, 2)])
def test_what_a_call_makes_belongs_to_its_stream(g, monkeypatch, stream, owner):
    """A workspace or an output that the binding makes is memory of the stream that the kernels run on: as
    memory of another one it would be handed out again, or still be in use there, while they run. Outputs are
    also known to the current stream, on which the caller reads them. (1 is another name of stream 0.)"""
    shapes = [(2, 8)]
    plan = g.ar_ortho_plan(shapes)
    g.ar_ortho_workspace(plan), g.ar_loss_workspace(2, 1), g.ar_loss_workspace(2, 2)
    x, labels, row = (Device(t) for t in (torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64), torch.zeros(2)))
    start = Device(torch.tensor([0, 1, 2]))
    now, made, calls = [64], [], []

    class Library:
        def __getattr__(self, name):
            return lambda *args: calls.append((name, args[-1])) or 0

    class Under:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            now.append(self.s.cuda_stream)

        def __exit__(self, *_):
            now.pop()

    real = torch.empty

    def empty(*shape, device, **kw):
        made.append(Made(real(*shape, **kw), now[-1]))
        return made[-1]

    monkeypatch.setattr(g._lib, "load", Library)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: Stream(now[-1]))
    monkeypatch.setattr(torch.cuda, "stream", Under)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    outputs = list(g.ar_policy_loss(x, labels, row, row, stream=stream))
    outputs += g.ar_preference_loss(x, labels, row, start, stream=stream)
    outputs.append(g.ar_token_logp(x, labels, stream=stream))
    outputs += g.ar_orthogonalize(plan, [x], stream=stream)
    g.ar_muon_step(plan, [x], [x], [x], lr=0.1, stream=stream)
    assert [c[0] for c in calls] == ["ar_policy_loss", "ar_preference_loss", "ar_token_logp", "ar_orthogonalize",
                                     "ar_muon_step"]
    assert all(c[1] == (64 if stream is None else stream) for c in calls)
    assert len(outputs) == 9 and len(made) == 13  # four workspaces
    assert all(m.stream == owner for m in made)
    assert all(m.told == ([64] if owner != 64 and any(m is o for o in outputs) else []) for m in made)
