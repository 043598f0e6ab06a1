"""GB300 gradient all-reduce over N virtual ranks held in one GPU's memory.

A thin Python binding of libar_gb300.so: the functions below carry the C
ABI's names (include/ar.h) and only marshal arguments -- torch tensors or raw
integer device pointers in, status codes out as exceptions. Every step of the
all-reduce runs in the library's CUDA kernels; there is no Python or CPU
fallback, and importing a function whose library is missing raises.
"""

from __future__ import annotations

import ctypes
import functools

from . import _lib

# ---- enums of include/ar.h
AR_OK, AR_EINVAL, AR_EUNSUPPORTED, AR_ENOMEM, AR_ECUDA, AR_ETIMEOUT = range(6)
AR_F32, AR_BF16 = 0, 1
AR_RING, AR_RABENSEIFNER, AR_HIER, AR_FUSED, AR_AUTO = 0, 1, 2, 3, 4
AR_ORDER_RING, AR_ORDER_RANK, AR_ORDER_TREE, AR_ORDER_HIER = 0, 1, 2, 3
AR_ALLREDUCE, AR_REDUCE_SCATTER, AR_ALLGATHER = 0, 1, 2
AR_KERNEL_AUTO, AR_KERNEL_LOADS, AR_KERNEL_BULK = 0, 1, 2
AR_MAX_RANKS = 64
AR_MAX_BUCKET_TENSORS = 32

AR_RECDOUBLING, AR_DBTREE, AR_TORUS = 5, 6, 7
ALGOS = {"ring": AR_RING, "rabenseifner": AR_RABENSEIFNER, "hier": AR_HIER, "fused": AR_FUSED, "auto": AR_AUTO,
         "recdoubling": AR_RECDOUBLING, "dbtree": AR_DBTREE, "torus": AR_TORUS}
ALGO_NAMES = {v: k for k, v in ALGOS.items()}
AR_DEVICE_ALPHA_S, AR_DEVICE_BW, AR_DEVICE_CTA_STEP_S, AR_DEVICE_CTA_STEP_MEM_S = 1.5e-6, 6.0e12, 0.28e-6, 0.75e-6
ORDERS = {"ring": AR_ORDER_RING, "rank": AR_ORDER_RANK, "tree": AR_ORDER_TREE, "hier": AR_ORDER_HIER}
DTYPES = {"f32": AR_F32, "bf16": AR_BF16}
COLLECTIVES = {"allreduce": AR_ALLREDUCE, "reduce_scatter": AR_REDUCE_SCATTER, "allgather": AR_ALLGATHER}
KERNELS = {"auto": AR_KERNEL_AUTO, "loads": AR_KERNEL_LOADS, "bulk": AR_KERNEL_BULK}
LOSS_MEANS = {"token": 0, "sequence": 1}
PREFERENCE_FORMS = {"sigmoid": 0, "square": 1}
PRECISIONS = {"auto": 0, "half": 1, "split": 2}
ADJUSTS = {"none": 0, "shape": 1, "rms": 2}
AR_MAX_MATRICES = 192
KERNEL_NAMES = {v: k for k, v in KERNELS.items()}


class ArError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {ar_status_string(status)}" if what else ar_status_string(status))


def _check(status: int, what: str):
    if status != AR_OK:
        raise ArError(status, what)


def _ptr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _ptrs(xs):
    return _lib.ptr_array([_ptr(x) for x in xs])


def _stream(stream) -> int:
    if stream is None:
        import torch

        if torch.cuda.is_initialized():  # without the Stream object, which takes longer to make than a call to enqueue
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


# ---------------------------------------------------------------- plans


class Plan:
    """An ar_plan_t*; destroyed with the object."""

    def __init__(self, handle: int, desc: dict):
        self.handle = handle
        self.desc = desc

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h:
            try:
                _lib.load().ar_plan_destroy(h)
            except Exception:
                pass

    @property
    def stats(self) -> dict:
        return ar_plan_stats(self)


def ar_plan(n_ranks: int, count: int, dtype="f32", algo="fused", group_size: int = 0, order="ring",
            scale: float = 1.0, collective="allreduce", sm_budget: int = 0, kernel="auto",
            torus_dims=(0, 0, 0)) -> Plan:
    """Validate the descriptor and build the schedule (host only)."""
    dims = (list(torus_dims) + [0, 0, 0])[:3]
    d = _lib.ArDesc(int(n_ranks), int(count), DTYPES.get(dtype, dtype), ALGOS.get(algo, algo),
                    int(group_size), ORDERS.get(order, order), float(scale),
                    COLLECTIVES.get(collective, collective), int(sm_budget), KERNELS.get(kernel, kernel),
                    (_lib.c_int * 3)(*[int(v) for v in dims]))
    h = _lib.c_void_p()
    _check(_lib.load().ar_plan(d, h), "ar_plan")
    return Plan(h.value, dict(n_ranks=n_ranks, count=count, dtype=dtype, algo=algo, group_size=group_size,
                              order=order, scale=scale, collective=collective, sm_budget=sm_budget,
                              kernel=kernel, torus_dims=tuple(dims)))


def ar_plan_desc(plan: Plan) -> dict:
    """The plan's descriptor as the library holds it (AR_AUTO resolved)."""
    d = _lib.ArDesc()
    _check(_lib.load().ar_plan_desc(plan.handle, d), "ar_plan_desc")
    return {"n_ranks": d.n_ranks, "count": d.count, "dtype": d.dtype, "algo": ALGO_NAMES.get(d.algo, d.algo),
            "group_size": d.group_size, "order": d.order, "scale": d.scale, "collective": d.collective,
            "sm_budget": d.sm_budget, "kernel": KERNEL_NAMES.get(d.kernel, d.kernel),
            "torus_dims": tuple(d.torus_dims)}


def fabric(alpha, bw_local, bw_net=None, ranks_per_server=0, in_network=False, shared_memory=False):
    """An ar_fabric: seconds per round, bytes/s inside and between servers."""
    return _lib.ArFabric(float(alpha), float(bw_local), float(bw_net if bw_net is not None else bw_local),
                         int(ranks_per_server), int(bool(in_network)), int(bool(shared_memory)))


def ar_plan_predict(plan: Plan, fab) -> float:
    """Predicted seconds of one ar_execute of the plan on a fabric (round model)."""
    t = ctypes.c_double()
    _check(_lib.load().ar_plan_predict(plan.handle, fab, t), "ar_plan_predict")
    return t.value


def ar_select(n_ranks, count, fab, dtype="f32", order="ring", scale=1.0, collective="allreduce"):
    """(algorithm name, group size, predicted seconds) of the fastest algorithm on a fabric."""
    d = _lib.ArDesc(int(n_ranks), int(count), DTYPES.get(dtype, dtype), AR_FUSED, 0, ORDERS.get(order, order),
                    float(scale), COLLECTIVES.get(collective, collective), 0)
    a, gs, t = _lib.c_int(), _lib.c_int(), ctypes.c_double()
    _check(_lib.load().ar_select(d, fab, a, gs, t), "ar_select")
    return ALGO_NAMES[a.value], gs.value, t.value


def ar_plan_stats(plan: Plan) -> dict:
    s = _lib.ArStats()
    _check(_lib.load().ar_plan_stats(plan.handle, s), "ar_plan_stats")
    return {f: getattr(s, f) for f, _ in _lib.ArStats._fields_}


def ar_plan_transfers(plan: Plan, step: int):
    """(op, [(src, dst, first, end), ...]) of one step of a step plan."""
    lib = _lib.load()
    op, n = _lib.c_int(), _lib.c_int()
    _check(lib.ar_plan_transfers(plan.handle, step, op, n, None, 0), "ar_plan_transfers")
    buf = (ctypes.c_int64 * max(1, 4 * n.value))()
    _check(lib.ar_plan_transfers(plan.handle, step, op, n, buf, n.value), "ar_plan_transfers")
    rows = [tuple(buf[4 * i: 4 * i + 4]) for i in range(n.value)]
    return ("reduce" if op.value == 0 else "copy"), rows


def ar_execute(plan: Plan, bufs, outs=None, workspace=None, stream=None):
    """Enqueue the all-reduce of the N device buffers ``bufs`` (in place unless ``outs``)."""
    o = _ptrs(outs) if outs is not None else None
    _check(_lib.load().ar_execute(plan.handle, _ptrs(bufs), o, _ptr(workspace), _stream(stream)),
           "ar_execute")


def ar_execute_host(plan: Plan, host_in, host_out, dev_bufs, workspace=None, stream=None):
    """All-reduce host buffers through device staging buffers; returns when done."""
    _check(_lib.load().ar_execute_host(plan.handle, _ptrs(host_in), _ptrs(host_out), _ptrs(dev_bufs),
                                       _ptr(workspace), _stream(stream)), "ar_execute_host")


AR_STATIC_WORKSPACE_BYTES = 64 << 20


def ar_execute_noalloc(plan: Plan, bufs, outs=None, stream=None):
    """ar_execute for callers that cannot allocate device memory: the workspace
    comes from a fixed array inside the library (AR_STATIC_WORKSPACE_BYTES).
    Calls share that array, so calls that overlap on the GPU race."""
    o = _ptrs(outs) if outs is not None else None
    _check(_lib.load().ar_execute_noalloc(plan.handle, _ptrs(bufs), o, _stream(stream)), "ar_execute_noalloc")


class Bound:
    """An ar_bound_t*: a plan bound to its buffers (a persistent collective).
    Keeps the buffers alive; destroyed with the object."""

    def __init__(self, handle: int, keep):
        self.handle = handle
        self._keep = keep

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h:
            try:
                _lib.load().ar_bound_destroy(h)
            except Exception:
                pass

    def execute(self, stream=None):
        ar_execute_bound(self, stream)


def ar_bind(plan: Plan, bufs, outs=None, workspace=None) -> Bound:
    """Validate the buffers once and record the plan's launches (see include/ar.h)."""
    o = _ptrs(outs) if outs is not None else None
    h = _lib.c_void_p()
    _check(_lib.load().ar_bind(plan.handle, _ptrs(bufs), o, _ptr(workspace), h), "ar_bind")
    return Bound(h.value, (list(bufs), None if outs is None else list(outs), workspace))


def ar_execute_bound(bound: Bound, stream=None):
    """Replay a bound all-reduce on ``stream`` (an int handle skips the torch lookup)."""
    _check(_lib.load().ar_execute_bound(bound.handle, _stream(stream)), "ar_execute_bound")


# ---------------------------------------------------------------- buckets


def _counts(counts):
    return (_lib.c_size_t * len(counts))(*[int(c) for c in counts])


def ar_bucket_plan(counts, elem_bytes: int, cap_bytes: int):
    """Returns (bucket_of_tensor list, n_buckets)."""
    n = len(counts)
    out = (_lib.c_int * n)()
    nb = _lib.c_int()
    _check(_lib.load().ar_bucket_plan(_counts(counts), n, int(elem_bytes), int(cap_bytes), out, nb),
           "ar_bucket_plan")
    return list(out), nb.value


class TensorTable:
    """The [rank][tensor] pointer table and element counts of the bucket calls,
    marshalled once. Pass it in place of the nested tensor list when the same
    gradients are synchronised again and again (as DDP does every step): the
    per-call cost is then independent of the number of tensors."""

    def __init__(self, tensors, counts=None):
        self.n_ranks = len(tensors)
        self.n_tensors = len(tensors[0])
        if counts is None:
            counts = [t.numel() for t in tensors[0]]
        self.counts = list(counts)
        self.c_ptrs = _lib.ptr_array([_ptr(t) for row in tensors for t in row])
        self.c_counts = _counts(self.counts)


def _marshal(tensors, counts):
    if isinstance(tensors, TensorTable):
        return tensors.n_ranks, tensors.c_ptrs, tensors.c_counts, tensors.n_tensors
    return len(tensors), _lib.ptr_array([_ptr(t) for row in tensors for t in row]), _counts(counts), len(counts)


def _buckets(bucket):
    """Bucket buffers: a list of tensors/pointers, or an already marshalled pointer array."""
    return bucket if isinstance(bucket, ctypes.Array) else _ptrs(bucket)


def ar_bucket_pack(tensors, counts, t_begin: int, t_end: int, in_dtype, bucket, stream=None):
    n, ptrs, cnt, nt = _marshal(tensors, counts)
    _check(_lib.load().ar_bucket_pack(n, ptrs, cnt, nt, t_begin, t_end, DTYPES.get(in_dtype, in_dtype),
                                      _buckets(bucket), _stream(stream)), "ar_bucket_pack")


def ar_bucket_unpack(bucket, scale: float, out_dtype, tensors, counts, t_begin: int, t_end: int,
                     stream=None):
    n, ptrs, cnt, nt = _marshal(tensors, counts)
    _check(_lib.load().ar_bucket_unpack(n, _buckets(bucket), float(scale), DTYPES.get(out_dtype, out_dtype),
                                        ptrs, cnt, nt, t_begin, t_end, _stream(stream)), "ar_bucket_unpack")


def ar_bucket_allreduce(tensors, counts, t_begin: int, t_end: int, dtype, scale: float, stream=None,
                        sm_budget: int = 0, kernel="auto"):
    n, ptrs, cnt, nt = _marshal(tensors, counts)
    _check(_lib.load().ar_bucket_allreduce(n, ptrs, cnt, nt, t_begin, t_end, DTYPES.get(dtype, dtype),
                                           float(scale), int(sm_budget), KERNELS.get(kernel, kernel),
                                           _stream(stream)), "ar_bucket_allreduce")


# ---------------------------------------------------------------- compression

AR_COMPRESS_MIN_BLOCK, AR_COMPRESS_MAX_BLOCK = 16, 1024


def ar_compress_sizes(count: int, block: int):
    """(number of scales, message bytes) of one rank's compressed message."""
    ns, mb = _lib.c_size_t(), _lib.c_size_t()
    _check(_lib.load().ar_compress_sizes(int(count), int(block), ns, mb), "ar_compress_sizes")
    return ns.value, mb.value


def ar_compress(grads, codes, scales, block: int, dtype="f32", residuals=None, count=None, stream=None):
    """Blockwise INT8 compression of every rank's gradient (with error feedback
    when ``residuals`` is given: read as e, overwritten with the new residual)."""
    n = len(grads)
    count = grads[0].numel() if count is None else count
    res = _ptrs(residuals) if residuals is not None else None
    _check(_lib.load().ar_compress(n, int(count), int(block), DTYPES.get(dtype, dtype), _ptrs(grads), res,
                                   _ptrs(codes), _ptrs(scales), _stream(stream)), "ar_compress")


def ar_compressed_reduce(codes, scales, outs, block: int, scale: float = 1.0, out_dtype="f32", count=None,
                         stream=None):
    """Sum the ranks' compressed messages in rank order into every ``outs[r]``."""
    n = len(codes)
    count = codes[0].numel() if count is None else count
    _check(_lib.load().ar_compressed_reduce(n, int(count), int(block), _ptrs(codes), _ptrs(scales), float(scale),
                                            DTYPES.get(out_dtype, out_dtype), _ptrs(outs), _stream(stream)),
           "ar_compressed_reduce")


def ar_compressed_allreduce(grads, block: int, dtype="f32", residuals=None, scale: float = 1.0, outs=None,
                            count=None, stream=None):
    """Compression and reduction in one pass (in place unless ``outs``)."""
    n = len(grads)
    count = grads[0].numel() if count is None else count
    res = _ptrs(residuals) if residuals is not None else None
    o = _ptrs(outs) if outs is not None else None
    _check(_lib.load().ar_compressed_allreduce(n, int(count), int(block), DTYPES.get(dtype, dtype), _ptrs(grads),
                                               res, float(scale), o, _stream(stream)), "ar_compressed_allreduce")


# ---------------------------------------------------------------- losses
# Calls run on `stream` (default: the current one). Outputs and workspaces that
# are not given are made for that stream; on another one the caller orders the
# streams before it reads the outputs, as for any call.


_KINDS: dict = {}  # torch type -> the library's, once torch is needed


def _torch_kinds() -> dict:
    if not _KINDS:
        import torch

        _KINDS.update({torch.float32: AR_F32, torch.bfloat16: AR_BF16})
    return _KINDS


def _dtype_of(t) -> int:
    """The library's type of a torch tensor; TypeError for any other type."""
    kind = _torch_kinds().get(t.dtype)
    if kind is None:
        raise TypeError(f"float32 or bfloat16 wanted, got {t.dtype}")
    return kind


def _vector(t, dtype, n: int, what: str) -> int:
    """The address of a contiguous device vector of one type and length."""
    if t.dtype is not dtype or t.dim() != 1 or t.shape[0] != n or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous {dtype} CUDA tensor of {n} elements wanted, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _row_major(t, what: str) -> int:
    """The row stride of a 2-D device tensor whose rows are contiguous and share no memory."""
    if t.dim() == 2 and t.is_cuda:
        (rows, cols), (ld, step) = t.shape, t.stride()
        if step == 1 or cols <= 1:
            if ld >= cols:
                return ld
            if rows <= 1:  # (the stride of a single row means nothing)
                return cols
    raise ValueError(f"{what}: a 2-D CUDA tensor with contiguous rows that share no memory wanted, got shape "
                     f"{tuple(t.shape)}, strides {t.stride()} on {t.device}")


def _logits(logits, labels, temperature):
    import torch

    ld = _row_major(logits, "logits")
    rows, vocab = logits.shape
    return _lib.ArLogits(logits.data_ptr(), rows, vocab, ld, _dtype_of(logits),
                         _vector(labels, torch.int64, rows, "labels"), temperature)


def _empty(shape, dtype, like, stream, read: bool = True):
    """A new tensor beside `like` for a call on `stream`: memory of that stream, so that the allocator
    neither hands it out again nor has it in use elsewhere while the call runs. What the caller reads on
    the current stream is known to that one too."""
    import torch

    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    handle = _stream(stream)
    if handle == 1:  # another name of the default stream
        handle = 0
    if handle == _stream(None):
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(torch.cuda.ExternalStream(handle, device=like.device)):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    if read:
        t.record_stream(torch.cuda.current_stream(like.device))
    return t


def _gradient(logits, dlogits, grad: bool, stream):
    """(tensor or None, address, row stride) of the gradient of the logits."""
    if dlogits is None:
        if not grad:
            return None, 0, 0
        dlogits = _empty(logits.shape, logits.dtype, logits, stream)
    elif dlogits.dtype is not logits.dtype or dlogits.shape != logits.shape:
        raise ValueError("dlogits: the logits' type and shape wanted")
    return dlogits, dlogits.data_ptr(), _row_major(dlogits, "dlogits")


def _output(t, n: int, like, what: str, stream):
    """An fp32 vector to write to, and its address."""
    import torch

    if t is None:
        t = _empty(n, torch.float32, like, stream)
        return t, t.data_ptr()
    return t, _vector(t, torch.float32, n, what)


@functools.lru_cache(maxsize=1024)
def ar_loss_workspace(rows: int, n_seq: int) -> int:
    """Device bytes that the two losses need for `rows` tokens in `n_seq` sequences."""
    b = _lib.c_size_t()
    _check(_lib.load().ar_loss_workspace(int(rows), int(n_seq), b), "ar_loss_workspace")
    return b.value


def _room(workspace, need: int, like, stream):
    """A workspace of at least `need` bytes, and its address."""
    if workspace is None:
        import torch

        workspace = _empty(need, torch.uint8, like, stream, read=False)
    elif (not workspace.is_cuda or not workspace.is_contiguous()
          or workspace.numel() * workspace.element_size() < need):
        raise ValueError(f"workspace: a contiguous CUDA tensor of at least {need} bytes wanted, got "
                         f"{workspace.numel() * workspace.element_size()} bytes on {workspace.device}, strides "
                         f"{workspace.stride()}")
    return workspace, workspace.data_ptr()


def ar_token_logp(logits, labels, temperature: float = 1.0, logp=None, stream=None):
    """Log-probabilities of the labelled tokens, [rows] fp32 (0 where the label
    is negative). `logits` [rows, vocab] fp32 or bf16, any row stride; `labels` int64."""
    d = _logits(logits, labels, temperature)
    logp, out = _output(logp, d.rows, logits, "logp", stream)
    _check(_lib.load().ar_token_logp(d, out, _stream(stream)), "ar_token_logp")
    return logp


def ar_policy_loss(logits, labels, old_logp, advantages, seq_start=None, ref_logp=None, clip_low: float = 0.2,
                   clip_high: float = 0.2, kl_coef: float = 0.0, temperature: float = 1.0, reduction="token",
                   denominator: float = 0.0, grad_scale: float = 1.0, grad: bool = True, stats=None, logp=None,
                   dlogits=None, workspace=None, stream=None):
    """Clipped policy loss with a KL term, and its gradient (see include/ar.h).

    Per-token `old_logp`, `advantages` and optional `ref_logp` are fp32 [rows];
    `seq_start` int64 [n_seq + 1] row offsets (None: one sequence). `dlogits`
    may be the logits themselves. Returns (stats [loss, surrogate, kl, clipped
    share], logp, dlogits or None)."""
    import torch

    d = _logits(logits, labels, temperature)
    rows, f32 = d.rows, torch.float32
    old, adv = _vector(old_logp, f32, rows, "old_logp"), _vector(advantages, f32, rows, "advantages")
    ref = 0 if ref_logp is None else _vector(ref_logp, f32, rows, "ref_logp")
    n_seq, start = 1, 0
    if seq_start is not None:
        n_seq = seq_start.shape[0] - 1 if seq_start.dim() else 0
        start = _vector(seq_start, torch.int64, n_seq + 1, "seq_start")
    dlogits, d_at, dld = _gradient(logits, dlogits, grad, stream)
    stats, stats_at = _output(stats, 4, logits, "stats", stream)
    logp, logp_at = _output(logp, rows, logits, "logp", stream)
    workspace, room = _room(workspace, ar_loss_workspace(rows, max(n_seq, 0)), logits, stream)
    desc = _lib.ArPolicyDesc(clip_low, clip_high, kl_coef, LOSS_MEANS.get(reduction, reduction), denominator, grad_scale)
    _check(_lib.load().ar_policy_loss(d, old, ref, adv, start, n_seq, desc, stats_at, logp_at, d_at, dld, room,
                                      _stream(stream)), "ar_policy_loss")
    return stats, logp, dlogits


def ar_preference_loss(logits, labels, ref_logp, seq_start, beta: float = 0.1, label_smoothing: float = 0.0,
                       loss="sigmoid", target: float = 0.5, length_normalized: bool = False,
                       temperature: float = 1.0, denominator: float = 0.0, grad_scale: float = 1.0,
                       grad: bool = True, stats=None, ratios=None, logp=None, dlogits=None, workspace=None,
                       stream=None):
    """Preference loss over paired log ratios, and its gradient (see include/ar.h).

    Sequences 2i and 2i + 1 of `seq_start` (int64 [n_seq + 1]) are the chosen
    and the rejected answer of pair i; `ref_logp` fp32 [rows]. Returns (stats
    [loss, chosen reward, rejected reward, accuracy], ratios, logp, dlogits or
    None)."""
    import torch

    d = _logits(logits, labels, temperature)
    rows, n_seq = d.rows, seq_start.shape[0] - 1 if seq_start.dim() else 0
    ref = _vector(ref_logp, torch.float32, rows, "ref_logp")
    start = _vector(seq_start, torch.int64, n_seq + 1, "seq_start")
    dlogits, d_at, dld = _gradient(logits, dlogits, grad, stream)
    stats, stats_at = _output(stats, 4, logits, "stats", stream)
    ratios, ratios_at = _output(ratios, max(n_seq, 0), logits, "ratios", stream)
    logp, logp_at = _output(logp, rows, logits, "logp", stream)
    workspace, room = _room(workspace, ar_loss_workspace(rows, max(n_seq, 0)), logits, stream)
    desc = _lib.ArPreferenceDesc(beta, PREFERENCE_FORMS.get(loss, loss), label_smoothing, target,
                                 1 if length_normalized else 0, denominator, grad_scale)
    _check(_lib.load().ar_preference_loss(d, ref, start, n_seq, desc, stats_at, ratios_at, logp_at, d_at, dld, room,
                                          _stream(stream)), "ar_preference_loss")
    return stats, ratios, logp, dlogits


# ---------------------------------------------------------------- optimiser


class OrthoPlan:
    """An ar_ortho_plan_t*; destroyed with the object."""

    def __init__(self, handle: int, shapes, in_dtype: int, out_dtype: int):
        self.handle, self.shapes, self.in_dtype, self.out_dtype = handle, shapes, in_dtype, out_dtype
        self.workspace_bytes = None

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h:
            try:
                _lib.load().ar_ortho_plan_destroy(h)
            except Exception:
                pass


def ar_ortho_plan(shapes, in_dtype="f32", out_dtype="f32", steps: int = 5, coefficients=None, eps: float = 1e-7,
                  precision="auto") -> OrthoPlan:
    """Plan the orthogonalised update of matrices of the given (rows, cols).

    `in_dtype`: matrices or gradients; `out_dtype`: results or weights.
    `coefficients`: `steps` triples (a, b, c), default the quintic of the Muon
    optimiser; see include/ar.h."""
    shapes = [(int(r), int(c)) for r, c in shapes]
    n = len(shapes)
    dims = [(ctypes.c_int64 * max(1, n))(*[s[d] for s in shapes]) for d in (0, 1)]
    coef = None
    if coefficients is not None:
        flat = [float(v) for row in coefficients for v in row]
        if len(flat) != 3 * steps:
            raise ValueError(f"coefficients: {steps} triples wanted")
        coef = (_lib.c_float * len(flat))(*flat)
    ins, outs = DTYPES.get(in_dtype, in_dtype), DTYPES.get(out_dtype, out_dtype)
    d = _lib.ArOrthoDesc(n, dims[0], dims[1], ins, outs, int(steps), coef, float(eps),
                         PRECISIONS.get(precision, precision))
    h = _lib.c_void_p()
    _check(_lib.load().ar_ortho_plan(d, h), "ar_ortho_plan")
    return OrthoPlan(h.value, shapes, ins, outs)


def ar_ortho_workspace(plan: OrthoPlan) -> int:
    """Device bytes that a call with the plan needs."""
    if plan.workspace_bytes is None:
        b = _lib.c_size_t()
        _check(_lib.load().ar_ortho_workspace(plan.handle, b), "ar_ortho_workspace")
        plan.workspace_bytes = b.value
    return plan.workspace_bytes


def _matrices(plan: OrthoPlan, tensors, dtype: int, what: str):
    if tensors is None:
        return None
    if len(tensors) != len(plan.shapes):
        raise ValueError(f"{what}: {len(plan.shapes)} matrices wanted, got {len(tensors)}")
    arr = (_lib.ArMatrix * max(1, len(tensors)))()
    for i, (t, shape) in enumerate(zip(tensors, plan.shapes)):
        ld = _row_major(t, f"{what}[{i}]")
        if tuple(t.shape) != shape or _dtype_of(t) != dtype:
            raise ValueError(f"{what}[{i}]: the plan has {shape} of type {dtype}, got {tuple(t.shape)} {t.dtype}")
        arr[i].data, arr[i].ld = _ptr(t), ld
    return arr


def ar_orthogonalize(plan: OrthoPlan, matrices, outs=None, workspace=None, stream=None):
    """Newton-Schulz orthogonalisation of every matrix of the plan; returns `outs`
    (new tensors by default; may be `matrices` themselves where the types agree)."""
    if outs is None:
        import torch

        kind = torch.bfloat16 if plan.out_dtype == AR_BF16 else torch.float32
        outs = [_empty(m.shape, kind, m, stream) for m in matrices]
    a, b = _matrices(plan, matrices, plan.in_dtype, "matrices"), _matrices(plan, outs, plan.out_dtype, "outs")
    workspace, room = _room(workspace, ar_ortho_workspace(plan), matrices[0], stream)
    _check(_lib.load().ar_orthogonalize(plan.handle, a, b, room, _stream(stream)), "ar_orthogonalize")
    return outs


def ar_muon_step(plan: OrthoPlan, params, grads, momenta, lr: float, momentum: float = 0.95, weight_decay: float = 0.0,
                 nesterov: bool = True, adjust="shape", grad_scale: float = 1.0, params_out=None, momenta_out=None,
                 workspace=None, stream=None):
    """One step of the orthogonalised optimiser on every matrix of the plan (see
    include/ar.h); `params` and `momenta` (fp32) are updated in place unless
    `params_out` / `momenta_out` are given."""
    p, g = _matrices(plan, params, plan.out_dtype, "params"), _matrices(plan, grads, plan.in_dtype, "grads")
    m = _matrices(plan, momenta, AR_F32, "momenta")
    po, mo = _matrices(plan, params_out, plan.out_dtype, "params_out"), _matrices(plan, momenta_out, AR_F32, "momenta_out")
    workspace, room = _room(workspace, ar_ortho_workspace(plan), params[0], stream)
    d = _lib.ArMuonDesc(float(lr), float(momentum), float(weight_decay), int(bool(nesterov)),
                        ADJUSTS.get(adjust, adjust), float(grad_scale))
    _check(_lib.load().ar_muon_step(plan.handle, d, p, g, m, po, mo, room, _stream(stream)), "ar_muon_step")


# ---------------------------------------------------------------- status


def ar_device_status(clear: bool = True) -> int:
    return _lib.load().ar_device_status(1 if clear else 0)


def ar_plan_query(plan: Plan) -> int:
    """The plan's sticky asynchronous status (AR_OK or AR_ETIMEOUT), read
    without synchronising; see include/ar.h."""
    return _lib.load().ar_plan_query(plan.handle)


def ar_selftest_wait_timeout(polls: int = 1000, stream=None):
    """Run the bounded-wait self-test kernel (see include/ar.h)."""
    _check(_lib.load().ar_selftest_wait_timeout(int(polls), _stream(stream)), "ar_selftest_wait_timeout")


def ar_selftest_scale_quotient() -> int:
    """Mismatches of the division-free block scale against the IEEE division
    over every non-negative float (see include/ar.h)."""
    n = ctypes.c_ulonglong(0)
    _check(_lib.load().ar_selftest_scale_quotient(ctypes.byref(n)), "ar_selftest_scale_quotient")
    return n.value


def ar_status_string(status: int) -> str:
    return _lib.load().ar_status_string(int(status)).decode()


def ar_version() -> int:
    return _lib.load().ar_version()


# ---------------------------------------------------------------- convenience


def workspace_for(plan: Plan, device=None):
    """A torch byte tensor of the plan's workspace size (None when it needs none)."""
    nbytes = plan.stats["workspace_bytes"]
    if nbytes == 0:
        return None
    import torch

    return torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
