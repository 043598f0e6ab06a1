"""The operators on both sides of a post-training step: what is measured, and on what.

In front of the losses, the rollouts; behind the gradient exchange, the way to the weights:

* verification of drafted tokens: drafts ``x_j`` of a cheap policy ``q`` against the target ``p``, from given uniform
  numbers: ``x_j`` stands if ``u_j < p_j(x_j) / q_j(x_j)``; behind the first that does not, one token is drawn from
  ``max(p - q, 0)`` (from ``p`` where all drafts stand) as the first index whose running sum passes ``u`` times the
  total. Drafts without a distribution count as ``q = 1``. The greedy form compares with the largest logit;
* the global norm of many gradient tensors, and the coefficient that clips it;
* clipping: the norm, and the scaled gradients;
* the AdamW step behind the norm, for the parameters that an orthogonalised step is not for.

``own`` false: elementary torch operations in 32 bits (64 for long sums and for the running sums of a draw), rounded
once at the end. ``own`` true: the library's entry points. ``exact`` is the definition in 64 bits, written another way.
"""

import math
import random

import torch

own = False

BETAS, EPS = (0.9, 0.95), 1e-8
NORM_EPS = 1e-6
GRAD_STD = 1e-3

# the repository's 16-layer transformer (hidden 2048, ffn 8192, vocabulary 32000): one layer, and all of it
LAYER = "2048*2,2048x2048*4,2048x8192*2,8192x2048"
MODEL = "32000x2048,2048*32,2048x2048*64,2048x8192*32,8192x2048*16"

MAX_ELEMENTS = 1 << 26  # of a drawn list of tensors
MAX_LOGITS = (64 * 9 + 64 * 8) * 131072


def listed():
    return [
        # the norm of an adapter's gradients: a few small tensors, latency
        dict(name="norm_small", op="norm", shapes="256x256,256*3,77x33", mat="bf16", vec="f32", kind="l2", scale=1.0,
             clip=True, packed=False),
        # the norm of all gradients of the transformer after a sum over 8 ranks, fp32 gains among bf16 matrices
        dict(name="norm_model", op="norm", shapes=MODEL, mat="bf16", vec="f32", kind="l2", scale=0.125, clip=False,
             packed=False),
        # the same adapter, clipped
        dict(name="clip_small", op="clip", shapes="256x256,256*3,77x33", mat="bf16", vec="f32", kind="l2", scale=1.0,
             clip=True, packed=False),
        # an uneven set by its largest entry: odd lengths, single elements, many small tensors, one behind the other
        dict(name="clip_uneven", op="clip", shapes="1000x333,77x2049,1,12345679,513*200,1536x640*2,7", mat="f32",
             vec="bf16", kind="max", scale=0.25, clip=True, packed=True),
        # one layer's fp32 gradients, clipped
        dict(name="clip_layer", op="clip", shapes=LAYER, mat="f32", vec="f32", kind="l2", scale=1.0, clip=True,
             packed=False),
        # the gains of the whole transformer, fp32: 33 short vectors, latency
        dict(name="adamw_gains", op="adamw", shapes="2048*33", grad="f32", param="f32", master=False, scale=1.0,
             clip=False, step=1000, decay=0.0, packed=False),
        # embedding and head with the gains: bf16 gradients and weights, fp32 masters
        dict(name="adamw_embedding", op="adamw", shapes="32000x2048*2,2048*33", grad="bf16", param="bf16", master=True,
             scale=0.125, clip=True, step=3, decay=0.1, packed=False),
        # fp32 throughout, odd lengths, one behind the other
        dict(name="adamw_uneven", op="adamw", shapes="32003x515,12345679,513*200,1", grad="f32", param="f32",
             master=False, scale=0.25, clip=True, step=57, decay=0.01, packed=True),
        # one answer and four drafts, fp32 logits, as a sampler verifies them at every step: latency
        dict(name="verify_step", op="verify", seqs=1, most=4, ragged=False, vocab=32000, pad=0, dtype="f32", tau=0.7,
             mode="sample", draft=True),
        # a batch of answers under a large vocabulary, eight drafts each, some ruled out by a grammar
        dict(name="verify_batch", op="verify", seqs=64, most=8, ragged=False, vocab=131072, pad=0, dtype="bf16",
             tau=1.0, mode="sample", draft=True),
        # drafts looked up in the prompt, without a distribution: uneven numbers of them, an odd, padded head
        dict(name="verify_lookup", op="verify", seqs=97, most=10, ragged=True, vocab=32003, pad=61, dtype="bf16",
             tau=0.9, mode="sample", draft=False),
        # greedy decoding, odd fp32 vocabulary
        dict(name="verify_greedy", op="verify", seqs=32, most=5, ragged=True, vocab=50021, pad=0, dtype="f32", tau=1.0,
             mode="greedy", draft=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "clip", "adamw", "verify", "verify"])
    if op == "verify":
        vocab = _log_int(rng, 300, 131072)
        dtype = rng.choice(["f32", "bf16"])
        mode = rng.choice(["sample", "sample", "sample", "greedy"])
        draft = mode == "sample" and rng.random() < 0.7
        most = rng.randint(1, 12)
        seqs = _log_int(rng, 1, 256)
        seqs = max(1, min(seqs, MAX_LOGITS // vocab // (2 * most + 1) // (2 if dtype == "f32" else 1)))
        return dict(op=op, seqs=seqs, most=most, ragged=rng.random() < 0.5, vocab=vocab,
                    pad=rng.choice([0, 0, 1, 8, 32]), dtype=dtype, tau=rng.choice([1.0, 1.0, 0.8]), mode=mode,
                    draft=draft)
    shapes, left = [], _log_int(rng, 1 << 10, MAX_ELEMENTS)
    for _ in range(rng.randint(1, 8)):
        if rng.random() < 0.5:
            n, times = _log_int(rng, 1, 20000), _log_int(rng, 1, 100)
            text = "%d*%d" % (n, times)
        else:
            r, c, times = _log_int(rng, 1, 8192), _log_int(rng, 1, 8192), 1
            n, text = r * c, "%dx%d" % (r, c)
        left -= n * times
        if shapes and left < 0:
            break
        if left < 0:
            text = "%d" % (left + n * times)
        shapes.append(text)
    case = dict(op=op, shapes=",".join(shapes), scale=rng.choice([1.0, 0.125, 0.3]), clip=rng.random() < 0.6,
                packed=rng.random() < 0.5)
    if op == "adamw":
        case.update(grad=rng.choice(["f32", "bf16"]), param=rng.choice(["f32", "bf16"]), master=False,
                    step=_log_int(rng, 1, 10000), decay=rng.choice([0.0, 0.1]))
        case["master"] = case["param"] == "bf16" and rng.random() < 0.6
    else:
        case.update(mat=rng.choice(["f32", "bf16"]), vec=rng.choice(["f32", "bf16"]),
                    kind=rng.choice(["l2", "l2", "max"]))
    return case


# ---------------------------------------------------------------- inputs


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _shapes(text):
    out = []
    for part in text.split(","):
        shape, _, times = part.partition("*")
        out += [tuple(int(v) for v in shape.split("x"))] * int(times or 1)
    return out


def _views(shapes, kinds, packed):
    """Tensors of the given shapes and types as parts of one buffer a type, and those buffers: one behind the other,
    or every one at a multiple of 512 bytes, as a flattened model has them."""
    ends, places = {}, []
    for shape, kind in zip(shapes, kinds):
        at = ends.get(kind, 0)
        if not packed:
            at = (at + 255) // 256 * 256
        places.append(at)
        ends[kind] = at + math.prod(shape)
    flat = {k: torch.zeros(n, dtype=k, device="cuda") for k, n in ends.items()}
    return [flat[k][at:at + math.prod(v)].view(v) for v, k, at in zip(shapes, kinds, places)], list(flat.values())


def _prepare_tensors(case, seed, gen):
    shapes = _shapes(case["shapes"])
    rng = random.Random(seed)
    f32 = [torch.float32] * len(shapes)

    def like(kinds):
        return _views(shapes, kinds, case["packed"])

    def normal(kinds, stds):
        views = like(kinds)[0]
        for v, std in zip(views, stds):
            v.copy_(torch.randn(v.shape, generator=gen, device="cuda") * std)
        return views

    # gradients: every tensor has its own magnitude, as the layers of a model have
    stds = [GRAD_STD * 10 ** rng.uniform(-1, 0.5) for _ in shapes]
    if case["op"] == "adamw":
        kinds = [_dtype(case["grad"])] * len(shapes)
    else:
        kinds = [_dtype(case["vec"] if len(v) == 1 else case["mat"]) for v in shapes]
    s = {"case": case, "grads": normal(kinds, stds)}
    if case.get("kind") == "max":
        near = 4 * max(stds)
    else:
        near = math.sqrt(sum(math.prod(v) * d * d for v, d in zip(shapes, stds)))
    s["max_norm"] = near * case["scale"] * (0.25 if case["clip"] else 8.0)
    if case["op"] == "clip":
        s["outs"], s["outs_flat"] = like(kinds)
    if case["op"] == "adamw":
        weights = [_dtype(case["param"])] * len(shapes)
        s["masters"] = normal(f32, [0.02] * len(shapes))
        s["params"] = like(weights)[0]
        for w, master in zip(s["params"], s["masters"]):
            w.copy_(master)
        # moments as earlier steps with such gradients leave them; the first step finds zeros
        old = 0.0 if case["step"] == 1 else case["scale"]
        s["exp_avgs"] = normal(f32, [0.3 * old * d for d in stds])
        s["exp_avg_sqs"] = normal(f32, [old * d for d in stds])
        for v in s["exp_avg_sqs"]:
            v.square_()
        for k in ("params", "exp_avgs", "exp_avg_sqs") + (("masters",) if case["master"] else ()):
            s[k + "_out"], s[k + "_out_flat"] = like(weights if k == "params" else f32)
        if not case["master"]:
            del s["masters"]
    if own:
        import gradient_sync_gb300 as g

        for k, v in list(s.items()):
            if isinstance(v, list) and not k.endswith("_flat"):
                s[k + "_list"] = g.TensorList(v)
        s["workspace"] = torch.empty(g.ar_grad_workspace(s["grads_list"]), dtype=torch.uint8, device="cuda")
        s["stats"] = torch.empty(4, device="cuda")
        s["norms"] = torch.empty(len(shapes), device="cuda")
    return s


def _drafts(case):
    """How many drafts there are: equal numbers, or in the mean half of the most."""
    return max(1, case["seqs"] * case["most"] // (2 if case["ragged"] else 1))


def _prepare_verify(case, seed, gen):
    S, V, tau = case["seqs"], case["vocab"], case["tau"]
    rng = random.Random(seed)
    N, counts = _drafts(case), [0 if case["ragged"] else case["most"]] * S
    for place in rng.sample(range(S * case["most"]), N) if case["ragged"] else []:
        counts[place // case["most"]] += 1
    start = [0]
    for c in counts:
        start.append(start[-1] + c)
    kind = _dtype(case["dtype"])
    draft_rows = torch.tensor([start[i] + i + j for i in range(S) for j in range(counts[i])], device="cuda")
    final_rows = torch.tensor([start[i + 1] + i for i in range(S)], device="cuda")

    # a head's logits: scores of standard deviation 2, a few likely tokens raised by up to 10; some ruled out (-inf)
    target = torch.empty(N + S, V + case["pad"], dtype=kind, device="cuda")
    for lo in range(0, N + S, 128):
        part = torch.randn(min(128, N + S - lo), V + case["pad"], generator=gen, device="cuda").mul_(2.0)
        likely = torch.randint(0, V, (part.shape[0], 12), generator=gen, device="cuda")
        part.scatter_add_(1, likely, 10.0 * torch.rand(likely.shape, generator=gen, device="cuda"))
        target[lo:lo + 128] = part
    ruled = torch.rand(V, generator=gen, device="cuda") < 0.05
    ruled[0] = False
    target = target[:, :V]
    target.masked_fill_(ruled, -math.inf)
    s = {"case": case, "target": target, "draft_start": torch.tensor(start, device="cuda")}

    drafts = torch.empty(N, dtype=torch.long, device="cuda")
    ratio = torch.empty(N, dtype=torch.float64, device="cuda")
    draft_logits = torch.empty(N, V + case["pad"], dtype=kind, device="cuda")[:, :V] if case["draft"] else None

    def random_like(v):
        return torch.rand(v.shape, generator=gen, device="cuda")

    for lo in range(0, N, 128):
        rows = draft_rows[lo:lo + 128]
        x = target[rows].float()
        if case["draft"]:  # the cheap policy: the target's scores, blurred; its drafts are drawn from it
            y = (x + 0.8 * torch.randn(x.shape, generator=gen, device="cuda")).to(kind)
            draft_logits[lo:lo + 128] = y
            at = (y.float() / tau - torch.log(-torch.log(random_like(x) * 0.999999 + 5e-7))).argmax(1)
            lq = y.double().div_(tau).log_softmax(1).gather(1, at[:, None])[:, 0]
        else:  # looked up: often a likely token, sometimes any
            at = (x / tau - torch.log(-torch.log(random_like(x) * 0.999999 + 5e-7))).argmax(1)
            if case["mode"] == "greedy":
                at = (x == x.max(1, keepdim=True).values).float().argmax(1)
            other = torch.randint(0, V, at.shape, generator=gen, device="cuda")
            at = torch.where(random_like(at) < (0.8 if case["mode"] == "greedy" else 0.6), at, other)
            lq = 0.0
            if case["mode"] != "greedy":  # and sometimes the most likely one
                at = torch.where(random_like(at) < 0.5, x.argmax(1), at)
        drafts[lo:lo + 128] = at
        if case["mode"] != "greedy":
            ratio[lo:lo + 128] = (x.double().div_(tau).log_softmax(1).gather(1, at[:, None])[:, 0] - lq).exp()
    s.update(drafts=drafts, draft_logits=draft_logits, uniforms=None)
    if case["mode"] != "greedy":
        u = random_like(torch.empty(N + S))
        # no number on the very edge of a decision, where rounding would take it: first those that accept ...
        ud = u[draft_rows].double()
        ud = torch.where((ud - ratio).abs() < 2e-3 * ratio, ratio * (1 - 4e-3), ud)
        u[draft_rows] = ud.float().clamp_(max=0.9999999)
        stands = (u[draft_rows].double() < ratio).tolist()
        # ... then those that draw: inside the drawn token's share, of a token that has more than 1e-5
        for i in range(S):
            a = next((j for j in range(counts[i]) if not stands[start[i] + j]), counts[i])
            p = target[start[i] + i + a].double().div_(tau).softmax(0)
            if a < counts[i]:
                if case["draft"]:
                    p = (p - draft_logits[start[i] + a].double().div_(tau).softmax(0)).clamp_(min=0)
                else:
                    p[drafts[start[i] + a]] = 0
            p /= p.sum()
            upto = p.cumsum(0)
            v = u[final_rows[i]].double()
            at = torch.searchsorted(upto, v, right=True).clamp_(max=V - 1)
            at = torch.where(p[at] > 1e-5, at, p.argmax())
            below = upto[at] - p[at]
            u[final_rows[i]] = torch.minimum(torch.maximum(v, below + 0.1 * p[at]), below + 0.9 * p[at]).float()
        s["uniforms"] = u
    s["tokens"] = torch.empty(N + S, dtype=torch.long, device="cuda")
    s["accepted"] = torch.empty(S, dtype=torch.long, device="cuda")
    s["logp"] = torch.empty(N + S, device="cuda")
    if own:
        import gradient_sync_gb300 as g

        s["workspace"] = torch.empty(g.ar_verify_workspace(N, S, V), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (_prepare_verify if case["op"] == "verify" else _prepare_tensors)(case, seed, gen)


# ---------------------------------------------------------------- plain forms


def _norm_plain(s):
    case, grads = s["case"], s["grads"]
    if case.get("kind") == "max":
        norms = torch.stack([v.float().abs().max() for v in grads]) * case["scale"]
        norm = norms.max()
    else:
        squares = torch.stack([v.float().square().sum(dtype=torch.float64) for v in grads]) * case["scale"] ** 2
        norms, norm = squares.sqrt().float(), squares.sum().sqrt()
    coef = (s["max_norm"] / (norm + NORM_EPS)).clamp(max=1.0)
    finite = torch.isfinite(norm)
    coef = torch.where(finite, coef, torch.zeros_like(coef)).float()
    clipped = (coef < 1).float()
    return {"stats": torch.stack([norm.float(), coef, clipped, finite.float()]), "norms": norms}


def _clip_plain(s):
    out = _norm_plain(s)
    factor = out["stats"][1] * s["case"]["scale"]
    for v, o in zip(s["grads"], s["outs"]):
        o.copy_(torch.where(factor != 0, v.float() * factor, torch.zeros_like(factor)))
    return {**out, "outs": s["outs_flat"]}


def _adamw_rates(case):
    t, lr = case["step"], 3e-3
    return lr, 1 - BETAS[0] ** t, math.sqrt(1 - BETAS[1] ** t)


def _adamw_plain(s):
    case = s["case"]
    out = _norm_plain(s)
    factor = out["stats"][1] * case["scale"]
    lr, c1, c2 = _adamw_rates(case)
    olds = s["masters"] if case["master"] else s["params"]
    for i, (w, g, m, v) in enumerate(zip(olds, s["grads"], s["exp_avgs"], s["exp_avg_sqs"])):
        g = g.float() * factor
        m1 = s["exp_avgs_out"][i].copy_(BETAS[0] * m + (1 - BETAS[0]) * g)
        v1 = s["exp_avg_sqs_out"][i].copy_(BETAS[1] * v + (1 - BETAS[1]) * g * g)
        w = w.float() * (1 - lr * case["decay"]) - (lr / c1) * m1 / (v1.sqrt() / c2 + EPS)
        s["params_out"][i].copy_(w)
        if case["master"]:
            s["masters_out"][i].copy_(w)
    return {**out, **_updated(s)}


def _updated(s):
    return {k: s[k + "_out_flat"] for k in ("params", "exp_avgs", "exp_avg_sqs", "masters") if k + "_out" in s}


def _log_probs_plain(x, tau):
    x = x.float() / tau
    x = x - x.max(1, keepdim=True).values
    return x - torch.log(torch.exp(x).sum(1, keepdim=True))


def _first_largest(x):
    index = torch.arange(x.shape[1], device=x.device)
    return torch.where(x == x.max(1, keepdim=True).values, index, x.shape[1]).min(1).values


def _verify_plain(s):
    case, x, drafts, start = s["case"], s["target"], s["drafts"], s["draft_start"]
    N, S = drafts.numel(), case["seqs"]
    index, seqs = torch.arange(N, device=x.device), torch.arange(S, device=x.device)
    which = torch.searchsorted(start[1:].contiguous(), index, right=True)
    rows = index + which
    logp = _log_probs_plain(x, case["tau"])
    if case["mode"] == "greedy":
        best = _first_largest(x)
        stands = best[rows] == drafts
    else:
        ratio = logp[rows].gather(1, drafts[:, None])[:, 0]
        if case["draft"]:
            ratio = ratio - _log_probs_plain(s["draft_logits"], case["tau"]).gather(1, drafts[:, None])[:, 0]
        stands = s["uniforms"][rows] < torch.exp(ratio)
    counts = start[1:] - start[:-1]
    place = index - start[which]
    accepted = counts.scatter_reduce(0, which, torch.where(stands, counts[which], place), "amin")
    at = start[:-1] + seqs + accepted
    if case["mode"] == "greedy":
        token = best[at]
    else:
        # the draw's running sums in 64 bits: a border between two tokens may lie anywhere
        r = torch.softmax(x[at].double() / case["tau"], 1)
        stopped = accepted < counts
        back = (start[:-1] + accepted).clamp(max=N - 1)
        if case["draft"]:
            q = torch.softmax(s["draft_logits"][back].double() / case["tau"], 1)
        else:
            q = torch.zeros_like(r).scatter_(1, drafts[back][:, None], 1.0)
        r = torch.where(stopped[:, None], (r - q).clamp_(min=0), r)
        upto = r.cumsum(1)
        u = s["uniforms"][start[1:] + seqs].double()
        token = (upto <= u[:, None] * upto[:, -1:]).sum(1)
    row = torch.arange(N + S, device=x.device)
    of = torch.searchsorted(start[1:] + seqs, row)
    place = row - start[of] - of
    tokens = torch.full_like(row, -1)
    tokens[rows] = drafts
    tokens = torch.where(place < accepted[of], tokens, torch.full_like(tokens, -1))
    tokens[at] = token
    picked = logp.gather(1, tokens.clamp(min=0)[:, None])[:, 0]
    return {"accepted": accepted, "tokens": tokens, "logp": torch.where(tokens >= 0, picked, torch.zeros_like(picked))}


# ---------------------------------------------------------------- one pass


def run(s):
    case = s["case"]
    if not own:
        return {"norm": _norm_plain, "clip": _clip_plain, "adamw": _adamw_plain, "verify": _verify_plain}[case["op"]](s)
    import gradient_sync_gb300 as g

    if case["op"] == "verify":
        accepted, tokens, logp = g.ar_verify_drafts(
            s["target"], s["drafts"], s["uniforms"], s["draft_start"], draft_logits=s["draft_logits"],
            temperature=case["tau"], mode=case["mode"], accepted=s["accepted"], tokens=s["tokens"], logp=s["logp"],
            workspace=s["workspace"])
        return {"accepted": accepted, "tokens": tokens, "logp": logp}
    ways = dict(kind=case.get("kind", "l2"), grad_scale=case["scale"], stats=s["stats"], norms=s["norms"],
                workspace=s["workspace"])
    if case["op"] == "clip":
        stats, norms, _ = g.ar_grad_clip(s["grads_list"], s["max_norm"], outs=s["outs_list"], **ways)
        return {"stats": stats, "norms": norms, "outs": s["outs_flat"]}
    stats, norms = g.ar_grad_norm(s["grads_list"], s["max_norm"], **ways)
    if case["op"] == "norm":
        return {"stats": stats, "norms": norms}
    lr, _, _ = _adamw_rates(case)
    g.ar_adamw_step(s["params_list"], s["grads_list"], s["exp_avgs_list"], s["exp_avg_sqs_list"], lr=lr,
                    step=case["step"], betas=BETAS, eps=EPS, weight_decay=case["decay"], grad_scale=case["scale"],
                    clip=stats, masters=s.get("masters_list"), params_out=s["params_out_list"],
                    exp_avgs_out=s["exp_avgs_out_list"], exp_avg_sqs_out=s["exp_avg_sqs_out_list"],
                    masters_out=s.get("masters_out_list"))
    return {"stats": stats, "norms": norms, **_updated(s)}


# ---------------------------------------------------------------- the work of one pass


def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "verify":
        # every row once: the target's, and the drafts' where they have any
        drafts = _drafts(case)
        rows = drafts * (2 if case["draft"] else 1) + case["seqs"]
        return {"bytes": rows * case["vocab"] * size[case["dtype"]] + 32 * (drafts + case["seqs"]),
                "flops": 4 * rows * case["vocab"]}
    moved = flops = 0
    for shape in _shapes(case["shapes"]):
        n = math.prod(shape)
        if case["op"] == "adamw":
            moved += n * (size[case["grad"]] + 16 + 2 * size[case["param"]])
            if case["master"]:
                moved += n * (8 - size[case["param"]])  # the weights themselves are written only
            flops += 16 * n
        else:
            moved += n * size[case["vec"] if len(shape) == 1 else case["mat"]] * (2 if case["op"] == "clip" else 1)
            flops += n * (3 if case["op"] == "clip" else 2)
    return {"bytes": moved, "flops": flops}


# ---------------------------------------------------------------- the definition in 64 bits


def _exact_tensors(case, s):
    c = case["scale"]
    order = math.inf if case.get("kind") == "max" else 2
    norms = torch.stack([torch.linalg.vector_norm(v.double() * c, order) for v in s["grads"]])
    norm = torch.linalg.vector_norm(norms, order)
    coef = min(1.0, s["max_norm"] / (float(norm) + NORM_EPS))
    out = {"stats": torch.tensor([float(norm), coef, float(coef < 1), 1.0], dtype=torch.float64, device="cuda"),
           "norms": norms}

    def wide(flats, views, values):
        """The buffers in 64 bits, with these values where the views lie."""
        to = {v.dtype: torch.zeros(v.numel(), dtype=torch.float64, device="cuda") for v in flats}
        for v, value in zip(views, values):
            to[v.dtype][v.storage_offset():v.storage_offset() + v.numel()] = value.reshape(-1)
        return list(to.values())

    grads = [v.double() * (c * coef) for v in s["grads"]] if case["op"] != "norm" else []
    if case["op"] == "clip":
        out["outs"] = wide(s["outs_flat"], s["outs"], grads)
    if case["op"] == "adamw":
        lr, c1, c2 = _adamw_rates(case)
        new = {"params": [], "exp_avgs": [], "exp_avg_sqs": []}
        for w, g, m, v in zip(s["masters"] if case["master"] else s["params"], grads, s["exp_avgs"], s["exp_avg_sqs"]):
            m1 = m.double() + (1 - BETAS[0]) * (g - m.double())
            v1 = v.double() + (1 - BETAS[1]) * (g * g - v.double())
            step = (m1 / c1) / ((v1 / (c2 * c2)).sqrt() + EPS)
            new["params"].append(w.double() - lr * (case["decay"] * w.double() + step))
            new["exp_avgs"].append(m1)
            new["exp_avg_sqs"].append(v1)
        if case["master"]:
            new["masters"] = new["params"]
        out.update({k: wide(s[k + "_out_flat"], s[k + "_out"], v) for k, v in new.items()})
    return out


def _exact_verify(case, s):
    start, drafts = s["draft_start"].tolist(), s["drafts"].tolist()
    S, N = case["seqs"], len(drafts)
    u = s["uniforms"].tolist() if s["uniforms"] is not None else None
    tokens, logp, accepted = [-1] * (N + S), [0.0] * (N + S), []
    for i in range(S):
        lo, hi = start[i], start[i + 1]
        p = torch.softmax(s["target"][lo + i:hi + i + 1].double() / case["tau"], 1)
        q = torch.softmax(s["draft_logits"][lo:hi].double() / case["tau"], 1) if case["draft"] else None
        for j in range(hi - lo + 1):
            row, x = lo + i + j, drafts[lo + j] if lo + j < hi else -1
            if case["mode"] == "greedy":
                best = int((s["target"][row] == s["target"][row].max()).nonzero()[0])
                if x == best:
                    tokens[row], logp[row] = x, math.log(p[j, x])
                    continue
                r = None
            else:
                r = p[j]
                if x >= 0:
                    qx = float(q[j, x]) if case["draft"] else 1.0
                    if u[row] * qx < float(p[j, x]):
                        tokens[row], logp[row] = x, math.log(p[j, x])
                        continue
                    one = torch.zeros_like(r)
                    one[x] = 1.0
                    r = torch.maximum(r - (q[j] if case["draft"] else one), torch.zeros_like(r))
                upto = torch.cumsum(r, 0)
                best = int(torch.searchsorted(upto, (u[hi + i] * upto[-1]).reshape(1), right=True))
            tokens[row], logp[row] = best, math.log(p[j, best])
            accepted.append(j)
            break
    return {"accepted": torch.tensor(accepted, device="cuda"), "tokens": torch.tensor(tokens, device="cuda"),
            "logp": torch.tensor(logp, dtype=torch.float64, device="cuda")}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_verify(case, s) if case["op"] == "verify" else _exact_tensors(case, s)
