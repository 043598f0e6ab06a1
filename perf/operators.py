"""The operators around the gradient exchange of a post-training step: what is measured, and on what.

Five operators, in the order in which a step uses them:

* token log-probabilities: ``logp[t] = logits[t, label[t]] / tau - logsumexp(logits[t] / tau)``;
* the clipped policy loss with a KL term, with the gradient of its logits;
* the preference loss over paired log ratios, with the gradient of its logits;
* the orthogonalised update: five Newton-Schulz steps ``X <- a X + (b A + c A A) X``, ``A = X X^T``, from
  ``X = U / (|U|_F + eps)``;
* the whole optimiser step around it: momentum, orthogonalisation, decayed weight update.

``own`` false: elementary torch operations in 32 bits, rounded once at the end. ``own`` true: the library's entry
points. ``exact`` is the definition in 64 bits, written another way: gradients by differentiation of the loss, the
Newton-Schulz steps on the side of the columns.
"""

import math

import torch

own = False

STEPS = 5
A, B, C = 3.4445, -4.7750, 2.0315  # the coefficients of every Newton-Schulz step (the library's default)
EPS = 1e-7
CLIP_LOW, CLIP_HIGH = 0.2, 0.28
MU, LR, DECAY = 0.95, 0.02, 0.01

# one layer of the repository's 16-layer transformer (hidden 2048, ffn 8192): Wq, Wk, Wv, Wo, W1, W3, W2
LAYER = "2048x2048*4,2048x8192*2,8192x2048"
# its gate projection workload, one matrix of 192 MiB in fp32
GATE = "12288x4096"

MAX_LOGITS = 16384 * 32000


def listed():
    return [
        # the log-probabilities of a batch of 16 sampled tokens, as a sampler asks for them at each step: latency
        dict(name="logp_step", op="logp", tokens=16, seqs=1, vocab=32000, pad=0, dtype="f32", tau=0.7),
        # scoring rollouts under the reference policy: an odd vocabulary, some of it ruled out (-inf)
        dict(name="logp_score", op="logp", tokens=6007, seqs=12, vocab=50021, pad=0, dtype="bf16", tau=1.0),
        # a micro-batch of four short answers: latency
        dict(name="policy_small", op="policy", tokens=64, seqs=4, vocab=32000, pad=0, dtype="bf16", tau=1.0,
             kl=0.05, per="token"),
        # fp32 logits of an odd, padded head; each answer counts the same, whatever its length
        dict(name="policy_odd", op="policy", tokens=3001, seqs=23, vocab=32003, pad=61, dtype="f32", tau=0.9,
             kl=0.0, per="sequence"),
        # a full batch of long answers at the transformer's vocabulary
        dict(name="policy_batch", op="policy", tokens=16384, seqs=32, vocab=32000, pad=0, dtype="bf16", tau=1.0,
             kl=0.05, per="token"),
        # one pair of short answers, fp32 logits: latency
        dict(name="pref_small", op="pref", tokens=48, seqs=2, vocab=32000, pad=0, dtype="f32", tau=1.0,
             form="sigmoid", mean=False),
        # eight pairs of about 512 tokens an answer
        dict(name="pref_batch", op="pref", tokens=8192, seqs=16, vocab=32000, pad=0, dtype="bf16", tau=1.0,
             form="sigmoid", mean=False),
        # two pairs over a large vocabulary, squared form on length-normalised ratios
        dict(name="pref_wide", op="pref", tokens=3500, seqs=4, vocab=131072, pad=0, dtype="bf16", tau=1.0,
             form="square", mean=True),
        # one small projection: latency
        dict(name="ortho_small", op="ortho", shapes="256x256", src="bf16", dst="bf16"),
        # an uneven set: tall, wide, odd and thin matrices, fp32 throughout
        dict(name="ortho_uneven", op="ortho", shapes="1000x333,77x2049,2048x2048,1x512,1536x640*2", src="f32",
             dst="f32"),
        # the step of one transformer layer: fp32 summed gradients, bf16 weights
        dict(name="muon_layer", op="muon", shapes=LAYER, src="f32", dst="bf16", nesterov=True),
        # the step of the 192 MiB gate projection, fp32 weights
        dict(name="muon_gate", op="muon", shapes=GATE, src="f32", dst="f32", nesterov=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logp", "policy", "pref", "ortho", "muon"])
    if op in ("ortho", "muon"):
        shapes, left = [], 1.2e12  # flops of the products of one pass, below the listed largest
        for _ in range(rng.randint(1, 6)):
            r, c = _log_int(rng, 16, 4096), _log_int(rng, 16, 4096)
            left -= _ortho_flops(r, c)
            if shapes and left < 0:
                break
            shapes.append("%dx%d" % (r, c))
        case = dict(op=op, shapes=",".join(shapes), src=rng.choice(["f32", "bf16"]), dst=rng.choice(["f32", "bf16"]))
        if op == "muon":
            case["nesterov"] = rng.random() < 0.5
        return case
    vocab = _log_int(rng, 1000, 131072)
    dtype = rng.choice(["f32", "bf16"])
    most = MAX_LOGITS // 2 // vocab // (2 if dtype == "f32" else 1)
    tokens = _log_int(rng, 4, min(16384, most))
    seqs = 2 * max(1, min(16, tokens // rng.randint(8, 200)))
    case = dict(op=op, tokens=tokens, seqs=seqs, vocab=vocab, pad=rng.choice([0, 0, 1, 8, 32]), dtype=dtype,
                tau=rng.choice([1.0, 1.0, 0.8]))
    if op == "policy":
        case.update(kl=rng.choice([0.0, 0.05]), per=rng.choice(["token", "sequence"]))
    if op == "pref":
        case.update(form=rng.choice(["sigmoid", "square"]), mean=rng.random() < 0.5)
    return case


# ---------------------------------------------------------------- inputs


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _shapes(text):
    out = []
    for part in text.split(","):
        shape, _, times = part.partition("*")
        r, c = shape.split("x")
        out += [(int(r), int(c))] * int(times or 1)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = {"case": case}
    if case["op"] in ("ortho", "muon"):
        shapes = _shapes(case["shapes"])
        # gradients: a few strong directions over noise, as the gradients of trained projections have
        grads = []
        for r, c in shapes:
            k = min(r, c, 16)
            u, v = normal(r, k), normal(k, c)
            weight = torch.linspace(1.0, 0.2, k, device="cuda")
            grads.append((((u * weight) @ v * 0.5 + normal(r, c)) * 1e-3).to(_dtype(case["src"])))
        s["grads"] = grads
        if case["op"] == "muon":
            s["params"] = [(normal(r, c) * 0.02).to(_dtype(case["dst"])) for r, c in shapes]
            s["momenta"] = [normal(r, c) * 2e-3 for r, c in shapes]
            s["params_out"] = [torch.empty_like(p) for p in s["params"]]
            s["momenta_out"] = [torch.empty_like(m) for m in s["momenta"]]
        else:
            s["outs"] = [torch.empty(r, c, dtype=_dtype(case["dst"]), device="cuda") for r, c in shapes]
        if own:
            import gradient_sync_gb300 as g

            s["plan"] = g.ar_ortho_plan(shapes, case["src"], case["dst"])
            s["workspace"] = torch.empty(g.ar_ortho_workspace(s["plan"]), dtype=torch.uint8, device="cuda")
        return s

    T, V, S = case["tokens"], case["vocab"], case["seqs"]
    # a head's logits: scores of standard deviation 2, the sampled token's raised by 0 to 14; rows V + pad apart
    whole = normal(T, V + case["pad"]).mul_(2.0)
    logits = whole[:, :V]
    labels = torch.randint(0, V, (T,), generator=gen, device="cuda")
    rows = torch.arange(T, device="cuda")
    logits[rows, labels] += 14.0 * torch.rand(T, generator=gen, device="cuda")
    if case["op"] == "logp":  # entries that a grammar rules out
        ruled = torch.rand(V, generator=gen, device="cuda") < 0.05
        keep = logits[rows, labels]
        logits.masked_fill_(ruled, -math.inf)
        logits[rows, labels] = keep
    whole = whole.to(_dtype(case["dtype"]))
    logits = whole[:, :V]
    # answers of uneven length; the first tokens of each belong to its prompt and carry no label
    cuts = torch.randint(0, T + 1, (S - 1,), generator=gen, device="cuda").sort().values
    even = torch.arange(1, S, device="cuda") * T // S
    cuts = (cuts + 3 * even) // 4
    seq_start = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)])
    which = torch.searchsorted(seq_start[1:].contiguous(), rows, right=True)
    place = rows - seq_start[which]
    length = (seq_start[1:] - seq_start[:-1])[which]
    labels = torch.where(place * 4 < length, torch.full_like(labels, -100), labels)
    s.update(logits=logits, labels=labels, seq_start=seq_start)
    s["logp"] = torch.empty(T, device="cuda")
    if case["op"] != "logp":
        now = torch.empty(T, device="cuda")
        for lo in range(0, T, 2048):
            x = logits[lo:lo + 2048].float() / case["tau"]
            at = labels[lo:lo + 2048].clamp(min=0)
            now[lo:lo + 2048] = x.gather(1, at[:, None])[:, 0] - x.logsumexp(1)
        s["ref_logp"] = now + 0.3 * normal(T)
        s["dlogits"] = torch.empty_strided(logits.shape, logits.stride(), dtype=logits.dtype, device="cuda")
    if case["op"] == "policy":
        # the policy has moved since the rollout; no ratio on the very edge of the clip, where rounding would decide
        ratio = torch.exp(0.15 * normal(T))
        for edge in (1 - CLIP_LOW, 1 + CLIP_HIGH):
            ratio = torch.where((ratio - edge).abs() < 2e-3, torch.full_like(ratio, edge + 4e-3), ratio)
        s["old_logp"] = now - ratio.log()
        s["advantages"] = normal(S)[which].contiguous()
    if own:
        import gradient_sync_gb300 as g

        s["workspace"] = torch.empty(g.ar_loss_workspace(T, S), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms


def _logp_plain(s):
    x = s["logits"].float() / s["case"]["tau"]
    top = x.max(1, keepdim=True).values
    x = x - top
    e = torch.exp(x)
    total = e.sum(1, keepdim=True)
    valid = s["labels"] >= 0
    at = torch.where(valid, s["labels"], torch.zeros_like(s["labels"]))
    logp = x.gather(1, at[:, None])[:, 0] - torch.log(total)[:, 0]
    return torch.where(valid, logp, torch.zeros_like(logp)), e, total, valid, at


def _dlogits_plain(s, e, total, valid, at, coef):
    """coef[t] * (onehot - softmax) / tau, rounded once into the gradient's type."""
    coef = torch.where(valid, coef, torch.zeros_like(coef)) / s["case"]["tau"]
    d = e * (-coef[:, None] / total)
    d.scatter_add_(1, at[:, None], coef[:, None])
    d = torch.where(valid[:, None], d, torch.zeros_like(d))
    s["dlogits"].copy_(d)
    return s["dlogits"]


def _segments(s):
    """Each token's sequence, the number of labelled tokens of each sequence, and sums over sequences."""
    start, T = s["seq_start"], s["labels"].numel()
    which = torch.searchsorted(start[1:].contiguous(), torch.arange(T, device=start.device), right=True)

    def total(v):
        return torch.zeros(start.numel() - 1, device=v.device).index_add_(0, which, v)

    return which, total((s["labels"] >= 0).float()), total


def _policy_plain(s):
    case = s["case"]
    logp, e, total, valid, at = _logp_plain(s)
    which, count, _ = _segments(s)
    zero = torch.zeros_like(logp)
    ratio = torch.exp(torch.where(valid, logp - s["old_logp"], zero))
    adv = s["advantages"]
    free, held = ratio * adv, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * adv
    back = torch.where(valid, s["ref_logp"] - logp, zero)
    kl = torch.exp(back) - back - 1
    surrogate = -torch.minimum(free, held)
    if case["per"] == "token":
        w = 1 / count.sum().clamp(min=1) * valid.float()
    else:
        w = valid.float() / (count[which].clamp(min=1) * (count > 0).sum().clamp(min=1))
    coef = torch.where(free <= held, -free, zero) + case["kl"] * (1 - torch.exp(back))
    stats = [(w * surrogate).sum(), (w * kl).sum(), (w * (held < free)).sum()]
    if not case["kl"]:
        stats[1] = stats[1] * 0
    stats = torch.stack([stats[0] + case["kl"] * stats[1], *stats])
    return {"stats": stats, "logp": logp, "dlogits": _dlogits_plain(s, e, total, valid, at, w * coef)}


def _pref_plain(s):
    case = s["case"]
    logp, e, total, valid, at = _logp_plain(s)
    which, count, add = _segments(s)
    over = count.clamp(min=1) if case["mean"] else torch.ones_like(count)
    ratios = add(torch.where(valid, logp - s["ref_logp"], torch.zeros_like(logp))) / over
    beta, smooth = 0.1, 0.05
    good, bad = ratios[0::2], ratios[1::2]
    pairs = good.numel()
    z = beta * (good - bad)
    if case["form"] == "sigmoid":
        def softplus(v):
            return torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0)

        loss = (1 - smooth) * softplus(-z) + smooth * softplus(z)
        slope = -(1 - smooth) / (1 + torch.exp(z)) + smooth / (1 + torch.exp(-z))
    else:
        loss = (z - 0.5) ** 2
        slope = 2 * (z - 0.5)
    one = slope * beta / pairs
    per_seq = torch.stack([one, -one], 1).reshape(-1) / over
    stats = torch.stack([loss.mean(), beta * good.mean(), beta * bad.mean(), (good > bad).float().mean()])
    return {"stats": stats, "ratios": ratios, "logp": logp,
            "dlogits": _dlogits_plain(s, e, total, valid, at, per_seq[which])}


def _newton_schulz_plain(u):
    x = u.float()
    turned = x.shape[0] > x.shape[1]
    if turned:
        x = x.T
    x = x / (x.square().sum().sqrt() + EPS)
    for _ in range(STEPS):
        a = x @ x.T
        x = A * x + (B * a + C * (a @ a)) @ x
    return x.T if turned else x


def _adjust(r, c):
    return math.sqrt(max(1.0, r / c))


def _ortho_plain(s):
    for g, o in zip(s["grads"], s["outs"]):
        o.copy_(_newton_schulz_plain(g))
    return s["outs"]


def _muon_plain(s):
    for g, m, p, mo, po in zip(s["grads"], s["momenta"], s["params"], s["momenta_out"], s["params_out"]):
        torch.add(g.float(), m, alpha=MU, out=mo)
        u = g.float() + MU * mo if s["case"]["nesterov"] else mo
        po.copy_(p.float() * (1 - LR * DECAY) - LR * _adjust(*p.shape) * _newton_schulz_plain(u))
    return {"params": s["params_out"], "momenta": s["momenta_out"]}


# ---------------------------------------------------------------- one pass


def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "logp":
            return _logp_plain(s)[0]
        return {"policy": _policy_plain, "pref": _pref_plain, "ortho": _ortho_plain, "muon": _muon_plain}[case["op"]](s)
    import gradient_sync_gb300 as g

    if case["op"] == "logp":
        return g.ar_token_logp(s["logits"], s["labels"], temperature=case["tau"], logp=s["logp"])
    if case["op"] == "policy":
        stats, logp, d = g.ar_policy_loss(
            s["logits"], s["labels"], s["old_logp"], s["advantages"], s["seq_start"],
            ref_logp=s["ref_logp"] if case["kl"] else None, clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
            kl_coef=case["kl"], temperature=case["tau"], reduction=case["per"], logp=s["logp"], dlogits=s["dlogits"],
            workspace=s["workspace"])
        return {"stats": stats, "logp": logp, "dlogits": d}
    if case["op"] == "pref":
        stats, ratios, logp, d = g.ar_preference_loss(
            s["logits"], s["labels"], s["ref_logp"], s["seq_start"], beta=0.1, label_smoothing=0.05,
            loss=case["form"], target=0.5, length_normalized=case["mean"], temperature=case["tau"], logp=s["logp"],
            dlogits=s["dlogits"], workspace=s["workspace"])
        return {"stats": stats, "ratios": ratios, "logp": logp, "dlogits": d}
    if case["op"] == "ortho":
        return g.ar_orthogonalize(s["plan"], s["grads"], outs=s["outs"], workspace=s["workspace"])
    g.ar_muon_step(s["plan"], s["params"], s["grads"], s["momenta"], lr=LR, momentum=MU, weight_decay=DECAY,
                   nesterov=case["nesterov"], adjust="shape", params_out=s["params_out"],
                   momenta_out=s["momenta_out"], workspace=s["workspace"])
    return {"params": s["params_out"], "momenta": s["momenta_out"]}


# ---------------------------------------------------------------- the work of one pass


def _ortho_flops(r, c):
    """Products of the Newton-Schulz steps, the two symmetric ones counted at one triangle."""
    m, n = min(r, c), max(r, c)
    return STEPS * (m * m * n + m ** 3 + 2 * m * m * n)


def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] in ("ortho", "muon"):
        n = sum(r * c for r, c in _shapes(case["shapes"]))
        moved = n * (size[case["src"]] + size[case["dst"]])
        if case["op"] == "muon":
            moved += n * (8 + size[case["dst"]])
        return {"bytes": moved, "flops": sum(_ortho_flops(r, c) for r, c in _shapes(case["shapes"]))}
    logits = case["tokens"] * case["vocab"]
    back = case["op"] != "logp"
    return {"bytes": logits * size[case["dtype"]] * (2 if back else 1) + case["tokens"] * 24,
            "flops": logits * (6 if back else 4)}


# ---------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("ortho", "muon"):
        def orthogonal(u):
            wide = u.shape[0] <= u.shape[1]
            y = (u.T if wide else u) / (torch.linalg.vector_norm(u) + EPS)  # at least as many rows as columns
            eye = torch.eye(y.shape[1], dtype=torch.float64, device=y.device)
            for _ in range(STEPS):
                gram = y.T @ y
                y = y @ (A * eye + gram @ (B * eye + C * gram))
            return y.T if wide else y

        if case["op"] == "ortho":
            return [orthogonal(g.double()) for g in s["grads"]]
        params, momenta = [], []
        for g, m, p in zip(s["grads"], s["momenta"], s["params"]):
            m1 = g.double() + MU * m.double()
            u = g.double() + MU * m1 if case["nesterov"] else m1
            momenta.append(m1)
            params.append(p.double() * (1 - LR * DECAY) - LR * _adjust(*p.shape) * orthogonal(u))
        return {"params": params, "momenta": momenta}

    T, S = case["tokens"], case["seqs"]
    start = s["seq_start"].tolist()
    which = torch.empty(T, dtype=torch.long, device="cuda")
    for i in range(S):
        which[start[i]:start[i + 1]] = i
    has = s["labels"] >= 0
    x = s["logits"].double()
    lse = torch.logsumexp(x / case["tau"], 1)
    at = s["labels"].clamp(min=0)
    picked = x.gather(1, at[:, None])[:, 0] / case["tau"] - lse
    logp = torch.where(has, picked, torch.zeros_like(picked))
    if case["op"] == "logp":
        return logp
    leaf = logp.clone().requires_grad_()
    number = torch.zeros(S, dtype=torch.float64, device="cuda").index_add_(0, which, has.double())
    if case["op"] == "policy":
        parts, adv = [], s["advantages"].double()
        old, ref = s["old_logp"].double(), s["ref_logp"].double()
        w = has / has.sum() if case["per"] == "token" else has / (number[which].clamp(min=1) * (number > 0).sum())
        ratio = torch.exp((leaf - old) * has)
        lowest = torch.where(adv >= 0, torch.minimum(ratio, ratio * 0 + 1 + CLIP_HIGH),
                             torch.maximum(ratio, ratio * 0 + 1 - CLIP_LOW))
        parts.append((-adv * lowest * w).sum())
        gap = (ref - leaf) * has
        parts.append((w * (torch.expm1(gap) - gap)).sum() * (1.0 if case["kl"] else 0.0))
        loss = parts[0] + case["kl"] * parts[1]
        out = {"stats": [loss, parts[0], parts[1], (w * ((lowest != ratio))).sum()]}
    else:
        gap = (leaf - s["ref_logp"].double()) * has
        ratios = torch.zeros(S, dtype=torch.float64, device="cuda").index_add(0, which, gap)
        ratios = ratios / number.clamp(min=1) if case["mean"] else ratios
        pair = ratios.reshape(-1, 2)
        z = 0.1 * (pair[:, 0] - pair[:, 1])
        if case["form"] == "sigmoid":
            loss = -(0.95 * torch.nn.functional.logsigmoid(z) + 0.05 * torch.nn.functional.logsigmoid(-z)).mean()
        else:
            loss = ((z - 0.5) ** 2).mean()
        out = {"stats": [loss, 0.1 * pair[:, 0].mean(), 0.1 * pair[:, 1].mean(),
                         (pair[:, 0] > pair[:, 1]).double().mean()], "ratios": ratios.detach()}
    (slope,) = torch.autograd.grad(loss, leaf)
    slope = slope * has / case["tau"]
    x = torch.softmax(x / case["tau"], 1).mul_(-slope[:, None])
    x[torch.arange(T, device="cuda"), at] += slope
    out["stats"] = torch.stack([v.detach() for v in out["stats"]])
    return {**out, "logp": logp, "dlogits": x}
