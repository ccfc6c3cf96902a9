"""What is measured of the losses of post-training over a batch of logits: the log-probabilities of
given tokens (with the entropy, and their gradient), the clipped policy loss with a KL term, the
preference loss of paired sequences, and distillation from a teacher's top logits.

`run` computes a case in its plain form (elementary torch operations in 32 bits; sums over a
sequence and the teacher's remaining mass in 64) or, with `own`, through the package's public
functions. `exact` states the same results from the definitions in 64 bits.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_IGNORED = -100


def _scale(case):
    """What a training step multiplies its loss by: 4096 where the gradient is held in fp16, and
    T^2 for a distillation at temperature T, whose gradients else shrink with it."""
    scale = 4096.0 if case["dtype"] == "f16" else 1.0
    return scale * case["temperature"] ** 2 if case["op"] == "distill" else scale


# ---------------------------------------------------------------- cases

def listed():
    return [
        # scoring a few tokens of one sequence (latency)
        {"name": "logp_few", "op": "logp", "B": 1, "T": 16, "V": 32000, "dtype": "bf16",
         "temperature": 1.0, "entropy": False, "train": False, "sliced": False},
        # the old policy's log-probabilities of a batch of sampled sequences
        {"name": "logp_rollout", "op": "logp", "B": 16, "T": 512, "V": 128256, "dtype": "bf16",
         "temperature": 0.7, "entropy": True, "train": False, "sliced": False},
        # a loss of the user's own over log-probabilities and entropies, odd sizes
        {"name": "logp_train_odd", "op": "logp", "B": 3, "T": 341, "V": 32003, "dtype": "f16",
         "temperature": 1.0, "entropy": True, "train": True, "sliced": False},
        # two short answers (latency of a training step's loss)
        {"name": "policy_few", "op": "policy", "B": 2, "T": 37, "V": 32000, "dtype": "bf16",
         "temperature": 1.0, "kl": 0.05, "entropy": 0.0, "per_token": False, "sliced": False},
        # a training step over 8 x 512 tokens, one advantage a sequence, a KL term
        {"name": "policy_group", "op": "policy", "B": 8, "T": 512, "V": 131072, "dtype": "bf16",
         "temperature": 1.0, "kl": 0.04, "entropy": 0.0, "per_token": False, "sliced": False},
        # fp32 logits without their last position, an advantage a token, an entropy bonus
        {"name": "policy_f32", "op": "policy", "B": 4, "T": 255, "V": 65536, "dtype": "f32",
         "temperature": 0.9, "kl": 0.0, "entropy": 0.01, "per_token": True, "sliced": True},
        # two pairs of short answers (latency)
        {"name": "pref_few", "op": "pref", "B": 2, "T": 48, "V": 32000, "dtype": "bf16",
         "loss": "sigmoid", "smoothing": 0.0, "average": False, "packed": False},
        # a training step over four pairs of 512 tokens
        {"name": "pref_pairs", "op": "pref", "B": 4, "T": 512, "V": 128256, "dtype": "bf16",
         "loss": "sigmoid", "smoothing": 0.1, "average": False, "packed": False},
        # pairs of ragged lengths without padding, odd vocabulary, averages over the lengths
        {"name": "pref_packed", "op": "pref", "B": 7, "T": 150, "V": 32003, "dtype": "f16",
         "loss": "ipo", "smoothing": 0.0, "average": True, "packed": True},
        # a few tokens against a short list (latency)
        {"name": "distill_few", "op": "distill", "B": 1, "T": 32, "V": 32000, "dtype": "bf16",
         "K": 8, "temperature": 1.0, "tail": False, "sliced": False},
        # a training step over 8 x 512 tokens against the teacher's 64 best
        {"name": "distill_top64", "op": "distill", "B": 8, "T": 512, "V": 131072, "dtype": "bf16",
         "K": 64, "temperature": 2.0, "tail": False, "sliced": False},
        # fp32, odd sizes, the teacher's remaining mass as one more outcome
        {"name": "distill_tail", "op": "distill", "B": 3, "T": 333, "V": 50003, "dtype": "f32",
         "K": 100, "temperature": 1.0, "tail": True, "sliced": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("logp", "logp", "policy", "policy", "pref", "pref", "distill", "distill"))
    V = _log(rng, 1000, 131072)
    V = max(1000, V // 64 * 64) if rng.random() < 0.5 else V  # whole vectors, or any
    rows = _log(rng, 16, max(17, min(8192, 2 ** 29 // V)))
    case = {"op": op, "V": V, "dtype": rng.choice(("bf16", "bf16", "f16", "f32"))}
    if op == "pref":
        case["B"] = max(1, min(_log(rng, 1, 16), rows // 8))
        case["T"] = max(4, rows // (2 * case["B"]))
        return {**case, "loss": rng.choice(("sigmoid", "ipo")),
                "smoothing": rng.choice((0.0, 0.1)), "average": rng.random() < 0.5,
                "packed": rng.random() < 0.5}
    case["B"] = max(1, min(_log(rng, 1, 16), rows // 8))
    case["T"] = max(4, rows // case["B"])
    case["sliced"] = rng.random() < 0.3
    case["temperature"] = rng.choice((1.0, 1.0, 0.7, 2.0))
    if op == "logp":
        return {**case, "entropy": rng.random() < 0.5, "train": rng.random() < 0.5}
    if op == "policy":
        return {**case, "kl": rng.choice((0.0, 0.04)), "entropy": rng.choice((0.0, 0.01)),
                "per_token": rng.random() < 0.5}
    return {**case, "K": _log(rng, 4, 128), "tail": rng.random() < 0.5}


def _counted(case):
    """Rows whose token counts: an eighth of the positions is padding or prompt (none of a
    packed batch, whose rows are tokens of the answers only)."""
    if case["op"] == "pref":
        rows = 2 * case["B"] * case["T"]
        return rows if case["packed"] else rows - 2 * case["B"] * (case["T"] // 8)
    return case["B"] * (case["T"] - case["T"] // 8)


def work(case):
    b = 4 if case["dtype"] == "f32" else 2
    rows = case["B"] * case["T"] * (2 if case["op"] == "pref" else 1)
    read = _counted(case) * case["V"]  # rows that do not count need not be read
    grad = rows * case["V"] if case["op"] != "logp" or case["train"] else 0
    small = {"logp": 16, "policy": 36, "pref": 8}.get(case["op"]) or 12 * case["K"]
    return {"bytes": (read + grad) * b + rows * small, "flops": 4 * read + 4 * grad}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    t = _TYPES[case["dtype"]]

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    op, V, T = case["op"], case["V"], case["T"]
    B = case["B"] * (2 if op == "pref" else 1)
    sliced = case.get("sliced", False)
    # logits of a model: a spread of a few units, some tokens far ahead
    logits = torch.empty(B, T + (1 if sliced else 0), V, dtype=t, device=dev)
    tokens = torch.empty(B, T, dtype=torch.int64, device=dev)
    logp = torch.empty(B, T, device=dev)
    for i in range(B):
        x = normal(logits.shape[1], V).mul_(2.0)
        ahead = torch.randint(V, (x.shape[0], 4), generator=g, device=dev)
        x.scatter_add_(1, ahead, 4.0 + 8.0 * uniform(*ahead.shape))
        logits[i] = x.to(t)
        # sampled from the model's distribution
        z = logits[i, :T].float()
        tokens[i] = (z - torch.log(-torch.log(uniform(T, V).clamp_(1e-20, 1 - 6e-8)))).argmax(1)
        z = z / case.get("temperature", 1.0)
        logp[i] = z.gather(1, tokens[i][:, None])[:, 0] - torch.logsumexp(z, 1)
    skip = T // 8
    if skip and not case.get("packed", False):  # a prompt's tokens, and padding behind the answer
        front = torch.randint(skip + 1, (B, 1), generator=g, device=dev)
        at = torch.arange(T, device=dev)[None]
        tokens.masked_fill_((at < front) | (at >= T - skip + front), _IGNORED)
    s = {"case": case, "tokens": tokens}
    x = logits[:, :T] if sliced else logits
    if op == "logp":
        s["d_logp"], s["d_entropy"] = normal(B, T), 0.1 * normal(B, T)
    elif op == "policy":
        # ratios around 1, some past the clip's borders; none within 1e-3 of a border, where a
        # rounding would decide which side a row falls on
        d = 0.2 * normal(B, T)
        for border in (math.log1p(-0.2), math.log1p(0.25)):
            d = torch.where((d - border).abs() < 1e-3, d + 0.01, d)
        s["old"] = logp - d
        s["ref"] = logp - 0.3 * normal(B, T) if case["kl"] else None
        # rewards of both signs whose mean is away from zero (near it, the relative error of a
        # mean loss would say nothing)
        a = uniform(B, T) if case["per_token"] else uniform(B)
        s["advantages"] = torch.where(uniform(*a.shape) < 0.3, -0.5 * a, 1.0 + a)
    elif op == "pref":
        lengths = torch.full((B,), T)
        if case["packed"]:  # ragged lengths, the same number of rows in all
            cut = torch.Generator().manual_seed(seed)
            move = torch.randint(T // 2 + 1, (B // 2,), generator=cut)
            lengths[:B // 2] -= move
            lengths[B // 2:] += move.flip(0)
            s["tokens"] = tokens.reshape(-1)
            x = logits.reshape(-1, V)
        s["offsets"] = torch.cat((torch.zeros(1, dtype=torch.int64), lengths.cumsum(0))).to(dev)
        gone = (s["tokens"] == _IGNORED).reshape(-1)
        sums = _segments(logp.reshape(-1).masked_fill(gone, 0.0).double(), s["offsets"])
        if case["average"]:
            sums = sums / _segments((~gone).double(), s["offsets"]).clamp(min=1.0)
        # the reference model scores a sequence a few units (of an average, tenths) apart
        s["ref"] = (sums + (0.2 if case["average"] else 4.0) * normal(B)).float()
    else:
        T0 = case["temperature"]
        K = case["K"]
        s["teacher"] = torch.empty(B, T, K, dtype=t, device=dev)
        s["index"] = torch.empty(B, T, K, dtype=torch.int64, device=dev)
        s["teacher_lse"] = torch.empty(B, T, device=dev) if case["tail"] else None
        for i in range(B):
            z = (x[i].float() * 0.9 + normal(T, V)).to(t)
            s["teacher"][i], s["index"][i] = torch.topk(z, K, dim=1)
            if case["tail"]:
                s["teacher_lse"][i] = torch.logsumexp(z.double() / T0, 1).float()
        s["index"].masked_fill_((tokens == _IGNORED)[..., None], -1)
    train = op != "logp" or case["train"]
    s["logits"] = x.detach().requires_grad_(train)
    return s


def _segments(v, offsets):
    """Sums of v (64 bits) over the rows between one offset and the next."""
    c = torch.cat((v.new_zeros(1), v.cumsum(0)))[offsets]
    return c[1:] - c[:-1]


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if own:
        return {"logp": _own_logp, "policy": _own_policy, "pref": _own_pref,
                "distill": _own_distill}[case["op"]](s, case)
    with torch.no_grad():
        return {"logp": _plain_logp, "policy": _plain_policy, "pref": _plain_pref,
                "distill": _plain_distill}[case["op"]](s, case)


def _own_logp(s, case):
    import softmax_cross_entropy_gb300 as gbce
    out = gbce.token_log_probs(s["logits"], s["tokens"], temperature=case["temperature"],
                               return_entropy=case["entropy"])
    parts = [out.log_probs, out.entropy] if case["entropy"] else [out]
    res = dict(zip(("log_probs", "entropy"), parts))
    if case["train"]:
        up = [s["d_logp"], s["d_entropy"]][:len(parts)]
        res["dlogits"], = torch.autograd.grad(parts, s["logits"], up)
    return res


def _own_policy(s, case):
    import softmax_cross_entropy_gb300 as gbce
    out = gbce.policy_loss(s["logits"], s["tokens"], s["advantages"], s["old"],
                           ref_log_probs=s["ref"], clip_low=0.2, clip_high=0.25,
                           kl_coef=case["kl"], entropy_coef=case["entropy"],
                           temperature=case["temperature"], scale=_scale(case),
                           return_stats=True)
    dlogits, = torch.autograd.grad(out.loss, s["logits"])
    return {"loss": out.loss, "log_probs": out.log_probs, "entropy": out.entropy,
            "kl": out.kl, "dlogits": dlogits}


def _own_pref(s, case):
    import softmax_cross_entropy_gb300 as gbce
    out = gbce.preference_loss(s["logits"], s["tokens"],
                               offsets=s["offsets"] if case["packed"] else None,
                               ref_log_probs=s["ref"], beta=0.1, loss_type=case["loss"],
                               # (the plain form of "ipo" has no smoothing)
                               label_smoothing=case["smoothing"] * (case["loss"] == "sigmoid"),
                               length_average=case["average"], scale=_scale(case),
                               return_scores=True)
    dlogits, = torch.autograd.grad(out.loss, s["logits"])
    return {"loss": out.loss, "scores": out.scores, "dlogits": dlogits}


def _own_distill(s, case):
    import softmax_cross_entropy_gb300 as gbce
    loss = gbce.distillation_loss(s["logits"], s["teacher"], s["index"],
                                  teacher_lse=s["teacher_lse"],
                                  temperature=case["temperature"],
                                  scale=_scale(case))
    dlogits, = torch.autograd.grad(loss, s["logits"])
    return {"loss": loss, "dlogits": dlogits}


# ---------------------------------------------------------------- plain forms

def _softmax_parts(s, case):
    """(log p over the vocabulary, which rows count, their tokens' places, log p of the tokens)."""
    z = s["logits"].float() / case.get("temperature", 1.0)
    z = z - z.amax(-1, keepdim=True)
    z = z - torch.log(torch.exp(z).sum(-1, keepdim=True))
    if "tokens" not in s:
        return z, None, None, None
    keep = s["tokens"] != _IGNORED
    at = torch.where(keep, s["tokens"], 0)[..., None]
    return z, keep, at, torch.where(keep, z.gather(-1, at)[..., 0], 0.0)


def _gradient(s, case, z, at, c, h, entropy):
    """d(sum c log p_token + h entropy) / d logits, rounded once to the logits' type."""
    p = torch.exp(z)
    d = -(p * c[..., None])
    if h is not None:
        d = d - p * (z + entropy[..., None]) * h[..., None]
    d.scatter_add_(-1, at, c[..., None])
    return (d / case.get("temperature", 1.0)).to(s["logits"].dtype)


def _entropy(z, keep):
    return torch.where(keep, -(torch.exp(z) * z).sum(-1), 0.0)


def _plain_logp(s, case):
    z, keep, at, lp = _softmax_parts(s, case)
    res = {"log_probs": lp}
    if case["entropy"]:
        res["entropy"] = _entropy(z, keep)
    if case["train"]:
        c = torch.where(keep, s["d_logp"], 0.0)
        h = torch.where(keep, s["d_entropy"], 0.0) if case["entropy"] else None
        res["dlogits"] = _gradient(s, case, z, at, c, h, res.get("entropy"))
    return res


def _plain_policy(s, case):
    z, keep, at, lp = _softmax_parts(s, case)
    entropy = _entropy(z, keep)
    n = keep.sum()
    a = s["advantages"] if case["per_token"] else s["advantages"][:, None]
    r = torch.exp(lp - s["old"])
    free = torch.where(a >= 0, r <= 1.25, r >= 0.8)  # not cut by the clip
    loss = -torch.minimum(r * a, r.clamp(0.8, 1.25) * a) - case["entropy"] * entropy
    c = torch.where(free, -a * r, 0.0)
    kl = torch.zeros_like(lp)
    if case["kl"]:
        e = torch.exp(s["ref"] - lp)
        kl = torch.where(keep, e - (s["ref"] - lp) - 1.0, 0.0)
        loss = loss + case["kl"] * kl
        c = c + case["kl"] * (1.0 - e)
    scale = _scale(case) / n
    c = torch.where(keep, c, 0.0) * scale
    h = keep * (-case["entropy"]) * scale if case["entropy"] else None
    return {"loss": (torch.where(keep, loss, 0.0).double().sum() * scale).float(), "log_probs": lp,
            "entropy": entropy, "kl": kl, "dlogits": _gradient(s, case, z, at, c, h, entropy)}


def _plain_pref(s, case):
    z, keep, at, lp = _softmax_parts(s, case)
    flat = lp.reshape(-1).double()
    scores = _segments(flat, s["offsets"])
    n = _segments(keep.reshape(-1).double(), s["offsets"])
    if case["average"]:
        scores = scores / n.clamp(min=1.0)
    B = case["B"]
    delta = (scores[:B] - scores[B:]) - (s["ref"][:B].double() - s["ref"][B:].double())
    if case["loss"] == "ipo":
        gap = delta - 1.0 / (2 * 0.1)
        loss, d = gap * gap, 2.0 * gap
    else:
        e = case["smoothing"]
        q = 1.0 / (1.0 + torch.exp(-0.1 * delta))
        loss = -(1 - e) * torch.log(q) - e * torch.log(1.0 - q)
        d = 0.1 * (q - 1.0 + e)
    d = torch.cat((d, -d)) * (_scale(case) / B)
    if case["average"]:
        d = d / n.clamp(min=1.0)
    sizes = s["offsets"][1:] - s["offsets"][:-1]
    c = torch.repeat_interleave(d, sizes, output_size=flat.numel()).reshape(lp.shape).float()
    return {"loss": (loss.mean() * _scale(case)).float(), "scores": scores.float(),
            "dlogits": _gradient(s, case, z, at, torch.where(keep, c, 0.0), None, None)}


def _plain_distill(s, case):
    z = _softmax_parts({"logits": s["logits"]}, case)[0]
    keep = s["index"][..., 0] >= 0
    at = torch.where(keep[..., None], s["index"], 0)
    own_rows = keep[..., None].float()
    n = keep.sum()
    t = s["teacher"].double() / case["temperature"]
    p = torch.exp(z)
    if case["tail"]:
        lq = t - s["teacher_lse"].double()[..., None]
        q = torch.exp(lq)
        rest = (1.0 - q.sum(-1)).clamp(min=1e-300)
        others = p.scatter(-1, at, 0.0)
        left = others.sum(-1)
        row = (q * (lq - z.gather(-1, at))).sum(-1) + rest * (torch.log(rest) - torch.log(left))
        d = others * (1.0 - (rest / left).float())[..., None]
        d.scatter_(-1, at, p.gather(-1, at) - q.float())
    else:
        lq = t - t.amax(-1, keepdim=True)
        lq = lq - torch.log(torch.exp(lq).sum(-1, keepdim=True))
        q = torch.exp(lq)
        row = (q * (lq - z.gather(-1, at))).sum(-1)
        d = p.scatter_add(-1, at, -q.float())
    scale = _scale(case)
    loss = scale * torch.where(keep, row, 0.0).sum() / n
    d = torch.where(own_rows > 0, d, 0.0) * (scale / case["temperature"] / n)
    return {"loss": loss.float(), "dlogits": d.to(s["logits"].dtype)}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"logp": _exact_logp, "policy": _exact_policy, "pref": _exact_pref,
            "distill": _exact_distill}[case["op"]](s, case)


def _rows(s):
    """The logits' rows and the batch's shape."""
    shape = s["logits"].shape[:-1]
    return s["logits"].detach().reshape(-1, s["logits"].shape[-1]), shape


def _token_scores(s, case, part):
    """log p of the tokens and the entropies of some rows, by autograd's own softmax."""
    x, _ = _rows(s)
    x = x[part].double().requires_grad_()
    full = torch.log_softmax(x / case.get("temperature", 1.0), 1)
    t = s["tokens"].reshape(-1)[part]
    lp = full.gather(1, t.clamp(min=0)[:, None])[:, 0]
    return x, t != _IGNORED, lp, -(full.exp() * full).sum(1)


def _parts(rows, V):
    step = max(1, 2 ** 26 // V)
    return [slice(i, min(rows, i + step)) for i in range(0, rows, step)]


def _exact_logp(s, case):
    x0, shape = _rows(s)
    lps, ents, grads = [], [], []
    for part in _parts(x0.shape[0], case["V"]):
        with torch.set_grad_enabled(case["train"]):
            x, keep, lp, ent = _token_scores(s, case, part)
            if case["train"]:
                total = (lp * s["d_logp"].reshape(-1)[part].double())[keep].sum()
                if case["entropy"]:
                    total = total + (ent * s["d_entropy"].reshape(-1)[part].double())[keep].sum()
                grads.append(torch.autograd.grad(total, x)[0])
        lps.append(torch.where(keep, lp, 0.0).detach())
        ents.append(torch.where(keep, ent, 0.0).detach())
    res = {"log_probs": torch.cat(lps).reshape(shape)}
    if case["entropy"]:
        res["entropy"] = torch.cat(ents).reshape(shape)
    if case["train"]:
        res["dlogits"] = torch.cat(grads).reshape(*shape, -1)
    return res


def _exact_policy(s, case):
    x0, shape = _rows(s)
    n = int((s["tokens"] != _IGNORED).sum())
    adv = s["advantages"] if case["per_token"] else s["advantages"][:, None].expand(shape)
    adv, old = adv.reshape(-1).double(), s["old"].reshape(-1).double()
    ref = None if s["ref"] is None else s["ref"].reshape(-1).double()
    got = {"log_probs": [], "entropy": [], "kl": [], "dlogits": []}
    loss = 0.0
    for part in _parts(x0.shape[0], case["V"]):
        x, keep, lp, ent = _token_scores(s, case, part)
        ratio = (lp - old[part]).exp()
        gain = torch.min(ratio * adv[part], torch.clamp(ratio, 1 - 0.2, 1 + 0.25) * adv[part])
        kl = torch.zeros_like(lp)
        if ref is not None:
            gap = ref[part] - lp
            kl = torch.expm1(gap) - gap
        total = (case["kl"] * kl - gain - case["entropy"] * ent)[keep].sum() / n * _scale(case)
        got["dlogits"].append(torch.autograd.grad(total, x)[0])
        loss = loss + total.detach()
        for name, v in (("log_probs", lp), ("entropy", ent), ("kl", kl)):
            got[name].append(torch.where(keep, v, 0.0).detach())
    res = {k: torch.cat(v).reshape(*shape, *v[0].shape[1:]) for k, v in got.items()}
    return {"loss": loss, **res}


def _exact_pref(s, case):
    x0, shape = _rows(s)
    parts = _parts(x0.shape[0], case["V"])
    with torch.no_grad():
        lp = torch.cat([torch.where(keep, v, 0.0)
                        for _, keep, v, _ in (_token_scores(s, case, p) for p in parts)])
    lp.requires_grad_()
    keep = (s["tokens"] != _IGNORED).reshape(-1)
    ends = s["offsets"].tolist()
    scores = torch.stack([lp[a:b].sum() / (keep[a:b].sum().clamp(min=1) if case["average"] else 1)
                          for a, b in zip(ends, ends[1:])])
    B = case["B"]
    ref = s["ref"].double()
    h = (scores[:B] - ref[:B]) - (scores[B:] - ref[B:])
    if case["loss"] == "ipo":
        loss = ((h - 5.0) ** 2).mean()
    else:
        f = torch.nn.functional.logsigmoid
        loss = -((1 - case["smoothing"]) * f(0.1 * h) + case["smoothing"] * f(-0.1 * h)).mean()
    loss = loss * _scale(case)
    c, = torch.autograd.grad(loss, lp)
    grads = []
    for part in parts:
        x, keep, v, _ = _token_scores(s, case, part)
        grads.append(torch.autograd.grad((v * c[part])[keep].sum(), x)[0])
    return {"loss": loss.detach(), "scores": scores.detach(),
            "dlogits": torch.cat(grads).reshape(*shape, -1)}


def _exact_distill(s, case):
    x0, shape = _rows(s)
    K, T0 = case["K"], case["temperature"]
    index, teacher = s["index"].reshape(-1, K), s["teacher"].reshape(-1, K)
    n = int((index[:, 0] >= 0).sum())
    loss, grads = 0.0, []
    for part in _parts(x0.shape[0], case["V"]):
        x = x0[part].double().requires_grad_()
        full = torch.log_softmax(x / T0, 1)
        keep = index[part][:, 0] >= 0
        at = index[part].clamp(min=0)
        t = teacher[part].double() / T0
        if case["tail"]:
            q = (t - s["teacher_lse"].reshape(-1)[part].double()[:, None]).exp()
            q = torch.cat((q, (1 - q.sum(1, keepdim=True)).clamp(min=1e-300)), 1)
            rest = full.scatter(1, at, -math.inf).logsumexp(1, keepdim=True)
            p = torch.cat((full.gather(1, at), rest), 1)
        else:
            q, p = torch.softmax(t, 1), full.gather(1, at)
        total = _scale(case) * (q * (q.log() - p)).sum(1)[keep].sum() / n
        grads.append(torch.autograd.grad(total, x)[0])
        loss = loss + total.detach()
    return {"loss": loss, "dlogits": torch.cat(grads).reshape(*shape, -1)}
