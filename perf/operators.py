"""What is measured of the operators around the cross-entropy: the gated feed-forward block (its
forward, its forward with the gradients, its form for a few tokens), dropout from a counter-based
generator (alone, and with the residual sum), and one step of beam search (the selection over
beams and vocabulary, then the reordering of the beams' states).

`run` computes a case in its plain form (elementary torch operations in 32 bits, in 64 for the
scores of the beams) or, with `own`, through the package's public functions. `exact` states the
same results from the definitions in 64 bits.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of one sequence: the block's latency when generating
        {"name": "ffn_token", "op": "ffn", "train": False, "rows": 1, "H": 4096, "I": 12288,
         "act": "silu", "dtype": "bf16", "p": 0.0, "residual": True},
        # a batch of sequences generating together (batch 5, 8 beams)
        {"name": "ffn_tokens_40", "op": "ffn", "train": False, "rows": 40, "H": 2048, "I": 8192,
         "act": "gelu_tanh", "dtype": "f16", "p": 0.0, "residual": True},
        # a prompt of odd length
        {"name": "ffn_prompt_1023", "op": "ffn", "train": False, "rows": 1023, "H": 4096,
         "I": 12288, "act": "silu", "dtype": "bf16", "p": 0.0, "residual": False},
        # a training step of the block over 8 x 512 tokens
        {"name": "ffn_train_4096", "op": "ffn", "train": True, "rows": 4096, "H": 4096,
         "I": 12288, "act": "silu", "dtype": "bf16", "p": 0.1, "residual": True},
        # a training step of a small model with sizes that fill no tile
        {"name": "ffn_train_odd", "op": "ffn", "train": True, "rows": 333, "H": 1000, "I": 2731,
         "act": "gelu", "dtype": "f16", "p": 0.1, "residual": False},
        # dropout on a small odd activation (launch latency)
        {"name": "dropout_small", "op": "dropout", "rows": 127, "cols": 1001, "dtype": "f16",
         "p": 0.5, "residual": False},
        # the residual branch of a training step, 8 x 512 tokens and its gradient
        {"name": "dropout_residual", "op": "dropout", "rows": 4096, "cols": 4096, "dtype": "bf16",
         "p": 0.1, "residual": True},
        # a large fp32 activation
        {"name": "dropout_f32", "op": "dropout", "rows": 16384, "cols": 8192, "dtype": "f32",
         "p": 0.2, "residual": False},
        # one sequence, four beams: the latency of a step
        {"name": "beam_one", "op": "beam", "B": 1, "K": 4, "V": 32000, "M": 8, "dtype": "bf16",
         "finished": 0, "masked": False, "heads": 4, "length": 64, "dim": 64},
        # a serving batch, some beams finished, a cache to reorder
        {"name": "beam_serving", "op": "beam", "B": 16, "K": 8, "V": 128256, "M": 16,
         "dtype": "bf16", "finished": 1, "masked": False, "heads": 8, "length": 512, "dim": 128},
        # odd sizes, forbidden tokens, a beam with every token forbidden
        {"name": "beam_masked", "op": "beam", "B": 7, "K": 5, "V": 32003, "M": 10, "dtype": "f16",
         "finished": 1, "masked": True, "heads": 3, "length": 77, "dim": 40},
        # a large batch of fp32 logits
        {"name": "beam_large", "op": "beam", "B": 64, "K": 8, "V": 131072, "M": 16,
         "dtype": "f32", "finished": 0, "masked": False, "heads": 8, "length": 128, "dim": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("ffn", "ffn", "ffn_train", "dropout", "beam", "beam"))
    if kind in ("ffn", "ffn_train"):
        train = kind == "ffn_train"
        step = rng.choice((1, 8, 64))  # sizes of every kind: odd ones, whole vectors, whole tiles
        H = max(step, _log(rng, 200, 4096) // step * step)
        I = max(step, _log(rng, 400, 12288) // step * step)
        return {"op": "ffn", "train": train, "rows": _log(rng, 24 if train else 1, 4096),
                "H": H, "I": I, "act": rng.choice(("silu", "gelu", "gelu_tanh")),
                "dtype": rng.choice(("bf16", "f16")), "p": rng.choice((0.0, 0.1)) if train else 0.0,
                "residual": rng.random() < 0.5}
    if kind == "dropout":
        return {"op": "dropout", "rows": _log(rng, 16, 16384), "cols": _log(rng, 64, 8192),
                "dtype": rng.choice(("bf16", "f16", "f32")), "p": rng.choice((0.05, 0.1, 0.3, 0.5)),
                "residual": rng.random() < 0.5}
    B, K = _log(rng, 1, 48), rng.randint(1, 10)
    return {"op": "beam", "B": B, "K": K, "V": _log(rng, 1000, 131072), "M": rng.choice((K, 2 * K)),
            "dtype": rng.choice(("bf16", "f16", "f32")), "finished": rng.randint(0, min(2, K - 1)),
            "masked": rng.random() < 0.4, "heads": rng.randint(1, 8), "length": _log(rng, 8, 256),
            "dim": rng.choice((33, 40, 64, 128))}


def work(case):
    if case["op"] == "ffn":
        b, rows, H, I = 2, case["rows"], case["H"], case["I"]
        tokens, weights = rows * H * b, 3 * H * I * b
        res = tokens if case["residual"] else 0
        if not case["train"]:
            return {"bytes": 2 * tokens + res + weights, "flops": 6 * rows * H * I}
        # x, residual, dy and the weights in; y, dx and the weights' gradients out
        return {"bytes": 4 * tokens + res + 2 * weights, "flops": 18 * rows * H * I}
    if case["op"] == "dropout":
        n = case["rows"] * case["cols"] * (4 if case["dtype"] == "f32" else 2)
        # x, dy (and the residual) in; y and dx out
        return {"bytes": n * (5 if case["residual"] else 4), "flops": 0}
    b = 4 if case["dtype"] == "f32" else 2
    rows = case["B"] * case["K"]
    logits = case["B"] * (case["K"] - case["finished"]) * case["V"] * b
    states = 2 * rows * case["heads"] * case["length"] * case["dim"] * 2
    return {"bytes": logits + 2 * states + rows * 5 + case["B"] * case["M"] * 20,
            "flops": 3 * case["B"] * (case["K"] - case["finished"]) * case["V"]}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    t = _TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=t):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dtype)

    if case["op"] == "ffn":
        rows, H, I = case["rows"], case["H"], case["I"]
        s = {"x": normal(rows, H), "w_gate": normal(I, H, scale=H ** -0.5),
             "w_up": normal(I, H, scale=H ** -0.5), "w_down": normal(H, I, scale=I ** -0.5),
             "residual": normal(rows, H) if case["residual"] else None,
             "dy": normal(rows, H) if case["train"] else None}
        if case["train"]:
            for k in ("x", "w_gate", "w_up", "w_down", "residual"):
                if s[k] is not None:
                    s[k].requires_grad_()
    elif case["op"] == "dropout":
        rows, cols = case["rows"], case["cols"]
        s = {"x": normal(rows, cols).requires_grad_(), "dy": normal(rows, cols),
             "residual": normal(rows, cols).requires_grad_() if case["residual"] else None}
    else:
        B, K, V = case["B"], case["K"], case["V"]
        logits = normal(B, K, V, scale=3.0)
        if case["masked"]:  # a third of the vocabulary forbidden, and one beam's whole row
            logits.masked_fill_(torch.rand(V, generator=g, device=dev) < 0.33, -math.inf)
            logits[B // 2, K - 1] = -math.inf
        finished = torch.zeros(B, K, dtype=torch.bool, device=dev)
        finished[:, :case["finished"]] = True
        cache = (B * K, case["heads"], case["length"], case["dim"])
        s = {"logits": logits, "finished": finished,
             "scores": -10.0 * torch.rand(B, K, generator=g, device=dev),
             "states": [normal(*cache, dtype=torch.bfloat16) for _ in range(2)]}
    s["case"] = case
    s["seed"] = seed * 7919 + 12345  # dropout's seed: an input like the others
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if case["op"] == "ffn":
        return _own_ffn(s, case) if own else _plain_ffn(s, case)
    if case["op"] == "dropout":
        return _own_dropout(s, case) if own else _plain_dropout(s, case)
    return _own_beam(s, case) if own else _plain_beam(s, case)


def _own_ffn(s, case):
    import softmax_cross_entropy_gb300 as gbce
    y = gbce.gated_feed_forward(s["x"], s["w_gate"], s["w_up"], s["w_down"],
                                activation=case["act"], residual=s["residual"],
                                dropout_p=case["p"], seed=s["seed"])
    if not case["train"]:
        return {"y": y}
    leaves = ["x", "w_gate", "w_up", "w_down"] + (["residual"] if case["residual"] else [])
    grads = torch.autograd.grad(y, [s[k] for k in leaves], s["dy"])
    return {"y": y, **{"d" + k: d for k, d in zip(leaves, grads)}}


def _own_dropout(s, case):
    import softmax_cross_entropy_gb300 as gbce
    y = gbce.dropout(s["x"], case["p"], s["seed"], residual=s["residual"])
    leaves = ["x"] + (["residual"] if case["residual"] else [])
    grads = torch.autograd.grad(y, [s[k] for k in leaves], s["dy"])
    return {"y": y, **{"d" + k: d for k, d in zip(leaves, grads)}}


def _own_beam(s, case):
    import softmax_cross_entropy_gb300 as gbce
    best = gbce.beam_search_step(s["logits"], s["scores"], num_candidates=case["M"],
                                 finished=s["finished"], pad_token=1)
    gbce.beam_reorder(s["states"], best.beams[:, :case["K"]], inplace=True)
    return {"scores": best.scores, "beams": best.beams, "tokens": best.tokens,
            "states": s["states"]}


# ---------------------------------------------------------------- plain forms

_LOW = 0xFFFFFFFF


def _random_words(n, seed, dev):
    """n 32-bit numbers (in int64) of Philox 4x32 with 10 rounds, key = seed, word i from lane
    i mod 4 of the counter i // 4. A product of two 32-bit numbers keeps its 64 bits in int64,
    whatever its sign, so a shift and a mask give its halves."""
    groups = (n + 3) // 4
    i = torch.arange(groups, dtype=torch.int64, device=dev)
    c0, c1 = i & _LOW, i >> 32
    c2, c3 = torch.zeros_like(i), torch.zeros_like(i)
    k0, k1 = seed & _LOW, (seed >> 32) & _LOW
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((b >> 32) & _LOW) ^ c1 ^ k0, b & _LOW,
                          ((a >> 32) & _LOW) ^ c3 ^ k1, a & _LOW)
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    return torch.stack((c0, c1, c2, c3), 1).reshape(-1)[:n]


def _factor(shape, p, seed, dev):
    """What dropout multiplies by: 0 or 1 / (1 - p)."""
    if p == 0.0:
        return torch.ones((), device=dev)
    kept = _random_words(math.prod(shape), seed, dev).reshape(shape) >= int(p * 2.0 ** 32)
    return kept * (1.0 / (1.0 - p))


def _act(g, name):
    """The activation and its derivative."""
    if name == "silu":
        q = 1.0 / (1.0 + torch.exp(-g))
        return g * q, q * (1.0 + g * (1.0 - q))
    if name == "gelu":
        c = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * c, c + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return (0.5 * g * (1.0 + t),
            0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * g * g))


def _plain_ffn(s, case):
    with torch.no_grad():
        t = s["x"].dtype
        x, wg, wu, wd = (s[k].float() for k in ("x", "w_gate", "w_up", "w_down"))
        g, u = x @ wg.T, x @ wu.T
        a, slope = _act(g, case["act"])
        h = a * u
        f = _factor(s["x"].shape, case["p"], s["seed"], x.device)
        y = (h @ wd.T) * f
        if case["residual"]:
            y = y + s["residual"].float()
        if not case["train"]:
            return {"y": y.to(t)}
        d = s["dy"].float() * f
        dh = d @ wd
        dg, du = dh * u * slope, dh * a
        out = {"y": y.to(t), "dx": (dg @ wg + du @ wu).to(t), "dw_gate": (dg.T @ x).to(t),
               "dw_up": (du.T @ x).to(t), "dw_down": (d.T @ h).to(t)}
        if case["residual"]:
            out["dresidual"] = s["dy"]
        return out


def _plain_dropout(s, case):
    with torch.no_grad():
        t = s["x"].dtype
        f = _factor(s["x"].shape, case["p"], s["seed"], s["x"].device)
        y = s["x"].float() * f
        if case["residual"]:
            y = y + s["residual"].float()
        out = {"y": y.to(t), "dx": (s["dy"].float() * f).to(t)}
        if case["residual"]:
            out["dresidual"] = s["dy"]
        return out


def _plain_beam(s, case):
    B, K, V, M = (case[k] for k in ("B", "K", "V", "M"))
    x = s["logits"].double()
    top = x.amax(2, keepdim=True)
    lse = top + torch.log(torch.exp(x - top).sum(2, keepdim=True))
    new = x - lse  # NaN where a row has no token left
    new = torch.where(torch.isnan(new), -math.inf, new)
    only = torch.full((V,), -math.inf, dtype=torch.float64, device=x.device)
    only[1] = 0.0  # a finished beam goes on with the padding token alone
    new = torch.where(s["finished"][..., None], only, new) + s["scores"].double()[..., None]
    new = new.reshape(B, K * V)
    # the best M and some more, so that equal ones at the end are put in order too
    some = min(K * V, M + 64)
    val, at = torch.topk(new, some, dim=1)
    at, by = torch.sort(at, dim=1)
    val, by = torch.sort(val.gather(1, by), dim=1, descending=True, stable=True)
    val, at = val[:, :M], at.gather(1, by)[:, :M]
    none = val == -math.inf
    beams = torch.where(none, -1, at // V)
    tokens = torch.where(none, 1, at % V)
    first = torch.arange(B, device=x.device)[:, None] * K
    stay = torch.arange(K, device=x.device)[None]
    rows = (first + torch.where(beams[:, :K] < 0, stay, beams[:, :K])).reshape(-1)
    for state in s["states"]:
        state.copy_(state[rows])
    return {"scores": val.float(), "beams": beams, "tokens": tokens, "states": s["states"]}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "ffn":
            return _exact_ffn(s, case)
        if case["op"] == "dropout":
            return _exact_dropout(s, case)
        return _exact_beam(s, case)


def _exact_mask(shape, p, seed, dev):
    """Philox 4x32-10 again, its products from 16-bit halves: bit i is whether element i stays."""
    n = math.prod(shape)
    ctr = torch.arange((n + 3) // 4, device=dev)
    x = [ctr % 2 ** 32, ctr // 2 ** 32, 0 * ctr, 0 * ctr]
    key = [seed % 2 ** 32, seed // 2 ** 32 % 2 ** 32]

    def mul(m, v):  # (high, low) 32 bits of m v
        low, mid = m * (v & 0xFFFF), m * (v >> 16)  # below 2^48 each
        mid = mid + (low >> 16)
        return mid >> 16, ((mid & 0xFFFF) << 16) | (low & 0xFFFF)

    for r in range(10):
        h0, l0 = mul(0xD2511F53, x[0])
        h1, l1 = mul(0xCD9E8D57, x[2])
        x = [h1 ^ x[1] ^ ((key[0] + r * 0x9E3779B9) % 2 ** 32), l1,
             h0 ^ x[3] ^ ((key[1] + r * 0xBB67AE85) % 2 ** 32), l0]
    words = torch.stack(x, dim=-1).flatten()[:n].reshape(shape)
    return words >= math.floor(p * 2 ** 32)


def _dropped(v, p, seed):
    if p == 0.0:
        return v
    return torch.where(_exact_mask(v.shape, p, seed, v.device), v / (1.0 - p), 0.0)


def _exact_ffn(s, case):
    x, wg, wu, wd = (s[k].detach().double() for k in ("x", "w_gate", "w_up", "w_down"))
    g, u = torch.einsum("rh,ih->ri", x, wg), torch.einsum("rh,ih->ri", x, wu)
    if case["act"] == "silu":
        q = torch.sigmoid(g)
        a, da = g * q, q + g * q * (1 - q)
    elif case["act"] == "gelu":
        cdf = 0.5 * torch.erfc(-g / math.sqrt(2))
        a, da = g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    else:  # 0.5 (1 + tanh z) is the logistic function of 2 z
        z2 = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        q = torch.sigmoid(z2)
        a, da = g * q, q + g * q * (1 - q) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * g * g)
    y = _dropped(torch.einsum("ri,hi->rh", a * u, wd), case["p"], s["seed"])
    if case["residual"]:
        y = y + s["residual"].double()
    if not case["train"]:
        return {"y": y}
    dz = _dropped(s["dy"].double(), case["p"], s["seed"])
    dh = torch.einsum("rh,hi->ri", dz, wd)
    out = {"y": y,
           "dx": torch.einsum("ri,ih->rh", dh * u * da, wg) + torch.einsum("ri,ih->rh", dh * a, wu),
           "dw_gate": torch.einsum("ri,rh->ih", dh * u * da, x),
           "dw_up": torch.einsum("ri,rh->ih", dh * a, x),
           "dw_down": torch.einsum("rh,ri->hi", dz, a * u)}
    if case["residual"]:
        out["dresidual"] = s["dy"].double()
    return out


def _exact_dropout(s, case):
    y = _dropped(s["x"].detach().double(), case["p"], s["seed"])
    out = {"dx": _dropped(s["dy"].double(), case["p"], s["seed"])}
    if case["residual"]:
        y = y + s["residual"].detach().double()
        out["dresidual"] = s["dy"].double()
    return {"y": y, **out}


def _exact_beam(s, case):
    """One batch entry after another: log-softmax, the sums, a stable sort of the best."""
    B, K, V, M = (case[k] for k in ("B", "K", "V", "M"))
    scores, beams, tokens, rows = [], [], [], []
    for b in range(B):
        total = torch.log_softmax(s["logits"][b].double(), 1).nan_to_num(nan=-math.inf)
        total = total + s["scores"][b].double()[:, None]
        for k in range(case["finished"]):
            total[k] = -math.inf
            total[k, 1] = s["scores"][b, k].double()
        total = total.reshape(-1)
        bound = torch.topk(total, min(M, K * V)).values[-1]
        at = torch.nonzero(total >= bound).reshape(-1)  # in order of the index
        at = at[torch.sort(total[at], descending=True, stable=True).indices][:M]
        val = total[at]
        gone = torch.isinf(val)
        scores.append(val)
        beams.append(torch.where(gone, -1, at // V))
        tokens.append(torch.where(gone, 1, at % V))
        stay = torch.arange(K, device=at.device)
        rows.append(b * K + torch.where(beams[b][:K] < 0, stay, beams[b][:K]))
    pick = torch.cat(rows)
    return {"scores": torch.stack(scores), "beams": torch.stack(beams),
            "tokens": torch.stack(tokens), "states": [t.double()[pick] for t in s["states"]]}
