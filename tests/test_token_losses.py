"""Log-probabilities of tokens, the policy, preference and distillation losses:
the references' own pins and the refusals (CPU), and the kernels against the
definitions in 64 bits (GPU)."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import token_losses_ref as ref

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
IGN = -100


# ---------------------------------------------------------------- CPU: the references

def _fd(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("T", [1.0, 0.7])
def test_reference_gradients_are_those_of_differences(T):
    rng = np.random.default_rng(3)
    x = rng.normal(size=(4, 5)) * 2
    tok = np.array([1, IGN, 4, 0])
    gl, gh = rng.normal(size=4), rng.normal(size=4)
    f = lambda v: (lambda lp, h, _: (lp * gl + h * gh).sum())(*ref.log_probs(v, tok, T, IGN))
    assert np.allclose(ref.log_probs(x, tok, T, IGN, gl, gh)[2], _fd(f, x), atol=1e-8)
    adv, old, rl = rng.normal(size=4), rng.normal(size=4) - 1.5, rng.normal(size=4) - 1.5
    args = (tok, adv, old, rl, np.array([1.0, 2.0, 0.5, 0.0]), 0.2, 0.3, 0.1, 0.05, T, IGN, 1.5)
    for red in ("mean", "sum"):
        p = lambda v: ref.policy(v, *args, red)[0]
        assert np.allclose(ref.policy(x, *args, red)[5], _fd(p, x), atol=1e-7)
    idx = np.array([[1, 2], [-1, 3], [4, -1], [0, 0]])
    v = rng.normal(size=(4, 2))
    for lse in (None, np.full(4, 3.0)):
        q = lambda u: ref.distill(u, v, idx, lse, None, T, 1.0, "mean")[0]
        assert np.allclose(ref.distill(x, v, idx, lse, None, T, 1.0, "mean")[1], _fd(q, x), atol=1e-7)
    for kind, av in itertools.product(("sigmoid", "hinge", "ipo"), (False, True)):
        b = [(0, 2), (2, 4)]
        a = (tok, b, np.array([0.3, -0.2]), kind, 0.4, 0.0, 0.1 if kind == "sigmoid" else 0.0, av, IGN,
             1.0, "mean")
        q = lambda u: ref.preference(u, *a)[0]
        assert np.allclose(ref.preference(x, *a)[2], _fd(q, x), atol=1e-7)


# ---------------------------------------------------------------- CPU: refusals

def _x(**over):
    from softmax_cross_entropy_gb300 import _lib
    a = dict(data=64, grad=128, dtype=_lib.CE_BF16, temperature=1.0, rows=4, V=8, inner=4,
             outer_stride=0, row_stride=8)
    a.update(over)
    return ctypes.byref(_lib.Rows(*(a[k] for k, _ in _lib.Rows._fields_)))


_BAD_ROWS = [dict(dtype=5), dict(rows=-1), dict(V=0), dict(inner=0), dict(temperature=0.0),
             dict(temperature=float("nan")), dict(temperature=float("inf")), dict(row_stride=7),
             dict(inner=2, outer_stride=15), dict(inner=1, outer_stride=7), dict(data=None),
             dict(data=65), dict(grad=130)]


def _calls(**o):
    """Each entry point with valid arguments, as a function of ce_rows."""
    from softmax_cross_entropy_gb300 import _lib as L
    n = L.ce_rows_workspace_bytes()

    def arg(name, default):
        return o.get(name, default)

    return {
        "logp": lambda x: L.ce_token_logp(x, arg("tokens", 16), IGN, arg("flags", 0),
                                          arg("logp", 16), None, arg("kept", None), None),
        "logp_bwd": lambda x: L.ce_token_logp_bwd(x, arg("tokens", 16), IGN, arg("flags", 0),
                                                  arg("kept", 16), None, None, None),
        "policy": lambda x: L.ce_policy_loss(
            x, arg("tokens", 16), IGN, arg("flags", 0), arg("adv", 16), arg("adv_rows", 1), None,
            None, None, arg("lo", 0.2), arg("hi", 0.2), arg("kl", 0.0), arg("ent", 0.0),
            arg("scale", 1.0), arg("red", 2), arg("loss", 16), None, None, None, None,
            arg("ws", 16), arg("ws_bytes", n), None),
        "distill": lambda x: L.ce_distill_loss(
            x, arg("teacher", 16), arg("tdt", 1), arg("index", 16), arg("K", 4), None,
            arg("flags", 0), None, arg("scale", 1.0), arg("red", 2), arg("loss", 16),
            arg("ws", 16), arg("ws_bytes", n), None),
        "pref": lambda x: L.ce_preference_loss(
            x, arg("tokens", 16), IGN, arg("flags", 0), arg("pairs", 2), arg("offsets", None), None,
            arg("kind", 0), arg("beta", 0.1), arg("margin", 0.0), arg("smooth", 0.0), 0,
            arg("scale", 1.0), arg("red", 2), arg("loss", 16), None, None, arg("kept", 16),
            arg("ws", 16), arg("ws_bytes", n), None),
        "pref_bwd": lambda x: L.ce_preference_loss_bwd(
            x, arg("tokens", 16), IGN, arg("flags", 0), arg("pairs", 2), arg("offsets", None),
            arg("kept", 16), arg("dscore", 16), arg("g", 16), 0, None),
        "scale": lambda x: L.ce_rows_scale(x, arg("g", 16), 0, None),
    }


@pytest.mark.parametrize("over", _BAD_ROWS)
@pytest.mark.parametrize("call", ["logp", "logp_bwd", "policy", "distill", "pref", "pref_bwd", "scale"])
def test_library_refuses_rows(call, over):
    from softmax_cross_entropy_gb300 import _lib
    assert _calls()[call](_x(**over)) == _lib.CE_ERR_INVALID_ARG


@pytest.mark.parametrize("call", ["logp", "logp_bwd", "policy", "distill", "pref", "pref_bwd", "scale"])
def test_library_refuses_large_vocabularies(call):
    from softmax_cross_entropy_gb300 import _lib
    big = dict(V=2**19 + 1, row_stride=2**20)
    assert _calls()[call](_x(**big)) == _lib.CE_ERR_UNSUPPORTED
    assert _calls()[call](_x(rows=2**41)) == _lib.CE_ERR_UNSUPPORTED


_NAN, _INF = float("nan"), float("inf")


@pytest.mark.parametrize("call,over", [
    ("logp", dict(tokens=None)), ("logp", dict(logp=None)), ("logp", dict(flags=1)),
    ("logp", dict(kept=8)), ("logp_bwd", dict(tokens=None)), ("logp_bwd", dict(kept=None)),
    ("logp_bwd", dict(kept=8)), ("logp_bwd", dict(flags=2)),
    ("policy", dict(tokens=None)), ("policy", dict(adv=None)), ("policy", dict(adv_rows=0)),
    ("policy", dict(lo=-0.1)), ("policy", dict(lo=1.1)), ("policy", dict(lo=_NAN)),
    ("policy", dict(hi=-0.1)), ("policy", dict(hi=_NAN)), ("policy", dict(kl=_INF)),
    ("policy", dict(ent=_NAN)), ("policy", dict(scale=_INF)), ("policy", dict(red=3)),
    ("policy", dict(loss=None)), ("policy", dict(ws=None)), ("policy", dict(ws=24)),
    ("policy", dict(ws_bytes=100)), ("policy", dict(flags=32)),
    ("distill", dict(teacher=None)), ("distill", dict(index=None)), ("distill", dict(tdt=3)),
    ("distill", dict(K=0)), ("distill", dict(scale=_NAN)), ("distill", dict(red=-1)),
    ("distill", dict(loss=None)), ("distill", dict(ws=None)), ("distill", dict(ws_bytes=0)),
    ("pref", dict(tokens=None)), ("pref", dict(pairs=-1)), ("pref", dict(pairs=3)),
    ("pref", dict(pairs=0)), ("pref", dict(kind=3)), ("pref", dict(beta=0.0)),
    ("pref", dict(beta=_NAN)), ("pref", dict(margin=_INF)), ("pref", dict(smooth=1.5)),
    ("pref", dict(smooth=0.1, kind=1)), ("pref", dict(margin=0.5, kind=2)), ("pref", dict(red=7)),
    ("pref", dict(loss=None)), ("pref", dict(kept=None)), ("pref", dict(kept=24)),
    ("pref", dict(ws=None)), ("pref", dict(scale=_NAN)),
    ("pref_bwd", dict(kept=None)), ("pref_bwd", dict(dscore=None)), ("pref_bwd", dict(g=None)),
    ("pref_bwd", dict(pairs=3)), ("scale", dict(g=None)),
])
def test_library_refuses(call, over):
    from softmax_cross_entropy_gb300 import _lib
    assert _calls(**over)[call](_x()) == _lib.CE_ERR_INVALID_ARG


def test_library_refuses_long_lists():
    from softmax_cross_entropy_gb300 import _lib
    assert _calls(K=257)["distill"](_x()) == _lib.CE_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", ["logp_bwd", "pref_bwd", "scale"])
def test_library_refuses_a_backward_without_a_gradient(call):
    from softmax_cross_entropy_gb300 import _lib
    assert _calls()[call](_x(grad=None)) == _lib.CE_ERR_INVALID_ARG


def test_library_takes_empty_batches_without_a_reduction():
    from softmax_cross_entropy_gb300 import _lib
    x = _x(rows=0, data=None, grad=None)
    assert _calls()["logp"](x) == _lib.CE_OK
    assert _calls(red=0)["policy"](x) == _lib.CE_OK
    assert _calls(red=0)["distill"](x) == _lib.CE_OK
    assert _calls(red=0, pairs=0)["pref"](x) == _lib.CE_OK


@pytest.mark.parametrize("make,want", [
    (lambda x: x, (28, 28, 0, 10)), (lambda x: x[:, :-1], (24, 6, 70, 10)),
    (lambda x: x[:, 1:], (24, 6, 70, 10)), (lambda x: x[::2], (14, 7, 140, 10)),
    (lambda x: x[:, :1], (4, 4, 0, 70)), (lambda x: x[:, :, :5], (28, 28, 0, 10)),
    (lambda x: x[:, ::2, :5], (16, 4, 70, 20)), (lambda x: x[:0], (0, 1, 0, 10)),
    (lambda x: x.transpose(0, 1), None), (lambda x: x[:1].expand(3, 7, 10), None),
    (lambda x: x[:, :, ::2], None), (lambda x: x.reshape(2, 2, 7, 10)[:, :, :6], (24, 6, 70, 10)),
    (lambda x: x.reshape(2, 2, 7, 10)[:, :1, :6], (12, 6, 140, 10)),
])
def test_layout_of_views(make, want):
    from softmax_cross_entropy_gb300.token_losses import _rows_of
    x = torch.arange(280.0).reshape(4, 7, 10)
    v = make(x)
    got = _rows_of(v)
    assert got == want
    if want:  # the rows that the layout names are v's
        rows, inner, outer, step = got
        flat, off = x.reshape(-1), v.storage_offset()
        for r, row in enumerate(v.reshape(-1, v.shape[-1])):
            at = off + (r // inner) * outer + (r % inner) * step
            assert torch.equal(flat[at:at + v.shape[-1]], row)


@pytest.mark.parametrize("make", [lambda x: x, lambda x: x[:, :-1], lambda x: x[:, 1:],
                                  lambda x: x.reshape(-1)[3:3 + 6 * 9].reshape(6, 9)])
def test_gradient_has_the_layout_of_the_logits(make):
    from softmax_cross_entropy_gb300.token_losses import _gradient_like, _rows_of
    x = make(torch.zeros(4, 7, 9, dtype=torch.bfloat16))
    g = _gradient_like(x, _rows_of(x))
    assert g.shape == x.shape and g.stride() == x.stride() and g.dtype == x.dtype
    assert (g.data_ptr() - x.data_ptr()) % 16 == 0


def _wrappers():
    import softmax_cross_entropy_gb300 as gbce
    return {"token_log_probs": lambda x, t: gbce.token_log_probs(x, t),
            "policy_loss": lambda x, t: gbce.policy_loss(x, t, torch.ones(t.shape, device=t.device)),
            "preference_loss": lambda x, t: gbce.preference_loss(x, t),
            "distillation_loss": lambda x, t: gbce.distillation_loss(
                x, torch.zeros(*t.shape, 3, device=t.device), t[..., None].expand(*t.shape, 3))}


@pytest.mark.parametrize("name", ["token_log_probs", "policy_loss", "preference_loss",
                                  "distillation_loss"])
def test_wrappers_refuse(name, monkeypatch):
    from softmax_cross_entropy_gb300 import token_losses
    f = _wrappers()[name]
    x, t = torch.zeros(2, 3, 8), torch.zeros(2, 3, dtype=torch.int64)
    with pytest.raises(ValueError):
        f(x, t)  # not on CUDA
    monkeypatch.setattr(token_losses, "require_cuda", lambda *a: None)
    with pytest.raises(TypeError):
        f(x.double(), t)
    with pytest.raises(ValueError):
        f(x[..., :0], t)
    with pytest.raises(ValueError):
        f(x, t[:1])
    with pytest.raises(TypeError):
        f(x, t.to(torch.int16))


def test_wrappers_refuse_options(monkeypatch):
    import softmax_cross_entropy_gb300 as gbce
    from softmax_cross_entropy_gb300 import token_losses
    monkeypatch.setattr(token_losses, "require_cuda", lambda *a: None)
    x, t = torch.zeros(2, 3, 8), torch.zeros(2, 3, dtype=torch.int64)
    a = torch.zeros(2, 3)

    def bad(kind, f, *args, **kw):
        with pytest.raises(kind):
            f(*args, **kw)

    for T in (0.0, -1.0, _NAN, _INF):
        bad(ValueError, gbce.token_log_probs, x, t, temperature=T)
        bad(ValueError, gbce.policy_loss, x, t, a, temperature=T)
    for kw in (dict(reduction="avg"), dict(clip_low=2.0), dict(clip_high=-1.0), dict(kl_coef=_INF),
               dict(scale=_NAN), dict(weight=a[:1]), dict(old_log_probs=a.long()),
               dict(ref_log_probs=a.clone().requires_grad_())):
        bad((ValueError, TypeError), gbce.policy_loss, x, t, a, **kw)
    bad(ValueError, gbce.policy_loss, x, t, a[:1])
    bad(ValueError, gbce.policy_loss, x, t, torch.zeros(3))
    bad(ValueError, gbce.policy_loss, x, t, torch.zeros(()))
    bad(ValueError, gbce.policy_loss, x, t, 1.0)
    bad(ValueError, gbce.policy_loss, x, t, torch.zeros(2, 3, 1))
    bad(ValueError, gbce.preference_loss, x[:1], t[:1])
    bad(ValueError, gbce.preference_loss, x[0], t[0])
    bad(ValueError, gbce.preference_loss, x[0], t[0], offsets=torch.tensor([0, 3]))
    bad(ValueError, gbce.preference_loss, x[0], t[0], offsets=torch.tensor([0.0, 1.0, 3.0]))
    bad(ValueError, gbce.preference_loss, x, t, offsets=torch.tensor([0, 1, 3]))
    for kw in (dict(loss_type="dpo"), dict(beta=0.0), dict(label_smoothing=2.0),
               dict(loss_type="ipo", margin=1.0), dict(loss_type="hinge", label_smoothing=0.1),
               dict(ref_log_probs=torch.zeros(3)), dict(reduction="max")):
        bad(ValueError, gbce.preference_loss, x, t, **kw)
    v, i = torch.zeros(2, 3, 4), torch.zeros(2, 3, 4, dtype=torch.int64)
    bad(ValueError, gbce.distillation_loss, x, v, i[..., :3])
    bad(ValueError, gbce.distillation_loss, x, v[..., :0], i[..., :0])
    bad(TypeError, gbce.distillation_loss, x, v.double(), i)
    bad(ValueError, gbce.distillation_loss, x, v.clone().requires_grad_(), i)
    bad(ValueError, gbce.distillation_loss, x, v, i, teacher_lse=a[:1])
    for f, args in ((gbce.token_log_probs, (t,)), (gbce.policy_loss, (t, a)),
                    (gbce.distillation_loss, (v, i))):
        bad(ValueError, f, torch.zeros(2, 8, 3).transpose(1, 2), *args, inplace=True)
        bad(ValueError, f, torch.zeros(1, 1, 8).expand(2, 3, 8), *args, inplace=True)


def test_tangents_and_second_derivatives_are_refused(monkeypatch):
    # (the library's calls are stand-ins here)
    import softmax_cross_entropy_gb300 as gbce
    from softmax_cross_entropy_gb300 import _lib, token_losses
    from torch.autograd import forward_ad
    monkeypatch.setattr(token_losses, "require_cuda", lambda *a: None)
    monkeypatch.setattr(token_losses, "on", lambda d: __import__("contextlib").nullcontext())
    monkeypatch.setattr(token_losses, "stream", lambda d: None)
    for name in ("ce_token_logp", "ce_token_logp_bwd", "ce_policy_loss", "ce_distill_loss",
                 "ce_preference_loss", "ce_preference_loss_bwd", "ce_rows_scale"):
        monkeypatch.setattr(_lib, name, lambda *a: _lib.CE_OK)
    x, t = torch.zeros(2, 3, 8), torch.zeros(2, 3, dtype=torch.int64)
    for name, f in _wrappers().items():
        with forward_ad.dual_level():
            with pytest.raises(NotImplementedError):
                f(forward_ad.make_dual(x, torch.ones_like(x)), t)
        leaf = x.clone().requires_grad_()
        out = f(leaf, t)
        with pytest.raises(RuntimeError, match="once"):
            torch.autograd.grad(out.sum(), leaf, create_graph=True)
        out = f(leaf, t)
        torch.autograd.grad(out.sum(), leaf, retain_graph=True)
        if name in ("policy_loss", "distillation_loss"):  # their gradient was given away
            with pytest.raises(RuntimeError, match="earlier backward"):
                torch.autograd.grad(out.sum(), leaf)
        else:
            torch.autograd.grad(out.sum(), leaf)


# ---------------------------------------------------------------- GPU

@pytest.fixture(autouse=True)
def no_device_errors(request):
    """Nothing was recorded on the device: no wait ran out, no token out of range."""
    yield
    if request.node.get_closest_marker("gpu"):
        import softmax_cross_entropy_gb300 as gbce
        from softmax_cross_entropy_gb300 import _lib
        assert gbce.device_status() == _lib.CE_OK


def put(x64, dtype, how="plain"):
    """(logits on the GPU, the values they hold in 64 bits [rows, V])."""
    t = torch.from_numpy(x64).to(DT[dtype])
    held = t.double().numpy().reshape(-1, t.shape[-1])
    B, T, V = t.shape
    if how == "plain":
        g = t.cuda()
    elif how in ("front", "back"):  # a view without the last, or the first, position
        full = torch.full((B, T + 1, V), float("nan"), dtype=t.dtype, device="cuda")
        g = full[:, :-1] if how == "front" else full[:, 1:]
        g.copy_(t)
    elif how == "odd":  # an unaligned base
        flat = torch.full((t.numel() + 3,), float("nan"), dtype=t.dtype, device="cuda")
        g = flat[3:].view(B, T, V)
        g.copy_(t)
    elif how == "wide":  # rows with a gap behind them
        full = torch.full((B, T, V + 5), float("nan"), dtype=t.dtype, device="cuda")
        g = full[..., :V]
        g.copy_(t)
    else:  # classes not contiguous: a copy is made
        g = t.cuda().transpose(1, 2).contiguous().transpose(1, 2)
    return g, held


def logits64(rng, B, T, V, mask=0.0, low=False):
    x = rng.normal(size=(B, T, V)) * 2.5
    x[..., rng.integers(V)] += 6.0
    if mask and V > 3:
        gone = rng.random(V) < mask
        gone[0] = False
        x[..., gone] = -3.0e38 if low else -np.inf
    return x


def logp_tol(lp, V, span=20.0):
    """How far a log-probability may be off. The sum S: an element is 2^arg with arg rounded three
    times (2^-24 of arg each, |arg| up to log2(e) span for elements that count: 3 * 2^-24 * 29 <
    2^-17.5 in log2 units, weighted by what they contribute; of the elements within a few units of
    the mean contribution arg is below 12: 2^-19) and ex2's error (2^-22); adding V elements by 128
    lanes or more rounds V / 128 + 16 times (2^-24 each). The logarithm and the result: 2^-23 of
    them."""
    return 2.0 ** -19 + (V / 128 + 16) * 2.0 ** -24 + 2.0 ** -23 * (np.abs(lp) + np.log(V) + 1)


def grad_tol(g, p, size, dtype, V):
    """size [rows]: the coefficients' magnitude. The element p_j has the relative error of S's
    (logp_tol), of the kept maximum's difference times c (2^-22 of arg <= 40) and ex2: below
    2^-17 in all, and its coefficient one of 2^-17 more (a ratio's exponent is lp's error). Then
    one rounding to the type. ex2 gives 0 for results below 2^-126, fp32's smallest normal: an
    element that small is off by up to 2^-126 times its coefficient (bf16 and fp32, which have
    subnormals below it, show that)."""
    eps = torch.finfo(DT[dtype]).eps / 2
    tiny = torch.finfo(DT[dtype]).smallest_normal * eps
    rel = 2.0 ** -16 + V / 128 * 2.0 ** -24
    return np.abs(g) * eps + size[:, None] * (p * rel + 2.0 ** -126) + tiny


def tokens_for(rng, B, T, V, skip=0.2):
    t = rng.integers(0, V, size=(B, T))
    t[rng.random((B, T)) < skip] = IGN
    return t


def cuda(a, dtype=None):
    t = torch.as_tensor(np.asarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def close(got, want, tol, what=""):
    got = got.detach().double().cpu().numpy()
    want = np.asarray(want)
    got = got.reshape(want.shape)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    off = np.abs(got - want)[fine]
    tol = np.broadcast_to(tol, want.shape)[fine]
    worst = np.argmax(off - tol) if off.size else 0
    assert (off <= tol).all(), f"{what}: off by {off[worst]:.3e}, may be {tol[worst]:.3e}"


def plus_zero(t):
    """Every element is exact +0."""
    return torch.all(t == 0) and not torch.any(torch.signbit(t))


def probs(held, T):
    return np.stack([ref.softmax_row(r, T)[2] for r in held])


SIZES = [(1, 1, 1), (2, 3, 2), (1, 5, 7), (3, 2, 8), (2, 2, 33), (2, 9, 1000), (1, 3, 4096),
         (2, 4, 4099), (1, 3, 16384), (2, 2, 32003), (1, 2, 65536), (1, 2, 131072), (1, 2, 262145)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,T,V", SIZES)
@pytest.mark.parametrize("entropy", [False, True])
def test_log_probs(B, T, V, dtype, entropy):
    import softmax_cross_entropy_gb300 as gbce
    rng = np.random.default_rng(V + B)
    temp = 0.7 if V % 2 else 1.0
    x, held = put(logits64(rng, B, T, V, mask=0.3 if V > 1000 else 0.0), dtype,
                  ("plain", "front", "odd", "wide", "copy")[(V + T) % 5])
    tok = tokens_for(rng, B, T, V)
    gl, gh = rng.normal(size=(B, T)), rng.normal(size=(B, T))
    flat = tok.reshape(-1)
    x = x.detach().requires_grad_()
    got = gbce.token_log_probs(x, cuda(tok, torch.int32 if V % 3 else None), temperature=temp,
                               return_entropy=entropy)
    lp, h = got if entropy else (got, None)
    want = ref.log_probs(held, flat, temp, IGN, gl.reshape(-1), gh.reshape(-1) if entropy else None)
    close(lp, want[0].reshape(B, T), logp_tol(np.where(np.isfinite(want[0]), want[0], 0), V).reshape(B, T), "lp")
    outs, ups = [lp], [cuda(gl).float()]
    if entropy:  # the sum of p arg: arg's own roundings and clamped p, times H's size
        close(h, want[1].reshape(B, T), logp_tol(want[1], V).reshape(B, T) * 2, "entropy")
        outs.append(h)
        ups.append(cuda(gh).float())
    (dx,) = torch.autograd.grad(outs, x, ups)
    size = np.abs(gl.reshape(-1))
    if entropy:
        size = size + np.abs(gh.reshape(-1)) * (np.log(V) + 45)
    p = probs(held, temp)
    onto = np.zeros_like(p)
    for r, t in enumerate(flat):
        if t >= 0:
            onto[r, t] = 1.0
    # (at the token g_lp (1 - p): the coefficient's own rounding, 2^-22)
    tol = grad_tol(want[2], p + onto * 2.0 ** -6, size / temp, dtype, V)
    close(dx.reshape(-1, V), want[2], tol, "dx")
    gone = dx.reshape(-1, V)[torch.as_tensor(flat == IGN)]
    assert plus_zero(gone)
    # the same call without a gradient, and again: the same bits
    with torch.no_grad():
        again = gbce.token_log_probs(x, cuda(tok), temperature=temp, return_entropy=entropy)
    assert torch.equal(again[0] if entropy else again, lp)


def _policy_case(rng, B, T, V, dtype, how, mask=0.0):
    x, held = put(logits64(rng, B, T, V, mask), dtype, how)
    tok = tokens_for(rng, B, T, V)
    if mask:  # no token at -inf
        for b, s in np.ndindex(B, T):
            if tok[b, s] >= 0 and not np.isfinite(held.reshape(B, T, V)[b, s, tok[b, s]]):
                tok[b, s] = 0
    return x, held, tok


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,T,V", SIZES)
@pytest.mark.parametrize("red,kl,ent,stats", [("mean", 0.1, 0.0, True), ("sum", 0.0, 0.02, False),
                                              ("none", 0.1, 0.02, True), ("mean", 0.0, 0.0, False)])
def test_policy(B, T, V, dtype, red, kl, ent, stats):
    import softmax_cross_entropy_gb300 as gbce
    rng = np.random.default_rng(V * 7 + B)
    temp = 1.3 if V % 2 else 1.0
    how = ("plain", "front", "odd", "wide", "back")[(V + T) % 5]
    x, held, tok = _policy_case(rng, B, T, V, dtype, how, 0.3 if V > 1000 else 0.0)
    flat = tok.reshape(-1)
    lp = ref.log_probs(held, flat, temp, IGN)[0]
    d = rng.normal(size=B * T) * 0.3
    for border in (np.log1p(-0.2), np.log1p(0.3)):  # (no ratio where a rounding picks the side)
        d = np.where(np.abs(d - border) < 1e-3, d + 5e-3, d)
    old = np.float32(lp - d).astype(np.float64)
    rl = np.float32(lp - rng.normal(size=B * T) * 0.3).astype(np.float64) if kl else None
    per_token = V % 2 == 0
    adv = np.float32(rng.normal(size=(B, T) if per_token else (B,))).astype(np.float64)
    w = np.float32(rng.random(B * T)).astype(np.float64) if red == "sum" else None
    scale = 64.0
    wide = np.broadcast_to(adv if per_token else adv[:, None], (B, T)).reshape(-1)
    want = ref.policy(held, flat, wide, old, rl, w, 0.2, 0.3, kl, ent, temp, IGN, scale, red)
    x = x.detach().requires_grad_()
    shape = lambda a: None if a is None else cuda(a).float().reshape(B, T)
    out = gbce.policy_loss(x, cuda(tok), cuda(adv).float(), shape(old), ref_log_probs=shape(rl),
                           weight=shape(w), clip_low=0.2, clip_high=0.3, kl_coef=kl,
                           entropy_coef=ent, temperature=temp, scale=scale, reduction=red,
                           return_stats=stats)
    loss = out.loss if stats else out
    tlp = logp_tol(lp, V)
    # a row's loss: the ratio's and the KL's exponents are off as lp is, expf by 2^-22 more
    ratio = np.exp(d)
    one = (np.abs(wide) * ratio * 2 + kl * (np.exp(lp * 0 + 1) * 4)) * (tlp + 2.0 ** -21) + ent * 2 * tlp + 2.0 ** -22
    f = np.zeros(B * T)
    keep = flat != IGN
    ww = np.ones(B * T) if w is None else w
    f[keep] = (scale * ww / (ww[keep].sum() if red == "mean" else 1.0))[keep]
    tol = one * np.abs(f)
    if red == "none":
        close(loss, want[0].reshape(B, T), (tol + np.abs(want[0]) * 2.0 ** -22).reshape(B, T), "loss")
    else:
        close(loss, want[0], tol.sum() + np.abs(np.nan_to_num(want[0])) * 2.0 ** -22, "loss")
    if stats:
        close(out.log_probs, want[1].reshape(B, T), tlp.reshape(B, T), "lp")
        close(out.entropy, want[2].reshape(B, T), 2 * logp_tol(want[2], V).reshape(B, T), "entropy")
        g = 0 if rl is None else np.abs(rl - lp)
        close(out.kl, want[3].reshape(B, T), (np.expm1(g) * (tlp + 2.0 ** -22) + 2.0 ** -23).reshape(B, T)
              if rl is not None else 0.0, "kl")
        assert np.array_equal(out.clipped.cpu().numpy().reshape(-1), want[4])
    up = torch.ones_like(loss)
    if red == "none":
        up = cuda(rng.integers(0, 3, size=(B, T))).float()
    (dx,) = torch.autograd.grad(loss, x, up)
    rows_up = up.double().cpu().numpy().reshape(-1) if red == "none" else np.ones(B * T)
    wdx = want[5] * rows_up[:, None]
    c, hcoef = want[6]
    p = probs(held, temp)
    onto = np.zeros_like(p)
    onto[np.nonzero(keep)[0], flat[keep]] = 1.0
    size = (np.abs(f) * (np.abs(wide) * ratio + kl * 3) + np.abs(hcoef) * (np.log(V) + 45)) * rows_up / temp
    # (at the token the slope itself: off by lp's error and expf's, 2^-21, relative)
    tol = grad_tol(wdx, p + onto * (tlp + 2.0 ** -20)[:, None] * 2.0 ** 16, size, dtype, V)
    if red == "none":  # rounded once in the forward, and once more by the factor
        tol = tol * 2
    close(dx.reshape(-1, V), wdx, tol, "dx")
    assert plus_zero(dx.reshape(-1, V)[torch.as_tensor(~keep)])


def _list_case(rng, B, T, V, K, dtype, how, tail, dup):
    x, held = put(logits64(rng, B, T, V), dtype, how)
    rows = B * T
    index = np.stack([rng.permutation(V)[:K] if K <= V else rng.integers(0, V, size=K)
                      for _ in range(rows)])
    if dup and K > 2:
        index[:, K // 2] = index[:, 0]
        index[0, -1] = index[0, 0]
    teacher = torch.as_tensor(rng.normal(size=(rows, K)) * 2).to(DT[dtype])
    index[rng.random((rows, K)) < 0.1] = -1
    index[rng.random(rows) < 0.2, 0] = -7
    lse = None
    if tail:  # the list holds between half and nearly all of the mass
        v = np.where(index >= 0, teacher.double().numpy(), -np.inf)
        lse = np.log(np.exp(v).sum(1) + 1e-300) + rng.uniform(0.001, 0.7, size=rows)
        lse = np.float32(lse).astype(np.float64)
    return x, held, index, teacher, lse


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,T,V", SIZES)
@pytest.mark.parametrize("K,tail,red", [(1, False, "mean"), (8, True, "mean"), (64, False, "none"),
                                        (100, True, "sum"), (256, True, "none")])
def test_distillation(B, T, V, dtype, K, tail, red):
    import softmax_cross_entropy_gb300 as gbce
    if K > V and K > 8:
        pytest.skip("a list longer than the vocabulary")
    rng = np.random.default_rng(V * 11 + K)
    temp = 1.0 if tail else 2.0
    how = ("plain", "front", "odd", "wide", "back")[(V + K) % 5]
    x, held, index, teacher, lse = _list_case(rng, B, T, V, K, dtype, how, tail, K % 8 == 0)
    w = np.float32(rng.random(B * T) + 0.1).astype(np.float64) if red == "sum" else None
    scale = 64.0
    want, wdx, keep = ref.distill(held, teacher.double().numpy(), index, lse, w, temp, scale, red)
    x = x.detach().requires_grad_()
    loss = gbce.distillation_loss(
        x, teacher.cuda().reshape(B, T, K),
        cuda(index, torch.int32 if K % 3 else None).reshape(B, T, K),
        teacher_lse=None if lse is None else cuda(lse).float().reshape(B, T), temperature=temp,
        weight=None if w is None else cuda(w).float().reshape(B, T), scale=scale, reduction=red)
    (dx,) = torch.autograd.grad(loss, x, torch.ones_like(loss))
    ww = np.ones(B * T) if w is None else w
    f = np.where(keep, scale * ww / (ww[keep].sum() if red == "mean" else 1.0), 0.0)
    # a row's loss: q (log q - log p) with both logarithms off as log-probabilities are, q by
    # 2^-22; the remaining mass is held in 64 bits, its logarithm's error is that of the mass
    # outside the list (a sum of its own: relative 2^-18) times its share
    row = 3 * logp_tol(np.full(B * T, 25.0), V) + 2.0 ** -18
    tol = row * f
    if red == "none":
        close(loss, want.reshape(B, T), (tol + np.abs(want) * 2.0 ** -22).reshape(B, T), "loss")
    else:
        close(loss, want, tol.sum() + np.abs(np.nan_to_num(want)) * 2.0 ** -22, "loss")
    p = probs(held, temp)
    # mass and q add to one term each: p (mass) - q, and outside the list p (mass - rest / left)
    onto = np.zeros_like(p)
    left = np.ones(B * T)
    for r in range(B * T):
        ok = index[r] >= 0
        onto[r, index[r][ok]] = 1.0
        left[r] = max(p[r][onto[r] == 0].sum(), 1e-30)
    out = p * (1 + (1 - onto) * (1.0 / left[:, None] if tail else 0.0))
    close(dx.reshape(-1, V), wdx, grad_tol(wdx, out + onto * 2.0 ** -5, f / temp, dtype, V), "dx")
    assert plus_zero(dx.reshape(-1, V)[torch.as_tensor(~keep)])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("P,T,V", [(1, 1, 2), (2, 5, 33), (3, 40, 1000), (1, 300, 257), (2, 3, 32003),
                                   (1, 2, 131072)])
@pytest.mark.parametrize("kind,average,red,packed", [
    ("sigmoid", False, "mean", False), ("sigmoid", True, "none", True), ("ipo", True, "mean", True),
    ("hinge", False, "sum", False), ("ipo", False, "none", False), ("hinge", True, "mean", True)])
def test_preference(P, T, V, dtype, kind, average, red, packed):
    import softmax_cross_entropy_gb300 as gbce
    rng = np.random.default_rng(V * 3 + P)
    how = ("plain", "front", "odd", "wide", "back")[(V + P) % 5]
    x, held = put(logits64(rng, 2 * P, T, V), dtype, "plain" if packed else how)
    rows = 2 * P * T
    tok = tokens_for(rng, 2 * P, T, V).reshape(-1)
    if packed:  # rows in front of the first and behind the last sequence, an empty sequence
        cut = np.sort(rng.integers(0, rows + 1, size=2 * P - 1))
        off = np.concatenate([[min(1, cut[0])], cut, [max(cut[-1], rows - 1)]])
        bounds = list(zip(off[:-1], off[1:]))
    else:
        bounds = [(s * T, (s + 1) * T) for s in range(2 * P)]
    smooth = 0.1 if kind == "sigmoid" else 0.0
    margin = 0.0 if kind == "ipo" else 0.3
    rs = np.float32(rng.normal(size=2 * P)).astype(np.float64)
    beta, scale = 0.25, 32.0
    want = ref.preference(held, tok, bounds, rs, kind, beta, margin, smooth, average, IGN, scale, red)
    x = x.detach()
    x = (x.reshape(rows, V) if packed else x).requires_grad_()
    out = gbce.preference_loss(x, cuda(tok) if packed else cuda(tok).reshape(2 * P, T),
                               offsets=cuda(off) if packed else None, ref_log_probs=cuda(rs).float(),
                               beta=beta, loss_type=kind, label_smoothing=smooth, margin=margin,
                               length_average=average, scale=scale, reduction=red,
                               return_scores=True)
    lp = ref.log_probs(held, tok, 1.0, IGN)[0]
    per = logp_tol(lp, V)
    err = np.array([per[a:b].mean() if average and b > a else per[a:b].sum() for a, b in bounds])
    # a score adds its tokens' errors (64 bits) and rounds once
    close(out.scores, want[1], err + np.abs(want[1]) * 2.0 ** -23, "scores")
    d = (want[1][:P] - want[1][P:]) - (rs[:P] - rs[P:])
    steep = 2 * np.abs(d - 0.5 / beta) + err.max() * 2 if kind == "ipo" else beta
    f = scale / (P if red == "mean" else 1)
    tol = steep * (err[:P] + err[P:]) * f
    if red == "none":
        close(out.loss, want[0], tol + np.abs(want[0]) * 2.0 ** -22, "loss")
    else:
        close(out.loss, want[0], tol.sum() + np.abs(want[0]) * 2.0 ** -22, "loss")
    up = torch.ones_like(out.loss) if red != "none" else cuda(rng.integers(0, 3, size=P)).float()
    (dx,) = torch.autograd.grad(out.loss, x, up)
    g = want[3].copy()
    size = np.zeros(rows)
    curve = np.broadcast_to(2.0 if kind == "ipo" else beta * beta, (P,)) * (err[:P] + err[P:]) * f
    for s, (a, b) in enumerate(bounds):
        k = float(up[s % P]) if red == "none" else 1.0
        n = max(1, (tok[a:b] != IGN).sum()) if average else 1
        g[a:b] *= k
        size[a:b] = curve[s % P] / n * k  # the derivative's own error
    p = probs(held, 1.0)
    wdx = -p * g[:, None]
    onto = np.zeros_like(p)
    ok = np.nonzero(tok >= 0)[0]
    wdx[ok, tok[ok]] += g[ok]
    onto[ok, tok[ok]] = 1.0
    tol = grad_tol(wdx, p + onto * 2.0 ** -5, np.abs(g), dtype, V) + size[:, None] * (p + onto)
    close(dx.reshape(-1, V), wdx, tol, "dx")
    if packed:
        assert plus_zero(dx[:off[0]]) and plus_zero(dx[off[-1]:])


# ---- values that are not finite, or are the type's lowest

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [40, 5000, 70001])
def test_masked_and_infinite_values(V, dtype):
    import softmax_cross_entropy_gb300 as gbce
    low = torch.finfo(DT[dtype]).min
    x = torch.zeros(8, V, dtype=DT[dtype], device="cuda")
    x[0] = low                       # all at the type's lowest value: uniform
    x[1] = -np.inf                   # nothing left: NaN
    x[2, 1:] = -np.inf               # one class left: certain
    x[3, 5] = np.inf                 # NaN
    x[4, 7] = float("nan")           # NaN
    x[5] = float("nan")              # ignored: not read
    x[6, ::2] = low
    x[7, ::2] = -np.inf
    tok = torch.tensor([3, 3, 0, 3, 3, IGN, 1, 2], device="cuda")
    x.requires_grad_()
    lp, h = gbce.token_log_probs(x, tok, return_entropy=True)
    half = V // 2
    logV, logh = np.log(V), np.log(half)
    want = np.array([-logV, np.nan, 0.0, np.nan, np.nan, 0.0, -logh, -np.inf])
    close(lp, want, logp_tol(10.0, V), "lp")
    close(h, np.array([logV, np.nan, 0.0, np.nan, np.nan, 0.0, logh, logh]), 2 * logp_tol(10.0, V), "h")
    (dx,) = torch.autograd.grad([lp, h], x, [torch.ones(8, device="cuda"), torch.zeros(8, device="cuda")])
    assert torch.isnan(dx[[1, 3, 4]]).all() and plus_zero(dx[5])
    assert torch.equal(dx[2], torch.zeros_like(dx[2]))
    assert (dx[6, ::2] == 0).all() and (dx[7, 4::2] == 0).all() and float(dx[7, 2].float()) == 1.0
    good = [0, 2, 5, 6]
    adv = torch.ones(8, device="cuda")
    loss = gbce.policy_loss(x[good], tok[good], adv[good], reduction="none", entropy_coef=0.1)
    assert torch.isfinite(loss).all() and float(loss[2]) == 0.0
    g, = torch.autograd.grad(loss.sum(), x)
    assert torch.isfinite(g[good].float()).all() and plus_zero(g[5])
    # a teacher that names classes the student has at -inf: infinite, and a finite gradient
    idx = torch.tensor([[0, 1]], device="cuda").expand(8, 2)
    t = torch.zeros(8, 2, dtype=DT[dtype], device="cuda")
    loss = gbce.distillation_loss(x[[0, 7]], t[:2], idx[:2], reduction="none")
    assert np.isclose(float(loss[0]), np.log(0.5) + logV, rtol=1e-5) and float(loss[1]) == np.inf
    g, = torch.autograd.grad(loss.sum(), x)
    assert torch.isfinite(g[[0, 7]].float()).all()
    t[:, 0] = -np.inf  # the teacher gives it nothing: no term
    loss = gbce.distillation_loss(x[[0, 7]].detach(), t[:2], idx[:2], reduction="none")
    assert np.allclose(loss.cpu().numpy(), [logV, logh], rtol=1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [6, 4099])
def test_a_list_of_every_class_has_no_remaining_mass(V):
    import softmax_cross_entropy_gb300 as gbce
    rng = np.random.default_rng(1)
    K = min(V, 256)
    x = torch.full((3, V), -np.inf, device="cuda")
    x[:, :K] = cuda(rng.normal(size=(3, K))).float()
    v = cuda(rng.normal(size=(3, K))).float()
    idx = torch.arange(K, device="cuda").expand(3, K)
    lse = torch.logsumexp(v.double(), 1).float() + 1e-6  # (a rounding above the list's)
    x.requires_grad_()
    loss = gbce.distillation_loss(x, v, idx, teacher_lse=lse)
    g, = torch.autograd.grad(loss, x)
    want, wdx, _ = ref.distill(x.detach().double().cpu().numpy(), v.double().cpu().numpy(),
                               idx.cpu().numpy(), lse.double().cpu().numpy(), None, 1.0, 1.0, "mean")
    close(loss, want, 3 * logp_tol(10.0, V))
    close(g, wdx, 2.0 ** -18)


@pytest.mark.gpu
@pytest.mark.parametrize("red", ["mean", "sum", "none"])
def test_nothing_counts(red):
    import softmax_cross_entropy_gb300 as gbce
    x = torch.full((2, 3, 50), float("nan"), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    tok = torch.full((2, 3), IGN, device="cuda")
    a = torch.ones(2, 3, device="cuda")
    idx = torch.full((2, 3, 4), -1, device="cuda")
    for f in (lambda: gbce.policy_loss(x, tok, a, reduction=red),
              lambda: gbce.distillation_loss(x, torch.zeros(2, 3, 4, device="cuda"), idx, reduction=red)):
        loss = f()
        g, = torch.autograd.grad(loss, x, torch.ones_like(loss))
        assert plus_zero(g)
        assert torch.isnan(loss) if red == "mean" else (loss == 0).all()
    loss = gbce.preference_loss(x, tok, reduction=red)  # two empty sequences: equal scores
    g, = torch.autograd.grad(loss, x, torch.ones_like(loss))
    assert plus_zero(g) and np.isclose(float(loss.sum()), np.log(2), rtol=1e-6)


@pytest.mark.gpu
@pytest.mark.parametrize("red", ["mean", "sum", "none"])
def test_empty_batches(red):
    import softmax_cross_entropy_gb300 as gbce
    x = torch.zeros(0, 3, 50, device="cuda", requires_grad=True)
    tok = torch.zeros(0, 3, dtype=torch.int64, device="cuda")
    f32 = dict(device="cuda")
    assert gbce.token_log_probs(x, tok).shape == (0, 3)
    for loss in (gbce.policy_loss(x, tok, torch.zeros(0, 3, **f32), reduction=red),
                 gbce.distillation_loss(x, torch.zeros(0, 3, 2, **f32),
                                        torch.zeros(0, 3, 2, dtype=torch.int64, **f32), reduction=red),
                 gbce.preference_loss(x, tok, reduction=red)):
        if red == "none":
            assert loss.numel() == 0
        else:
            assert torch.isnan(loss) if red == "mean" else float(loss) == 0.0
        g, = torch.autograd.grad(loss, x, torch.ones_like(loss))
        assert g.shape == x.shape


@pytest.mark.gpu
def test_out_of_range_tokens_are_reported():
    import softmax_cross_entropy_gb300 as gbce
    from softmax_cross_entropy_gb300 import _lib
    x = torch.randn(4, 100, device="cuda")
    assert gbce.device_status() == _lib.CE_OK
    for bad in (100, -1, 2 ** 40):
        tok = torch.tensor([1, bad, 2, IGN], device="cuda")
        lp = gbce.token_log_probs(x, tok)
        assert gbce.device_status() == _lib.CE_ERR_TARGET_RANGE and float(lp[1]) == 0.0
        loss = gbce.policy_loss(x, tok, torch.ones(4, device="cuda"))
        assert gbce.device_status() == _lib.CE_ERR_TARGET_RANGE
        assert np.isclose(float(loss), -1.0)  # two rows count
    idx = torch.tensor([[1, 100], [100, 1], [-1, 100], [3, -5]], device="cuda")
    loss = gbce.distillation_loss(x, torch.zeros(4, 2, device="cuda"), idx, reduction="none")
    assert gbce.device_status() == _lib.CE_ERR_TARGET_RANGE
    want = ref.distill(x.double().cpu().numpy(), np.zeros((4, 2)), idx.cpu().numpy(), None, None, 1.0,
                       1.0, "none")[0]
    close(loss, want, logp_tol(10.0, 100))
    gbce.distillation_loss(x[3:], torch.zeros(1, 2, device="cuda"), idx[3:])
    assert gbce.device_status() == _lib.CE_OK


# ---- how they are called

def _four(x, tok, **kw):
    """Each loss on logits x [4, T, V] and its own arguments, made from a fixed seed."""
    import softmax_cross_entropy_gb300 as gbce
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    shape = tok.shape
    adv = torch.randn(shape, generator=g, device="cuda")
    old = torch.randn(shape, generator=g, device="cuda") * 0.1 - 5
    idx = torch.randint(x.shape[-1], (*shape, 9), generator=g, device="cuda")
    val = torch.randn(*shape, 9, generator=g, device="cuda")
    return {"logp": lambda x: gbce.token_log_probs(x, tok, **kw).sum(),
            "policy": lambda x: gbce.policy_loss(x, tok, adv, old, ref_log_probs=old, kl_coef=0.1, **kw),
            "pref": lambda x: gbce.preference_loss(x, tok, **kw),
            "distill": lambda x: gbce.distillation_loss(x, val, idx, **kw)}


ALL = ["logp", "policy", "pref", "distill"]


@pytest.mark.gpu
@pytest.mark.parametrize("name", ALL)
@pytest.mark.parametrize("view", [False, True])
def test_in_place(name, view):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    tok = torch.randint(1001, (4, 6), generator=g, device="cuda")
    tok[0, 2] = IGN
    full = torch.randn(4, 7, 1001, generator=g, device="cuda").bfloat16()
    x = full[:, :-1] if view else full[:, :-1].contiguous()
    leaf = x.detach().requires_grad_()
    want, = torch.autograd.grad(_four(leaf, tok)[name](leaf), leaf)
    held = full[:, -1].clone()
    at = x.detach().requires_grad_()
    mid = at.view_as(at)  # an intermediate result, as a model's logits are
    loss = _four(mid, tok, inplace=True)[name](mid)
    got, = torch.autograd.grad(loss, at)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)
    if view:
        assert torch.equal(full[:, -1], held)  # what lies between the rows is left alone


@pytest.mark.gpu
@pytest.mark.parametrize("name", ALL)
def test_in_place_is_seen_by_other_users_of_the_logits(name):
    tok = torch.zeros(4, 3, dtype=torch.int64, device="cuda")
    leaf = torch.randn(4, 3, 64, device="cuda", requires_grad=True)
    x = leaf * 1.0
    other = x.exp()          # (saves its own result)
    square = x * x           # saves x
    loss = _four(x, tok, inplace=True)[name](x)
    torch.autograd.grad(loss, x, retain_graph=True)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        torch.autograd.grad(square.sum(), leaf)
    torch.autograd.grad(other.sum(), leaf)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ALL)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_factors_on_the_loss(name, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    tok = torch.randint(515, (4, 5), generator=g, device="cuda")
    x = torch.randn(4, 5, 515, generator=g, device="cuda").to(DT[dtype]).requires_grad_()
    f = _four(x, tok)[name]
    one, = torch.autograd.grad(f(x), x)
    four, = torch.autograd.grad(f(x) * 4.0, x)  # (a power of two: no rounding)
    assert torch.equal(one * 4, four)
    with torch.enable_grad():
        (f(x) * 0.5 + f(x) * 0.5).backward()
    assert torch.allclose(x.grad.float(), one.float(), rtol=2.0 ** -7, atol=0)


@pytest.mark.gpu
@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("B,T,V,dtype", [(8, 700, 1000, "bf16"), (6, 601, 4099, "f16"),
                                         (4, 600, 9000, "f32"), (2, 700, 40000, "bf16"),
                                         (2, 300, 70001, "f32"), (2, 250, 131072, "bf16"),
                                         (2, 9, 524288, "f32")])
def test_runs_of_rows_that_do_not_count(B, T, V, dtype, entropy):
    """Many rows a CTA, prompts and padding among them in runs."""
    check_all(B, T, V, dtype, entropy)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [1, 2, 3, 4, 5, 7, 8, 11, 16])
@pytest.mark.parametrize("B,T,V,dtype", [(4, 333, 1500, "bf16"), (2, 400, 9001, "f32")])
def test_every_cluster_size(C, B, T, V, dtype, monkeypatch):
    """One to sixteen CTAs a row, the last of them with little or nothing of it."""
    monkeypatch.setenv("GBCE_ROWS_CLUSTER", str(C))
    check_all(B, T, V, dtype, C % 2 == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("spread,T", [(300.0, 1.0), (3000.0, 1.0), (20000.0, 50.0), (4.0, 1e-3),
                                      (60000.0, 1000.0), (2.0, 100.0)])
def test_large_logits_and_extreme_temperatures(dtype, spread, T):
    import softmax_cross_entropy_gb300 as gbce
    rng = np.random.default_rng(int(spread))
    V = 5000
    x64 = np.clip(rng.normal(size=(1, 6, V)) * spread, -65000, 65000)
    x64[0, 1] -= x64[0, 1].max() + spread  # every logit far below zero
    x64 = np.clip(x64, -65000, 65000)
    x, held = put(x64, dtype)
    tok = held.argmax(1)
    tok[2] = 17
    x.requires_grad_()
    g = rng.normal(size=6)
    want = ref.log_probs(held, tok, T, IGN, g, np.zeros(6))
    lp, h = gbce.token_log_probs(x, cuda(tok).reshape(1, 6), temperature=T, return_entropy=True)
    close(lp, want[0].reshape(1, 6), logp_tol(want[0], V).reshape(1, 6), "lp")
    close(h, want[1].reshape(1, 6), 2 * logp_tol(want[1], V).reshape(1, 6), "h")
    dx, = torch.autograd.grad(lp, x, cuda(g).float().reshape(1, 6))
    p = probs(held, T)
    onto = np.zeros_like(p)
    onto[np.arange(6), tok] = 1.0
    close(dx.reshape(6, V), want[2], grad_tol(want[2], p + onto * 2.0 ** -6, np.abs(g) / T, dtype, V), "dx")
    # the losses whose forward forms the gradient: the same rows, coefficients 1
    loss = gbce.policy_loss(x, cuda(tok).reshape(1, 6), torch.ones(1, 6, device="cuda"),
                            temperature=T, reduction="sum", entropy_coef=1e-30)
    dx, = torch.autograd.grad(loss, x)
    wdx = ref.log_probs(held, tok, T, IGN, -np.ones(6), -1e-30 * np.ones(6))[2]
    close(dx.reshape(6, V), wdx, grad_tol(wdx, p + onto * 2.0 ** -6, np.ones(6) / T, dtype, V), "policy dx")


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["logp", "policy", "pref", "distill"])
@pytest.mark.parametrize("V", [3000, 70000])
def test_a_wait_that_runs_out_is_reported(name, V, monkeypatch):
    """CTA 0 leaves its first copy out: the waits for it give up, nothing else happens, and the next
    call is right."""
    import softmax_cross_entropy_gb300 as gbce
    from softmax_cross_entropy_gb300 import _lib
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    tok = torch.randint(V, (4, 50), generator=g, device="cuda")
    x = torch.randn(4, 50, V, generator=g, device="cuda").bfloat16().requires_grad_()
    f = _four(x, tok)[name]
    want = f(x)
    monkeypatch.setenv("GBCE_WAIT_TIMEOUT_MS", "20")
    monkeypatch.setenv("GBCE_TEST_STALL_COPY", "1")
    f(x)
    assert gbce.device_status() == _lib.CE_ERR_TIMEOUT
    monkeypatch.delenv("GBCE_TEST_STALL_COPY")
    got = f(x)
    assert gbce.device_status() == _lib.CE_OK and torch.equal(got, want)


def check_all(B, T, V, dtype, entropy):
    """Every loss on one batch against 64 bits."""
    import softmax_cross_entropy_gb300 as gbce
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    x = (torch.randn(B, T, V, generator=g, device="cuda") * 2).to(DT[dtype]).requires_grad_()
    tok = torch.randint(V, (B, T), generator=g, device="cuda")
    start = torch.randint(T // 3, (B, 1), generator=g, device="cuda")
    at = torch.arange(T, device="cuda")[None]
    tok[(at < start) | (at > start + T // 2)] = IGN
    tok[:, T // 2] = IGN
    keep = tok != IGN
    K = 20
    idx = torch.randint(V, (B, T, K), generator=g, device="cuda")
    idx[~keep] = -1
    val = torch.randn(B, T, K, generator=g, device="cuda")
    adv = torch.randn(B, T, generator=g, device="cuda")
    lsm = torch.log_softmax(x.detach().double(), -1)
    p = lsm.exp()
    onto = torch.zeros_like(p).scatter_(-1, tok.clamp(min=0)[..., None], 1.0)
    lp = torch.where(keep, lsm.gather(-1, tok.clamp(min=0)[..., None])[..., 0], 0.0)
    h = torch.where(keep, -(p * lsm).sum(-1), 0.0)
    n = int(keep.sum())
    near = dict(rtol=2.0 ** -19, atol=2.0 ** -18)

    def same(dx, c, hc=None):
        want = c[..., None] * (onto - p)
        size = c.abs()
        if hc is not None:
            want = want - hc[..., None] * p * (lsm + h[..., None])
            size = size + hc.abs() * 30
        eps = torch.finfo(DT[dtype]).eps / 2
        tiny = torch.finfo(DT[dtype]).smallest_normal * eps
        tol = want.abs() * eps + size[..., None] * (p + onto * 2.0 ** -5) * 2.0 ** -14 + tiny
        assert bool(((dx.double() - want).abs() <= tol).all())
        assert plus_zero(dx[~keep])

    got = gbce.token_log_probs(x, tok, return_entropy=entropy)
    glp, gh = got if entropy else (got, None)
    assert torch.allclose(glp.double(), lp, **near)
    assert gh is None or torch.allclose(gh.double(), h, **near)
    up = torch.randn(B, T, generator=g, device="cuda")
    ups = [up, up * 0.1] if entropy else [up]
    dx, = torch.autograd.grad([glp, gh] if entropy else [glp], x, ups)
    c = torch.where(keep, up.double(), 0.0)
    same(dx, c, c * 0.1 if entropy else None)
    coef = 0.02 if entropy else 0.0
    for scale in (64.0,):
        loss = gbce.policy_loss(x, tok, adv, entropy_coef=coef, scale=scale)
        want = torch.where(keep, -adv.double() - coef * h, 0.0).sum() * scale / n
        assert torch.allclose(loss.double(), want, rtol=2.0 ** -18, atol=scale * 2.0 ** -18)
        dx, = torch.autograd.grad(loss, x)
        f = keep * scale / n
        same(dx, -adv.double() * f, -coef * f.double() if entropy else None)
    with torch.no_grad():
        assert torch.equal(gbce.policy_loss(x, tok, adv, entropy_coef=coef, scale=64.0), loss)
    # distillation: the list's mass, and with the remaining mass as one outcome more
    lse = torch.logsumexp(val.double(), -1).float() + 0.5 if entropy else None
    lq = val.double() - (torch.logsumexp(val.double(), -1) if lse is None else lse.double())[..., None]
    q = lq.exp()
    j = idx.clamp(min=0)
    rows = (q * (lq - lsm.gather(-1, j))).sum(-1)
    want = p * q.sum(-1, keepdim=True)
    want = want.scatter_add(-1, j, -q)
    if lse is not None:
        rest = 1 - q.sum(-1)
        others = p.scatter(-1, j, 0.0)
        left = others.sum(-1)
        rows = rows + rest * (rest.log() - left.log())
        want = want + rest[..., None] * p - others * (rest / left)[..., None]
    loss = gbce.distillation_loss(x, val, idx, teacher_lse=lse, scale=64.0)
    total = torch.where(keep, rows, 0.0).sum() * 64 / n
    assert torch.allclose(loss.double(), total, rtol=2.0 ** -18)
    dx, = torch.autograd.grad(loss, x)
    want = torch.where(keep[..., None], want, 0.0) * 64 / n
    eps = torch.finfo(DT[dtype]).eps / 2
    tiny = torch.finfo(DT[dtype]).smallest_normal * eps
    named = torch.zeros_like(p).scatter_(-1, j, 1.0)
    tol = want.abs() * eps + 64 / n * (2 * p + named * 2.0 ** -5) * 2.0 ** -14 + tiny
    assert bool(((dx.double() - want).abs() <= tol).all())
    assert plus_zero(dx[~keep])
    with torch.no_grad():
        assert torch.equal(gbce.distillation_loss(x, val, idx, teacher_lse=lse, scale=64.0), loss)
    # pairs
    out = gbce.preference_loss(x, tok, beta=0.1, scale=64.0, return_scores=True)
    s = lp.sum(1)
    assert torch.allclose(out.scores.double(), s, rtol=2.0 ** -20, atol=n * 2.0 ** -20)
    d = s[:B // 2] - s[B // 2:]
    dx, = torch.autograd.grad(out.loss, x)
    sl = 0.1 * (torch.sigmoid(0.1 * d) - 1) * 64 / (B // 2)
    c = torch.where(keep, torch.cat([sl, -sl])[:, None].double(), 0.0)
    same(dx, c)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ALL)
def test_captured_and_replayed(name):
    """Captured with its backward on a side stream, two graphs at once, new inputs between replays."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    tok = torch.randint(4000, (4, 8), generator=g, device="cuda")
    xs = [torch.randn(4, 8, 4000, generator=g, device="cuda").bfloat16().requires_grad_() for _ in range(2)]
    new = [torch.randn(4, 8, 4000, generator=g, device="cuda").bfloat16() for _ in range(2)]
    fs = [_four(x, tok)[name] for x in xs]
    want = []
    for x, f, n in zip(xs, fs, new):
        leaf = n.clone().requires_grad_()
        loss = f(leaf)
        want.append((loss.detach().clone(), torch.autograd.grad(loss, leaf)[0]))
    del loss
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for x, f in zip(xs, fs):
            torch.autograd.grad(f(x), x)  # warm-up
    torch.cuda.synchronize()
    for x, f in zip(xs, fs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            loss = f(x)
            outs.append((loss, *torch.autograd.grad(loss, x)))
        graphs.append(graph)
    for x, n in zip(xs, new):
        x.detach().copy_(n)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (loss, dx), (wl, wdx) in zip(outs, want):
        assert torch.equal(loss, wl) and torch.equal(dx, wdx)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ALL)
def test_streams_at_once(name):
    """Calls on several streams at once give what they give one after another."""
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    tok = torch.randint(9000, (4, 20), generator=g, device="cuda")
    xs = [torch.randn(4, 20, 9000, generator=g, device="cuda", requires_grad=True) for _ in range(4)]
    f = _four(xs[0], tok)[name]
    want = []
    for x in xs:
        loss = f(x)
        want.append((loss.detach().clone(), torch.autograd.grad(loss, x)[0]))
    torch.cuda.synchronize()
    got = [None] * 4
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        for i, (s, x) in enumerate(zip(streams, xs)):
            with torch.cuda.stream(s):
                loss = f(x)
                got[i] = (loss.detach(), torch.autograd.grad(loss, x)[0])
    torch.cuda.synchronize()
    for (a, b), (c, d) in zip(got, want):
        assert torch.equal(a, c) and torch.equal(b, d)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ALL)
def test_offsets_past_32_bits(name):
    """Rows behind the 2^31st element of the logits."""
    V = 262144
    rows = 2 ** 31 // V + 8
    x = torch.zeros(4, rows // 4, V, dtype=torch.bfloat16, device="cuda")
    tok = torch.full((4, rows // 4), IGN, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(12)
    last = torch.randn(2, V, generator=gen, device="cuda").bfloat16()
    x[3, -2:] = last
    tok[3, -2:] = torch.tensor([5, V - 1], device="cuda")
    x.requires_grad_()
    f = _four(x, tok)[name]
    if name == "distill":
        import softmax_cross_entropy_gb300 as gbce
        idx = torch.full((*tok.shape, 3), -1, device="cuda")
        idx[3, -2:] = torch.tensor([7, 9, V - 3], device="cuda")
        val = torch.zeros(*tok.shape, 3, device="cuda")
        f = lambda x: gbce.distillation_loss(x, val, idx)
        small = lambda x: gbce.distillation_loss(x, val[3:, -2:], idx[3:, -2:])
    loss = f(x)
    dx, = torch.autograd.grad(loss, x)
    assert plus_zero(dx[:3]) and plus_zero(dx[3, :-2])
    leaf = last[None].clone().requires_grad_()
    if name == "logp":
        import softmax_cross_entropy_gb300 as gbce
        want = gbce.token_log_probs(leaf, tok[3:, -2:]).sum()
    elif name == "distill":
        want = small(leaf)
    else:  # the token's own row: a multiple of onehot - p
        p = torch.softmax(last.double(), 1)
        p[0, 5] -= 1
        p[1, V - 1] -= 1
        d = dx[3, -2:].double()
        for a, b in zip(d, p):
            k = float((a @ b) / (b @ b))
            assert abs(k) > 0 and float((a - k * b).norm() / a.norm()) < 2.0 ** -8
        return
    wdx, = torch.autograd.grad(want, leaf)
    # two rows are shared by more CTAs than many are, whose sums add up in another order (2^-20 of
    # each); the gradients of the two are then at most a step apart
    assert torch.allclose(loss, want, rtol=2.0 ** -20)
    assert torch.allclose(dx[3:, -2:].float(), wdx.float(), rtol=2.0 ** -7, atol=2.0 ** -126)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ALL)
def test_saved_tensors_with_other_strides(name):
    """Hooks on saved tensors (here: kept on the host meanwhile) give back contiguous copies of the
    logits, or of the gradient, whose rows were apart."""
    g = torch.Generator(device="cuda")
    g.manual_seed(10)
    tok = torch.randint(999, (4, 6), generator=g, device="cuda")
    full = torch.randn(4, 8, 1003, generator=g, device="cuda").bfloat16()
    x = full[:, 1:-1, :999].detach().requires_grad_()
    f = _four(x, tok)[name]
    want, = torch.autograd.grad(f(x) * 2.0, x)
    with torch.autograd.graph.save_on_cpu():
        loss = f(x) * 2.0
    got, = torch.autograd.grad(loss, x)
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_sequences_without_rows():
    import softmax_cross_entropy_gb300 as gbce
    x = torch.zeros(4, 0, 50, device="cuda", requires_grad=True)
    out = gbce.preference_loss(x, torch.zeros(4, 0, dtype=torch.int64, device="cuda"),
                               return_scores=True)
    g, = torch.autograd.grad(out.loss, x)
    assert np.isclose(float(out.loss), np.log(2), rtol=1e-6) and (out.scores == 0).all()
    assert g.shape == x.shape


@pytest.mark.gpu
@pytest.mark.parametrize("V", [777, 5431, 41003, 90001])
def test_first_call_of_a_size_may_be_captured(V):
    """Sizes that no call has had, captured at once (whatever a layout needs is asked for then)."""
    import softmax_cross_entropy_gb300 as gbce
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    x = torch.randn(2, 5, V, generator=g, device="cuda").half()
    tok = torch.randint(V, (2, 5), generator=g, device="cuda")
    adv = torch.randn(2, 5, generator=g, device="cuda")
    idx = torch.randint(V, (2, 5, 6), generator=g, device="cuda")
    val = torch.randn(2, 5, 6, generator=g, device="cuda")
    calls = [lambda: gbce.token_log_probs(x, tok), lambda: gbce.policy_loss(x, tok, adv),
             lambda: gbce.preference_loss(x, tok), lambda: gbce.distillation_loss(x, val, idx)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs, graph = [], torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = [f() for f in calls]
    graph.replay()
    torch.cuda.synchronize()
    for f, got in zip(calls, outs):
        assert torch.equal(f(), got)


@pytest.mark.gpu
def test_shares_of_a_training_step():
    """A run of them together: scores of the old and the reference policy, the policy loss on the
    new logits (on-policy its ratio is 1), a preference loss and a distillation added up."""
    import softmax_cross_entropy_gb300 as gbce
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    hidden = torch.randn(4, 12, 64, generator=g, device="cuda")
    head = (torch.randn(2000, 64, generator=g, device="cuda") * 0.2).requires_grad_()
    tok = torch.randint(2000, (4, 12), generator=g, device="cuda")
    tok[:, :3] = IGN
    logits = hidden @ head.T
    with torch.no_grad():
        old = gbce.token_log_probs(logits, tok)
        base = gbce.token_log_probs(hidden @ (head * 0.9).T, tok)
        top = torch.topk(hidden @ (head * 1.1).T, 32)
    adv = torch.randn(4, generator=g, device="cuda")
    out = gbce.policy_loss(logits, tok, adv, old, ref_log_probs=base, kl_coef=0.05, return_stats=True)
    assert torch.equal(out.log_probs, old) and not out.clipped.any()
    pref = gbce.preference_loss(logits, tok, ref_log_probs=base.sum(1), return_scores=True)
    kd = gbce.distillation_loss(logits, top.values, top.indices)
    (out.loss + pref.loss + kd).backward()
    got = head.grad.clone()
    # the same in 64 bits from their definitions
    h64 = head.detach().double().requires_grad_()
    z = hidden.double() @ h64.T
    lsm = torch.log_softmax(z, -1)
    keep = tok != IGN
    lp = lsm.gather(-1, tok.clamp(min=0)[..., None])[..., 0]
    a = adv.double()[:, None]
    gap = base.double() - lp
    rows = -(lp - old.double()).exp() * a + 0.05 * (gap.exp() - gap - 1)
    s = torch.where(keep, lp, 0.0).sum(1)
    delta = (s[:2] - s[2:]) - (base.double().sum(1)[:2] - base.double().sum(1)[2:])
    q = torch.softmax(top.values.double(), -1)
    d = (q * (q.log() - lsm.gather(-1, top.indices))).sum(-1).mean()
    total = rows[keep].mean() - torch.nn.functional.logsigmoid(0.1 * delta).mean() + d
    total.backward()
    err = float((got.double() - h64.grad).norm() / h64.grad.norm())
    # (the fp32 products of 64 terms and the logits' roundings: some 2^-20 each)
    assert err < 2.0 ** -16
