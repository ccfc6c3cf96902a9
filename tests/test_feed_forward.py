"""The gated feed-forward block: refusals (CPU), and the kernels against the
formulas in 64 bits (GPU)."""
import contextlib
import ctypes
import math

import numpy as np
import pytest
import torch

from philox_ref import keep

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def act64(g, name):
    """(act, slope) in 64 bits."""
    if name == "silu":
        q = torch.sigmoid(g)
        return g * q, q + g * q * (1 - q)
    if name == "gelu":
        c = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 0.134145 * g * g)


def mask64(rows, O, p, seed, offset=0):
    if p == 0.0:
        return torch.ones(rows, O, dtype=torch.float64, device="cuda")
    kept = torch.from_numpy(keep(rows * O, p, seed, offset)).cuda().reshape(rows, O)
    return kept.double() * (0.0 if p == 1.0 else 1.0 / (1.0 - p))


def reference(x, wg, wu, wd, act, f, res=None, dy=None):
    """Outputs and gradients in 64 bits, and for each the sum of the absolute
    values that its last product adds (what a relative error of its factors is
    scaled by)."""
    x, wg, wu, wd = (t.detach().double() for t in (x, wg, wu, wd))
    g, u = x @ wg.T, x @ wu.T
    a, s = act64(g, act)
    h = a * u
    y = (h @ wd.T) * f
    size = {"y": (h.abs() @ wd.abs().T) * f}
    if res is not None:
        y = y + res.detach().double()
    out = {"y": y}
    if dy is None:
        return out, size
    dz = dy.double() * f
    dh = dz @ wd
    dg, du = dh * u * s, dh * a
    out.update(dx=dg @ wg + du @ wu, dw_gate=dg.T @ x, dw_up=du.T @ x, dw_down=dz.T @ h)
    # an error of fp32's size in g and u (terms 2^-24 of the projections' sizes) reaches act'(g)
    # and act(g) too: counted with the sizes of dz Wd, u and g
    adh = dz.abs() @ wd.abs()
    bg = adh * (u.abs() * 1.13 * (1 + 1.5 * g.abs()))
    bu = adh * (a.abs() + 1.13 * g.abs())
    size.update(dx=bg @ wg.abs() + bu @ wu.abs(), dw_gate=bg.T @ x.abs(), dw_up=bu.T @ x.abs(),
                dw_down=dz.abs().T @ h.abs())
    return out, size


# The kernel rounds h once before y's product, and dg or du before the gradients': half a step
# (eps / 2) of a factor, and products that accumulate in fp32: n terms are added with at most n 2^-24 of their sizes. The result's own
# rounding is half a step of the value.
def check(got, want, size, dt, roundings, terms):
    eps = torch.finfo(dt).eps
    bound = size * (roundings * eps / 2 * 1.02 + terms * 2.0 ** -24) + \
        want.abs() * eps / 2 * 1.02 + torch.finfo(dt).smallest_normal
    err = (got.detach().double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    # what the bound leaves room for, a systematic error, would show in the norm: the roundings are
    # independent, so the error is of the order of one of them (2^-8 of the norm, or eps)
    norm = want.norm()
    if norm > 0 and want.numel() >= 64:
        assert float(err.norm() / norm) <= 3 * eps


def make(rows, H, I, O, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + rows + 3 * H + 5 * I + 7 * O)
    n = lambda *s, k=1.0: (torch.randn(*s, generator=g, device="cuda") * k).to(DT[dtype])  # noqa: E731
    return (n(rows, H), n(I, H, k=H ** -0.5), n(I, H, k=H ** -0.5), n(O, I, k=I ** -0.5),
            n(rows, O), n(rows, O))


# ---------------------------------------------------------------- CPU

def fwd(**over):
    from softmax_cross_entropy_gb300 import _lib
    a = dict(x=256, w_gate=256, w_up=256, w_down=256, residual=None, dtype=_lib.CE_BF16, rows=4,
             H=64, I=64, O=64, act=0, p=0.0, seed=0, offset=0, state=None, y=256, h=256, s=None,
             a=None, workspace=None, workspace_bytes=0, stream=None)
    a.update(over)
    return _lib.ce_ffn_fwd(**a)


def bwd(**over):
    from softmax_cross_entropy_gb300 import _lib
    a = dict(dy=256, x=256, w_gate=256, w_up=256, w_down=256, h=256, s=256, a=256,
             dtype=_lib.CE_F16, rows=4, H=64, I=64, O=64, act=1, p=0.1, seed=0, offset=0,
             state=None, dx=256, dw_gate=256, dw_up=256, dw_down=256, workspace=256,
             workspace_bytes=1 << 20, stream=None)
    a.update(over)
    return _lib.ce_ffn_bwd(**a)


BAD = [dict(dtype=3), dict(rows=-1), dict(H=0), dict(I=-8), dict(O=0), dict(act=3), dict(act=-1),
       dict(p=-0.5), dict(p=2.0), dict(p=float("nan")), dict(x=None), dict(w_gate=None),
       dict(w_up=None), dict(w_down=None)]


@pytest.mark.parametrize("over", BAD + [dict(y=None), dict(h=None), dict(s=256), dict(h=264), dict(H=60, workspace=None)])
def test_forward_refuses(over):
    from softmax_cross_entropy_gb300 import _lib
    ws = dict(workspace=4096, workspace_bytes=1 << 30) if "workspace" not in over else {}
    assert fwd(**{**ws, **over}) == _lib.CE_ERR_INVALID_ARG


@pytest.mark.parametrize("over", BAD + [dict(dy=None), dict(h=None), dict(s=None), dict(a=None), dict(x=257),
                                        dict(dw_up=None), dict(workspace=None),
                                        dict(workspace=264), dict(workspace_bytes=100)])
def test_backward_refuses(over):
    from softmax_cross_entropy_gb300 import _lib
    assert bwd(**over) == _lib.CE_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [dict(dtype=0), dict(x=264), dict(w_down=258), dict(w_gate=272 + 2),
                                  dict(rows=2 ** 31)])
def test_sizes_and_types_it_does_not_take(over):
    from softmax_cross_entropy_gb300 import _lib
    assert fwd(**over) == _lib.CE_ERR_UNSUPPORTED
    assert bwd(**over) == _lib.CE_ERR_UNSUPPORTED


def test_wrapper_refuses_cpu_tensors():
    import softmax_cross_entropy_gb300 as gbce
    t = torch.zeros(8, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        gbce.gated_feed_forward(t, t, t, t)


UP, DOWN, DH, DX, DW = range(5)  # the block's products


def tiles_of(product, rows, H, I, O, sms=152):
    """((rows, columns, SMs) of a tile, the tiles that the busiest SM or pair works on)."""
    from softmax_cross_entropy_gb300 import _lib
    t = (ctypes.c_int64 * 4)()
    assert _lib.ce_ffn_tiles(product, rows, H, I, O, sms, t) == _lib.CE_OK
    return tuple(t[:3]), -(-t[3] // (sms // t[2]))


# Sizes at which each product takes each of its tile shapes, several tiles an SM (or pair) where
# the shape is ever taken so: {product: (tile, tiles of the busiest at least)}. Edges are ragged,
# those with odd sizes store rows that are not whole vectors.
ONE = {128: (128, 256, 1), 256: (256, 256, 1)}
PAIR = {w: (256, w, 2) for w in (192, 224, 256)}
SHAPES = [
    (300, 72, 38993, 72, {UP: ((128, 128, 1), 6), DH: (ONE[128], 4), DW: (ONE[128], 6)}),
    (300, 38984, 72, 38984, {DOWN: (ONE[128], 4), DX: (ONE[128], 4), DW: (ONE[128], 5)}),
    (297, 38993, 71, 38993, {DOWN: (ONE[128], 4), DX: (ONE[128], 4)}),
    (500, 72, 39000, 72, {UP: ((256, 128, 2), 8), DH: (PAIR[256], 4)}),
    (497, 72, 7000, 72, {UP: ((256, 96, 2), 2)}),
    (500, 72, 136, 38000, {DOWN: (PAIR[256], 4)}),
    (500, 72, 136, 39000, {DOWN: (PAIR[224], 5)}),
    (499, 72, 136, 13999, {DOWN: (PAIR[192], 2)}),
    (500, 23000, 504, 72, {DX: (PAIR[256], 3), DW: (PAIR[256], 5)}),
    (499, 19152, 504, 19152, {DX: (ONE[256], 1), DW: (ONE[256], 3)}),
    (500, 57496, 72, 72, {DX: (ONE[256], 3)}),
    (499, 57491, 72, 72, {DX: (ONE[256], 3)})]


@pytest.mark.parametrize("rows,H,I,O,forms", SHAPES)
def test_sizes_take_the_tiles_they_are_meant_for(rows, H, I, O, forms):
    for product, (tile, least) in forms.items():
        got, most = tiles_of(product, rows, H, I, O)
        assert got == tile and most >= least, (product, got, most)


@pytest.mark.parametrize("sms", [2, 3, 151, 152])
def test_long_epilogues_never_take_the_shape_that_does_not_overlap_them(sms):
    for product in (UP, DOWN, DH):
        for n in range(1, 400):
            rows, _, shared = tiles_of(product, 512, 256, 128 * n, 128 * n, sms)[0]
            assert rows == 128 or shared == 2


def test_tiles_refuses():
    from softmax_cross_entropy_gb300 import _lib
    t = (ctypes.c_int64 * 4)()
    for bad in ((-1, 4, 8, 8, 8, 152, t), (5, 4, 8, 8, 8, 152, t), (0, -1, 8, 8, 8, 152, t),
                (0, 4, 0, 8, 8, 152, t), (0, 4, 8, 8, 8, 0, t), (0, 4, 8, 8, 8, 152, None)):
        assert _lib.ce_ffn_tiles(*bad) == _lib.CE_ERR_INVALID_ARG


@pytest.fixture
def stubbed(monkeypatch):
    """The wrapper on CPU tensors, its library call a plain copy."""
    from softmax_cross_entropy_gb300 import feed_forward

    def forward(x, w_gate, w_up, w_down, residual, act, p, seed, offset, state, grad):
        return x.detach().clone(), x.detach(), torch.zeros(2, *x.shape) if grad else None

    monkeypatch.setattr(feed_forward, "_refuse", lambda *a: None)
    monkeypatch.setattr(feed_forward, "_forward", forward)
    return feed_forward


def test_tangents_are_refused_not_dropped(stubbed):
    from torch.autograd import forward_ad
    t = torch.randn(8, 8).bfloat16()
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(t, torch.ones_like(t))
        for i in range(5):
            args = [t] * 5
            args[i] = dual
            with pytest.raises(NotImplementedError):
                stubbed.gated_feed_forward(*args[:4], residual=args[4])
            with pytest.raises(NotImplementedError), torch.no_grad():
                stubbed.gated_feed_forward(*args[:4], residual=args[4])
        assert torch.equal(stubbed.gated_feed_forward(t, t, t, t), t)


def test_a_gradient_with_a_tangent_is_refused(stubbed):
    from torch.autograd import forward_ad
    t = torch.randn(8, 8).bfloat16()
    with forward_ad.dual_level():
        x = t.clone().requires_grad_()
        y = stubbed.gated_feed_forward(x, t, t, t)
        with pytest.raises(RuntimeError, match="once"):
            torch.autograd.grad(y, [x], forward_ad.make_dual(t, torch.ones_like(t)))


@pytest.mark.parametrize("p", [0.0, 0.5, 1.0])
def test_a_seed_tensor_may_change_before_the_backward(stubbed, monkeypatch, p):
    calls = []
    monkeypatch.setattr(stubbed._lib, "ce_ffn_bwd_workspace_bytes", lambda *a: 1)
    monkeypatch.setattr(stubbed._lib, "ce_ffn_bwd", lambda *a: calls.append(a) or 0)
    monkeypatch.setattr(stubbed, "stream", lambda device: 0)
    monkeypatch.setattr(stubbed, "on", lambda device: contextlib.nullcontext())
    t = torch.randn(8, 8).bfloat16()
    x = t.clone().requires_grad_()
    seed = torch.tensor([3, 4])
    y = stubbed.gated_feed_forward(x, t, t, t, dropout_p=p, seed=seed)
    seed += 1
    torch.autograd.grad(y.sum(), [x])
    assert len(calls) == 1


# ---------------------------------------------------------------- GPU

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("rows,H,I,O", [
    (1, 8, 8, 8), (2, 64, 128, 64), (3, 200, 72, 40), (16, 256, 512, 256), (17, 1000, 24, 136),
    (1, 2048, 4096, 2048), (40, 1024, 2048, 1000), (63, 4096, 640, 264),
    (33, 72, 1000, 264), (64, 512, 640, 512), (129, 136, 264, 8), (300, 384, 320, 640),
    (515, 256, 1032, 256), (1000, 64, 72, 4096)])
def test_forward(dtype, act, rows, H, I, O):
    import softmax_cross_entropy_gb300 as gbce
    x, wg, wu, wd, _, _ = make(rows, H, I, O, dtype)
    y = gbce.gated_feed_forward(x, wg, wu, wd, activation=act)
    want, size = reference(x, wg, wu, wd, act, mask64(rows, O, 0.0, 0))
    check(y, want["y"], size["y"], DT[dtype], 1, H + I)
    assert gbce.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("rows,H,I,O,p,residual", [
    (1, 8, 8, 8, 0.0, False), (5, 64, 128, 72, 0.3, True), (70, 264, 136, 264, 0.0, True),
    (130, 128, 256, 128, 0.1, False), (257, 520, 392, 520, 0.1, True), (512, 512, 1024, 512, 0.5, True),
    (64, 64, 64, 64, 1.0, True)])
def test_training_step(dtype, act, rows, H, I, O, p, residual):
    import softmax_cross_entropy_gb300 as gbce
    dt = DT[dtype]
    x, wg, wu, wd, res, dy = make(rows, H, I, O, dtype)
    leaves = [t.requires_grad_() for t in (x, wg, wu, wd)] + ([res.requires_grad_()] if residual else [])
    y = gbce.gated_feed_forward(x, wg, wu, wd, activation=act, dropout_p=p, seed=99, offset=7,
                                residual=res if residual else None)
    grads = torch.autograd.grad(y, leaves, dy)
    want, size = reference(x, wg, wu, wd, act, mask64(rows, O, p, 99, 7), res if residual else None, dy)
    check(y, want["y"], size["y"], dt, 1, H + I)
    for name, got, n in zip(("dx", "dw_gate", "dw_up", "dw_down"), grads, (O + 2 * I, O + rows, O + rows, rows)):
        check(got, want[name], size[name], dt, 1, n + H)
    if residual:
        assert torch.equal(grads[4], dy)
    assert gbce.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gradients_against_differences(act):
    # (f(t + d) - f(t - d)) / 2 of the 64-bit formulas along the kernel's own gradient direction
    import softmax_cross_entropy_gb300 as gbce
    args = [t.requires_grad_() for t in make(40, 64, 96, 64, "f16")[:4]]
    dy = make(40, 64, 96, 64, "f16", 1)[5]
    grads = torch.autograd.grad(gbce.gated_feed_forward(*args, activation=act), args, dy)

    def loss(step):
        x, wg, wu, wd = (t.detach().double() + step * d.double() for t, d in zip(args, grads))
        return float((((act64(x @ wg.T, act)[0] * (x @ wu.T)) @ wd.T) * dy.double()).sum())

    total = sum(float(d.double().square().sum()) for d in grads)
    step = 1e-4 / math.sqrt(total)
    diff = (loss(step) - loss(-step)) / (2 * step)
    # the direction is the gradient itself: the derivative along it is its squared norm, up to the
    # gradients' own relative error (a few eps) and the difference's second order
    assert abs(diff / total - 1.0) <= 4 * torch.finfo(torch.float16).eps


@pytest.mark.gpu
@pytest.mark.parametrize("rows,H,I,O", [(1, 7, 9, 5), (37, 33, 65, 33), (130, 1001, 131, 77),
                                        (300, 65, 131, 77), (513, 128, 203, 300),
                                        (600, 200, 96, 130), (1000, 64, 70, 4093)])
@pytest.mark.parametrize("p,residual", [(0.0, False), (0.25, True)])
def test_odd_sizes(rows, H, I, O, p, residual):
    import softmax_cross_entropy_gb300 as gbce
    x, wg, wu, wd, res, dy = make(rows, H, I, O, "bf16")
    leaves = [t.requires_grad_() for t in (x, wg, wu, wd)] + ([res.requires_grad_()] if residual else [])
    y = gbce.gated_feed_forward(x, wg, wu, wd, dropout_p=p, seed=5, residual=res if residual else None)
    want, size = reference(x, wg, wu, wd, "silu", mask64(rows, O, p, 5), res if residual else None, dy)
    check(y, want["y"], size["y"], torch.bfloat16, 1, H + I)
    for name, got in zip(("dx", "dw_gate", "dw_up", "dw_down"), torch.autograd.grad(y, leaves, dy)):
        assert got.shape == want[name].shape
        check(got, want[name], size[name], torch.bfloat16, 1, H + 2 * I + O + rows)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,H,I,O,forms", SHAPES)
def test_every_tile_shape_and_several_tiles_an_sm(dtype, rows, H, I, O, forms):
    import softmax_cross_entropy_gb300 as gbce
    dt = DT[dtype]
    x, wg, wu, wd, res, dy = make(rows, H, I, O, dtype)
    leaves = [t.requires_grad_() for t in (x, wg, wu, wd)]
    p = 0.25 if rows * O < 1 << 23 else 0.0  # (the reference's words are formed on the CPU)
    y = gbce.gated_feed_forward(x, wg, wu, wd, dropout_p=p, seed=21, residual=res)
    grads = torch.autograd.grad(y, leaves, dy)
    want, size = reference(x, wg, wu, wd, "silu", mask64(rows, O, p, 21), res, dy)
    check(y, want["y"], size["y"], dt, 1, H + I)
    for name, got, n in zip(("dx", "dw_gate", "dw_up", "dw_down"), grads, (O + 2 * I, O + rows, O + rows, rows)):
        check(got, want[name], size[name], dt, 1, n + H)
    # the bounds above grow with the terms of a product: a tile or a run of rows that is wrong
    # shows in its own norm, which holds one rounding of its factors and one of the result
    eps = torch.finfo(dt).eps
    for name, got in zip(("y", "dx", "dw_gate", "dw_up", "dw_down"), (y, *grads)):
        err = (got.detach().double() - want[name]).square()
        ref = want[name].square()
        for dim in (0, 1):
            for e, r in zip(err.split(32, dim), ref.split(32, dim)):
                if r.numel() >= 4096:
                    assert float(e.sum()) <= (3 * eps) ** 2 * float(r.sum()), (name, dim)
    assert gbce.device_status() == 0


@pytest.mark.gpu
def test_leading_dimensions_strides_and_no_rows():
    import softmax_cross_entropy_gb300 as gbce
    x, wg, wu, wd, res, _ = make(24, 64, 128, 64, "bf16")
    y = gbce.gated_feed_forward(x, wg, wu, wd, residual=res)
    y3 = gbce.gated_feed_forward(x.view(2, 3, 4, 64), wg, wu, wd, residual=res.view(2, 3, 4, 64))
    assert torch.equal(y3.view(24, 64), y)
    yt = gbce.gated_feed_forward(x.t().contiguous().t(), wg.t().contiguous().t(), wu, wd, residual=res)
    assert torch.equal(yt, y)
    odd = torch.empty(24 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(24, 64).copy_(x)
    assert torch.equal(gbce.gated_feed_forward(odd, wg, wu, wd, residual=res), y)
    one = gbce.gated_feed_forward(x[3], wg, wu, wd)
    assert one.shape == (64,)
    e = x[:0].requires_grad_()
    w = wg.detach().requires_grad_()
    ye = gbce.gated_feed_forward(e, w, wu, wd)
    assert ye.shape == (0, 64)
    ge, gw = torch.autograd.grad(ye.sum(), [e, w])
    assert ge.shape == (0, 64) and torch.equal(gw, torch.zeros_like(w))


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [40, 400])
def test_unaligned_residual_and_gradient(rows):
    import softmax_cross_entropy_gb300 as gbce
    x, wg, wu, wd, res, dy = make(rows, 64, 128, 64, "f16")

    def shifted(t):  # the same values on a base that is not 16-byte aligned
        return torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)

    outs = []
    for r, d in ((res, dy), (shifted(res), shifted(dy))):
        a = [t.detach().requires_grad_() for t in (x, wg, wu, wd)]
        y = gbce.gated_feed_forward(*a, residual=r, dropout_p=0.3, seed=2)
        outs.append([y.detach(), *torch.autograd.grad(y, a, d)])
    for p, q in zip(*outs):
        assert torch.equal(p, q)


@pytest.mark.gpu
def test_two_graphs_replayed_at_once():
    # each graph has its own workspace: replays on two streams do not meet
    import softmax_cross_entropy_gb300 as gbce
    sets = [make(40, 256, 512, 256, "bf16", i) for i in range(2)]
    want = [gbce.gated_feed_forward(*s[:4], residual=s[4]) for s in sets]
    graphs, outs = [], []
    for s in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(gbce.gated_feed_forward(*s[:4], residual=s[4]))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.gpu
@pytest.mark.parametrize("which", [(0,), (1,), (2, 3), (3,), (0, 3), (4,)])
def test_some_gradients_only(which):
    import softmax_cross_entropy_gb300 as gbce
    args = list(make(72, 64, 136, 64, "bf16")[:5])
    dy = make(72, 64, 136, 64, "bf16", 2)[5]

    def grads(idx):
        a = [t.detach().clone().requires_grad_(i in idx) for i, t in enumerate(args)]
        y = gbce.gated_feed_forward(*a[:4], residual=a[4], dropout_p=0.2, seed=1)
        return torch.autograd.grad(y, [a[i] for i in idx], dy)

    every = grads((0, 1, 2, 3, 4))
    for i, g in zip(which, grads(which)):
        assert torch.equal(g, every[i])


@pytest.mark.gpu
def test_rows_do_not_touch_each_other_and_results_repeat():
    import softmax_cross_entropy_gb300 as gbce
    x, wg, wu, wd, res, _ = make(200, 128, 256, 128, "bf16")
    y = gbce.gated_feed_forward(x, wg, wu, wd, residual=res)
    assert torch.equal(gbce.gated_feed_forward(x, wg, wu, wd, residual=res), y)
    x2 = x.clone()
    x2[100] = float("nan")
    y2 = gbce.gated_feed_forward(x2, wg, wu, wd, residual=res)
    rest = torch.arange(200, device="cuda") != 100
    assert torch.equal(y2[rest], y[rest]) and bool(y2[100].isnan().all())


@pytest.mark.gpu
def test_large_gates_saturate():
    import softmax_cross_entropy_gb300 as gbce
    # g = +-3008: act(g) is g or 0, its slope 1 or 0
    x = torch.full((8, 64), 1.0, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    sign = torch.tensor([1.0, -1.0], device="cuda").repeat(32)[:, None]
    wg = (sign * 47.0).expand(64, 64).bfloat16().contiguous()
    wu = torch.full((64, 64), 1 / 64, device="cuda", dtype=torch.bfloat16)
    wd = torch.full((64, 64), 1 / 64, device="cuda", dtype=torch.bfloat16)
    for act in ("silu", "gelu", "gelu_tanh"):
        y = gbce.gated_feed_forward(x, wg, wu, wd, activation=act)
        # 32 gates of 3008, the others 0
        assert torch.equal(y.detach().float(), torch.full_like(y, 1504.0).float())
        (dx,) = torch.autograd.grad(y.sum(), [x])
        # dh = 1: dg = 1 (u = act' = 1) or 0, du = 3008 or 0: 32 (47 + 3008 / 64)
        assert torch.equal(dx.float(), torch.full_like(dx, 3008.0).float())
    # gates of 1e20, whose squares overflow
    y = gbce.gated_feed_forward(x * 1e20 / 47.0 / 64.0, wg, wu, wd, activation="gelu_tanh")
    (dx,) = torch.autograd.grad(y.sum(), [x])
    assert bool(y.isfinite().all()) and bool(dx.isfinite().all())


@pytest.mark.gpu
def test_seed_tensor_changed_before_the_backward_and_captured_step():
    import softmax_cross_entropy_gb300 as gbce
    x, wg, wu, wd, res, dy = make(40, 64, 128, 64, "bf16")
    leaves = [t.requires_grad_() for t in (x, wg, wu, wd)]
    state = torch.tensor([3, 4], dtype=torch.int64, device="cuda")

    def step(seed, offset=0):
        y = gbce.gated_feed_forward(x, wg, wu, wd, dropout_p=0.5, seed=seed, offset=offset, residual=res)
        if isinstance(seed, torch.Tensor):
            seed += 1
        return [y.detach(), *torch.autograd.grad(y, leaves, dy)]

    want = [step(s, s + 1) for s in range(3, 7)]
    for a, b in zip(step(state), want[0]):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            outs = step(state)
    torch.cuda.synchronize()
    for w in want[1:]:
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, w):
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [40, 300])
@pytest.mark.parametrize("p", [0.0, 1.0])
def test_seed_tensor_where_no_words_are_drawn(rows, p):
    import softmax_cross_entropy_gb300 as gbce
    x, wg, wu, wd, res, dy = make(rows, 64, 128, 64, "bf16")
    leaves = [t.requires_grad_() for t in (x, wg, wu, wd)]
    state = torch.tensor([3, 4], dtype=torch.int64, device="cuda")
    outs = []
    for seed in (3, state):
        y = gbce.gated_feed_forward(x, wg, wu, wd, dropout_p=p, seed=seed, residual=res)
        state += 1
        outs.append([y.detach(), *torch.autograd.grad(y, leaves, dy)])
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_calls_on_two_streams_at_once():
    import softmax_cross_entropy_gb300 as gbce
    sets = [make(96, 256, 512, 256, "f16", i) for i in range(3)]
    want = [gbce.gated_feed_forward(*s[:4], residual=s[4]) for s in sets]
    few = [gbce.gated_feed_forward(s[0][:4], *s[1:4]) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append((gbce.gated_feed_forward(*s[:4], residual=s[4]),
                            gbce.gated_feed_forward(s[0][:4], *s[1:4])))
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(got):
        assert torch.equal(a, want[i % 3]) and torch.equal(b, few[i % 3])


@pytest.mark.gpu
def test_block_then_loss_then_beams():
    """Together as they would be used: a training step of block + fused linear cross-entropy, whose
    gradients reach the block's weights, then beams over the same model's logits."""
    import softmax_cross_entropy_gb300 as gbce
    torch.manual_seed(0)
    H, V, rows = 64, 512, 48
    block = gbce.GatedFeedForward(H, 128, dropout_p=0.1, device="cuda")
    emb = (torch.randn(V, H, device="cuda") * 0.5).bfloat16().requires_grad_()
    tokens = torch.randint(0, V, (rows,), device="cuda")
    target = torch.randint(0, V, (rows,), device="cuda")
    x = emb[tokens]
    hidden = block(x, residual=x, seed=11)
    loss = gbce.fused_linear_cross_entropy(hidden, emb, target)
    loss.backward()
    # the same in 64 bits
    p64 = [t.detach().double().requires_grad_() for t in (emb, block.gate, block.up, block.down)]
    e, wg, wu, wd = p64
    x64 = e[tokens]
    g = x64 @ wg.T
    y = ((g * torch.sigmoid(g) * (x64 @ wu.T)) @ wd.T) * mask64(rows, H, 0.1, 11) + x64
    ref = torch.nn.functional.cross_entropy(y @ e.T, target)
    ref.backward()
    assert abs(float(loss) - float(ref)) <= 2e-3 * float(ref)
    for got, want in zip((emb, block.gate, block.up, block.down), p64):
        assert float((got.grad.double() - want.grad).norm() / want.grad.norm()) <= 0.02
    # generating: 2 sequences x 4 beams, the token form of the block, a step of beam search
    block.eval()
    B, K = 2, 4
    last = torch.randint(0, V, (B, K), device="cuda")
    scores = torch.zeros(B, K, device="cuda")
    history = torch.zeros(B * K, 4, dtype=torch.int64, device="cuda")
    for step in range(4):
        x = emb.detach()[last]
        logits = block(x, residual=x) @ emb.detach().T
        best = gbce.beam_search_step(logits, scores, finished=None)
        total = (scores[..., None].double() + torch.log_softmax(logits.double(), 2)).reshape(B, -1)
        assert torch.allclose(best.scores.double(), total.topk(K, 1).values, atol=1e-4)
        gbce.beam_reorder(history, best.beams, inplace=True)
        last, scores = best.tokens, best.scores
        history[:, step] = last.reshape(-1)
    assert bool((scores[:, :-1] >= scores[:, 1:]).all())


@pytest.mark.gpu
def test_wrapper_refuses():
    import softmax_cross_entropy_gb300 as gbce
    x, wg, wu, wd, res, _ = make(8, 64, 128, 64, "bf16")
    f = gbce.gated_feed_forward
    with pytest.raises(TypeError):
        f(x.float(), wg.float(), wu.float(), wd.float())
    with pytest.raises(TypeError):
        f(x, wg.half(), wu, wd)
    with pytest.raises(ValueError):
        f(x, wg, wu[:64], wd)
    with pytest.raises(ValueError):
        f(x, wg, wu, wd.t())
    with pytest.raises(ValueError):
        f(x, wg, wu, wd, residual=res[:4])
    with pytest.raises(ValueError):
        f(x, wg, wu, wd, activation="tanh")
    with pytest.raises(ValueError):
        f(x, wg, wu, wd, dropout_p=0.5)
