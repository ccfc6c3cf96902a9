"""Dropout from counter-based words: the reference's own pins, the refusals
(CPU), and the kernel against the definition in 64 bits (GPU)."""
import numpy as np
import pytest
import torch

from philox_ref import keep, philox

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- CPU

def test_reference_reproduces_the_published_known_answers():
    # the known-answer vectors of the generator's authors (philox4x32, 10 rounds)
    zero = [int(v) for v in philox((0, 0, 0, 0), (0, 0))]
    assert zero == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = [int(v) for v in philox((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2)]
    assert ones == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


@pytest.mark.parametrize("over", [dict(dtype=3), dict(n=-1), dict(p=-0.1), dict(p=1.1),
                                  dict(p=float("nan")), dict(x=None), dict(y=None)])
def test_library_refuses(over):
    from softmax_cross_entropy_gb300 import _lib
    a = dict(x=16, residual=None, y=32, dtype=_lib.CE_F32, n=4, p=0.5, seed=1, offset=0,
             state=None, used=None, stream=None)
    a.update(over)
    assert _lib.ce_dropout(**a) == _lib.CE_ERR_INVALID_ARG


def test_wrapper_refuses_cpu_tensors():
    import softmax_cross_entropy_gb300 as gbce
    with pytest.raises(ValueError):
        gbce.dropout(torch.zeros(4), 0.5, 1)


def test_tangents_are_refused_not_dropped(monkeypatch):
    # a dual tensor does not require a gradient (the library's call is a copy here)
    import softmax_cross_entropy_gb300 as gbce
    from softmax_cross_entropy_gb300 import philox_dropout
    from torch.autograd import forward_ad
    monkeypatch.setattr(philox_dropout, "require_cuda", lambda *a: None)
    monkeypatch.setattr(philox_dropout, "_call", lambda x, *a: x.detach().clone())
    x = torch.randn(5)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones(5))
        for args in ((dual, None), (x, dual)):
            with pytest.raises(NotImplementedError):
                gbce.dropout(args[0], 0.0, 1, residual=args[1])
            with pytest.raises(NotImplementedError), torch.no_grad():
                gbce.dropout(args[0], 0.0, 1, residual=args[1])
        assert torch.equal(gbce.dropout(x, 0.0, 1), x)
    assert torch.equal(gbce.dropout(x, 0.0, 1), x)


def test_a_gradient_with_a_tangent_is_refused(monkeypatch):
    import softmax_cross_entropy_gb300 as gbce
    from softmax_cross_entropy_gb300 import philox_dropout
    from torch.autograd import forward_ad
    monkeypatch.setattr(philox_dropout, "require_cuda", lambda *a: None)
    monkeypatch.setattr(philox_dropout, "_call", lambda x, *a: x.detach().clone())
    x, dy = torch.randn(5, requires_grad=True), torch.randn(5)
    with forward_ad.dual_level():
        y = gbce.dropout(x, 0.0, 1)
        with pytest.raises(RuntimeError, match="once"):
            torch.autograd.grad(y, [x], forward_ad.make_dual(dy, torch.ones(5)), retain_graph=True)
        assert torch.equal(torch.autograd.grad(y, [x], dy)[0], dy)


# ---------------------------------------------------------------- GPU

def expected(x, res, kept, p):
    """(y, bound): y in 64 bits, and how far the kernel may be off: the scale and the product are
    rounded to fp32 (2^-24 each of the product), the sum to fp32, and the result to its type
    (half a step, eps / 2; below the smallest normal, half the smallest step)."""
    s = np.where(kept, x / (1.0 - p) if p < 1 else 0.0, 0.0)
    y = s + (res if res is not None else 0.0)
    return y, s


def check(got, x, res, kept, p, dt):
    y, s = expected(x, res, kept, p)
    info = torch.finfo(dt)
    half = info.eps / 2
    bound = 2.0 ** -24 * (2.01 * np.abs(s) + np.abs(y)) + half * 1.01 * np.abs(y) + \
        info.smallest_normal * half
    assert np.all(np.abs(got.detach().double().cpu().numpy().reshape(-1) - y) <= bound)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [1, 3, 4, 7, 8, 16, 1001, 4096, 70001])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
def test_forward_and_backward(dtype, n, p, residual, shift):
    import softmax_cross_entropy_gb300 as gbce
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(n + 7)
    seed, offset = 0x123456789ABCDEF, 0x100000003

    def make():  # shift 1: a contiguous tensor whose base is not 16-byte aligned
        return torch.randn(n + shift, generator=g, device="cuda").to(dt)[shift:]

    x, dy = make().requires_grad_(), make()
    res = make().requires_grad_() if residual else None
    y = gbce.dropout(x, p, seed, offset, residual=res)
    kept = keep(n, p, seed, offset)
    f64 = lambda t: None if t is None else t.detach().double().cpu().numpy()  # noqa: E731
    check(y, f64(x), f64(res), kept, p, dt)
    grads = torch.autograd.grad(y, [x] + ([res] if residual else []), dy)
    check(grads[0], f64(dy), None, kept, p, dt)
    if residual:
        assert torch.equal(grads[1], dy)


@pytest.mark.gpu
def test_dropped_elements_leave_nothing():
    import softmax_cross_entropy_gb300 as gbce
    kept = torch.from_numpy(keep(4096, 0.5, 9)).cuda()
    for bad in (float("inf"), float("-inf"), float("nan")):
        x = torch.ones(4096, device="cuda")
        x[~kept] = bad
        y = gbce.dropout(x, 0.5, 9)
        assert torch.equal(y, torch.where(kept, 2.0, 0.0))
        assert torch.equal(gbce.dropout(torch.full_like(x, bad), 1.0, 9), torch.zeros_like(x))


@pytest.mark.gpu
def test_shapes_strides_and_empty():
    import softmax_cross_entropy_gb300 as gbce
    x = torch.randn(6, 5, 8, device="cuda").transpose(0, 2)
    y = gbce.dropout(x, 0.3, 4)
    assert y.shape == x.shape
    kept = torch.from_numpy(keep(240, 0.3, 4)).cuda().reshape(8, 5, 6)
    torch.testing.assert_close(y, torch.where(kept, x / 0.7, 0.0), rtol=2 ** -22, atol=0)
    assert gbce.dropout(torch.empty(0, 3, device="cuda"), 0.3, 4).shape == (0, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("bits,state", [(32, False), (33, True), (34, False), (34, True)])
def test_elements_past_32_bits(bits, state):
    # a launch's last element (2^33), the block counter's low word (2^34)
    import softmax_cross_entropy_gb300 as gbce
    n = 2 ** bits + 13
    seed = torch.tensor([77, 5], device="cuda") if state else 77
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = gbce.dropout(x, 0.5, seed)
    for first in (2 ** bits - 64, 2 ** (bits - 1) - 32):
        kept = keep(77, 0.5, 77, 5 if state else 0, first)
        assert np.array_equal(y[first:first + 77].float().cpu().numpy(), np.where(kept, 2.0, 0.0))
    del x, y
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_same_leaf_as_input_and_residual():
    import softmax_cross_entropy_gb300 as gbce
    x = torch.randn(1000, device="cuda", requires_grad=True)
    gbce.dropout(x, 0.25, 3, residual=x).sum().backward()
    kept = torch.from_numpy(keep(1000, 0.25, 3)).cuda()
    assert torch.equal(x.grad, 1.0 + torch.where(kept, torch.tensor(1 / 0.75, device="cuda"), 0.0))


@pytest.mark.gpu
def test_seed_tensor_and_its_update_before_the_backward():
    import softmax_cross_entropy_gb300 as gbce
    state = torch.tensor([41, 6], dtype=torch.int64, device="cuda")
    x = torch.ones(513, device="cuda", requires_grad=True)
    y = gbce.dropout(x, 0.5, state, offset=2)
    state += 1
    y.sum().backward()
    want = torch.from_numpy(np.where(keep(513, 0.5, 41, 8), 2.0, 0.0)).float().cuda()
    assert torch.equal(y.detach(), want) and torch.equal(x.grad, want)


@pytest.mark.gpu
def test_captured_step_draws_anew():
    import softmax_cross_entropy_gb300 as gbce
    state = torch.tensor([5, 0], dtype=torch.int64, device="cuda")
    x = torch.ones(2048, device="cuda", dtype=torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = gbce.dropout(x, 0.5, state)
    for i in range(3):
        state.copy_(torch.tensor([5, i]))
        graph.replay()
        assert np.array_equal(y.float().cpu().numpy(), np.where(keep(2048, 0.5, 5, i), 2.0, 0.0))


@pytest.mark.gpu
def test_another_stream():
    import softmax_cross_entropy_gb300 as gbce
    s = torch.cuda.Stream()
    x = torch.ones(4096, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = gbce.dropout(x, 0.5, 12)
    s.synchronize()
    assert np.array_equal(y.cpu().numpy(), np.where(keep(4096, 0.5, 12), 2.0, 0.0))


@pytest.mark.gpu
def test_wrapper_refuses():
    import softmax_cross_entropy_gb300 as gbce
    x = torch.ones(8, device="cuda")
    with pytest.raises(ValueError):
        gbce.dropout(x, 1.5, 1)
    with pytest.raises(ValueError):
        gbce.dropout(x, 0.5, None)
    with pytest.raises(ValueError):
        gbce.dropout(x, 0.5, torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        gbce.dropout(x, 0.5, 1, residual=torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        gbce.dropout(x, 0.5, 1, residual=torch.ones(8, device="cuda", dtype=torch.float16))
    with pytest.raises(TypeError):
        gbce.dropout(x.double(), 0.5, 1)


@pytest.mark.gpu
def test_second_derivatives_are_refused():
    import softmax_cross_entropy_gb300 as gbce
    x = torch.ones(8, device="cuda", requires_grad=True)
    with pytest.raises(RuntimeError, match="once"):
        torch.autograd.grad(gbce.dropout(x, 0.5, 1).sum(), [x], create_graph=True)
