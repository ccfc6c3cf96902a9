"""The beam search step and the reordering of states: refusals (CPU), and the
kernels against a stable sort of the definition in 64 bits (GPU)."""
import contextlib
import ctypes
import math

import numpy as np
import pytest
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def reference(logits, scores, M, finished=None, pad=0):
    """(scores in 64 bits, beams, tokens) by the definition."""
    x = logits.double().cpu().numpy()
    s = scores.double().cpu().numpy()
    B, K, V = x.shape
    x = np.where(np.isnan(x), -np.inf, x)
    out = (np.full((B, M), -np.inf), np.full((B, M), -1), np.full((B, M), pad))
    for b in range(B):
        tot = np.full((K, V), -np.inf)
        for k in range(K):
            if not np.isfinite(s[b, k]):
                continue
            if finished is not None and bool(finished[b, k]):
                tot[k, pad] = s[b, k]
                continue
            m = x[b, k].max()
            if not np.isfinite(m):
                continue
            tot[k] = s[b, k] + ((x[b, k] - m) - math.log(np.exp(x[b, k] - m).sum()))
        tot = tot.reshape(-1)
        order = np.argsort(-tot, kind="stable")[:M]
        order = order[tot[order] > -np.inf]
        out[0][b, :len(order)] = tot[order]
        out[1][b, :len(order)] = order // V
        out[2][b, :len(order)] = order % V
    return out


def compare(got, want):
    assert np.array_equal(got.beams.cpu().numpy(), want[1])
    assert np.array_equal(got.tokens.cpu().numpy(), want[2])
    g = got.scores.double().cpu().numpy()
    none = np.isinf(want[0])
    assert np.array_equal(np.isinf(g), none)
    # the fp32 output's half step, and 2^-20 of the log-sum-exp: each fp32 exponential is off by
    # a few 2^-24 relative (the product with log2 e, the exponent), and their sum by less than
    # 2^-24 for each of the ~12 levels of additions a term goes through
    w = np.where(none, 0.0, want[0])
    assert np.all(np.abs(np.where(none, 0.0, g) - w) <= 2.0 ** -24 * np.abs(w) * 1.01 + 2.0 ** -20)


# ---------------------------------------------------------------- CPU

def select(**over):
    from softmax_cross_entropy_gb300 import _lib
    a = dict(logits=256, dtype=_lib.CE_F32, B=2, K=4, V=100, scores=512, finished=None,
             pad_token=0, M=8, out_scores=768, out_beams=1024, out_tokens=1280, workspace=4096,
             workspace_bytes=1 << 20, stream=None)
    a.update(over)
    return _lib.ce_beam_select(**a)


@pytest.mark.parametrize("over", [
    dict(dtype=3), dict(B=-1), dict(K=0), dict(V=0), dict(M=0), dict(pad_token=-1),
    dict(pad_token=100), dict(logits=None), dict(scores=None), dict(out_scores=None),
    dict(out_beams=None), dict(out_tokens=None), dict(workspace=None), dict(workspace=4100),
    dict(workspace_bytes=16), dict(logits=258)])
def test_select_refuses(over):
    from softmax_cross_entropy_gb300 import _lib
    assert select(**over) == _lib.CE_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [dict(K=33), dict(M=65), dict(V=2 ** 31 - 1), dict(B=2 ** 21)])
def test_select_sizes_it_does_not_take(over):
    from softmax_cross_entropy_gb300 import _lib
    assert select(**over) == _lib.CE_ERR_UNSUPPORTED
    assert _lib.ce_beam_workspace_bytes(0, over.get("B", 2), over.get("K", 4), over.get("V", 100),
                                        over.get("M", 8)) == 0


def test_select_of_no_entries_is_a_no_op():
    from softmax_cross_entropy_gb300 import _lib
    assert select(B=0, logits=None, workspace=None) == _lib.CE_OK


def reorder(n=1, beams=64, row=None, B=2, K=4, **over):
    from softmax_cross_entropy_gb300 import _lib
    at = (_lib.BeamState * 1)()
    f = dict(src=256, dst=512, src_row=16, src_block=0, dst_row=16, dst_block=0, blocks=1,
             block_bytes=16)
    f.update(over)
    for k, v in f.items():
        setattr(at[0], k, v)
    return _lib.ce_beam_reorder(at if n else None, n, beams, K if row is None else row, B, K, None)


@pytest.mark.parametrize("over", [
    dict(n=-1), dict(B=-1), dict(K=0), dict(row=3), dict(beams=None), dict(src=None), dict(dst=None),
    dict(blocks=-1), dict(block_bytes=-1), dict(dst=256, dst_row=32),
    dict(dst=256, dst_block=8)])
def test_reorder_refuses(over):
    from softmax_cross_entropy_gb300 import _lib
    assert reorder(**over) == _lib.CE_ERR_INVALID_ARG


def test_reorder_sizes():
    from softmax_cross_entropy_gb300 import _lib
    assert reorder(K=33) == _lib.CE_ERR_UNSUPPORTED
    assert reorder(n=0) == _lib.CE_OK and reorder(B=0) == _lib.CE_OK


def test_reorder_refuses_one_state_twice():
    from softmax_cross_entropy_gb300 import _lib
    one = (256, 512, 16, 0, 16, 0, 1, 16)
    at = (_lib.BeamState * 2)(one, (256 + 64, *one[1:]))
    assert _lib.ce_beam_reorder(at, 2, 64, 4, 2, 4, None) == _lib.CE_ERR_INVALID_ARG


def test_wrapper_refuses_cpu_tensors():
    import softmax_cross_entropy_gb300 as gbce
    with pytest.raises(ValueError):
        gbce.beam_search_step(torch.zeros(1, 2, 3), torch.zeros(1, 2))
    with pytest.raises(ValueError):
        gbce.beam_reorder(torch.zeros(2, 3), torch.zeros(1, 2, dtype=torch.int64))


def host_reorder(states, n, beams, beams_row, B, K, stream):
    """ce_beam_reorder by its definition on host memory."""
    if beams_row < K:
        return 1  # CE_ERR_INVALID_ARG
    for s in list(states)[:n]:
        for b in range(B):
            take = (ctypes.c_int64 * K).from_address(beams + 8 * b * beams_row)
            rows = [[ctypes.string_at(s.src + (b * K + (f if 0 <= f < K else j)) * s.src_row +
                                      o * s.src_block, s.block_bytes) for o in range(s.blocks)]
                    for j, f in enumerate(take)]
            for j, row in enumerate(rows):
                for o, block in enumerate(row):
                    ctypes.memmove(s.dst + (b * K + j) * s.dst_row + o * s.dst_block, block, s.block_bytes)
    return 0


@pytest.fixture
def on_host(monkeypatch):
    """The wrapper on CPU tensors, the library's reordering on host memory."""
    import softmax_cross_entropy_gb300 as gbce
    from softmax_cross_entropy_gb300 import beam_search
    monkeypatch.setattr(beam_search, "require_cuda", lambda *a: None)
    monkeypatch.setattr(beam_search, "on", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(beam_search, "stream", lambda device: 0)
    monkeypatch.setattr(beam_search._lib, "ce_beam_reorder", host_reorder)
    return gbce


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("kind", ["conj", "neg", "conj_strided", "neg_strided"])
def test_states_that_defer_a_conjugation_or_negation(on_host, inplace, kind):
    z = torch.randn(6, 5, dtype=torch.complex64)
    z = z[:, :4] if "strided" in kind else z
    t = z.conj() if "conj" in kind else z.conj().imag
    assert t.is_conj() or t.is_neg()
    beams = torch.tensor([[1, 1, 0], [2, -1, 0]])
    want = t.clone()[[1, 1, 0, 5, 4, 3]]
    got = on_host.beam_reorder(t, beams, inplace=inplace)
    assert (got is t) == inplace and torch.equal(got, want)


@pytest.mark.parametrize("beams", [
    torch.tensor([[1], [0], [1]]).t(), torch.tensor([1, 0, 1]).as_strided((1, 3), (0, 1)),
    torch.tensor([1, 9, 0, 9, 1]).as_strided((1, 3), (1, 2)), torch.tensor([[1, 0, 1, 7]])[:, :3]])
def test_beams_of_one_entry_whatever_their_strides(on_host, beams):
    state = torch.randn(3, 4)
    assert torch.equal(on_host.beam_reorder(state, beams), state[[1, 0, 1]])


def test_beams_that_are_part_of_a_state(on_host):
    # the history of the chosen beams [T, B, K] is a state like the others
    B, K, T = 2, 3, 4
    parents = torch.randint(0, K, (T, B, K))
    parents[2] = torch.tensor([[1, 1, 0], [2, 0, 0]])
    history, cache = parents.permute(1, 2, 0), torch.randn(B * K, 5)
    rows = [1, 1, 0, 5, 3, 3]
    want = [history.clone().reshape(B * K, T)[rows].reshape(B, K, T), cache[rows]]
    on_host.beam_reorder([history, cache], parents[2], inplace=True)
    assert torch.equal(history, want[0]) and torch.equal(cache, want[1])
    whole = parents[2].clone()
    want = whole.reshape(B * K)[rows].reshape(B, K)
    on_host.beam_reorder([whole, cache], torch.tensor([[1, 1, 0], [2, 0, 0]]), inplace=True)
    assert torch.equal(whole, want)


def test_wrappers_take_the_values_of_negated_views():
    from softmax_cross_entropy_gb300 import _tensors, feed_forward
    for t in (torch.tensor([1 + 2j]).conj().imag, torch._neg_view(torch.arange(16.0))):
        assert t.is_neg() and t.is_contiguous()
        for f in (_tensors.plain, feed_forward.aligned):
            assert not f(t).is_neg() and torch.equal(f(t), t)


def test_states_with_tangents_are_not_changed_in_place(monkeypatch):
    import softmax_cross_entropy_gb300 as gbce
    from softmax_cross_entropy_gb300 import beam_search
    from torch.autograd import forward_ad
    monkeypatch.setattr(beam_search, "require_cuda", lambda *a: None)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(torch.randn(2, 3), torch.ones(2, 3))
        with pytest.raises(ValueError, match="tangent"):
            gbce.beam_reorder(dual, torch.zeros(1, 2, dtype=torch.int64), inplace=True)


# ---------------------------------------------------------------- GPU

def inputs(B, K, V, dtype, seed=0, scale=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(B, K, V, generator=g, device="cuda") * scale).to(DT[dtype])
    return x, -10 * torch.rand(B, K, generator=g, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,K,V,M", [
    (1, 1, 1, 1), (1, 1, 3, 5), (2, 3, 2, 16), (3, 4, 7, 8), (2, 5, 33, 10), (1, 4, 1000, 8),
    (2, 8, 1023, 16), (1, 1, 50001, 64), (3, 7, 4097, 33), (2, 32, 257, 64), (9, 16, 515, 32),
    (1, 2, 131072, 4), (40, 5, 8191, 10), (1, 32, 30001, 64)])
def test_selection(dtype, B, K, V, M):
    import softmax_cross_entropy_gb300 as gbce
    x, s = inputs(B, K, V, dtype, seed=V + K)
    compare(gbce.beam_search_step(x, s, num_candidates=M), reference(x, s, M))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 5000, 64000])
@pytest.mark.parametrize("kind", ["equal", "ascending", "descending", "two_values", "zeros"])
def test_ties_and_orders(dtype, V, kind):
    # one beam an entry, so that equal logits are exactly equal scores
    import softmax_cross_entropy_gb300 as gbce
    i = torch.arange(V, device="cuda")
    row = {"equal": torch.full((V,), -2.5, device="cuda"), "ascending": i * 1e-3,
           "descending": i * -1e-3, "two_values": (i % 7 == 3).float() * 4,
           # -0 and +0 are the same logit
           "zeros": torch.where(i % 2 == 0, -0.0, 0.0)}[kind]
    x = row.to(DT[dtype]).expand(2, 1, V).contiguous()
    s = torch.zeros(2, 1, device="cuda")
    for M in (1, 31, 32, 33, 64):
        compare(gbce.beam_search_step(x, s, num_candidates=M), reference(x, s, M))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [4096, 4097, 65001, 65003])
def test_equal_beams_take_the_lowest_first(dtype, V):
    # odd V: the equal rows start at different places of a 16-byte vector
    import softmax_cross_entropy_gb300 as gbce
    x, _ = inputs(2, 1, V, dtype)
    x = x.expand(2, 6, V).contiguous()
    s = torch.full((2, 6), -1.5, device="cuda")
    compare(gbce.beam_search_step(x, s, num_candidates=12), reference(x, s, 12))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [5, 1001, 33000])
def test_masks_and_what_is_not_finite(dtype, V):
    import softmax_cross_entropy_gb300 as gbce
    x, s = inputs(7, 4, V, dtype, seed=V)
    low = torch.finfo(DT[dtype]).min
    x[0, 0] = -math.inf                # no token left
    x[0, 1, 1:] = -math.inf            # one token left
    x[1] = -math.inf                   # no token in the whole entry
    x[2, :, ::2] = math.nan            # NaN counts as masked
    x[3, 2, V // 2] = math.inf         # no finite log-sum-exp: no candidates
    x[4, 1] = low                      # the type's lowest value is a value: all equal
    x[4, 2, : V // 2] = low
    s[5, 0], s[5, 1], s[5, 3] = -math.inf, math.nan, math.inf  # dead beams
    s[6] = -math.inf
    compare(gbce.beam_search_step(x, s, num_candidates=8), reference(x, s, 8))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 8, 40])
def test_finished_beams(M):
    import softmax_cross_entropy_gb300 as gbce
    x, s = inputs(4, 4, 3001, "bf16")
    fin = torch.zeros(4, 4, dtype=torch.bool, device="cuda")
    fin[0, 1] = fin[1, :] = fin[2, 0] = fin[3, 3] = True
    s[1, 2] = -math.inf       # finished and dead
    x[0, 1] = math.nan        # not read
    s[3, 3] = -1e30           # far behind
    got = gbce.beam_search_step(x, s, num_candidates=M, finished=fin, pad_token=17)
    compare(got, reference(x, s, M, fin, 17))


@pytest.mark.gpu
def test_two_streams_at_once_and_a_captured_step():
    import softmax_cross_entropy_gb300 as gbce
    ins = [inputs(3, 4, 20011, "bf16", seed=i) for i in range(4)]
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    outs = []
    for (x, s), st in zip(ins, streams):
        with torch.cuda.stream(st):
            outs.append(gbce.beam_search_step(x, s, num_candidates=8))
    torch.cuda.synchronize()
    for (x, s), o in zip(ins, outs):
        compare(o, reference(x, s, 8))
    x, s = (t.clone() for t in ins[0])
    cache = torch.randn(12, 5, 8, device="cuda")
    kept = cache.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        best = gbce.beam_search_step(x, s)
        gbce.beam_reorder(cache, best.beams, inplace=True)
    for xi, si in ins[1:3]:
        x.copy_(xi)
        s.copy_(si)
        cache.copy_(kept)
        graph.replay()
        want = reference(xi, si, 4)
        compare(best, want)
        rows = (np.arange(3)[:, None] * 4 + want[1]).reshape(-1)
        assert torch.equal(cache, kept[torch.from_numpy(rows).cuda()])


def plain_reorder(state, beams):
    B, K = beams.shape
    b = torch.where((beams < 0) | (beams >= K), torch.arange(K, device=beams.device), beams)
    rows = (torch.arange(B, device=beams.device)[:, None] * K + b).reshape(-1)
    return state.reshape(B * K, *state.shape[2 if state.shape[:2] == (B, K) else 1:])[rows] \
        .reshape(state.shape)


@pytest.mark.gpu
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.int64, torch.bool])
@pytest.mark.parametrize("B,K,shape", [(1, 1, (3,)), (2, 4, (1,)), (3, 5, (7, 3)),
                                       (2, 16, (4, 9, 16)), (1, 32, (2, 64)), (5, 8, (3, 33, 40))])
def test_reorder(inplace, dtype, B, K, shape):
    import softmax_cross_entropy_gb300 as gbce
    g = torch.Generator(device="cuda").manual_seed(3)
    beams = torch.randint(-1, K + 1, (B, K), generator=g, device="cuda")
    a = torch.randint(0, 100, (B * K, *shape), generator=g, device="cuda").to(dtype)
    b = torch.randint(0, 100, (B, K, *shape), generator=g, device="cuda").to(dtype)
    want = [plain_reorder(t, beams) for t in (a, b)]
    got = gbce.beam_reorder([a, b], beams, inplace=inplace)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (got[0] is a) == inplace


@pytest.mark.gpu
@pytest.mark.parametrize("inplace", [False, True])
def test_reorder_of_strided_states(inplace):
    import softmax_cross_entropy_gb300 as gbce
    beams = torch.tensor([[1, 1, 0], [2, -1, 0]], device="cuda")
    cache = torch.randn(6, 4, 32, 8, device="cuda")           # [B K, heads, length, dim]
    heads = torch.randn(4, 6, 10, 8, device="cuda")           # heads first
    odd = torch.randn(6 * 7 + 1, device="cuda").half()[1:].view(6, 7)
    before = [t.clone() for t in (cache, heads, odd)]
    views = [cache[:, :, :19], heads.transpose(0, 1), odd]
    want = [plain_reorder(v.clone(), beams) for v in views]
    got = gbce.beam_reorder(views, beams, inplace=inplace)
    for w, v in zip(want, got):
        assert torch.equal(w, v)
    assert torch.equal(cache[:, :, 19:], before[0][:, :, 19:])  # behind the last position
    if not inplace:
        assert torch.equal(cache, before[0]) and torch.equal(heads, before[1])


@pytest.mark.gpu
@pytest.mark.parametrize("inplace", [False, True])
def test_reorder_of_one_beam(inplace):
    # the beams' dimension of one has a stride of its own (here 5 * 8, rows are 9 * 8 apart)
    import softmax_cross_entropy_gb300 as gbce
    cache = torch.randn(4, 9, 8, device="cuda")
    state = cache[:, :5].unsqueeze(1)
    want = state.clone()
    got = gbce.beam_reorder(state, torch.tensor([[0], [-1], [0], [0]], device="cuda"), inplace=inplace)
    assert got.shape == want.shape and torch.equal(got, want)


@pytest.mark.gpu
def test_reorder_in_place_is_seen_by_autograd():
    import softmax_cross_entropy_gb300 as gbce
    beams = torch.tensor([[1, 0, 2]], device="cuda")
    state = torch.randn(3, 8, device="cuda")
    w = torch.randn(3, 8, device="cuda", requires_grad=True)
    y = (w * state).sum()
    gbce.beam_reorder([state], beams, inplace=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        t = torch.randn(3, 8, device="cuda")
        want = t[[1, 0, 2]]
        assert torch.equal(gbce.beam_reorder(t, beams, inplace=True), want)


@pytest.mark.gpu
def test_reorder_of_the_beams_own_history():
    import softmax_cross_entropy_gb300 as gbce
    B, K, T = 64, 8, 16
    parents = torch.randint(0, K, (T, B, K), device="cuda")
    history, cache = parents.permute(1, 2, 0), torch.randn(B * K, 4096, device="cuda")
    want = [plain_reorder(t.clone(), parents[5].clone()) for t in (history, cache)]
    gbce.beam_reorder([history, cache], parents[5], inplace=True)
    assert torch.equal(history, want[0]) and torch.equal(cache, want[1])


@pytest.mark.gpu
def test_values_of_conjugated_and_negated_views():
    import softmax_cross_entropy_gb300 as gbce
    z = torch.randn(3, 4, dtype=torch.complex64, device="cuda")
    beams = torch.tensor([[1, 0, 2]], device="cuda")
    for t in (z.conj(), z.conj().imag):
        assert torch.equal(gbce.beam_reorder(t, beams), t.clone()[[1, 0, 2]])
    x = torch._neg_view(torch.randn(2, 3, 40, device="cuda"))
    s = torch._neg_view(torch.rand(2, 3, device="cuda"))
    compare(gbce.beam_search_step(x, s), reference(x.clone(), s.clone(), 3))
    assert torch.equal(gbce.dropout(x, 0.0, 1, residual=x), 2 * x.clone())


@pytest.mark.gpu
def test_no_entries():
    import softmax_cross_entropy_gb300 as gbce
    best = gbce.beam_search_step(torch.empty(0, 3, 7, device="cuda"), torch.empty(0, 3, device="cuda"))
    assert best.scores.shape == best.beams.shape == best.tokens.shape == (0, 3)
    assert gbce.beam_reorder(torch.empty(0, 5, device="cuda"), best.beams).shape == (0, 5)


@pytest.mark.gpu
@pytest.mark.parametrize("V,dtype", [(2 ** 20, "f32"), (2 ** 20 - 3, "bf16")])
def test_the_largest_vocabulary(V, dtype):
    import softmax_cross_entropy_gb300 as gbce
    x, s = inputs(1, 3, V, dtype)
    compare(gbce.beam_search_step(x, s, num_candidates=64), reference(x, s, 64))


@pytest.mark.gpu
@pytest.mark.parametrize("B,K,M", [(1, 32, 64), (1, 1, 64), (2, 2, 33)])
def test_the_most_parts(B, K, M):
    # 32 beams of 94 parts, one row in as many as the GPU is given, and few rows between
    import softmax_cross_entropy_gb300 as gbce
    x, s = inputs(B, K, 2 ** 20, "f32", seed=K)
    got = gbce.beam_search_step(x, s, num_candidates=M)
    # only a beam's best M can be among them: the rest counts in its log-sum-exp alone
    val, at = x.topk(M, dim=2)
    lse = torch.logsumexp(x.double(), 2)
    tot = (s.double()[..., None] + (val.double() - lse[..., None])).cpu().numpy().reshape(B, -1)
    at = (torch.arange(K, device="cuda")[:, None] * 2 ** 20 + at).cpu().numpy().reshape(B, -1)
    order = np.lexsort((at, -tot))[:, :M]
    tot, at = np.take_along_axis(tot, order, 1), np.take_along_axis(at, order, 1)
    compare(got, (tot, at // 2 ** 20, at % 2 ** 20))


@pytest.mark.gpu
def test_logits_past_32_bits():
    import softmax_cross_entropy_gb300 as gbce
    B, K, V = 66, 32, 2 ** 20 - 1
    x = torch.empty(B, K, V, dtype=torch.bfloat16, device="cuda").normal_()
    s = -torch.rand(B, K, device="cuda")
    s[1:-1] = -math.inf  # entries whose logits are not read
    got = gbce.beam_search_step(x, s, num_candidates=4)
    last = gbce.BeamCandidates(*(t[-1:] for t in got))
    compare(last, reference(x[-1:], s[-1:], 4))
    assert bool((got.beams[1:-1] == -1).all())
    del x
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_many_equal_logits_next_to_better_ones():
    # more logits reach the bound than a part lists: equal ones, in several beams and parts
    import softmax_cross_entropy_gb300 as gbce
    x = torch.zeros(3, 4, 70001, device="cuda")
    x[0, :, ::3] = 1.0
    x[1, 2, 69990:] = 5.0
    x[2, 1, 5] = x[2, 3, 70000] = 2.0
    s = torch.tensor([[-1.0, -1.5, -1.25, -3.0]], device="cuda").expand(3, 4).contiguous()
    for M in (3, 16, 40):
        for t in (x, x.bfloat16()):
            compare(gbce.beam_search_step(t, s, num_candidates=M), reference(t, s, M))


@pytest.mark.gpu
def test_reorder_by_a_part_of_the_candidates():
    import softmax_cross_entropy_gb300 as gbce
    g = torch.Generator(device="cuda").manual_seed(1)
    every = torch.randint(-1, 4, (5, 8), generator=g, device="cuda")
    state = torch.randn(20, 6, device="cuda")
    for beams in (every[:, :4], every[:, 2:6], every.t()[:5, :4], every[:1, :4].expand(5, 4)):
        assert torch.equal(gbce.beam_reorder(state, beams), plain_reorder(state, beams))


@pytest.mark.gpu
def test_reorder_of_many_states_and_of_none():
    import softmax_cross_entropy_gb300 as gbce
    beams = torch.tensor([[3, 0, 0, 1]], device="cuda")
    states = [torch.randn(4, 3 + i, device="cuda") for i in range(37)]
    want = [plain_reorder(t, beams) for t in states]
    gbce.beam_reorder(states, beams, inplace=True)
    assert all(torch.equal(a, b) for a, b in zip(states, want))
    assert gbce.beam_reorder([], beams) == []
    assert gbce.beam_reorder(torch.empty(4, 0, device="cuda"), beams).shape == (4, 0)


@pytest.mark.gpu
def test_reorder_offsets_past_32_bits():
    import softmax_cross_entropy_gb300 as gbce
    state = torch.zeros(4, 2 ** 31 + 16, dtype=torch.uint8, device="cuda")
    state[:, -5:] = torch.arange(4, device="cuda", dtype=torch.uint8)[:, None] + 1
    gbce.beam_reorder(state, torch.tensor([[3, 3, 0, 2]], device="cuda"), inplace=True)
    assert state[:, -1].tolist() == [4, 4, 1, 3] and state[:, -6].tolist() == [0, 0, 0, 0]


@pytest.mark.gpu
def test_wrapper_refuses():
    import softmax_cross_entropy_gb300 as gbce
    x, s = inputs(2, 3, 10, "f32")
    for bad in (dict(scores=s.double()), dict(scores=s[:1]), dict(pad_token=10),
                dict(num_candidates=0), dict(finished=torch.zeros(2, 3, device="cuda"))):
        with pytest.raises(ValueError):
            gbce.beam_search_step(**{"logits": x, "scores": s, **bad})
    with pytest.raises(TypeError):
        gbce.beam_search_step(x.double(), s)
    with pytest.raises(gbce.CEError):
        gbce.beam_search_step(x, s, num_candidates=65)
    beams = torch.zeros(2, 3, dtype=torch.int64, device="cuda")
    for state in (torch.zeros(5, 4, device="cuda"), torch.zeros(6, 1, device="cuda").expand(6, 4),
                  torch.zeros(1, 4, device="cuda").expand(6, 4),
                  torch.zeros(6, 8, 9, 10, device="cuda")[:, ::2, :, ::2],
                  torch.zeros(6, 4, device="cuda", requires_grad=True)):
        with pytest.raises(ValueError):
            gbce.beam_reorder(state, beams, inplace=True)
    with pytest.raises(ValueError):
        gbce.beam_reorder(torch.zeros(6, 4, device="cuda"), beams.int())
    twice = torch.zeros(6, 4, device="cuda")
    with pytest.raises(ValueError):
        gbce.beam_reorder([twice, twice], beams, inplace=True)


@pytest.mark.gpu
def test_three_steps_find_the_best_sequences_of_the_kept_prefixes():
    # a model whose next logits depend on the last token alone; the states that are reordered are
    # the sequences so far
    import softmax_cross_entropy_gb300 as gbce
    V = K = 5
    g = torch.Generator().manual_seed(0)
    table = torch.randn(V + 1, V, generator=g, dtype=torch.float32)
    lp = torch.log_softmax(table.double(), 1)
    every = {(a, b, c): float(lp[V, a] + lp[a, b] + lp[b, c])
             for a in range(V) for b in range(V) for c in range(V)}
    dev_table = table.cuda()
    last = torch.full((1, K), V, device="cuda")
    scores = torch.full((1, K), -math.inf, device="cuda")
    scores[0, 0] = 0.0
    history = torch.zeros(K, 3, dtype=torch.int64, device="cuda")
    for step in range(2):
        best = gbce.beam_search_step(dev_table[last], scores)
        gbce.beam_reorder(history, best.beams, inplace=True)
        last, scores = best.tokens, best.scores
        history[:, step] = last[0]
    best = gbce.beam_search_step(dev_table[last], scores, num_candidates=3)
    prefixes = {tuple(r) for r in history[:, :2].tolist()}
    within = sorted((v, k) for k, v in every.items() if k[:2] in prefixes)[::-1][:3]
    found = [(*history[int(b)][:2].tolist(), int(t)) for b, t in zip(best.beams[0], best.tokens[0])]
    assert found == [k for _, k in within]
    assert np.allclose(best.scores[0].cpu().numpy(), [v for v, _ in within], atol=1e-5)
