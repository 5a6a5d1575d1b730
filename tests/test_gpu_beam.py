"""qmv_beam_select against the definition.

The scores are fp32 steps on a log-sum-exp whose own error is below 2^-20 of
1 + |lse| (fp32 sums of at most 2^18 exponentials, each within 2^-22, added in
blocks), so scores are held to 2^-20 (1 + |lse|) + 2^-22 |c|.  Which entries win
is checked exactly where the definition decides it by whole steps (ties,
infinities) and by the scores' tolerance elsewhere."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _select(dev, logits, scores, num, **kw):
    import torch

    import bit_affine_quantized_amd as qm
    s, p, t = qm.qmv_beam_select(logits, torch.from_numpy(scores).to(dev), num, **kw)
    torch.cuda.synchronize()
    return s.double().cpu().numpy(), p.cpu().numpy(), t.cpu().numpy()


def _check(dev, x, scores, num, f32):
    """x: torch [B, W, V] on the device; all finite logits, no ties across rows needed."""
    got, par, tok = _select(dev, x, scores, num)
    X = x.double().cpu().numpy()
    B, W, V = X.shape
    m = X.max(-1, keepdims=True)
    lse = m + np.log(np.exp(X - m).sum(-1, keepdims=True))
    c = (scores.astype(np.float64)[..., None] + (X - lse)).reshape(B, W * V)
    tol = 2.0 ** -20 * (1 + np.abs(lse).max()) + 2.0 ** -22 * np.abs(got[np.isfinite(got)]).max(initial=1.0)
    for b in range(B):
        order = np.argsort(-c[b], kind="stable")[:num]
        np.testing.assert_allclose(got[b], c[b][order], rtol=0, atol=tol)
        at = par[b].astype(np.int64) * V + tok[b]
        assert len(set(at.tolist())) == num and np.all((tok[b] >= 0) & (tok[b] < V) & (par[b] >= 0) & (par[b] < W))
        np.testing.assert_allclose(c[b][at], got[b], rtol=0, atol=tol)
        for i in range(num - 1):                       # best first, exact ties by index
            assert got[b, i] > got[b, i + 1] or (got[b, i] == got[b, i + 1] and at[i] < at[i + 1])
        sure = np.abs(np.diff(np.sort(-c[b])[:num + 1])).min(initial=1.0) > 4 * tol if W * V > num else True
        if sure:
            np.testing.assert_array_equal(at, order)


@pytest.mark.parametrize("B,W,V,num", [(1, 1, 1, 1), (1, 1, 7, 7), (2, 3, 5, 15), (1, 4, 32000, 8), (3, 2, 4096, 4), (2, 2, 4097, 5),
                                       (1, 1, 50001, 32), (2, 8, 131072, 16), (1, 40, 300, 32), (5, 1, 255, 1), (1, 7, 257, 14),
                                       (2, 5, 150000, 10), (1, 300, 5000, 32)])
@pytest.mark.parametrize("f32", [True, False])
def test_random(dev, B, W, V, num, f32):
    import torch
    g = torch.Generator(device=dev)
    g.manual_seed(V + W)
    x = torch.randn(B, W, V, generator=g, device=dev) * 2.5
    x = x if f32 else x.to(torch.bfloat16)
    scores = (-20 * np.random.default_rng(W).random((B, W))).astype(np.float32)
    _check(dev, x, scores, num, f32)


def test_all_equal_logits_take_the_lowest_indices(dev):
    import torch
    for f32 in (True, False):
        for V in (10, 9000):
            x = torch.full((2, 3, V), 1.5, device=dev, dtype=torch.float32 if f32 else torch.bfloat16)
            _, par, tok = _select(dev, x, np.zeros((2, 3), np.float32), 5)
            assert np.all(par == 0) and np.array_equal(tok, np.tile(np.arange(5), (2, 1)))


def test_logits_a_rounding_apart_share_a_score(dev):
    """Logits far below the score's rounding: every candidate has the same
    score, so the lowest indices win, wherever the larger logits are."""
    import torch
    V = 9000
    x = torch.rand(2, 2, V, generator=torch.Generator(device=dev).manual_seed(1), device=dev) * 1e-9
    got, par, tok = _select(dev, x, np.full((2, 2), -3.0, np.float32), 6)
    assert np.all(par == 0) and np.array_equal(tok, np.tile(np.arange(6), (2, 1)))
    assert np.all(got == got[0, 0])
    # two levels: 40 logits stand out by more than the rounding, the rest do not
    x2 = x.clone()
    x2[:, 1, 100:140] += 1.0
    _, par, tok = _select(dev, x2, np.full((2, 2), -3.0, np.float32), 30)
    assert np.all(par == 1) and np.array_equal(tok, np.tile(np.arange(100, 130), (2, 1)))


def test_dead_beams_and_first_step(dev):
    """Only beam 0 is alive: all winners are its; with no live beam the lowest
    indices come back at -infinity."""
    import torch
    x = torch.randn(2, 4, 5000, generator=torch.Generator(device=dev).manual_seed(2), device=dev)
    s = np.full((2, 4), -np.inf, np.float32)
    s[:, 0] = 0.0
    got, par, tok = _select(dev, x, s, 8)
    assert np.all(par == 0) and np.all(np.isfinite(got))
    s[:] = -np.inf
    got, par, tok = _select(dev, x, s, 8)
    assert np.all(got == -np.inf) and np.all(par == 0) and np.array_equal(tok, np.tile(np.arange(8), (2, 1)))


def test_masked_vocabulary(dev):
    """-infinity logits (constrained decoding): fewer open tokens than winners,
    a row with none, and rows of the lowest finite value."""
    import torch
    V = 10000
    x = torch.full((2, 2, V), float("-inf"), device=dev)
    x[0, 0, 7777], x[0, 0, 12], x[0, 1, 9999] = 1.0, 2.0, 0.5
    x[1, 1] = torch.finfo(torch.float32).min
    got, par, tok = _select(dev, x, np.zeros((2, 2), np.float32), 5)
    lse = np.log(np.exp(1.0) + np.exp(2.0))
    np.testing.assert_allclose(got[0], [0.0, 2 - lse, 1 - lse, -np.inf, -np.inf], atol=1e-5)
    assert list(zip(par[0], tok[0])) == [(1, 9999), (0, 12), (0, 7777), (0, 0), (0, 1)]
    assert np.all(par[1] == 1) and np.array_equal(tok[1], np.arange(5))


def test_nan_and_infinite_logits(dev):
    """A row with a NaN or a +infinity has no scores; the others are unhurt."""
    import torch
    x = torch.randn(1, 3, 6000, generator=torch.Generator(device=dev).manual_seed(3), device=dev)
    clean = x.clone()
    x[0, 0, 5000] = float("nan")
    x[0, 2, 17] = float("inf")
    s = np.zeros((1, 3), np.float32)
    got, par, tok = _select(dev, x, s, 6)
    want = _select(dev, clean[:, 1:2].contiguous(), s[:, :1].copy(), 6)
    assert np.all(par == 1) and np.array_equal(tok, want[2]) and np.array_equal(got, want[0])


def test_strided_rows_other_stream_and_graph(dev):
    import torch

    import bit_affine_quantized_amd as qm
    g = torch.Generator(device=dev).manual_seed(4)
    wide = torch.randn(2, 4, 33000, generator=g, device=dev).to(torch.bfloat16)
    x, s = wide[:, :, :32001], torch.randn(2, 4, generator=g, device=dev)
    want = qm.qmv_beam_select(x.contiguous(), s, 8)
    got = qm.qmv_beam_select(x, s, 8)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(qm.qmv_beam_select_workspace_bytes(2, 4, 32001, 8), dtype=torch.uint8, device=dev)
    out = tuple(torch.empty_like(t) for t in want)
    torch.cuda.synchronize()
    qm.qmv_beam_select(x, s, 8, out=out, workspace=ws, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qm.qmv_beam_select(x, s, 8, out=out, workspace=ws)
    for _ in range(3):
        for t in out:
            t.zero_()
        ws.fill_(0x55)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals(dev):
    import torch

    import bit_affine_quantized_amd as qm
    x, s = torch.zeros(1, 2, 100, device=dev), torch.zeros(1, 2, device=dev)
    for bad, what in [(dict(logits=x.half()), "bf16 or fp32"), (dict(logits=x[0]), "3 axes"), (dict(scores=s.double()), "float32"),
                      (dict(scores=s[:, :1]), "shape"), (dict(logits=x.transpose(1, 2)), "contiguous"),
                      (dict(logits=torch.zeros(2, 4, 100, device=dev)[:, :2], scores=torch.zeros(2, 2, device=dev)), "one stride")]:
        with pytest.raises(ValueError, match=what):
            qm.qmv_beam_select(**{**dict(logits=x, scores=s, num=2), **bad})
    for num in (0, 33):
        with pytest.raises(qm.QmvError, match="num="):
            qm.qmv_beam_select(x, s, num)
    with pytest.raises(qm.QmvError, match="num="):
        qm.qmv_beam_select(x[:, :, :3], s, 7)
    with pytest.raises(qm.QmvError, match="workspace"):
        qm.qmv_beam_select(x, s, 2, workspace=torch.empty(16, dtype=torch.uint8, device=dev))


def test_many_logits_above_the_bound(dev):
    """Half of every run of 512 logits far above the rest, in runs of eight: more
    candidates than one list holds, so they are taken one by one."""
    import torch
    g = torch.Generator(device=dev).manual_seed(6)
    for W, V, num, f32 in ((1, 4096, 32, True), (2, 16384, 32, True), (1, 20000, 24, False)):
        x = torch.rand(1, W, V, generator=g, device=dev)
        at = torch.arange(V, device=dev)
        x = torch.where(at // 8 % 64 < num + 1, x * 4 + 10, x)
        x = x if f32 else x.to(torch.bfloat16)
        _check(dev, x, np.zeros((1, W), np.float32), num, f32)


def test_equal_logits_that_overflow_one_list(dev):
    """A row of equal logits whose last chunk has 1105 of them: one thread's
    single logit is past the list's end, where the others' do not fit."""
    import torch
    for V in (50257, 1025, 1040, 2049, 4096 + 1105):
        for f32 in (True, False):
            x = torch.zeros(2, V, device=dev, dtype=torch.float32 if f32 else torch.bfloat16).view(1, 2, V)
            for num in (1, 32):
                got, par, tok = _select(dev, x, np.zeros((1, 2), np.float32), num)
                assert np.all(par == 0) and np.array_equal(tok[0], np.arange(num)), (V, f32, num)
                np.testing.assert_allclose(got, -np.log(V), rtol=0, atol=2.0 ** -20 * (1 + np.log(V)))


def _by_definition(x, scores, num):
    """(beams, tokens) by fp32 steps on the given fp32 logits, for rows whose
    log-sum-exp is NaN or far above the logits' differences."""
    B, W, V = x.shape
    with np.errstate(invalid="ignore"):
        m = x.max(-1, keepdims=True)
        lse = (m + np.log(np.exp((x - m).astype(np.float64)).sum(-1, keepdims=True))).astype(np.float32)
        c = scores[..., None] + (x - lse)
    c = np.where(np.isnan(c), -np.inf, c).reshape(B, W * V)
    at = np.argsort(-c, axis=-1, kind="stable")[:, :num]
    return at // V, at % V


def test_a_row_with_a_nan_among_equal_logits(dev):
    """Its log-sum-exp is NaN, so every candidate counts as -infinity and the
    lowest indices win, the NaN's own among them."""
    import torch
    for V in (40, 9000, 50257):
        for f32 in (True, False):
            for bad in (float("nan"), float("inf"), float("-inf")):
                for where in ([0], [3], list(range(0, 40, 2)), [V - 1]):
                    for W in (1, 2):                       # a second beam of nothing but NaN
                        x = torch.full((1, W, V), float("nan"), device=dev)
                        x[0, 0] = 1.5
                        x[0, 0, where] = bad
                        x = x if f32 else x.to(torch.bfloat16)
                        scores = np.array([[0.0, 5.0]], np.float32)[:, :W]
                        got, par, tok = _select(dev, x, scores, 5)
                        want = _by_definition(x.float().cpu().numpy(), scores, 5)
                        assert np.array_equal(par, want[0]) and np.array_equal(tok, want[1]), (V, f32, bad, where[0], W, tok)
                        if bad != float("-inf"):
                            assert np.all(got == -np.inf)


def test_lower_logits_that_round_to_equal_ones_scores(dev):
    """More equal logits than a list holds, and before them others a rounding
    lower: all have one score, so the lowest indices win."""
    import torch
    for V in (300, 9000):
        for f32 in (True, False):
            x = torch.full((1, 2, V), 2.0 ** -30, device=dev)
            x[0, :, :7] = 2.0 ** -31
            x[0, :, 20:25] = -2.0 ** -30
            x = x if f32 else x.to(torch.bfloat16)
            for num in (1, 4, 12):
                _, par, tok = _select(dev, x, np.full((1, 2), -1.0, np.float32), num)
                assert np.all(par == 0) and np.array_equal(tok[0], np.arange(num)), (V, f32, num, tok)


def test_ties_found_across_rows_and_past_one_sweep_step(dev):
    """Ties whose lowest indices lie late in a row, at a row's ragged end and in
    the next rows, behind winners that the lists hold."""
    import torch
    B, W, V = 1, 3, 20003
    for f32 in (True, False):
        x = torch.full((B, W, V), -30.0, device=dev)
        for w, where in ((0, [9000, 9001, 16383, 20002]), (1, [0, 7, 8, 12345]), (2, list(range(5000, 5100)))):
            x[0, w, where] = 2.0 ** -30
        x[0, 2, 100:104] = 2.0 ** -31                          # a rounding lower, the same score, left out of a full list
        x[0, 1, 20000:20002] = 1.0
        x = x if f32 else x.to(torch.bfloat16)
        # scores that bring every row's ties to one value: two rows a whole number of steps apart would not do
        lse = torch.logsumexp(x.double(), -1)
        scores = lse.float() - 8.0
        for num in (1, 2, 5, 9, 14, 30):
            _, par, tok = _select(dev, x, scores.cpu().numpy(), num)
            c = (scores.double()[..., None] + (x.double() - lse[..., None])).reshape(-1).cpu().numpy()
            c = np.round(c * 2 ** 18)                          # the ties are exact in fp32: 2^-30 is far below a step
            got = c[par[0].astype(np.int64) * V + tok[0]]
            assert np.array_equal(got, np.sort(c)[::-1][:num]) and len({*zip(par[0], tok[0])}) == num, (f32, num)


def test_few_lanes_hold_most_candidates(dev):
    """Peaked rows, fifteen strong tokens in every run of 4096: more candidates
    above the join's bound than it ranks at once."""
    import torch
    g = torch.Generator(device=dev).manual_seed(8)
    W, V = 300, 5000
    x = torch.randn(1, W, V, generator=g, device=dev) * 0.01 - 20
    for start in (0, 4096):
        x[0, :, start + 10:start + 25] = torch.rand(W, 15, generator=g, device=dev) * 0.5
    scores = (-0.25 * np.random.default_rng(3).random((1, W))).astype(np.float32)
    _check(dev, x, scores, 32, True)


def test_a_finished_item_costs_no_more_than_a_live_one(dev):
    """Scores of -infinity throughout: every candidate ties, and the lowest
    indices are found at once instead of by sweeps over all logits."""
    import torch

    import bit_affine_quantized_amd as qm
    x = torch.randn(2, 8, 131072, generator=torch.Generator(device=dev).manual_seed(9), device=dev)
    live = torch.zeros(2, 8, device=dev)
    done = live.clone()
    done[1] = float("-inf")

    def best_time(s):
        times = []
        for _ in range(12):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            out = qm.qmv_beam_select(x, s, 16)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times), out
    t0, _ = best_time(live)
    t1, (got, par, tok) = best_time(done)
    assert bool((got[1] == float("-inf")).all()) and bool((par[1] == 0).all()) and tok[1].tolist() == list(range(16))
    assert t1 < 4 * t0, (t0, t1)


def test_late_ties_in_index_order(dev):
    """One live row: two winners above, then ties from a late index on, of which
    the lowest ones are a rounding below those that the lists hold."""
    import torch
    for V, f32 in ((20003, True), (40001, False), (9000, True)):
        for W in (1, 3):
            ties = [8190, 8191, 8192, 8193] + list(range(8300, 8330)) + [V - 2, V - 1]
            x = torch.full((1, W, V), -30.0, device=dev)
            x[0, W - 1, ties] = 2.0 ** -30
            x[0, W - 1, ties[:6]] = 2.0 ** -31
            x[0, W - 1, [17, V - 5]] = torch.tensor([1.0, 2.0], device=dev)
            x = x if f32 else x.to(torch.bfloat16)
            scores = np.full((1, W), -np.inf, np.float32)
            scores[0, W - 1] = -1.0
            for num in (1, 2, 3, 5, 11, 30, 32):
                _, par, tok = _select(dev, x, scores, num)
                assert np.all(par == W - 1) and tok[0].tolist() == ([V - 5, 17] + ties)[:num], (V, f32, W, num, tok)


def test_masked_and_equal_rows_cost_no_more(dev):
    """-infinity in most of the vocabulary, or one value throughout: the ties at
    a chunk's bound do not overflow its list."""
    import torch

    import bit_affine_quantized_amd as qm
    g = torch.Generator(device=dev).manual_seed(10)
    x = (torch.randn(16, 8, 131072, generator=g, device=dev) * 2.5).to(torch.bfloat16)
    s = torch.zeros(16, 8, device=dev)
    few = torch.full_like(x, float("-inf"))
    few[:, :, 100:200] = x[:, :, 100:200]
    half = x.clone()
    half[:, :, 65536:] = float("-inf")

    def best_time(logits):
        times = []
        for _ in range(12):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            qm.qmv_beam_select(logits, s, 16)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)
    t0 = best_time(x)
    for other in (few, half, torch.zeros_like(x)):
        t = best_time(other)
        assert t < 3 * t0, (t0, t)


@pytest.mark.parametrize("V", [1, 8, 9, 100, 257, 3000, 4096, 4097, 9001])
@pytest.mark.parametrize("f32", [True, False])
def test_masked_rows_with_nan_among_them(dev, V, f32):
    """Few open tokens, -infinity and NaN in every mixture, short rows and short
    last chunks: what ties at -infinity is taken by its index, NaN's too."""
    import torch
    rng = np.random.default_rng(V)
    for kind in range(8):
        W = 2
        x = np.full((1, W, V), -np.inf, np.float32)
        if kind in (1, 4, 5, 6):                               # a few open, one exact step apart
            at = rng.permutation(V)[:max(1, min(V, 5 + kind))]
            x[0, 0, at] = np.arange(len(at), dtype=np.float32) * 0.5
        if kind in (2, 4):
            x[0, 0, rng.random(V) < 0.3] = np.nan
        if kind in (3, 5):
            x[0, 1] = np.nan
        if kind == 6:
            x[0, 1, V // 2:] = np.nan
        if kind == 7:
            x[0, :, :V - V // 8] = np.nan
        scores = np.array([[-1.0, -np.inf if kind == 6 else -2.0]], np.float32)
        t = torch.from_numpy(x).to(dev)
        t = t if f32 else t.to(torch.bfloat16)
        for num in {1, min(4, 2 * V), min(32, 2 * V)}:
            got, par, tok = _select(dev, t, scores, num)
            want = _by_definition(x, scores, num)
            assert np.array_equal(par, want[0]) and np.array_equal(tok, want[1]), (kind, num, par, tok, want)
