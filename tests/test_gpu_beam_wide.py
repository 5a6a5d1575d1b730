"""qmv_beam_select on batches so large that a thread of the scan takes 32 or 64
logits (tests/test_gpu_beam.py runs 16): ragged and one-logit last chunks, ties,
lists that overflow, masked and NaN rows, both types."""
import numpy as np
import pytest

from tests.test_gpu_beam import _by_definition, _check, _select

pytestmark = pytest.mark.gpu

# items x beams: at 131071 tokens 9.4 and 16.8 million logits
SIZES = [(9, 8), (16, 8)]


def _logits(dev, B, W, V, seed, f32):
    import torch
    x = torch.randn(B, W, V, generator=torch.Generator(device=dev).manual_seed(seed), device=dev) * 2.5
    return x if f32 else x.to(torch.bfloat16)


@pytest.mark.parametrize("B,W", SIZES)
@pytest.mark.parametrize("V", [131071, 131073])
@pytest.mark.parametrize("f32", [True, False])
def test_random(dev, B, W, V, f32):
    x = _logits(dev, B, W, V, V + B, f32)
    scores = (-20 * np.random.default_rng(W).random((B, W))).astype(np.float32)
    for num in (1, 16, 32):
        _check(dev, x, scores, num, f32)


@pytest.mark.parametrize("B,W", SIZES)
@pytest.mark.parametrize("f32", [True, False])
def test_ties_masks_and_nan(dev, B, W, f32):
    """One item each: equal logits; a lower value that rounds to their score; few
    open tokens; none; a NaN; NaN throughout; finished beams."""
    import torch
    V = 131073
    x = _logits(dev, B, W, V, 5, f32)
    scores = np.zeros((B, W), np.float32)
    x[0] = 1.25
    x[1] = 2.0 ** -30
    x[1, :, 3:9] = 2.0 ** -31
    x[2] = float("-inf")
    x[2, 3, [131072, 70000, 5]] = torch.tensor([3.0, 2.0, 1.0], device=dev, dtype=x.dtype)
    x[3] = float("-inf")
    x[4] = 0.5
    x[4, 0, 7] = float("nan")
    x[5] = float("nan")
    scores[6] = -np.inf
    scores[0], scores[1], scores[4] = [-np.arange(W)] * 3
    got, par, tok = _select(dev, x, scores, 32)
    for b in (0, 1, 3, 5, 6):
        assert np.all(par[b] == 0) and np.array_equal(tok[b], np.arange(32)), (b, tok[b])
    assert list(zip(par[2], tok[2]))[:5] == [(3, 131072), (3, 70000), (3, 5), (0, 0), (0, 1)]
    assert np.all(par[4] == 1) and np.array_equal(tok[4], np.arange(32))
    assert np.all(got[[3, 5, 6]] == -np.inf)
    want = _by_definition(x[4:5].float().cpu().numpy(), scores[4:5], 32)
    assert np.array_equal(want[0][0], par[4]) and np.array_equal(want[1][0], tok[4])


@pytest.mark.parametrize("B,W", SIZES)
@pytest.mark.parametrize("f32", [True, False])
def test_lists_that_overflow(dev, B, W, f32):
    """Runs of eight far above the rest, as many as winners and one in 64: more
    logits above the bound than a list holds."""
    import torch
    V = 131071
    at = torch.arange(V, device=dev)
    for num in (8, 32):
        x = torch.rand(B, W, V, generator=torch.Generator(device=dev).manual_seed(num), device=dev)
        x = torch.where(at // 8 % 64 < num + 1, x * 4 + 10, x)
        x = x if f32 else x.to(torch.bfloat16)
        _check(dev, x, np.zeros((B, W), np.float32), num, f32)
