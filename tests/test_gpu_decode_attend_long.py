"""qmv_kv_attend where a wave has many tiles and a call many sequences: chunks of
several tiles a wave, at the cap on their size and past 32 tiles a wave (where
page numbers are fetched again), and more than 64 sequences, empty ones among
them.  Many heads make the chunks long; sequences share a few pages, so the
caches are small.  Against the float64 definition, computed on the device."""
import numpy as np
import pytest

from tests import decode_ref as ref

pytestmark = pytest.mark.gpu


def _definition(q, k64, v64, tables, lens, scale, mask):
    """float64 tensors: q [B, Hq, D], pages [P, heads, page, D] -> y, lse, attention [B, heads, slots]."""
    import torch
    B, Hq, D = q.shape
    heads, page = k64.shape[1:3]
    G = Hq // heads
    y, lse = torch.zeros_like(q), torch.full((B, Hq), float("-inf"), dtype=q.dtype, device=q.device)
    got = torch.zeros(B, heads, tables.shape[1] * page, dtype=q.dtype, device=q.device)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        at = tables[b, :-(-n // page)].long()
        K, V = (x[at].transpose(0, 1).reshape(heads, -1, D)[:, :n].contiguous() for x in (k64, v64))
        s = scale * torch.matmul(q[b].view(heads, G, D), K.transpose(1, 2).contiguous())
        if mask is not None:
            s = s + mask[b, 0, :n].double()
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m.masked_fill(m == float("-inf"), 0.0))
        total = p.sum(-1, keepdim=True)
        lse[b] = (m + total.log()).view(Hq)
        p = p / total.masked_fill(total == 0, 1.0)
        y[b] = torch.matmul(p, V).view(Hq, D)
        got[b, :, :n] = p.sum(1)
    return y, lse, got


def _run(dev, lens, heads, G, D, page, bits=16, gs=64, extras=False, spare=0, seed=0):
    import torch

    import bit_affine_quantized_amd as qm
    rng = np.random.default_rng(seed)
    B, pages = len(lens), 37
    cache = ref.Cache(dev, pages, heads, page, D, bits, gs, seed=seed)
    cols = -(-max(lens) // page) + spare
    tables = rng.integers(0, pages, (B, cols)).astype(np.int32)
    for b, n in enumerate(lens):
        tables[b, -(-n // page):] = -1
    q = ref.bf16_round(rng.standard_normal((B, heads * G, D)))
    t, S = torch.from_numpy(tables).to(dev), cols * page
    mask = w = w_out = None
    if extras:
        m = rng.standard_normal((B, 1, S)).astype(np.float32)
        m[rng.random(m.shape) < 0.2] = -np.inf
        m[:, :, 300:2000] = -np.inf                    # whole tiles without a slot
        m[rng.random(m.shape) < 0.001] = np.finfo(np.float32).min
        m[B // 2] = -np.inf
        mask = torch.from_numpy(m).to(dev)
        w = torch.rand(B, heads, S, device=dev)
        w_out = torch.empty_like(w)
    y, lse = qm.qmv_kv_attend(q.to(dev), cache.k, cache.v, t, torch.tensor(lens, dtype=torch.int32, device=dev), mask=mask,
                              weights=w, weights_out=w_out, return_lse=True, out_dtype=torch.float32, **cache.kw)
    torch.cuda.synchronize()
    scale = D ** -0.5
    k64, v64 = (torch.from_numpy(x).to(dev) for x in (cache.k64, cache.v64))
    ry, rl, got = _definition(q.double().to(dev), k64, v64, t, lens, scale, mask)
    ref.check_attend(y.double().cpu().numpy(), lse.double().cpu().numpy(), ry.cpu().numpy(), rl.cpu().numpy(), q.double().numpy(),
                     cache, scale, max(lens), False)
    if extras:
        ds = ref.score_error(q.double().numpy(), cache, scale)
        np.testing.assert_allclose(w_out.double().cpu().numpy(), (w.double() + got).cpu().numpy(), rtol=0,
                                   atol=G * (2 * ds + 2.0 ** -18 + 2.0 ** -24) + 2.0 ** -23)


@pytest.mark.parametrize("heads,G,D,page,bits,gs", [(64, 1, 128, 16, 16, 64), (96, 2, 128, 64, 8, 64), (128, 1, 64, 32, 4, 32),
                                                    (32, 3, 256, 48, 16, 64), (64, 1, 256, 16, 8, 32), (64, 4, 256, 128, 4, 128),
                                                    (64, 1, 128, 24, 16, 64), (96, 1, 128, 7, 8, 128), (32, 17, 128, 16, 4, 64),
                                                    (32, 17, 128, 40, 8, 32)])
@pytest.mark.parametrize("extras", [False, True])
def test_chunks_of_many_tiles(dev, heads, G, D, page, bits, gs, extras):
    """About 8 shares: one sequence at an equal share, at the cap of 2048 slots,
    and a batch whose chunks pass 4096."""
    _run(dev, [9001], heads, G, D, page, bits, gs, extras, seed=1)
    _run(dev, [23456, 0, 5, 20001], heads, G, D, page, bits, gs, extras, spare=3, seed=2)
    if G < 8:
        _run(dev, [40000, 39999, 0, 1, 33333, 128, 40000, 40000, 4097], heads, G, D, page, bits, gs, extras, seed=3)


@pytest.mark.parametrize("B", [64, 65, 128, 129, 200])
@pytest.mark.parametrize("page,bits", [(16, 16), (24, 16), (16, 8), (7, 4)])
def test_many_sequences(dev, B, page, bits):
    rng = np.random.default_rng(B)
    lens = [int(n) for n in np.where(rng.random(B) < 0.3, 0, rng.integers(1, 3000, B))]
    lens[-1], lens[63] = 2999, 1111
    _run(dev, lens, 2, 4, 64, page, bits, 32, B % 2 == 1, seed=B)


@pytest.mark.parametrize("lens", [[0] * 70 + [1300], [1300] + [0] * 129, [0] * 200 + [1]])
def test_mostly_empty(dev, lens):
    _run(dev, lens, 4, 2, 128, 16, spare=100, extras=True, seed=7)
