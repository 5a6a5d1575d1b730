"""How many bits of a probability reach the output.  Queries of zero make the
scores the mask, so the keys' product, whose own tolerance is wider, plays no
part.

A probability (times the row's scale, for codes) enters the values' product as two
bf16 terms: the first is the value cut to 8 bits, the rest rounded to 8.  In units
of the value's power of two that leaves an error uniform in +-2^-16 at most, root
mean square 2^-16 / sqrt(3) of the value, independent from token to token.  On
codes it multiplies the value's distance from its middle code, on bf16 rows the
value.  The rows here are centred on the middle code (or zero), so over many
outputs the error's root mean square is at most 2^-16 / sqrt(3) of the output's
own; fp32 sums, the exponential and the rounding of its argument (scores up to 32
apart: 2^-24 * 64 = 2^-18) add less than 2^-17 of it, being shared by a row's
outputs.  Held to 2^-16."""
import numpy as np
import pytest

from tests import decode_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,D,gs", [(16, 64, 0), (16, 128, 0), (16, 256, 0)] +
                         [(b, D, g) for b in (8, 4) for D in (64, 128, 256) for g in (32, 64, 128) if g <= D])
@pytest.mark.parametrize("G,page", [(1, 16), (8, 16), (12, 16), (3, 24)])
def test_root_mean_square_error(dev, bits, D, gs, G, page):
    import torch

    import bit_affine_quantized_amd as qm
    heads, lens = 2, [1999, 640, 73]
    tables, pages = ref.tables_for(lens, page, D + bits)
    cache = ref.Cache(dev, pages, heads, page, D, bits, gs or 64, seed=G + bits)
    v64 = cache.v64
    if bits != 16:                                             # centred on the middle code, moved by a little
        w, s, z = cache.v
        mid = ((1 << bits) - 1) / 2
        z = (-mid * s.float() * (1 + 0.01 * torch.randn(s.shape, generator=torch.Generator(device=dev).manual_seed(1), device=dev))).to(torch.bfloat16)
        cache.v = (w, s, z)
        v64 = cache.values(cache.v)
    S = tables.shape[1] * page
    mask = (np.random.default_rng(3).standard_normal((3, heads * G, S)) * 2).astype(np.float32)
    q = torch.zeros(3, heads * G, D, dtype=torch.bfloat16, device=dev)
    y, lse = qm.qmv_kv_attend(q, cache.k, cache.v, torch.from_numpy(tables).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev),
                              mask=torch.from_numpy(mask).to(dev), return_lse=True, out_dtype=torch.float32, **cache.kw)
    ry, rl, _ = ref.attend(q.double().cpu().numpy(), np.zeros_like(cache.k64), v64, tables, lens, page, D ** -0.5, mask)
    y = y.double().cpu().numpy()
    for b in range(3):
        err = np.sqrt(np.mean((y[b] - ry[b]) ** 2)) / np.sqrt(np.mean(ry[b] ** 2))
        print("%d bits D %d gs %d G %d length %d: %.2e" % (bits, D, gs, G, lens[b], err))
        assert err <= 2.0 ** -16, (b, err)
    np.testing.assert_allclose(lse.double().cpu().numpy(), rl, rtol=2.0 ** -22, atol=2.0 ** -18)
