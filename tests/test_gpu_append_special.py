"""qmv_kv_append of codes against qmv_pack on the device, for groups with
infinities, NaN, denormals, the largest finite values, and zeros of both signs:
the same codes, scales and biases (NaN as any NaN)."""
import numpy as np
import pytest

from tests import decode_ref as ref

pytestmark = pytest.mark.gpu

SPECIAL = {
    "nan": [0x7FC0], "negative nan": [0xFFC0], "signalling nan": [0x7F81, 0xFF81], "inf": [0x7F80], "negative inf": [0xFF80], "both inf": [0x7F80, 0xFF80],
    "inf and nan": [0x7F80, 0x7FC0], "denormal": [0x0001, 0x007F, 0x8001], "largest": [0x7F7F], "largest and lowest": [0x7F7F, 0xFF7F],
    "lowest": [0xFF7F], "zeros": [0x0000, 0x8000], "smallest normal": [0x0080, 0x8080], "tiny": [0x33D7, 0x33D6, 0xB3D7],
}


@pytest.mark.parametrize("bits,gs", [(8, 32), (8, 64), (8, 128), (4, 32), (4, 64), (4, 128)])
@pytest.mark.parametrize("kind", list(SPECIAL))
def test_special_values(dev, bits, gs, kind):
    import torch

    import bit_affine_quantized_amd as qm
    T, heads, D, page = 96, 2, 128, 16
    rng = np.random.default_rng(len(kind))
    raw = ref.bf16_round(rng.standard_normal((T, 2 * heads, D))).view(torch.int16).numpy().view(np.uint16).copy()
    put = rng.choice(np.array(SPECIAL[kind], np.uint16), raw.shape)
    share = np.array([0.0, 0.02, 0.3, 1.0])[np.arange(T) % 4][:, None, None]    # none, few, some, all values of a token
    raw = np.where(rng.random(raw.shape) < share, put, raw)
    x = torch.from_numpy(raw.view(np.int16)).view(torch.bfloat16).to(dev)
    cache = ref.Cache(dev, 6, heads, page, D, bits, gs)
    tables = torch.arange(6, dtype=torch.int32, device=dev)[None]
    for n in (T, 5):                                                        # as a prompt, as single tokens
        qm.qmv_kv_append(x[:n, :heads], x[:n, heads:], cache.k, cache.v, tables, torch.arange(n, dtype=torch.int32, device=dev),
                         rows=torch.zeros(n, dtype=torch.int32, device=dev), **cache.kw)
        for pool, src in ((cache.k, x[:n, :heads]), (cache.v, x[:n, heads:])):
            want = qm.qmv_pack(src.float().reshape(-1, D).contiguous(), gs, bits)
            for got, w in zip(pool, want):
                got = got.transpose(1, 2).reshape(6 * page, heads, -1)[:n].reshape(n * heads, -1)
                if got.dtype == torch.bfloat16:
                    assert torch.equal(got.isnan(), w.isnan())
                    got, w = (t.masked_fill(t.isnan(), 0.0).view(torch.int16) for t in (got, w))
                assert torch.equal(got, w.view(got.dtype))
