"""The decode operators on another stream than the current one, without a
workspace or outputs of the caller's: what a call allocates belongs to its
stream, and work queued on the current stream right after it does not touch it."""
import numpy as np
import pytest

from tests import decode_ref as ref

pytestmark = pytest.mark.gpu


def _calls(dev):
    """name -> a call with every result it makes, of sizes that need a workspace."""
    import torch

    import bit_affine_quantized_amd as qm
    lens = [2000, 700, 1500]
    tables, pages = ref.tables_for(lens, 16, 1)
    cache = ref.Cache(dev, pages, 2, 16, 128)
    q = ref.bf16_round(np.random.default_rng(1).standard_normal((3, 8, 128))).to(dev)
    t, n = torch.from_numpy(tables).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    S = tables.shape[1] * 16
    g = torch.Generator(device=dev).manual_seed(2)
    w = torch.rand(3, 2, S, generator=g, device=dev)
    w_out = torch.empty_like(w)
    pos = torch.arange(S, dtype=torch.int32, device=dev).expand(3, 2, S).contiguous()
    logits = torch.randn(2, 4, 50000, generator=g, device=dev)
    scores = torch.zeros(2, 4, device=dev)
    beams = torch.from_numpy(np.arange(8, dtype=np.int32).reshape(2, 2, 2)).to(dev)
    spare = torch.tensor([[8, 9], [10, 11]], dtype=torch.int32, device=dev)
    parents = torch.tensor([[1, 0], [1, 1]], dtype=torch.int32, device=dev)
    fill = torch.full((2, 2), 24, dtype=torch.int32, device=dev)

    def evict(**kw):
        k, v = cache.k.clone(), cache.v.clone()
        torch.cuda.synchronize()
        return *qm.qmv_kv_evict(k, v, t, n, w, pos, n, 300, recent=20, **kw), k, v

    return {
        "attend": lambda **kw: (*qm.qmv_kv_attend(q, cache.k, cache.v, t, n, weights=w, weights_out=w_out, return_lse=True, **kw), w_out),
        "evict": evict,
        "select": lambda **kw: qm.qmv_beam_select(logits, scores, 8, **kw),
        "reorder": lambda **kw: qm.qmv_beam_reorder(cache.k, cache.v, beams, fill, parents, spare, **kw),
    }


@pytest.mark.parametrize("name", ["attend", "evict", "select", "reorder"])
def test_allocations_belong_to_the_stream(dev, name, monkeypatch):
    import torch

    from bit_affine_quantized_amd import decode
    call = _calls(dev)[name]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    had = {b["address"] for seg in torch.cuda.memory_snapshot() for b in seg["blocks"] if b["state"] == "active_allocated"}
    pointers = []

    def seen(fn, *args, real=decode._call):
        if not fn.endswith("_bytes"):
            pointers.extend(a for a in args if isinstance(a, int) and a > 1 << 32)
        return real(fn, *args)
    monkeypatch.setattr(decode, "_call", seen)
    call(stream=s)
    monkeypatch.undo()
    torch.cuda.synchronize()
    own = [p for p in pointers if p not in had and p != s.cuda_stream]
    assert own
    for p in own:
        seg = [g for g in torch.cuda.memory_snapshot() if g["address"] <= p < g["address"] + g["total_size"]]
        assert len(seg) == 1 and seg[0]["stream"] == s.cuda_stream


@pytest.mark.parametrize("name", ["attend", "evict", "select", "reorder"])
def test_work_queued_right_after_on_the_current_stream(dev, name):
    """Tensors of all small and middle sizes are taken and filled on the current
    stream while the call runs on its own."""
    import torch
    call = _calls(dev)[name]
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        got = call(stream=s)
        held = [torch.empty(1 << k, dtype=torch.uint8, device=dev).fill_(0x7F) for k in range(8, 25) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del held
