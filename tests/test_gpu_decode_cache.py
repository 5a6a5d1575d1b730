"""qmv_kv_append, qmv_kv_evict and qmv_beam_reorder against their definitions:
what they write is compared bit for bit, and so is everything they must leave."""
import numpy as np
import pytest

import oracle
from tests import decode_ref as ref
from tests.parity import bf16_to_np_bits, u32_to_np

pytestmark = pytest.mark.gpu


def _bits(t):
    """A device tensor's memory as whole numbers, row by row."""
    import torch
    return t.detach().cpu().contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).numpy()


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("bits,D,gs", [(16, 64, 64), (16, 128, 64), (16, 256, 64), (8, 64, 32), (8, 128, 64), (8, 256, 128),
                                       (4, 64, 64), (4, 128, 32), (4, 128, 128), (4, 256, 64)])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "padded"])
def test_append(dev, bits, D, gs, layout):
    import torch

    import bit_affine_quantized_amd as qm
    heads, page, S = 3, 7, 40
    cache = ref.Cache(dev, 16, heads, page, D, bits, gs, layout, seed=bits)
    tables = np.array([[3, 1, 7, 9, 10], [0, 15, 5, 2, -1], [8, 99, 6, -1, -1]], np.int32)
    rows = np.array([0, 0, 1, 2, 2, 0, 1, 9, -1, 1, 2], np.int32)
    slots = np.array([6, 7, 0, 13, 14, 34, 27, 3, 3, -1, 8], np.int32)   # the last two: skipped; rows 9, -1 and page 99 do not exist
    T = len(rows)
    fused = ref.bf16_round(np.random.default_rng(5).standard_normal((T, 3 * heads, D)) * 3)
    fused[1, heads + 1] = 0                                # an all-zero row
    fused[2, 2 * heads:] = -fused[2, 2 * heads:].abs()     # all negative
    fused[3, 2 * heads, :gs] = 0.25
    f = fused.to(dev)
    k, v = f[:, heads:2 * heads], f[:, 2 * heads:]
    w = torch.full((3, heads, S), 5.0, device=dev)
    pos = torch.full((3, heads, S), 77, dtype=torch.int32, device=dev)
    tpos = torch.arange(1000, 1000 + T, dtype=torch.int32, device=dev)
    before = [_bits(t).copy() for t in cache.parts()]
    qm.qmv_kv_append(k, v, cache.k, cache.v, torch.from_numpy(tables).to(dev), torch.from_numpy(slots).to(dev),
                     rows=torch.from_numpy(rows).to(dev), weights=w, positions=pos, token_positions=tpos, **cache.kw)
    torch.cuda.synchronize()
    want_w, want_p = np.full((3, heads, S), 5.0), np.full((3, heads, S), 77)
    for t in range(T):
        b, s = int(rows[t]), int(slots[t])
        if s < 0 or not 0 <= b < 3:
            continue
        want_w[b, :, s], want_p[b, :, s] = 0.0, 1000 + t
        p = int(tables[b, s // page])
        if not 0 <= p < 16:
            continue
        for half, src in ((0, fused[t, heads:2 * heads]), (1, fused[t, 2 * heads:])):
            if bits == 16:
                before[half][p, :, s % page] = src.view(torch.int16).numpy()
            else:
                wq, sc, bi = oracle.quantize_pack(src.float().numpy(), gs, bits)
                base = 3 * half
                before[base][p, :, s % page] = wq.view(np.int32)
                before[base + 1][p, :, s % page] = sc.view(np.int16)
                before[base + 2][p, :, s % page] = bi.view(np.int16)
    for got, want in zip(cache.parts(), before):
        np.testing.assert_array_equal(_bits(got), want)
    np.testing.assert_array_equal(w.cpu().numpy(), want_w)
    np.testing.assert_array_equal(pos.cpu().numpy(), want_p)


def test_append_one_token_per_sequence_then_attend(dev):
    """The decode step's form: no rows, slots = lengths; the token attends to itself."""
    import torch

    import bit_affine_quantized_amd as qm
    cache = ref.Cache(dev, 4, 2, 16, 128, fill=float("nan"))
    tables = torch.tensor([[0], [1], [2]], dtype=torch.int32, device=dev)
    kv = ref.bf16_round(np.random.default_rng(0).standard_normal((3, 4, 128))).to(dev)
    n = torch.zeros(3, dtype=torch.int32, device=dev)
    qm.qmv_kv_append(kv[:, :2], kv[:, 2:], cache.k, cache.v, tables, n)
    q = ref.bf16_round(np.random.default_rng(1).standard_normal((3, 6, 128))).to(dev)
    y = qm.qmv_kv_attend(q, cache.k, cache.v, tables, n + 1)
    assert torch.equal(y.view(3, 2, 3, 128), kv[:, 2:][:, :, None].expand(3, 2, 3, 128))


def test_append_nothing_and_refusals(dev):
    import torch

    import bit_affine_quantized_amd as qm
    c = ref.Cache(dev, 4, 2, 16, 128)
    t = torch.zeros(1, 4, dtype=torch.int32, device=dev)
    kv = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device=dev)
    n = torch.zeros(1, dtype=torch.int32, device=dev)
    qm.qmv_kv_append(kv[:0], kv[:0], c.k, c.v, t, n[:0])
    for bad, what in [
            (dict(k=kv.float()), "bfloat16"), (dict(k=kv[:, :1]), "must be"), (dict(slots=n.long()), "int32"),
            (dict(slots=torch.zeros(2, dtype=torch.int32, device=dev)), "shape"),
            (dict(k=kv.expand(3, 2, 128), v=kv.expand(3, 2, 128), slots=torch.zeros(3, dtype=torch.int32, device=dev)), "give rows"),
            (dict(weights=torch.zeros(1, 3, 8, device=dev)), "weights must"),
            (dict(weights=torch.zeros(1, 2, 8, device=dev), positions=torch.zeros(1, 2, 9, dtype=torch.int32, device=dev)), "one layout")]:
        with pytest.raises(ValueError, match=what):
            qm.qmv_kv_append(**{**dict(k=kv, v=kv, k_cache=c.k, v_cache=c.v, block_tables=t, slots=n), **bad})
    odd = torch.zeros(2 * 128 + 1, dtype=torch.bfloat16, device=dev)[1:].view(1, 2, 128)
    with pytest.raises(qm.QmvError, match="aligned"):
        qm.qmv_kv_append(odd, kv, c.k, c.v, t, n)


# ------------------------------------------------------------------ evict
def _evict_case(dev, lens, budget, recent, heads=2, D=128, page=16, bits=16, gs=64, layout="hnd", seed=0, S=None,
                weights=None, positions=None, spoil_table=False):
    import torch

    import bit_affine_quantized_amd as qm
    rng = np.random.default_rng(seed)
    tables, pages = ref.tables_for(lens, page, seed, 1)
    if spoil_table:
        tables = tables.copy()
        tables[0, 1] = -1
    cache = ref.Cache(dev, pages, heads, page, D, bits, gs, layout, seed)
    B, S = len(lens), S or max(max(lens), 1)
    w = rng.random((B, heads, S)).astype(np.float32) ** 6 if weights is None else weights
    pos = np.stack([[rng.permutation(S) for _ in range(heads)] for _ in range(B)]).astype(np.int32) if positions is None else positions
    nxt = np.array(lens, np.int32)
    before = [_bits(t).copy() for t in cache.parts()]
    got = qm.qmv_kv_evict(cache.k, cache.v, torch.from_numpy(tables).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev),
                          torch.from_numpy(w).to(dev), torch.from_numpy(pos).to(dev), torch.from_numpy(nxt).to(dev), budget,
                          recent=recent, **cache.kw)
    torch.cuda.synchronize()
    want_w, want_p = w.copy(), pos.copy()
    cap = tables.shape[1] * page
    for i, (new, moves) in enumerate(ref.evict(lens, w, pos, nxt, budget, recent, cap)):
        b, h = divmod(i, heads)
        for s, d in moves:
            ps, pd = tables[b, s // page], tables[b, d // page]
            if 0 <= ps < pages and 0 <= pd < pages:
                for t in before:
                    t[pd, h, d % page] = t[ps, h, s % page]
            want_w[b, h, d], want_p[b, h, d] = w[b, h, s], pos[b, h, s]
        want_w[b, h, new:], want_p[b, h, new:] = 0.0, -1
    np.testing.assert_array_equal(got[0].cpu().numpy(), [max(0, min(n, S, cap, budget)) for n in lens])
    np.testing.assert_array_equal(got[1].cpu().numpy().view(np.int32), want_w.view(np.int32))
    np.testing.assert_array_equal(got[2].cpu().numpy(), want_p)
    for t, x in zip(cache.parts(), before):
        np.testing.assert_array_equal(_bits(t), x)


@pytest.mark.parametrize("lens,budget,recent", [
    ([1], 1, 0), ([2], 1, 1), ([0, 5, 64], 5, 2), ([65, 64, 63, 200], 64, 16), ([1000, 3], 999, 0), ([1500], 1, 0),
    ([1025, 1024, 2049], 100, 100), ([3000], 2900, 64), ([5000], 313, 17), ([9000, 4096], 4097, 1000), ([20000], 700, 0),
    ([33000, 70], 32768, 5)])
def test_evict(dev, lens, budget, recent):
    _evict_case(dev, lens, budget, recent)


@pytest.mark.parametrize("bits,D,gs,page,layout", [(8, 128, 64, 16, "nhd"), (4, 64, 32, 24, "hnd"), (4, 256, 128, 7, "padded"),
                                                   (16, 64, 64, 1, "padded"), (16, 256, 64, 64, "nhd")])
def test_evict_row_types(dev, bits, D, gs, page, layout):
    _evict_case(dev, [150, 90, 10], 60, 10, heads=3, D=D, page=page, bits=bits, gs=gs, layout=layout)


@pytest.mark.parametrize("kind", ["equal", "zero", "few", "nan", "inf", "signed"])
@pytest.mark.parametrize("n", [300, 2500])
def test_evict_ties_and_odd_weights(dev, kind, n):
    rng = np.random.default_rng(1)
    w = rng.random((1, 2, n)).astype(np.float32)
    if kind == "equal":
        w[:] = 0.125
    elif kind == "zero":
        w[:] = np.where(rng.random(w.shape) < 0.5, 0.0, -0.0)
    elif kind == "few":
        w = rng.integers(0, 3, w.shape).astype(np.float32)
    elif kind == "nan":
        w[rng.random(w.shape) < 0.1] = np.nan
        w[:, :, ::7] = -np.nan
    elif kind == "inf":
        w[rng.random(w.shape) < 0.1] = np.inf
        w[rng.random(w.shape) < 0.3] = -np.inf
    else:
        w = rng.standard_normal(w.shape).astype(np.float32)
    _evict_case(dev, [n], n // 3, 20, weights=w)


def test_evict_more_protected_than_the_budget_and_short_bookkeeping(dev):
    """Positions that repeat protect more entries than fit: the lowest slots
    stay.  Bookkeeping narrower than the length: slots past it do not count."""
    _evict_case(dev, [100], 20, 20, positions=np.full((1, 2, 100), 99, np.int32))
    _evict_case(dev, [100, 50], 20, 5, S=60)
    _evict_case(dev, [100, 50], 20, 5, S=400)
    _evict_case(dev, [100, 50], 20, 5, spoil_table=True)


def test_evict_refusals(dev):
    import torch

    import bit_affine_quantized_amd as qm
    c = ref.Cache(dev, 4, 2, 16, 128)
    n = torch.ones(1, dtype=torch.int32, device=dev)
    ok = dict(k_cache=c.k, v_cache=c.v, block_tables=torch.zeros(1, 4, dtype=torch.int32, device=dev), lengths=n,
              weights=torch.zeros(1, 2, 64, device=dev), positions=torch.zeros(1, 2, 64, dtype=torch.int32, device=dev),
              next_positions=n, budget=8)
    for bad, what in [(dict(positions=torch.zeros(1, 2, 64, device=dev)), "int32"), (dict(lengths=n.long()), "int32"),
                      (dict(weights=torch.zeros(1, 3, 64, device=dev)), "must be"),
                      (dict(positions=torch.zeros(1, 2, 128, dtype=torch.int32, device=dev)[:, :, :64]), "one layout")]:
        with pytest.raises(ValueError, match=what):
            qm.qmv_kv_evict(**{**ok, **bad})
    for bad, what in [(dict(budget=0), "budget"), (dict(recent=9), "recent"), (dict(recent=-1), "recent"),
                      (dict(out=(n, torch.empty(1, 2, 64, device=dev), torch.empty(1, 2, 64, dtype=torch.int32, device=dev))), "outputs"),
                      (dict(workspace=torch.empty(16, dtype=torch.uint8, device=dev)), "workspace")]:
        with pytest.raises(qm.QmvError, match=what):
            qm.qmv_kv_evict(**{**ok, **bad})


# ------------------------------------------------------------------ reorder
@pytest.mark.parametrize("bits,page,n,layout", [(16, 16, 37, "hnd"), (16, 16, 48, "nhd"), (8, 7, 20, "padded"), (4, 24, 5, "hnd"),
                                                (16, 1, 3, "hnd"), (16, 128, 300, "hnd")])
def test_reorder(dev, bits, page, n, layout):
    import torch

    import bit_affine_quantized_amd as qm
    B, W, M, heads, D = 2, 3, 4, 3, 128
    cols = n // page + 2
    pages = B * W * cols + B * M
    cache = ref.Cache(dev, pages, heads, page, D, bits, 64, layout)
    rng = np.random.default_rng(n)
    order = rng.permutation(pages).astype(np.int32)
    tables, spare = order[:B * W * cols].reshape(B, W, cols), order[B * W * cols:].reshape(B, M)
    lens = np.full((B, W), n, np.int32)
    lens[1] = [0, max(0, n - 1), n]
    parents = np.array([[2, 0, 0, 1, 9], [1, 5, -1, 0, 9]], np.int32)   # 5 and -1 do not exist
    before = [_bits(t).copy() for t in cache.parts()]
    t2, n2 = qm.qmv_beam_reorder(cache.k, cache.v, torch.from_numpy(tables).to(dev), torch.from_numpy(lens).to(dev),
                                 torch.from_numpy(parents).to(dev)[:, :M], torch.from_numpy(spare).to(dev), **cache.kw)
    torch.cuda.synchronize()
    want_t, want_n = np.full((B, M, cols), -1, np.int32), np.zeros((B, M), np.int32)
    for b in range(B):
        for i in range(M):
            p = parents[b, i]
            k = int(lens[b, p]) if 0 <= p < W else 0
            full, tail = divmod(k, page)
            if 0 <= p < W:
                want_t[b, i, :full] = tables[b, p, :full]
                for t in before:
                    t[spare[b, i], :, :tail] = t[tables[b, p, full], :, :tail]
            want_t[b, i, full] = spare[b, i]
            want_n[b, i] = k
    np.testing.assert_array_equal(t2.cpu().numpy(), want_t)
    np.testing.assert_array_equal(n2.cpu().numpy(), want_n)
    for t, x in zip(cache.parts(), before):
        np.testing.assert_array_equal(_bits(t), x)


def test_reorder_full_table_and_bad_pages(dev):
    """A parent that fills its table leaves no column for the free page; page
    numbers that do not exist copy nothing."""
    import torch

    import bit_affine_quantized_amd as qm
    cache = ref.Cache(dev, 6, 2, 4, 64)
    tables = torch.tensor([[[0, 1], [2, 77]]], dtype=torch.int32, device=dev)
    lens = torch.tensor([[8, 6]], dtype=torch.int32, device=dev)
    before = [_bits(t).copy() for t in cache.parts()]
    t2, n2 = qm.qmv_beam_reorder(cache.k, cache.v, tables, lens, torch.tensor([[0, 1]], dtype=torch.int32, device=dev),
                                 torch.tensor([[4, 5]], dtype=torch.int32, device=dev))
    assert t2.tolist() == [[[0, 1], [2, 5]]] and n2.tolist() == [[8, 6]]
    for t, x in zip(cache.parts(), before):
        np.testing.assert_array_equal(_bits(t), x)


def test_reorder_refusals(dev):
    import torch

    import bit_affine_quantized_amd as qm
    c = ref.Cache(dev, 4, 2, 16, 128)
    z = torch.zeros(1, 2, dtype=torch.int32, device=dev)
    ok = dict(k_cache=c.k, v_cache=c.v, block_tables=torch.zeros(1, 2, 4, dtype=torch.int32, device=dev), lengths=z,
              parents=z, spare_pages=z)
    for bad, what in [(dict(parents=z.long()), "int32"), (dict(spare_pages=z[:, :1]), "shape"), (dict(lengths=z[:, :1]), "shape"),
                      (dict(block_tables=torch.zeros(1, 4, dtype=torch.int32, device=dev)), "3 axes")]:
        with pytest.raises(ValueError, match=what):
            qm.qmv_beam_reorder(**{**ok, **bad})
    with pytest.raises(qm.QmvError, match="outputs"):
        qm.qmv_beam_reorder(**ok, out=(ok["block_tables"], torch.zeros_like(z)))


@pytest.mark.parametrize("bits,gs", [(8, 32), (8, 64), (8, 128), (4, 32), (4, 64), (4, 128)])
def test_append_codes_equal_the_quantizer_in_bulk(dev, bits, gs):
    """Tens of thousands of groups, quotients on exact halves among them, equal
    the packing oracle's bits; odd token counts end inside a line of 16."""
    import torch

    import bit_affine_quantized_amd as qm
    T, heads, D, page = 1003, 4, 128, 64
    rng = np.random.default_rng(bits + gs)
    new = rng.standard_normal((T, 2 * heads, D)).astype(np.float32) * np.exp(rng.standard_normal((T, 2 * heads, 1))).astype(np.float32)
    top = (1 << bits) - 1
    half = rng.integers(0, min(top, 127), (T // 4, 2 * heads, D)) + 0.5           # with ends 0 and `top` the scale is one
    half[..., ::gs], half[..., 1::gs] = 0.0, top
    new[::4][:T // 4] = half * np.exp2(rng.integers(-20, 20, (T // 4, 2 * heads, 1)))
    new[5::16] *= np.float32(1e-6)
    x = ref.bf16_round(new)
    tables = rng.permutation(17)[None, :16].astype(np.int32)
    cache = ref.Cache(dev, 17, heads, page, D, bits, gs)
    xd = x.to(dev)
    qm.qmv_kv_append(xd[:, :heads], xd[:, heads:], cache.k, cache.v, torch.from_numpy(tables).to(dev),
                     torch.arange(T, dtype=torch.int32, device=dev), rows=torch.zeros(T, dtype=torch.int32, device=dev), **cache.kw)
    at = torch.from_numpy(tables[0].astype(np.int64)).to(dev)
    for pool, src in ((cache.k, x[:, :heads]), (cache.v, x[:, heads:])):
        wq, sc, bi = oracle.quantize_pack(src.float().numpy().reshape(T * heads, D), gs, bits)
        for t, want in zip(pool, (wq.view(np.int32), sc.view(np.int16), bi.view(np.int16))):
            got = _bits(t[at].transpose(1, 2).reshape(16 * page, heads, -1)[:T])
            np.testing.assert_array_equal(got.reshape(T * heads, -1), want)


def _groups_near_halves(bits, gs):
    """bf16 patterns [n, gs]: every pair of a largest value in [1, 2) and a
    smallest one up to 200 steps below it, with the values between them whose
    quotients come closest to a half."""
    top = np.float32((1 << bits) - 1)
    value = lambda p: (p.astype(np.uint32) << 16).view(np.float32)  # noqa: E731
    out = []
    for hi in range(0x3F80, 0x4000):
        lo = np.arange(hi - 200, hi)
        h, low = value(np.full(200, hi)), value(lo)
        s = -((h - low) / top)
        s = h / np.trunc(h / s - np.float32(0.5))                         # rounded away from zero, as it is negative
        x = np.arange(hi - 200, hi + 1)
        q = ((value(x) - h[0])[None] / s[:, None]).astype(np.float64)
        far = np.where(x[None] >= lo[:, None], np.abs(q - np.floor(q) - 0.5), 9.0)
        take = np.argsort(far, 1, kind="stable")[:, :gs - 2]
        pick = np.where(np.take_along_axis(far, take, 1) < 1.0, x[take], hi)
        out.append(np.concatenate([np.full((200, 1), hi), lo[:, None], pick], 1))
    return np.concatenate(out).astype(np.uint16)


@pytest.mark.parametrize("bits,gs", [(8, 32), (8, 64), (8, 128), (4, 32), (4, 64), (4, 128)])
def test_append_codes_of_groups_without_a_zero(dev, bits, gs):
    """Groups whose values all lie above zero (or all below), one to 200 bf16
    steps apart: the bias is many times the range away.  Among their quotients
    are those closest to a half, where a code changes."""
    import torch

    import bit_affine_quantized_amd as qm
    heads, D, page = 4, 128, 64
    groups = _groups_near_halves(bits, gs)
    T = len(groups) * gs // (2 * heads * D)
    rng = np.random.default_rng(bits + gs)
    groups = groups[rng.permutation(len(groups))[:T * 2 * heads * D // gs]]
    groups = np.where(rng.random((len(groups), 1)) < 0.1, groups ^ 0x8000, groups)
    x = torch.from_numpy(groups.astype(np.uint16).view(np.int16).reshape(T, 2 * heads, D)).view(torch.bfloat16)
    pages = -(-T // page)
    tables = rng.permutation(pages + 1)[None, :pages].astype(np.int32)
    cache = ref.Cache(dev, pages + 1, heads, page, D, bits, gs)
    xd = x.to(dev)
    qm.qmv_kv_append(xd[:, :heads], xd[:, heads:], cache.k, cache.v, torch.from_numpy(tables).to(dev),
                     torch.arange(T, dtype=torch.int32, device=dev), rows=torch.zeros(T, dtype=torch.int32, device=dev), **cache.kw)
    at = torch.from_numpy(tables[0].astype(np.int64)).to(dev)
    for pool, src in ((cache.k, x[:, :heads]), (cache.v, x[:, heads:])):
        wq, sc, bi = oracle.quantize_pack(src.float().numpy().reshape(T * heads, D), gs, bits)
        for t, want in zip(pool, (wq.view(np.int32), sc.view(np.int16), bi.view(np.int16))):
            got = _bits(t[at].transpose(1, 2).reshape(pages * page, heads, -1)[:T])
            np.testing.assert_array_equal(got.reshape(T * heads, -1), want)


def test_bookkeeping_of_one_sequence_or_one_head(dev):
    """An axis of size one may have any stride: weights and positions of one
    sequence made in different ways have one layout."""
    import torch

    import bit_affine_quantized_amd as qm
    for B, heads in ((1, 2), (2, 1), (1, 1)):
        S, n = 64, 48
        cache = ref.Cache(dev, 4 * B, heads, 16, 128)
        tables = torch.arange(4 * B, dtype=torch.int32, device=dev).view(B, 4)
        lengths = torch.full((B,), n, dtype=torch.int32, device=dev)
        w = torch.rand(B, heads, S, device=dev)
        pos = torch.arange(S, dtype=torch.int32, device=dev).expand(B, heads, S).contiguous()
        want = [t.clone() for t in qm.qmv_kv_evict(cache.k.clone(), cache.v.clone(), tables, lengths, w, pos, lengths, 20, recent=4)]
        odd_w = torch.empty_strided((B, heads, S), (9999 if B == 1 else heads * S, 7777 if heads == 1 else S, 1), device=dev).copy_(w)
        odd_p = pos
        assert odd_w.stride() != odd_p.stride()
        got = qm.qmv_kv_evict(cache.k.clone(), cache.v.clone(), tables, lengths, odd_w, odd_p, lengths, 20, recent=4)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        kv = ref.bf16_round(np.random.default_rng(0).standard_normal((B, 2 * heads, 128))).to(dev)
        qm.qmv_kv_append(kv[:, :heads], kv[:, heads:], cache.k, cache.v, tables, lengths, weights=odd_w, positions=odd_p,
                         token_positions=lengths + 100)
        assert bool((odd_w[:, :, n] == 0).all()) and bool((odd_p[:, :, n] == n + 100).all())
        q = ref.bf16_round(np.random.default_rng(1).standard_normal((B, heads, 128))).to(dev)
        out = torch.empty(B, heads, S, device=dev)
        qm.qmv_kv_attend(q, cache.k, cache.v, tables, lengths + 1, weights=odd_w, weights_out=out)
        assert bool(((out - odd_w).sum(-1) - 1).abs().max() < 1e-3)


def test_evict_bookkeeping_of_the_most_slots(dev):
    """Bookkeeping as wide as is accepted (8.6 GB an array): what lies past the
    new length is cleared up to the last slot."""
    import torch

    import bit_affine_quantized_amd as qm
    S, n = 2 ** 31 - 1 - 65536, 100
    cache = ref.Cache(dev, 8, 1, 16, 128)
    tables = torch.arange(8, dtype=torch.int32, device=dev)[None]
    lengths = torch.tensor([n], dtype=torch.int32, device=dev)
    w = torch.ones(1, 1, S, device=dev)
    pos = torch.ones(1, 1, S, dtype=torch.int32, device=dev)
    got = qm.qmv_kv_evict(cache.k, cache.v, tables, lengths, w, pos, lengths, 60)
    assert int(got[0]) == 60
    assert bool((got[1][..., :60] == 1).all()) and bool((got[2][..., :60] == 1).all())
    for t, want in ((got[1], 0), (got[2], -1)):
        for a in range(0, S, 1 << 28):
            part = t[0, 0, max(a, 60):min(S, a + (1 << 28))]
            assert int(part.min()) == want and int(part.max()) == want
    del w, pos, got, t, part
    torch.cuda.empty_cache()
