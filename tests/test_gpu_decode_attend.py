"""qmv_kv_attend against the float64 definition (tests/decode_ref.py, where the
tolerances are derived): row types, head layouts, page sizes, lengths, masks,
strides, and what lies in memory that no sequence uses."""
import numpy as np
import pytest

from tests import decode_ref as ref

pytestmark = pytest.mark.gpu


def _run(dev, lens, heads=2, G=4, D=128, page=16, bits=16, gs=64, layout="hnd", mask=None, weights=False, f32=True,
         scale=None, seed=0, spare=1, q_gain=1.0, max_length=None, spoil=True, tables=None, **kw):
    """One call and its check; mask: None or float32 [B|1, Hq|1, slots]."""
    import torch

    import bit_affine_quantized_amd as qm
    B = len(lens)
    if tables is None:
        tables, pages = ref.tables_for(lens, page, seed, spare)
    else:
        pages = int(tables.max()) + 1
    cache = ref.Cache(dev, pages, heads, page, D, bits, gs, layout, seed)
    if spoil:
        cache.spoil(tables, lens)
    rng = np.random.default_rng(seed + 1)
    q = ref.bf16_round(rng.standard_normal((B, heads * G, D)) * q_gain)
    sc = D ** -0.5 if scale is None else scale
    S = tables.shape[1] * page
    w = w_out = None
    if weights:
        w = torch.rand(B, heads, S, device=dev)
        w_out = torch.empty_like(w)
    out = qm.qmv_kv_attend(q.to(dev), cache.k, cache.v, torch.from_numpy(tables).to(dev),
                           torch.tensor(lens, dtype=torch.int32, device=dev), scale=scale,
                           mask=None if mask is None else torch.from_numpy(mask).to(dev), weights=w, weights_out=w_out,
                           return_lse=True, out_dtype=torch.float32 if f32 else None, max_length=max_length,
                           **cache.kw, **kw)
    torch.cuda.synchronize()
    cut = [n if max_length is None else min(n, max_length) for n in lens]
    q64 = q.double().numpy()
    ry, rl, probs = ref.attend(q64, cache.k64, cache.v64, tables, cut, page, sc, mask)
    y, lse = (t.double().cpu().numpy() for t in out)
    ref.check_attend(y, lse, ry, rl, q64, cache, sc, max(max(cut), 1), not f32,
                     f"lens={lens} heads={heads} G={G} D={D} page={page} bits={bits} gs={gs}")
    if weights:
        want = w.double().cpu().numpy()
        for b, p in enumerate(probs):
            want[b, :, :p.shape[1]] += p.reshape(heads, G, -1).sum(1)
        ds = ref.score_error(q64, cache, sc)
        np.testing.assert_allclose(w_out.double().cpu().numpy(), want, rtol=0,
                                   atol=G * (2 * ds + 2.0 ** -18 + 2.0 ** -24) + 2.0 ** -23)
    return out


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 500, 1025, 5000])
def test_lengths(dev, n):
    _run(dev, [n])


@pytest.mark.parametrize("bits,D,gs", [(16, 64, 0), (16, 128, 0), (16, 256, 0)] +
                         [(b, D, g) for b in (8, 4) for D in (64, 128, 256) for g in (32, 64, 128) if g <= D])
@pytest.mark.parametrize("G", [1, 8, 12])
def test_row_types_and_groups(dev, bits, D, gs, G):
    _run(dev, [0, 1, 77, 300], G=G, D=D, bits=bits, gs=gs or 64, weights=True, seed=D + bits + G)


@pytest.mark.parametrize("heads,G", [(1, 1), (3, 2), (1, 3), (5, 5), (2, 7), (1, 9), (2, 16), (1, 17), (1, 40)])
def test_head_layouts(dev, heads, G):
    _run(dev, [65, 3, 200], heads=heads, G=G, weights=True, seed=G)


@pytest.mark.parametrize("page", [1, 3, 7, 8, 16, 24, 32, 48, 100, 128, 1000])
@pytest.mark.parametrize("bits", [16, 8])
def test_page_sizes(dev, page, bits):
    _run(dev, [1, 95, 260, 2 * page], page=page, bits=bits, seed=page)


@pytest.mark.parametrize("layout", ["nhd", "padded"])
@pytest.mark.parametrize("bits", [16, 8, 4])
def test_layouts(dev, layout, bits):
    _run(dev, [130, 0, 41], heads=3, layout=layout, bits=bits, page=32)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("shape", ["row", "batch", "heads", "full"])
def test_masks(dev, f32, shape):
    lens, heads, G, page = [70, 33, 1, 150], 2, 4, 16
    S = (-(-150 // page) + 1) * page
    rng = np.random.default_rng(5)
    m = rng.standard_normal({"row": (1, 1, S), "batch": (4, 1, S), "heads": (1, 8, S), "full": (4, 8, S)}[shape]).astype(np.float32)
    m[rng.random(m.shape) < 0.3] = -np.inf
    m[rng.random(m.shape) < 0.1] = np.finfo(np.float32).min
    m[..., 150:] = np.nan                             # past every length: never read
    _run(dev, lens, heads=heads, G=G, mask=m, weights=True, f32=f32)


def test_mask_that_leaves_nothing(dev):
    """A row of -inf everywhere, one open slot, and the lowest value everywhere
    (which is a number: all slots then weigh the same)."""
    lens, S = [40, 40, 40], 64
    m = np.zeros((3, 1, S), np.float32)
    m[0] = -np.inf
    m[1] = -np.inf
    m[1, 0, 17] = 3.0
    m[2] = np.finfo(np.float32).min
    y, lse = _run(dev, lens, mask=m, weights=True)
    assert bool((y[0] == 0).all()) and bool((lse[0] == float("-inf")).all())


def test_nan_and_infinity_in_masked_rows(dev):
    """Rows masked for every query head of their key-value head take no part,
    whatever they hold."""
    import torch

    import bit_affine_quantized_amd as qm
    tables, pages = ref.tables_for([90], 16, 1, 1)
    rng = np.random.default_rng(2)
    for bad in (float("nan"), float("inf")):
        cache = ref.Cache(dev, pages, 2, 16, 128)
        m = np.zeros((1, 1, 112), np.float32)
        hit = rng.permutation(90)[:30]
        m[0, 0, hit] = -np.inf
        for t in hit:
            cache.k[tables[0, t // 16], :, t % 16] = bad
            cache.v[tables[0, t // 16], :, t % 16] = bad
        q = ref.bf16_round(rng.standard_normal((1, 8, 128)))
        y, lse = qm.qmv_kv_attend(q.to(dev), cache.k, cache.v, torch.from_numpy(tables).to(dev),
                                  torch.tensor([90], dtype=torch.int32, device=dev), mask=torch.from_numpy(m).to(dev),
                                  return_lse=True, out_dtype=torch.float32)
        ry, rl, _ = ref.attend(q.double().numpy(), cache.k64, cache.v64, tables, [90], 16, 128 ** -0.5, m)
        ref.check_attend(y.double().cpu().numpy(), lse.double().cpu().numpy(), ry, rl, q.double().numpy(), cache,
                         128 ** -0.5, 90, False)


def test_large_scores(dev):
    """Scores in the hundreds: the running maximum has to move."""
    _run(dev, [300, 1000, 37], q_gain=60.0, seed=3)
    _run(dev, [300], scale=-2.5, seed=4)
    _run(dev, [300], scale=0.0, seed=4)


def test_page_numbers_that_do_not_exist(dev):
    """Slots of a missing page take no part; nothing is read there."""
    tables, _ = ref.tables_for([200, 64, 100], 16, 7, 0, extra_pages=0)
    tables = tables.copy()
    pages = int(tables.max()) + 1
    tables[0, 3], tables[0, 12], tables[1, :] = -1, pages + 5, 2 ** 31 - 1
    tables[2, 0] = -2 ** 31
    cap = int(tables[tables < pages].max())
    keep = np.where(tables > cap, -7, tables)          # the same meaning, for the definition
    import torch

    import bit_affine_quantized_amd as qm
    cache = ref.Cache(dev, pages, 2, 16, 128)
    q = ref.bf16_round(np.random.default_rng(1).standard_normal((3, 8, 128)))
    lens = [200, 64, 100]
    w = torch.zeros(3, 2, 208, device=dev)
    y, lse = qm.qmv_kv_attend(q.to(dev), cache.k, cache.v, torch.from_numpy(tables).to(dev),
                              torch.tensor(lens, dtype=torch.int32, device=dev), return_lse=True, weights=w,
                              out_dtype=torch.float32)
    ry, rl, probs = ref.attend(q.double().numpy(), cache.k64, cache.v64, keep, lens, 16, 128 ** -0.5)
    ref.check_attend(y.double().cpu().numpy(), lse.double().cpu().numpy(), ry, rl, q.double().numpy(), cache,
                     128 ** -0.5, 200, False)
    for b, p in enumerate(probs):
        np.testing.assert_allclose(w[b, :, :p.shape[1]].double().cpu().numpy(), p.reshape(2, 4, -1).sum(1), atol=1e-4)


def test_lengths_out_of_range_and_max_length(dev):
    _run(dev, [100, 37, 80], max_length=64)            # cut
    _run(dev, [100, 37, 80], max_length=100, spare=40)  # a wide table
    _run(dev, [100, 37], max_length=10000)             # more than the table holds
    import torch

    import bit_affine_quantized_amd as qm
    cache = ref.Cache(dev, 3, 2, 16, 128)
    tables = np.array([[0, 1], [2, -1]], np.int32)
    q = ref.bf16_round(np.random.default_rng(1).standard_normal((2, 8, 128)))
    y = qm.qmv_kv_attend(q.to(dev), cache.k, cache.v, torch.from_numpy(tables).to(dev),
                         torch.tensor([1000, -3], dtype=torch.int32, device=dev), out_dtype=torch.float32)
    ry, rl, _ = ref.attend(q.double().numpy(), cache.k64, cache.v64, tables, [32, 0], 16, 128 ** -0.5)
    ref.check_attend(y.double().cpu().numpy(), None, ry, rl, q.double().numpy(), cache, 128 ** -0.5, 32, False)


def test_strided_q_shared_pages_and_weights_in_place(dev):
    """q as a slice of a fused projection; two sequences reading the same
    pages; weights added in place with a batch stride."""
    import torch

    import bit_affine_quantized_amd as qm
    heads, G, D, page = 2, 4, 128, 16
    cache = ref.Cache(dev, 8, heads, page, D)
    tables = np.array([[0, 1, 2, 3], [0, 1, 5, 6]], np.int32)
    lens = [60, 45]
    fused = ref.bf16_round(np.random.default_rng(3).standard_normal((2, heads * (G + 2), D))).to(dev)
    q = fused[:, :heads * G]
    big = torch.rand(2, heads, 128, device=dev)
    w = big[:, :, 32:96]
    before = big.clone()
    y = qm.qmv_kv_attend(q, cache.k, cache.v, torch.from_numpy(tables).to(dev),
                         torch.tensor(lens, dtype=torch.int32, device=dev), weights=w, out_dtype=torch.float32)
    q64 = q.double().cpu().numpy()
    ry, rl, probs = ref.attend(q64, cache.k64, cache.v64, tables, lens, page, D ** -0.5)
    ref.check_attend(y.double().cpu().numpy(), None, ry, rl, q64, cache, D ** -0.5, 60, False)
    want = before.double().cpu().numpy()
    for b, p in enumerate(probs):
        want[b, :, 32:32 + p.shape[1]] += p.reshape(heads, G, -1).sum(1)
    np.testing.assert_allclose(big.double().cpu().numpy(), want, rtol=0, atol=1e-4)


def test_offsets_past_32_bits(dev):
    """Pools over 4 GiB: the sequence lies in their last pages."""
    import torch

    import bit_affine_quantized_amd as qm
    pages, heads, page, D, n = 70001, 2, 64, 256, 150
    k = torch.empty(pages, heads, page, D, dtype=torch.bfloat16, device=dev)
    v = torch.empty_like(k)
    tail = ref.Cache(dev, 3, heads, page, D, seed=9)
    k[-3:], v[-3:] = tail.k, tail.v
    tables = np.array([[2, 0, 1]], np.int32)
    q = ref.bf16_round(np.random.default_rng(1).standard_normal((1, 8, D)))
    y = qm.qmv_kv_attend(q.to(dev), k, v, torch.from_numpy(tables + pages - 3).to(dev),
                         torch.tensor([n], dtype=torch.int32, device=dev), out_dtype=torch.float32)
    ry, rl, _ = ref.attend(q.double().numpy(), tail.k64, tail.v64, tables, [n], page, D ** -0.5)
    ref.check_attend(y.double().cpu().numpy(), None, ry, rl, q.double().numpy(), tail, D ** -0.5, n, False)


def test_other_stream_same_bits_and_graph(dev):
    """On a stream of its own, twice, and replayed from a graph: the same bits."""
    import torch

    import bit_affine_quantized_amd as qm
    lens = [777, 64, 2049]
    tables, pages = ref.tables_for(lens, 16, 1)
    cache = ref.Cache(dev, pages, 2, 16, 128)
    q = ref.bf16_round(np.random.default_rng(1).standard_normal((3, 8, 128))).to(dev)
    t, n = torch.from_numpy(tables).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    w = torch.zeros(3, 2, tables.shape[1] * 16, device=dev)
    w_out = torch.empty_like(w)
    need = qm.qmv_kv_attend_workspace_bytes(cache.k, cache.v, t, 8, weights=True)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    y = torch.empty(3, 8, 128, dtype=torch.bfloat16, device=dev)

    def call(**kw):
        qm.qmv_kv_attend(q, cache.k, cache.v, t, n, weights=w, weights_out=w_out, y=y, workspace=ws, **kw)
    call()
    torch.cuda.synchronize()
    want_y, want_w = y.clone(), w_out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y.zero_()
    torch.cuda.synchronize()
    call(stream=s)
    s.synchronize()
    assert torch.equal(y, want_y) and torch.equal(w_out, want_w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        y.zero_()
        w_out.zero_()
        ws.fill_(0x7F)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(w_out, want_w)


def test_weights_narrower_and_wider_than_the_table(dev):
    import torch

    import bit_affine_quantized_amd as qm
    cache = ref.Cache(dev, 6, 2, 16, 128)
    tables, lens = np.array([[0, 1, 2, 3, 4]], np.int32), [70]
    q = ref.bf16_round(np.random.default_rng(1).standard_normal((1, 2, 128)))
    _, _, probs = ref.attend(q.double().numpy(), cache.k64, cache.v64, tables, lens, 16, 128 ** -0.5)
    for S in (50, 70, 200):
        w = torch.ones(1, 2, S, device=dev)
        out = torch.full_like(w, 7.0)
        qm.qmv_kv_attend(q.to(dev), cache.k, cache.v, torch.from_numpy(tables).to(dev),
                         torch.tensor(lens, dtype=torch.int32, device=dev), weights=w, weights_out=out)
        want = np.ones((1, 2, S))
        want[0, :, :70] += probs[0].reshape(2, 70)[:, :S]
        np.testing.assert_allclose(out.double().cpu().numpy(), want, rtol=0, atol=1e-4)


def test_refusals(dev):
    import torch

    import bit_affine_quantized_amd as qm
    c = ref.Cache(dev, 4, 2, 16, 128)
    q = torch.zeros(1, 8, 128, dtype=torch.bfloat16, device=dev)
    t = torch.zeros(1, 4, dtype=torch.int32, device=dev)
    n = torch.ones(1, dtype=torch.int32, device=dev)
    ok = dict(q=q, k_cache=c.k, v_cache=c.v, block_tables=t, lengths=n)
    for bad, what in [
            (dict(q=q.float()), "bfloat16"), (dict(q=q[:, :7]), "multiple of 2"), (dict(q=q[:, :, :64]), "q must"),
            (dict(q=q.cpu()), "device"), (dict(lengths=n.long()), "int32"), (dict(lengths=torch.ones(2, dtype=torch.int32, device=dev)), "shape"),
            (dict(block_tables=t.long()), "int32"), (dict(block_tables=torch.zeros(2, 4, dtype=torch.int32, device=dev)), "rows"),
            (dict(v_cache=c.v[:2]), "one shape"), (dict(v_cache=c.v.transpose(1, 2).contiguous().transpose(1, 2)), "strides"),
            (dict(k_cache=(c.k,)), "both"), (dict(mask=torch.zeros(3, 1, 64, device=dev)), "does not fit"),
            (dict(mask=torch.zeros(1, 1, 64, device=dev).double()), "float32"),
            (dict(weights=torch.zeros(1, 3, 64, device=dev)), "weights must"),
            (dict(weights_out=torch.zeros(1, 2, 64, device=dev)), "goes with"),
            (dict(out_dtype=torch.float16), "out_dtype"), (dict(y=torch.zeros(1, 8, 64, device=dev, dtype=torch.bfloat16)), "shape"),
            (dict(k_cache=(t, t, t), v_cache=(t, t, t), bits=3), "bits 8 or 4")]:
        with pytest.raises(ValueError, match=what):
            qm.qmv_kv_attend(**{**ok, **bad})
    for bad, what in [
            (dict(mask=torch.zeros(1, 1, 63, device=dev)), "63 columns"), (dict(max_length=-1), "max_length"),
            (dict(workspace=torch.empty(16, dtype=torch.uint8, device=dev), weights=torch.zeros(1, 2, 64, device=dev)), "workspace"),
            (dict(q=torch.zeros(8 * 128 + 4, dtype=torch.bfloat16, device=dev)[4:].view(1, 8, 128)), "aligned")]:
        with pytest.raises(qm.QmvError, match=what):
            qm.qmv_kv_attend(**{**ok, **bad})


def test_weights_in_other_layouts(dev):
    """Heads before sequences, a head of its own, one sequence: any strides will
    do as long as no two slots are one place; shared slots are refused."""
    import torch

    import bit_affine_quantized_amd as qm
    for B, heads in ((2, 2), (1, 3), (3, 1), (1, 1)):
        lens = [40, 64, 9][:B]
        tables, pages = ref.tables_for(lens, 16, B)
        cache = ref.Cache(dev, pages, heads, 16, 128, seed=B)
        q = ref.bf16_round(np.random.default_rng(1).standard_normal((B, heads * 2, 128)))
        _, _, probs = ref.attend(q.double().numpy(), cache.k64, cache.v64, tables, lens, 16, 128 ** -0.5)
        want = np.ones((B, heads, 80))
        for b, p in enumerate(probs):
            want[b, :, :p.shape[1]] += p.reshape(heads, 2, -1).sum(1)
        call = dict(q=q.to(dev), k_cache=cache.k, v_cache=cache.v, block_tables=torch.from_numpy(tables).to(dev),
                    lengths=torch.tensor(lens, dtype=torch.int32, device=dev))
        for w in (torch.ones(heads, B, 80, device=dev).transpose(0, 1), torch.ones(B, heads + 1, 100, device=dev)[:, 1:, 20:]):
            qm.qmv_kv_attend(weights=w, **call)
            np.testing.assert_allclose(w.double().cpu().numpy(), want, rtol=0, atol=1e-4)
        if B * heads > 1:
            with pytest.raises(qm.QmvError, match="overlap"):
                qm.qmv_kv_attend(weights=torch.ones(1, 1, 80, device=dev).expand(B, heads, 80), **call)
