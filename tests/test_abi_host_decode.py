"""C-ABI checks of the decode operators that need no GPU: bad arguments are
refused before any HIP call, and workspaces are sized as documented."""
import ctypes

import pytest

import bit_affine_quantized_amd as q
from bit_affine_quantized_amd import decode

FAKE = 0x10000   # never dereferenced: validation runs first


def cache(**kw):
    c = dict(k=FAKE, v=FAKE, ks=FAKE, kb=FAKE, vs=FAKE, vb=FAKE, pages=8, page_rows=64, head_rows=16, slot_rows=1, heads=4,
             page=16, D=128, bits=16, gs=0)
    c.update(kw)
    return decode._CACHE.pack(*c.values())


def err():
    return q.lib().qmv_last_error().decode()


BAD_CACHES = [
    (dict(k=0), q.QMV_EINVAL, "null k or v"), (dict(v=0), q.QMV_EINVAL, "null k or v"), (dict(k=FAKE + 8), q.QMV_EINVAL, "aligned"),
    (dict(bits=5), q.QMV_EINVAL, "bits=5"), (dict(D=96), q.QMV_EUNSUPPORTED, "head_dim=96"), (dict(D=0), q.QMV_EUNSUPPORTED, "head_dim=0"),
    (dict(bits=8, gs=48), q.QMV_EINVAL, "group_size=48"), (dict(bits=4, gs=128, D=64), q.QMV_EINVAL, "multiple"),
    (dict(bits=8, gs=64, ks=0), q.QMV_EINVAL, "null scales"), (dict(bits=4, gs=32, vb=FAKE + 2), q.QMV_EINVAL, "aligned"),
    (dict(pages=0), q.QMV_EINVAL, "positive"), (dict(heads=0), q.QMV_EINVAL, "positive"), (dict(page=0), q.QMV_EINVAL, "positive"),
    (dict(page=1 << 21), q.QMV_EINVAL, "page_size"), (dict(page_rows=0), q.QMV_EINVAL, "strides"), (dict(head_rows=-1), q.QMV_EINVAL, "strides"),
]


def append(c=None, **kw):
    a = dict(k=FAKE, k_t=512, k_h=128, v=FAKE, v_t=512, v_h=128, c=cache() if c is None else c, tables=FAKE, ld=4, cols=4, B=2, rows=None, slots=FAKE,
             T=2, w=None, pos=None, tp=None, mb=0, mh=0, S=0)
    a.update(kw)
    return q.lib().qmv_kv_append(*a.values(), None)


def attend(c=None, **kw):
    a = dict(q=FAKE, q_b=2048, q_h=128, c=cache() if c is None else c, tables=FAKE, ld=4, cols=4, lengths=FAKE, B=2, group=4, scale=1.0, mask=None, mb=0,
             mh=0, mcols=0, win=None, wout=None, wb=0, wh=0, S=0, y=FAKE, lse=None, most=0, out=0, ws=None, wsb=0)
    a.update(kw)
    return q.lib().qmv_kv_attend(*a.values(), None)


def evict(c=None, **kw):
    a = dict(c=cache() if c is None else c, tables=FAKE, ld=4, cols=4, lengths=FAKE, B=2, w=FAKE, pos=FAKE, mb=256, mh=64, S=64, nxt=FAKE, budget=32,
             recent=4, lo=FAKE + 64, wo=FAKE + 64, po=FAKE + 64, ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return q.lib().qmv_kv_evict(*a.values(), None)


def select(**kw):
    a = dict(x=FAKE, dt=0, ld=100, s=FAKE, B=1, W=2, V=100, num=4, os=FAKE, op=FAKE, ot=FAKE, ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return q.lib().qmv_beam_select(*a.values(), None)


def reorder(c=None, **kw):
    a = dict(c=cache() if c is None else c, tables=FAKE, lengths=FAKE, B=1, W=2, cols=4, parents=FAKE, pld=3, M=3, spare=FAKE, to=FAKE + 64, lo=FAKE + 64)
    a.update(kw)
    return q.lib().qmv_beam_reorder(*a.values(), None)


@pytest.mark.parametrize("call", [append, attend, evict, reorder])
@pytest.mark.parametrize("kw,code,msg", BAD_CACHES)
def test_bad_caches(call, kw, code, msg):
    assert call(cache(**kw)) == code and msg in err()


@pytest.mark.parametrize("call", [append, attend, evict, reorder])
def test_null_cache(call):
    assert call(c=0) == q.QMV_EINVAL and "null cache" in err()


@pytest.mark.parametrize("kw,msg", [
    (dict(tables=None), "block_tables"), (dict(B=0), "positive"), (dict(cols=0), "positive"), (dict(ld=3), "stride"), (dict(k=None), "null"),
    (dict(slots=None), "null"), (dict(T=-1), "T=-1"), (dict(k=FAKE + 8), "aligned"), (dict(v_t=12), "aligned"), (dict(w=FAKE), "S=0"),
    (dict(cols=1 << 28, ld=1 << 28), "too large")])
def test_append_refusals(kw, msg):
    assert append(**kw) == q.QMV_EINVAL and msg in err()


def test_append_of_nothing_is_fine():
    assert append(T=0, k=None, v=None, slots=None) == q.QMV_OK and err() == ""


@pytest.mark.parametrize("kw,msg", [
    (dict(q=None), "null"), (dict(lengths=None), "null"), (dict(y=None), "null"), (dict(q=FAKE + 2), "aligned"), (dict(q_h=4), "aligned"),
    (dict(out=2), "out_dtype"), (dict(group=0), "group"), (dict(group=1025), "group"), (dict(most=-1), "max_length"), (dict(B=0), "B=0"),
    (dict(win=FAKE), "go together"), (dict(win=FAKE, wout=FAKE), "S=0"), (dict(win=FAKE, wout=FAKE, S=64), "workspace"),
    (dict(win=FAKE, wout=FAKE, S=64, ws=FAKE + 4, wsb=1 << 30), "aligned"), (dict(mask=FAKE, mcols=63), "63 columns"), (dict(tables=None), "block_tables")])
def test_attend_refusals(kw, msg):
    assert attend(**kw) == q.QMV_EINVAL and msg in err()


def test_attend_of_more_than_can_be_numbered():
    assert attend(B=1 << 20, cols=1 << 16, ld=1 << 16, c=cache(page=1024)) == q.QMV_EUNSUPPORTED and "too many" in err()


@pytest.mark.parametrize("kw,msg", [
    (dict(budget=0), "budget"), (dict(recent=33), "recent"), (dict(recent=-1), "recent"), (dict(S=0), "S=0"), (dict(w=None), "null"),
    (dict(nxt=None), "null"), (dict(lo=FAKE), "outputs"), (dict(wo=FAKE), "outputs"), (dict(po=FAKE), "outputs"), (dict(wsb=16), "workspace"),
    (dict(ws=FAKE + 8), "aligned"), (dict(ws=None), "workspace")])
def test_evict_refusals(kw, msg):
    assert evict(**kw) == q.QMV_EINVAL and msg in err()


@pytest.mark.parametrize("kw,msg", [
    (dict(num=0), "num=0"), (dict(num=33), "num=33"), (dict(V=1, ld=1), "num=4"), (dict(W=0), "positive"), (dict(V=0), "positive"),
    (dict(W=5000), "too many"), (dict(W=4096, V=1 << 21, ld=1 << 21), "too many"), (dict(dt=2), "logits_dtype"), (dict(x=None), "null"),
    (dict(ot=None), "null"), (dict(ld=99), "stride"), (dict(x=FAKE + 1), "misaligned"), (dict(wsb=16), "workspace"), (dict(ws=FAKE + 8), "aligned")])
def test_select_refusals(kw, msg):
    assert select(**kw) == q.QMV_EINVAL and msg in err()


@pytest.mark.parametrize("kw,msg", [
    (dict(W=0), "positive"), (dict(M=0), "positive"), (dict(parents=None), "null"), (dict(spare=None), "null"), (dict(pld=2), "stride"),
    (dict(to=FAKE), "outputs"), (dict(lo=FAKE), "outputs"), (dict(M=1 << 21, pld=1 << 21), "too large")])
def test_reorder_refusals(kw, msg):
    assert reorder(**kw) == q.QMV_EINVAL and msg in err()


def _attend_bytes(B, cols, group, weights=0, most=0, **kw):
    out = ctypes.c_size_t(7)
    rc = q.lib().qmv_kv_attend_workspace_bytes(cache(**kw), B, cols, group, weights, most, ctypes.byref(out))
    return rc, out.value


def test_attend_workspace_sizes():
    # up to 640 slots, or 1024 from 128 heads in all on: one launch, no partial results
    assert _attend_bytes(4, 40, 4) == (q.QMV_OK, 0) and _attend_bytes(32, 64, 4) == (q.QMV_OK, 0)
    for B, cols in ((4, 41), (32, 65)):
        rc, split = _attend_bytes(B, cols, 4)
        assert rc == q.QMV_OK and split > 0
        assert _attend_bytes(B, cols, 4, most=512) == (q.QMV_OK, 0)
    rc, w = _attend_bytes(4, 64, 4, weights=1)
    assert rc == q.QMV_OK and w >= 4 * 16 * 1024 * 4                    # a score for every slot and query head
    assert _attend_bytes(0, 64, 4)[0] == q.QMV_EINVAL and _attend_bytes(1, 64, 0)[0] == q.QMV_EINVAL
    assert q.lib().qmv_kv_attend_workspace_bytes(cache(), 1, 64, 4, 0, 0, None) == q.QMV_EINVAL


def test_other_workspace_sizes():
    assert q.qmv_kv_evict_workspace_bytes(2, 4, 100, 50) >= 2 * 4 * 2 * 50 * 4
    assert q.qmv_kv_evict_workspace_bytes(2, 4, 100, 100) < q.qmv_kv_evict_workspace_bytes(2, 4, 100, 99)
    assert q.qmv_beam_select_workspace_bytes(1, 4, 32000, 8) >= 4 * 4 * 8 * 8
    for bad in (dict(B=0), dict(heads=0), dict(S=0), dict(budget=0)):
        with pytest.raises(q.QmvError):
            q.qmv_kv_evict_workspace_bytes(**{**dict(B=2, heads=4, S=100, budget=50), **bad})


@pytest.mark.parametrize("wb,wh", [(0, 64), (256, 0), (256, 63), (255, 64), (63, 128), (64, 127), (0, 0), (-255, 64), (256, -63)])
def test_attend_refuses_weights_that_overlap(wb, wh):
    size = _attend_bytes(2, 4, 4, weights=1)[1]
    assert attend(win=FAKE, wout=FAKE, S=64, wb=wb, wh=wh, ws=FAKE, wsb=size) == q.QMV_EINVAL and "overlap" in err()


def test_sizes_that_pass_64_or_32_bits_are_refused():
    out = ctypes.c_size_t(7)
    for B, heads, S, budget in ((1 << 24, 127, (1 << 31) - 65537, 1 << 30), (1 << 24, 64, 1 << 30, 1 << 29), (1 << 10, 1 << 10, (1 << 20) + 1, 5)):
        assert q.lib().qmv_kv_evict_workspace_bytes(B, heads, S, budget, ctypes.byref(out)) == q.QMV_EUNSUPPORTED and "too many" in err()
    assert q.lib().qmv_kv_evict_workspace_bytes(1 << 10, 1 << 10, 1 << 20, 5, ctypes.byref(out)) == q.QMV_OK and out.value > 0
    big = dict(page=1 << 20, cols=1 << 50, ld=1 << 50)
    for call in (append, attend):
        c = cache(page=big["page"])
        assert call(c, cols=big["cols"], ld=big["ld"]) == q.QMV_EINVAL and ("too large" in err() or "out of range" in err())
    assert _attend_bytes(1, 1 << 50, 4, page=1 << 20)[0] == q.QMV_EINVAL
    assert reorder(cache(heads=1 << 12, page=1 << 20)) == q.QMV_EUNSUPPORTED and "too many" in err()
