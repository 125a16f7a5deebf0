"""Host side of the decoder operators without a GPU: every refusal happens
before any HIP call, with its status and a message (pointers are made up)."""
from __future__ import annotations

import ctypes

import pytest

OK_PTR = 0x100000
NULL, SHAPE, ALIGN, VALUE, WORKSPACE = 1, 2, 3, 4, 6


@pytest.fixture(scope="module")
def tl():
    import ternary_weight_linear_amd as tl
    tl.lib()
    return tl


def norm(tl, **kw):
    a = dict(x=OK_PTR, xt=0, xs=256, r=OK_PTR, rs=256, ro=OK_PTR, ros=256, rt=1, w=OK_PTR, wt=0, eps=1e-6, T=3, k=256,
             q=OK_PTR, s=OK_PTR, layout=0, y=OK_PTR, ys=256)
    a.update(kw)
    return tl.lib().tern_rmsnorm(*a.values(), None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(x=None)), (NULL, dict(w=None)), (NULL, dict(q=None)), (NULL, dict(s=None)), (NULL, dict(r=None)),
    (NULL, dict(ro=None)), (NULL, dict(q=None, s=None, y=None)),
    (VALUE, dict(xt=2)), (VALUE, dict(rt=-1)), (VALUE, dict(wt=7)), (VALUE, dict(layout=2)), (VALUE, dict(eps=-1e-9)),
    (VALUE, dict(eps=float("nan"))), (VALUE, dict(eps=float("inf"))),
    (SHAPE, dict(T=0)), (SHAPE, dict(T=(1 << 19) + 1)), (SHAPE, dict(k=0)), (SHAPE, dict(k=8)), (SHAPE, dict(k=32784)),
    (SHAPE, dict(k=48, layout=1)), (SHAPE, dict(xs=255)), (SHAPE, dict(rs=0)), (SHAPE, dict(ros=128)), (SHAPE, dict(ys=-256)),
    (ALIGN, dict(x=OK_PTR + 8)), (ALIGN, dict(q=OK_PTR + 4)), (ALIGN, dict(y=OK_PTR + 2)), (ALIGN, dict(xs=258)),
    (ALIGN, dict(rs=260)), (ALIGN, dict(ys=260)), (ALIGN, dict(s=OK_PTR + 2))])
def test_rmsnorm_refuses(tl, want, kw):
    assert norm(tl, **kw) == want
    assert tl.lib().tern_last_error() != b""


def structs(tl, cache=(), batch=()):
    c = dict(k=OK_PTR, v=OK_PTR, k_scale=OK_PTR, v_scale=OK_PTR, pages=4, heads=2, dim=128)
    b = dict(q_begin=OK_PTR, kv_len=OK_PTR, page_table=OK_PTR, seqs=2, max_q=3, max_kv=128, table_width=2)
    c.update(dict(cache))
    b.update(dict(batch))
    return tl._KvCache(*c.values()), tl._KvBatch(*b.values())


BAD = [
    (NULL, dict(k=None), {}), (NULL, dict(v_scale=None), {}), (NULL, {}, dict(kv_len=None)),
    (NULL, {}, dict(page_table=None)), (SHAPE, dict(dim=96), {}), (SHAPE, dict(heads=0), {}),
    (SHAPE, dict(heads=1025), {}), (SHAPE, dict(pages=0), {}), (SHAPE, {}, dict(seqs=0)), (SHAPE, {}, dict(seqs=65536)),
    (SHAPE, {}, dict(max_q=0)), (SHAPE, {}, dict(max_kv=0)), (SHAPE, {}, dict(max_kv=129)),
    (SHAPE, {}, dict(table_width=0)), (ALIGN, dict(k=OK_PTR + 8), {}), (ALIGN, dict(k_scale=OK_PTR + 2), {}),
    (ALIGN, {}, dict(q_begin=OK_PTR + 1)),
]


@pytest.mark.parametrize("want,cache,batch", BAD)
def test_every_cache_call_checks_cache_and_batch(tl, want, cache, batch):
    L = tl.lib()
    c, b = structs(tl, cache, batch)
    assert L.tern_kv_append(c, b, 3, OK_PTR, 256, OK_PTR, 256, None, 0, 0, None, 0, None, None, None) == want
    assert L.tern_kv_read(c, b, 3, OK_PTR, OK_PTR, None) == want
    assert L.tern_kv_attn(c, b, 3, OK_PTR, 1024, 8, 1.0, 0, 0, OK_PTR, None, 0, None) == want
    assert L.tern_kv_attn_workspace_bytes(c, b, 3, 8, 0, 0) == ctypes.c_size_t(-1).value
    assert L.tern_last_error() != b""


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(k=None)), (NULL, dict(v=None)), (NULL, dict(q=None)), (NULL, dict(qo=None)), (SHAPE, dict(tokens=0)),
    (SHAPE, dict(ks=255)), (SHAPE, dict(vs=0)), (SHAPE, dict(qs=1023)), (SHAPE, dict(heads=0)), (VALUE, dict(type=2)),
    (ALIGN, dict(k=OK_PTR + 8)), (ALIGN, dict(vs=258)), (ALIGN, dict(qo=OK_PTR + 8))])
def test_append_refuses(tl, want, kw):
    a = dict(tokens=3, k=OK_PTR, ks=256, v=OK_PTR, vs=256, q=OK_PTR, qs=1024, heads=8, qo=OK_PTR, type=0)
    a.update(kw)
    c, b = structs(tl)
    assert tl.lib().tern_kv_append(c, b, *a.values(), None, None, None) == want


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(table=None)), (NULL, dict(axis=None)), (SHAPE, dict(pairs=0)), (SHAPE, dict(pairs=6)),
    (SHAPE, dict(pairs=68)), (SHAPE, dict(max_pos=0)), (SHAPE, dict(axes=0)), (SHAPE, dict(axes=256)),
    (ALIGN, dict(table=OK_PTR + 4))])
def test_append_refuses_rope(tl, want, kw):
    r = dict(table=OK_PTR, axis=OK_PTR, pairs=64, max_pos=10, axes=3)
    r.update(kw)
    c, b = structs(tl)
    got = tl.lib().tern_kv_append(c, b, 3, OK_PTR, 256, OK_PTR, 256, None, 0, 0, None, 0, tl._Rope(*r.values()), OK_PTR, None)
    assert got == want
    good = tl._Rope(OK_PTR, OK_PTR, 64, 10, 3)
    assert tl.lib().tern_kv_append(c, b, 3, OK_PTR, 256, OK_PTR, 256, None, 0, 0, None, 0, good, None, None) == NULL


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(q=None)), (NULL, dict(out=None)), (SHAPE, dict(heads=1)), (SHAPE, dict(heads=7)), (SHAPE, dict(qs=1023)),
    (VALUE, dict(scale=0.0)), (VALUE, dict(scale=-1.0)), (VALUE, dict(scale=float("nan"))),
    (VALUE, dict(scale=float("inf"))), (VALUE, dict(window=-1)), (VALUE, dict(sinks=-1)), (ALIGN, dict(q=OK_PTR + 8)),
    (ALIGN, dict(qs=1028)), (ALIGN, dict(out=OK_PTR + 4))])
def test_attention_refuses(tl, want, kw):
    a = dict(q=OK_PTR, qs=1024, heads=8, scale=1.0, window=0, sinks=0, out=OK_PTR)
    a.update(kw)
    c, b = structs(tl)
    assert tl.lib().tern_kv_attn(c, b, 3, *a.values(), None, 0, None) == want


def test_attention_workspace(tl):
    L = tl.lib()
    c, b = structs(tl, {}, dict(table_width=1 << 14, max_kv=1 << 20))
    need = L.tern_kv_attn_workspace_bytes(c, b, 3, 8, 0, 0)
    assert 0 < need < 1 << 30
    for ws, n, want in ((None, need, WORKSPACE), (OK_PTR, need - 1, WORKSPACE), (OK_PTR + 8, need, ALIGN)):
        assert L.tern_kv_attn(c, b, 3, OK_PTR, 1024, 8, 1.0, 0, 0, OK_PTR, ws, n, None) == want
    # a window that no sequence reaches is none; a short one needs few pages
    assert L.tern_kv_attn_workspace_bytes(c, b, 3, 8, 1 << 20, 0) == need
    assert L.tern_kv_attn_workspace_bytes(c, b, 3, 8, 64, 4) == 0
    assert L.tern_kv_attn_workspace_bytes(c, b, 3, 8, 2 ** 31 - 1, 2 ** 31 - 1) == need


def test_read_refuses(tl):
    c, b = structs(tl)
    L = tl.lib()
    assert L.tern_kv_read(c, b, 3, None, None, None) == NULL
    assert L.tern_kv_read(c, b, 0, OK_PTR, None, None) == SHAPE
    assert L.tern_kv_read(c, b, 3, OK_PTR + 8, None, None) == ALIGN


def test_rope_table_and_sections(tl):
    with pytest.raises(ValueError):
        tl.Rope.make(4, 8, sections=(3, 3))
    with pytest.raises(ValueError):
        tl.Rope.make(4, 8, sections=(9, -1))


def test_attention_refuses_row_counts_past_32_bits(tl):
    L = tl.lib()
    c, b = structs(tl, dict(heads=1), dict(max_q=1 << 19))
    assert L.tern_kv_attn_workspace_bytes(c, b, 3, 4096, 0, 0) == ctypes.c_size_t(-1).value
    assert b"too large" in L.tern_last_error()
