"""Host side of the recurrent block's operators without a GPU: every refusal
happens before any HIP call, with its status and a message (pointers are made up)."""
from __future__ import annotations

import ctypes

import pytest

P = 0x100000
NULL, SHAPE, ALIGN, VALUE, WORKSPACE = 1, 2, 3, 4, 6
NONE = ctypes.c_size_t(-1).value


@pytest.fixture(scope="module")
def tl():
    import ternary_weight_linear_amd as tl
    tl.lib()
    return tl


def batch(tl, **kw):
    b = dict(begin=P, src=P, dst=P, seqs=2, max_q=3)
    b.update(kw)
    return tl._StateBatch(*b.values())


def conv(tl, b=None, **kw):
    a = dict(rows=6, x=P, type=0, xs=64, ch=64, width=4, w=P, bias=P, wt=0, silu=1, state=P, slots=2, y=2 * P, ys=64)
    a.update(kw)
    return tl.lib().tern_causal_conv(b if b is not None else batch(tl), *a.values(), None)


def scan(tl, seqs=None, **kw):
    a = dict(rows=6, heads=4, dim=64, groups=2, n=128, x=P, xs=256, b=P, bs=256, c=P, cs=256, dt=P, dtt=0, dts=4, bias=P,
             softplus=1, a=P, d=P, state=P, slots=2, y=2 * P, ws=None, wb=0)
    a.update(kw)
    return tl.lib().tern_scan(seqs if seqs is not None else batch(tl), *a.values(), None)


BAD = [(NULL, dict(begin=None)), (NULL, dict(src=None)), (NULL, dict(dst=None)), (SHAPE, dict(seqs=0)),
       (SHAPE, dict(seqs=65536)), (SHAPE, dict(max_q=0)), (SHAPE, dict(max_q=(1 << 19) + 1)), (ALIGN, dict(begin=P + 2)),
       (ALIGN, dict(src=P + 1)), (ALIGN, dict(dst=P + 2))]


@pytest.mark.parametrize("want,kw", BAD)
def test_every_state_call_checks_the_batch(tl, want, kw):
    assert conv(tl, batch(tl, **kw)) == want
    assert tl.lib().tern_last_error() != b""
    assert scan(tl, batch(tl, **kw)) == want
    assert tl.lib().tern_scan_workspace_bytes(batch(tl, **kw), 6, 4, 64, 2, 128) == NONE


def test_no_batch(tl):
    assert tl.lib().tern_causal_conv(None, 6, P, 0, 64, 64, 4, P, P, 0, 1, P, 2, P, 64, None) == NULL
    assert tl.lib().tern_scan_workspace_bytes(None, 6, 4, 64, 2, 128) == NONE


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(x=None)), (NULL, dict(w=None)), (NULL, dict(state=None)), (NULL, dict(y=None)),
    (VALUE, dict(type=2)), (VALUE, dict(wt=-1)), (VALUE, dict(y=P)), (SHAPE, dict(rows=0)), (SHAPE, dict(rows=(1 << 19) + 1)),
    (SHAPE, dict(ch=0)), (SHAPE, dict(ch=60)), (SHAPE, dict(ch=(1 << 20) + 8, xs=1 << 21, ys=1 << 21)),
    (SHAPE, dict(width=1)), (SHAPE, dict(width=5)), (SHAPE, dict(xs=63)), (SHAPE, dict(ys=0)), (SHAPE, dict(slots=0)),
    (ALIGN, dict(x=P + 8)), (ALIGN, dict(xs=66)), (ALIGN, dict(ys=68)), (ALIGN, dict(y=2 * P + 8)), (ALIGN, dict(w=P + 4)),
    (ALIGN, dict(bias=P + 8)), (ALIGN, dict(state=P + 8))])
def test_conv_refuses(tl, want, kw):
    assert conv(tl, **kw) == want
    assert tl.lib().tern_last_error() != b""


def test_conv_refuses_grids_that_one_launch_cannot_hold(tl):
    b = batch(tl, seqs=65535, max_q=1 << 19)
    assert conv(tl, b, rows=1 << 19, ch=1 << 20, xs=1 << 20, ys=1 << 20) == SHAPE


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(x=None)), (NULL, dict(b=None)), (NULL, dict(c=None)), (NULL, dict(dt=None)), (NULL, dict(a=None)),
    (NULL, dict(state=None)), (NULL, dict(y=None)), (VALUE, dict(dtt=2)), (VALUE, dict(y=P)), (SHAPE, dict(rows=0)),
    (SHAPE, dict(heads=0)), (SHAPE, dict(heads=65536)), (SHAPE, dict(groups=0)), (SHAPE, dict(groups=3)),
    (SHAPE, dict(dim=48)), (SHAPE, dict(n=32)), (SHAPE, dict(xs=255)), (SHAPE, dict(bs=255)), (SHAPE, dict(cs=0)),
    (SHAPE, dict(xs=(1 << 22) + 8)), (SHAPE, dict(bs=(1 << 22) + 8)), (SHAPE, dict(cs=(1 << 22) + 8)),
    (SHAPE, dict(dts=3)), (SHAPE, dict(slots=0)), (ALIGN, dict(x=P + 8)), (ALIGN, dict(b=P + 8)), (ALIGN, dict(cs=260)),
    (ALIGN, dict(state=P + 4)), (ALIGN, dict(y=2 * P + 2)), (ALIGN, dict(dt=P + 2)), (ALIGN, dict(bias=P + 2)),
    (ALIGN, dict(a=P + 1)), (ALIGN, dict(d=P + 2))])
def test_scan_refuses(tl, want, kw):
    assert scan(tl, **kw) == want
    assert tl.lib().tern_last_error() != b""


def test_scan_refuses_too_many_heads_for_a_launch(tl):
    b = batch(tl, seqs=65535)
    assert tl.lib().tern_scan_workspace_bytes(b, 6, 65535, 64, 1, 128) == NONE
    assert b"too large" in tl.lib().tern_last_error()


def test_scan_asks_for_its_workspace(tl):
    size = tl.lib().tern_scan_workspace_bytes
    assert size(batch(tl, max_q=8), 6, 4, 64, 2, 128) == 0
    for b, rows in ((batch(tl, max_q=9), 18), (batch(tl, seqs=1, max_q=5000), 5000)):
        need = size(b, rows, 4, 64, 2, 128)
        assert 0 < need < 1 << 30
        kw = dict(rows=rows, ws=P, wb=need)
        assert scan(tl, b, **{**kw, "ws": None}) == WORKSPACE
        assert scan(tl, b, **{**kw, "wb": need - 1}) == WORKSPACE
        assert scan(tl, b, **{**kw, "ws": P + 8}) == ALIGN
    # segments of a long prompt of few heads hold a state each
    assert size(batch(tl, seqs=1, max_q=5000), 5000, 4, 64, 2, 128) - size(batch(tl, seqs=1, max_q=32), 5000, 4, 64, 2, 128) >= 2 * 4 * 4 * 64 * 128


def gated(tl, **kw):
    a = dict(x=P, xt=1, xs=256, z=P, zt=0, zs=256, w=P, wt=0, group=64, first=1, eps=1e-6, T=3, k=256, q=P, s=P, layout=1,
             y=P, ys=256)
    a.update(kw)
    return tl.lib().tern_rmsnorm_gated(*a.values(), None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(x=None)), (NULL, dict(z=None)), (NULL, dict(w=None)), (NULL, dict(q=None)), (NULL, dict(s=None)),
    (NULL, dict(q=None, s=None, y=None)), (VALUE, dict(xt=2)), (VALUE, dict(zt=-1)), (VALUE, dict(wt=3)),
    (VALUE, dict(layout=2)), (VALUE, dict(eps=-1.0)), (VALUE, dict(eps=float("nan"))), (SHAPE, dict(T=0)),
    (SHAPE, dict(T=(1 << 19) + 1)), (SHAPE, dict(k=0)), (SHAPE, dict(k=32832, xs=40000, zs=40000, ys=40000)),
    (SHAPE, dict(group=0)), (SHAPE, dict(group=48)), (SHAPE, dict(group=192)), (SHAPE, dict(group=8, layout=0)),
    (SHAPE, dict(group=16)), (SHAPE, dict(group=-64)), (SHAPE, dict(xs=255)), (SHAPE, dict(zs=0)), (SHAPE, dict(ys=128)),
    (ALIGN, dict(x=P + 8)), (ALIGN, dict(z=P + 4)), (ALIGN, dict(w=P + 8)), (ALIGN, dict(xs=260)), (ALIGN, dict(zs=258)),
    (ALIGN, dict(q=P + 8)), (ALIGN, dict(y=P + 2)), (ALIGN, dict(ys=260)), (ALIGN, dict(s=P + 2))])
def test_gated_norm_refuses(tl, want, kw):
    assert gated(tl, **kw) == want
    assert tl.lib().tern_last_error() != b""


def post(tl, **kw):
    a = dict(x=P, xt=0, xs=256, pw=P, gate=P, gt=0, gs=0, scale=0.5, r=P, rs=256, ro=P, ros=256, rt=1, w=P, wt=0, eps=1e-6,
             T=3, k=256, q=P, s=P, layout=0, y=P, ys=256)
    a.update(kw)
    return tl.lib().tern_rmsnorm_post(*a.values(), None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(x=None)), (NULL, dict(pw=None)), (NULL, dict(r=None)), (NULL, dict(ro=None)), (NULL, dict(w=None)),
    (NULL, dict(w=None, q=None, s=None)), (NULL, dict(w=None, y=None)), (NULL, dict(q=None)), (NULL, dict(s=None)),
    (NULL, dict(q=None, s=None, y=None)), (VALUE, dict(xt=2)), (VALUE, dict(gt=5)), (VALUE, dict(rt=-1)),
    (VALUE, dict(wt=2)), (VALUE, dict(scale=float("nan"))), (VALUE, dict(scale=float("inf"))), (VALUE, dict(eps=-1.0)),
    (VALUE, dict(layout=3)), (SHAPE, dict(T=0)), (SHAPE, dict(k=24)), (SHAPE, dict(k=48, layout=1)), (SHAPE, dict(xs=0)),
    (SHAPE, dict(gs=128)), (SHAPE, dict(gs=-256)), (SHAPE, dict(rs=255)), (SHAPE, dict(ros=0)), (SHAPE, dict(ys=255)),
    (ALIGN, dict(x=P + 8)), (ALIGN, dict(pw=P + 8)), (ALIGN, dict(gate=P + 4)), (ALIGN, dict(gs=258)), (ALIGN, dict(r=P + 8)),
    (ALIGN, dict(ro=P + 8)), (ALIGN, dict(rs=260)), (ALIGN, dict(ros=260)), (ALIGN, dict(w=P + 8)), (ALIGN, dict(q=P + 8))])
def test_post_norm_refuses(tl, want, kw):
    assert post(tl, **kw) == want
    assert tl.lib().tern_last_error() != b""
