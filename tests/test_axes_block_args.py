"""What uw_block_norm, uw_rope_axes and uw_kv4_append_axes refuse, before any device work: checked on the CPU by calling
the C ABI with addresses that are never read, and the Python binding with tensors of the wrong shape, type, stride
or place."""
import ctypes

import pytest
import torch

OK, INVALID, SHAPE, SMALL, UNSUPPORTED = 0, 1, 2, 3, 7
P = 1 << 20      # stands for an aligned device address
NAN, INF = float("nan"), float("inf")


def _status(what, *args, **kw):
    with pytest.raises(RuntimeError) as e:
        what(*args, **kw)
    return e.value.status


def test_block_arguments(uw):
    def call(b=None, **change):
        block = dict(pw=P, g=P, gs=0, off=0.0, rs=1.0, bs=1.0, eps=1e-5)
        block.update(b or {})
        a = dict(x=P, xs=64, r=P, rs=64, h=P, hs=64, w=P, n=2, d=64, y=P, ys=64)
        a.update(change)
        blk = uw.Block(*block.values())
        status = uw.load().uw_block_norm(blk, *a.values(), None)
        assert uw.load().uw_block_norm_e4m3(blk, *a.values(), P, None) == status
        return status

    for change, want in ((dict(x=None), INVALID), (dict(r=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID),
                         (dict(n=-1), INVALID), (dict(d=0), SHAPE), (dict(d=-4), SHAPE), (dict(xs=63), INVALID),
                         (dict(rs=63), INVALID), (dict(hs=63), INVALID), (dict(ys=63), INVALID), (dict(x=P + 1), INVALID),
                         (dict(r=P + 1), INVALID), (dict(h=P + 1), INVALID), (dict(w=P + 1), INVALID),
                         (dict(n=1 << 31), UNSUPPORTED), (dict(n=1, d=1 << 31), UNSUPPORTED), (dict(n=0), OK),
                         (dict(n=0, x=None, r=None, h=None, y=None), OK)):
        assert call(**change) == want, change
    for block in (dict(pw=P + 1), dict(g=P + 1), dict(gs=-64), dict(gs=63), dict(off=NAN), dict(rs=INF), dict(bs=NAN),
                  dict(eps=-1.0), dict(eps=NAN)):
        assert call(block) == INVALID, block
    lib, blk = uw.load(), uw.Block(P, P, 0, 0.0, 1.0, 1.0, 1e-5)
    args = [P, 64, P, 64, P, 64, P, 2, 64, P, 64]
    assert lib.uw_block_norm(None, *args, None) == INVALID
    assert lib.uw_block_norm_e4m3(blk, *args, None, None) == INVALID
    assert lib.uw_block_norm_e4m3(blk, *args, P + 2, None) == INVALID
    assert lib.uw_block_norm(blk, *args[:9], P + 1, 64, None) == INVALID
    assert lib.uw_block_norm(blk, P, 64, P, 64, None, 0, None, 2, 64, None, 0, None) == INVALID   # neither h nor y
    assert lib.uw_block_norm_e4m3(blk, P, 64, P, 64, P, 64, None, 2, 64, None, 0, P, None) == INVALID


def test_block_tensors(uw):
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    y, scale = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4)
    half, other = x.half(), torch.zeros(4, 32, dtype=torch.bfloat16)
    good = dict(x=x, residual=x, weight=w, residual_out=x, y=x, post_weight=w, gate=w)
    for change, want in ((dict(x=torch.zeros(2, 2, 64, dtype=torch.bfloat16)), SHAPE), (dict(residual=half), SHAPE),
                         (dict(residual=other), SHAPE), (dict(residual_out=other), SHAPE), (dict(y=y), SHAPE),
                         (dict(y=None), INVALID), (dict(weight=None), INVALID), (dict(weight=w.half()), SHAPE),
                         (dict(weight=w[:32]), SMALL), (dict(weight=torch.zeros(128, dtype=torch.bfloat16)[::2]), SMALL),
                         (dict(post_weight=w.half()), SHAPE), (dict(post_weight=w[:63]), SMALL), (dict(gate=w.half()), SHAPE),
                         (dict(gate=w[:8]), SMALL), (dict(gate=other), SHAPE), (dict(gate=x[None]), SHAPE),
                         (dict(residual=x.t().contiguous().t()), INVALID), (dict(scale=scale), SHAPE),
                         (dict(scale=scale[:3], y=y), SMALL), (dict(scale=scale.double(), y=y), SHAPE),
                         ({}, INVALID)):      # the last: all right but for not being on the GPU
        assert _status(uw.block_norm, **{**good, **change}) == want, change


def _rows(uw, dev=P, ts=1024, hs=128):
    return uw.Kv4Rows(dev, ts, hs)


def _rope(uw, **change):
    a = dict(pos=P, stride=8, n=3, rot=128, axis=bytes([0] * 16 + [1] * 24 + [2] * 24), cos=P, sin=P, len=100, inter=0)
    a.update(change)
    return uw.Rope(*a.values())


BAD_ROPES = [(dict(pos=None), INVALID), (dict(pos=P + 2), INVALID), (dict(stride=2), INVALID), (dict(stride=-8), INVALID),
             (dict(n=0), INVALID), (dict(n=-1), INVALID), (dict(n=5), UNSUPPORTED), (dict(n=2), INVALID),
             (dict(axis=None), INVALID), (dict(axis=bytes([3] * 64)), INVALID), (dict(cos=None), INVALID),
             (dict(sin=None), INVALID), (dict(cos=P + 4), INVALID), (dict(sin=P + 8), INVALID), (dict(len=-1), INVALID),
             (dict(rot=-16), INVALID), (dict(rot=24), UNSUPPORTED), (dict(rot=144), UNSUPPORTED)]


def test_rope_arguments(uw):
    def call(rope=None, **change):
        a = dict(n=3, q=_rows(uw), hq=4, qo=_rows(uw), k=_rows(uw), hk=2, ko=_rows(uw), d=128, ws=P, size=256)
        a.update(change)
        return uw.load().uw_rope_axes(_rope(uw, **(rope or {})), *a.values(), None)

    for rope, want in BAD_ROPES + [(dict(rot=0), UNSUPPORTED)]:
        assert call(rope) == want, rope
    bad = _rows(uw, P + 2)
    for change, want in ((dict(n=-1), INVALID), (dict(n=1 << 31), UNSUPPORTED), (dict(q=None), INVALID), (dict(qo=None), INVALID),
                         (dict(hq=0), INVALID), (dict(hq=-1), INVALID), (dict(k=None), INVALID), (dict(ko=None), INVALID),
                         (dict(hk=0), INVALID), (dict(q=bad), INVALID), (dict(qo=bad), INVALID), (dict(k=bad), INVALID),
                         (dict(ko=_rows(uw, 0)), INVALID), (dict(q=_rows(uw, P, 4, 128)), INVALID),
                         (dict(q=_rows(uw, P, 1024, 60)), INVALID), (dict(k=_rows(uw, P, -1024)), INVALID),
                         (dict(d=0), SHAPE), (dict(d=132), UNSUPPORTED), (dict(d=120), UNSUPPORTED),
                         (dict(q=None, hq=0, qo=None, k=None, hk=0, ko=None), SHAPE), (dict(hq=1 << 17), UNSUPPORTED),
                         (dict(ws=None), INVALID), (dict(ws=P + 16), INVALID), (dict(size=255), SMALL), (dict(n=0), OK)):
        assert call(**change) == want, change
    assert uw.load().uw_rope_axes(None, 3, _rows(uw), 4, _rows(uw), None, 0, None, 128, P, 256, None) == INVALID


def test_append_axes_arguments(uw):
    cache = uw.Kv4CacheDesc(P, P, 10, 4, 4, 2, 2, 128, 16)

    def call(rope=None, **change):
        a = dict(start=P, len=P, n=3, r=_rope(uw, **(rope or {})), q=_rows(uw), hq=4, qo=_rows(uw), k=_rows(uw),
                 v=_rows(uw), ko=_rows(uw), ws=P, size=256)
        a.update(change)
        return uw.load().uw_kv4_append_axes(ctypes.byref(cache), *a.values(), None)

    for rope, want in BAD_ROPES:
        assert call(rope) == want, rope
    for change, want in ((dict(r=None), INVALID), (dict(start=None), INVALID), (dict(n=-1), INVALID), (dict(q=None), INVALID),
                         (dict(qo=None), INVALID), (dict(hq=0), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
                         (dict(ko=_rows(uw, P + 2)), INVALID), (dict(ko=_rows(uw, P, 4)), INVALID), (dict(ws=None), INVALID),
                         (dict(size=255), SMALL), (dict(n=0), OK), (dict(n=0, ko=None), OK)):
        assert call(**change) == want, change
    cache.head_dim = 96
    assert call() == UNSUPPORTED


def test_rope_tensors(uw):
    q, k = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    c, ws = torch.zeros(10, 32), torch.zeros(256, dtype=torch.uint8)
    good = dict(q=q, k=k, pos=torch.zeros(3, 5, dtype=torch.int32), pair_axis=bytes(32), q_out=q, k_out=k, cos=c, sin=c, ws=ws)
    assert _status(uw.rope_axes, **good) == INVALID      # not on the GPU
    for change, want in ((dict(q_out=None), INVALID), (dict(k_out=None), INVALID), (dict(q=None, k=None, q_out=None, k_out=None), SHAPE),
                         (dict(q=q[0]), SHAPE), (dict(q_out=k), SHAPE), (dict(k=k.half()), SHAPE), (dict(k_out=k[:4]), SHAPE),
                         (dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), INVALID),
                         (dict(pos=torch.zeros(3, 5)), SHAPE), (dict(pos=torch.zeros(3, 4, dtype=torch.int32)), SHAPE),
                         (dict(pos=torch.zeros(5, dtype=torch.int32)), SHAPE),
                         (dict(pos=torch.zeros(5, 3, dtype=torch.int32).t()), SHAPE), (dict(pair_axis=bytes(31)), SHAPE),
                         (dict(cos=c[:, :31]), SHAPE), (dict(sin=c.double()), SHAPE), (dict(cos=c[:9]), SHAPE),
                         (dict(cos=torch.zeros(32, 10).t(), sin=torch.zeros(32, 10).t()), INVALID)):
        assert _status(uw.rope_axes, **{**good, **change}) == want, change
    pages = torch.zeros(3, uw.kv4_page_bytes(2, 64, 16), dtype=torch.uint8)
    cache = uw.kv4_cache(pages, torch.zeros(1, 2, dtype=torch.int32), 2, 64, 16)
    more = dict(good, cache=cache, start=torch.zeros(2, dtype=torch.int32), length=torch.zeros(1, dtype=torch.int32), v=k)
    assert _status(uw.kv4_append_axes, **more) == INVALID
    for change, want in ((dict(q_out=None), INVALID), (dict(v=q), SHAPE), (dict(k_out=q), SHAPE), (dict(q=k, q_out=q), SHAPE),
                         (dict(start=torch.zeros(1, dtype=torch.int32)), SMALL), (dict(length=torch.zeros(1)), SMALL),
                         (dict(pos=torch.zeros(3, 4, dtype=torch.int32)), SHAPE), (dict(pair_axis=bytes(33)), SHAPE)):
        assert _status(uw.kv4_append_axes, **{**more, **change}) == want, change
