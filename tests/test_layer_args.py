"""What the entry points around the matmuls refuse, before any device work:
checked on the CPU by calling the C ABI with addresses that are never read, and
the Python binding with tensors of the wrong shape, type or stride."""
import ctypes

import pytest
import torch

OK, INVALID, SHAPE, SMALL, UNSUPPORTED = 0, 1, 2, 3, 7
P = 1 << 20      # stands for an aligned device address


@pytest.fixture
def cache(uw):
    return uw.Kv4CacheDesc(P, P, 10, 4, 4, 2, 2, 128, 16)


def _rows(uw, dev=P, ts=1024, hs=128):
    return uw.Kv4Rows(dev, ts, hs)


def test_page_bytes(uw):
    assert uw.kv4_page_bytes(8, 128, 64) == 8 * 64 * 136
    assert uw.kv4_page_bytes(1, 64, 16) == 16 * 72
    n = ctypes.c_size_t()
    fn = uw.load().uw_kv4_page_bytes
    for args, want in (((0, 128, 16), SHAPE), ((1, 128, 0), SHAPE), ((1, 96, 16), UNSUPPORTED),
                       ((1, 128, 24), UNSUPPORTED), ((1, 128, 8), UNSUPPORTED), ((1, 128, 512), UNSUPPORTED)):
        assert fn(*args, ctypes.byref(n)) == want
    assert fn(1, 128, 16, None) == INVALID


def _append(uw, c, **change):
    a = dict(start=P, len=P, n=3, q=_rows(uw), hq=4, qo=_rows(uw), k=_rows(uw), v=_rows(uw), cos=P, sin=P, rope=100,
             rot=128, inter=0, ws=P, size=256)
    a.update(change)
    return uw.load().uw_kv4_append(ctypes.byref(c) if c is not None else None, *a.values(), None)


def _attention(uw, c, **change):
    a = dict(start=P, len=P, n=3, q=_rows(uw), hq=4, out=_rows(uw), lse=None, mn=1, ml=100, scale=0.0, causal=1,
             window=0, ws=P, size=1 << 40)
    a.update(change)
    return uw.load().uw_kv4_attention(ctypes.byref(c) if c is not None else None, *a.values(), None)


@pytest.mark.parametrize("field,value,want", [
    ("pages_dev", 0, INVALID), ("pages_dev", P + 8, INVALID), ("table_dev", 0, INVALID), ("table_dev", P + 2, INVALID),
    ("n_pages", -1, INVALID), ("n_pages", 1 << 40, UNSUPPORTED), ("table_stride", 3, INVALID),
    ("table_width", -1, INVALID), ("table_width", 1 << 28, INVALID), ("n_seqs", -1, INVALID), ("kv_heads", 0, SHAPE),
    ("head_dim", 96, UNSUPPORTED), ("head_dim", 0, SHAPE), ("page_size", 48, UNSUPPORTED), ("page_size", 0, SHAPE)])
def test_cache_descriptor(uw, cache, field, value, want):
    setattr(cache, field, value)
    assert _append(uw, cache) == want
    assert _attention(uw, cache) == want
    r = _rows(uw)
    assert uw.load().uw_kv4_read(ctypes.byref(cache), P, P, 3, r, r, P, 256, None) == want


def test_length_limit(uw, cache):
    cache.n_seqs, cache.table_width, cache.table_stride = 1, 1 << 28, 1 << 28
    assert _attention(uw, cache) == UNSUPPORTED       # positions past 31 bits


def test_append_arguments(uw, cache):
    bad = _rows(uw, P + 2)
    for change, want in ((dict(start=None), INVALID), (dict(len=None), INVALID), (dict(n=-1), INVALID),
                         (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(hq=0), INVALID),
                         (dict(hq=-1), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
                         (dict(k=bad), INVALID), (dict(v=_rows(uw, P, 4, 128)), INVALID),
                         (dict(q=_rows(uw, P, 1024, 60)), INVALID), (dict(qo=_rows(uw, 0)), INVALID),
                         (dict(k=_rows(uw, P, -1024)), INVALID), (dict(cos=None), INVALID), (dict(sin=None), INVALID),
                         (dict(cos=P + 2), INVALID), (dict(rope=-1), INVALID), (dict(rot=-16), INVALID),
                         (dict(rot=8), UNSUPPORTED), (dict(rot=144), UNSUPPORTED), (dict(ws=None), INVALID),
                         (dict(ws=P + 16), INVALID), (dict(size=255), SMALL), (dict(n=1 << 31), UNSUPPORTED)):
        assert _append(uw, cache, **change) == want, change
    assert _append(uw, None) == INVALID
    assert _append(uw, cache, n=0) == OK              # nothing to do
    cache.n_seqs = 0
    assert _append(uw, cache) == OK


def test_attention_arguments(uw, cache):
    for change, want in ((dict(start=None), INVALID), (dict(n=-1), INVALID), (dict(q=None), INVALID),
                         (dict(out=None), INVALID), (dict(q=_rows(uw, P + 8)), INVALID),
                         (dict(out=_rows(uw, P, 1020)), INVALID), (dict(hq=3), SHAPE), (dict(hq=0), SHAPE),
                         (dict(lse=P + 2), INVALID), (dict(mn=-1), INVALID), (dict(ml=-1), INVALID),
                         (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
                         (dict(scale=float("inf")), INVALID), (dict(window=-1), INVALID), (dict(ws=None), INVALID),
                         (dict(size=255), SMALL)):
        assert _attention(uw, cache, **change) == want, change
    n = ctypes.c_size_t()
    assert uw.load().uw_kv4_workspace_size(ctypes.byref(cache), 4, ctypes.byref(n)) == OK
    assert n.value >= 256
    if n.value > 256:
        assert _attention(uw, cache, size=n.value - 1) == SMALL
    assert uw.load().uw_kv4_workspace_size(ctypes.byref(cache), 5, ctypes.byref(n)) == SHAPE
    assert uw.load().uw_kv4_workspace_size(None, 4, ctypes.byref(n)) == INVALID
    assert _attention(uw, cache, n=0) == OK
    cache.n_seqs = 0
    assert _attention(uw, cache) == OK


def test_rmsnorm_arguments(uw):
    def call(**change):
        a = dict(x=P, xs=64, r=P, rs=64, h=P, hs=64, w=P, n=2, d=64, eps=1e-5, y=P, ys=64)
        a.update(change)
        status = uw.load().uw_rmsnorm(*a.values(), None)
        a8 = list(a.values()) + [P, None]
        assert uw.load().uw_rmsnorm_e4m3(*a8) == status
        return status

    for change, want in ((dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID),
                         (dict(r=None), INVALID), (dict(n=-1), INVALID), (dict(d=0), SHAPE), (dict(d=-4), SHAPE),
                         (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(xs=63), INVALID),
                         (dict(ys=63), INVALID), (dict(rs=63), INVALID), (dict(hs=63), INVALID),
                         (dict(x=P + 1), INVALID), (dict(w=P + 1), INVALID), (dict(n=1 << 31), UNSUPPORTED),
                         (dict(d=1 << 31, n=1), UNSUPPORTED), (dict(n=0), OK)):
        assert call(**change) == want, change
    base = [P, 64, None, 0, None, 0, P, 2, 64, 1e-5, P, 64]
    assert uw.load().uw_rmsnorm_e4m3(*base, None, None) == INVALID
    assert uw.load().uw_rmsnorm_e4m3(*base, P + 2, None) == INVALID


class _Recorder:
    def __init__(self, lib):
        self.calls, self.lib = [], lib

    def __getattr__(self, name):
        if name in ("uw_kv4_page_bytes", "uw_kv4_workspace_size"):
            return getattr(self.lib, name)

        def fn(*args):
            self.calls.append(name)
            return 0
        return fn


@pytest.fixture
def fake(uw, monkeypatch):
    rec = _Recorder(uw.load())
    monkeypatch.setattr(uw, "_lib", rec)
    return rec


def _refused(uw, status, fn, *args, **kw):
    with pytest.raises(uw.UwError) as e:
        fn(*args, **kw)
    assert e.value.status == status


def _bits(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_binding_rmsnorm(uw, fake):
    x, w, y = _bits(4, 64), _bits(64), _bits(4, 64)
    uw.rmsnorm(x, w, y, stream=0)
    uw.rmsnorm(_bits(64), w, _bits(64), stream=0)
    uw.rmsnorm(_bits(4, 80)[:, :64], w, y, residual=x, residual_out=x, stream=0)
    q, s = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4)
    uw.rmsnorm(x, w, q, scale=s, stream=0)
    assert fake.calls == ["uw_rmsnorm"] * 3 + ["uw_rmsnorm_e4m3"]
    _refused(uw, SHAPE, uw.rmsnorm, x, w, _bits(3, 64), stream=0)
    _refused(uw, SHAPE, uw.rmsnorm, x, w, q, stream=0)                        # 8-bit y without scales
    _refused(uw, SHAPE, uw.rmsnorm, x, w, y, scale=s, stream=0)               # BF16 y with scales
    _refused(uw, SHAPE, uw.rmsnorm, x.float(), w, y, stream=0)
    _refused(uw, SHAPE, uw.rmsnorm, x, w, y, residual=_bits(4, 32), stream=0)
    _refused(uw, INVALID, uw.rmsnorm, _bits(64, 4).t(), w, y, stream=0)
    _refused(uw, SMALL, uw.rmsnorm, x, _bits(63), y, stream=0)
    _refused(uw, SMALL, uw.rmsnorm, x, w, q, scale=torch.zeros(3), stream=0)
    assert len(fake.calls) == 4


def test_binding_cache(uw, fake):
    hk, d, page = 2, 64, 16
    size = uw.kv4_page_bytes(hk, d, page)
    pages, table = torch.zeros(3, size, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.int32)
    c = uw.kv4_cache(pages, table, hk, d, page)
    assert c.desc.n_pages == 3 and c.desc.n_seqs == 2 and c.desc.table_width == 4 and c.desc.table_stride == 4
    assert uw.kv4_cache(pages, table[:, :3], hk, d, page).desc.table_stride == 4
    _refused(uw, SHAPE, uw.kv4_cache, pages[:, 1:], table, hk, d, page)
    _refused(uw, SHAPE, uw.kv4_cache, pages.view(-1)[:-1], table, hk, d, page)
    _refused(uw, SHAPE, uw.kv4_cache, pages, table.long(), hk, d, page)
    _refused(uw, SHAPE, uw.kv4_cache, pages, table[0], hk, d, page)
    _refused(uw, SHAPE, uw.kv4_cache, pages, table.t().contiguous().t(), hk, d, page)
    start, length, ws = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(256)
    qkv = _bits(5, 8, d)
    q, k, v, out = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], _bits(5, 4, d)
    cos = torch.zeros(9, 32)
    uw.kv4_append(c, start, length, q, k, v, out, cos, cos, ws, stream=0)
    uw.kv4_append(c, start, length, None, k, v, None, None, None, ws, stream=0)
    uw.kv4_read(c, start, length, _bits(5, 2, d), _bits(5, 2, d), ws, stream=0)
    uw.kv4_attention(c, start, length, q, out, ws, stream=0)
    assert fake.calls == ["uw_kv4_append"] * 2 + ["uw_kv4_read", "uw_kv4_attention"]
    for status, fn, args in (
            (SMALL, uw.kv4_append, (c, start[:2], length, q, k, v, out, cos, cos, ws)),
            (SMALL, uw.kv4_append, (c, start, length[:1], q, k, v, out, cos, cos, ws)),
            (SHAPE, uw.kv4_append, (c, start, length, q, k[:4], v, out, cos, cos, ws)),
            (SHAPE, uw.kv4_append, (c, start, length, q, k.float(), v, out, cos, cos, ws)),
            (SHAPE, uw.kv4_append, (c, start, length, q, k, v, out[:, :3], cos, cos, ws)),
            (SHAPE, uw.kv4_append, (c, start, length, q, k, v, out, cos, cos[:8], ws)),
            (SHAPE, uw.kv4_append, (c, start, length, q, k, v, out, cos.bfloat16(), cos.bfloat16(), ws)),
            (INVALID, uw.kv4_append, (c, start, length, q, k, v, out, cos.t().contiguous().t(), cos, ws)),
            (INVALID, uw.kv4_append, (c, start, length, q, k, _bits(5, d, 2).transpose(1, 2), out, cos, cos, ws)),
            (SHAPE, uw.kv4_read, (c, start, length, _bits(5, 3, d), _bits(5, 2, d), ws)),
            (SHAPE, uw.kv4_attention, (c, start, length, q, _bits(4, 4, d), ws)),
            (SHAPE, uw.kv4_attention, (c, start, length, q.flatten(1), out, ws)),
            (SMALL, uw.kv4_attention, (c, start, length[:1], q, out, ws))):
        _refused(uw, status, fn, *args, stream=0)
    _refused(uw, SMALL, uw.kv4_attention, c, start, length, q, out, ws, lse=torch.zeros(19), stream=0)
    assert len(fake.calls) == 4
