"""uw_kv4_append_axes without a rotation: what is not looked at need not be there.  Checked before any device work, by calls
without tokens and addresses that are never read."""
import ctypes

import pytest
import torch

OK, INVALID, SHAPE = 0, 1, 2
P = 1 << 20      # stands for an aligned device address


def _rows(uw):
    return uw.Kv4Rows(P, 128, 128)


def _rope(uw, **change):
    a = dict(pos=P, stride=8, n=3, rot=128, axis=bytes([0] * 16 + [1] * 24 + [2] * 24), cos=P, sin=P, len=100, inter=0)
    a.update(change)
    return uw.Rope(*a.values())


def test_no_rotation_needs_no_positions(uw):
    cache = uw.Kv4CacheDesc(P, P, 10, 4, 4, 2, 2, 128, 16)

    def call(tokens, **change):
        return uw.load().uw_kv4_append_axes(ctypes.byref(cache), P, P, tokens, _rope(uw, **change), None, 0, None, _rows(uw),
                                            _rows(uw), None, P, 256, None)

    nothing = dict(pos=None, stride=0, n=0, axis=None, cos=None, sin=None, len=0)
    assert call(0, rot=0, **nothing) == OK
    assert call(0, **nothing) == INVALID
    for change in (dict(n=0), dict(n=9), dict(stride=-1), dict(pos=P + 1), dict(axis=None)):
        assert call(0, rot=0, **change) == OK, change
    assert uw.load().uw_rope_axes(_rope(uw, rot=0, **nothing), 0, _rows(uw), 4, _rows(uw), None, 0, None, 128, P, 256,
                                  None) == INVALID      # (nothing to do there: no tables)


def test_no_tables_in_the_binding(uw):
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    pages = torch.zeros(3, uw.kv4_page_bytes(2, 64, 16), dtype=torch.uint8)
    cache = uw.kv4_cache(pages, torch.zeros(1, 2, dtype=torch.int32), 2, 64, 16)
    good = dict(cache=cache, start=torch.zeros(2, dtype=torch.int32), length=torch.zeros(1, dtype=torch.int32), pos=None,
                pair_axis=b"", q=None, k=k, v=k, q_out=None, cos=None, sin=None, ws=torch.zeros(256, dtype=torch.uint8))
    c = torch.zeros(10, 32)
    for change, want in (({}, INVALID),       # (not on the GPU)
                         (dict(pair_axis=bytes(32)), SHAPE), (dict(cos=c, sin=c), SHAPE), (dict(cos=c[:, :0]), SHAPE),
                         (dict(pair_axis=bytes(32), cos=c, sin=c), SHAPE)):
        with pytest.raises(RuntimeError) as e:
            uw.kv4_append_axes(**{**good, **change})
        assert e.value.status == want, change
