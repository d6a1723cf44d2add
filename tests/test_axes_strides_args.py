"""Rotation by axes: which axis strides are taken, before any device work, by calls that end before a launch (no tokens,
or more work than one takes) with addresses that are never read."""
OK, INVALID, UNSUPPORTED = 0, 1, 7
P = 1 << 20      # stands for an aligned device address
HUGE = 2 ** 31 - 1


def _rows(uw):
    return uw.Kv4Rows(P, 128, 128)


def _rope(uw, **change):
    a = dict(pos=P, stride=8, n=3, rot=128, axis=bytes([0] * 16 + [1] * 24 + [2] * 24), cos=P, sin=P, len=100, inter=0)
    a.update(change)
    return uw.Rope(*a.values())


def test_axis_strides(uw):
    def call(tokens, heads, **change):
        return uw.load().uw_rope_axes(_rope(uw, **change), tokens, _rows(uw), heads, _rows(uw), None, 0, None, 128, P, 256, None)

    assert call(0, 4, stride=0) == OK
    # all axes alike, or each behind the other: taken, and refused for the size only
    assert call(HUGE, 1 << 16, stride=0) == UNSUPPORTED and call(HUGE, 1 << 16, stride=HUGE) == UNSUPPORTED
    for stride in (1, 7, HUGE - 1, -1):
        assert call(HUGE, 1 << 16, stride=stride) == INVALID, stride
    assert call(HUGE, 1 << 16, stride=1, n=1, axis=bytes(64)) == UNSUPPORTED
