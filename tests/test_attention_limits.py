"""uw_attention: the largest calls that it takes, before any device work."""
import pytest

SMALL, UNSUPPORTED = 3, 7
P = 1 << 20      # stands for an aligned device address


@pytest.mark.parametrize("group", [1, 7, 256])
def test_rows_of_a_kv_head(uw, group):
    """The last 256 numbers below 2^31 are no row numbers: a tile's threads count past its rows."""
    def call(n):
        r = uw.Kv4Rows(P, 64, 64)
        # (a workspace of no bytes: what is not refused for its rows is refused for that)
        return uw.load().uw_attention(P, P, 1, n, 5, r, group, r, r, 1, 64, r, None, 0.0, 1, 0, P, 0, None)

    most = (2 ** 31 - 1 - 256) // group
    assert call(most) == SMALL and call(most + 1) == UNSUPPORTED and call((2 ** 31 - 1) // group) == UNSUPPORTED
