"""uw_kv4_attention at the ends of its arguments' ranges, against the same
64-bit attention and the same bounds as in test_gpu_kv4_attention.py."""
import pytest

from tests.test_gpu_kv4_attention import _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 30])
@pytest.mark.parametrize("new,lens", [([6], [2]), ([1, 6, 3], [40, 2, 0]), ([200, 9], [150, 3])])
@pytest.mark.parametrize("causal,hints", [(True, True), (True, False), (False, True)])
def test_windows_of_any_size(uw, new, lens, window, causal, hints):
    """A window as good as none, with more new tokens than the sequence holds (their first positions are negative)."""
    _run(uw, 3, 8, 2, 128, 16, new, lens, causal, window, hints=hints)


@pytest.mark.parametrize("count,hq,hk,new", [(4000, 8, 8, 1), (3000, 20, 4, 2), (2500, 8, 8, 5)])
def test_more_items_than_a_warp_lists_at_once(uw, count, hq, hk, new):
    """Many short sequences: each warp of the kernel for few rows goes through several lists of items."""
    lens = [new + (7 * i) % 37 for i in range(count)]
    _run(uw, count, hq, hk, 64, 16, [new] * count, lens)
