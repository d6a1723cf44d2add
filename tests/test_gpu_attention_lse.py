"""uw_attention's statistics, log(sum exp(scale q.k)), against the formula in 64 bits, by comparisons that a NaN fails."""
import pytest
import torch

from tests.test_gpu_attention import Case, _reference

pytestmark = pytest.mark.gpu


def check_strictly(c, out, lse):
    """Every row of a sequence within its bound (no NaN), -inf and 0 where it sees no key."""
    o, l, o_tol, l_tol = _reference(c.q, c.k, c.v, c.new, c.kv, **c.opts)
    n = sum(c.new)
    o, l, o_tol, l_tol = o[:n], l[:n], o_tol[:n], l_tol[:n]
    assert not o.isnan().any() and not l.isnan().any()
    none = l.isneginf()
    assert (lse[:n][none] == -float("inf")).all() and (out[:n][none] == 0).all()
    assert ((out[:n].double() - o).abs() <= o_tol + 1e-38).all()
    assert ((lse[:n].double() - l).abs() <= l_tol)[~none].all()


@pytest.mark.parametrize("new,kv", [([37], [37]), ([300, 1, 0, 65], [300, 1, 0, 65]), ([1999, 301, 77], [1999, 301, 77]),
                                    ([4, 3, 200], [0, 1, 100]), ([1], [20001]), ([513], [2049])])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (3, 1, 64), (4, 4, 64)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50)])
def test_statistics(uw, new, kv, hq, hk, d, causal, window):
    c = Case(uw, new, kv, hq, hk, d, causal, window, seed=sum(kv) + d)
    check_strictly(c, *c.run())


@pytest.mark.parametrize("way", ["up", "down", "jumps", "masked"])
@pytest.mark.parametrize("d", [64, 128])
def test_statistics_with_maxima_that_move(uw, way, d):
    n = 700
    c = Case(uw, [n], [n], 4, 2, d, causal=way != "down", seed=5, spare=0)
    at = torch.arange(n, device="cuda").float()
    level = {"up": at, "down": -at, "jumps": 300.0 * ((at // 50) % 3), "masked": 3 * at}[way]
    c.q[..., 0], c.k[..., 0] = 16.0, level[:, None].bfloat16()
    c.k[..., 1:] *= 0.1
    check_strictly(c, *c.run())
