"""uw_kv4_append_axes without a rotation, with positions and tables and without."""
import numpy as np
import pytest
import torch

from tests import _kv4 as ref
from tests.test_gpu_rope_axes import _dev, _ws

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1, 40])
@pytest.mark.parametrize("given", ["nothing", "positions", "empty tables"])
def test_append_without_a_rotation(uw, t, given):
    """rot_dim 0: q and k as they come, the cache as uw_kv4_append leaves it, positions (if there are any) not looked at."""
    rng = np.random.default_rng(t)
    hq, hk, d, page = 4, 2, 64, 16
    x = _dev(ref.bf16(rng.standard_normal((t, hq + 2 * hk, d))))
    start, length = _dev(np.array([0, t], np.int32)), _dev(np.array([t], np.int32))
    pages, got = -(-t // page), []
    pos = None if given == "nothing" else torch.full((3, t), -5, dtype=torch.int32, device="cuda")
    none = torch.empty(7, 0, device="cuda") if given == "empty tables" else None
    for axes in (False, True):
        pool = torch.zeros(pages, hk, page * (d + 8), dtype=torch.uint8, device="cuda")
        cache = uw.kv4_cache(pool, torch.arange(pages, dtype=torch.int32, device="cuda")[None], hk, d, page)
        q, k, ws = torch.zeros(t, hq, d, dtype=torch.int16, device="cuda"), None, _ws(uw)
        qkv = (x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:])
        if axes:
            k = torch.zeros(t, hk, d, dtype=torch.int16, device="cuda")
            uw.kv4_append_axes(cache, start, length, pos, b"", *qkv, q, none, none, ws, k_out=k)
            assert torch.equal(k, qkv[1])
        else:
            uw.kv4_append(cache, start, length, *qkv, q, None, None, ws)
        assert uw.check_status(ws) == 0
        got.append((q, pool))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]) and torch.equal(got[0][0], x[:, :hq])
