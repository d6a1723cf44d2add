"""Positions that all axes share: an axis stride of 0."""
import numpy as np
import pytest
import torch

from tests import _kv4 as ref
from tests.test_gpu_rope_axes import _axis, _bits, _dev, _tables, _turned, _ws

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1, 2, 77])
@pytest.mark.parametrize("axes", [2, 3, 4])
def test_one_row_of_positions_for_all_axes(uw, t, axes):
    rng = np.random.default_rng(t + axes)
    hq, hk, d = 4, 2, 128
    cos, sin = _tables(rng, 100, d // 2)
    axis, line = _axis(rng, d // 2, axes, "any"), rng.integers(0, 100, t).astype(np.int32)
    x = ref.bf16(rng.standard_normal((t, hq + hk, d)))
    want = _turned(x, np.stack([line] * axes), axis, cos, sin, False)
    xd, q, ws = _dev(x), torch.empty(t, hq, d, dtype=torch.int16, device="cuda"), _ws(uw)
    k = torch.empty(t, hk, d, dtype=torch.int16, device="cuda")
    pos = _dev(line).expand(axes, t)
    assert pos.stride(0) == 0
    uw.rope_axes(xd[:, :hq], xd[:, hq:], pos, bytes(axis.tolist()), q, k, _dev(cos), _dev(sin), ws)
    assert uw.check_status(ws) == 0
    assert np.array_equal(_bits(q), want[:, :hq]) and np.array_equal(_bits(k), want[:, hq:])
