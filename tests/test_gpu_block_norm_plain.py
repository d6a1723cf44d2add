"""uw_block_norm without a norm after the block, a gate and scales beside uw_rmsnorm: the same h, and both y within the bound
of one formula (their sums run in different orders, so a last bit may differ)."""
import pytest
import torch

from tests.test_gpu_block_norm import Inputs, _bits, _check_y, _dev, _normed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,d", [(5, 300), (40, 1000), (3, 4096), (300, 4097), (2, 8200), (2, 17000)])
def test_plain_call_beside_the_residual_norm(uw, n, d):
    i = Inputs(n, d, False, "none", 0.0, d)
    x, r, w = _dev(i.x), _dev(i.r), _dev(i.w)
    h, y, h2, y2 = (torch.empty_like(x) for _ in range(4))
    uw.block_norm(x, r, w, h, y, 1e-5)
    uw.rmsnorm(x, w, y2, 1e-5, residual=r, residual_out=h2)
    assert torch.equal(h, h2)
    want = _normed(_bits(h), i.w, 0.0, 1e-5)
    _check_y(_bits(y), want)
    _check_y(_bits(y2), want)
    a, b = y.view(torch.bfloat16).double(), y2.view(torch.bfloat16).double()
    assert ((a - b).abs() <= b.abs() * 2.0 ** -7).all()     # a step
