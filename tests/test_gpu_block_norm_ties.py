"""uw_block_norm with a scale that fp32 does not hold exactly but whose product with x and the gate is short in decimals:
sums that lie just between two BF16 values go to the even one, sums that are 0 come out as 0."""
import numpy as np
import pytest
import torch

from tests._kv4 import bf16, f32
from tests.test_gpu_block_norm import _bits, _dev

pytestmark = pytest.mark.gpu


def between(rng, shape):
    """x, gate, r and h with 0.22 gate x + 0.5 r between two BF16 values, h the even one.  In units of 2^-16: gate x is 2 (25 a b),
    0.22 of it 11 a b, 0.5 r a multiple of 128, and their sum an odd number S in 256 .. 511, between two even ones."""
    a, b = 2 * rng.integers(0, 5, shape) + 1, 2 * rng.integers(64, 128, shape) + 1
    z = 11 * a * b
    s = z % 128 + 128 * rng.integers(2, 4, shape)
    even = np.where((s - 1) // 2 % 2 == 0, s - 1, s + 1)
    sign = 1 - 2 * rng.integers(0, 2, shape)
    return sign * 25 * a / 2.0 ** 7, b / 2.0 ** 8, sign * 2 * (s - z) / 2.0 ** 16, sign * even / 2.0 ** 16


def nothing(rng, shape):
    """The same with a sum of 0: 0.22 x = 2.75 k."""
    k = rng.integers(1, 11, shape) * (1 - 2 * rng.integers(0, 2, shape))
    return 12.5 * k, np.ones(shape), -5.5 * k, np.zeros(shape)


def held(v):
    """BF16 bits of values that it holds."""
    bits = bf16(v)
    assert np.array_equal(f32(bits).reshape(v.shape), v)
    return bits


@pytest.mark.parametrize("n,d", [(3, 64), (40, 1000), (3, 1001), (1, 4096), (400, 4096), (3, 4097), (400, 8192), (400, 16384),
                                 (2, 16383), (2, 17000)])
@pytest.mark.parametrize("make", [between, nothing])
@pytest.mark.parametrize("e4m3", [False, True])
def test_sums_between_two_values(uw, n, d, make, e4m3):
    x, g, r, want = make(np.random.default_rng(d), (n, d))
    w, h = _dev(bf16(np.ones(d))), torch.empty(n, d, dtype=torch.int16, device="cuda")
    y = torch.empty(n, d, dtype=torch.uint8 if e4m3 else torch.int16, device="cuda")
    scale = torch.empty(n, device="cuda") if e4m3 else None
    uw.block_norm(_dev(held(x)), _dev(held(r)), w, h, y, 1e-5, gate=_dev(held(g)), residual_scale=0.5, block_scale=0.22,
                  scale=scale)
    assert np.array_equal(f32(_bits(h)).reshape(n, d), want)
    if make is nothing:
        uw.block_norm(_dev(held(x)), _dev(held(r)), w, h, y, 1e-5, residual_scale=0.5, block_scale=0.22, scale=scale)
        assert np.array_equal(f32(_bits(h)).reshape(n, d), want)
