"""uw_rmsnorm_e4m3 where h * weight passes fp32: such a row is NaN throughout, its scale too, and no other row is."""
import numpy as np
import pytest
import torch

from tests._kv4 import bf16

pytestmark = pytest.mark.gpu


def _dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda()


# a warp a row, a CTA a row (16-byte steps and rows that begin anywhere), value by value
@pytest.mark.parametrize("d", [64, 333, 4096, 4097, 16400])
@pytest.mark.parametrize("infinite", [False, True])
def test_products_past_fp32(uw, d, infinite):
    rng = np.random.default_rng(d)
    x = rng.standard_normal((4, d)).astype(np.float32)
    w = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32)
    x[2] *= 1e10
    x[2, d // 3] = 3e10
    w[d // 3] = np.inf if infinite else 1e30          # times 3e10: past fp32's 3.4e38
    x[3] = 0
    scale = torch.empty(4, dtype=torch.float32, device="cuda")
    q = torch.empty(4, d, dtype=torch.float8_e4m3fn, device="cuda")
    uw.rmsnorm(_dev(bf16(x)), _dev(bf16(w)), q, 1e-5, scale=scale)
    torch.cuda.synchronize()
    bad = [True] * 4 if infinite else [False, False, True, False]
    s, e = scale.cpu().numpy(), q.float().cpu().numpy()
    for i in range(4):
        assert np.isnan(s[i]) == bad[i] and np.isfinite(s[i]) != bad[i]
        assert np.isnan(e[i]).all() if bad[i] else np.isfinite(e[i]).all()
