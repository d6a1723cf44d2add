"""uw_attention around the counts of sequences at which a share's begin is found in another way (256 and 512), with empty
sequences among them and one that is much longer than the others: every sequence against 64 bits."""
import numpy as np
import pytest
import torch

from tests.test_gpu_attention import Case
from tests.test_gpu_attention_lse import check_strictly

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count", [2, 129, 200, 255, 256, 257, 400, 511, 512, 513, 1025])
@pytest.mark.parametrize("hq,hk,d,causal", [(4, 2, 64, True), (2, 1, 128, False)])
@pytest.mark.parametrize("long_at", ["first", "middle", "last"])
def test_counts_of_sequences(uw, count, hq, hk, d, causal, long_at):
    rng = np.random.default_rng(count)
    new = [int(n) for n in rng.integers(0, 5, count)]
    new[{"first": 0, "middle": count // 2, "last": count - 1}[long_at]] = 1500
    c = Case(uw, new, new, hq, hk, d, causal, seed=count)
    check_strictly(c, *c.run())


@pytest.mark.parametrize("count", [255, 300, 600])
def test_all_but_one_are_empty(uw, count):
    new = [0] * count
    new[count - 3] = 700
    c = Case(uw, new, new, 8, 2, 128, seed=count)
    check_strictly(c, *c.run())


@pytest.mark.parametrize("count", [255, 300])
def test_single_tokens_over_other_counts_of_keys(uw, count):
    rng = np.random.default_rng(count)
    kv = [int(n) for n in rng.integers(0, 300, count)]
    kv[7] = 9000
    c = Case(uw, [1] * count, kv, 8, 1, 64, seed=count)
    check_strictly(c, *c.run())
    torch.cuda.synchronize()
