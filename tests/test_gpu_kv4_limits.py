"""uw_kv4_attention at the ends of its arguments' ranges, against the same
64-bit attention and the same bounds as in test_gpu_kv4_attention.py."""
import numpy as np
import pytest
import torch

from tests import _kv4 as ref
from tests.test_gpu_kv4_attention import _cache, _dev, _run

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


@pytest.mark.parametrize("new,page,short", [(1, 16, 0), (1, 16, 5), (3, 64, 0), (200, 16, 0), (200, 256, 9)])
@pytest.mark.parametrize("causal", [True, False])
def test_positions_up_to_31_bits(uw, new, page, short, causal):
    """A sequence that ends at the last position its table can name: the same as its last keys alone, the
    window leaving out all others (whose page numbers are none)."""
    hq, hk, d, window = 4, 2, 64, 40
    held = 512                                        # keys whose pages are there
    width = (2 ** 31 - 1) // page
    length = width * page - short
    rng = np.random.default_rng(new + page)
    pages, few = _cache(rng, hk, d, page, [held - short])
    qb = ref.bf16(rng.standard_normal((new, hq, d)))
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, width - few.shape[1]:] = _dev(few[0])
    cache = uw.kv4_cache(_dev(pages.bytes), table, hk, d, page)
    ws = torch.empty(uw.kv4_workspace_size(cache, hq), dtype=torch.uint8, device="cuda")
    uw.workspace_init(ws)
    start, ln = _dev(np.array([0, new], np.int32)), _dev(np.array([length], np.int32))
    q, lse = _dev(qb), torch.empty(new, hq, device="cuda")
    out = torch.empty_like(q)
    uw.kv4_attention(cache, start, ln, q, out, ws, new, length, causal=causal, window=window, lse=lse)
    k = torch.empty(new, hk, d, dtype=torch.int16, device="cuda")
    v = torch.empty_like(k)
    uw.kv4_read(cache, start, ln, k, v, ws)
    assert uw.check_status(ws) == 0
    o_ref, lse_ref, bound = ref.attention(ref.f32(qb).reshape(qb.shape), pages, few, [new], [held - short], hk, causal,
                                          window, d ** -0.5)
    o = ref.f32(out.cpu().numpy().view(np.uint16)).reshape(qb.shape)
    assert np.all(np.abs(o - o_ref) <= 2.0 ** -8 * np.abs(o_ref) + 1.1 * 2.0 ** -8 * bound + 1e-30)
    assert np.all(np.abs(lse.cpu().numpy() - lse_ref) <= 2.0 ** -10)
    for which, got in ((0, k), (1, v)):
        for h in range(hk):
            want = ref.bf16(ref.value(*pages.get(which, few[0], held - short, h)))[-new:]
            assert np.array_equal(got[:, h].cpu().numpy().view(np.uint16), want)


@pytest.mark.parametrize("new,count,hq,hk,d", [([20, 40], 260, 32, 8, 128), ([9, 9, 9, 17], 400, 64, 4, 64),
                                               ([33, 20, 128, 65, 25], 150, 12, 4, 128), ([8, 8, 30], 360, 128, 8, 64)])
@pytest.mark.parametrize("window", [0, 1])
def test_short_items_beside_full_ones(uw, new, count, hq, hk, d, window):
    """Items of up to 128 rows, which the lower half of the kernel for many rows passes over, then ones of more,
    many of both a CTA."""
    new = [new[i % len(new)] for i in range(count)]
    lens = [n + (11 * i) % 50 for i, n in enumerate(new)]
    _run(uw, count + window, hq, hk, d, 16, new, lens, False, window, hints=False)
