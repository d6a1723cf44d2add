"""uw_kv4_append with q rotated in place (q_out is q): the same bits as into
another tensor, in a projection's output whose k and v lie beside q."""
import numpy as np
import pytest
import torch

from tests import _kv4 as ref

pytestmark = pytest.mark.gpu

# hq, hk, D, new, pairs, interleaved: one token, drafted ones, and long calls in which a warp takes several heads in turn
CASES = [(32, 8, 128, [1], 64, False), (32, 8, 128, [1], 64, True), (5, 1, 64, [3, 0, 2], 32, False),
         (32, 8, 128, [1500, 300], 64, False), (32, 8, 128, [1800], 64, True), (12, 4, 64, [2000, 77], 32, False),
         (12, 4, 64, [1999], 8, True), (40, 8, 128, [1200], 32, False), (7, 7, 64, [900], 0, False)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "q%dkv%dd%d-%s-%d-%d" % (*c[:3], "+".join(map(str, c[3])), *c[4:]))
def test_rotation_in_place(uw, case):
    hq, hk, d, new, pairs, interleaved = case
    page, t = 64, sum(new)
    rng = np.random.default_rng(t + pairs)
    qkv = ref.bf16(rng.standard_normal((t, hq + 2 * hk, d)))
    lens = [n + 5 for n in new]
    table, pool = ref.random_table(rng, lens, page)
    angle = np.arange(max(lens))[:, None] * 10000.0 ** (-np.arange(pairs) / max(pairs, 1))
    cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    dev = lambda a: torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()  # noqa: E731
    pages = torch.zeros(pool, hk, page * (d + 8), dtype=torch.uint8, device="cuda")
    cache = uw.kv4_cache(pages, dev(table), hk, d, page)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    uw.workspace_init(ws)
    x = dev(qkv)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    uw.kv4_append(cache, dev(ref.starts(new)), dev(np.array(lens, np.int32)), q, k, v, q,
                  *((dev(cos), dev(sin)) if pairs else (None, None)), ws, interleaved=interleaved)
    assert uw.check_status(ws) == 0
    want, at = qkv.copy(), 0
    for n, m in zip(new, lens):
        pos = m - n + np.arange(n)
        want[at:at + n, :hq] = ref.rotate(qkv[at:at + n, :hq], cos[pos], sin[pos], interleaved)
        at += n
    assert np.array_equal(x.cpu().numpy().view(np.uint16), want)     # and k and v as they were
