"""uw_kv4_append and uw_kv4_read: the rotated q bits, the pages' bytes and the
values read back equal the formulas computed step by step in fp32 (numpy), bit
for bit; whatever a call does not append to keeps its bytes."""
import numpy as np
import pytest
import torch

from tests import _kv4 as ref

pytestmark = pytest.mark.gpu


def _dev(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


def _bits(t):
    """BF16 bits; every NaN as the quiet one (which NaN a conversion gives is not part of the interface)."""
    b = t.contiguous().cpu().numpy().view(np.uint16)
    return np.where((b & 0x7FFF) > 0x7F80, np.uint16(0x7FC0), b)


def _workspace(uw, nbytes=256):
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    uw.workspace_init(ws)
    return ws


def _table(positions, pairs):
    angle = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(pairs) / max(pairs, 1))
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


def _run(uw, rng, hq, hk, d, page, new, lens, pairs, interleaved, qkv=None, extra=0):
    t = int(sum(new)) + extra
    if qkv is None:
        qkv = ref.bf16(rng.standard_normal((t, hq + 2 * hk, d)) * rng.uniform(0.1, 4, (1, hq + 2 * hk, 1)))
    table, pool = ref.random_table(rng, lens, page)
    cos, sin = _table(max(max(lens), 1), pairs)
    want = ref.Pages(pool, hk, d, page, fill=0xA5)
    pages = _dev(want.bytes.copy())
    qd = _dev(qkv)
    out = _dev(np.full((t, max(hq, 1), d), 0x1234, np.uint16))
    start, length, tab = _dev(ref.starts(new)), _dev(np.array(lens, np.int32)), _dev(table)
    ws = _workspace(uw)
    cache = uw.kv4_cache(pages, tab, hk, d, page)
    rope = (_dev(cos), _dev(sin)) if pairs else (None, None)
    q, k, v = qd[:, :hq], qd[:, hq:hq + hk], qd[:, hq + hk:]
    uw.kv4_append(cache, start, length, q if hq else None, k, v, out if hq else None, *rope, ws,
                  interleaved=interleaved)
    ko = _dev(np.full((t, hk, d), 0x1234, np.uint16))
    vo = ko.clone()
    uw.kv4_read(cache, start, length, ko, vo, ws)
    assert uw.check_status(ws) == 0
    q_want = np.full((t, max(hq, 1), d), 0x1234, np.uint16)
    kv_want = np.full((2, t, hk, d), 0x1234, np.uint16)
    at = 0
    for s, (n, m) in enumerate(zip(new, lens)):
        pos = m - n + np.arange(n)
        x = ref.rotate(qkv[at:at + n, :hq + hk], cos[pos], sin[pos], interleaved)
        if hq:
            q_want[at:at + n] = x[:, :hq]
        for which, src in ((0, x[:, hq:]), (1, qkv[at:at + n, hq + hk:])):
            code, par = ref.quantise(src)
            val = ref.value(code, par)
            for i in range(n):
                for h in range(hk):
                    want.put(which, table[s, pos[i] // page], pos[i] % page, h, code[i, h], par[i, h])
            kv_want[which, at:at + n] = ref.bf16(val)
        at += n
    if hq:
        assert np.array_equal(_bits(out), q_want)
    assert np.array_equal(pages.cpu().numpy(), want.bytes)
    for got, exp in ((ko, kv_want[0]), (vo, kv_want[1])):
        assert np.array_equal(_bits(got), exp)


CASES = [
    # hq, hk, D, page, new, lens, pairs, interleaved
    (32, 8, 128, 16, [1], [1], 64, False),
    (32, 8, 128, 16, [1], [1025], 64, False),
    (32, 8, 128, 64, [1, 1, 1, 1, 1], [17, 64, 65, 1, 500], 64, True),
    (8, 8, 64, 32, [3, 0, 70, 1], [3, 40, 100, 33], 32, False),
    (6, 2, 64, 16, [5, 33], [5, 48], 32, True),
    (4, 1, 128, 256, [300], [300], 64, False),
    (5, 5, 128, 128, [2, 2], [130, 2], 32, False),      # half of the dimensions rotated
    (3, 1, 64, 16, [19], [20], 8, True),                # a quarter
    (7, 7, 64, 16, [4], [9], 0, False),                 # none
    (0, 2, 128, 16, [20], [21], 64, False),             # keys and values alone
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "q%dkv%dd%dp%d" % c[:4])
def test_append_and_read(uw, case):
    _run(uw, np.random.default_rng(sum(case[4]) + case[3]), *case)


def test_many_sequences(uw):
    """More sequences than one round of the search covers, empty ones among them."""
    rng = np.random.default_rng(11)
    new = [int(n) for n in rng.integers(0, 3, 1100)]
    lens = [n + int(m) for n, m in zip(new, rng.integers(0, 40, 1100))]
    _run(uw, rng, 2, 1, 64, 16, new, lens, 32, False)


def test_tokens_of_no_sequence_are_left_alone(uw):
    _run(uw, np.random.default_rng(3), 4, 2, 128, 16, [3, 2], [30, 2], 64, False, extra=6)


def test_long_call(uw):
    """Several heads a warp."""
    _run(uw, np.random.default_rng(4), 12, 4, 128, 64, [900, 1, 700], [900, 77, 1001], 64, False)


def test_extreme_vectors(uw):
    """Constant, zero, subnormal, largest finite and not finite vectors; one large value among small ones."""
    rng = np.random.default_rng(5)
    d, hk, t = 128, 1, 12
    qkv = ref.bf16(rng.standard_normal((t, 3, d)))
    for i, row in enumerate([0x0000, 0x3F80, 0xBF80, 0x0001, 0x7F7F, 0x8000]):
        qkv[i, 1:] = row
    qkv[4, 1:, ::2] = 0xFF7F                    # range beyond the largest fp32
    qkv[3, 1:, 5] = 0x0003                      # a range of two smallest steps
    qkv[6, 1:, 7] = 0x7F80
    qkv[7, 1:, 9] = 0xFF80
    qkv[8, 1:, 11] = 0x7FC1
    qkv[9, 1:] = ref.bf16(np.full(d, 1e-3))
    qkv[9, 1:, 3] = 0x4780                      # 65536
    _run(uw, rng, 1, hk, d, 16, [t], [t], 0, False, qkv=qkv)


def test_bad_device_values_touch_nothing_and_are_reported(uw):
    hk, d, page = 2, 64, 16
    x = _dev(ref.bf16(np.random.default_rng(1).standard_normal((2, 4, d))))
    cos = torch.ones(64, 32, device="cuda")

    def run(table, start, length, rows=64):
        pages = torch.full((3, hk, page * (d + 8)), 7, dtype=torch.uint8, device="cuda")
        cache = uw.kv4_cache(pages, _dev(np.array(table, np.int32)), hk, d, page)
        ws = _workspace(uw)
        q = torch.zeros(2, 2, d, dtype=torch.int16, device="cuda")
        uw.kv4_append(cache, _dev(np.array(start, np.int32)), _dev(np.array(length, np.int32)), x[:, :2], x[:, :2],
                      x[:, 2:], q, cos[:rows], cos[:rows], ws)
        status = uw.check_status(ws)
        assert uw.check_status(ws) == 0
        return status, bool((pages == 7).all())

    assert run([[0, 1]], [0, 2], [20]) == (0, False)
    assert run([[0, 3]], [0, 2], [20]) == (4, True)       # a page past the pool
    assert run([[0, -1]], [0, 2], [20]) == (4, True)      # a page before it
    assert run([[0, 1]], [0, 2], [33]) == (4, True)       # a length past the table
    assert run([[0, 1]], [0, 2], [-1]) == (4, True)
    assert run([[0, 1]], [0, 3], [20]) == (4, True)       # a start past the call's tokens
    assert run([[0, 1]], [1, 0], [20]) == (4, True)
    assert run([[0, 1]], [0, 2], [20], rows=18) == (4, True)   # positions past the rotation table
    status, untouched = run([[0, 1]], [0, 2], [1])        # more new tokens than the sequence holds
    assert status == 4 and not untouched                   # the second, at position 0, is appended


def test_cache_past_two_and_four_gigabytes(uw):
    """Pages whose byte offsets pass 31 and 32 bits."""
    hk, d, page = 8, 128, 256
    size = uw.kv4_page_bytes(hk, d, page)
    n_pages = (1 << 32) // size + 3
    pages = torch.zeros(n_pages, size, dtype=torch.uint8, device="cuda")
    table = _dev(np.array([[n_pages - 1, (1 << 31) // size + 1]], np.int32))
    cache = uw.kv4_cache(pages, table, hk, d, page)
    rng = np.random.default_rng(2)
    x = ref.bf16(rng.standard_normal((300, 2 * hk, d)))
    xd, ws = _dev(x), _workspace(uw)
    start, length = _dev(np.array([0, 300], np.int32)), _dev(np.array([300], np.int32))
    uw.kv4_append(cache, start, length, None, xd[:, :hk], xd[:, hk:], None, None, None, ws)
    k = torch.empty(300, hk, d, dtype=torch.int16, device="cuda")
    v = torch.empty_like(k)
    uw.kv4_read(cache, start, length, k, v, ws)
    assert uw.check_status(ws) == 0
    for got, src in ((k, x[:, :hk]), (v, x[:, hk:])):
        assert np.array_equal(_bits(got), ref.bf16(ref.value(*ref.quantise(src))))
    assert int(pages[0].max()) == 0
