"""Rotation by positions on several axes (uw_rope_axes, uw_kv4_append_axes) against the formula step by step in
fp32: exact, as in the append, since every product and the sum are rounded alike."""
import numpy as np
import pytest
import torch

from tests import _kv4 as ref

pytestmark = pytest.mark.gpu


def _dev(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


def _bits(t):
    return t.contiguous().cpu().numpy().view(np.uint16)


def _ws(uw):
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    uw.workspace_init(ws)
    return ws


def _tables(rng, rows, pairs):
    angle = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(pairs) / max(pairs, 1))
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


def _turned(bits, pos, axis, cos, sin, interleaved):
    pair = np.arange(len(axis))
    at = pos[axis].T     # [tokens, pairs]
    return ref.rotate(bits, cos[at, pair], sin[at, pair], interleaved)


def _axis(rng, pairs, axes, kind):
    if kind == "sections":
        cuts = np.sort(rng.integers(0, pairs + 1, axes - 1))
        return np.repeat(np.arange(axes), np.diff(np.concatenate([[0], cuts, [pairs]])))
    return rng.integers(0, axes, pairs) if kind == "any" else np.arange(pairs) % axes


@pytest.mark.parametrize("t,hq,hk,d,rot,axes,kind", [
    (1, 32, 8, 128, 128, 3, "sections"), (37, 4, 4, 64, 64, 2, "sections"), (9, 5, 1, 128, 128, 4, "turns"),
    (130, 16, 16, 80, 80, 2, "any"), (3, 3, 2, 72, 64, 3, "any"), (700, 7, 1, 128, 96, 3, "turns"), (5, 1, 1, 16, 16, 1, "any"),
    (2, 2, 3, 256, 256, 4, "any"), (2000, 24, 8, 128, 128, 3, "sections"), (4, 130, 2, 48, 48, 2, "turns"),
    (3, 2, 2, 264, 16, 2, "any")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_axes(uw, t, hq, hk, d, rot, axes, kind, interleaved):
    rng = np.random.default_rng(t + d + axes)
    rows = 300
    cos, sin = _tables(rng, rows, rot // 2)
    axis = _axis(rng, rot // 2, axes, kind)
    pos = rng.integers(0, rows, (axes, t)).astype(np.int32)
    qkv = ref.bf16(rng.standard_normal((t, hq + hk, d)))
    x = _dev(qkv)
    q, k = torch.empty(t, hq, d, dtype=torch.int16, device="cuda"), torch.empty(t, hk, d, dtype=torch.int16, device="cuda")
    ws = _ws(uw)
    args = (_dev(pos), bytes(axis.tolist()))
    uw.rope_axes(x[:, :hq], x[:, hq:], *args, q, k, _dev(cos), _dev(sin), ws, interleaved=interleaved)
    assert uw.check_status(ws) == 0
    want = _turned(qkv, pos, axis, cos, sin, interleaved)
    assert np.array_equal(_bits(q), want[:, :hq]) and np.array_equal(_bits(k), want[:, hq:])
    # in place, one after the other
    uw.rope_axes(x[:, :hq], None, *args, x[:, :hq], None, _dev(cos), _dev(sin), ws, interleaved=interleaved)
    uw.rope_axes(None, x[:, hq:], *args, None, x[:, hq:], _dev(cos), _dev(sin), ws, interleaved=interleaved)
    assert uw.check_status(ws) == 0
    assert np.array_equal(_bits(x), want)


def test_strides_and_gaps(uw):
    """Heads and tokens apart from each other; what lies between them keeps its bits; rows of positions apart."""
    rng = np.random.default_rng(1)
    t, h, d, axes = 11, 3, 64, 3
    cos, sin = _tables(rng, 50, 32)
    axis, pos = _axis(rng, 32, axes, "any"), rng.integers(0, 50, (axes, t)).astype(np.int32)
    x = ref.bf16(rng.standard_normal((t, h, d)))
    wide = torch.full((t, h + 2, d + 8), 0x1234, dtype=torch.int16, device="cuda")
    src = wide[:, 1:1 + h, :d]
    src.copy_(_dev(x))
    out = torch.full((t + 1, h, d + 16), 0x1234, dtype=torch.int16, device="cuda")
    p = torch.full((axes, t + 9), -7, dtype=torch.int32, device="cuda")
    p[:, :t] = _dev(pos)
    ws = _ws(uw)
    uw.rope_axes(src, None, p[:, :t], bytes(axis.tolist()), out[:t, :, :d], None, _dev(cos), _dev(sin), ws)
    assert uw.check_status(ws) == 0
    assert np.array_equal(_bits(out[:t, :, :d]), _turned(x, pos, axis, cos, sin, False))
    assert (out[:t, :, d:] == 0x1234).all() and (out[t] == 0x1234).all()


def test_positions_outside_the_tables(uw):
    """Such tokens are left alone and reported, whichever axis it is; the others are done."""
    rng = np.random.default_rng(2)
    t, h, d = 6, 2, 64
    cos, sin = _tables(rng, 20, 32)
    pos = rng.integers(0, 20, (3, t)).astype(np.int32)
    bad = {1: (0, -1), 2: (1, 20), 4: (2, 2 ** 31 - 1)}
    for token, (a, p) in bad.items():
        pos[a, token] = p
    axis = _axis(rng, 32, 3, "sections")
    x = ref.bf16(rng.standard_normal((t, h, d)))
    out = torch.full((t, h, d), 0x55, dtype=torch.int16, device="cuda")
    ws = _ws(uw)
    uw.rope_axes(_dev(x), None, _dev(pos), bytes(axis.tolist()), out, None, _dev(cos), _dev(sin), ws)
    assert uw.check_status(ws) == 4
    good = np.array([i not in bad for i in range(t)])
    want = _turned(x, np.clip(pos, 0, 19), axis, cos, sin, False)
    assert np.array_equal(_bits(out)[good], want[good]) and np.all(_bits(out)[~good] == 0x55)


class Filled:
    """A cache with a call's tokens appended by axes, and what it should hold."""

    def __init__(self, uw, new, lens, hq, hk, d, page, rot, axes, kind, interleaved, with_q=True, in_place=False, seed=0):
        rng = np.random.default_rng(seed)
        t, rows = sum(new), 200
        table, pool = ref.random_table(rng, lens, page)
        self.pages = ref.Pages(pool, hk, d, page, fill=0xA5)
        cos, sin = _tables(rng, rows, rot // 2)
        axis = _axis(rng, rot // 2, axes, kind)
        pos = rng.integers(0, rows, (axes, t)).astype(np.int32)
        qkv = ref.bf16(rng.standard_normal((t, hq + 2 * hk, d)))
        self.turned = _turned(qkv[:, :hq + hk], pos, axis, cos, sin, interleaved)
        dev = torch.from_numpy(self.pages.bytes.copy()).cuda()
        cache = uw.kv4_cache(dev, torch.from_numpy(table).cuda(), hk, d, page)
        x = _dev(qkv)
        q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        self.q = q if in_place else torch.empty(t, hq, d, dtype=torch.int16, device="cuda")
        self.k = k if in_place else torch.empty(t, hk, d, dtype=torch.int16, device="cuda")
        ws = _ws(uw)
        uw.kv4_append_axes(cache, _dev(ref.starts(new)), _dev(np.array(lens, np.int32)), _dev(pos), bytes(axis.tolist()),
                           q if with_q else None, k, v, self.q if with_q else None, _dev(cos), _dev(sin), ws,
                           k_out=self.k, interleaved=interleaved)
        assert uw.check_status(ws) == 0
        at = 0
        for s, (n, m) in enumerate(zip(new, lens)):
            for i in range(n):
                p = m - n + i
                for which, vec in ((0, self.turned[at + i, hq:]), (1, qkv[at + i, hq + hk:])):
                    code, par = ref.quantise(vec)
                    for h in range(hk):
                        self.pages.put(which, table[s, p // page], p % page, h, code[h], par[h])
            at += n
        self.got = dev.cpu().numpy()
        self.hq = hq


@pytest.mark.parametrize("new,lens", [([1], [1]), ([1, 1, 1], [5, 1, 40]), ([3, 0, 5], [3, 9, 70]), ([90, 1], [90, 33])])
@pytest.mark.parametrize("hq,hk,d,page,rot,axes,kind", [
    (4, 2, 128, 16, 128, 3, "sections"), (6, 3, 64, 32, 64, 4, "any"), (1, 1, 128, 64, 96, 2, "turns"),
    (32, 8, 128, 16, 128, 3, "turns"), (5, 5, 64, 16, 48, 1, "any")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_axes(uw, new, lens, hq, hk, d, page, rot, axes, kind, interleaved):
    f = Filled(uw, new, lens, hq, hk, d, page, rot, axes, kind, interleaved, in_place=d == 64, seed=sum(lens) + d)
    assert np.array_equal(_bits(f.q), f.turned[:, :hq]) and np.array_equal(_bits(f.k), f.turned[:, hq:])
    assert np.array_equal(f.got, f.pages.bytes)


def test_append_axes_without_q(uw):
    f = Filled(uw, [7, 2], [20, 2], 0, 2, 128, 16, 128, 3, "any", False, with_q=False)
    assert np.array_equal(_bits(f.k), f.turned) and np.array_equal(f.got, f.pages.bytes)


def test_equal_positions_are_the_plain_append(uw):
    """All axes at the place in the sequence: uw_kv4_append's bits."""
    rng = np.random.default_rng(3)
    new, lens, hq, hk, d, page = [40, 1], [40, 17], 4, 2, 128, 16
    t = sum(new)
    table, pool = ref.random_table(rng, lens, page)
    cos, sin = (_dev(a) for a in _tables(rng, 64, d // 2))
    x = _dev(ref.bf16(rng.standard_normal((t, hq + 2 * hk, d))))
    pos = np.concatenate([np.arange(m - n, m) for n, m in zip(new, lens)]).astype(np.int32)
    start, length = _dev(ref.starts(new)), _dev(np.array(lens, np.int32))
    got = []
    for axes in (False, True):
        dev = torch.zeros(pool, hk, page * (d + 8), dtype=torch.uint8, device="cuda")
        cache = uw.kv4_cache(dev, torch.from_numpy(table).cuda(), hk, d, page)
        q, ws = torch.empty(t, hq, d, dtype=torch.int16, device="cuda"), _ws(uw)
        qkv = (x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:])
        if axes:
            uw.kv4_append_axes(cache, start, length, _dev(np.stack([pos] * 3)), bytes([0] * 20 + [1] * 20 + [2] * 24), *qkv, q,
                               cos, sin, ws)
        else:
            uw.kv4_append(cache, start, length, *qkv, q, cos, sin, ws)
        assert uw.check_status(ws) == 0
        got.append((q, dev))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_tokens_of_no_sequence_and_bad_positions(uw):
    """Tokens behind the last sequence keep their rows; a token whose position is not in the tables touches nothing."""
    rng = np.random.default_rng(4)
    hq, hk, d, page, t = 2, 1, 64, 16, 9
    cos, sin = (_dev(a) for a in _tables(rng, 10, 32))
    pages = torch.full((2, hk, page * (d + 8)), 0x77, dtype=torch.uint8, device="cuda")
    cache = uw.kv4_cache(pages, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), hk, d, page)
    pos = np.zeros((2, t), np.int32)
    pos[1, 2] = 10
    x = _dev(ref.bf16(rng.standard_normal((t, hq + 2 * hk, d))))
    q, k = torch.full((t, hq, d), 0x55, dtype=torch.int16, device="cuda"), torch.full((t, hk, d), 0x55, dtype=torch.int16, device="cuda")
    ws = _ws(uw)
    uw.kv4_append_axes(cache, _dev(np.array([0, 5], np.int32)), _dev(np.array([5], np.int32)), _dev(pos), bytes([0, 1] * 16),
                       x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], q, cos, sin, ws, k_out=k)
    assert uw.check_status(ws) == 4
    for out in (q, k):
        left = (out == 0x55).all(-1).all(-1).cpu().numpy()
        assert left.tolist() == [i == 2 or i >= 5 for i in range(t)]
    view = pages.cpu().numpy()[0, 0]
    codes = view[:page * d // 2].reshape(page, d // 2)
    assert np.all(codes[2] == 0x77) and np.all(codes[5:] == 0x77) and np.all(pages.cpu().numpy()[1] == 0x77)


def test_a_page_outside_the_pool(uw):
    """Nothing of the cache is touched and the call says so; q and k come out rotated all the same."""
    rng = np.random.default_rng(7)
    hq, hk, d, page, t = 3, 2, 128, 16, 20
    cos, sin = _tables(rng, 40, 64)
    axis, pos = _axis(rng, 64, 3, "sections"), rng.integers(0, 40, (3, t)).astype(np.int32)
    qkv = ref.bf16(rng.standard_normal((t, hq + 2 * hk, d)))
    pages = torch.full((2, hk, page * (d + 8)), 0x77, dtype=torch.uint8, device="cuda")
    cache = uw.kv4_cache(pages, _dev(np.array([[1, 2]], np.int32)), hk, d, page)     # page 2 is none of the pool's
    x, ws = _dev(qkv), _ws(uw)
    q, k = torch.zeros(t, hq, d, dtype=torch.int16, device="cuda"), torch.zeros(t, hk, d, dtype=torch.int16, device="cuda")
    uw.kv4_append_axes(cache, _dev(np.array([0, t], np.int32)), _dev(np.array([t], np.int32)), _dev(pos), bytes(axis.tolist()),
                       x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], q, _dev(cos), _dev(sin), ws, k_out=k)
    assert uw.check_status(ws) == 4
    want = _turned(qkv[:, :hq + hk], pos, axis, cos, sin, False)
    assert np.array_equal(_bits(q), want[:, :hq]) and np.array_equal(_bits(k), want[:, hq:])
    assert (pages[0] == 0x77).all() and not (pages[1] == 0x77).all()


def test_captured_and_replayed(uw):
    rng = np.random.default_rng(5)
    t, h, d = 50, 4, 128
    cos, sin = _tables(rng, 64, 64)
    axis = _axis(rng, 64, 3, "sections")
    x, out = torch.empty(t, h, d, dtype=torch.int16, device="cuda"), torch.empty(t, h, d, dtype=torch.int16, device="cuda")
    pos = torch.zeros(3, t, dtype=torch.int32, device="cuda")
    c, s, ws = _dev(cos), _dev(sin), _ws(uw)
    x.zero_()
    uw.rope_axes(x, None, pos, bytes(axis.tolist()), out, None, c, s, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        uw.rope_axes(x, None, pos, bytes(axis.tolist()), out, None, c, s, ws)
    for seed in (1, 2):
        r = np.random.default_rng(seed)
        xb, p = ref.bf16(r.standard_normal((t, h, d))), r.integers(0, 64, (3, t)).astype(np.int32)
        x.copy_(_dev(xb))
        pos.copy_(_dev(p))
        graph.replay()
        assert np.array_equal(_bits(out), _turned(xb, p, axis, cos, sin, False))


def test_no_tokens(uw):
    x = torch.empty(0, 2, 64, dtype=torch.int16, device="cuda")
    c, pos = torch.ones(4, 32, device="cuda"), torch.empty(2, 0, dtype=torch.int32, device="cuda")
    uw.rope_axes(x, x, pos, bytes(32), torch.empty_like(x), torch.empty_like(x), c, c, _ws(uw))
