"""uw_attention against the formula in 64 bits.

Bound on an output, from the formats: a probability is rounded to BF16 (2^-8 of it) and so is the output
(2^-8 of it); a score is a sum of D products in fp32 (in an order of the tensor cores', each step off by at
most 2^-23 of the running sum of magnitudes), which moves a probability and the sum under it by that much
times the softmax scale, each; exponentials and the rescaling by maxima 2^-20.  The lse is off by the score's error,
that of a sum of m / 64 + 64 steps and its own rounding."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _starts(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()


def _ws(uw, dim=128):
    ws = torch.empty(uw.attention_workspace_size(dim), dtype=torch.uint8, device="cuda")
    uw.workspace_init(ws)
    return ws


def _normal(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def _seen(n, m, causal, window):
    pos, key = m - n + torch.arange(n, device="cuda")[:, None], torch.arange(m, device="cuda")
    seen = torch.ones(n, m, dtype=torch.bool, device="cuda")
    if causal:
        seen &= key <= pos
    if window:
        # the keys max(0, p - window + 1) .. of a token at position p (or below 0: from 0)
        seen &= key > (pos.clamp(min=-1) - window)
    return seen


def _reference(q, k, v, new, kv, causal, window, scale):
    """o, lse, and their bounds, 64 bits; rows of no sequence NaN."""
    t, hq, d = q.shape
    hk = k.shape[1]
    scale = scale or d ** -0.5
    o = torch.full((t, hq, d), np.nan, dtype=torch.float64, device="cuda")
    lse = torch.full((t, hq), np.nan, dtype=torch.float64, device="cuda")
    o_tol, lse_tol = torch.zeros_like(o), torch.zeros_like(lse)
    a = b = 0
    for n, m in zip(new, kv):
        seen = _seen(n, m, causal, window)
        for h in range(hq):
            qd, kd, vd = (x.double() for x in (q[a:a + n, h], k[b:b + m, h * hk // hq], v[b:b + m, h * hk // hq]))
            s = torch.where(seen, qd @ kd.T * scale, -np.inf)
            top = s.amax(1, keepdim=True) if m else torch.full((n, 1), -np.inf, device="cuda", dtype=torch.float64)
            p = torch.exp(s - torch.where(top.isneginf(), 0.0, top))
            tot = p.sum(1, keepdim=True)
            pn = p / torch.where(tot == 0, 1.0, tot)
            o[a:a + n, h] = pn @ vd
            lse[a:a + n, h] = (tot.log() + top)[:, 0]
            rough = torch.where(seen, qd.abs() @ kd.abs().T, 0.0)
            off = (rough.amax(1, keepdim=True) if m else torch.zeros(n, 1, device="cuda").double()) * scale * (d + 8) * 2.0 ** -23
            o_tol[a:a + n, h] = (pn @ vd.abs()) * (2.0 ** -8 * 1.01 + 2 * off + 2.0 ** -20) + o[a:a + n, h].abs() * 2.0 ** -8 * 1.01
            lse_tol[a:a + n, h] = off[:, 0] + (m / 64 + 64) * 2.0 ** -24 + lse[a:a + n, h].abs() * 2.0 ** -22 + 2.0 ** -20
        a, b = a + n, b + m
    return o, lse, o_tol, lse_tol


def _check(out, lse, want):
    o, l, o_tol, l_tol = want
    ok = (out.double() - o).abs() <= o_tol + 1e-38
    assert ok[~o.isnan()].all(), "out: %g of the bound" % ((out.double() - o).abs() / o_tol)[~ok].max().item()
    if lse is not None:
        inf = l.isneginf()
        assert lse[inf].isneginf().all()
        bad = ((lse.double() - l).abs() > l_tol) & ~inf & ~l.isnan()
        assert not bad.any(), (lse.double() - l)[bad]


class Case:
    def __init__(self, uw, new, kv, hq, hk, d, causal=True, window=0, scale=0.0, seed=0, spare=3):
        t, m = sum(new) + spare, sum(kv) + spare
        self.uw, self.new, self.kv, self.opts = uw, new, kv, dict(causal=causal, window=window, scale=scale)
        self.q = (_normal(seed, t, hq, d) * 1.5).bfloat16()
        self.k = (_normal(seed + 1, m, hk, d) * (0.3 + _normal(seed + 2, 1, hk, d).abs())).bfloat16()
        self.v = (_normal(seed + 3, m, hk, d) * 2 + 0.5).bfloat16()
        self.ws = _ws(uw, d)

    def run(self, lse=True, ws=None):
        ws = self.ws if ws is None else ws
        q = self.q
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        l = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
        self.uw.attention(q, self.k, self.v, out, _starts(self.new), ws, kv_start=_starts(self.kv), lse=l, **self.opts)
        assert self.uw.check_status(ws) == 0
        return out, l

    def check(self, out, lse):
        _check(out, lse, _reference(self.q, self.k, self.v, self.new, self.kv, **self.opts))
        n = sum(self.new)
        assert (out[n:] == 7).all() and (lse is None or (lse[n:] == 7).all())  # rows behind the last sequence


LENGTHS = [[1], [2], [37], [64], [127, 1], [128], [129], [256], [300, 1, 0, 65], [1] * 40, [700], [31, 1000, 5]]


@pytest.mark.parametrize("new", LENGTHS)
@pytest.mark.parametrize("hq,hk,d", [(1, 1, 64), (4, 4, 128), (8, 2, 128), (8, 2, 64), (7, 1, 128), (6, 2, 64), (5, 1, 128),
                                     (16, 1, 64)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50)])
def test_whole_sequences(uw, new, hq, hk, d, causal, window):
    c = Case(uw, new, new, hq, hk, d, causal, window, seed=sum(new) + hq + d)
    c.check(*c.run())


@pytest.mark.parametrize("new,kv", [([1], [5000]), ([5], [20001]), ([100, 3], [400, 1000]), ([300], [10]), ([4, 3, 200], [0, 1, 100]),
                                    ([1, 0, 1], [0, 50, 0]), ([513], [2049]), ([2], [128]), ([130], [127])])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (3, 1, 64)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (False, 77), (True, 2 ** 31 - 1)])
def test_other_counts_of_keys(uw, new, kv, hq, hk, d, causal, window):
    c = Case(uw, new, kv, hq, hk, d, causal, window, seed=sum(kv) + d)
    c.check(*c.run())


@pytest.mark.parametrize("scale", [0.0, 0.02, 1.0, 2.0 ** -30])
def test_softmax_scales(uw, scale):
    c = Case(uw, [200, 90], [200, 90], 4, 2, 128, scale=scale)
    c.check(*c.run(lse=False))


@pytest.mark.parametrize("way", ["up", "down", "jumps", "masked"])
@pytest.mark.parametrize("d", [64, 128])
def test_maxima_that_move(uw, way, d):
    """Scores that rise by hundreds from key to key, fall, or jump: the running maximum is raised in every half tile."""
    n = 700
    c = Case(uw, [n], [n], 4, 2, d, causal=way != "down", seed=5, spare=0)
    at = torch.arange(n, device="cuda").float()
    level = {"up": at, "down": -at, "jumps": 300.0 * ((at // 50) % 3), "masked": 3 * at}[way]
    c.q[..., 0], c.k[..., 0] = 16.0, level[:, None].bfloat16()
    c.k[..., 1:] *= 0.1
    c.check(*c.run())


@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (3, 1, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_keys_and_values_that_are_not_finite(uw, hq, hk, d, bad):
    """What a token does not see takes no part in it, whatever its bits: later keys, keys before the window, other
    sequences' and those of none; what it sees does."""
    new = [300, 1, 140, 513]
    at = np.concatenate([[0], np.cumsum(new)])
    for window in (0, 60):
        c = Case(uw, new, new, hq, hk, d, window=window, seed=9)
        clean = c.run()
        # one value of V in each of some keys, of the spare rows too
        hit = [(0, 200), (1, 0), (2, 139), (3, 130), (3, 300)]
        for s, i in hit:
            c.v[at[s] + i, 0, i % d] = bad
        c.v[at[-1]:] = bad
        out, lse = c.run()
        assert torch.equal(lse, clean[1])
        want = clean[0].clone()
        for s, i in hit:
            last = new[s] if not window else min(new[s], i + window)
            want[at[s] + i:at[s] + last, :hq // hk, i % d] = bad
        assert torch.equal(out.isnan(), want.isnan()) and torch.equal(out[~out.isnan()], want[~want.isnan()])
        # a whole key
        c = Case(uw, new, new, hq, hk, d, window=window, seed=9)
        c.k[at[3] + 250], c.k[at[-1]:] = float("nan"), bad
        out, lse = c.run()
        rows = torch.zeros(len(out), dtype=torch.bool, device="cuda")
        rows[at[3] + 250:at[3] + (513 if not window else min(513, 250 + window))] = True
        assert out[rows].isnan().all() and lse[rows].isnan().all()
        assert torch.equal(out[~rows], clean[0][~rows]) and torch.equal(lse[~rows], clean[1][~rows])


def test_queries_that_are_not_finite(uw):
    c = Case(uw, [300], [300], 4, 2, 128, causal=False, seed=3)
    clean = c.run()
    c.q[17, 1, 5] = float("nan")
    out, lse = c.run()
    assert out[17, 1].isnan().all() and lse[17, 1].isnan()
    out[17, 1], lse[17, 1] = clean[0][17, 1], clean[1][17, 1]
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("d", [64, 128])
def test_strides(uw, d):
    """Slices of one projection, heads outside of tokens, a head that all kv heads share, rows apart."""
    t, hq, hk = 333, 6, 3
    ws, start = _ws(uw, d), _starts([200, 133])
    qkv = _normal(1, t, hq + 2 * hk, d).bfloat16()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    want = _reference(q, k, v, [200, 133], [200, 133], True, 0, 0)

    def run(q, k, v, out):
        uw.attention(q, k, v, out, start, ws)
        assert uw.check_status(ws) == 0
        return out

    plain = run(q, k, v, torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda"))
    _check(plain, None, want)
    by_heads = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    out = torch.full((hq, t + 1, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(run(*by_heads, out[:, :t, :d].transpose(0, 1)), plain)
    assert (out[:, t] == 7).all() and (out[..., d:] == 7).all()
    apart = [torch.zeros(t, x.shape[1], d + 24, dtype=torch.bfloat16, device="cuda")[..., :d].copy_(x) for x in (q, k, v)]
    assert torch.equal(run(*apart, torch.empty_like(plain)), plain)
    one = [x[:, 1:2].expand(t, hk, d) for x in (k, v)]
    _check(run(q, *one, torch.empty_like(plain)), None, _reference(q, *one, [200, 133], [200, 133], True, 0, 0))
    in_place = q.clone()
    assert torch.equal(run(in_place, k, v, in_place), plain)


def test_no_kv_start_is_the_tokens(uw):
    c = Case(uw, [77, 200], [77, 200], 4, 1, 64, spare=0)
    out, _ = c.run()
    again = torch.empty_like(out)
    uw.attention(c.q, c.k, c.v, again, _starts([77, 200]), c.ws)
    assert torch.equal(out, again)


def test_many_sequences(uw):
    """More sequences than a CTA has threads, most of them short, some empty; a share is many lists long."""
    rng = np.random.default_rng(0)
    new = [int(n) for n in rng.integers(0, 6, 1100)] + [300] + [int(n) for n in rng.integers(0, 3, 400)]
    c = Case(uw, new, new, 2, 1, 64, spare=0)
    out, lse = c.run()
    start = np.concatenate([[0], np.cumsum(new)])
    some = [i for i in (0, 1, 2, 500, 511, 512, 513, 1023, 1024, 1100, 1101, 1500)]
    for i in some:
        a, b = start[i], start[i + 1]
        if a < b:
            _check(out[a:b], lse[a:b], _reference(c.q[a:b], c.k[a:b], c.v[a:b], [b - a], [b - a], True, 0, 0))
    assert out.isfinite().all() and not (out == 7).all(-1).any()


def test_same_bits_twice_and_in_one_workspace(uw):
    """Calls of both head sizes and of any lengths after each other in one workspace."""
    big, small = Case(uw, [900, 5], [900, 5], 8, 2, 128, seed=1), Case(uw, [64, 3000], [64, 3000], 4, 1, 64, seed=2)
    want = [c.run(ws=_ws(uw)) for c in (big, small)]
    ws = _ws(uw)
    for _ in range(2):
        for c, w in zip((big, small), want):
            got = c.run(ws=ws)
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])


def test_starts_that_do_not_hold(uw):
    """A sequence outside the call's rows is left alone and reported; the others are done."""
    c = Case(uw, [10, 20, 30], [10, 20, 30], 4, 2, 64, spare=0)
    want, _ = c.run()
    for bad in ([0, 10, 30, 61], [-1, 10, 30, 60], [0, 10, 70, 60], [0, 10, 5, 60]):
        out = torch.full_like(want, 7.0)
        start = torch.tensor(bad, dtype=torch.int32).cuda()
        uw.attention(c.q, c.k, c.v, out, start, c.ws)
        assert uw.check_status(c.ws) == 4
        if bad[1:3] == [10, 30]:
            assert torch.equal(out[10:30], want[10:30])
            left = slice(30, 60) if bad[3] == 61 else slice(0, 10)
            assert (out[left] == 7).all()
    out = torch.full_like(want, 7.0)
    uw.attention(c.q, c.k, c.v, out, _starts([10, 20, 30]), c.ws, kv_start=torch.tensor([0, 10, 61, 60], dtype=torch.int32).cuda())
    assert uw.check_status(c.ws) == 4 and torch.equal(out[:10], want[:10]) and (out[10:] == 7).all()


def test_captured_and_replayed_with_other_lengths(uw):
    t, hq, hk, d = 600, 4, 2, 128
    q, k, v = (_normal(i, t, h, d).bfloat16() for i, h in ((1, hq), (2, hk), (3, hk)))
    out, lse, ws = torch.empty_like(q), torch.empty(t, hq, device="cuda"), _ws(uw)
    start = _starts([100, 200, 300])
    uw.attention(q, k, v, out, start, ws, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        uw.attention(q, k, v, out, start, ws, lse=lse)
    for new in ([600, 0, 0], [1, 598, 1], [0, 0, 250]):
        start.copy_(_starts(new))
        q.copy_(_normal(sum(new) + new[0], t, hq, d).bfloat16())
        graph.replay()
        assert uw.check_status(ws) == 0
        n = sum(new)
        _check(out[:n], lse[:n], _reference(q[:n], k[:n], v[:n], new, new, True, 0, 0))


def test_nothing_to_do(uw):
    ws = _ws(uw)
    q = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    uw.attention(q, q, q, torch.empty_like(q), _starts([0, 0]), ws)
    q = torch.ones(5, 4, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    uw.attention(q, q, q, out, torch.zeros(1, dtype=torch.int32, device="cuda"), ws)
    uw.attention(q, q, q, out, _starts([0]), ws)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert (out == 7).all()
    lse = torch.empty(5, 4, device="cuda")
    uw.attention(q, none, none, out, _starts([5]), ws, kv_start=_starts([0]), lse=lse)
    assert (out == 0).all() and lse.isneginf().all() and uw.check_status(ws) == 0


@pytest.mark.parametrize("hq,hk,d", [(320, 1, 64), (129, 1, 128), (600, 2, 128)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 9)])
def test_more_heads_than_a_tile_has_rows(uw, hq, hk, d, causal, window):
    c = Case(uw, [5, 0, 33], [5, 7, 140], hq, hk, d, causal, window, seed=hq)
    c.check(*c.run())


@pytest.mark.parametrize("hq,hk,d", [(8, 1, 128), (7, 1, 64)])
def test_over_the_queries_with_items_in_parts(uw, hq, hk, d):
    """out may be q: items that several CTAs share, and tiles that end inside the next sequence."""
    c = Case(uw, [1999, 301, 77], [1999, 301, 77], hq, hk, d, seed=3)
    want, l = c.run()
    c.check(want, l)
    start, n = _starts(c.new), sum(c.new)
    for _ in range(3):
        q = c.q.clone()
        uw.attention(q, c.k, c.v, q, start, c.ws, kv_start=start)
        assert torch.equal(q[:n], want[:n]) and torch.equal(q[n:], c.q[n:])


def test_two_streams_at_once(uw):
    cases = [Case(uw, [700, 64, 1], [700, 64, 1], 8, 2, 128, seed=5), Case(uw, [513, 900], [513, 900], 4, 4, 64, False, seed=6)]
    want = [c.run()[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[torch.full_like(c.q, 7.0) for _ in range(8)] for c in cases]
    starts = [_starts(c.new) for c in cases]
    torch.cuda.synchronize()
    for i in range(8):
        for c, s, out, start in zip(cases, streams, outs, starts):
            with torch.cuda.stream(s):
                uw.attention(c.q, c.k, c.v, out[i], start, c.ws, kv_start=start, **c.opts)
    torch.cuda.synchronize()
    for c, out, w in zip(cases, outs, want):
        assert uw.check_status(c.ws) == 0 and all(torch.equal(o, w) for o in out)
