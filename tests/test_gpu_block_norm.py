"""uw_block_norm and uw_block_norm_e4m3 against the formula in 64 bits.

Bounds, from the formats.  h is one rounding to BF16 (2^-8 of the value) of a sum in fp32: the
block's part has a sum of d squares in any order, at most d * 2^-24 off (its root half of that), and fewer
than 16 further roundings; the residual's part two.  y is held to the norm of the very h that came back:
fp32 arithmetic with the same sum and one rounding to BF16, or an e4m3 value within half a step (2^-4 of
the value, or 2^-10 of the scale for the smallest) of y / scale."""
import numpy as np
import pytest
import torch

from tests._kv4 import bf16, f32

pytestmark = pytest.mark.gpu


def _dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda()


def _bits(t):
    return t.contiguous().cpu().numpy().view(np.uint16)


def _f64(bits):
    return f32(bits).reshape(bits.shape).astype(np.float64)


class Inputs:
    def __init__(self, n, d, post, gate, offset, seed):
        rng = np.random.default_rng(seed)
        self.x = bf16(rng.standard_normal((n, d)) * (0.1 + rng.random((n, 1))))
        self.r = bf16(3 * rng.standard_normal((n, d)))
        self.w = bf16(1 - offset + 0.2 * rng.standard_normal(d))
        self.wp = bf16(1 - offset + 0.2 * rng.standard_normal(d)) if post else None
        self.g = {"none": None, "channel": bf16(rng.standard_normal(d)), "row": bf16(rng.standard_normal((n, d)))}[gate]
        self.offset = offset

    def h(self, eps, rs, bs):
        """h before its rounding, and how far fp32 may be off it."""
        z = _f64(self.x)
        if self.wp is not None:
            z = z / np.sqrt((z * z).mean(-1, keepdims=True) + eps) * (_f64(self.wp) + self.offset)
        if self.g is not None:
            z = z * _f64(self.g)
        z, r = np.float32(bs) * z, np.float32(rs) * _f64(self.r)
        return z + r, ((self.x.shape[-1] + 16) * np.abs(z) + 4 * np.abs(r)) * 2.0 ** -24


def _check_h(h_bits, want, slack):
    assert np.all(np.abs(_f64(h_bits) - want) <= 2.0 ** -8 * 1.001 * np.abs(want) + slack * 1.01 + 1e-38)


def _normed(h_bits, w_bits, offset, eps):
    f = _f64(h_bits)
    return f / np.sqrt((f * f).mean(-1, keepdims=True) + eps) * (_f64(w_bits) + offset)


def _rel(d):
    return 2.0 ** -8 * 1.001 + (d + 16) * 2.0 ** -24


def _check_y(y_bits, want):
    assert np.all(np.abs(_f64(y_bits) - want) <= _rel(want.shape[-1]) * np.abs(want) + 1e-38)


def _check_e4m3(q, scale, want):
    d = want.shape[-1]
    s = scale.cpu().numpy().astype(np.float64)
    s_ref = np.maximum(np.abs(want).max(1) / 448, 2.0 ** -126)
    assert np.all(np.abs(s - s_ref) <= (d + 24) * 2.0 ** -24 * s_ref)
    got = q.contiguous().view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64) * s[:, None]
    slack = (d + 24) * 2.0 ** -23
    assert np.all(np.abs(got - want) <= (2.0 ** -4 + slack) * np.abs(want) + 2.0 ** -10 * s[:, None])


def _opt(bits):
    return None if bits is None else _dev(bits)


# a warp's and a CTA's rows with partly filled last vectors; odd, short and longer rows
SHAPES = [(1, 8), (9, 64), (3, 264), (17, 512), (5, 1000), (8, 1024), (2, 1032), (257, 4096), (1, 4096), (3, 5120),
          (2, 8200), (2, 16384), (2, 16392), (1, 1), (4, 7), (5, 1023), (3, 4097), (2, 16383), (1, 40001)]


@pytest.mark.parametrize("n,d", SHAPES)
@pytest.mark.parametrize("post,gate,offset,rs,bs", [(True, "none", 0.0, 1.0, 1.0), (True, "channel", 1.0, 0.5, 0.25),
                                                    (False, "row", 0.0, 1.0, -1.5), (True, "row", 1.0, 1.0, 1.0),
                                                    (False, "none", 0.0, 1.0, 1.0)])
@pytest.mark.parametrize("bits", [16, 8])
def test_rows(uw, n, d, post, gate, offset, rs, bs, bits):
    i = Inputs(n, d, post, gate, offset, 7 * n + d)
    x, h = _dev(i.x), _dev(np.full((n, d), 0x7FC0, np.uint16))
    y = torch.empty(n, d, dtype=torch.int16 if bits == 16 else torch.uint8, device="cuda")
    scale = torch.empty(n, dtype=torch.float32, device="cuda")
    uw.block_norm(x, _dev(i.r), _dev(i.w), h, y, 1e-6, post_weight=_opt(i.wp), gate=_opt(i.g), residual_scale=rs,
                  block_scale=bs, weight_offset=offset, scale=None if bits == 16 else scale)
    _check_h(_bits(h), *i.h(1e-6, rs, bs))
    want = _normed(_bits(h), i.w, offset, 1e-6)
    if bits == 16:
        _check_y(_bits(y), want)
    else:
        _check_e4m3(y, scale, want)


@pytest.mark.parametrize("d", [1, 7, 9, 15, 263, 1018, 1025, 4099, 16377, 16384])
@pytest.mark.parametrize("alike", [True, False])
@pytest.mark.parametrize("bits", [16, 8])
def test_rows_that_begin_anywhere(uw, d, alike, bits):
    """Strided rows at the same or at different distances from 16-byte steps; what lies between them keeps its bits."""
    n, off = 7, 3
    i = Inputs(n, d, True, "row", 1.0, d)
    stride = {"x": d, "r": d + 8, "h": d + 16, "y": d, "g": d + (8 if alike else 5)}

    def spread(name, values, dtype):
        st = stride[name]
        buf = np.full(off + (n - 1) * st + d + 16, 0x34, dtype)
        rows = np.lib.stride_tricks.as_strided(buf[off:], (n, d), (st * buf.itemsize, buf.itemsize))
        if values is not None:
            rows[:] = values
        t = _dev(buf) if dtype == np.uint16 else torch.from_numpy(buf).cuda()
        return t, t[off:].as_strided((n, d), (st, 1))

    (_, x), (_, r), (_, g) = spread("x", i.x, np.uint16), spread("r", i.r, np.uint16), spread("g", i.g, np.uint16)
    (hb, h), (yb, y) = spread("h", None, np.uint16), spread("y", None, np.uint16 if bits == 16 else np.uint8)
    w, wp = (_dev(np.concatenate([np.zeros(2, np.uint16), v]))[2:] for v in (i.w, i.wp))
    scale = torch.empty(n, dtype=torch.float32, device="cuda")
    uw.block_norm(x, r, w, h, y, 1e-5, post_weight=wp, gate=g, weight_offset=1.0, scale=None if bits == 16 else scale)
    _check_h(_bits(h), *i.h(1e-5, 1.0, 1.0))
    want = _normed(_bits(h), i.w, 1.0, 1e-5)
    if bits == 16:
        _check_y(_bits(y), want)
    else:
        _check_e4m3(y, scale, want)
    for buf, name in ((hb, "h"), (yb, "y")):
        b, st = buf.cpu().numpy(), stride[name]
        used = (off + st * np.arange(n)[:, None] + np.arange(d)).ravel()
        assert np.all(np.delete(b, used) == 0x34)


@pytest.mark.parametrize("d", [512, 4096, 777, 20000])
@pytest.mark.parametrize("to", ["residual", "x"])
def test_in_place(uw, d, to):
    """h over the residual and y over x, and the other way round."""
    i = Inputs(6, d, True, "channel", 0.0, d)
    x, r = _dev(i.x), _dev(i.r)
    h, y = (r, x) if to == "residual" else (x, r)
    uw.block_norm(x, r, _dev(i.w), h, y, 1e-5, post_weight=_dev(i.wp), gate=_dev(i.g))
    _check_h(_bits(h), *i.h(1e-5, 1.0, 1.0))
    _check_y(_bits(y), _normed(_bits(h), i.w, 0.0, 1e-5))


@pytest.mark.parametrize("d", [520, 4096, 20000])
def test_without_y_and_without_h(uw, d):
    i = Inputs(3, d, True, "row", 0.0, d)
    x, r, w, wp, g = _dev(i.x), _dev(i.r), _dev(i.w), _dev(i.wp), _dev(i.g)
    h, y, h2, y2 = (torch.empty_like(x) for _ in range(4))
    uw.block_norm(x, r, w, h, y, 1e-5, post_weight=wp, gate=g)
    uw.block_norm(x, r, None, h2, None, 1e-5, post_weight=wp, gate=g)
    uw.block_norm(x, r, w, None, y2, 1e-5, post_weight=wp, gate=g)
    assert torch.equal(h, h2) and torch.equal(y, y2)


def test_one_vector_is_a_row(uw):
    i = Inputs(1, 640, True, "channel", 0.0, 3)
    x, r, w, wp, g = _dev(i.x[0]), _dev(i.r[0]), _dev(i.w), _dev(i.wp), _dev(i.g)
    h, y = torch.empty_like(x), torch.empty_like(x)
    uw.block_norm(x, r, w, h, y, 1e-5, post_weight=wp, gate=g)
    _check_h(_bits(h)[None], *i.h(1e-5, 1.0, 1.0))
    _check_y(_bits(y)[None], _normed(_bits(h)[None], i.w, 0.0, 1e-5))


def test_plain_call_is_the_residual_norm(uw):
    """Without a norm after the block, a gate and scales: uw_rmsnorm's bits."""
    for n, d in ((5, 300), (3, 4096), (2, 8200), (2, 17000)):
        i = Inputs(n, d, False, "none", 0.0, d)
        x, r, w = _dev(i.x), _dev(i.r), _dev(i.w)
        h, y, h2, y2 = (torch.empty_like(x) for _ in range(4))
        uw.block_norm(x, r, w, h, y, 1e-5)
        uw.rmsnorm(x, w, y2, 1e-5, residual=r, residual_out=h2)
        assert torch.equal(h, h2)
        _check_y(_bits(y), _normed(_bits(h2), i.w, 0.0, 1e-5))


@pytest.mark.parametrize("d", [64, 333, 4096, 20000])
def test_zero_and_non_finite_rows(uw, d):
    i = Inputs(6, d, True, "none", 0.0, d + 1)
    i.x[0] = 0                       # nothing from the block: h is the residual
    i.x[1, d // 2] = 0x7F80          # infinity: its own value is NaN (inf / inf), the others 0
    i.x[2, d - 1] = 0x7FC1           # NaN
    i.r[3, 0] = 0xFF80
    x, h = _dev(i.x), torch.empty(6, d, dtype=torch.int16, device="cuda")
    y, q = torch.empty_like(h), torch.empty(6, d, dtype=torch.uint8, device="cuda")
    scale = torch.empty(6, dtype=torch.float32, device="cuda")
    r, w, wp = _dev(i.r), _dev(i.w), _dev(i.wp)
    uw.block_norm(x, r, w, h, y, 1e-5, post_weight=wp)
    uw.block_norm(x, r, w, h, q, 1e-5, post_weight=wp, scale=scale)
    hb, yb = _f64(_bits(h)), _f64(_bits(y))
    assert np.array_equal(_bits(h)[0], i.r[0])
    assert np.isnan(hb[1, d // 2]) and np.array_equal(np.delete(_bits(h)[1], d // 2), np.delete(i.r[1], d // 2))
    assert np.isnan(hb[2]).all() and hb[3, 0] == -np.inf and np.isfinite(hb[3, 1:]).all()
    assert np.isnan(yb[1:3]).all() and np.isnan(yb[3, 0]) and np.all(yb[3, 1:] == 0)
    e = q.view(torch.float8_e4m3fn).float().cpu().numpy()
    assert np.isnan(e[1:4]).all() and np.isnan(scale.cpu().numpy()[1:4]).all()
    for k in (0, 4, 5):
        _check_y(_bits(y)[k:k + 1], _normed(_bits(h)[k:k + 1], i.w, 0.0, 1e-5))
        assert np.isfinite(e[k]).all()


def test_captured_and_replayed_on_another_stream(uw):
    i = Inputs(33, 2048, True, "channel", 0.0, 5)
    x, r, w, wp, g = _dev(i.x), _dev(i.r), _dev(i.w), _dev(i.wp), _dev(i.g)
    h, y = torch.empty_like(x), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        uw.block_norm(x, r, w, h, y, 1e-5, post_weight=wp, gate=g)
        with torch.cuda.graph(graph, stream=side):
            uw.block_norm(x, r, w, h, y, 1e-5, post_weight=wp, gate=g)
    torch.cuda.current_stream().wait_stream(side)
    other = Inputs(33, 2048, True, "channel", 0.0, 6)
    for t, v in ((x, other.x), (r, other.r), (w, other.w), (wp, other.wp), (g, other.g)):
        t.copy_(_dev(v))
    graph.replay()
    _check_h(_bits(h), *other.h(1e-5, 1.0, 1.0))
    _check_y(_bits(y), _normed(_bits(h), other.w, 0.0, 1e-5))


def test_no_rows(uw):
    x, w = torch.empty(0, 64, dtype=torch.int16, device="cuda"), torch.zeros(64, dtype=torch.int16, device="cuda")
    uw.block_norm(x, x, w, torch.empty_like(x), torch.empty_like(x), post_weight=w, gate=w)
