"""uw_rmsnorm and uw_rmsnorm_e4m3 against the formula in 64 bits.

Bounds, from the formats: h is one BF16 rounding of a sum (exact match against
fp32 addition).  y is fp32 arithmetic (a sum of d squares in any order, at most
d * 2^-24 off its root's half, a handful of roundings) and one rounding to BF16
(8 significant bits: 2^-8 of the value).  An e4m3 value is within half a step (2^-4 of the value,
or 2^-10 of the scale for the smallest) of y / scale."""
import numpy as np
import pytest
import torch

from tests._kv4 import bf16, f32

pytestmark = pytest.mark.gpu


def _dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda()


def _bits(t):
    return t.cpu().numpy().view(np.uint16)


def _reference(xb, rb, wb, eps):
    x = f32(xb).reshape(xb.shape)
    h = xb if rb is None else bf16(x + f32(rb).reshape(rb.shape))
    f = f32(h).reshape(h.shape).astype(np.float64)
    y = f / np.sqrt((f * f).mean(-1, keepdims=True) + eps) * f32(wb).astype(np.float64)
    return h, y


def _inputs(n, d, seed):
    rng = np.random.default_rng(seed)
    x = bf16(rng.standard_normal((n, d)))
    r = bf16(3 * rng.standard_normal((n, d)))
    w = bf16(1 + 0.2 * rng.standard_normal(d))
    return x, r, w


def _rel(d):
    return 2.0 ** -8 * 1.001 + (d + 16) * 2.0 ** -24


# register rows of a warp (up to 1024) and of a CTA (to 16384) with partly filled last vectors; odd and longer rows
SHAPES = [(1, 8), (9, 64), (3, 264), (17, 512), (5, 1000), (8, 1024), (2, 1032), (257, 4096), (1, 4096), (3, 5120),
          (3, 8192), (2, 14336), (2, 16384), (2, 16392), (1, 1), (4, 7), (5, 1023), (3, 4097), (2, 16383), (1, 40001)]


@pytest.mark.parametrize("n,d", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_bf16_rows(uw, n, d, residual):
    xb, rb, wb = _inputs(n, d, n + d)
    h_ref, y_ref = _reference(xb, rb if residual else None, wb, 1e-5)
    x, w, y = _dev(xb), _dev(wb), _dev(np.full((n, d), 0x7FC0, np.uint16))
    r = _dev(rb) if residual else None
    h = torch.empty_like(x) if residual else None
    uw.rmsnorm(x, w, y, 1e-5, residual=r, residual_out=h)
    torch.cuda.synchronize()
    if residual:
        assert np.array_equal(_bits(h), h_ref)
    err = np.abs(f32(_bits(y)).reshape(n, d) - y_ref)
    assert np.all(err <= _rel(d) * np.abs(y_ref) + 1e-38)


@pytest.mark.parametrize("n,d", SHAPES)
def test_e4m3_rows(uw, n, d):
    xb, rb, wb = _inputs(n, d, 7 * n + d)
    h_ref, y_ref = _reference(xb, rb, wb, 1e-6)
    x, r, w = _dev(xb), _dev(rb), _dev(wb)
    h, scale = torch.empty_like(x), torch.empty(n, dtype=torch.float32, device="cuda")
    q = torch.empty(n, d, dtype=torch.float8_e4m3fn, device="cuda")
    uw.rmsnorm(x, w, q, 1e-6, residual=r, residual_out=h, scale=scale)
    torch.cuda.synchronize()
    assert np.array_equal(_bits(h), h_ref)
    s = scale.cpu().numpy().astype(np.float64)
    s_ref = np.abs(y_ref).max(1) / 448
    assert np.all(np.abs(s - s_ref) <= ((d + 16) * 2.0 ** -24) * s_ref)
    got = q.float().cpu().numpy().astype(np.float64) * s[:, None]
    slack = (d + 16) * 2.0 ** -23
    assert np.all(np.abs(got - y_ref) <= (2.0 ** -4 + slack) * np.abs(y_ref) + 2.0 ** -10 * s[:, None])
    assert np.all(np.abs(q.float().cpu().numpy()).max(1) == 448)


@pytest.mark.parametrize("d,xs,rs,hs,ys,off", [(512, 640, 512, 520, 1024, 0), (4096, 4104, 4096, 8192, 4096, 0),
                                               (512, 513, 515, 512, 514, 0), (1032, 1040, 1040, 1040, 1040, 1),
                                               (7, 9, 8, 10, 7, 3)])
def test_strided_rows(uw, d, xs, rs, hs, ys, off):
    """Rows apart from each other and starting anywhere; what lies between them keeps its bits."""
    n = 5
    xb, rb, wb = _inputs(n, d, d + xs)
    h_ref, y_ref = _reference(xb, rb, wb, 1e-5)

    def spread(bits, stride):
        buf = np.full(off + n * stride + 8, 0x1234, np.uint16)
        view = buf[off:off + n * stride].reshape(n, stride)
        if bits is not None:
            view[:, :d] = bits
        t = _dev(buf)
        return t, t[off:off + n * stride].view(n, stride)[:, :d]

    (_, x), (_, r), (hb, h), (yb, y) = spread(xb, xs), spread(rb, rs), spread(None, hs), spread(None, ys)
    uw.rmsnorm(x, _dev(wb), y, 1e-5, residual=r, residual_out=h)
    torch.cuda.synchronize()
    assert np.array_equal(_bits(h.contiguous()), h_ref)
    err = np.abs(f32(_bits(y.contiguous())).reshape(n, d) - y_ref)
    assert np.all(err <= _rel(d) * np.abs(y_ref))
    for buf, stride in ((hb, hs), (yb, ys)):
        b = _bits(buf)
        gaps = b[off:off + n * stride].reshape(n, stride)[:, d:]
        assert np.all(gaps == 0x1234) and np.all(b[:off] == 0x1234) and np.all(b[off + n * stride:] == 0x1234)


@pytest.mark.parametrize("d", [1, 3, 6, 7, 9, 14, 15, 17, 263, 1018, 1025, 2047, 4099, 8201, 16377, 16384])
@pytest.mark.parametrize("off", [0, 1, 5])
@pytest.mark.parametrize("bits", [16, 8])
def test_rows_alike_that_begin_anywhere(uw, d, off, bits):
    """Rows of all tensors at the same odd distance from 16-byte steps, the weights at another."""
    n = 9
    xb, rb, wb = _inputs(n, d, d + off)
    h_ref, y_ref = _reference(xb, rb, wb, 1e-5)
    stride = {"x": d, "r": d + 8, "h": d + 16, "y": d}

    def spread(name, values, dtype):
        st = stride[name]
        buf = np.full(off + (n - 1) * st + d + 16, 0x34, dtype)
        rows = np.lib.stride_tricks.as_strided(buf[off:], (n, d), (st * buf.itemsize, buf.itemsize))
        if values is not None:
            rows[:] = values
        t = _dev(buf) if dtype == np.uint16 else torch.from_numpy(buf).cuda()
        return t, t[off:].as_strided((n, d), (st, 1))

    (_, x), (_, r), (hb, h) = spread("x", xb, np.uint16), spread("r", rb, np.uint16), spread("h", None, np.uint16)
    yb, y = spread("y", None, np.uint16 if bits == 16 else np.uint8)
    w = _dev(np.concatenate([np.zeros(2, np.uint16), wb]))[2:]
    scale = torch.empty(n, dtype=torch.float32, device="cuda")
    uw.rmsnorm(x, w, y, 1e-5, residual=r, residual_out=h, scale=None if bits == 16 else scale)
    torch.cuda.synchronize()
    assert np.array_equal(_bits(h.contiguous()), h_ref)
    if bits == 16:
        err = np.abs(f32(_bits(y.contiguous())).reshape(n, d) - y_ref)
        assert np.all(err <= _rel(d) * np.abs(y_ref))
    else:
        s = scale.cpu().numpy().astype(np.float64)[:, None]
        got = y.contiguous().view(torch.float8_e4m3fn).float().cpu().numpy() * s
        slack = (d + 16) * 2.0 ** -23
        assert np.all(np.abs(got - y_ref) <= (2.0 ** -4 + slack) * np.abs(y_ref) + 2.0 ** -10 * s)
    for buf, name in ((hb, "h"), (yb, "y")):
        b, st = buf.cpu().numpy(), stride[name]
        used = (off + st * np.arange(n)[:, None] + np.arange(d)).ravel()
        assert np.all(np.delete(b, used) == 0x34)


@pytest.mark.parametrize("d", [512, 4096, 777])
def test_in_place(uw, d):
    """The residual stream updated in place, the norm written over x."""
    xb, rb, wb = _inputs(6, d, d)
    h_ref, y_ref = _reference(xb, rb, wb, 1e-5)
    x, r = _dev(xb), _dev(rb)
    uw.rmsnorm(x, _dev(wb), x, 1e-5, residual=r, residual_out=r)
    torch.cuda.synchronize()
    assert np.array_equal(_bits(r), h_ref)
    assert np.all(np.abs(f32(_bits(x)).reshape(6, d) - y_ref) <= _rel(d) * np.abs(y_ref))


@pytest.mark.parametrize("d", [64, 4096, 333])
def test_zero_and_non_finite_rows(uw, d):
    xb, _, wb = _inputs(5, d, d + 1)
    xb[0] = 0
    xb[1, d // 2] = 0x7F80
    xb[2, d - 1] = 0x7FC1
    xb[4] = bf16(np.float32(1e-30) * f32(xb[4]))   # eps decides; far below BF16's smallest square
    _, y_ref = _reference(xb, None, wb, 1e-5)
    x, w, y = _dev(xb), _dev(wb), torch.empty(5, d, dtype=torch.int16, device="cuda")
    uw.rmsnorm(x, w, y, 1e-5)
    q = torch.empty(5, d, dtype=torch.uint8, device="cuda")
    scale = torch.empty(5, dtype=torch.float32, device="cuda")
    uw.rmsnorm(x, w, q, 1e-5, scale=scale)
    torch.cuda.synchronize()
    got = f32(_bits(y)).reshape(5, d)
    assert np.all(got[0] == 0)
    assert np.isnan(got[1, d // 2]) and np.all(np.delete(got[1], d // 2) == 0)
    assert np.isnan(got[2]).all()
    for i in (3, 4):
        assert np.all(np.abs(got[i] - y_ref[i]) <= _rel(d) * np.abs(y_ref[i]) + 1e-38)
    e = q.view(torch.float8_e4m3fn).float().cpu().numpy()
    s = scale.cpu().numpy()
    assert np.all(e[0] == 0) and s[0] == np.float32(2.0 ** -126)
    assert np.isnan(e[1:3]).all() and np.isnan(s[1:3]).all()
    assert np.isfinite(e[3:]).all() and np.isfinite(s[3:]).all()


def test_no_rows(uw):
    x = torch.empty(0, 64, dtype=torch.int16, device="cuda")
    uw.rmsnorm(x, torch.zeros(64, dtype=torch.int16, device="cuda"), torch.empty_like(x))
