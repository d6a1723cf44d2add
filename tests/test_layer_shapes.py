"""What the layer operators refuse beyond wrong sizes, on the CPU: tensors of
another rank, of which a call would take the first row only (against a stand-in for the
library that records which entry points were reached), and a softmax scale that
the kernels could not take (the C ABI itself, with addresses that are never read)."""
import ctypes

import pytest
import torch

OK, INVALID, SHAPE, SMALL, UNSUPPORTED = 0, 1, 2, 3, 7


class _Recorder:
    def __init__(self, lib):
        self.calls, self.lib = [], lib

    def __getattr__(self, name):
        if name in ("uw_kv4_page_bytes", "uw_kv4_workspace_size"):
            return getattr(self.lib, name)

        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


@pytest.fixture
def fake(uw, monkeypatch):
    rec = _Recorder(uw.load())
    monkeypatch.setattr(uw, "_lib", rec)
    return rec


def _refused(uw, status, fn, *args, **kw):
    with pytest.raises(uw.UwError) as e:
        fn(*args, **kw)
    assert e.value.status == status


def _bits(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("shape", [(2, 5, 64), (1, 1, 64), (3, 1, 64), (2, 2, 2, 64), (0, 3, 64)])
def test_rmsnorm_takes_rows_and_vectors_only(uw, fake, shape):
    x, w = _bits(*shape), _bits(64)
    q, s = torch.zeros(shape, dtype=torch.uint8), torch.zeros(64)
    _refused(uw, SHAPE, uw.rmsnorm, x, w, _bits(*shape), stream=0)
    _refused(uw, SHAPE, uw.rmsnorm, x, w, _bits(*shape), residual=x, residual_out=x, stream=0)
    _refused(uw, SHAPE, uw.rmsnorm, x, w, q, scale=s, stream=0)
    n = x.numel() // 64
    rows = _bits(n, 64)
    _refused(uw, SHAPE, uw.rmsnorm, rows, w, _bits(*shape), stream=0)
    _refused(uw, SHAPE, uw.rmsnorm, rows, w, _bits(n, 64), residual=x, stream=0)
    assert fake.calls == []
    uw.rmsnorm(x.view(n, 64), w, rows, stream=0)
    name, args = fake.calls.pop()
    assert name == "uw_rmsnorm" and args[7:9] == (n, 64)


def test_rmsnorm_of_a_single_number_is_refused(uw, fake):
    x = torch.zeros((), dtype=torch.bfloat16)
    _refused(uw, SHAPE, uw.rmsnorm, x, _bits(1), x, stream=0)
    assert fake.calls == []


@pytest.mark.parametrize("scale,want", [(2.0 ** 43, UNSUPPORTED), (1e30, UNSUPPORTED), (2.0 ** -127, UNSUPPORTED),
                                        (2.0 ** 42, OK), (2.0 ** -126, OK), (0.0, OK), (1.0, OK), (-0.0, OK)])
def test_softmax_scales(uw, scale, want):
    """No tokens: a scale that is taken needs no device."""
    p = 1 << 20
    cache, rows = uw.Kv4CacheDesc(p, p, 10, 4, 4, 2, 2, 128, 16), uw.Kv4Rows(p, 1024, 128)
    got = uw.load().uw_kv4_attention(ctypes.byref(cache), p, p, 0, rows, 4, rows, None, 1, 100, scale, 1, 0, p, 1 << 40,
                                     None)
    assert got == want


@pytest.fixture
def call(uw):
    """A right call of kv4_append: its arguments by name."""
    d = 64
    cache = uw.kv4_cache(torch.zeros(3, uw.kv4_page_bytes(2, d, 16), dtype=torch.uint8),
                         torch.zeros(2, 4, dtype=torch.int32), 2, d, 16)
    qkv, cos = _bits(5, 8, d), torch.zeros(9, 32)
    return dict(cache=cache, start=torch.zeros(3, dtype=torch.int32), length=torch.zeros(2, dtype=torch.int32),
                q=qkv[:, :4], k=qkv[:, 4:6], v=qkv[:, 6:], q_out=_bits(5, 4, d), cos=cos, sin=cos, ws=torch.zeros(256),
                stream=0)


@pytest.mark.parametrize("left_out", ["q", "q_out", "cos", "sin"])
def test_append_takes_pairs_of_arguments_only_together(uw, fake, call, left_out):
    """q without q_out or cosines without sines: refused, not taken as if neither had been given."""
    uw.kv4_append(**call)
    assert len(fake.calls) == 1
    call[left_out] = None
    _refused(uw, INVALID, uw.kv4_append, **call)
    assert len(fake.calls) == 1


def test_rmsnorm_refuses_other_types_of_the_same_size(uw, fake):
    """16-bit floats that are not BF16, fp32 weights, 8-bit floats that are not e4m3, scales that are not fp32."""
    x, w, y = _bits(4, 64), _bits(64), _bits(4, 64)
    q, s = torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.zeros(4)
    uw.rmsnorm(x, w, y, residual=x, residual_out=y, stream=0)
    uw.rmsnorm(x.view(torch.int16), w.view(torch.int16), y.view(torch.int16), stream=0)  # bits
    for out in (q, q.view(torch.uint8), q.view(torch.int8)):
        uw.rmsnorm(x, w, out, scale=s, stream=0)
    assert len(fake.calls) == 5
    _refused(uw, SHAPE, uw.rmsnorm, x.half(), w, y, stream=0)
    _refused(uw, SHAPE, uw.rmsnorm, x, w, y.half(), stream=0)
    _refused(uw, SHAPE, uw.rmsnorm, x, w, y, residual=x.half(), stream=0)
    _refused(uw, SHAPE, uw.rmsnorm, x, w, y, residual=x, residual_out=x.half(), stream=0)
    _refused(uw, SHAPE, uw.rmsnorm, x, w.float(), y, stream=0)
    _refused(uw, SHAPE, uw.rmsnorm, x, w.half(), y, stream=0)
    _refused(uw, SHAPE, uw.rmsnorm, x, w, q.view(torch.uint8).view(torch.float8_e5m2), scale=s, stream=0)
    _refused(uw, SHAPE, uw.rmsnorm, x, w, q, scale=s.double(), stream=0)
    _refused(uw, SHAPE, uw.rmsnorm, x, w, q, scale=s.int(), stream=0)
    assert len(fake.calls) == 5


def test_cache_calls_refuse_other_types_of_the_same_size(uw, fake, call):
    def changed(name, f):
        return dict(call, **{name: f(call[name])})

    for name, f in (("q", torch.Tensor.half), ("k", torch.Tensor.half), ("v", torch.Tensor.half),
                    ("q_out", torch.Tensor.half), ("cos", torch.Tensor.int), ("sin", torch.Tensor.int),
                    ("start", torch.Tensor.float), ("length", torch.Tensor.float)):
        with pytest.raises(uw.UwError):
            uw.kv4_append(**changed(name, f))
    with pytest.raises(uw.UwError):
        uw.kv4_cache(call["cache"].pages, call["cache"].table.float(), 2, 64, 16)
    c, start, length, ws = (call[n] for n in ("cache", "start", "length", "ws"))
    q, kv = _bits(5, 4, 64), _bits(5, 2, 64)
    _refused(uw, SHAPE, uw.kv4_read, c, start, length, kv.half(), kv, ws, stream=0)
    _refused(uw, SHAPE, uw.kv4_read, c, start, length, kv, kv.half(), ws, stream=0)
    _refused(uw, SHAPE, uw.kv4_attention, c, start, length, q.half(), q, ws, stream=0)
    _refused(uw, SHAPE, uw.kv4_attention, c, start, length, q, q.half(), ws, stream=0)
    _refused(uw, SHAPE, uw.kv4_attention, c, start, length, q, q, ws, lse=torch.zeros(20, dtype=torch.float64), stream=0)
    _refused(uw, SHAPE, uw.kv4_attention, c, start, length, q, q, ws, lse=torch.zeros(40, dtype=torch.bfloat16), stream=0)
    assert fake.calls == []
    uw.kv4_attention(c, start, length, q.view(torch.int16), q, ws, lse=torch.zeros(20), stream=0)
    assert len(fake.calls) == 1


def test_no_tokens_have_no_strides(uw, fake, call):
    """Views of no tokens, whatever their strides, are nothing to do; for tokens they have to be rows."""
    c, start, length, ws = (call[n] for n in ("cache", "start", "length", "ws"))
    odd = lambda n, h: torch.zeros(n, 64, h, dtype=torch.bfloat16).transpose(1, 2)  # noqa: E731
    uw.kv4_append(c, start, length, odd(0, 4), odd(0, 2), odd(0, 2), odd(0, 4), None, None, ws, stream=0)
    uw.kv4_read(c, start, length, odd(0, 2), odd(0, 2), ws, stream=0)
    uw.kv4_attention(c, start, length, odd(0, 4), odd(0, 4), ws, stream=0)
    assert len(fake.calls) == 3
    _refused(uw, INVALID, uw.kv4_read, c, start, length, odd(1, 2), odd(1, 2), ws, stream=0)
