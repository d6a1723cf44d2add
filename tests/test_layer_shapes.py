"""What the binding of the layer operators refuses beyond wrong sizes: tensors of
another rank, of which a call would take the first row only.  On the CPU,
against a stand-in for the library that records which entry points were reached."""
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
