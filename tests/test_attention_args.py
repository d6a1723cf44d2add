"""What uw_attention refuses, before any device work: checked on the CPU by calling the C ABI with addresses that
are never read, and the Python binding with tensors of the wrong shape, type, stride or place."""
import ctypes

import pytest
import torch

OK, INVALID, SHAPE, SMALL, UNSUPPORTED = 0, 1, 2, 3, 7
P = 1 << 20      # stands for an aligned device address


def _rows(uw, dev=P, ts=1024, hs=128):
    return uw.Kv4Rows(dev, ts, hs)


def test_workspace_size(uw):
    n, fn = ctypes.c_size_t(), uw.load().uw_attention_workspace_size
    sizes = []
    for dim in (64, 128):
        assert fn(dim, ctypes.byref(n)) == OK and n.value > 256
        sizes.append(n.value)
        assert uw.attention_workspace_size(dim) == n.value
    assert sizes[0] < sizes[1]
    assert fn(64, None) == INVALID and fn(0, ctypes.byref(n)) == SHAPE and fn(96, ctypes.byref(n)) == UNSUPPORTED


def test_arguments(uw):
    def call(**change):
        a = dict(start=P, kstart=P, seqs=2, n=3, keys=5, q=_rows(uw), hq=4, k=_rows(uw), v=_rows(uw), hk=2, d=128,
                 out=_rows(uw), lse=None, scale=0.0, causal=1, window=0, ws=P, size=1 << 40)
        a.update(change)
        return uw.load().uw_attention(*a.values(), None)

    bad = _rows(uw, P + 8)
    for change, want in ((dict(start=None), INVALID), (dict(start=P + 2), INVALID), (dict(kstart=P + 1), INVALID),
                         (dict(seqs=-1), INVALID), (dict(n=-1), INVALID), (dict(keys=-1), INVALID), (dict(kstart=None), SHAPE),
                         (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(out=None), INVALID),
                         (dict(q=bad), INVALID), (dict(k=bad), INVALID), (dict(v=bad), INVALID), (dict(out=bad), INVALID),
                         (dict(k=_rows(uw, 0)), INVALID), (dict(v=_rows(uw, P, 4)), INVALID),
                         (dict(q=_rows(uw, P, 1024, -128)), INVALID), (dict(k=_rows(uw, P, 0)), UNSUPPORTED),
                         (dict(v=_rows(uw, P, 0)), UNSUPPORTED), (dict(hq=0), SHAPE), (dict(hk=0), SHAPE), (dict(hq=5), SHAPE),
                         (dict(hq=-2, hk=-1), SHAPE), (dict(d=0), SHAPE), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
                         (dict(hq=1 << 18), UNSUPPORTED), (dict(n=1 << 31), UNSUPPORTED), (dict(keys=1 << 31), UNSUPPORTED),
                         (dict(n=1 << 30, hq=16, hk=1), UNSUPPORTED), (dict(lse=P + 2), INVALID), (dict(window=-1), INVALID),
                         (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
                         (dict(scale=3.3e38), UNSUPPORTED), (dict(scale=1e-45), UNSUPPORTED), (dict(ws=None), INVALID),
                         (dict(ws=P + 16), INVALID), (dict(size=uw.attention_workspace_size(128) - 1), SMALL),
                         (dict(n=0), OK), (dict(seqs=0), OK), (dict(seqs=0, start=None), OK),
                         (dict(n=0, start=None, kstart=None, keys=0), OK)):
        assert call(**change) == want, change


def test_tensors(uw):
    q, k = torch.zeros(7, 4, 64, dtype=torch.bfloat16), torch.zeros(7, 2, 64, dtype=torch.bfloat16)
    start = torch.tensor([0, 3, 7], dtype=torch.int32)
    good = dict(q=q, k=k, v=k, out=q, start=start, ws=torch.zeros(256, dtype=torch.uint8))
    for change, want in ((dict(q=q[0]), SHAPE), (dict(k=k[0]), SHAPE), (dict(v=q), SHAPE), (dict(v=k[:6]), SHAPE),
                         (dict(out=k), SHAPE), (dict(q=q.half()), SHAPE), (dict(k=k.float()), SHAPE),
                         (dict(k=torch.zeros(7, 2, 128, dtype=torch.bfloat16)), SHAPE),
                         (dict(v=k.transpose(1, 2).contiguous().transpose(1, 2)), INVALID), (dict(start=start.long()), SHAPE),
                         (dict(start=start[None]), SHAPE), (dict(start=torch.zeros(6, dtype=torch.int32)[::2]), SHAPE),
                         (dict(start=start[:0]), SHAPE), (dict(kv_start=start[:2]), SHAPE), (dict(kv_start=start.long()), SHAPE),
                         (dict(lse=torch.zeros(7, 4).double()), SHAPE), (dict(lse=torch.zeros(7, 3)), SMALL),
                         (dict(lse=torch.zeros(4, 7).t()), SMALL), ({}, INVALID)):   # the last: not on the GPU
        with pytest.raises(RuntimeError) as e:
            uw.attention(**{**good, **change})
        assert e.value.status == want, change
