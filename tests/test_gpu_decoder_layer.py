"""A whole decoder layer from compressed weights (examples/decoder_layer.py):
norm, projection, append, attention, projection, norm and MLP together, against
the same layer in 64 bits with every tensor rounded to BF16 where the layer
rounds it and keys and values quantised as the cache quantises them.

Bound: each of the layer's twelve or so roundings to BF16 is at most 2^-8 of its
value, and a code of a key or value that falls the other way is one step of its
vector's range; both reach the output through averages over at least 256
terms, so the relative error in the 2-norm is taken to stay under 2^-6."""
import os
import sys

import numpy as np
import pytest
import torch

from tests import _kv4 as ref

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

HIDDEN, MLP, HQ, HK, D = 512, 768, 8, 2, 64


def _r(x):
    """Rounded to BF16, as 64-bit values."""
    x = np.asarray(x)
    return ref.f32(ref.bf16(x.astype(np.float32))).astype(np.float64).reshape(x.shape)


def _bits(x):
    return ref.bf16(np.asarray(x, np.float32)).reshape(np.shape(x))


def _norm(x, w, eps):
    return _r(x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w)


class Reference:
    """The layer for one sequence, token after token appended."""

    def __init__(self, layer):
        self.layer = layer
        self.w = {n: ref.f32(m.w).reshape(m.w.shape).astype(np.float64) for n, m in layer.m.items()}
        self.norms = [n.float().cpu().numpy().astype(np.float64) for n in layer.norms]
        self.cos, self.sin = layer.cos.cpu().numpy(), layer.sin.cpu().numpy()
        self.k, self.v = np.zeros((0, HK, D)), np.zeros((0, HK, D))

    def forward(self, x, residual):
        h = x if residual is None else _r(x + residual)
        y = _norm(h, self.norms[0], self.layer.eps)
        qkv = _bits(_r(y @ self.w["qkv"].T)).reshape(len(x), HQ + 2 * HK, D)
        pos = len(self.k) + np.arange(len(x))
        qk = ref.rotate(qkv[:, :HQ + HK], self.cos[pos], self.sin[pos], False)
        self.k = np.concatenate([self.k, ref.value(*ref.quantise(qk[:, HQ:]))])
        self.v = np.concatenate([self.v, ref.value(*ref.quantise(qkv[:, HQ + HK:]))])
        q = ref.f32(qk[:, :HQ]).reshape(len(x), HQ, D).astype(np.float64)
        a = np.zeros((len(x), HQ, D))
        for i in range(HQ):
            s = q[:, i] @ self.k[:, i // (HQ // HK)].T / np.sqrt(D)
            s = np.where(np.arange(len(self.k)) <= pos[:, None], s, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            a[:, i] = p / p.sum(1, keepdims=True) @ self.v[:, i // (HQ // HK)]
        o = _r(_r(a).reshape(len(x), -1) @ self.w["o"].T)
        h2 = _r(h + o)
        y = _norm(h2, self.norms[1], self.layer.eps)
        g, u = _r(y @ self.w["gate"].T), _r(y @ self.w["up"].T)
        return _r(_r(g / (1 + np.exp(-g)) * u) @ self.w["down"].T), h2


def _host(t):
    return t.float().cpu().numpy().astype(np.float64)


def _close(got, want):
    err = np.linalg.norm(_host(got) - want) / np.linalg.norm(want)
    assert err < 2.0 ** -6, err


@pytest.fixture(scope="module")
def layer(uw):
    from decoder_layer import DecoderLayer
    return DecoderLayer(HIDDEN, MLP, HQ, HK, D, pages=40, page_size=16, max_tokens=300, max_positions=256, seed=3)


def _dev(x):
    return torch.from_numpy(ref.bf16(x.astype(np.float32)).view(np.int16)).cuda().view(torch.bfloat16)


def test_prompts_and_tokens_against_64_bits(layer):
    from decoder_layer import Sequences
    rng = np.random.default_rng(0)
    prompts = [130, 1, 40, 17]
    seqs = Sequences(layer, len(prompts), 140)
    refs = [Reference(layer) for _ in prompts]
    cuts = np.cumsum([0] + prompts)
    x = _r(rng.standard_normal((sum(prompts), HIDDEN)))
    out, h = layer.forward(_dev(x), None, *seqs.extend(prompts))
    layer.check()
    for i, r in enumerate(refs):
        want, want_h = r.forward(x[cuts[i]:cuts[i + 1]], None)
        _close(out[cuts[i]:cuts[i + 1]], want)
        _close(h[cuts[i]:cuts[i + 1]], want_h)
    for new in ([1, 1, 1, 1], [1, 3, 1, 2], [1, 1, 1, 1]):   # a step with drafted tokens among single ones
        n = sum(new)
        x, res = _r(rng.standard_normal((n, HIDDEN))), _r(rng.standard_normal((n, HIDDEN)))
        out, h = layer.forward(_dev(x), _dev(res), *seqs.extend(new))
        layer.check()
        at = 0
        for i, r in enumerate(refs):
            want, want_h = r.forward(x[at:at + new[i]], res[at:at + new[i]])
            _close(out[at:at + new[i]], want)
            _close(h[at:at + new[i]], want_h)
            at += new[i]


def test_prompt_at_once_and_token_by_token(layer):
    """The same tokens in one call and one by one: the kernels for many and for few rows, the matmuls of every
    batch size."""
    from decoder_layer import Sequences
    x = _dev(np.random.default_rng(1).standard_normal((90, HIDDEN)))
    whole, _ = layer.forward(x, None, *Sequences(layer, 1, 96).extend([90]))
    seqs = Sequences(layer, 1, 96)
    rows = [layer.forward(x[i:i + 1], None, *seqs.extend([1]))[0] for i in range(90)]
    layer.check()
    _close(torch.cat(rows), _host(whole))


def test_example_runs(uw, monkeypatch, capsys):
    import decoder_layer
    monkeypatch.setattr(sys, "argv", ["decoder_layer.py", "--hidden", "512", "--mlp", "768", "--q-heads", "4",
                                      "--kv-heads", "2", "--prompts", "70,1", "--tokens", "3"])
    decoder_layer.main()
    assert "one token each" in capsys.readouterr().out
