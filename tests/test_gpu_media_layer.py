"""A decoder layer that takes in images (examples/decoder_layer.py with sections and post_norms): compressed
projection, rotation by axes with append, attention over the prompts' own k and v, norms around the blocks, compressed
MLP, then single tokens over the cache, against the same layer in 64 bits.  The bound is that of
test_gpu_decoder_layer, with two more norms."""
import os
import sys

import numpy as np
import pytest
import torch

from tests import _kv4 as ref
from tests.test_gpu_decoder_layer import D, HIDDEN, HK, HQ, MLP, Reference, _bits, _close, _dev, _host, _norm, _r

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

SECTIONS = (8, 12, 12)


class MediaReference(Reference):
    """The layer for one sequence; k and v of the prompt as they were projected until its attention is done."""

    def __init__(self, layer):
        super().__init__(layer)
        self.post = [n.float().cpu().numpy().astype(np.float64) for n in layer.post]
        self.axis = np.frombuffer(layer.pair_axis, np.uint8)

    def _after(self, i, x):
        """The norm after a block, not rounded."""
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + self.layer.eps) * self.post[i]

    def forward(self, x, residual, pos, whole):
        h = x if residual is None else _r(residual + self._after(0, x))
        y = _norm(h, self.norms[0], self.layer.eps)
        qkv = _bits(_r(y @ self.w["qkv"].T)).reshape(len(x), HQ + 2 * HK, D)
        at, pair = pos[self.axis].T, np.arange(D // 2)
        qk = ref.rotate(qkv[:, :HQ + HK], self.cos[at, pair], self.sin[at, pair], False)
        place = len(self.k) + np.arange(len(x))
        held_k = np.concatenate([self.k, ref.value(*ref.quantise(qk[:, HQ:]))])
        held_v = np.concatenate([self.v, ref.value(*ref.quantise(qkv[:, HQ + HK:]))])
        k, v = held_k, held_v
        if whole:
            k, v = (ref.f32(b).reshape(b.shape).astype(np.float64) for b in (qk[:, HQ:], qkv[:, HQ + HK:]))
        self.k, self.v = held_k, held_v
        q = ref.f32(qk[:, :HQ]).reshape(len(x), HQ, D).astype(np.float64)
        a = np.zeros((len(x), HQ, D))
        for i in range(HQ):
            s = q[:, i] @ k[:, i // (HQ // HK)].T / np.sqrt(D)
            s = np.where(np.arange(len(k)) <= place[:, None], s, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            a[:, i] = p / p.sum(1, keepdims=True) @ v[:, i // (HQ // HK)]
        o = _r(_r(a).reshape(len(x), -1) @ self.w["o"].T)
        h2 = _r(h + self._after(1, o))
        y = _norm(h2, self.norms[1], self.layer.eps)
        g, u = _r(y @ self.w["gate"].T), _r(y @ self.w["up"].T)
        return _r(_r(g / (1 + np.exp(-g)) * u) @ self.w["down"].T), h2


@pytest.fixture(scope="module")
def layer(uw):
    from decoder_layer import DecoderLayer
    return DecoderLayer(HIDDEN, MLP, HQ, HK, D, pages=40, page_size=16, max_tokens=300, max_positions=256, seed=5,
                        sections=SECTIONS, post_norms=True)


def test_prompts_with_images_and_tokens_against_64_bits(layer):
    from decoder_layer import Sequences, media_positions
    rng = np.random.default_rng(0)
    prompts = [130, 1, 40, 17]
    seqs = Sequences(layer, len(prompts), 140)
    refs = [MediaReference(layer) for _ in prompts]
    cuts = np.cumsum([0] + prompts)
    x = _r(rng.standard_normal((sum(prompts), HIDDEN)))
    pos = media_positions(prompts, 3, image=5)
    assert not (pos[1] == pos[2]).all() and not (pos[0] == pos[1]).all()
    out, h = layer.forward(_dev(x), None, *seqs.extend(prompts), pos=pos.cuda(), whole=True)
    layer.check()
    pos = pos.numpy()
    for i, r in enumerate(refs):
        want, want_h = r.forward(x[cuts[i]:cuts[i + 1]], None, pos[:, cuts[i]:cuts[i + 1]], True)
        _close(out[cuts[i]:cuts[i + 1]], want)
        _close(h[cuts[i]:cuts[i + 1]], want_h)
    last = [pos[:, cuts[i]:cuts[i + 1]].max() for i in range(len(prompts))]
    for new in ([1, 1, 1, 1], [1, 3, 1, 2]):
        n, at = sum(new), 0
        x, res = _r(rng.standard_normal((n, HIDDEN))), _r(rng.standard_normal((n, HIDDEN)))
        p = np.concatenate([last[i] + 1 + np.arange(m) for i, m in enumerate(new)]).astype(np.int32)
        p = np.stack([p] * 3)
        last = [a + m for a, m in zip(last, new)]
        out, h = layer.forward(_dev(x), _dev(res), *seqs.extend(new), pos=torch.from_numpy(p).cuda())
        layer.check()
        for i, r in enumerate(refs):
            want, want_h = r.forward(x[at:at + new[i]], res[at:at + new[i]], p[:, at:at + new[i]], False)
            _close(out[at:at + new[i]], want)
            _close(h[at:at + new[i]], want_h)
            at += new[i]


def test_a_graph_of_the_whole_layer(layer):
    """Captured and replayed with other lengths, positions and values: the bits of calls one by one."""
    from decoder_layer import Sequences, media_positions
    prompts = [90, 30]
    x = torch.randn(120, HIDDEN, device="cuda").bfloat16()
    seqs = Sequences(layer, 2, 128)
    args = seqs.extend(prompts)
    pos = media_positions(prompts, 3, image=4).cuda()
    out, h = layer.forward(x, x, *args, pos=pos, whole=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, h = layer.forward(x, x, *args, pos=pos, whole=True)
    other = Sequences(layer, 2, 128)
    again = other.extend([50, 70])
    want_x, want_pos = torch.randn(120, HIDDEN, device="cuda").bfloat16(), media_positions([50, 70], 3, image=3).cuda()
    want, want_h = layer.forward(want_x, want_x, *again, pos=want_pos, whole=True)
    cache, start, length = args[:3]
    for to, of in ((x, want_x), (pos, want_pos), (start, again[1]), (length, again[2])):
        to.copy_(of)
    seqs.table.copy_(other.table)
    graph.replay()
    layer.check()
    assert torch.equal(out, want) and torch.equal(h, want_h)


def test_prompt_attends_to_what_was_projected(layer):
    """With post norms and sections but over the cache: near, and not the same."""
    from decoder_layer import Sequences, media_positions
    x = _dev(np.random.default_rng(1).standard_normal((90, HIDDEN)))
    pos = media_positions([90], 3, image=6).cuda()
    runs = [layer.forward(x, x, *Sequences(layer, 1, 96).extend([90]), pos=pos, whole=w)[0] for w in (True, False)]
    layer.check()
    assert not torch.equal(*runs)
    err = np.linalg.norm(_host(runs[0]) - _host(runs[1])) / np.linalg.norm(_host(runs[0]))
    assert err < 0.5, err


def test_example_runs(uw, monkeypatch, capsys):
    import decoder_layer
    monkeypatch.setattr(sys, "argv", ["decoder_layer.py", "--hidden", "512", "--mlp", "768", "--q-heads", "4",
                                      "--kv-heads", "2", "--prompts", "300,1", "--tokens", "3", "--sections", "16,24,24",
                                      "--post-norms"])
    decoder_layer.main()
    assert "one token each" in capsys.readouterr().out
