"""Workspaces that serve one call after another: what a call leaves in its
workspace does not reach the results of the next, whatever that one's shape."""
import os
import sys

import pytest
import torch

import workloads as wl

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def g(uw):
    from tests import _gpu
    return _gpu


def _normal(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("batch", [2, 3, 8, 15])
def test_chain_does_not_depend_on_the_call_before(g, uw, batch):
    """A chain whose wide and narrow matrices are both split along their columns."""
    dim, inner = 1024, 4096
    mats = [g.Compressed(wl.normal_weights(r, c, 0.02, i)) for i, (r, c) in
            enumerate([(inner, dim), (inner, dim), (dim, inner)])]
    chain = uw.mlp_matrices([(m.desc, m.blob_dev, None, None) for m in mats])
    ws = g.workspace(uw.mlp_workspace_size(chain, batch))
    for seed in (1, 2, 1):
        x = _normal(seed, batch, dim)
        y = torch.empty_like(x)
        uw.mlp_forward(chain, x, y, ws)
        assert uw.check_status(ws) == 0
        gate, up = (torch.from_numpy(m.matmul(x).view("int16")).cuda() for m in mats[:2])
        h = torch.empty_like(gate)
        uw.swiglu(gate, up, h)
        assert (g.host_bits(y.view(torch.int16)) == mats[2].matmul(h)).all()


def test_attention_workspace_serves_both_head_sizes(uw):
    """Heads of 64 and of 128 in turn, prompts long enough that items are joined through the workspace."""
    page, hq, hk, n = 64, 8, 2, 3001
    table = torch.arange(-(-n // page), dtype=torch.int32, device="cuda")[None]
    start, length = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, n], [n]))
    both = {}
    for d in (64, 128):
        pages = torch.zeros(table.shape[1], uw.kv4_page_bytes(hk, d, page), dtype=torch.uint8, device="cuda")
        both[d] = (uw.kv4_cache(pages, table, hk, d, page), _normal(d, n, hq + 2 * hk, d))
    need = max(uw.kv4_workspace_size(c, hq) for c, _ in both.values())
    shared = torch.empty(need, dtype=torch.uint8, device="cuda")
    uw.workspace_init(shared)

    def run(d, ws, tokens):
        cache, qkv = both[d]
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        uw.kv4_append(cache, start, length, None, k, v, None, None, None, ws)
        at = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
        out = torch.full((tokens, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        uw.kv4_attention(cache, at, length, q[:tokens], out, ws, tokens, n)
        assert uw.check_status(ws) == 0
        return out

    for tokens in (n, 1):
        for d in (64, 128, 64, 128):
            own = torch.empty(need, dtype=torch.uint8, device="cuda")
            uw.workspace_init(own)
            assert torch.equal(run(d, shared, tokens), run(d, own, tokens))


@pytest.mark.parametrize("tokens", [1, 3, 15, 40])
def test_layer_steps_do_not_depend_on_the_ones_before(uw, tokens):
    """Projections of 4096 and 1024 rows, which small batches split along their columns."""
    from decoder_layer import DecoderLayer, Sequences
    layer = DecoderLayer(1024, 1024, 16, 8, 128, pages=8, page_size=16, max_tokens=64, max_positions=64, seed=5)
    outs = []
    for seed in (1, 2, 1):
        out, h = layer.forward(_normal(seed, tokens, 1024), None, *Sequences(layer, 1, 64).extend([tokens]))
        layer.check()
        outs.append((out.clone(), h.clone()))
    assert not torch.equal(outs[0][0], outs[1][0])
    assert torch.equal(outs[0][0], outs[2][0]) and torch.equal(outs[0][1], outs[2][1])


@pytest.mark.parametrize("tokens", [129, 161, 299])
def test_layer_takes_every_batch_up_to_its_limit(uw, tokens):
    from decoder_layer import DecoderLayer, Sequences
    layer = DecoderLayer(1024, 1024, 8, 2, 128, pages=24, page_size=16, max_tokens=300, max_positions=300, seed=5)
    out, h = layer.forward(_normal(1, tokens, 1024), None, *Sequences(layer, 1, 300).extend([tokens]))
    layer.check()
    assert torch.isfinite(out.float()).all() and torch.isfinite(h.float()).all()
