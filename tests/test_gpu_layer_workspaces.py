"""Workspaces that serve one call after another: what a call leaves in its
workspace does not reach the results of the next, whatever that one's shape."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _normal(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


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
