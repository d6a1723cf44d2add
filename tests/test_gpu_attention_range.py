"""uw_attention at the end of its documented range: sums of many tiles whose scores lie far above the first keys'.

The first 32 keys score 0, all others 22.75, so a tile adds 128 e^22.75 (2^39.8) times its values to a sum that is kept
relative to the first keys: 600 of them pass 2^49, and values near 2^80 would pass fp32's range with it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

KEYS, HIGH = 600 * 128, 22.75


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [1.5 * 2.0 ** 79, -1.9921875 * 2.0 ** 79, 1.0])
def test_many_tiles_above_the_first_keys(uw, d, value):
    # as many heads as the GPU has SMs, all of one key and value head's data: a CTA takes a whole head
    heads = torch.cuda.get_device_properties(0).multi_processor_count
    q = torch.zeros(1, heads, d, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(KEYS, 1, d, dtype=torch.bfloat16, device="cuda")
    v = torch.full((KEYS, 1, d), value, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 8
    k[32:, 0, 0] = HIGH
    ws = torch.empty(uw.attention_workspace_size(d), dtype=torch.uint8, device="cuda")
    uw.workspace_init(ws)
    out, lse = torch.empty_like(q), torch.empty(1, heads, device="cuda")
    start, kv_start = torch.tensor([[0, 1], [0, KEYS]], dtype=torch.int32).cuda()
    uw.attention(q, k.expand(KEYS, heads, d), v.expand(KEYS, heads, d), out, start, ws, kv_start=kv_start, scale=0.125,
                 causal=False, lse=lse)
    assert uw.check_status(ws) == 0
    # a probability's rounding and the output's, 2^-8 each; sums of 600 tiles in fp32 are far below the remainder
    off = (out.double() / value - 1).abs()
    assert (off <= 2.0 ** -7 * 1.01).all(), off.max().item()
    want = torch.log(torch.tensor(32 + (KEYS - 32) * 2.718281828459045 ** HIGH, dtype=torch.float64)).item()
    assert ((lse.double() - want).abs() <= (KEYS / 64 + 64) * 2.0 ** -24 + want * 2.0 ** -21 + 2.0 ** -20).all()
