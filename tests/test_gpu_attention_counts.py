"""What a call of uw_attention finds in its workspace from the one before: counts of an item's parts that never came to
their end (the call ran out of time) do not mislead it, and its waits with a limit report themselves."""
import pytest
import torch

from tests.test_gpu_attention import Case

pytestmark = pytest.mark.gpu

UW_ERR_TIMEOUT = 6
CALL = 1024          # a call's number and a count share a word: number * 1024 + count


def _words(ws):
    """The calls' number and the counts of parts, a word for each CTA (behind the 256 bytes of the error word)."""
    n = torch.cuda.get_device_properties(0).multi_processor_count
    words = ws[256:256 + 8 * (1 + n)].view(torch.int64)
    return words[:1], words[1:]


@pytest.mark.parametrize("new,hq,hk,d", [([1999, 301, 77], 8, 2, 128), ([2048], 32, 8, 128), ([513, 900], 4, 4, 64)])
@pytest.mark.parametrize("left", [1, 2, 3, 151])
def test_counts_that_a_call_left_behind(uw, new, hq, hk, d, left):
    c = Case(uw, new, new, hq, hk, d, seed=3)
    want = c.run()
    c.check(*want)
    calls, counts = _words(c.ws)
    assert calls.item() == CALL
    parts = counts.clone()
    assert (parts % CALL > 0).any()                # some items lie in parts
    for _ in range(3):
        counts.fill_(calls.item() - CALL + left)   # as of the last call, whichever of its parts came
        got = c.run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert calls.item() == 4 * CALL


@pytest.mark.parametrize("tries", [1, 64, 4096])
def test_a_wait_that_runs_out(uw, tries):
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    uw.workspace_init(ws)
    uw.selftest_attention_wait(ws, tries)
    assert uw.check_status(ws) == UW_ERR_TIMEOUT
    assert uw.check_status(ws) == 0
    L = uw.load()
    assert L.uw_selftest_attention_wait(ws.data_ptr(), 256, 0, None) == 1
    assert L.uw_selftest_attention_wait(ws.data_ptr(), 256, (1 << 22) + 1, None) == 1
    assert L.uw_selftest_attention_wait(ws.data_ptr(), 255, 1, None) == 3
    c = Case(uw, [300, 1], [300, 1], 4, 2, 128)    # the context works on
    c.check(*c.run())
