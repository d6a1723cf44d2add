"""The shape of uw_attention's statistics in the Python binding: rows of heads, not heads of rows."""
import pytest
import torch

INVALID, SHAPE, SMALL = 1, 2, 3


def test_shape_of_the_statistics(uw):
    q, k = torch.zeros(7, 4, 64, dtype=torch.bfloat16), torch.zeros(7, 2, 64, dtype=torch.bfloat16)
    good = dict(q=q, k=k, v=k, out=q, start=torch.tensor([0, 3, 7], dtype=torch.int32), ws=torch.zeros(256, dtype=torch.uint8))
    for lse, want in ((torch.zeros(4, 7), SHAPE), (torch.zeros(28, 1), SHAPE), (torch.zeros(7, 4, 1), SHAPE),
                      (torch.zeros(14, 2), SHAPE), (torch.zeros(7, 3), SMALL),
                      # taken (and then not on the GPU): rows of heads, more of them than tokens, or all in a line
                      (torch.zeros(7, 4), INVALID), (torch.zeros(9, 4), INVALID), (torch.zeros(28), INVALID),
                      (torch.zeros(1, 7, 4), INVALID)):
        with pytest.raises(RuntimeError) as e:
            uw.attention(**good, lse=lse)
        assert e.value.status == want, tuple(lse.shape)
    # one head, or one token: either order is the same
    one = dict(good, q=q[:, :1], k=k[:, :1], v=k[:, :1], out=q[:, :1])
    few = dict(good, q=q[:1], k=k[:1], v=k[:1], out=q[:1])
    for args, lse in ((one, torch.zeros(1, 7)), (one, torch.zeros(7, 1)), (few, torch.zeros(4, 1)), (few, torch.zeros(1, 4))):
        with pytest.raises(RuntimeError) as e:
            uw.attention(**args, lse=lse)
        assert e.value.status == INVALID, tuple(lse.shape)
