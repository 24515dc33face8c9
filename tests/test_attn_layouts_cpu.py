"""Layouts of the attention block's tensors, as the binding hands them to the library, and what the library
refuses of them before any device work."""
import pytest
import torch

from partial_activation_sync_caat_b200 import caat as C


def heads4(t):
    return C._heads4(t, "q", torch.bfloat16, -1)[1:]


@pytest.mark.parametrize("shape,to", [((1, 1, 4, 64), (2, 100, 4, 64)), ((4, 64), (1, 100, 4, 64)), ((3, 1, 4, 64), (3, 100, 4, 64)),
                                      ((1, 1, 1, 64), (1, 2, 1, 64)), ((1, 1, 1, 64), (8, 16, 1, 64))])
def test_expanded_tokens_are_refused(shape, to):
    """Strides (0, 0) mean a contiguous tensor to the library, which an expanded one is not."""
    x = torch.zeros(shape, dtype=torch.bfloat16).expand(to)
    assert not x.is_contiguous()
    with pytest.raises(ValueError, match="share memory"):
        heads4(x)


def test_tokens_that_overlap_are_refused():
    x = torch.zeros(4096, dtype=torch.bfloat16).as_strided((2, 4, 2, 64), (1024, 64, 64, 1))
    with pytest.raises(ValueError, match="share memory"):
        heads4(x)


def test_strides_that_are_passed_on():
    x = torch.zeros(2, 5, 4, 64, dtype=torch.bfloat16)
    assert heads4(x) == (0, 0)
    assert heads4(x[:, :, :2]) == (5 * 256, 256)
    assert heads4(x[:, ::2]) == (5 * 256, 512)
    # one token, or one rank: that dimension has no stride to speak of
    assert heads4(x[:1].expand(1, 5, 4, 64)) == (0, 0)
    assert heads4(x[:, :1]) == (5 * 256, 256)
    assert heads4(x[:1, :, 1:]) == (5 * 256, 256)
    assert heads4(torch.zeros(0, 5, 4, 64, dtype=torch.bfloat16)) == (0, 0)
