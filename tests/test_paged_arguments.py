"""Arguments of the paged-cache binding that the kernels must never see, and those
that they have to take: nothing here reaches a GPU."""
import pytest
import torch

from sparse_attention_indexer_dsa_gb300 import paged

CPU = torch.device("cpu")


def _tokens(t, heads=4, head_dim=64):
    return paged._tokens(t, "k", CPU, (torch.bfloat16,), heads, head_dim)


def test_token_strides():
    """The stride handed on is one that the kernel can walk without leaving the tensor: 0 (packed) only
    where the tokens are packed."""
    base = torch.zeros((8, 6, 64), dtype=torch.bfloat16)
    t = base[:, :4].contiguous()
    assert _tokens(t) == (t.data_ptr(), 0)
    assert _tokens(base[:, 2:]) == (base[:, 2:].data_ptr(), 6 * 64)
    assert _tokens(base[:1, 2:]) == (base[:1, 2:].data_ptr(), 0)          # one token has no next one
    one = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    assert _tokens(one.expand(1, 4, 64)) == (one.data_ptr(), 0)
    assert _tokens(base[:0, 2:])[1] == 0


@pytest.mark.parametrize("view", [
    lambda: torch.zeros((1, 4, 64), dtype=torch.bfloat16).expand(8, 4, 64),
    lambda: torch.zeros((4, 64), dtype=torch.bfloat16).expand(2, 4, 64),
    lambda: torch.zeros(64 * 32, dtype=torch.bfloat16).as_strided((8, 4, 64), (64, 64, 1)),
    lambda: torch.zeros((8, 1, 64), dtype=torch.bfloat16).expand(8, 4, 64),
    lambda: torch.zeros((8, 64, 4), dtype=torch.bfloat16).transpose(1, 2),
])
def test_tokens_that_share_memory_are_refused(view):
    with pytest.raises(ValueError):
        _tokens(view())


def test_one_head_expanded_over_tokens_is_refused():
    with pytest.raises(ValueError):
        _tokens(torch.zeros((1, 1, 64), dtype=torch.bfloat16).expand(5, 1, 64), heads=1)
