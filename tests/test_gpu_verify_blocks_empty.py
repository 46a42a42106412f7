"""Attention over selected pages: lists of a sequence without tokens."""
import pytest
import torch

import speculative_decoding_tree_split_gb300 as ta

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ta.build()
    ta.load()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("T", [1, 3])
def test_blocks_of_an_empty_sequence_are_reported(T):
    def bf(*shape):
        return torch.zeros(*shape, device="cuda").bfloat16()
    q, k, v = bf(1, T, 2, 64), bf(4, 1, 16, 64), bf(4, 1, 16, 64)
    for row, want in (([-1, -1], 0), ([0, -1], ta.STATUS_BAD_PAGE), ([-1, 7], ta.STATUS_BAD_PAGE),
                      ([-1, -3], ta.STATUS_BAD_PAGE)):
        status = ints([0])
        blocks = ints([[row] if t == T - 1 else [[-1, -1]] for t in range(T)]).view(1, T, 1, 2)
        ta.verify_blocks(q, k, v, ints([[0, 1, 2, 3]]), ints([0]), blocks, bf(1, T, 1, 64),
                         bf(1, T, 1, 64), parents=ints([-1] * T), status=status)
        assert int(status) == want, row
