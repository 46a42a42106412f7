"""Numbers that 32 bits do not hold are refused, not cut."""
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


def test_numbers_past_32_bits():
    t, n, r = ints([[0, 1]]), ints([20]), ints([1, 1, 0, 0])
    big = 1 << 32
    for kw in (dict(reserve=big), dict(reserve=big + 1), dict(page_size=big + 16)):
        args = dict(dict(page_size=16, reserve=0), **kw)
        with pytest.raises(ValueError):
            ta.kv_fork([], t, n, r, ints([0]), **args)
    x, s = torch.zeros(1, 2, 10, device="cuda"), torch.zeros(1, 2, device="cuda")
    done = torch.zeros(1, 2, dtype=torch.bool, device="cuda")
    for eos in (big, big + 5, -big):
        with pytest.raises(ValueError):
            ta.beam_select(x, s, 2, finished=done, eos=eos)
    q = torch.zeros(1, 1, 4, 64, device="cuda", dtype=torch.bfloat16)
    bounds = torch.zeros(4, 2, 2, 64, device="cuda", dtype=torch.int8)
    exps = torch.full((4, 2), 127, device="cuda", dtype=torch.uint8)
    for kw in (dict(page_size=big + 16), dict(n_first=big), dict(n_last=big + 1),
               dict(n_first=-big)):
        args = dict(dict(page_size=16), **kw)
        with pytest.raises(ValueError):
            ta.select_blocks(q, bounds, exps, t, n, 2, **args)
