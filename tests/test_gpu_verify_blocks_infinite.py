"""Attention over selected pages where a value is infinite: rows that see one such value get
that infinity in its channel, rows that see both signs no number, others neither."""
import math

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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,G", [(1, 1), (1, 4), (4, 4)])
def test_infinite_values_of_pages(T, G, d):
    P, n = 16, 8
    g = torch.Generator("cuda").manual_seed(T + d)

    def bf(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()
    q, k, v = bf(1, T, G, d), bf(n, 1, P, d), bf(n, 1, P, d)
    tk, tv = bf(1, T, 1, d), bf(1, T, 1, d)
    blocks = ints([[1, 2, 3], [1, 3, 4], [2, 3, 5], [3, 4, 6]][:T]).view(1, T, 1, 3)
    args = (ints([list(range(n))]), ints([n * P]), blocks, tk, tv)
    parents = ints([-1] * T)
    before, l0 = ta.verify_blocks(q, k, v, *args, parents=parents)
    v[1, 0, 5, 7] = math.inf     # tokens 0 and 1
    v[2, 0, 3, 9] = -math.inf    # tokens 0 and 2
    v[1, 0, 1, 20] = math.inf    # both signs: tokens 0 and 1
    v[1, 0, 2, 20] = -math.inf
    after, l1 = ta.verify_blocks(q, k, v, *args, parents=parents)
    assert torch.equal(l0, l1)
    for t in range(T):
        has = blocks[0, t, 0].tolist()
        hit = set()
        if 1 in has:
            assert bool((after[0, t, :, 7] == math.inf).all())
            assert bool(after[0, t, :, 20].isnan().all())
            hit |= {7, 20}
        if 2 in has:
            assert bool((after[0, t, :, 9] == -math.inf).all())
            hit.add(9)
        keep = [i for i in range(d) if i not in hit]
        a, b = before[0, t][:, keep].double(), after[0, t][:, keep].double()
        # (sums in another order: at most a step of bf16)
        assert bool(((a - b).abs() <= a.abs() * 2.0 ** -7).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_infinite_values_of_tree_tokens(fp8):
    P, d, T, G, n = 16, 64, 3, 4, 4
    g = torch.Generator("cuda").manual_seed(2)

    def bf(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()
    q, tk, tv = bf(1, T, G, d), bf(1, T, 1, d), bf(1, T, 1, d)
    scales = {}
    if fp8:
        k, v = (torch.randint(0, 0x70, (n, 1, P, d), dtype=torch.uint8, device="cuda", generator=g)
                for _ in "kv")
        scales = {s: torch.full((n, 1, P), 119, dtype=torch.uint8, device="cuda")
                  for s in ("k_scales", "v_scales")}
    else:
        k, v = bf(n, 1, P, d), bf(n, 1, P, d)
    tv[0, 1, 0, 11] = -math.inf  # tokens 1 and 2 see it
    tv[0, 2, 0, 30] = math.inf   # token 2
    out, _ = ta.verify_blocks(q, k, v, ints([[0, 1, 2, 3]]), ints([n * P]),
                              ints([[0, 1], [1, 2], [2, 3]]).view(1, T, 1, 2), tk, tv,
                              parents=ints([-1, 0, 1]), **scales)
    assert int(out.isnan().sum()) == 0
    assert bool((out[0, 1:, :, 11] == -math.inf).all())
    assert bool((out[0, 2, :, 30] == math.inf).all())
    assert int(out.isinf().sum()) == 3 * G
