"""verify_fp8 where the queries of one node, or of one head of a group, are far
larger than the others': every row has the bits that its own queries give it.
Tolerances as in test_gpu_verify_fp8_sinks, with max|q| that of the row."""
import pytest
import torch

import speculative_decoding_tree_split_gb300 as ta
from test_gpu_verify_fp8_sinks import cache_of, close, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ta.build()
    ta.load()


@pytest.mark.parametrize("T,G,d", [(1, 4, 128), (6, 3, 64), (12, 4, 128), (8, 8, 128),
                                   (16, 5, 128), (16, 8, 64), (33, 4, 128)])
@pytest.mark.parametrize("gain", [2.0 ** 12, 2.0 ** 60, float("inf"), float("nan")])
def test_large_queries_leave_the_other_rows_alone(T, G, d, gain):
    B, L, Hkv = 2, 4096, 2
    g = torch.Generator("cuda").manual_seed(T * G)

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    k, v = rnd(B * L, Hkv, d).bfloat16(), (rnd(B * L, Hkv, d) + 0.5).bfloat16()
    cache, lens, cu = cache_of(B, L, Hkv, d, 64, k, v)
    q, tk, tv = (rnd(B, T, h, d).bfloat16() for h in (Hkv * G, Hkv, Hkv))
    q[:, T // 2, G // 2] *= gain       # a head of the first group, of one node
    q[:, T - 1, 2 * G - 1, 5] *= gain  # an element of the last row
    small = torch.ones(T, Hkv * G, dtype=torch.bool, device="cuda")
    small[T // 2, G // 2] = small[T - 1, 2 * G - 1] = False
    parents = ints(list(range(-1, T - 1)))
    status = ints([0])
    out, lse = ta.verify_fp8(q, *cache, lens, tk, tv, parents=parents, status=status)
    ck, cv = ta.kv_read_fp8(*cache, cu, B * L, status=status)
    assert int(status) == 0
    see = torch.ones(T, T, dtype=torch.bool, device="cuda").tril()
    for b in range(B):
        s = slice(b * L, (b + 1) * L)
        calm = torch.where(small[..., None], q[b], 0)  # what is compared
        o = torch.where(small[..., None], out[b], 0)
        x = torch.where(small, lse[b], 0)
        with_zero, zero_l = zero_rows(ck[s], cv[s], tk[b], tv[b], see, small, d)
        close(torch.where(small[..., None], o, with_zero), torch.where(small, x, zero_l), calm,
              ck[s], cv[s], tk[b], tv[b], see)


def zero_rows(k, v, tk, tv, see, small, d):
    """What rows of zero queries give (those that are left out above)."""
    from test_gpu_verify_fp8_sinks import attend
    q = torch.zeros(*small.shape, d, dtype=torch.bfloat16, device="cuda")
    out, lse, _, _ = attend(q, k, v, tk, tv, see)
    return out, lse
