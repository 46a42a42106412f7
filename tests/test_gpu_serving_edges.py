"""Serving operators: broadcast heads and tokens, both ways queries and results move, offsets
past 32 bits, two calls at once.  Tolerances as in test_gpu_prefill."""
import math

import pytest
import torch

import speculative_decoding_tree_split_gb300 as ta
from test_gpu_prefill import check, ints, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ta.build()
    ta.load()


def same(a, b):
    return torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (6, 2, 64)])
def test_one_head_of_keys_and_one_query_for_all(Hq, Hkv, d):
    cu = [0, 70, 71, 330]
    q, k, v = make(330, Hq, Hkv, d, 20)
    k1, v1 = k[:, :1].expand(-1, Hkv, -1), v[:, :1].expand(-1, Hkv, -1)
    out, lse = ta.prefill(q, k1, v1, ints(cu))
    check(q, k1, v1, cu, out, lse)
    q1 = q[:1].expand(330, -1, -1)          # every token asks the same
    out, lse = ta.prefill(q1, k, v, ints(cu))
    check(q1, k, v, cu, out, lse)
    assert same((out, lse), ta.prefill(q1.contiguous(), k, v, ints(cu)))
    q1 = q[:, :1].expand(-1, Hq, -1)        # every head
    out, lse = ta.prefill(q1, k, v, ints(cu))
    check(q1, k, v, cu, out, lse)
    with pytest.raises(ta.TreeAttnError):   # one key for all tokens
        ta.prefill(q, k[:1].expand(330, -1, -1), v, ints(cu))


@pytest.mark.parametrize("Hq,Hkv,d", [(1, 1, 128), (4, 2, 64), (16, 2, 128), (32, 1, 64),
                                      (64, 1, 128), (3, 1, 128)])
def test_queries_as_boxes_and_row_by_row_give_the_same_bits(Hq, Hkv, d):
    # -q at the scale -s is q at the scale s, and goes row by row
    cu = [0, 1, 40, 40, 297, 809]
    q, k, v = make(809, Hq, Hkv, d, 21, "fused")
    s = 1 / math.sqrt(d)
    a = ta.prefill(q, k, v, ints(cu), softmax_scale=s)
    assert same(a, ta.prefill(-q, k, v, ints(cu), softmax_scale=-s))
    check(q, k, v, cu, *a)


def test_results_past_32_bit_offsets():
    # 2^31 elements of q and out are passed at token 262144
    Hq, Hkv, d, n = 64, 8, 128, 205
    cu = list(range(0, 262144 + 2 * n, n))
    N = cu[-1]
    q, k, v = make(N, Hq, Hkv, d, 22)
    assert (N - n) * Hq * d > 2 ** 31
    status = ints([0])
    out, lse = ta.prefill(q, k, v, ints(cu), status=status)
    assert int(status) == 0
    for a in (cu[0], cu[-3], cu[-2]):
        check(q[a:a + n], k[a:a + n], v[a:a + n], [0, n], out[a:a + n], lse[a:a + n])
    again = ta.prefill(-q, k, v, ints(cu), softmax_scale=-1 / math.sqrt(d))
    assert same((out, lse), again)


def test_two_calls_at_once():
    # prompts attended on one stream while another writes, verifies and reads a cache
    cu = ints([0, 500, 1900])
    q, k, v = make(1900, 16, 2, 128, 23)
    want = ta.prefill(q, k, v, cu)
    B, T, Hkv, d, P, n = 2, 5, 2, 128, 64, 1500
    pages = B * 32
    g = torch.Generator("cuda").manual_seed(24)
    rows = [torch.randn(B * n, Hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2)]
    tree = [torch.randn(B, T, Hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2)]
    tq = torch.randn(B, T, 8, d, generator=g, device="cuda").bfloat16()
    bt = ints(list(range(pages))).view(B, 32)
    parents, zero, new = ints([-1, 0, 0, 1, 2]), ints([0, 0]), ints([0, n, 2 * n])

    def step(stream=None):
        cache = [torch.zeros(pages, Hkv, P, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
        cache += [torch.full((pages, Hkv, P), 127, dtype=torch.uint8, device="cuda")
                  for _ in range(2)] + [bt]
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        lens = ta.kv_append_fp8(*cache, zero, new, *rows, stream=stream)
        out = ta.verify_fp8(tq, *cache, lens, *tree, parents=parents, stream=stream)
        back = ta.kv_read_fp8(*cache, new, 2 * n, stream=stream)
        return cache, out + back

    alone = step()[1]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    kept = []
    for _ in range(6):
        kept.append((ta.prefill(q, k, v, cu), step(s)))
    torch.cuda.synchronize()
    for a, (_, b) in kept:
        assert same(a, want)
        assert all(torch.equal(x, y) for x, y in zip(b, alone))
