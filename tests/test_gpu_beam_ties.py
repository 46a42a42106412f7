"""Beams with the same logits and scores tie, whatever addresses their rows begin at, and the
place of a tensor in memory has no part in what is chosen."""
import pytest
import torch

import speculative_decoding_tree_split_gb300 as ta
from oracle import context

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ta.build()
    ta.load()


DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,W,V,k", [(3, 8, 50257, 16), (1, 3, 8193, 9), (20, 4, 8193, 8),
                                     (2, 8, 4099, 8), (6, 5, 131, 7)])
def test_equal_beams_tie_wherever_their_rows_begin(B, W, V, k, dtype):
    for seed in range(4):
        g = torch.Generator("cuda").manual_seed(V + seed)
        one = (3 * torch.randn(B, 1, V, generator=g, device="cuda")).to(dtype)
        x = one.expand(B, W, V).contiguous()  # (rows of an odd length begin anywhere)
        scores = (-5 * torch.rand(B, 1, generator=g, device="cuda")).expand(B, W).contiguous()
        got, rows, tokens = ta.beam_select(x, scores, k)
        for b in range(B):
            # all beams' first candidates, then their second ones (equal logits by token)
            _, at = torch.sort(one[b, 0].float(), descending=True, stable=True)
            y = one[b, 0].float()[at]
            want, i = [], 0
            while len(want) < k:
                same = int((y == y[i]).sum())
                want += [(w, int(v)) for w in range(W) for v in at[i:i + same].tolist()]
                i += same
            assert list(zip((rows[b] - b * W).tolist(), tokens[b].tolist())) == want[:k]
            for j in range(1, k):  # and so do their scores
                if bool(one[b, 0, tokens[b, j]] == one[b, 0, tokens[b, j - 1]]):
                    assert float(got[b, j]) == float(got[b, j - 1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,W,V,k", [(2, 8, 50257, 8), (1, 4, 8192, 8), (1, 2, 30001, 8)])
def test_the_same_at_every_offset(B, W, V, k, dtype):
    g = torch.Generator("cuda").manual_seed(V)
    x = (3 * torch.randn(B, W, V, generator=g, device="cuda")).to(dtype)
    scores = -5 * torch.rand(B, W, generator=g, device="cuda")
    want = ta.beam_select(x, scores, k)
    room = torch.empty(x.numel() + 8 + B * W * 8, dtype=dtype, device="cuda")
    for skip in range(1, 8):
        y = room[skip:skip + x.numel()].view(x.shape)
        y.copy_(x)
        got = ta.beam_select(y, scores, k)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), skip
        z = room[:B * W * (V + skip)].view(B, W, V + skip)[..., skip:]  # rows further apart
        z.copy_(x)
        got = ta.beam_select(z, scores, k)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), skip


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("skip", [0, 1, 3, 5])
def test_largest_logits_with_one_thread_and_numbers_beside_the_rows(dtype, skip):
    """The best of a row where one lane of a warp has them all, at every alignment; what lies
    before a row and behind it is larger still."""
    V, per = 3 * 4096 + 77, 16 // torch.empty(0, dtype=dtype).element_size()
    wide = torch.full((2, 3, V + 24), 60000.0, device="cuda").to(dtype)
    g = torch.Generator("cuda").manual_seed(skip)
    x = torch.randn(2, 3, V, generator=g, device="cuda")
    whole = x[..., :2 * 4096].view(2, 3, 2, 8, 16 // per, 32, per)
    whole[:, :, :, 5, :, 31] += 50  # a lane's vectors, the last of a warp
    whole[:, 1, :, 7, :, 0] += 60
    wide[..., skip:skip + V] = x.to(dtype)
    y = wide[..., skip:skip + V]
    scores = torch.tensor([[0.0, -70.0, -0.25]] * 2, device="cuda")
    got = ta.beam_select(y, scores, 40)
    for b in range(2):
        want = context.beams(y[b].cpu(), scores[b].cpu(), None, None, 40)
        assert got[1][b].tolist() == [b * 3 + w for _, w, _ in want]
        assert got[2][b].tolist() == [v for _, _, v in want]


def test_the_most_candidates():
    """W, K and V at their joint limit, and one token past it."""
    W = k = 64
    V = 131072
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(1, W, V, generator=g, device="cuda")
    s = -torch.rand(1, W, generator=g, device="cuda")
    got, rows, tokens = ta.beam_select(x, s, k)
    y = torch.log_softmax(x[0].double(), -1) + s[0].double()[:, None]
    best, at = torch.sort(y.view(-1), descending=True, stable=True)
    assert float((got[0].double() - best[:k]).abs().max()) <= 2.0 ** -20 + 2.0 ** -23 * float(
        best[:k].abs().max())
    mine = y[rows[0].long(), tokens[0].long()]
    # (order to the rounding of the sums)
    assert float((mine - best[:k]).abs().max()) <= 2.0 ** -20
    with pytest.raises(ta.TreeAttnError):
        ta.beam_select(torch.zeros(1, W, V + 1, device="cuda"), s, k)
