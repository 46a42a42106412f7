"""Beam search's selection against a plain one in 64 bits."""
import math

import pytest
import torch

import speculative_decoding_tree_split_gb300 as ta
from oracle import context

pytestmark = pytest.mark.gpu

INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ta.build()
    ta.load()


def check(logits, scores, k, finished=None, eos=None, **kw):
    got = ta.beam_select(logits, scores, k, finished=finished, eos=eos, **kw)
    B, W, _ = logits.shape
    for b in range(B):
        want = context.beams(logits[b].cpu(), scores[b].cpu(),
                             None if finished is None else finished[b].cpu(), eos, k)
        n = len(want)
        assert got[1][b].tolist() == [b * W + w for _, w, _ in want] + [-1] * (k - n)
        assert got[2][b].tolist() == [v for _, _, v in want] + [-1] * (k - n)
        s = got[0][b].double().cpu()
        assert bool((s[n:] == -INF).all())
        if n:
            # fp32 exponentials (2^-21 each, with their arguments) inside the logarithm, and one
            # rounding to fp32 of the score
            ref = torch.tensor([x for x, _, _ in want], dtype=torch.float64)
            assert bool(((s[:n] - ref).abs() <= 2.0 ** -20 + ref.abs() * 2.0 ** -23).all())
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("B,W,V,k", [(1, 1, 1, 1), (2, 1, 5, 9), (3, 4, 63, 4), (1, 4, 8185, 17),
                                     (2, 3, 8192, 16), (1, 2, 8193, 64), (2, 8, 20011, 8),
                                     (1, 64, 301, 64)])
def test_against_64_bits(B, W, V, k, dtype):
    g = torch.Generator("cuda").manual_seed(V + k)
    x = (3 * torch.randn(B, W, V, generator=g, device="cuda")).to(dtype)
    s = -20 * torch.rand(B, W, generator=g, device="cuda")
    check(x, s, k)
    done = torch.rand(B, W, generator=g, device="cuda") < 0.4
    check(x, s, k, finished=done, eos=V // 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties_go_to_the_lowest_place(dtype):
    x = torch.zeros(2, 3, 20000, device="cuda", dtype=dtype)
    x[0, :, 777:] = 1.0
    x[1, 1, 5] = -0.0
    check(x, torch.zeros(2, 3, device="cuda"), 64)
    s = torch.zeros(2, 3, device="cuda")
    s[:, 0] = -1.0
    check(x, s, 16)


def test_values_that_are_no_numbers():
    V = 9000
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn(6, 2, V, generator=g, device="cuda")
    x[0, 0, ::2] = math.nan
    x[0, 1, 5:] = -INF
    x[1, 0] = -INF
    x[1, 1, 3:] = -INF          # three candidates in all
    x[2] = math.nan             # none
    x[3, 0, 17] = INF
    x[3, 1, [40, 41]] = INF     # two that share a beam's whole probability
    x[4] = torch.finfo(torch.float32).min
    s = torch.zeros(6, 2, device="cuda")
    s[5, 0], s[5, 1] = math.nan, -INF
    check(x, s, 8)
    y = x.bfloat16()
    y[4] = torch.finfo(torch.bfloat16).min
    check(y, s, 8)
    done = torch.zeros(6, 2, dtype=torch.bool, device="cuda")
    done[2, 1] = done[1] = done[5] = True
    check(x, s, 3, finished=done, eos=0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_many_logits_of_the_largest_value(dtype):
    """As many as there are wanted, and more, in the first tile: +inf, and the type's largest."""
    g = torch.Generator("cuda").manual_seed(6)
    x = torch.randn(4, 2, 9000, generator=g, device="cuda").to(dtype)
    x[0] = INF
    x[1, 0] = INF
    x[2, 1, ::3] = INF
    x[3, :, 40:] = torch.finfo(dtype).max
    s = torch.tensor([[0.0, -1.0]], device="cuda").expand(4, 2).contiguous()
    for k in (1, 8, 64):
        check(x, s, k)
    check(-x, s, 8)


@pytest.mark.parametrize("order", ["up", "down", "one thread", "one group"])
def test_logits_whose_largest_lie_together(order):
    """The largest logits where one thread or one group of lanes holds all of them."""
    V = 16384
    x = torch.arange(V, device="cuda").float() / 64
    if order == "down":
        x = x.flip(0)
    elif order == "one thread":   # vectors of four logits, 256 threads
        x = x * 0 + torch.arange(V, device="cuda") * 1e-4
        x.view(2, 8, 256, 4)[:, :, 77] += 1000
    elif order == "one group":
        x.view(2, 8, 64, 16)[:, :, 9] += 1000
    for k in (8, 16, 17, 64):
        check(x[None, None].expand(1, 2, V), torch.tensor([[0.0, -0.5]], device="cuda"), k)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_slices_of_a_padded_vocabulary(dtype):
    g = torch.Generator("cuda").manual_seed(9)
    wide = torch.randn(3, 4, 8300, generator=g, device="cuda").to(dtype)
    wide[..., :3] = 1e4
    wide[..., 8290:] = 1e4
    x = wide[:, :, 3:8290]  # neither the rows nor their lengths end on a boundary
    s = torch.zeros(3, 4, device="cuda")
    check(x, s, 5)
    check(x.transpose(0, 1), torch.zeros(4, 3, device="cuda"), 5)
    check(x[:, :1].expand(3, 4, 8287), s - torch.arange(4, device="cuda"), 6)


def test_outputs_given_captured_and_on_another_stream():
    g = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(2, 4, 30000, generator=g, device="cuda")
    s = torch.zeros(2, 4, device="cuda")
    want = [t.clone() for t in check(x, s, 4)]
    outs = [torch.empty_like(t) for t in want]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    ta.beam_select(x, s, 4, scores_out=outs[0], rows_out=outs[1], tokens_out=outs[2],
                   stream=stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ta.beam_select(x, s, 4, scores_out=outs[0], rows_out=outs[1], tokens_out=outs[2])
    x.copy_(x.flip(2))
    graph.replay()
    torch.cuda.synchronize()
    again = ta.beam_select(x, s, 4)
    assert all(torch.equal(a, b) for a, b in zip(outs, again))
    assert not torch.equal(outs[2], want[2])


def test_refusals():
    x, s = torch.zeros(1, 2, 10, device="cuda"), torch.zeros(1, 2, device="cuda")
    done = torch.zeros(1, 2, dtype=torch.bool, device="cuda")
    for bad in (lambda: ta.beam_select(x.cpu(), s, 2),
                lambda: ta.beam_select(x, s.cpu(), 2),
                lambda: ta.beam_select(x, s[:, :1], 2),
                lambda: ta.beam_select(x.transpose(1, 2), s, 2),
                lambda: ta.beam_select(x, s, 2, finished=done),
                lambda: ta.beam_select(x, s, 2, finished=done[:, :1], eos=1)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ta.beam_select(x.double(), s, 2), lambda: ta.beam_select(x, s.half(), 2)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: ta.beam_select(x, s, 0), lambda: ta.beam_select(x, s, 65),
                lambda: ta.beam_select(x, s, 2, finished=done, eos=10),
                lambda: ta.beam_select(torch.zeros(1, 65, 4, device="cuda"),
                                       torch.zeros(1, 65, device="cuda"), 2)):
        with pytest.raises(ta.TreeAttnError):
            bad()
    assert [t.shape for t in ta.beam_select(x[:0], s[:0], 3)] == [(0, 3)] * 3


@pytest.mark.parametrize("W,V,k", [(16, 70000, 16), (8, 200001, 40), (64, 9000, 30)])
def test_many_candidates_and_scores_that_are_nearly_equal(W, V, k):
    """Joins of thousands of candidates, apart by little or by nothing, and far off."""
    g = torch.Generator("cuda").manual_seed(V)
    x = torch.randn(3, W, V, generator=g, device="cuda")
    x[0] = 0.0                                    # all equal in every beam
    x[0, 1] += 1.0
    x[1] = 1e-6 * torch.randint(0, 3, (W, V), generator=g, device="cuda")
    x[2, :, ::7] = torch.finfo(torch.float32).min
    x[2, 3] = 3e38
    s = torch.zeros(3, W, device="cuda")
    s[1] = -1e-6 * torch.arange(W, device="cuda")
    s[2] = -1e30 * torch.arange(W, device="cuda")
    got = ta.beam_select(x, s, k)
    for b in range(3):
        # (the plain one takes too long in Python: its order by sorting)
        y = x[b].double()
        y = y - y.amax(1, keepdim=True)
        y = y - y.exp().sum(1, keepdim=True).log() + s[b].double()[:, None]
        best, at = torch.sort(y.view(-1), descending=True, stable=True)
        rows, tokens = got[1][b].long() - b * W, got[2][b].long()
        mine = y[rows, tokens]
        # scores in order, the same as the best ones to the precision of the sums
        assert float((mine - best[:k]).abs().max()) <= 2.0 ** -20 + float(best[:k].abs().max()) * 2.0 ** -22
        assert len(set(zip(rows.tolist(), tokens.tolist()))) == k
        if b == 0:
            assert rows.tolist() == (at[:k] // V).tolist() and tokens.tolist() == (at[:k] % V).tolist()
