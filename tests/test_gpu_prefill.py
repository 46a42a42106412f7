"""prefill against causal attention written out in 64 bits.

Tolerances.  Let A = sum_j p_j |v_j| / l.  The probabilities enter P.V in bf16
(2^-8 each, at most) and the result is rounded to bf16 once:
    |out - ref| <= 2^-8 (|ref| + A) + 2^-18 max|v|.
Scores are exact products summed in fp32:
    |lse - ref| <= scale 2^-20 max|q| max_j sum|k_j| + 2^-18.
"""
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


def make(N, Hq, Hkv, d, seed=0, layout="dense", gain=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    q, k, v = (torch.randn(N, h, d, generator=g, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
    q = q * gain
    if layout == "fused":
        x = torch.cat([q, k, v], 1)
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if layout == "heads first":
        return tuple(x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
    return q, k, v


def check(q, k, v, cu, out, lse, scale=None):
    N, Hq, d = q.shape
    Hkv = k.shape[1]
    scale = 1 / math.sqrt(d) if scale is None else scale
    for a, b in zip(cu[:-1], cu[1:]):
        n = b - a
        if n == 0:
            continue
        hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
        for h in range(Hq):
            kk, vv = k[a:b, h * Hkv // Hq].double(), v[a:b, h * Hkv // Hq].double()
            x = (q[a:b, h].double() @ kk.T * scale).masked_fill_(hidden, -math.inf)
            top = torch.logsumexp(x, 1)
            p = (x - top[:, None]).exp()
            ref, A = p @ vv, p @ vv.abs()
            tol = 2.0 ** -8 * (ref.abs() + A) + 2.0 ** -18 * vv.abs().max()
            off = (out[a:b, h].double() - ref).abs()
            assert bool((off <= tol).all()), (a, h, float(off.max()))
            lt = (abs(scale) * 2.0 ** -20 * float(q[a:b, h].double().abs().max())
                  * float(kk.abs().sum(1).max()) + 2.0 ** -18)
            assert float((lse[a:b, h].double() - top).abs().max()) <= lt, (a, h)


CASES = [
    # lens, Hq, Hkv, d, layout
    ([1], 1, 1, 64, "dense"),
    ([1, 1, 1], 8, 2, 128, "fused"),
    ([2, 0, 3, 31, 0, 33], 4, 4, 64, "dense"),
    ([127, 128, 129], 4, 1, 128, "dense"),
    ([64, 255, 256, 257], 8, 2, 128, "fused"),
    ([300, 5, 511], 10, 2, 128, "heads first"),      # five query heads to a KV head
    ([513, 1, 700], 7, 1, 64, "fused"),              # seven
    ([1000], 24, 2, 128, "dense"),                   # twelve
    ([140, 70], 66, 1, 64, "dense"),                 # 66: a tile is a few tokens
    ([40, 3], 300, 1, 64, "dense"),                  # more query heads than a tile has rows
    ([2049], 2, 2, 64, "dense"),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_64_bits(i):
    lens, Hq, Hkv, d, layout = CASES[i]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    q, k, v = make(cu[-1], Hq, Hkv, d, i, layout)
    status = ints([0])
    out, lse = ta.prefill(q, k, v, ints(cu), status=status)
    assert int(status) == 0
    check(q, k, v, cu, out, lse)


@pytest.mark.parametrize("gain,scale", [(6.0, None), (1.0, -0.1), (1.0, 0.0)])
def test_wide_scores_and_other_scales(gain, scale):
    cu = [0, 400, 900]
    q, k, v = make(900, 4, 2, 128, 3, gain=gain)
    out, lse = ta.prefill(q, k, v, ints(cu), softmax_scale=scale)
    check(q, k, v, cu, out, lse, scale)


def test_scores_that_keep_rising():
    # every block of keys holds a new maximum, so sums are rescaled each time
    n, d = 1500, 64
    q, k, v = make(n, 2, 1, d, 4)
    q = q.abs() + 0.5
    k = (k.abs() * torch.linspace(0.1, 4, n, device="cuda")[:, None, None]).bfloat16()
    out, lse = ta.prefill(q, k, v, ints([0, n]))
    check(q, k, v, [0, n], out, lse)


@pytest.mark.parametrize("d", [64, 128])
def test_long(d):
    n = 8192 + 77
    q, k, v = make(n, 4, 2, d, 5)
    out, lse = ta.prefill(q, k, v, ints([0, n]))
    check(q, k, v, [0, n], out, lse)


def test_rows_of_no_sequence_are_left_alone_and_reach_nothing():
    # rows before, behind and of refused sequences hold NaN
    cu = [3, 50, 50, 180]
    q, k, v = make(200, 4, 2, 64, 6)
    for x in (q, k, v):
        x[:3] = float("nan")
        x[180:] = float("nan")
    out = torch.full((200, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((200, 4), 7.0, device="cuda")
    ta.prefill(q, k, v, ints(cu), out=out, lse=lse)
    check(q, k, v, cu, out, lse)
    for t in (out, lse):
        assert bool((t[:3] == 7).all()) and bool((t[180:] == 7).all())


def test_nan_and_infinity_stay_with_the_rows_that_see_them():
    cu = [0, 200, 420]
    q, k, v = make(420, 4, 2, 128, 7)
    clean, clean_l = ta.prefill(q, k, v, ints(cu))
    k[150, 1, 3] = float("nan")
    v[300, 0, 5] = float("inf")
    v[310, 1, 6] = float("nan")
    out, lse = ta.prefill(q, k, v, ints(cu))
    assert torch.equal(out[:150], clean[:150]) and torch.equal(lse[:150], clean_l[:150])
    assert torch.equal(out[150:200, :2], clean[150:200, :2])
    assert bool(out[150:200, 2:].isnan().all()) and bool(lse[150:200, 2:].isnan().all())
    assert torch.equal(out[200:300], clean[200:300])
    assert torch.equal(lse[200:], clean_l[200:])
    other = [c for c in range(128) if c != 5]
    assert torch.equal(out[300:, :2][..., other], clean[300:, :2][..., other])
    assert bool((out[300:420, :2, 5] == math.inf).all())
    assert torch.equal(out[200:310, 2:], clean[200:310, 2:])
    assert bool(out[310:, 2:, 6].isnan().all())


@pytest.mark.parametrize("cu", [[0, 40, 30, 100], [0, 50, 101, 100], [-1, 20, 60, 100],
                                [0, 30, 60, 120]])
def test_ranges_out_of_order_are_reported(cu):
    q, k, v = make(100, 2, 1, 64, 8)
    out = torch.full((100, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((100, 2), 7.0, device="cuda")
    status = ints([0])
    ta.prefill(q, k, v, ints(cu), out=out, lse=lse, status=status)
    assert int(status) == 3


def test_graph_replay_other_stream_and_repeated_calls():
    cu = ints([0, 300, 301, 800])
    q, k, v = make(800, 8, 2, 128, 9)
    first = ta.prefill(q, k, v, cu)
    again = ta.prefill(q, k, v, cu)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ta.prefill(q, k, v, cu, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(first[0], got[0])
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ta.prefill(q, k, v, cu, out=out, lse=lse, stream=s)
    cu.copy_(ints([0, 100, 600, 799]))
    want = ta.prefill(q, k, v, cu)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:799], want[0][:799]) and torch.equal(lse[:799], want[1][:799])


def test_the_binding_checks_its_arguments():
    q, k, v = make(20, 4, 2, 64, 10)
    cu = ints([0, 20])
    for a in ((q.float(), k, v, cu), (q, k[:19], v, cu), (q, k, v[:, :1], cu), (q, k, v, cu.long()),
              (q, k[..., :32], v, cu), (q.transpose(1, 2), k, v, cu), (q, k, v, cu[:0])):
        with pytest.raises((ValueError, TypeError)):
            ta.prefill(*a)
    with pytest.raises(ta.TreeAttnError):
        ta.prefill(q[:, :3], k, v, cu)
    with pytest.raises(ValueError):
        ta.prefill(q, k, v, cu, out=torch.empty(20, 4, 32, dtype=torch.bfloat16, device="cuda"))
