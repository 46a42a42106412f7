"""Bounds of cache pages and the selection by them, against plain definitions."""
import math
import random

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


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make_table(lens, P, r, spare=2):
    pages = [-(-n // P) for n in lens]
    ids = list(range(sum(pages) + spare))
    r.shuffle(ids)
    width = max(pages + [1])
    rows = []
    for n in pages:
        rows.append([ids.pop() for _ in range(n)] + [-1] * (width - n))
    return rows, sum(pages) + spare


def make_keys(n, H, P, d, fp8, g):
    if fp8:
        codes = torch.randint(0, 256, (n, H, P, d), dtype=torch.uint8, device="cuda", generator=g)
        return codes, torch.randint(71, 168, (n, H, P), dtype=torch.uint8, device="cuda", generator=g)
    x = torch.randn(n, H, P, d, device="cuda", generator=g)
    return (x * torch.exp2(torch.randint(-20, 20, (n, H, 1, 1), device="cuda", generator=g))
            ).bfloat16(), None


def values(k, ks):
    return context.row_values(k.cpu(), ks.cpu()) if ks is not None else k.cpu().double()


def check_bounds(k, ks, rows, lens, starts, P):
    n, H, _, d = k.shape
    bounds = torch.randint(-128, 127, (n, H, 2, d), dtype=torch.int8, device="cuda")
    exps = torch.randint(0, 255, (n, H), dtype=torch.uint8, device="cuda")
    want_b, want_e = bounds.cpu().clone(), exps.cpu().clone()
    status = ints([0])
    ta.kv_block_bounds(k, ints(rows), ints(lens), k_scales=ks,
                       starts=None if starts is None else ints(starts), bounds=bounds,
                       bounds_exp=exps, status=status)
    x = values(k, ks)
    for b, L in enumerate(lens):
        a = 0 if starts is None else starts[b]
        for j in range(a // P, -(-L // P)) if a < L else ():
            page = rows[b][j]
            for h in range(H):
                hi, lo, e = context.page_bounds(x[page, h, :min(P, L - j * P)])
                want_b[page, h, 0] = torch.tensor(hi, dtype=torch.int8)
                want_b[page, h, 1] = torch.tensor(lo, dtype=torch.int8)
                want_e[page, h] = e
    assert int(status) == 0
    assert torch.equal(exps.cpu(), want_e) and torch.equal(bounds.cpu(), want_b)
    return bounds, exps


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,P,d", [(1, 16, 64), (2, 32, 128), (3, 64, 64), (2, 64, 128), (1, 128, 128),
                                   (2, 128, 64)])
def test_bounds(H, P, d, fp8):
    r = random.Random(P + d)
    lens = [0, 1, P - 1, P, P + 1, 2 * P + 7, 3 * P - 2]
    rows, n = make_table(lens, P, r)
    g = torch.Generator("cuda").manual_seed(P)
    k, ks = make_keys(n, H, P, d, fp8, g)
    check_bounds(k, ks, rows, lens, None, P)
    check_bounds(k, ks, rows, lens, [0, 1, 3, P - 1, P, P + 3, 3 * P - 3], P)


def test_bounds_of_what_is_no_number():
    k = torch.randn(3, 1, 16, 64, device="cuda")
    k[0, 0, :, 0] = math.nan              # a channel without numbers
    k[0, 0, 3, 1] = math.nan
    k[0, 0, 4, 2], k[0, 0, 5, 3] = math.inf, -math.inf
    k[1, 0, :] = math.nan
    k[1, 0, 0, 7] = -math.inf             # only that
    k[2, 0, :] = 0
    k[2, 0, 9] = 2.0 ** -130
    k[2, 0, 10:] = math.nan               # behind the sequence's end
    check_bounds(k.bfloat16(), None, [[0], [1], [2]], [16, 16, 10], None, 16)
    codes = torch.randint(0, 256, (2, 1, 16, 64), dtype=torch.uint8, device="cuda")
    codes[0] = 0x7f                       # NaN
    codes[1, 0, 0] = 0
    check_bounds(codes, torch.full((2, 1, 16), 167, dtype=torch.uint8, device="cuda"), [[0], [1]],
                 [16, 1], None, 16)


def test_bounds_report_bad_data():
    k = torch.zeros(4, 1, 16, 64, device="cuda", dtype=torch.bfloat16)
    for rows, lens, starts, want in (([[0, 4]], [20], [0], ta.STATUS_BAD_PAGE),
                                     ([[0, -1]], [20], [0], ta.STATUS_BAD_PAGE),
                                     ([[0, 1]], [33], [0], ta.STATUS_BAD_SEQ_LEN),
                                     ([[0, 1]], [-1], [0], ta.STATUS_BAD_SEQ_LEN),
                                     ([[0, 1]], [20], [-1], ta.STATUS_BAD_SEQ_LEN)):
        status = ints([0])
        ta.kv_block_bounds(k, ints(rows), ints(lens), starts=ints(starts), status=status)
        assert int(status) == want


@pytest.mark.parametrize("fp8", [False, True])
def test_bounds_past_32_bits(fp8):
    """The last page's keys lie past 2^32 bytes."""
    n, H, P, d = (4300 if fp8 else 2150), 64, 128, 128
    k = torch.empty(n, H, P, d, device="cuda", dtype=torch.uint8 if fp8 else torch.bfloat16)
    ks = torch.full((n, H, P), 127, dtype=torch.uint8, device="cuda") if fp8 else None
    g = torch.Generator("cuda").manual_seed(2)
    last, _ = make_keys(1, H, P, d, fp8, g)
    k[n - 1] = last[0]
    bounds, exps = ta.kv_block_bounds(k, ints([[n - 1]]), ints([P - 5]), k_scales=ks)
    x = values(k[n - 1:], None if ks is None else ks[n - 1:])
    for h in (0, 41, 63):
        hi, lo, e = context.page_bounds(x[0, h, :P - 5])
        assert bounds[n - 1, h].tolist() == [hi, lo] and int(exps[n - 1, h]) == e


def make_bounds(n, H, d, g, spread=20):
    mid = torch.randint(-60, 60, (n, H, d), device="cuda", generator=g)
    wide = torch.randint(0, 67, (n, H, d), device="cuda", generator=g)
    b = torch.stack([mid + wide, mid - wide], 2).to(torch.int8)
    return b, torch.randint(127, 127 + spread, (n, H), dtype=torch.uint8, device="cuda", generator=g)


def check_select(q, bounds, exps, rows, lens, P, k, first, last, heads=None):
    B, T, Hq, d = q.shape
    H = bounds.shape[1]
    G = Hq // H
    status = ints([0])
    got = ta.select_blocks(q, bounds, exps, ints(rows), ints(lens), k, P, n_first=first, n_last=last,
                           status=status).cpu()
    assert int(status) == 0 and got.shape == (B, T, H, k)
    qc, bc, ec = q.cpu(), bounds.cpu(), exps.cpu()
    for b in range(B):
        pages = rows[b][:-(-lens[b] // P)]
        for t in range(T):
            for h in range(H) if heads is None else heads:
                want = context.choose(qc[b, t, h * G:(h + 1) * G], bc[pages, h], ec[pages, h], k,
                                      first, last)
                assert got[b, t, h].tolist() == want + [-1] * (k - len(want)), (b, t, h)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,G,T,P,k,first,last", [
    (1, 1, 1, 16, 1, 0, 0), (2, 4, 1, 64, 5, 1, 1), (1, 5, 3, 32, 7, 0, 2), (2, 8, 4, 16, 16, 2, 0),
    (1, 3, 17, 128, 9, 1, 1), (1, 16, 2, 16, 4, 0, 1), (1, 13, 64, 16, 3, 1, 1), (3, 2, 9, 64, 30, 30, 0),
    (1, 128, 2, 16, 6, 0, 0)])
def test_select(H, G, T, P, k, first, last, d):
    r = random.Random(H * 1000 + G * 10 + T)
    lens = [0, 1, 40 * P, 33 * P + 1, k * P, (k + 1) * P - 1, 17 * P]
    rows, n = make_table(lens, P, r)
    g = torch.Generator("cuda").manual_seed(G + T)
    bounds, exps = make_bounds(n, H, d, g)
    q = torch.randn(len(lens), T, H * G, d, device="cuda", generator=g).bfloat16()
    check_select(q, bounds, exps, rows, lens, P, k, first, last)


def test_select_ties_go_to_the_lowest_pages():
    P, n = 16, 300
    bounds = torch.full((n, 1, 2, 64), 3, dtype=torch.int8, device="cuda")
    exps = torch.full((n, 1), 120, dtype=torch.uint8, device="cuda")
    exps[[50, 60, 250]] = 121
    rows = [list(range(n))]
    for q in (torch.ones(1, 1, 4, 64, device="cuda"), torch.zeros(1, 1, 4, 64, device="cuda"),
              -torch.ones(1, 1, 4, 64, device="cuda")):
        for k in (1, 2, 5, 64, 299, 300, 301):
            check_select(q.bfloat16(), bounds, exps, rows, [n * P - 3], P, k, 0, 0)
            check_select(q.bfloat16(), bounds, exps, rows, [n * P - 3], P, k, 0, 1)


def test_select_queries_that_are_no_numbers():
    P = 16
    r = random.Random(4)
    lens = [40 * P]
    rows, n = make_table(lens, P, r)
    g = torch.Generator("cuda").manual_seed(8)
    bounds, exps = make_bounds(n, 1, 64, g)
    q = torch.randn(1, 6, 4, 64, device="cuda", generator=g)
    q[0, 0, 1, 3] = math.nan
    q[0, 1, 2, 5], q[0, 1, 0, 6] = math.inf, -math.inf
    q[0, 2] = math.nan
    q[0, 3] *= 2.0 ** 110
    q[0, 4] *= 2.0 ** -120
    q[0, 5] = math.inf
    check_select(q.bfloat16(), bounds, exps, rows, lens, P, 9, 1, 1)
    exps[::2], exps[1::2] = 27, 227  # the whole range of exponents
    check_select(q.bfloat16(), bounds, exps, rows, lens, P, 9, 0, 0)


@pytest.mark.parametrize("nb,T,k", [(3000, 1, 64), (9001, 3, 200), (40000, 2, 4096), (70000, 1, 5),
                                    (262144, 1, 33)])
def test_select_from_many_pages(nb, T, k):
    P = 16
    g = torch.Generator("cuda").manual_seed(nb)
    bounds, exps = make_bounds(nb, 1, 64, g, spread=3)
    rows = [torch.randperm(nb, generator=torch.Generator().manual_seed(1)).tolist()]
    q = torch.randn(1, T, 3, 64, device="cuda", generator=g).bfloat16()
    check_select(q, bounds, exps, rows, [nb * P - 7], P, k, 1, 2)


def test_select_reports_bad_data():
    g = torch.Generator("cuda").manual_seed(1)
    bounds, exps = make_bounds(8, 1, 64, g)
    q = torch.randn(1, 1, 1, 64, device="cuda", generator=g).bfloat16()
    for rows, lens, want in (([[0, 8, 1, 2]], [60], ta.STATUS_BAD_PAGE),
                             ([[0, -1, 1, 2]], [60], ta.STATUS_BAD_PAGE),
                             ([[0, 1, 2, 3]], [65], ta.STATUS_BAD_SEQ_LEN),
                             ([[0, 1, 2, 3]], [-2], ta.STATUS_BAD_SEQ_LEN)):
        status = ints([0])
        ta.select_blocks(q, bounds, exps, ints(rows), ints(lens), 2, 16, status=status)
        assert int(status) == want


def test_select_captured_and_replayed():
    P, lens = 64, [90 * 64, 30 * 64]
    r = random.Random(2)
    rows, n = make_table(lens, P, r)
    g = torch.Generator("cuda").manual_seed(3)
    bounds, exps = make_bounds(n, 2, 128, g)
    q = torch.randn(2, 4, 8, 128, device="cuda", generator=g).bfloat16()
    rows = ints(rows)
    out = torch.empty(2, 4, 2, 8, dtype=torch.int32, device="cuda")
    ta.select_blocks(q, bounds, exps, rows, ints(lens), 8, P, out=out)
    seq = ints(lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ta.select_blocks(q, bounds, exps, rows, seq, 8, P, out=out)
    q.neg_()
    seq.sub_(640)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ta.select_blocks(q, bounds, exps, rows, seq, 8, P))


def test_refusals():
    g = torch.Generator("cuda").manual_seed(1)
    bounds, exps = make_bounds(4, 2, 64, g)
    q = torch.zeros(1, 1, 4, 64, device="cuda", dtype=torch.bfloat16)
    t, s = ints([[0, 1]]), ints([20])
    for kw in (dict(n_select=0), dict(n_select=1), dict(n_select=4097), dict(page_size=24),
               dict(n_first=-1), dict(n_last=2)):
        args = dict(n_select=2, page_size=16)
        args.update(kw)
        with pytest.raises(ta.TreeAttnError):
            ta.select_blocks(q, bounds, exps, t, s, **args)
    with pytest.raises(ta.TreeAttnError):
        ta.select_blocks(q[:, :, :3].contiguous(), bounds, exps, t, s, 2, 16)
    for bad in (lambda: ta.select_blocks(q, bounds.cpu(), exps, t, s, 2, 16),
                lambda: ta.select_blocks(q, bounds[..., :32], exps, t, s, 2, 16),
                lambda: ta.select_blocks(q, bounds, exps[:3], t, s, 2, 16),
                lambda: ta.select_blocks(q, bounds, exps, ints([[0], [1]]), s, 2, 16),
                lambda: ta.select_blocks(q, bounds, exps, t, ints([1, 2]), 2, 16)):
        with pytest.raises(ValueError):
            bad()
    k = torch.zeros(4, 2, 16, 64, device="cuda", dtype=torch.bfloat16)
    codes, sc = k.to(torch.uint8), torch.zeros(4, 2, 16, device="cuda", dtype=torch.uint8)
    with pytest.raises(TypeError):
        ta.kv_block_bounds(codes, t, s)
    with pytest.raises(TypeError):
        ta.kv_block_bounds(k, t, s, k_scales=sc)
    with pytest.raises(ValueError):
        ta.kv_block_bounds(codes, t, s, k_scales=sc[:3])
    with pytest.raises(ValueError):
        ta.kv_block_bounds(k, t, s, bounds=bounds)
    with pytest.raises(ValueError):
        ta.kv_block_bounds(k, t, s, bounds=bounds[..., :32].contiguous(), bounds_exp=exps)
    with pytest.raises(ta.TreeAttnError):
        ta.kv_block_bounds(k[:, :, :8].contiguous(), t, s)
