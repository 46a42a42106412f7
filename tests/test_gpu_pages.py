"""Copying, forking and compacting the pages of a cache, against plain loops."""
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


def make_pools(n, g):
    """Pools of every kind of page size: multiples of 16 bytes and odd ones, short
    and longer than what a warp moves at a time, one that starts off a boundary."""
    def rand(*shape):
        return torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)
    off = rand(n * 48 + 8)[8:].view(n, 48)
    return [rand(n, 2, 16, 64).view(torch.int16), rand(n, 2, 16), rand(n, 5), rand(n, 3, 1367),
            rand(n, 24, 512), off]


def moved(pools, moves):
    out = []
    for p in pools:
        q = p.clone()
        for a, z in moves:
            q[z] = p[a]
        out.append(q)
    return out


def same(pools, want):
    return all(torch.equal(a, b) for a, b in zip(pools, want))


def test_copies_skip_and_count():
    n = 40
    g = torch.Generator("cuda").manual_seed(1)
    pools = make_pools(n, g)
    src = [3, -1, 7, 7, 11, 39, 0]
    dst = [20, 21, 22, 23, -1, 24, 25]
    for count, upto in ((None, 7), (ints([4]), 4), (ints([0]), 0), (ints([99]), 7), (ints([-3]), 0)):
        live = [p.clone() for p in pools]
        status = ints([0])
        ta.kv_copy_pages(live, ints(src), ints(dst), count=count, status=status)
        want = moved(pools, [(a, z) for a, z in zip(src[:upto], dst[:upto]) if a >= 0 and z >= 0])
        assert same(live, want) and int(status) == 0
    live = [p.clone() for p in pools]
    status = ints([0])
    ta.kv_copy_pages(live, ints([n, 2, 5]), ints([1, -2, 30]), status=status)
    assert same(live, moved(pools, [(5, 30)])) and int(status) == ta.STATUS_BAD_PAGE
    ta.kv_copy_pages([], ints([1]), ints([2]))
    ta.kv_copy_pages(pools, ints([]), ints([]))


def test_more_pools_than_one_launch_takes():
    g = torch.Generator("cuda").manual_seed(2)
    pools = [torch.randint(0, 99, (6, 32), dtype=torch.uint8, device="cuda", generator=g)
             for _ in range(250)]
    want = moved(pools, [(1, 4), (2, 5)])
    ta.kv_copy_pages(pools, ints([1, 2]), ints([4, 5]))
    assert same(pools, want)


def test_copies_past_32_bits():
    """A pool of 5 GB: the last page's bytes lie past 2^32."""
    n = 40000
    pool = torch.empty(n, 131072, dtype=torch.uint8, device="cuda")
    pool[n - 1].copy_(torch.arange(131072, device="cuda") % 251)
    pool[3] = 7
    pool[n - 2] = 1
    ta.kv_copy_pages([pool], ints([n - 1, 3]), ints([0, n - 2]))
    assert torch.equal(pool[0], pool[n - 1]) and bool((pool[n - 2] == 7).all())


def random_state(r, rows, P, width, num_pages, share=0.5, extra=0):
    """A table whose rows share full pages now and then (and once in a while a
    partly filled one), lengths of every kind, pages reserved behind some."""
    ids = list(range(num_pages))
    r.shuffle(ids)
    refs, table, lens = [0] * num_pages, [], []
    for i in range(rows):
        L = r.choice([0, 1, P - 1, P, P + 1, r.randrange(0, (width - 1) * P)])
        L = min(L, (width - 1) * P)
        mapped = min(width, -(-L // P) + r.choice([0, 0, 1, 2]))
        row = []
        if table and r.random() < share:
            other = r.randrange(len(table))
            common = min(lens[other] // P, L // P)
            row = table[other][:common]
            if r.random() < 0.3 and lens[other] == L and common < mapped and table[other][common] >= 0:
                row = row + [table[other][common]]  # a partly filled page in two rows
        while len(row) < mapped and ids:
            row.append(ids.pop())
        L = min(L, len(row) * P)
        for p in row:
            refs[p] += 1
        table.append(row + [-1] * (width - len(row)))
        lens.append(L)
    for _ in range(extra):  # pages that something else of the caller's holds
        if ids:
            refs[ids.pop()] += 1
    return table, lens, refs


def check_fork(table, lens, refs, src, reserve, P, pools, one=None):
    t0, r0 = ints(table).view(len(table), len(table[0])), ints(refs)
    status = ints([0])
    before = [p.clone() for p in pools]
    got = ta.kv_fork(pools, t0, ints(lens), r0, ints(src), P,
                     reserve=ints(reserve) if one is None else one, status=status)
    want_t, want_l, want_r, moves, short = context.fork(table, lens, refs, src, reserve, P)
    assert got[0].tolist() == want_t
    assert got[1].tolist() == want_l and got[2].tolist() == want_r
    assert int(status) == (ta.STATUS_NO_PAGE if short else 0)
    assert torch.equal(t0, ints(table).view(t0.shape)) and torch.equal(r0, ints(refs))
    assert same(pools, moved(before, moves))
    return got


@pytest.mark.parametrize("seed", range(8))
@pytest.mark.parametrize("rows,out,P,width,num_pages",
                         [(1, 4, 16, 6, 64), (9, 23, 32, 9, 200), (70, 300, 16, 70, 20000),
                          (5, 0, 64, 5, 40), (33, 65, 128, 33, 1000), (16, 16, 16, 90, 2048),
                          (16, 16, 16, 90, 2049), (3, 16, 32, 40, 33), (16, 5, 128, 2, 31)])
def test_fork_against_loops(rows, out, P, width, num_pages, seed):
    r = random.Random(seed * 100 + rows)
    g = torch.Generator("cuda").manual_seed(seed)
    table, lens, refs = random_state(r, rows, P, width, num_pages, extra=3)
    src = [r.choice([-1, -2, r.randrange(rows), r.randrange(rows)]) for _ in range(out)]
    pools = make_pools(num_pages, g) if num_pages <= 1000 else [
        torch.randint(0, 256, (num_pages, 32), dtype=torch.uint8, device="cuda", generator=g)]
    if seed % 2:
        reserve = [min(r.choice([-2, 0, 1, P, 3 * P + 1]), width * P - (lens[p] if p >= 0 else 0))
                   for p in src]
        check_fork(table, lens, refs, src, reserve, P, pools)
    else:
        one = min([r.choice([0, 1, P])] + [width * P - (lens[p] if p >= 0 else 0) for p in src])
        check_fork(table, lens, refs, src, [one] * out, P, pools, one=one)


@pytest.mark.parametrize("num_pages", [500, 3000])
def test_fork_of_more_pools_than_one_launch_takes_and_long_reserves(num_pages):
    g = torch.Generator("cuda").manual_seed(12)
    table = [list(range(10, 110)) + [-1] * 100, list(range(110, 113)) + [-1] * 197]
    lens, refs = [16 * 20 + 3, 47], [0] * num_pages
    for p in range(10, 113):
        refs[p] = 1
    pools = [torch.randint(0, 99, (num_pages, 16), dtype=torch.uint8, device="cuda", generator=g)
             for _ in range(250)]
    check_fork(table, lens, refs, [0, 1, 0, -2], [16 * 150, 1, 40, 16 * 33], 16, pools)


def test_fork_identity_release_and_new_rows():
    g = torch.Generator("cuda").manual_seed(5)
    table, lens, refs = [[4, 2, -1], [4, 7, 9], [1, -1, -1]], [20, 33, 16], [0] * 12
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] += 1
    pools = make_pools(12, g)
    got = check_fork(table, lens, refs, [0, 1, 2], [0, 0, 0], 16, pools)
    assert got[2].tolist() == refs  # nothing changes
    check_fork(table, lens, refs, [1], [0], 16, pools)          # two rows end
    check_fork(table, lens, refs, [-2, -1, 0], [17, 9, 0], 16, pools)
    status = ints([0])  # no rows yet
    got = ta.kv_fork(pools, torch.empty(0, 3, dtype=torch.int32, device="cuda"), ints([]),
                     ints([0, 2] + [0] * 10), ints([-2, -1, -2]), 16, reserve=ints([20, 0, 1]),
                     status=status)
    assert [t.tolist() for t in got] == [[[0, 2, -1], [-1] * 3, [3, -1, -1]], [0, 0, 0],
                                         [1, 2, 1, 1] + [0] * 8] and int(status) == 0


def test_fork_without_enough_pages():
    g = torch.Generator("cuda").manual_seed(6)
    table, lens = [[0, 1, 2], [3, -1, -1]], [40, 5]
    refs = [1, 1, 1, 1, 0, 0]
    pools = make_pools(6, g)
    # three copies of a partly filled page, two free pages: the last row ends early
    got = check_fork(table, lens, refs, [0, 0, 0, 1], [0, 0, 0, 0], 16, pools)
    assert got[1].tolist() == [40, 40, 40, 5]
    got = check_fork(table, lens, refs, [0, 0, 1, 0, 0], [0, 0, 20, 0, 0], 16, pools)
    assert got[1].tolist() == [40, 40, 5, 32, 32]
    assert got[0].tolist()[3] == [0, 1, -1]


def test_fork_reports_bad_data():
    g = torch.Generator("cuda").manual_seed(7)
    pools = make_pools(8, g)
    refs = ints([1, 1, 1, 0, 0, 0, 0, 0])
    for table, lens, src, reserve, want in (
            ([[0, 1], [2, -1]], [17, 3], [0, 2], 0, ta.STATUS_BAD_ROW),
            ([[0, 1], [2, -1]], [17, 3], [0, -3], 0, ta.STATUS_BAD_ROW),
            ([[0, 1], [2, -1]], [33, 3], [0], 0, ta.STATUS_BAD_SEQ_LEN),
            ([[0, 1], [2, -1]], [-1, 3], [0], 0, ta.STATUS_BAD_SEQ_LEN),
            ([[0, 1], [2, -1]], [17, 3], [0], 16, ta.STATUS_BAD_SEQ_LEN),
            ([[8, 1], [2, -1]], [17, 3], [0, 0], 0, ta.STATUS_BAD_PAGE),
            ([[0, 1], [2, -7]], [17, 3], [0], 0, ta.STATUS_BAD_PAGE)):
        status = ints([0])
        ta.kv_fork(pools, ints(table), ints(lens), refs, ints(src), 16, reserve=reserve,
                   status=status)
        assert int(status) == want, (table, lens, src, reserve)


@pytest.mark.parametrize("n,share,rows,width", [(1, 1.0, 1, 1), (2, 0.5, 1, 2), (64, 0.0, 2, 3),
                                                (64, 1.0, 4, 16), (300, 0.4, 7, 40),
                                                (9000, 0.3, 5, 800), (9000, 0.97, 3, 3000),
                                                (50000, 0.01, 2, 600)])
def test_compact_against_loops(n, share, rows, width):
    r = random.Random(n + rows)
    g = torch.Generator("cuda").manual_seed(n)
    used = r.sample(range(n), int(share * n))
    table = [[-1] * width for _ in range(rows)]
    refs = [0] * n
    for i, p in enumerate(used):
        refs[p] = r.randint(1, 3)
        if i // width < rows:
            table[i // width][i % width] = p
    pools = make_pools(n, g) if n <= 300 else [
        torch.randint(0, 256, (n, 32), dtype=torch.uint8, device="cuda", generator=g)]
    before = [p.clone() for p in pools]
    status = ints([0])
    t0 = ints(table)
    got = ta.kv_compact(pools, t0, ints(refs), status=status)
    want_t, want_r, want_n, moves = context.compact(table, refs)
    assert got[0].tolist() == want_t and got[1].tolist() == want_r and got[2].tolist() == [want_n]
    assert int(status) == 0 and same(pools, moved(before, moves))
    again = [p.clone() for p in before]
    ta.kv_compact(again, t0, ints(refs), block_table_out=t0)  # in place
    assert t0.tolist() == want_t and same(again, pools)


@pytest.mark.parametrize("n,holes", [(31, [0]), (32, [31]), (33, [32]), (33, [0, 31]), (8191, [5, 8190]),
                                     (8192, [0, 4096, 8191]), (8192, []), (8193, [1, 8192]),
                                     (8192, range(8191)), (8192, range(1, 8192)),
                                     (8193, range(0, 8193, 2)), (2047, [2046]), (2048, []),
                                     (2048, [0, 2047]), (2048, range(1, 2048)),
                                     (2048, range(0, 2048, 3)), (2049, [7])])
def test_compact_of_few_and_many_holes(n, holes):
    g = torch.Generator("cuda").manual_seed(n)
    refs = [p % 3 + 1 for p in range(n)]
    for p in holes:
        refs[p] = 0
    table = [[p if c else -1 for p, c in enumerate(refs)]]
    pools = [torch.randint(0, 99, (n, 48), dtype=torch.uint8, device="cuda", generator=g),
             torch.randint(0, 99, (n, 5), dtype=torch.uint8, device="cuda", generator=g)]
    want_t, want_r, want_n, moves = context.compact(table, refs)
    want = moved(pools, moves)
    got = ta.kv_compact(pools, ints(table), ints(refs))
    assert got[0].tolist() == want_t and got[1].tolist() == want_r and got[2].tolist() == [want_n]
    assert same(pools, want)


def test_compact_of_more_pools_than_one_launch_takes():
    g = torch.Generator("cuda").manual_seed(8)
    pools = [torch.randint(0, 99, (40, 16), dtype=torch.uint8, device="cuda", generator=g)
             for _ in range(250)]
    refs = [p % 2 for p in range(40)]
    table = [list(range(1, 40, 2))]
    want_t, want_r, want_n, moves = context.compact(table, refs)
    want = moved(pools, moves)
    got = ta.kv_compact(pools, ints(table), ints(refs))
    assert got[0].tolist() == want_t and got[1].tolist() == want_r and got[2].tolist() == [want_n]
    assert same(pools, want)


def test_compact_reports_entries_without_a_page():
    pools = [torch.zeros(8, 32, dtype=torch.uint8, device="cuda")]
    status = ints([0])
    got = ta.kv_compact(pools, ints([[6, 5, 8, -1, -2]]), ints([0, 0, 0, 0, 0, 0, 2, 0]),
                        status=status)
    assert got[0].tolist() == [[0, -1, -1, -1, -1]] and int(status) == ta.STATUS_BAD_PAGE


@pytest.mark.parametrize("rows,out,n", [(40, 100, 4000), (9, 16, 600)])
def test_captured_and_replayed_on_two_streams_at_once(rows, out, n):
    """Two captured forks with workspaces of their own, replayed at once, twice."""
    states = []
    for seed in range(2):
        r = random.Random(seed)
        table, lens, refs = random_state(r, rows, 16, 40, n)
        src = [r.randrange(-1, rows) for _ in range(out)]
        g = torch.Generator("cuda").manual_seed(seed)
        pool = torch.randint(0, 256, (n, 4096), dtype=torch.uint8, device="cuda", generator=g)
        want = context.fork(table, lens, refs, src, [0] * out, 16)
        states.append((ints(table), ints(lens), ints(refs), ints(src), pool, pool.clone(), want))
    graphs = []
    for t, l, c, s, pool, _, _ in states:
        ta.kv_fork([pool], t, l, c, s, 16)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = ta.kv_fork([pool], t, l, c, s, 16)
        graphs.append((graph, got))
    streams = [torch.cuda.Stream() for _ in states]
    for (t, l, c, s, pool, first, _) in states:
        pool.copy_(first)
    torch.cuda.synchronize()
    for _ in range(2):
        for (graph, _), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for (_, got), (_, _, _, _, pool, first, want) in zip(graphs, states):
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1]
        assert got[2].tolist() == want[2] and same([pool], moved([first], want[3]))


def test_refusals():
    pools = [torch.zeros(8, 32, dtype=torch.uint8, device="cuda")]
    t, l, c, s = ints([[0, -1]]), ints([3]), ints([1] + [0] * 7), ints([0, 0])
    with pytest.raises(ValueError):
        ta.kv_fork(pools, t, l, c, s, 16, page_refs_out=c)
    with pytest.raises(ValueError):
        ta.kv_fork(pools, t, l, c, ints([0]), 16, block_table_out=t)
    with pytest.raises(ta.TreeAttnError):
        ta.kv_fork(pools, t, l, c, s, 48)
    with pytest.raises(ValueError):
        ta.kv_fork(pools, t, l, c, s, 16, reserve=-1)
    with pytest.raises(ValueError):
        ta.kv_fork([pools[0][:4]], t, l, c, s, 16)
    with pytest.raises(ValueError):
        ta.kv_fork([torch.zeros(8, 32)], t, l, c, s, 16)
    with pytest.raises(ValueError):
        ta.kv_fork([pools[0].t()], t, l, c, s, 16)
    with pytest.raises(ta.TreeAttnError):
        ta.kv_fork(pools, t, l, c, ints([-1] * 17), 16,
                   workspace=torch.empty(256, dtype=torch.uint8, device="cuda")[:16])
    with pytest.raises(ValueError):
        ta.kv_compact(pools, t, c, page_refs_out=c)
    with pytest.raises(TypeError):
        ta.kv_copy_pages(pools, s.long(), s)
    with pytest.raises(ValueError):
        ta.kv_copy_pages(pools, s, ints([1]))
