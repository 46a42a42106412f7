"""The 8-bit paged cache on the GPU: every byte that append and commit write
against the definition in oracle/fp8_rows.py (bit-exact: a code is one
rounding of an exactly scaled value), every other byte left alone, and the
read-back exact."""
import numpy as np
import pytest
import torch

import speculative_decoding_tree_split_gb300 as ta
from oracle import fp8_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ta.build()
    ta.load()


def make_cache(caps, Hkv, d, P, seed=0, extra=2):
    """Pools of random bytes and a block table for caps[b] tokens each."""
    g = torch.Generator().manual_seed(seed)
    pages = [-(-c // P) for c in caps]
    n = sum(pages) + extra
    perm = torch.randperm(n, generator=g).int()
    bt = torch.full((len(caps), max(pages + [1])), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(pages):
        bt[b, :m] = perm[at:at + m]
        at += m

    def pool(*shape):
        return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)

    return [pool(n, Hkv, P, d), pool(n, Hkv, P, d), pool(n, Hkv, P), pool(n, Hkv, P), bt]


def rows(n, Hkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, Hkv, d, generator=g) * torch.exp(2 * torch.randn(n, Hkv, 1, generator=g))
    return x.bfloat16()


def edge_rows(x):
    """Some rows of x [N][H][d] made hard: zeros, infinities, NaN, huge, tiny."""
    n = x.shape[0]
    for i, v in enumerate((0.0, float("inf"), float("nan"), 3e38, 1e-38, -float("inf"), 448.0)):
        if i < n:
            x[i, 0, i] = v
    if n > 8:
        x[7] = 0.0
        x[8, -1] *= 1e-30
        x[8, -1, 3] = 1e-40  # subnormal in bf16
    return x


def put(cache, which, b, pos, x):
    P = cache[2 + which].shape[2]
    page = int(cache[4][b, pos // P])
    codes, scale = fp8_rows.encode(x.double().numpy())
    cache[which][page, :, pos % P] = torch.from_numpy(codes)
    cache[2 + which][page, :, pos % P] = torch.from_numpy(scale)


def dev(ts):
    return [t.cuda() for t in ts]


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cumulate(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return out


def assert_same(got, want):
    for name, a, b in zip(("k codes", "v codes", "k scales", "v scales"), got, want):
        a, b = a.cpu(), b
        if name.endswith("codes"):  # a NaN may carry either sign
            a, b = a.clone(), b.clone()
            a[(a & 127) == 127] = 127
            b[(b & 127) == 127] = 127
        assert torch.equal(a, b), (name, int((a != b).sum()))


APPENDS = [
    # lens, starts, Hkv, d, P, layout
    ([1], [0], 1, 64, 16, "dense"),
    ([5], [15], 2, 128, 16, "fused"),
    ([0, 17, 0, 1, 40], [3, 0, 9, 31, 64], 2, 64, 32, "dense"),
    ([100, 33, 129], [1, 127, 0], 3, 128, 128, "heads first"),
    ([70, 0, 300], [63, 64, 65], 8, 128, 64, "fused"),
    ([0, 0], [4, 5], 2, 64, 64, "dense"),
]


def lay_out(k, v, layout):
    if layout == "fused":
        kv = torch.cat([k, v], 1).cuda()
        return kv[:, :k.shape[1]], kv[:, k.shape[1]:]
    if layout == "heads first":
        return tuple(x.transpose(0, 1).contiguous().cuda().transpose(0, 1) for x in (k, v))
    return k.cuda(), v.cuda()


@pytest.mark.parametrize("lens,starts,Hkv,d,P,layout", APPENDS)
def test_append_is_bit_exact_and_writes_nothing_else(lens, starts, Hkv, d, P, layout):
    first, behind = 2, 3  # packed rows before the first and after the last sequence
    N = first + sum(lens) + behind
    k, v = edge_rows(rows(N, Hkv, d, 1)), edge_rows(rows(N, Hkv, d, 2))
    cache = make_cache([s + n for s, n in zip(starts, lens)], Hkv, d, P)
    cu = cumulate(lens, first)
    got = dev(cache)
    status = ints([0])
    kd, vd = lay_out(k, v, layout)
    new = ta.kv_append_fp8(*got, ints(starts), ints(cu), kd, vd, status=status)
    assert int(status) == 0
    assert new.tolist() == [s + n for s, n in zip(starts, lens)]
    for b, n in enumerate(lens):
        for j in range(n):
            put(cache, 0, b, starts[b] + j, k[cu[b] + j])
            put(cache, 1, b, starts[b] + j, v[cu[b] + j])
    assert_same(got, cache[:4])


@pytest.mark.parametrize("Hkv,d,P", [(1, 128, 64), (2, 64, 16)])
def test_append_and_read_of_many_tokens(Hkv, d, P):
    # enough tokens that the larger tile of the two kernels is used on any GPU
    # of up to 160 SMs, none of the ranges a multiple of it
    lens, starts = [9001, 0, 1, 2003, 17], [5, 0, 63, 1, P]
    N = sum(lens)
    assert N // 16 >= 4 * torch.cuda.get_device_properties(0).multi_processor_count
    cache = make_cache([s + n for s, n in zip(starts, lens)], Hkv, d, P)
    k, v = edge_rows(rows(N, Hkv, d, 21)), edge_rows(rows(N, Hkv, d, 22))
    got, status = dev(cache), ints([0])
    cu = cumulate(lens)
    ta.kv_append_fp8(*got, ints(starts), ints(cu), k.cuda(), v.cuda(), status=status)
    seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens))
    pos = torch.arange(N) - torch.tensor(cu)[seq] + torch.tensor(starts)[seq]
    page, off = cache[4][seq, pos // P].long(), pos % P
    values = []
    for w, x in enumerate((k, v)):
        codes, scale = fp8_rows.encode(x.double().numpy())
        values.append(fp8_rows.decode(codes, scale))
        cache[w][page, :, off] = torch.from_numpy(codes)
        cache[2 + w][page, :, off] = torch.from_numpy(scale)
    assert_same(got, cache[:4])
    back = ta.kv_read_fp8(*got, ints(cu), N, starts=ints(starts), status=status)
    assert int(status) == 0
    for x, want in zip(back, values):
        assert np.array_equal(x.double().cpu().numpy(), want, equal_nan=True)


def test_append_takes_float8_pools():
    cache = make_cache([9], 1, 64, 16)
    x = rows(9, 1, 64, 3)
    got = dev(cache)
    codes = [got[0].view(torch.float8_e4m3fn), got[1].view(torch.float8_e4m3fn)]
    ta.kv_append_fp8(*codes, *got[2:], ints([0]), ints([0, 9]), x.cuda(), x.cuda())
    for j in range(9):
        put(cache, 0, 0, j, x[j])
        put(cache, 1, 0, j, x[j])
    assert_same(got, cache[:4])


@pytest.mark.parametrize("case", ["page", "past the table", "negative length", "descending",
                                  "past the rows"])
def test_append_skips_what_fails_and_says_so(case):
    # two sequences of 20 tokens; the first is sound, the second is not
    lens, starts, P = [20, 20], [0, 0], 16
    cache = make_cache([20, 20], 2, 64, P)
    cu = cumulate(lens)
    k = rows(40, 2, 64, 4)
    want_status, want_new, good = 3, [20, 20], 20
    if case == "page":
        cache[4][1, 1] = cache[0].shape[0]
        want_status, good = 2, 36
    elif case == "past the table":
        starts[1] = 20  # the block table holds 32 positions
        want_new, good = [20, 40], 32
    elif case == "negative length":
        starts[1] = -1
        want_new = [20, -1]
    elif case == "descending":
        cu[2] = 10
        want_new = [20, 0]
    else:
        cu[2] = 41
        want_new = [20, 0]
    got = dev(cache)
    status = ints([0])
    new = ta.kv_append_fp8(*got, ints(starts), ints(cu), k.cuda(), k.cuda(), status=status)
    assert int(status) == want_status
    assert new.tolist() == want_new
    for i in range(good):
        b, j = (0, i) if i < 20 else (1, starts[1] + i - 20)
        for w in (0, 1):
            put(cache, w, b, j, k[i])
    assert_same(got, cache[:4])


@pytest.mark.parametrize("T,Hkv,d,P", [(1, 1, 64, 16), (4, 8, 128, 64), (33, 2, 128, 16),
                                       (64, 3, 64, 128)])
def test_commit_is_bit_exact_and_writes_nothing_else(T, Hkv, d, P):
    B = 5
    g = torch.Generator().manual_seed(T)
    L = [0, P - 1, P, 3 * P + 5, 77]
    n = [0, T, 1] + torch.randint(0, T + 1, (2,), generator=g).tolist()
    path = torch.full((B, T), -1, dtype=torch.int32)
    for b in range(B):
        path[b, :n[b]] = torch.randperm(T, generator=g)[:n[b]].sort().values.int()
    cache = make_cache([x + T for x in L], Hkv, d, P)
    tk = edge_rows(rows(B * T, Hkv, d, 5)).view(B, T, Hkv, d)
    tv = edge_rows(rows(B * T, Hkv, d, 6)).view(B, T, Hkv, d)
    got = dev(cache)
    status = ints([0])
    new = ta.kv_commit_fp8(*got, ints(L), path.cuda(), ints(n), tk.cuda(), tv.cuda(), status=status)
    assert int(status) == 0
    assert new.tolist() == [x + y for x, y in zip(L, n)]
    for b in range(B):
        for j in range(n[b]):
            put(cache, 0, b, L[b] + j, tk[b, path[b, j]])
            put(cache, 1, b, L[b] + j, tv[b, path[b, j]])
    assert_same(got, cache[:4])


def test_commit_skips_what_fails_and_says_so():
    cache = make_cache([40, 40, 40], 2, 64, 16)
    x = rows(12, 2, 64, 7).view(3, 4, 2, 64)
    path = torch.tensor([[0, 4, 2, -1], [0, 1, 2, 3], [0, 1, 2, 3]], dtype=torch.int32)
    for lens, n, want, new in (([0, 0, 0], [3, 0, 0], 5, [3, 0, 0]),
                               ([0, 0, 0], [0, 5, 0], 5, [0, 0, 0]),
                               ([0, 46, 0], [0, 4, 0], 3, [0, 50, 0]),
                               ([0, -3, 0], [0, 4, 0], 3, [0, -3, 0])):
        got, status = dev(cache), ints([0])
        out = ta.kv_commit_fp8(*got, ints(lens), path.cuda(), ints(n), x.cuda(), x.cuda(),
                               status=status)
        assert int(status) == want and out.tolist() == new, (lens, n)
        ref = [t.clone() for t in cache]
        for b in range(3):
            for k in range(n[b] if n[b] <= 4 else 0):
                j = int(path[b, k])
                if 0 <= j < 4 and 0 <= lens[b] + k < 48 and lens[b] >= 0:
                    put(ref, 0, b, lens[b] + k, x[b, j])
                    put(ref, 1, b, lens[b] + k, x[b, j])
        assert_same(got, ref[:4])


@pytest.mark.parametrize("lens,starts,Hkv,d,P,layout", APPENDS)
def test_read_is_exact_and_leaves_other_rows(lens, starts, Hkv, d, P, layout):
    cache = make_cache([s + n for s, n in zip(starts, lens)], Hkv, d, P)
    # scales that append can write
    for w in (2, 3):
        cache[w] = (cache[w].int() % 97 + 71).to(torch.uint8)
    first, behind = 1, 2
    cu = cumulate(lens, first)
    N = cu[-1] + behind
    outs = [torch.full((N, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    status = ints([0])
    got = ta.kv_read_fp8(*dev(cache), ints(cu), N, starts=ints(starts), k_out=outs[0],
                         v_out=outs[1], status=status)
    assert int(status) == 0
    for w in (0, 1):
        want = np.full((N, Hkv, d), 7.0)
        for b, n in enumerate(lens):
            for j in range(n):
                pos = starts[b] + j
                page = int(cache[4][b, pos // P])
                want[cu[b] + j] = fp8_rows.decode(cache[w][page, :, pos % P].numpy(),
                                                  cache[2 + w][page, :, pos % P].numpy())
        g = got[w].double().cpu().numpy()
        assert np.array_equal(np.isnan(g), np.isnan(want))
        assert np.array_equal(g[~np.isnan(g)], want[~np.isnan(want)])


def test_read_reports_bad_positions():
    cache = make_cache([32], 1, 64, 16)
    for starts, table, want in (([1], None, 3), ([-1], None, 3), ([0], -1, 2)):
        c = [t.clone() for t in cache]
        if table is not None:
            c[4][0, 1] = table
        status = ints([0])
        ta.kv_read_fp8(*dev(c), ints([0, 32]), 32, starts=ints(starts), status=status)
        assert int(status) == want


def test_written_rows_read_back_within_half_a_step():
    lens, P, Hkv, d = [50, 7], 16, 2, 128
    k, v = rows(57, Hkv, d, 8), rows(57, Hkv, d, 9)
    got = dev(make_cache(lens, Hkv, d, P))
    cu = ints([0, 50, 57])
    ta.kv_append_fp8(*got, ints([0, 0]), cu, k.cuda(), v.cuda())
    for x, y in zip((k, v), ta.kv_read_fp8(*got, cu, 57)):
        x, y = x.double(), y.double().cpu()
        top = x.abs().amax(-1, keepdim=True)
        # half a step: 2^-4 of the value, or of the smallest normal code's
        # 2^-6 * 2^s < top * 2^-13 (448 * 2^s < 2 * top)
        assert bool(((x - y).abs() <= 2.0 ** -4 * torch.maximum(x.abs(), top * 2.0 ** -13)).all())


def test_append_and_read_in_a_replayed_graph_and_on_another_stream():
    lens, P, Hkv, d = [33, 18], 32, 2, 64
    cache = make_cache([x + 40 for x in lens], Hkv, d, P)
    got = dev(cache)
    k, v = rows(51, Hkv, d, 10).cuda(), rows(51, Hkv, d, 11).cuda()
    cu, sl, new = ints([0, 33, 51]), ints([0, 0]), ints([0, 0])
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        ta.kv_append_fp8(*got, sl, cu, k, v, seq_lens_out=new, stream=s)
        ta.kv_read_fp8(*got, cu, 51, k_out=ko, v_out=vo, starts=sl, stream=s)

    step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for seed in (12, 13):
        k.copy_(rows(51, Hkv, d, seed))
        v.copy_(rows(51, Hkv, d, seed + 50))
        sl.copy_(ints([seed % 5, 7]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in ((k, ko), (v, vo)):
            codes, scale = fp8_rows.encode(x.double().cpu().numpy())
            assert np.array_equal(y.double().cpu().numpy(), fp8_rows.decode(codes, scale))
        assert new.tolist() == [seed % 5 + 33, 7 + 18]


def test_the_binding_checks_its_arguments():
    cache = dev(make_cache([32], 2, 64, 16))
    x = rows(8, 2, 64, 14).cuda()
    cu, sl = ints([0, 8]), ints([0])
    bad = [
        dict(k=x[:, :1]), dict(k=x[:7]), dict(k=x.float()), dict(k=x.transpose(1, 2)),
        dict(cu=ints([0, 4, 8])), dict(sl=ints([0, 0])), dict(cu=cu.long()),
        dict(ks=cache[2][:, :1].contiguous()),
    ]
    for kw in bad:
        a = dict(k=x, cu=cu, sl=sl, ks=cache[2])
        a.update(kw)
        with pytest.raises((ValueError, TypeError)):
            ta.kv_append_fp8(cache[0], cache[1], a["ks"], cache[3], cache[4], a["sl"], a["cu"],
                             a["k"], x)
    with pytest.raises(ta.TreeAttnError):  # the new lengths must be an array of their own
        ta.kv_append_fp8(*cache, sl, cu, x, x, seq_lens_out=sl)
    with pytest.raises(ValueError):
        ta.kv_read_fp8(*cache, cu, -1)
    with pytest.raises(ta.TreeAttnError):  # rows 8 bytes off a 16-byte boundary
        y = torch.zeros(8 * 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(8, 2, 64)
        ta.kv_append_fp8(*cache, sl, cu, y, y)
