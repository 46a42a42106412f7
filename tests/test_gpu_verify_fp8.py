"""verify_fp8 against the fp64 oracle on the values that the cache stands for.

Tolerances.  Let A = sum_j p_j |v_j| / l.  The probabilities enter P.V with at
most half a step of 8 bits (2^-8 each; those below 2^-14 of the largest a fixed
2^-18 of it), the tree's in fp32, and the result is rounded to bf16 once:
    |out - ref| <= 2^-8 (|ref| + A) + 2^-18 n max|v|,
never more than the library's bar of 1e-2.  A score is a sum of d products in
fp32 of a query held to 2^-17 of the tile's largest element, so
    |lse - ref| <= scale (2^-17 max|q| + 2^-20 |q|) max_j sum|k_j| + 2^-18,
never more than the bar of 1e-3.
"""
import dataclasses
import math

import numpy as np
import pytest
import torch

import speculative_decoding_tree_split_gb300 as ta
from oracle import fp8_rows
from workloads import CONFIGS, Config, make_workload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ta.build()
    ta.load()


def quantised(wl, garbage=True):
    """(pools, the workload with the values the pools stand for).  Slots that
    hold no committed token get bytes of NaN codes and absurd scales."""
    pools, values = [], []
    for x in (wl.k_pages, wl.v_pages):
        codes, scale = fp8_rows.encode(x.double().numpy())
        values.append(torch.from_numpy(fp8_rows.decode(codes, scale)).bfloat16())
        pools.append((torch.from_numpy(codes), torch.from_numpy(scale)))
    if garbage:
        P = wl.cfg.page
        used = torch.zeros(wl.num_pages, P, dtype=torch.bool)
        for b, L in enumerate(wl.seq_lens.tolist()):
            for p in range(0, L, P):
                used[int(wl.block_table[b, p // P]), :min(P, L - p)] = True
        for codes, scale in pools:
            for page, slot in (~used).nonzero().tolist():
                codes[page, :, slot] = 127
                scale[page, :, slot] = 255
    return ([pools[0][0], pools[1][0], pools[0][1], pools[1][1]],
            dataclasses.replace(wl, k_pages=values[0], v_pages=values[1]))


def run(wl, pools, status_want=0, **kw):
    d = torch.device("cuda")
    status = torch.zeros(1, dtype=torch.int32, device=d)
    if "mask" not in kw and "parents" not in kw:
        kw["parents"] = wl.parents.to(d)
    out, lse = ta.verify_fp8(wl.q.to(d), *[p.to(d) for p in pools], wl.block_table.to(d),
                             wl.seq_lens.to(d), wl.tree_k.to(d), wl.tree_v.to(d),
                             softmax_scale=wl.scale, status=status, **kw)
    assert int(status) == status_want
    return out, lse


def check(oracle, wl, pools, mask=None, **kw):
    out, lse = run(wl, pools, **kw)
    close(oracle, wl, out, lse, mask)


def close(oracle, wl, out, lse, mask=None):
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    if mask is None:
        mask = oracle.tree_mask(wl.parents.tolist())
    c = wl.cfg
    ref, ref_l = oracle.verify(wl, mask)
    A, _ = oracle.verify(dataclasses.replace(wl, v_pages=wl.v_pages.abs(), tree_v=wl.tree_v.abs()),
                         mask)
    n = int(wl.seq_lens.max()) + c.T
    vmax = float(max(wl.v_pages.abs().max() if wl.v_pages.numel() else 0, wl.tree_v.abs().max()))
    tol = np.minimum(2.0 ** -8 * (np.abs(ref) + A) + 2.0 ** -18 * n * vmax, 1e-2 * max(1.0, vmax / 4))
    assert np.isfinite(out).all() and (np.abs(out - ref) <= tol).all(), np.abs(out - ref).max()
    ksum = float(max(wl.k_pages.float().abs().sum(-1).max() if wl.k_pages.numel() else 0,
                     wl.tree_k.float().abs().sum(-1).max()))
    qmax = float(wl.q.float().abs().max())
    lt = min(abs(wl.scale) * (2.0 ** -17 + 2.0 ** -20) * qmax * ksum + 2.0 ** -18, 1e-3)
    assert np.array_equal(np.isfinite(lse), np.isfinite(ref_l))
    ok = np.isfinite(lse)
    assert (np.abs(lse - ref_l)[ok] <= lt).all(), (np.abs(lse - ref_l)[ok].max(), lt)


def cfg(B, Hq, Hkv, d, page, T, tree="random"):
    return Config("case", B=B, Hq=Hq, Hkv=Hkv, d=d, L=64, page=page, T=T, tree=tree, max_depth=T,
                  max_branch=4, seed=B * 1000 + Hq + T)


CASES = [
    # cfg, committed lengths
    (cfg(1, 1, 1, 64, 16, 1), [1]),
    (cfg(3, 4, 1, 64, 16, 1), [0, 17, 300]),
    (cfg(2, 8, 2, 128, 64, 1), [63, 1025]),
    (cfg(4, 8, 2, 128, 16, 4), [0, 1, 128, 129]),
    (cfg(2, 32, 8, 128, 64, 12), [500, 1000]),
    (cfg(3, 10, 2, 128, 32, 16), [64, 127, 700]),      # five query heads to a KV head
    (cfg(2, 40, 8, 128, 64, 16), [300, 257]),          # 80 rows to a tile
    (cfg(1, 14, 2, 128, 128, 15), [333]),              # 105 rows
    (cfg(2, 16, 2, 64, 32, 16), [40, 200]),            # 128 rows
    (cfg(1, 8, 1, 128, 64, 33), [300]),                # 264 rows: three row blocks
    (cfg(1, 16, 2, 64, 16, 64), [130]),                # 512 rows
    (cfg(5, 2, 2, 64, 128, 7), [5, 0, 256, 128, 511]),
    (cfg(1, 3, 1, 128, 64, 64, "chain"), [2000]),
    (cfg(2, 8, 1, 128, 32, 4), [77, 900]),             # 32 rows
    (cfg(2, 8, 2, 64, 64, 8), [64, 391]),              # 32 rows
    (cfg(1, 12, 1, 64, 16, 4), [700]),                 # 48 rows
    (cfg(2, 16, 2, 128, 64, 8), [1, 555]),             # 64 rows
    (cfg(2, 8, 1, 64, 128, 8), [200, 333]),            # 64 rows
    (cfg(1, 10, 2, 64, 32, 16), [1023]),               # 80 rows
    (cfg(70, 4, 1, 64, 16, 2), [(37 * i) % 90 for i in range(70)]),  # many short sequences
    (cfg(300, 1, 1, 128, 64, 1), [(29 * i) % 150 for i in range(300)]),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_the_oracle(oracle, i):
    c, lens = CASES[i]
    wl = make_workload(c, seq_lens=lens, extra_pages=3)
    pools, wl = quantised(wl)
    check(oracle, wl, pools)


@pytest.mark.parametrize("name", ["tiny", "llama8b"])
def test_full_size(oracle, name):
    wl = make_workload(CONFIGS[name])
    pools, wl = quantised(wl)
    check(oracle, wl, pools)


def test_mask_parents_and_per_sequence_trees_agree(oracle):
    c = cfg(3, 8, 2, 128, 32, 9)
    wl = make_workload(c, seq_lens=[100, 0, 333], per_sequence_trees=True)
    pools, wl = quantised(wl)
    masks = ta.mask_build_batched(wl.parents.cuda())
    built = torch.empty_like(masks)
    o1, l1 = run(wl, pools, parents=wl.parents.cuda(), mask_out=built)
    o2, l2 = run(wl, pools, mask=masks)
    assert torch.equal(built, masks) and torch.equal(o1, o2) and torch.equal(l1, l2)
    for b in range(3):
        one = wl.sequence(b)
        close(oracle, one, o1[b:b + 1], l1[b:b + 1])


def test_rows_without_any_key(oracle):
    c = cfg(2, 4, 2, 64, 16, 3)
    wl = make_workload(c, seq_lens=[0, 20])
    pools, wl = quantised(wl)
    mask = torch.tensor([0, 3, 0], dtype=torch.int64)  # nodes 0 and 2 see no tree token
    out, lse = run(wl, pools, mask=mask.cuda())
    assert float(out[0, [0, 2]].abs().max()) == 0
    assert bool((lse[0, [0, 2]] == -math.inf).all())
    one = wl.sequence(1)
    close(oracle, one, out[1:], lse[1:], mask=mask.numpy().astype(np.uint64))


def test_many_keys_of_uneven_size(oracle):
    # Scores of a wide spread (the running maximum moves often), values whose
    # scales differ by token, and a first token that draws the attention but
    # holds nothing.
    c = cfg(2, 16, 2, 128, 64, 5)
    wl = make_workload(c, seq_lens=[3000, 1300], extra_pages=1)
    g = torch.Generator().manual_seed(1)
    wl.q.mul_(4.0)
    n, H, P, d = wl.k_pages.shape
    wl.v_pages.mul_(torch.exp2(torch.randint(-6, 3, (n, H, P, 1), generator=g).float()).bfloat16())
    for b in range(2):
        wl.v_pages[wl.block_table[b, 0], :, 0] = 0
        wl.k_pages[wl.block_table[b, 0], :, 0] = wl.q[b, 0, ::8].sign() * 1.5
    pools, wl = quantised(wl)
    check(oracle, wl, pools)


@pytest.mark.parametrize("shift", [-50, -20, 20, 30])
def test_values_far_from_one(oracle, shift):
    # The whole value cache in other units: the result moves with it.
    c = cfg(1, 8, 2, 128, 64, 4)
    wl = make_workload(c, seq_lens=[400])
    f = 2.0 ** shift
    pools, wl1 = quantised(wl)
    for p in pools[3:]:
        p[p != 255] += shift
    big = dataclasses.replace(wl1, tree_v=(wl1.tree_v.float() * f).bfloat16())
    out, lse = run(big, pools)
    o = dataclasses.replace(wl1)
    close(oracle, o, out.float() / f, lse)


def test_negative_scale(oracle):
    c = cfg(1, 8, 2, 128, 64, 4)
    wl = dataclasses.replace(make_workload(c, seq_lens=[500]), scale=-0.05)
    pools, wl = quantised(wl)
    check(oracle, wl, pools)


def test_nan_of_a_committed_row_reaches_only_its_sequence_and_head():
    c = cfg(2, 4, 2, 64, 16, 2)
    wl = make_workload(c, seq_lens=[200, 200])
    pools, wl = quantised(wl)
    clean, clean_l = run(wl, pools)
    page = int(wl.block_table[1, 3])
    pools[0][page, 1, 5, 7] = 127  # NaN in one key row of sequence 1, KV head 1
    out, lse = run(wl, pools)
    assert torch.equal(out[0], clean[0]) and torch.equal(lse[0], clean_l[0])
    assert torch.equal(out[1, :, :2], clean[1, :, :2])
    assert bool(out[1, :, 2:].isnan().all()) and bool(lse[1, :, 2:].isnan().all())


@pytest.mark.parametrize("T,G,d", [(5, 2, 64), (40, 3, 128)])
def test_nan_and_infinity_of_a_tree_token_reach_only_rows_that_see_it(T, G, d):
    c = cfg(2, 2 * G, 2, d, 16, T)
    wl = make_workload(c, seq_lens=[0, 50])
    pools, wl = quantised(wl)
    clean, clean_l = run(wl, pools)
    masks = [int(m) for m in ta.mask_build(wl.parents.cuda()).cpu()]
    # a leaf's key is NaN, a leaf's value infinite in one place, another's NaN
    leaves = [j for j in range(T) if sum((m >> j) & 1 for m in masks) == 1]
    k_bad, v_inf, v_nan = leaves[0], leaves[-1], leaves[len(leaves) // 2]
    tk, tv = wl.tree_k.clone(), wl.tree_v.clone()
    tk[:, k_bad, :, 3] = float("nan")
    tv[:, v_inf, :, 7] = -float("inf")
    tv[:, v_nan, :, 9] = float("nan")
    out, lse = run(dataclasses.replace(wl, tree_k=tk, tree_v=tv), pools)
    for t in range(T):
        if (masks[t] >> k_bad) & 1:
            assert bool(out[:, t].isnan().all()) and bool(lse[:, t].isnan().all())
            continue
        assert torch.equal(lse[:, t], clean_l[:, t])
        want = clean[:, t].clone()
        if (masks[t] >> v_inf) & 1:
            want[..., 7] = -math.inf
        if (masks[t] >> v_nan) & 1:
            want[..., 9] = math.nan
        assert torch.equal(out[:, t].isnan(), want.isnan()), t
        ok = ~want.isnan()
        assert torch.equal(out[:, t][ok], want[ok]), t


def test_bad_data_is_reported():
    c = cfg(2, 4, 2, 64, 16, 2)
    wl = make_workload(c, seq_lens=[100, 40])
    pools, wl = quantised(wl)
    for page in (wl.num_pages, -1):
        bt = wl.block_table.clone()
        bt[0, 2] = page
        run(dataclasses.replace(wl, block_table=bt), pools, status_want=2)
    for n in (-1, wl.max_pages_per_seq * 16 + 1):
        sl = wl.seq_lens.clone()
        sl[1] = n
        run(dataclasses.replace(wl, seq_lens=sl), pools, status_want=3)
    run(wl, pools, status_want=1, parents=torch.tensor([-1, 1], dtype=torch.int32, device="cuda"))


def test_matches_verification_over_the_read_back_cache(oracle):
    c = cfg(3, 8, 2, 128, 64, 6)
    lens = [700, 64, 129]
    wl = make_workload(c, seq_lens=lens)
    pools, wl = quantised(wl)
    out, lse = run(wl, pools)
    d = torch.device("cuda")
    o2, l2 = ta.verify_tree(wl.q.to(d), wl.k_pages.to(d), wl.v_pages.to(d), wl.block_table.to(d),
                            wl.seq_lens.to(d), wl.tree_k.to(d), wl.tree_v.to(d),
                            wl.parents.to(d), softmax_scale=wl.scale)
    # two results within the bars of the same exact one
    assert float((out.float() - o2.float()).abs().max()) <= 2e-2
    assert float((lse - l2).abs().max()) <= 2e-3
    close(oracle, wl, out, lse)


def test_graph_replay_and_repeated_calls_give_the_same_bits():
    c = cfg(2, 32, 8, 128, 64, 8)
    wl = make_workload(c, seq_lens=[1000, 700])
    pools, wl = quantised(wl)
    d = torch.device("cuda")
    x = [wl.q.to(d), *[p.to(d) for p in pools], wl.block_table.to(d), wl.seq_lens.to(d),
         wl.tree_k.to(d), wl.tree_v.to(d)]
    par = wl.parents.to(d)
    first = ta.verify_fp8(*x, parents=par)
    again = ta.verify_fp8(*x, parents=par)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(ta.workspace_size(2, 32, 8, 128, 8, 0, 64), dtype=torch.uint8, device=d)
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    graphs = []
    for _ in range(2):  # two graphs that share a workspace, replayed one after the other
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            ta.verify_fp8(*x, parents=par, out=out, lse=lse, workspace=ws, stream=s)
        graphs.append(graph)
    for graph in graphs * 2:
        out.zero_()
        lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_another_stream_with_tensors_of_the_calls_own():
    c = cfg(1, 8, 2, 64, 16, 3)
    wl = make_workload(c, seq_lens=[150])
    pools, wl = quantised(wl)
    want = run(wl, pools)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = run_on(wl, pools, s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def run_on(wl, pools, stream):
    d = torch.device("cuda")
    x = [wl.q.to(d), *[p.to(d) for p in pools], wl.block_table.to(d), wl.seq_lens.to(d),
         wl.tree_k.to(d), wl.tree_v.to(d)]
    par = wl.parents.to(d)
    stream.wait_stream(torch.cuda.current_stream())
    out = ta.verify_fp8(*x, parents=par, stream=stream)
    stream.synchronize()
    return out


def test_the_binding_checks_its_arguments():
    c = cfg(2, 4, 2, 64, 16, 3)
    wl = make_workload(c, seq_lens=[30, 40])
    pools, wl = quantised(wl)
    d = torch.device("cuda")
    base = dict(q=wl.q.to(d), kp=pools[0].to(d), vp=pools[1].to(d), ks=pools[2].to(d),
                vs=pools[3].to(d), bt=wl.block_table.to(d), sl=wl.seq_lens.to(d),
                tk=wl.tree_k.to(d), tv=wl.tree_v.to(d))
    par = wl.parents.to(d)
    bad = [
        (dict(), dict()),                                              # no tree
        (dict(), dict(parents=par, mask=ta.mask_build(par))),          # two trees
        (dict(), dict(parents=par[:2])),
        (dict(), dict(parents=par.long())),
        (dict(q=base["q"].float()), dict(parents=par)),
        (dict(tk=base["tk"][:, :2].contiguous()), dict(parents=par)),
        (dict(ks=base["ks"][:, :1].contiguous()), dict(parents=par)),
        (dict(sl=base["sl"][:1]), dict(parents=par)),
        (dict(), dict(parents=par, out=torch.empty(1, 3, 4, 64, dtype=torch.bfloat16, device=d))),
        (dict(), dict(mask=ta.mask_build(par), mask_out=ta.mask_build(par))),
    ]
    for change, kw in bad:
        a = dict(base)
        a.update(change)
        with pytest.raises((ValueError, TypeError)):
            ta.verify_fp8(*a.values(), **kw)
    with pytest.raises(ta.TreeAttnError):
        ta.verify_fp8(*base.values(), parents=par,
                      workspace=torch.empty(256, dtype=torch.uint8, device=d))
