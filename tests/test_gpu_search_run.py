"""Beam search over selected pages, as a server runs it: prompts into the cache, beams
forked from them, each step selecting pages, attending, choosing continuations and
reordering the cache -- with sequences that end and begin and a compaction on the way --
against the same search over plain rows of keys and values, in 64 bits."""
import math

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


def bits(t):
    return t.view(torch.uint8)


@pytest.mark.parametrize("fp8,d,P", [(True, 128, 16), (False, 64, 32)])
def test_search(fp8, d, P):
    Hkv, G, W, V, steps, k = 2, 4, 3, 50, 2 * P + 3, 4
    lens = [5 * P + 3, 9, 7 * P]
    B, N, n = len(lens), sum(lens), 120
    g = torch.Generator("cuda").manual_seed(d)

    def bf(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    if fp8:
        cache = [torch.full((n, Hkv, P, d), 255, dtype=torch.uint8, device="cuda") for _ in "kv"]
        cache += [torch.full((n, Hkv, P), 255, dtype=torch.uint8, device="cuda") for _ in "kv"]
    else:
        cache = [torch.full((n, Hkv, P, d), math.nan, dtype=torch.bfloat16, device="cuda")
                 for _ in "kv"]
    scales = dict(k_scales=cache[2], v_scales=cache[3]) if fp8 else {}
    bounds = [torch.zeros(n, Hkv, 2, d, dtype=torch.int8, device="cuda"),
              torch.zeros(n, Hkv, dtype=torch.uint8, device="cuda")]
    pools = cache + bounds
    status = ints([0])
    # New rows for the prompts, then their tokens.
    table = torch.empty(0, 12, dtype=torch.int32, device="cuda")
    table, seq, refs = ta.kv_fork(pools, table, ints([]), ints([0] * n), ints([-2] * B), P,
                                  reserve=ints(lens), status=status)
    pk, pv = bf(N, Hkv, d), bf(N, Hkv, d)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)

    def append(table, seq, k, v, counts):
        """Tokens behind the rows, and the bounds of the pages that they touch."""
        if fp8:
            c = [0]
            for x in counts:
                c.append(c[-1] + x)
            new = ta.kv_append_fp8(*cache, table, seq, ints(c), k, v, status=status)
        else:
            new = seq + ints(counts)
            at = 0
            for r, (s, m) in enumerate(zip(seq.tolist(), counts)):
                for j in range(m):
                    page = int(table[r, (s + j) // P])
                    cache[0][page, :, (s + j) % P] = k[at]
                    cache[1][page, :, (s + j) % P] = v[at]
                    at += 1
        ta.kv_block_bounds(cache[0], table, new, k_scales=cache[2] if fp8 else None, starts=seq,
                           bounds=bounds[0], bounds_exp=bounds[1], status=status)
        return new

    seq = append(table, seq, pk, pv, lens)
    # Every prompt's W beams, and the same as plain rows.
    src = ints([b for b in range(B) for _ in range(W)])
    table, seq, refs = ta.kv_fork(pools, table, seq, refs, src, P, reserve=1, status=status)
    plain = [[(pk[cu[b]:cu[b + 1]], pv[cu[b]:cu[b + 1]])] * W for b in range(B)]
    scores = torch.full((B, W), -math.inf, device="cuda")
    scores[:, 0] = 0.0  # all beams are the same yet
    finished = torch.zeros(B, W, dtype=torch.bool, device="cuda")
    parents = ints([-1])
    for step in range(steps):
        q, tk, tv = bf(B * W, 1, Hkv * G, d), bf(B * W, 1, Hkv, d), bf(B * W, 1, Hkv, d)
        blocks = ta.select_blocks(q, *bounds, table, seq, k, P, status=status)
        out, lse = ta.verify_blocks(q, cache[0], cache[1], table, seq, blocks, tk, tv,
                                    parents=parents, status=status, **scales)
        if step % 8 == 0 or step > steps - 3:
            for r in range(B * W):
                b, w = divmod(r, W)
                if not plain[b]:
                    continue
                keys, values = plain[b][w]
                assert int(seq[r]) == keys.shape[0]
                for h in range(Hkv):
                    see = [p * P + j for p in blocks[r, 0, h].tolist() if p >= 0
                           for j in range(min(P, int(seq[r]) - p * P))]
                    ks = torch.cat([keys[see, h], tk[r, :, h]]).double()
                    vs = torch.cat([values[see, h], tv[r, :, h]]).double()
                    qh = q[r, 0, h * G:(h + 1) * G]
                    ref, ref_l = context.attend(qh, ks, vs, 1 / math.sqrt(d))
                    # 8-bit rows: each value within 2^-4 of itself, or of the row's largest 2^-9
                    # of that; bf16 rows: rounding of the result alone
                    o = out[r, 0, h * G:(h + 1) * G].double()
                    assert float((o - ref).abs().max()) <= (0.4 if fp8 else 2e-2)
                    assert float((lse[r, 0, h * G:(h + 1) * G] - ref_l).abs().max()) <= (
                        0.3 if fp8 else 1e-3)
                    # the selection's bounds are those of the row's own pages
                    if not fp8:
                        nb = -(-int(seq[r]) // P)
                        hi, lo, e = zip(*(context.page_bounds(keys[j * P:(j + 1) * P, h].double())
                                          for j in range(nb)))
                        own = torch.tensor([hi, lo]).permute(1, 0, 2).to(torch.int8)
                        want = context.choose(qh.cpu(), own, torch.tensor(e), k, 1, 1)
                        assert blocks[r, 0, h].tolist() == want + [-1] * (k - len(want))
        # The token is written, then the beams go on.
        seq = append(table, seq, tk[:, 0], tv[:, 0], [1] * (B * W))
        plain = [[(torch.cat([x, tk[b * W + w]]), torch.cat([y, tv[b * W + w]]))
                  for w, (x, y) in enumerate(plain[b])] for b in range(B)]
        logits = 2 * torch.randn(B, W, V, generator=g, device="cuda")
        before = scores.clone()
        scores, rows, tokens = ta.beam_select(logits, before, W, finished=finished, eos=0)
        for b in range(B):
            if not plain[b]:
                continue
            want = context.beams(logits[b].cpu(), before[b].cpu(), finished[b].cpu(), 0, W)
            assert [(b * W + w, v) for _, w, v in want] == list(zip(rows[b].tolist(),
                                                                    tokens[b].tolist()))
        src = rows.view(-1).clone()
        if step >= P:
            src[:W] = -1  # the first prompt has ended
            plain[0] = []
        plain = [[plain[b][int(r) - b * W] for r in rows[b]] if plain[b] else [] for b in range(B)]
        finished = finished.gather(1, (rows - W * ints(range(B))[:, None]).clamp(0).long())
        finished[1, W - 1] |= step == 5
        table, seq, refs = ta.kv_fork(pools, table, seq, refs, src, P, reserve=1, status=status)
        if step == P:
            seq[:W] = 0
        if step % 7 == 3:
            table, refs, used = ta.kv_compact(pools, table, refs, status=status)
            m = int(used)
            assert bool((refs[:m] > 0).all()) and bool((refs[m:] == 0).all())
        assert torch.equal(refs, torch.bincount(table[table >= 0].long(), minlength=n).int())
        if not plain[0]:
            scores[0] = -math.inf
            # rows without a sequence: a table of their own for the steps that still run over them
            table, seq, refs = ta.kv_fork(pools, table, seq, refs,
                                          ints([-2] * W + list(range(W, B * W))), P, reserve=1,
                                          status=status)
    assert int(status) == 0
