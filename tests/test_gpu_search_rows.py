"""Beam search over selected pages of an 8-bit cache, against plain rows that hold what the
cache holds (each row rounded once by the plain rule): results to the precision of the
attention itself, and the selection by the bounds of those rows."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_tree_split_gb300 as ta
from oracle import context, fp8_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ta.build()
    ta.load()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def held(x):
    """Rows [n][H][d] as the 8-bit cache holds them, fp64 on the CPU."""
    x = x.double().cpu().numpy()
    return torch.from_numpy(np.ascontiguousarray(fp8_rows.decode(*fp8_rows.encode(x))))


@pytest.mark.parametrize("d,P", [(128, 16), (64, 32)])
def test_search_over_rounded_rows(d, P):
    Hkv, G, W, V, steps, k = 2, 4, 4, 61, P + 7, 4
    lens = [6 * P + 3, 11, 5 * P]
    B, N, n = len(lens), sum(lens), 130
    g = torch.Generator("cuda").manual_seed(d + 1)

    def bf(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    def values(m):
        """Values of tokens whose sizes differ by up to 2^24."""
        e = torch.randint(-12, 13, (m, Hkv, 1), generator=g, device="cuda").float()
        return (bf(m, Hkv, d).float() * torch.exp2(e)).bfloat16()
    cache = [torch.full((n, Hkv, P, d), 255, dtype=torch.uint8, device="cuda") for _ in "kv"]
    cache += [torch.full((n, Hkv, P), 255, dtype=torch.uint8, device="cuda") for _ in "kv"]
    bounds = [torch.zeros(n, Hkv, 2, d, dtype=torch.int8, device="cuda"),
              torch.zeros(n, Hkv, dtype=torch.uint8, device="cuda")]
    pools, status = cache + bounds, ints([0])
    table, seq, refs = ta.kv_fork(pools, torch.empty(0, 12, dtype=torch.int32, device="cuda"),
                                  ints([]), ints([0] * n), ints([-2] * B), P, reserve=ints(lens),
                                  status=status)

    def append(table, seq, k, v, counts):
        cu = [0]
        for x in counts:
            cu.append(cu[-1] + x)
        new = ta.kv_append_fp8(*cache, table, seq, ints(cu), k, v, status=status)
        ta.kv_block_bounds(cache[0], table, new, k_scales=cache[2], starts=seq, bounds=bounds[0],
                           bounds_exp=bounds[1], status=status)
        return new
    pk, pv = bf(N, Hkv, d), values(N)
    seq = append(table, seq, pk, pv, lens)
    table, seq, refs = ta.kv_fork(pools, table, seq, refs,
                                  ints([b for b in range(B) for _ in range(W)]), P, reserve=1,
                                  status=status)
    hk, hv = held(pk), held(pv)
    cu = [sum(lens[:b]) for b in range(B + 1)]
    plain = [(hk[cu[b]:cu[b + 1]], hv[cu[b]:cu[b + 1]]) for b in range(B) for _ in range(W)]
    scores = torch.full((B, W), -math.inf, device="cuda")
    scores[:, 0] = 0.0
    for step in range(steps):
        q, tk, tv = bf(B * W, 1, Hkv * G, d), bf(B * W, 1, Hkv, d), values(B * W)[:, None].contiguous()
        blocks = ta.select_blocks(q, *bounds, table, seq, k, P, status=status)
        out, lse = ta.verify_blocks(q, cache[0], cache[1], table, seq, blocks, tk, tv,
                                    parents=ints([-1]), k_scales=cache[2], v_scales=cache[3],
                                    status=status)
        if step % 5 == 0 or step > steps - 3:
            for r, (keys, vals) in enumerate(plain):
                L = int(seq[r])
                assert L == keys.shape[0]
                for h in range(Hkv):
                    qh = q[r, 0, h * G:(h + 1) * G].cpu()
                    hi, lo, e = zip(*(context.page_bounds(keys[j:j + P, h]) for j in range(0, L, P)))
                    own = torch.tensor([hi, lo]).permute(1, 0, 2).to(torch.int8)
                    want = context.choose(qh, own, torch.tensor(e), k, 1, 1)
                    assert blocks[r, 0, h].tolist() == want + [-1] * (k - len(want))
                    see = [i for j in want for i in range(j * P, min(j * P + P, L))]
                    ks = torch.cat([keys[see, h], tk[r, :, h].double().cpu()])
                    vs = torch.cat([vals[see, h], tv[r, :, h].double().cpu()])
                    ref, ref_l = context.attend(qh, ks, vs, 1 / math.sqrt(d))
                    # d products of a score in fp32 (e), probabilities in fp16 (2^-12 of
                    # themselves, or 2^-31 of the row's largest p max|v| a key), results in bf16
                    p = torch.exp(qh.double() @ ks.t() / math.sqrt(d) - ref_l[:, None])
                    err = float((qh.double().abs() @ ks.abs().t()).max()) / math.sqrt(d) * 2.0 ** -21
                    err += 2.0 ** -20
                    largest = (p * vs.abs().amax(1)).amax(1)[:, None]
                    tol = p @ vs.abs() * (2 * err + 2.0 ** -11) + largest * len(see) * 2.0 ** -31
                    o = out[r, 0, h * G:(h + 1) * G].double().cpu()
                    assert bool(((o - ref).abs() <= tol + ref.abs() * 2.0 ** -8).all())
                    l = lse[r, 0, h * G:(h + 1) * G].double().cpu()
                    assert bool(((l - ref_l).abs() <= err + ref_l.abs() * 2.0 ** -22 + 2.0 ** -20).all())
        seq = append(table, seq, tk[:, 0], tv[:, 0], [1] * (B * W))
        hk, hv = held(tk[:, 0]), held(tv[:, 0])
        plain = [(torch.cat([x, hk[r:r + 1]]), torch.cat([y, hv[r:r + 1]]))
                 for r, (x, y) in enumerate(plain)]
        logits = 2 * torch.randn(B, W, V, generator=g, device="cuda")
        before = scores
        scores, rows, tokens = ta.beam_select(logits, before, W)
        for b in range(B):
            want = context.beams(logits[b].cpu(), before[b].cpu(), None, None, W)
            assert [(b * W + w, v) for _, w, v in want] == list(zip(rows[b].tolist(),
                                                                    tokens[b].tolist()))
        plain = [plain[r] for r in rows.view(-1).tolist()]
        table, seq, refs = ta.kv_fork(pools, table, seq, refs, rows.view(-1), P, reserve=1,
                                      status=status)
        if step % 4 == 1:
            table, refs, used = ta.kv_compact(pools, table, refs, status=status)
        assert torch.equal(refs, torch.bincount(table[table >= 0].long(), minlength=n).int())
    assert int(status) == 0
