"""The operators together, as a server runs them: prompts through prefill and
into the 8-bit cache, draft trees verified over it, the accepted path committed
into it, and the next step verified again -- each step against 64-bit
attention over what the cache then stands for."""
import math

import pytest
import torch

import speculative_decoding_tree_split_gb300 as ta
from workloads import random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ta.build()
    ta.load()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d,P,Hq,Hkv,T", [(128, 64, 8, 2, 6), (64, 16, 5, 1, 9)])
def test_prompt_to_second_verification(d, P, Hq, Hkv, T):
    lens = [1, 70, 333]
    B, N = len(lens), sum(lens)
    cu = [0, 1, 71, 404]
    g = torch.Generator("cuda").manual_seed(d)

    def bf(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    qkv = bf(N, Hq + 2 * Hkv, d)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    out, lse = ta.prefill(q, k, v, ints(cu))
    for a, b in zip(cu[:-1], cu[1:]):  # the last token sees its whole prompt
        x = torch.einsum("hd,nhd->hn", q[b - 1].double(),
                         k[a:b].double().repeat_interleave(Hq // Hkv, 1)) / math.sqrt(d)
        ref = torch.einsum("hn,nhd->hd", x.softmax(1),
                           v[a:b].double().repeat_interleave(Hq // Hkv, 1))
        assert float((out[b - 1].double() - ref).abs().max()) <= 1e-2
        assert float((lse[b - 1].double() - x.logsumexp(1)).abs().max()) <= 1e-3

    steps = 2
    pages = [-(-(n + steps * T) // P) for n in lens]
    order = torch.randperm(sum(pages) + 1).int()
    bt = torch.full((B, max(pages)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        bt[b, :n] = order[at:at + n]
        at += n
    bt = bt.cuda()
    n = sum(pages) + 1
    cache = [torch.full((n, Hkv, P, d), 255, dtype=torch.uint8, device="cuda") for _ in "kv"]
    cache += [torch.full((n, Hkv, P), 255, dtype=torch.uint8, device="cuda") for _ in "kv"]
    cache.append(bt)
    status = ints([0])
    seq = ta.kv_append_fp8(*cache, ints([0] * B), ints(cu), k, v, status=status)
    assert seq.tolist() == lens
    for step in range(steps):
        parents = random_tree(T, 4, 3, torch.Generator().manual_seed(step)).cuda()
        tq, tk, tv = bf(B, T, Hq, d), bf(B, T, Hkv, d), bf(B, T, Hkv, d)
        mask = torch.empty(T, dtype=torch.int64, device="cuda")
        out, lse = ta.verify_fp8(tq, *cache, seq, tk, tv, parents=parents, mask_out=mask,
                                 status=status)
        total = [int(x) for x in seq]
        ccu = ints([sum(total[:b]) for b in range(B + 1)])
        ck, cv = ta.kv_read_fp8(*cache, ccu, sum(total), status=status)
        see = torch.tensor([[(int(m) >> j) & 1 for j in range(T)] for m in mask.tolist()],
                           device="cuda").bool()
        for b in range(B):
            a, e = int(ccu[b]), int(ccu[b + 1])
            kk = torch.cat([ck[a:e], tk[b]]).double().repeat_interleave(Hq // Hkv, 1)
            vv = torch.cat([cv[a:e], tv[b]]).double().repeat_interleave(Hq // Hkv, 1)
            x = torch.einsum("thd,nhd->thn", tq[b].double(), kk) / math.sqrt(d)
            x[..., e - a:] = x[..., e - a:].masked_fill(~see[:, None], -math.inf)
            ref = torch.einsum("thn,nhd->thd", x.softmax(2), vv)
            assert float((out[b].double() - ref).abs().max()) <= 1e-2
            assert float((lse[b].double() - x.logsumexp(2)).abs().max()) <= 1e-3
        draft = torch.randint(0, 2, (B, T), generator=g, device="cuda", dtype=torch.int32)
        target = torch.randint(0, 2, (B, T), generator=g, device="cuda", dtype=torch.int32)
        length, path, _ = ta.greedy_accept(mask, draft, target)
        new = ta.kv_commit_fp8(*cache, seq, path, length, tk, tv, status=status)
        assert torch.equal(new, seq + length)
        # what was committed reads back as the accepted rows, to half a step
        m = int(length.sum())
        lcu = torch.cat([ints([0]), length.cumsum(0).int()])
        rk, _ = ta.kv_read_fp8(*cache, lcu, m, starts=seq, status=status)
        want = torch.cat([tk[b, path[b, :int(length[b])].long()] for b in range(B)]).double()
        top = want.abs().amax(-1, keepdim=True)
        assert bool(((rk.double() - want).abs()
                     <= 2.0 ** -4 * torch.maximum(want.abs(), top * 2.0 ** -13)).all())
        seq = new
    assert int(status) == 0
