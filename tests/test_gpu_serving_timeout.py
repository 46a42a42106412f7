"""A pipeline wait that runs out in the pass over the 8-bit cache and in the
prompt attention: with a limit of 1 ns, far below the microseconds a tile takes
to arrive, the call reports TREE_ATTN_STATUS_TIMEOUT, lets its copies and MMAs in
flight finish and returns; with the limit restored, the same call on the same
stream gives the bits it gave before."""
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


def _times_out(run):
    seen = []
    assert ta.set_wait_limit_ns(1) == ta.DEFAULT_WAIT_NS
    try:
        for _ in range(3):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            run(status)
            torch.cuda.synchronize()
            seen.append(int(status))
            if seen[-1] == ta.STATUS_TIMEOUT:
                break
    finally:
        assert ta.set_wait_limit_ns(0) == 1
    assert ta.STATUS_TIMEOUT in seen and set(seen) <= {0, ta.STATUS_TIMEOUT}, seen


@pytest.mark.parametrize("d,P,T,Hq", [(128, 64, 4, 8), (64, 16, 16, 10)])
def test_verify_fp8(d, P, T, Hq):
    g = torch.Generator("cuda").manual_seed(d)
    B, Hkv, L = 3, 2, 6000
    pages = -(-L // P)
    n = B * pages

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    pool = [torch.randint(0, 120, (n, Hkv, P, d), generator=g, device="cuda", dtype=torch.uint8)
            for _ in "kv"]
    scale = [torch.randint(116, 120, (n, Hkv, P), generator=g, device="cuda", dtype=torch.uint8)
             for _ in "kv"]
    bt = torch.arange(n, device="cuda", dtype=torch.int32).view(B, pages)
    sl = torch.full((B,), L, device="cuda", dtype=torch.int32)
    x = (rnd(B, T, Hq, d), *pool, *scale, bt, sl, rnd(B, T, Hkv, d), rnd(B, T, Hkv, d))
    par = torch.arange(-1, T - 1, device="cuda", dtype=torch.int32)
    want = ta.verify_fp8(*x, parents=par)
    torch.cuda.synchronize()
    _times_out(lambda status: ta.verify_fp8(*x, parents=par, status=status))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ta.verify_fp8(*x, parents=par, status=status)
    assert int(status) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("d", [128, 64])
def test_prefill(d):
    g = torch.Generator("cuda").manual_seed(d)
    cu = torch.tensor([0, 3000, 3001, 9000], dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn(9000, h, d, generator=g, device="cuda").bfloat16() for h in (8, 2, 2))
    want = ta.prefill(q, k, v, cu)
    torch.cuda.synchronize()
    _times_out(lambda status: ta.prefill(q, k, v, cu, status=status))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ta.prefill(q, k, v, cu, status=status)
    assert int(status) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
