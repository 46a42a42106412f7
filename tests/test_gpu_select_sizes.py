"""Selection at the corners of its documented range: the widest tables with the largest groups."""
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


@pytest.mark.parametrize("d,G,width,T", [(128, 128, 262144, 1), (128, 97, 262143, 2),
                                         (128, 104, 243713, 1), (64, 128, 262144, 3),
                                         (128, 96, 262144, 1)])
def test_wide_tables_and_large_groups(d, G, width, T):
    P, k, nb = 16, 33, width - 5
    g = torch.Generator("cuda").manual_seed(G)
    mid = torch.randint(-60, 60, (width, 1, d), device="cuda", generator=g)
    half = torch.randint(0, 67, (width, 1, d), device="cuda", generator=g)
    bounds = torch.stack([mid + half, mid - half], 2).to(torch.int8)
    exps = torch.randint(127, 130, (width, 1), dtype=torch.uint8, device="cuda", generator=g)
    row = torch.randperm(width, device="cuda", generator=g).int()[None]
    q = torch.randn(1, T, G, d, device="cuda", generator=g).bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ta.select_blocks(q, bounds, exps, row, torch.tensor([nb * P - 7], dtype=torch.int32,
                                                              device="cuda"), k, P, n_first=1,
                           n_last=2, status=status)
    assert int(status) == 0
    page = row[0, :nb].long()
    hi, lo = bounds[page, 0, 0].double(), bounds[page, 0, 1].double()
    for t in range(T):
        c = context.query_codes(q[0, t].cpu()).double().cuda()
        score = (c.clamp_min(0) @ hi.t() + c.clamp_max(0) @ lo.t()).amax(0)  # whole numbers
        score *= torch.pow(2.0, exps[page, 0].double() - 127)
        score[0] = score[nb - 2:] = torch.inf
        best = torch.sort(score, descending=True, stable=True).indices[:k]
        assert torch.equal(got[0, t, 0].long(), torch.sort(best).values)
