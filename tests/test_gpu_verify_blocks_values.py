"""Attention over selected pages of an 8-bit cache whose value scales lie far apart: what a
row gets is held to that row's own largest value, whatever other tokens list."""
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


class Cache:
    """Sequences of 24 pages of an 8-bit cache; page 0 of each has value scales 2^far above
    the others'.  Queries are positive, page 0's keys negative where `faint`: each of its
    keys then has e^-60 of a probability, or so."""

    B, H, G, pages, k = 40, 4, 4, 24, 20

    def __init__(self, P, T, d, far, faint, seed, low=100):
        g = torch.Generator("cuda").manual_seed(seed)
        self.P, self.T, self.d = P, T, d
        n = self.B * self.pages
        self.rows = torch.randperm(n, generator=g, device="cuda").int().view(self.B, self.pages)
        c = torch.randint(0, 256, (2, n, self.H, P, d), dtype=torch.uint8, device="cuda", generator=g)
        c[(c & 0x7f) == 0x7f] = 0x30
        c[..., 0] = 0x7e  # (rows as the cache holds them: their largest code is large)
        self.k_pages, self.v_pages = c
        self.ks = torch.full((n, self.H, P), 119, dtype=torch.uint8, device="cuda")
        self.vs = torch.randint(low, low + 3, (n, self.H, P), dtype=torch.uint8, device="cuda",
                                generator=g)
        first = self.rows[:, 0].long()
        self.vs[first] = self.vs[first] + far

        def bf(*shape):
            return torch.randn(*shape, generator=g, device="cuda").bfloat16()
        self.q = bf(self.B, T, self.H * self.G, d)
        if faint:
            self.q.abs_()
            self.k_pages[first] = 0xbd  # -1.625, times 2^2 or 2^3: q.k / sqrt(d) is about -60
            self.ks[first] = 129 if d == 128 else 130
        self.tk = bf(self.B, T, self.H, d)
        self.tv = (bf(self.B, T, self.H, d) * 2.0 ** (low - 119)).bfloat16()

    def check(self, blocks):
        B, H, G, T, P, d = self.B, self.H, self.G, self.T, self.P, self.d
        status = ints([0])
        lens = ints([self.pages * P] * B)
        out, lse = ta.verify_blocks(self.q, self.k_pages, self.v_pages, self.rows, lens, blocks,
                                    self.tk, self.tv, parents=ints([-1] * T), k_scales=self.ks,
                                    v_scales=self.vs, status=status)
        assert int(status) == 0
        worst = 0.0
        for b in range(0, B, 7):
            for t in range(T):
                for h in range(H):
                    page = self.rows[b, blocks[b, t, h].long()].long()
                    ks = context.row_values(self.k_pages[page, h], self.ks[page, h]).view(-1, d)
                    vs = context.row_values(self.v_pages[page, h], self.vs[page, h]).view(-1, d)
                    n = ks.shape[0]
                    ks = torch.cat([ks, self.tk[b, t:t + 1, h].double()])
                    vs = torch.cat([vs, self.tv[b, t:t + 1, h].double()])
                    q = self.q[b, t, h * G:(h + 1) * G].double()
                    ref, ref_l = context.attend(q, ks, vs, 1 / math.sqrt(d))
                    p = torch.exp(q @ ks.t() / math.sqrt(d) - ref_l[:, None])
                    # Scores: d products in fp32 (2^-24 of the sum of magnitudes each, as e), which
                    # p and the sum follow; p to fp16: 2^-12 of itself, or 2^-31 of the row's
                    # largest p max|v| a key; the result to bf16.
                    e = float((q.abs() @ ks.abs().t()).max()) / math.sqrt(d) * 2.0 ** -21 + 2.0 ** -20
                    part = p @ vs.abs()
                    largest = (p[:, :n] * vs[:n].abs().amax(1)).amax(1)
                    tol = part * (2 * e + 2.0 ** -11) + largest[:, None] * n * 2.0 ** -31
                    o = out[b, t, h * G:(h + 1) * G].double()
                    ratio = (o - ref).abs() / (tol + ref.abs() * 2.0 ** -8)
                    worst = max(worst, float(ratio.max()))
                    l = lse[b, t, h * G:(h + 1) * G].double()
                    assert bool(((l - ref_l).abs() <= e + ref_l.abs() * 2.0 ** -22 + 2.0 ** -20).all())
        assert worst <= 1.0, worst


def lists(T, others, seed):
    """Page lists [B][T][H][k]: the last `others` tokens list page 0, the first ones do not."""
    r = random.Random(seed)
    out = []
    for _ in range(Cache.B):
        for t in range(T):
            for _ in range(Cache.H):
                if t >= T - others:
                    out.append([0] + sorted(r.sample(range(1, Cache.pages), Cache.k - 1)))
                else:
                    out.append(sorted(r.sample(range(1, Cache.pages), Cache.k)))
    return ints(out).view(Cache.B, T, Cache.H, Cache.k)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [16, 128])
@pytest.mark.parametrize("far", [20, 24, 32, 40])
def test_a_large_value_scale_in_a_page_that_only_another_token_lists(far, P, d):
    Cache(P, 4, d, far, False, far + P).check(lists(4, 1, far))


@pytest.mark.parametrize("P", [16, 128])
@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("far", [20, 24, 32, 40])
def test_a_large_value_scale_of_keys_that_hardly_count(far, T, P):
    Cache(P, T, 128, far, True, far + P).check(lists(T, T, far))


@pytest.mark.parametrize("faint", [False, True])
@pytest.mark.parametrize("T", [1, 4])
def test_the_widest_range_of_value_scales(T, faint):
    """All that the cache's bytes allow: 2^-56 to 2^40."""
    Cache(16, T, 64, 94, faint, 7, low=71).check(lists(T, 1, 3))
