"""Tree attention over selected pages against 64-bit attention over the same rows."""
import math
import random

import pytest
import torch

import speculative_decoding_tree_split_gb300 as ta
from oracle import context
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


class Case:
    """A cache with sequences of the given lengths, in random pages; what lies
    behind their ends is NaN (bf16) or any code and scale."""

    def __init__(self, lens, Hkv, G, d, P, T, k, fp8, seed=0, gain=1.0):
        r = random.Random(seed)
        g = torch.Generator("cuda").manual_seed(seed)
        self.lens, self.P, self.fp8, self.Hkv, self.G, self.d, self.T = lens, P, fp8, Hkv, G, d, T
        B = len(lens)
        pages = [-(-n // P) for n in lens]
        n = sum(pages) + 2
        ids = list(range(n))
        r.shuffle(ids)
        width = max(pages + [1])
        self.rows = [[ids.pop() for _ in range(m)] + [-1] * (width - m) for m in pages]

        def bf(*shape):
            return torch.randn(*shape, generator=g, device="cuda").bfloat16()

        def pool():
            if fp8:
                c = torch.randint(0, 256, (n, Hkv, P, d), dtype=torch.uint8, device="cuda", generator=g)
                c[(c & 0x7f) == 0x7f] = 0x30  # no NaN among committed rows
                s = torch.randint(116, 122, (n, Hkv, P), dtype=torch.uint8, device="cuda", generator=g)
                return c, s
            return bf(n, Hkv, P, d), None
        (self.k, self.ks), (self.v, self.vs) = pool(), pool()
        for b, L in enumerate(lens):
            if L % P:
                page = self.rows[b][L // P]
                for x, s in ((self.k, self.ks), (self.v, self.vs)):
                    x[page, :, L % P:] = 0x7f if fp8 else math.nan
                    if fp8:
                        s[page, :, L % P:] = 255
        self.q = (bf(B, T, Hkv * G, d) * gain).contiguous()
        self.tk, self.tv = bf(B, T, Hkv, d), bf(B, T, Hkv, d)
        self.parents = random_tree(T, 5, 3, torch.Generator().manual_seed(seed)).int().cuda()
        lists = []
        for b in range(B):
            for _ in range(T * Hkv):
                m = min(k, pages[b])
                row = r.sample(range(pages[b]), m) + [-1] * (k - m)
                if r.random() < 0.5:
                    r.shuffle(row)  # in any order, -1 anywhere
                lists.append(row)
        self.blocks = ints(lists).view(B, T, Hkv, k)

    def values(self, pool, scales, page, h, n):
        x = pool[page, h, :n]
        return (context.row_values(x, scales[page, h, :n]) if self.fp8 else x.double()).cpu()

    def sees(self, b, t):
        up = self.parents if self.parents.dim() == 1 else self.parents[b]
        out, j = [], t
        while j >= 0:
            out.append(j)
            j = int(up[j])
        return out

    def call(self, **kw):
        args = dict(parents=self.parents)
        args.update(kw)
        return ta.verify_blocks(self.q, self.k, self.v, ints(self.rows), ints(self.lens), self.blocks,
                                self.tk, self.tv, k_scales=self.ks, v_scales=self.vs, **args)

    def check(self, sees=None, scale=None, **kw):
        status = ints([0])
        out, lse = self.call(status=status, softmax_scale=scale, **kw)
        assert int(status) == 0
        out, lse = out.double().cpu(), lse.double().cpu()
        scale = scale or 1 / math.sqrt(self.d)
        G = self.G
        for b, L in enumerate(self.lens):
            for t in range(self.T):
                tree = (sees or self.sees)(b, t)
                for h in range(self.Hkv):
                    ks = [self.tk[b, tree, h].double().cpu()]
                    vs = [self.tv[b, tree, h].double().cpu()]
                    for j in sorted(set(self.blocks[b, t, h].tolist())):  # twice counts once
                        if j >= 0:
                            n, page = min(self.P, L - j * self.P), self.rows[b][j]
                            ks.append(self.values(self.k, self.ks, page, h, n))
                            vs.append(self.values(self.v, self.vs, page, h, n))
                    rows = slice(h * G, (h + 1) * G)
                    ks, vs = torch.cat(ks), torch.cat(vs)
                    ref, ref_l = context.attend(self.q[b, t, rows].cpu(), ks, vs, scale)
                    # A score is a sum of d products in fp32 (relative 2^-24 each, of sum |q k|),
                    # its exponent's argument and ex2 about as much: with `e` the bound on a
                    # score's error the probabilities are off by e, the result by 2 e max|v| at
                    # most; the 8-bit form rounds probabilities to 2^-12 of themselves; then
                    # half a bf16 step.
                    size = (self.q[b, t, rows].cpu().double().abs() @ ks.abs().t() * abs(scale))
                    e = float(size.max() if size.numel() else 0) * 2.0 ** -21 + 2.0 ** -20
                    top = float(vs.abs().max()) if vs.numel() else 0.0
                    tol = 2 * (e + (2.0 ** -12 if self.fp8 else 2.0 ** -17)) * top
                    o, l = out[b, t, rows], lse[b, t, rows]
                    assert bool(((o - ref).abs() <= tol + ref.abs() * 2.0 ** -8).all()), (b, t, h)
                    if ks.shape[0]:
                        assert bool(((l - ref_l).abs() <= e + ref_l.abs() * 2.0 ** -22).all()), (b, t, h)
                    else:
                        assert bool((l == -math.inf).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hkv,G,d,P,T,k", [
    (2, 4, 128, 64, 1, 4), (1, 1, 64, 16, 1, 1), (2, 5, 128, 16, 3, 7), (1, 8, 64, 128, 2, 2),
    (1, 12, 128, 32, 2, 3), (1, 16, 64, 64, 1, 3), (1, 40, 128, 16, 1, 9), (2, 2, 64, 32, 17, 5),
    (1, 3, 128, 16, 64, 2), (1, 4, 128, 64, 1, 40)])
def test_against_64_bits(Hkv, G, d, P, T, k, fp8):
    lens = [0, 1, P - 1, P, 2 * P + 5, 47 * P + 3]
    Case(lens, Hkv, G, d, P, T, k, fp8, seed=P + T).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_masks(d, fp8):
    c = Case([0, 100, 31], 2, 4, d, 16, 6, 3, fp8, seed=3)
    bits = [0, 1, 0b100110, 0b111111, 1 << 5, 0]
    low = 0xffffffffffffffc0  # bits past T are ignored
    one = torch.tensor([x | low if x | low < 1 << 63 else (x | low) - (1 << 64) for x in bits],
                       device="cuda")
    c.check(lambda b, t: [j for j in range(6) if bits[t] >> j & 1], mask=one, parents=None)
    each = torch.tensor([bits, bits[::-1], [63] * 6], device="cuda")
    c.check(lambda b, t: [j for j in range(6) if int(each[b, t]) >> j & 1], mask=each, parents=None)
    c.parents = torch.stack([random_tree(6, 4, 2, torch.Generator().manual_seed(i)).int()
                             for i in range(3)]).cuda()
    c.check()
    c.blocks.fill_(-1)  # the tree alone
    c.check()
    c.blocks = c.blocks[..., :0].contiguous()
    c.check(lambda b, t: [j for j in range(6) if bits[t] >> j & 1], mask=one, parents=None)


@pytest.mark.parametrize("fp8", [False, True])
def test_scores_far_apart_and_a_first_key_that_draws_most(fp8):
    c = Case([700, 64], 1, 4, 128, 64, 2, 11, fp8, seed=5, gain=30.0)
    c.check()
    c = Case([700], 1, 4, 128, 64, 2, 11, fp8, seed=6)
    page = c.rows[0][0]
    if fp8:
        c.ks[page, 0, 0] += 6
        c.k[page, 0, 0] &= 0x7f
    else:
        c.k[page, 0, 0] = c.k[page, 0, 0].abs() * 40
    c.q.abs_()
    c.check()
    c.check(scale=-0.3)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_scale_of_zero_gives_the_mean(fp8):
    c = Case([70], 1, 4, 64, 16, 2, 3, fp8, seed=17)
    out, lse = c.call(softmax_scale=0.0)
    for t in range(2):
        vs = [c.tv[0, c.sees(0, t), 0].double().cpu()]
        for j in c.blocks[0, t, 0].tolist():
            if j >= 0:
                vs.append(c.values(c.v, c.vs, c.rows[0][j], 0, min(16, 70 - 16 * j)))
        vs = torch.cat(vs)
        assert float((out[0, t].double().cpu() - vs.mean(0)).abs().max()) <= float(
            vs.mean(0).abs().max()) * 2.0 ** -8 + float(vs.abs().max()) * 2.0 ** -11
        assert float((lse[0, t] - math.log(vs.shape[0])).abs().max()) <= 1e-5


def test_value_scales_far_apart():
    c = Case([640], 2, 4, 128, 64, 2, 10, True, seed=8)
    for j, page in enumerate(c.rows[0]):
        c.vs[page] = [71, 120, 167, 90, 71, 100, 130, 80, 167, 71][j]
        c.ks[page] = 100 + j
    out, lse = c.call()
    for h in range(2):
        for t in range(2):
            ks, vs = [c.tk[0, c.sees(0, t), h].double()], [c.tv[0, c.sees(0, t), h].double()]
            for j in c.blocks[0, t, h].tolist():
                ks.append(context.row_values(c.k[c.rows[0][j], h], c.ks[c.rows[0][j], h]))
                vs.append(context.row_values(c.v[c.rows[0][j], h], c.vs[c.rows[0][j], h]))
            q = c.q[0, t, 4 * h:4 * h + 4]
            ref, ref_l = context.attend(q, torch.cat(ks), torch.cat(vs), 1 / math.sqrt(128))
            o = out[0, t, 4 * h:4 * h + 4].double()
            # 2^-12 of the probabilities, and half a bf16 step, relative to the largest value's part
            p = torch.exp((q.double() @ torch.cat(ks).t()) / math.sqrt(128) - ref_l[:, None])
            part = p @ torch.cat(vs).abs()
            assert bool(((o - ref).abs() <= part * 2.0 ** -11 + ref.abs() * 2.0 ** -8).all())


def test_a_value_that_is_no_number_reaches_the_rows_that_list_its_page():
    c = Case([64, 64], 1, 4, 64, 16, 1, 2, False, seed=9)
    c.blocks[0, 0, 0] = ints([0, 1])
    c.blocks[1, 0, 0] = ints([2, 3])
    before, _ = c.call()
    c.v[c.rows[0][2], 0, 3] = math.nan
    c.v[c.rows[0][3], 0, 5] = math.inf
    c.v[c.rows[1][2], 0, 3, 7] = math.nan
    after, _ = c.call()
    assert torch.equal(before[0], after[0])
    assert bool(after[1, 0, :, 7].isnan().all())
    keep = [i for i in range(64) if i != 7]
    assert torch.equal(before[1, 0][:, keep], after[1, 0][:, keep])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_value_that_is_no_number_stays_with_the_tokens_that_see_it(fp8, d):
    """Tokens that are worked on together, of which some list a page (see a tree token)
    with such a value."""
    c = Case([64], 1, 4, d, 16, 4, 2, fp8, seed=15)
    c.parents = ints([-1, 0, 0, 2])
    for t, pages in enumerate(([0, 1], [1, 2], [0, 2], [1, 3])):
        c.blocks[0, t, 0] = ints(pages)
    before, _ = c.call()
    page = c.rows[0][2]
    if fp8:
        c.v[page, 0, 5, 3] = 0x7f
    else:
        c.v[page, 0, 5, 3] = math.nan
        c.v[page, 0, 7, 9] = math.inf
    after, _ = c.call()
    bad = {1, 2}
    for t in range(4):
        assert torch.equal(before[0, t], after[0, t]) == (t not in bad)
    assert bool(after[0, 1:3, :, 3].isnan().all()) and int(after[0, :, :, 3].isnan().sum()) == 8
    keep = [i for i in range(d) if i not in (3, 9)]
    assert torch.equal(before[0, 1:3][..., keep], after[0, 1:3][..., keep])
    c.v[page, 0] = 0
    before, _ = c.call()
    c.tv[0, 2, 0, 11] = math.nan  # tokens 2 and 3 see it
    after, _ = c.call()
    assert torch.equal(before[0, :2], after[0, :2])
    assert bool(after[0, 2:, :, 11].isnan().all())
    keep = [i for i in range(d) if i != 11]
    assert torch.equal(before[0, 2:][..., keep], after[0, 2:][..., keep])


@pytest.mark.parametrize("fp8", [False, True])
def test_lists_over_many_pages_and_cache_rows_off_32_byte_boundaries(fp8):
    P, L = 16, 20000 * 16 - 5  # pages of a sequence in more than one stretch
    c = Case([L, 70], 1, 2, 64, P, 3, 6, fp8, seed=16)
    c.blocks[0, :, 0] = ints([[0, 8191, 8192, 16383, 16384, 19999], [19999, 4, 8192, -1, 4, 12000],
                              [7, 8, 9, 16384, 16385, 16386]])
    c.check()
    for name in "kv":  # the same pools 16 bytes further on
        x = getattr(c, name)
        room = torch.empty(x.nbytes + 16, dtype=torch.uint8, device="cuda")
        y = room[16:].view(x.dtype).view(x.shape)
        y.copy_(x)
        setattr(c, name, y)
    assert c.k.data_ptr() % 32 == 16
    c.check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,G", [(1, 1), (5, 4)])
def test_the_longest_lists(T, G, fp8):
    Case([16 * 4100, 31], 1, G, 128, 16, T, 4096, fp8, seed=23).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_all_pages_are_the_whole_cache_and_twice_counts_once(fp8):
    c = Case([300, 17], 2, 4, 128, 16, 5, 19, fp8, seed=10)
    for b, L in enumerate(c.lens):
        nb = -(-L // 16)
        c.blocks[b] = ints(list(range(nb)) + [-1] * (19 - nb))
    out, lse = c.call()
    args = (ints(c.rows), ints(c.lens), c.tk, c.tv)
    want = (ta.verify_fp8(c.q, c.k, c.v, c.ks, c.vs, *args, parents=c.parents) if fp8 else
            ta.verify_tree(c.q, c.k, c.v, *args, c.parents))
    assert float((out.double() - want[0].double()).abs().max()) <= (5e-2 if fp8 else 2e-2)
    assert float((lse - want[1]).abs().max()) <= 1e-3
    c.blocks[0, :, :, 1] = 0
    c.blocks[1, :, :, 1] = 0
    c.check()
    c = Case([300], 2, 4, 128, 16, 1, 19, fp8, seed=20)
    c.blocks[0, 0, 0, :4] = ints([3, 3, -1, 3])
    c.check()


def test_blocks_outside_the_sequence_are_skipped_and_reported():
    c = Case([40, 16], 1, 2, 64, 16, 1, 3, False, seed=11)
    c.blocks[0, 0, 0] = ints([0, 2, -1])
    c.blocks[1, 0, 0] = ints([0, -1, -1])
    want = c.call()
    for bad in (3, 100, -2):
        c.blocks[0, 0, 0, 2] = bad
        status = ints([0])
        got = c.call(status=status)
        assert int(status) == ta.STATUS_BAD_PAGE
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.blocks[0, 0, 0, 2] = -1
    for lens, code in (([49, 16], ta.STATUS_BAD_SEQ_LEN), ([-1, 16], ta.STATUS_BAD_SEQ_LEN)):
        c.lens, status = lens, ints([0])
        c.call(status=status)
        assert int(status) == code
    c.lens, c.rows[0][0], status = [40, 16], 99, ints([0])
    c.call(status=status)
    assert int(status) == ta.STATUS_BAD_PAGE
    c.rows[0][0] = 0
    c = Case([40], 1, 2, 64, 16, 3, 2, False, seed=12)
    for parents in ([-1, 0, 2], [-1, -2, 0], [0, 0, 1]):
        status = ints([0])
        c.call(parents=ints(parents), status=status)
        assert int(status) == ta.STATUS_BAD_PARENT


def test_pool_past_32_bits():
    """The last page lies past 2^32 bytes of the pools."""
    n, H, P, d = 2150, 64, 128, 128
    g = torch.Generator("cuda").manual_seed(1)
    k, v = (torch.empty(n, H, P, d, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    for x in (k, v):
        x[n - 1] = torch.randn(H, P, d, device="cuda", generator=g)
    q, tk, tv = (torch.randn(1, 1, H, d, device="cuda", generator=g).bfloat16() for _ in range(3))
    blocks = ints([0]).expand(1, 1, H, 1).contiguous()
    out, _ = ta.verify_blocks(q, k, v, ints([[n - 1]]), ints([100]), blocks, tk, tv, parents=ints([-1]))
    for h in (0, 63):
        ref, _ = context.attend(q[0, 0, h:h + 1], torch.cat([k[n - 1, h, :100], tk[0, :, h]]).double(),
                                torch.cat([v[n - 1, h, :100], tv[0, :, h]]).double(), 1 / math.sqrt(d))
        assert float((out[0, 0, h] - ref[0]).abs().max()) <= 1e-2


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_replayed_and_on_another_stream(fp8):
    c = Case([500, 33], 2, 4, 128, 16, 2, 8, fp8, seed=13)
    rows, lens = ints(c.rows), ints(c.lens)
    out, lse = torch.empty_like(c.q), torch.empty(2, 2, 8, device="cuda")

    def call(**kw):
        return ta.verify_blocks(c.q, c.k, c.v, rows, lens, c.blocks, c.tk, c.tv, parents=c.parents,
                                k_scales=c.ks, v_scales=c.vs, **kw)
    want = [t.clone() for t in call()]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    call(out=out, lse=lse, stream=stream)
    stream.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=out, lse=lse)
    c.q.neg_()
    graph.replay()
    torch.cuda.synchronize()
    again = call()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert not torch.equal(out, want[0])


def test_refusals():
    c = Case([40], 1, 2, 64, 16, 1, 2, False, seed=14)
    f = Case([40], 1, 2, 64, 16, 1, 2, True, seed=14)
    with pytest.raises(ValueError):
        c.call(mask=torch.ones(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        c.call(parents=None)
    with pytest.raises(ValueError):
        c.call(parents=ints([-1, 0]))
    c.ks = f.ks
    with pytest.raises(ValueError):
        c.call()
    c.vs = f.vs
    with pytest.raises(TypeError):
        c.call()
    f.ks = f.vs = None
    with pytest.raises(TypeError):
        f.call()
    c.ks = c.vs = None
    c.blocks = c.blocks.long()
    with pytest.raises(TypeError):
        c.call()
    c.blocks = c.blocks.int()[:, :, :, :1].expand(1, 1, 1, 2)
    with pytest.raises(ValueError):
        c.call()
    c.blocks = ints([-1] * 4097).view(1, 1, 1, 4097)
    with pytest.raises(ta.TreeAttnError):
        c.call()
    c.blocks = ints([0]).view(1, 1, 1, 1)
    with pytest.raises(ta.TreeAttnError):
        c.call(softmax_scale=math.nan)
    with pytest.raises(ValueError):
        c.call(out=torch.empty(1, 1, 2, 32, device="cuda", dtype=torch.bfloat16))
