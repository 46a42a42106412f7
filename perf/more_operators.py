"""The measured cases of the operators for long contexts and several hypotheses.

What a server does to its paged cache beside filling it and attending over it:

* ``bounds``: for each (page, KV head) the largest and the smallest key of every
  channel, in 8 bits, rounded outwards; written when tokens arrive.
* ``select``: for each query the pages whose bounds allow the largest scores.
* ``attend``: attention of a draft tree (T = 1: plain decoding) over the selected
  pages, plus the tree tokens its mask allows; cache in bf16 or in 8-bit rows.
* ``fork``: the rows of the next step from the rows of this one -- beams that go
  on from the same parent share its full pages and get a copy of the last one,
  rows that end give their pages back, rows that grow get new pages.
* ``compact``: used pages moved to the front of the pool.
* ``beam``: the best continuations over all beams and the vocabulary.

``run`` gives the framework's calls when ``own`` is set and otherwise the same
results from elementary tensor operations.
"""
import math
import random

import torch

own = False

E_MIN, E_MAX = -100, 100          # exponents of bounds and of query codes
S_MIN, S_MAX, CODE_MAX = -56, 40, 448.0  # of the 8-bit cache's rows


def listed():
    return [
        # Bounds of one prompt of 8192 tokens that a Llama-3.1-8B layer took in.
        dict(name="bounds_prompt_8b", op="bounds", B=1, lo=8192, hi=8192, new=8192, Hkv=8, d=128,
             page=64, fp8=False),
        # The step after verification at the large batch: the pages that up to 4
        # new tokens of each sequence touch (latency counts).
        dict(name="bounds_step_b64", op="bounds", B=64, lo=512, hi=16384, new=4, Hkv=8, d=128,
             page=64, fp8=True),
        # One token of one long sequence chooses 64 of 512 pages.
        dict(name="select_decode_b1", op="select", B=1, lo=32768, hi=32768, T=1, Hq=32, Hkv=8,
             d=128, page=64, k=64),
        # The 4-token drafts of 64 sequences choose among up to 1024 small pages.
        dict(name="select_chain_b64", op="select", B=64, lo=512, hi=16384, T=4, Hq=32, Hkv=8,
             d=128, page=16, k=64),
        # One token of a sequence of 131072 tokens over 64 of its 2048 pages, bf16 cache.
        dict(name="attend_decode_128k", op="attend", B=1, lo=131072, hi=131072, T=1, Hq=32, Hkv=8,
             d=128, page=64, k=64, fp8=False),
        # The drafts of the large batch over 32 pages each, 8-bit cache.
        dict(name="attend_chain_b64", op="attend", B=64, lo=512, hi=16384, T=4, Hq=32, Hkv=8,
             d=128, page=64, k=32, fp8=True),
        # Eight beams of one prompt take their next step (one layer's pools).
        dict(name="fork_b1_w8", op="fork", B=1, W=8, lo=8200, hi=8200, Hkv=8, d=128, page=64,
             layers=1, fp8=False, reserve=1, done=0),
        # 32 prompts with eight beams each, four layers' 8-bit pools, some prompts done.
        dict(name="fork_b32_w8", op="fork", B=32, W=8, lo=512, hi=4096, Hkv=8, d=128, page=64,
             layers=4, fp8=True, reserve=4, done=3),
        # A small pool with holes.
        dict(name="compact_256", op="compact", pages=256, used=100, B=8, Hkv=8, d=128, page=64,
             layers=1, fp8=False),
        # Two layers' pools after most of a batch has ended.
        dict(name="compact_4096", op="compact", pages=4096, used=1600, B=48, Hkv=8, d=128, page=64,
             layers=2, fp8=True),
        # Four beams of one sequence, a vocabulary of 32000 (latency counts).
        dict(name="beam_b1_w4", op="beam", B=1, W=4, V=32000, k=4, dtype="bf16", done=False),
        # 64 sequences of eight beams, fp32 logits over 128000 tokens, some beams finished.
        dict(name="beam_b64_w8", op="beam", B=64, W=8, V=128000, k=8, dtype="fp32", done=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["bounds", "select", "attend", "attend", "fork", "compact", "beam"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8])
    fp8 = rng.random() < 0.5
    if op == "beam":
        W = _spread(rng, 1, 16)
        V = _spread(rng, 64, 160_000)
        B = _spread(rng, 1, max(1, min(96, 60_000_000 // (W * V))))
        return dict(op=op, B=B, W=W, V=V, k=min(_spread(rng, 1, 32), V), done=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if op in ("fork", "compact"):
        layers = rng.choice([1, 2, 4])
        most = 400_000_000 // (layers * 2 * Hkv * page * d * 2)  # pages in all
        if op == "compact":
            pages = _spread(rng, 16, max(16, min(8192, most)))
            used = rng.randrange(1, pages)
            return dict(op=op, pages=pages, used=used, B=_spread(rng, 1, 64), Hkv=Hkv, d=d, page=page,
                        layers=layers, fp8=fp8)
        W = _spread(rng, 1, 16)
        B = _spread(rng, 1, max(1, min(48, most // (W * 4 + 8))))
        hi = _spread(rng, 1, max(1, min(16384, (most // B - 2 * W) * page)))
        return dict(op=op, B=B, W=W, lo=max(1, hi // 3), hi=hi, Hkv=Hkv, d=d, page=page,
                    layers=layers, fp8=fp8, reserve=rng.choice([0, 1, 4, 8, 33]),
                    done=rng.randrange(0, B) if rng.random() < 0.5 else 0)
    G = rng.choice([1, 2, 4, 5, 8, 16])
    if op == "attend":
        T = rng.choice([1, 1, 1, 2, 4, 7, 12])
        k = _spread(rng, 1, 64)
        hi = _spread(rng, 1, 65536)
        B = _spread(rng, 1, max(1, min(64, 500_000 // hi, 4_000_000 // (T * Hkv * k * page))))
        return dict(op=op, B=B, lo=rng.choice([0, max(1, hi // 2), hi]), hi=hi, T=T, Hq=Hkv * G,
                    Hkv=Hkv, d=d, page=page, k=k, fp8=fp8)
    if op == "select":
        T = rng.choice([1, 1, 2, 4, 7, 16, 64])
        hi = _spread(rng, 8 * page, 131072)
        most = 160_000_000 // (hi // page * T * Hkv * G + 1)
        B = _spread(rng, 1, max(1, min(64, 500_000 // hi, most)))
        c = dict(op=op, B=B, lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi, T=T, Hq=Hkv * G, Hkv=Hkv,
                 d=d, page=page)
        nb = max(_lens(c)) // page  # some sequence has a choice to make
        if nb < 8:
            c["lo"], nb = hi, hi // page
        return dict(c, k=_spread(rng, 3, min(256, nb // 2)))
    hi = _spread(rng, 1, 16384)
    B = _spread(rng, 1, max(1, min(96, 200_000 // hi)))
    return dict(op=op, B=B, lo=rng.choice([0, max(1, hi // 2), hi]), hi=hi,
                new=rng.choice([1, 4, page, 16384]), Hkv=Hkv, d=d, page=page, fp8=fp8)


def _lens(case):
    """The case's sequence lengths (of the case alone, so that work() knows them)."""
    r = random.Random("lens %d %d %d" % (case["B"], case["lo"], case["hi"]))
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    if sum(n) == 0:
        n[0] = 1
    return n


def _listed_blocks(case):
    """Page lists of every (sequence, token, KV head): tokens of one sequence
    share most of theirs, the first page and the last are always among them."""
    r = random.Random("blocks %r" % sorted(case.items()))
    out = []
    for n in _lens(case):
        nb = -(-n // case["page"])
        m = min(case["k"], nb)
        heads = [sorted(r.sample(range(nb), m)) for _ in range(case["Hkv"])]
        rows = []
        for _ in range(case["T"]):
            for base in heads:
                kept = r.sample(base, m - m // 4)
                pick = set(kept[:m])
                while len(pick) < m:
                    pick.add(r.randrange(nb))
                if m > 1:
                    for must in (0, nb - 1):
                        if must not in pick:
                            pick.remove(r.choice(sorted(pick - {0, nb - 1})))
                            pick.add(must)
                row = sorted(pick)
                rows.append(row + [-1] * (case["k"] - len(row)))
        out.append(rows)
    return out


def _parents(case):
    """fork: the parent row of every new row (of the case alone); -1: no row."""
    r = random.Random("parents %r" % sorted(case.items()))
    B, W = case["B"], case["W"]
    done = set(r.sample(range(B), case["done"]))
    out = []
    for b in range(B):
        best = r.sample(range(W), max(1, (W + 1) // 2))  # half of the beams go on
        out += [-1] * W if b in done else [b * W + r.choice(best) for _ in range(W)]
    return out


def _used(case):
    """compact: which pages of the pool are in use."""
    r = random.Random("used %r" % sorted(case.items()))
    return sorted(r.sample(range(case["pages"]), case["used"]))


def _tree(T, r):
    """A draft tree: node 0 the root, each later node below an earlier one."""
    return [-1] + [r.randrange(max(0, i - 4), i) for i in range(1, T)]


def _dev():
    return torch.device("cuda")


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=_dev())


def _pow2(e):
    """2^e of whole numbers e as fp32."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """[..., d] -> (e4m3 codes [..., d], exponent bytes [...]) of the 8-bit cache."""
    a = x.float()
    amax = a.abs().amax(-1)
    m, e = torch.frexp(amax / CODE_MAX)
    s = torch.where(m == 0.5, e - 1, e).clamp(S_MIN, S_MAX)
    y = (a * _pow2(-s)[..., None]).clamp(-CODE_MAX, CODE_MAX)
    return y.to(torch.float8_e4m3fn), (s + 127).to(torch.uint8)


def _tables(counts, spare, g):
    """A block table that gives row b counts[b] pages, in random order, unused
    entries -1; and the number of pages."""
    total = max(1, sum(counts)) + spare
    perm = torch.randperm(total, generator=g, device=_dev()).int().cpu()
    bt = torch.full((len(counts), max(1, max(counts))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(counts):
        bt[b, :n] = perm[at:at + n]
        at += n
    return bt.to(_dev()), total


def _key_pool(n, H, P, d, fp8, g):
    """Keys or values of n pages: channels of unequal size, tokens of unequal norm.
    (pool bf16, None) or (codes, scale bytes)."""
    gain = torch.exp(0.4 * torch.randn(H, 1, d, generator=g, device=_dev()))
    pool = torch.empty(n, H, P, d, device=_dev(), dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16)
    scales = torch.empty(n, H, P, device=_dev(), dtype=torch.uint8) if fp8 else None
    step = max(1, (1 << 26) // (H * P * d))
    for at in range(0, n, step):
        m = min(step, n - at)
        x = torch.randn(m, H, P, d, generator=g, device=_dev()) * gain
        x *= torch.exp(0.3 * torch.randn(m, H, P, 1, generator=g, device=_dev()))
        if fp8:
            pool[at:at + m], scales[at:at + m] = _quantise(x)
        else:
            pool[at:at + m] = x
    return pool, scales


def _queries(B, T, Hq, d, g):
    x = torch.randn(B, T, Hq, d, generator=g, device=_dev())
    x *= torch.exp(0.4 * torch.randn(Hq, d, generator=g, device=_dev()))
    return x.bfloat16()


def prepare(case, seed):
    g = torch.Generator(device=_dev()).manual_seed(int(seed) * 7919 + 29)
    r = random.Random(int(seed))
    op = case["op"]
    s = dict(op=op, case=dict(case))
    if op == "beam":
        B, W, V, k = (case[w] for w in ("B", "W", "V", "k"))
        dt = dict(bf16=torch.bfloat16, fp16=torch.float16, fp32=torch.float32)[case["dtype"]]
        x = torch.empty(B, W, V, device=_dev(), dtype=dt)
        for b in range(B):  # logits: a wide bulk and a few tokens that stand out
            y = 2.0 * torch.randn(W, V, generator=g, device=_dev())
            n = min(V, 16)
            at = torch.randint(0, V, (W, n), generator=g, device=_dev())
            y.scatter_add_(1, at, 6.0 + 3.0 * torch.rand(W, n, generator=g, device=_dev()))
            x[b] = y
        scores = -torch.sort(30.0 * torch.rand(B, W, generator=g, device=_dev()), dim=1).values
        s.update(logits=x, scores=scores, k=k, eos=V // 3)
        s["finished"] = torch.rand(B, W, generator=g, device=_dev()) < 0.2 if case["done"] else None
        return s
    H, d, P = case["Hkv"], case["d"], case["page"]
    if op in ("fork", "compact"):
        fp8, layers, B = case["fp8"], case["layers"], case["B"]
        if op == "fork":
            _fork_state(case, s, r)
        else:
            used = _used(case)
            order = list(used)
            r.shuffle(order)
            cut = random.Random("cuts %r" % sorted(case.items()))
            cuts = sorted(cut.randint(0, len(order)) for _ in range(B - 1))
            rows = [order[a:b] for a, b in zip([0] + cuts, cuts + [len(order)])]
            wide = max(1, max(map(len, rows)))
            s["bt"] = _ints([x + [-1] * (wide - len(x)) for x in rows])
            s["refs"] = torch.zeros(case["pages"], dtype=torch.int32, device=_dev())
            s["refs"][torch.tensor(used, device=_dev())] = 1
        n = s["refs"].numel()
        s["pools"] = []
        for _ in range(2 * layers):
            if fp8:
                pool = torch.randint(0, 127, (n, H, P, d), generator=g, device=_dev(), dtype=torch.uint8)
                s["pools"].append(pool.view(torch.float8_e4m3fn))
                s["pools"].append(torch.randint(100, 140, (n, H, P), generator=g, device=_dev(),
                                                dtype=torch.uint8))
            else:
                pool = torch.empty(n, H, P, d, device=_dev(), dtype=torch.bfloat16)
                s["pools"].append(pool.normal_(generator=g))
        return s
    B, lens = case["B"], _lens(case)
    s["lens"] = lens
    s["seq_lens"] = _ints(lens)
    s["bt"], n = _tables([-(-x // P) for x in lens], 0, g)
    if op == "bounds":
        s["k_pages"], s["k_scales"] = _key_pool(n, H, P, d, case["fp8"], g)
        s["starts"] = _ints([max(0, x - case["new"]) for x in lens])
        s["bounds"] = torch.zeros(n, H, 2, d, dtype=torch.int8, device=_dev())
        s["bounds_exp"] = torch.zeros(n, H, dtype=torch.uint8, device=_dev())
        return s
    T, Hq, k = case["T"], case["Hq"], case["k"]
    s["q"] = _queries(B, T, Hq, d, g)
    if op == "select":
        # the bounds that a cache of such keys has, one channel's apart from the next one's
        gain = torch.exp(0.4 * torch.randn(H, d, generator=g, device=_dev()))
        mid = 0.6 * torch.randn(n, H, d, generator=g, device=_dev()) * gain
        wide = 2.2 * gain * torch.exp(0.15 * torch.randn(n, H, d, generator=g, device=_dev()))
        s["bounds"], s["bounds_exp"] = _code_bounds(mid + wide, mid - wide)
        s["first"], s["last"] = (1, 1) if k >= 2 else (0, 1)
        return s
    s["k_pages"], s["k_scales"] = _key_pool(n, H, P, d, case["fp8"], g)
    s["v_pages"], s["v_scales"] = _key_pool(n, H, P, d, case["fp8"], g)
    s["tree_k"] = torch.randn(B, T, H, d, generator=g, device=_dev()).bfloat16()
    s["tree_v"] = torch.randn(B, T, H, d, generator=g, device=_dev()).bfloat16()
    s["blocks"] = _ints(_listed_blocks(case)).view(B, T, H, k)
    s["parents"] = _ints(_tree(T, r))
    return s


def _fork_state(case, s, r):
    """Beams as a search leaves them: those of one prompt share its full pages,
    and each holds its own last page."""
    B, W, P = case["B"], case["W"], case["page"]
    lens = _lens(case)
    full = [n // P for n in lens]
    total = sum(full) + B * W * (2 + -(-(case["reserve"] + 1) // P)) + 8
    ids = list(range(total))
    r.shuffle(ids)
    at, rows, refs = 0, [], [0] * total
    for b in range(B):
        shared = ids[at:at + full[b]]
        at += full[b]
        for p in shared:
            refs[p] = W
        for _ in range(W):
            own_pages = ids[at:at + 1]
            at += 1
            refs[own_pages[0]] = 1
            rows.append(shared + own_pages)
    wide = max(map(len, rows)) + -(-case["reserve"] // P) + 1
    s["bt"] = _ints([x + [-1] * (wide - len(x)) for x in rows])
    s["refs"] = _ints(refs)
    s["seq_lens"] = _ints([n for n in lens for _ in range(W)])
    s["src"] = _ints(_parents(case))


# The plain forms.

def _code_bounds(hi, lo):
    """Largest and smallest values [..., d] (fp32) -> codes int8 [..., 2, d] and
    exponent bytes [...]."""
    amax = torch.maximum(hi.abs(), lo.abs()).amax(-1)
    m, e = torch.frexp(amax)  # amax = m * 2^e, m in [0.5, 1)
    e = torch.where(m <= 127.0 / 128.0, e - 7, e - 6)
    e = torch.where(amax == 0, E_MIN, e).clamp(E_MIN, E_MAX)
    inv = _pow2(-e)[..., None]
    codes = torch.stack([torch.ceil(hi * inv), torch.floor(lo * inv)], -2)
    return codes.clamp(-127, 127).to(torch.int8), (e + 127).to(torch.uint8)


def _plain_bounds(s):
    P, lens, new = s["case"]["page"], s["lens"], s["case"]["new"]
    first = [max(0, n - new) // P for n in lens]
    count = [-(-n // P) - a for a, n in zip(first, lens)]
    seq = torch.repeat_interleave(torch.arange(len(lens), device=_dev()),
                                  torch.tensor(count, device=_dev()), output_size=sum(count))
    shift = torch.tensor([a - sum(count[:b]) for b, a in enumerate(first)], device=_dev())
    slot = torch.arange(sum(count), device=_dev()) + shift[seq]
    for at in range(0, sum(count), 4096):  # in pieces: less memory at a time
        b, j = seq[at:at + 4096], slot[at:at + 4096]
        page = s["bt"][b, j].long()
        x = s["k_pages"][page].float()
        if s["k_scales"] is not None:
            x *= _pow2(s["k_scales"][page].int() - 127)[..., None]
        here = (j[:, None] * P + torch.arange(P, device=_dev())) < s["seq_lens"][b][:, None]
        gone = ~here[:, None, :, None]
        codes, e = _code_bounds(x.masked_fill(gone, -math.inf).amax(2),
                                x.masked_fill(gone, math.inf).amin(2))
        s["bounds"][page], s["bounds_exp"][page] = codes, e
    return s["bounds"], s["bounds_exp"]


def _plain_select(s):
    q, P, k = s["q"].float(), s["case"]["page"], s["case"]["k"]
    B, T, Hq, d = q.shape
    H = s["bounds"].shape[1]
    G, nb = Hq // H, s["bt"].shape[1]
    rows = q.view(B, T, H, G, d)
    amax = rows.abs().amax((-1, -2))
    m, f = torch.frexp(amax)
    f = torch.where(m <= 127.0 / 128.0, f - 7, f - 6)
    f = torch.where(amax == 0, E_MIN, f).clamp(E_MIN, E_MAX)
    qc = torch.round(rows * _pow2(-f)[..., None, None]).clamp(-127, 127)
    count = ((s["seq_lens"] + P - 1) // P)[:, None, None, None]
    slot = torch.arange(nb, device=q.device)
    pages = s["bt"].clamp_min(0).long()
    # whole numbers below 2^24 in every product and sum: exact in fp32
    x = s["bounds"][pages].float().permute(0, 2, 3, 4, 1)  # [B][H][2][d][nb]
    c = qc.permute(0, 2, 1, 3, 4).reshape(B, H, T * G, d)
    dots = c.clamp_min(0) @ x[:, :, 0] + c.clamp_max(0) @ x[:, :, 1]
    size = _pow2(s["bounds_exp"][pages].int() - 127).transpose(1, 2)[:, :, None]
    score = dots.view(B, H, T, G, nb).amax(3) * size
    score.masked_fill_((slot < s["first"]) | (slot >= count - s["last"]), math.inf)
    score.masked_fill_(slot >= count, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :k]
    order = torch.where(order < count, order, nb)
    order = torch.sort(order, dim=-1).values
    order = torch.where(order < count, order, -1).int()
    if nb < k:
        order = torch.cat([order, order.new_full((B, H, T, k - nb), -1)], -1)
    return order.transpose(1, 2).contiguous()


def _ancestors(parents):
    """[T][T] truth values: whether column j is row i or an ancestor of it."""
    T = parents.numel()
    up = torch.nn.functional.one_hot(parents.long() + 1, T + 1)[:, 1:].float()
    reach = up + torch.eye(T, device=parents.device)
    n = 1
    while n < T:
        reach = (reach @ reach > 0).float()
        n *= 2
    return reach > 0


def _plain_attend(s):
    q, P = s["q"].float(), s["case"]["page"]
    B, T, Hq, d = q.shape
    H = s["tree_k"].shape[2]
    G, k = Hq // H, s["blocks"].shape[3]
    see = _ancestors(s["parents"])
    head = torch.arange(H, device=q.device)[None, None, :, None]
    out, lse = [], []
    step = max(1, (1 << 28) // (T * H * k * P * d))
    for at in range(0, B, step):  # some sequences at a time: less memory
        blocks = s["blocks"][at:at + step].long()  # [n][T][H][k]
        n = blocks.shape[0]
        table = s["bt"][at:at + step].clamp_min(0).long()
        page = table.gather(1, blocks.clamp_min(0).view(n, -1)).view_as(blocks)
        pos = blocks[..., None] * P + torch.arange(P, device=q.device)
        held = (blocks[..., None] >= 0) & (pos < s["seq_lens"][at:at + step, None, None, None, None])
        held = held.view(n, T, H, 1, k * P)

        def rows(which):  # [n][T][H][k * P + T][d]
            x = s[which + "_pages"][page, head].float()
            if s[which + "_scales"] is not None:
                x *= _pow2(s[which + "_scales"][page, head].int() - 127)[..., None]
            x = x.view(n, T, H, k * P, d).masked_fill_(~held.transpose(3, 4), 0.0)
            tree = s["tree_" + which][at:at + step].float().transpose(1, 2)
            return torch.cat([x, tree[:, None].expand(n, T, H, T, d)], 3)

        x = q[at:at + step].view(n, T, H, G, d) @ rows("k").transpose(3, 4)
        x *= 1.0 / math.sqrt(d)
        ok = torch.cat([held, see[:, None, None].expand(n, T, H, 1, T)], 4)
        x.masked_fill_(~ok, -math.inf)
        top = x.amax(-1, keepdim=True)
        x.sub_(top).exp_()
        total = x.sum(-1, keepdim=True)
        out.append(((x @ rows("v")) / total).view(n, T, Hq, d).bfloat16())
        lse.append((total.log() + top).view(n, T, Hq))
    return torch.cat(out), torch.cat(lse)


def _counted(table, n):
    """How often each of n pages stands in a table (-1: nowhere)."""
    c = torch.zeros(n + 1, dtype=torch.int32, device=table.device)
    at = torch.where(table >= 0, table, n).long().view(-1)
    return c.scatter_add_(0, at, torch.ones_like(at, dtype=torch.int32))[:n]


def _plain_fork(s):
    bt, lens, refs, src = s["bt"].long(), s["seq_lens"].long(), s["refs"], s["src"].long()
    P, n, wide = s["case"]["page"], s["refs"].numel(), s["bt"].shape[1]
    live = src >= 0
    up = src.clamp_min(0)
    L = torch.where(live, lens[up], 0)
    rows = torch.where(live[:, None], bt[up], -1)
    me = torch.arange(src.numel(), device=src.device)
    first = torch.full((bt.shape[0],), src.numel(), device=src.device)
    first = first.scatter_reduce(0, up[live], me[live], "amin")
    eldest = live & (first[up] == me)
    slot = torch.arange(wide, device=src.device)
    need = torch.where(live, (L + s["case"]["reserve"] + P - 1) // P, 0)
    shared = slot < (L // P)[:, None]
    tail = ~shared & (slot < need[:, None])
    keep = tail & eldest[:, None] & (rows >= 0) & (refs[rows.clamp_min(0)] == 1)
    fresh = tail & ~keep
    free = torch.sort(torch.where(refs == 0, torch.arange(n, device=src.device), n)).values
    rank = (fresh.view(-1).long().cumsum(0) - 1).view_as(fresh)
    new = torch.where(fresh, free[rank.clamp(0, n - 1)], -1)
    table = torch.where(shared | keep, rows, new)
    refs = refs - _counted(bt, n) + _counted(table, n)
    last = (L // P).clamp_max(wide - 1)[:, None]
    copied = (fresh.gather(1, last) & (L % P != 0)[:, None])[:, 0]
    a, z = rows.gather(1, last)[copied, 0], table.gather(1, last)[copied, 0]
    for pool in s["pools"]:
        bits = pool.view(torch.uint8)
        bits[z] = bits[a]
    return table.int(), L.int(), refs, s["pools"]


def _plain_compact(s):
    refs = s["refs"]
    n = refs.numel()
    used = refs > 0
    m = used.sum()
    page = torch.arange(n, device=refs.device)
    move, hole = used & (page >= m), ~used & (page < m)
    to = torch.where(used, page, -1)
    holes = torch.sort(torch.where(hole, page, n)).values
    to = torch.where(move, holes[(move.long().cumsum(0) - 1).clamp_min(0)], to)
    table = torch.where(s["bt"] >= 0, to[s["bt"].clamp_min(0).long()], -1).int()
    new = torch.zeros(n + 1, dtype=torch.int32, device=refs.device)
    new[torch.where(used, to, n)] = refs
    a, z = page[move], to[move]
    for pool in s["pools"]:
        bits = pool.view(torch.uint8)
        bits[z] = bits[a]
    return table, new[:n], m.int().view(1), s["pools"]


def _plain_beam(s):
    x, k, eos = s["logits"].double(), s["k"], s["eos"]
    B, W, V = x.shape
    top = x.amax(-1, keepdim=True)
    x.sub_(top)
    x -= x.exp().sum(-1, keepdim=True).log()
    x += s["scores"].double()[..., None]
    if s["finished"] is not None:  # a finished beam stands for itself alone
        only = torch.full_like(x, -math.inf)
        only[..., eos] = s["scores"].double()
        x = torch.where(s["finished"][..., None], only, x)
    best, at = torch.sort(x.view(B, W * V), dim=1, descending=True, stable=True)
    best, at = best[:, :k], at[:, :k]
    some = best > -math.inf
    row = torch.arange(B, device=x.device)[:, None] * W + at // V
    token = torch.where(some, at % V, -1).int()
    return best.float(), torch.where(some, row, -1).int(), token


def run(s):
    op = s["op"]
    if own:
        import speculative_decoding_tree_split_gb300 as ta
        if op == "bounds":
            return ta.kv_block_bounds(s["k_pages"], s["bt"], s["seq_lens"], k_scales=s["k_scales"],
                                      starts=s["starts"], bounds=s["bounds"],
                                      bounds_exp=s["bounds_exp"])
        if op == "select":
            return ta.select_blocks(s["q"], s["bounds"], s["bounds_exp"], s["bt"], s["seq_lens"],
                                    s["case"]["k"], s["case"]["page"], n_first=s["first"],
                                    n_last=s["last"])
        if op == "attend":
            return ta.verify_blocks(s["q"], s["k_pages"], s["v_pages"], s["bt"], s["seq_lens"],
                                    s["blocks"], s["tree_k"], s["tree_v"], parents=s["parents"],
                                    k_scales=s["k_scales"], v_scales=s["v_scales"])
        if op == "fork":
            bt, lens, refs = ta.kv_fork(s["pools"], s["bt"], s["seq_lens"], s["refs"], s["src"],
                                        s["case"]["page"], reserve=s["case"]["reserve"])
            return bt, lens, refs, s["pools"]
        if op == "compact":
            bt, refs, n_used = ta.kv_compact(s["pools"], s["bt"], s["refs"])
            return bt, refs, n_used, s["pools"]
        return ta.beam_select(s["logits"], s["scores"], s["k"], finished=s["finished"],
                              eos=s["eos"])
    return dict(bounds=_plain_bounds, select=_plain_select, attend=_plain_attend, fork=_plain_fork,
                compact=_plain_compact, beam=_plain_beam)[op](s)


def _copies(case):
    """fork: how many rows get a copy of their last page."""
    lens, seen, n = _lens(case), set(), 0
    for p in _parents(case):
        if p >= 0 and lens[p // case["W"]] % case["page"]:
            n += p in seen
            seen.add(p)
    return n


def work(case):
    op = case["op"]
    if op == "beam":
        B, W, V, k = (case[w] for w in ("B", "W", "V", "k"))
        size = 4 if case["dtype"] == "fp32" else 2
        return dict(bytes=B * W * V * size + 5 * B * W + 12 * B * k, flops=3 * B * W * V)
    H, d, P = case["Hkv"], case["d"], case["page"]
    if op in ("fork", "compact"):
        one = H * P * ((d + 1) if case["fp8"] else 2 * d) * 2 * case["layers"]  # of one page
        if op == "compact":
            used = _used(case)
            moves = sum(p >= len(used) for p in used)
            return dict(bytes=2 * moves * one + 8 * case["pages"] + 8 * len(used), flops=0)
        lens, src = _lens(case), _parents(case)
        table = sum(-(-(lens[p // case["W"]] + case["reserve"]) // P) for p in src if p >= 0)
        pages = sum(n // P for n in lens) + case["B"] * case["W"]
        return dict(bytes=2 * _copies(case) * one + 8 * (table + pages + 2 * len(src)), flops=0)
    lens = _lens(case)
    row = d + 1 if case.get("fp8") else 2 * d
    if op == "bounds":
        tokens = pages = 0
        for n in lens:
            if n:
                first = max(0, n - case["new"]) // P
                pages += -(-n // P) - first
                tokens += n - first * P
        return dict(bytes=H * (tokens * row + pages * (2 * d + 1)) + 4 * pages, flops=0)
    B, T, Hq, k = case["B"], case["T"], case["Hq"], case["k"]
    nb = [-(-n // P) for n in lens]
    if op == "select":
        return dict(bytes=sum(nb) * (H * (2 * d + 1) + 4) + B * T * (Hq * d * 2 + H * k * 4),
                    flops=4 * d * Hq * T * sum(nb))
    tokens = seen = 0
    for b, rows in enumerate(_listed_blocks(case)):
        def held(blocks):
            return sum(min(P, lens[b] - j * P) for j in blocks if j >= 0)
        for h in range(H):
            tokens += held(set().union(*(rows[t * H + h] for t in range(T))))
        seen += sum(held(x) for x in rows)
    return dict(bytes=2 * tokens * row + B * T * (2 * Hq + 2 * H) * d * 2 + B * T * Hq * 4
                + 4 * (B * T * H * k + sum(nb)),
                flops=4 * d * (Hq // H) * (seen + B * H * T * (T + 1) // 2))


# The same from the definitions, in 64 bits, with code of its own.

def _two_to(e):
    """2^e of whole numbers e in 64 bits, put together from the bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _least_exponent(big):
    """The least e of [E_MIN, E_MAX] with big <= 127 * 2^e."""
    e = torch.full(big.shape, E_MAX, dtype=torch.long, device=big.device)
    guess = torch.floor(torch.log2(big.clamp_min(1e-200) / 127)).long()
    for step in (2, 1, 0, -1, -2):
        c = (guess + step).clamp(E_MIN, E_MAX)
        e = torch.where(127 * _two_to(c) >= big, torch.minimum(e, c), e)
    return e


def _exact_keys(s, which, page):
    """Rows of pages [...]: [..., Hkv][P][d] in 64 bits."""
    x = s[which + "_pages"][page].double()
    if s[which + "_scales"] is not None:
        x = x * _two_to(s[which + "_scales"][page].long() - 127)[..., None]
    return x


def _exact_bounds(s):
    P, new = s["case"]["page"], s["case"]["new"]
    out, exps = s["bounds"].clone(), s["bounds_exp"].clone()
    for b, n in enumerate(s["lens"]):
        pages = s["bt"][b].tolist()
        for j in range(max(0, n - new) // P, -(-n // P)):
            x = _exact_keys(s, "k", pages[j])[:, :n - j * P]
            hi, lo = x.max(1).values, x.min(1).values
            e = _least_exponent(torch.maximum(hi, -lo).max(1).values)
            unit = _two_to(e)[:, None]
            out[pages[j], :, 0] = torch.ceil(hi / unit).to(torch.int8)
            out[pages[j], :, 1] = torch.floor(lo / unit).to(torch.int8)
            exps[pages[j]] = (e + 127).to(torch.uint8)
    return out, exps


def _exact_select(s):
    P, k = s["case"]["page"], s["case"]["k"]
    B, T, Hq, d = s["q"].shape
    H = s["bounds"].shape[1]
    out = torch.full((B, T, H, k), -1, dtype=torch.int32)
    for b, L in enumerate(s["seq_lens"].tolist()):
        nb = (L + P - 1) // P
        if nb == 0:
            continue
        pages = s["bt"][b, :nb].long()
        x = s["bounds"][pages].double()
        size = _two_to(s["bounds_exp"][pages].long() - 127)
        for t in range(T):
            for h in range(H):
                q = s["q"][b, t, h * (Hq // H):(h + 1) * (Hq // H)].double()
                q = torch.round(q / _two_to(_least_exponent(q.abs().max().view(1))))
                each = torch.maximum(q[:, None] * x[:, h, 0], q[:, None] * x[:, h, 1]).sum(-1)
                score = (each.max(0).values * size[:, h]).tolist()
                forced = [j for j in range(nb) if j < s["first"] or j >= nb - s["last"]]
                rest = sorted(set(range(nb)) - set(forced), key=lambda j: (-score[j], j))
                pick = sorted((forced + rest)[:k])
                out[b, t, h, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
    return out.to(_dev())


def _exact_attend(s):
    P = s["case"]["page"]
    B, T, Hq, d = s["q"].shape
    H = s["tree_k"].shape[2]
    G = Hq // H
    up, lens, table = s["parents"].tolist(), s["seq_lens"].tolist(), s["bt"].tolist()
    out = torch.empty(B, T, Hq, d, dtype=torch.float64, device=_dev())
    lse = torch.empty(B, T, Hq, dtype=torch.float64, device=_dev())
    lists = s["blocks"].tolist()
    for b in range(B):
        for t in range(T):
            line, j = [], t
            while j >= 0:
                line.append(j)
                j = up[j]
            line = torch.tensor(line, device=_dev())
            for h in range(H):
                blocks = [j for j in lists[b][t][h] if j >= 0]
                page = torch.tensor([table[b][j] for j in blocks], dtype=torch.long, device=_dev())
                held = torch.cat([torch.arange(P) < lens[b] - j * P for j in blocks]
                                 or [torch.zeros(0, dtype=torch.bool)]).to(_dev())
                kv = []
                for w in "kv":
                    x = s[w + "_pages"][page, h].double()
                    if s[w + "_scales"] is not None:
                        x = x * _two_to(s[w + "_scales"][page, h].long() - 127)[..., None]
                    kv.append(torch.cat([x.view(-1, d)[held], s["tree_" + w][b, line, h].double()]))
                z = s["q"][b, t, h * G:(h + 1) * G].double() @ kv[0].T / math.sqrt(d)
                whole = torch.logsumexp(z, 1)
                lse[b, t, h * G:(h + 1) * G] = whole
                out[b, t, h * G:(h + 1) * G] = torch.exp(z - whole[:, None]) @ kv[1]
    return out, lse


def _exact_fork(s):
    P, reserve = s["case"]["page"], s["case"]["reserve"]
    old, lens, refs = s["bt"].tolist(), s["seq_lens"].tolist(), s["refs"].tolist()
    free = iter([p for p, c in enumerate(refs) if c == 0])
    table, new_lens, moves, seen = [], [], [], set()
    for p in s["src"].tolist():
        row = [-1] * len(old[0])
        L = lens[p] if p >= 0 else 0
        if p >= 0:
            for j in range(-(-(L + reserve) // P)):
                has = old[p][j]
                if j < L // P or (p not in seen and has >= 0 and refs[has] == 1):
                    row[j] = has
                else:
                    row[j] = next(free)
                    if j * P < L:
                        moves.append((has, row[j]))
            seen.add(p)
        table.append(row)
        new_lens.append(L)
    count = list(refs)
    for rows, sign in ((old, -1), (table, 1)):
        for row in rows:
            for p in row:
                if p >= 0:
                    count[p] += sign
    return _ints(table), _ints(new_lens), _ints(count), _moved(s["pools"], moves)


def _moved(pools, moves):
    out = []
    for pool in pools:
        pool = pool.clone()
        for a, z in moves:
            pool[z].copy_(pool[a])
        out.append(pool)
    return out


def _exact_compact(s):
    refs = s["refs"].tolist()
    m = sum(c > 0 for c in refs)
    holes = iter([p for p in range(m) if refs[p] == 0])
    to = {p: p if p < m else next(holes) for p, c in enumerate(refs) if c > 0}
    new = [0] * len(refs)
    for p, z in to.items():
        new[z] = refs[p]
    table = [[to[p] if p >= 0 else -1 for p in row] for row in s["bt"].tolist()]
    moves = [(p, z) for p, z in to.items() if p != z]
    return _ints(table), _ints(new), _ints([m]), _moved(s["pools"], moves)


def _exact_beam(s):
    B, W, V = s["logits"].shape
    k, eos = s["k"], s["eos"]
    scores = s["scores"].double().tolist()
    done = s["finished"].tolist() if s["finished"] is not None else [[False] * W] * B
    got = [], [], []
    for b in range(B):
        some = []
        for w in range(W):
            if done[b][w]:
                some.append((-scores[b][w], w, eos))
                continue
            x = torch.log_softmax(s["logits"][b, w].double(), 0)
            best = torch.topk(x, min(V, k)).values[-1]
            at = (x >= best).nonzero()[:, 0]
            some += [(-(scores[b][w] + y), w, v) for y, v in zip(x[at].tolist(), at.tolist())]
        some = sorted(some)[:k]
        some += [(math.inf, -1 - b * W, -1)] * (k - len(some))
        got[0].append([-y for y, _, _ in some])
        got[1].append([b * W + w for _, w, _ in some])
        got[2].append([v for _, _, v in some])
    return torch.tensor(got[0], dtype=torch.float64, device=_dev()), _ints(got[1]), _ints(got[2])


def exact(case, seed):
    s = prepare(case, seed)
    return dict(bounds=_exact_bounds, select=_exact_select, attend=_exact_attend, fork=_exact_fork,
                compact=_exact_compact, beam=_exact_beam)[s["op"]](s)
