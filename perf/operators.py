"""The measured cases of the serving operators around tree verification.

Four operators that belong together in a server that verifies draft trees:

* ``append`` / ``commit``: K/V rows written into a paged cache of 8-bit floats
  (e4m3) with one power-of-two scale for each (token, KV head) row -- a
  prompt's or a step's tokens, or the accepted path of a draft tree.
* ``read``: a stretch of every sequence read back out of that cache as bf16.
* ``verify``: attention of a draft tree (T = 1: plain decoding) over the
  committed tokens of that cache plus the tree tokens its mask allows.
* ``prefill``: causal attention over whole prompts of different lengths, packed
  one after the other, with grouped heads.

A cache row x (d values) is held as codes c (e4m3) and one exponent s with
x ~ c * 2^s: s is the smallest integer with max|x| <= 448 * 2^s over the finite
values, held within [-56, 40] and stored as the byte s + 127.

``run`` gives the framework's calls when ``own`` is set and otherwise the same
results from elementary tensor operations in 32 bits.
"""
import math
import random

import torch

own = False

S_MIN, S_MAX, CODE_MAX = -56, 40, 448.0


def listed():
    return [
        # A Llama-3.1-8B layer takes in one prompt of 8192 tokens: k and v are
        # slices of the fused projection's output.
        dict(name="append_prompt_8b", op="append", B=1, lo=8192, hi=8192, start=0, Hkv=8, d=128,
             page=64, fused=True),
        # The 64 sequences of the large-batch workload take in a chunk each, of
        # any length from none to 8191, behind what they hold already.
        dict(name="append_ragged_b64", op="append", B=64, lo=0, hi=8191, start=1000, Hkv=8, d=128,
             page=64, fused=False),
        # The step after verification at that batch: the accepted path of a
        # 4-token draft chain is written (latency counts).
        dict(name="commit_b64_t4", op="commit", B=64, lo=512, hi=4096, T=4, Hkv=8, d=128, page=64),
        # One 8192-token sequence read back whole (a prefix handed to a bf16 user).
        dict(name="read_8b", op="read", B=1, lo=8192, hi=8192, start=0, Hkv=8, d=128, page=64),
        # The Llama-3.1-70B batch, read back from an odd position on.
        dict(name="read_ragged_b16", op="read", B=16, lo=1024, hi=8192, start=37, Hkv=8, d=128,
             page=64),
        # Plain decoding of three sequences with 64-wide heads and small pages.
        dict(name="verify_decode_d64", op="verify", B=3, lo=1, hi=4099, T=1, Hq=8, Hkv=2, d=64,
             page=16),
        # The Llama-3.1-8B verification layer (one sequence; latency counts).
        dict(name="verify_8b", op="verify", B=1, lo=8192, hi=8192, T=12, Hq=32, Hkv=8, d=128,
             page=64),
        # The Maverick-shaped layer: five query heads to a KV head, 32768 tokens.
        dict(name="verify_maverick", op="verify", B=4, lo=32768, hi=32768, T=16, Hq=40, Hkv=8,
             d=128, page=64),
        # The large-batch chain: 64 sequences of 512 to 16384 tokens.
        dict(name="verify_chain_b64", op="verify", B=64, lo=512, hi=16384, T=4, Hq=32, Hkv=8,
             d=128, page=64),
        # A batch of prompts from one token to 2048, Llama-3.1-70B heads, q, k
        # and v slices of the fused projection's output.
        dict(name="prefill_ragged_b16", op="prefill", B=16, lo=1, hi=2048, Hq=64, Hkv=8, d=128,
             fused=True),
        # One prompt of 8192 tokens through a Llama-3.1-8B layer.
        dict(name="prefill_8b", op="prefill", B=1, lo=8192, hi=8192, Hq=32, Hkv=8, d=128,
             fused=False),
        # The longest: one prompt of 16384 tokens.
        dict(name="prefill_16k", op="prefill", B=1, lo=16384, hi=16384, Hq=32, Hkv=8, d=128,
             fused=False),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "commit", "read", "verify", "verify", "prefill"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8])
    if op == "prefill":
        G = rng.choice([1, 2, 4, 5, 8])
        hi = _spread(rng, 16, 8192)
        # padded score elements of the plain form: those of 16384^2 x 32 at most
        B = _spread(rng, 1, max(1, min(32, (32 * 16384 ** 2 // 2) // (hi * hi * Hkv * G))))
        return dict(op=op, B=B, lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi, Hq=Hkv * G, Hkv=Hkv,
                    d=d, fused=rng.random() < 0.5)
    hi = _spread(rng, 1, 16384)
    B = _spread(rng, 1, max(1, min(96, 300_000 // hi)))
    lo = rng.choice([1, max(1, hi // 2), hi])
    if op == "verify":
        T = rng.choice([1, 2, 4, 7, 8, 12, 16, 33, 64])
        G = rng.choice([1, 2, 4, 5, 8])
        return dict(op=op, B=B, lo=lo, hi=hi, T=T, Hq=Hkv * G, Hkv=Hkv, d=d, page=page)
    if op == "commit":
        return dict(op=op, B=B, lo=lo, hi=hi, T=rng.choice([1, 3, 4, 8, 16, 33, 64]), Hkv=Hkv, d=d,
                    page=page)
    start = rng.choice([0, rng.randrange(1, 200)])
    c = dict(op=op, B=B, lo=rng.choice([0, lo]), hi=hi, start=start, Hkv=Hkv, d=d, page=page)
    return c if op == "read" else dict(c, fused=rng.random() < 0.5)


def _lens(case):
    """The case's sequence lengths (of the case alone, so that work() knows them)."""
    r = random.Random("lens %d %d %d" % (case["B"], case["lo"], case["hi"]))
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    if sum(n) == 0:
        n[0] = 1
    return n


def _accepted(case):
    r = random.Random("accepted %d %d" % (case["B"], case["T"]))
    return [r.randint(1, case["T"]) for _ in range(case["B"])]


def _tree(T, r):
    """A draft tree: node 0 the root, each later node below an earlier one."""
    return [-1] + [r.randrange(max(0, i - 4), i) for i in range(1, T)]


def _dev():
    return torch.device("cuda")


def _rows(n, H, d, g, gain):
    """n rows of H heads of keys or values: channels of unequal size (`gain`
    [H][d]) and tokens of unequal norm."""
    x = torch.randn(n, H, d, generator=g, device=_dev())
    x *= gain
    x *= torch.exp(0.3 * torch.randn(n, H, 1, generator=g, device=_dev()))
    return x.bfloat16()


def _gain(H, d, g):
    return torch.exp(0.4 * torch.randn(H, d, generator=g, device=_dev()))


def _pow2(e):
    """2^e of whole numbers e as fp32."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """bf16 [..., d] -> (codes as float8_e4m3fn [..., d], exponent bytes [...])."""
    a = x.float()
    amax = torch.where(torch.isfinite(a), a.abs(), 0.0).amax(-1)
    m, e = torch.frexp(amax / CODE_MAX)
    s = torch.where(m == 0.5, e - 1, e).clamp(S_MIN, S_MAX)
    s = torch.where(amax == 0, S_MIN, s)
    y = (a * _pow2(-s)[..., None]).clamp(-CODE_MAX, CODE_MAX)
    return y.to(torch.float8_e4m3fn), (s + 127).to(torch.uint8)


def _positions(lens, start):
    """(sequence, position) of every packed token."""
    n = torch.tensor(lens, device=_dev())
    seq = torch.repeat_interleave(torch.arange(len(lens), device=_dev()), n)
    first = torch.cumsum(n, 0) - n
    return seq, torch.arange(sum(lens), device=_dev()) - first[seq] + start


def _paged(case, caps, g):
    """Empty pools (any bytes) and a block table that covers caps[b] tokens of
    sequence b, its pages in random order, unused entries -1."""
    P, H, d = case["page"], case["Hkv"], case["d"]
    pages = [-(-c // P) for c in caps]
    total = max(1, sum(pages))
    perm = torch.randperm(total, generator=g, device=_dev()).int()
    bt = torch.full((len(caps), max(1, max(pages))), -1, dtype=torch.int32)
    perm_h = perm.cpu()
    at = 0
    for b, n in enumerate(pages):
        bt[b, :n] = perm_h[at:at + n]
        at += n

    def pool(*shape):
        return torch.randint(0, 256, shape, generator=g, device=_dev(), dtype=torch.uint8)

    return dict(k_pages=pool(total, H, P, d).view(torch.float8_e4m3fn),
                v_pages=pool(total, H, P, d).view(torch.float8_e4m3fn),
                k_scales=pool(total, H, P), v_scales=pool(total, H, P), bt=bt.to(_dev()))


def _put(s, which, seq, pos, x):
    """Rows x [N][H][d] into the pools at positions pos of sequences seq."""
    P = s["k_scales"].shape[2]
    page, off = s["bt"][seq, pos // P].long(), pos % P
    codes, scale = _quantise(x)
    s[which + "_pages"].view(torch.uint8)[page, :, off] = codes.view(torch.uint8)
    s[which + "_scales"][page, :, off] = scale


def _get(s, which, seq, pos):
    """Rows [..., H, d] at positions pos of sequences seq, as fp32."""
    P = s["k_scales"].shape[2]
    page, off = s["bt"][seq, pos // P].clamp_min(0).long(), pos % P
    codes = s[which + "_pages"].view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn).float()
    return codes * _pow2(s[which + "_scales"][page, :, off].int() - 127)[..., None]


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=_dev())


def _cu(lens):
    return _ints([sum(lens[:i]) for i in range(len(lens) + 1)])


def prepare(case, seed):
    g = torch.Generator(device=_dev()).manual_seed(int(seed) * 7919 + 13)
    r = random.Random(int(seed))
    lens, op, d = _lens(case), case["op"], case["d"]
    Hkv, N = case["Hkv"], sum(lens)
    s = dict(op=op, case=dict(case), lens=lens, cu=_cu(lens))
    gk, gv = _gain(Hkv, d, g), _gain(Hkv, d, g)
    if op == "prefill":
        Hq = case["Hq"]
        q = _rows(N, Hq, d, g, _gain(Hkv, d, g).repeat_interleave(Hq // Hkv, 0))
        k, v = _rows(N, Hkv, d, g, gk), _rows(N, Hkv, d, g, gv)
        if case["fused"]:
            qkv = torch.cat([q, k, v], 1)
            q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        return dict(s, q=q, k=k, v=v)
    T = case.get("T", 0)
    start = case.get("start", 0)
    caps = [n + start + T for n in lens]
    s.update(_paged(case, caps, g))
    s["T"], s["start"] = T, start
    if op == "append":
        k, v = _rows(N, Hkv, d, g, gk), _rows(N, Hkv, d, g, gv)
        if case["fused"]:
            kv = torch.cat([k, v], 1)
            k, v = kv[:, :Hkv], kv[:, Hkv:]
        return dict(s, k=k, v=v, seq_lens=_ints([start] * case["B"]))
    s["seq_lens"] = _ints(lens)
    if op == "commit":
        B = case["B"]
        s["tree_k"] = _rows(B * T, Hkv, d, g, gk).view(B, T, Hkv, d)
        s["tree_v"] = _rows(B * T, Hkv, d, g, gv).view(B, T, Hkv, d)
        n = _accepted(case)
        path = [[0] + sorted(r.sample(range(1, T), m - 1)) + [-1] * (T - m) for m in n]
        return dict(s, accept_len=_ints(n), accept_path=_ints(path))
    for which, gain in (("k", gk), ("v", gv)):
        seq, pos = _positions([n + start for n in lens], 0)
        for at in range(0, seq.numel(), 1 << 17):  # the rows in pieces: less memory at a time
            sl, ps = seq[at:at + (1 << 17)], pos[at:at + (1 << 17)]
            _put(s, which, sl, ps, _rows(sl.numel(), Hkv, d, g, gain))
    if op == "read":
        return dict(s, starts=_ints([start] * case["B"]))
    B, Hq = case["B"], case["Hq"]
    s["q"] = _rows(B * T, Hq, d, g, _gain(Hkv, d, g).repeat_interleave(Hq // Hkv, 0)).view(B, T, Hq, d)
    s["tree_k"] = _rows(B * T, Hkv, d, g, gk).view(B, T, Hkv, d)
    s["tree_v"] = _rows(B * T, Hkv, d, g, gv).view(B, T, Hkv, d)
    return dict(s, parents=_ints(_tree(T, r)))


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


def _softmax_rows(x, values):
    """(softmax over the last axis of x [.., M, n]) @ values [.., n, d], and the
    logarithm of its sum; x is overwritten."""
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    return (x @ values) / total, (total.log() + top)[..., 0]


def _plain_verify(s):
    q, T = s["q"].float(), s["T"]
    B, _, Hq, d = q.shape
    Hkv = s["tree_k"].shape[2]
    G, n = Hq // Hkv, max(s["lens"])
    pos = torch.arange(n, device=q.device).expand(B, n)
    held = (pos < s["seq_lens"][:, None])
    seq = torch.arange(B, device=q.device)[:, None].expand(B, n)

    def keys(which):  # [B][Hkv][n + T][d], zero where the sequence has ended
        x = torch.where(held[..., None, None], _get(s, which, seq, pos), 0.0)
        return torch.cat([x, s["tree_" + which].float()], 1).transpose(1, 2).contiguous()

    rows = q.view(B, T, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, d)
    x = rows @ keys("k").transpose(2, 3)
    x *= 1.0 / math.sqrt(d)
    see = torch.cat([held[:, None].expand(B, T, n), _ancestors(s["parents"]).expand(B, T, T)], 2)
    x.masked_fill_(~see.repeat_interleave(G, 1)[:, None], -math.inf)
    out, lse = _softmax_rows(x, keys("v"))
    out = out.view(B, Hkv, T, G, d).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, d)
    return out.bfloat16(), lse.view(B, Hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, Hq)


def _plain_prefill(s):
    q, k, v = s["q"], s["k"], s["v"]
    N, Hq, d = q.shape
    Hkv, B, n = k.shape[1], len(s["lens"]), max(s["lens"])
    G = Hq // Hkv
    seq, pos = _positions(s["lens"], 0)

    def padded(x):  # [B][H][n][d]
        y = torch.zeros(B, n, x.shape[1], d, device=x.device)
        y[seq, pos] = x.float()
        return y.transpose(1, 2).contiguous()

    x = padded(q).view(B, Hkv, G * n, d) @ padded(k).transpose(2, 3)
    x *= 1.0 / math.sqrt(d)
    at = torch.arange(n, device=q.device)
    x.view(B, Hkv, G, n, n).masked_fill_(at[None, :] > at[:, None], -math.inf)
    out, lse = _softmax_rows(x, padded(v))
    out = out.view(B, Hq, n, d).transpose(1, 2)[seq, pos]
    return out.bfloat16(), lse.view(B, Hq, n).transpose(1, 2)[seq, pos]


def run(s):
    op = s["op"]
    if own:
        import speculative_decoding_tree_split_gb300 as ta
        if op == "prefill":
            return ta.prefill(s["q"], s["k"], s["v"], s["cu"])
        cache = (s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["bt"])
        if op == "append":
            new = ta.kv_append_fp8(*cache, s["seq_lens"], s["cu"], s["k"], s["v"])
            return cache[:4] + (new,)
        if op == "commit":
            new = ta.kv_commit_fp8(*cache, s["seq_lens"], s["accept_path"], s["accept_len"],
                                   s["tree_k"], s["tree_v"])
            return cache[:4] + (new,)
        if op == "read":
            return ta.kv_read_fp8(*cache, s["cu"], sum(s["lens"]), starts=s["starts"])
        return ta.verify_fp8(s["q"], *cache, s["seq_lens"], s["tree_k"], s["tree_v"],
                             parents=s["parents"])
    if op == "prefill":
        return _plain_prefill(s)
    if op == "append":
        seq, pos = _positions(s["lens"], s["start"])
        _put(s, "k", seq, pos, s["k"])
        _put(s, "v", seq, pos, s["v"])
        new = s["seq_lens"] + (s["cu"][1:] - s["cu"][:-1])
        return s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], new
    if op == "commit":
        T = s["T"]
        b, j = (torch.arange(T, device=_dev()) < s["accept_len"][:, None]).nonzero(as_tuple=True)
        node = s["accept_path"][b, j].long()
        pos = s["seq_lens"][b].long() + j
        _put(s, "k", b, pos, s["tree_k"][b, node])
        _put(s, "v", b, pos, s["tree_v"][b, node])
        new = s["seq_lens"] + s["accept_len"]
        return s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], new
    if op == "read":
        seq, pos = _positions(s["lens"], s["start"])
        return _get(s, "k", seq, pos).bfloat16(), _get(s, "v", seq, pos).bfloat16()
    return _plain_verify(s)


def work(case):
    lens, op, d, Hkv, B = _lens(case), case["op"], case["d"], case["Hkv"], case["B"]
    N = sum(lens)
    row = d + 1  # bytes of a cache row: codes and the scale
    if op == "prefill":
        Hq = case["Hq"]
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return dict(bytes=N * (2 * Hq + 2 * Hkv) * d * 2 + N * Hq * 4 + 4 * (B + 1),
                    flops=4 * d * Hq * pairs)
    if op in ("append", "read"):
        return dict(bytes=N * Hkv * 2 * (2 * d + row) + 4 * B, flops=0)
    if op == "commit":
        n = sum(_accepted(case))
        return dict(bytes=n * Hkv * 2 * (2 * d + row) + 4 * (n + 3 * B), flops=0)
    T, Hq = case["T"], case["Hq"]
    table = sum(-(-n // case["page"]) for n in lens)
    return dict(bytes=N * Hkv * 2 * row + B * T * (2 * Hq + 2 * Hkv) * d * 2 + B * T * Hq * 4
                + 4 * (table + B + T), flops=4 * d * Hq * T * (N + B * (T + 1) // 2))


# The same from the definitions, in 64 bits, with code of its own.

def _two_to(e):
    """2^e of whole numbers e in 64 bits, put together from the bits (a pow() may
    be off by a last bit, which would move ties)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_row(x):
    """Codes (fp64 values) and exponent bytes of the rows of x, by the definition."""
    x = x.double()
    fine = x.abs().nan_to_num(0.0, 0.0, 0.0)
    big = fine.max(-1).values
    s = torch.ceil(torch.log2(big.clamp_min(1e-300) / CODE_MAX)).clamp(S_MIN, S_MAX)
    s = torch.where(CODE_MAX * _two_to(s) < big, s + 1, s)
    s = torch.where(CODE_MAX * _two_to(s - 1) >= big, s - 1, s).clamp(S_MIN, S_MAX)
    y = (x / _two_to(s)[..., None]).clamp(-CODE_MAX, CODE_MAX)
    # e4m3: steps of an eighth of the value's power of two, at least 2^-9
    step = _two_to(torch.frexp(y.abs().clamp_min(2.0 ** -6))[1] - 4)
    return torch.round(y / step) * step, (s + 127).to(torch.uint8)


def _exact_cache(s, spots):
    """The four pools after rows (b, position, k, v) have been written."""
    pools = [s["k_pages"].to(torch.float64), s["v_pages"].to(torch.float64),
             s["k_scales"].clone(), s["v_scales"].clone()]
    P = s["k_scales"].shape[2]
    b, pos, k, v = spots
    page, off = s["bt"][b, torch.div(pos, P, rounding_mode="floor")].long(), pos.remainder(P)
    for i, x in enumerate((k, v)):
        codes, scale = _exact_row(x)
        pools[i][page, :, off] = codes
        pools[2 + i][page, :, off] = scale
    return pools


def _exact_rows(s, which, b, lo, hi):
    """Cache rows lo..hi of sequence b in 64 bits: [hi - lo][Hkv][d]."""
    P = s["k_scales"].shape[2]
    first, last = lo // P, -(-hi // P)
    pages = s["bt"][b, first:last].long()
    codes = s[which + "_pages"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()
    scale = _two_to(s[which + "_scales"][pages].long() - 127)
    x = (codes * scale[..., None]).transpose(1, 2).flatten(0, 1)
    return x[lo - first * P:hi - first * P]


def _exact_attend(q, k, v, see):
    """q [T][Hq][d], k and v [n][Hkv][d], see [T][n] or None -> out, lse in 64 bits."""
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    out, lse = [], []
    for h in range(Hq):
        x = q[:, h].double() @ k[:, h * Hkv // Hq].double().T / math.sqrt(d)
        if see is not None:
            x = x.masked_fill_(~see, -math.inf)
        top = torch.logsumexp(x, 1)
        lse.append(top)
        out.append(x.sub_(top[:, None]).exp_() @ v[:, h * Hkv // Hq].double())
    return torch.stack(out, 1), torch.stack(lse, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op, lens = s["op"], s["lens"]
    if op == "append":
        b = torch.cat([torch.full((n,), i, dtype=torch.long) for i, n in enumerate(lens)]).to(_dev())
        at = torch.cat([torch.arange(n) for n in lens]).to(_dev()) + s["start"]
        new = s["seq_lens"] + _ints(lens)
        return (*_exact_cache(s, (b, at, s["k"], s["v"])), new)
    if op == "commit":
        n, path = s["accept_len"].tolist(), s["accept_path"].tolist()
        spots = [(i, lens[i] + j, path[i][j]) for i in range(len(n)) for j in range(n[i])]
        b, at, node = (torch.tensor(c, device=_dev()) for c in zip(*spots))
        new = s["seq_lens"] + s["accept_len"]
        return (*_exact_cache(s, (b, at, s["tree_k"][b, node], s["tree_v"][b, node])), new)
    if op == "read":
        return tuple(torch.cat([_exact_rows(s, w, b, s["start"], s["start"] + n)
                                for b, n in enumerate(lens)]) for w in "kv")
    outs, at = [], 0
    for b, n in enumerate(lens):
        if op == "prefill":
            see = torch.ones(n, n, dtype=torch.bool, device=_dev()).tril()
            outs.append(_exact_attend(*(s[w][at:at + n] for w in "qkv"), see))
            at += n
            continue
        T, up = s["T"], s["parents"].tolist()
        see = torch.zeros(T, n + T, dtype=torch.bool)
        see[:, :n] = True
        for i in range(T):
            j = i
            while j >= 0:
                see[i, n + j] = True
                j = up[j]
        k, v = (torch.cat([_exact_rows(s, w, b, 0, n), s["tree_" + w][b].double()]) for w in "kv")
        outs.append(_exact_attend(s["q"][b], k, v, see.to(_dev())))
    join = torch.cat if op == "prefill" else torch.stack
    return join([o for o, _ in outs]), join([x for _, x in outs])
