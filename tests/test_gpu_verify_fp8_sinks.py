"""verify_fp8 where one key holds much of a row's weight and the rest is spread
over thousands of small probabilities (a first token that draws the attention, a
retrieved one in the middle), with values that do not average out, against 64
bits over the cache as it reads back.  There are at least as many units as SMs,
so that a unit's keys are not cut into short pieces.

Tolerances.  Let A = sum_j p_j |v_j| / l and M = max_j p_j max|v_j| / l.  A
probability is rounded to fp16 (half a step: 2^-11 of it, or half of 2^-24 where
the p 2^(value scale) that the kernel holds is that small; the largest is at
least 2^7, a code is at most 448 and the largest of a row at least 224), has
2 dx from the errors dx of its score and of the sum, and the result is
rounded to bf16 once:
    |out - ref| <= 2^-8 |ref| + (1 + 2^-7) ((2^-11 + 2 dx) A + n 2^-31 M),
    dx = scale (2^-17 + 2^-20) max|q| max_j sum|k_j| + 2^-18.
|lse - ref| <= dx.
"""
import math

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


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def attend(q, k, v, tk, tv, see):
    """q [T][Hq][d], k and v [n][Hkv][d], tk and tv [T][Hkv][d], see [T][T] in 64
    bits: out, lse, sum p |v| / l and max p max|v| / l."""
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    G, n = Hq // Hkv, k.shape[0]
    out, A = torch.empty(2, T, Hq, d, dtype=torch.float64, device="cuda")
    lse, M = torch.empty(2, T, Hq, dtype=torch.float64, device="cuda")
    for h in range(Hkv):
        g = slice(h * G, (h + 1) * G)
        kk, vv = torch.cat([k[:, h], tk[:, h]]).double(), torch.cat([v[:, h], tv[:, h]]).double()
        x = q[:, g].double() @ kk.T / math.sqrt(d)
        x[..., n:].masked_fill_(~see[:, None], -math.inf)
        lse[:, g] = torch.logsumexp(x, 2)
        p = (x - lse[:, g, None]).exp()
        out[:, g], A[:, g] = p @ vv, p @ vv.abs()
        M[:, g] = (p * vv.abs().amax(1)).amax(2)
    return out, lse, A, M


def close(out, lse, q, k, v, tk, tv, see):
    ref, ref_l, A, M = attend(q, k, v, tk, tv, see)
    d = q.shape[2]
    ksum = max(float(k.float().abs().sum(2).max()), float(tk.float().abs().sum(2).max()))
    dx = ((2.0 ** -17 + 2.0 ** -20) / math.sqrt(d) * ksum * q.double().abs().amax(2)
          + 2.0 ** -18)
    tol = (2.0 ** -8 * ref.abs() + (1 + 2.0 ** -7)
           * ((2.0 ** -11 + 2 * dx[..., None]) * A + k.shape[0] * 2.0 ** -31 * M[..., None]))
    off = (out.double() - ref).abs()
    assert bool((off <= tol).all()), (float(off.max()), float((off / tol).max()))
    off = (lse.double() - ref_l).abs()
    assert bool((off <= dx).all()), float(off.max())


def cache_of(B, L, Hkv, d, P, k, v):
    """B sequences of L tokens [B * L][Hkv][d], written by the library."""
    per = -(-L // P)
    n = B * per
    pools = [torch.full((n, Hkv, P, d), 255, dtype=torch.uint8, device="cuda") for _ in "kv"]
    pools += [torch.full((n, Hkv, P), 255, dtype=torch.uint8, device="cuda") for _ in "kv"]
    bt = torch.randperm(n, generator=torch.Generator().manual_seed(n)).int().view(B, per).cuda()
    cu = torch.arange(B + 1, device="cuda", dtype=torch.int32) * L
    lens = ta.kv_append_fp8(*pools, bt, torch.zeros(B, dtype=torch.int32, device="cuda"), cu, k, v)
    return (*pools, bt), lens, cu


CASES = [
    # keys, weight of the one key, spread of the others' scores (nats), the one
    # key's position, its value, T, G, d
    (4096, 0.9, 0.5, 0, "as others", 1, 1, 128),
    (16384, 0.5, 0.5, 0, "as others", 4, 4, 128),
    (16384, 0.5, 0.3, 8000, "as others", 1, 4, 64),
    (16384, 0.9, 1.0, 0, "a tenth", 2, 8, 128),
    (16384, 0.5, 0.5, 5000, "one wide channel", 4, 8, 128),
    (16384, 0.5, 1.0, 0, "as others", 16, 3, 128),     # 48 rows
    (16384, 0.5, 0.5, 0, "as others", 8, 8, 64),       # 64 rows
    (16384, 0.5, 0.5, 0, "as others", 16, 5, 128),     # 80 rows
    (16384, 0.3, 0.5, 9001, "as others", 16, 8, 128),  # 128 rows
    (16384, 0.5, 0.5, 0, "as others", 16, 8, 64),
    (32768, 0.3, 1.0, 0, "as others", 4, 4, 128),
    (32768, 0.5, 0.0, 20000, "as others", 1, 2, 64),   # the others all alike
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_one_large_probability_among_many_small_ones(i):
    L, weight, spread, at, value, T, G, d = CASES[i]
    Hkv, P = 4, 64
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B = -(-sms // Hkv)
    g = torch.Generator("cuda").manual_seed(100 + i)

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    # queries close to a common direction of each KV head; the one key lies along it
    e = rnd(B, 1, Hkv, 1, d).sign()
    q = (e + 0.05 * rnd(B, T, Hkv, G, d)).reshape(B, T, Hkv * G, d).bfloat16()
    k = (spread * rnd(B, L, Hkv, d)).bfloat16()
    v = (rnd(B, L, Hkv, d) + 0.5).bfloat16()
    score = math.log(weight / (1 - weight)) + math.log(L) + spread ** 2 / 2
    k[:, at] = (e[:, 0, :, 0] * score / math.sqrt(d)).bfloat16()
    if value == "a tenth":
        v[:, at] *= 0.1
    elif value == "one wide channel":
        v[:, at, :, 3] = 4096.0
    cache, lens, cu = cache_of(B, L, Hkv, d, P, k.view(B * L, Hkv, d), v.view(B * L, Hkv, d))
    tk, tv = rnd(B, T, Hkv, d).bfloat16(), (rnd(B, T, Hkv, d) + 0.5).bfloat16()
    parents = ints(list(range(-1, T - 1)))  # a chain: node i sees nodes 0 .. i
    status = ints([0])
    out, lse = ta.verify_fp8(q, *cache, lens, tk, tv, parents=parents, status=status)
    ck, cv = ta.kv_read_fp8(*cache, cu, B * L, status=status)
    assert int(status) == 0
    see = torch.ones(T, T, dtype=torch.bool, device="cuda").tril()
    for b in range(B):
        close(out[b], lse[b], q[b], ck[b * L:(b + 1) * L], cv[b * L:(b + 1) * L], tk[b], tv[b],
              see)
