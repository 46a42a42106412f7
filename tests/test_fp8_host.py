"""The 8-bit cache, verification over it and the prompt attention, as far as
the host goes: the row format's definition, and every refusal (CPU only)."""
import numpy as np
import pytest
import torch

import speculative_decoding_tree_split_gb300 as ta
from oracle import fp8_rows

A = 1 << 20  # a fake, never dereferenced device address


@pytest.fixture(scope="module")
def lib():
    ta.build()
    return ta.load()


# ---------------------------------------------------------------------------
# the row format's definition
# ---------------------------------------------------------------------------
def test_code_values_are_e4m3s():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    got = fp8_rows.code_values()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


def test_encode_agrees_with_a_conversion_of_the_scaled_row():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(500, 64, generator=g) * torch.exp(6 * torch.randn(500, 1, generator=g))
    x = x.bfloat16().double()
    codes, byte = fp8_rows.encode(x.numpy())
    y = (x * torch.exp2(127 - torch.from_numpy(byte).double())[:, None]).float()
    assert float(y.abs().max()) <= 448
    want = y.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes, want)
    # the exponent is the smallest that fits
    top = x.abs().amax(1).numpy()
    s = byte.astype(int) - 127
    assert (top <= 448 * 2.0 ** s).all()
    assert ((s == fp8_rows.S_MIN) | (top > 448 * 2.0 ** (s - 1))).all()


def test_encode_edges():
    inf, nan = float("inf"), float("nan")
    rows = np.array([[0.0, -0.0], [448.0, 449.0], [448.0, 1.0], [inf, 2.0], [nan, -1.0],
                     [2.0 ** 120, 1.0], [2.0 ** -120, 0.0], [nan, -inf]])
    codes, byte = fp8_rows.encode(rows)
    assert list(byte.astype(int) - 127) == [-56, 1, 0, -7, -8, 40, -56, -56]
    v = fp8_rows.decode(codes, byte)
    assert v[0, 0] == 0 and v[0, 1] == 0 and codes[0, 1] == 128
    assert v[1, 0] == 448 and v[1, 1] == 448       # 449 / 2 rounds down to 224
    assert v[3, 0] == 448 * 2.0 ** -7 and v[3, 1] == 2
    assert np.isnan(v[4, 0]) and v[4, 1] == -1
    assert v[5, 0] == 448 * 2.0 ** 40 and v[5, 1] == 0
    assert v[6, 0] == 0
    assert np.isnan(v[7, 0]) and v[7, 1] == -448 * 2.0 ** -56


# ---------------------------------------------------------------------------
# refusals of the C entries
# ---------------------------------------------------------------------------
def _append(lib, **kw):
    a = dict(kp=A, vp=A, ks=A, vs=A, bt=A, maxp=4, sl=A, cu=A, k=A, v=A, st=(16, 16, 16, 16),
             out=A + 256, B=2, N=8, Hkv=2, d=128, P=64, NP=8, status=None)
    a.update(kw)
    return lib.tree_kv_append_fp8(a["kp"], a["vp"], a["ks"], a["vs"], a["bt"], a["maxp"], a["sl"],
                                  a["cu"], a["k"], a["v"], *a["st"], a["out"], a["B"], a["N"],
                                  a["Hkv"], a["d"], a["P"], a["NP"], a["status"], None)


def test_append_refusals(lib):
    for kw in (dict(d=96), dict(P=48), dict(maxp=0), dict(NP=0), dict(Hkv=0), dict(B=-1),
               dict(N=-1), dict(out=A), dict(NP=1 << 24, Hkv=8)):
        assert _append(lib, **kw) == -2, kw
    for name in ("kp", "vp", "ks", "vs", "bt", "sl", "cu", "k", "v"):
        assert _append(lib, **{name: None}) == -1, name
    for kw in (dict(kp=A + 8), dict(vs=A + 4), dict(bt=A + 2), dict(sl=A + 1), dict(cu=A + 2),
               dict(k=A + 8), dict(out=A + 258), dict(status=A + 2), dict(st=(4, 16, 16, 16)),
               dict(st=(16, 16, 16, 12))):
        assert _append(lib, **kw) == -3, kw
    assert _append(lib, B=0, kp=None) == 0


def _commit(lib, **kw):
    a = dict(kp=A, vp=A, ks=A, vs=A, bt=A, maxp=4, sl=A, path=A, n=A, tk=A, tv=A, out=A + 256,
             B=2, Hkv=2, d=128, T=4, P=64, NP=8, status=None)
    a.update(kw)
    return lib.tree_kv_commit_fp8(a["kp"], a["vp"], a["ks"], a["vs"], a["bt"], a["maxp"], a["sl"],
                                  a["path"], a["n"], a["tk"], a["tv"], a["out"], a["B"], a["Hkv"],
                                  a["d"], a["T"], a["P"], a["NP"], a["status"], None)


def test_commit_refusals(lib):
    for kw in (dict(d=96), dict(T=0), dict(T=65), dict(P=8), dict(out=A), dict(B=-1)):
        assert _commit(lib, **kw) == -2, kw
    for name in ("kp", "vp", "ks", "vs", "bt", "sl", "path", "n", "tk", "tv"):
        assert _commit(lib, **{name: None}) == -1, name
    for kw in (dict(ks=A + 8), dict(tk=A + 8), dict(path=A + 2), dict(n=A + 1)):
        assert _commit(lib, **kw) == -3, kw
    assert _commit(lib, B=0, kp=None) == 0


def _read(lib, **kw):
    a = dict(kp=A, vp=A, ks=A, vs=A, bt=A, maxp=4, starts=None, cu=A, ko=A, vo=A, B=2, N=8, Hkv=2,
             d=128, P=64, NP=8, status=None)
    a.update(kw)
    return lib.tree_kv_read_fp8(a["kp"], a["vp"], a["ks"], a["vs"], a["bt"], a["maxp"],
                                a["starts"], a["cu"], a["ko"], a["vo"], a["B"], a["N"], a["Hkv"],
                                a["d"], a["P"], a["NP"], a["status"], None)


def test_read_refusals(lib):
    for kw in (dict(d=32), dict(P=256), dict(N=-1), dict(NP=0)):
        assert _read(lib, **kw) == -2, kw
    for name in ("kp", "vp", "ks", "vs", "bt", "cu", "ko", "vo"):
        assert _read(lib, **{name: None}) == -1, name
    for kw in (dict(ko=A + 8), dict(starts=A + 2), dict(cu=A + 2)):
        assert _read(lib, **kw) == -3, kw
    assert _read(lib, B=0, kp=None) == 0
    assert _read(lib, N=0, ko=None) == 0


def _verify(lib, **kw):
    a = dict(q=A, kp=A, vp=A, ks=A, vs=A, bt=A, maxp=4, sl=A, tk=A, tv=A, mask=A, ms=0, par=None,
             ps=0, mo=None, out=A, lse=A, B=2, Hq=8, Hkv=2, d=128, T=4, P=64, NP=8, scale=0.1,
             ws=A, wsb=1 << 40, status=None)
    a.update(kw)
    return lib.tree_attn_verify_fp8(
        a["q"], a["kp"], a["vp"], a["ks"], a["vs"], a["bt"], a["maxp"], a["sl"], a["tk"], a["tv"],
        a["mask"], a["ms"], a["par"], a["ps"], a["mo"], a["out"], a["lse"], a["B"], a["Hq"],
        a["Hkv"], a["d"], a["T"], a["P"], a["NP"], a["scale"], a["ws"], a["wsb"], a["status"], None)


def test_verify_refusals(lib):
    for kw in (dict(T=0), dict(T=65), dict(Hq=6, Hkv=4), dict(d=96), dict(P=48), dict(maxp=0),
               dict(NP=0), dict(NP=1 << 24, Hkv=8, Hq=8), dict(scale=float("nan")), dict(ms=3),
               dict(par=A), dict(mask=None, par=A, ps=2)):
        assert _verify(lib, **kw) == -2, kw
    for name in ("q", "kp", "vp", "ks", "vs", "bt", "sl", "tk", "tv", "mask", "out", "lse"):
        assert _verify(lib, **{name: None}) == -1, name
    for kw in (dict(q=A + 8), dict(kp=A + 8), dict(vs=A + 8), dict(bt=A + 2), dict(mask=A + 4),
               dict(mask=None, par=A + 2), dict(mask=None, par=A, mo=A + 4), dict(lse=A + 2),
               dict(status=A + 1)):
        assert _verify(lib, **kw) == -3, kw
    assert _verify(lib, B=0, q=None) == 0


def _prefill(lib, **kw):
    a = dict(q=A, k=A, v=A, st=(16,) * 6, cu=A, out=A, lse=A, B=2, N=8, Hq=8, Hkv=2, d=128,
             scale=0.1, status=None)
    a.update(kw)
    return lib.tree_attn_prefill(a["q"], a["k"], a["v"], *a["st"], a["cu"], a["out"], a["lse"],
                                 a["B"], a["N"], a["Hq"], a["Hkv"], a["d"], a["scale"],
                                 a["status"], None)


def test_prefill_refusals(lib):
    for kw in (dict(d=96), dict(Hq=6, Hkv=4), dict(Hq=1, Hkv=2), dict(N=-1), dict(B=-1),
               dict(scale=float("inf"))):
        assert _prefill(lib, **kw) == -2, kw
    for name in ("q", "k", "v", "cu", "out", "lse"):
        assert _prefill(lib, **{name: None}) == -1, name
    for kw in (dict(q=A + 8), dict(out=A + 8), dict(lse=A + 2), dict(cu=A + 2), dict(status=A + 1),
               dict(st=(16, 16, 16, 4, 16, 16))):
        assert _prefill(lib, **kw) == -3, kw
    assert _prefill(lib, B=0, q=None) == 0
    assert _prefill(lib, N=0, q=None) == 0


def test_prefill_refuses_strides_it_cannot_walk(lib):
    for i in range(6):  # negative ones, of q, k and v
        st = [16] * 6
        st[i] = -16
        assert _prefill(lib, st=tuple(st)) == -2, i
    for i in (2, 4):    # one key or value for all tokens
        st = [16] * 6
        st[i] = 0
        assert _prefill(lib, st=tuple(st)) == -2, i
    assert _prefill(lib, N=1 << 30, Hq=16, Hkv=2) == -2  # rows past 32 bits


def test_the_binding_refuses_cpu_tensors():
    z = torch.zeros
    pools = (z(2, 1, 16, 64, dtype=torch.uint8), z(2, 1, 16, 64, dtype=torch.uint8),
             z(2, 1, 16, dtype=torch.uint8), z(2, 1, 16, dtype=torch.uint8),
             z(1, 2, dtype=torch.int32))
    row = z(4, 1, 64, dtype=torch.bfloat16)
    one, two = z(1, dtype=torch.int32), z(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        ta.kv_append_fp8(*pools, one, two, row, row)
    with pytest.raises(ValueError):
        ta.kv_commit_fp8(*pools, one, z(1, 4, dtype=torch.int32), one, row[None], row[None])
    with pytest.raises(ValueError):
        ta.kv_read_fp8(*pools, two, 4)
    with pytest.raises(ValueError):
        ta.verify_fp8(row[None], *pools, one, row[None], row[None], parents=one)
    with pytest.raises(ValueError):
        ta.prefill(row, row, row, two)
    with pytest.raises(TypeError):
        ta.prefill([1], row, row, two)
