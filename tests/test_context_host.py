"""The C entries of the operators for long contexts and several hypotheses refuse bad
arguments on the host, before any CUDA call (CPU only)."""
import ctypes

import pytest

import speculative_decoding_tree_split_gb300 as ta

A = 0x10000  # a fake device address, never dereferenced


@pytest.fixture(scope="module")
def lib():
    ta.build()
    return ta.load()


def pools(*ptrs, size=64):
    return (ctypes.c_void_p * len(ptrs))(*ptrs), (ctypes.c_size_t * len(ptrs))(*[size] * len(ptrs))


def copy(lib, ptrs=(A,), size=64, **kw):
    p, s = pools(*ptrs, size=size)
    a = dict(pools=p, bytes=s, n_pools=len(ptrs), src=A, dst=A, count=None, n=3, pages=8, status=None)
    a.update(kw)
    return lib.tree_kv_copy_pages(a["pools"], a["bytes"], a["n_pools"], a["src"], a["dst"], a["count"],
                                  a["n"], a["pages"], a["status"], None)


def test_copy_pages(lib):
    for kw in (dict(n=-1), dict(n=1 << 30), dict(pages=1 << 30), dict(pages=0), dict(n_pools=-1), dict(size=0), dict(size=(1 << 31) + 1)):
        assert copy(lib, **kw) == -2
    for kw in (dict(src=None), dict(dst=None), dict(pools=None), dict(bytes=None), dict(ptrs=(A, None))):
        assert copy(lib, **kw) == -1
    for kw in (dict(src=A + 1), dict(dst=A + 2), dict(count=A + 2), dict(status=A + 1)):
        assert copy(lib, **kw) == -3
    assert copy(lib, n=0, src=None) == 0 and copy(lib, n_pools=0) == 0


def fork(lib, **kw):
    p, s = pools(A)
    need = lib.tree_kv_fork_workspace_size(2, 3, 2049)
    a = dict(pools=p, bytes=s, n_pools=1, bt=A, maxp=4, lens=A, refs=A, src=A, reserve=None, all=0,
             bt_out=2 * A, lens_out=2 * A, refs_out=2 * A, rows_in=2, rows_out=3, P=16, pages=2049, ws=A,
             ws_bytes=need, status=None)
    a.update(kw)
    return lib.tree_kv_fork(a["pools"], a["bytes"], a["n_pools"], a["bt"], a["maxp"], a["lens"],
                            a["refs"], a["src"], a["reserve"], a["all"], a["bt_out"], a["lens_out"],
                            a["refs_out"], a["rows_in"], a["rows_out"], a["P"], a["pages"], a["ws"],
                            a["ws_bytes"], a["status"], None)


def test_fork(lib):
    need = lib.tree_kv_fork_workspace_size(2, 3, 2049)
    assert need > 0 and lib.tree_kv_fork_workspace_size(-1, 3, 8) == 0
    assert lib.tree_kv_fork_workspace_size(2, 3, 0) == 0
    assert lib.tree_kv_fork_workspace_size(16, 16, 2048) == 0
    assert lib.tree_kv_fork_workspace_size(17, 3, 8) > 0 and lib.tree_kv_fork_workspace_size(2, 17, 8) > 0
    for kw in (dict(rows_in=-1), dict(rows_out=1 << 24), dict(rows_out=1 << 16, maxp=1 << 15), dict(maxp=0), dict(pages=0), dict(P=24),
               dict(all=-1), dict(bt_out=A), dict(lens_out=A), dict(refs_out=A), dict(n_pools=-1)):
        assert fork(lib, **kw) == -2, kw
    for name in ("bt", "lens", "refs", "src", "bt_out", "lens_out", "refs_out", "pools"):
        assert fork(lib, **{name: None}) == -1, name
    for name in ("bt", "lens", "refs", "src", "reserve", "bt_out", "lens_out", "refs_out", "status"):
        assert fork(lib, **{name: 3 * A + 2}) == -3, name
    for kw in (dict(ws=None), dict(ws=A + 16), dict(ws_bytes=need - 1)):
        assert fork(lib, **kw) == -4


def compact(lib, **kw):
    p, s = pools(A)
    a = dict(pools=p, bytes=s, n_pools=1, bt=A, maxp=4, refs=A, bt_out=2 * A, refs_out=2 * A, n=A,
             rows=2, pages=8, ws=A, ws_bytes=lib.tree_kv_compact_workspace_size(8), status=None)
    a.update(kw)
    return lib.tree_kv_compact(a["pools"], a["bytes"], a["n_pools"], a["bt"], a["maxp"], a["refs"],
                               a["bt_out"], a["refs_out"], a["n"], a["rows"], a["pages"], a["ws"],
                               a["ws_bytes"], a["status"], None)


def test_compact(lib):
    need = lib.tree_kv_compact_workspace_size(2049)
    assert need > 0 and lib.tree_kv_compact_workspace_size(2048) == 0
    assert lib.tree_kv_compact_workspace_size(0) == 0
    for kw in (dict(rows=-1), dict(maxp=0), dict(pages=0), dict(refs_out=A), dict(n_pools=-1)):
        assert compact(lib, **kw) == -2, kw
    for name in ("bt", "refs", "bt_out", "refs_out", "n", "pools"):
        assert compact(lib, **{name: None}) == -1, name
    for name in ("bt", "refs", "bt_out", "refs_out", "n", "status"):
        assert compact(lib, **{name: 3 * A + 2}) == -3, name
    for kw in (dict(ws=None), dict(ws=A + 16), dict(ws_bytes=need - 1)):
        assert compact(lib, **dict(dict(pages=2049, ws_bytes=need), **kw)) == -4


def beam(lib, **kw):
    a = dict(x=A, dtype=0, bs=400, ws=100, scores=A, done=None, eos=-1, so=A, ro=A, to=A, B=20, W=4,
             V=100, K=4, work=A, bytes=lib.tree_beam_workspace_size(20, 4, 100, 4))
    a.update(kw)
    return lib.tree_beam_select(a["x"], a["dtype"], a["bs"], a["ws"], a["scores"], a["done"], a["eos"],
                                a["so"], a["ro"], a["to"], a["B"], a["W"], a["V"], a["K"], a["work"],
                                a["bytes"], None)


def test_beam(lib):
    need = lib.tree_beam_workspace_size(20, 4, 100, 4)
    assert need > 0 and lib.tree_beam_workspace_size(2, 4, 100, 4) == 0
    assert lib.tree_beam_workspace_size(1, 4, 40000, 4) > 0
    for sizes in ((2, 0, 100, 4), (2, 65, 100, 4), (2, 4, 0, 4), (2, 4, 100, 65), (2, 4, 100, 0),
                  (20000, 4, 100, 4), (1, 64, 1 << 20, 64)):
        assert lib.tree_beam_workspace_size(*sizes) == 0
    for kw in (dict(B=-1), dict(W=0), dict(W=65), dict(V=0), dict(K=0), dict(K=65), dict(dtype=3),
               dict(dtype=-1), dict(bs=-1), dict(ws=-1), dict(done=A, eos=-1), dict(done=A, eos=100),
               dict(B=20000)):
        assert beam(lib, **kw) == -2, kw
    for name in ("x", "scores", "so", "ro", "to"):
        assert beam(lib, **{name: None}) == -1, name
    for kw in (dict(x=A + 1), dict(x=A + 2, dtype=2), dict(scores=A + 2), dict(so=A + 1),
               dict(ro=A + 2), dict(to=A + 2)):
        assert beam(lib, **kw) == -3, kw
    for kw in (dict(work=None), dict(work=A + 16), dict(bytes=need - 1)):
        assert beam(lib, **kw) == -4, kw
    assert beam(lib, B=0, x=None) == 0


def bounds(lib, **kw):
    a = dict(k=A, ks=None, bt=A, maxp=4, starts=None, lens=A, out=A, exps=A, B=2, H=2, d=64, P=16,
             pages=8, status=None)
    a.update(kw)
    return lib.tree_kv_block_bounds(a["k"], a["ks"], a["bt"], a["maxp"], a["starts"], a["lens"],
                                    a["out"], a["exps"], a["B"], a["H"], a["d"], a["P"], a["pages"],
                                    a["status"], None)


def test_bounds(lib):
    for kw in (dict(B=-1), dict(B=65536), dict(H=0), dict(d=96), dict(P=8), dict(maxp=0), dict(pages=0),
               dict(pages=1 << 27), dict(maxp=1 << 28), dict(maxp=1 << 20, H=1 << 10, pages=1)):
        assert bounds(lib, **kw) == -2, kw
    for name in ("k", "bt", "lens", "out", "exps"):
        assert bounds(lib, **{name: None}) == -1, name
    for kw in (dict(k=A + 8), dict(out=A + 8), dict(bt=A + 1), dict(lens=A + 2), dict(starts=A + 2),
               dict(status=A + 2)):
        assert bounds(lib, **kw) == -3, kw
    assert bounds(lib, B=0, k=None) == 0


def select(lib, **kw):
    a = dict(q=A, b=A, e=A, bt=A, maxp=4, lens=A, out=A, B=2, Hq=8, H=2, d=64, T=2, P=16, pages=8, k=3,
             first=1, last=1, status=None)
    a.update(kw)
    return lib.tree_select_blocks(a["q"], a["b"], a["e"], a["bt"], a["maxp"], a["lens"], a["out"],
                                  a["B"], a["Hq"], a["H"], a["d"], a["T"], a["P"], a["pages"], a["k"],
                                  a["first"], a["last"], a["status"], None)


def test_select(lib):
    for kw in (dict(B=-1), dict(H=0), dict(Hq=7), dict(Hq=0), dict(Hq=258), dict(d=32), dict(T=0),
               dict(T=65), dict(P=48), dict(maxp=0), dict(maxp=262145), dict(pages=0), dict(k=0),
               dict(k=4097), dict(first=-1), dict(last=-1), dict(first=2, last=2),
               dict(first=2147483647, last=2147483647)):
        assert select(lib, **kw) == -2, kw
    for name in ("q", "b", "e", "bt", "lens", "out"):
        assert select(lib, **{name: None}) == -1, name
    for kw in (dict(q=A + 8), dict(b=A + 4), dict(bt=A + 2), dict(lens=A + 1), dict(out=A + 2),
               dict(status=A + 2)):
        assert select(lib, **kw) == -3, kw
    assert select(lib, B=0, q=None) == 0


def attend(lib, **kw):
    a = dict(q=A, k=A, v=A, ks=None, vs=None, bt=A, maxp=4, lens=A, blocks=A, n=3, tk=A, tv=A, mask=A,
             ms=0, par=None, ps=0, out=A, lse=A, B=2, Hq=8, H=2, d=64, T=2, P=16, pages=8, scale=0.1,
             status=None)
    a.update(kw)
    return lib.tree_attn_verify_blocks(
        a["q"], a["k"], a["v"], a["ks"], a["vs"], a["bt"], a["maxp"], a["lens"], a["blocks"], a["n"],
        a["tk"], a["tv"], a["mask"], a["ms"], a["par"], a["ps"], a["out"], a["lse"], a["B"], a["Hq"],
        a["H"], a["d"], a["T"], a["P"], a["pages"], a["scale"], a["status"], None)


def test_verify_blocks(lib):
    for kw in (dict(B=-1), dict(H=0), dict(Hq=7), dict(Hq=0), dict(d=32), dict(T=0), dict(T=65),
               dict(P=48), dict(maxp=0), dict(pages=0), dict(pages=1 << 27), dict(n=-1), dict(n=4097),
               dict(scale=float("inf")), dict(par=A), dict(ms=1), dict(mask=None, par=A, ps=3),
               dict(ks=A), dict(vs=A)):
        assert attend(lib, **kw) == -2, kw
    for name in ("q", "k", "v", "bt", "lens", "blocks", "tk", "tv", "mask", "out", "lse"):
        assert attend(lib, **{name: None}) == -1, name
    for kw in (dict(q=A + 8), dict(k=A + 8), dict(v=A + 2), dict(bt=A + 2), dict(lens=A + 1),
               dict(blocks=A + 2), dict(ks=A + 8, vs=A), dict(ks=A, vs=A + 4), dict(tk=A + 8), dict(tv=A + 8), dict(mask=A + 4),
               dict(mask=None, par=A + 2), dict(out=A + 8), dict(lse=A + 2), dict(status=A + 2)):
        assert attend(lib, **kw) == -3, kw
    assert attend(lib, B=0, q=None) == 0


def test_binding_refuses_cpu_tensors():
    import torch
    t = torch.zeros(2, 2, dtype=torch.int32)
    for call in (lambda: ta.kv_fork([], t, t[0], t[0], t[0], 16), lambda: ta.kv_compact([], t, t[0]),
                 lambda: ta.kv_copy_pages([], t[0], t[1]),
                 lambda: ta.beam_select(torch.zeros(1, 1, 2), torch.zeros(1, 1), 1),
                 lambda: ta.kv_block_bounds(torch.zeros(1, 1, 16, 64).bfloat16(), t, t[0]),
                 lambda: ta.select_blocks(torch.zeros(1, 1, 1, 64).bfloat16(), t, t, t, t[0], 1, 16)):
        with pytest.raises(ValueError):
            call()
