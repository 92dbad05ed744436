"""Host checks of the paged-cache entry points, without a GPU (fake, never
dereferenced addresses), and the sequential tables the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import rope_aware_kv_b200 as tri
from rope_aware_kv_b200 import build as tri_build
from tests import paged_ref as R

P = ctypes.c_void_p
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    tri_build.build()
    return tri.load()


def _decode(lib, **o):
    a = dict(q=1 << 36, k=1 << 37, v=1 << 38, dt=tri.TRI_BF16, S=2, L=3, H=4, layer=-1, G=7, d=128, table=1 << 39,
             rows=16, ppu=8, pages=1000, nv=16, scale=0.1, out=1 << 35, lse=None, ws=1 << 34, wb=BIG)
    a.update(o)
    return lib.tri_decode_attention_paged(P(a["q"]), P(a["k"]), P(a["v"]), a["dt"], a["S"], a["L"], a["H"], a["layer"],
                                          a["G"], a["d"], P(a["table"]), a["rows"], a["ppu"], a["pages"], P(a["nv"]),
                                          ctypes.c_float(a["scale"]), P(a["out"]), P(a["lse"]), P(a["ws"]), a["wb"],
                                          None)


def test_decode_refuses(lib):
    need = lib.tri_decode_paged_workspace_bytes(24, 7)
    assert need > 256 + 24 * 4
    assert lib.tri_decode_paged_workspace_bytes(0, 7) == 256
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(nv=None), dict(table=None),
                dict(S=0), dict(L=0), dict(H=0), dict(layer=3), dict(layer=-2), dict(rows=0), dict(ppu=0),
                dict(pages=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(q=(1 << 36) + 4), dict(k=(1 << 37) + 8), dict(out=(1 << 35) + 4), dict(lse=2), dict(nv=18),
                dict(table=(1 << 39) + 2)):
        assert _decode(lib, **bad) == 1, bad
    for bad in (dict(G=0), dict(G=9), dict(d=64), dict(dt=5), dict(rows=1 << 22, pages=1 << 10), dict(ppu=1 << 30),
                dict(S=1 << 30), dict(rows=1 << 20, ppu=1 << 12, pages=4)):
        assert _decode(lib, **bad) == 2, bad
    assert _decode(lib, wb=need - 1) == 3
    assert _decode(lib, ws=None) == 3
    assert _decode(lib, ws=(1 << 34) + 4) == 3


def _append(lib, **o):
    a = dict(k=1 << 36, v=1 << 37, pos=1 << 33, S=2, L=3, H=4, layer=1, cap=128, rows=16, ppu=8, pages=1000, refs=16,
             nv=16, pc=16, kn=1 << 38, vn=1 << 39, pn=16, add=16, n=5, ws=1 << 34, wb=BIG, dt=tri.TRI_F32, d=128)
    a.update(o)
    return lib.tri_append_paged(P(a["k"]), P(a["v"]), P(a["pos"]), a["dt"], a["S"], a["L"], a["H"], a["layer"], a["cap"],
                                a["d"], P(1 << 35), a["rows"], a["ppu"], a["pages"], P(a["refs"]), P(a["nv"]),
                                P(a["pc"]), P(a["kn"]), P(a["vn"]), P(a["pn"]), P(a["add"]), a["n"], P(a["ws"]),
                                a["wb"], None)


def test_append_refuses(lib):
    pool = 1000 * 16 * 512
    for bad in (dict(k=None), dict(nv=None), dict(n=-1), dict(cap=0), dict(cap=129), dict(kn=None), dict(v=None),
                dict(vn=None), dict(pos=None), dict(pn=None), dict(pos=None, pn=None), dict(pc=20), dict(k=(1 << 36) + 8),
                dict(kn=(1 << 38) + 4), dict(add=18), dict(refs=18), dict(kn=(1 << 36) + pool - 512),
                dict(vn=(1 << 37) - 512), dict(v=(1 << 36) + 512), dict(layer=3), dict(S=0)):
        assert _append(lib, **bad) == 1, bad
    assert _append(lib, d=64) == 2 and _append(lib, dt=9) == 2 and _append(lib, n=1 << 30) == 2
    assert _append(lib, wb=lib.tri_append_paged_workspace_bytes(8) - 1) == 3
    assert _append(lib, layer=-1, wb=lib.tri_append_paged_workspace_bytes(24) - 1) == 3


def test_pages_refuse(lib):
    need = lib.tri_pages_workspace_bytes(24, 8, 1000)
    assert need > 2 * 4 * 1000

    def fit(k=1 << 36, v=1 << 37, S=2, U=24, d=128, t=1 << 35, rows=16, refs=16, nv=16, add=16, n=5, nf=16, wb=need,
            dt=tri.TRI_BF16):
        return lib.tri_pages_fit(P(k), P(v), dt, S, U, d, P(t), rows, 8, 1000, P(refs), P(nv), P(add), n, 0, P(nf),
                                 P(1 << 34), wb, None)
    for bad in (dict(k=None), dict(refs=None), dict(nv=None), dict(t=None), dict(n=-1), dict(S=5), dict(U=0),
                dict(rows=0), dict(k=(1 << 36) + 2), dict(refs=18), dict(nf=18), dict(v=(1 << 36) + 4096)):
        assert fit(**bad) == 1, bad
    assert fit(d=64) == 2 and fit(dt=3) == 2 and fit(rows=1 << 24) == 2 and fit(wb=need - 1) == 3

    def fork(t=1 << 35, refs=16, S=2, U=24, src=16, dst=16, n=2, nv=16, pos=1 << 33, cap=128, pc=16, wb=need):
        return lib.tri_pages_fork(P(t), 16, 8, 1000, P(refs), S, U, P(src), P(dst), n, P(nv), P(pos), cap, P(pc),
                                  P(1 << 34), wb, None)
    for bad in (dict(t=None), dict(refs=None), dict(nv=None), dict(src=None), dict(dst=None), dict(n=-1), dict(S=7),
                dict(cap=129), dict(cap=0), dict(pc=20), dict(src=18)):
        assert fork(**bad) == 1, bad
    assert fork(n=1025) == 2 and fork(wb=need - 1) == 3

    def compact(k=1 << 36, v=None, t=1 << 35, refs=16, nl=16, wb=need, d=128):
        return lib.tri_pages_compact(P(k), P(v), tri.TRI_BF16, 24, d, P(t), 16, 8, 1000, P(refs), P(nl), P(1 << 34), wb,
                                     None)
    for bad in (dict(k=None), dict(refs=None), dict(t=None), dict(nl=18), dict(v=(1 << 36) + 16)):
        assert compact(**bad) == 1, bad
    assert compact(d=256) == 2 and compact(wb=need - 1) == 3


def test_sequential_tables_by_hand():
    """The sequential counterpart on a case worked out by hand: three holders
    of page 0; two of them write it and get copies, all of them and the last
    keeps it."""
    t = np.array([[0, 1], [0, -1], [0, -1]], np.int32)
    refs = np.array([3, 1, 0, 0, 0], np.int32)
    p = R.Pages(t, refs, np.array([4, 3, 2]), 3, 4)
    assert p.fit([0, 1, 1]) == 2  # page 1 given back: 4 free, two of them copies of page 0
    assert p.table.tolist() == [[0, -1], [1, -1], [2, -1]] and p.refs.tolist() == [1, 1, 1, 0, 0]
    assert p.copied == [(0, 1, 3), (0, 2, 2)]
    p = R.Pages(t, refs, np.array([4, 3, 2]), 3, 4)
    assert p.fit([0, 0, 0], own=True) == 2  # the last holder keeps page 0
    assert p.table.tolist() == [[1, -1], [2, -1], [0, -1]] and p.refs.tolist() == [1, 1, 1, 0, 0]
    assert p.fork([1, 0], [0, 1]) == 0 and p.table.tolist() == [[2, -1], [1, -1], [0, -1]]
    assert p.fork([-1], [1]) == 0 and p.refs.tolist() == [1, 0, 1, 0, 0]
    assert p.compact() == 2 and p.table.tolist() == [[1, -1], [-1, -1], [0, -1]]
    p.check()


def test_decode_refuses_a_scale_whose_base_2_form_overflows(lib):
    """scale * log2(e) is what the scores are multiplied with: as infinity it
    would turn a score of 0 into NaN."""
    for scale in (2.4e38, 3.4e38):
        with np.errstate(over="ignore"):
            assert np.isfinite(np.float32(scale)) and np.isinf(np.float32(scale) * np.float32(1.4426950408889634))
        assert _decode(lib, scale=scale) == 1
    assert _decode(lib, scale=2.3e38, ws=None) == 3
