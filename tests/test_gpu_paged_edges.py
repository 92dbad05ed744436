"""Paged-cache calls at their edges: entries and counts out of range, forks of
many sequences, and how near the attention comes to float64 where the scores
are exact."""
import subprocess
import sys

import numpy as np
import pytest
import torch

import rope_aware_kv_b200 as tri
from rope_aware_kv_b200 import build as tri_build
from tests import paged_ref as R
from tests.test_gpu_paged import BF16, DEV, F32, _cache, _i32, _rows, _state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tri_build.build()
    tri.load()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("moves", [True, False])
def test_compact_flags_bad_entries(moves):
    """Entries below -1 or past the pool are left and flagged, whether or not
    a page moves; the others follow their pages."""
    page = 8
    table = np.array([[0, 4, -1], [1, -9, 6]] if moves else [[0, 1, -1], [2, -9, 6]], np.int32)
    refs = np.zeros(6, np.int32)
    refs[table[(table >= 0) & (table < 6)]] = 1
    k = torch.randn((6, page, R.D), device=DEV).to(BF16)
    want = k.clone()
    if moves:
        want[2] = k[4]
    t, c = _i32(table), _i32(refs)
    ws = tri.workspace(tri.tri_pages_workspace_bytes(2, 3, 6))
    assert tri.tri_pages_compact(k, None, t, c, ws=ws).item() == 3
    assert tri.tri_check_device_error(ws) == tri.FLAG_INDEX_RANGE
    assert t.cpu().tolist() == ([[0, 2, -1], [1, -9, 6]] if moves else [[0, 1, -1], [2, -9, 6]])
    assert c.cpu().tolist() == [1, 1, 1, 0, 0, 0]
    assert torch.equal(k, want)
    t = _i32(np.where((table < -1) | (table >= 6), -1, table))  # the same without them: no flag
    c = _i32(refs)
    tri.tri_pages_compact(want, None, t, c, ws=ws)
    assert tri.tri_check_device_error(ws) == 0


@pytest.mark.parametrize("crossed", [False, True])
def test_fork_flags_bad_entries_of_the_destination(crossed):
    """An entry of a replaced sequence that names no page is dropped and
    flagged; its valid entries give their pages back."""
    page = 4
    table = np.array([[0, 1, -1], [2, 9, -7], [3, -1, -1]], np.int32)
    refs = _i32([1, 1, 1, 1, 0])
    t, c, n = _i32(table), refs.clone(), _i32([6, 3, 4])
    src, dst = ([0, 1], [1, 2]) if crossed else ([0], [1])
    ws = tri.workspace(tri.tri_pages_workspace_bytes(3, 3, 5))
    tri.tri_pages_fork(t, c, page, 3, n, _i32(src), _i32(dst), ws=ws)
    assert tri.tri_check_device_error(ws) == tri.FLAG_INDEX_RANGE
    assert t.cpu().tolist() == [[0, 1, -1], [0, 1, -1], [2, -1, -1] if crossed else [3, -1, -1]]
    assert c.cpu().tolist() == ([2, 2, 1, 0, 0] if crossed else [2, 2, 0, 1, 0])
    assert n.cpu().tolist() == [6, 6, 3 if crossed else 4]
    tri.tri_pages_fork(t, c, page, 3, n, _i32(src), _i32(dst), ws=ws)  # nothing bad is left
    assert tri.tri_check_device_error(ws) == 0


@pytest.mark.parametrize("src,dst", [([0], [1]), ([0, 1], [1, 2]), ([0, 0], [0, 1]), ([1, 0], [0, 1])])
def test_fork_clamps_row_counts(src, dst):
    """A source's count past its pages' rows, or below 0, is clamped and
    flagged, and the clamped count is what the destination gets."""
    page, ppu = 4, 3
    for bad, good in ((ppu * page + 7, ppu * page), (-5, 0)):
        table = np.array([[0, 1, 2], [3, 4, -1], [5, -1, -1]], np.int32)
        t, c = _i32(table), _i32([1, 1, 1, 1, 1, 1, 0])
        n = np.array([bad, 6, 3], np.int32)
        pos = np.arange(3 * 10, dtype=np.int32).reshape(3, 10)
        ref = R.Pages(table, np.array([1, 1, 1, 1, 1, 1, 0], np.int32), np.array([good, 6, 3], np.int32), 3, page)
        want_pos = pos.copy()
        ref.fork(src, dst, want_pos)
        nd, ps = _i32(n), _i32(pos)
        ws = tri.workspace(tri.tri_pages_workspace_bytes(3, ppu, 7))
        tri.tri_pages_fork(t, c, page, 3, nd, _i32(src), _i32(dst), pos=ps, ws=ws)
        assert tri.tri_check_device_error(ws) == tri.FLAG_NVALID_RANGE
        assert np.array_equal(t.cpu().numpy(), ref.table) and np.array_equal(c.cpu().numpy(), ref.refs)
        assert np.array_equal(ps.cpu().numpy(), want_pos)
        for s in dst:
            assert nd[s].item() == ref.n_valid[s]


# One call of tri_pages_fit and one of each attention kernel through plain CUDA
# runtime calls, before and after the device's context is made anew.
_RESET = r"""
import ctypes, sys
import rope_aware_kv_b200 as tri
lib = tri.load()
P = ctypes.c_void_p
rt = ctypes.CDLL(sys.argv[1])

def buf(n):
    p = P()
    assert rt.cudaMalloc(ctypes.byref(p), ctypes.c_size_t(n)) == 0
    assert rt.cudaMemset(p, 0, ctypes.c_size_t(n)) == 0
    return p

def calls():
    big, small = [buf(1 << 20) for _ in range(4)], [buf(4096) for _ in range(4)]
    q, k, v, ws = big
    table, refs, n, out = small
    got = [lib.tri_pages_fit(k, v, tri.TRI_BF16, 1, 1, 128, table, 8, 1, 4, refs, n, None, 1, 0, None, ws, 1 << 20, None)]
    for rows in (8, 4):
        wb = lib.tri_decode_paged_workspace_bytes(1, 1)
        w = buf(wb)
        got.append(lib.tri_decode_attention_paged(q, k, v, tri.TRI_BF16, 1, 1, 1, -1, 1, 128, table, rows, 1, 4, n,
                                                  ctypes.c_float(0.1), out, None, w, wb, None))
    got.append(rt.cudaDeviceSynchronize())
    return got

print(calls())
assert rt.cudaDeviceReset() == 0
print(calls())
"""


def test_calls_after_a_device_reset():
    """A context made anew by cudaDeviceReset is followed (in a process of its
    own, through the C entry points)."""
    with open("/proc/self/maps") as f:
        runtime = next(x.split()[-1] for x in f if "libcudart" in x)
    r = subprocess.run([sys.executable, "-c", _RESET, runtime], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split("\n")[:2] == ["[0, 0, 0, 0]"] * 2, (r.stdout, r.stderr[-2000:])


@pytest.mark.parametrize("n_seq,per_seq,page,ppu,n_fork,seed", [
    (8, 6, 16, 40, 4, 0), (12, 5, 4, 300, 7, 1), (64, 8, 16, 130, 32, 2), (700, 2, 8, 30, 600, 3),
    (2048, 1, 8, 20, 1024, 4), (1024, 1, 4, 70, 1024, 5)])
def test_fork_of_sequences_that_are_only_read(n_seq, per_seq, page, ppu, n_fork, seed):
    """Forks none of whose destinations is another fork's source: repeated
    sources, emptied sequences, sequences that stay themselves, over several
    (layer, head) pairs and more columns than one job takes."""
    n_pages = n_seq * per_seq * ppu + 3
    cap = ppu * page - 1
    table, refs, nv = _state(n_seq, per_seq, page, ppu, n_pages, seed, high=cap)
    for u in range(len(nv)):  # rows whose pages are there
        nv[u] = min(int(nv[u]), page * int((table[u] >= 0).sum()), cap)
    rng = np.random.default_rng(seed + 70)
    order = rng.permutation(n_seq)
    only_read, dst = order[:n_seq - n_fork], order[n_seq - n_fork:].copy()
    if len(only_read):
        src = rng.choice(only_read, n_fork)
        src[0] = src[-1]
    else:  # every sequence is a destination: all stay themselves or are emptied
        src = dst.copy()
    src[rng.random(n_fork) < 0.15] = -1
    stays = rng.random(n_fork) < 0.2
    src[stays] = dst[stays]
    for f in range(n_fork):
        assert src[f] == dst[f] or dst[f] not in src
    assert len(set(dst.tolist())) == n_fork
    pos = rng.integers(0, 30000, (n_seq * per_seq, cap)).astype(np.int32)
    p_cur = rng.integers(0, 30000, n_seq).astype(np.int64)
    ref = R.Pages(table, refs, nv, n_seq, page)
    wpos, wcur = pos.copy(), p_cur.copy()
    assert ref.fork(src.tolist(), dst.tolist(), wpos, wcur) == 0
    ref.check()
    ws = tri.workspace(tri.tri_pages_workspace_bytes(*table.shape, n_pages))
    for _ in range(3):
        t, c, n, ps = _i32(table), _i32(refs), _i32(nv), _i32(pos)
        pc = torch.as_tensor(p_cur, device=DEV)
        tri.tri_pages_fork(t, c, page, n_seq, n, _i32(src), _i32(dst), pos=ps, p_cur=pc, ws=ws)
        assert tri.tri_check_device_error(ws) == 0
        assert np.array_equal(t.cpu().numpy(), ref.table) and np.array_equal(c.cpu().numpy(), ref.refs)
        assert np.array_equal(n.cpu().numpy(), ref.n_valid)
        assert np.array_equal(ps.cpu().numpy(), wpos) and np.array_equal(pc.cpu().numpy(), wcur)


def test_fork_1024_crossed():
    """The most forks of one call, every destination the next one's source."""
    n_seq, page, ppu = 1024, 4, 40
    n_pages = n_seq * ppu + 3
    table, refs, nv = _state(n_seq, 1, page, ppu, n_pages, 9, high=ppu * page)
    for u in range(n_seq):
        nv[u] = min(int(nv[u]), page * int((table[u] >= 0).sum()))
    dst = np.random.default_rng(1).permutation(n_seq)
    src = np.roll(dst, 1)
    ref = R.Pages(table, refs, nv, n_seq, page)
    assert ref.fork(src.tolist(), dst.tolist()) == 0
    t, c, n = _i32(table), _i32(refs), _i32(nv)
    ws = tri.workspace(tri.tri_pages_workspace_bytes(*table.shape, n_pages))
    tri.tri_pages_fork(t, c, page, n_seq, n, _i32(src), _i32(dst), ws=ws)
    assert tri.tri_check_device_error(ws) == 0
    assert np.array_equal(t.cpu().numpy(), ref.table) and np.array_equal(c.cpu().numpy(), ref.refs)
    assert np.array_equal(n.cpu().numpy(), ref.n_valid)
