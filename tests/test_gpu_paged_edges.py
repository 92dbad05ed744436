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
from tests.test_gpu_paged import BF16, DEV, F32, _cache, _check_decode, _i32, _rows, _state

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


def _exact_scores(n, G, page, dtype, seed):
    """One unit of n rows whose scores are whole numbers times 2^-8 in any
    order of summation; every 32 rows hold each head's largest score at their
    front, so the running maximum never changes and no weight is rescaled; and V has one
    row a dim, whose element is 1, so out[h, d] is one row's weight over the
    sum of all.  Returns q, k, v, table and the dims' rows."""
    rng = np.random.default_rng(seed)
    q = rng.choice([-2, -1, 1, 2], (G, R.D))
    kk = rng.integers(-2, 3, (n, R.D))
    tops = [j0 + h for j0 in range(0, n, 32) for h in range(G)]
    for j in tops:
        if j < n:
            kk[j] = 2 * np.sign(q[j % 32])
    s = kk @ q.T
    assert all(s[j0 + h, h] == s[:, h].max() for j0 in range(0, n, 32) for h in range(G)
               if j0 + h < n)
    rest = np.setdiff1d(np.arange(n), tops)
    dims = min(len(rest), R.D)
    at = np.sort(rng.choice(rest, dims, replace=False))
    k, v, table, _ = _cache([n], page, dtype, seed)
    for j in range(n):
        v[int(table[0, j // page]), j % page] = 0.0
        k[int(table[0, j // page]), j % page] = torch.as_tensor(kk[j], device=DEV).to(dtype)
    for d, j in enumerate(at):
        v[int(table[0, j // page]), j % page, d] = 1.0
    return torch.as_tensor(q[None], device=DEV).to(dtype), k, v, table, s, at


@pytest.mark.parametrize("dtype,page,n", [(BF16, 128, 128), (BF16, 8, 100), (BF16, 64, 640), (BF16, 128, 1280),
                                          (BF16, 20, 128), (BF16, 20, 640), (F32, 64, 128), (F32, 24, 1280)])
@pytest.mark.parametrize("G", [1, 7, 8])
def test_decode_weights_are_float32(dtype, page, n, G):
    """Each weight by itself.  With exact scores a weight over the sum is off by

      exp2: 2 ulp, at most 4 eps (eps = 2^-24, half an ulp's most);
      its argument x = s scale log2(e) - max, 0 >= x > -4: one rounding of at
        most 2^-23, times ln 2: 1.4 eps; log2(e) is off by 1.4e-8 of itself,
        times 4 ln 2: 0.7 eps;
      the split into three bf16 terms 2^-27, and the sum of the terms, the
        accumulator, the reciprocal and the product with it, a rounding each:
        4.2 eps;
      the sum of the weights: the same factor for every row of a head.

    So but for that factor at most 10.3 eps, and their root mean square no more.
    Weights in two terms of bf16, on the same scores, are off by three times
    that."""
    eps = 2.0 ** -24
    q, k, v, table, s, at = _exact_scores(n, G, page, dtype, 100 * G + n + page)
    scale = 2.0 ** -8
    x = (s - s.max(0)) * scale / np.log(2.0)
    assert x.min() > -4
    p = np.exp2(x)
    one = torch.as_tensor(p).bfloat16().double()
    two = one + (torch.as_tensor(p) - one).bfloat16().double()
    assert np.sqrt(((two.numpy() / p - 1)[at] ** 2).mean()) > 25 * eps
    want = (p / p.sum(0))[at].T
    out = tri.tri_decode_attention_paged(q, k, v, _i32(table), 1, 1, 1, _i32([n]), scale=scale)[0].double().cpu().numpy()
    dims = len(at)
    assert not out[:, dims:].any()
    rel = out[:, :dims] / want - 1
    own = rel - rel.mean(1, keepdims=True)
    # The factor: the weights' own bound twice (in the sum, and the mean of
    # these), and a rounding for each of at most n / 4 + 40 steps of a sum.
    assert np.abs(rel.mean(1)).max() <= (2 * 10.3 + n / 4 + 40) * eps
    assert np.abs(own).max() <= 2 * 10.3 * eps
    assert np.sqrt((own ** 2).mean()) <= 10.3 * eps


@pytest.mark.parametrize("dtype,page", [(BF16, 128), (BF16, 64), (BF16, 20), (F32, 64)])
@pytest.mark.parametrize("n", [3, 130, 1025, 9000])
def test_decode_error_next_to_plain_float32(dtype, page, n):
    """The relative error (Euclidean, over all units) is at most 4 times that of
    elementary float32 operations.  The kernels round no more often than those;
    a tensor-core sum that truncates errs to one side, 2 eps a step of 16
    products: 8 steps, 16 eps of a score's partial sums, where 128 roundings
    add up to sqrt(128) eps / sqrt(3) = 6.5 eps: 2.5 times; and likewise for the
    8 steps of a tile's values."""
    U, G = 6, 4
    k, v, table, _ = _cache([n] * U, page, dtype, n + page)
    q = (torch.randn((U, G, R.D), device=DEV, generator=torch.Generator(DEV).manual_seed(n)) * 2).to(dtype)
    out = tri.tri_decode_attention_paged(q, k, v, _i32(table), 1, 1, U, _i32([n] * U))
    assert not torch.backends.cuda.matmul.allow_tf32
    err, plain, size = 0.0, 0.0, 0.0
    for u in range(U):
        kr, vr = _rows(k, table, u, n), _rows(v, table, u, n)
        x = q[u].double() @ kr.double().T * R.D ** -0.5
        want = torch.softmax(x, 1) @ vr.double()
        y = (q[u].float() @ kr.float().T) * R.D ** -0.5
        w = torch.exp(y - y.amax(1, keepdim=True))
        ours = (w @ vr.float()) / w.sum(1, keepdim=True)
        err += ((out[u].double() - want) ** 2).sum().item()
        plain += ((ours.double() - want) ** 2).sum().item()
        size += (want ** 2).sum().item()
    assert err ** 0.5 <= 4 * plain ** 0.5, (err / size, plain / size)


@pytest.mark.parametrize("dtype,page", [(BF16, 128), (BF16, 20), (F32, 64)])
@pytest.mark.parametrize("n", [129, 400])
def test_decode_huge_values_without_weight(dtype, page, n):
    """Values of 1e38 in rows whose weight is 0 in float32, the last of them
    alone in its tile, leave nothing in the output."""
    G = 4
    k, v, table, _ = _cache([n], page, dtype, n)
    q = torch.randn((1, G, R.D), device=DEV, generator=torch.Generator(DEV).manual_seed(4)).to(dtype)
    away = -30.0 * q[0].float().sum(0)
    for x, j in enumerate((0, n // 2, n - 1)):
        k[int(table[0, j // page]), j % page] = away.to(dtype)
        v[int(table[0, j // page]), j % page] = (torch.full((R.D,), 1e38, device=DEV) * (-1) ** x).to(dtype)
    gone = (0, n // 2, n - 1)
    s = (q[0].double() @ _rows(k, table, 0, n).double().T * R.D ** -0.5).cpu().numpy()
    for j in gone:
        assert np.all(s[:, j] < s.max(1) - 110)  # exp(-110) < 2^-158, below float32's least 2^-149
    keep = [j for j in range(n) if j not in gone]
    lse = torch.zeros((1, G), device=DEV)
    out = tri.tri_decode_attention_paged(q, k, v, _i32(table), 1, 1, 1, _i32([n]), lse=lse)
    o, ls, to, tl = R.attention(q[0].double().cpu().numpy(), _rows(k, table, 0, n).double().cpu().numpy()[keep],
                                _rows(v, table, 0, n).double().cpu().numpy()[keep], float(np.float32(R.D ** -0.5)))
    assert np.all(np.abs(out[0].double().cpu().numpy() - o) <= to)
    assert np.all(np.abs(lse[0].double().cpu().numpy() - ls) <= tl)


def _many_units(kind):
    rng = np.random.default_rng(7)
    if kind == "0 or 1":
        return np.repeat(rng.integers(0, 2, 52), 8)
    if kind == "one in 40":
        return np.where(rng.random(2000) < 1 / 40, rng.integers(1, 33, 2000), 0)
    if kind == "short":
        return rng.integers(0, 41, 6000)
    n = np.where(rng.random(3000) < 1 / 15, rng.integers(1, 300, 3000), 0)
    n[[0, 40, 41, 700, 2999]] = [900, 0, 33, 1300, 64]
    return n


@pytest.mark.parametrize("dtype,page", [(F32, 32), (F32, 24), (BF16, 20), (BF16, 128)])
@pytest.mark.parametrize("kind", ["0 or 1", "one in 40", "short", "gaps"])
def test_decode_ranges_of_many_units(kind, dtype, page):
    """A CTA's range that spans more units than a warp looks at at once: many
    short ones, or long stretches of units without a row."""
    n = _many_units(kind).astype(np.int32)
    k, v, table, _ = _cache(n, page, dtype, 3)
    q = torch.randn((len(n), 3, R.D), device=DEV, generator=torch.Generator(DEV).manual_seed(5)).to(dtype)
    _check_decode(q, k, v, table, n, 1, 1, len(n))
