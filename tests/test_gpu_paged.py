"""Paged-cache operators through the C ABI: decode attention, append and the
page calls, against float64 attention and sequential tables (paged_ref).

Rows that no call may read (past n_valid, free pages) hold NaN, so a masked
row that leaks shows; keys at the first and last row and at page and tile
borders are turned towards the query, so a row that is missed shows.  The
tolerances of the attention are derived in paged_ref.attention."""
import ctypes

import numpy as np
import pytest
import torch

import rope_aware_kv_b200 as tri
from rope_aware_kv_b200 import build as tri_build
from tests import paged_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tri_build.build()
    tri.load()
    yield
    torch.cuda.empty_cache()


def _cache(rows_of, page, dtype, seed, ppu=None, spare=3, fill=float("nan")):
    """A cache with the given rows of each unit, pages scattered over a pool
    whose other rows hold `fill`; also the units' rows in float64."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    U = len(rows_of)
    held = [-(-n // page) for n in rows_of]
    ppu = ppu or max(1, max(held))
    n_pages = sum(held) + spare
    perm = rng.permutation(n_pages)
    table = np.full((U, ppu), -1, np.int32)
    refs = np.zeros(n_pages, np.int32)
    k = torch.full((n_pages, page, R.D), fill, dtype=dtype, device=DEV)
    v = torch.full((n_pages, page, R.D), fill, dtype=dtype, device=DEV)
    x = 0
    for u, n in enumerate(rows_of):
        for s in range(held[u]):
            p = int(perm[x])
            x += 1
            table[u, s], refs[p] = p, 1
            r = min(page, n - s * page)
            k[p, :r] = torch.randn((r, R.D), generator=g, device=DEV).to(dtype)
            v[p, :r] = torch.randn((r, R.D), generator=g, device=DEV).to(dtype)
    return k, v, table, refs


def _rows(pool, table, u, n):
    page = pool.shape[1]
    p = torch.as_tensor(table[u, :-(-n // page)].astype(np.int64), device=DEV)
    return pool.index_select(0, p).flatten(0, 1)[:n]


def _i32(x):
    return torch.as_tensor(np.asarray(x, np.int32), device=DEV)


def _check_decode(q, k, v, table, rows_of, n_seq, L, H, layer=-1, scale=None, **kw):
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    ws = kw.pop("ws", None)
    if ws is None:
        ws = tri.workspace(tri.tri_decode_paged_workspace_bytes(q.shape[0], q.shape[1]))
    out = tri.tri_decode_attention_paged(q, k, v, _i32(table), n_seq, L, H, _i32(rows_of),
                                         layer=layer, scale=scale, lse=lse, ws=ws, **kw)
    assert tri.tri_check_device_error(ws) == 0
    out_h, lse_h = out.double().cpu().numpy(), lse.double().cpu().numpy()
    sc = float(np.float32(R.D ** -0.5 if scale is None else scale))
    for i, u in enumerate(R.unit_list(n_seq, L, H, layer)):
        n = int(rows_of[u])
        o, ls, to, tl = R.attention(q[i].double().cpu().numpy(),
                                    _rows(k, table, u, n).double().cpu().numpy(),
                                    _rows(v, table, u, n).double().cpu().numpy(), sc)
        if n == 0:
            assert not out_h[i].any() and np.all(lse_h[i] == -np.inf)
            continue
        assert np.all(np.abs(out_h[i] - o) <= to), (u, n, np.max(np.abs(out_h[i] - o) / to))
        assert np.all(np.abs(lse_h[i] - ls) <= tl), (u, n, np.max(np.abs(lse_h[i] - ls) / tl))
    return out


def _spike(q, k, table, rows_of, units, page):
    """Turn the keys at borders towards their unit's queries."""
    for i, u in enumerate(units):
        n = int(rows_of[u])
        G = q.shape[1]
        for x, j in enumerate(sorted({0, n - 1, page - 1, page, 127, 128, 31, 32, n // 2})):
            if 0 <= j < n:
                k[int(table[u, j // page]), j % page] = (q[i, x % G].float() * 0.8).to(k.dtype)


LENGTHS = [1, 2, 31, 32, 33, 63, 127, 128, 129, 255, 257, 700, 0, 1025, 3]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("G,page", [(1, 128), (2, 8), (3, 64), (4, 16), (5, 1), (6, 24), (7, 32), (8, 100), (8, 128),
                                    (7, 256), (4, 640), (8, 13)])
def test_decode_parity(dtype, G, page):
    """Every group size; pages of one row, odd ones, ones that end inside a
    tile and ones larger than it; lengths around the tile borders and 0."""
    n_seq, L, H = 5, 1, 3
    rows_of = LENGTHS
    k, v, table, _ = _cache(rows_of, page, dtype, G * 1000 + page)
    q = torch.randn((15, G, R.D), device=DEV, generator=torch.Generator(DEV).manual_seed(page)).to(dtype)
    _spike(q, k, table, rows_of, range(15), page)
    _check_decode(q, k, v, table, rows_of, n_seq, L, H)
    _check_decode(q, k, v, table, rows_of, n_seq, L, H, scale=0.3)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows_of,page", [([9000], 128), ([40000, 1], 64), ([1, 20011], 24), ([0, 0], 128),
                                          ([1], 128), ([5, 0, 30000, 64], 32)])
def test_decode_split_long(dtype, rows_of, page):
    """Few units, so one is split over many CTAs and joined."""
    k, v, table, _ = _cache(rows_of, page, dtype, sum(rows_of))
    q = torch.randn((len(rows_of), 4, R.D), device=DEV, generator=torch.Generator(DEV).manual_seed(3)).to(dtype)
    _spike(q, k, table, rows_of, range(len(rows_of)), page)
    a = _check_decode(q, k, v, table, rows_of, 1, 1, len(rows_of))
    b = _check_decode(q, k, v, table, rows_of, 1, 1, len(rows_of))
    assert torch.equal(a, b)


@pytest.mark.parametrize("page", [128, 12])
def test_decode_many_units_and_layers(page):
    """More units than CTAs, and one layer of several."""
    n_seq, L, H, G = 40, 3, 5, 2
    rng = np.random.default_rng(5)
    rows_of = rng.integers(0, 160, n_seq * L * H).astype(np.int32)
    k, v, table, _ = _cache(rows_of, page, BF16, 12, ppu=-(-160 // page) + 2)
    g = torch.Generator(DEV).manual_seed(3)
    q = torch.randn((n_seq * L * H, G, R.D), device=DEV, generator=g).to(BF16)
    whole = _check_decode(q, k, v, table, rows_of, n_seq, L, H)
    for layer in range(L):
        units = R.unit_list(n_seq, L, H, layer)
        part = _check_decode(q[units].contiguous(), k, v, table, rows_of, n_seq, L, H, layer=layer)
        err = (part - whole[units]).abs().max().item()
        assert err <= 1e-4


@pytest.mark.parametrize("dtype,page", [(BF16, 128), (BF16, 20), (F32, 64)])
def test_decode_masked_values_and_extremes(dtype, page):
    """Rows past n_valid hold infinities; scores reach far below and above
    the others; a value row of the largest numbers carries no weight that a
    rounding could give it."""
    rows_of = [130, 1, 400]
    k, v, table, _ = _cache(rows_of, page, dtype, 5, fill=float("inf"))
    q = torch.randn((3, 4, R.D), device=DEV, generator=torch.Generator(DEV).manual_seed(4)).to(dtype)
    for u, n in enumerate(rows_of):
        for j, f in ((0, -30.0), (n // 2, 12.0), (n - 1, 11.5)):
            k[int(table[u, j // page]), j % page] = (q[u, 1].float() * f).to(dtype)
    _check_decode(q, k, v, table, rows_of, 1, 1, 3)


@pytest.mark.parametrize("dtype,page", [(BF16, 128), (BF16, 20), (F32, 64)])
def test_decode_missing_pages_and_bad_counts(dtype, page):
    """A page that is not in the pool carries no weight and is flagged; counts
    out of range are clamped and flagged."""
    n = 3 * page + 5
    k, v, table, _ = _cache([n, n, n], page, dtype, 8, ppu=4)
    q = torch.randn((3, 3, R.D), device=DEV, generator=torch.Generator(DEV).manual_seed(4)).to(dtype)
    holed = table.copy()
    holed[0, 1], holed[1, 3], holed[2, 0] = -1, len(k) + 7, -5
    ws = tri.workspace(tri.tri_decode_paged_workspace_bytes(3, 3))
    out = tri.tri_decode_attention_paged(q, k, v, _i32(holed), 1, 1, 3, _i32([n, n, n]), ws=ws)
    assert tri.tri_check_device_error(ws) == tri.FLAG_INDEX_RANGE
    for u, gone in ((0, 1), (1, 3), (2, 0)):
        keep = [j for j in range(n) if j // page != gone]
        o, _, to, _ = R.attention(q[u].double().cpu().numpy(),
                                  _rows(k, table, u, n).double().cpu().numpy()[keep],
                                  _rows(v, table, u, n).double().cpu().numpy()[keep], float(np.float32(R.D ** -0.5)))
        assert np.all(np.abs(out[u].double().cpu().numpy() - o) <= to)
    # every page missing: as a unit without rows
    lse = torch.zeros((3, 3), device=DEV)
    out = tri.tri_decode_attention_paged(q, k, v, torch.full_like(_i32(holed), -1), 1, 1, 3, _i32([n, 1, n]), ws=ws,
                                         lse=lse)
    assert tri.tri_check_device_error(ws) == tri.FLAG_INDEX_RANGE
    assert not out.any() and torch.all(lse == -torch.inf)
    full = [4 * page] * 3
    k2, v2, t2, _ = _cache(full, page, dtype, 9)
    a = tri.tri_decode_attention_paged(q, k2, v2, _i32(t2), 1, 1, 3, _i32([4 * page, 4 * page + 9, -3]), ws=ws)
    assert tri.tri_check_device_error(ws) == tri.FLAG_NVALID_RANGE
    b = tri.tri_decode_attention_paged(q, k2, v2, _i32(t2), 1, 1, 3, _i32([4 * page, 4 * page, 0]), ws=ws)
    assert torch.equal(a, b)


def test_decode_equals_contiguous_call():
    """On a cache whose pages lie in order the paged call agrees with
    tri_decode_attention."""
    U, G, cap = 6, 7, 1000
    g = torch.Generator(DEV).manual_seed(1)
    q = torch.randn((U, G, R.D), device=DEV, generator=g).to(BF16)
    k = torch.randn((U, cap, R.D), device=DEV, generator=g).to(BF16)
    v = torch.randn((U, cap, R.D), device=DEV, generator=g).to(BF16)
    nv = _i32([1000, 0, 1, 999, 257, 500])
    table = torch.arange(U * 10, dtype=torch.int32, device=DEV).view(U, 10)
    a = tri.tri_decode_attention(q, k, v, n_valid=nv)
    b = tri.tri_decode_attention_paged(q, k.view(U * 10, 100, R.D), v.view(U * 10, 100, R.D), table, 1, 1, U, nv)
    assert (a - b).abs().max().item() <= 1e-4


def test_decode_graph_streams_and_shared_workspace():
    """Captured and replayed with other contents; two captured calls on one
    workspace; a call on another stream without a workspace of its own."""
    rows_of = [300, 0, 1025, 77]
    k, v, table, _ = _cache(rows_of, 64, BF16, 2)
    t, nv = _i32(table), _i32(rows_of)
    g = torch.Generator(DEV).manual_seed(1)
    q = torch.randn((4, 4, R.D), device=DEV, generator=g).to(BF16)
    want = tri.tri_decode_attention_paged(q, k, v, t, 2, 1, 2, nv)
    nv2 = _i32([5, 300, 1000, 0])
    t2 = t[[3, 0, 2, 1]].contiguous()
    want2 = tri.tri_decode_attention_paged(q, k, v, t2, 2, 1, 2, nv2.clone().clamp_(max=64))
    ws = tri.workspace(tri.tri_decode_paged_workspace_bytes(4, 4))
    qs, ts, ns = q.clone(), t.clone(), nv.clone()
    o1, o2 = torch.empty_like(want), torch.empty_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tri.tri_decode_attention_paged(qs, k, v, ts, 2, 1, 2, ns, out=o1, ws=ws)
        tri.tri_decode_attention_paged(qs, k, v, t, 2, 1, 2, nv, out=o2, ws=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o1, want) and torch.equal(o2, want)
    ts.copy_(t2)
    ns.copy_(nv2.clamp(max=64))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o1, want2) and torch.equal(o2, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [tri.tri_decode_attention_paged(q, k, v, t, 2, 1, 2, nv, stream=side) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("dtype,page", [(BF16, 128), (BF16, 20), (F32, 64)])
def test_decode_infinite_value_rows(dtype, page):
    """An infinite value in a row of the cache makes that dim infinite in every
    head that gives the row weight, and no other dim."""
    n = 300
    k, v, table, _ = _cache([n], page, dtype, 6)
    q = torch.randn((1, 5, R.D), device=DEV, generator=torch.Generator(DEV).manual_seed(4)).to(dtype)
    for j, d, x in ((0, 3, float("inf")), (150, 64, float("-inf")), (299, 127, float("inf"))):
        v[int(table[0, j // page]), j % page, d] = x
    out = tri.tri_decode_attention_paged(q, k, v, _i32(table), 1, 1, 1, _i32([n]))[0]
    assert torch.all(out[:, [3, 127]] == float("inf")) and torch.all(out[:, 64] == float("-inf"))
    rest = [d for d in range(R.D) if d not in (3, 64, 127)]
    o, _, to, _ = R.attention(q[0].double().cpu().numpy(), _rows(k, table, 0, n).double().cpu().numpy(),
                              _rows(v, table, 0, n).double().cpu().numpy()[:, rest], float(np.float32(R.D ** -0.5)), rest)
    assert np.all(np.abs(out[:, rest].double().cpu().numpy() - o) <= to)


@pytest.mark.parametrize("page", [64, 20])
def test_far_rows(page):
    """Rows whose elements lie past 2^31: attention, append, fit's copies and
    compaction at the far end of a pool of 4.6 GB."""
    n_pages = 18_000_000 // page
    k = torch.empty((n_pages, page, R.D), dtype=BF16, device=DEV)
    v = torch.empty_like(k)
    n = 3 * page + 7
    table = np.array([[n_pages - 1, n_pages - 5, 2, n_pages - 2, -1], [0, n_pages - 3, 1, n_pages - 4, -1]], np.int32)
    g = torch.Generator(DEV).manual_seed(3)
    for p in table[table >= 0]:
        k[int(p)] = torch.randn((page, R.D), device=DEV, generator=g).to(BF16)
        v[int(p)] = torch.randn((page, R.D), device=DEV, generator=g).to(BF16)
    q = torch.randn((2, 4, R.D), device=DEV, generator=g).to(BF16)
    _check_decode(q, k, v, table, [n, n - 1], 1, 1, 2)
    # a third unit shares the first one's pages and gets copies of them
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    t = _i32(np.concatenate([table, table[:1]]))
    refs.index_add_(0, t[t >= 0].long(), torch.ones(int((t >= 0).sum()), dtype=torch.int32, device=DEV))
    refs[3:n_pages - 9] += (refs[3:n_pages - 9] == 0).int()  # only a few pages at each end are free
    nv = _i32([n, n - 1, n])
    free = tri.tri_pages_fit(k, v, t, refs, 3, nv, own=True)
    assert free.item() == 4 - 4 and int(t[0].max()) == n_pages - 6  # the far free pages, lowest first
    th = t.cpu().numpy()
    for u in (0, 2):
        assert torch.equal(_rows(k, th, 0, n), _rows(k, th, 2, n)) and torch.equal(_rows(v, th, 0, n), _rows(v, th, 2, n))
    _check_decode(q, k, v, th[:2], [n, n - 1], 1, 1, 2)
    kn = torch.randn((3, 2, R.D), device=DEV, generator=g).to(BF16)
    want = [torch.cat([_rows(k, th, u, int(m)), kn[u]]) for u, m in enumerate([n, n - 1, n])]
    tri.tri_append_paged(k, v, None, t, 3, 1, 1, nv, kn, kn, None, page_refs=refs)
    assert nv.cpu().tolist() == [n + 2, n + 1, n + 2]
    for u, m in enumerate([n + 2, n + 1, n + 2]):
        assert torch.equal(_rows(k, th, u, m), want[u])
    # most of the pool is freed, and what is left moves to its front
    refs[3:n_pages - 9] = 0
    refs.zero_().index_add_(0, t[t >= 0].long(), torch.ones(int((t >= 0).sum()), dtype=torch.int32, device=DEV))
    live = tri.tri_pages_compact(k, v, t, refs)
    assert live.item() == 12 and int(t.max()) == 11
    for u, m in enumerate([n + 2, n + 1, n + 2]):
        assert torch.equal(_rows(k, t.cpu().numpy(), u, m), want[u])
    _check_decode(q, k, v, t.cpu().numpy()[:2], [n + 2, n + 1], 1, 1, 2)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def _pool_with_pages(n_valid, room, page, dtype, seed, ppu):
    """Pages for n_valid + room rows of each unit; every row of the pool random."""
    k, v, table, refs = _cache([n + r for n, r in zip(n_valid, room)], page, dtype, seed, ppu=ppu, fill=0.5)
    return k, v, table, refs


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page,n_new,layer", [(128, 1, -1), (16, 1, 1), (1, 5, -1), (24, 8, 0), (32, 9, -1),
                                              (100, 300, 1), (7, 65, -1)])
def test_append_rows(dtype, page, n_new, layer):
    """Rows, positions, counts and p_cur; every other byte stays."""
    n_seq, L, H, cap = 4, 2, 3, 700
    U = n_seq * L * H
    rng = np.random.default_rng(page + n_new)
    nv = rng.integers(0, 300, U).astype(np.int32)
    nv[0], nv[1] = 0, page
    add = rng.integers(0, n_new + 1, n_seq).astype(np.int32)
    add[0], add[-1] = n_new, 0
    per = L * H
    ppu = -(-cap // page)
    k, v, table, refs = _pool_with_pages(nv, [int(add[u // per]) for u in range(U)], page, dtype, 5, ppu)
    pos = torch.randint(0, 100, (U, cap), dtype=torch.int32, device=DEV)
    units = R.unit_list(n_seq, L, H, layer)
    g = torch.Generator(DEV).manual_seed(9)
    kn = torch.randn((len(units), n_new, R.D), device=DEV, generator=g).to(dtype)
    vn = torch.randn((len(units), n_new, R.D), device=DEV, generator=g).to(dtype)
    pn = torch.randint(1000, 9000, (len(units), n_new), dtype=torch.int32, device=DEV)
    p_cur = torch.tensor([3, 8999, 100000, 5], dtype=torch.int64, device=DEV)
    want_k, want_v, want_pos, want_n, want_c = k.clone(), v.clone(), pos.clone(), nv.copy(), p_cur.cpu().numpy()
    for i, u in enumerate(units):
        s = u // per
        for x in range(int(add[s])):
            j = int(nv[u]) + x
            want_k[int(table[u, j // page]), j % page] = kn[i, x]
            want_v[int(table[u, j // page]), j % page] = vn[i, x]
            want_pos[u, j] = pn[i, x]
            want_c[s] = max(want_c[s], int(pn[i, x]) + 1)
        want_n[u] += add[s]
    n = _i32(nv)
    ws = tri.workspace(tri.tri_append_paged_workspace_bytes(len(units)))
    tri.tri_append_paged(k, v, pos, _i32(table), n_seq, L, H, n, kn, vn, pn, layer=layer, n_add=_i32(add),
                         page_refs=_i32(refs), p_cur=p_cur, ws=ws)
    assert tri.tri_check_device_error(ws) == 0
    assert torch.equal(k, want_k) and torch.equal(v, want_v) and torch.equal(pos, want_pos)
    assert np.array_equal(n.cpu().numpy(), want_n) and np.array_equal(p_cur.cpu().numpy(), want_c)


@pytest.mark.parametrize("n_new", [2, 40])
def test_append_refuses_units(n_new):
    """Units whose rows do not fit, whose page is missing or shared, stay as
    they are; the others are appended."""
    page, cap, U = 16, 128, 5
    nv = np.array([20, 100, 20, 20, 20], np.int32)
    nv[1] = cap - n_new + 1
    k, v, table, refs = _pool_with_pages(nv, [n_new] * U, page, BF16, 5, 12)
    table[2, (20 + n_new - 1) // page] = -1
    refs[table[3, 20 // page]] = 2
    k0, v0, n = k.clone(), v.clone(), _i32(nv)
    kn = torch.randn((U, n_new, R.D), device=DEV).to(BF16)
    ws = tri.workspace(tri.tri_append_paged_workspace_bytes(U))
    pos = torch.zeros((U, cap), dtype=torch.int32, device=DEV)
    pn = torch.ones((U, n_new), dtype=torch.int32, device=DEV)
    tri.tri_append_paged(k, v, pos, _i32(table), 1, 1, U, n, kn, kn, pn, page_refs=_i32(refs), ws=ws)
    assert tri.tri_check_device_error(ws) == (tri.FLAG_NVALID_RANGE | tri.FLAG_INDEX_RANGE | tri.FLAG_SHARED_PAGE)
    grown = [True, False, False, False, True]
    assert n.cpu().tolist() == [int(x) + n_new * y for x, y in zip(nv, grown)]
    for u in (0, 4):
        for x in range(n_new):
            j = int(nv[u]) + x
            k0[int(table[u, j // page]), j % page] = kn[u, x]
            v0[int(table[u, j // page]), j % page] = kn[u, x]
    assert torch.equal(k, k0) and torch.equal(v, v0)
    assert pos.sum().item() == 2 * n_new
    # keys only, no positions, nothing to add
    tri.tri_append_paged(k, None, None, _i32(table), 1, 1, U, n, kn[:, :0].contiguous(), None, None, ws=ws)
    assert tri.tri_check_device_error(ws) == 0 and torch.equal(k, k0)


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------

def _state(n_seq, per_seq, page, ppu, n_pages, seed, low=0, high=None):
    """Random tables: some units share pages, some hold more than their rows
    need, some less."""
    rng = np.random.default_rng(seed)
    U = n_seq * per_seq
    table = np.full((U, ppu), -1, np.int32)
    refs = np.zeros(n_pages, np.int32)
    nv = rng.integers(low, (high or ppu * page) + 1, U).astype(np.int32)
    free = list(rng.permutation(n_pages))
    for u in range(U):
        held = -(-int(nv[u]) // page) + int(rng.integers(-1, 3))
        for s in range(max(0, min(ppu, held))):
            if rng.random() < 0.4 and u:
                p = table[int(rng.integers(0, u)), s]  # the same slot of an earlier unit
                if p >= 0:
                    table[u, s] = p
                    refs[p] += 1
                    continue
            if not free:
                break
            p = int(free.pop())
            table[u, s] = p
            refs[p] = 1
    return table, refs, nv


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("n_seq,per_seq,page,ppu,n_pages,dtype", [
    (1, 1, 16, 1, 1, BF16), (3, 2, 16, 5, 80, BF16), (4, 6, 128, 4, 260, F32), (7, 11, 3, 40, 6000, BF16),
    (2, 1, 1, 9, 60, F32), (16, 20, 8, 12, 9000, BF16)])
def test_fit(own, n_seq, per_seq, page, ppu, n_pages, dtype):
    for seed in range(3):
        table, refs, nv = _state(n_seq, per_seq, page, ppu, n_pages, seed, high=(ppu - 1) * page)
        rng = np.random.default_rng(seed)
        add = rng.integers(0, page + 1, n_seq).astype(np.int32)
        if n_pages == 1:
            nv[:], add[:] = 0, 1
        ref = R.Pages(table, refs, nv, n_seq, page)
        n_free = ref.fit([int(x) for x in add], own)
        assert n_free >= 0
        ref.check()
        k = torch.randn((n_pages, page, R.D), device=DEV).to(dtype)
        v = torch.randn((n_pages, page, R.D), device=DEV).to(dtype)
        wk, wv = k.clone(), v.clone()
        for a, b, r in ref.copied:
            wk[b, :r], wv[b, :r] = k[a, :r], v[a, :r]
        t, c = _i32(table), _i32(refs)
        ws = tri.workspace(tri.tri_pages_workspace_bytes(*table.shape, n_pages))
        got = tri.tri_pages_fit(k, v, t, c, n_seq, _i32(nv), n_new=page, n_add=_i32(add), own=own, ws=ws)
        assert tri.tri_check_device_error(ws) == 0
        assert np.array_equal(t.cpu().numpy(), ref.table) and np.array_equal(c.cpu().numpy(), ref.refs)
        assert got.item() == n_free
        assert torch.equal(k, wk) and torch.equal(v, wv)
        # once more with nothing to add: gives back what was taken for rows to come, copies nothing
        ref.copied = []
        n_free = ref.fit([0] * n_seq)
        got = tri.tri_pages_fit(k, None, t, c, n_seq, _i32(nv))
        assert np.array_equal(t.cpu().numpy(), ref.table) and np.array_equal(c.cpu().numpy(), ref.refs)
        assert got.item() == n_free and torch.equal(k, wk) and not ref.copied


def test_fit_short_pool_and_bad_entries():
    """Nothing is taken from a pool that is too small, but what is not needed
    is given back; entries and counts out of range are flagged."""
    page, n_pages = 8, 6
    table = np.array([[0, 1, 2], [3, -1, -1]], np.int32)
    refs = np.array([1, 1, 1, 1, 0, 0], np.int32)
    nv = [9, 8]
    k = torch.randn((n_pages, page, R.D), device=DEV).to(BF16)
    k0 = k.clone()
    t, c = _i32(table), _i32(refs)
    ws = tri.workspace(tri.tri_pages_workspace_bytes(2, 3, n_pages))
    got = tri.tri_pages_fit(k, None, t, c, 2, _i32(nv), n_new=15, n_add=_i32([15, 15]), ws=ws)  # wants 0 + 2 of 2
    assert got.item() == 0 and tri.tri_check_device_error(ws) == 0
    assert t.cpu().tolist() == [[0, 1, 2], [3, 4, 5]]
    t, c = _i32(np.array([[0, 1, 2], [3, -1, -1], [-1, -1, -1]])), _i32(refs)
    ws = tri.workspace(tri.tri_pages_workspace_bytes(3, 3, n_pages))
    got = tri.tri_pages_fit(k, None, t, c, 3, _i32([9, 8, 0]), n_new=16, n_add=_i32([0, 16, 16]), ws=ws)
    assert got.item() == -1 and tri.tri_check_device_error(ws) == tri.FLAG_NO_PAGES
    assert t.cpu().tolist() == [[0, 1, -1], [3, -1, -1], [-1, -1, -1]]
    assert c.cpu().tolist() == [1, 1, 0, 1, 0, 0]
    t = _i32(np.array([[0, 77, -1], [3, -9, -1], [-1, -1, -1]]))
    c = _i32([1, 0, 0, 1, 0, 0])
    tri.tri_pages_fit(k, None, t, c, 3, _i32([9, 8, 99]), n_add=_i32([0, 0, 4]), n_new=3, ws=ws)
    assert tri.tri_check_device_error(ws) == tri.FLAG_INDEX_RANGE | tri.FLAG_NVALID_RANGE
    assert t.cpu().tolist() == [[0, 1, -1], [3, -1, -1], [2, 4, 5]]
    assert torch.equal(k, k0)


@pytest.mark.parametrize("n_seq,per_seq,page,ppu,n_fork", [(1, 1, 16, 1, 1), (4, 6, 16, 5, 4), (6, 2, 3, 50, 6),
                                                         (9, 112, 128, 3, 5), (300, 1, 4, 40, 300)])
def test_fork(n_seq, per_seq, page, ppu, n_fork):
    """Permutations, repeated sources, emptied sequences, repeated and bad
    indices; sources that are also destinations."""
    n_pages = n_seq * per_seq * ppu + 3
    cap = ppu * page - (page > 2)
    for seed in range(4):
        table, refs, nv = _state(n_seq, per_seq, page, ppu, n_pages, seed, high=cap)
        for u in range(len(nv)):  # rows whose pages are there
            nv[u] = min(int(nv[u]), page * int((table[u] >= 0).sum()), cap)
        rng = np.random.default_rng(seed + 50)
        dst = rng.permutation(n_seq)[:n_fork]
        src = rng.integers(-1, n_seq, n_fork)
        if seed == 1:
            src = np.roll(dst, 1)
        if seed == 3 and n_fork > 2:
            dst[1], src[2], dst[0] = dst[2], n_seq, dst[0]
        pos = rng.integers(0, 30000, (n_seq * per_seq, cap)).astype(np.int32)
        p_cur = rng.integers(0, 30000, n_seq).astype(np.int64)
        ref = R.Pages(table, refs, nv, n_seq, page)
        wpos, wcur = pos.copy(), p_cur.copy()
        skipped = ref.fork(src.tolist(), dst.tolist(), wpos, wcur)
        ref.check()
        t, c, n, ps = _i32(table), _i32(refs), _i32(nv), _i32(pos)
        pc = torch.as_tensor(p_cur, device=DEV)
        ws = tri.workspace(tri.tri_pages_workspace_bytes(*table.shape, n_pages))
        tri.tri_pages_fork(t, c, page, n_seq, n, _i32(src), _i32(dst), pos=ps, p_cur=pc, ws=ws)
        assert tri.tri_check_device_error(ws) == (tri.FLAG_INDEX_RANGE if skipped else 0)
        assert np.array_equal(t.cpu().numpy(), ref.table) and np.array_equal(c.cpu().numpy(), ref.refs)
        assert np.array_equal(n.cpu().numpy(), ref.n_valid)
        assert np.array_equal(ps.cpu().numpy(), wpos) and np.array_equal(pc.cpu().numpy(), wcur)


@pytest.mark.parametrize("U,page,ppu,n_pages,dtype", [(1, 16, 1, 1, BF16), (5, 16, 6, 100, BF16), (40, 3, 30, 4000, F32),
                                                    (6, 128, 4, 31, BF16), (1, 8, 2, 5000, BF16)])
def test_compact(U, page, ppu, n_pages, dtype):
    for seed in range(3):
        table, refs, nv = _state(1, U, page, ppu, n_pages, seed)
        ref = R.Pages(table, refs, nv, 1, page)
        live = ref.compact()
        ref.check()
        k = torch.randn((n_pages, page, R.D), device=DEV).to(dtype)
        v = torch.randn((n_pages, page, R.D), device=DEV).to(dtype)
        wk, wv = k.clone(), v.clone()
        for a, b, _ in ref.copied:
            wk[b], wv[b] = k[a], v[a]
        t, c = _i32(table), _i32(refs)
        ws = tri.workspace(tri.tri_pages_workspace_bytes(*table.shape, n_pages))
        got = tri.tri_pages_compact(k, v, t, c, ws=ws)
        assert tri.tri_check_device_error(ws) == 0
        assert got.item() == live
        assert np.array_equal(t.cpu().numpy(), ref.table) and np.array_equal(c.cpu().numpy(), ref.refs)
        assert torch.equal(k, wk) and torch.equal(v, wv)
        assert tri.tri_pages_compact(k, None, t, c).item() == live  # nothing left to move
        assert np.array_equal(t.cpu().numpy(), ref.table) and torch.equal(k, wk)


def test_fit_same_page_twice_in_a_unit():
    """A page named by two slots of one unit, and by all slots of another."""
    table = np.array([[0, 0, 1], [2, 2, 2]], np.int32)
    refs = np.array([2, 1, 3, 0, 0, 0, 0], np.int32)
    nv = np.array([11, 12], np.int32)
    ref = R.Pages(table, refs, nv, 2, 4)
    n_free = ref.fit([0, 0], own=True)
    ref.check()
    k = torch.randn((7, 4, R.D), device=DEV)
    wk = k.clone()
    for a, b, r in ref.copied:
        wk[b, :r] = k[a, :r]
    t, c = _i32(table), _i32(refs)
    assert tri.tri_pages_fit(k, None, t, c, 2, _i32(nv), own=True).item() == n_free == 1
    assert np.array_equal(t.cpu().numpy(), ref.table) and np.array_equal(c.cpu().numpy(), ref.refs)
    assert torch.equal(k, wk)


@pytest.mark.parametrize("n_new", [3, 30])
def test_append_counts_out_of_range(n_new):
    """n_add above n_new appends n_new rows, below 0 none; both are flagged."""
    k, v, table, refs = _cache([100, 100, 100], 32, F32, 3, fill=0.0)
    nv = _i32([10, 20, 30])
    kn = torch.randn((3, n_new, R.D), device=DEV)
    ws = tri.workspace(tri.tri_append_paged_workspace_bytes(3))
    tri.tri_append_paged(k, v, None, _i32(table), 3, 1, 1, nv, kn, kn, None, n_add=_i32([n_new + 5, -2, 1]),
                         page_refs=_i32(refs), ws=ws)
    assert tri.tri_check_device_error(ws) == tri.FLAG_NVALID_RANGE
    assert nv.cpu().tolist() == [10 + n_new, 20, 31]
    assert torch.equal(_rows(k, table, 0, 10 + n_new)[10:], kn[0]) and torch.equal(_rows(v, table, 2, 31)[30:], kn[2, :1])


def test_page_calls_captured():
    """fit, append, attention, fork and compact of one step in a graph, on one
    workspace and a side stream, replayed from two states: what the calls
    give one by one."""
    n_seq, L, H, page, ppu, n_pages = 4, 2, 2, 16, 8, 200
    per, U = L * H, n_seq * L * H
    states = [_state(n_seq, per, page, ppu, n_pages, seed, high=100) for seed in (1, 2)]
    g = torch.Generator(DEV).manual_seed(5)
    kn = torch.randn((U, 1, R.D), device=DEV, generator=g).to(BF16)
    q = torch.randn((U, 2, R.D), device=DEV, generator=g).to(BF16)
    k0 = torch.randn((n_pages, page, R.D), device=DEV, generator=g).to(BF16)
    src, dst = _i32([0, 1, -1]), _i32([1, 0, 3])
    k, v = k0.clone(), k0.clone()
    t, c, nv = _i32(states[0][0]), _i32(states[0][1]), _i32(states[0][2])
    out = torch.zeros((U, 2, R.D), device=DEV)
    n_free, n_live = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = tri.workspace(max(tri.tri_pages_workspace_bytes(U, ppu, n_pages), tri.tri_append_paged_workspace_bytes(U),
                           tri.tri_decode_paged_workspace_bytes(U, 2)))

    def step():
        tri.tri_pages_fit(k, v, t, c, n_seq, nv, n_new=1, n_free=n_free, ws=ws)
        tri.tri_append_paged(k, v, None, t, n_seq, L, H, nv, kn, kn, None, page_refs=c, ws=ws)
        tri.tri_decode_attention_paged(q, k, v, t, n_seq, L, H, nv, out=out, ws=ws)
        tri.tri_pages_fork(t, c, page, n_seq, nv, src, dst, ws=ws)
        tri.tri_pages_compact(k, v, t, c, n_live=n_live, ws=ws)

    def start(state):
        for x, y in zip((t, c, nv), state):
            x.copy_(_i32(y))
        k.copy_(k0)
        v.copy_(k0)

    want = []
    for s in states:
        start(s)
        step()
        want.append([x.clone() for x in (t, c, nv, k, v, out, n_free, n_live)])
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    for s, w in list(zip(states, want)) * 2:
        start(s)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((t, c, nv, k, v, out, n_free, n_live), w):
            assert torch.equal(x, y)


# ---------------------------------------------------------------------------
# together, as a serving loop uses them
# ---------------------------------------------------------------------------

def test_serving_loop_equals_contiguous_caches():
    """Prefill of a padded batch, decode steps, a fork, more steps, own pages,
    a prune, the pages given back, compaction and another step: the paged cache
    holds the rows of contiguous caches driven by the contiguous calls, and its
    attention agrees with theirs."""
    n_seq, L, H, G, page, cap, B = 3, 2, 2, 4, 128, 640, 200
    U, per = n_seq * L * H, L * H
    ppu = cap // page
    n_pages = U * ppu
    g = torch.Generator(DEV).manual_seed(11)
    rnd = lambda *s: torch.randn(s, device=DEV, generator=g).to(BF16)  # noqa: E731
    kp = torch.full((n_pages, page, R.D), float("nan"), dtype=BF16, device=DEV)
    vp = torch.full_like(kp, float("nan"))
    table = torch.full((U, ppu), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    nv = torch.zeros(U, dtype=torch.int32, device=DEV)
    pos = torch.zeros((U, cap), dtype=torch.int32, device=DEV)
    p_cur = torch.zeros(n_seq, dtype=torch.int64, device=DEV)
    kc, vc = torch.zeros((U, cap, R.D), dtype=BF16, device=DEV), torch.zeros((U, cap, R.D), dtype=BF16, device=DEV)
    n_c, pos_c = nv.clone(), pos.clone()
    ws = tri.workspace(max(tri.tri_pages_workspace_bytes(U, ppu, n_pages), tri.tri_append_paged_workspace_bytes(U),
                           tri.tri_decode_paged_workspace_bytes(U, G)))

    def ok(flags=0):
        assert tri.tri_check_device_error(ws) == flags

    def step():
        """One token of every sequence, layer by layer."""
        tri.tri_pages_fit(kp, vp, table, refs, n_seq, nv, n_new=1, ws=ws)
        ok()
        pn = p_cur.int().repeat_interleave(H)[:, None].contiguous()
        new = [(rnd(n_seq * H, 1, R.D), rnd(n_seq * H, 1, R.D), rnd(n_seq * H, G, R.D)) for _ in range(L)]
        for layer, (kn, vn, q) in enumerate(new):
            tri.tri_append_paged(kp, vp, pos, table, n_seq, L, H, nv, kn, vn, pn, layer=layer, page_refs=refs,
                                 p_cur=p_cur, ws=ws)
            ok()
        k1 = torch.stack([x[0].view(n_seq, H, 1, R.D) for x in new], 1).reshape(U, 1, R.D)
        v1 = torch.stack([x[1].view(n_seq, H, 1, R.D) for x in new], 1).reshape(U, 1, R.D)
        p1 = pn.view(n_seq, 1, H, 1).expand(n_seq, L, H, 1).reshape(U, 1).contiguous()
        tri.tri_append(kc, vc, pos_c, n_seq, n_c, k1.contiguous(), v1.contiguous(), p1)
        for layer, (_, _, q) in enumerate(new):
            units = R.unit_list(n_seq, L, H, layer)
            a = tri.tri_decode_attention_paged(q, kp, vp, table, n_seq, L, H, nv, layer=layer, ws=ws)
            ok()
            b = tri.tri_decode_attention(q, kc[units].contiguous(), vc[units].contiguous(), n_valid=n_c[units])
            assert (a - b).abs().max().item() <= 1e-4

    def same():
        assert torch.equal(nv, n_c)
        th = table.cpu().numpy()
        for u in range(U):
            n = int(nv[u])
            assert torch.equal(_rows(kp, th, u, n), kc[u, :n]) and torch.equal(_rows(vp, th, u, n), vc[u, :n])
            assert torch.equal(pos[u, :n], pos_c[u, :n])
        named = torch.bincount(table[table >= 0].long(), minlength=n_pages)
        assert torch.equal(named.int(), refs)

    # prefill: 300, 129 and 0 rows
    add = _i32([300, 129, 0])
    tri.tri_pages_fit(kp, vp, table, refs, n_seq, nv, n_new=300, n_add=add, ws=ws)
    ok()
    kn, vn = rnd(U, 300, R.D), rnd(U, 300, R.D)
    pn = torch.arange(300, dtype=torch.int32, device=DEV).expand(U, 300).contiguous()
    tri.tri_append_paged(kp, vp, pos, table, n_seq, L, H, nv, kn, vn, pn, n_add=add, page_refs=refs, p_cur=p_cur, ws=ws)
    ok()
    for u in range(U):
        n = [300, 129, 0][u // per]
        kc[u, :n], vc[u, :n], pos_c[u, :n] = kn[u, :n], vn[u, :n], pn[u, :n]
        n_c[u] = n
    assert p_cur.cpu().tolist() == [300, 129, 0]
    same()
    for _ in range(3):
        step()
    same()
    # sequence 2 becomes a continuation of 0, then both write
    tri.tri_pages_fork(table, refs, page, n_seq, nv, _i32([0]), _i32([2]), pos=pos, p_cur=p_cur, ws=ws)
    ok()
    for x in (kc, vc, pos_c, n_c):
        x[2 * per:] = x[:per]
    same()
    assert (refs == 2).sum().item() == per * 3
    for _ in range(2):
        step()
    same()
    assert (refs == 2).sum().item() == per * 2  # the two full pages stay shared
    # every sequence grows past the budget, then a prune
    tri.tri_pages_fit(kp, vp, table, refs, n_seq, nv, n_new=90, own=True, ws=ws)
    ok()
    assert refs.max().item() == 1
    kn, vn = rnd(U, 90, R.D), rnd(U, 90, R.D)
    pn = (p_cur.int().repeat_interleave(per)[:, None] + torch.arange(90, dtype=torch.int32, device=DEV)).contiguous()
    tri.tri_append_paged(kp, vp, pos, table, n_seq, L, H, nv, kn, vn, pn, page_refs=refs, p_cur=p_cur, ws=ws)
    ok()
    tri.tri_append(kc, vc, pos_c, n_seq, n_c, kn, vn, pn)
    same()
    stats = tri.tri_calibrate(rnd(L * H * G, 256, R.D)).view(L, H * G, 64, 4)
    nk, nk_c = torch.empty_like(nv), torch.empty_like(nv)
    kept, kept_c = (torch.empty((U, B), dtype=torch.int32, device=DEV) for _ in range(2))
    cfg = tri.config(path=tri.PATH_SPLIT)
    tri.tri_prune_paged_inplace(cfg, kp, vp, pos, table, cap, n_seq, L, H, G, p_cur, stats, B, nk, n_valid=nv, kept=kept)
    tri.tri_prune_inplace(cfg, kc, vc, pos_c, n_seq, L, H, G, p_cur, stats, B, nk_c, n_valid=n_c, kept=kept_c)
    assert torch.equal(kept, kept_c)
    nv, n_c = nk, nk_c
    free = tri.tri_pages_fit(kp, vp, table, refs, n_seq, nv, ws=ws)
    ok()
    assert free.item() == n_pages - U * 2
    same()
    live = tri.tri_pages_compact(kp, vp, table, refs, ws=ws)
    ok()
    assert live.item() == U * 2 and int(table.max()) == U * 2 - 1 and not refs[U * 2:].any()
    same()
    step()
    same()
    # a sequence ends
    tri.tri_pages_fork(table, refs, page, n_seq, nv, _i32([-1]), _i32([1]), pos=pos, p_cur=p_cur, ws=ws)
    ok()
    n_c[per:2 * per] = 0
    same()
    assert refs.sum().item() == 2 * per * 2


def test_refusals():
    """Host checks of the paged calls (no launch)."""
    lib = tri.load()
    P = ctypes.c_void_p
    assert lib.tri_pages_compact(P(1 << 36), None, tri.TRI_BF16, 1, 128, P(1 << 37), 16, 4, 0, P(1 << 38), None,
                                 P(1 << 39), 1 << 20, None) == 1
    k, v, table, refs = _cache([40, 3], 16, BF16, 1)
    t, c, n = _i32(table), _i32(refs), _i32([40, 3])
    q = torch.zeros((2, 4, R.D), dtype=BF16, device=DEV)
    call = lambda **o: tri.tri_decode_attention_paged(*[o.get(x, y) for x, y in (  # noqa: E731
        ("q", q), ("k", k), ("v", v), ("t", t), ("S", 1), ("L", 1), ("H", 2), ("n", n))], **o.get("kw", {}))
    call()
    for bad in (dict(q=q.float()), dict(q=q[:1]), dict(t=t.long()), dict(t=t.cpu()), dict(n=n[:1]), dict(H=3),
                dict(v=v[:1]), dict(v=v.float()), dict(kw=dict(layer=1)), dict(kw=dict(layer=-2)),
                dict(kw=dict(scale=-1.0)), dict(kw=dict(scale=float("inf"))), dict(kw=dict(out=torch.zeros(2, 4, 128))),
                dict(kw=dict(ws=torch.empty(16, dtype=torch.uint8, device=DEV))),
                dict(q=torch.zeros((2, 9, R.D), dtype=BF16, device=DEV)), dict(k=k[:, :, :64].contiguous(), v=v[:, :, :64].contiguous()),
                dict(q=q.transpose(0, 1))):
        with pytest.raises((tri.TriError, TypeError, ValueError)):
            call(**bad)
    kn = torch.zeros((2, 2, R.D), dtype=BF16, device=DEV)
    with pytest.raises(tri.TriError):  # values without a value pool
        tri.tri_append_paged(k, None, None, t, 1, 1, 2, n, kn, kn, None)
    with pytest.raises(tri.TriError):  # p_cur without positions
        tri.tri_append_paged(k, v, None, t, 1, 1, 2, n, kn, kn, None, p_cur=torch.zeros(1, dtype=torch.int64, device=DEV))
    with pytest.raises(tri.TriError):  # new rows inside the pool
        tri.tri_append_paged(k, v, None, t, 1, 1, 2, n, k.view(-1, 128)[:4].view(2, 2, 128), kn, None)
    with pytest.raises(tri.TriError):  # positions wider than the pages
        tri.tri_append_paged(k, v, torch.zeros((2, 49), dtype=torch.int32, device=DEV), t, 1, 1, 2, n, kn, kn,
                             torch.zeros((2, 2), dtype=torch.int32, device=DEV))
    with pytest.raises(tri.TriError):  # one pool for keys and values
        tri.tri_pages_fit(k, k, t, c, 1, n)
    with pytest.raises(tri.TriError):  # 2 units are not 3 sequences
        tri.tri_pages_fit(k, v, t, c, 3, n, n_add=_i32([0, 0, 0]))
    with pytest.raises(tri.TriError):
        tri.tri_pages_fork(t, c, 16, 2, n, _i32([0] * 1025), _i32([1] * 1025))
    with pytest.raises(ValueError):
        tri.tri_pages_fork(t, c, 16, 2, n, _i32([0]), _i32([1, 0]))
