"""Measured calls of the paged-cache operators: decode attention over a paged
KV cache, appending to it, and the page calls (fit, fork, compact).

Each case is one call (or its plain torch form when ``own`` is false) on a
cache whose pages are scattered over a pool.  Units are ordered
[n_seq][n_layers][n_kvheads]; a page table row lists the pages of one unit,
-1 where there is none; ``page_refs`` counts the table entries that name a page.
"""
import random

import torch

import rope_aware_kv_b200 as tri

own = False

D = 128          # head_dim
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One sequence's next token in one layer of the 28-layer 4-KV-head
        # model right after a prune to 2048 rows: the smallest call, latency.
        dict(name="decode 1 seq pruned", op="decode", dtype="bf16", n_seq=1, n_layers=28, kv=4, G=7, layer=13,
             page=128, low=2049, high=2176),
        # A serving batch of 16 sequences of that model, windows of different
        # ages, 64-row pages.
        dict(name="decode 16 seqs", op="decode", dtype="bf16", n_seq=16, n_layers=4, kv=4, G=7, layer=2, page=64,
             low=1500, high=3200),
        # The long-prefill model (8 KV heads, 4 query heads each) before its
        # first prune: 4 sequences of up to 131072 rows.
        dict(name="decode 4 long seqs", op="decode", dtype="bf16", n_seq=4, n_layers=1, kv=8, G=4, layer=0, page=128,
             low=98304, high=131072),
        # float32 cache, pages of 24 rows, a padded batch: some sequences hold
        # nothing or one row.
        dict(name="decode 24 ragged seqs f32", op="decode", dtype="f32", n_seq=24, n_layers=2, kv=4, G=8, layer=1,
             page=24, low=0, high=4099),
        # The next token's rows of every layer of 16 sequences.
        dict(name="append one token", op="append", dtype="bf16", n_seq=16, n_layers=28, kv=4, page=128, low=200,
             high=600, n_new=1),
        # A prefill of 4 prompts of different lengths in a padded batch.
        dict(name="append prompts", op="append", dtype="f32", n_seq=4, n_layers=4, kv=8, page=128, low=0, high=131,
             n_new=4096),
        # Room for the next token of 16 sequences, every layer: most units
        # need nothing, some a page, some give back what a prune left.
        dict(name="fit one token", op="fit", dtype="bf16", n_seq=16, n_layers=28, kv=4, page=32, low=1500, high=2175,
             n_new=1, shared=0, own=0),
        # Forked sequences made private before an in-place prune.
        dict(name="fit own before prune", op="fit", dtype="bf16", n_seq=8, n_layers=8, kv=8, page=128, low=1500,
             high=2176, n_new=0, shared=1, own=1),
        # Beam reorder of 4 beams of one sequence.
        dict(name="fork 4 beams", op="fork", dtype="bf16", n_seq=4, n_layers=28, kv=4, page=128, low=1900, high=2176,
             n_fork=4),
        # 32 of 64 sequences replaced by continuations of the other ones.
        dict(name="fork 32 seqs", op="fork", dtype="bf16", n_seq=64, n_layers=28, kv=4, page=16, low=1500, high=2176,
             n_fork=32),
        # A half-empty pool of one layer's small pages.
        dict(name="compact small pages", op="compact", dtype="bf16", n_seq=8, n_layers=1, kv=4, page=16, low=400,
             high=1100, spare=1.0),
        # A pool after many sequences have ended: 40 % free.
        dict(name="compact pool", op="compact", dtype="f32", n_seq=16, n_layers=8, kv=4, page=128, low=900,
             high=2176, spare=0.7),
    ]


def _log(rng, a, b):
    return int(round(a * (b / a) ** rng.random()))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "fit", "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    page = rng.choice([rng.randint(1, 40), 16, 32, 64, 128, 128, 256, 8 * rng.randint(1, 40)])
    if op == "decode":
        n_seq, kv, n_layers = _log(rng, 1, 64), rng.randint(1, 8), rng.randint(1, 3)
        most = max(64, min(131072, 3_200_000 // (n_seq * kv * n_layers) // (2 if dtype == "f32" else 1)))
        high = _log(rng, 1, most)
        return dict(op=op, dtype=dtype, n_seq=n_seq, n_layers=n_layers, kv=kv, G=rng.randint(1, 8),
                    layer=rng.randint(-1, n_layers - 1), page=page, low=rng.choice([0, high // 2, high]), high=high)
    n_seq, n_layers, kv = _log(rng, 2, 24), _log(rng, 1, 16), rng.randint(1, 8)
    units = n_seq * n_layers * kv
    if op == "append":
        high = _log(rng, 1, max(1, min(2000, 600_000 // units)))
        return dict(op=op, dtype=dtype, n_seq=n_seq, n_layers=n_layers, kv=kv, page=page, low=high // 3, high=high,
                    n_new=_log(rng, 1, max(2, min(4096, 400_000 // units))))
    high = max(2, _log(rng, 100, 2176) if units < 800 else _log(rng, 50, 900))
    base = dict(op=op, dtype=dtype, n_seq=n_seq, n_layers=n_layers, kv=kv, page=max(page, 8), low=high // 2, high=high)
    if op == "fit":
        return dict(base, n_new=rng.choice([0, 1, 1, rng.randint(2, 200)]), shared=rng.randint(0, 1),
                    own=rng.randint(0, 1))
    if op == "fork":
        return dict(base, n_fork=rng.randint(1, n_seq))
    return dict(base, spare=round(rng.uniform(0.05, 2.0), 2))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(case):
    """Rows of each sequence: a function of the case alone."""
    rng = random.Random("%s %d %d %d" % (case["op"], case["n_seq"], case["low"], case["high"]))
    got = [rng.randint(case["low"], case["high"]) for _ in range(case["n_seq"])]
    if case["low"] == 0 and case["n_seq"] >= 4:
        got[1], got[2] = 0, 1
    return got


def _adds(case):
    """New rows of each sequence in the padded batch."""
    rng = random.Random("add %d %d" % (case["n_seq"], case["n_new"]))
    if case["n_new"] <= 1:
        return [case["n_new"]] * case["n_seq"]
    return [rng.randint(1, case["n_new"]) for _ in range(case["n_seq"])]


def _ceil(a, b):
    return -(-a // b)


def _held(case):
    """Rows that each sequence's pages cover at the start of the call."""
    rows = _lengths(case)
    if case["op"] == "append":
        return [n + a for n, a in zip(rows, _adds(case))]
    if case["op"] == "fit":  # every fourth sequence still has the pages a prune emptied
        return [n + (case["high"] // 4 if s % 4 == 3 else 0) for s, n in enumerate(rows)]
    return rows


def _cap(case):
    most = case["high"] + case.get("n_new", 0) + (case["high"] // 4 if case["op"] == "fit" else 0)
    return max(1, most)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed * 1000003 + 17)
    dt = TYPES[case["dtype"]]
    S, L, H, page = case["n_seq"], case["n_layers"], case["kv"], case["page"]
    U, cap = S * L * H, _cap(case)
    ppu = _ceil(cap, page)
    rows = _lengths(case)
    n_valid = torch.tensor(rows, dtype=torch.int32, device=DEV).repeat_interleave(L * H)
    held = torch.tensor([_ceil(n, page) for n in _held(case)], device=DEV).repeat_interleave(L * H)
    used = int(held.sum())
    if case["op"] == "fit":  # room for what the call can ask for
        n_pages = used + U * (_ceil(case["n_new"], page) + 2) + (used if case["shared"] else 0)
    else:
        n_pages = max(1, int(used * (1.0 + case.get("spare", 0.1))))
    slot = torch.arange(ppu, device=DEV)[None, :]
    perm = torch.randperm(n_pages, generator=gen, device=DEV)
    first = (torch.cumsum(held, 0) - held)[:, None]
    at = torch.where(slot < held[:, None], first + slot, 0)
    table = torch.where(slot < held[:, None], perm[at], -1)
    if case.get("shared") and S >= 2:  # the second half of the sequences are forks of the first
        half = (S // 2) * L * H
        table[half:2 * half] = table[:half]
        n_valid[half:2 * half] = n_valid[:half]
    refs = torch.zeros(n_pages + 1, dtype=torch.int64, device=DEV)
    refs.index_add_(0, torch.where(table >= 0, table, n_pages).reshape(-1),
                    torch.ones(U * ppu, dtype=torch.int64, device=DEV))
    # What calls change is held in one buffer, so that a pass can begin from
    # the same state as the one before it.
    start = torch.cat([table.reshape(-1).int(), refs[:n_pages].int(), n_valid])
    live = start.clone()
    s = dict(case=case, start=start, live=live, table=live[:U * ppu].view(U, ppu),
             refs=live[U * ppu:U * ppu + n_pages], n_valid=live[U * ppu + n_pages:])
    if case["op"] != "fork":  # fork touches no K or V row
        s["k"] = torch.randn((n_pages, page, D), generator=gen, device=DEV, dtype=dt)
        s["v"] = torch.randn((n_pages, page, D), generator=gen, device=DEV, dtype=dt)
    if case["op"] == "decode":
        Uq = U if case["layer"] < 0 else S * H
        s["q"] = (torch.randn((Uq, case["G"], D), generator=gen, device=DEV) * 2.0).to(dt)
    if case["op"] in ("append", "fork"):
        s["pos"] = torch.randint(0, 32768, (U, cap), generator=gen, device=DEV, dtype=torch.int32)
        s["p_cur"] = torch.tensor(rows, dtype=torch.int64, device=DEV)
    if case["op"] == "append":
        n = case["n_new"]
        s["n_add"] = torch.tensor(_adds(case), dtype=torch.int32, device=DEV)
        s["k_new"] = torch.randn((U, n, D), generator=gen, device=DEV, dtype=dt)
        s["v_new"] = torch.randn((U, n, D), generator=gen, device=DEV, dtype=dt)
        s["pos_new"] = (n_valid[:, None] + torch.arange(n, device=DEV, dtype=torch.int32)[None, :]).contiguous()
    if case["op"] == "fit":
        s["n_add"] = torch.tensor(_adds(case), dtype=torch.int32, device=DEV)
    if case["op"] == "fork":
        # The best beams (about half) go on and take the other ones' places:
        # a beam that is both read and replaced stays itself, so that the same
        # call can be made again.
        rng = random.Random(seed)
        best = rng.sample(range(S), max(1, S // 2))
        dst = sorted(rng.sample(range(S), case["n_fork"]))
        src = [d if d in best else rng.choice(best) for d in dst]
        s["dst"] = torch.tensor(dst, dtype=torch.int32, device=DEV)
        s["src"] = torch.tensor(src, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# the calls
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if op != "decode":  # the others change the tables and counts
        s["live"].copy_(s["start"])
    return (_OWN if own else _PLAIN)[op](s)


def _ws(s, nbytes):
    """The workspace that a user's program keeps for the call."""
    if "ws" not in s:
        s["ws"] = tri.workspace(nbytes)
    return s["ws"]


def _decode_own(s):
    c = s["case"]
    ws = _ws(s, tri.tri_decode_paged_workspace_bytes(s["q"].shape[0], c["G"]))
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
    out = tri.tri_decode_attention_paged(s["q"], s["k"], s["v"], s["table"], c["n_seq"], c["n_layers"], c["kv"],
                                         s["n_valid"], layer=c["layer"], lse=lse, ws=ws)
    return dict(out=out, lse=lse)


def _append_own(s):
    c = s["case"]
    ws = _ws(s, tri.tri_append_paged_workspace_bytes(s["table"].shape[0]))
    tri.tri_append_paged(s["k"], s["v"], s["pos"], s["table"], c["n_seq"], c["n_layers"], c["kv"], s["n_valid"],
                         s["k_new"], s["v_new"], s["pos_new"], n_add=s["n_add"], page_refs=s["refs"],
                         p_cur=s["p_cur"], ws=ws)
    return {k: s[k] for k in ("k", "v", "pos", "n_valid", "p_cur")}


def _fit_own(s):
    c = s["case"]
    ws = _ws(s, tri.tri_pages_workspace_bytes(*s["table"].shape, s["refs"].numel()))
    n_free = tri.tri_pages_fit(s["k"], s["v"], s["table"], s["refs"], c["n_seq"], s["n_valid"], n_new=c["n_new"],
                               n_add=s["n_add"], own=bool(c["own"]), ws=ws)
    return dict(table=s["table"], refs=s["refs"], n_free=n_free, k=s["k"], v=s["v"])


def _fork_own(s):
    c = s["case"]
    ws = _ws(s, tri.tri_pages_workspace_bytes(*s["table"].shape, s["refs"].numel()))
    tri.tri_pages_fork(s["table"], s["refs"], c["page"], c["n_seq"], s["n_valid"], s["src"], s["dst"], pos=s["pos"],
                       p_cur=s["p_cur"], ws=ws)
    return {k: s[k] for k in ("table", "refs", "n_valid", "pos", "p_cur")}


def _compact_own(s):
    ws = _ws(s, tri.tri_pages_workspace_bytes(*s["table"].shape, s["refs"].numel()))
    n_live = tri.tri_pages_compact(s["k"], s["v"], s["table"], s["refs"], ws=ws)
    return dict(table=s["table"], refs=s["refs"], n_live=n_live, k=s["k"], v=s["v"])


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _decode_plain(s):
    c = s["case"]
    S, L, H, page = c["n_seq"], c["n_layers"], c["kv"], c["page"]
    table, n = s["table"].long(), s["n_valid"].long()
    if c["layer"] >= 0:
        table = table.view(S, L, H, -1)[:, c["layer"]].reshape(S * H, -1)
        n = n.view(S, L, H)[:, c["layer"]].reshape(-1)
    j = torch.arange(_cap(c), device=DEV)
    inside = j[None, :] < n[:, None]
    at = (table[:, j // page] * page + (j % page)[None, :]).clamp_(min=0)
    k = s["k"].view(-1, D)[at].float()
    logits = torch.matmul(s["q"].float(), k.transpose(1, 2)) * D ** -0.5
    del k
    logits = torch.where(inside[:, None, :], logits, -torch.inf)
    m = logits.amax(2, keepdim=True)
    p = torch.exp(logits - torch.where(m > -torch.inf, m, 0.0))
    den = p.sum(2, keepdim=True)
    v = torch.where(inside[:, :, None], s["v"].view(-1, D)[at], 0.0).float()
    out = torch.matmul(p, v) / torch.where(den > 0, den, 1.0)
    return dict(out=out, lse=(m + torch.log(den))[:, :, 0])


def _append_plain(s):
    c = s["case"]
    per, page = c["n_layers"] * c["kv"], c["page"]
    add = s["n_add"].long().repeat_interleave(per)
    i = torch.arange(c["n_new"], device=DEV)
    u, i = torch.nonzero(i[None, :] < add[:, None], as_tuple=True)
    j = s["n_valid"].long()[u] + i
    at = s["table"].long()[u, j // page] * page + j % page
    s["k"].view(-1, D)[at] = s["k_new"][u, i]
    s["v"].view(-1, D)[at] = s["v_new"][u, i]
    s["pos"][u, j] = s["pos_new"][u, i]
    seq = u // per
    s["p_cur"].scatter_reduce_(0, seq, s["pos_new"][u, i].long() + 1, "amax")
    s["n_valid"].add_(add.int())
    return {k: s[k] for k in ("k", "v", "pos", "n_valid", "p_cur")}


def _fit_plain(s):
    c = s["case"]
    table, refs, page = s["table"], s["refs"], c["page"]
    U, ppu = table.shape
    n_pages = refs.numel()
    n = s["n_valid"].long()[:, None]
    add = s["n_add"].long().repeat_interleave(U // c["n_seq"])[:, None]
    keep = (n + add + page - 1) // page
    slot = torch.arange(ppu, device=DEV)[None, :]
    ids = torch.arange(U * ppu, device=DEV).view(U, ppu)
    t = table.long()
    gone = (t >= 0) & (slot >= keep)
    r = torch.cat([refs.long(), refs.new_zeros(1).long()])
    r.scatter_add_(0, torch.where(gone, t, n_pages).view(-1), -torch.ones(U * ppu, dtype=torch.int64, device=DEV))
    t = torch.where(gone, -1, t)
    # shared pages that will be written; the last writer keeps the page where every holder writes it
    written = (t >= 0) & (slot < keep) & (r[t] > 1) & (bool(c["own"]) | ((slot >= n // page) & (add > 0)))
    to = torch.where(written, t, n_pages).view(-1)
    writers = torch.zeros(n_pages + 1, dtype=torch.int64, device=DEV).scatter_add_(0, to, torch.ones_like(to))
    last = torch.full((n_pages + 1,), -1, dtype=torch.int64, device=DEV).scatter_reduce_(0, to, ids.view(-1), "amax")
    copied = written & ~((writers[t] == r[t]) & (last[t] == ids))
    need = copied | ((t < 0) & (slot < keep))
    free = torch.nonzero(r[:n_pages] == 0)[:, 0]
    u, b = torch.nonzero(need, as_tuple=True)
    got, old = free[:u.numel()], t[u, b]
    r.scatter_add_(0, torch.where(old >= 0, old, n_pages), -torch.ones_like(old))
    r[got] = 1
    # rows below n_valid of the copied pages
    i = torch.arange(page, device=DEV)[None, :]
    w, i = torch.nonzero((old >= 0)[:, None] & (b[:, None] * page + i < n[u]), as_tuple=True)
    s["k"].view(-1, D)[got[w] * page + i] = s["k"].view(-1, D)[old[w] * page + i]
    s["v"].view(-1, D)[got[w] * page + i] = s["v"].view(-1, D)[old[w] * page + i]
    t[u, b] = got
    table.copy_(t)
    refs.copy_(r[:n_pages])
    n_free = torch.full((1,), free.numel() - u.numel(), dtype=torch.int32, device=DEV)
    return dict(table=table, refs=refs, n_free=n_free, k=s["k"], v=s["v"])


def _fork_plain(s):
    c = s["case"]
    S, page, n_pages = c["n_seq"], c["page"], s["refs"].numel()
    table = s["table"].view(S, -1, s["table"].shape[1])
    n_valid, pos = s["n_valid"].view(S, -1), s["pos"].view(S, table.shape[1], -1)
    src, dst = s["src"].long(), s["dst"].long()
    old, n = table[dst], n_valid[src]
    slot = torch.arange(table.shape[2], device=DEV)
    new = torch.where(slot * page < n[:, :, None], table[src], -1)
    r = torch.cat([s["refs"], s["refs"].new_zeros(1)])
    one = torch.ones(old.numel(), dtype=torch.int32, device=DEV)
    r.index_add_(0, torch.where(old >= 0, old, n_pages).view(-1), -one)
    r.index_add_(0, torch.where(new >= 0, new, n_pages).view(-1), one)
    s["refs"].copy_(r[:n_pages])
    table[dst] = new
    row = torch.arange(pos.shape[2], device=DEV)
    pos[dst] = torch.where(row < n[:, :, None], pos[src], pos[dst])
    n_valid[dst] = n
    s["p_cur"][dst] = s["p_cur"][src]
    return {k: s[k] for k in ("table", "refs", "n_valid", "pos", "p_cur")}


def _compact_plain(s):
    table, refs = s["table"], s["refs"]
    ids = torch.arange(refs.numel(), device=DEV)
    live = refs != 0
    n_live = live.sum()
    src = torch.nonzero(live & (ids >= n_live))[:, 0]
    dst = torch.nonzero(~live & (ids < n_live))[:, 0]
    s["k"][dst] = s["k"][src]
    s["v"][dst] = s["v"][src]
    to = ids.int()
    to[src] = dst.int()
    table.copy_(torch.where(table >= 0, to[table.long()], table))
    refs[dst] = refs[src]
    refs[src] = 0
    return dict(table=table, refs=refs, n_live=n_live.int().view(1), k=s["k"], v=s["v"])


_OWN = dict(decode=_decode_own, append=_append_own, fit=_fit_own, fork=_fork_own, compact=_compact_own)
_PLAIN = dict(decode=_decode_plain, append=_append_plain, fit=_fit_plain, fork=_fork_plain, compact=_compact_plain)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    row = D * (2 if case["dtype"] == "bf16" else 4)
    S, per, page = case["n_seq"], case["n_layers"] * case["kv"], case["page"]
    rows, held = _lengths(case), _held(case)
    U, ppu = S * per, _ceil(_cap(case), page)
    pages = sum(_ceil(n, page) for n in held) * per
    if case["op"] == "decode":
        heads = per if case["layer"] < 0 else case["kv"]
        keys, units = sum(rows) * heads, S * heads
        return {"bytes": 2 * row * keys + units * case["G"] * (row + 4 * D + 4)
                + 4 * heads * sum(_ceil(n, page) for n in rows) + 4 * units, "flops": 4 * D * case["G"] * keys}
    if case["op"] == "append":
        new = sum(_adds(case)) * per
        return {"bytes": new * 2 * (2 * row + 4) + 8 * U + 4 * U, "flops": 0}
    if case["op"] == "fit":  # the tables and counts once, and the rows that are copied, read and written
        copied = 0
        if case["shared"] and S >= 2:
            now = rows[:S // 2]
            copied = sum(n if case["own"] else (n % page if a else 0) for n, a in zip(now, _adds(case))) * per
        return {"bytes": 4 * U * ppu + 4 * pages + 4 * U + 2 * 2 * row * copied, "flops": 0}
    if case["op"] == "fork":
        n = sum(rows) * case["n_fork"] * per / S
        return {"bytes": 2 * 4 * n + 4 * 4 * n / page, "flops": 0}
    n_pages = max(1, int(pages * (1.0 + case["spare"])))
    moved = pages * (n_pages - pages) / n_pages  # live pages behind the border, on average
    return {"bytes": moved * page * row * 2 * 2 + 4 * n_pages + 4 * U * ppu, "flops": 0}


def exact(case, seed):
    if case["op"] != "decode":
        return None  # rows and whole numbers that are moved, none computed
    s = prepare(case, seed)
    S, L, H, G = case["n_seq"], case["n_layers"], case["kv"], case["G"]
    layers = range(L) if case["layer"] < 0 else [case["layer"]]
    units = [(q * L + l) * H + h for q in range(S) for l in layers for h in range(H)]
    table, n_valid = s["table"].tolist(), s["n_valid"].tolist()
    out = torch.zeros((len(units), G, D), dtype=torch.float64, device=DEV)
    lse = torch.full((len(units), G), -float("inf"), dtype=torch.float64, device=DEV)
    for i, u in enumerate(units):
        n = n_valid[u]
        if n == 0:
            continue
        pages = torch.tensor(table[u][:_ceil(n, case["page"])], device=DEV)
        k = s["k"].index_select(0, pages).double().flatten(0, 1)[:n]
        v = s["v"].index_select(0, pages).double().flatten(0, 1)[:n]
        x = s["q"][i].double() @ k.T / 128.0 ** 0.5
        lse[i] = torch.logsumexp(x, 1)
        out[i] = torch.softmax(x, 1) @ v
    return dict(out=out, lse=lse)
