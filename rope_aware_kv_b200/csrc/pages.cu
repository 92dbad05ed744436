// pages.cu -- a paged cache's rows and pages: append, fit (release, allocate,
// copy on write), fork and compact.
//
// The state is the page table ([n_units][per_unit], -1: no page) and, per
// page of the pool, the number of table entries that name it (0: free).
// Whole numbers decide everything and every choice goes by index (the i-th
// request in (unit, slot) order gets the i-th free page), so results do not
// depend on the order in which CTAs run; the atomics are integer additions
// and maxima.  All kernels move rows or small integer tables once: they are
// bound by HBM for large calls and by launches for small ones.
#include "paged_core.cuh"
#include "tri_launch.h"

namespace tri {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

static unsigned grid_for(int64_t items, int64_t per_cta, int64_t most) {
    const int64_t g = (items + per_cta - 1) / per_cta;
    return static_cast<unsigned>(g < 1 ? 1 : g < most ? g : most);
}

// Rows that sequence `seq` adds, clamped to [0, n_new].
__device__ __forceinline__ int64_t rows_added(const int32_t* n_add, int64_t seq, int64_t n_new,
                                              uint32_t* flag) {
    if (!n_add) return n_new;
    int64_t x = n_add[seq];
    if (x < 0 || x > n_new) {
        raise_flag(flag, TRI_FLAG_NVALID_RANGE);
        x = x < 0 ? 0 : n_new;
    }
    return x;
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
// A warp looks unit i over: where its new rows begin, or -1 when they do not
// fit, a page is missing, or a page is shared (the unit is then left as it
// is).  All lanes return the same values.
struct AppendUnit {
    int64_t unit;
    int64_t first;  // -1: refused
    int64_t add;
};

__device__ AppendUnit append_check(const AppendPagedArgs& a, int64_t i, int lane) {
    AppendUnit r;
    r.unit = slice_unit(a.sl, i);
    const int64_t per_seq = a.pc.n_units / a.pc.n_seq;
    r.add = rows_added(a.n_add, r.unit / per_seq, a.n_new, lane == 0 ? a.flag : nullptr);
    const int64_t n = a.n_valid[r.unit];
    r.first = n;
    if (n < 0 || n + r.add > a.cap) {
        if (lane == 0) raise_flag(a.flag, TRI_FLAG_NVALID_RANGE);
        r.first = -1;
        return r;
    }
    if (r.add == 0) return r;
    uint32_t bad = 0;
    const int64_t s1 = (n + r.add - 1) / a.pc.rows;
    for (int64_t slot = n / a.pc.rows + lane; slot <= s1; slot += 32) {
        const int64_t pg = page_of(a.pc, r.unit, slot);
        if (pg < 0)
            bad |= TRI_FLAG_INDEX_RANGE;
        else if (a.refs && a.refs[pg] > 1)
            bad |= TRI_FLAG_SHARED_PAGE;
    }
    bad = __reduce_or_sync(0xffffffffu, bad);
    if (bad) {
        if (lane == 0) raise_flag(a.flag, bad);
        r.first = -1;
    }
    return r;
}

// New count of the unit and 1 + its largest new position.
__device__ void append_account(const AppendPagedArgs& a, int64_t i, const AppendUnit& r, int lane) {
    if (r.first < 0 || r.add == 0) return;
    if (lane == 0) a.n_valid[r.unit] = static_cast<int32_t>(r.first + r.add);
    if (!a.p_cur) return;
    int32_t best = INT32_MIN;
    for (int64_t x = lane; x < r.add; x += 32) best = max(best, a.pos_new[i * a.n_new + x]);
    best = __reduce_max_sync(0xffffffffu, best);
    if (lane == 0)
        atomicMax(reinterpret_cast<long long*>(a.p_cur) + r.unit / (a.pc.n_units / a.pc.n_seq),
                  static_cast<long long>(best) + 1);
}

// A warp copies new rows [x0, x1) of unit i, whose new rows begin at `first`:
// half a warp moves a bf16 row (a whole one a float32 row) as 16-byte vectors.
template <int kVec>
__device__ void append_rows(const AppendPagedArgs& a, int64_t i, int64_t u, int64_t first,
                            int64_t x0, int64_t x1, int lane) {
    constexpr int kPer = 32 / kVec;  // rows of one array in one instruction
    uint4* k = static_cast<uint4*>(a.k);
    uint4* v = static_cast<uint4*>(a.v);
    const uint4* kn = static_cast<const uint4*>(a.k_new);
    const uint4* vn = static_cast<const uint4*>(a.v_new);
    for (int64_t b = x0; b < x1; b += 32) {
        const int64_t x = b + lane;
        const int64_t row = x < x1 ? paged_row(a.pc, u, first + x) : 0;
        if (a.pos && x < x1) a.pos[u * a.cap + first + x] = a.pos_new[i * a.n_new + x];
        const int m = static_cast<int>(min(x1 - b, static_cast<int64_t>(32)));
        for (int r = 0; r < m; r += kPer) {
            const int mine = r + lane / kVec;
            const int64_t dst = __shfl_sync(0xffffffffu, row, mine < m ? mine : 0);
            if (mine < m && dst >= 0) {
                const int64_t src = (i * a.n_new + b + mine) * kVec + lane % kVec;
                k[dst * kVec + lane % kVec] = ld_stream(kn + src);
                if (v) v[dst * kVec + lane % kVec] = ld_stream(vn + src);
            }
        }
    }
}

// Few new rows a unit: one warp does all of a unit.
constexpr int kAppendFew = 8;

template <int kVec>
__global__ void __launch_bounds__(kThreads) append_few_kernel(const AppendPagedArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (i >= a.sl.n) return;
    const AppendUnit r = append_check(a, i, lane);
    if (r.first < 0) return;
    append_rows<kVec>(a, i, r.unit, r.first, 0, r.add, lane);
    append_account(a, i, r, lane);
}

// Many: the units are looked over first (one warp each), then every CTA
// copies kAppendChunk rows of one unit.
constexpr int kAppendChunk = 64;

__global__ void __launch_bounds__(kThreads) append_look_kernel(const AppendPagedArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (i >= a.sl.n) return;
    const AppendUnit r = append_check(a, i, lane);
    if (lane == 0) a.first[i] = static_cast<int32_t>(r.first);
    append_account(a, i, r, lane);
}

template <int kVec>
__global__ void __launch_bounds__(kThreads) append_copy_kernel(const AppendPagedArgs a, int chunks) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i = blockIdx.x / chunks;
    const int64_t first = a.first[i];
    if (first < 0) return;
    const int64_t u = slice_unit(a.sl, i);
    const int64_t add = rows_added(a.n_add, u / (a.pc.n_units / a.pc.n_seq), a.n_new, nullptr);
    constexpr int kRows = kAppendChunk / kWarps;
    const int64_t x0 = static_cast<int64_t>(blockIdx.x % chunks) * kAppendChunk + warp * kRows;
    append_rows<kVec>(a, i, u, first, x0, min(x0 + kRows, add), lane);
}

template <int kVec>
static cudaError_t launch_append_t(const AppendPagedArgs& a, cudaStream_t s) {
    const unsigned units = grid_for(a.sl.n, kWarps, INT32_MAX);
    if (a.n_new <= kAppendFew) {
        append_few_kernel<kVec><<<units, kThreads, 0, s>>>(a);
        note_launch(s);
        return cudaGetLastError();
    }
    append_look_kernel<<<units, kThreads, 0, s>>>(a);
    note_launch(s);
    const int64_t chunks = (a.n_new + kAppendChunk - 1) / kAppendChunk;
    append_copy_kernel<kVec><<<static_cast<unsigned>(a.sl.n * chunks), kThreads, 0, s>>>(
        a, static_cast<int>(chunks));
    note_launch(s);
    return cudaGetLastError();
}

cudaError_t launch_append_paged(tri_dtype dt, const AppendPagedArgs& a, cudaStream_t s) {
    return dt == TRI_BF16 ? launch_append_t<kD * 2 / 16>(a, s) : launch_append_t<kD * 4 / 16>(a, s);
}

// ---------------------------------------------------------------------------
// counting and listing by chunks
// ---------------------------------------------------------------------------
// Sum of `x` over the CTA, in every thread.
__device__ __forceinline__ uint32_t cta_sum(uint32_t x) {
    __shared__ uint32_t w[kWarps];
    x = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = x;
    __syncthreads();
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) t += w[i];
    return t;
}

// Number of set `x` in the threads before this one, and of the whole CTA.
__device__ __forceinline__ uint32_t cta_rank(bool x, uint32_t* total) {
    __shared__ uint32_t w[kWarps];
    const uint32_t bal = __ballot_sync(0xffffffffu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = __popc(bal);
    __syncthreads();
    uint32_t before = __popc(bal & ((1u << (threadIdx.x & 31)) - 1u)), t = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < static_cast<int>(threadIdx.x >> 5)) before += w[i];
        t += w[i];
    }
    *total = t;
    return before;
}

// Sums of counts[0 .. at) and counts[0 .. n), in every thread.
__device__ __forceinline__ uint2 cta_prefix(const uint32_t* counts, int stride, int64_t n, int64_t at) {
    uint32_t before = 0, all = 0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
        const uint32_t c = __ldcg(counts + i * stride);
        all += c;
        if (i < at) before += c;
    }
    return make_uint2(cta_sum(before), cta_sum(all));
}

// ---------------------------------------------------------------------------
// fit
// ---------------------------------------------------------------------------
// What the call wants of one table slot.
struct SlotWish {
    bool kept;     // the slot's page stays (or is asked for)
    bool written;  // its rows will be written
    int64_t rows;  // rows below n_valid that it holds
};

__device__ __forceinline__ SlotWish slot_wish(const FitArgs& a, int64_t u, int64_t slot,
                                              uint32_t* flag) {
    const int64_t cap = a.pc.per_unit * a.pc.rows;
    const int64_t n = clamp_nvalid(a.n_valid, u, cap, flag);
    const int64_t add = rows_added(a.n_add, u / (a.pc.n_units / a.pc.n_seq), a.n_new, flag);
    if (n + add > cap) raise_flag(flag, TRI_FLAG_NVALID_RANGE);
    SlotWish w;
    const int64_t row0 = slot * a.pc.rows;
    w.kept = row0 < n + add;
    w.written = w.kept && (a.own || (add > 0 && row0 + a.pc.rows > n));
    const int64_t r = n - row0;
    w.rows = r < 0 ? 0 : r < a.pc.rows ? r : a.pc.rows;
    return w;
}

// Pages behind the last kept row are given back; pages that are shared and
// will be written are marked.  A count that falls below 2 while this runs can
// only make marks that the next kernel finds needless.
__global__ void __launch_bounds__(kThreads) fit_mark_kernel(const FitArgs a) {
    const int64_t slots = a.pc.n_units * a.pc.per_unit;
    for (int64_t id = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; id < slots;
         id += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t u = id / a.pc.per_unit, slot = id - u * a.pc.per_unit;
        const int64_t pg = a.pc.table[id];
        const SlotWish w = slot_wish(a, u, slot, slot == 0 ? a.flag : nullptr);
        if (pg < 0 || pg >= a.pc.n_pages) {
            if (pg != -1) {
                raise_flag(a.flag, TRI_FLAG_INDEX_RANGE);
                a.pc.table[id] = -1;
            }
            continue;
        }
        if (!w.kept) {
            atomicSub(a.refs + pg, 1);
            a.pc.table[id] = -1;
        } else if (w.written && __ldcg(a.refs + pg) > 1) {
            atomicAdd(a.writers + pg, 1u);
            atomicMax(a.last + pg, static_cast<uint32_t>(id) + 1u);
        }
    }
}

// Whether the slot asks for a page (0: no, 1: it has none, 2: its page is
// shared and it gets a copy).  Where every holder of a page writes it, the
// last of them keeps it.
__device__ __forceinline__ int slot_need(const FitArgs& a, int64_t id, int64_t* page) {
    const int64_t u = id / a.pc.per_unit, slot = id - u * a.pc.per_unit;
    const int64_t pg = a.pc.table[id];
    const SlotWish w = slot_wish(a, u, slot, nullptr);
    *page = pg;
    if (!w.kept) return 0;
    if (pg < 0) return 1;
    const int32_t refs = a.refs[pg];
    if (!w.written || refs <= 1) return 0;
    return a.writers[pg] == static_cast<uint32_t>(refs) && a.last[pg] == id + 1 ? 0 : 2;
}

__global__ void __launch_bounds__(kThreads) fit_count_kernel(const FitArgs a, int slot_chunks) {
    if (static_cast<int>(blockIdx.x) < slot_chunks) {
        const int64_t slots = a.pc.n_units * a.pc.per_unit;
        uint32_t need = 0, copy = 0;
        for (int q = 0; q < kPageChunk / kThreads; ++q) {
            const int64_t id = blockIdx.x * static_cast<int64_t>(kPageChunk) + q * kThreads + threadIdx.x;
            int64_t pg;
            const int w = id < slots ? slot_need(a, id, &pg) : 0;
            need += w > 0;
            copy += w == 2;
        }
        need = cta_sum(need);
        copy = cta_sum(copy);
        if (threadIdx.x == 0) a.slot_counts[blockIdx.x] = make_uint2(need, copy);
    } else {
        const int64_t c = blockIdx.x - slot_chunks;
        uint32_t free = 0;
        for (int q = 0; q < kPageChunk / kThreads; ++q) {
            const int64_t p = c * kPageChunk + q * kThreads + threadIdx.x;
            free += p < a.pc.n_pages && a.refs[p] == 0;
        }
        free = cta_sum(free);
        if (threadIdx.x == 0) a.page_counts[c] = free;
    }
}

// The requests and the free pages in index order.  Nothing is served when
// there are fewer free pages than requests.
__global__ void __launch_bounds__(kThreads)
fit_list_kernel(const FitArgs a, int slot_chunks, int page_chunks) {
    const bool slots_side = static_cast<int>(blockIdx.x) < slot_chunks;
    const int64_t c = slots_side ? blockIdx.x : blockIdx.x - slot_chunks;
    const uint32_t* counts = reinterpret_cast<const uint32_t*>(a.slot_counts);
    const uint2 need = cta_prefix(counts, 2, slot_chunks, slots_side ? c : 0);
    const uint2 free = cta_prefix(a.page_counts, 1, page_chunks, slots_side ? 0 : c);
    const bool served = need.y <= free.y;
    if (blockIdx.x == 0) {
        const uint2 copy = cta_prefix(counts + 1, 2, slot_chunks, 0);
        if (threadIdx.x == 0) {
            a.totals[0] = served ? need.y : 0;
            a.totals[1] = served ? copy.y : 0;
            if (!served) raise_flag(a.flag, TRI_FLAG_NO_PAGES);
            if (a.n_free) *a.n_free = static_cast<int32_t>(free.y) - static_cast<int32_t>(need.y);
        }
    }
    if (!served || need.y == 0) return;
    if (slots_side) {
        if (a.slot_counts[c].x == 0) return;
        const int64_t slots = a.pc.n_units * a.pc.per_unit;
        uint32_t base = need.x, copy_base = cta_prefix(counts + 1, 2, slot_chunks, c).x;
        for (int q = 0; q < kPageChunk / kThreads; ++q) {
            const int64_t id = c * kPageChunk + q * kThreads + threadIdx.x;
            int64_t pg = -1;
            const int w = id < slots ? slot_need(a, id, &pg) : 0;
            uint32_t n, nc;
            const uint32_t r = base + cta_rank(w > 0, &n);
            const uint32_t rc = copy_base + cta_rank(w == 2, &nc);
            if (w > 0) {
                a.need_slot[r] = static_cast<int32_t>(id);
                a.need_old[r] = w == 2 ? static_cast<int32_t>(pg) : -1;
            }
            if (w == 2) a.copy_rank[rc] = static_cast<int32_t>(r);
            base += n;
            copy_base += nc;
        }
    } else {
        uint32_t base = free.x;
        for (int q = 0; q < kPageChunk / kThreads && base < need.y; ++q) {
            const int64_t p = c * kPageChunk + q * kThreads + threadIdx.x;
            const bool is_free = p < a.pc.n_pages && a.refs[p] == 0;
            uint32_t n;
            const uint32_t r = base + cta_rank(is_free, &n);
            if (is_free && r < need.y) a.free_page[r] = static_cast<int32_t>(p);
            base += n;
        }
    }
}

// A CTA copies `rows` rows of kVec 16-byte vectors, 8 loads a thread in
// flight.
__device__ __forceinline__ void copy_vectors(uint4* dst, const uint4* src, int64_t n) {
    for (int64_t b = 0; b < n; b += 8 * kThreads) {
        uint4 x[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int64_t e = b + q * kThreads + threadIdx.x;
            if (e < n) x[q] = ld_stream(src + e);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int64_t e = b + q * kThreads + threadIdx.x;
            if (e < n) dst[e] = x[q];
        }
    }
}

// Table entries and counts of the served requests, then the copies: a CTA
// takes the K or the V rows of one page at a time.
template <int kVec>
__global__ void __launch_bounds__(kThreads) fit_serve_kernel(const FitArgs a) {
    const uint32_t need = a.totals[0], copies = a.totals[1];
    for (int64_t r = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; r < need;
         r += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int32_t pg = a.free_page[r], old = a.need_old[r];
        a.pc.table[a.need_slot[r]] = pg;
        a.refs[pg] = 1;
        if (old >= 0) atomicSub(a.refs + old, 1);
    }
    for (int64_t c = blockIdx.x; c < 2 * static_cast<int64_t>(copies); c += gridDim.x) {
        const int32_t r = a.copy_rank[c >> 1];
        const int64_t id = a.need_slot[r], old = a.need_old[r], pg = a.free_page[r];
        const int64_t u = id / a.pc.per_unit;
        const SlotWish w = slot_wish(a, u, id - u * a.pc.per_unit, nullptr);
        uint4* x = static_cast<uint4*>(c & 1 ? a.v : a.k);
        if (!x) continue;
        copy_vectors(x + pg * a.pc.rows * kVec, x + old * a.pc.rows * kVec, w.rows * kVec);
    }
}

cudaError_t launch_pages_fit(tri_dtype dt, const FitArgs& a, int n_sm, cudaStream_t s) {
    const int64_t slots = a.pc.n_units * a.pc.per_unit;
    const int slot_chunks = static_cast<int>((slots + kPageChunk - 1) / kPageChunk);
    const int page_chunks = static_cast<int>((a.pc.n_pages + kPageChunk - 1) / kPageChunk);
    fit_mark_kernel<<<grid_for(slots, kThreads, 8LL * n_sm), kThreads, 0, s>>>(a);
    note_launch(s);
    fit_count_kernel<<<slot_chunks + page_chunks, kThreads, 0, s>>>(a, slot_chunks);
    note_launch(s);
    fit_list_kernel<<<slot_chunks + page_chunks, kThreads, 0, s>>>(a, slot_chunks, page_chunks);
    note_launch(s);
    if (dt == TRI_BF16)
        fit_serve_kernel<kD * 2 / 16><<<8 * n_sm, kThreads, 0, s>>>(a);
    else
        fit_serve_kernel<kD * 4 / 16><<<8 * n_sm, kThreads, 0, s>>>(a);
    note_launch(s);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
// Every fork reads its source as it was on entry, though a sequence may be
// read by some forks and replaced by another (beams that change places).  The
// columns of the tables are independent of one another: a CTA takes some
// columns of one (layer, head) for ALL forks, reads the sources' entries into
// shared memory and only then writes the destinations'.  The row counts, which
// every CTA reads, are replaced by the CTA that finishes last.
constexpr int kForkCells = 8192;  // entries that a CTA holds

__global__ void __launch_bounds__(kThreads) pages_fork_kernel(const ForkArgs a, int table_cols,
                                                              int table_jobs, int pos_cols,
                                                              int pos_jobs) {
    extern __shared__ __align__(16) unsigned char smem[];
    int32_t* cell = reinterpret_cast<int32_t*>(smem);
    int32_t* src = cell + kForkCells;  // -1: empties, -2: skipped
    int32_t* dst = src + kMaxForks;
    __shared__ bool last;
    const int tid = threadIdx.x;
    const int F = static_cast<int>(a.n_fork);
    const int64_t per_seq = a.pc.n_units / a.pc.n_seq;  // (layer, head) pairs
    for (int f = tid; f < F; f += kThreads) {
        src[f] = a.src[f];
        dst[f] = a.dst[f];
    }
    __syncthreads();
    // A fork out of range is skipped, and so is one whose destination an
    // earlier fork has.
    bool skip[kMaxForks / kThreads];
#pragma unroll
    for (int q = 0; q < kMaxForks / kThreads; ++q) {
        const int f = q * kThreads + tid;
        skip[q] = false;
        if (f < F) {
            skip[q] = src[f] < -1 || src[f] >= a.pc.n_seq || dst[f] < 0 || dst[f] >= a.pc.n_seq;
            for (int g = 0; g < f && !skip[q]; ++g) skip[q] = dst[g] == dst[f];
        }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kMaxForks / kThreads; ++q) {
        const int f = q * kThreads + tid;
        if (f < F && skip[q]) {
            src[f] = -2;
            if (blockIdx.x == 0) raise_flag(a.flag, TRI_FLAG_INDEX_RANGE);
        }
    }
    __syncthreads();
    const int64_t cap = a.pc.per_unit * a.pc.rows;
    const int64_t jobs = per_seq * (table_jobs + pos_jobs);
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const bool pos = job >= per_seq * table_jobs;
        const int64_t j = pos ? job - per_seq * table_jobs : job;
        const int64_t lh = j % per_seq;
        const int64_t col0 = j / per_seq * (pos ? pos_cols : table_cols);
        const int64_t width = pos ? a.cap : a.pc.per_unit;
        const int cols = static_cast<int>(min(static_cast<int64_t>(pos ? pos_cols : table_cols), width - col0));
        for (int e = tid; e < F * cols; e += kThreads) {
            const int f = e / cols, c = e - f * cols;
            if (src[f] == -2) continue;
            if (src[f] < 0) {
                cell[e] = -1;
                continue;
            }
            const int64_t u = src[f] * per_seq + lh;
            const int64_t n = clamp_nvalid(a.n_valid, u, cap, nullptr);
            if (pos) {
                cell[e] = col0 + c < n ? a.pos[u * a.cap + col0 + c] : -1;
                continue;
            }
            int32_t pg = -1;
            if ((col0 + c) * a.pc.rows < n) {
                pg = static_cast<int32_t>(page_of(a.pc, u, col0 + c));
                if (pg < 0) raise_flag(a.flag, TRI_FLAG_INDEX_RANGE);
            }
            cell[e] = pg;
        }
        __syncthreads();
        for (int e = tid; e < F * cols; e += kThreads) {
            const int f = e / cols, c = e - f * cols;
            if (src[f] == -2) continue;
            const int64_t u = dst[f] * per_seq + lh;
            if (pos) {
                if (src[f] < 0) continue;
                const int64_t n = clamp_nvalid(a.n_valid, src[f] * per_seq + lh, cap, nullptr);
                if (col0 + c < n) a.pos[u * a.cap + col0 + c] = cell[e];
                continue;
            }
            const int64_t old = page_of(a.pc, u, col0 + c);
            if (cell[e] != old) {
                if (cell[e] >= 0) atomicAdd(a.refs + cell[e], 1);
                if (old >= 0) atomicSub(a.refs + old, 1);
            }
            a.pc.table[u * a.pc.per_unit + col0 + c] = cell[e];
        }
        __syncthreads();
    }
    // ---- the counts, when every CTA has read them ----
    __threadfence();
    __syncthreads();
    if (tid == 0) last = atomicAdd(a.done, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    const int step = kForkCells / F;  // (layer, head) pairs at a time
    for (int64_t lh0 = 0; lh0 < per_seq; lh0 += step) {
        const int cols = static_cast<int>(min(static_cast<int64_t>(step), per_seq - lh0));
        for (int e = tid; e < F * cols; e += kThreads) {
            const int f = e / cols, c = e - f * cols;
            cell[e] = src[f] >= 0 ? a.n_valid[src[f] * per_seq + lh0 + c] : 0;
        }
        __syncthreads();
        for (int e = tid; e < F * cols; e += kThreads) {
            const int f = e / cols, c = e - f * cols;
            if (src[f] != -2) a.n_valid[dst[f] * per_seq + lh0 + c] = cell[e];
        }
        __syncthreads();
    }
    if (!a.p_cur) return;
    int64_t now[kMaxForks / kThreads];
#pragma unroll
    for (int q = 0; q < kMaxForks / kThreads; ++q) {
        const int f = q * kThreads + tid;
        now[q] = f < F && src[f] >= 0 ? a.p_cur[src[f]] : 0;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kMaxForks / kThreads; ++q) {
        const int f = q * kThreads + tid;
        if (f < F && src[f] != -2) a.p_cur[dst[f]] = now[q];
    }
}

cudaError_t launch_pages_fork(const ForkArgs& a, cudaStream_t s) {
    const int64_t most = kForkCells / a.n_fork;
    const int table_cols = static_cast<int>(a.pc.per_unit < most ? a.pc.per_unit : most);
    const int64_t pos_width = a.pos ? a.cap : 0;
    const int pos_cols = static_cast<int>(pos_width < most ? (pos_width ? pos_width : 1) : most);
    const int64_t per_seq = a.pc.n_units / a.pc.n_seq;
    const int table_jobs = static_cast<int>((a.pc.per_unit + table_cols - 1) / table_cols);
    const int pos_jobs = static_cast<int>((pos_width + pos_cols - 1) / pos_cols);
    constexpr size_t smem = (kForkCells + 2 * kMaxForks) * sizeof(int32_t);
    pages_fork_kernel<<<grid_for(per_seq * (table_jobs + pos_jobs), 1, 65535), kThreads, smem, s>>>(
        a, table_cols, table_jobs, pos_cols, pos_jobs);
    note_launch(s);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------
// With L live pages, the live pages at L and behind go, in order, to the free
// pages below L, in order (there are as many of one as of the other).
__global__ void __launch_bounds__(kThreads) compact_count_kernel(const CompactPagesArgs a) {
    uint32_t live = 0;
    for (int q = 0; q < kPageChunk / kThreads; ++q) {
        const int64_t p = blockIdx.x * static_cast<int64_t>(kPageChunk) + q * kThreads + threadIdx.x;
        live += p < a.pc.n_pages && a.refs[p] != 0;
    }
    live = cta_sum(live);
    if (threadIdx.x == 0) a.page_counts[blockIdx.x] = live;
}

__global__ void __launch_bounds__(kThreads) compact_list_kernel(const CompactPagesArgs a, int chunks) {
    const int64_t c = blockIdx.x;
    const uint2 live = cta_prefix(a.page_counts, 1, chunks, c);
    const int64_t L = live.y;
    // Live pages below L: whole chunks, then the chunk that L lies in.
    const int64_t cl = L / kPageChunk;
    uint32_t below = cta_prefix(a.page_counts, 1, chunks, cl).x, part = 0;
    for (int64_t p = cl * kPageChunk + threadIdx.x; p < L; p += kThreads) part += a.refs[p] != 0;
    below += cta_sum(part);
    if (c == 0 && threadIdx.x == 0) {
        a.totals[0] = static_cast<uint32_t>(L);
        a.totals[1] = static_cast<uint32_t>(L) - below;
        if (a.n_live) *a.n_live = static_cast<int32_t>(L);
    }
    uint32_t base = live.x;
    for (int q = 0; q < kPageChunk / kThreads; ++q) {
        const int64_t p = c * kPageChunk + q * kThreads + threadIdx.x;
        const bool is_live = p < a.pc.n_pages && a.refs[p] != 0;
        uint32_t n;
        const uint32_t r = base + cta_rank(is_live, &n);  // live pages before p
        if (p < a.pc.n_pages) {
            if (p < L && !is_live) a.to[p - r] = static_cast<int32_t>(p);
            if (p >= L && is_live) {
                a.from[r - below] = static_cast<int32_t>(p);
                a.rank[p] = static_cast<int32_t>(r - below);
            }
        }
        base += n;
    }
}

// The moving pages' rows and counts, and the table entries that name them.
template <int kVec>
__global__ void __launch_bounds__(kThreads) compact_move_kernel(const CompactPagesArgs a) {
    const int64_t L = a.totals[0], moves = a.totals[1];
    if (moves == 0) return;
    const int64_t slots = a.pc.n_units * a.pc.per_unit;
    for (int64_t id = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; id < slots;
         id += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t pg = a.pc.table[id];
        if (pg < L || pg >= a.pc.n_pages) continue;
        // An entry whose page's count is 0 names no listed page: left, flagged.
        const int64_t r = a.rank[pg];
        if (r >= 0 && r < moves && a.from[r] == pg)
            a.pc.table[id] = a.to[r];
        else
            raise_flag(a.flag, TRI_FLAG_INDEX_RANGE);
    }
    for (int64_t c = blockIdx.x; c < 2 * moves; c += gridDim.x) {
        const int64_t from = a.from[c >> 1], to = a.to[c >> 1];
        if ((c & 1) == 0 && threadIdx.x == 0) {
            a.refs[to] = a.refs[from];
            a.refs[from] = 0;
        }
        uint4* x = static_cast<uint4*>(c & 1 ? a.v : a.k);
        if (!x) continue;
        copy_vectors(x + to * a.pc.rows * kVec, x + from * a.pc.rows * kVec, a.pc.rows * kVec);
    }
}

cudaError_t launch_pages_compact(tri_dtype dt, const CompactPagesArgs& a, int n_sm,
                                 cudaStream_t s) {
    const int chunks = static_cast<int>((a.pc.n_pages + kPageChunk - 1) / kPageChunk);
    compact_count_kernel<<<chunks, kThreads, 0, s>>>(a);
    note_launch(s);
    compact_list_kernel<<<chunks, kThreads, 0, s>>>(a, chunks);
    note_launch(s);
    if (dt == TRI_BF16)
        compact_move_kernel<kD * 2 / 16><<<8 * n_sm, kThreads, 0, s>>>(a);
    else
        compact_move_kernel<kD * 4 / 16><<<8 * n_sm, kThreads, 0, s>>>(a);
    note_launch(s);
    return cudaGetLastError();
}

}  // namespace tri
