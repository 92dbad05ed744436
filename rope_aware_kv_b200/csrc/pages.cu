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

// Warps that move rows with bulk copies, and the shared memory of each.
constexpr int kEngines = 8;
constexpr int kWindow = 8192;
struct CopyShared {
    unsigned char window[kEngines][kWindow];
    uint64_t landed[kEngines];
};

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

// New rows [x0, x0 + m) (at most 8) of unit i in a warp's registers: half a warp
// holds a bf16 row (a whole one a float32 row) as 16-byte vectors, all rows of
// both arrays in flight before the first store.
constexpr int kAppendFew = 8;

template <int kVec>
struct NewRows {
    static constexpr int kPer = 32 / kVec;  // rows of one array in one instruction
    static constexpr int kIter = kAppendFew / kPer;
    uint4 k[kIter], v[kIter];

    __device__ __forceinline__ void read(const AppendPagedArgs& a, int64_t i, int64_t x0, int m, int lane) {
        const int64_t src = (i * a.n_new + x0) * kVec + lane;
#pragma unroll
        for (int r = 0; r < kIter; ++r)
            if (r * 32 + lane < m * kVec) k[r] = ld_stream(static_cast<const uint4*>(a.k_new) + src + r * 32);
        if (!a.v) return;
#pragma unroll
        for (int r = 0; r < kIter; ++r)
            if (r * 32 + lane < m * kVec) v[r] = ld_stream(static_cast<const uint4*>(a.v_new) + src + r * 32);
    }
    // Into rows row0, row0 + 1, ... of unit u.
    __device__ __forceinline__ void write(const AppendPagedArgs& a, int64_t u, int64_t row0, int m, int lane) {
        const int64_t row = lane < m ? paged_row(a.pc, u, row0 + lane) : -1;
#pragma unroll
        for (int r = 0; r < kIter; ++r) {
            const int64_t dst = __shfl_sync(0xffffffffu, row, r * kPer + lane / kVec);
            if (r * 32 + lane >= m * kVec || dst < 0) continue;
            static_cast<uint4*>(a.k)[dst * kVec + lane % kVec] = k[r];
            if (a.v) static_cast<uint4*>(a.v)[dst * kVec + lane % kVec] = v[r];
        }
    }
};

// Few new rows a unit (what a warp's registers hold): one warp does all of a
// unit, in one launch.  1792 units of 1 bf16 row: 8.5 us against 14.5 us by the
// other two kernels, of 8 float32 rows 10.4 against 16.8 us; 448 units: alike.
template <int kVec>
__global__ void __launch_bounds__(kThreads) append_few_kernel(const AppendPagedArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (i >= a.sl.n) return;
    const AppendUnit r = append_check(a, i, lane);
    if (r.first < 0) return;
    const int m = static_cast<int>(r.add);
    NewRows<kVec> rows;
    rows.read(a, i, 0, m, lane);
    rows.write(a, r.unit, r.first, m, lane);
    if (a.pos && lane < m) a.pos[r.unit * a.cap + r.first + lane] = a.pos_new[i * a.n_new + lane];
    append_account(a, i, r, lane);
}

// Many: the units are looked over first (a CTA each, since a unit's positions
// and pages are many), then every warp copies 8 rows of one unit, which it reads
// while the look is under way.  (Bulk copies, 8 KB a window, took 130 us where
// this takes 90: a ragged batch has many short windows.)
__global__ void __launch_bounds__(kThreads) append_look_kernel(const AppendPagedArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x;
    const int64_t i = blockIdx.x;
    const int64_t u = slice_unit(a.sl, i);
    const int64_t seq = u / (a.pc.n_units / a.pc.n_seq);
    const int64_t add = rows_added(a.n_add, seq, a.n_new, tid == 0 ? a.flag : nullptr);
    const int64_t n = a.n_valid[u];
    uint32_t bad = n < 0 || n + add > a.cap ? TRI_FLAG_NVALID_RANGE : 0;
    int32_t best = INT32_MIN;
    if (!bad && add > 0) {
        const int64_t s1 = (n + add - 1) / a.pc.rows;
        for (int64_t slot = n / a.pc.rows + tid; slot <= s1; slot += kThreads) {
            const int64_t pg = page_of(a.pc, u, slot);
            if (pg < 0)
                bad |= TRI_FLAG_INDEX_RANGE;
            else if (a.refs && a.refs[pg] > 1)
                bad |= TRI_FLAG_SHARED_PAGE;
        }
        if (a.p_cur) {
#pragma unroll 8
            for (int64_t x = tid; x < add; x += kThreads) best = max(best, a.pos_new[i * a.n_new + x]);
        }
    }
    const int any = __syncthreads_or(bad != 0);
    if (bad) raise_flag(a.flag, bad);
    if (tid == 0) {
        a.first[i] = any ? -1 : static_cast<int32_t>(n);
        if (!any) a.n_valid[u] = static_cast<int32_t>(n + add);
    }
    if (any || add == 0) return;
    if (a.pos) {
#pragma unroll 8
        for (int64_t x = tid; x < add; x += kThreads) a.pos[u * a.cap + n + x] = a.pos_new[i * a.n_new + x];
    }
    if (!a.p_cur) return;
    best = __reduce_max_sync(0xffffffffu, best);
    if ((tid & 31) == 0 && best != INT32_MIN)
        atomicMax(reinterpret_cast<long long*>(a.p_cur) + seq, static_cast<long long>(best) + 1);
}

template <int kVec>
__global__ void __launch_bounds__(kThreads) append_copy_kernel(const AppendPagedArgs a, int chunks) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i = blockIdx.x / chunks;
    const int64_t u = slice_unit(a.sl, i);
    const int64_t add = rows_added(a.n_add, u / (a.pc.n_units / a.pc.n_seq), a.n_new, nullptr);
    const int64_t x0 = (static_cast<int64_t>(blockIdx.x % chunks) * kWarps + warp) * kAppendFew;
    const int m = static_cast<int>(max(min(add - x0, static_cast<int64_t>(kAppendFew)), static_cast<int64_t>(0)));
    NewRows<kVec> rows;
    rows.read(a, i, x0, m, lane);
    // For the look kernel; by every warp, so that this kernel does not end
    // before that one has.
    wait_for_clear();
    if (m == 0) return;
    const int64_t first = __ldcg(a.first + i);
    if (first >= 0) rows.write(a, u, first + x0, m, lane);
}

template <int kVec>
static cudaError_t launch_append_t(const AppendPagedArgs& a, cudaStream_t s) {
    if (a.n_new <= kAppendFew) {
        append_few_kernel<kVec><<<grid_for(a.sl.n, kWarps, INT32_MAX), kThreads, 0, s>>>(a);
        note_launch(s);
        return cudaGetLastError();
    }
    append_look_kernel<<<static_cast<unsigned>(a.sl.n), kThreads, 0, s>>>(a);
    note_launch(s);
    const int64_t chunks = (a.n_new + kWarps * kAppendFew - 1) / (kWarps * kAppendFew);
    const cudaError_t e = launch_early(append_copy_kernel<kVec>, static_cast<unsigned>(a.sl.n * chunks), kThreads, 0,
                                       s, a, static_cast<int>(chunks));
    if (e == cudaSuccess) note_launch(s);
    return e;
}

cudaError_t launch_append_paged(tri_dtype dt, const AppendPagedArgs& a, cudaStream_t s) {
    return dt == TRI_BF16 ? launch_append_t<kD * 2 / 16>(a, s) : launch_append_t<kD * 4 / 16>(a, s);
}

// ---------------------------------------------------------------------------
// one grid, several phases (fit, compact)
// ---------------------------------------------------------------------------
// fit and compact are cooperative kernels: their phases (count, list, serve)
// depend on one another over the whole pool, and a barrier of the grid costs
// less than a launch.  CTA c of C owns the c-th C-th of the slots and of the
// pages, so ranks over the pool are prefix sums of C counts.
constexpr int kGridThreads = 512;
constexpr int kGridWarps = kGridThreads / 32;

// All CTAs of the grid have arrived (their writes are visible); `round` counts
// the barriers.  Gives up after 2 s (TRI_FLAG_TIMEOUT): false, and the kernel
// returns.
__device__ bool grid_barrier(uint32_t* count, int round, uint32_t* flag) {
    __shared__ bool ok;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(count, 1u);
        const uint32_t want = static_cast<uint32_t>(round) * gridDim.x;
        const uint64_t t0 = globaltimer_ns();
        ok = true;
        while (true) {
            uint32_t now;
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(now) : "l"(count) : "memory");
            if (now >= want) break;
            if (globaltimer_ns() - t0 > kWaitLimitNs) {
                raise_flag(flag, TRI_FLAG_TIMEOUT);
                ok = false;
                break;
            }
        }
    }
    __syncthreads();
    return ok;
}

// Part c of n things dealt to the CTAs of the grid.
__device__ __forceinline__ int64_t part_begin(int64_t n, int64_t c) { return n * c / gridDim.x; }

// Sum of `x` over the CTA, in every thread.
__device__ __forceinline__ uint32_t cta_sum(uint32_t x) {
    __shared__ uint32_t w[kGridWarps];
    x = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = x;
    __syncthreads();
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < kGridWarps; ++i) t += w[i];
    return t;
}

// Number of set `x` in the threads before this one, and of the whole CTA.
__device__ __forceinline__ uint32_t cta_rank(bool x, uint32_t* total) {
    __shared__ uint32_t w[kGridWarps];
    const uint32_t bal = __ballot_sync(0xffffffffu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = __popc(bal);
    __syncthreads();
    uint32_t before = __popc(bal & ((1u << (threadIdx.x & 31)) - 1u)), t = 0;
#pragma unroll
    for (int i = 0; i < kGridWarps; ++i) {
        if (i < static_cast<int>(threadIdx.x >> 5)) before += w[i];
        t += w[i];
    }
    *total = t;
    return before;
}

// Sums of the CTAs' counts x, y, z before CTA `at` and of all CTAs, by one
// warp for the CTA.
struct PageSums {
    uint32_t x, y, z, all_x, all_y, all_z;
};
__device__ __forceinline__ PageSums sum_counts(const uint4* counts, uint32_t at) {
    __shared__ PageSums out;
    __syncthreads();
    if (threadIdx.x < 32) {
        PageSums s = {};
        for (uint32_t c = threadIdx.x; c < gridDim.x; c += 32) {
            const uint4 v = __ldcg(counts + c);
            s.all_x += v.x;
            s.all_y += v.y;
            s.all_z += v.z;
            if (c < at) {
                s.x += v.x;
                s.y += v.y;
                s.z += v.z;
            }
        }
        s.x = __reduce_add_sync(0xffffffffu, s.x);
        s.y = __reduce_add_sync(0xffffffffu, s.y);
        s.z = __reduce_add_sync(0xffffffffu, s.z);
        s.all_x = __reduce_add_sync(0xffffffffu, s.all_x);
        s.all_y = __reduce_add_sync(0xffffffffu, s.all_y);
        s.all_z = __reduce_add_sync(0xffffffffu, s.all_z);
        if (threadIdx.x == 0) out = s;
    }
    __syncthreads();
    return out;
}

// Copies of whole or part pages, of K and then of V, as one flat run of bytes
// (`page_bytes` a page) cut into windows.  kEngines warps a CTA move a window at
// a time each, through their own shared memory with bulk copies, lane x the
// part of the window that lies in its x-th page, so pages of any size keep 64 KB
// an SM in flight.  page(c) gives copy c's source and destination page and its
// bytes.  A compaction that moves 698 MB takes 126 us (6.2 TB/s for the rows);
// more in flight is slower (133 us with 192 KB), and so are loads and stores
// through registers (161 us with 64 KB).
struct PageCopy {
    int32_t from, to;
    int64_t bytes;
};

template <typename Page>
__device__ __forceinline__ void copy_pages(void* k, void* v, int64_t copies, int64_t page_bytes,
                                           uint32_t* flag, Page page) {
    extern __shared__ __align__(16) unsigned char smem[];
    CopyShared& sm = *reinterpret_cast<CopyShared*>(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp >= kEngines) return;
    unsigned char* window = sm.window[warp];
    uint64_t* landed = &sm.landed[warp];
    if (lane == 0) {
        mbar_init(landed, 1);
        fence_barrier_init();
    }
    __syncwarp();
    uint32_t phase = 0;
    const int64_t all = copies * page_bytes;
    const int64_t window_bytes = min(static_cast<int64_t>(kWindow), 31 * page_bytes);  // 32 pages at most
    const int64_t windows = (all + window_bytes - 1) / window_bytes;
    for (int64_t w = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x; w < windows * (v ? 2 : 1);
         w += static_cast<int64_t>(gridDim.x) * kEngines) {
        const bool second = w >= windows;
        char* pool = static_cast<char*>(second ? v : k);
        const int64_t b0 = (second ? w - windows : w) * window_bytes, b1 = min(b0 + window_bytes, all);
        const int64_t c = b0 / page_bytes + lane;
        const int64_t at = max(b0, c * page_bytes);
        // This lane's part: bytes [at, at + n) of the run, off within page c.
        int64_t off = 0, n = 0;
        PageCopy p = {0, 0, 0};
        if (at < b1) {
            p = page(c);
            off = at - c * page_bytes;
            n = max(min(min(b1 - at, page_bytes - off), p.bytes - off), static_cast<int64_t>(0));
        }
        const uint32_t bytes = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(n));
        bulk_wait_read<0>();  // this lane's last part has left the window
        __syncwarp();
        if (bytes == 0) continue;
        if (lane == 0) mbar_arrive_expect_tx(landed, bytes);
        __syncwarp();
        if (n > 0)
            bulk_load_hint(window + (at - b0), pool + p.from * page_bytes + off, static_cast<uint32_t>(n), landed,
                           policy_evict_first());
        const bool ok = mbar_wait(landed, phase, flag);
        if (!__all_sync(0xffffffffu, ok)) {
            // Copies may still be in flight: once more (bounded as well), so
            // that none lands in the window of a CTA that has ended.
            mbar_wait(landed, phase, flag);
            break;
        }
        phase ^= 1;
        if (n > 0) bulk_store(pool + p.to * page_bytes + off, window + (at - b0), static_cast<uint32_t>(n));
        bulk_commit();
    }
    bulk_wait_all();
}

template <typename Args>
static cudaError_t launch_grid(void (*fn)(Args), const Args& a, int ctas, cudaStream_t s) {
    void* args[1] = {const_cast<Args*>(&a)};
    const void* f = reinterpret_cast<const void*>(fn);
    constexpr size_t smem = sizeof(CopyShared);
    cudaError_t e = allow_smem(f, smem);
    if (e != cudaSuccess) return e;
    e = cudaLaunchCooperativeKernel(f, dim3(ctas), dim3(kGridThreads), args, smem, s);
    if (e == cudaSuccess) note_launch(s);
    return e;
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
    const uint32_t seq = static_cast<uint32_t>(u) / static_cast<uint32_t>(a.pc.n_units / a.pc.n_seq);
    const int64_t add = rows_added(a.n_add, seq, a.n_new, flag);
    if (n + add > cap) raise_flag(flag, TRI_FLAG_NVALID_RANGE);
    SlotWish w;
    const int64_t row0 = slot * a.pc.rows;
    w.kept = row0 < n + add;
    w.written = w.kept && (a.own || (add > 0 && row0 + a.pc.rows > n));
    const int64_t r = n - row0;
    w.rows = r < 0 ? 0 : r < a.pc.rows ? r : a.pc.rows;
    return w;
}

// Whether the slot asks for a page (0: no, 1: it has none, 2: its page is
// shared and it gets a copy).  Where every holder of a page writes it, the
// last of them keeps it.
__device__ __forceinline__ int slot_need(const FitArgs& a, int64_t id, int64_t* page) {
    const uint32_t per = static_cast<uint32_t>(a.pc.per_unit);
    const uint32_t u = static_cast<uint32_t>(id) / per, slot = static_cast<uint32_t>(id) - u * per;
    const int64_t pg = __ldcg(a.pc.table + id);
    const SlotWish w = slot_wish(a, u, slot, nullptr);
    *page = pg;
    if (!w.kept) return 0;
    if (pg < 0) return 1;
    const int32_t refs = __ldcg(a.refs + pg);
    if (!w.written || refs <= 1) return 0;
    return __ldcg(a.writers + pg) == static_cast<uint32_t>(refs) && __ldcg(a.last + pg) == id + 1 ? 0 : 2;
}

template <int kRow>  // bytes of a row
__global__ void __launch_bounds__(kGridThreads, 1) pages_fit_kernel(const FitArgs a) {
    const int tid = threadIdx.x;
    const int64_t c = blockIdx.x;
    const int64_t slots = a.pc.n_units * a.pc.per_unit;
    const uint32_t per = static_cast<uint32_t>(a.pc.per_unit);
    const int64_t s0 = part_begin(slots, c), s1 = part_begin(slots, c + 1);
    const int64_t p0 = part_begin(a.pc.n_pages, c), p1 = part_begin(a.pc.n_pages, c + 1);
    // ---- pages behind the last kept row are given back; pages that are
    // shared and will be written are marked.  (A count that falls below 2
    // meanwhile only leaves a mark that nobody needs.) ----
    for (int64_t id = s0 + tid; id < s1; id += kGridThreads) {
        const uint32_t u = static_cast<uint32_t>(id) / per, slot = static_cast<uint32_t>(id) - u * per;
        const int64_t pg = a.pc.table[id];
        const SlotWish w = slot_wish(a, u, slot, slot == 0 ? a.flag : nullptr);
        if (pg < 0 || pg >= a.pc.n_pages) {
            if (pg != -1) {
                raise_flag(a.flag, TRI_FLAG_INDEX_RANGE);
                a.pc.table[id] = -1;
            }
        } else if (!w.kept) {
            atomicSub(a.refs + pg, 1);
            a.pc.table[id] = -1;
        } else if (w.written && __ldcg(a.refs + pg) > 1) {
            atomicAdd(a.writers + pg, 1u);
            atomicMax(a.last + pg, static_cast<uint32_t>(id) + 1u);
        }
    }
    if (!grid_barrier(a.barrier, 1, a.flag)) return;
    // ---- requests, copies among them, free pages ----
    uint32_t need = 0, copy = 0, free = 0;
    for (int64_t id = s0 + tid; id < s1; id += kGridThreads) {
        int64_t pg;
        const int w = slot_need(a, id, &pg);
        need += w > 0;
        copy += w == 2;
    }
    for (int64_t p = p0 + tid; p < p1; p += kGridThreads) free += __ldcg(a.refs + p) == 0;
    need = cta_sum(need);
    copy = cta_sum(copy);
    free = cta_sum(free);
    if (tid == 0) a.counts[c] = make_uint4(need, copy, free, 0);
    if (!grid_barrier(a.barrier, 2, a.flag)) return;
    // ---- both lists in index order; nothing is served when there are fewer
    // free pages than requests ----
    const PageSums sum = sum_counts(a.counts, static_cast<uint32_t>(c));
    if (c == 0 && tid == 0) {
        if (sum.all_x > sum.all_z) raise_flag(a.flag, TRI_FLAG_NO_PAGES);
        if (a.n_free) *a.n_free = static_cast<int32_t>(sum.all_z) - static_cast<int32_t>(sum.all_x);
    }
    if (sum.all_x == 0 || sum.all_x > sum.all_z) return;
    if (need > 0) {
        uint32_t base = sum.x, copy_base = sum.y;
        for (int64_t b = s0; b < s1; b += kGridThreads) {
            const int64_t id = b + tid;
            int64_t pg = -1;
            const int w = id < s1 ? slot_need(a, id, &pg) : 0;
            uint32_t n, nc;
            const uint32_t r = base + cta_rank(w > 0, &n);
            const uint32_t rc = copy_base + cta_rank(w == 2, &nc);
            if (w > 0) {
                a.need_slot[r] = static_cast<int32_t>(id);
                a.need_old[r] = w == 2 ? static_cast<int32_t>(pg) : -1;
            }
            if (w == 2) {
                const uint32_t u = static_cast<uint32_t>(id) / per;
                const int64_t rows = slot_wish(a, u, id - static_cast<int64_t>(u) * per, nullptr).rows;
                a.copies[rc] = make_int4(static_cast<int32_t>(pg), static_cast<int32_t>(r),
                                         static_cast<int32_t>(rows), 0);
            }
            base += n;
            copy_base += nc;
        }
    }
    uint32_t base = sum.z;
    for (int64_t b = p0; b < p1 && base < sum.all_x; b += kGridThreads) {
        const int64_t p = b + tid;
        const bool is_free = p < p1 && __ldcg(a.refs + p) == 0;
        uint32_t n;
        const uint32_t r = base + cta_rank(is_free, &n);
        if (is_free && r < sum.all_x) a.free_page[r] = static_cast<int32_t>(p);
        base += n;
    }
    if (!grid_barrier(a.barrier, 3, a.flag)) return;
    // ---- table entries and counts of the requests, and the copies ----
    for (int64_t r = c * kGridThreads + tid; r < sum.all_x; r += static_cast<int64_t>(gridDim.x) * kGridThreads) {
        const int32_t pg = __ldcg(a.free_page + r), old = __ldcg(a.need_old + r);
        a.pc.table[__ldcg(a.need_slot + r)] = pg;
        a.refs[pg] = 1;
        if (old >= 0) atomicSub(a.refs + old, 1);
    }
    copy_pages(a.k, a.v, sum.all_y, a.pc.rows * kRow, a.flag, [&](int64_t x) {
        const int4 y = __ldcg(a.copies + x);
        return PageCopy{y.x, __ldcg(a.free_page + y.y), static_cast<int64_t>(y.z) * kRow};
    });
}

int page_ctas(int n_sm) { return n_sm; }

cudaError_t launch_pages_fit(tri_dtype dt, const FitArgs& a, int n_sm, cudaStream_t s) {
    return dt == TRI_BF16 ? launch_grid(pages_fit_kernel<kD * 2>, a, page_ctas(n_sm), s)
                          : launch_grid(pages_fit_kernel<kD * 4>, a, page_ctas(n_sm), s);
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
// Every fork reads its source as it was on entry, though a sequence may be
// read by some forks and replaced by another (beams that change places).  The
// columns of the tables are independent of one another: a CTA takes some
// columns of one (layer, head) for ALL forks, reads the sources' entries into
// shared memory and only then writes the destinations'.  Where a destination is
// the source of another fork, the row counts of a (layer, head), which all its
// jobs read, are replaced by the CTA that finishes the last of them; else by its
// first job, without fences and atomics (31 against 34 us for 32 of 64 sequences).
// Every CTA looks all forks over by itself, each fork against the others, and the
// columns of a job are 8192 / n_fork: right for a batch of sequences, while from a
// few hundred forks on both cost more than the tables.  3584 units of 16 entries
// take 9 us as 32 forks, 42 as 256, 105 as 512, 305 as 1024; with positions of 2048
// rows a unit and 28 (layer, head) pairs 1024 forks take 2.05 ms (floor 78 us).
constexpr int kForkCells = 8192;  // entries that a CTA holds
constexpr int kForkLoads = 4;

__global__ void __launch_bounds__(kThreads) pages_fork_kernel(const ForkArgs a, int table_bits,
                                                              int table_jobs, int pos_bits,
                                                              int pos_jobs) {
    extern __shared__ __align__(16) unsigned char smem[];
    int32_t* cell = reinterpret_cast<int32_t*>(smem);
    int32_t* src = cell + kForkCells;  // -1: empties, -2: skipped
    int32_t* dst = src + kMaxForks;
    int32_t* rows = dst + kMaxForks;   // rows of the source unit
    __shared__ bool last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool crossed = false;  // a destination is the source of another fork
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
    for (int f = tid; f < F; f += kThreads) {
        if (src[f] == -2 || src[f] == dst[f]) continue;
        for (int g = 0; g < F && !crossed; ++g) crossed = g != f && src[g] == dst[f];
    }
    crossed = __syncthreads_or(crossed);
    if (a.p_cur && blockIdx.x == 0) {
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
    const int64_t cap = a.pc.per_unit * a.pc.rows;
    const int64_t jobs = per_seq * (table_jobs + pos_jobs);
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const bool pos = job >= per_seq * table_jobs;
        const int64_t j = pos ? job - per_seq * table_jobs : job;
        const int64_t lh = j % per_seq;
        const int bits = pos ? pos_bits : table_bits;  // 2^bits columns
        const int col0 = static_cast<int>(j / per_seq) << bits;
        const int64_t width = pos ? a.cap : a.pc.per_unit;
        const int cols = static_cast<int>(min(int64_t(1) << bits, width - col0));
        __syncthreads();
        for (int f = tid; f < F; f += kThreads)
            rows[f] = src[f] < 0 ? 0 : clamp_nvalid(a.n_valid, src[f] * per_seq + lh, cap, a.flag);
        // A warp takes a fork at a time, its lanes neighbouring columns.  The
        // sources go straight to shared memory, all of them in flight, and
        // without waiting for their counts.
        int32_t* table = pos ? a.pos : a.pc.table;
        for (int f = warp; f < F; f += kWarps) {
            if (src[f] < 0 || (pos && src[f] == dst[f])) continue;
            const int32_t* from = table + (src[f] * per_seq + lh) * width + col0;
            int32_t* to = cell + (f << bits);
            for (int c = lane; c < cols; c += 32)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to + c)), "l"(from + c)
                             : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        for (int f = warp; f < F; f += kWarps) {
            if (src[f] == -2 || (pos && src[f] == dst[f])) continue;
            int32_t* to = table + (dst[f] * per_seq + lh) * width + col0;
            const int32_t* from = cell + (f << bits);
            if (pos) {
                const int n = min(rows[f] - col0, cols);
                for (int c = lane; c < n; c += 32) to[c] = from[c];
                continue;
            }
            for (int c0 = lane; c0 < cols; c0 += 32 * kForkLoads) {
                int32_t old[kForkLoads];
#pragma unroll
                for (int q = 0; q < kForkLoads; ++q)
                    if (c0 + 32 * q < cols) old[q] = to[c0 + 32 * q];
#pragma unroll
                for (int q = 0; q < kForkLoads; ++q) {
                    const int c = c0 + 32 * q;
                    if (c >= cols) continue;
                    // A page that holds rows of the source, or none.
                    const bool held = static_cast<int64_t>(col0 + c) * a.pc.rows < rows[f];
                    int32_t now = held ? from[c] : -1;
                    if (now < 0 || now >= a.pc.n_pages) {
                        if (held) raise_flag(a.flag, TRI_FLAG_INDEX_RANGE);
                        now = -1;
                    }
                    if (now == old[q]) continue;
                    if (now >= 0) atomicAdd(a.refs + now, 1);
                    if (old[q] >= 0 && old[q] < a.pc.n_pages)
                        atomicSub(a.refs + old[q], 1);
                    else if (old[q] != -1)
                        raise_flag(a.flag, TRI_FLAG_INDEX_RANGE);
                    to[c] = now;
                }
            }
        }
        // ---- the counts: by the first job, or when every job of the (layer,
        // head) has read them ----
        if (crossed) {
            __syncthreads();
            if (tid == 0) {
                __threadfence();
                last = atomicAdd(a.done + lh, 1u) == static_cast<uint32_t>(table_jobs + pos_jobs) - 1;
            }
            __syncthreads();
            if (!last) continue;
        } else if (pos || col0 != 0) {
            continue;
        }
        __syncthreads();
        for (int f = tid; f < F; f += kThreads)
            cell[f] = src[f] >= 0 ? clamp_nvalid(a.n_valid, src[f] * per_seq + lh, cap, nullptr) : 0;
        __syncthreads();
        // (A sequence that stays itself is written only where its count is
        // clamped, to what every job reads of it before and after; always
        // written, 32 forks took 1 us more.)
        for (int f = tid; f < F; f += kThreads) {
            if (src[f] == -2) continue;
            int32_t* n = a.n_valid + dst[f] * per_seq + lh;
            if (src[f] != dst[f] || *n != cell[f]) *n = cell[f];
        }
    }
}

cudaError_t launch_pages_fork(const ForkArgs& a, int n_sm, cudaStream_t s) {
    const int64_t per_seq = a.pc.n_units / a.pc.n_seq;
    // Columns of a job, a power of two: as few as leave an SM at most 4 jobs
    // (5 CTAs fit it), 32 at least, and no more than fit the cells.
    const int64_t pos_width = a.pos ? a.cap : 0;
    auto bits = [&](int64_t width) {
        int b = 5;
        while ((int64_t(1) << b) < width && ((a.pc.per_unit + pos_width) >> b) * per_seq > 4 * n_sm) ++b;
        while (b > 0 && (a.n_fork << b) > kForkCells) --b;
        return b;
    };
    const int table_bits = bits(a.pc.per_unit), pos_bits = bits(pos_width);
    const int table_jobs = static_cast<int>((a.pc.per_unit + (int64_t(1) << table_bits) - 1) >> table_bits);
    const int pos_jobs = static_cast<int>((pos_width + (int64_t(1) << pos_bits) - 1) >> pos_bits);
    constexpr size_t smem = (kForkCells + 3 * kMaxForks) * sizeof(int32_t);
    static_assert(smem <= 48 * 1024, "more than the default limit");
    pages_fork_kernel<<<grid_for(per_seq * (table_jobs + pos_jobs), 1, 5LL * n_sm), kThreads, smem, s>>>(
        a, table_bits, table_jobs, pos_bits, pos_jobs);
    note_launch(s);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------
// With L live pages, the live pages at L and behind go, in order, to the free
// pages below L, in order (there are as many of one as of the other).
template <int kRow>  // bytes of a row
__global__ void __launch_bounds__(kGridThreads, 1) pages_compact_kernel(const CompactPagesArgs a) {
    const int tid = threadIdx.x;
    const int64_t c = blockIdx.x;
    const int64_t p0 = part_begin(a.pc.n_pages, c), p1 = part_begin(a.pc.n_pages, c + 1);
    uint32_t live = 0;
    for (int64_t p = p0 + tid; p < p1; p += kGridThreads) live += a.refs[p] != 0;
    live = cta_sum(live);
    if (tid == 0) a.counts[c] = make_uint4(live, 0, 0, 0);
    if (!grid_barrier(a.barrier, 1, a.flag)) return;
    const PageSums sum = sum_counts(a.counts, static_cast<uint32_t>(c));
    const int64_t L = sum.all_x;
    // Live pages below L: those of whole parts, then of the part that L lies in.
    int64_t cl = L * gridDim.x / a.pc.n_pages;
    while (cl + 1 < gridDim.x && part_begin(a.pc.n_pages, cl + 1) <= L) ++cl;
    while (cl > 0 && part_begin(a.pc.n_pages, cl) > L) --cl;
    uint32_t some = 0;
    for (int64_t p = part_begin(a.pc.n_pages, cl) + tid; p < L; p += kGridThreads) some += a.refs[p] != 0;
    const uint32_t below = sum_counts(a.counts, static_cast<uint32_t>(cl)).x + cta_sum(some);
    const int64_t moves = L - below;
    if (c == 0 && tid == 0 && a.n_live) *a.n_live = static_cast<int32_t>(L);
    uint32_t base = sum.x;
    for (int64_t b = p0; b < p1 && moves > 0; b += kGridThreads) {
        const int64_t p = b + tid;
        const bool is_live = p < p1 && a.refs[p] != 0;
        uint32_t n;
        const uint32_t r = base + cta_rank(is_live, &n);  // live pages before p
        if (p < p1) {
            if (p < L && !is_live) a.to[p - r] = static_cast<int32_t>(p);
            if (p >= L && is_live) {
                a.from[r - below] = static_cast<int32_t>(p);
                a.rank[p] = static_cast<int32_t>(r - below);
            }
        }
        base += n;
    }
    if (moves > 0 && !grid_barrier(a.barrier, 2, a.flag)) return;
    // ---- the table entries that name the moving pages, their counts and rows
    // (no page moves: the entries are only looked at) ----
    const int64_t slots = a.pc.n_units * a.pc.per_unit;
    for (int64_t id = c * kGridThreads + tid; id < slots; id += static_cast<int64_t>(gridDim.x) * kGridThreads) {
        const int64_t pg = a.pc.table[id];
        if (pg < -1 || pg >= a.pc.n_pages) {
            raise_flag(a.flag, TRI_FLAG_INDEX_RANGE);
            continue;
        }
        if (pg < L) continue;
        // An entry whose page's count is 0 names no listed page: left, flagged.
        const int64_t r = __ldcg(a.rank + pg);
        if (r >= 0 && r < moves && __ldcg(a.from + r) == pg)
            a.pc.table[id] = __ldcg(a.to + r);
        else
            raise_flag(a.flag, TRI_FLAG_INDEX_RANGE);
    }
    for (int64_t m = c * kGridThreads + tid; m < moves; m += static_cast<int64_t>(gridDim.x) * kGridThreads) {
        const int32_t from = __ldcg(a.from + m), to = __ldcg(a.to + m);
        a.refs[to] = a.refs[from];
        a.refs[from] = 0;
    }
    const int64_t page_bytes = a.pc.rows * kRow;
    copy_pages(a.k, a.v, moves, page_bytes, a.flag, [&](int64_t x) {
        return PageCopy{__ldcg(a.from + x), __ldcg(a.to + x), page_bytes};
    });
}

cudaError_t launch_pages_compact(tri_dtype dt, const CompactPagesArgs& a, int n_sm,
                                 cudaStream_t s) {
    return dt == TRI_BF16 ? launch_grid(pages_compact_kernel<kD * 2>, a, page_ctas(n_sm), s)
                          : launch_grid(pages_compact_kernel<kD * 4>, a, page_ctas(n_sm), s);
}

}  // namespace tri
