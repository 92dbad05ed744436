// decode_paged_tc.cu -- decode attention over a bf16 paged cache on the
// tensor cores (the formulas stand in decode_paged.cu).
//
// A tile is 128 keys of one unit; the tiles of a CTA are one stream over its
// units.  One warp brings a tile's K and V rows in as TMA boxes, each within one
// page, into a ring of kTcStages tiles (192 KB in flight), one warp issues the
// products, and four warps (one thread a key, then one thread a dim) do the rest:
//   S [128 keys x 16]  = K [128 x 128] Q^T             tcgen05, K rows as A;
//                        the G <= 8 heads are columns, the rest zeros;
//   weights            p = 2^(scale log2(e) s - m): the tile's maxima by a
//                        transposing butterfly and four words a warp in
//                        shared memory, running maxima m kept by every thread;
//   O [128 dims x 32]  = V^T [128 x 128] P              tcgen05, V rows as A
//                        (M-major), P [keys x 32] as B (N-major).
// P is split into three bf16 terms, p = p1 + p2 + p3 to 2^-26, in columns
// 0-7, 8-15 and 16-23: M = 128 wants 16 columns at least, so the 32 cost a
// few cycles more and the weights keep float32's precision.  Q and V are bf16
// already, products are exact and sums are float32.  O of each tile is added
// to float32 accumulators in registers with the rescale of the running
// maximum, so nothing in tensor memory is rescaled.
//
// S runs up to two tiles ahead (one over a change of unit), and O of a tile is
// read after the next tile's weights, so no warp waits for a product that it
// has just asked for; a unit's Q, row count and page entries are read while
// the unit before it is worked on.
//
// Bound: K and V are read once (512 bytes a key), so HBM: 64 KB a tile arrive in
// 1.5 us at an SM's share of it.  4 sequences x 8 heads of 98 to 131 K rows (1.73
// GB) take 258 us, 6.7 TB/s; 7168 units of 2176 rows 1.17 ms; 64 units of about
// 2300 rows (76 MB) 25 us, of which 13 are ramp, join and launch.  What is read
// is whole boxes (the largest power of two of rows, 128 at most, that divides a
// page), so a unit's last box brings rows behind its end too: 1792 units of 130
// rows in pages of 128 read 237 MB for 119 MB of rows.  That is the smaller part
// of what short units lose: they take 56 us, and 50 in pages of 8 rows (125 MB);
// 20 rows a unit 42 and 38.  The rest is what a tile costs that is its unit's
// only one (weights, values and results one after the other).  With the products
// issued by one of the four warps a tile took 1.8 us, and 1792 units of 130 rows
// 96 us.
#include "paged_core.cuh"
#include "tri_launch.h"

namespace tri {

constexpr int kTcStages = 3;
constexpr int kTcMath = 128;               // threads of the math warps
constexpr int kTcThreads = kTcMath + 64;   // and a loading and an issuing warp
constexpr int kTcMat = kTcTile * kD * 2;   // K or V of a tile: [8-row group][64-dim half][8 x 128 bytes]
constexpr int kTcGroup = 2048;             // bytes of an 8-row group, and of
constexpr int kTcHalf = 1024;              //   one half of it
constexpr int kTcPRow = 64;                // bytes of a key's weights: 32 bf16

struct __align__(1024) TcShared {
    unsigned char k[kTcStages][kTcMat];
    unsigned char v[kTcStages][kTcMat];
    unsigned char q[2][2][16 * 128];    // [unit in turn][64-dim half][16 rows], swizzled
    unsigned char p[kTcTile * kTcPRow]; // [key][32 columns], swizzled
    float wmax[2][4][8];                // [tile in turn][warp][head]
    float wsum[4][8];
    uint64_t k_full[kTcStages], k_empty[kTcStages], v_full[kTcStages], v_empty[kTcStages];
    uint64_t s_full[2], o_full;
    uint64_t p_full;                    // Q of the first tile; then P of a tile (and Q of the next)
    uint32_t q_next;                    // bit 0: Q of the next tile; bit 1: the one behind it has it too
    uint32_t tmem;
    int abort[2];                       // [tile in turn]: a wait gave up before the tile's barrier
    int failed;
};

// ---- tcgen05 ----
__device__ __forceinline__ void tc_alloc(uint32_t* smem, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tc_dealloc(uint32_t tmem, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// 8 columns of this thread's lane.
__device__ __forceinline__ void tc_load8(uint32_t addr, float (&x)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7])
                 : "r"(addr));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tc_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptor: leading and stride byte offsets, version 1,
// swizzle 128 bytes (2) or 64 bytes (4).
__device__ __forceinline__ uint64_t tc_desc(const void* p, uint32_t lead, uint32_t stride,
                                            uint64_t swizzle) {
    return static_cast<uint64_t>((smem_u32(p) & 0x3ffff) >> 4) |
           (static_cast<uint64_t>(lead >> 4) << 16) | (static_cast<uint64_t>(stride >> 4) << 32) |
           (1ull << 46) | (swizzle << 61);
}

// float32 result, bf16 operands, M = 128, N columns.
constexpr uint32_t tc_idesc(uint32_t n, bool a_m_major, bool b_n_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_m_major ? 1u << 15 : 0u) |
           (b_n_major ? 1u << 16 : 0u) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// S = K Q^T: both operands K-major (dims contiguous) in 128-byte rows, 8-row
// groups 2048 (K) and 1024 (Q) bytes apart; 16 dims are 32 bytes.  (A
// descriptor's address counts 16-byte units in its lowest bits.)
__device__ __forceinline__ void issue_scores(uint64_t k, uint64_t q, uint32_t tmem) {
    constexpr uint32_t idesc = tc_idesc(16, false, false);
#pragma unroll
    for (int x = 0; x < kD / 16; ++x) {
        const int half = x >> 2, off = (x & 3) * 32;
        tc_mma(tmem, k + ((half * kTcHalf + off) >> 4), q + ((half * 2048 + off) >> 4), idesc, x > 0);
    }
}

// O = V^T P: V (A, M contiguous) with its 64-dim halves 1024 and its 8-key
// groups 2048 bytes apart; P (B, N contiguous) 64-byte keys, 8-key groups 512
// bytes apart; 16 keys a step.
__device__ __forceinline__ void issue_values(uint64_t v, uint64_t p, uint32_t tmem) {
    constexpr uint32_t idesc = tc_idesc(32, true, true);
#pragma unroll
    for (int x = 0; x < kTcTile / 16; ++x)
        tc_mma(tmem, v + ((x * 2 * kTcGroup) >> 4), p + ((x * 16 * kTcPRow) >> 4), idesc, x > 0);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&x);
}

// A box of the 4-D view {64 dims, 8 rows, 2 halves, groups} of a pool: whole
// groups, each 2048 contiguous bytes here and there.
__device__ __forceinline__ void tma_load_groups(void* dst, const CUtensorMap* map, uint64_t* bar,
                                                int32_t group, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %3, %3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(group), "l"(policy)
        : "memory");
}

// Maxima or sums of 8 values over a warp by a transposing butterfly: lane x
// gets value x >> 2.
template <typename Op>
__device__ __forceinline__ float reduce8(float (&x)[8], Op op) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        const int o = 16 >> q, c = 4 >> q;
        const bool up = lane & o;
#pragma unroll
        for (int h = 0; h < c; ++h) {
            const float keep = up ? x[h + c] : x[h];
            const float give = up ? x[h] : x[h + c];
            x[h] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
    }
    x[0] = op(x[0], __shfl_xor_sync(0xffffffffu, x[0], 2));
    return op(x[0], __shfl_xor_sync(0xffffffffu, x[0], 1));
}

using TcUnit = UnitCursor<kTcTile>;

template <int G>
__global__ void __launch_bounds__(kTcThreads, 1)
decode_paged_tc_kernel(const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const int box_rows,
                       const PageDivide divide, const DecodePagedArgs a) {
    extern __shared__ unsigned char smem_raw[];
    TcShared& sm = *reinterpret_cast<TcShared*>(
        smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == kTcMath) {
        for (int i = 0; i < kTcStages; ++i) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_empty[i], 1);
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.v_empty[i], 1);
        }
        mbar_init(&sm.s_full[0], 1);
        mbar_init(&sm.s_full[1], 1);
        mbar_init(&sm.o_full, 1);
        mbar_init(&sm.p_full, kTcMath / 32);
        sm.abort[0] = sm.abort[1] = sm.failed = 0;
        fence_barrier_init();
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    const SplitPlan p = plan_split<kTcThreads>(a, kTcTile, 1);  // (synchronises the CTA)
    // The loading warp goes on while the others get their tensor memory.
    uint32_t tmem = 0;
    if (warp != kTcMath / 32) {
        if (warp == 0) tc_alloc(&sm.tmem, 64);
        // Columns 24 .. 31 of the weights stay zeros.
        if (tid < kTcMath)
            *reinterpret_cast<uint4*>(sm.p + tid * kTcPRow + ((3 ^ ((tid >> 1) & 3)) * 16)) =
                make_uint4(0, 0, 0, 0);
        tc_fence_before();
        named_sync(2, kTcMath + 32);
        tc_fence_after();
        tmem = sm.tmem;
    }
    const uint32_t s_cols = tmem, o_cols = tmem + 32;
    const uint32_t n_it = p.end - p.begin;  // tiles of this CTA
    auto aborted = [&] {
        return (*reinterpret_cast<volatile int*>(&sm.abort[0]) | *reinterpret_cast<volatile int*>(&sm.abort[1])) != 0;
    };

    if (warp == kTcMath / 32) {
        // ---- the loading warp: lane b brings box b ----
        const int n_boxes = kTcTile / box_rows;
        const uint64_t pol = policy_evict_first();
        TcUnit cur = {};
        // Page entry of this lane's box of tile t (read a tile ahead).
        auto look_up = [&](const TcUnit& w, uint32_t t) -> int32_t {
            return lane < n_boxes ? w.page(divide, (t - w.tile0) * kTcTile + lane * box_rows) : -1;
        };
        int32_t page = -1;
        if (n_it) {
            cur.first(a, p.unit, p.tile0, p.rows, p.end);
            page = look_up(cur, p.begin);
        }
        uint32_t it = 0;
        for (; it < n_it; ++it) {
            const uint32_t t = p.begin + it;
            const int stage = it % kTcStages;
            const uint32_t parity = ((it / kTcStages) & 1) ^ 1;
            const uint32_t j = (t - cur.tile0) * kTcTile + lane * box_rows;
            const bool wanted = lane < n_boxes && j < cur.n;
            if (t + 1 == cur.t1 && it + 1 < n_it) cur = cur.next(a, p.end);
            const int32_t page_next = it + 1 < n_it ? look_up(cur, t + 1) : -1;
            const bool load = page >= 0 && page < a.pc.n_pages;
            if (wanted && !load) {
                wait_for_clear();
                raise_flag(a.flag, TRI_FLAG_INDEX_RANGE);
            }
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, load)) * box_rows * 256;
            const int off = lane * box_rows * 256;
            const uint32_t in_page = j - divide.slot(j) * divide.rows;
            const int32_t group = static_cast<int32_t>((static_cast<int64_t>(page) * divide.rows + in_page) >> 3);
            bool ok = mbar_wait(&sm.k_empty[stage], parity, a.flag);
            ok = __all_sync(0xffffffffu, ok && !aborted());
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&sm.k_full[stage], bytes);
            __syncwarp();
            if (load) tma_load_groups(sm.k[stage] + off, &kmap, &sm.k_full[stage], group, pol);
            ok = mbar_wait(&sm.v_empty[stage], parity, a.flag);
            ok = __all_sync(0xffffffffu, ok);
            if (lane == 0) mbar_arrive_expect_tx(&sm.v_full[stage], ok ? bytes : 0);
            __syncwarp();
            if (ok && load) tma_load_groups(sm.v[stage] + off, &vmap, &sm.v_full[stage], group, pol);
            page = page_next;
        }
        // Nothing of this warp is in flight when the CTA ends.
        for (uint32_t x = it < kTcStages ? 0 : it - kTcStages; x < it; ++x) {
            mbar_wait(&sm.k_full[x % kTcStages], (x / kTcStages) & 1, a.flag);
            mbar_wait(&sm.v_full[x % kTcStages], (x / kTcStages) & 1, a.flag);
        }
    } else if (warp == kTcMath / 32 + 1) {
        // ---- the issuing warp: one thread ----
        if (lane == 0 && n_it) {
            const uint64_t kd = tc_desc(sm.k, 16, kTcGroup, 2), qd = tc_desc(sm.q, 16, 1024, 2);
            const uint64_t vd = tc_desc(sm.v, kTcHalf, kTcGroup, 2), pd = tc_desc(sm.p, 16, 512, 4);
            uint32_t asked = 0;  // scores issued: of tiles 0 .. asked - 1
            uint32_t given = 0;  // values issued
            auto scores = [&](uint32_t qb) {
                const uint32_t x = asked++, stage = x % kTcStages;
                if (!mbar_wait(&sm.k_full[stage], (x / kTcStages) & 1, a.flag)) return false;
                tc_fence_after();
                issue_scores(kd + stage * (kTcMat >> 4), qd + qb * (4096 >> 4), s_cols + (x & 1) * 16);
                tc_commit(&sm.s_full[x & 1]);
                tc_commit(&sm.k_empty[stage]);
                return true;
            };
            bool ok = mbar_wait(&sm.p_full, 0, a.flag);
            uint32_t w = *reinterpret_cast<volatile uint32_t*>(&sm.q_next);
            ok = ok && scores(w & 1);
            if (ok && (w & 2)) ok = scores(w & 1);
            for (uint32_t it = 0; ok && it < n_it; ++it) {
                const int stage = it % kTcStages;
                ok = mbar_wait(&sm.p_full, (it + 1) & 1, a.flag) &&
                     mbar_wait(&sm.v_full[stage], (it / kTcStages) & 1, a.flag);
                if (!ok) break;
                w = *reinterpret_cast<volatile uint32_t*>(&sm.q_next);
                tc_fence_after();
                issue_values(vd + stage * (kTcMat >> 4), pd, o_cols);
                tc_commit(&sm.o_full);
                tc_commit(&sm.v_empty[stage]);
                ++given;
                if (asked == it + 1 && asked < n_it) ok = scores(w & 1);
                if (ok && asked == it + 2 && (w & 2)) ok = scores(w & 1);
            }
            // The products are done, and their last arrivals are in, before the
            // CTA gives its tensor memory back and ends (also when a wait gave up).
            for (uint32_t x = asked < kTcStages ? 0 : asked - kTcStages; x < asked; ++x)
                mbar_wait(&sm.k_empty[x % kTcStages], (x / kTcStages) & 1, a.flag);
            for (uint32_t x = given < kTcStages ? 0 : given - kTcStages; x < given; ++x)
                mbar_wait(&sm.v_empty[x % kTcStages], (x / kTcStages) & 1, a.flag);
        }
        __syncwarp();
    } else {
        const uint32_t lanes = static_cast<uint32_t>(warp) * 32 << 16;  // this warp's TMEM lanes
        SplitUnit split0 = {}, split1 = {};
        int n_split = 0;
        uint32_t qb = 0;
        bool ok = true;
        float m[G], l[G], acc[G], al[G];
        // Q of unit i, rows >= G zero: chunks tid and tid + 128 of its 16 x 16;
        // 16-byte chunk c of a 128-byte row r lies at c ^ (r & 7).
        uint4 qx[2];
        auto read_q = [&](uint32_t i) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int e = tid + x * kTcMath, r = e >> 4, c = e & 15;
                qx[x] = make_uint4(0, 0, 0, 0);
                if (r < G)
                    qx[x] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                                 (static_cast<int64_t>(i) * G + r) * kD) +
                                  c);
            }
        };
        auto store_q = [&](uint32_t b) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int e = tid + x * kTcMath, r = e >> 4, c = e & 15;
                *reinterpret_cast<uint4*>(sm.q[b][c >> 3] + r * 128 + ((c & 7) ^ (r & 7)) * 16) = qx[x];
            }
        };
        // What this warp wrote (and read of tensor memory) is handed to the
        // issuing warp.
        auto hand_over = [&] {
            fence_proxy_async();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full);
        };
        // O of the tile x that was last handed over, into the accumulators.
        auto take_values = [&](uint32_t x) {
            ok = mbar_wait(&sm.o_full, x & 1, a.flag) && ok;
            tc_fence_after();
            float o1[8], o2[8], o3[8];
            tc_load8(o_cols + lanes, o1);
            tc_load8(o_cols + 8 + lanes, o2);
            tc_load8(o_cols + 16 + lanes, o3);
            tc_load_wait();
#pragma unroll
            for (int h = 0; h < G; ++h) {
                // An infinite value times a term of zero is no part of the sum.
                const float rest = isfinite(o1[h]) ? o2[h] + o3[h] : 0.f;
                acc[h] = fmaf(acc[h], al[h], o1[h] + rest);
            }
        };
        TcUnit cur = {};
        int32_t page = -1;  // entry of this thread's key (read a tile ahead)
        if (n_it) {
            read_q(p.unit);
            cur.first(a, p.unit, p.tile0, p.rows, p.end);
            page = cur.page(divide, (p.begin - cur.tile0) * kTcTile + tid);
            store_q(0);
            if (tid == 0) sm.q_next = p.begin + 1 < cur.t1 ? 2 : 0;
            hand_over();
        }
        bool begins = true;  // the tile is its unit's first in the range
        for (uint32_t it = 0; it < n_it; ++it) {
            const uint32_t t = p.begin + it;
            const int stage = it % kTcStages;
            const bool ends = t + 1 == cur.t1, more = it + 1 < n_it;
            const bool valid = page >= 0 && page < a.pc.n_pages;
            TcUnit nxt = cur;
            if (ends && more) {
                nxt = cur.next(a, p.end);
                read_q(nxt.i);
            }
            page = more ? nxt.page(divide, (t + 1 - nxt.tile0) * kTcTile + tid) : -1;
            ok = mbar_wait(&sm.s_full[it & 1], (it >> 1) & 1, a.flag) && ok;
            tc_fence_after();
            float s[8];
            tc_load8(s_cols + (it & 1) * 16 + lanes, s);
            tc_load_wait();
            // ---- maxima of the warp's 32 keys ----
            float x[8];
#pragma unroll
            for (int h = 0; h < 8; ++h) x[h] = h < G && valid ? s[h] * a.scale_log2 : -INFINITY;
            const float wm = reduce8(x, [](float u, float v) { return fmaxf(u, v); });
            if ((lane & 3) == 0) sm.wmax[it & 1][warp][lane >> 2] = wm;
            if (!ok) *reinterpret_cast<volatile int*>(&sm.abort[it & 1]) = 1;
            named_sync(1, kTcMath);
            if (*reinterpret_cast<volatile int*>(&sm.abort[it & 1])) {
                ok = false;
                break;
            }
            if (begins) {
#pragma unroll
                for (int h = 0; h < G; ++h) {
                    m[h] = -INFINITY;
                    l[h] = acc[h] = 0.f;
                }
            }
            float al_now[G];
#pragma unroll
            for (int h = 0; h < G; ++h) {
                const float mt = fmaxf(fmaxf(sm.wmax[it & 1][0][h], sm.wmax[it & 1][1][h]),
                                       fmaxf(sm.wmax[it & 1][2][h], sm.wmax[it & 1][3][h]));
                const float m_new = fmaxf(m[h], mt);
                const float base = m_new == -INFINITY ? 0.f : m_new;
                al_now[h] = exp2f(m[h] - base);
                // (one rounding of the small difference, not of the large product)
                const float w = valid ? exp2f(fmaf(s[h], a.scale_log2, -base)) : 0.f;
                l[h] = fmaf(l[h], al_now[h], w);
                m[h] = m_new;
                s[h] = w;
            }
            // The tile before this one; from here on P may be written again.
            if (!begins) take_values(it - 1);
#pragma unroll
            for (int h = 0; h < G; ++h) al[h] = al_now[h];
            // ---- P: three bf16 terms; chunk c of key t's 64 bytes lies at c ^ ((t >> 1) & 3) ----
            unsigned char* prow = sm.p + tid * kTcPRow;
            const int sw = (tid >> 1) & 3;
#pragma unroll
            for (int term = 0; term < 3; ++term) {
                uint32_t w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float lo = 2 * c < G ? s[2 * c] : 0.f;
                    const float hi = 2 * c + 1 < G ? s[2 * c + 1] : 0.f;
                    w[c] = pack_bf16(lo, hi);
                    if (2 * c < G) s[2 * c] = lo - bf16_lo(w[c]);
                    if (2 * c + 1 < G) s[2 * c + 1] = hi - bf16_hi(w[c]);
                }
                *reinterpret_cast<uint4*>(prow + ((term ^ sw) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            // Rows that carry no weight hold anything: zeros, since 0 * inf is
            // not 0.  (The chunks in an order that spreads the lanes' banks.)
            if (!__all_sync(0xffffffffu, valid)) {
                ok = mbar_wait(&sm.v_full[stage], (it / kTcStages) & 1, a.flag) && ok;
                if (!valid) {
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        *reinterpret_cast<uint4*>(sm.v[stage] + (tid >> 3) * kTcGroup + (c >> 3) * kTcHalf +
                                                  (tid & 7) * 128 + ((c + tid) & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
            }
            if (ends && more) {
                qb ^= 1;
                store_q(qb);
            }
            if (tid == 0) sm.q_next = qb | (t + 2 < nxt.t1 ? 2u : 0u);
            hand_over();
            begins = ends;
            if (!ends) continue;
            // ---- the unit's sums over the keys, and its results ----
            take_values(it);
#pragma unroll
            for (int h = 0; h < 8; ++h) x[h] = h < G ? l[h] : 0.f;
            const float ws = reduce8(x, [](float u, float v) { return u + v; });
            if ((lane & 3) == 0) sm.wsum[warp][lane >> 2] = ws;
            named_sync(1, kTcMath);
            const bool whole = cur.tile0 >= p.begin && cur.t1 == cur.tile0 + cur.n_tiles;
            const uint32_t slot = part_slot(p, blockIdx.x, cur.tile0);
            // Lane h finishes head h's sum, maximum and reciprocal.
            const int hl = lane & 7;
            const float den = (sm.wsum[0][hl] + sm.wsum[1][hl]) + (sm.wsum[2][hl] + sm.wsum[3][hl]);
            const float inv = !whole ? 1.f : den == 0.f ? 0.f : 1.f / den;
            float ml = 0.f;
#pragma unroll
            for (int h = 0; h < G; ++h) ml = hl == h ? m[h] : ml;
            float* to = whole ? a.out + static_cast<int64_t>(cur.i) * G * kD
                              : a.part + static_cast<int64_t>(slot) * G * kD;
#pragma unroll
            for (int h = 0; h < G; ++h) to[h * kD + tid] = acc[h] * __shfl_sync(0xffffffffu, inv, h);
            if (tid < G) {
                if (!whole)
                    a.part_ml[slot * G + tid] = make_float2(ml, den);
                else if (a.lse)
                    a.lse[static_cast<int64_t>(cur.i) * G + tid] = lse_of(ml, den);
            }
            if (!whole) {
                split1 = split_unit(p, cur.i, cur.tile0, cur.n_tiles);
                if (n_split++ == 0) split0 = split1;
            }
            cur = nxt;
        }
        if (!ok) *reinterpret_cast<volatile int*>(&sm.failed) = 1;
        named_sync(1, kTcMath);
        if (!*reinterpret_cast<volatile int*>(&sm.failed))
            join_split_units<kTcMath / 32, 1, 32>(a, G, n_split, split0, split1);
    }
    wait_for_clear();
    write_empty_units(a, G);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tc_dealloc(tmem, 64);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int decode_paged_box_rows(int64_t page_rows) {
    int g = kTcTile;
    while (g >= 8 && page_rows % g != 0) g >>= 1;
    return g >= 8 ? g : 0;
}

template <int G>
static cudaError_t launch_tc(const CUtensorMap& kmap, const CUtensorMap& vmap, int box_rows,
                             const DecodePagedArgs& a, int n_sm, cudaStream_t s) {
    constexpr size_t smem = sizeof(TcShared) + 1024;
    static_assert(smem <= 227 * 1024, "tile ring too large");
    auto* fn = decode_paged_tc_kernel<G>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), smem);
    if (e != cudaSuccess) return e;
    e = launch_decode_paged_clear(a, s);
    if (e != cudaSuccess) return e;
    e = launch_early(fn, decode_paged_ctas(n_sm), kTcThreads, smem, s, kmap, vmap, box_rows,
                     page_divide(a.pc.rows), a);
    if (e == cudaSuccess) note_launch(s);
    return e;
}

cudaError_t launch_decode_paged_tc(int G, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                   int box_rows, const DecodePagedArgs& a, int n_sm,
                                   cudaStream_t s) {
    switch (G) {
#define TRI_DCASE(g) \
    case g: return launch_tc<g>(kmap, vmap, box_rows, a, n_sm, s);
        TRI_DCASE(1) TRI_DCASE(2) TRI_DCASE(3) TRI_DCASE(4)
        TRI_DCASE(5) TRI_DCASE(6) TRI_DCASE(7) TRI_DCASE(8)
#undef TRI_DCASE
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace tri
