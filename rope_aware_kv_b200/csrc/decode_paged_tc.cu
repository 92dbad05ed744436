// decode_paged_tc.cu -- decode attention over a bf16 paged cache on the
// tensor cores (the formulas stand in decode_paged.cu).
//
// A tile is 128 keys of one unit.  One warp brings its K and V rows in as TMA
// boxes, each within one page, into a ring of kStages tiles (192 KB in
// flight); four warps (one thread a key, then one thread a dim) work on it:
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
// maximum, so nothing in tensor memory is rescaled.  S of the next tile is
// issued together with O of this one.
//
// Bound: K and V rows are read once (512 bytes a key), so HBM; the math of a
// tile takes about half of the time that its 64 KB take to arrive.
#include "paged_core.cuh"
#include "tri_launch.h"

namespace tri {

constexpr int kTcStages = 3;
constexpr int kTcMath = 128;               // threads of the math warps
constexpr int kTcThreads = kTcMath + 32;   // and one loading warp
constexpr int kTcHalf = kTcTile * 128;     // 64 dims of the tile's rows: 16 KB
constexpr int kTcMat = 2 * kTcHalf;        // K or V of a tile
constexpr int kTcPRow = 64;                // bytes of a key's weights: 32 bf16

struct __align__(1024) TcShared {
    unsigned char k[kTcStages][kTcMat];
    unsigned char v[kTcStages][kTcMat];
    unsigned char q[2][16 * 128];       // [64-dim half][16 rows], swizzled
    unsigned char p[kTcTile * kTcPRow]; // [key][32 columns], swizzled
    float wmax[4][8];
    float wsum[4][8];
    uint64_t k_full[kTcStages], k_empty[kTcStages], v_full[kTcStages], v_empty[kTcStages];
    uint64_t s_full[2], o_full;
    uint32_t tmem;
    int abort;
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
// groups 1024 bytes apart; 16 dims are 32 bytes.
__device__ __forceinline__ void issue_scores(TcShared& sm, int stage, uint32_t tmem) {
    constexpr uint32_t idesc = tc_idesc(16, false, false);
#pragma unroll
    for (int x = 0; x < kD / 16; ++x) {
        const int half = x >> 2, off = (x & 3) * 32;
        tc_mma(tmem, tc_desc(sm.k[stage] + half * kTcHalf + off, 16, 1024, 2),
               tc_desc(sm.q[half] + off, 16, 1024, 2), idesc, x > 0);
    }
}

// O = V^T P: V's 64-dim halves (A, M contiguous) kTcHalf bytes apart, 8-key
// groups 1024 bytes apart; P (B, N contiguous) 64-byte keys, 8-key groups 512
// bytes apart; 16 keys a step.
__device__ __forceinline__ void issue_values(TcShared& sm, int stage, uint32_t tmem) {
    constexpr uint32_t idesc = tc_idesc(32, true, true);
#pragma unroll
    for (int x = 0; x < kTcTile / 16; ++x)
        tc_mma(tmem, tc_desc(sm.v[stage] + x * 2048, kTcHalf, 1024, 2),
               tc_desc(sm.p + x * 16 * kTcPRow, 16, 512, 4), idesc, x > 0);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&x);
}

template <int G>
__global__ void __launch_bounds__(kTcThreads, 1)
decode_paged_tc_kernel(const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const int box_rows,
                       const DecodePagedArgs a) {
    extern __shared__ unsigned char smem_raw[];
    TcShared& sm = *reinterpret_cast<TcShared*>(
        smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t cap = a.pc.per_unit * a.pc.rows;
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
        sm.abort = 0;
        fence_barrier_init();
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    const SplitPlan p = plan_split<kTcThreads>(a, kTcTile, 1);  // (synchronises the CTA)
    // The loading warp goes on while the others get their tensor memory.
    uint32_t tmem = 0;
    if (warp < kTcMath / 32) {
        if (warp == 0) tc_alloc(&sm.tmem, 64);
        // Columns 24 .. 31 of the weights stay zeros.
        *reinterpret_cast<uint4*>(sm.p + tid * kTcPRow + ((3 ^ ((tid >> 1) & 3)) * 16)) =
            make_uint4(0, 0, 0, 0);
        tc_fence_before();
        named_sync(1, kTcMath);
        tc_fence_after();
        tmem = sm.tmem;
    }

    uint32_t it = 0;  // tiles of this CTA so far
    uint32_t t = p.begin, i = p.unit, tile0 = p.tile0;
    if (warp == kTcMath / 32) {
        // ---- the loading warp: lane b brings box b ----
        const int n_boxes = kTcTile / box_rows;
        const uint64_t pol = policy_evict_first();
        for (; t < p.end; ++i) {
            const int64_t u = slice_unit(a.sl, i);
            const uint32_t n = i == p.unit ? p.rows : clamp_nvalid(a.n_valid, u, cap, nullptr);
            const uint32_t n_tiles = static_cast<uint32_t>(n + kTcTile - 1) / kTcTile;
            if (n_tiles == 0) continue;
            const uint32_t t1 = min(tile0 + n_tiles, p.end);
            for (; t < t1; ++t, ++it) {
                const int stage = it % kTcStages;
                const uint32_t parity = ((it / kTcStages) & 1) ^ 1;
                const int64_t j = static_cast<int64_t>(t - tile0) * kTcTile + lane * box_rows;
                int64_t row = lane < n_boxes && j < cap ? paged_row(a.pc, u, j) : -1;
                if (lane < n_boxes && j < n && row < 0) {
                    wait_for_clear();
                    raise_flag(a.flag, TRI_FLAG_INDEX_RANGE);
                }
                if (j >= n) row = -1;
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, row >= 0)) * box_rows * 256;
                const int off = lane * box_rows * 128;
                bool ok = mbar_wait(&sm.k_empty[stage], parity, a.flag);
                ok = __all_sync(0xffffffffu, ok && !*reinterpret_cast<volatile int*>(&sm.abort));
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&sm.k_full[stage], bytes);
                __syncwarp();
                if (row >= 0) {
                    const int32_t y = static_cast<int32_t>(row);
                    tma_load_2d_hint(sm.k[stage] + off, &kmap, &sm.k_full[stage], 0, y, pol);
                    tma_load_2d_hint(sm.k[stage] + kTcHalf + off, &kmap, &sm.k_full[stage], 64, y, pol);
                }
                ok = mbar_wait(&sm.v_empty[stage], parity, a.flag);
                ok = __all_sync(0xffffffffu, ok);
                if (lane == 0) mbar_arrive_expect_tx(&sm.v_full[stage], ok ? bytes : 0);
                __syncwarp();
                if (ok && row >= 0) {
                    const int32_t y = static_cast<int32_t>(row);
                    tma_load_2d_hint(sm.v[stage] + off, &vmap, &sm.v_full[stage], 0, y, pol);
                    tma_load_2d_hint(sm.v[stage] + kTcHalf + off, &vmap, &sm.v_full[stage], 64, y, pol);
                }
            }
            if (t < t1) break;  // gave up
            tile0 += n_tiles;
        }
        // Nothing of this warp is in flight when the CTA ends.
        for (uint32_t x = it < kTcStages ? 0 : it - kTcStages; x < it; ++x) {
            mbar_wait(&sm.k_full[x % kTcStages], (x / kTcStages) & 1, a.flag);
            mbar_wait(&sm.v_full[x % kTcStages], (x / kTcStages) & 1, a.flag);
        }
    } else {
        const uint32_t lanes = static_cast<uint32_t>(warp) * 32 << 16;  // this warp's TMEM lanes
        const uint32_t s_cols = tmem, o_cols = tmem + 32;
        const uint32_t page_rows = static_cast<uint32_t>(a.pc.rows);
        SplitUnit split0 = {}, split1 = {};
        int n_split = 0;
        bool ok = true;
        while (t < p.end) {
            const int64_t u = slice_unit(a.sl, i);
            const uint32_t n = i == p.unit ? p.rows : clamp_nvalid(a.n_valid, u, cap, nullptr);
            const uint32_t n_tiles = static_cast<uint32_t>(n + kTcTile - 1) / kTcTile;
            if (n_tiles == 0) {
                ++i;
                continue;
            }
            const uint32_t t1 = min(tile0 + n_tiles, p.end);
            const bool from_start = t == tile0;
            // ---- Q, rows >= G zero; 16-byte chunk c of a 128-byte row r lies at c ^ (r & 7) ----
            for (int e = tid; e < 16 * 16; e += kTcMath) {
                const int r = e >> 4, c = e & 15;
                uint4 x = make_uint4(0, 0, 0, 0);
                if (r < G)
                    x = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                             (static_cast<int64_t>(i) * G + r) * kD) +
                              c);
                *reinterpret_cast<uint4*>(sm.q[c >> 3] + r * 128 + ((c & 7) ^ (r & 7)) * 16) = x;
            }
            float m[G], l[G], acc[G];
#pragma unroll
            for (int h = 0; h < G; ++h) {
                m[h] = -INFINITY;
                l[h] = acc[h] = 0.f;
            }
            fence_proxy_async();
            named_sync(1, kTcMath);
            auto start_scores = [&](uint32_t x) {
                ok = mbar_wait(&sm.k_full[x % kTcStages], (x / kTcStages) & 1, a.flag) && ok;
                tc_fence_after();
                issue_scores(sm, x % kTcStages, s_cols + (x & 1) * 16);
                tc_commit(&sm.s_full[x & 1]);
                tc_commit(&sm.k_empty[x % kTcStages]);
            };
            if (tid == 0) start_scores(it);
            // Whether this thread's key of tile x has a row (looked up a tile ahead).
            auto has_row = [&](uint32_t x) {
                const uint32_t j = (x - tile0) * kTcTile + tid;
                return x < t1 && j < n && page_of(a.pc, u, j / page_rows) >= 0;
            };
            bool valid = has_row(t);
            for (; t < t1; ++t, ++it) {
                const int stage = it % kTcStages;
                const uint32_t parity = (it / kTcStages) & 1;
                const bool valid_next = has_row(t + 1);
                ok = mbar_wait(&sm.s_full[it & 1], (it >> 1) & 1, a.flag) && ok;
                tc_fence_after();
                float s[8];
                tc_load8(s_cols + (it & 1) * 16 + lanes, s);
                tc_load_wait();
                tc_fence_before();
                // ---- maxima of the warp's 32 keys: 8 values, halved 3 times ----
                float x[8];
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    x[h] = h < G && valid ? s[h] * a.scale_log2 : -INFINITY;
                }
#pragma unroll
                for (int q = 0; q < 3; ++q) {
                    const int o = 16 >> q, c = 4 >> q;
                    const bool up = lane & o;
#pragma unroll
                    for (int h = 0; h < c; ++h) {
                        const float keep = up ? x[h + c] : x[h];
                        const float give = up ? x[h] : x[h + c];
                        x[h] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, o));
                    }
                }
                x[0] = fmaxf(x[0], __shfl_xor_sync(0xffffffffu, x[0], 2));
                x[0] = fmaxf(x[0], __shfl_xor_sync(0xffffffffu, x[0], 1));
                if ((lane & 3) == 0) sm.wmax[warp][lane >> 2] = x[0];
                const bool part_tile = !__all_sync(0xffffffffu, valid);
                if (part_tile) ok = mbar_wait(&sm.v_full[stage], parity, a.flag) && ok;
                if (!ok) *reinterpret_cast<volatile int*>(&sm.abort) = 1;
                named_sync(1, kTcMath);
                if (*reinterpret_cast<volatile int*>(&sm.abort)) break;
                float al[G];
#pragma unroll
                for (int h = 0; h < G; ++h) {
                    const float mt = fmaxf(fmaxf(sm.wmax[0][h], sm.wmax[1][h]),
                                           fmaxf(sm.wmax[2][h], sm.wmax[3][h]));
                    const float m_new = fmaxf(m[h], mt);
                    const float base = m_new == -INFINITY ? 0.f : m_new;
                    al[h] = exp2f(m[h] - base);
                    // (one rounding of the small difference, not of the large product)
                    const float w = valid ? exp2f(fmaf(s[h], a.scale_log2, -base)) : 0.f;
                    l[h] = fmaf(l[h], al[h], w);
                    m[h] = m_new;
                    s[h] = w;
                }
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
                // Rows that carry no weight hold anything: zeros, since 0 * inf is not 0.
                if (!valid) {
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        *reinterpret_cast<uint4*>(sm.v[stage] + (c >> 3) * kTcHalf + tid * 128 +
                                                  (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
                named_sync(1, kTcMath);
                if (tid == 0) {
                    ok = mbar_wait(&sm.v_full[stage], parity, a.flag) && ok;
                    tc_fence_after();
                    issue_values(sm, stage, o_cols);
                    tc_commit(&sm.o_full);
                    tc_commit(&sm.v_empty[stage]);
                    if (t + 1 < t1) start_scores(it + 1);
                }
                __syncwarp();
                ok = mbar_wait(&sm.o_full, it & 1, a.flag) && ok;
                tc_fence_after();
                float o1[8], o2[8], o3[8];
                tc_load8(o_cols + lanes, o1);
                tc_load8(o_cols + 8 + lanes, o2);
                tc_load8(o_cols + 16 + lanes, o3);
                tc_load_wait();
                tc_fence_before();
#pragma unroll
                for (int h = 0; h < G; ++h) {
                    // An infinite value times a term of zero is no part of the sum.
                    const float rest = isfinite(o1[h]) ? o2[h] + o3[h] : 0.f;
                    acc[h] = fmaf(acc[h], al[h], o1[h] + rest);
                }
                valid = valid_next;
            }
            // ---- the unit's sums over the keys ----
#pragma unroll
            for (int h = 0; h < G; ++h) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], o);
                if (lane == 0) sm.wsum[warp][h] = l[h];
            }
            if (!ok) *reinterpret_cast<volatile int*>(&sm.abort) = 1;
            named_sync(1, kTcMath);
            if (*reinterpret_cast<volatile int*>(&sm.abort)) break;
            const bool whole = from_start && t1 == tile0 + n_tiles;
            const uint32_t slot = part_slot(p, blockIdx.x, tile0);
#pragma unroll
            for (int h = 0; h < G; ++h) {
                const float den = (sm.wsum[0][h] + sm.wsum[1][h]) + (sm.wsum[2][h] + sm.wsum[3][h]);
                if (whole) {
                    a.out[(static_cast<int64_t>(i) * G + h) * kD + tid] = den == 0.f ? 0.f : acc[h] / den;
                    if (a.lse && tid == 0) a.lse[static_cast<int64_t>(i) * G + h] = lse_of(m[h], den);
                } else {
                    a.part[(slot * G + h) * kD + tid] = acc[h];
                    if (tid == 0) a.part_ml[slot * G + h] = make_float2(m[h], den);
                }
            }
            if (!whole) {
                split1 = split_unit(p, i, tile0, n_tiles);
                if (n_split++ == 0) split0 = split1;
            }
            named_sync(1, kTcMath);  // wsum and Q are rewritten by the next unit
            tile0 += n_tiles;
            ++i;
        }
        if (!*reinterpret_cast<volatile int*>(&sm.abort))
            join_split_units<kTcMath / 32, 1, 16>(a, G, n_split, split0, split1);
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
    struct Key {};
    cudaError_t e = allow_smem<Key>(reinterpret_cast<const void*>(fn), smem);
    if (e != cudaSuccess) return e;
    e = launch_decode_paged_clear(a, s);
    if (e != cudaSuccess) return e;
    e = launch_early(fn, decode_paged_ctas(n_sm), kTcThreads, smem, s, kmap, vmap, box_rows, a);
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
