// decode_paged.cu -- attention of the next token over a paged cache.
//
// For each unit (sequence, layer, KV head) and each of its G query heads h:
//   o_h = sum_{j < n} a_j v_j,  a_j = exp(s_j - m) / sum_{j' < n} exp(s_j' - m),
//   s_j = scale * (q_h . k_j),  m = max_j s_j,  lse_h = m + log sum_j exp(s_j - m),
// row j of the unit found through its page table (jaedaily.cn tutorial,
// KV-compression objective: the softmax renormalised over the kept rows).
//
// rows kernel (any page size, both types).  Warps are independent: a warp
// takes 32 keys at a time in groups of 4, its lanes holding 4 of the 128 dims
// each.  Every lane copies its own 4 dims of the keys and values of the next
// groups into a private shared-memory ring (cp.async, so no barrier is needed:
// a lane reads back what it copied; a row without a page copies zeros).  The
// 4 G partial dot products of a group are summed over the lanes by a
// transposing butterfly (one shuffle per halved value instead of five per
// value), which leaves one (key, head) score per lane for the online softmax;
// the weights go back to all lanes by shuffle for the value product.  Scores,
// running maxima, sums and accumulators are float32.
#include "paged_core.cuh"
#include "tri_launch.h"

namespace tri {

__global__ void __launch_bounds__(256) decode_clear_kernel(uint32_t* flag, uint32_t* counters, int64_t n) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t i = blockIdx.x * 256ll + threadIdx.x;
    if (i == 0) *flag = 0;
    if (i < n) counters[i] = 0;
}

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kRowTile = 32;    // keys a warp takes at a time
constexpr int kGroup = 4;       // keys whose scores are formed together
constexpr int kRing = 6;        // groups in a warp's ring

constexpr int row_group_pad(int G) { return G <= 1 ? 1 : G <= 2 ? 2 : G <= 4 ? 4 : 8; }

template <typename T>
constexpr size_t row_ring_bytes() {
    return static_cast<size_t>(kRowWarps) * kRing * kGroup * 2 * kD * sizeof(T);
}
template <int G>
constexpr size_t row_red_bytes() {
    return static_cast<size_t>(kRowWarps) * G * (kD + 2) * sizeof(float);
}

// This lane's 4 dims of one row: global -> shared, zeros where the row has no
// page.
template <typename T>
__device__ __forceinline__ void copy_lane(void* dst, const T* src, bool valid) {
    constexpr int kBytes = 4 * sizeof(T);
    const int n = valid ? kBytes : 0;
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
                     "r"(n)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(dst)), "l"(src),
                     "r"(n)
                     : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void load4(const float* p, float2& a, float2& b) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    a = make_float2(x.x, x.y);
    b = make_float2(x.z, x.w);
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float2& a, float2& b) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    a = make_float2(bf16_lo(x.x), bf16_hi(x.x));
    b = make_float2(bf16_lo(x.y), bf16_hi(x.y));
}

template <typename T, int G>
__global__ void __launch_bounds__(kRowThreads, 1) decode_paged_rows_kernel(const DecodePagedArgs a) {
    constexpr int GP = row_group_pad(G);
    constexpr int NV = kGroup * GP;  // values of a group's butterfly
    extern __shared__ __align__(16) unsigned char smem[];
    T* ring = reinterpret_cast<T*>(smem);
    float* red = reinterpret_cast<float*>(smem + row_ring_bytes<T>());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t cap = a.pc.per_unit * a.pc.rows;
    const SplitPlan p = plan_split<kRowThreads>(a, kRowTile, kRowWarps);
    SplitUnit split[2] = {};
    int n_split = 0;
    // This lane's slice of the warp's ring: [kRing][kGroup][K, V] of 4 dims.
    T* mine = ring + (static_cast<int64_t>(warp) * kRing * kGroup * 2 * 32 + lane) * 4;
    auto cell = [&](int slot, int key, int kv) {
        return mine + ((slot * kGroup + key) * 2 + kv) * 32 * 4;
    };
    const T* kp = static_cast<const T*>(a.k) + lane * 4;
    const T* vp = static_cast<const T*>(a.v) + lane * 4;

    uint32_t t = p.begin, i = p.unit, tile0 = p.tile0;
    while (t < p.end) {
        const int64_t u = slice_unit(a.sl, i);
        const int64_t n = clamp_nvalid(a.n_valid, u, cap, nullptr);
        const uint32_t n_tiles = static_cast<uint32_t>(n + kRowTile - 1) / kRowTile;
        if (n_tiles == 0) {
            ++i;
            continue;
        }
        const int64_t b1 = min(n_tiles, p.end - tile0);  // tiles [t - tile0, b1) of the unit
        const int64_t b0 = t - tile0;
        float2 q[G][2], acc[G][2];
#pragma unroll
        for (int h = 0; h < G; ++h) {
            const T* qh = static_cast<const T*>(a.q) + (static_cast<int64_t>(i) * G + h) * kD + lane * 4;
            load4(qh, q[h][0], q[h][1]);
            acc[h][0] = acc[h][1] = make_float2(0.f, 0.f);
        }
        // This lane's score of a group: key lane / (32 / NV) / GP, head % GP.
        const int vi = lane / (32 / NV);
        const int my_key = vi / GP, my_head = vi % GP;
        float m = -INFINITY, l = 0.f;  // of my_head; l over my_key's keys only

        // Tiles b0 + warp, b0 + warp + kRowWarps, ...; their groups in one
        // running order g = 0, 1, ... for the ring.
        const int64_t mt = b1 - b0 > warp ? (b1 - b0 - warp + kRowWarps - 1) / kRowWarps : 0;
        const int64_t n_groups = mt * (kRowTile / kGroup);
        int64_t row_next = -1;  // physical row of this lane's key of the tile being loaded
        auto issue = [&](int64_t g) {
            if (g < n_groups) {
                const int gi = static_cast<int>(g % (kRowTile / kGroup));
                if (gi == 0) {
                    const int64_t j = (b0 + warp + g / (kRowTile / kGroup) * kRowWarps) * kRowTile + lane;
                    row_next = -1;
                    if (j < n) {
                        row_next = paged_row(a.pc, u, j);
                        if (row_next < 0) {
                            wait_for_clear();
                            raise_flag(a.flag, TRI_FLAG_INDEX_RANGE);
                        }
                    }
                }
                const int slot = static_cast<int>(g % kRing);
#pragma unroll
                for (int key = 0; key < kGroup; ++key) {
                    const int64_t r = __shfl_sync(0xffffffffu, row_next, gi * kGroup + key);
                    const int64_t off = (r < 0 ? 0 : r) * kD;
                    copy_lane(cell(slot, key, 0), kp + off, r >= 0);
                    copy_lane(cell(slot, key, 1), vp + off, r >= 0);
                }
            }
            copy_commit();
        };
        // Rows of the tile being used: looked up again rather than kept for
        // the whole ring (the table entries are in L1).
        int64_t row_now = -1;
        for (int g = 0; g < kRing - 1; ++g) issue(g);
        for (int64_t g = 0; g < n_groups; ++g) {
            const int gi = static_cast<int>(g % (kRowTile / kGroup));
            if (gi == 0) {
                const int64_t j = (b0 + warp + g / (kRowTile / kGroup) * kRowWarps) * kRowTile + lane;
                row_now = j < n ? paged_row(a.pc, u, j) : -1;
            }
            copy_wait<kRing - 2>();
            const int slot = static_cast<int>(g % kRing);
            // ---- partial dot products, then the transposing butterfly ----
            float s[NV];
#pragma unroll
            for (int key = 0; key < kGroup; ++key) {
                float2 k0, k1;
                load4(cell(slot, key, 0), k0, k1);
#pragma unroll
                for (int h = 0; h < GP; ++h) {
                    if (h < G) {
                        float2 d = __ffma2_rn(k0, q[h < G ? h : 0][0], make_float2(0.f, 0.f));
                        d = __ffma2_rn(k1, q[h < G ? h : 0][1], d);
                        s[key * GP + h] = d.x + d.y;
                    } else {
                        s[key * GP + h] = 0.f;
                    }
                }
            }
            int o = 16;
#pragma unroll
            for (int count = NV; count > 1; count >>= 1) {
                const bool up = lane & o;
#pragma unroll
                for (int x = 0; x < count / 2; ++x) {
                    const float keep = up ? s[x + count / 2] : s[x];
                    const float give = up ? s[x] : s[x + count / 2];
                    s[x] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
                o >>= 1;
            }
#pragma unroll
            for (; o > 0; o >>= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
            const bool valid = __shfl_sync(0xffffffffu, row_now, gi * kGroup + my_key) >= 0;
            const float sc = valid ? s[0] * a.scale_log2 : -INFINITY;
            // ---- online softmax of my_head ----
            float mx = sc;
#pragma unroll
            for (int x = GP * (32 / NV); x < 32; x <<= 1)
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const float m_new = fmaxf(m, mx);
            const float base = m_new == -INFINITY ? 0.f : m_new;
            const float pr = valid ? exp2f(sc - base) : 0.f;
            if (__any_sync(0xffffffffu, m_new != m)) {
                const float al = exp2f(m - base);
                l *= al;
#pragma unroll
                for (int h = 0; h < G; ++h) {
                    const float ah = __shfl_sync(0xffffffffu, al, h * (32 / NV));
                    acc[h][0].x *= ah;
                    acc[h][0].y *= ah;
                    acc[h][1].x *= ah;
                    acc[h][1].y *= ah;
                }
                m = m_new;
            }
            l += pr;
            // ---- values ----
#pragma unroll
            for (int key = 0; key < kGroup; ++key) {
                float2 v0, v1;
                load4(cell(slot, key, 1), v0, v1);
#pragma unroll
                for (int h = 0; h < G; ++h) {
                    const float w = __shfl_sync(0xffffffffu, pr, (key * GP + h) * (32 / NV));
                    acc[h][0] = __ffma2_rn(make_float2(w, w), v0, acc[h][0]);
                    acc[h][1] = __ffma2_rn(make_float2(w, w), v1, acc[h][1]);
                }
            }
            issue(g + kRing - 1);
        }
        copy_wait<0>();
        // ---- the warps' results, joined in warp order ----
        // l of my_head: over the keys of a group (lanes GP * (32 / NV) apart).
#pragma unroll
        for (int x = GP * (32 / NV); x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        float* rw = red + warp * G * (kD + 2);
#pragma unroll
        for (int h = 0; h < G; ++h) {
            float2* d = reinterpret_cast<float2*>(rw + h * (kD + 2) + 2 + lane * 4);
            d[0] = acc[h][0];
            d[1] = acc[h][1];
        }
        if (lane % (32 / NV) == 0 && my_key == 0 && my_head < G) {
            rw[my_head * (kD + 2)] = m;
            rw[my_head * (kD + 2) + 1] = l;
        }
        __syncthreads();
        const bool whole = b0 == 0 && b1 == n_tiles;
        const uint32_t slot = part_slot(p, blockIdx.x, tile0);
        for (int e = tid; e < G * kD; e += kRowThreads) {
            const int h = e / kD, d = e % kD;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, red[(w * G + h) * (kD + 2)]);
            float num = 0.f, den = 0.f;
#pragma unroll
            for (int w = 0; w < kRowWarps; ++w) {
                const float* x = red + (w * G + h) * (kD + 2);
                const float f = x[0] == -INFINITY ? 0.f : exp2f(x[0] - M);
                num = fmaf(f, x[2 + d], num);
                den = fmaf(f, x[1], den);
            }
            if (whole) {
                a.out[(static_cast<int64_t>(i) * G + h) * kD + d] = den == 0.f ? 0.f : num / den;
                if (a.lse && d == 0) a.lse[static_cast<int64_t>(i) * G + h] = lse_of(M, den);
            } else {
                a.part[(slot * G + h) * kD + d] = num;
                if (d == 0) a.part_ml[slot * G + h] = make_float2(M, den);
            }
        }
        if (!whole) {
            split[0] = n_split ? split[0] : SplitUnit{i, tile0, n_tiles, false};
            split[1] = SplitUnit{i, tile0, n_tiles, false};
            ++n_split;
        }
        __syncthreads();  // red is rewritten by the next unit
        t = tile0 + b1;
        tile0 += n_tiles;
        ++i;
    }
    join_split_units<kRowWarps, 0>(a, G, p, n_split, split);
    write_empty_units(a, G);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int decode_paged_ctas(int n_sm) { return n_sm; }

cudaError_t launch_decode_paged_clear(const DecodePagedArgs& a, cudaStream_t s) {
    decode_clear_kernel<<<static_cast<unsigned>((a.sl.n + 255) / 256), 256, 0, s>>>(a.flag, a.counters,
                                                                                   a.sl.n);
    note_launch(s);
    return cudaGetLastError();
}

template <typename T, int G>
static cudaError_t launch_rows(const DecodePagedArgs& a, int n_sm, cudaStream_t s) {
    constexpr size_t smem = row_ring_bytes<T>() + row_red_bytes<G>();
    auto* fn = decode_paged_rows_kernel<T, G>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    e = launch_decode_paged_clear(a, s);
    if (e != cudaSuccess) return e;
    e = launch_early(fn, decode_paged_ctas(n_sm), kRowThreads, smem, s, a);
    if (e == cudaSuccess) note_launch(s);
    return e;
}

template <typename T>
static cudaError_t launch_rows_t(int G, const DecodePagedArgs& a, int n_sm, cudaStream_t s) {
    switch (G) {
#define TRI_DCASE(g) \
    case g: return launch_rows<T, g>(a, n_sm, s);
        TRI_DCASE(1) TRI_DCASE(2) TRI_DCASE(3) TRI_DCASE(4)
        TRI_DCASE(5) TRI_DCASE(6) TRI_DCASE(7) TRI_DCASE(8)
#undef TRI_DCASE
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_decode_paged_rows(tri_dtype dt, int G, const DecodePagedArgs& a, int n_sm,
                                     cudaStream_t s) {
    return dt == TRI_BF16 ? launch_rows_t<__nv_bfloat16>(G, a, n_sm, s)
                          : launch_rows_t<float>(G, a, n_sm, s);
}

}  // namespace tri
