// paged_core.cuh -- device helpers of the paged-cache kernels.
#pragma once

#include <atomic>

#include "paged.h"
#include "tri_internal.cuh"

namespace tri {

// Cache unit of the call's i-th unit.
__device__ __forceinline__ int64_t slice_unit(const UnitSlice& sl, int64_t i) {
    // (counts of units, slots and rows fit 32 bits: cheaper divisions)
    if (sl.layer < 0) return i;
    const uint32_t heads = static_cast<uint32_t>(sl.n_kvheads);
    const uint32_t seq = static_cast<uint32_t>(i) / heads, head = static_cast<uint32_t>(i) - seq * heads;
    return (seq * sl.n_layers + sl.layer) * heads + head;
}

// Page of slot `slot` of unit u, or -1.
__device__ __forceinline__ int64_t page_of(const PagedCache& pc, int64_t u, int64_t slot) {
    const int64_t pg = pc.table[u * pc.per_unit + slot];
    return pg >= 0 && pg < pc.n_pages ? pg : -1;
}

// Physical row of row j of unit u, or -1 when its page is not in the pool.
__device__ __forceinline__ int64_t paged_row(const PagedCache& pc, int64_t u, int64_t j) {
    const uint32_t rows = static_cast<uint32_t>(pc.rows);
    const uint32_t slot = static_cast<uint32_t>(j) / rows;
    const int64_t pg = page_of(pc, u, slot);
    return pg < 0 ? -1 : pg * pc.rows + (static_cast<uint32_t>(j) - slot * rows);
}

// ---------------------------------------------------------------------------
// Split of the call's keys over the CTAs.  The units' rows are cut into tiles
// of `tile` keys and the tiles of all units, end to end, are dealt to the
// CTAs in equal contiguous ranges, so ragged lengths balance; a unit that
// lies in several ranges is joined by the CTA that finishes it last.
// ---------------------------------------------------------------------------
struct SplitPlan {
    uint32_t share;   // tiles of a CTA; the first `longer` ones have one more
    uint32_t longer;
    uint32_t begin;   // this CTA's tiles
    uint32_t end;
    uint32_t unit;    // first unit of the range
    uint32_t tile0;   // its first tile
};

__device__ __forceinline__ uint32_t range_begin(const SplitPlan& p, uint32_t c) {
    return c * p.share + min(c, p.longer);
}
// The CTA whose range holds tile t.
__device__ __forceinline__ uint32_t cta_of_tile(const SplitPlan& p, uint32_t t) {
    const uint32_t edge = p.longer * (p.share + 1);
    return t < edge ? t / (p.share + 1) : p.longer + (t - edge) / p.share;
}

// Computed by every thread of the CTA together (kThreads of them, a multiple
// of 32): each sums the tiles of its share of the units, a block scan places
// the shares, and the thread whose share holds the CTA's first tile finds its
// unit.  At least `min_tiles` tiles a CTA, while the call has that many.
// (The host has checked that the tiles of the call fit 31 bits.)
template <int kThreads>
__device__ SplitPlan plan_split(const DecodePagedArgs& a, int tile, uint32_t min_tiles) {
    __shared__ uint32_t warp_sum[kThreads / 32];
    __shared__ uint32_t found[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t cap = a.pc.per_unit * a.pc.rows;
    const uint32_t units = static_cast<uint32_t>(a.sl.n);
    const uint32_t per = (units + kThreads - 1) / kThreads;
    const uint32_t i0 = min(tid * per, units), i1 = min(i0 + per, units);
    auto tiles = [&](uint32_t i) -> uint32_t {
        return static_cast<uint32_t>(clamp_nvalid(a.n_valid, slice_unit(a.sl, i), cap, nullptr) + (tile - 1)) / tile;
    };
    uint32_t sum = 0;
#pragma unroll 4
    for (uint32_t i = i0; i < i1; ++i) sum += tiles(i);
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    uint32_t before = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    SplitPlan p;
    const uint32_t ctas = max(min((total + min_tiles - 1) / min_tiles, gridDim.x), 1u);
    const uint32_t c = blockIdx.x;
    p.share = total / ctas;
    p.longer = total - p.share * ctas;
    p.begin = c < ctas ? range_begin(p, c) : total;
    p.end = c < ctas ? range_begin(p, c + 1) : total;
    if (p.begin < p.end && before <= p.begin && p.begin < before + sum) {
        uint32_t t = before;
        for (uint32_t i = i0; i < i1; ++i) {
            const uint32_t nt = per == 1 ? sum : tiles(i);
            if (p.begin < t + nt) {
                found[0] = i;
                found[1] = t;
                break;
            }
            t += nt;
        }
    }
    __syncthreads();
    p.unit = found[0];
    p.tile0 = found[1];
    return p;
}

// The first kernel of the call clears the flag word and the counters and lets
// the second one start at once; that one waits here before it touches them.
__device__ __forceinline__ void wait_for_clear() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Let fn use `bytes` of dynamic shared memory; asked of the runtime once per
// kernel (Key: a type that names it) and device.
template <typename Key>
cudaError_t allow_smem(const void* fn, size_t bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Launch a kernel that may start before the previous one of the stream has
// ended (it waits with wait_for_clear).
template <typename... P, typename... A>
cudaError_t launch_early(void (*fn)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t s,
                         const A&... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

// Units without a row: zeros and an lse of -inf, spread over the grid; counts
// out of range are flagged.  (After wait_for_clear.)
__device__ __forceinline__ void write_empty_units(const DecodePagedArgs& a, int G) {
    const int64_t cap = a.pc.per_unit * a.pc.rows;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = blockIdx.x + static_cast<int64_t>(gridDim.x) * threadIdx.x; i < a.sl.n;
         i += step) {
        if (clamp_nvalid(a.n_valid, slice_unit(a.sl, i), cap, a.flag) > 0) continue;
        float4* o = reinterpret_cast<float4*>(a.out + i * G * kD);
        for (int e = 0; e < G * kD / 4; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.lse)
            for (int h = 0; h < G; ++h) a.lse[i * G + h] = -INFINITY;
    }
}

// log2-domain running maximum and sum -> natural logarithm of the softmax's
// denominator.
__device__ __forceinline__ float lse_of(float m, float l) {
    return l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : (l == 0.f ? -INFINITY : l);
}

// Partial result of a unit's segment: slot 2 c of CTA c, or 2 c + 1 for a unit
// that begins inside the CTA's range.
__device__ __forceinline__ uint32_t part_slot(const SplitPlan& p, uint32_t c, uint32_t tile0) {
    return 2 * c + (tile0 <= range_begin(p, c) ? 0 : 1);
}

// A CTA's range holds at most two units that lie in other ranges too: its
// first and its last.
struct SplitUnit {
    uint32_t i, tile0, n_tiles;
    bool last;  // this CTA joins it
};

// The heads h0, h0 + step, ... (kHeads of them at most, below `heads`) of the
// split units, joined by one warp: head q is head q % G of unit q / G.  Lane c
// holds the maximum and sum of the c-th of 32 CTAs, every lane 4 dims of the
// accumulators; the accumulators of kAhead CTAs of all kHeads are requested
// at a time.
template <int kHeads, int kAhead>
__device__ void join_heads(const DecodePagedArgs& a, int G, const SplitPlan& p,
                           const SplitUnit (&split)[2], int heads, int h0, int step) {
    const int lane = threadIdx.x & 31;
    struct Head {
        uint32_t i, c0, n, slot0, h;  // n = 0: none
    } hd[kHeads];
    uint32_t most = 0;
#pragma unroll
    for (int r = 0; r < kHeads; ++r) {
        const int q = h0 + r * step;
        const SplitUnit& s = split[q >= G && q < heads ? 1 : 0];
        hd[r].i = s.i;
        hd[r].h = q >= G ? q - G : q;
        hd[r].c0 = cta_of_tile(p, s.tile0);
        hd[r].n = q < heads && s.last ? cta_of_tile(p, s.tile0 + s.n_tiles - 1) - hd[r].c0 + 1 : 0;
        hd[r].slot0 = part_slot(p, hd[r].c0, s.tile0);
        most = max(most, hd[r].n);
    }
    // Slot of the unit's x-th CTA; x past the last one repeats it.
    auto slot = [&](const Head& d, uint32_t x) -> uint32_t {
        x = min(x, d.n - 1);
        return (x == 0 ? d.slot0 : 2 * (d.c0 + x)) * G + d.h;
    };
    float M[kHeads], den[kHeads];
    float4 acc[kHeads];
#pragma unroll
    for (int r = 0; r < kHeads; ++r) {
        M[r] = -INFINITY;
        den[r] = 0.f;
        acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll 1
    for (uint32_t cb = 0; cb < most; cb += 32) {
        float2 x[kHeads];
        float w[kHeads];
        float4 v[kHeads][kAhead];
#pragma unroll
        for (int r = 0; r < kHeads; ++r)
            if (hd[r].n) x[r] = __ldcg(a.part_ml + slot(hd[r], cb + lane));
        auto request = [&](uint32_t b) {
#pragma unroll
            for (int r = 0; r < kHeads; ++r)
#pragma unroll
                for (int y = 0; y < kAhead; ++y)
                    if (hd[r].n)
                        v[r][y] = __ldcg(reinterpret_cast<const float4*>(
                                             a.part + static_cast<int64_t>(slot(hd[r], b + y)) * kD) + lane);
        };
        request(cb);
#pragma unroll
        for (int r = 0; r < kHeads; ++r) {
            const bool in = cb + lane < hd[r].n;
            float m = in ? x[r].x : -INFINITY;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            m = fmaxf(m, M[r]);
            const float base = m == -INFINITY ? 0.f : m;
            const float f = exp2f(M[r] - base);
            w[r] = in ? exp2f(x[r].x - base) : 0.f;
            float l = in ? w[r] * x[r].y : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            M[r] = m;
            den[r] = fmaf(den[r], f, l);
            acc[r] = make_float4(acc[r].x * f, acc[r].y * f, acc[r].z * f, acc[r].w * f);
        }
#pragma unroll 1
        for (uint32_t b = 0; b < 32 && cb + b < most; b += kAhead) {
#pragma unroll
            for (int r = 0; r < kHeads; ++r) {
#pragma unroll
                for (int y = 0; y < kAhead; ++y) {
                    const float g = __shfl_sync(0xffffffffu, w[r], b + y);
                    if (cb + b + y >= hd[r].n) continue;
                    acc[r].x = fmaf(g, v[r][y].x, acc[r].x);
                    acc[r].y = fmaf(g, v[r][y].y, acc[r].y);
                    acc[r].z = fmaf(g, v[r][y].z, acc[r].z);
                    acc[r].w = fmaf(g, v[r][y].w, acc[r].w);
                }
            }
            if (b + kAhead < 32 && cb + b + kAhead < most) request(cb + b + kAhead);
        }
    }
#pragma unroll
    for (int r = 0; r < kHeads; ++r) {
        if (!hd[r].n) continue;
        const int64_t row = static_cast<int64_t>(hd[r].i) * G + hd[r].h;
        const float d = den[r];
        reinterpret_cast<float4*>(a.out + row * kD)[lane] =
            d == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                     : make_float4(acc[r].x / d, acc[r].y / d, acc[r].z / d, acc[r].w / d);
        if (a.lse && lane == 0) a.lse[row] = lse_of(M[r], d);
    }
}

// The partials of this CTA's n_split split units are written; of each unit the
// CTA that arrives last joins the partials in CTA order,
//   out = sum_c 2^(m_c - M) acc_c / sum_c 2^(m_c - M) l_c.
// Called once, at the end, by the kWarps * 32 threads of named barrier kBar,
// so the fence and the atomics are paid once.  What bounds it is the latency
// of its loads: with many heads to join from few CTAs each a warp takes four
// heads at a time, else two with more CTAs at a time.
// (kAhead: as the kernel's registers allow.)
template <int kWarps, int kBar, int kAhead>
__device__ void join_split_units(const DecodePagedArgs& a, int G, const SplitPlan& p, int n_split,
                                 SplitUnit (&split)[2]) {
    __shared__ bool last[2];
    const int tid = threadIdx.x, warp = tid >> 5;
    wait_for_clear();
    named_sync(kBar, kWarps * 32);
    uint32_t most = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        if (x >= n_split) break;
        const uint32_t more =
            cta_of_tile(p, split[x].tile0 + split[x].n_tiles - 1) - cta_of_tile(p, split[x].tile0);
        most = max(most, more + 1);
        if (tid == x * 32) {
            __threadfence();
            last[x] = atomicAdd(a.counters + split[x].i, 1u) == more;
            __threadfence();
        }
    }
    named_sync(kBar, kWarps * 32);
    bool any = false;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        split[x].last = x < n_split && last[x];
        any = any || split[x].last;
    }
    if (!any) return;
    const int heads = n_split * G;
    if (most <= 4) {
#pragma unroll 1
        for (int q = warp; q < heads; q += 4 * kWarps) join_heads<4, 4>(a, G, p, split, heads, q, kWarps);
    } else {
#pragma unroll 1
        for (int q = warp; q < heads; q += 2 * kWarps) join_heads<2, kAhead>(a, G, p, split, heads, q, kWarps);
    }
}

}  // namespace tri
