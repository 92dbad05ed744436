// paged_core.cuh -- device helpers of the paged-cache kernels.
#pragma once

#include "paged.h"
#include "tri_internal.cuh"

namespace tri {

// Cache unit of the call's i-th unit.
__device__ __forceinline__ int64_t slice_unit(const UnitSlice& sl, int64_t i) {
    if (sl.layer < 0) return i;
    const int64_t seq = i / sl.n_kvheads, head = i - seq * sl.n_kvheads;
    return (seq * sl.n_layers + sl.layer) * sl.n_kvheads + head;
}

// Page of slot `slot` of unit u, or -1.
__device__ __forceinline__ int64_t page_of(const PagedCache& pc, int64_t u, int64_t slot) {
    const int64_t pg = pc.table[u * pc.per_unit + slot];
    return pg >= 0 && pg < pc.n_pages ? pg : -1;
}

// Physical row of row j of unit u, or -1 when its page is not in the pool.
__device__ __forceinline__ int64_t paged_row(const PagedCache& pc, int64_t u, int64_t j) {
    const int64_t slot = j / pc.rows;
    const int64_t pg = page_of(pc, u, slot);
    return pg < 0 ? -1 : pg * pc.rows + (j - slot * pc.rows);
}

// ---------------------------------------------------------------------------
// Split of the call's keys over the CTAs.  The units' rows are cut into tiles
// of `tile` keys and the tiles of all units, end to end, are dealt to the
// CTAs in equal contiguous ranges, so ragged lengths balance; a unit that
// lies in several ranges is joined by the CTA that finishes it last.
// ---------------------------------------------------------------------------
struct SplitPlan {
    int64_t total;   // tiles of all units
    int ctas;        // CTAs with a range
    int64_t begin;   // this CTA's tiles
    int64_t end;
    int64_t unit;    // first unit of the range
    int64_t tile0;   // its first tile
};

__device__ __forceinline__ int64_t range_begin(int64_t total, int ctas, int c) {
    return total * c / ctas;
}
// The CTA whose range holds tile t.
__device__ __forceinline__ int cta_of_tile(int64_t total, int ctas, int64_t t) {
    return static_cast<int>(((t + 1) * ctas - 1) / total);
}

// Computed by every thread of the CTA together (kThreads of them, a multiple
// of 32): each sums the tiles of its share of the units, a block scan places
// the shares, and the thread whose share holds the CTA's first tile finds its
// unit.  At least `min_tiles` tiles a CTA, while the call has that many.
template <int kThreads>
__device__ SplitPlan plan_split(const DecodePagedArgs& a, int tile, int min_tiles) {
    __shared__ int64_t warp_sum[kThreads / 32];
    __shared__ int64_t found[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t cap = a.pc.per_unit * a.pc.rows;
    const int64_t per = (a.sl.n + kThreads - 1) / kThreads;
    const int64_t i0 = tid * per < a.sl.n ? tid * per : a.sl.n;
    const int64_t i1 = i0 + per < a.sl.n ? i0 + per : a.sl.n;
    uint32_t* flag = blockIdx.x == 0 ? a.flag : nullptr;
    int64_t sum = 0;
    for (int64_t i = i0; i < i1; ++i)
        sum += (clamp_nvalid(a.n_valid, slice_unit(a.sl, i), cap, flag) + tile - 1) / tile;
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) warp_sum[warp] = incl;
    if (tid == 0) found[0] = a.sl.n;
    __syncthreads();
    int64_t before = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    SplitPlan p;
    p.total = total;
    const int64_t want = (total + min_tiles - 1) / min_tiles;
    p.ctas = static_cast<int>(want < gridDim.x ? want : gridDim.x);
    const int c = blockIdx.x;
    p.begin = c < p.ctas ? range_begin(total, p.ctas, c) : total;
    p.end = c < p.ctas ? range_begin(total, p.ctas, c + 1) : total;
    if (p.begin < p.end && before <= p.begin && p.begin < before + sum) {
        int64_t t = before;
        for (int64_t i = i0; i < i1; ++i) {
            const int64_t nt =
                (clamp_nvalid(a.n_valid, slice_unit(a.sl, i), cap, nullptr) + tile - 1) / tile;
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

// Units without a row: zeros and an lse of -inf, spread over the grid.
__device__ __forceinline__ void write_empty_units(const DecodePagedArgs& a, int G) {
    const int64_t cap = a.pc.per_unit * a.pc.rows;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = blockIdx.x + static_cast<int64_t>(gridDim.x) * threadIdx.x; i < a.sl.n;
         i += step) {
        if (clamp_nvalid(a.n_valid, slice_unit(a.sl, i), cap, nullptr) > 0) continue;
        float4* o = reinterpret_cast<float4*>(a.out + i * G * kD);
        for (int e = 0; e < G * kD / 4; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.lse)
            for (int h = 0; h < G; ++h) a.lse[i * G + h] = -INFINITY;
    }
}

__device__ __forceinline__ float ld_cg(const float* p) { return __ldcg(p); }

// log2-domain running maximum and sum -> natural logarithm of the softmax's
// denominator.
__device__ __forceinline__ float lse_of(float m, float l) {
    return l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : (l == 0.f ? -INFINITY : l);
}

// The tiles [begin, end) of unit i (first tile tile0, n_tiles tiles) are done
// and their (maximum, sum, accumulator) is written to this CTA's partial
// slot.  The CTA that arrives last joins the unit's partials in CTA order:
// out = sum_c 2^(m_c - M) acc_c / sum_c 2^(m_c - M) l_c.
// Called by the kThreads threads of named barrier kBar.
template <int kThreads, int kBar>
__device__ void join_split_unit(const DecodePagedArgs& a, int G, const SplitPlan& p, int64_t i,
                                int64_t tile0, int64_t n_tiles) {
    __shared__ bool last;
    const int tid = threadIdx.x;
    const int c0 = cta_of_tile(p.total, p.ctas, tile0);
    const int c1 = cta_of_tile(p.total, p.ctas, tile0 + n_tiles - 1);
    __threadfence();
    named_sync(kBar, kThreads);
    if (tid == 0) last = atomicAdd(a.counters + i, 1u) == static_cast<uint32_t>(c1 - c0);
    named_sync(kBar, kThreads);
    if (!last) return;
    __threadfence();
    for (int e = tid; e < G * kD; e += kThreads) {
        const int h = e / kD, d = e % kD;
        float M = -INFINITY;
        for (int c = c0; c <= c1; ++c) {
            const int slot = tile0 <= range_begin(p.total, p.ctas, c) ? 0 : 1;
            M = fmaxf(M, ld_cg(a.part + ((static_cast<int64_t>(c) * 2 + slot) * G + h) * (2 + kD)));
        }
        float num = 0.f, den = 0.f;
        for (int c = c0; c <= c1; ++c) {
            const int slot = tile0 <= range_begin(p.total, p.ctas, c) ? 0 : 1;
            const float* x = a.part + ((static_cast<int64_t>(c) * 2 + slot) * G + h) * (2 + kD);
            const float m = ld_cg(x);
            const float w = m == -INFINITY ? 0.f : exp2f(m - M);
            num = fmaf(w, ld_cg(x + 2 + d), num);
            den = fmaf(w, ld_cg(x + 1), den);
        }
        a.out[(i * G + h) * kD + d] = den == 0.f ? 0.f : num / den;
        if (a.lse && d == 0) a.lse[i * G + h] = lse_of(M, den);
    }
}

}  // namespace tri
