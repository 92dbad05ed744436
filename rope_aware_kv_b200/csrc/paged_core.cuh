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

// log2-domain running maximum and sum -> natural logarithm of the softmax's
// denominator.
__device__ __forceinline__ float lse_of(float m, float l) {
    return l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : (l == 0.f ? -INFINITY : l);
}

// Partial result of a unit's segment: slot 2 c of CTA c, or 2 c + 1 for a unit
// that begins inside the CTA's range.
__device__ __forceinline__ int64_t part_slot(const SplitPlan& p, int c, int64_t tile0) {
    return 2 * static_cast<int64_t>(c) + (tile0 <= range_begin(p.total, p.ctas, c) ? 0 : 1);
}

// This CTA's partial of unit i (first tile tile0, n_tiles tiles) is written;
// the CTA that arrives last joins the unit's partials in CTA order,
//   out = sum_c 2^(m_c - M) acc_c / sum_c 2^(m_c - M) l_c.
// Called by the kWarps * 32 threads of named barrier kBar.  A lane has 4 dims
// of every head; the warps take the CTAs in turn, so the loads of a warp are
// independent of one another, and are joined in warp order through red
// ((kWarps - 1) * G * 128 floats of shared memory).
template <int kWarps, int kBar, int G>
__device__ void join_split_unit(const DecodePagedArgs& a, const SplitPlan& p, int64_t i,
                                int64_t tile0, int64_t n_tiles, float* red) {
    __shared__ bool last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c0 = cta_of_tile(p.total, p.ctas, tile0);
    const int c1 = cta_of_tile(p.total, p.ctas, tile0 + n_tiles - 1);
    __threadfence();
    named_sync(kBar, kWarps * 32);
    if (tid == 0) last = atomicAdd(a.counters + i, 1u) == static_cast<uint32_t>(c1 - c0);
    named_sync(kBar, kWarps * 32);
    if (!last) return;
    __threadfence();
    float M[G], den[G];
    float4 acc[G];
#pragma unroll
    for (int h = 0; h < G; ++h) {
        M[h] = -INFINITY;
        den[h] = 0.f;
        acc[h] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int c = c0 + lane; c <= c1; c += 32) {
        const float2* ml = a.part_ml + part_slot(p, c, tile0) * G;
#pragma unroll
        for (int h = 0; h < G; ++h) M[h] = fmaxf(M[h], __ldcg(ml + h).x);
    }
#pragma unroll
    for (int h = 0; h < G; ++h) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M[h] = fmaxf(M[h], __shfl_xor_sync(0xffffffffu, M[h], o));
    }
    for (int cb = c0; cb <= c1; cb += 32) {
        float w[G];
        const bool in = cb + lane <= c1;
        const float2* ml = a.part_ml + part_slot(p, in ? cb + lane : cb, tile0) * G;
#pragma unroll
        for (int h = 0; h < G; ++h) {
            const float2 x = __ldcg(ml + h);
            w[h] = in && x.x != -INFINITY ? exp2f(x.x - M[h]) : 0.f;
            if (in) den[h] = fmaf(w[h], x.y, den[h]);
        }
        const int m = min(32, c1 - cb + 1);
#pragma unroll 2
        for (int x = warp; x < m; x += kWarps) {
            const float4* src =
                reinterpret_cast<const float4*>(a.part + part_slot(p, cb + x, tile0) * G * kD) + lane;
#pragma unroll
            for (int h = 0; h < G; ++h) {
                const float4 v = __ldcg(src + h * 32);
                const float f = __shfl_sync(0xffffffffu, w[h], x);
                acc[h].x = fmaf(f, v.x, acc[h].x);
                acc[h].y = fmaf(f, v.y, acc[h].y);
                acc[h].z = fmaf(f, v.z, acc[h].z);
                acc[h].w = fmaf(f, v.w, acc[h].w);
            }
        }
    }
#pragma unroll
    for (int h = 0; h < G; ++h) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) den[h] += __shfl_xor_sync(0xffffffffu, den[h], o);
        if (warp > 0) reinterpret_cast<float4*>(red)[((warp - 1) * G + h) * 32 + lane] = acc[h];
    }
    named_sync(kBar, kWarps * 32);
    if (warp > 0) return;
#pragma unroll
    for (int h = 0; h < G; ++h) {
        float4 o = acc[h];
#pragma unroll
        for (int x = 0; x < kWarps - 1; ++x) {
            const float4 v = reinterpret_cast<const float4*>(red)[(x * G + h) * 32 + lane];
            o.x += v.x;
            o.y += v.y;
            o.z += v.z;
            o.w += v.w;
        }
        const float d = den[h];
        reinterpret_cast<float4*>(a.out + (i * G + h) * kD)[lane] =
            d == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                     : make_float4(o.x / d, o.y / d, o.z / d, o.w / d);
        if (a.lse && lane == 0) a.lse[i * G + h] = lse_of(M[h], d);
    }
}

}  // namespace tri
