// paged_core.cuh -- device helpers of the paged-cache kernels.
#pragma once

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
    uint32_t rows;    // its rows
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
    __shared__ uint32_t found[3];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t cap = a.pc.per_unit * a.pc.rows;
    const uint32_t units = static_cast<uint32_t>(a.sl.n);
    const uint32_t per = (units + kThreads - 1) / kThreads;
    const uint32_t i0 = min(tid * per, units), i1 = min(i0 + per, units);
    auto rows_of = [&](uint32_t i) -> uint32_t {
        return clamp_nvalid(a.n_valid, slice_unit(a.sl, i), cap, nullptr);
    };
    uint32_t sum = 0, n0 = 0;
#pragma unroll 4
    for (uint32_t i = i0; i < i1; ++i) {
        const uint32_t n = rows_of(i);
        if (i == i0) n0 = n;
        sum += (n + (tile - 1)) / tile;
    }
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
            const uint32_t n = i == i0 ? n0 : rows_of(i), nt = (n + (tile - 1)) / tile;
            if (p.begin < t + nt) {
                found[0] = i;
                found[1] = t;
                found[2] = n;
                break;
            }
            t += nt;
        }
    }
    __syncthreads();
    p.unit = found[0];
    p.tile0 = found[1];
    p.rows = found[2];
    return p;
}

// j / page_rows for j < 2^31 by a multiplication: with 2^l >= d > 2^(l-1) and
// m = floor(2^(31+l) / d) + 1, the product m d exceeds 2^(31+l) by at most 2^l,
// so floor(j m / 2^(31+l)) is exact.  (d = 1 has no such m: m = 0.)
struct PageDivide {
    uint32_t m, shift, rows;
    __device__ __forceinline__ uint32_t slot(uint32_t j) const { return m ? __umulhi(j, m) >> shift : j; }
};
inline PageDivide page_divide(int64_t rows) {
    PageDivide d = {0, 0, static_cast<uint32_t>(rows)};
    if (rows == 1) return d;
    uint32_t l = 1;
    while ((1ull << l) < d.rows) ++l;
    d.m = static_cast<uint32_t>((1ull << (31 + l)) / d.rows + 1);
    d.shift = l - 1;
    return d;
}

// A unit of a range of tiles that ends at `end`, and the row counts of the two
// units behind it (read ahead).
template <int kTile>
struct UnitCursor {
    uint32_t i, tile0, n, n_tiles;
    uint32_t t1;           // its tiles in the range end here
    uint32_t n1, n2;
    const int32_t* pages;  // its page table row

    __device__ static uint32_t rows_of(const DecodePagedArgs& a, uint32_t i) {
        if (i >= static_cast<uint32_t>(a.sl.n)) return 0;
        return clamp_nvalid(a.n_valid, slice_unit(a.sl, i), a.pc.per_unit * a.pc.rows, nullptr);
    }
    __device__ void set(const DecodePagedArgs& a, uint32_t end, uint32_t rows) {
        n = rows;
        n_tiles = (n + kTile - 1) / kTile;
        t1 = min(tile0 + n_tiles, end);
        pages = a.pc.table + slice_unit(a.sl, i) * a.pc.per_unit;
    }
    __device__ void first(const DecodePagedArgs& a, uint32_t unit, uint32_t unit_tile0, uint32_t rows,
                          uint32_t end) {
        i = unit;
        tile0 = unit_tile0;
        set(a, end, rows);
        n1 = rows_of(a, i + 1);
        n2 = rows_of(a, i + 2);
    }
    // The next unit with rows (there is one while t1 < end).
    __device__ UnitCursor next(const DecodePagedArgs& a, uint32_t end) const {
        UnitCursor x;
        x.tile0 = tile0 + n_tiles;
        x.i = i + 1;
        x.n1 = n2;
        uint32_t rows = n1;
        while (rows == 0 && x.i + 1 < static_cast<uint32_t>(a.sl.n)) {
            rows = x.n1;
            ++x.i;
            x.n1 = rows_of(a, x.i + 1);
        }
        x.i = min(x.i, static_cast<uint32_t>(a.sl.n) - 1);
        x.set(a, end, rows);
        x.n2 = rows_of(a, x.i + 2);
        return x;
    }
    // Page entry of row j, -1 past the last row.
    __device__ int32_t page(const PageDivide& d, uint32_t j) const { return j < n ? pages[d.slot(j)] : -1; }
};

// A kernel that was launched early (launch_early) waits here for the one before
// it: the attention for the clearing of the flag word and the counters, before
// it touches them.  Every warp of such a kernel does, else it could end, and
// what follows it begin, before the other one is done.
__device__ __forceinline__ void wait_for_clear() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Let fn use `bytes` of dynamic shared memory.  Asked at every call, like the
// other kernels': an answer kept from an earlier one would outlive the context
// that it was given for (cudaDeviceReset).
inline cudaError_t allow_smem(const void* fn, size_t bytes) {
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
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
// first and its last.  The partials of such a unit: n of them, of CTAs c0,
// c0 + 1, ..., the first in slot0, the others in slots 2 c.
struct SplitUnit {
    uint32_t i, c0, n, slot0;
};
__device__ __forceinline__ SplitUnit split_unit(const SplitPlan& p, uint32_t i, uint32_t tile0,
                                                uint32_t n_tiles) {
    SplitUnit s;
    s.i = i;
    s.c0 = cta_of_tile(p, tile0);
    s.n = cta_of_tile(p, tile0 + n_tiles - 1) - s.c0 + 1;
    s.slot0 = part_slot(p, s.c0, tile0);
    return s;
}
// Row of head h of the unit's x-th partial; x past the last one repeats it.
__device__ __forceinline__ uint32_t part_row(const SplitUnit& s, uint32_t x, int G, int h) {
    x = min(x, s.n - 1);
    return (x == 0 ? s.slot0 : 2 * (s.c0 + x)) * G + h;
}

__device__ __forceinline__ void fma4(float4& acc, float f, const float4& v) {
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
}

__device__ __forceinline__ void write_joined(const DecodePagedArgs& a, int64_t row, const float4& o, float M,
                                             float den) {
    const int lane = threadIdx.x & 31;
    reinterpret_cast<float4*>(a.out + row * kD)[lane] =
        den == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                   : make_float4(o.x / den, o.y / den, o.z / den, o.w / den);
    if (a.lse && lane == 0) a.lse[row] = lse_of(M, den);
}

// Heads of units of at most kFew partials, by one warp, kHeads of them at a
// time (n = 0: none): a lane has 4 dims and, by itself, all maxima and sums, so
// nothing is exchanged and all loads are in flight together.
constexpr int kFew = 4;
template <int kHeads>
__device__ void join_few(const DecodePagedArgs& a, int G, const SplitUnit (&s)[kHeads],
                         const int (&h)[kHeads]) {
    const int lane = threadIdx.x & 31;
    float2 x[kHeads][kFew];
    float4 v[kHeads][kFew];
#pragma unroll
    for (int r = 0; r < kHeads; ++r) {
#pragma unroll
        for (int y = 0; y < kFew; ++y) {
            if (s[r].n == 0) continue;
            const int64_t row = part_row(s[r], y, G, h[r]);
            x[r][y] = __ldcg(a.part_ml + row);
            v[r][y] = __ldcg(reinterpret_cast<const float4*>(a.part + row * kD) + lane);
        }
    }
#pragma unroll
    for (int r = 0; r < kHeads; ++r) {
        if (s[r].n == 0) continue;
        float M = x[r][0].x;
#pragma unroll
        for (int y = 1; y < kFew; ++y) M = fmaxf(M, x[r][y].x);
        const float base = M == -INFINITY ? 0.f : M;
        float den = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int y = 0; y < kFew; ++y) {
            if (y >= static_cast<int>(s[r].n)) continue;
            const float w = exp2f(x[r][y].x - base);
            den = fmaf(w, x[r][y].y, den);
            fma4(acc, w, v[r][y]);
        }
        write_joined(a, static_cast<int64_t>(s[r].i) * G + h[r], acc, M, den);
    }
}

// One head of a unit of any number of partials: lane c holds the maximum and
// sum of the c-th of 32, every lane 4 dims; kAhead accumulators are requested
// at a time.
template <int kAhead>
__device__ void join_many(const DecodePagedArgs& a, int G, const SplitUnit& s, int h) {
    const int lane = threadIdx.x & 31;
    float M = -INFINITY, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (uint32_t cb = 0; cb < s.n; cb += 32) {
        const float2 x = __ldcg(a.part_ml + part_row(s, cb + lane, G, h));
        float4 v[kAhead];
        auto request = [&](uint32_t c) {
#pragma unroll
            for (int y = 0; y < kAhead; ++y)
                v[y] = __ldcg(reinterpret_cast<const float4*>(
                                  a.part + static_cast<int64_t>(part_row(s, c + y, G, h)) * kD) + lane);
        };
        request(cb);
        const bool in = cb + lane < s.n;
        float m = in ? x.x : -INFINITY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = fmaxf(m, M);
        const float base = m == -INFINITY ? 0.f : m;
        const float f = exp2f(M - base);
        const float w = in ? exp2f(x.x - base) : 0.f;
        float l = in ? w * x.y : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        M = m;
        den = fmaf(den, f, l);
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll 1
        for (uint32_t b = 0; b < 32 && cb + b < s.n; b += kAhead) {
#pragma unroll
            for (int y = 0; y < kAhead; ++y) {
                const float g = __shfl_sync(0xffffffffu, w, b + y);
                if (cb + b + y < s.n) fma4(acc, g, v[y]);
            }
            if (b + kAhead < 32 && cb + b + kAhead < s.n) request(cb + b + kAhead);
        }
    }
    write_joined(a, static_cast<int64_t>(s.i) * G + h, acc, M, den);
}

// The partials of this CTA's n_split split units are written; of each unit the
// CTA that arrives last joins the partials in CTA order,
//   out = sum_c 2^(m_c - M) acc_c / sum_c 2^(m_c - M) l_c,
// a head a warp.  Called once, at the end, by the kWarps * 32 threads of named
// barrier kBar, so the fence and the atomics are paid once.  Bound by the
// latency of its loads.
template <int kWarps, int kBar, int kAhead>
__device__ void join_split_units(const DecodePagedArgs& a, int G, int n_split,
                                 const SplitUnit& s0, const SplitUnit& s1) {
    __shared__ bool last[2];
    const int tid = threadIdx.x, warp = tid >> 5;
    wait_for_clear();
    named_sync(kBar, kWarps * 32);
    if ((tid & 31) == 0 && warp < n_split) {
        const uint32_t i = warp ? s1.i : s0.i, n = warp ? s1.n : s0.n;
        __threadfence();
        last[warp] = atomicAdd(a.counters + i, 1u) == n - 1;
        __threadfence();
    }
    named_sync(kBar, kWarps * 32);
    // Head q: head q of the first unit that this CTA joins, or q - G of the other.
    const bool j0 = n_split > 0 && last[0], j1 = n_split > 1 && last[1];
    const int heads = (j0 ? G : 0) + (j1 ? G : 0);
    constexpr int kAtOnce = kAhead >= 16 ? 4 : 2;
#pragma unroll 1
    for (int q0 = warp; q0 < heads; q0 += kWarps * kAtOnce) {
        SplitUnit s[kAtOnce];
        int h[kAtOnce];
#pragma unroll
        for (int r = 0; r < kAtOnce; ++r) {
            const int q = q0 + r * kWarps;
            s[r] = j0 && q < G ? s0 : s1;
            h[r] = q >= G ? q - G : q;
            if (q >= heads || s[r].n > kFew) s[r].n = 0;
        }
        join_few(a, G, s, h);
    }
#pragma unroll 1
    for (int q = warp; q < heads; q += kWarps) {
        const SplitUnit s = j0 && q < G ? s0 : s1;
        if (s.n > kFew) join_many<kAhead>(a, G, s, q >= G ? q - G : q);
    }
}

}  // namespace tri
