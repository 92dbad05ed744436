// decode_paged.cu -- attention of the next token over a paged cache.
//
// For each unit (sequence, layer, KV head) and each of its G query heads h:
//   o_h = sum_{j < n} a_j v_j,  a_j = exp(s_j - m) / sum_{j' < n} exp(s_j' - m),
//   s_j = scale * (q_h . k_j),  m = max_j s_j,  lse_h = m + log sum_j exp(s_j - m),
// row j of the unit found through its page table (jaedaily.cn tutorial,
// KV-compression objective: the softmax renormalised over the kept rows).
//
// rows kernel (any page size, both types).  A CTA's tiles of 32 keys are cut
// into one contiguous run a warp; a warp streams its run, over changes of unit,
// through its own shared-memory ring in groups of 8 keys, copied row by row
// (cp.async; a row without a page copies zeros).  Units that lie in a warp's run
// are finished by it; the others' pieces are joined at the CTA's end.
//   scores   8 lanes share a key, 16 of its dims each, interleaved by 16-byte
//            chunks so that the lanes' reads fall on different banks; a lane
//            has two keys of the group at a time, which halves the reads of
//            Q.  The 8 lanes' partial sums of all heads are summed by a
//            transposing butterfly (7 shuffles for 8 heads and 8 lanes, where
//            32 lanes of 4 dims took 31), which leaves a lane the scores of
//            one head for its keys and the online softmax.
//   values   a lane has 4 dims; the weights come back through 256 bytes of
//            shared memory as pairs of heads, so a packed FFMA2 multiplies
//            two heads' weights with one dim.
// Scores, running maxima, sums and accumulators are float32.
//
// Bound: about 65 instructions a key and warp at 8 heads.  Over long float32
// caches (1.07 GB, pages of 24 rows) that keeps up with 88 % of the copy rate
// at 8 heads and 93 % at one; bf16 rows, twice as many a byte, with 51 % and 76 %
// (4 heads).  24 ragged sequences (174 MB) take 45 us: rows at full rate for 24,
// the rest is the ramp, runs of 3 and 4 tiles side by side, and the joins.
#include "paged_core.cuh"
#include "tri_launch.h"

namespace tri {

// The attention starts while this runs (wait_for_clear): on the device it hides
// behind the plan, where a memset in front of the kernel costs 0.5 to 1.3 us of
// the calls of 25 us and more (and saves the host 1 us of 22).
__global__ void __launch_bounds__(256) decode_clear_kernel(uint32_t* flag, uint32_t* counters, int64_t n) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t i = blockIdx.x * 256ll + threadIdx.x;
    if (i == 0) *flag = 0;
    if (i < n) counters[i] = 0;
}

constexpr int kRowThreads = 320;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kRowTile = 32;    // keys a warp takes at a time
constexpr int kGroup = 8;       // keys whose scores are formed together
constexpr int kRingBytes = 16384;  // of a warp: 2 groups of float32 rows, 4 of bf16

constexpr int row_heads_pad(int G) { return G <= 2 ? 2 : G <= 4 ? 4 : 8; }

// A warp's piece of a unit: the accumulators of every head (maxima and sums
// stay in shared memory).
constexpr size_t row_piece_floats(int G) { return static_cast<size_t>(G) * kD; }
struct RowPiece {
    uint32_t i, tile0, n_tiles;
    bool any;
};

struct RowShared {
    float p[kRowWarps][kGroup * 8];          // weights [key][head]
    float q[kRowWarps][TRI_MAX_GROUP * kD];  // [head][piece][lane of 8][4 dims]
    unsigned char ring[kRowWarps][kRingBytes];
    RowPiece piece[2 * kRowWarps];           // [warp][of the unit its run begins in, of its last unit]
    float2 piece_ml[2 * kRowWarps][TRI_MAX_GROUP];
};

__device__ __forceinline__ void copy16(void* dst, const void* src, bool valid) {
    const int n = valid ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 4 dims as two pairs.
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

// The same from global memory that nothing writes meanwhile.
__device__ __forceinline__ void read4(const float* p, float2& a, float2& b) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(p));
    a = make_float2(x.x, x.y);
    b = make_float2(x.z, x.w);
}
__device__ __forceinline__ void read4(const __nv_bfloat16* p, float2& a, float2& b) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
    a = make_float2(bf16_lo(x.x), bf16_hi(x.x));
    b = make_float2(bf16_lo(x.y), bf16_hi(x.y));
}

template <typename T, int G>
__global__ void __launch_bounds__(kRowThreads, 1) decode_paged_rows_kernel(const PageDivide divide, const DecodePagedArgs a) {
    constexpr int GP = row_heads_pad(G);     // heads of the butterfly
    constexpr int HP = (G + 1) / 2;          // pairs of heads
    constexpr int kRowBytes = kD * sizeof(T);
    constexpr int kGroupBytes = kGroup * 2 * kRowBytes;  // [K, V][key][row]
    constexpr int kRing = kRingBytes / kGroupBytes;
    constexpr int kChunkDims = 16 / sizeof(T);           // dims of a 16-byte chunk
    constexpr int kGroups = kRowTile / kGroup;
    constexpr size_t kPiece = row_piece_floats(G);
    extern __shared__ __align__(16) unsigned char smem[];
    RowShared& sm = *reinterpret_cast<RowShared*>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sub = lane & 7, quad = lane >> 3;  // lane of a key, key of four
    const SplitPlan p = plan_split<kRowThreads>(a, kRowTile, kRowWarps);
    unsigned char* ring = sm.ring[warp];
    float* pw = sm.p[warp];
    float* qw = sm.q[warp];
    // Pieces: the first one of a warp goes to global memory while the ring is
    // in use, the last one takes the ring's place.
    float* first_piece = a.pieces + (static_cast<int64_t>(blockIdx.x) * kRowWarps + warp) * kPiece;
    float* last_piece = reinterpret_cast<float*>(ring);
    const char* kp = static_cast<const char*>(a.k);
    const char* vp = static_cast<const char*>(a.v);

    // ---- this warp's run of tiles [t0, t1) and its first unit ----
    const uint32_t len = p.end - p.begin;
    const uint32_t t0 = p.begin + len * warp / kRowWarps, t1 = p.begin + len * (warp + 1) / kRowWarps;
    using Cursor = UnitCursor<kRowTile>;
    Cursor cur = {};
    if (t0 < t1) {
        uint32_t i = p.unit, tile0 = p.tile0, rows = p.rows;
        while (t0 >= tile0 + (rows + kRowTile - 1) / kRowTile) {  // 32 units at a time
            const uint32_t n = Cursor::rows_of(a, i + lane);
            const uint32_t nt = (n + kRowTile - 1) / kRowTile;
            uint32_t incl = nt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, t0 < tile0 + incl);
            if (past || i + 32 >= static_cast<uint32_t>(a.sl.n)) {
                const int w = past ? __ffs(past) - 1 : 31;
                i = min(i + w, static_cast<uint32_t>(a.sl.n) - 1);
                tile0 += __shfl_sync(0xffffffffu, incl - nt, w);
                rows = __shfl_sync(0xffffffffu, n, w);
                break;
            }
            // (Unit i + 32 has not been looked at: it is among the next 32.)
            tile0 += __shfl_sync(0xffffffffu, incl, 31);
            i += 32;
            rows = 0;
        }
        cur.first(a, i, tile0, rows, t1);
    }
    if (lane < 2) sm.piece[2 * warp + lane].any = false;

    // Q of a unit: piece r of lane s holds the 4 dims that it multiplies r-th.
    auto load_q = [&](uint32_t i) {
        const T* q = static_cast<const T*>(a.q) + static_cast<int64_t>(i) * G * kD + 4 * lane;
        float2 x[G][2];
#pragma unroll
        for (int h = 0; h < G; ++h) read4(q + h * kD, x[h][0], x[h][1]);
        const int chunk = 4 * lane / kChunkDims, part = lane % (kChunkDims / 4);  // dims 4 lane ..
        const int r = (chunk >> 3) * (kChunkDims / 4) + part;
        __syncwarp();
#pragma unroll
        for (int h = 0; h < G; ++h)
            *reinterpret_cast<float4*>(&qw[h * kD + (r * 8 + (chunk & 7)) * 4]) =
                make_float4(x[h][0].x, x[h][0].y, x[h][1].x, x[h][1].y);
        __syncwarp();
    };
    float2 acc[4][HP];  // [dim][pair of heads]
    // This lane's head; its l is over its own keys.
    const int my_head = sub / (8 / GP);
    float m = -INFINITY, l = 0.f;
    auto begin_unit = [&](uint32_t i) {
        load_q(i);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int h = 0; h < HP; ++h) acc[x][h] = make_float2(0.f, 0.f);
        m = -INFINITY;
        l = 0.f;
    };
    // The unit `w` ends in this run (or the run ends in it).
    auto end_unit = [&](const Cursor& w) {
        float sum = l;
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const bool whole = w.tile0 >= t0 && w.tile0 + w.n_tiles <= t1;
        const bool final = w.t1 == t1;
        float* to = final ? last_piece : first_piece;
        if (whole) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            float* o = a.out + static_cast<int64_t>(w.i) * G * kD + lane * 4;
#pragma unroll
            for (int h = 0; h < G; ++h) {
                const float f = __shfl_sync(0xffffffffu, inv, h * (8 / GP));
                const int x = h / 2;
                *reinterpret_cast<float4*>(o + h * kD) =
                    h & 1 ? make_float4(acc[0][x].y * f, acc[1][x].y * f, acc[2][x].y * f, acc[3][x].y * f)
                          : make_float4(acc[0][x].x * f, acc[1][x].x * f, acc[2][x].x * f, acc[3][x].x * f);
            }
            if (a.lse && quad == 0 && sub % (8 / GP) == 0 && my_head < G)
                a.lse[static_cast<int64_t>(w.i) * G + my_head] = lse_of(m, sum);
            return;
        }
        __syncwarp();  // (the ring's last reads)
#pragma unroll
        for (int h = 0; h < G; ++h) {
            const int x = h / 2;
            *reinterpret_cast<float4*>(to + h * kD + lane * 4) =
                h & 1 ? make_float4(acc[0][x].y, acc[1][x].y, acc[2][x].y, acc[3][x].y)
                      : make_float4(acc[0][x].x, acc[1][x].x, acc[2][x].x, acc[3][x].x);
        }
        const int e = 2 * warp + (final ? 1 : 0);
        if (quad == 0 && sub % (8 / GP) == 0 && my_head < G) sm.piece_ml[e][my_head] = make_float2(m, sum);
        if (lane == 0) sm.piece[e] = RowPiece{w.i, w.tile0, w.n_tiles, true};
    };

    // ---- the stream: groups g = 0, 1, ... of tiles t0, t0 + 1, ... ----
    const uint32_t n_groups = (t1 - t0) * kGroups;
    // Physical row of this lane's key of tile t of unit w, from its page
    // entry `page` (read a tile ahead of the first copy); -1: none.
    Cursor ahead = cur;  // the unit of the tile to be issued next
    auto key_of = [&](const Cursor& w, uint32_t t) { return (t - w.tile0) * kRowTile + lane; };
    int32_t page_ahead = t0 < t1 ? ahead.page(divide, key_of(ahead, t0)) : -1;
    int32_t row_issue = -1;
    uint32_t have = 0, have_issue = 0;  // keys with a row, of the tile used and the one issued
    auto issue = [&](uint32_t g) {
        if (g < n_groups) {
            const int gi = g % kGroups;
            if (gi == 0) {
                const uint32_t t = t0 + g / kGroups, j = key_of(ahead, t);
                const bool ok = page_ahead >= 0 && page_ahead < a.pc.n_pages;
                row_issue = ok ? static_cast<int32_t>(page_ahead * divide.rows + (j - divide.slot(j) * divide.rows)) : -1;
                if (!ok && j < ahead.n) {
                    wait_for_clear();
                    raise_flag(a.flag, TRI_FLAG_INDEX_RANGE);
                }
                have_issue = __ballot_sync(0xffffffffu, ok);
                if (t + 1 < t1) {
                    if (t + 1 == ahead.t1) ahead = ahead.next(a, t1);
                    page_ahead = ahead.page(divide, key_of(ahead, t + 1));
                }
            }
            unsigned char* slot = ring + (g % kRing) * kGroupBytes;
            constexpr int kLanes = kRowBytes / 16;  // of one row
#pragma unroll
            for (int x = 0; x < kGroup; x += 32 / kLanes) {
                const int key = x + lane / kLanes, off = lane % kLanes * 16;
                const int32_t r = __shfl_sync(0xffffffffu, row_issue, gi * kGroup + key);
                const int64_t src = static_cast<int64_t>(r < 0 ? 0 : r) * kRowBytes + off;
                copy16(slot + key * kRowBytes + off, kp + src, r >= 0);
                copy16(slot + (kGroup + key) * kRowBytes + off, vp + src, r >= 0);
            }
        }
        copy_commit();
    };
    if (n_groups) begin_unit(cur.i);  // (while the first page entry is on its way)
    for (int g = 0; g < kRing; ++g) issue(g);
    // (The ring is at most one tile ahead, so the tile in use is the one
    // issued or the one before it.)
    uint32_t have_next = have_issue;
    static_assert(kRing <= kGroups, "ring longer than a tile");
    for (uint32_t g = 0; g < n_groups; ++g) {
        const int gi = g % kGroups;
        if (gi == 0) {
            have = have_next;
            if (t0 + g / kGroups == cur.t1) {
                end_unit(cur);
                cur = cur.next(a, t1);
                begin_unit(cur.i);
            }
        }
        copy_wait<kRing - 1>();
        __syncwarp();
        const unsigned char* slot = ring + (g % kRing) * kGroupBytes;
        // ---- partial dot products of keys quad and quad + 4 ----
        float2 s0[G], s1[G];
#pragma unroll
        for (int h = 0; h < G; ++h) s0[h] = s1[h] = make_float2(0.f, 0.f);
        const T* k0 = reinterpret_cast<const T*>(slot + quad * kRowBytes);
        const T* k1 = reinterpret_cast<const T*>(slot + (quad + 4) * kRowBytes);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int dim = (sub + 8 * (r / (kChunkDims / 4))) * kChunkDims + r % (kChunkDims / 4) * 4;
            float2 x0, x1, y0, y1;
            load4(k0 + dim, x0, x1);
            load4(k1 + dim, y0, y1);
#pragma unroll
            for (int h = 0; h < G; ++h) {
                float2 q0, q1;
                load4(&qw[h * kD + (r * 8 + sub) * 4], q0, q1);
                s0[h] = __ffma2_rn(x0, q0, s0[h]);
                s0[h] = __ffma2_rn(x1, q1, s0[h]);
                s1[h] = __ffma2_rn(y0, q0, s1[h]);
                s1[h] = __ffma2_rn(y1, q1, s1[h]);
            }
        }
        // ---- the transposing butterfly over the key's 8 lanes ----
        float sa[GP], sb[GP];
#pragma unroll
        for (int h = 0; h < GP; ++h) {
            sa[h] = h < G ? s0[h < G ? h : 0].x + s0[h < G ? h : 0].y : 0.f;
            sb[h] = h < G ? s1[h < G ? h : 0].x + s1[h < G ? h : 0].y : 0.f;
        }
        int o = 4;
#pragma unroll
        for (int count = GP; count > 1; count >>= 1) {
            const bool up = sub & o;
#pragma unroll
            for (int x = 0; x < count / 2; ++x) {
                const float ka = up ? sa[x + count / 2] : sa[x], ga = up ? sa[x] : sa[x + count / 2];
                const float kb = up ? sb[x + count / 2] : sb[x], gb = up ? sb[x] : sb[x + count / 2];
                sa[x] = ka + __shfl_xor_sync(0xffffffffu, ga, o);
                sb[x] = kb + __shfl_xor_sync(0xffffffffu, gb, o);
            }
            o >>= 1;
        }
#pragma unroll
        for (; o > 0; o >>= 1) {
            sa[0] += __shfl_xor_sync(0xffffffffu, sa[0], o);
            sb[0] += __shfl_xor_sync(0xffffffffu, sb[0], o);
        }
        // ---- online softmax of my_head ----
        const uint32_t bits = have >> (gi * kGroup + quad);
        const bool va = bits & 1, vb = bits & 16;
        float mx = fmaxf(va ? sa[0] * a.scale_log2 : -INFINITY, vb ? sb[0] * a.scale_log2 : -INFINITY);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float m_new = fmaxf(m, mx);
        const float base = m_new == -INFINITY ? 0.f : m_new;
        // (one rounding of the small difference, not of the large product)
        const float wa = va ? exp2f(fmaf(sa[0], a.scale_log2, -base)) : 0.f;
        const float wb = vb ? exp2f(fmaf(sb[0], a.scale_log2, -base)) : 0.f;
        if (__any_sync(0xffffffffu, m_new != m)) {
            const float al = exp2f(m - base);
            l *= al;
#pragma unroll
            for (int h = 0; h < HP; ++h) {
                const float a0 = __shfl_sync(0xffffffffu, al, 2 * h * (8 / GP));
                const float a1 = __shfl_sync(0xffffffffu, al, (2 * h + 1) * (8 / GP));
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    acc[x][h].x *= a0;
                    acc[x][h].y *= a1;
                }
            }
            m = m_new;
        }
        l += wa + wb;
        if (sub % (8 / GP) == 0) {
            pw[quad * GP + my_head] = wa;
            pw[(quad + 4) * GP + my_head] = wb;
        }
        __syncwarp();
        // ---- values ----
#pragma unroll
        for (int key = 0; key < kGroup; ++key) {
            float2 v01, v23;
            load4(reinterpret_cast<const T*>(slot + (kGroup + key) * kRowBytes) + lane * 4, v01, v23);
            float2 w[GP / 2];
#pragma unroll
            for (int h = 0; h < GP / 2; h += 2) {
                if constexpr (GP >= 4)
                    load4(pw + key * GP + 2 * h, w[h], w[h + 1 < GP / 2 ? h + 1 : h]);
                else
                    w[h] = *reinterpret_cast<const float2*>(pw + key * GP);
            }
#pragma unroll
            for (int h = 0; h < HP; ++h) {
                acc[0][h] = __ffma2_rn(w[h], make_float2(v01.x, v01.x), acc[0][h]);
                acc[1][h] = __ffma2_rn(w[h], make_float2(v01.y, v01.y), acc[1][h]);
                acc[2][h] = __ffma2_rn(w[h], make_float2(v23.x, v23.x), acc[2][h]);
                acc[3][h] = __ffma2_rn(w[h], make_float2(v23.y, v23.y), acc[3][h]);
            }
        }
        __syncwarp();  // the group's slot and the weights are rewritten
        issue(g + kRing);
        if ((g + kRing) % kGroups == 0) have_next = have_issue;
    }
    copy_wait<0>();
    if (n_groups) end_unit(cur);
    // ---- the pieces, in the order of the warps; those of one unit follow one
    // another.  A warp takes a head of a unit: a lane has 4 dims. ----
    __syncthreads();
    SplitUnit split0 = {}, split1 = {};
    int n_split = 0, turn = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < 2 * kRowWarps;) {
        const RowPiece w = sm.piece[e0];
        if (!w.any) {
            ++e0;
            continue;
        }
        int e1 = e0 + 1;
        while (e1 < 2 * kRowWarps && (!sm.piece[e1].any || sm.piece[e1].i == w.i)) ++e1;
        const bool whole = w.tile0 >= p.begin && w.tile0 + w.n_tiles <= p.end;
        const uint32_t slot = part_slot(p, blockIdx.x, w.tile0);
#pragma unroll 1
        for (int h = 0; h < G; ++h) {
            if (turn++ % kRowWarps != warp) continue;
            float M = -INFINITY;
            for (int x = e0; x < e1; ++x)
                if (sm.piece[x].any) M = fmaxf(M, sm.piece_ml[x][h].x);
            const float base = M == -INFINITY ? 0.f : M;
            float den = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int x = e0; x < e1; ++x) {
                if (!sm.piece[x].any) continue;
                const float2 ml = sm.piece_ml[x][h];
                const float f = exp2f(ml.x - base);
                const float* from = x & 1 ? reinterpret_cast<const float*>(sm.ring[x >> 1])
                                          : a.pieces + (static_cast<int64_t>(blockIdx.x) * kRowWarps + (x >> 1)) * kPiece;
                den = fmaf(f, ml.y, den);
                fma4(o, f, reinterpret_cast<const float4*>(from + h * kD)[lane]);
            }
            if (whole) {
                write_joined(a, static_cast<int64_t>(w.i) * G + h, o, M, den);
            } else {
                reinterpret_cast<float4*>(a.part + (static_cast<int64_t>(slot) * G + h) * kD)[lane] = o;
                if (lane == 0) a.part_ml[slot * G + h] = make_float2(M, den);
            }
        }
        if (!whole) {
            split1 = split_unit(p, w.i, w.tile0, w.n_tiles);
            if (n_split++ == 0) split0 = split1;
        }
        e0 = e1;
    }
    join_split_units<kRowWarps, 0, 8>(a, G, n_split, split0, split1);
    write_empty_units(a, G);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int decode_paged_ctas(int n_sm) { return n_sm; }

size_t decode_paged_piece_bytes(int G) { return kRowWarps * row_piece_floats(G) * sizeof(float); }

cudaError_t launch_decode_paged_clear(const DecodePagedArgs& a, cudaStream_t s) {
    decode_clear_kernel<<<static_cast<unsigned>((a.sl.n + 255) / 256), 256, 0, s>>>(a.flag, a.counters,
                                                                                   a.sl.n);
    note_launch(s);
    return cudaGetLastError();
}

template <typename T, int G>
static cudaError_t launch_rows(const DecodePagedArgs& a, int n_sm, cudaStream_t s) {
    constexpr size_t smem = sizeof(RowShared);
    static_assert(row_piece_floats(G) * 4 <= kRingBytes && smem <= 227 * 1024, "shared memory");
    auto* fn = decode_paged_rows_kernel<T, G>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), smem);
    if (e != cudaSuccess) return e;
    e = launch_decode_paged_clear(a, s);
    if (e != cudaSuccess) return e;
    e = launch_early(fn, decode_paged_ctas(n_sm), kRowThreads, smem, s, page_divide(a.pc.rows), a);
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
