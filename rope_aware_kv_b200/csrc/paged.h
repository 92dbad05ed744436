// paged.h -- launchers of the paged-cache operators: decode attention through
// a page table (decode_paged.cu), append and the page calls (pages.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/tri.h"

namespace tri {

// A paged cache: row j of unit u is row j % rows of page table[u * per_unit +
// j / rows]; entries outside [0, n_pages) hold no page.
struct PagedCache {
    int32_t* table;
    int64_t per_unit;
    int64_t rows;
    int64_t n_pages;
    int64_t n_seq;
    int64_t n_units;
};

// The units of one call: all of them (layer < 0) or one layer's, in the unit
// order [n_seq][n_layers][n_kvheads].
struct UnitSlice {
    int64_t n;          // units of the call
    int64_t n_layers;
    int64_t n_kvheads;
    int64_t layer;
};

// decode_paged.cu
struct DecodePagedArgs {
    const void* q;           // [sl.n][G][128]
    const void* k;           // [n_pages][rows][128]
    const void* v;
    PagedCache pc;
    UnitSlice sl;
    const int32_t* n_valid;  // [n_units]
    float scale_log2;        // scale * log2(e)
    float* out;              // [sl.n][G][128]
    float* lse;              // [sl.n][G] or null
    uint32_t* counters;      // [sl.n]: segments of a unit that are done
    // Partial results of split units, two slots a CTA: accumulators
    // [2 * ctas][G][128] and (maximum, sum) [2 * ctas][G].
    float* part;
    float2* part_ml;
    float* pieces;           // scratch of the row kernel, decode_paged_piece_bytes a CTA
    uint32_t* flag;
};
int decode_paged_ctas(int n_sm);
size_t decode_paged_piece_bytes(int G);
// The first kernel of the call: clears the flag word and the counters while
// the second one begins.
cudaError_t launch_decode_paged_clear(const DecodePagedArgs& a, cudaStream_t s);
// Any page size, both types.
cudaError_t launch_decode_paged_rows(tri_dtype dt, int G, const DecodePagedArgs& a, int n_sm,
                                     cudaStream_t s);

// decode_paged_tc.cu: bf16 pages of a multiple of 8 rows, through the tensor
// cores.  kmap, vmap: the pools as {64 dims, 8 rows, 2 halves, groups of 8
// rows}, boxes of box_rows rows (box_rows / 8 groups), 128-byte swizzle.
constexpr int kTcTile = 128;  // keys of one tile
int decode_paged_box_rows(int64_t page_rows);  // 0: not served
cudaError_t launch_decode_paged_tc(int G, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                   int box_rows, const DecodePagedArgs& a, int n_sm,
                                   cudaStream_t s);

// pages.cu
struct AppendPagedArgs {
    void* k;
    void* v;                  // null: keys only
    int32_t* pos;             // [n_units][cap] or null
    int64_t cap;
    PagedCache pc;
    UnitSlice sl;
    const int32_t* refs;      // null: no page is shared
    int32_t* n_valid;
    int64_t* p_cur;           // [n_seq] or null
    const void* k_new;        // [sl.n][n_new][128]
    const void* v_new;
    const int32_t* pos_new;   // [sl.n][n_new]
    const int32_t* n_add;     // [n_seq] or null
    int64_t n_new;
    int32_t* first;           // scratch [sl.n]: row the unit's new rows begin at, -1: refused
    uint32_t* flag;
};
cudaError_t launch_append_paged(tri_dtype dt, const AppendPagedArgs& a, cudaStream_t s);

int page_ctas(int n_sm);  // CTAs of fit and compact

struct FitArgs {
    void* k;
    void* v;
    PagedCache pc;
    int32_t* refs;
    const int32_t* n_valid;
    const int32_t* n_add;     // [n_seq] or null
    int64_t n_new;
    int own;
    int32_t* n_free;          // or null
    // scratch
    uint32_t* writers;        // [n_pages], zero on entry: slots of the page that will be written
    uint32_t* last;           // [n_pages], zero on entry: 1 + the last of them
    uint4* counts;            // [ctas]: pages asked for, of them copies, free pages
    int32_t* need_slot;       // [min(slots, pages)]: the i-th request's slot
    int32_t* need_old;        //   and the page it copies (-1: none)
    int4* copies;             // [min(slots, pages)]: page that is copied, request, rows
    int32_t* free_page;       // [min(slots, pages)]: the i-th free page
    uint32_t* barrier;        // zero on entry
    uint32_t* flag;
};
cudaError_t launch_pages_fit(tri_dtype dt, const FitArgs& a, int n_sm, cudaStream_t s);

constexpr int kMaxForks = 1024;

struct ForkArgs {
    PagedCache pc;
    int32_t* refs;
    int32_t* n_valid;
    int32_t* pos;             // [n_units][cap] or null
    int64_t cap;
    int64_t* p_cur;           // [n_seq] or null
    const int32_t* src;
    const int32_t* dst;
    int64_t n_fork;
    uint32_t* done;           // [n_units / n_seq], zero on entry: jobs that are done
    uint32_t* flag;
};
cudaError_t launch_pages_fork(const ForkArgs& a, int n_sm, cudaStream_t s);

struct CompactPagesArgs {
    void* k;
    void* v;
    PagedCache pc;
    int32_t* refs;
    int32_t* n_live;          // or null
    // scratch
    uint4* counts;            // [ctas]: live pages
    int32_t* from;            // [n_pages / 2]: the i-th page that moves
    int32_t* to;              //   and where it goes
    int32_t* rank;            // [n_pages]: i of a page that moves
    uint32_t* barrier;        // zero on entry
    uint32_t* flag;
};
cudaError_t launch_pages_compact(tri_dtype dt, const CompactPagesArgs& a, int n_sm,
                                 cudaStream_t s);

}  // namespace tri
