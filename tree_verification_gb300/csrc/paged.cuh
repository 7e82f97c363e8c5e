// Shared by the paged-cache kernels: argument checks, page lookup, the attention plan's layout.
#pragma once

#include <cuda_fp16.h>

#include <cstddef>

#include "common.cuh"

namespace graft {
namespace paged {

constexpr int HD = GRAFT_HEAD_DIM;

// Host checks of a cache's sizes; `tables` adds the arrays that reserve, fork and free need.
int check_cache(const GraftPagedCache* c);
int check_tables(const GraftPagedCache* c);

inline int log2_exact(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Copy on write holds for every writer: where the cache says who holds its pages, a sequence's rows are written only
// to pages among its own (entry k of its block-table row, k < held) that no other sequence holds.
__device__ __forceinline__ bool guarded(const GraftPagedCache& c) { return c.held != nullptr && c.page_refs != nullptr; }

// Does sequence b take part in the call?
__device__ __forceinline__ bool takes_part(const GraftPagedCache& c, int b) { return c.active == nullptr || c.active[b] != 0; }

// ---------------------------------------------------------------- the attention plan
// A work item of the attention is one entry (a block of query rows of one sequence) and one KV head,
// against a range of keys.  The plan is one buffer:
//   PlanHead | few entries | their unit prefix sums | the CTAs' first units |
//   wide row blocks, unsorted | wide items of whole rounds | the CTAs' last items | where each CTA's lie |
//   row blocks split by keys
// "Few" entries (paged_few.cu): sequences of at most few_rows query rows (new rows x group).  "Wide" ones
// (paged_wide.cu): all others, in blocks of two tiles of tile_tokens new rows.
struct PlanHead {
    int32_t magic, N, Hq, Hkv, n_seqs, max_new, tree, page_rows, max_pages, num_pages, few_rows, ctas;
    int32_t few_ctas;    // CTAs of the few kernel that have work
    int32_t rounds;      // whole rounds of wide items: every CTA takes one of each
    int32_t n_groups;    // row blocks split by keys
    int32_t tiles;       // tiles of such a row block at most
    int32_t reserved[15];
};
constexpr int32_t kPlanMagic = 0x47503033;

struct Entry {
    int32_t b;       // sequence
    int32_t q0;      // its first new row
    int32_t n, L;    // new rows, rows before them
    int32_t row0;    // first query row of the block (row = new row x group + head of the group)
    int32_t rows;    // query rows of the block
    int32_t keys;    // keys that any of them may see
    int32_t units;   // of 16 keys
};

constexpr int kBlockKeys = 128;

struct Wide {
    int32_t b, q0, n, L;  // sequence, its first new row, new rows, rows before them
    int32_t tok0;         // first new row of the block
    int32_t two;          // the block has a second tile
    int32_t blk0, nblk;   // range of 128-key blocks
    int32_t keys;         // keys that any row of the block may see
    int32_t kvh;          // KV head
    int32_t part;         // partial rows of the range, -1: the rows are written to O
    int32_t pad;
};

// A row block of one KV head whose key ranges are joined: partial rows part0, part0 + step, ...
struct Group {
    int32_t q0, n, tok0, tiles, kvh, ranges, part0, step;
};

// Where a CTA of the few kernel starts: everything its first item needs, in one read.  Either a CTA takes an even
// run of all units, over whatever items they belong to (step 0), or a share of one item alone.
struct Start {
    Entry e;
    int32_t entry, head, unit, count;  // units of the CTA
    int32_t ctas;                      // step 0: CTAs that share all units
    int32_t step, cta0, pieces;        // the item's pieces: CTAs cta0, cta0 + step, ...
    int64_t item_first;                // step 0: the item's first unit among all
    int64_t total;                     // step 0: all units
};

constexpr int kHeadBytes = offsetof(PlanHead, reserved);  // of the head's fields

struct PlanShape {
    int max_few;   // bound on the few entries
    int ctas;      // CTAs of the few kernel at most
    int few_warps; // warps of such a CTA
    int few_rows;  // query rows of a few entry at most (16 or 32)
    int few, wide; // whether the calls launch either kernel
    int sms;
    int tile_tokens;  // new rows of a 128-row tile
    int max_pairs;    // bound on the wide row blocks
    int max_groups;   // bound on the row blocks split by keys, 0: nothing is split
    size_t off_few, off_prefix, off_start, off_pairs, off_wide, off_last, off_where, off_group, bytes;
};

// CTA k of `ctas` takes units [first_unit(k), first_unit(k + 1)).
__host__ __device__ __forceinline__ int64_t first_unit(int64_t units, int ctas, int k) {
    const int64_t each = units / ctas, left = units % ctas;
    return each * k + (k < left ? k : left);
}
// The CTA that takes unit u.
__host__ __device__ __forceinline__ int unit_cta(int64_t units, int ctas, int64_t u) {
    const int64_t each = units / ctas, left = units % ctas, big = left * (each + 1);
    return (int)(u < big ? u / (each + 1) : left + (u - big) / each);
}

PlanShape plan_shape(const GraftPagedCache* c, int N, int Hq, int max_new);

// Partial results of cut items: every CTA has at most two (its first item's end, its last item's start).
constexpr int kFewRows = 32;
struct FewWs {
    int32_t* count;  // [2 x SMs] arrivals at the item that is cut and starts in a CTA, zero between calls
    float* o;        // [ctas][2][kFewRows][128]
    float2* ml;      // [ctas][2][kFewRows]: maximum (log2 units), sum
};

struct AttnArgs {
    GraftPagedCache c;
    const void* K;
    const void* V;
    const char* plan;
    const void* Q;
    int64_t q_stride;
    const uint64_t* mask;
    void* O;
    float scale;
    int N, Hq, G, max_new, page_shift;
    int after_wide;  // the few kernel runs beside the wide one
    uint64_t wait_ns;  // bound on every pipeline wait of the wide kernel (0.5 s unless tuned)
    PlanShape shape;
    FewWs few;
    float* wide_o;    // [partial row blocks][2][32][128][4] normalised: four dims of the 128 rows side by side
    float* wide_lse;  // [partial row blocks][2][128] log2-sum-exp
};

int wide_launch(const AttnArgs& a, cudaStream_t st);
int join_launch(const AttnArgs& a, cudaStream_t st);
int few_launch(const AttnArgs& a, cudaStream_t st);

// Is the plan one for these arguments?  (The lengths and row counts in it were checked when it was made.)
__device__ __forceinline__ bool plan_fits(const AttnArgs& a, const PlanHead& h) {
    return h.magic == kPlanMagic && h.N == a.N && h.Hq == a.Hq && h.Hkv == a.c.Hkv && h.n_seqs == a.c.n_seqs &&
           h.max_new == a.max_new && h.tree == (a.mask != nullptr) && h.page_rows == a.c.page_rows &&
           h.max_pages == a.c.max_pages && h.num_pages == a.c.num_pages && h.few_rows == a.shape.few_rows &&
           h.ctas == a.shape.ctas;
}

// ---------------------------------------------------------------- element types
template <int DT>
struct Elem;
template <>
struct Elem<GRAFT_BF16> {
    using T = __nv_bfloat16;
    using T2 = __nv_bfloat162;
    static __device__ __forceinline__ float2 up(uint32_t w) {
        return __bfloat1622float2(*reinterpret_cast<const T2*>(&w));
    }
    static __device__ __forceinline__ uint32_t down(float x, float y) {
        const T2 v = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    // either half of the pair is infinite or NaN: its exponent bits are all set
    static __device__ __forceinline__ bool odd(uint32_t w) {
        return ((w & 0x7f80u) == 0x7f80u) || ((w & 0x7f800000u) == 0x7f800000u);
    }
};
template <>
struct Elem<GRAFT_FP16> {
    using T = __half;
    using T2 = __half2;
    static __device__ __forceinline__ float2 up(uint32_t w) { return __half22float2(*reinterpret_cast<const T2*>(&w)); }
    static __device__ __forceinline__ uint32_t down(float x, float y) {
        const T2 v = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    static __device__ __forceinline__ bool odd(uint32_t w) {
        return ((w & 0x7c00u) == 0x7c00u) || ((w & 0x7c000000u) == 0x7c000000u);
    }
};

}  // namespace paged
}  // namespace graft
