// Log probabilities of given tokens, with entropy, rank and top alternatives, from rows of given logits.
//
//   z = x / T, m = max z, s = sum e^(z - m), t = sum (z - m) e^(z - m):
//   log p(v) = (z_v - m) - ln s,  H = ln s - t / s,
//   rank(v) = #{x > x_v} + #{x = x_v at lower ids},  the top k by (x descending, id ascending).
//
// Every logit of the rows asked for is read once (4 or 2 bytes) and costs about ten instructions: HBM bounds fp32, the
// issue of instructions 16-bit logits (1024 rows of 151936: fp32 109 us, 5.7 TB/s; bf16 69 us, 4.5 TB/s).
// logprob_part_kernel lays the rows' chunks (32 fp32 or 64 16-bit logits a thread) side by side and gives every team of
// threads an even run of them, so all end together whatever the number of rows; the next chunk comes through a ring in
// shared memory (cp.async, each thread its own pieces: no barrier) while one is worked on.  A thread keeps its own
// maximum and sums over its run's part of a row: a chunk's by themselves, then added to the part's in two numbers.  A
// team is a CTA; where rows are short (kShort), a warp that takes whole rows, without barriers.  logprob_join_kernel
// adds up the pieces of rows that a run's edges cut, in their order.
//
// Top alternatives cost the pass one store a thread and chunk, a bound of the chunk's largest of the thread's logits.
// Once a segment (kSeg chunks, or a row's end) a threshold is taken that at least k of the threads' largest reach; the
// pieces above it (some 50) are read once more, all threads at once; what passes goes to a buffer in shared memory and
// finds its place by counting (20 alternatives of the rows above: 126 us; 209 with candidates pushed and merged a chunk
// at a time).  Where more pass than the buffer holds (long runs of equal or of rising logits), the segment is gone
// through chunk by chunk instead.
#include <climits>
#include <cmath>
#include <type_traits>

#include <cuda_fp16.h>

#include "common.cuh"

namespace graft {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// CTAs an SM, of 128 registers.  (Three of 80, tried with chunks half as long, left spills in the 16-bit kernels: 1024 rows
// of 151936 in fp32 138 us, 134 with two; bf16 161 and 120.)
constexpr int kResident = 2;
constexpr int kSeg = 40;       // chunks of a segment
constexpr int kMaxRows = 128;  // rows of a CTA's runs at most
constexpr int kShort = 4096;   // logits of a row that a warp takes
constexpr float kFloor = -150.f;  // log2 of a weight that is zero in 32 bits
// log2 of the largest weight before the sums are moved to a new maximum.  (ln s and t / s cancel where a token is all but
// certain: at 16 an entropy near 0 was off by 11 x 2^-24.)
constexpr float kSlack = 2.f;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int DT>
constexpr int kElems = DT == GRAFT_F32 ? 4 : 8;  // of 16 bytes
// 16-byte pieces of a chunk a thread, and chunks in shared memory (one worked on, one on its way).  When it was chosen, 1024
// rows of 151936 with 20 alternatives, eight pieces and four (and four chunks): fp32 126 and 131 us, bf16 98 and 100; 1999
// rows of 32768 in bf16 39 and 43 (of 8192, half a chunk, 19 and 15.5).
constexpr int kVecs = 8, kStages = 2;
constexpr int kRing = kStages * kVecs * kThreads * 16;

struct Args {
    const char* logits;
    const char* logits_end;
    int64_t stride;  // bytes
    const int32_t* rows;
    const int32_t* tokens;
    int64_t R;
    int N, V, block, top, chunks;  // chunks of a row
    int ctas;
    float c1;     // log2(e) / T
    float inv_T, inv_T_rest;  // 1 / T
    float* logprob;
    float* entropy;
    int32_t* rank;
    int32_t* top_id;
    float* top_logprob;
    int32_t* status;
    // workspace
    int32_t* n_rows;    // rows that are asked for
    float4* sums;       // [N + ctas] of a piece: m, s, t, bits of the count of better tokens
    int2* entry;        // [N + ctas]: the entry (its complement where it has no token), bits of its token's logit
    uint64_t* keys;     // [N + ctas][top]
};

// (32-bit where it fits: a 64-bit division takes a hundred instructions)
__device__ __forceinline__ int64_t quotient(int64_t x, int y) {
    return ((uint64_t)x >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}
// How `units` are shared out: part k of `parts` takes [first(k), first(k + 1)).
struct Shares {
    int64_t each;
    int left, parts;
    __device__ __forceinline__ Shares(int64_t units, int64_t most) {
        parts = (int)(units < most ? units : most);
        each = parts > 0 ? quotient(units, parts) : 0;
        left = (int)(units - each * parts);
    }
    __device__ __forceinline__ int64_t first(int k) const { return each * k + (k < left ? k : left); }
    __device__ __forceinline__ int of(int64_t u) const {
        const int64_t big = left * (each + 1);
        return (int)(u < big ? quotient(u, (int)(each + 1)) : left + quotient(u - big, (int)each));
    }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// A logit and its id as a number that rises with the logit and falls with the id; 0: none.
__device__ __forceinline__ uint64_t key_of(float x, int id) {
    const uint32_t b = __float_as_uint(x + 0.f);
    const uint32_t o = b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
    return (uint64_t)o << 32 | (uint32_t)~id;
}
__device__ __forceinline__ float key_value(uint64_t k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ int key_id(uint64_t k) { return (int)~(uint32_t)k; }

// The best 32 of two falling lists, in falling order.
__device__ __forceinline__ uint64_t merge_keys(uint64_t a, uint64_t b, int lane) {
    const uint64_t r = __shfl_sync(0xffffffffu, b, 31 - lane);
    uint64_t k = a > r ? a : r;
#pragma unroll
    for (int step = 16; step > 0; step >>= 1) {
        const uint64_t o = __shfl_xor_sync(0xffffffffu, k, step);
        k = ((lane & step) == 0) == (k > o) ? k : o;
    }
    return k;
}
// A warp's 32 values in falling order.
__device__ __forceinline__ float sort_values(float v, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int step = size >> 1; step > 0; step >>= 1) {
            const float o = __shfl_xor_sync(0xffffffffu, v, step);
            const bool high = ((lane & step) == 0) == ((lane & size) == 0);
            v = high ? fmaxf(v, o) : fminf(v, o);
        }
    return v;
}

// Maxima, sums and counts (m, s, t, n) of kLanes neighbouring lanes added up: the sums are moved to the largest maximum.
template <int kLanes>
__device__ __forceinline__ void add_lanes(float4& v, float c1) {
    float m = v.x;
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    // (a lane of -inf alone has sums of zero, or NaN)
    const float d = v.x == -INFINITY ? 0.f : (v.x - m) * c1, f = ex2(d);
    v.z = f * (v.z + max_nan(d, kFloor) * v.y);
    v.y *= f;
    v.x = m;
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) {
        v.y += __shfl_xor_sync(0xffffffffu, v.y, d);
        v.z += __shfl_xor_sync(0xffffffffu, v.z, d);
        v.w += __shfl_xor_sync(0xffffffffu, v.w, d);
    }
}

// A pair of logits in 32 bits.
template <int DT>
__device__ __forceinline__ float2 pair(const uint4& w, int i) {
    const uint32_t* p = &w.x;
    if (DT == GRAFT_F32) return make_float2(__uint_as_float(p[2 * i]), __uint_as_float(p[2 * i + 1]));
    const uint32_t x = p[i];
    if (DT == GRAFT_BF16) return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
}
template <int DT>
__device__ __forceinline__ float load_logit(const char* row, int id) {
    if (DT == GRAFT_F32) return reinterpret_cast<const float*>(row)[id];
    const unsigned short h = reinterpret_cast<const unsigned short*>(row)[id];
    return DT == GRAFT_BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}
// Two 16-bit logits in a word.
template <int DT>
struct Two {
    using T = __nv_bfloat162;
    static __device__ __forceinline__ T both(float x) { return __floats2bfloat162_rn(x, x); }
    static __device__ __forceinline__ float2 up(T x) { return __bfloat1622float2(x); }
};
template <>
struct Two<GRAFT_FP16> {
    using T = __half2;
    static __device__ __forceinline__ T both(float x) { return __floats2half2_rn(x, x); }
    static __device__ __forceinline__ float2 up(T x) { return __half22float2(x); }
};
// The largest of kN x 16 bytes of logits (NaN aside).
template <int DT, int kN>
__device__ __forceinline__ float largest(const uint4* w) {
    if constexpr (DT == GRAFT_F32) {
        float m[kN];
#pragma unroll
        for (int x = 0; x < kN; ++x)
            m[x] = fmaxf(fmaxf(__uint_as_float(w[x].x), __uint_as_float(w[x].y)),
                         fmaxf(__uint_as_float(w[x].z), __uint_as_float(w[x].w)));
#pragma unroll
        for (int x = 1; x < kN; ++x) m[0] = fmaxf(m[0], m[x]);
        return m[0];
    } else {
        typename Two<DT>::T m[kN];
#pragma unroll
        for (int x = 0; x < kN; ++x) {
            const auto* p = reinterpret_cast<const typename Two<DT>::T*>(&w[x].x);
            m[x] = __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3]));
        }
#pragma unroll
        for (int x = 1; x < kN; ++x) m[0] = __hmax2(m[0], m[x]);
        const float2 f = Two<DT>::up(m[0]);
        return fmaxf(f.x, f.y);
    }
}
// The largest number of the logits' type below x (of -inf: itself).
template <int DT>
__device__ __forceinline__ float below(float x) {
    const uint32_t step = DT == GRAFT_BF16 ? 0x10000u : 1u;
    const uint32_t b = __float_as_uint(x);
    if (DT == GRAFT_FP16) {
        const uint32_t h = __half_as_ushort(__float2half_rn(x));
        const uint32_t p = h == 0u || h == 0x8000u ? 0x8001u : h >> 15 ? (h == 0xfc00u ? h : h + 1) : h - 1;
        return __half2float(__ushort_as_half((unsigned short)p));
    }
    if (x == 0.f) return __uint_as_float(0x80000000u + step);
    if (x == -INFINITY) return x;
    return __uint_as_float(b >> 31 ? b + step : b - step);
}
// How many of 16 bytes of logits lie above x, added to n: two counts, of 16-bit logits in 16 bits (exact up to 2^8).
template <int DT>
__device__ __forceinline__ void count_above(const uint4& w, float x, float2& n) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float2 v = pair<DT>(w, e);
        float2 y;
        asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(y.x) : "f"(v.x), "f"(x));
        asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(y.y) : "f"(v.y), "f"(x));
        n = __fadd2_rn(n, y);
    }
}
template <int DT>
__device__ __forceinline__ void count_above(const uint4& w, float x, typename Two<DT>::T& n) {
    const auto* p = reinterpret_cast<const typename Two<DT>::T*>(&w.x);
    const auto y = Two<DT>::both(x);
#pragma unroll
    for (int e = 0; e < 4; ++e) n = __hadd2(n, __hgt2(p[e], y));
}
// 16 bytes of logits from id on that reach past the row's ends: -inf there.  `have`: they were read; else they reach
// past the logits' own ends and are read one by one.  (Out of line: rare, and long.)
template <int DT>
__device__ __noinline__ uint4 ragged(uint4 v, bool have, const char* row, int id, int V) {
    uint32_t* w = &v.x;
#pragma unroll
    for (int e = 0; e < kElems<DT>; ++e) {
        const bool in = id + e >= 0 && id + e < V;
        if (DT == GRAFT_F32) {
            if (!in) w[e] = 0xff800000u;
            else if (!have) w[e] = reinterpret_cast<const uint32_t*>(row)[id + e];
        } else {
            uint32_t h = (w[e >> 1] >> (16 * (e & 1))) & 0xffffu;
            if (!in) h = DT == GRAFT_BF16 ? 0xff80u : 0xfc00u;
            else if (!have) h = reinterpret_cast<const unsigned short*>(row)[id + e];
            w[e >> 1] = (e & 1) ? (w[e >> 1] & 0xffffu) | h << 16 : (w[e >> 1] & 0xffff0000u) | h;
        }
    }
    return v;
}
// How many of 16 bytes of logits from their e0-th on equal x.
template <int DT>
__device__ __noinline__ float count_equal(uint4 w, int e0, float x) {
    float n = 0.f;
#pragma unroll
    for (int e = 0; e < kElems<DT>; ++e) {
        const float2 p = pair<DT>(w, e / 2);
        n += e >= e0 && ((e & 1) ? p.y : p.x) == x ? 1.f : 0.f;
    }
    return n;
}
// How many of 16 bytes of logits from id on go ahead of token tok, of logit x (NaN as -inf).
template <int DT>
__device__ __noinline__ float count_ahead(uint4 w, int id, int tok, float x) {
    float n = 0.f;
#pragma unroll
    for (int e = 0; e < kElems<DT>; ++e) {
        const float2 p = pair<DT>(w, e / 2);
        const float v = fmaxf((e & 1) ? p.y : p.x, -INFINITY);
        n += v > x || (v == x && id + e >= 0 && id + e < tok) ? 1.f : 0.f;
    }
    return n;
}

// The law of a row from its maximum and the sum of its weights relative to that.
struct Law {
    float m, whole, rest;  // ln s in two parts
    bool lawful;
    // a row of -inf alone has no law, nor has one with NaN or +inf: NaN
    // The last few operations keep what they round off, as logits, maxima and ln s may be larger than what is left of
    // them: (x - m) / T in two parts, ln s = e ln 2 + ln f with e 2839 / 4096 exact.
    __device__ __forceinline__ Law(float m, float s) : m(m), lawful(m > -INFINITY && s < INFINITY) {
        constexpr float kLn2 = 2839.f / 4096.f, kLn2Rest = 3.1946184945309e-5f;
        int e;
        float f = frexpf(s, &e);
        if (f < 0.70710678f) {  // (near one: of a certain token, s = 1, ln s is 0)
            f *= 2.f;
            --e;
        }
        rest = lawful ? e * kLn2Rest + logf(f) : NAN;
        whole = e * kLn2;
    }
    __device__ __forceinline__ float logp(const Args& a, float x) const {
        const float d = x - m, q = d * a.inv_T;
        if (!(fabsf(q) < INFINITY)) return q - rest;
        const float back = d + m, lost = x - back + (m - (back - d));  // of x - m
        const float left = fmaf(d, a.inv_T, -q) + d * a.inv_T_rest + lost * a.inv_T;
        const float sum = q - whole, gone = sum - q;
        return sum + (((q - (sum - gone)) + (-whole - gone)) + (left - rest));
    }
};

// The outputs of entry n but its alternatives: its token's logit (ok: it has one), the sums of the weights relative to
// the maximum, the better tokens' number.
__device__ __forceinline__ void answer(const Args& a, const Law& law, int n, bool ok, float given, float s, float t, int cnt) {
    a.logprob[n] = ok ? law.logp(a, given) : 0.f;
    if (a.entropy != nullptr) a.entropy[n] = law.whole + law.rest - 0.693147181f * (t / s);
    if (a.rank != nullptr) a.rank[n] = ok ? cnt : -1;
}

// The outputs of entry n, by a warp, with a key a lane.
__device__ __forceinline__ void finish(const Args& a, int n, bool ok, float given, float m, float s, float t, int cnt,
                                       uint64_t list) {
    const int lane = threadIdx.x & 31;
    const Law law(m, s);
    if (lane == 0) answer(a, law, n, ok, given, s, t, cnt);
    if (a.top > 0) {
        int id = key_id(list);
        float lp = list != 0 ? law.logp(a, key_value(list)) : 0.f;
        const unsigned have = __ballot_sync(0xffffffffu, list != 0);
        const int known = __popc(have);
        if (known < a.top) {
            // Fewer tokens above -inf than places: all of them are listed, the lowest other ids follow.
            uint64_t used = 0;
            for (int k = 0; k < known; ++k) {
                const int x = __shfl_sync(0xffffffffu, id, k);
                if (x < 64) used |= 1ull << x;
            }
            if (lane >= known) {
                int skip = lane - known;
                id = 0;
                while ((used >> id & 1) || skip-- > 0) ++id;
                lp = law.lawful ? -INFINITY : NAN;
            }
        }
        if (lane < a.top) {
            a.top_id[(int64_t)n * a.top + lane] = id;
            a.top_logprob[(int64_t)n * a.top + lane] = lp;
        }
    }
}

template <int DT, bool kWarpTeam>
__global__ void __launch_bounds__(kThreads, kResident)
logprob_part_kernel(const __grid_constant__ Args a) {
    constexpr int E = kElems<DT>;
    constexpr int kBytes = DT == GRAFT_F32 ? 4 : 2;
    constexpr int kTeams = kWarpTeam ? kWarps : 1;       // of a CTA
    constexpr int kTeam = kThreads / kTeams;             // threads of a team
    constexpr int kMaxChunks = kWarpTeam ? kShort / (32 * kVecs * E) + 1 : kSeg;
    extern __shared__ __align__(16) unsigned char s_ring[];  // [stage][piece][thread] 16 bytes
    __shared__ int s_entry[kMaxRows], s_tok[kMaxRows];
    __shared__ const char* s_row[kMaxRows];
    __shared__ int s_may[kMaxRows];  // which of its pieces may be read
    __shared__ float2 s_xt[kMaxRows];  // the given token's logit, and the largest number below it
    constexpr int kCap = kWarpTeam ? 1024 : 256;
    __shared__ unsigned short s_max[kMaxChunks][kThreads];  // a segment's largest, by chunk and thread: upper bf16 bounds
    constexpr int kParts = kWarpTeam ? 1 : kWarps;
    __shared__ float4 s_part[kMaxRows][kParts];  // the sums of the rows' parts, by warp
    __shared__ float4 s_total[kThreads];  // a thread's sums over its part's chunks, and what they round off
    __shared__ uint64_t s_cand[kCap + kTeams * 32];  // candidates, and the best so far behind them
    __shared__ uint64_t s_list[kTeams][32];          // the best so far, best first; 0: none
    __shared__ int s_hit[kCap];                      // chunk and thread whose largest reaches the threshold
    __shared__ int s_n[kTeams][2], s_hits[kTeams][2], s_scan[kWarps];
    __shared__ float s_reach[32];
    __shared__ uint64_t s_best[kWarps];
    griddep_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
    // ---- which rows
    // A row number is good if it lies within the logits and, with blocks, within its block.  (Where the logits hold all
    // of the entries' blocks, as they do in a step, that takes no division.)
    const bool whole = a.block > 0 && a.R >= ((int64_t)a.N + a.block - 1) / a.block * a.block;
    auto good = [&](int n, int64_t r) {
        if (r < 0) return false;
        if (a.block == 0) return r < a.R;
        return r < a.block && (whole || (int64_t)(n / a.block) * a.block + r < a.R);
    };
    // With `rows`: kLook entries a lane side by side, kThreads x kLook at a time.  have[x]: the warp's entries that
    // have a row among the x-th 32.
    constexpr int kLook = 16, kLot = kThreads * kLook;
    int n_rows = a.N;
    int32_t given[kLook];
    unsigned have[kLook];
    auto entry_of = [&](int n0, int x) { return n0 + (warp * kLook + x) * 32 + lane; };
    auto look = [&](int n0) {  // how many rows the warps before this one have, and how many there are
#pragma unroll
        for (int x = 0; x < kLook; ++x) given[x] = entry_of(n0, x) < a.N ? a.rows[entry_of(n0, x)] : -1;
        int mine = 0;
#pragma unroll
        for (int x = 0; x < kLook; ++x) {
            have[x] = __ballot_sync(0xffffffffu, good(entry_of(n0, x), given[x]));
            mine += __popc(have[x]);
        }
        __syncthreads();
        if (lane == 0) s_scan[warp] = mine;
        __syncthreads();
        int2 n = make_int2(0, 0);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) n.x += s_scan[w];
            n.y += s_scan[w];
        }
        return n;
    };
    int2 seen = make_int2(0, 0);
    if (a.rows != nullptr) {
        n_rows = 0;
        const int each = (a.N + (int)gridDim.x - 1) / (int)gridDim.x;  // entries without a row: every CTA sees to its share
        for (int n0 = 0; n0 < a.N; n0 += kLot) {
            seen = look(n0);
            n_rows += seen.y;
#pragma unroll
            for (int x = 0; x < kLook; ++x) {
                const int n = entry_of(n0, x);
                if (n >= a.N || (have[x] >> lane & 1) || n < cta * each || n >= (cta + 1) * each) continue;
                if (given[x] != -1) flag_status(a.status, GRAFT_STATUS_ROW);
                a.logprob[n] = 0.f;
                if (a.entropy != nullptr) a.entropy[n] = 0.f;
                if (a.rank != nullptr) a.rank[n] = -1;
                for (int k = 0; k < a.top; ++k) {
                    a.top_id[(int64_t)n * a.top + k] = -1;
                    a.top_logprob[(int64_t)n * a.top + k] = 0.f;
                }
            }
        }
    }
    if (cta == 0 && tid == 0) *a.n_rows = n_rows;
    // The teams' runs: units of a chunk, or of a row where a warp takes it whole.
    const int per_row = kWarpTeam ? 1 : a.chunks;
    const Shares shares((int64_t)n_rows * per_row, (int64_t)gridDim.x * kTeams);
    const int teams = shares.parts, t_first = cta * kTeams;  // the CTA's first team
    if (t_first >= teams) return;
    const int64_t cta_u0 = shares.first(t_first), cta_u1 = shares.first(min(t_first + kTeams, teams));
    const int cta_r0 = (int)quotient(cta_u0, per_row), cta_r1 = (int)quotient(cta_u1 - 1, per_row);
    auto take = [&](int r, int n, int64_t at) {
        s_entry[r - cta_r0] = n;
        s_row[r - cta_r0] = a.logits + at * a.stride;
    };
    if (a.rows == nullptr) {
        for (int r = cta_r0 + tid; r <= cta_r1; r += kThreads) take(r, r, r);
    } else {
        for (int n0 = 0, r0 = 0; n0 < a.N; n0 += kLot) {
            if (a.N > kLot) seen = look(n0);  // (else they are at hand)
            int r = r0 + seen.x;
#pragma unroll
            for (int x = 0; x < kLook; ++x) {
                const int n = entry_of(n0, x), at = r + __popc(have[x] & ((1u << lane) - 1u));
                if ((have[x] >> lane & 1) && at >= cta_r0 && at <= cta_r1)
                    take(at, n, a.block > 0 ? (int64_t)(n / a.block) * a.block + given[x] : given[x]);
                r += __popc(have[x]);
            }
            r0 += seen.y;
        }
    }
    if (tid < 2 * kTeams) s_n[tid >> 1][tid & 1] = s_hits[tid >> 1][tid & 1] = 0;
    __syncthreads();
    auto offset_of = [&](const char* row) { return (int)(reinterpret_cast<uintptr_t>(row) & 15) / kBytes; };
    // A row's chunks start at the 16 bytes that its first logit lies in.
    auto start_of = [&](const char* row) {
        return reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(row) & ~(uintptr_t)15);
    };
    static_assert(kMaxRows <= kThreads, "a row a thread");
    const bool listed_row = tid <= cta_r1 - cta_r0;
    if (listed_row) {
        // What of other rows lies in a row's first and last 16 bytes may be read, what lies around the logits may not: the
        // first piece of the first row, the last one of the last.  (Bit 0: not the first; above it: how many from there.)
        const char* row = s_row[tid];
        const int first = start_of(row) < a.logits, pieces = (offset_of(row) + a.V + E - 1) / E;
        const int64_t there = (a.logits_end - start_of(row)) / 16;
        s_may[tid] = max((there < pieces ? (int)there : pieces) - first, 0) << 1 | first;
    }
    __syncthreads();
    const int team = kWarpTeam ? warp : 0;
    const bool idle = t_first + team >= teams;  // (warps of the last CTA)
    const int ttid = kWarpTeam ? lane : tid;
    auto sync = [&]() {
        if (kWarpTeam) __syncwarp();
        else __syncthreads();
    };
    constexpr int kTeamCap = kCap / kTeams;
    uint64_t* cand = s_cand + team * (kTeamCap + 32);

    // ---- the run: chunk c of row j of the list
    const int64_t u0 = shares.first(t_first + (idle ? 0 : team));
    int left = idle ? 0 : (int)(shares.first(t_first + team + 1) - u0) * (kWarpTeam ? a.chunks : 1);  // chunks
    const int row0 = (int)quotient(u0, per_row);
    const int j0 = row0 - cta_r0, c0 = (int)(u0 - (int64_t)row0 * per_row);
    int j = j0, c = c0;
    constexpr int kChunk = kVecs * kTeam * E;  // logits
    // chunks of a row that lie within it: [x, y)
    auto inside_of = [&](int off) { return make_int2(off != 0, (a.V + off) / kChunk); };
    auto readable = [&](const char* p) { return p >= a.logits && p + 16 <= a.logits_end; };
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(s_ring)) + tid * 16;
    constexpr uint32_t kStageBytes = kVecs * kThreads * 16;
    int j_in = j, c_in = c, in = left;
    uint32_t dst = ring;
    const char* src = start_of(s_row[j]) + ((int64_t)c * (kVecs * kTeam) + ttid) * 16;
    int2 in_may, in_whole;  // of the row: pieces of 16 bytes, x and [x, x + y) of them; chunks wholly among them, [x, y)
    auto begin_in = [&](int j) {
        const int may = s_may[j];
        in_may = make_int2(may & 1, may >> 1);
        in_whole = make_int2(in_may.x, (in_may.x + in_may.y) / (kVecs * kTeam));
    };
    begin_in(j);
    auto issue = [&]() {  // the next chunk's copies (a thread's own pieces: it waits for them alone)
        if (in > 0) {
            if (c_in >= in_whole.x && c_in < in_whole.y) {
#pragma unroll
                for (int x = 0; x < kVecs; ++x) cp_async16(dst + x * kThreads * 16, src + x * kTeam * 16);
            } else {
                const unsigned piece = (unsigned)(c_in * kVecs * kTeam + ttid) - in_may.x;
#pragma unroll
                for (int x = 0; x < kVecs; ++x)
                    if (piece + x * kTeam < (unsigned)in_may.y) cp_async16(dst + x * kThreads * 16, src + x * kTeam * 16);
            }
            --in;
            src += kVecs * kTeam * 16;
            if (++c_in == a.chunks) {
                c_in = 0;
                ++j_in;
                if (in > 0) {
                    src = start_of(s_row[j_in]) + ttid * 16;
                    begin_in(j_in);
                }
            }
        }
        dst = dst + kStageBytes == ring + kStages * kStageBytes ? ring : dst + kStageBytes;
        cp_commit();
    };
    static_assert(kStages == 2, "one chunk ahead");
    // The tokens and their logits: a read each among the first copies (behind all of them they took 6 us).
    const int my_tok = listed_row ? a.tokens[s_entry[tid]] : -1;
    issue();
    if (listed_row) {
        const bool ok = my_tok >= 0 && my_tok < a.V;
        const float v = ok ? fmaxf(load_logit<DT>(s_row[tid], my_tok), -INFINITY) : INFINITY;  // (NaN ranks with -inf)
        s_tok[tid] = ok ? my_tok : -1;
        s_xt[tid] = make_float2(v, below<DT>(v));
        if (!ok && my_tok != -1) flag_status(a.status, GRAFT_STATUS_TOKEN_RANGE);
    }
    __syncthreads();
    if (idle) return;  // (warps alone from here on)

    // ---- the row at hand
    const char* row = nullptr;
    int off = 0, tok = -1;
    int2 in_row = make_int2(0, 0);   // chunks within the row
    int tok_chunk = -1;              // the given token's
    int one_by_one = -1;             // up to this chunk better tokens are counted one by one
    float2 xt = make_float2(INFINITY, INFINITY);
    auto begin_row = [&]() {
        row = s_row[j];
        off = offset_of(row);
        in_row = inside_of(off);
        tok = s_tok[j];
        if (tok >= 0 && a.rank != nullptr) {
            xt = s_xt[j];
            tok_chunk = (tok + off) / kChunk;
            one_by_one = xt.x > -INFINITY ? -1 : tok_chunk;  // (there is no number below -inf to compare with)
        } else {
            xt = make_float2(INFINITY, INFINITY);
            tok_chunk = one_by_one = -1;
        }
    };
    begin_row();
    int stage = 0;
    float m = -INFINITY;
    float2 cnt = make_float2(0.f, 0.f);
    s_total[tid] = make_float4(0.f, 0.f, 0.f, 0.f);
    float seg_max = -INFINITY;
    int turn = 0, c_part = c, c_seg = c;  // the part's and the segment's first chunk
    while (true) {
        const int c2 = c + 1 == a.chunks ? 0 : c + 1;
        auto id_of = [&](int c, int x) { return ((c * kVecs + x) * kTeam + ttid) * E - off; };
        issue();
        cp_wait<kStages - 1>();
        uint4 cur[kVecs];
#pragma unroll
        for (int x = 0; x < kVecs; ++x)
            cur[x] = *reinterpret_cast<const uint4*>(s_ring + ((stage * kVecs + x) * kThreads + tid) * 16);
        stage = stage + 1 == kStages ? 0 : stage + 1;
        if (c < in_row.x || c >= in_row.y) {
#pragma unroll
            for (int x = 0; x < kVecs; ++x) {
                const int id = id_of(c, x);
                if (id >= a.V) {
                    constexpr uint32_t kNone = DT == GRAFT_F32 ? 0xff800000u : DT == GRAFT_BF16 ? 0xff80ff80u : 0xfc00fc00u;
                    cur[x] = make_uint4(kNone, kNone, kNone, kNone);
                } else if (id < 0 || id + E > a.V) {
                    cur[x] = ragged<DT>(cur[x], readable(row + (int64_t)id * kBytes), row, id, a.V);
                }
            }
        }
        // ---- maximum, sums
        const float top = fmaxf(largest<DT, kVecs>(cur), -INFINITY);  // (of NaN alone: -inf)
        // The sums are relative to a maximum that moves only when weights would pass 2^kSlack.
        if (!((top - m) * a.c1 <= kSlack) && top > m) {
            if (m != -INFINITY) {
                const float d = (m - top) * a.c1, f = ex2(d), dd = max_nan(d, kFloor);
                const float4 v = s_total[tid];
                s_total[tid] = make_float4(f * v.x, f * (v.y + dd * v.x), f * v.z, f * (v.w + dd * v.z));
            }
            m = top;
        }
        {
            // A chunk's sums by themselves, then added to those of the chunks before, which keep what they round off: over a
            // long row of alike weights one chain of sums went one way (ln s of 2^20 logits 3e-5 off, of 2^24 3e-4).
            float2 s = make_float2(0.f, 0.f), t = s;
            const float base = m == -INFINITY ? 0.f : -m;
            const float2 base2 = make_float2(base, base), c12 = make_float2(a.c1, a.c1);
#pragma unroll
            for (int x = 0; x < kVecs; ++x) {
                if (x == kVecs / 2 && (c * kVecs + x) * kTeam * E - off >= a.V) break;  // (the row ends in the first half)
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    float2 d = __fmul2_rn(__fadd2_rn(pair<DT>(cur[x], e), base2), c12);
                    d.x = max_nan(d.x, kFloor);
                    d.y = max_nan(d.y, kFloor);
                    const float2 w = make_float2(ex2(d.x), ex2(d.y));
                    s = __fadd2_rn(s, w);
                    t = __ffma2_rn(d, w, t);
                }
            }
            const float4 v = s_total[tid];
            const float2 before = make_float2(v.x, v.y);
            const float2 more = __fadd2_rn(make_float2(s.x + s.y, t.x + t.y), make_float2(-v.z, -v.w));
            const float2 sum = __fadd2_rn(before, more);
            const float2 over = make_float2((sum.x - v.x) - more.x, (sum.y - v.y) - more.y);
            s_total[tid] = make_float4(sum.x, sum.y, over.x, over.y);
        }
        // ---- tokens ahead of the given one
        if (c > one_by_one) {
            // A piece that starts ahead of the token counts equal ones too; of the token's own, those from the token on
            // are taken off again.  (A likely token has few ahead of it: most chunks have none.)
            if (__any_sync(0xffffffffu, top > (c <= tok_chunk ? xt.y : xt.x))) {
                if constexpr (DT == GRAFT_F32) {
#pragma unroll
                    for (int x = 0; x < kVecs; ++x) count_above<DT>(cur[x], id_of(c, x) < tok ? xt.y : xt.x, cnt);
                } else {
                    auto n = Two<DT>::both(0.f);
#pragma unroll
                    for (int x = 0; x < kVecs; ++x) count_above<DT>(cur[x], id_of(c, x) < tok ? xt.y : xt.x, n);
                    cnt = __fadd2_rn(cnt, Two<DT>::up(n));
                }
                if (c == tok_chunk) {
#pragma unroll
                    for (int x = 0; x < kVecs; ++x)
                        if (id_of(c, x) < tok && tok < id_of(c, x) + E)
                            cnt.x -= count_equal<DT>(cur[x], tok - id_of(c, x), xt.x);
                }
            }
        } else {
#pragma unroll
            for (int x = 0; x < kVecs; ++x) cnt.x += count_ahead<DT>(cur[x], id_of(c, x), tok, xt.x);
        }
        if (a.top > 0) {
            const uint32_t b = __float_as_uint(top);
            s_max[c - c_seg][tid] = (unsigned short)((b >> 31 ? b : b + 0xffffu) >> 16);
            seg_max = fmaxf(seg_max, top);
        }
        const bool ends = c2 == 0 || left == 1;  // the part's last chunk
        if (ends) {
            const float4 sums = s_total[tid];
            float4 v = make_float4(m, sums.x - sums.z, sums.y - sums.w, cnt.x + cnt.y);
            add_lanes<32>(v, a.c1);
            if (lane == 0) s_part[j][kWarpTeam ? 0 : warp] = v;
        }
        // ---- alternatives
        if (a.top > 0 && (ends || c - c_seg == kSeg - 1)) {
            const float v = sort_values(seg_max, lane);
            float tau;
            if (kWarpTeam) {
                tau = __shfl_sync(0xffffffffu, v, a.top - 1);
            } else {
                // Reached by at least k threads' largest: what 8 / 2^i warps reach 2^i ceil(k / 8) times each, for i
                // up to 3 (short segments leave warps without logits), the largest of these.
                const int each = (a.top + kWarps - 1) / kWarps;
                const float q = __shfl_sync(0xffffffffu, v, min((each << (lane & 3)) - 1, 31));
                if (lane < 4) s_reach[lane * kWarps + warp] = q;
                __syncthreads();
                const float r = s_reach[lane];  // of warp lane & 7, 2^(lane / 8) ceil(k / 8) times
                int ahead = 0;
#pragma unroll
                for (int d = 1; d < kWarps; ++d) {
                    const int o = (lane & 24) | ((lane + d) & 7);
                    const float w = __shfl_sync(0xffffffffu, r, o);
                    ahead += w > r || (w == r && o < lane);
                }
                tau = ahead == (kWarps >> (lane >> 3)) - 1 ? r : -INFINITY;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) tau = fmaxf(tau, __shfl_xor_sync(0xffffffffu, tau, d));
            }
            // (of equal logits the lower id goes first, so a full list's last has to be passed, the threshold reached)
            bool listed = c_seg != c_part;  // the list holds what came before
            float kth = -INFINITY;          // its last, if it is full
            auto last_listed = [&]() {
                const uint64_t last = s_list[team][a.top - 1];
                return last != 0 ? key_value(last) : -INFINITY;
            };
            if (listed) kth = last_listed();
            auto passes = [&](float v) { return v >= tau && v > kth; };
            if (passes(seg_max)) {
#pragma unroll 8
                for (int x = 0; x <= c - c_seg; ++x) {
                    if (!passes(__uint_as_float((uint32_t)s_max[x][tid] << 16))) continue;
                    const int at = atomicAdd(&s_hits[team][turn], 1);
                    if (at < kTeamCap) s_hit[team * kTeamCap + at] = x * kTeam + ttid;
                }
            }
            sync();
            // A thread reads one piece of one of them again: all at once, as the reads queue behind the copies under way.
            const int hits = s_hits[team][turn];
            for (int y = ttid; y < min(hits, kTeamCap) * kVecs; y += kTeam) {
                const int hit = s_hit[team * kTeamCap + y / kVecs], x = hit / kTeam;
                const int id = (((c_seg + x) * kVecs + y % kVecs) * kTeam + hit % kTeam) * E - off;
                uint4 again = make_uint4(0, 0, 0, 0);
                if (id >= 0 && id + E <= a.V) again = *reinterpret_cast<const uint4*>(row + (int64_t)id * kBytes);
                else again = ragged<DT>(again, false, row, id, a.V);
                if (!passes(largest<DT, 1>(&again))) continue;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float2 p = pair<DT>(again, e / 2);
                    const float v = (e & 1) ? p.y : p.x;
                    if (passes(v)) {
                        const int at = atomicAdd(&s_n[team][turn], 1);
                        if (at < kTeamCap) cand[at] = key_of(v, id + e);
                    }
                }
            }
            sync();
            // (the other counters are cleared here: all have read them, and none adds to them before the next barrier)
            int n = hits > kTeamCap ? kTeamCap + 1 : s_n[team][turn];
            if (kWarpTeam) __syncwarp();
            if (ttid == 0) s_n[team][turn ^ 1] = s_hits[team][turn ^ 1] = 0;
            turn ^= 1;
            // The best of the list and n candidates, by their ranks among each other (0 is nobody's key: any order).
            auto merge = [&](int n) {
                if (listed) {
                    if (ttid < a.top) cand[n + ttid] = s_list[team][ttid];
                    n += a.top;
                    sync();
                }
                for (int x = ttid; x < max(n, a.top); x += kTeam) {
                    const uint64_t mine = x < n ? cand[x] : 0;
                    int rank = x < n ? 0 : x;
                    if (x < n) {
#pragma unroll 4
                        for (int y = 0; y < n; ++y) {
                            const uint64_t o = cand[y];
                            rank += o > mine || (o == mine && y < x);
                        }
                    }
                    if (rank < a.top) s_list[team][rank] = mine;
                }
                listed = true;
                sync();
            };
            if (n <= kTeamCap) {
                merge(n);
            } else {
                // More than the buffer holds: chunk by chunk, the best that pass one by one, each chunk against the
                // list as the last one left it.
                for (int cc = c_seg; cc <= c; ++cc) {
                    const int lo = max(cc * kChunk - off, 0), hi = min((cc + 1) * kChunk - off, a.V);
                    n = 0;
                    for (uint64_t last = ~0ull; n < a.top; ++n) {
                        uint64_t best = 0;
                        for (int id = lo + ttid; id < hi; id += kTeam) {
                            const float v = load_logit<DT>(row, id);
                            const uint64_t key = key_of(v, id);
                            if (passes(v) && key < last && key > best) best = key;
                        }
#pragma unroll
                        for (int d = 16; d > 0; d >>= 1) {
                            const uint64_t o = __shfl_xor_sync(0xffffffffu, best, d);
                            best = o > best ? o : best;
                        }
                        if (!kWarpTeam) {
                            __syncthreads();
                            if (lane == 0) s_best[warp] = best;
                            __syncthreads();
#pragma unroll
                            for (int w = 0; w < kWarps; ++w) best = s_best[w] > best ? s_best[w] : best;
                        }
                        if (best == 0) break;
                        last = best;
                        if (ttid == 0) cand[n] = best;
                    }
                    sync();
                    merge(n);
                    kth = last_listed();
                    sync();
                }
            }
            seg_max = -INFINITY;
            c_seg = c + 1;
        }
        if (ends) {
            if ((kWarpTeam || warp == 0) && lane < a.top)
                a.keys[((int64_t)(cta_r0 + j) + cta) * a.top + lane] = s_list[team][lane];
            m = seg_max = -INFINITY;
            cnt = make_float2(0.f, 0.f);
            s_total[tid] = make_float4(0.f, 0.f, 0.f, 0.f);
            c_part = c_seg = c2;
        }
        c = c2;
        if (--left == 0) break;
        if (c2 == 0) {
            ++j;
            begin_row();
        }
    }
    // The rows end here, side by side.  (One by one in the run, by a warp that the others waited for, that took 4000 to 7000
    // cycles a row: 1999 rows of 32003 in bf16 51 us, 45.5 here.)
    sync();
    auto given_of = [&](int x) {
        return make_int2(s_tok[x] >= 0 ? s_entry[x] : ~s_entry[x], __float_as_int(s_xt[x].x));
    };
    auto is_whole = [&](int x) { return (x > j0 || c0 == 0) && (x < j || c == 0); };
    if (a.top > 0) {
#pragma unroll 1
        for (int x = j0 + (kWarpTeam ? 0 : warp); x <= j; x += kParts) {
            float4 v = s_part[x][kWarpTeam ? 0 : lane & 7];
            if (!kWarpTeam) add_lanes<kWarps>(v, a.c1);
            const int64_t slot = (int64_t)(cta_r0 + x) + cta;
            if (is_whole(x)) {
                const uint64_t list = lane < a.top ? a.keys[slot * a.top + lane] : 0;
                finish(a, s_entry[x], s_tok[x] >= 0, s_xt[x].x, v.x, v.y, v.z, (int)v.w, list);
            } else if (lane == 0) {
                a.sums[slot] = make_float4(v.x, v.y, v.z, __int_as_float((int)v.w));
                a.entry[slot] = given_of(x);
            }
        }
        return;
    }
    for (int x = j0 + ttid; x <= j; x += kTeam) {
        float4 v = s_part[x][0];
#pragma unroll
        for (int w = 1; w < kParts; ++w) v.x = fmaxf(v.x, s_part[x][w].x);
        const float m = v.x;
        v.y = v.z = v.w = 0.f;
#pragma unroll
        for (int w = 0; w < kParts; ++w) {
            const float4 o = s_part[x][w];
            const float d = o.x == -INFINITY ? 0.f : (o.x - m) * a.c1, f = ex2(d);
            v.y += f * o.y;
            v.z += f * (o.z + max_nan(d, kFloor) * o.y);
            v.w += o.w;
        }
        if (is_whole(x)) {
            answer(a, Law(v.x, v.y), s_entry[x], s_tok[x] >= 0, s_xt[x].x, v.y, v.z, (int)v.w);
        } else {
            const int64_t slot = (int64_t)(cta_r0 + x) + cta;
            a.sums[slot] = make_float4(v.x, v.y, v.z, __int_as_float((int)v.w));
            a.entry[slot] = given_of(x);
        }
    }
}

constexpr int kJoinWarps = 4;

// Adds up the pieces of the rows that are cut: a CTA a row.  A warp merges every fourth piece's alternatives, the
// first one adds the sums.
template <int DT>
__global__ void __launch_bounds__(kJoinWarps * 32)
logprob_join_kernel(const __grid_constant__ Args a) {
    griddep_enter();
    __shared__ uint64_t s_keys[kJoinWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n_rows = *a.n_rows;
    const Shares shares((int64_t)n_rows * a.chunks, a.ctas);
    for (int r = blockIdx.x; r < n_rows; r += gridDim.x) {
        const int c0 = shares.of((int64_t)r * a.chunks), c1 = shares.of((int64_t)(r + 1) * a.chunks - 1);
        const int64_t slot0 = (int64_t)r + c0;
        const int pieces = c1 - c0 + 1;
        if (pieces == 1) continue;
        const int2 e = a.entry[slot0];
        uint64_t list = 0;
        if (a.top > 0) {
            for (int p = warp; p < pieces; p += kJoinWarps)
                list = merge_keys(list, lane < a.top ? a.keys[(slot0 + p) * a.top + lane] : 0, lane);
            s_keys[warp][lane] = list;
            __syncthreads();
            if (warp == 0)
                for (int w = 1; w < kJoinWarps && w < pieces; ++w) list = merge_keys(list, s_keys[w][lane], lane);
            __syncthreads();
        }
        if (warp != 0) continue;
        float m = -INFINITY;
        for (int p = lane; p < pieces; p += 32) m = fmaxf(m, a.sums[slot0 + p].x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        float s = 0.f, t = 0.f;
        int cnt = 0;
        for (int p = lane; p < pieces; p += 32) {
            const float4 v = a.sums[slot0 + p];
            cnt += __float_as_int(v.w);
            if (v.x == -INFINITY) {
                s += v.y;  // (0, or NaN)
            } else {
                const float d = (v.x - m) * a.c1, f = ex2(d);
                s += f * v.y;
                t += f * (v.z + max_nan(d, kFloor) * v.y);
            }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, d);
            t += __shfl_xor_sync(0xffffffffu, t, d);
            cnt += __shfl_xor_sync(0xffffffffu, cnt, d);
        }
        finish(a, e.x < 0 ? ~e.x : e.x, e.x >= 0, __int_as_float(e.y), m, s, t, cnt, list);
    }
}

// CTAs of a call at most: as many as the SMs hold at once; where those would have longer lists of rows than they keep, more.
int most_ctas(int N) {
    const int sms = device_sm_count(), most = kResident * (sms > 0 ? sms : 152), least = N / (kMaxRows - 16) + 1;
    return most > least ? most : least;
}

template <int DT>
int launch(Args& a, cudaStream_t st) {
    const bool warps = a.V <= kShort;
    const int64_t chunk = (int64_t)(warps ? 32 : kThreads) * kVecs * kElems<DT>;
    // (a row may start inside 16 bytes)
    const bool aligned = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && (a.R <= 1 || a.stride % 16 == 0);
    a.chunks = (int)((a.V + (aligned ? 0 : kElems<DT> - 1) + chunk - 1) / chunk);
    const int64_t units = warps ? ((int64_t)a.N + kWarps - 1) / kWarps : (int64_t)a.N * a.chunks;
    a.ctas = (int)(units < a.ctas ? units : a.ctas);
    const auto kernel = warps ? logprob_part_kernel<DT, true> : logprob_part_kernel<DT, false>;
    static bool attr_set[64][2] = {};
    int dev = 0;
    if (!cuda_ok(cudaGetDevice(&dev))) return GRAFT_ERR_CUDA;
    if (dev < 0 || dev >= 64 || !attr_set[dev][warps]) {
        if (!cuda_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing)) ||
            !cuda_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                          cudaSharedmemCarveoutMaxShared)))
            return GRAFT_ERR_CUDA;
        if (dev >= 0 && dev < 64) attr_set[dev][warps] = true;
    }
    launch_pdl(kernel, dim3(a.ctas), dim3(kThreads), kRing, st, a);
    count_launches(1);
    if (!warps) {
        const int sms = device_sm_count();
        launch_pdl(logprob_join_kernel<DT>, dim3(a.N < 8 * sms ? a.N : 8 * sms), dim3(kJoinWarps * 32), 0, st, a);
        count_launches(1);
    }
    return launch_status();
}

void carve(WsCarver& w, int N, int top, int ctas, Args* a) {
    int32_t* n = w.take<int32_t>(1);
    float4* sums = w.take<float4>((size_t)N + ctas);
    int2* entry = w.take<int2>((size_t)N + ctas);
    uint64_t* keys = w.take<uint64_t>(((size_t)N + ctas) * top);
    if (a != nullptr) {
        a->n_rows = n;
        a->sums = sums;
        a->entry = entry;
        a->keys = keys;
    }
}

int check(int N, int V, int top) {
    if (N < 0 || V < 1 || top < 0 || top > V) return GRAFT_ERR_INVALID_ARG;
    if (N > 65535 || V > (1 << 24) || top > GRAFT_MAX_TOP_LOGPROBS) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    return GRAFT_OK;
}

}  // namespace
}  // namespace graft

using namespace graft;

extern "C" int graft_token_logprobs_workspace_size(int N, int V, int top, size_t* bytes) {
    if (bytes == nullptr) return GRAFT_ERR_INVALID_ARG;
    const int rc = check(N, V, top);
    if (rc != GRAFT_OK) return rc;
    WsCarver w(nullptr);
    carve(w, N, top, most_ctas(N), nullptr);
    *bytes = w.bytes();
    return GRAFT_OK;
}

extern "C" int graft_token_logprobs(int N, int V, int64_t n_logit_rows, int dtype, const void* logits, int64_t row_stride,
                                    const int32_t* rows, int block, const int32_t* tokens, float temperature, int top,
                                    float* logprob, float* entropy, int32_t* rank, int32_t* top_id, float* top_logprob,
                                    int32_t* status, void* ws, size_t ws_bytes, graft_stream_t stream) {
    const int rc = check(N, V, top);
    if (rc != GRAFT_OK) return rc;
    if (dtype != GRAFT_BF16 && dtype != GRAFT_FP16 && dtype != GRAFT_F32) return GRAFT_ERR_INVALID_ARG;
    if (!(temperature > 0.f) || !std::isnormal(temperature) || block < 0 || n_logit_rows < 0) return GRAFT_ERR_INVALID_ARG;
    if (n_logit_rows >= (1LL << 31)) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    if (N == 0) return GRAFT_OK;
    if (logits == nullptr || tokens == nullptr || logprob == nullptr) return GRAFT_ERR_INVALID_ARG;
    if (top > 0 && (top_id == nullptr || top_logprob == nullptr)) return GRAFT_ERR_INVALID_ARG;
    if (rows == nullptr && (n_logit_rows < N || block != 0)) return GRAFT_ERR_INVALID_ARG;
    const int size = dtype == GRAFT_F32 ? 4 : 2;
    if (row_stride < V || row_stride > (1LL << 40) || reinterpret_cast<uintptr_t>(logits) % size != 0)
        return GRAFT_ERR_INVALID_ARG;
    Args a{};
    a.ctas = most_ctas(N);
    WsCarver sizer(nullptr);
    carve(sizer, N, top, a.ctas, nullptr);
    if (!ws_ok(ws, ws_bytes, sizer.bytes())) return GRAFT_ERR_WORKSPACE;
    WsCarver w(ws);
    carve(w, N, top, a.ctas, &a);
    a.logits = static_cast<const char*>(logits);
    a.stride = row_stride * size;
    a.logits_end = a.logits + (n_logit_rows > 0 ? (n_logit_rows - 1) * a.stride + (int64_t)V * size : 0);
    a.rows = rows;
    a.tokens = tokens;
    a.R = n_logit_rows;
    a.N = N;
    a.V = V;
    a.block = block;
    a.top = top;
    a.c1 = (float)(1.4426950408889634074 / (double)temperature);
    a.inv_T = (float)(1.0 / (double)temperature);
    a.inv_T_rest = (float)(1.0 / (double)temperature - (double)a.inv_T);
    a.logprob = logprob;
    a.entropy = entropy;
    a.rank = rank;
    a.top_id = top_id;
    a.top_logprob = top_logprob;
    a.status = status;
    cudaStream_t st = (cudaStream_t)stream;
    if (dtype == GRAFT_F32) return launch<GRAFT_F32>(a, st);
    return dtype == GRAFT_BF16 ? launch<GRAFT_BF16>(a, st) : launch<GRAFT_FP16>(a, st);
}
