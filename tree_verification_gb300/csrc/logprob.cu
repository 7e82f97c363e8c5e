// Log probabilities of given tokens, with entropy, rank and top alternatives, from rows of given logits.
//
//   z = x / T, m = max z, s = sum e^(z - m), t = sum (z - m) e^(z - m):
//   log p(v) = (z_v - m) - ln s,  H = ln s - t / s,
//   rank(v) = #{x > x_v} + #{x = x_v at lower ids},  the top k by (x descending, id ascending).
//
// HBM bound: every logit of the rows asked for is read once (4 or 2 bytes) and costs about ten instructions.
// logprob_part_kernel lays the rows' chunks (kVecs x 16 bytes a thread) side by side and gives every CTA an even
// run of them, so all end together whatever the number of rows; the next chunk's loads are in flight while one is
// worked on.  A thread keeps its own maximum and sums over its run's part of a row (one pass, no CTA barrier for
// them); logprob_join_kernel adds up the pieces of each row, in their order, in 64 bits.
//
// Top alternatives: a CTA holds the best k of its part of the row so far, in one warp's registers.  Until
// the list is full a chunk's threshold is a value that at least k of the threads' maxima reach; then logits have to
// pass the k-th best.  What passes goes to a buffer in shared memory and is merged
// when the buffer fills or the part ends: a sort of 32 by one warp.  Where more pass than the buffer holds (long
// runs of equal or rising logits) the chunk's best are drawn one by one instead.
#include <climits>
#include <cmath>

#include <cuda_fp16.h>

#include "common.cuh"

namespace graft {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 4;       // 16-byte loads a thread and chunk
constexpr int kResident = 3;   // CTAs an SM
constexpr int kCap = 512;      // candidates held
constexpr int kMerge = 64;     // candidates that wait for a merge at most
constexpr int kMaxRows = 1024; // rows of a CTA's run at most
constexpr float kFloor = -150.f;  // log2 of a weight that is zero in 32 bits

template <int DT>
constexpr int kElems = DT == GRAFT_F32 ? 4 : 8;  // of 16 bytes

struct Args {
    const char* logits;
    int64_t stride;  // bytes
    const int32_t* rows;
    const int32_t* tokens;
    int64_t R;
    int N, V, block, top, chunks;  // chunks of a row
    int ctas;
    float c1;           // log2(e) / T
    double inv_T;
    float* logprob;
    float* entropy;
    int32_t* rank;
    int32_t* top_id;
    float* top_logprob;
    int32_t* status;
    // workspace
    int32_t* n_rows;    // rows that are asked for
    float4* sums;       // [N + ctas] of a piece: m, s, t, bits of the count of better tokens
    int32_t* entry;     // [N + ctas]
    uint64_t* keys;     // [N + ctas][top]
};

// Units of `units` that CTA k of `ctas` takes: [first(k), first(k + 1)).
__device__ __forceinline__ int64_t first_of(int64_t units, int ctas, int k) {
    const int64_t each = units / ctas, left = units % ctas;
    return each * k + (k < left ? k : left);
}
__device__ __forceinline__ int cta_of(int64_t units, int ctas, int64_t u) {
    const int64_t each = units / ctas, left = units % ctas, big = left * (each + 1);
    return (int)(u < big ? u / (each + 1) : left + (u - big) / each);
}

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

__device__ __forceinline__ uint64_t exchange(uint64_t k, int lane, int step, bool down) {
    const uint64_t o = __shfl_xor_sync(0xffffffffu, k, step);
    const bool upper = (lane & step) == 0;
    return (upper == down) == (k > o) ? k : o;
}
// A warp's 32 keys in falling order.
__device__ __forceinline__ uint64_t sort_keys(uint64_t k, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int step = size >> 1; step > 0; step >>= 1) k = exchange(k, lane, step, (lane & size) == 0);
    return k;
}
// The best 32 of two falling lists, in falling order.
__device__ __forceinline__ uint64_t merge_keys(uint64_t a, uint64_t b, int lane) {
    const uint64_t r = __shfl_sync(0xffffffffu, b, 31 - lane);
    uint64_t k = a > r ? a : r;
#pragma unroll
    for (int step = 16; step > 0; step >>= 1) k = exchange(k, lane, step, true);
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

// Maximum and sums of two parts of a row: t and s of the lower maximum are moved to the higher one.
__device__ __forceinline__ void add_part(float& m, float& s, float& t, float m2, float s2, float t2, float c1) {
    if (m2 == -INFINITY) {  // (nothing but -inf there; NaN sums are kept)
        s += s2;
        t += t2;
        return;
    }
    if (m == -INFINITY) {
        s += s2;
        t += t2;
        m = m2;
        return;
    }
    const float hi = fmaxf(m, m2), d1 = (m - hi) * c1, d2 = (m2 - hi) * c1;
    const float f1 = ex2(d1), f2 = ex2(d2);
    t = f1 * (t + max_nan(d1, kFloor) * s) + f2 * (t2 + max_nan(d2, kFloor) * s2);
    s = f1 * s + f2 * s2;
    m = hi;
}

template <int DT>
__device__ __forceinline__ float element(const uint4& w, int e) {
    const uint32_t* p = &w.x;
    if (DT == GRAFT_F32) return __uint_as_float(p[e]);
    const uint32_t x = p[e >> 1];
    if (DT == GRAFT_BF16) return __uint_as_float((e & 1) ? x & 0xffff0000u : x << 16);
    const unsigned short h = (unsigned short)((e & 1) ? x >> 16 : x);
    return __half2float(__ushort_as_half(h));
}

template <int DT>
__global__ void __launch_bounds__(kThreads, kResident)
logprob_part_kernel(const __grid_constant__ Args a) {
    constexpr int E = kElems<DT>;
    constexpr int kBytes = DT == GRAFT_F32 ? 4 : 2;
    __shared__ int s_entry[kMaxRows], s_row[kMaxRows], s_tok[kMaxRows];
    __shared__ uint64_t s_cand[kCap];
    // Candidates of a chunk are counted in one of three places in turn: the one after next is cleared behind a
    // chunk's barrier, when all have read it and none adds to it as yet.
    __shared__ int s_n[3], s_scan[kWarps];
    __shared__ float s_tau, s_red[kWarps][3], s_reach[32];
    __shared__ int s_cnt[kWarps];
    __shared__ uint64_t s_best[kWarps];
    griddep_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
    // ---- which rows
    auto row_of = [&](int n) -> int64_t {  // of entry n, -1: none
        if (a.rows == nullptr) return n;
        const int64_t r = a.rows[n];
        if (r < 0) return -1;
        const int64_t at = a.block > 0 ? (int64_t)(n / a.block) * a.block + r : r;
        return (a.block > 0 && r >= a.block) || at >= a.R ? -1 : at;
    };
    int n_rows = a.N, mine = 0, before = 0, e0 = 0, e1 = 0;
    if (a.rows != nullptr) {
        const int each = (a.N + kThreads - 1) / kThreads;
        e0 = min(tid * each, a.N);
        e1 = min(e0 + each, a.N);
        for (int n = e0; n < e1; ++n) {
            const bool ok = row_of(n) >= 0;
            mine += ok;
            if (!ok && cta == 0 && a.rows[n] != -1) flag_status(a.status, GRAFT_STATUS_ROW);
        }
        int x = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) s_scan[warp] = x;
        __syncthreads();
        n_rows = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) before = n_rows + x - mine;
            n_rows += s_scan[w];
        }
        // entries without a row
        for (int n = cta; n < a.N; n += gridDim.x) {
            if (row_of(n) >= 0) continue;
            if (tid == 0) {
                a.logprob[n] = 0.f;
                if (a.entropy != nullptr) a.entropy[n] = 0.f;
                if (a.rank != nullptr) a.rank[n] = -1;
            }
            if (tid < a.top) {
                a.top_id[(int64_t)n * a.top + tid] = -1;
                a.top_logprob[(int64_t)n * a.top + tid] = 0.f;
            }
        }
    }
    if (cta == 0 && tid == 0) *a.n_rows = n_rows;
    const int64_t units = (int64_t)n_rows * a.chunks;
    const int ctas = (int)(units < gridDim.x ? units : gridDim.x);
    if (cta >= ctas) return;
    const int64_t u0 = first_of(units, ctas, cta), u1 = first_of(units, ctas, cta + 1);
    const int r0 = (int)(u0 / a.chunks), r1 = (int)((u1 - 1) / a.chunks);
    auto take = [&](int r, int n) {
        const int tok = a.tokens[n];
        s_entry[r - r0] = n;
        s_row[r - r0] = (int)row_of(n);
        const bool ok = tok >= 0 && tok < a.V;
        s_tok[r - r0] = ok ? tok : -1;
        if (!ok && tok != -1) flag_status(a.status, GRAFT_STATUS_TOKEN_RANGE);
    };
    if (a.rows == nullptr) {
        for (int r = r0 + tid; r <= r1; r += kThreads) take(r, r);
    } else {
        for (int n = e0, r = before; n < e1; ++n)
            if (row_of(n) >= 0) {
                if (r >= r0 && r <= r1) take(r, n);
                ++r;
            }
    }
    if (tid < 3) s_n[tid] = 0;
    __syncthreads();

    // ---- the run: chunk c of row j of the list
    int j = 0, c = (int)(u0 - (int64_t)r0 * a.chunks);
    auto start_of = [&](int j, int& off) -> const char* {  // 16-byte aligned, `off` elements before the row
        const char* p = a.logits + (int64_t)s_row[j] * a.stride;
        const uintptr_t x = reinterpret_cast<uintptr_t>(p);
        off = (int)(x & 15) / kBytes;
        return reinterpret_cast<const char*>(x & ~(uintptr_t)15);
    };
    auto fetch = [&](int j, int c, uint4* buf) {
        int off;
        const char* p = start_of(j, off);
#pragma unroll
        for (int x = 0; x < kVecs; ++x) {
            const int g = (c * kVecs + x) * kThreads + tid;
            const int id = g * E - off;
            if (id >= 0 && id + E <= a.V) {
                buf[x] = __ldcs(reinterpret_cast<const uint4*>(p) + g);
            } else {
                uint32_t* w = &buf[x].x;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const bool in = id + e >= 0 && id + e < a.V;
                    if (DT == GRAFT_F32) {
                        w[e] = in ? reinterpret_cast<const uint32_t*>(p)[(int64_t)g * E + e] : 0xff800000u;
                    } else {
                        const uint32_t h = in ? reinterpret_cast<const unsigned short*>(p)[(int64_t)g * E + e]
                                              : (DT == GRAFT_BF16 ? 0xff80u : 0xfc00u);
                        w[e >> 1] = (e & 1) ? w[e >> 1] | h << 16 : h;
                    }
                }
            }
        }
    };
    auto given = [&](int j) -> float {
        const int tok = s_tok[j];
        if (tok < 0) return INFINITY;
        const char* p = a.logits + (int64_t)s_row[j] * a.stride + (int64_t)tok * kBytes;
        if (DT == GRAFT_F32) return *reinterpret_cast<const float*>(p);
        const unsigned short h = *reinterpret_cast<const unsigned short*>(p);
        return DT == GRAFT_BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
    };
    uint4 cur[kVecs], nxt[kVecs];
    fetch(j, c, cur);
    float xt = given(j), xt_next = xt;
    float m = -INFINITY, s = 0.f, t = 0.f;
    int cnt = 0;
    uint64_t list = 0;  // warp 0: the best so far, one a lane
    float tau = -INFINITY;  // what later logits have to pass; -inf: fewer than k are listed
    int waiting = 0;    // candidates in the buffer
    int turn = 0;
    for (int64_t u = u0; u < u1; ++u) {
        int j2 = j, c2 = c + 1;
        if (c2 == a.chunks) {
            c2 = 0;
            ++j2;
        }
        if (u + 1 < u1) {
            fetch(j2, c2, nxt);
            if (j2 != j) xt_next = given(j2);
        }
        int off;
        start_of(j, off);
        const int tok = s_tok[j];
        const int id_first = (c * kVecs * kThreads + tid) * E - off;
        auto id_of = [&](int x) { return id_first + x * kThreads * E; };
        // ---- maximum, sums
        float top = -INFINITY;
#pragma unroll
        for (int x = 0; x < kVecs; ++x)
#pragma unroll
            for (int e = 0; e < E; ++e) top = fmaxf(top, element<DT>(cur[x], e));
        if (top > m) {
            if (m != -INFINITY) {
                const float d = (m - top) * a.c1, f = ex2(d);
                t = f * (t + max_nan(d, kFloor) * s);
                s *= f;
            }
            m = top;
        }
        const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int x = 0; x < kVecs; ++x)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float d = max_nan((element<DT>(cur[x], e) - base) * a.c1, kFloor);
                const float w = ex2(d);
                s += w;
                t += d * w;
            }
        // ---- tokens ahead of the given one
        if (tok >= 0) {
#pragma unroll
            for (int x = 0; x < kVecs; ++x) {
                const int id = id_of(x);
                if (id > tok) {
#pragma unroll
                    for (int e = 0; e < E; ++e) cnt += element<DT>(cur[x], e) > xt;
                } else if (id >= 0 && id + E <= tok) {
#pragma unroll
                    for (int e = 0; e < E; ++e) cnt += element<DT>(cur[x], e) >= xt;
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float v = element<DT>(cur[x], e);
                        cnt += v > xt || (v == xt && id + e >= 0 && id + e < tok);
                    }
                }
            }
        }
        // ---- alternatives
        const bool ends = c + 1 == a.chunks || u + 1 == u1;
        if (a.top > 0) {
            const bool open = tau == -INFINITY;
            if (open) {
                // Reached by at least k threads' maxima: what 8 / 2^i warps reach 2^i ceil(k / 8) times each, for i up
                // to 3 (short rows leave warps without logits), the largest of these.
                const float v = sort_values(top, lane);
                const int each = (a.top + kWarps - 1) / kWarps;
                const float q = __shfl_sync(0xffffffffu, v, min((each << (lane & 3)) - 1, 31));
                if (lane < 4) s_reach[lane * kWarps + warp] = q;
                __syncthreads();
                const float r = s_reach[lane];  // of warp lane & 7, 2^(lane / 8) ceil(k / 8) times
                int above = 0;
#pragma unroll
                for (int d = 1; d < kWarps; ++d) {
                    const int o = (lane & 24) | ((lane + d) & 7);
                    const float w = __shfl_sync(0xffffffffu, r, o);
                    above += w > r || (w == r && o < lane);
                }
                tau = above == (kWarps >> (lane >> 3)) - 1 ? r : -INFINITY;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) tau = fmaxf(tau, __shfl_xor_sync(0xffffffffu, tau, d));
            }
            // (of equal logits the lower id goes first, so a full list's last has to be passed; a chunk's own threshold
            // to be reached)
            auto passes = [&](float v) { return open ? v >= tau && v > -INFINITY : v > tau; };
            if (passes(top)) {
#pragma unroll
                for (int x = 0; x < kVecs; ++x)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float v = element<DT>(cur[x], e);
                        if (passes(v)) {
                            const int at = waiting + atomicAdd(&s_n[turn], 1);
                            if (at < kCap) s_cand[at] = key_of(v, id_of(x) + e);
                        }
                    }
            }
            __syncthreads();
            int n = waiting + s_n[turn];
            const int after = turn == 0 ? 2 : turn - 1;  // (the place after next)
            if (tid == 0) s_n[after] = 0;
            turn = turn == 2 ? 0 : turn + 1;
            if (n > kCap) {
                // The chunk's best that pass, one by one.  (Rare: long runs of equal or rising logits.)
                n = waiting;
                uint64_t last = ~0ull;
                for (int k = 0; k < a.top; ++k) {
                    uint64_t best = 0;
#pragma unroll 1
                    for (int x = 0; x < kVecs; ++x) {
                        const uint4 w = x == 0 ? cur[0] : x == 1 ? cur[1] : x == 2 ? cur[2] : cur[3];
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            const float v = element<DT>(w, e);
                            const uint64_t key = key_of(v, id_of(x) + e);
                            if (passes(v) && key < last && key > best) best = key;
                        }
                    }
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) {
                        const uint64_t o = __shfl_xor_sync(0xffffffffu, best, d);
                        best = o > best ? o : best;
                    }
                    __syncthreads();
                    if (lane == 0) s_best[warp] = best;
                    __syncthreads();
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) best = s_best[w] > best ? s_best[w] : best;
                    if (best == 0) break;
                    last = best;
                    if (tid == 0) s_cand[n] = best;
                    ++n;
                }
                __syncthreads();
            }
            if (n >= kMerge || (n > 0 && (open || ends))) {
                if (warp == 0) {
                    for (int at = 0; at < n; at += 32)
                        list = merge_keys(list, sort_keys(at + lane < n ? s_cand[at + lane] : 0, lane), lane);
                    const uint64_t kth = __shfl_sync(0xffffffffu, list, a.top - 1);
                    if (lane == 0) s_tau = kth != 0 ? key_value(kth) : -INFINITY;
                }
                __syncthreads();
                tau = s_tau;
                n = 0;
            } else if (open) {
                tau = -INFINITY;  // (nothing above -inf as yet)
            }
            waiting = n;
        }
        // ---- the part's end
        if (ends) {
            float m2 = m, s2 = s, t2 = t;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                const float mo = __shfl_xor_sync(0xffffffffu, m2, d), so = __shfl_xor_sync(0xffffffffu, s2, d),
                            to = __shfl_xor_sync(0xffffffffu, t2, d);
                add_part(m2, s2, t2, mo, so, to, a.c1);
                cnt += __shfl_xor_sync(0xffffffffu, cnt, d);
            }
            __syncthreads();
            if (lane == 0) {
                s_red[warp][0] = m2;
                s_red[warp][1] = s2;
                s_red[warp][2] = t2;
                s_cnt[warp] = cnt;
            }
            __syncthreads();
            const int64_t slot = (int64_t)(r0 + j) + cta;
            if (tid == 0) {
#pragma unroll
                for (int w = 1; w < kWarps; ++w) {
                    add_part(m2, s2, t2, s_red[w][0], s_red[w][1], s_red[w][2], a.c1);
                    cnt += s_cnt[w];
                }
                a.sums[slot] = make_float4(m2, s2, t2, __int_as_float(cnt));
                a.entry[slot] = s_entry[j];
            }
            if (tid < a.top) a.keys[slot * a.top + tid] = list;
            m = -INFINITY;
            s = t = 0.f;
            cnt = 0;
            list = 0;
            tau = -INFINITY;
        }
        j = j2;
        c = c2;
        xt = xt_next;
#pragma unroll
        for (int x = 0; x < kVecs; ++x) cur[x] = nxt[x];
    }
}

constexpr int kJoinWarps = 4;

// Adds up the pieces of each row: a CTA a row.  A warp merges every fourth piece's alternatives, the first one adds the sums.
template <int DT>
__global__ void __launch_bounds__(kJoinWarps * 32)
logprob_join_kernel(const __grid_constant__ Args a) {
    griddep_enter();
    __shared__ uint64_t s_keys[kJoinWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n_rows = *a.n_rows;
    const int64_t units = (int64_t)n_rows * a.chunks;
    const int ctas = (int)(units < a.ctas ? units : a.ctas);
    for (int r = blockIdx.x; r < n_rows; r += gridDim.x) {
        const int c0 = cta_of(units, ctas, (int64_t)r * a.chunks), c1 = cta_of(units, ctas, (int64_t)(r + 1) * a.chunks - 1);
        const int64_t slot0 = (int64_t)r + c0;
        const int pieces = c1 - c0 + 1;
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
        double s = 0, t = 0;  // t in units of ln
        int cnt = 0;
        for (int p = lane; p < pieces; p += 32) {
            const float4 v = a.sums[slot0 + p];
            cnt += __float_as_int(v.w);
            if (v.x == -INFINITY) {
                s += v.y;  // (0, or NaN)
            } else {
                const double d = ((double)v.x - m) * a.inv_T, f = exp(d);
                s += f * v.y;
                t += f * (0.69314718055994530942 * v.z + (f > 0 ? d * v.y : 0.0));
            }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, d);
            t += __shfl_xor_sync(0xffffffffu, t, d);
            cnt += __shfl_xor_sync(0xffffffffu, cnt, d);
        }
        // a row of -inf alone has no law, nor has one with NaN or +inf: NaN
        const double ln_s = m == -INFINITY ? (double)NAN : log(s);
        const int n = a.entry[slot0];
        auto logp = [&](float x) -> float {
            if (isnan(ln_s)) return NAN;
            return (float)(((double)x - m) * a.inv_T - ln_s);
        };
        if (lane == 0) {
            const int tok = a.tokens[n];
            const bool ok = tok >= 0 && tok < a.V;
            float x = 0.f;
            if (ok) {
                int64_t row = n;
                if (a.rows != nullptr) row = (a.block > 0 ? (int64_t)(n / a.block) * a.block : 0) + a.rows[n];
                const char* p = a.logits + row * a.stride;
                if (DT == GRAFT_F32) x = reinterpret_cast<const float*>(p)[tok];
                if (DT == GRAFT_BF16) x = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[tok]);
                if (DT == GRAFT_FP16) x = __half2float(reinterpret_cast<const __half*>(p)[tok]);
            }
            a.logprob[n] = ok ? logp(x) : 0.f;
            if (a.entropy != nullptr) a.entropy[n] = isnan(ln_s) ? NAN : (float)(ln_s - t / s);
            if (a.rank != nullptr) a.rank[n] = ok ? cnt : -1;
        }
        if (a.top > 0) {
            int id = key_id(list);
            float lp = list != 0 ? logp(key_value(list)) : 0.f;
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
                    lp = isnan(ln_s) ? NAN : -INFINITY;
                }
            }
            if (lane < a.top) {
                a.top_id[(int64_t)n * a.top + lane] = id;
                a.top_logprob[(int64_t)n * a.top + lane] = lp;
            }
        }
    }
}

template <int DT>
int launch(Args& a, cudaStream_t st) {
    constexpr int64_t chunk = (int64_t)kThreads * kVecs * kElems<DT>;
    a.chunks = (int)((a.V + kElems<DT> - 1 + chunk - 1) / chunk);  // (a row may start inside 16 bytes)
    const int64_t units = (int64_t)a.N * a.chunks;
    const int grid = (int)(units < a.ctas ? units : a.ctas);
    a.ctas = grid;
    launch_pdl(logprob_part_kernel<DT>, dim3(grid), dim3(kThreads), 0, st, a);
    const int sms = device_sm_count();
    launch_pdl(logprob_join_kernel<DT>, dim3(a.N < 8 * sms ? a.N : 8 * sms), dim3(kJoinWarps * 32), 0, st, a);
    count_launches(2);
    return launch_status();
}

int most_ctas() {
    const int sms = device_sm_count();
    return kResident * (sms > 0 ? sms : 152);
}

void carve(WsCarver& w, int N, int top, int ctas, Args* a) {
    int32_t* n = w.take<int32_t>(1);
    float4* sums = w.take<float4>((size_t)N + ctas);
    int32_t* entry = w.take<int32_t>((size_t)N + ctas);
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
    if (N > 65535 || V > (1 << 30) || top > GRAFT_MAX_TOP_LOGPROBS) return GRAFT_ERR_UNSUPPORTED_SHAPE;
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
    carve(w, N, top, most_ctas(), nullptr);
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
    if (!(temperature > 0.f) || !std::isfinite(temperature) || block < 0 || n_logit_rows < 0) return GRAFT_ERR_INVALID_ARG;
    if (n_logit_rows >= (1LL << 31)) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    if (N == 0) return GRAFT_OK;
    if (logits == nullptr || tokens == nullptr || logprob == nullptr) return GRAFT_ERR_INVALID_ARG;
    if (top > 0 && (top_id == nullptr || top_logprob == nullptr)) return GRAFT_ERR_INVALID_ARG;
    if (rows == nullptr && (n_logit_rows < N || block != 0)) return GRAFT_ERR_INVALID_ARG;
    const int size = dtype == GRAFT_F32 ? 4 : 2;
    if (row_stride < V || row_stride > (1LL << 40) || reinterpret_cast<uintptr_t>(logits) % size != 0)
        return GRAFT_ERR_INVALID_ARG;
    Args a{};
    a.ctas = most_ctas();
    WsCarver sizer(nullptr);
    carve(sizer, N, top, a.ctas, nullptr);
    if (!ws_ok(ws, ws_bytes, sizer.bytes())) return GRAFT_ERR_WORKSPACE;
    WsCarver w(ws);
    carve(w, N, top, a.ctas, &a);
    a.logits = static_cast<const char*>(logits);
    a.stride = row_stride * size;
    a.rows = rows;
    a.tokens = tokens;
    a.R = n_logit_rows;
    a.N = N;
    a.V = V;
    a.block = block;
    a.top = top;
    a.c1 = (float)(1.4426950408889634074 / (double)temperature);
    a.inv_T = 1.0 / (double)temperature;
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
