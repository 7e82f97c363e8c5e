// Attention of a few query rows a KV head over a paged cache: single tokens,
// short chunks and small trees (new rows x group up to 16 or 32 at a time).
//
//   o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),  s_j = scale log2(e) q.k_j
//
// with a running maximum m and sum (one pass over the keys).  Such calls read
// 512 bytes of K and V a key and head for at most 32 rows' products, so HBM
// bounds them; the work is split by keys, evenly over the CTAs, whatever the
// sequences' lengths: the plan lays the 16-key units of all (entry, KV head)
// items side by side and gives every CTA an equal run of them.  Within a run
// each warp takes every kWarps-th unit, streams it through its own ring of
// kStages units in shared memory with cp.async (no CTA barrier inside a run:
// a warp waits for its own copies alone), and keeps its rows' O in registers
// (mma.sync m16n8k16, 32-bit accumulators: 16 rows are too few to fill a
// tcgen05 tile, and the products take a quarter of the time the bytes do).
// A page row index costs a lookup per unit; a lane holds one, 32 units ahead.
//
// Items that a run's edges cut are joined by the CTA that arrives last (a
// counter an item): it reads the pieces' 32-bit partial rows in their order,
// so the result does not depend on which CTA that is.
#include <cmath>

#include "paged.cuh"

namespace graft {
namespace paged {
namespace {

constexpr int kStages = 3;
constexpr int kAhead = 4;                          // units a warp brings into L2 ahead of the grid wait
constexpr int kUnit = 16;                          // keys of a unit
constexpr int kUnitBytes = kUnit * HD * 2;         // of K, or of V
constexpr int kRowPad = 132;                       // floats of a staged partial row: 4 banks apart

// W: warps of a CTA, RT: 16-row tiles of a warp
constexpr int ring_bytes(int W, int RT) {
    const int ring = W * kStages * 2 * kUnitBytes, merge = W * RT * 16 * kRowPad * 4;
    return ring > merge ? ring : merge;
}
// ring (or staged rows) | Q of two row tiles | maxima and sums
constexpr int q_bytes(int RT) { return RT > 1 ? RT * 16 * HD * 2 : 0; }
constexpr int smem_bytes(int W, int RT) { return ring_bytes(W, RT) + q_bytes(RT) + W * RT * 16 * 8; }

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// byte offset of 16-byte chunk ch (0..15) of row r in a [rows][128] 16-bit tile
__device__ __forceinline__ uint32_t swz(int r, int ch) { return (uint32_t)(r * (HD * 2) + ((ch ^ (r & 7)) << 4)); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    const int n = valid ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr)
                 : "memory");
}
template <int DT>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    if (DT == GRAFT_BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};\n"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};\n"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float safe(float m) { return m == -INFINITY ? 0.f : m; }
// Weights are 2^(s - m + lift).  fp16 reaches down to 2^-24 only: lifted by 2^7 the small weights of a long
// context keep their bits (and the largest, 2^(8 + 7), still fits); sums and O carry the same factor.
template <int DT>
constexpr float kLift = DT == GRAFT_FP16 ? 7.f : 0.f;

// Joins the warps' staged rows r (the sum of the weights in l); a lane takes four dims.
template <int W, int RT>
__device__ __forceinline__ void join_warps(const float* s_part, const float2* s_ml, int r, float4& acc, float& m,
                                           float& l) {
    const int lane = threadIdx.x & 31;
    m = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) m = fmaxf(m, s_ml[w * RT * 16 + r].x);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    l = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const float2 ml = s_ml[w * RT * 16 + r];
        if (ml.x == -INFINITY && ml.y == 0.f) continue;  // saw no key
        const float x = ex2(ml.x - safe(m));
        const float4 v = *reinterpret_cast<const float4*>(s_part + (w * RT * 16 + r) * kRowPad + lane * 4);
        acc.x += x * v.x;
        acc.y += x * v.y;
        acc.z += x * v.z;
        acc.w += x * v.w;
        l += x * ml.y;
    }
}

template <int DT>
__device__ __forceinline__ void put_row(const AttnArgs& a, const Entry& e, int kvh, int r, const float4& acc, float l) {
    using E = Elem<DT>;
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const int row = e.row0 + r, tok = row / a.G, g = row - tok * a.G;
    typename E::T* dst = static_cast<typename E::T*>(a.O) + ((int64_t)(e.q0 + tok) * a.Hq + kvh * a.G + g) * HD +
                         (threadIdx.x & 31) * 4;
    *reinterpret_cast<uint2*>(dst) = make_uint2(E::down(acc.x * inv, acc.y * inv), E::down(acc.z * inv, acc.w * inv));
}

// Joins an item's pieces, by the CTA that arrived last.  The pieces' rows come to shared memory with cp.async, as
// many as the ring holds at a time (all reads in flight at once, little code: this part runs cold), then a thread
// sums four dims of a row over them.  More pieces than fit: the sums so far take the first place of the next lot.
template <int DT, int RT, int W>
__device__ __forceinline__ void join_pieces(const AttnArgs& a, const Start& at, unsigned char* smem) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_rows = at.e.rows, step = at.step, kvh = at.head, c0 = at.cta0, pieces = at.pieces;
    const int row_floats = n_rows * HD;
    const int cap = ring_bytes(W, RT) / (n_rows * (HD * 4 + 8));
    float* s_o = reinterpret_cast<float*>(smem);                            // [cap][n_rows][128]
    float2* s_ml = reinterpret_cast<float2*>(s_o + (size_t)cap * row_floats);  // [cap][n_rows]
    int have = 0;
    for (int p0 = 0; p0 < pieces;) {
        const int n = min(cap - have, pieces - p0);
        // a run's last item (the one that it starts) has the CTA's second slot
        auto slot_of = [&](int q) -> int64_t { return step > 0 ? (c0 + q * step) * 2 : (c0 + q) * 2 + (q == 0 ? 1 : 0); };
        for (int p = warp; p < n; p += W) {
            const float* src = a.few.o + slot_of(p0 + p) * kFewRows * HD;
            const uint32_t dst = smem_u32(s_o + (size_t)(have + p) * row_floats);
#pragma unroll 4
            for (int i = lane; i < n_rows * 32; i += 32) cp_async16(dst + i * 16, src + i * 4, true);
        }
        for (int x = tid; x < n * n_rows; x += W * 32) {
            const int p = x / n_rows, r = x - p * n_rows;
            s_ml[have * n_rows + x] = __ldcg(a.few.ml + slot_of(p0 + p) * kFewRows + r);
        }
        cp_commit();
        cp_wait<0>();
        __syncthreads();
        p0 += n;
        const int all = have + n;
        for (int r = warp; r < n_rows; r += W) {
            // a lane weighs one piece, and sums four dims over all
            float m = -INFINITY, l = 0.f;
            for (int p = lane; p < all; p += 32) m = fmaxf(m, s_ml[p * n_rows + r].x);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int q0 = 0; q0 < all; q0 += 32) {
                float f = 0.f;
                if (q0 + lane < all) {
                    const float2 ml = s_ml[(q0 + lane) * n_rows + r];
                    f = ex2(ml.x - safe(m));
                    l += f * ml.y;
                }
                const int n = min(all - q0, 32);
#pragma unroll 8
                for (int p = 0; p < n; ++p) {
                    const float g = __shfl_sync(0xffffffffu, f, p);
                    const float4 v =
                        *reinterpret_cast<const float4*>(s_o + (size_t)(q0 + p) * row_floats + r * HD + lane * 4);
                    acc.x += g * v.x;
                    acc.y += g * v.y;
                    acc.z += g * v.z;
                    acc.w += g * v.w;
                }
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
            if (p0 == pieces) {
                put_row<DT>(a, at.e, kvh, r, acc, l);
            } else {
                *reinterpret_cast<float4*>(s_o + r * HD + lane * 4) = acc;
                __syncwarp();  // (a row's maxima are read by the warp that sums the row alone)
                if (lane == 0) s_ml[r] = make_float2(m, l);
            }
        }
        have = 1;
        __syncthreads();
    }
}

template <int DT, int RT, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, 8 / kWarps)
few_kernel(const __grid_constant__ AttnArgs a) {
    using E = Elem<DT>;
    using T = typename E::T;
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cta = blockIdx.x;
    const Entry* entries = reinterpret_cast<const Entry*>(a.plan + a.shape.off_few);
    // The run's state is the CTA's, not a thread's: shared memory holds it, the registers are for O and Q.
    __shared__ Start s_at, s_pending[2];
    __shared__ PlanHead s_head;
    __shared__ int s_n_pending;
    float* s_part = reinterpret_cast<float*>(smem);
    float2* s_ml = reinterpret_cast<float2*>(smem + ring_bytes(kWarps, RT) + q_bytes(RT));
    const uint32_t ring = smem_u32(smem) + warp * (kStages * 2 * kUnitBytes);
    const uint32_t s_q = smem_u32(smem + ring_bytes(kWarps, RT));
    unsigned char* ring_p = smem + warp * (kStages * 2 * kUnitBytes);
    const T* Kp = static_cast<const T*>(a.K);
    const T* Vp = static_cast<const T*>(a.V);
    const T* Qp = static_cast<const T*>(a.Q);
    const float sl2 = a.scale * 1.4426950408889634f;
    const int64_t key_stride = (int64_t)a.c.Hkv * HD;

    // ---- the item at hand
    int u0 = 0, u1 = 0, kvh = 0, keys = 0, L = 0, n_new = 0;
    int mine = 0;                 // this warp's units (may be <= 0)
    int pages = -1, pages_at = 0; // pages of this warp's units pages_at .. pages_at + 31, one a lane
    const int32_t* table = a.c.block_table;
    const Entry& e = s_at.e;
    auto begin = [&]() {
        keys = e.keys;
        L = e.L;
        n_new = e.n;
        u0 = s_at.unit;
        u1 = min(e.units, u0 + s_at.count);
        kvh = s_at.head;
        table = a.c.block_table + (int64_t)e.b * a.c.max_pages;
        mine = (u1 - u0 - warp + kWarps - 1) / kWarps;
    };
    auto fetch_pages = [&](int i0, bool flag) {
        const int u = u0 + warp + (i0 + lane) * kWarps;
        int p = -1;
        if (u < u1) {
            p = __ldcg(table + ((u * kUnit) >> a.page_shift));
            if (p < 0 || p >= a.c.num_pages) {
                p = -1;
                if (flag) flag_status(a.c.status, GRAFT_STATUS_PAGE);
            }
        }
        return p;
    };
    auto load = [&](int i) {
        if (i < mine) {
            if (i - pages_at >= 32) {
                pages_at = i;
                pages = fetch_pages(i, true);
            }
            const int key0 = (u0 + warp + i * kWarps) * kUnit;
            const int page = __shfl_sync(0xffffffffu, pages, i - pages_at);
            const int64_t row = ((int64_t)max(page, 0) << a.page_shift) + (key0 & (a.c.page_rows - 1));
            const int64_t off = (row * a.c.Hkv + kvh) * HD;
            const uint32_t k = ring + (i % kStages) * 2 * kUnitBytes, v = k + kUnitBytes;
#pragma unroll
            for (int x = 0; x < kUnit * 16 / 32; ++x) {
                const int r = x * 2 + (lane >> 4), ch = lane & 15;
                const bool ok = page >= 0 && key0 + r < keys;
                const int64_t o = off + (ok ? r * key_stride : 0) + ch * 8;
                cp_async16(k + swz(r, ch), Kp + o, ok);
                cp_async16(v + swz(r, ch), Vp + o, ok);
            }
        }
        cp_commit();
    };

    // ---- before the previous kernel has finished
    // The plan and the pages are read ahead of the grid wait and the first units brought into L2: a guess, since
    // whatever runs before may still write them.  Every index is checked, the reads are read again after the wait,
    // and a guess that does not hold is dropped; nothing but L2's contents depends on it (L2 is where all writes
    // meet, so a line brought in early is not stale).
    constexpr int kHeadWords = sizeof(PlanHead) / 4, kStartWords = sizeof(Start) / 4;
    static_assert(kHeadWords + kStartWords <= kWarps * 32, "one word a thread");
    const int32_t* word = tid < kHeadWords
                              ? reinterpret_cast<const int32_t*>(a.plan) + tid
                              : reinterpret_cast<const int32_t*>(a.plan + a.shape.off_start) + cta * kStartWords +
                                    (tid - kHeadWords);
    int32_t* s_word = tid < kHeadWords ? reinterpret_cast<int32_t*>(&s_head) + tid
                                       : reinterpret_cast<int32_t*>(&s_at) + (tid - kHeadWords);
    const bool has_word = tid < kHeadWords + kStartWords;
    int32_t guess = 0;
    if (has_word) *s_word = guess = __ldcg(word);
    if (tid == 0) s_n_pending = 0;
    __syncthreads();
    const bool sound = plan_fits(a, s_head) && cta < s_head.few_ctas && e.b >= 0 && e.b < a.c.n_seqs && e.keys > 0 &&
                 e.L >= 0 && e.keys <= (int64_t)a.c.max_pages * a.c.page_rows &&
                 e.units == (e.keys - 1) / kUnit + 1 && s_at.unit >= 0 && s_at.unit < e.units && s_at.count > 0 &&
                 s_at.head >= 0 && s_at.head < a.c.Hkv && e.row0 == 0 && e.rows > 0 && e.rows <= RT * 16 && e.q0 >= 0 &&
                 e.q0 < a.N && (e.rows - 1) / a.G < a.N - e.q0;
    if (sound) {
        begin();
        pages = fetch_pages(0, false);
        if (warp == 0 && lane < e.rows) {
            const int tok = lane / a.G;
            const T* q = Qp + (int64_t)(e.q0 + tok) * a.q_stride + (kvh * a.G + lane - tok * a.G) * HD;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
            asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 64));
        }
        for (int i = 0; i < min(mine, kAhead); ++i) {
            const int key0 = (u0 + warp + i * kWarps) * kUnit;
            const int page = __shfl_sync(0xffffffffu, pages, i);
            if (page < 0) continue;
            const int64_t row = ((int64_t)page << a.page_shift) + (key0 & (a.c.page_rows - 1));
            const T* at = Kp + ((row + (lane >> 1)) * a.c.Hkv + kvh) * HD + (lane & 1) * 64;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
            asm volatile("prefetch.global.L2 [%0];" ::"l"(Vp + (at - Kp)));
        }
    }
    if (!a.after_wide) griddep_wait();
    griddep_launch_dependents();
    // Beside the wide kernel (two row tiles) the wait comes last, so that this kernel's end is that of both; all that
    // it reads comes from L2, past lines that an earlier kernel left in the SM's L1.
    auto leave = [&]() {
        if (a.after_wide) griddep_wait();
    };
    // reads the plan anew; false: nothing to do
    auto reread = [&]() -> bool {
        cp_wait<0>();
        __syncthreads();
        if (has_word) *s_word = __ldcg(word);
        __syncthreads();
        if (!plan_fits(a, s_head)) {
            if (cta == 0 && tid == 0) flag_status(a.c.status, GRAFT_STATUS_PLAN);
            return false;
        }
        if (cta >= s_head.few_ctas) return false;
        begin();
        pages = fetch_pages(0, true);
        return true;
    };
    if (!sound && !reread()) {
        leave();
        return;
    }
    bool guessed = sound;  // the first item is as yet a guess

    while (true) {
        // Q: rows past the block read as zeros.  One row tile's fragments stay in registers, straight from
        // memory; two tiles' would not fit beside O, so they go through shared memory, read again every unit.
        uint32_t qf[RT > 1 ? 1 : 8][4];
        if (RT > 1) {
            for (int x = tid; x < RT * 16 * 16; x += kWarps * 32) {
                const int r = x >> 4, ch = x & 15;
                const int row = e.row0 + r, tok = row / a.G, g = row - tok * a.G;
                const bool ok = r < e.rows;
                cp_async16(s_q + swz(r, ch),
                           Qp + (ok ? (int64_t)(e.q0 + tok) * a.q_stride + (kvh * a.G + g) * HD + ch * 8 : 0), ok);
            }
            cp_commit();
        }
        int limit[RT][2];        // keys below it are seen
        uint64_t anc[RT][2];     // new rows seen (tree)
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = t * 16 + (lane >> 2) + h * 8;
                const int row = e.row0 + r, tok = row / a.G;
                const int g = row - tok * a.G;
                const bool ok = r < e.rows;
                if (RT == 1) {
                    const T* q = Qp + (ok ? (int64_t)(e.q0 + tok) * a.q_stride + (kvh * a.G + g) * HD : 0);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const int col = kk * 16 + (lane & 3) * 2;
                        qf[kk][h] = ok ? *reinterpret_cast<const uint32_t*>(q + col) : 0u;
                        qf[kk][h + 2] = ok ? *reinterpret_cast<const uint32_t*>(q + col + 8) : 0u;
                    }
                }
                anc[t][h] = 0;
                if (!ok) {
                    limit[t][h] = 0;
                } else if (a.mask != nullptr) {
                    limit[t][h] = e.L;
                    const uint64_t* m = a.mask + e.q0 + tok;
                    anc[t][h] = RT > 1 ? __ldcg(reinterpret_cast<const unsigned long long*>(m)) : *m;
                } else {
                    limit[t][h] = e.L + tok + 1;
                }
            }
        float m_run[RT][2], l_run[RT][2], o[RT][16][4];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            m_run[t][0] = m_run[t][1] = -INFINITY;
            l_run[t][0] = l_run[t][1] = 0.f;
#pragma unroll
            for (int d = 0; d < 16; ++d) o[t][d][0] = o[t][d][1] = o[t][d][2] = o[t][d][3] = 0.f;
        }

        // (Q's reads, and those that check the guess, go ahead of the units': a unit's bytes take the SM's read
        // port for longer than any of them)
        // (without a status bit as yet: a guess that does not hold may name a sequence whose pages are gone)
        const int now = guessed ? fetch_pages(0, false) : pages;
        const int32_t again = guessed && has_word ? __ldcg(word) : guess;
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) load(i);
        if (guessed) {
            guessed = false;
            if (__syncthreads_or(again != guess)) {
                if (!reread()) {
                    leave();
                    return;
                }
                continue;
            }
            if (now < 0 && u0 + warp + lane * kWarps < u1) flag_status(a.c.status, GRAFT_STATUS_PAGE);
            if (__any_sync(0xffffffffu, now != pages)) {
                cp_wait<0>();
                __syncwarp();
                pages = now;
#pragma unroll 1
                for (int i = 0; i < kStages - 1; ++i) load(i);
            }
        }
        if (RT > 1) {
            cp_wait<0>();  // Q, and the first units with it
            __syncthreads();
        }
#pragma unroll 1
        for (int i = 0; i < mine; ++i) {
            load(i + kStages - 1);
            cp_wait<kStages - 1>();
            __syncwarp();
            const uint32_t tK = ring + (i % kStages) * 2 * kUnitBytes, tV = tK + kUnitBytes;
            const int key0 = (u0 + warp + i * kWarps) * kUnit;
            float s[RT][2][4];
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int n = 0; n < 2; ++n) s[t][n][0] = s[t][n][1] = s[t][n][2] = s[t][n][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                uint32_t b0, b1, b2, b3;
                const int m = lane >> 3;
                ldsm_x4(tK + swz((m >> 1) * 8 + (lane & 7), kk * 2 + (m & 1)), b0, b1, b2, b3);
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    uint32_t* q = qf[RT > 1 ? 0 : kk];
                    if (RT > 1) ldsm_x4(s_q + swz(t * 16 + (lane & 15), kk * 2 + (lane >> 4)), q[0], q[1], q[2], q[3]);
                    mma16816<DT>(s[t][0], q, b0, b1);
                    mma16816<DT>(s[t][1], q, b2, b3);
                }
            }
            const bool edge = key0 + kUnit > L;  // the unit holds new rows, or ends the keys
            auto sees = [&](int t, int h, int key) -> bool {
                if (key < limit[t][h]) return true;
                const int j = key - L;
                return a.mask != nullptr && j >= 0 && j < n_new && ((anc[t][h] >> j) & 1ull);
            };
            bool up = false;
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int h = x >> 1;
                        float v = s[t][n][x] * sl2;
                        if (edge) v = sees(t, h, key0 + n * 8 + (lane & 3) * 2 + (x & 1)) ? v : -INFINITY;
                        s[t][n][x] = v;
                        up |= v > m_run[t][h] + 8.f;
                    }
            // the maximum moves only when a score passes it by 8 (weights stay below 2^8: 16-bit P and the
            // 32-bit sums carry them), so most units need no row maximum and leave O alone
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float mx = fmaxf(fmaxf(s[t][0][2 * h], s[t][0][2 * h + 1]),
                                         fmaxf(s[t][1][2 * h], s[t][1][2 * h + 1]));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        const float m = fmaxf(m_run[t][h], mx);
                        const float alpha = ex2(m_run[t][h] - safe(m));
                        m_run[t][h] = m;
                        l_run[t][h] *= alpha;
#pragma unroll
                        for (int d = 0; d < 16; ++d) {
                            o[t][d][2 * h] *= alpha;
                            o[t][d][2 * h + 1] *= alpha;
                        }
                    }
            }
            uint32_t p[RT][4];
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float m = safe(m_run[t][h]) - kLift<DT>;
                        const uint32_t w = E::down(ex2(s[t][n][2 * h] - m), ex2(s[t][n][2 * h + 1] - m));
                        // the sum adds the rounded weights that the product uses: they add up to one
                        const float2 f = E::up(w);
                        l_run[t][h] += f.x + f.y;
                        p[t][n * 2 + h] = w;
                    }
            if (edge) {
                // A new row of V may hold infinities or NaN that some rows do not see, and 0 * NaN is NaN:
                // such elements are added to the rows that see them and taken out of the product.
                bool odd = false;
#pragma unroll
                for (int x = 0; x < kUnitBytes / 512; ++x) {
                    const uint4 v = *reinterpret_cast<const uint4*>(ring_p + (tV - ring) + x * 512 + lane * 16);
                    odd |= E::odd(v.x) || E::odd(v.y) || E::odd(v.z) || E::odd(v.w);
                }
                if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
                    for (int key = 0; key < kUnit; ++key)
#pragma unroll 1
                        for (int d = 0; d < 16; ++d) {
                            const uint32_t w = *reinterpret_cast<const uint32_t*>(ring_p + (tV - ring) + swz(key, d) +
                                                                                  (lane & 3) * 4);
                            if (!E::odd(w)) continue;
                            float2 f = E::up(w);
                            if (isfinite(f.x)) f.x = 0.f;
                            if (isfinite(f.y)) f.y = 0.f;
                            for (int t = 0; t < RT; ++t)
                                for (int h = 0; h < 2; ++h)
                                    if (sees(t, h, key0 + key)) {
#pragma unroll
                                        for (int dd = 0; dd < 16; ++dd)
                                            if (dd == d) {
                                                o[t][dd][2 * h] += f.x;
                                                o[t][dd][2 * h + 1] += f.y;
                                            }
                                    }
                        }
                    __syncwarp();
#pragma unroll 1
                    for (int x = lane; x < kUnitBytes / 4; x += 32) {
                        uint32_t* w = reinterpret_cast<uint32_t*>(ring_p + (tV - ring)) + x;
                        const float2 f = E::up(*w);
                        *w = (isfinite(f.x) ? (*w & 0xffffu) : 0u) | (isfinite(f.y) ? (*w & 0xffff0000u) : 0u);
                    }
                    __syncwarp();
                }
            }
#pragma unroll
            for (int dp = 0; dp < 8; ++dp) {
                uint32_t b0, b1, b2, b3;
                const int m = lane >> 3;
                ldsm_x4_t(tV + swz((m & 1) * 8 + (lane & 7), dp * 2 + (m >> 1)), b0, b1, b2, b3);
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    mma16816<DT>(o[t][2 * dp], p[t], b0, b1);
                    mma16816<DT>(o[t][2 * dp + 1], p[t], b2, b3);
                }
            }
            __syncwarp();
        }
        cp_wait<0>();
        __syncthreads();  // every ring is free: the partial rows take its place
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l_run[t][h] += __shfl_xor_sync(0xffffffffu, l_run[t][h], 1);
                l_run[t][h] += __shfl_xor_sync(0xffffffffu, l_run[t][h], 2);
                const int r = t * 16 + (lane >> 2) + h * 8;
                if (r < e.rows) {
                    float* dst = s_part + (warp * RT * 16 + r) * kRowPad + (lane & 3) * 2;
#pragma unroll
                    for (int d = 0; d < 16; ++d)
                        *reinterpret_cast<float2*>(dst + d * 8) = make_float2(o[t][d][2 * h], o[t][d][2 * h + 1]);
                    if ((lane & 3) == 0) s_ml[warp * RT * 16 + r] = make_float2(m_run[t][h], l_run[t][h]);
                }
            }
        __syncthreads();

        const int step = s_at.step;
        int c0 = s_at.cta0, pieces = s_at.pieces;
        if (step == 0) {
            c0 = unit_cta(s_at.total, s_at.ctas, s_at.item_first);
            pieces = unit_cta(s_at.total, s_at.ctas, s_at.item_first + e.units - 1) - c0 + 1;
        }
        if (pieces == 1) {
            for (int r = warp; r < e.rows; r += kWarps) {
                float4 acc;
                float m, l;
                join_warps<kWarps, RT>(s_part, s_ml, r, acc, m, l);
                put_row<DT>(a, e, kvh, r, acc, l);
            }
        } else {
            constexpr int rows = kFewRows;
            const int slot = step > 0 ? cta * 2 : cta * 2 + (cta == c0 ? 1 : 0);
            for (int r = warp; r < e.rows; r += kWarps) {
                float4 acc;
                float m, l;
                join_warps<kWarps, RT>(s_part, s_ml, r, acc, m, l);
                *reinterpret_cast<float4*>(a.few.o + ((int64_t)slot * rows + r) * HD + lane * 4) = acc;
                if (lane == 0) a.few.ml[(int64_t)slot * rows + r] = make_float2(m, l);
            }
            __threadfence();
            __syncthreads();
            int32_t* count = a.few.count + c0;  // (a CTA is the first of one cut item at most)
            if (tid == 0) {
                const int before = atomicAdd(count, 1);
                if (before >= pieces) flag_status(a.c.status, GRAFT_STATUS_WORKSPACE);
                if (before == pieces - 1) {
                    // the last to arrive: it joins the pieces, after its run (a run cuts at most two items), when
                    // O's registers are free for the reads
                    *count = 0;
                    Start& p = s_pending[s_n_pending++];
                    p = s_at;
                    p.cta0 = c0;
                    p.pieces = pieces;
                }
            }
        }
        __syncthreads();  // the staged rows are read: the next item's copies may overwrite them
        const int left = s_at.count - (u1 - u0);
        if (left <= 0) break;
        // the run goes on with the next head, or the next entry's first
        __syncthreads();
        if (tid == 0) {
            s_at.count = left;
            s_at.unit = 0;
            s_at.item_first += s_at.e.units;
            if (++s_at.head == a.c.Hkv) {
                s_at.head = 0;
                const Entry* next = entries + ++s_at.entry;
                if (RT > 1) {
                    const int4 lo = __ldcg(reinterpret_cast<const int4*>(next));
                    const int4 hi = __ldcg(reinterpret_cast<const int4*>(next) + 1);
                    s_at.e = Entry{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                } else {
                    s_at.e = *next;
                }
            }
        }
        __syncthreads();
        begin();
        pages = fetch_pages(0, true);
        pages_at = 0;
    }
    // (the pieces are read from L2, after the barrier behind the counter's atomic; their writers fenced before it)
    for (int k = 0; k < s_n_pending; ++k) {
        join_pieces<DT, RT, kWarps>(a, s_pending[k], smem);
    }
    leave();
}

template <int DT, int RT, int W>
int launch(const AttnArgs& a, cudaStream_t st) {
    static bool attr_set[64] = {};
    int dev = 0;
    if (!cuda_ok(cudaGetDevice(&dev))) return GRAFT_ERR_CUDA;
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        if (!cuda_ok(cudaFuncSetAttribute(few_kernel<DT, RT, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          smem_bytes(W, RT))))
            return GRAFT_ERR_CUDA;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    launch_pdl(few_kernel<DT, RT, W>, dim3(a.shape.ctas), dim3(W * 32), smem_bytes(W, RT), st, a);
    count_launches(1);
    return launch_status();
}

template <int DT>
int launch_type(const AttnArgs& a, cudaStream_t st) {
    if (a.shape.few_warps == 4)
        return a.shape.few_rows == 16 ? launch<DT, 1, 4>(a, st) : launch<DT, 2, 4>(a, st);
    return a.shape.few_rows == 16 ? launch<DT, 1, 8>(a, st) : launch<DT, 2, 8>(a, st);
}

}  // namespace

int few_launch(const AttnArgs& a, cudaStream_t st) {
    return a.c.dtype == GRAFT_BF16 ? launch_type<GRAFT_BF16>(a, st) : launch_type<GRAFT_FP16>(a, st);
}

}  // namespace paged
}  // namespace graft
