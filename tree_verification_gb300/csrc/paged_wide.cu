// Attention of many query rows a KV head over a paged cache, on the tcgen05
// tensor cores: prompt chunks and draft trees.
//
//   o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),  s_j = scale log2(e) q.k_j
//
// A work item is 256 query rows (two tiles of T = 128 / G new rows with their
// G heads; one tile where the rest of the sequence fits it) of one sequence
// and KV head against a range of 128-key blocks; the plan lists the items,
// longest first, deals whole rounds of them to one persistent CTA per SM in a
// snake, and splits what is left over by keys, so that all end together.
// Tensor-core bound: 4 x 128 x 128 products a row and key block; two tiles
// share every K and V block, so a block's 64 KB serve 256 rows.
//
// Warps: one producer, one MMA issuer (one thread), eight of softmax (one per
// 32 rows).  TMEM holds S_0, S_1, O_0, O_1; P overwrites S as packed 16-bit
// pairs and feeds the PV product from there.  The pipeline (rings, barriers,
// the order of the products) is that of the dense persistent kernel
// (attention_tcp.cu).  What pages and ragged chunks change:
//   * a block of K or V comes in pieces, one TMA box per page (a block inside
//     a page of 128 rows or more is one box); the producer's lanes each hold a page number,
//     fetched one block ahead, and issue their own box.  A page that the
//     item's keys do not reach, or outside the pool, is a box out of bounds:
//     zeros.
//   * causal and tree masks cover only the blocks that reach past the first
//     new row; the keep-bits of a row's 128 keys are built once a block.
//   * rows of a tile that hold no query row (G not a power of two) are zero
//     from the start and never loaded.
//   * with a window (kWindow, graft_paged_attention_window) an item's blocks are
//     those of the first tokens and those from its earliest row's window on;
//     the blocks that some row's window starts in or behind are masked and
//     cleaned like those with new rows, and a row that has seen nothing as yet
//     takes a block's maximum anew.  (16 trees at group 16 over 4096 keys 137
//     us; 4100 prompt rows over 1024, where 4 of an item's 10.5 blocks are
//     masked, 121.)
//   * V elements that are infinite or NaN in blocks with masked keys are
//     taken out in shared memory (0 * NaN is NaN) and given to the rows that
//     do see them after the item's rows are written.
//
// Every mbarrier wait is bounded; on timeout the CTA raises
// GRAFT_STATUS_TIMEOUT, stops issuing work, drains what it issued (again
// with a bound) and frees its TMEM before returning.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <type_traits>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace graft {
namespace paged {
namespace {

using namespace tc;

constexpr int BN = kBlockKeys;
constexpr int SK = 2;  // K ring depth
constexpr int SV = 3;  // V ring depth
constexpr int NTHREADS = 320;
// A K or V block lies as 16 groups of 8 keys, a group as its two halves of 64 dims (8 rows of 128 bytes each,
// 128-byte swizzle): groups 2 KB apart, halves 1 KB.  So one box brings a page's rows with all their dims, and
// both products still find their operand at one stride.
constexpr uint32_t HALF_BYTES = 1024, GROUP_BYTES = 2048;
constexpr uint32_t BLK_BYTES = (BN / 8) * GROUP_BYTES;
constexpr uint32_t Q_TILE_BYTES = 2 * 128 * 64 * 2;  // 128 rows x 128 dims
constexpr uint32_t OFF_Q = 0;
constexpr uint32_t OFF_K = OFF_Q + 2 * Q_TILE_BYTES;
constexpr uint32_t OFF_V = OFF_K + SK * BLK_BYTES;
constexpr uint32_t OFF_BAR = OFF_V + SV * BLK_BYTES;
constexpr int BAR_Q = 0;                 // an item's Q tiles landed (one phase per item)
constexpr int BAR_KF = 1;                // [SK] K block landed
constexpr int BAR_KE = BAR_KF + SK;      // [SK] K block consumed by the S products
constexpr int BAR_VF = BAR_KE + SK;      // [SV] V block landed
constexpr int BAR_VE = BAR_VF + SV;      // [SV] V block consumed by the PV products
constexpr int BAR_S = BAR_VE + SV;       // [tile] S_t ready in TMEM
constexpr int BAR_P = BAR_S + 2;         // [tile] P_t written to TMEM (128 arrivals)
// [tile] an item's MMAs completed: tile 0's one phase per item, tile 1's one phase per item of two tiles.  (Tile 1
// takes no part in the others and so holds none of them back: a phase for each could pass it by.)
constexpr int BAR_DONE = BAR_P + 2;
constexpr int BAR_OFREE = BAR_DONE + 2;  // [tile] an item's O_t read out of TMEM (128 arrivals)
constexpr int BAR_DRAIN = BAR_OFREE + 2;  // after an abort: everything issued has completed
constexpr int N_BARS = BAR_DRAIN + 1;
constexpr uint32_t OFF_MISC = OFF_BAR + N_BARS * 8;  // tmem slot, abort flag, odd flags
constexpr uint32_t SMEM_BYTES = OFF_MISC + 64 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
constexpr uint32_t TM_S = 0;    // + tile * 128
constexpr uint32_t TM_O = 256;  // + tile * 128
constexpr float RESCALE_LOG2 = 8.f;
// Pipeline waits are bounded by kWaitNs (a.wait_ns in the failure-path tests); the teardown's waits on the loads
// (kDrainNs) and products (kWaitNs) in flight keep fixed bounds.
constexpr uint64_t kWaitNs = 500000000ull;
constexpr uint64_t kDrainNs = 100000000ull;

struct Maps {
    CUtensorMap q, k, v;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ bool aborted(const volatile uint32_t* flag) { return *flag != 0; }
__device__ __forceinline__ void raise_abort(volatile uint32_t* flag, int32_t* status) {
    *flag = 1;
    flag_status(status, GRAFT_STATUS_TIMEOUT);
}
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
// kind::f16 with 32-bit accumulation; fp16 or bf16 operands (both alike), M 128
template <int DT>
__host__ __device__ constexpr uint32_t idesc(int N, bool b_mn) {
    return (1u << 4) | (DT == GRAFT_BF16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? (1u << 16) : 0u) |
           ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void* tmap, uint32_t bar, int c0, int c1, int c2,
                                            int c3, int c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, "
        "%6, %7}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}
// a pair of weights rounded, and their sum in 32 bits
template <int DT>
__device__ __forceinline__ float2 add_pair(float2 acc, uint32_t w) {
    if (DT == GRAFT_BF16) return add_bf16x2_f32(acc, w);
    float x = acc.x, y = acc.y;
    const unsigned short lo = (unsigned short)(w & 0xffffu), hi = (unsigned short)(w >> 16);
    asm("add.rn.f32.f16 %0, %1, %0;" : "+f"(x) : "h"(lo));
    asm("add.rn.f32.f16 %0, %1, %0;" : "+f"(y) : "h"(hi));
    return make_float2(x, y);
}

// What a row sees of the 128 keys from kb on: keys below `limit`, and new row j (key L + j) where bit j of anc is set.
__device__ __forceinline__ void keep_bits(uint32_t* w, int kb, int limit, int L, uint64_t anc) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int n = limit - (kb + 32 * x);
        uint32_t m = n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : ((1u << n) - 1u));
        const int s = kb + 32 * x - L;  // the word's first key is new row s
        if (s >= 0)
            m |= s < 64 ? (uint32_t)(anc >> s) : 0u;
        else if (s > -32)
            m |= (uint32_t)(anc << -s);
        w[x] = m;
    }
}

// The same with a window: of the keys below the limit, those from `low` on and the first tokens'.
__device__ __forceinline__ void hide_bits(uint32_t* w, int kb, int first, int low) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int from = max(first - (kb + 32 * x), 0), to = min(low - (kb + 32 * x), 32);
        if (from >= to) continue;
        const uint32_t below = to >= 32 ? 0xffffffffu : (1u << to) - 1u;
        w[x] &= ~(below & ~((1u << from) - 1u));
    }
}

// Infinite and NaN elements of V that row r sees among keys [k0, k1): added to the row's 128 dims where they
// were written (16-bit rows of O, or 32-bit partial rows, four dims every 512 floats).  Rare, so out of line and straight from memory.
template <int DT, bool kWindow>
__device__ __noinline__ void add_odd(const GraftPagedCache& c, const void* V, const int32_t* table, int page_shift,
                                     int kvh, int k0, int k1, int limit, int first, int low, int L, uint64_t anc,
                                     void* row16, float* row32) {
    using E = Elem<DT>;
    for (int key = k0; key < k1; ++key) {
        const int j = key - L;
        if (!((key < limit && (!kWindow || key >= low || key < first)) || (j >= 0 && j < 64 && ((anc >> j) & 1ull)))) continue;
        const int page = table[key >> page_shift];
        if (page < 0 || page >= c.num_pages) continue;
        const int64_t at = ((((int64_t)page << page_shift) + (key & (c.page_rows - 1))) * c.Hkv + kvh) * HD;
        const uint32_t* v = reinterpret_cast<const uint32_t*>(static_cast<const typename E::T*>(V) + at);
        for (int x = 0; x < HD / 2; ++x) {
            if (!E::odd(v[x])) continue;
            float2 f = E::up(v[x]);
            if (isfinite(f.x)) f.x = 0.f;
            if (isfinite(f.y)) f.y = 0.f;
            if (row32 != nullptr) {
                float* o = row32 + (x >> 1) * 512 + (x & 1) * 2;
                o[0] += f.x;
                o[1] += f.y;
            } else {
                uint32_t* o = static_cast<uint32_t*>(row16) + x;
                const float2 g = E::up(*o);
                *o = E::down(g.x + f.x, g.y + f.y);
            }
        }
    }
}

// kTestWaits: pipeline waits bounded by a.wait_ns (the failure-path tests); otherwise by a constant.
template <int DT, bool kTestWaits, bool kWindow>
__global__ void __launch_bounds__(NTHREADS, 1)
wide_kernel(const __grid_constant__ Maps maps, const __grid_constant__ AttnArgs a) {
    using E = Elem<DT>;
    // See paged_few.cu: small weights keep their bits.  (Lifted by 2^3 in windows, so that fewer blocks are weighed twice,
    // weights below 2^-17 of the largest lost bits, which show where the largest is that of a first token whose values are
    // small.)
    constexpr float kLift = DT == GRAFT_FP16 ? 7.f : 0.f;
    // Most that the weights of a block and row may sum to by an old maximum.  In windows, where heads of scores 3 apart
    // weighed many a block twice, it is what 128 finite weights can: a block is weighed again where one overflows (chunks of
    // up to 2048 rows over 1024 keys: 131 us, 138 by 2^15, 126 with the lift of 2^3).
    constexpr float kMaxSum = DT == GRAFT_FP16 ? (kWindow ? BN * 65504.f : 32768.f) : 65536.f;
    const uint64_t wait_ns = kTestWaits ? a.wait_ns : kWaitNs;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + OFF_MISC);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(gbase + OFF_MISC + 4);
    // Stamp (place in the deal + 1) of the last item in whose blocks V held infinities or NaN: [0..1] by parity
    // among the items of two tiles, [2..3] among the others.  Tile 0 sets it before it signals P_0 and a word is
    // set again two items of its kind later, which takes the P of every thread that may still read it.
    volatile uint32_t* odd_item = reinterpret_cast<volatile uint32_t*>(gbase + OFF_MISC + 8);
    auto bar = [&](int i) { return base + OFF_BAR + 8u * (uint32_t)i; };

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.G, T = a.shape.tile_tokens;
    // an item's block v lies at block v, or v + gap behind the first tokens' blocks
    const int behind = kWindow ? window_units(a.first, BN) : 0;
    auto block_at = [&](int v, int gap) { return kWindow && v >= behind ? v + gap : v; };

    // Prologue that touches no global memory: it overlaps the previous kernel's tail.
    if (tid == 0) {
        for (int i = 0; i < N_BARS; ++i) {
            uint32_t cnt = 1;
            if (i == BAR_P || i == BAR_P + 1 || i == BAR_OFREE || i == BAR_OFREE + 1) cnt = 128;
            mbar_init(bar(i), cnt);
        }
        *abort_flag = 0;
        for (int i = 0; i < 4; ++i) odd_item[i] = 0;
        fence_mbar_init();
    } else if (tid == 32) {
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc(base + OFF_MISC, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    if (T * G < 128) {
        // rows that no box writes
        for (uint32_t x = tid; x < 2 * Q_TILE_BYTES / 16; x += NTHREADS)
            *reinterpret_cast<uint4*>(gbase + OFF_Q + x * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    griddep_wait();
    griddep_launch_dependents();
    const PlanHead& head = *reinterpret_cast<const PlanHead*>(a.plan);
    const Wide* wide = reinterpret_cast<const Wide*>(a.plan + a.shape.off_wide);
    const Wide* last = reinterpret_cast<const Wide*>(a.plan + a.shape.off_last);
    // (the first item's line is on its way while the head is read)
    asm volatile("prefetch.global.L1 [%0];" ::"l"(last + blockIdx.x));
    const int* where = reinterpret_cast<const int*>(a.plan + a.shape.off_where) + blockIdx.x;
    const int where0 = where[0], where1 = where[1];
    const bool fits = plan_fits(a, head);
    if (!fits && blockIdx.x == 0 && tid == 0) flag_status(a.c.status, GRAFT_STATUS_PLAN);
    const int rounds = fits ? head.rounds : 0, n_mine = fits ? rounds + where1 - where0 : 0;
    // this CTA's k-th item: one of every round, dealt in a snake, then its last ones
    auto item_at = [&](int k) -> const Wide* {
        if (k < rounds) return wide + (k * (int)gridDim.x + ((k & 1) ? (int)(gridDim.x - 1 - blockIdx.x) : (int)blockIdx.x));
        return last + (where0 + k - rounds);
    };
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    int k_issued = 0, v_issued = 0, q_issued = 0;
    if (warp == 0) {
        // ------------------------------------------------------------ producer: every lane issues its own boxes
        const int page_box = min(a.c.page_rows, BN);  // rows of a box
        const int pieces = BN / page_box;
        const bool issues = lane < pieces;
        struct Cur {
            int k, j;      // place in the deal (-1: past the end), block
            int kvh;
            int blk0, nblk, keys, tok, two, b;  // of the item
            int gap, low;  // (window)
            int row;       // first pool row / 8 of this lane's box of block j (out of bounds: zeros)
        };
        auto lookup = [&](Cur& c) {
            if (c.k < 0 || !issues) return;
            const int key = block_at(c.blk0 + c.j, c.gap) * BN + lane * page_box;
            int row = 0x7fffffff >> 3;
            if (key < c.keys && (!kWindow || key < a.first || key + page_box > c.low)) {
                const int page = a.c.block_table[(int64_t)c.b * a.c.max_pages + (key >> a.page_shift)];
                if (page >= 0 && page < a.c.num_pages)
                    row = ((page << a.page_shift) + (key & (a.c.page_rows - 1))) >> 3;
                else
                    flag_status(a.c.status, GRAFT_STATUS_PAGE);
            }
            c.row = row;
        };
        auto seek = [&](Cur& c) {
            if (c.k >= n_mine) {
                c.k = -1;
                return;
            }
            const Wide w = *item_at(c.k);
            c.kvh = w.kvh;
            c.j = 0;
            c.blk0 = w.blk0;
            c.nblk = w.nblk;
            c.keys = w.keys;
            c.tok = w.q0 + w.tok0;
            c.two = w.two;
            c.b = w.b;
            if (kWindow) {
                c.gap = w.gap;
                c.low = w.L + (a.mask != nullptr ? 0 : w.tok0) - a.window + 1;
            }
        };
        auto advance = [&](Cur& c) {
            if (c.k < 0) return;
            if (++c.j < c.nblk) return;
            ++c.k;
            seek(c);
        };
        auto load = [&](Cur& c, const CUtensorMap* map, uint32_t dst, uint32_t full) {
            if (lane == 0) mbar_expect_tx(full, BLK_BYTES);
            __syncwarp();
            if (issues)
                tma_load_5d(dst + lane * (page_box / 8) * GROUP_BYTES, map, full, 0, 0, 0, c.row, c.kvh);
            advance(c);
            lookup(c);
        };
        auto load_q = [&](const Cur& c) {
            ++q_issued;
            const int tiles = c.two ? 2 : 1;
            if (lane == 0) {
                mbar_expect_tx(bar(BAR_Q), (uint32_t)(tiles * 2 * T * G * 128));
                for (int t = 0; t < tiles; ++t)
                    for (int h = 0; h < 2; ++h)
                        tma_load_3d(base + OFF_Q + t * Q_TILE_BYTES + h * (Q_TILE_BYTES / 2), &maps.q, bar(BAR_Q),
                                    h * 64, c.kvh * G, c.tok + t * T);
            }
        };
        Cur kc{};
        seek(kc);
        Cur cc = kc;
        if (kc.k >= 0) load_q(kc);
        lookup(kc);
        Cur vc = kc;
        auto load_k = [&]() {
            load(kc, &maps.k, base + OFF_K + (k_issued % SK) * BLK_BYTES, bar(BAR_KF + k_issued % SK));
            ++k_issued;
        };
        auto load_v = [&]() {
            load(vc, &maps.v, base + OFF_V + (v_issued % SV) * BLK_BYTES, bar(BAR_VF + v_issued % SV));
            ++v_issued;
        };
        for (int s = 0; s < SK && kc.k >= 0; ++s) load_k();
        for (int s = 0; s < SV && vc.k >= 0; ++s) load_v();
        for (int g = 0; cc.k >= 0; ++g) {
            Cur nx = cc;
            advance(nx);
            const bool next_q = nx.k >= 0 && nx.j == 0;  // block g ends its item: the next Q follows
            bool ok = true;
            if (kc.k >= 0 || next_q) {
                ok = __all_sync(0xffffffffu,
                                mbar_wait(bar(BAR_KE + g % SK), (g / SK) & 1, wait_ns) && !aborted(abort_flag));
                if (!ok) break;
                if (next_q) load_q(nx);
                if (kc.k >= 0) load_k();
            }
            if (vc.k >= 0) {
                ok = __all_sync(0xffffffffu,
                                mbar_wait(bar(BAR_VE + g % SV), (g / SV) & 1, wait_ns) && !aborted(abort_flag));
                if (!ok) break;
                load_v();
            }
            cc = nx;
        }
        if (cc.k >= 0 && lane == 0 && !aborted(abort_flag)) raise_abort(abort_flag, a.c.status);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (lane 0 alone)
        if (lane == 0) {
            const uint32_t idS = idesc<DT>(BN, false);
            const uint32_t idO = idesc<DT>(HD, true);
            const uint64_t q_desc = sdesc_sw128(base + OFF_Q, 16, 1024);
            const uint64_t k_desc = sdesc_sw128(base + OFF_K, 16, GROUP_BYTES);
            const uint64_t v_desc = sdesc_sw128(base + OFF_V, HALF_BYTES, GROUP_BYTES);
            int kst = 0, kph = 0;
            int vst = 0, vph = 0;
            uint32_t pph0 = 0, pph1 = 0;  // phases of the tiles' P barriers
            // The barrier that the next group of products needs is tested, without blocking, just before
            // the last two products of a group (see attention_tcp.cu).
            struct Pre {
                int bar;
                uint32_t ph;
            };
            const Pre none{-1, 0u};
            auto test_pre = [&](Pre pre) -> bool { return pre.bar < 0 || mbar_test_now(bar(pre.bar), pre.ph); };
            auto wait_pre = [&](Pre pre, bool ready) -> bool {
                return ready || mbar_wait(bar(pre.bar), pre.ph, wait_ns);
            };
            auto group_S = [&](int t, bool last, Pre nxt) -> bool {
                bool ready = false;
                const uint64_t kd = k_desc + ((kst * BLK_BYTES) >> 4);
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    if (kk == HD / 16 - 2) ready = test_pre(nxt);
                    const uint32_t off = (kk >> 2) * HALF_BYTES + (kk & 3) * 32;
                    const uint32_t qoff = t * Q_TILE_BYTES + (kk >> 2) * (Q_TILE_BYTES / 2) + (kk & 3) * 32;
                    mma_bf16_ss(tmem + TM_S + t * 128, q_desc + (qoff >> 4), kd + (off >> 4), idS, kk > 0);
                }
                mma_commit(bar(BAR_S + t));
                if (last) {
                    mma_commit(bar(BAR_KE + kst));
                    if (++kst == SK) { kst = 0; kph ^= 1; }
                }
                return ready;
            };
            auto group_PV = [&](int t, bool last, bool first, Pre nxt) -> bool {
                bool ready = false;
                const uint64_t vd = v_desc + ((vst * BLK_BYTES) >> 4);
                const uint32_t p = tmem + TM_S + t * 128;
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk) {
                    if (kk == BN / 16 - 2) ready = test_pre(nxt);
                    mma_bf16_ts(tmem + TM_O + t * 128, p + kk * 8, vd + ((kk * 2 * GROUP_BYTES) >> 4), idO, !first || kk > 0);
                }
                if (last) mma_commit(bar(BAR_VE + vst));
                return ready;
            };
            bool ok = true;
            int q = 0, q1 = 0;  // items issued; those of two tiles
            // one item's products; a copy each for one and two tiles, so that the loop decides nothing
            auto run_item = [&](auto two_tiles, int nblk) {
                constexpr bool two = decltype(two_tiles)::value;
                ok = mbar_wait(bar(BAR_Q), q & 1, wait_ns) && !aborted(abort_flag) &&
                     mbar_wait(bar(BAR_KF + kst), kph, wait_ns);
                if (!ok) return;
                tc_fence_after();
                Pre vf{BAR_VF + vst, (uint32_t)vph};
                bool vf_ready = group_S(0, !two, two ? none : vf);
                if (two) vf_ready = group_S(1, true, vf);
                for (int j = 0; j < nblk && ok; ++j) {
                    const bool more = j + 1 < nblk;
                    ok = wait_pre(vf, vf_ready) && mbar_wait(bar(BAR_P), pph0, wait_ns);
                    // the item's first PV overwrites O_t: the previous item's epilogue must have read it
                    if (ok && j == 0 && q > 0) ok = mbar_wait(bar(BAR_OFREE), (q - 1) & 1, wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const Pre kf{BAR_KF + kst, (uint32_t)kph};
                    const Pre p1 = two ? Pre{BAR_P + 1, pph1} : none;
                    const int vst_next = vst + 1 == SV ? 0 : vst + 1;
                    const int vph_next = vst + 1 == SV ? vph ^ 1 : vph;
                    const Pre vn{BAR_VF + vst_next, (uint32_t)vph_next};
                    bool p1_ready;
                    if (more) {
                        const bool kf_ready = group_PV(0, !two, j == 0, kf);
                        ok = wait_pre(kf, kf_ready);
                        if (!ok) break;
                        tc_fence_after();
                        p1_ready = group_S(0, !two, two ? p1 : vn);
                    } else {
                        p1_ready = group_PV(0, !two, j == 0, p1);
                    }
                    vf_ready = !two && more ? p1_ready : false;
                    if (two) {
                        ok = wait_pre(p1, p1_ready);
                        if (ok && j == 0 && q1 > 0) ok = mbar_wait(bar(BAR_OFREE + 1), (q1 - 1) & 1, wait_ns);
                        if (!ok) break;
                        tc_fence_after();
                        group_PV(1, true, j == 0, none);
                        vf_ready = more ? group_S(1, true, vn) : false;
                        pph1 ^= 1u;
                    }
                    vf = vn;
                    vst = vst_next;
                    vph = vph_next;
                    pph0 ^= 1u;
                }
                if (two) mma_commit(bar(BAR_DONE + 1));
                mma_commit(bar(BAR_DONE));
                ++q;
                q1 += two;
            };
            for (int k = 0; ok && k < n_mine; ++k) {
                const Wide& w = *item_at(k);
                if (w.two != 0)
                    run_item(std::true_type{}, w.nblk);
                else
                    run_item(std::false_type{}, w.nblk);
            }
            if (!ok && !aborted(abort_flag)) raise_abort(abort_flag, a.c.status);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax + epilogue
        const int t = (warp - 2) >> 2;
        const int quad = warp & 3;
        const int r = quad * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        const uint32_t sbuf = tmem + lane_base + TM_S + t * 128;
        const float sl2 = a.scale * 1.4426950408889634f;
        const int rtok = r / G, rg = r - rtok * G;
        bool ok = true;
        int q = 0, n_two = 0;  // items passed; those of two tiles (phase of DONE: tile 0's, tile 1's)
        int g = 0, gv = 0;     // blocks of this tile, blocks of the CTA
        for (int k = 0; ok && k < n_mine; ++k) {
            const Wide* at = item_at(k);
            // The block loop holds only counts; an edge block reads the item and the row's mask again, and so
            // does the epilogue.
            int nblk, edge;
            int front = 0;          // (window) blocks before it some row does not see whole
            bool searching = false;  // (window) the row may see its first key in a later block
            bool two;
            {
                const Wide& w = *at;
                nblk = w.nblk;
                two = w.two != 0;
                // first block that some row of the tile does not see whole
                edge = (a.mask != nullptr ? w.L : min(w.L + w.tok0 + t * T + 1, w.keys)) / BN - w.blk0;
                if (kWindow) {
                    edge -= w.gap;
                    const int rows = a.mask != nullptr ? w.n : min(w.tok0 + (two ? 2 * T : T), w.n);
                    const int low = w.L + rows - a.window;  // of the last row
                    if (low > 0) front = (low + BN - 1) / BN - w.gap - w.blk0;
                    searching = rtok < T && w.tok0 + t * T + rtok < w.n;
                }
            }
            // (low, with a window: of the keys below the limit, those from it on and the first tokens' are seen)
            auto row_of = [&](const Wide& w, int& tok, int& limit, int& low, uint64_t& anc) -> bool {
                tok = w.tok0 + t * T + rtok;
                const bool row_ok = rtok < T && tok < w.n;
                limit = low = 0;
                anc = 0;
                if (row_ok) {
                    limit = a.mask != nullptr ? w.L : w.L + tok + 1;
                    if (a.mask != nullptr)
                        anc = a.mask[w.q0 + tok] & (w.n >= 64 ? ~0ull : ((1ull << w.n) - 1ull));
                    if (kWindow) {
                        low = max(a.mask != nullptr ? min(window_low(anc, a.window, w.L), w.L) : limit - a.window, 0);
                        anc = window_mask(anc, a.window, a.first, w.L);
                    }
                }
                return row_ok;
            };
            if (t == 1 && !two) {
                gv += nblk;
                ++q;
                continue;
            }
            auto odd_word = [&]() { return odd_item + (two ? (n_two & 1) : 2 + ((q - n_two) & 1)); };
            // (Without a window a row that sees none of the range's first block sees none of the range: new rows see a run
            // of keys from the front, and a tree's 64 keys lie in one block unless prefix keys come first; so the maximum
            // of a row that is still -inf after the first block stays so, and its weights are 0.  With one a row may see
            // its first key in a later block: there it takes that block's maximum anew.)
            float m_used = -INFINITY, l_sum = 0.f;
            {
                for (int j = 0; j < nblk; ++j) {
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(bar(BAR_S + t), g & 1, wait_ns) && !aborted(abort_flag));
                    if (!ok) break;
                    ++g;
                    tc_fence_after();
                    if (j >= edge || (kWindow && j < front)) {
                        // Masked scores are written back as -inf, in a pass of their own over S in tensor memory:
                        // the block loop proper carries no masking code (inlined it cost all blocks 4%).
                        const Wide& w = *at;
                        int tok, limit, low;
                        uint64_t anc;
                        row_of(w, tok, limit, low, anc);
                        uint32_t keep[4];
                        const int kb = block_at(w.blk0 + j, w.gap) * BN;
                        keep_bits(keep, kb, limit, w.L, anc);
                        if (kWindow) hide_bits(keep, kb, a.first, low);
#pragma unroll
                        for (int x = 0; x < BN / 32; ++x) {
                            float s[32];
                            tmem_ld32(sbuf + x * 32, s);
                            tmem_wait_ld();
#pragma unroll
                            for (int y = 0; y < 32; ++y) s[y] = ((keep[x] >> y) & 1u) ? s[y] : -INFINITY;
                            tmem_st32(sbuf + x * 32, s);
                        }
                        tmem_wait_st();
                    }
                    if (t == 0 && (j >= edge || (kWindow && j < front))) {
                        // Tile 0 cleans the V block before either tile's PV reads it: rows past the last key
                        // (their pages may hold anything) and infinite or NaN elements that masked rows would
                        // multiply by zero.
                        const int vb = gv + j;
                        ok = __all_sync(0xffffffffu, mbar_wait(bar(BAR_VF + vb % SV), (vb / SV) & 1, wait_ns));
                        if (!ok) break;
                        uint8_t* v0 = gbase + OFF_V + (vb % SV) * BLK_BYTES;
                        const Wide& w = *at;
                        const int kb = block_at(w.blk0 + j, w.gap) * BN, keys = w.keys;
                        const int lo = kWindow && j < front ? 0 : max(w.L - kb, 0), n = BN - lo;
                        // (a thread's pieces: every eighth row from its first on, one group apart)
                        const int r0 = lo + r / 16, c16 = r % 16;
                        uint8_t* first = v0 + (r0 >> 3) * GROUP_BYTES + (c16 >> 3) * HALF_BYTES + (r0 & 7) * 128 +
                                         (c16 & 7) * 16;
                        bool look = true;
                        if constexpr (kWindow) {
                            // Whole blocks are cleaned, most without need: zero times any of a thread's elements is zero,
                            // or there is something to take out.  (Chunks over 1024 keys 141 -> 131 us.)
                            typename E::T2 zeros = E::pack(0u);
#pragma unroll 4
                            for (int x = 0; x < n - r / 16; x += 8) {
                                const uint4 v = *reinterpret_cast<const uint4*>(first + (x >> 3) * GROUP_BYTES);
                                zeros = __hfma2(E::pack(v.x), E::pack(0u), zeros);
                                zeros = __hfma2(E::pack(v.y), E::pack(0u), zeros);
                                zeros = __hfma2(E::pack(v.z), E::pack(0u), zeros);
                                zeros = __hfma2(E::pack(v.w), E::pack(0u), zeros);
                            }
                            look = kb + BN > keys || E::odd(*reinterpret_cast<const uint32_t*>(&zeros));
                        }
                        bool odd = false;
                        for (int x = 0; look && x < n - r / 16; x += 8) {
                            const int rr = r0 + x;
                            uint4* p = reinterpret_cast<uint4*>(first + (x >> 3) * GROUP_BYTES);
                            uint4 v = *p;
                            if (kb + rr >= keys) {
                                *p = make_uint4(0, 0, 0, 0);
                            } else if (E::odd(v.x) || E::odd(v.y) || E::odd(v.z) || E::odd(v.w)) {
                                odd = true;
                                uint32_t* e = &v.x;
#pragma unroll
                                for (int y = 0; y < 4; ++y) {
                                    const float2 f = E::up(e[y]);
                                    e[y] = (isfinite(f.x) ? (e[y] & 0xffffu) : 0u) |
                                           (isfinite(f.y) ? (e[y] & 0xffff0000u) : 0u);
                                }
                                *p = v;
                            }
                        }
                        if (odd) *odd_word() = (uint32_t)k + 1;
                        fence_proxy_async_smem();
                    }
                    float alpha = 1.f;
                    bool rescale = false;
                    float2 acc;
                    float packed[BN / 2];
                    const bool anew = kWindow && j > 0 && __any_sync(0xffffffffu, searching && m_used == -INFINITY);
                    // An item's first block takes its maximum; a later block is weighed against the running
                    // maximum and stands if its row sum stays small; otherwise it is weighed again with its
                    // own maximum (S is still in TMEM).
                    for (int pass = 0; pass < 2; ++pass) {
                        float s[BN];
#pragma unroll
                        for (int x = 0; x < BN / 32; ++x) tmem_ld32(sbuf + x * 32, s + x * 32);
                        tmem_wait_ld();
                        const bool full = j == 0 || pass == 1 || anew;
                        if (full) {
                            float m8[8];
#pragma unroll
                            for (int x = 0; x < 8; ++x) {
                                float m = fmaxf(s[x], s[x + 8]);
#pragma unroll
                                for (int y = 16; y < BN; y += 16) m = fmaxf(m, fmaxf(s[x + y], s[x + y + 8]));
                                m8[x] = m;
                            }
                            const float mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                                                   fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7]))) * sl2;
                            if (j == 0) {
                                m_used = mx;
                            } else if (__any_sync(0xffffffffu, mx > m_used + RESCALE_LOG2)) {
                                const float m_new = fmaxf(mx, m_used);
                                alpha = (m_used == -INFINITY) ? 1.f : ex2(m_used - m_new);
                                m_used = m_new;
                                // (a row that saw its first key has nothing to move)
                                rescale = !kWindow || __any_sync(0xffffffffu, alpha != 1.f);
                            }
                        }
                        const float neg_m = kLift - ((m_used == -INFINITY) ? 0.f : m_used);
                        const float2 sc2 = make_float2(sl2, sl2), nm2 = make_float2(neg_m, neg_m);
                        acc = make_float2(0.f, 0.f);
#pragma unroll
                        for (int x = 0; x < BN; x += 2) {
                            const float2 v = __ffma2_rn(make_float2(s[x], s[x + 1]), sc2, nm2);
                            const uint32_t w = E::down(ex2(v.x), ex2(v.y));
                            acc = add_pair<DT>(acc, w);  // the rounded weights that the product uses
                            packed[x / 2] = __uint_as_float(w);
                        }
                        if (full || !__any_sync(0xffffffffu, !(acc.x + acc.y <= kMaxSum))) break;
                    }
#pragma unroll
                    for (int hh = 0; hh < 4; ++hh) tmem_st16(sbuf + hh * 16, packed + hh * 16);
                    if (rescale) {
                        for (int c0 = 0; c0 < HD; c0 += 32) {
                            float o[32];
                            tmem_ld32(tmem + lane_base + TM_O + t * 128 + c0, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 32; ++x) o[x] *= alpha;
                            tmem_st32(tmem + lane_base + TM_O + t * 128 + c0, o);
                        }
                    }
                    l_sum = l_sum * alpha + (acc.x + acc.y);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(bar(BAR_P + t));
                }
                if (!ok) break;
            }
            // ------------------------------------------------------------ epilogue of the item
            ok = __all_sync(0xffffffffu, mbar_wait(bar(BAR_DONE + t), (t == 0 ? q : n_two) & 1, wait_ns) &&
                                             !aborted(abort_flag));
            if (!ok) break;
            tc_fence_after();
            {
                const Wide w = *at;
                const int kvh = w.kvh;
                int tok, limit, low;
                uint64_t anc;
                const bool row_ok = row_of(w, tok, limit, low, anc);
                const float inv = l_sum != 0.f ? 1.f / l_sum : 0.f;
                const bool direct = w.part < 0;
                typename E::T* orow =
                    static_cast<typename E::T*>(a.O) + ((int64_t)(w.q0 + tok) * a.Hq + kvh * G + rg) * HD;
                // partial rows lie four dims at a time, the tile's 128 rows side by side: a warp's store is one run
                const int64_t pblk = (int64_t)w.part * 2 + t;
                float* part = a.wide_o + (direct ? 0 : pblk * 128 * HD + r * 4);
                for (int c0 = 0; c0 < HD; c0 += 32) {
                    float o[32];
                    tmem_ld32(tmem + lane_base + TM_O + t * 128 + c0, o);
                    tmem_wait_ld();
                    if (c0 == HD - 32) {
                        tc_fence_before();
                        mbar_arrive(bar(BAR_OFREE + t));
                    }
                    if (!row_ok) continue;
                    if (direct) {
#pragma unroll
                        for (int x = 0; x < 32; x += 16) {
                            uint32_t v[8];
#pragma unroll
                            for (int y = 0; y < 8; ++y) v[y] = E::down(o[x + 2 * y] * inv, o[x + 2 * y + 1] * inv);
                            st_global_v8(orow + c0 + x, v);
                        }
                    } else {
#pragma unroll
                        for (int x = 0; x < 32; x += 4)
                            *reinterpret_cast<float4*>(part + ((c0 + x) / 4) * 512) =
                                make_float4(o[x] * inv, o[x + 1] * inv, o[x + 2] * inv, o[x + 3] * inv);
                    }
                }
                if (row_ok && !direct)
                    a.wide_lse[pblk * 128 + r] = l_sum == 0.f ? -INFINITY : m_used + log2f(l_sum) - kLift;
                if (*odd_word() == (uint32_t)k + 1 && row_ok) {
                    // (from the first block that tile 0 cleaned: what lies before is in the products as it is)
                    const int edge0 = (a.mask != nullptr ? w.L : min(w.L + w.tok0 + 1, w.keys)) / BN;
                    const int32_t* table = a.c.block_table + (int64_t)w.b * a.c.max_pages;
                    if (!kWindow) {
                        add_odd<DT, false>(a.c, a.V, table, a.page_shift, kvh, max(max(w.blk0, edge0) * BN, w.L),
                                           min((w.blk0 + w.nblk) * BN, w.keys), limit, 0, 0, w.L, anc,
                                           direct ? orow : nullptr, direct ? nullptr : part);
                    } else {
                        for (int j = 0; j < w.nblk; ++j) {
                            const int kb = block_at(w.blk0 + j, w.gap) * BN;
                            const bool all = j < front;  // (cleaned from its first row on)
                            if (!all && j < edge0 - w.gap - w.blk0) continue;
                            add_odd<DT, true>(a.c, a.V, table, a.page_shift, kvh, all ? kb : max(kb, w.L),
                                              min(kb + BN, w.keys), limit, a.first, low, w.L, anc,
                                              direct ? orow : nullptr, direct ? nullptr : part);
                        }
                    }
                }
            }
            gv += nblk;
            ++q;
            n_two += two;
        }
        if (!ok && !aborted(abort_flag)) raise_abort(abort_flag, a.c.status);
    }
    // ---------------------------------------------------------------- teardown
    // (the products are complete when their last item is: the epilogue waited for it)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // All warps are through, so the flag is final.  (The producer may end with loads in flight that a warp which
    // gives up later never waits for: looked at before the barrier, the flag could still be down, and the CTA would
    // leave with its loads outstanding.)
    if (aborted(abort_flag)) {
        if (warp == 0 && lane == 0) {
            if (q_issued > 0) mbar_wait(bar(BAR_Q), (q_issued - 1) & 1, kDrainNs);
            for (int st = 0; st < SK; ++st) {
                const int n = (k_issued - st + SK - 1) / SK;
                if (n > 0) mbar_wait(bar(BAR_KF + st), (n - 1) & 1, kDrainNs);
            }
            for (int st = 0; st < SV; ++st) {
                const int n = (v_issued - st + SV - 1) / SV;
                if (n > 0) mbar_wait(bar(BAR_VF + st), (n - 1) & 1, kDrainNs);
            }
        }
        if (warp == 1 && lane == 0) {
            // (a commit and a barrier of their own: several phases of DONE may be pending, which one parity cannot
            // tell apart)
            mma_commit(bar(BAR_DRAIN));
            mbar_wait(bar(BAR_DRAIN), 0, kWaitNs);
        }
        __syncthreads();
    }
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Joins the key ranges of split row blocks: O = sum_c 2^(lse_c - lse) O_c.  A thread takes eight dims of a row, a
// warp 32 rows side by side (its reads are runs of 512 bytes, and each lane weighs its own row); a batch of
// ranges' reads is issued together.
constexpr int kBatch = 10;
template <int DT>
__device__ __forceinline__ void join_rows(const AttnArgs& a, const Group& gr, int part) {
    using E = Elem<DT>;
    // eight parts a tile, of two groups of eight dims each
    const int t = part >> 3, r = threadIdx.x & 127, c = (part & 7) * 2 + (threadIdx.x >> 7);
    const int T = a.shape.tile_tokens;
    const int tok = gr.tok0 + t * T + r / a.G;
    if (r / a.G >= T || tok >= gr.n || t >= gr.tiles) return;
    const int64_t blk = (int64_t)gr.part0 * 2 + t;
    const float* lse = a.wide_lse + blk * 128 + r;
    const float* po = a.wide_o + blk * 128 * HD + c * 1024 + r * 4;
    const int64_t step = (int64_t)gr.step * 2 * 128;
    float m = -INFINITY, l = 0.f;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int c0 = 0; c0 < gr.ranges; c0 += kBatch) {
        float lc[kBatch];
        float4 v[kBatch][2];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int x = c0 + u;
            lc[u] = -INFINITY;
            v[u][0] = v[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (x < gr.ranges) {
                lc[u] = lse[x * step];
                v[u][0] = *reinterpret_cast<const float4*>(po + x * step * HD);
                v[u][1] = *reinterpret_cast<const float4*>(po + x * step * HD + 512);
            }
        }
        float mb = m;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) mb = fmaxf(mb, lc[u]);
        const float base = mb == -INFINITY ? 0.f : mb;
        const float s = ex2(m - base);
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[x] *= s;
        l *= s;
        m = mb;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const float w = ex2(lc[u] - base);  // 0 for a range of which the row saw no key: its partial row is 0
            const float* f = &v[u][0].x;
#pragma unroll
            for (int x = 0; x < 8; ++x) acc[x] += w * f[x];
            l += w;
        }
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    typename E::T* dst =
        static_cast<typename E::T*>(a.O) + ((int64_t)(gr.q0 + tok) * a.Hq + gr.kvh * a.G + r % a.G) * HD + c * 8;
    *reinterpret_cast<uint4*>(dst) = make_uint4(E::down(acc[0] * inv, acc[1] * inv), E::down(acc[2] * inv, acc[3] * inv),
                                                E::down(acc[4] * inv, acc[5] * inv), E::down(acc[6] * inv, acc[7] * inv));
}

template <int DT>
__global__ void __launch_bounds__(256, 2)
join_kernel(const __grid_constant__ AttnArgs a) {
    // The next kernel may start now: it waits for this one, which waits for the attention's (15.9 -> 15.8 us a call
    // for one request's tree).
    griddep_launch_dependents();
    // The plan is read ahead of the grid wait: the kernels before this one are the attention's, of which the first let
    // the next start after its own wait, and so after the plan was written.  From L2, as a line of an older plan may
    // still lie in the SM's L1, and in one trip: the head's words, and the first task's row block at both places where
    // it can lie (15.9 -> 15.7 us, 40000 keys 45.2 -> 44.4).
    const Group* groups = reinterpret_cast<const Group*>(a.plan + a.shape.off_group);
    __shared__ int32_t s_words[32];
    static_assert(kHeadBytes <= 64 && sizeof(Group) == 32, "16 + 8 + 8 words");
    if (threadIdx.x < 32) {
        const int x = threadIdx.x, g = min((int)blockIdx.x / (x < 24 ? 8 : 16), a.shape.max_groups - 1);
        s_words[x] = __ldcg(x < 16 ? reinterpret_cast<const int32_t*>(a.plan) + x
                                   : reinterpret_cast<const int32_t*>(groups + g) + (x & 7));
    }
    __syncthreads();
    const PlanHead& head = *reinterpret_cast<const PlanHead*>(s_words);
    const int each = 8 * head.tiles, tasks = plan_fits(a, head) ? head.n_groups * each : 0;
    int task = blockIdx.x;
    Group gr = *reinterpret_cast<const Group*>(s_words + (head.tiles == 1 ? 16 : 24));
    griddep_wait();
    while (task < tasks) {
        join_rows<DT>(a, gr, task % each);
        task += gridDim.x;
        if (task < tasks) gr = groups[task / each];
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

bool encode(CUtensorMap* m, int dtype, int rank, const void* ptr, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
    auto enc = encoder();
    if (enc == nullptr) return false;
    cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return enc(m, dtype == GRAFT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
               const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DT, bool kWindow>
int launch(const AttnArgs& a, const Maps& m, cudaStream_t st) {
    static bool attr_set[64][2] = {};
    int dev = 0;
    if (!cuda_ok(cudaGetDevice(&dev))) return GRAFT_ERR_CUDA;
    const bool test_waits = a.wait_ns != kWaitNs;
    const auto kernel = test_waits ? wide_kernel<DT, true, kWindow> : wide_kernel<DT, false, kWindow>;
    if (dev < 0 || dev >= 64 || !attr_set[dev][test_waits]) {
        if (!cuda_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES)))
            return GRAFT_ERR_CUDA;
        if (dev >= 0 && dev < 64) attr_set[dev][test_waits] = true;
    }
    launch_pdl(kernel, dim3(a.shape.sms), dim3(NTHREADS), SMEM_BYTES, st, m, a);
    count_launches(1);
    return launch_status();
}

}  // namespace

int wide_launch(const AttnArgs& a, cudaStream_t st) {
    Maps m;
    const cuuint64_t es = 2;
    {
        // Q: (dim, head, new row)
        const cuuint64_t dims[3] = {HD, (cuuint64_t)a.Hq, (cuuint64_t)a.N};
        const cuuint64_t strides[2] = {HD * es, (cuuint64_t)a.q_stride * es};
        const cuuint32_t box[3] = {64, (cuuint32_t)a.G, (cuuint32_t)a.shape.tile_tokens};
        if (!encode(&m.q, a.c.dtype, 3, a.Q, dims, strides, box)) return GRAFT_ERR_CUDA;
    }
    {
        // pools: (dim of a half, row of a group, half, group, KV head)
        const cuuint64_t row = (cuuint64_t)a.c.Hkv * HD * es;
        const cuuint64_t dims[5] = {64, 8, 2, (cuuint64_t)a.c.num_pages * a.c.page_rows / 8, (cuuint64_t)a.c.Hkv};
        const cuuint64_t strides[4] = {row, 64 * es, 8 * row, HD * es};
        const cuuint32_t box[5] = {64, 8, 2, (cuuint32_t)(a.c.page_rows < BN ? a.c.page_rows : BN) / 8, 1};
        if (!encode(&m.k, a.c.dtype, 5, a.K, dims, strides, box)) return GRAFT_ERR_CUDA;
        if (!encode(&m.v, a.c.dtype, 5, a.V, dims, strides, box)) return GRAFT_ERR_CUDA;
    }
    if (a.window > 0) return a.c.dtype == GRAFT_BF16 ? launch<GRAFT_BF16, true>(a, m, st) : launch<GRAFT_FP16, true>(a, m, st);
    return a.c.dtype == GRAFT_BF16 ? launch<GRAFT_BF16, false>(a, m, st) : launch<GRAFT_FP16, false>(a, m, st);
}

int join_launch(const AttnArgs& a, cudaStream_t st) {
    const auto kernel = a.c.dtype == GRAFT_BF16 ? join_kernel<GRAFT_BF16> : join_kernel<GRAFT_FP16>;
    // (four CTAs an SM at most: where nothing turns out to be split they only come and go)
    const int tasks = 16 * a.shape.max_groups, most = 4 * a.shape.sms;
    launch_pdl(kernel, dim3(tasks < most ? tasks : most), dim3(256), 0, st, a);
    count_launches(1);
    return launch_status();
}

}  // namespace paged
}  // namespace graft
