// Rotary positions of Q and K, and the new K and V rows into their pages.
//
// Pair (x, y) of a head turns by a = position * w:
//   x' = f (x cos a - y sin a),  y' = f (x sin a + y cos a).
// Far positions: a's whole turns are dropped exactly.  w / 2 pi is held as a
// 64-bit fraction of a turn, W = round(w / 2 pi * 2^64); position * W modulo
// 2^64 is then the fraction of the turn itself (whole turns overflow away),
// off by at most |position| (2^-65 + 2^-52 w / 2 pi) turns, the second term
// the rounding of w / 2 pi: 2^-23 turns at position 2^31, as good as a 64-bit
// product.  Its upper 32 bits go to sincospi.  No 64-bit floating product a
// position.
//
// Memory bound: every element is read and written once.  A CTA takes one to
// three rows with all their heads, so a row's cosines are computed once
// and serve Hq + Hkv heads; each thread's loads (32 bytes a unit: the two
// 16-byte chunks whose dims pair up) are issued before the CTA looks up the
// sequences and pages, so the look-up's dependent reads run behind them; the
// page's number is read while the cosines are computed.
#include <climits>
#include <cmath>

#include "paged.cuh"

namespace graft {
namespace paged {
namespace {

constexpr int kThreads = 128;
constexpr int kTokens = 3;    // rows of a CTA at most
constexpr int kResident = 5;  // CTAs an SM holds at once
constexpr int kStep = kThreads / 8;  // heads that the CTA's threads hold at once

struct RopeArgs {
    GraftPagedCache c;
    uint4* K_pool;
    uint4* V_pool;
    const int32_t* q_start;
    const int32_t* pos;
    const double* inv_freq;
    const uint4* Q;
    const uint4* K;
    const uint4* V;
    uint4* Q_out;
    int64_t qs, ks, vs, qos;  // row strides in 16-byte chunks
    int N, Hq, rot, page_shift;
    int tokens;  // rows of a CTA
    bool inter;
    float factor;
};

struct Place {
    int b;      // sequence, -1: the row is no sequence's
    int first;  // its first new row
    int L;      // rows before them
    int held;   // pages that it holds (all, where the cache does not say)
};

// The sequence of a row, by a warp: 32 probes at a time until 32 sequences are left, whose starts, ends and
// lengths are read at once (up to 32 sequences: one read's latency).
__device__ __forceinline__ Place find_seq(const RopeArgs& a, int row) {
    const int lane = threadIdx.x & 31;
    int lo = 0, len = a.c.n_seqs;  // the last b with q_start[b] <= row lies in [lo, lo + len), or there is none
    while (len > 32) {
        const int step = (len + 31) / 32;
        const int at = lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, at < len && a.q_start[lo + at] <= row);
        const int hit = m == 0 ? 0 : 31 - __clz(m);
        lo += hit * step;
        len = min(step, len - hit * step);
    }
    int first = 0, end = 0, L = 0, held = INT_MAX;
    const bool have = lane < len;
    if (have) {
        first = a.q_start[lo + lane];
        end = a.q_start[lo + lane + 1];
        L = a.c.lengths[lo + lane];
        if (guarded(a.c)) held = a.c.held[lo + lane];
        if (!takes_part(a.c, lo + lane)) end = first;
    }
    const unsigned m = __ballot_sync(0xffffffffu, have && first <= row);
    const int hit = m == 0 ? 0 : 31 - __clz(m);
    Place p;
    p.first = __shfl_sync(0xffffffffu, first, hit);
    p.L = __shfl_sync(0xffffffffu, L, hit);
    p.held = __shfl_sync(0xffffffffu, held, hit);
    p.b = m != 0 && row < __shfl_sync(0xffffffffu, end, hit) ? lo + hit : -1;
    return p;
}

template <int DT>
__device__ __forceinline__ uint32_t turn2(uint32_t a, uint32_t& b, float2 cs0, float2 cs1) {
    using E = Elem<DT>;
    const float2 x = E::up(a), y = E::up(b);
    b = E::down(x.x * cs0.y + y.x * cs0.x, x.y * cs1.y + y.y * cs1.x);
    return E::down(x.x * cs0.x - y.x * cs0.y, x.y * cs1.x - y.y * cs1.y);
}
template <int DT>
__device__ __forceinline__ uint32_t turn1(uint32_t a, float2 cs) {
    using E = Elem<DT>;
    const float2 x = E::up(a);
    return E::down(x.x * cs.x - x.y * cs.y, x.x * cs.y + x.y * cs.x);
}

// kAhead: heads that a thread reads at a time, the first ones before the look-up
template <int DT, int kAhead>
__global__ void __launch_bounds__(kThreads, kResident)
rope_append_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ float2 s_cs[kTokens][HD / 2];
    __shared__ int64_t s_dst[kTokens];  // cache row in the pool, -1: not written
    __shared__ int s_live[kTokens], s_pos[kTokens];
    griddep_enter();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int t0 = blockIdx.x * a.tokens;
    const int nt = min(a.tokens, a.N - t0);
    const int heads = a.Hq + 2 * a.c.Hkv, turned = a.Hq + a.c.Hkv;
    const int rot_units = a.rot / 16;
    // A head is 8 units of two 16-byte chunks; a thread keeps its place i in the head and takes every kStep-th head,
    // so that a row's cosines come to its registers once.  The rotated units of the half layout pair chunk i with
    // chunk i + rot / 16.
    const int i = tid & 7, h_first = tid >> 3;
    const bool rotates = i < rot_units;
    const int c0 = rotates && !a.inter ? i : 2 * i, c1 = rotates && !a.inter ? i + rot_units : 2 * i + 1;
    uint4 buf[kAhead][2];
    auto fetch = [&](int t, int h0) {
        const int64_t row = t0 + t;
        const uint4* q = a.Q + row * a.qs;
        const uint4* k = a.K + row * a.ks - a.Hq * 16;
        const uint4* v = a.V + row * a.vs - turned * 16;
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const int h = h0 + x * kStep;
            if (h < heads) {
                const uint4* src = (h < a.Hq ? q : h < turned ? k : v) + h * 16;
                buf[x][0] = src[h < turned ? c0 : 2 * i];
                buf[x][1] = src[h < turned ? c1 : 2 * i + 1];
            }
        }
    };
    fetch(0, h_first);
    // one warp a row; what the cosines need first, the page behind them
    int page_at = -1;  // entry of the block table
    int64_t r = 0;
    if (warp < nt) {
        const int row = t0 + warp;
        const int given = a.pos != nullptr ? a.pos[row] : 0;
        const Place p = find_seq(a, row);
        r = (int64_t)p.L + ((int64_t)row - p.first);
        if (lane == 0) {
            s_live[warp] = p.b >= 0;
            s_pos[warp] = a.pos != nullptr ? given : (int)r;
            if (p.b >= 0) {
                if (p.L < 0 || p.first < 0 || (r >> a.page_shift) >= a.c.max_pages)
                    flag_status(a.c.status, GRAFT_STATUS_LENGTH);
                else if ((r >> a.page_shift) >= p.held)
                    flag_status(a.c.status, GRAFT_STATUS_PAGE);
                else
                    page_at = p.b * a.c.max_pages + (int)(r >> a.page_shift);
            }
        }
    }
    __syncthreads();
    const int page = page_at >= 0 ? a.c.block_table[page_at] : 0;
    const bool in_pool = page >= 0 && page < a.c.num_pages;
    // (a third dependent read, beside the cosines)
    const int refs = guarded(a.c) && page_at >= 0 && in_pool ? a.c.page_refs[page] : 1;
    // (the warps that look nothing up come first: a step of 32 layers over one request 721 -> 715 us, held pages checked)
    for (int x = tid ^ (kThreads / 2); x < nt * (a.rot / 2); x += kThreads) {
        const int t = (x >= a.rot / 2) + (x >= a.rot), p = x - t * (a.rot / 2);
        // 2^64 / 2 pi; a frequency of a turn or more per position keeps only its fraction
        const double turns = a.inv_freq[p] * 0.15915494309189533577;
        const uint64_t w = (uint64_t)__double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
        const uint64_t f = w * (uint64_t)(int64_t)s_pos[t];
        float s, c;
        sincospif((float)(int32_t)(f >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
        s_cs[t][p] = make_float2(c * a.factor, s * a.factor);
    }
    if (warp < nt && lane == 0) {
        const bool ours = in_pool && refs == 1;
        if (page_at >= 0 && !ours) flag_status(a.c.status, GRAFT_STATUS_PAGE);
        s_dst[warp] = page_at >= 0 && ours ? ((int64_t)page << a.page_shift) + (r & (a.c.page_rows - 1)) : -1;
    }
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
        if (!s_live[t]) {
            if (t + 1 < nt) fetch(t + 1, h_first);
            continue;
        }
        float4 cs[4];
        if (rotates) {
            const float4* s = reinterpret_cast<const float4*>(&s_cs[t][i * 8]);
#pragma unroll
            for (int k = 0; k < 4; ++k) cs[k] = s[k];
        }
        const int64_t dst = s_dst[t];
        uint4* q = a.Q_out + (int64_t)(t0 + t) * a.qos;
        uint4* k = a.K_pool + (dst * a.c.Hkv - a.Hq) * 16;
        uint4* v = a.V_pool + (dst * a.c.Hkv - turned) * 16;
        for (int h0 = h_first; h0 < heads; h0 += kAhead * kStep) {
            if (h0 > h_first) fetch(t, h0);
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const int h = h0 + x * kStep;
                if (h >= heads) continue;
                uint4 x0 = buf[x][0], x1 = buf[x][1];
                if (rotates && h < turned) {
                    uint32_t* w0 = &x0.x;
                    uint32_t* w1 = &x1.x;
                    if (a.inter) {
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            w0[2 * z] = turn1<DT>(w0[2 * z], make_float2(cs[z].x, cs[z].y));
                            w0[2 * z + 1] = turn1<DT>(w0[2 * z + 1], make_float2(cs[z].z, cs[z].w));
                            w1[2 * z] = turn1<DT>(w1[2 * z], make_float2(cs[z + 2].x, cs[z + 2].y));
                            w1[2 * z + 1] = turn1<DT>(w1[2 * z + 1], make_float2(cs[z + 2].z, cs[z + 2].w));
                        }
                    } else {
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            w0[z] = turn2<DT>(w0[z], w1[z], make_float2(cs[z].x, cs[z].y), make_float2(cs[z].z, cs[z].w));
                    }
                }
                if (h >= a.Hq && dst < 0) continue;
                uint4* to = (h < a.Hq ? q : h < turned ? k : v) + h * 16;
                to[h < turned ? c0 : 2 * i] = x0;
                to[h < turned ? c1 : 2 * i + 1] = x1;
            }
        }
        if (t + 1 < nt) fetch(t + 1, h_first);
    }
}

}  // namespace

int check_cache(const GraftPagedCache* c) {
    if (c == nullptr) return GRAFT_ERR_INVALID_ARG;
    if (c->dtype != GRAFT_BF16 && c->dtype != GRAFT_FP16) return GRAFT_ERR_INVALID_ARG;
    if (c->Hkv < 1 || c->num_pages < 1 || c->n_seqs < 1 || c->max_pages < 1 || c->n_layers < 0)
        return GRAFT_ERR_INVALID_ARG;
    if (c->head_dim != HD || c->Hkv > 1024) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    const int p = c->page_rows;
    if (p < 16 || p > GRAFT_MAX_PAGE_ROWS || (p & (p - 1)) != 0) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    if (c->n_seqs > GRAFT_MAX_SEQS || c->n_layers > 16384) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    if ((int64_t)c->num_pages * p >= (1LL << 31) || (int64_t)c->max_pages * p > (1LL << 30) ||
        (int64_t)c->n_seqs * c->max_pages >= (1LL << 31))
        return GRAFT_ERR_UNSUPPORTED_SHAPE;
    if (c->block_table == nullptr || c->lengths == nullptr) return GRAFT_ERR_INVALID_ARG;
    return GRAFT_OK;
}

int check_tables(const GraftPagedCache* c) {
    const int rc = check_cache(c);
    if (rc != GRAFT_OK) return rc;
    if (c->held == nullptr || c->page_refs == nullptr) return GRAFT_ERR_INVALID_ARG;
    return GRAFT_OK;
}

}  // namespace paged
}  // namespace graft

using namespace graft;
using namespace graft::paged;

extern "C" int graft_rope_inv_freq(int rot_dim, double base, int scaling, double stretch, double low, double high,
                                   double original, double* out, float* factor) {
    if (out == nullptr || rot_dim < 2 || rot_dim % 2 != 0 || !(base > 0.0) || !std::isfinite(base) || scaling < 0 ||
        scaling > 3)
        return GRAFT_ERR_INVALID_ARG;
    if (rot_dim > HD) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    if (scaling != 0 && (!(stretch > 0.0) || !std::isfinite(stretch))) return GRAFT_ERR_INVALID_ARG;
    if (scaling >= 2 && (!(low > 0.0) || !(high > low) || !(original > 0.0) || !std::isfinite(high) ||
                         !std::isfinite(original)))
        return GRAFT_ERR_INVALID_ARG;
    if (scaling == 3 && base == 1.0) return GRAFT_ERR_INVALID_ARG;  // every pair turns alike: no ramp
    const double two_pi = 6.283185307179586477;
    double ramp_low = 0, ramp_high = 1;
    if (scaling == 3) {
        // the pair index at which a pair turns r times in the original context
        auto at = [&](double r) { return rot_dim * std::log(original / (two_pi * r)) / (2 * std::log(base)); };
        ramp_low = std::fmax(std::floor(at(high)), 0.0);
        ramp_high = std::fmin(std::ceil(at(low)), (double)(rot_dim - 1));
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double w = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == 1) {
            w /= stretch;
        } else if (scaling == 2) {
            const double wave = two_pi / w;
            const double keep = std::fmin(std::fmax((original / wave - low) / (high - low), 0.0), 1.0);
            w = (1 - keep) * w / stretch + keep * w;
        } else if (scaling == 3) {
            const double ramp =
                std::fmin(std::fmax((i - ramp_low) / std::fmax(ramp_high - ramp_low, 1e-3), 0.0), 1.0);
            w = w * (1 - ramp) + w / stretch * ramp;
        }
        out[i] = w;
    }
    if (factor != nullptr) *factor = scaling == 3 ? (float)(0.1 * std::log(stretch) + 1.0) : 1.f;
    return GRAFT_OK;
}

extern "C" int graft_rope_append(const GraftPagedCache* cache, void* K_pool, void* V_pool, int N, int Hq,
                                 const int32_t* q_start, const int32_t* pos, const double* inv_freq, int rot_dim,
                                 int interleaved, float factor, const void* Q, int64_t q_stride, const void* K,
                                 int64_t k_stride, const void* V, int64_t v_stride, void* Q_out, int64_t qo_stride,
                                 graft_stream_t stream) {
    const int rc = check_cache(cache);
    if (rc != GRAFT_OK) return rc;
    if (N < 0 || Hq < 0) return GRAFT_ERR_INVALID_ARG;
    if (Hq > 8192) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    if (rot_dim < 0 || rot_dim > HD || rot_dim % 16 != 0) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    if (N == 0) return GRAFT_OK;
    if (q_start == nullptr || K == nullptr || V == nullptr || K_pool == nullptr || V_pool == nullptr)
        return GRAFT_ERR_INVALID_ARG;
    if (Hq > 0 && (Q == nullptr || Q_out == nullptr)) return GRAFT_ERR_INVALID_ARG;
    if (rot_dim > 0 && inv_freq == nullptr) return GRAFT_ERR_INVALID_ARG;
    if (!(aligned16(Q) && aligned16(K) && aligned16(V) && aligned16(Q_out) && aligned16(K_pool) && aligned16(V_pool)))
        return GRAFT_ERR_INVALID_ARG;
    if (k_stride % 8 != 0 || v_stride % 8 != 0 || k_stride < (int64_t)cache->Hkv * HD ||
        v_stride < (int64_t)cache->Hkv * HD)
        return GRAFT_ERR_INVALID_ARG;
    if (Hq > 0 && (q_stride % 8 != 0 || qo_stride % 8 != 0 || q_stride < (int64_t)Hq * HD || qo_stride < (int64_t)Hq * HD))
        return GRAFT_ERR_INVALID_ARG;
    RopeArgs a{};
    a.c = *cache;
    a.K_pool = static_cast<uint4*>(K_pool);
    a.V_pool = static_cast<uint4*>(V_pool);
    a.q_start = q_start;
    a.pos = pos;
    a.inv_freq = inv_freq;
    a.Q = static_cast<const uint4*>(Q);
    a.K = static_cast<const uint4*>(K);
    a.V = static_cast<const uint4*>(V);
    a.Q_out = static_cast<uint4*>(Q_out);
    a.qs = q_stride / 8;
    a.ks = k_stride / 8;
    a.vs = v_stride / 8;
    a.qos = qo_stride / 8;
    a.N = N;
    a.Hq = Hq;
    a.rot = rot_dim;
    a.page_shift = log2_exact(cache->page_rows);
    a.inter = interleaved != 0;
    a.factor = factor;
    // As few rows a CTA as make one wave of CTAs, up to three; else two, which share a look-up (48 heads, one, two,
    // three rows: 64 rows 6.2, 8.2 us; 704 rows 7.5, 8.2; 1280 rows 9.1, 9.9 with three; 1600 to 2240 rows, a wave of
    // three, 11.1 to 13.7, with two 11.8 to 15.0; 2304 rows, past it, 16.5 with three, 14.9 with two).
    const int64_t wave = (int64_t)kResident * device_sm_count();
    a.tokens = N <= wave ? 1 : N > 2 * wave && N <= 3 * wave ? 3 : 2;
    const dim3 grid((unsigned)((N + a.tokens - 1) / a.tokens));
    // (a row's heads in one go where three or five a thread do; 4096 rows of 48 heads: 21.4 us, 23.9 with five)
    const bool three = Hq + 2 * cache->Hkv <= 3 * kStep;
    const auto kernel = cache->dtype == GRAFT_BF16
                            ? (three ? rope_append_kernel<GRAFT_BF16, 3> : rope_append_kernel<GRAFT_BF16, 5>)
                            : (three ? rope_append_kernel<GRAFT_FP16, 3> : rope_append_kernel<GRAFT_FP16, 5>);
    launch_pdl(kernel, grid, dim3(kThreads), 0, (cudaStream_t)stream, a);
    count_launches(1);
    return launch_status();
}
