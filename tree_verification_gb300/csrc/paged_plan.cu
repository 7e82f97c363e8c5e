// The attention plan of a paged cache's step, and the attention's entry points.
//
// The host knows a step's row count and the most rows of one sequence, not the
// lengths: those are on the device.  One CTA turns them into work items once
// a step, and every layer's attention reads its share from the plan, so no
// attention CTA searches or sorts.
#include "paged.cuh"

namespace graft {
namespace paged {
namespace {

constexpr int kPlanThreads = 1024;

template <class T>
__device__ __forceinline__ T scan_block(T v, T* s_warp, T* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        T w = s_warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    const T before = warp > 0 ? s_warp[warp - 1] : 0;
    *total = s_warp[31];
    __syncthreads();
    return before + x - v;
}

__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const __grid_constant__ GraftPagedCache c, int N, int Hq, const int32_t* __restrict__ q_start, int max_new,
            int tree, char* plan, PlanShape shape) {
    __shared__ int64_t s_warp[32];
    griddep_enter();
    const int tid = threadIdx.x, G = Hq / c.Hkv;
    Entry* few = reinterpret_cast<Entry*>(plan + shape.off_few);
    int64_t* prefix = reinterpret_cast<int64_t*>(plan + shape.off_prefix);
    Start* start = reinterpret_cast<Start*>(plan + shape.off_start);
    int n_few = 0;
    for (int b0 = 0; b0 < c.n_seqs; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int q0 = 0, n = 0, L = 0, count = 0;
        if (b < c.n_seqs) {
            q0 = q_start[b];
            const int64_t q1 = q_start[b + 1];
            L = c.lengths[b];
            const int64_t rows = q1 - q0;
            if (q0 < 0 || rows < 0 || q1 > N || rows > max_new || L < 0 ||
                (int64_t)L + rows > (int64_t)c.max_pages * c.page_rows) {
                flag_status(c.status, GRAFT_STATUS_LENGTH);
            } else {
                n = (int)rows;
                count = (n * G + shape.few_rows - 1) / shape.few_rows;
            }
        }
        int64_t total;
        int64_t at = n_few + scan_block<int64_t>(count, s_warp, &total);
        // (sequences that do not overlap have at most shape.max_few blocks; starts that do not rise could
        // claim more, and those are left out)
        for (int j = 0; j < count; ++j, ++at) {
            if (at >= shape.max_few) {
                flag_status(c.status, GRAFT_STATUS_LENGTH);
                break;
            }
            Entry e;
            e.b = b;
            e.q0 = q0;
            e.n = n;
            e.L = L;
            e.row0 = j * shape.few_rows;
            e.rows = min(n * G - e.row0, shape.few_rows);
            e.keys = tree ? L + n : L + (e.row0 + e.rows - 1) / G + 1;
            e.units = (e.keys + 15) / 16;
            few[at] = e;
        }
        n_few = (int)min((int64_t)shape.max_few, n_few + total);
    }
    __syncthreads();
    int64_t units = 0;
    for (int e0 = 0; e0 < n_few; e0 += kPlanThreads) {
        const int e = e0 + tid;
        int64_t total;
        const int64_t before = scan_block<int64_t>(e < n_few ? (int64_t)few[e].units * c.Hkv : 0, s_warp, &total);
        if (e < n_few) prefix[e] = units + before;
        units += total;
    }
    __syncthreads();
    // at least kMinUnits units a CTA: a CTA's own start and end cost more than the keys it would save another
    constexpr int64_t kMinUnits = 8;
    const int64_t want = (units + kMinUnits - 1) / kMinUnits;
    const int ctas = (int)(want < shape.ctas ? want : shape.ctas);
    for (int k = tid; k <= shape.ctas; k += kPlanThreads) {
        Start s{n_few, 0, 0, 0};
        if (k < ctas) {
            const int64_t u = first_unit(units, ctas, k);
            int lo = 0, hi = n_few;  // the entry with prefix[lo] <= u < prefix[lo + 1]
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (prefix[mid] <= u) lo = mid;
                else hi = mid;
            }
            const int64_t in = u - prefix[lo];
            s.entry = lo;
            s.head = (int)(in / few[lo].units);
            s.unit = (int)(in % few[lo].units);
        }
        start[k] = s;
    }
    if (tid == 0) {
        PlanHead h{};
        h.magic = kPlanMagic;
        h.N = N;
        h.Hq = Hq;
        h.Hkv = c.Hkv;
        h.n_seqs = c.n_seqs;
        h.max_new = max_new;
        h.tree = tree;
        h.page_rows = c.page_rows;
        h.max_pages = c.max_pages;
        h.num_pages = c.num_pages;
        h.few_rows = shape.few_rows;
        h.ctas = shape.ctas;
        h.n_few = n_few;
        h.few_ctas = ctas;
        h.few_units = units;
        *reinterpret_cast<PlanHead*>(plan) = h;
    }
}

int check_attention(const GraftPagedCache* c, int N, int Hq, int max_new) {
    const int rc = check_cache(c);
    if (rc != GRAFT_OK) return rc;
    if (N < 0 || Hq < 1 || max_new < 0 || Hq % c->Hkv != 0) return GRAFT_ERR_INVALID_ARG;
    if (Hq / c->Hkv > 64 || Hq > 8192) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    if ((int64_t)N * Hq >= (1LL << 31)) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    return GRAFT_OK;
}

FewWs carve_few(WsCarver& w, const GraftPagedCache* c, const PlanShape& s) {
    FewWs f;
    f.o = w.take<float>((size_t)s.ctas * 2 * kFewRows * HD);
    f.ml = w.take<float2>((size_t)s.ctas * 2 * kFewRows);
    f.count = w.take<int32_t>((size_t)s.max_few * c->Hkv);
    return f;
}

}  // namespace

PlanShape plan_shape(const GraftPagedCache* c, int N, int Hq, int max_new) {
    PlanShape s;
    const int G = Hq / c->Hkv;
    int sms = device_sm_count();
    if (sms <= 0) sms = 148;
    s.ctas = 2 * sms;
    s.few_rows = (int64_t)max_new * G <= 16 ? 16 : 32;
    // sequences with rows: at most n_seqs and at most N; each ends in at most one block that is not full
    const int64_t seqs = c->n_seqs < N ? c->n_seqs : N;
    s.max_few = (int)(((int64_t)N * G) / s.few_rows + seqs);
    s.off_few = align_up(sizeof(PlanHead), kWsAlign);
    s.off_prefix = align_up(s.off_few + sizeof(Entry) * (size_t)s.max_few, kWsAlign);
    s.off_start = align_up(s.off_prefix + sizeof(int64_t) * (size_t)s.max_few, kWsAlign);
    s.bytes = align_up(s.off_start + sizeof(Start) * (size_t)(s.ctas + 1), kWsAlign);
    return s;
}

}  // namespace paged
}  // namespace graft

using namespace graft;
using namespace graft::paged;

extern "C" int graft_paged_plan_size(const GraftPagedCache* cache, int N, int Hq, int max_new, size_t* bytes) {
    if (bytes == nullptr) return GRAFT_ERR_INVALID_ARG;
    const int rc = check_attention(cache, N, Hq, max_new);
    if (rc != GRAFT_OK) return rc;
    *bytes = plan_shape(cache, N, Hq, max_new).bytes;
    return GRAFT_OK;
}

extern "C" int graft_paged_plan(const GraftPagedCache* cache, int N, int Hq, const int32_t* q_start, int max_new,
                                int tree, void* plan, size_t plan_bytes, graft_stream_t stream) {
    const int rc = check_attention(cache, N, Hq, max_new);
    if (rc != GRAFT_OK) return rc;
    if (tree && max_new > GRAFT_MAX_KMAX) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    if (q_start == nullptr) return GRAFT_ERR_INVALID_ARG;
    const PlanShape s = plan_shape(cache, N, Hq, max_new);
    if (!ws_ok(plan, plan_bytes, s.bytes)) return GRAFT_ERR_WORKSPACE;
    launch_pdl(plan_kernel, dim3(1), dim3(kPlanThreads), 0, (cudaStream_t)stream, *cache, N, Hq, q_start, max_new,
               tree != 0 ? 1 : 0, static_cast<char*>(plan), s);
    count_launches(1);
    return launch_status();
}

extern "C" int graft_paged_attention_workspace_size(const GraftPagedCache* cache, int N, int Hq, int max_new,
                                                    size_t* bytes) {
    if (bytes == nullptr) return GRAFT_ERR_INVALID_ARG;
    const int rc = check_attention(cache, N, Hq, max_new);
    if (rc != GRAFT_OK) return rc;
    WsCarver w(nullptr);
    carve_few(w, cache, plan_shape(cache, N, Hq, max_new));
    *bytes = w.bytes();
    return GRAFT_OK;
}

extern "C" int graft_paged_attention(const GraftPagedCache* cache, const void* K_pool, const void* V_pool, int N,
                                     int Hq, int max_new, const void* plan, size_t plan_bytes, const void* Q,
                                     int64_t q_stride, const uint64_t* mask, float scale, void* O, void* ws,
                                     size_t ws_bytes, graft_stream_t stream) {
    const int rc = check_attention(cache, N, Hq, max_new);
    if (rc != GRAFT_OK) return rc;
    if (mask != nullptr && max_new > GRAFT_MAX_KMAX) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    if (N == 0) return GRAFT_OK;
    if (K_pool == nullptr || V_pool == nullptr || Q == nullptr || O == nullptr) return GRAFT_ERR_INVALID_ARG;
    if (!(aligned16(K_pool) && aligned16(V_pool) && aligned16(Q) && aligned16(O))) return GRAFT_ERR_INVALID_ARG;
    if (q_stride % 8 != 0 || q_stride < (int64_t)Hq * HD) return GRAFT_ERR_INVALID_ARG;
    if (!(scale > 0.f)) return GRAFT_ERR_INVALID_ARG;
    AttnArgs a{};
    a.shape = plan_shape(cache, N, Hq, max_new);
    if (!ws_ok(plan, plan_bytes, a.shape.bytes)) return GRAFT_ERR_WORKSPACE;
    WsCarver sizer(nullptr);
    carve_few(sizer, cache, a.shape);
    if (!ws_ok(ws, ws_bytes, sizer.bytes())) return GRAFT_ERR_WORKSPACE;
    WsCarver w(ws);
    a.few = carve_few(w, cache, a.shape);
    a.c = *cache;
    a.K = K_pool;
    a.V = V_pool;
    a.plan = static_cast<const char*>(plan);
    a.Q = Q;
    a.q_stride = q_stride;
    a.mask = mask;
    a.O = O;
    a.scale = scale;
    a.N = N;
    a.Hq = Hq;
    a.G = Hq / cache->Hkv;
    a.max_new = max_new;
    a.page_shift = log2_exact(cache->page_rows);
    return few_launch(a, (cudaStream_t)stream);
}
