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
constexpr int kBuckets = 1024;  // of wide entries by their blocks

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

// The shortest piece length >= least at which the n items of s_units units, cut into such pieces, make at most
// `slots` pieces in all (at length `most`, the longest item's, they do): each warp tries one of 32 lengths.
__device__ __forceinline__ int piece_length(const int* s_units, int n, int slots, int least, int most, int* s_fits) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int lo = least, hi = max(most, least);
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        const int len = min(lo + warp * step, hi);
        int64_t items = 0;
        for (int i = lane; i < n; i += 32) items += (s_units[i] + len - 1) / len;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) items += __shfl_xor_sync(0xffffffffu, items, d);
        if (lane == 0) s_fits[warp] = items <= slots;
        __syncthreads();
        const unsigned m = __ballot_sync(0xffffffffu, s_fits[lane] != 0);
        __syncthreads();
        const int hit = m != 0 ? __ffs(m) - 1 : 32;  // the first length tried that fits
        hi = min(lo + hit * step, hi);
        lo = hit > 0 ? min(lo + (hit - 1) * step + 1, hi) : hi;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const __grid_constant__ GraftPagedCache c, int N, int Hq, const int32_t* __restrict__ q_start, int max_new,
            int tree, char* plan, PlanShape shape) {
    __shared__ int64_t s_warp[32];
    __shared__ int s_hist[kBuckets];
    __shared__ int s_first[kPlanThreads];  // units of the items, then their first pieces
    __shared__ int s_max, s_few_max, s_fits[32];
    griddep_wait();
    const int tid = threadIdx.x, G = Hq / c.Hkv;
    Entry* few = reinterpret_cast<Entry*>(plan + shape.off_few);
    int64_t* prefix = reinterpret_cast<int64_t*>(plan + shape.off_prefix);
    Start* start = reinterpret_cast<Start*>(plan + shape.off_start);
    Wide* pairs = reinterpret_cast<Wide*>(plan + shape.off_pairs);
    Wide* wide = reinterpret_cast<Wide*>(plan + shape.off_wide);
    Group* groups = reinterpret_cast<Group*>(plan + shape.off_group);
    const int pair = 2 * shape.tile_tokens;
    int n_few = 0, n_pairs = 0;
    if (tid == 0) s_max = 1;
    s_hist[tid] = 0;
    for (int b0 = 0; b0 < c.n_seqs; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int q0 = 0, n = 0, L = 0, count = 0, wcount = 0;
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
                if (n > 0 && shape.few && (n * G <= shape.few_rows || !shape.wide))
                    count = 1;
                else
                    wcount = (n + pair - 1) / pair;
            }
        }
        // (sequences that do not overlap have at most max_few and max_pairs blocks; starts that do not rise
        // could claim more, and those are left out)
        int64_t total;
        int64_t at = n_few + scan_block<int64_t>(count, s_warp, &total);
        if (count > 0) {
            if (at >= shape.max_few) {
                flag_status(c.status, GRAFT_STATUS_LENGTH);
            } else {
                Entry e;
                e.b = b;
                e.q0 = q0;
                e.n = n;
                e.L = L;
                e.row0 = 0;
                e.rows = n * G;
                e.keys = L + n;
                e.units = (e.keys + 15) / 16;
                few[at] = e;
            }
        }
        n_few = (int)min((int64_t)shape.max_few, n_few + total);
        if (!shape.wide) continue;
        at = n_pairs + scan_block<int64_t>(wcount, s_warp, &total);
        int most = 1;
        for (int j = 0; j < wcount; ++j, ++at) {
            if (at >= shape.max_pairs) {
                flag_status(c.status, GRAFT_STATUS_LENGTH);
                break;
            }
            Wide w{};
            w.b = b;
            w.q0 = q0;
            w.n = n;
            w.L = L;
            w.tok0 = j * pair;
            w.two = n - w.tok0 > shape.tile_tokens;
            w.keys = tree ? L + n : L + min(w.tok0 + pair, n);
            w.nblk = (w.keys + kBlockKeys - 1) / kBlockKeys;
            w.part = -1;
            pairs[at] = w;
            most = max(most, w.nblk);
        }
        if (wcount > 0) atomicMax(&s_max, most);
        n_pairs = (int)min((int64_t)shape.max_pairs, n_pairs + total);
    }
    __syncthreads();
    // ---- wide entries: split by keys where they would leave SMs without work, else sorted, longest first
    int n_wide = n_pairs, n_groups = 0;
    if (n_pairs > 0 && shape.max_groups > 0 && n_pairs * c.Hkv < shape.sms) {
        // Where single tiles would still fit one wave the items are single tiles: twice the key ranges' length, half
        // the partial rows (64-node tree at group 4 over 4096 keys: see the table of measurements).
        int64_t tiles;
        scan_block<int64_t>(tid < n_pairs ? 1 + pairs[tid].two : 0, s_warp, &tiles);
        const int slots = shape.sms / c.Hkv;
        const bool single = tiles <= slots;
        Wide w{};
        int mine = 0;
        const int e = single ? tid >> 1 : tid;
        if (e < n_pairs) {
            w = pairs[e];
            const int t = single ? tid & 1 : 0;
            if (t == 0 || w.two) {
                if (single) {
                    w.tok0 += t * shape.tile_tokens;
                    w.keys = tree ? w.L + w.n : w.L + min(w.tok0 + shape.tile_tokens, w.n);
                    w.nblk = (w.keys + kBlockKeys - 1) / kBlockKeys;
                    w.two = 0;
                }
                mine = w.nblk;
            }
        }
        int64_t blocks;
        scan_block<int64_t>(mine, s_warp, &blocks);
        // the shortest range (two blocks at least) at which the items fit one wave
        s_first[tid] = mine;
        __syncthreads();
        const int len = piece_length(s_first, single ? 2 * n_pairs : n_pairs, slots,
                                     (int)max((int64_t)2, (blocks + slots - 1) / slots), s_max, s_fits);
        int64_t items;
        const int64_t first = scan_block<int64_t>((mine + len - 1) / len, s_warp, &items);
        int64_t splits, split_parts;
        const int ranges = (mine + len - 1) / len;
        const int64_t group = scan_block<int64_t>(ranges > 1, s_warp, &splits);
        const int64_t part = scan_block<int64_t>(ranges > 1 ? ranges : 0, s_warp, &split_parts);
        if (ranges > 0) {
            const int nblk = w.nblk, each = nblk / ranges, left = nblk % ranges;
            if (ranges > 1)
                groups[group] = Group{w.q0, w.n, w.tok0, 1 + w.two, ranges, (int)part * c.Hkv, {0, 0}};
            for (int j = 0; j < ranges; ++j) {
                w.blk0 = each * j + min(j, left);
                w.nblk = each + (j < left);
                w.part = ranges > 1 ? (int)(part + j) * c.Hkv : -1;
                wide[first + j] = w;
            }
        }
        n_wide = (int)items;
        n_groups = (int)splits;
    } else if (n_pairs > 0) {
        const int64_t most = s_max;
        auto bucket = [&](int nblk) { return (int)(((most - nblk) * (kBuckets - 1)) / most); };
        for (int e = tid; e < n_pairs; e += kPlanThreads) atomicAdd(&s_hist[bucket(pairs[e].nblk)], 1);
        __syncthreads();
        int64_t total;
        const int before = (int)scan_block<int64_t>(s_hist[tid], s_warp, &total);
        s_hist[tid] = before;
        __syncthreads();
        for (int e = tid; e < n_pairs; e += kPlanThreads) {
            const Wide w = pairs[e];
            wide[atomicAdd(&s_hist[bucket(w.nblk)], 1)] = w;
        }
    }
    int64_t units = 0;
    if (tid == 0) s_few_max = 1;
    __syncthreads();
    for (int e0 = 0; e0 < n_few; e0 += kPlanThreads) {
        const int e = e0 + tid;
        int64_t total;
        const int64_t before = scan_block<int64_t>(e < n_few ? (int64_t)few[e].units * c.Hkv : 0, s_warp, &total);
        if (e < n_few) prefix[e] = units + before;
        if (e < n_few) atomicMax(&s_few_max, few[e].units);
        units += total;
    }
    __syncthreads();
    // Where every item can have CTAs of its own (items no more than CTAs), pieces of one length: a CTA that ends
    // one item and starts the next pays the latencies of both, about as long as kSwitch units take.  A unit a
    // warp at least.
    const int kSwitch = 5 * shape.few_warps / 2;
    int ctas = 0;
    bool own_ctas = false;
    if (units > 0 && (int64_t)n_few * c.Hkv <= shape.ctas) {
        const int mine = tid < n_few ? few[tid].units : 0;
        // an SM's share left free for every item: the CTAs that join pieces hold theirs longest, and the next
        // call's CTAs find room elsewhere (decode of one sequence: 10.4 -> 9.0 us a call)
        int slots = shape.ctas / c.Hkv;
        if (n_few * 8 <= slots) slots -= n_few;
        const int64_t even = (units + shape.ctas - 1) / shape.ctas;
        s_first[tid] = mine;
        __syncthreads();
        const int len = piece_length(s_first, n_few, slots, (int)max((int64_t)shape.few_warps, even), s_few_max, s_fits);
        int64_t items;
        const int64_t first = scan_block<int64_t>((mine + len - 1) / len, s_warp, &items);
        if (len <= even + kSwitch || len == shape.few_warps) {
            own_ctas = true;
            ctas = (int)items * c.Hkv;
            if (tid < n_few) s_first[tid] = (int)first;
            __syncthreads();
            for (int k = tid; k < ctas; k += kPlanThreads) {
                const int piece = k / c.Hkv;
                int lo = 0, hi = n_few;  // the entry with s_first[lo] <= piece < s_first[lo + 1]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (s_first[mid] <= piece) lo = mid;
                    else hi = mid;
                }
                Start s{};
                s.e = few[lo];
                s.entry = lo;
                s.head = k - piece * c.Hkv;
                s.pieces = (s.e.units + len - 1) / len;
                const int j = piece - s_first[lo], each = s.e.units / s.pieces, left = s.e.units % s.pieces;
                s.unit = each * j + min(j, left);
                s.count = each + (j < left);
                s.ctas = ctas;
                s.step = c.Hkv;
                s.cta0 = s_first[lo] * c.Hkv + s.head;
                start[k] = s;
            }
        }
    }
    if (!own_ctas) {
        const int64_t want = (units + shape.few_warps - 1) / shape.few_warps;
        ctas = (int)(want < shape.ctas ? want : shape.ctas);
        for (int k = tid; k < ctas; k += kPlanThreads) {
            const int64_t u = first_unit(units, ctas, k);
            int lo = 0, hi = n_few;  // the entry with prefix[lo] <= u < prefix[lo + 1]
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (prefix[mid] <= u) lo = mid;
                else hi = mid;
            }
            const int64_t in = u - prefix[lo];
            Start s{};
            s.e = few[lo];
            s.entry = lo;
            s.head = (int)(in / s.e.units);
            s.unit = (int)(in % s.e.units);
            s.item_first = prefix[lo] + (int64_t)s.head * s.e.units;
            s.count = (int)(first_unit(units, ctas, k + 1) - u);
            s.ctas = ctas;
            s.total = units;
            start[k] = s;
        }
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
        h.n_wide = n_wide;
        h.n_groups = n_groups;
        *reinterpret_cast<PlanHead*>(plan) = h;
    }
    // the attention reads the plan ahead of its grid wait, as a guess that is checked after it: it starts when the
    // plan is written, so that the guess holds
    __threadfence();
    griddep_launch_dependents();
}

int check_attention(const GraftPagedCache* c, int N, int Hq, int max_new) {
    const int rc = check_cache(c);
    if (rc != GRAFT_OK) return rc;
    if (N < 0 || Hq < 1 || max_new < 0 || Hq % c->Hkv != 0) return GRAFT_ERR_INVALID_ARG;
    if (Hq / c->Hkv > 64 || Hq > 8192) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    if ((int64_t)N * Hq >= (1LL << 31)) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    return GRAFT_OK;
}

// Partial rows first, in sizes of the device's alone, then the counters (see FewWs).  Split row blocks have at
// most one range a slot of the wave, and one more a block.
void carve(WsCarver& w, const GraftPagedCache* c, const PlanShape& s, AttnArgs* a) {
    FewWs f;
    const size_t slots = (size_t)s.sms * 2 * 2;  // two a CTA, at most two CTAs an SM
    f.o = w.take<float>(slots * kFewRows * HD);
    f.ml = w.take<float2>(slots * kFewRows);
    const size_t parts = (size_t)s.sms * 2;
    float* wo = w.take<float>(parts * 2 * 128 * HD);
    float* wl = w.take<float>(parts * 2 * 128);
    f.count = w.take<int32_t>((size_t)s.max_few * c->Hkv);
    if (a != nullptr) {
        a->few = f;
        a->wide_o = wo;
        a->wide_lse = wl;
    }
}

}  // namespace

PlanShape plan_shape(const GraftPagedCache* c, int N, int Hq, int max_new) {
    PlanShape s;
    const int G = Hq / c->Hkv;
    int sms = device_sm_count();
    if (sms <= 0) sms = 148;
    s.sms = sms;
    s.few_rows = (int64_t)max_new * G <= 16 ? 16 : 32;
    // Up to 32 query rows the few kernel reads K and V at HBM speed; past that its products take longer than
    // the bytes.  A step whose rows are all taken by full sequences (N = n_seqs x max_new) has no short ones.
    s.wide = (int64_t)max_new * G > kFewRows;
    s.few = !s.wide || (int64_t)N < (int64_t)c->n_seqs * max_new;
    s.tile_tokens = 128 / G;
    // sequences with rows: at most n_seqs and at most N; each ends in at most one block that is not full
    const int64_t seqs = c->n_seqs < N ? c->n_seqs : N;
    s.max_few = s.few ? (int)seqs : 0;
    // Many items: two CTAs of four warps an SM, so that one streams while the other joins its warps and starts
    // anew.  Few: one of eight, whose runs are twice as long and cut an item into half as many pieces.
    s.few_warps = seqs * c->Hkv >= 2 * sms ? 4 : 8;
    s.ctas = sms * 8 / s.few_warps;
    const int full_pairs = N / (2 * s.tile_tokens);
    s.max_pairs = s.wide ? (int)(full_pairs + seqs) : 0;
    // where even the full row blocks fill the SMs nothing is split
    const bool split = s.wide && (int64_t)full_pairs * c->Hkv < sms;
    s.max_wide = s.max_pairs + (split ? sms / c->Hkv : 0);
    s.max_groups = split ? (2 * s.max_pairs < sms / c->Hkv ? 2 * s.max_pairs : sms / c->Hkv) : 0;
    s.off_few = align_up(sizeof(PlanHead), kWsAlign);
    s.off_prefix = align_up(s.off_few + sizeof(Entry) * (size_t)s.max_few, kWsAlign);
    s.off_start = align_up(s.off_prefix + sizeof(int64_t) * (size_t)s.max_few, kWsAlign);
    s.off_pairs = align_up(s.off_start + sizeof(Start) * (size_t)s.ctas, kWsAlign);
    s.off_wide = align_up(s.off_pairs + sizeof(Wide) * (size_t)s.max_pairs, kWsAlign);
    s.off_group = align_up(s.off_wide + sizeof(Wide) * (size_t)s.max_wide, kWsAlign);
    s.bytes = align_up(s.off_group + sizeof(Group) * (size_t)s.max_groups, kWsAlign);
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
    carve(w, cache, plan_shape(cache, N, Hq, max_new), nullptr);
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
    if ((reinterpret_cast<uintptr_t>(O) & 31) != 0) return GRAFT_ERR_INVALID_ARG;  // rows leave in 32-byte pieces
    if (!(scale > 0.f)) return GRAFT_ERR_INVALID_ARG;
    AttnArgs a{};
    a.shape = plan_shape(cache, N, Hq, max_new);
    if (!ws_ok(plan, plan_bytes, a.shape.bytes)) return GRAFT_ERR_WORKSPACE;
    WsCarver sizer(nullptr);
    carve(sizer, cache, a.shape, nullptr);
    if (!ws_ok(ws, ws_bytes, sizer.bytes())) return GRAFT_ERR_WORKSPACE;
    WsCarver w(ws);
    carve(w, cache, a.shape, &a);
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
    if (a.shape.few) {
        const int rc2 = few_launch(a, (cudaStream_t)stream);
        if (rc2 != GRAFT_OK) return rc2;
    }
    return a.shape.wide ? wide_launch(a, (cudaStream_t)stream) : GRAFT_OK;
}
