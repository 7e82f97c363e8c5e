// Pages of a cache: accepted rows compacted, pages reserved (copy on write), forked and freed.
//
// All state is on the device (block table, lengths, held counts, reference
// counts), so a captured step can run them; nothing depends on the order in
// which threads arrive.  A free page is one with no references, and the
// lowest free ones are taken first: the result is a function of the state
// alone, with no free list whose order would carry the history.
#include "paged.cuh"

namespace graft {
namespace paged {
namespace {

// ---------------------------------------------------------------- compaction
// A CTA takes one sequence in every G-th layer, two layers at a time, so that
// the look-up (two dependent reads) is paid once for both.  A thread owns 16-byte
// columns of a row; it moves rows in rising order, kBatch loads (in two
// layers) before their stores: the path rises strictly, so path[t] >= t, and
// a row is overwritten only after every move that reads it has read it (moves
// never read below their own t).
constexpr int kMoveThreads = 256;
constexpr int kBatch = 3;

// Where move t of sequence b reads and writes (rows of the pool), or the status bits that forbid it.
__device__ __forceinline__ int find_move(const GraftPagedCache& c, int Kmax, int p, int before, int L, int b, int t,
                                         int page_shift, int64_t* src, int64_t* dst) {
    if (p <= before || p >= Kmax) return GRAFT_STATUS_TREE;
    const int64_t from = (int64_t)L + p, to = (int64_t)L + t;
    if ((from >> page_shift) >= c.max_pages) return GRAFT_STATUS_LENGTH;
    const int32_t* row = c.block_table + (int64_t)b * c.max_pages;
    const int ps = row[from >> page_shift], pd = row[to >> page_shift];
    if (ps < 0 || ps >= c.num_pages || pd < 0 || pd >= c.num_pages) return GRAFT_STATUS_PAGE;
    if (guarded(c) && ((from >> page_shift) >= c.held[b] || c.page_refs[ps] != 1 || c.page_refs[pd] != 1))
        return GRAFT_STATUS_PAGE;
    *src = ((int64_t)ps << page_shift) + (from & (c.page_rows - 1));
    *dst = ((int64_t)pd << page_shift) + (to & (c.page_rows - 1));
    return 0;
}

__global__ void __launch_bounds__(kMoveThreads)
compact_rows_kernel(const __grid_constant__ GraftPagedCache c, int Kmax, const int32_t* __restrict__ path,
                    const int32_t* __restrict__ acc_len, int32_t* lengths_out, int page_shift) {
    __shared__ int64_t s_src[GRAFT_MAX_KMAX], s_dst[GRAFT_MAX_KMAX];
    griddep_enter();
    const int b = blockIdx.y, t = threadIdx.x;
    const int per = c.Hkv * (HD / 8);  // 16-byte columns of a row
    // everything that depends on nothing is read at once: the path, the lengths, the first pools
    int p = 0, before = -1;
    if (t < Kmax) {
        p = path[(int64_t)b * Kmax + t];
        if (t > 0) before = path[(int64_t)b * Kmax + t - 1];
    }
    const int L = c.lengths[b], given = acc_len[b];
    const bool idle = !takes_part(c, b);
    const int n = idle ? 0 : given;
    auto pool_of = [&](int l, int x) -> uint4* {
        return l < c.n_layers && x < 2 * per ? static_cast<uint4*>((x < per ? c.K_layers : c.V_layers)[l]) : nullptr;
    };
    const int G = gridDim.x;
    uint4* pool0 = pool_of(blockIdx.x, t);
    uint4* pool1 = pool_of(blockIdx.x + G, t);
    int bad = (n < 0 || n > Kmax) ? GRAFT_STATUS_TREE : L < 0 && !idle ? GRAFT_STATUS_LENGTH : 0;
    if (!bad && t < n) bad = find_move(c, Kmax, p, before, L, b, t, page_shift, &s_src[t], &s_dst[t]);
    if (bad && blockIdx.x == 0) flag_status(c.status, bad);
    const int stop = __syncthreads_or(bad);
    if (blockIdx.x == 0 && t == 0 && lengths_out != nullptr) lengths_out[b] = stop ? L : L + n;
    if (stop) return;
    // moves that stay where they are (the root's, and those of a path that starts 0, 1, ...) come first
    int first = 0;
    while (first < n && s_src[first] == s_dst[first]) ++first;
    // a thread's column in two layers at a time
    for (int x = t; x < 2 * per; x += kMoveThreads) {
        const int col = x < per ? x : x - per;
        for (int l = blockIdx.x; l < c.n_layers; l += 2 * G) {
            for (int t0 = first; t0 < n; t0 += kBatch) {
                uint4 v[2][kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    if (t0 + k < n) {
                        v[0][k] = pool0[s_src[t0 + k] * per + col];
                        if (pool1 != nullptr) v[1][k] = pool1[s_src[t0 + k] * per + col];
                    }
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    if (t0 + k < n) {
                        pool0[s_dst[t0 + k] * per + col] = v[0][k];
                        if (pool1 != nullptr) pool1[s_dst[t0 + k] * per + col] = v[1][k];
                    }
            }
            const int next_l = l + 2 * G < c.n_layers ? l + 2 * G : (int)blockIdx.x;
            const int next_x = l + 2 * G < c.n_layers ? x : x + kMoveThreads;
            pool0 = pool_of(next_l, next_x);
            pool1 = pool_of(next_l + G, next_x);
        }
    }
}

// Lengths advanced in place: a launch of its own, after every CTA of the moves has read them.
__global__ void __launch_bounds__(GRAFT_MAX_KMAX)
compact_lengths_kernel(const __grid_constant__ GraftPagedCache c, int Kmax, const int32_t* __restrict__ path,
                       const int32_t* __restrict__ acc_len, int page_shift) {
    griddep_enter();
    const int b = blockIdx.x, t = threadIdx.x;
    const int L = c.lengths[b], n = takes_part(c, b) ? acc_len[b] : 0;
    int64_t src, dst;
    bool bad = n < 0 || n > Kmax || L < 0;
    if (!bad && t < n) {
        const int before = t > 0 ? path[(int64_t)b * Kmax + t - 1] : -1;
        bad = find_move(c, Kmax, path[(int64_t)b * Kmax + t], before, L, b, t, page_shift, &src, &dst) != 0;
    }
    if (!__syncthreads_or(bad) && t == 0) c.lengths[b] = L + n;
}

// ---------------------------------------------------------------- free, fork
__global__ void __launch_bounds__(256)
free_kernel(const __grid_constant__ GraftPagedCache c, int n, const int32_t* __restrict__ seqs) {
    griddep_enter();
    const int i = blockIdx.x, b = seqs[i];
    int bad = b < 0 || b >= c.n_seqs;
    for (int j = threadIdx.x; j < i; j += blockDim.x) bad |= seqs[j] == b;
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) flag_status(c.status, GRAFT_STATUS_SEQUENCE);
        return;
    }
    const int held = min(max(c.held[b], 0), c.max_pages);
    int32_t* row = c.block_table + (int64_t)b * c.max_pages;
    for (int k = threadIdx.x; k < c.max_pages; k += blockDim.x) {
        if (k < held) {
            const int p = row[k];
            if (p < 0 || p >= c.num_pages) {
                flag_status(c.status, GRAFT_STATUS_PAGE);
            } else if (atomicSub(c.page_refs + p, 1) <= 0) {
                atomicAdd(c.page_refs + p, 1);  // held by nobody: the count stays
                flag_status(c.status, GRAFT_STATUS_PAGE);
            }
        }
        row[k] = -1;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        c.held[b] = 0;
        c.lengths[b] = 0;
    }
}

__global__ void __launch_bounds__(256)
fork_kernel(const __grid_constant__ GraftPagedCache c, int n, const int32_t* __restrict__ src_seq,
            const int32_t* __restrict__ dst_seq, int page_shift) {
    griddep_enter();
    const int i = blockIdx.x, src = src_seq[i], dst = dst_seq[i];
    int bad = src < 0 || src >= c.n_seqs || dst < 0 || dst >= c.n_seqs;
    for (int j = threadIdx.x; j < n; j += blockDim.x) bad |= dst_seq[j] == src || (j < i && dst_seq[j] == dst);
    bad = __syncthreads_or(bad);
    // (no other fork writes src; another of the same dst has left this one out)
    if (!bad) bad = c.held[dst] != 0 || c.lengths[dst] != 0;
    if (bad) {
        if (threadIdx.x == 0) flag_status(c.status, GRAFT_STATUS_SEQUENCE);
        return;
    }
    const int L = c.lengths[src];
    const int64_t count = L < 0 ? -1 : ((int64_t)L + c.page_rows - 1) >> page_shift;
    if (count < 0 || count > c.held[src] || count > c.max_pages) {
        if (threadIdx.x == 0) flag_status(c.status, GRAFT_STATUS_LENGTH);
        return;
    }
    const int32_t* from = c.block_table + (int64_t)src * c.max_pages;
    int32_t* to = c.block_table + (int64_t)dst * c.max_pages;
    bad = 0;
    for (int k = threadIdx.x; k < count; k += blockDim.x) bad |= from[k] < 0 || from[k] >= c.num_pages;
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) flag_status(c.status, GRAFT_STATUS_PAGE);
        return;
    }
    for (int k = threadIdx.x; k < c.max_pages; k += blockDim.x) {
        const int p = k < count ? from[k] : -1;
        if (p >= 0) atomicAdd(c.page_refs + p, 1);
        to[k] = p;
    }
    if (threadIdx.x == 0) {
        c.held[dst] = (int)count;
        c.lengths[dst] = L;
    }
}

// ---------------------------------------------------------------- reserve
// A sequence's new rows start inside a page that it holds: the one page whose rows may have to be copied.
struct Tail {
    int32_t src, dst, rows, pad;  // rows 0: nothing to copy
};

struct ReserveWs {
    Tail* tail;      // [n_seqs]
    int32_t* fresh;  // [num_pages] the free pages that are handed out, lowest first
    int32_t* old;    // [num_pages] the page that fresh page i replaces, -1: none
};

constexpr int kPlanThreads = 1024;

// Exclusive prefix sum over the block; *total receives the sum.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = s_warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    const int before = warp > 0 ? s_warp[warp - 1] : 0;
    *total = s_warp[31];
    __syncthreads();
    return before + x - v;
}

// One CTA.  Demands are counted and summed in the order of the sequences,
// the lowest free pages found (in tiles of the reference counts, until the
// demand is met) and handed out; the replaced pages' references fall last,
// so that "shared" means the same to every sequence of the call.  Latency
// bound: what depends on nothing is read at once (a thread's sequence and its
// share of the first tile), and the pages found first stay in shared memory.
// The search is linear in the pages held below the free ones: one page each
// for 64 sequences of a pool nine tenths full takes 4.3 us with 4096 pages,
// 7.1 with 16384, 17.7 with 65536.
constexpr int kTile = kPlanThreads * 4;
constexpr int kFreshInSmem = 2048;
__global__ void __launch_bounds__(kPlanThreads, 1)
reserve_kernel(const __grid_constant__ GraftPagedCache c, const int32_t* __restrict__ new_rows, ReserveWs w,
               int page_shift) {
    __shared__ int s_warp[32];
    __shared__ int s_first[GRAFT_MAX_SEQS], s_need[GRAFT_MAX_SEQS];  // rank of the first new page, their number
    __shared__ int s_fresh[kFreshInSmem];
    griddep_enter();
    const int tid = threadIdx.x;
    auto read_tile = [&](int p0) {  // which of this thread's four pages are free, as bits
        int bits = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int p = p0 + tid * 4 + k;
            bits |= (p < c.num_pages && c.page_refs[p] == 0) << k;
        }
        return bits;
    };
    int free = read_tile(0);
    int demand = 0;
    for (int b0 = 0; b0 < c.n_seqs; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int need = 0, bad = 0;
        const bool mine = b < c.n_seqs;
        const int rows = mine && takes_part(c, b) ? new_rows[b] : 0, held = mine ? c.held[b] : 0;
        const int64_t L = mine ? c.lengths[b] : 0;
        if (rows != 0) {
            const int64_t pages = (L + rows + c.page_rows - 1) >> page_shift;
            const int64_t first = L >> page_shift;
            if (L < 0 || rows < 0 || held < 0 || pages > c.max_pages || held > c.max_pages || held < first) {
                bad = GRAFT_STATUS_LENGTH;
            } else {
                const int32_t* row = c.block_table + (int64_t)b * c.max_pages;
                need = max((int)pages - held, 0);
                for (int k = (int)first; k < min(held, (int)pages); ++k) {
                    const int p = row[k];
                    const int refs = p >= 0 && p < c.num_pages ? c.page_refs[p] : 0;
                    if (refs < 1) bad = GRAFT_STATUS_PAGE;
                    need += refs > 1;
                }
            }
            if (bad) {
                flag_status(c.status, bad);
                need = 0;
            }
        }
        int total;
        const int before = block_scan(need, s_warp, &total);
        if (mine) {
            s_first[b] = demand + before;
            s_need[b] = bad ? -1 : need;
        }
        demand += total;
    }
    int found = 0;
    for (int p0 = 0; p0 < c.num_pages && found < demand; p0 += kTile) {
        if (p0 > 0) free = read_tile(p0);
        int total;
        int at = found + block_scan(__popc(free), s_warp, &total);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (free >> k & 1) {
                if (at < kFreshInSmem)
                    s_fresh[at] = p0 + tid * 4 + k;
                else
                    w.fresh[at] = p0 + tid * 4 + k;
                w.old[at] = -1;
                ++at;
            }
        found += total;
    }
    __syncthreads();
    for (int b = tid; b < c.n_seqs; b += kPlanThreads) {
        Tail tail{0, 0, 0, 0};
        const int rows = takes_part(c, b) ? new_rows[b] : 0;
        if (rows > 0 && s_need[b] >= 0) {
            const int64_t L = c.lengths[b];
            const int held = c.held[b], pages = (int)((L + rows + c.page_rows - 1) >> page_shift);
            const int first = (int)(L >> page_shift);
            int32_t* row = c.block_table + (int64_t)b * c.max_pages;
            int at = s_first[b];
            if (at + s_need[b] > found) {
                flag_status(c.status, GRAFT_STATUS_CACHE_OVERFLOW);
            } else {
                for (int k = first; k < pages; ++k) {
                    const int old = k < held ? row[k] : -1;
                    if (old >= 0 && c.page_refs[old] <= 1) continue;
                    const int p = at < kFreshInSmem ? s_fresh[at] : w.fresh[at];
                    w.old[at++] = old;
                    c.page_refs[p] = 1;
                    row[k] = p;
                    if (old >= 0 && k == first) tail = Tail{old, p, (int)(L & (c.page_rows - 1)), 0};
                }
                if (pages > held) c.held[b] = pages;
            }
        }
        w.tail[b] = tail;
    }
    __syncthreads();
    for (int i = tid; i < min(found, demand); i += kPlanThreads)
        if (w.old[i] >= 0) atomicSub(c.page_refs + w.old[i], 1);
}

// Rows of the replaced last pages, every layer: a CTA copies up to kCopyRows rows of K or V of one sequence.  (CTAs
// that took several layers each, the next one's rows read before this one's were written, were slower: 30 against
// 26 us for a turnover of 48 samples in 36 layers.)
constexpr int kCopyRows = 16;
constexpr int kCopyThreads = 256;
constexpr int kCopyBatch = 8;
__global__ void __launch_bounds__(kCopyThreads)
copy_tails_kernel(const __grid_constant__ GraftPagedCache c, const Tail* __restrict__ tails, int pieces,
                  int page_shift) {
    griddep_enter();
    const int b = blockIdx.x / pieces, r0 = (blockIdx.x - b * pieces) * kCopyRows;
    uint4* pool = static_cast<uint4*>(((blockIdx.y & 1) ? c.V_layers : c.K_layers)[blockIdx.y >> 1]);
    const Tail tail = tails[b];
    const int rows = min(tail.rows - r0, kCopyRows);
    if (rows <= 0) return;
    const int per = c.Hkv * (HD / 8);
    const uint4* from = pool + (((int64_t)tail.src << page_shift) + r0) * per;
    uint4* to = pool + (((int64_t)tail.dst << page_shift) + r0) * per;
    const int n = rows * per;  // rows of a page lie side by side
    for (int x = threadIdx.x; x < n; x += kCopyThreads * kCopyBatch) {
        uint4 v[kCopyBatch];
#pragma unroll
        for (int k = 0; k < kCopyBatch; ++k)
            if (x + k * kCopyThreads < n) v[k] = from[x + k * kCopyThreads];
#pragma unroll
        for (int k = 0; k < kCopyBatch; ++k)
            if (x + k * kCopyThreads < n) to[x + k * kCopyThreads] = v[k];
    }
}

ReserveWs carve_reserve(WsCarver& c, const GraftPagedCache* cache) {
    ReserveWs w;
    w.tail = c.take<Tail>(cache->n_seqs);
    w.fresh = c.take<int32_t>(cache->num_pages);
    w.old = c.take<int32_t>(cache->num_pages);
    return w;
}

}  // namespace
}  // namespace paged
}  // namespace graft

using namespace graft;
using namespace graft::paged;

extern "C" int graft_pages_compact(const GraftPagedCache* cache, int Kmax, const int32_t* path, const int32_t* acc_len,
                                   int32_t* lengths_out, graft_stream_t stream) {
    const int rc = check_cache(cache);
    if (rc != GRAFT_OK) return rc;
    if (Kmax < 1 || path == nullptr || acc_len == nullptr || lengths_out == nullptr) return GRAFT_ERR_INVALID_ARG;
    if (Kmax > GRAFT_MAX_KMAX) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    if (cache->n_layers > 0 && (cache->K_layers == nullptr || cache->V_layers == nullptr)) return GRAFT_ERR_INVALID_ARG;
    const int shift = log2_exact(cache->page_rows);
    const bool in_place = lengths_out == cache->lengths;
    cudaStream_t st = (cudaStream_t)stream;
    // CTAs a sequence: one a layer where they all fit the GPU at once, else one for two layers (64 sequences in 36
    // layers: 10.2 us; 11.4 when it was chosen, one a layer then 15.5, one for six layers 12.6)
    const int n_layers = cache->n_layers > 0 ? cache->n_layers : 1;
    const int G = (int64_t)n_layers * cache->n_seqs <= 4LL * device_sm_count() ? n_layers : (n_layers + 1) / 2;
    launch_pdl(compact_rows_kernel, dim3(G, cache->n_seqs), dim3(kMoveThreads), 0, st, *cache, Kmax, path, acc_len,
               in_place ? nullptr : lengths_out, shift);
    count_launches(1);
    if (in_place) {
        launch_pdl(compact_lengths_kernel, dim3(cache->n_seqs), dim3(GRAFT_MAX_KMAX), 0, st, *cache, Kmax, path,
                   acc_len, shift);
        count_launches(1);
    }
    return launch_status();
}

extern "C" int graft_pages_reserve_workspace_size(const GraftPagedCache* cache, size_t* bytes) {
    if (bytes == nullptr) return GRAFT_ERR_INVALID_ARG;
    const int rc = check_tables(cache);
    if (rc != GRAFT_OK) return rc;
    WsCarver c(nullptr);
    carve_reserve(c, cache);
    *bytes = c.bytes();
    return GRAFT_OK;
}

extern "C" int graft_pages_reserve(const GraftPagedCache* cache, const int32_t* new_rows, void* ws, size_t ws_bytes,
                                   graft_stream_t stream) {
    const int rc = check_tables(cache);
    if (rc != GRAFT_OK) return rc;
    if (new_rows == nullptr) return GRAFT_ERR_INVALID_ARG;
    if (cache->n_layers > 0 && (cache->K_layers == nullptr || cache->V_layers == nullptr)) return GRAFT_ERR_INVALID_ARG;
    WsCarver sizer(nullptr);
    carve_reserve(sizer, cache);
    if (!ws_ok(ws, ws_bytes, sizer.bytes())) return GRAFT_ERR_WORKSPACE;
    WsCarver c(ws);
    const ReserveWs w = carve_reserve(c, cache);
    const int shift = log2_exact(cache->page_rows);
    cudaStream_t st = (cudaStream_t)stream;
    launch_pdl(reserve_kernel, dim3(1), dim3(kPlanThreads), 0, st, *cache, new_rows, w, shift);
    count_launches(1);
    if (cache->n_layers > 0) {
        const int pieces = (cache->page_rows + kCopyRows - 1) / kCopyRows;
        launch_pdl(copy_tails_kernel, dim3(cache->n_seqs * pieces, cache->n_layers * 2), dim3(kCopyThreads), 0, st,
                   *cache, static_cast<const Tail*>(w.tail), pieces, shift);
        count_launches(1);
    }
    return launch_status();
}

extern "C" int graft_pages_fork(const GraftPagedCache* cache, int n, const int32_t* src, const int32_t* dst,
                                graft_stream_t stream) {
    const int rc = check_tables(cache);
    if (rc != GRAFT_OK) return rc;
    if (n < 0) return GRAFT_ERR_INVALID_ARG;
    if (n > GRAFT_MAX_SEQS) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    if (n == 0) return GRAFT_OK;
    if (src == nullptr || dst == nullptr) return GRAFT_ERR_INVALID_ARG;
    launch_pdl(fork_kernel, dim3(n), dim3(256), 0, (cudaStream_t)stream, *cache, n, src, dst,
               log2_exact(cache->page_rows));
    count_launches(1);
    return launch_status();
}

extern "C" int graft_pages_free(const GraftPagedCache* cache, int n, const int32_t* seqs, graft_stream_t stream) {
    const int rc = check_tables(cache);
    if (rc != GRAFT_OK) return rc;
    if (n < 0) return GRAFT_ERR_INVALID_ARG;
    if (n > GRAFT_MAX_SEQS) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    if (n == 0) return GRAFT_OK;
    if (seqs == nullptr) return GRAFT_ERR_INVALID_ARG;
    launch_pdl(free_kernel, dim3(n), dim3(256), 0, (cudaStream_t)stream, *cache, n, seqs);
    count_launches(1);
    return launch_status();
}
