// The attention plan of a paged cache's step, and the attention's entry points.
//
// The host knows a step's row count and the most rows of one sequence, not the
// lengths: those are on the device.  One CTA turns them into work items once
// a step, and every layer's attention reads its share from the plan, so no
// attention CTA searches or sorts.
#include <type_traits>

#include "paged.cuh"

namespace graft {
namespace paged {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 1024;  // of wide row blocks by their length
// (in blocks of a two-tile item's time, about 1.7 us)
constexpr int kItemCost = 2;           // an item's start and end
constexpr int kMinGain = 16;           // what splitting the last items costs: second pieces, partial rows, their join
constexpr int kSnap = 3;               // blocks of a piece at least
constexpr float kTileTime = 0.85f;     // a block of a single tile
constexpr float kPairCost = 2.f;       // twice the partial rows

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

// A length at which n items of `units` units in all make at most `slots` pieces: rounding up adds less than one a
// piece to units / length.
__device__ __forceinline__ int longest_piece(int64_t units, int n, int slots, int most) {
    if (slots <= n) return most;
    return (int)min((int64_t)most, (units + slots - n - 1) / (slots - n));
}

// Is a sequence's block of rows for the few kernel?
__device__ __forceinline__ bool is_few(const PlanShape& shape, int rows) {
    return rows > 0 && shape.few && (rows <= shape.few_rows || !shape.wide);
}

constexpr int kFewInSmem = 512;

template <bool kWindow, class ReadSeq>
__device__ __forceinline__ void plan_few(const GraftPagedCache& c, int Hq, int window, int first, char* plan,
                                         const PlanShape& shape, ReadSeq read_seq) {
    __shared__ int64_t s_warp[32];
    __shared__ Entry s_few[kFewInSmem];
    __shared__ int64_t s_prefix[kFewInSmem];
    __shared__ int s_units[kPlanThreads], s_most, s_fits[32];
    const int tid = threadIdx.x, G = Hq / c.Hkv;
    Entry* few = reinterpret_cast<Entry*>(plan + shape.off_few);
    int64_t* prefix = reinterpret_cast<int64_t*>(plan + shape.off_prefix);
    Start* start = reinterpret_cast<Start*>(plan + shape.off_start);
    int n_few = 0;
    int64_t units = 0;  // over entries and heads
    if (tid == 0) s_most = 1;
    for (int b0 = 0; b0 < c.n_seqs; b0 += kPlanThreads) {
        int q0, n, L;
        read_seq(b0 + tid, q0, n, L);
        const bool mine = is_few(shape, n * G);
        const int gap = kWindow ? window_gap(L - window + 1, first, 16) : 0;
        const Entry e{b0 + tid, q0, n, L, 0, n * G, L + n, (L + n + 15) / 16 - gap};
        int64_t total, all;
        const int at = n_few + (int)scan_block<int64_t>(mine, s_warp, &total);
        const int64_t before = units + scan_block<int64_t>(mine ? (int64_t)e.units * c.Hkv : 0, s_warp, &all);
        // (sequences that do not overlap number max_few at most; starts that do not rise could claim more)
        if (mine && at < shape.max_few) {
            few[at] = e;
            prefix[at] = before;
            if (at < kFewInSmem) {
                s_few[at] = e;
                s_prefix[at] = before;
            }
            atomicMax(&s_most, e.units);
        } else if (mine) {
            flag_status(c.status, GRAFT_STATUS_LENGTH);
        }
        n_few = (int)min((int64_t)shape.max_few, n_few + total);
        units += all;
    }
    __syncthreads();
    auto entry_at = [&](int i) { return i < kFewInSmem ? s_few[i] : few[i]; };
    auto prefix_at = [&](int i) { return i < kFewInSmem ? s_prefix[i] : prefix[i]; };
    // (without those left out, if any were)
    if (n_few > 0) units = prefix_at(n_few - 1) + (int64_t)entry_at(n_few - 1).units * c.Hkv;
    // Where every item can have CTAs of its own (items no more than CTAs), pieces of one length: a CTA that ends
    // one item and starts the next pays the latencies of both, about as long as kSwitch units take.  A unit a
    // warp at least.
    const int kSwitch = 5 * shape.few_warps / 2;
    int ctas = 0;
    bool own_ctas = false;
    if (units > 0 && n_few <= kFewInSmem && (int64_t)n_few * c.Hkv <= shape.ctas) {
        const int mine = tid < n_few ? s_few[tid].units : 0;
        // an SM's share left free for every item: the CTAs that join pieces hold theirs longest, and the next
        // call's CTAs find room elsewhere (decode of one sequence: 10.4 -> 9.0 us a call)
        // (not where the runs are long and every SM counts: 65536 keys, 49 against 51 us)
        int slots = shape.ctas / c.Hkv;
        const int64_t even = (units + shape.ctas - 1) / shape.ctas;
        if (n_few * 8 <= slots && even <= 8 * shape.few_warps) slots -= n_few;
        s_units[tid] = mine;
        __syncthreads();
        const int len = piece_length(s_units, n_few, slots, (int)max((int64_t)shape.few_warps, even),
                                     longest_piece(units / c.Hkv, n_few, slots, s_most), s_fits);
        int64_t items;
        const int first = (int)scan_block<int64_t>((mine + len - 1) / len, s_warp, &items);
        if (len <= even + kSwitch || len == shape.few_warps) {
            own_ctas = true;
            ctas = (int)items * c.Hkv;
            s_units[tid] = first;
            __syncthreads();
            for (int k = tid; k < ctas; k += kPlanThreads) {
                const int piece = k / c.Hkv;
                int lo = 0, hi = n_few;  // the entry with s_units[lo] <= piece < s_units[lo + 1]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (s_units[mid] <= piece) lo = mid;
                    else hi = mid;
                }
                Start s{};
                s.e = s_few[lo];
                s.entry = lo;
                s.head = k - piece * c.Hkv;
                s.pieces = (s.e.units + len - 1) / len;
                const int j = piece - s_units[lo], each = s.e.units / s.pieces, left = s.e.units % s.pieces;
                s.unit = each * j + min(j, left);
                s.count = each + (j < left);
                s.ctas = ctas;
                s.step = c.Hkv;
                s.cta0 = s_units[lo] * c.Hkv + s.head;
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
                if (prefix_at(mid) <= u) lo = mid;
                else hi = mid;
            }
            const int64_t in = u - prefix_at(lo);
            Start s{};
            s.e = entry_at(lo);
            s.entry = lo;
            s.head = (int)(in / s.e.units);
            s.unit = (int)(in % s.e.units);
            s.item_first = prefix_at(lo) + (int64_t)s.head * s.e.units;
            s.count = (int)(first_unit(units, ctas, k + 1) - u);
            s.ctas = ctas;
            s.total = units;
            start[k] = s;
        }
    }
    if (tid == 0) reinterpret_cast<PlanHead*>(plan)->few_ctas = ctas;
}

template <bool kWindow, class ReadSeq>
__device__ __forceinline__ void plan_wide(const GraftPagedCache& c, int N, int Hq, int tree, int window, int first,
                                          char* plan, const PlanShape& shape, ReadSeq read_seq) {
    __shared__ int64_t s_warp[32];
    __shared__ int s_hist[kBuckets], s_first[kPlanThreads], s_max, s_fits[32];
    const int tid = threadIdx.x, G = Hq / c.Hkv;
    Wide* pairs = reinterpret_cast<Wide*>(plan + shape.off_pairs);
    Wide* wide = reinterpret_cast<Wide*>(plan + shape.off_wide);
    Wide* last = reinterpret_cast<Wide*>(plan + shape.off_last);
    int32_t* where = reinterpret_cast<int32_t*>(plan + shape.off_where);
    Group* groups = reinterpret_cast<Group*>(plan + shape.off_group);
    const int pair = 2 * shape.tile_tokens;
    auto count_blocks = [&](Wide& w) {  // from its keys and first row
        w.gap = kWindow ? window_gap(w.L + (tree ? 0 : w.tok0) - window + 1, first, kBlockKeys) : 0;
        w.nblk = (w.keys + kBlockKeys - 1) / kBlockKeys - w.gap;
    };
    int n_pairs = 0;
    if (tid == 0) s_max = 1;
    for (int b0 = 0; b0 < c.n_seqs; b0 += kPlanThreads) {
        int q0, n, L;
        read_seq(b0 + tid, q0, n, L);
        const int count = is_few(shape, n * G) ? 0 : (n + pair - 1) / pair;
        int64_t total;
        int64_t at = n_pairs + scan_block<int64_t>(count, s_warp, &total);
        int most = 1;
        for (int j = 0; j < count; ++j, ++at) {
            if (at >= shape.max_pairs) {  // (as in plan_few)
                flag_status(c.status, GRAFT_STATUS_LENGTH);
                break;
            }
            Wide w{};
            w.b = b0 + tid;
            w.q0 = q0;
            w.n = n;
            w.L = L;
            w.tok0 = j * pair;
            w.two = n - w.tok0 > shape.tile_tokens;
            w.keys = tree ? L + n : L + min(w.tok0 + pair, n);
            count_blocks(w);
            w.part = -1;
            pairs[at] = w;
            most = max(most, w.nblk);
        }
        if (count > 0) atomicMax(&s_max, most);
        n_pairs = (int)min((int64_t)shape.max_pairs, n_pairs + total);
    }
    __syncthreads();
    const int P = shape.sms;
    int rounds = 0, n_groups = 0, most_tiles = 2;
    if (n_pairs == 0) {
        for (int k = tid; k <= P; k += kPlanThreads) where[k] = 0;
    } else if (shape.max_groups > 0 && n_pairs * c.Hkv * 3 <= P) {
        // ---- Three SMs an item or more: all are split by keys into ranges of about one length, one a CTA, so short that
        // they just fit (two blocks at least).  The row blocks may be cut into their single tiles for that: half the
        // partial rows, but a tile alone takes kTileTime of two tiles' time a block; the estimate decides (one
        // request's 64-node tree at group 4 over 4096 keys: 15.8 us in single tiles, 16.9 in pairs, over 40000 59 and
        // 45; 300 rows of a prompt over 6000: 76 and 40).
        const int slots = P / c.Hkv;
        auto block_of = [&](bool single, int e) {
            Wide w = pairs[single ? e >> 1 : e];
            const int t = single ? e & 1 : 0;
            if (t == 1 && !w.two) {
                w.nblk = 0;
            } else if (single) {
                w.tok0 += t * shape.tile_tokens;
                w.keys = tree ? w.L + w.n : w.L + min(w.tok0 + shape.tile_tokens, w.n);
                count_blocks(w);
                w.two = 0;
            }
            return w;
        };
        auto length_of = [&](bool single, int count, int64_t tiles) {
            s_first[tid] = tid < count ? block_of(single, tid).nblk : 0;
            int64_t blocks;
            scan_block<int64_t>(s_first[tid], s_warp, &blocks);
            return piece_length(s_first, count, slots, (int)max((int64_t)2, (blocks + slots - 1) / slots),
                                longest_piece(blocks, (int)tiles, slots, s_max), s_fits);
        };
        int64_t tiles;
        scan_block<int64_t>(tid < n_pairs ? 1 + pairs[tid].two : 0, s_warp, &tiles);
        int len = length_of(false, n_pairs, n_pairs);
        bool single = false;
        if (tiles <= slots) {
            const int alone = length_of(true, 2 * n_pairs, tiles);
            single = alone * kTileTime <= len + kPairCost;
            if (single) {
                len = alone;
                most_tiles = 1;
            }
        }
        const int n = single ? 2 * n_pairs : n_pairs;
        Wide w{};
        if (tid < n) w = block_of(single, tid);
        const int ranges = (w.nblk + len - 1) / len;
        // three sums in one: ranges, split blocks, their ranges
        int64_t sums;
        const int64_t mine3 =
            (int64_t)ranges | (int64_t)(ranges > 1) << 20 | (int64_t)(ranges > 1 ? ranges : 0) << 40;
        const int64_t before3 = scan_block<int64_t>(mine3, s_warp, &sums);
        const int first = (int)(before3 & 0xfffff), group = (int)(before3 >> 20 & 0xfffff), part = (int)(before3 >> 40);
        const int items = (int)(sums & 0xfffff) * c.Hkv;
        n_groups = (int)(sums >> 20 & 0xfffff) * c.Hkv;
        s_first[tid] = first;
        s_hist[tid] = part;
        if (ranges > 1)
            for (int h = 0; h < c.Hkv; ++h)
                groups[group * c.Hkv + h] =
                    Group{w.q0, w.n, w.tok0, 1 + w.two, h, ranges, part * c.Hkv + h, c.Hkv};
        __syncthreads();
        for (int k = tid; k < items; k += kPlanThreads) {
            const int r = k / c.Hkv;
            int lo = 0, hi = n;  // the block with s_first[lo] <= r < s_first[lo + 1]
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (s_first[mid] <= r) lo = mid;
                else hi = mid;
            }
            Wide x = block_of(single, lo);
            const int count = (x.nblk + len - 1) / len, j = r - s_first[lo];
            const int each = x.nblk / count, left = x.nblk % count;
            x.blk0 = each * j + min(j, left);
            x.nblk = each + (j < left);
            x.kvh = k - r * c.Hkv;
            x.part = count > 1 ? (s_hist[lo] + j) * c.Hkv + x.kvh : -1;
            last[k] = x;
        }
        for (int k = tid; k <= P; k += kPlanThreads) where[k] = min(k, items);
    } else {
        // ---- Items in the order of their blocks, the longest first, the heads of a row block side by side (their K
        // and V lie in the same pages).  The order decides what is split, so it is the same every time (equal
        // blocks by their place); past what one pass ranks nothing is split, and equal blocks may change places.
        const bool ranked = n_pairs <= kPlanThreads;
        auto put = [&](int at, Wide w) {
            for (int h = 0; h < c.Hkv; ++h) {
                w.kvh = h;
                wide[(int64_t)at * c.Hkv + h] = w;
            }
        };
        if (ranked) {
            s_first[tid] = tid < n_pairs ? pairs[tid].nblk : 0;
            __syncthreads();
            if (tid < n_pairs) {
                const int mine = s_first[tid];
                int rank = 0;
                for (int j = 0; j < n_pairs; ++j) rank += s_first[j] > mine || (s_first[j] == mine && j < tid);
                s_hist[rank] = mine;
                put(rank, pairs[tid]);
            }
        } else {
            const int64_t most = s_max;
            auto bucket = [&](int nblk) { return (int)(((most - nblk) * (kBuckets - 1)) / most); };
            s_hist[tid] = 0;
            __syncthreads();
            for (int e = tid; e < n_pairs; e += kPlanThreads) atomicAdd(&s_hist[bucket(pairs[e].nblk)], 1);
            __syncthreads();
            int64_t total;
            const int before = (int)scan_block<int64_t>(s_hist[tid], s_warp, &total);
            s_hist[tid] = before;
            __syncthreads();
            for (int e = tid; e < n_pairs; e += kPlanThreads) {
                const Wide w = pairs[e];
                put(atomicAdd(&s_hist[bucket(w.nblk)], 1), w);
            }
        }
        __syncthreads();
        const int n_items = n_pairs * c.Hkv;
        rounds = n_items / P;
        const int rem = n_items - rounds * P;  // < P
        const Wide* rest = wide + (int64_t)rounds * P;
        // ---- The items past the whole rounds: split over all CTAs where their even share is kMinGain blocks below
        // the longest (group 16 over 8192 keys: 10 trees, eight items past one round, 201 -> 123 us; 5 trees, 80
        // items, 102 -> 78; 8 trees, 128 items, 104 whole and 120 split).
        auto blocks_of = [&](int i) { return s_hist[i / c.Hkv]; };  // of item i (ranked)
        const int mine = ranked && tid < rem ? blocks_of(rounds * P + tid) : 0;
        int64_t blocks;
        const int before = (int)scan_block<int64_t>(mine, s_warp, &blocks);
        if (shape.max_groups > 0 && ranked && rem > 0 && blocks_of(rounds * P) >= blocks / P + kMinGain) {
            s_first[tid] = tid < rem ? before : (int)blocks;  // an item's place on the line of their blocks
            // what a CTA has done when the rounds end, an item's own cost included
            int load = 0;
            for (int k = 0; k < rounds && tid < P; ++k) load += blocks_of(k * P + ((k & 1) ? P - 1 - tid : tid)) + kItemCost;
            // the level that the rest fills every CTA up to (those above it take nothing)
            bool takes = tid < P;
            int64_t level = 0, sum;
            for (int it = 0; it < 2; ++it) {
                scan_block<int64_t>(takes ? (int64_t)load << 11 | 1 : 0, s_warp, &sum);
                level = ((sum >> 11) + blocks) / (sum & 2047);
                takes = takes && load <= level;
            }
            // (the shares' sum is off by rounding and by what dropped out last: the cuts are scaled to the blocks; the
            // share of a few blocks over a level floor would be none at all, so then they go to the first CTAs alone)
            int64_t share = takes ? level - load : 0;
            const int64_t both = scan_block<int64_t>(share << 11 | takes, s_warp, &sum);
            int64_t ahead = both >> 11, shares = sum >> 11;
            const int64_t takers = sum & 2047, few_takers = (blocks + kSnap - 1) / kSnap;
            if (few_takers < takers) {
                const int64_t rank = both & 2047;
                share = takes && rank < few_takers;
                ahead = min(rank, few_takers);
                shares = few_takers;
            }
            const int64_t from = ahead * blocks / shares, to = (ahead + share) * blocks / shares;
            auto item_of = [&](int x) {  // the item whose blocks hold x
                int lo = 0, hi = rem;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (s_first[mid] <= x) lo = mid;
                    else hi = mid;
                }
                return lo;
            };
            auto end_of = [&](int i) { return i + 1 < rem ? s_first[i + 1] : (int)blocks; };
            auto snap = [&](int64_t x) {  // a cut keeps kSnap blocks on both sides, or moves to the item's edge
                if (x >= blocks) return (int)blocks;
                const int i = item_of((int)x), s = s_first[i], e = end_of(i);
                return x - s < kSnap ? s : e - x < kSnap ? e : (int)x;
            };
            const int lo = tid < P ? snap(from) : (int)blocks;
            const int hi = tid == P - 1 ? (int)blocks : tid < P ? snap(to) : (int)blocks;
            int i0 = 0, pieces = 0, cuts = 0;
            bool head = false;  // the last piece starts an item that goes on in the next CTA
            if (lo < hi) {
                i0 = item_of(lo);
                const int i1 = item_of(hi - 1);
                pieces = i1 - i0 + 1;
                head = hi < end_of(i1) && s_first[i1] >= lo;
                cuts = (lo > s_first[i0] || hi < end_of(i0)) + (i1 > i0 && hi < end_of(i1));
            }
            __syncthreads();
            s_hist[tid] = lo < hi ? lo : -1;  // where a CTA's share starts
            int64_t total;
            const int64_t before3 = scan_block<int64_t>((int64_t)pieces | (int64_t)cuts << 20 | (int64_t)head << 40,
                                                        s_warp, &total);
            const int at = (int)(before3 & 0xfffff), group = (int)(before3 >> 40);
            int part = (int)(before3 >> 20 & 0xfffff);
            n_groups = (int)(total >> 40);
            if (tid < P) where[tid] = at;
            if (tid == 0) where[P] = (int)(total & 0xfffff);
            for (int j = 0; j < pieces; ++j) {
                const int i = i0 + j, s = s_first[i], e = end_of(i);
                const int p0 = max(lo, s), p1 = min(hi, e);
                Wide x = rest[i];
                x.blk0 = p0 - s;
                x.nblk = p1 - p0;
                const bool cut = p0 > s || p1 < e;
                if (cut && p0 == s) {
                    int ranges = 1;
                    for (int k = tid + 1; k < P && s_hist[k] < e; ++k) ranges += s_hist[k] >= 0;
                    groups[group] = Group{x.q0, x.n, x.tok0, 1 + x.two, x.kvh, ranges, part, 1};
                }
                x.part = cut ? part++ : -1;
                last[at + j] = x;
            }
        } else {
            // one of them a CTA, the longest to those that the snake served last
            if (tid < rem) last[(rounds & 1) ? rem - 1 - tid : tid] = rest[tid];
            for (int k = tid; k <= P; k += kPlanThreads)
                where[k] = (rounds & 1) ? min(max(k - (P - rem), 0), rem) : min(k, rem);
        }
    }
    if (tid == 0) {
        PlanHead& h = *reinterpret_cast<PlanHead*>(plan);
        h.rounds = rounds;
        h.n_groups = n_groups;
        h.tiles = most_tiles;
    }
}

// Block 0 plans the few entries, block 1 the wide items (a grid of one block has only the one kind).
template <bool kFew, bool kWide, bool kWindow>
__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const __grid_constant__ GraftPagedCache c, int N, int Hq, const int32_t* __restrict__ q_start, int max_new,
            int tree, int window, int first, char* plan, const __grid_constant__ PlanShape shape) {
    griddep_wait();
    const bool wide_block = kWide && (!kFew || blockIdx.x > 0);
    // Every block checks all sequences, the first one sets the status.
    auto read_seq = [&](int b, int& q0, int& n, int& L) {
        q0 = n = L = 0;
        if (b >= c.n_seqs || !takes_part(c, b)) return;
        const int64_t from = q_start[b], to = q_start[b + 1], len = c.lengths[b];
        const int64_t rows = to - from;
        if (from < 0 || rows < 0 || to > N || rows > max_new || len < 0 ||
            len + rows > (int64_t)c.max_pages * c.page_rows) {
            if (blockIdx.x == 0) flag_status(c.status, GRAFT_STATUS_LENGTH);
            return;
        }
        q0 = (int)from;
        n = (int)rows;
        L = (int)len;
    };
    if constexpr (kWide)
        if (wide_block) plan_wide<kWindow>(c, N, Hq, tree, window, first, plan, shape, read_seq);
    if constexpr (kFew)
        if (!wide_block) plan_few<kWindow>(c, Hq, window, first, plan, shape, read_seq);
    if (threadIdx.x == 0 && blockIdx.x == 0) {
        PlanHead& h = *reinterpret_cast<PlanHead*>(plan);
        h.magic = kPlanMagic;
        h.N = N;
        h.heads = plan_heads(Hq, c.Hkv);
        h.n_seqs = c.n_seqs;
        h.max_new = max_new;
        h.rows = plan_rows(shape.few_rows, c.page_rows, tree);
        h.max_pages = c.max_pages;
        h.num_pages = c.num_pages;
        h.ctas = shape.ctas;
        h.window = window;
        h.first = first;
    }
    // The attention reads the plan ahead of its grid wait, as a guess that is checked after it.  A CTA's first thread
    // to let it start does so for all, so a barrier comes before: every thread has made its writes, and the guess
    // holds (lengths rising by one a pass, 64 sequences: 0 of 222528 CTAs dropped it, 104511 without the barrier;
    // with a fence as well plan and attention of one sequence take 1.3 us longer).
    __syncthreads();
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

// Counters first, at a place and of a number that no argument changes: calls of other shapes and caches that share a
// workspace never write over them.  Then the partial rows.
void carve(WsCarver& w, const PlanShape& s, AttnArgs* a) {
    FewWs f;
    f.count = w.take<int32_t>((size_t)s.sms * 2);
    const size_t slots = (size_t)s.sms * 2 * 2;  // two a CTA, at most two CTAs an SM
    f.o = w.take<float>(slots * kFewRows * HD);
    f.ml = w.take<float2>(slots * kFewRows);
    const size_t parts = s.max_groups > 0 ? (size_t)s.sms * 2 : 0;  // a wave's cuts leave at most two pieces each
    float* wo = w.take<float>(parts * 2 * 128 * HD);
    float* wl = w.take<float>(parts * 2 * 128);
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
    const int64_t most_pairs = seqs * ((max_new - 1) / (2 * s.tile_tokens) + 1);
    s.max_pairs = s.wide ? (int)(full_pairs + seqs < most_pairs ? full_pairs + seqs : most_pairs) : 0;
    // Many rounds even themselves out; up to eight, what is left over may be split by keys.
    const int64_t full_items = (int64_t)full_pairs * c->Hkv, most_blocks = 2LL * s.max_pairs * c->Hkv;
    s.max_groups = s.wide && full_items < 8LL * sms ? (int)(most_blocks < sms ? most_blocks : sms) : 0;
    s.off_few = align_up(sizeof(PlanHead), kWsAlign);
    s.off_prefix = align_up(s.off_few + sizeof(Entry) * (size_t)s.max_few, kWsAlign);
    s.off_start = align_up(s.off_prefix + sizeof(int64_t) * (size_t)s.max_few, kWsAlign);
    s.off_pairs = align_up(s.off_start + sizeof(Start) * (size_t)s.ctas, kWsAlign);
    s.off_wide = align_up(s.off_pairs + sizeof(Wide) * (size_t)s.max_pairs, kWsAlign);
    s.off_last = align_up(s.off_wide + sizeof(Wide) * (size_t)s.max_pairs * c->Hkv, kWsAlign);
    s.off_where = align_up(s.off_last + (s.wide ? sizeof(Wide) * 2 * (size_t)sms : 0), kWsAlign);
    s.off_group = align_up(s.off_where + (s.wide ? sizeof(int32_t) * (size_t)(sms + 1) : 0), kWsAlign);
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

// window 0: none
static int plan_call(const GraftPagedCache* cache, int N, int Hq, const int32_t* q_start, int max_new, int tree, int window,
                     int first, void* plan, size_t plan_bytes, graft_stream_t stream) {
    const int rc = check_attention(cache, N, Hq, max_new);
    if (rc != GRAFT_OK) return rc;
    if (tree && max_new > GRAFT_MAX_KMAX) return GRAFT_ERR_UNSUPPORTED_SHAPE;
    if (q_start == nullptr) return GRAFT_ERR_INVALID_ARG;
    const PlanShape s = plan_shape(cache, N, Hq, max_new);
    if (!ws_ok(plan, plan_bytes, s.bytes)) return GRAFT_ERR_WORKSPACE;
    const auto pick = [&](auto win) {
        constexpr bool W = decltype(win)::value;
        return !s.wide ? plan_kernel<true, false, W> : s.few ? plan_kernel<true, true, W> : plan_kernel<false, true, W>;
    };
    const auto kernel = window > 0 ? pick(std::true_type{}) : pick(std::false_type{});
    launch_pdl(kernel, dim3(s.few && s.wide ? 2 : 1), dim3(kPlanThreads), 0, (cudaStream_t)stream, *cache, N, Hq,
               q_start, max_new, tree != 0 ? 1 : 0, window, first, static_cast<char*>(plan), s);
    count_launches(1);
    return launch_status();
}

extern "C" int graft_paged_plan(const GraftPagedCache* cache, int N, int Hq, const int32_t* q_start, int max_new,
                                int tree, void* plan, size_t plan_bytes, graft_stream_t stream) {
    return plan_call(cache, N, Hq, q_start, max_new, tree, 0, 0, plan, plan_bytes, stream);
}

extern "C" int graft_paged_plan_window(const GraftPagedCache* cache, int N, int Hq, const int32_t* q_start, int max_new,
                                       int tree, int window, int first, void* plan, size_t plan_bytes,
                                       graft_stream_t stream) {
    if (window < 1 || first < 0) return GRAFT_ERR_INVALID_ARG;
    return plan_call(cache, N, Hq, q_start, max_new, tree, window, first, plan, plan_bytes, stream);
}

extern "C" int graft_paged_attention_workspace_size(const GraftPagedCache* cache, int N, int Hq, int max_new,
                                                    size_t* bytes) {
    if (bytes == nullptr) return GRAFT_ERR_INVALID_ARG;
    const int rc = check_attention(cache, N, Hq, max_new);
    if (rc != GRAFT_OK) return rc;
    WsCarver w(nullptr);
    carve(w, plan_shape(cache, N, Hq, max_new), nullptr);
    *bytes = w.bytes();
    return GRAFT_OK;
}

extern "C" int graft_paged_attention(const GraftPagedCache* cache, const void* K_pool, const void* V_pool, int N,
                                     int Hq, int max_new, const void* plan, size_t plan_bytes, const void* Q,
                                     int64_t q_stride, const uint64_t* mask, float scale, void* O, void* ws,
                                     size_t ws_bytes, graft_stream_t stream) {
    return graft_paged_attention_ex(cache, K_pool, V_pool, N, Hq, max_new, plan, plan_bytes, Q, q_stride, mask, scale, O,
                                    nullptr, ws, ws_bytes, stream);
}

static int attention_call(const GraftPagedCache* cache, const void* K_pool, const void* V_pool, int N, int Hq, int max_new,
                          int window, int first, const void* plan, size_t plan_bytes, const void* Q, int64_t q_stride,
                          const uint64_t* mask, float scale, void* O, const GraftAttnTuning* tuning, void* ws,
                          size_t ws_bytes, graft_stream_t stream) {
    const int rc = check_attention(cache, N, Hq, max_new);
    if (rc != GRAFT_OK) return rc;
    if (tuning != nullptr) {
        if (tuning->tiles != 0 || tuning->min_chunk != 0 || tuning->persist_ctas != 0 || tuning->split != 0 ||
            tuning->wait_ns < 0)
            return GRAFT_ERR_INVALID_ARG;
        for (int r : tuning->reserved)
            if (r != 0) return GRAFT_ERR_INVALID_ARG;
    }
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
    carve(sizer, a.shape, nullptr);
    if (!ws_ok(ws, ws_bytes, sizer.bytes())) return GRAFT_ERR_WORKSPACE;
    WsCarver w(ws);
    carve(w, a.shape, &a);
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
    a.window = window;
    a.first = first;
    a.page_shift = log2_exact(cache->page_rows);
    a.wait_ns = tuning != nullptr && tuning->wait_ns > 0 ? (uint64_t)tuning->wait_ns : 500000000ull;
    cudaStream_t st = (cudaStream_t)stream;
    if (!a.shape.wide) return few_launch(a, st);
    // Steps of both kinds: the few kernel comes second and does not wait for the first, which has waited for all
    // that came before; its CTAs take the SMs that the wide items leave one by one.
    int rc2 = wide_launch(a, st);
    if (rc2 == GRAFT_OK && a.shape.few) {
        a.after_wide = 1;
        rc2 = few_launch(a, st);
    }
    if (rc2 == GRAFT_OK && a.shape.max_groups > 0) rc2 = join_launch(a, st);
    return rc2;
}

extern "C" int graft_paged_attention_ex(const GraftPagedCache* cache, const void* K_pool, const void* V_pool, int N,
                                        int Hq, int max_new, const void* plan, size_t plan_bytes, const void* Q,
                                        int64_t q_stride, const uint64_t* mask, float scale, void* O,
                                        const GraftAttnTuning* tuning, void* ws, size_t ws_bytes,
                                        graft_stream_t stream) {
    return attention_call(cache, K_pool, V_pool, N, Hq, max_new, 0, 0, plan, plan_bytes, Q, q_stride, mask, scale, O,
                          tuning, ws, ws_bytes, stream);
}

extern "C" int graft_paged_attention_window(const GraftPagedCache* cache, const void* K_pool, const void* V_pool, int N,
                                            int Hq, int max_new, int window, int first, const void* plan,
                                            size_t plan_bytes, const void* Q, int64_t q_stride, const uint64_t* mask,
                                            float scale, void* O, const GraftAttnTuning* tuning, void* ws,
                                            size_t ws_bytes, graft_stream_t stream) {
    if (window < 1 || first < 0) return GRAFT_ERR_INVALID_ARG;
    return attention_call(cache, K_pool, V_pool, N, Hq, max_new, window, first, plan, plan_bytes, Q, q_stride, mask,
                          scale, O, tuning, ws, ws_bytes, stream);
}
