// sz_evict.cu -- eviction from the 4-bit cache by accumulated attention
// weight, in place.
//
// Each (sequence, kv head) keeps the `keep` tokens that come first in the
// order: protected (position >= next position - recent), then larger weight,
// then lower slot.  The i-th evicted slot below `keep` (a hole) receives the
// i-th surviving token from `keep` on, so that only those tokens move: an
// attention does not depend on the order of its tokens, and their positions
// travel with them.  Sources and targets are disjoint, so the moves need no
// order among themselves.
//
// First kernel, one cluster of blocks per (sequence, kv head): weights as
// 32-bit keys whose unsigned order is theirs, held in registers (warp after
// warp takes a contiguous run of slots), a radix selection of the keep-th
// largest (11, 11 and 10 bits), then three passes in slot order: ties that
// survive, holes and movers are counted, then numbered.  The blocks of a
// cluster join their histograms and counts through each other's shared
// memory.  Second kernel: the moves, eight lanes each.  Both are bound by
// latency: 8 bytes a slot are read, and few tokens move (8 sequences of 32,768
// tokens, 4 heads, cut by a page: 14 us for the selection, 4 us for the moves,
// against 1.3 us for their bytes).
#include <type_traits>

#include "sz_cache.cuh"
#include "sz_params.h"

namespace sz {
namespace {

constexpr uint32_t kThreads = 1024;
constexpr uint32_t kWarps = kThreads / 32;
constexpr uint32_t kMaxCluster = 8;
constexpr uint32_t kBins = 2048;
constexpr uint32_t kCopies = 4;  // of the first histogram: keys of neighbouring lanes often share a bin
constexpr uint32_t kProtected = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// All threads of the cluster; shared memory written before is seen after.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Two words of this block's shared memory (8-byte aligned) as block `rank` of
// the cluster holds them.
__device__ __forceinline__ uint2 peer_pair(const uint32_t* p, uint32_t rank) {
    uint32_t a;
    uint2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

// Their sums over the cluster's n blocks, with the loads under way together;
// `before`, if given: over the first `rank` of them.
__device__ __forceinline__ uint2 peer_sums(const uint32_t* p, uint32_t n, uint32_t rank = 0, uint2* before = nullptr) {
    uint2 v[kMaxCluster], sum{0, 0};
#pragma unroll
    for (uint32_t r = 0; r < kMaxCluster; r++) v[r] = r < n ? peer_pair(p, r) : uint2{0, 0};
#pragma unroll
    for (uint32_t r = 0; r < kMaxCluster; r++) {
        if (before && r == rank) *before = sum;
        sum.x += v[r].x, sum.y += v[r].y;
    }
    return sum;
}

// Unsigned order of the key = order of the weight; NaN counts as -infinity,
// -0 as 0.  At most 0xFF800000 (+infinity), so protected tokens come first.
__device__ __forceinline__ uint32_t key_of(float w) {
    if (w != w) w = -__builtin_huge_valf();
    const uint32_t b = __float_as_uint(w + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct Slots {
    const EvictParams& p;
    uint32_t b, h;
    __device__ __forceinline__ bool find(uint32_t slot, uint64_t& at) const {
        const int32_t page = p.table[(uint64_t)b * p.table_width + (slot >> p.pool.lg_page)];
        if ((uint32_t)page >= p.pool.pages) return false;
        at = (((uint64_t)(uint32_t)page * p.pool.heads + h) << p.pool.lg_page) + (slot & ((1u << p.pool.lg_page) - 1u));
        return true;
    }
    // Keys of slots i0, i0 + 32, ... below `to`; 0 past it.  only_safe: there
    // are at least `keep` protected tokens, which compete by weight, and no
    // other stays (key 0).  All loads of a kind are under way together.
    template <int N>
    __device__ __forceinline__ void keys(uint32_t i0, uint32_t to, int64_t safe_from, bool only_safe, uint32_t* out) const {
        uint64_t at[N];
        int32_t page[N], pos[N];
        float weight[N];
        bool bad = false;
        const int32_t* row = p.table + (uint64_t)b * p.table_width;
#pragma unroll
        for (int j = 0; j < N; j++) page[j] = i0 + 32 * j < to ? row[(i0 + 32 * j) >> p.pool.lg_page] : 0;
#pragma unroll
        for (int j = 0; j < N; j++) {
            const bool ok = (uint32_t)page[j] < p.pool.pages;
            bad |= !ok;
            at[j] = (((uint64_t)(ok ? (uint32_t)page[j] : 0u) * p.pool.heads + h) << p.pool.lg_page) +
                    ((i0 + 32 * j) & ((1u << p.pool.lg_page) - 1u));
        }
#pragma unroll
        for (int j = 0; j < N; j++) pos[j] = p.pos[at[j]];
#pragma unroll
        for (int j = 0; j < N; j++) weight[j] = p.weight[at[j]];
#pragma unroll
        for (int j = 0; j < N; j++) {
            const bool safe = (int64_t)pos[j] >= safe_from;
            const uint32_t k = safe == only_safe ? key_of(weight[j]) : safe ? kProtected : 0u;
            out[j] = i0 + 32 * j < to && (uint32_t)page[j] < p.pool.pages ? k : 0u;
        }
        if (bad && p.status) atomicMax(p.status, kStatusInvalid);
    }
};

// KEYS: keys that a thread holds, 32 * KEYS to a warp; 0: more than fit, read
// again for every pass.
template <int KEYS>
__global__ void __launch_bounds__(kThreads, 1) evict_select_kernel(const EvictParams p) {
    __shared__ alignas(8) uint32_t s_bins[kCopies * kBins];
    __shared__ uint32_t s_count[2][kWarps];
    __shared__ alignas(8) uint32_t s_sum[2][2];  // of the block: ties; holes and movers
    __shared__ alignas(8) uint32_t s_safe[2];    // the block's protected tokens (and 0)
    __shared__ uint32_t s_pick[3];  // a bin, how many of its keys survive, how many it has
    wait_for_previous();
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    const uint32_t rank = cluster_rank(), blocks = cluster_size();
    const Slots slots{p, blockIdx.z, blockIdx.y};
    const uint32_t list = blockIdx.z * p.pool.heads + blockIdx.y;
    const int32_t len = p.lens[slots.b], next_pos = p.next_pos[slots.b];
    const bool ok = len >= 0 && (uint64_t)len <= (uint64_t)p.table_width << p.pool.lg_page;
    const uint32_t n = ok ? (uint32_t)len : 0u;
    if (tid == 0 && rank == 0) {
        if (!ok && p.status) atomicMax(p.status, kStatusInvalid);
        if (blockIdx.y == 0) p.new_lens[slots.b] = (int32_t)min(n, p.keep);
        if (n <= p.keep) p.moves[list] = 0;
    }
    if (n <= p.keep) return;  // the whole cluster
    const int64_t safe_from = (int64_t)next_pos - (int64_t)p.recent;

    // This warp's slots [from, to), in order of block and warp.
    const uint32_t runs = blocks * kWarps;
    const uint32_t run = ((n + runs - 1) / runs + 31u) & ~31u;
    const uint64_t first = (uint64_t)(rank * kWarps + warp) * run;
    const uint32_t from = (uint32_t)min(first, (uint64_t)n), to = (uint32_t)min(first + run, (uint64_t)n);
    uint32_t keys[KEYS ? KEYS : 1];
    bool only_safe = false;
    auto load_keys = [&]() {
        if constexpr (KEYS > 0) {
            constexpr int kBatch = KEYS < 8 ? KEYS : 8;
#pragma unroll
            for (int j = 0; j < KEYS; j += kBatch)
                slots.keys<kBatch>(from + 32 * j + lane, to, safe_from, only_safe, keys + j);
        }
    };
    // Calls f(slot, key, whether there is such a slot) for the warp's slots in
    // order, 32 at a time, by whole warps.
    auto each = [&](auto f) {
        if constexpr (KEYS > 0) {
#pragma unroll
            for (int j = 0; j < KEYS; j++) {
                const uint32_t i0 = from + 32 * j;
                if (i0 < to) f(i0 + lane, keys[j], i0 + lane < to);
            }
        } else {
            for (uint32_t i0 = from; i0 < to; i0 += 32) {
                uint32_t k;
                slots.keys<1>(i0 + lane, to, safe_from, only_safe, &k);
                f(i0 + lane, k, i0 + lane < to);
            }
        }
    };
    // Turns two counts per warp into what the warps and blocks before this one
    // have; returns the first's sum over the cluster.  k: a place of s_sum of
    // its own.
    auto place = [&](uint32_t& x, uint32_t& y, int k) {
        if (lane == 0) s_count[0][warp] = x, s_count[1][warp] = y;
        __syncthreads();
        const uint32_t cx = s_count[0][lane], cy = s_count[1][lane];
        x = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? cx : 0u);
        y = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? cy : 0u);
        uint32_t all_x = __reduce_add_sync(0xFFFFFFFFu, cx), all_y = __reduce_add_sync(0xFFFFFFFFu, cy);
        if (blocks == 1) {
            __syncthreads();  // s_count is written again by the next call
            return all_x;
        }
        if (tid == 0) s_sum[k][0] = all_x, s_sum[k][1] = all_y;
        cluster_sync();
        uint2 before{0, 0};
        all_x = peer_sums(s_sum[k], blocks, rank, &before).x;
        x += before.x, y += before.y;
        return all_x;
    };

    // ---- the threshold: `need` of the tokens whose key equals it survive ----
    // Each level has bins of its own, so that none are cleared while another
    // block reads them: levels 1 and 2 take the first one's spare copies.
    load_keys();
    uint32_t apart = kProtected;  // keys that do not compete
    uint32_t threshold = 0, need = 0;
    uint32_t fixed = 0;  // mask of the bits chosen so far
    bool all_pass = false;
    for (int level = 0; level < 3 && !all_pass; level++) {
        const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
        const uint32_t width = level == 2 ? 1024 : 2048;
        uint32_t* own = s_bins + level * kBins;
        for (uint32_t i = tid; i < (level == 0 ? kCopies : 1) * kBins; i += kThreads) own[i] = 0;
        if (level == 0 && tid < 2) s_safe[tid] = 0;
        __syncthreads();
        uint32_t* bins = own + (level == 0 ? lane % kCopies * kBins : 0);
        uint32_t safe = 0;
        // N keys of a lane, 32 slots apart.  A warp whose keys all share a bin
        // (equal weights) adds once.
        auto tally = [&](auto n_keys, const uint32_t* k, uint32_t i0) {
            constexpr int N = decltype(n_keys)::value;
            uint32_t every = 0xFFFFFFFFu, some = 0, count = 0, bin[N];
#pragma unroll
            for (int j = 0; j < N; j++) {
                bool in = i0 + 32 * j + lane < to;
                if (level == 0) safe += in && k[j] == kProtected;
                in = in && k[j] != apart && (k[j] & fixed) == threshold;
                bin[j] = in ? (k[j] >> shift) & (width - 1) : 0xFFFFFFFFu;
                every &= bin[j], some |= in ? bin[j] : 0u, count += in;
            }
            every = __reduce_and_sync(0xFFFFFFFFu, every);
            some = __reduce_or_sync(0xFFFFFFFFu, some);
            if (every == some) {
                count = __reduce_add_sync(0xFFFFFFFFu, count);
                if (lane == 0) atomicAdd(&own[some], count);
            } else if (count) {
#pragma unroll
                for (int j = 0; j < N; j++)
                    if (bin[j] != 0xFFFFFFFFu) atomicAdd(&bins[bin[j]], 1u);
            }
        };
        if constexpr (KEYS > 0) {
            constexpr int kBatch = KEYS < 8 ? KEYS : 8;
#pragma unroll
            for (int j = 0; j < KEYS; j += kBatch) tally(std::integral_constant<int, kBatch>{}, keys + j, from + 32 * j);
        } else {
            each([&](uint32_t i, uint32_t k, bool) { tally(std::integral_constant<int, 1>{}, &k, i - lane); });
        }
        if (level == 0) {
            safe = __reduce_add_sync(0xFFFFFFFFu, safe);
            if (lane == 0 && safe) atomicAdd(s_safe, safe);
        }
        __syncthreads();
        // The counts of two neighbouring bins: thread t has bins 2 t and 2 t + 1
        // from the top, of all blocks.
        const uint32_t pair = 2 * tid < width ? width - 2 - 2 * tid : 0u;
        uint2 two = *reinterpret_cast<const uint2*>(&own[pair]);
        if (level == 0) {
#pragma unroll
            for (uint32_t c = 1; c < kCopies; c++) {
                const uint2 o = *reinterpret_cast<const uint2*>(&own[c * kBins + pair]);
                two.x += o.x, two.y += o.y;
            }
        }
        uint32_t all_safe = s_safe[0];
        if (blocks > 1) {
            if (level == 0) *reinterpret_cast<uint2*>(&own[pair]) = two;
            cluster_sync();
            two = peer_sums(&own[pair], blocks);
            if (level == 0) all_safe = peer_sums(s_safe, blocks).x;
        }
        if (2 * tid >= width) two = uint2{0, 0};
        if (level == 0 && !only_safe) {
            need = p.keep - all_safe;
            if (all_safe >= p.keep) {
                // The protected tokens are enough: they compete, and no other
                // stays.  Once more from the start.
                only_safe = true;
                apart = 0;
                need = p.keep;
                if (blocks > 1)
                    cluster_sync();
                else
                    __syncthreads();
                load_keys();
                level = -1;
                continue;
            }
        }
        // The bin that holds the need-th largest.
        uint32_t upto = two.y + two.x;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
            if (lane >= (uint32_t)d) upto += o;
        }
        if (lane == 31) s_count[0][warp] = upto;
        __syncthreads();
        const uint32_t others = s_count[0][lane];
        upto += __reduce_add_sync(0xFFFFFFFFu, lane < warp ? others : 0u);
        const uint32_t past = upto - two.y - two.x;  // in higher bins
        if (past < need && need <= upto) {
            const bool second = need > past + two.y;
            s_pick[0] = width - 1 - 2 * tid - (second ? 1u : 0u);
            s_pick[1] = need - past - (second ? two.y : 0u);
            s_pick[2] = second ? two.x : two.y;
        }
        __syncthreads();
        threshold |= s_pick[0] << shift;
        fixed |= (width - 1) << shift;
        need = s_pick[1];
        // All keys of the bin survive: with the lower bits at 0 the threshold
        // lets them pass, and none has to be told from another.
        all_pass = need == s_pick[2];
    }

    // ---- survivors, holes and movers, in slot order ----
    const uint32_t below = (1u << lane) - 1u;
    uint32_t ties_before = 0, none = 0;
    if (all_pass) {
        need = 0xFFFFFFFFu;
    } else {
        each([&](uint32_t, uint32_t k, bool in) { ties_before += __popc(__ballot_sync(0xFFFFFFFFu, in && k == threshold)); });
        place(ties_before, none, 0);
    }
    // Whether a slot's token stays, for the slots in order.
    uint32_t tie = ties_before;
    auto stays = [&](uint32_t k, bool in) {
        bool yes = in && k >= threshold;
        if (!all_pass) {
            const uint32_t eq = __ballot_sync(0xFFFFFFFFu, in && k == threshold);
            yes = yes && (k != threshold || tie + __popc(eq & below) < need);
            tie += __popc(eq);
        }
        return yes;
    };
    // The lane's holes and movers: counted, and kept a bit each (KEYS of them) or
    // found again for the second pass.
    uint32_t moving = 0, bit = 0, hole = 0, mover = 0;
    each([&](uint32_t i, uint32_t k, bool in) {
        const bool yes = stays(k, in), is_hole = in && i < p.keep && !yes, is_mover = i >= p.keep && yes;
        hole += is_hole, mover += is_mover;
        if constexpr (KEYS > 0) moving |= (uint32_t)(is_hole || is_mover) << bit++;
    });
    hole = __reduce_add_sync(0xFFFFFFFFu, hole);
    mover = __reduce_add_sync(0xFFFFFFFFu, mover);
    const uint32_t holes = place(hole, mover, 1);
    if (tid == 0 && rank == 0) p.moves[list] = min(holes, p.max_moves);
    uint32_t* to_list = p.pairs + 2ull * list * p.max_moves;
    uint32_t* from_list = to_list + p.max_moves;
    bit = 0;
    tie = ties_before;
    each([&](uint32_t i, uint32_t k, bool in) {
        bool moves;
        if constexpr (KEYS > 0) {
            moves = moving >> bit++ & 1u;
        } else {
            const bool yes = stays(k, in);
            moves = in && (i < p.keep) != yes;
        }
        const bool is_hole = moves && i < p.keep;
        const uint32_t both = __ballot_sync(0xFFFFFFFFu, moves);
        if (!both) return;
        const uint32_t h = __ballot_sync(0xFFFFFFFFu, is_hole), m = both ^ h;
        const uint32_t at = is_hole ? hole + __popc(h & below) : mover + __popc(m & below);
        if (moves && at < p.max_moves) (is_hole ? to_list : from_list)[at] = i;
        hole += __popc(h);
        mover += __popc(m);
    });
    if (blocks > 1) cluster_sync();  // no block leaves while another reads its counts
}

constexpr uint32_t kTogether = 4;  // moves of a warp at a time, 8 lanes each
constexpr uint32_t kMoveThreads = 128;

// The lists' moves in groups of up to kTogether, one list after the other, in
// equal runs to the warps: few lists may have all the moves.  About 30,000
// moves in 16 of 128 lists take 7.5 us; with blocks set aside for each list
// and a move's words spread over a whole warp they took 12.7, with blocks of
// 256 threads 7.9, of 512 9.1.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
    using C = Cell<D>;
    constexpr uint32_t kSegments = kMoveThreads;
    __shared__ uint32_t s_start[kSegments];  // groups before segment s of the lists
    __shared__ uint32_t s_moves[kSegments];  // of its list, in segments of one list
    __shared__ uint32_t s_warp[kMoveThreads / 32];
    wait_for_previous();
    const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t lists = p.batch * p.pool.heads, segment = (lists + kSegments - 1) / kSegments;
    auto moves = [&](uint32_t list) { return list < lists ? p.moves[list] : 0u; };
    auto groups = [](uint32_t n) { return (n + kTogether - 1) / kTogether; };
    auto scan = [&](uint32_t v) {  // inclusive, over the warp
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
            if (lane >= (uint32_t)d) v += o;
        }
        return v;
    };
    uint32_t own = 0, last = 0;
    for (uint32_t e = 0; e < segment; e++) own += groups(last = moves(tid * segment + e));
    uint32_t upto = scan(own);
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    uint32_t total = 0;
#pragma unroll
    for (uint32_t w = 0; w < kMoveThreads / 32; w++) {
        if (w < warp) upto += s_warp[w];
        total += s_warp[w];
    }
    s_start[tid] = upto - own;
    s_moves[tid] = segment == 1 ? last : 0u;
    __syncthreads();

    // This warp's run, and the last segment that starts at or before it.
    const uint32_t workers = gridDim.x * (kMoveThreads / 32), share = (total + workers - 1) / workers;
    const uint64_t first = (uint64_t)(blockIdx.x * (kMoveThreads / 32) + warp) * share;
    if (first >= total) return;
    uint32_t left = min(share, total - (uint32_t)first);
    uint32_t at_or_before = 0;
#pragma unroll
    for (uint32_t e = 0; e < kSegments / 32; e++) at_or_before += s_start[lane + 32 * e] <= (uint32_t)first;
    const uint32_t seg = __reduce_add_sync(0xFFFFFFFFu, at_or_before) - 1;
    uint32_t list = seg * segment, group = (uint32_t)first - s_start[seg], n = s_moves[seg];
    // Eight lanes a move.  Lane q of them has an eighth of K's bytes, which are
    // in a row; row q of V, a word for each 32 channels next to the word of the
    // token's even or odd neighbour (loaded with it, stored alone); a scale
    // word in the first D / 16; and the weight or the position.
    constexpr uint32_t kGroups = D / 32;
    using KPart = std::conditional_t<D == 128, uint2, uint32_t>;
    struct alignas(4 * kGroups) VPart {
        uint32_t pair[kGroups];
    };
    const uint32_t e = lane / 8, q = lane % 8;
    for (; left; left--, group++) {
        while (group * kTogether >= n) {  // on to the list that holds the group, 32 at a time
            group -= groups(n);
            list += n ? 1 : 0;
            n = 0;
            if (list >= lists) return;
            const uint32_t count = moves(list + lane), here = groups(count), sum = scan(here);
            const uint32_t holds = __ballot_sync(0xFFFFFFFFu, sum > group);
            if (!holds) {
                group -= __shfl_sync(0xFFFFFFFFu, sum, 31);
                list += 32;
                continue;
            }
            const uint32_t to = __ffs(holds) - 1;
            group -= __shfl_sync(0xFFFFFFFFu, sum - here, to);
            list += to;
            n = __shfl_sync(0xFFFFFFFFu, count, to);
        }
        const Slots slots{p, list / p.pool.heads, list % p.pool.heads};
        const uint32_t* to_list = p.pairs + 2ull * list * p.max_moves;
        const uint32_t k = group * kTogether + e;
        uint64_t to = 0, from = 0;
        bool good = k < n;
        const uint32_t target_slot = good ? to_list[k] : 0u, source_slot = good ? to_list[p.max_moves + k] : 0u;
        good &= slots.find(target_slot, to);
        good &= slots.find(source_slot, from);
        if (!good) continue;
        const uint8_t* source = p.pool.base + (from >> 4) * C::kBytes;
        uint8_t* target = p.pool.base + (to >> 4) * C::kBytes;
        const uint16_t* source_word = reinterpret_cast<const uint16_t*>(source);
        uint16_t* target_word = reinterpret_cast<uint16_t*>(target);
        const uint32_t st = (uint32_t)from & 15u, tt = (uint32_t)to & 15u;
        const uint32_t scale = q % kGroups, value = q < kGroups ? 0 : D / 2;
        const KPart k_part = reinterpret_cast<const KPart*>(source_word + C::k_word(st, 0, 0))[q];
        const VPart v_part = *reinterpret_cast<const VPart*>(source_word + C::v_word(st & ~1u, 0, q));
        uint16_t scale_word = 0;
        float weight = 0.f;
        int32_t pos = 0;
        if (q < 2 * kGroups) scale_word = source_word[C::scale_word(st, scale) + value];
        if (q == 0) weight = p.weight[from];
        if (q == 1) pos = p.pos[from];
        reinterpret_cast<KPart*>(target_word + C::k_word(tt, 0, 0))[q] = k_part;
#pragma unroll
        for (uint32_t i = 0; i < kGroups; i++) target_word[C::v_word(tt, i, q)] = (uint16_t)(v_part.pair[i] >> 16 * (st & 1u));
        if (q < 2 * kGroups) target_word[C::scale_word(tt, scale) + value] = scale_word;
        if (q == 0) p.weight[to] = weight;
        if (q == 1) p.pos[to] = pos;
    }
}

cudaError_t launch_select(void (*kern)(EvictParams), const EvictParams& p, uint32_t cluster, cudaStream_t s) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {cluster, 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster, p.pool.heads, p.batch);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t s) {
    int sms = 0, per_sm = 0;
    cudaError_t err = kernel_fit(reinterpret_cast<const void*>(evict_select_kernel<0>), kThreads, 0, &sms, &per_sm);
    if (err != cudaSuccess) return err;
    // As many blocks a list as fit on the device at once, while a thread has more
    // than 8 keys (8,192 tokens, 8 heads: 9.7 us in one block, 12.2 in two, whose
    // barriers cost more than the keys; 16,384: 14.6 us in one block, 12.9 in
    // two, 13.1 in four), and at least as many as hold the longest sequence's
    // keys, 32 a thread (beyond 8 blocks the keys are read again for every pass:
    // 4 heads of 524,288 tokens 160 us, 8 of 262,144 35).  16 keys have a kernel
    // of their own: 32 spill, and 32 lists of 65,536 tokens take 19.4 us with
    // it, 30.1 without; 8 of 16,384 in one block 14.6 and 24.8.
    const uint64_t lists = (uint64_t)p.pool.heads * p.batch, longest = (uint64_t)p.table_width << p.pool.lg_page;
    uint32_t cluster = 1;
    while (cluster < kMaxCluster && longest > 8ull * cluster * kThreads &&
           (lists * cluster * 2 <= (uint64_t)sms || longest > 32ull * cluster * kThreads))
        cluster *= 2;
    const uint64_t keys = (longest + (uint64_t)cluster * kThreads - 1) / ((uint64_t)cluster * kThreads);
    err = launch_select(keys <= 2    ? evict_select_kernel<2>
                        : keys <= 8  ? evict_select_kernel<8>
                        : keys <= 16 ? evict_select_kernel<16>
                        : keys <= 32 ? evict_select_kernel<32>
                                     : evict_select_kernel<0>,
                        p, cluster, s);
    if (err != cudaSuccess) return err;
    void (*move)(EvictParams) = p.pool.dim == 64 ? evict_move_kernel<64> : evict_move_kernel<128>;
    err = kernel_fit(reinterpret_cast<const void*>(move), kMoveThreads, 0, &sms, &per_sm);
    if (err != cudaSuccess) return err;
    constexpr uint32_t per_block = kMoveThreads / 32 * kTogether;
    const uint64_t blocks = (lists * p.max_moves + per_block - 1) / per_block, most = (uint64_t)sms * per_sm;
    return launch_dependent(move, dim3((uint32_t)(blocks < most ? blocks : most)), dim3(kMoveThreads), 0, s, p);
}

}  // namespace sz
