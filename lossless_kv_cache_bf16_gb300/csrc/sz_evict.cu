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
// First kernel, one block per (sequence, kv head): weights as 32-bit keys
// whose unsigned order is theirs, a radix selection of the keep-th largest
// (11, 11 and 10 bits), then three passes in slot order over contiguous runs
// of slots, one per warp: ties that survive, holes and movers are counted,
// then numbered.  Second kernel: the moves, one warp each.
#include "sz_cache.cuh"
#include "sz_params.h"

namespace sz {
namespace {

constexpr uint32_t kThreads = 1024;
constexpr uint32_t kWarps = kThreads / 32;
constexpr uint32_t kKeysShared = 51200;  // keys that fit in shared memory; longer sequences read theirs again per pass
constexpr uint32_t kBins = 2048;
constexpr uint32_t kProtected = 0xFFFFFFFFu;

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
    // only_safe: there are at least `keep` protected tokens, which compete by
    // weight, and no other stays (key 0).
    __device__ __forceinline__ uint32_t key(uint32_t slot, int64_t safe_from, bool only_safe) const {
        uint64_t at;
        if (!find(slot, at)) {
            if (p.status) atomicMax(p.status, kStatusInvalid);
            return 0;
        }
        const bool safe = (int64_t)p.pos[at] >= safe_from;
        return safe == only_safe ? key_of(p.weight[at]) : safe ? kProtected : 0u;
    }
};

// Sums of the counts of the warps before this one.
__device__ __forceinline__ void warp_offsets(uint32_t (*s_count)[3], uint32_t warp, uint32_t (&off)[3]) {
#pragma unroll
    for (int k = 0; k < 3; k++) off[k] = 0;
    for (uint32_t w = 0; w < warp; w++)
#pragma unroll
        for (int k = 0; k < 3; k++) off[k] += s_count[w][k];
}

__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictParams p, const uint32_t shared_keys) {
    extern __shared__ uint32_t s_keys[];
    __shared__ uint32_t s_bins[kBins];
    __shared__ uint32_t s_count[kWarps][3];
    __shared__ uint32_t s_pick[2];
    wait_for_previous();
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    const Slots slots{p, blockIdx.y, blockIdx.x};
    const uint32_t list = blockIdx.y * p.pool.heads + blockIdx.x;
    const int32_t len = p.lens[slots.b];
    const bool ok = len >= 0 && (uint64_t)len <= (uint64_t)p.table_width << p.pool.lg_page;
    const uint32_t n = ok ? (uint32_t)len : 0u;
    if (tid == 0) {
        if (!ok && p.status) atomicMax(p.status, kStatusInvalid);
        if (blockIdx.x == 0) p.new_lens[slots.b] = (int32_t)min(n, p.keep);
        if (n <= p.keep) p.moves[list] = 0;
    }
    if (n <= p.keep) return;
    const int64_t safe_from = (int64_t)p.next_pos[slots.b] - (int64_t)p.recent;
    const bool cached = n <= shared_keys;

    // ---- keys, and the protected ones' number ----
    uint32_t safe = 0;
    for (uint32_t i = tid; i < n; i += kThreads) {
        const uint32_t k = slots.key(i, safe_from, false);
        if (cached) s_keys[i] = k;
        safe += k == kProtected;
    }
    safe = __reduce_add_sync(0xFFFFFFFFu, safe);
    if (lane == 0) s_count[warp][0] = safe;
    __syncthreads();
    safe = 0;
    for (uint32_t w = 0; w < kWarps; w++) safe += s_count[w][0];
    const bool only_safe = safe >= p.keep;
    if (only_safe && cached) {
        __syncthreads();
        for (uint32_t i = tid; i < n; i += kThreads) s_keys[i] = slots.key(i, safe_from, true);
        __syncthreads();
    }
    auto key = [&](uint32_t i) { return cached ? s_keys[i] : slots.key(i, safe_from, only_safe); };

    // ---- the threshold: `need` of the tokens whose key equals it survive ----
    const uint32_t apart = only_safe ? 0u : kProtected;  // keys that do not compete
    uint32_t threshold = 0, need = only_safe ? p.keep : p.keep - safe;
    uint32_t fixed = 0;  // mask of the bits chosen so far
    for (int level = 0; level < 3; level++) {
        const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
        const uint32_t width = level == 2 ? 1024 : 2048;
        for (uint32_t i = tid; i < kBins; i += kThreads) s_bins[i] = 0;
        __syncthreads();
        for (uint32_t i0 = warp * 32; i0 < n; i0 += kThreads) {
            const uint32_t i = i0 + lane;
            const uint32_t k = i < n ? key(i) : apart;
            const bool in = k != apart && (k & fixed) == threshold;
            const uint32_t bin = (k >> shift) & (width - 1);
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, in);
            if (!who) continue;
            // A warp whose keys share a bin (equal weights) adds once.
            const uint32_t lead = __ffs(who) - 1;
            const uint32_t bin0 = __shfl_sync(0xFFFFFFFFu, bin, lead);
            if (__all_sync(0xFFFFFFFFu, !in || bin == bin0)) {
                if (lane == lead) atomicAdd(&s_bins[bin0], __popc(who));
            } else if (in) {
                atomicAdd(&s_bins[bin], 1u);
            }
        }
        __syncthreads();
        // Warp 0 finds the bin that holds the need-th largest: each lane sums
        // a run of bins, top lane first.
        if (warp == 0) {
            const uint32_t per = width / 32, hi = width - lane * per;
            uint32_t sum = 0;
            for (uint32_t j = 1; j <= per; j++) sum += s_bins[hi - j];
            uint32_t upto = sum;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
                if (lane >= (uint32_t)d) upto += o;
            }
            const uint32_t past = __ballot_sync(0xFFFFFFFFu, upto >= need);
            if (past && lane == (uint32_t)(__ffs(past) - 1)) {
                uint32_t left = need - (upto - sum), j = 1;
                while (j < per && s_bins[hi - j] < left) left -= s_bins[hi - j], j++;
                s_pick[0] = hi - j;
                s_pick[1] = left;
            }
        }
        __syncthreads();
        threshold |= s_pick[0] << shift;
        fixed |= (width - 1) << shift;
        need = s_pick[1];
    }

    // ---- survivors, holes and movers, in slot order ----
    const uint32_t run = ((n + kWarps - 1) / kWarps + 31u) & ~31u;
    const uint32_t from = min(warp * run, n), to = min(from + run, n);
    uint32_t ties = 0;
    for (uint32_t i0 = from; i0 < to; i0 += 32)
        ties += __popc(__ballot_sync(0xFFFFFFFFu, i0 + lane < to && key(i0 + lane) == threshold));
    if (lane == 0) s_count[warp][0] = ties, s_count[warp][1] = 0, s_count[warp][2] = 0;
    __syncthreads();
    uint32_t off[3];
    warp_offsets(s_count, warp, off);
    const uint32_t ties_before = off[0];
    __syncthreads();
    uint32_t* to_list = p.pairs + 2ull * list * p.max_moves;
    uint32_t* from_list = to_list + p.max_moves;
    uint32_t holes = 0, movers = 0;
    const uint32_t below = (1u << lane) - 1u;
    for (int write = 0; write < 2; write++) {
        uint32_t tie = ties_before, hole = holes, mover = movers;
        for (uint32_t i0 = from; i0 < to; i0 += 32) {
            const uint32_t i = i0 + lane;
            const uint32_t k = i < to ? key(i) : 0u;
            const uint32_t eq = __ballot_sync(0xFFFFFFFFu, i < to && k == threshold);
            const bool stays = i < to && (k > threshold || (k == threshold && tie + __popc(eq & below) < need));
            tie += __popc(eq);
            const uint32_t hb = __ballot_sync(0xFFFFFFFFu, i < to && i < p.keep && !stays);
            const uint32_t mb = __ballot_sync(0xFFFFFFFFu, i >= p.keep && stays);
            if (write) {
                const uint32_t hi = hole + __popc(hb & below), mi = mover + __popc(mb & below);
                if (hb >> lane & 1u && hi < p.max_moves) to_list[hi] = i;
                if (mb >> lane & 1u && mi < p.max_moves) from_list[mi] = i;
            }
            hole += __popc(hb);
            mover += __popc(mb);
        }
        if (write) break;
        if (lane == 0) s_count[warp][1] = hole, s_count[warp][2] = mover;
        __syncthreads();
        warp_offsets(s_count, warp, off);
        holes = off[1], movers = off[2];
        if (tid == 0) {
            uint32_t all = 0;
            for (uint32_t w = 0; w < kWarps; w++) all += s_count[w][1];
            p.moves[list] = min(all, p.max_moves);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictParams p) {
    using C = Cell<D>;
    wait_for_previous();
    const uint32_t lane = threadIdx.x & 31u;
    const Slots slots{p, blockIdx.z, blockIdx.y};
    const uint32_t list = blockIdx.z * p.pool.heads + blockIdx.y;
    const uint32_t n = p.moves[list];
    const uint32_t* to_list = p.pairs + 2ull * list * p.max_moves;
    for (uint32_t k = blockIdx.x * 8 + threadIdx.x / 32; k < n; k += gridDim.x * 8) {
        const uint32_t slot[2] = {to_list[k], to_list[p.max_moves + k]};
        uint64_t at[2];
        if (!slots.find(slot[0], at[0]) || !slots.find(slot[1], at[1])) continue;
        uint16_t* cell[2];
        uint32_t tok[2];
#pragma unroll
        for (int e = 0; e < 2; e++) {
            cell[e] = reinterpret_cast<uint16_t*>(p.pool.base + (at[e] >> 4) * C::kBytes);
            tok[e] = (uint32_t)at[e] & 15u;
        }
        // Lane l: K and V word l (of D / 4), and a scale word in the first D / 16 lanes.
        uint16_t v[3];
        const uint32_t i = lane / 8, r = lane % 8, j = lane % (D / 32);
        if (lane < D / 4) {
            v[0] = cell[1][C::k_word(tok[1], i, r)];
            v[1] = cell[1][C::v_word(tok[1], i, r)];
        }
        if (lane < D / 16) v[2] = cell[1][C::scale_word(tok[1], j) + (lane < D / 32 ? 0 : D / 2)];
        if (lane < D / 4) {
            cell[0][C::k_word(tok[0], i, r)] = v[0];
            cell[0][C::v_word(tok[0], i, r)] = v[1];
        }
        if (lane < D / 16) cell[0][C::scale_word(tok[0], j) + (lane < D / 32 ? 0 : D / 2)] = v[2];
        if (lane == 0) p.weight[at[0]] = p.weight[at[1]];
        if (lane == 1) p.pos[at[0]] = p.pos[at[1]];
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t s) {
    int sms = 0, per_sm = 0;
    const size_t smem = 4ull * kKeysShared;
    cudaError_t err = kernel_fit(reinterpret_cast<const void*>(evict_select_kernel), kThreads, smem, &sms, &per_sm);
    if (err != cudaSuccess) return err;
    const uint64_t longest = (uint64_t)p.table_width << p.pool.lg_page;
    const size_t take = longest < kKeysShared ? 4 * longest : smem;
    err = launch_dependent(evict_select_kernel, dim3(p.pool.heads, p.batch), dim3(kThreads), take, s, p, (uint32_t)(take / 4));
    if (err != cudaSuccess) return err;
    const uint32_t blocks = (p.max_moves + 31) / 32;
    return launch_dependent(p.pool.dim == 64 ? evict_move_kernel<64> : evict_move_kernel<128>,
                            dim3(blocks < 64 ? blocks : 64, p.pool.heads, p.batch), dim3(256), 0, s, p);
}

}  // namespace sz
