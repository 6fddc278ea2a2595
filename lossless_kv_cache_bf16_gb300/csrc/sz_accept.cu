// sz_accept.cu -- the accepted tokens of a tree move up behind the context, in
// place.
//
// Token path[i] of a sequence's tree goes from slot length + path[i] to slot
// length + i.  The path ascends, so that a target can be the source of another
// move and nothing else: one block takes all the moves of a (sequence, kv head),
// eight lanes a move, and holds every word in registers before it stores the
// first one.  Bound by latency: three dependent loads (path, table, token) and a
// few kilobytes a block.  Measured (GB300): 256 sequences of 64 nodes, 8 heads of
// 64 channels: 7.9 us, 7.5 with half the threads and two rounds, 7.1 with a
// quarter; 64 sequences of 32 nodes: 2.9, and 4.0 with a quarter.
#include <type_traits>

#include "sz_cache.cuh"
#include "sz_params.h"

namespace sz {
namespace {

constexpr uint32_t kLanes = 8;  // of a move

template <int D>
__global__ void __launch_bounds__(kLanes* kMaxNodes) accept_kernel(const AcceptParams p) {
    using C = Cell<D>;
    constexpr uint32_t kGroups = D / 32;
    using KPart = std::conditional_t<D == 128, uint2, uint32_t>;  // an eighth of K's codes
    wait_for_previous();
    const uint32_t b = blockIdx.y, h = blockIdx.x, i = threadIdx.x / kLanes, q = threadIdx.x % kLanes;
    const int32_t len = p.lens[b], accepted = p.accepted[b];
    const uint64_t room = (uint64_t)p.table_width << p.pool.lg_page;
    const int32_t* path = p.path + (uint64_t)b * p.nodes;
    const bool len_ok = len >= 0 && (uint64_t)len <= room, count_ok = accepted >= 0 && (uint32_t)accepted <= p.nodes;
    bool ok = len_ok && count_ok;
    uint64_t from = 0, to = 0;       // cells, as byte offsets in the pool
    uint64_t from_at = 0, to_at = 0; // entries of the tables beside it
    uint32_t from_t = 0, to_t = 0;   // tokens of the cells
    bool move = false;
    if (ok && i < (uint32_t)accepted) {
        const int32_t node = path[i];
        // Ascending numbers are at least their index.
        ok = node >= (int32_t)i && (uint32_t)node < p.nodes && (i == 0 || path[i - 1] < node) &&
             (uint64_t)len + (uint32_t)node < room;
        move = ok && node != (int32_t)i;
        if (move) {
            auto locate = [&](uint32_t slot, uint64_t& cell, uint64_t& at, uint32_t& t) {
                const int32_t page = p.table[(uint64_t)b * p.table_width + (slot >> p.pool.lg_page)];
                const uint32_t off = slot & ((1u << p.pool.lg_page) - 1u);
                ok &= (uint32_t)page < p.pool.pages;
                cell = cell_offset<D>(p.pool, (uint32_t)page, h, off);
                at = (((uint64_t)(uint32_t)page * p.pool.heads + h) << p.pool.lg_page) + off;
                t = off & 15u;
            };
            locate((uint32_t)len + (uint32_t)node, from, from_at, from_t);
            locate((uint32_t)len + i, to, to_at, to_t);
        }
    }
    ok = __syncthreads_and(ok);
    if (h == 0 && threadIdx.x == 0) {
        p.new_lens[b] = ok ? len + accepted : len_ok ? len : 0;
        if (!ok && p.status) atomicMax(p.status, kStatusInvalid);
    }
    if (!ok) return;
    // Lane q has an eighth of K's bytes, which are in a row; row q of V, a word
    // for each 32 channels; a scale word in the first D / 16; and the weight or
    // the position.
    KPart k{};
    uint16_t v[kGroups] = {}, scale = 0;
    uint32_t entry = 0;
    const uint32_t scale_part = q >= kGroups, scale_group = q % kGroups;
    if (move) {
        const uint16_t* cell = reinterpret_cast<const uint16_t*>(p.pool.base + from);
        k = reinterpret_cast<const KPart*>(cell + C::k_word(from_t, 0, 0))[q];
#pragma unroll
        for (uint32_t e = 0; e < kGroups; e++) v[e] = cell[C::v_word(from_t, e, q)];
        if (q < 2 * kGroups) scale = cell[C::scale_word(from_t, scale_group) + scale_part * (D / 2)];
        if (q == 0 && p.weight) entry = __float_as_uint(p.weight[from_at]);
        if (q == 1 && p.pos) entry = (uint32_t)p.pos[from_at];
    }
    __syncthreads();
    if (move) {
        uint16_t* cell = reinterpret_cast<uint16_t*>(p.pool.base + to);
        reinterpret_cast<KPart*>(cell + C::k_word(to_t, 0, 0))[q] = k;
#pragma unroll
        for (uint32_t e = 0; e < kGroups; e++) cell[C::v_word(to_t, e, q)] = v[e];
        if (q < 2 * kGroups) cell[C::scale_word(to_t, scale_group) + scale_part * (D / 2)] = scale;
        if (q == 0 && p.weight) p.weight[to_at] = __uint_as_float(entry);
        if (q == 1 && p.pos) p.pos[to_at] = (int32_t)entry;
    }
}

}  // namespace

cudaError_t launch_accept(const AcceptParams& p, cudaStream_t s) {
    const uint32_t threads = (kLanes * p.nodes + 31) / 32 * 32;
    return launch_dependent(p.pool.dim == 64 ? accept_kernel<64> : accept_kernel<128>, dim3(p.pool.heads, p.batch), dim3(threads),
                            0, s, p);
}

}  // namespace sz
