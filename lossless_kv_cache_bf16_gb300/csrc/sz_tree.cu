// sz_tree.cu -- attention of a tree of drafted tokens per sequence over the
// 4-bit paged cache: o = sum_j p_j v_j / sum_j p_j, p_j = exp(scale q.k_j -
// max), over the context and the nodes that a node's mask names.
//
// What bounds it: a token and kv head cost 9 D / 8 bytes of cache and, for each
// of its R = nodes * group query rows, 4 D flops: below some 100 rows the stream
// of the cache, above the matrix unit.
//
// Both products run on the fifth-generation tensor cores with the cache as the
// left operand, 128 tokens (a tile) at a time, so that their time grows with
// the rows, not with a padded 128 of them:
//   S^T = K Q^T   128 tokens x N rows, K from tensor memory, Q^T from shared
//   O^T += V^T P^T   D channels x N rows, V^T from tensor memory, P^T from shared
// Codes never pass through shared memory again: warps read a raw cell, turn it
// into 16-bit values and store them as tensor-memory operands.  The order of
// k (channels, tokens) inside an operand is free as long as both sides agree: it
// is the one in which a lane's words of a cell are its fragment's registers.
//   K: (code - 8) * scale as fp16, 3 bits times 8 bits, the token's scales
//   divided by a power of two of the token's own.  The four bits of a code, 4
//   places up, are a subnormal number, so that one fused multiply-add makes two
//   values, exact as long as the scales lie within 2^12 of the largest one (and
//   otherwise to 2^-19 of that).  The power and the row's (queries are scaled
//   the same way) come back as factors of S.
//   V: (code - 8) * scale as bf16, one rounding; weights are rounded to bf16.
//
// Roles of a block's warps (one block an SM): softmax (a thread a token, a
// group of four warps for NC of the rows), K and V (two sets of four each, for
// every other tile), one that copies raw tiles into a ring, two that prepare
// queries, one that issues the matrix instructions: S of tile n + 1 before O of
// tile n.  All walk the same list of segments.
//
// Softmax.  A row's maximum lies across threads, so that a tile only asks
// whether any weight would pass 2^80: one vote of the group.  Only then (the
// first tile, and rarely after) the maxima are formed and O is rescaled.  Sums
// of weights stay in registers, a share per thread, until the item's end.
//
// Work split.  The list of (sequence, kv head, tile of rows, tile of tokens),
// with kItemCost more entries per item, is cut into one equal run per block.
// Items over several blocks are joined by a second kernel, in list order:
// results do not depend on timing.
//
// Measured (GB300, 128 channels): 16 sequences of 32,768 tokens, 8 nodes, 7 query
// heads per kv head, 4 kv heads: 128 us, 304 MB at 2.4 TB/s.  4 sequences of
// 32,768, 64 nodes: 208 us, 120 GFLOP at 579 TFLOP/s.  16 ragged sequences up to
// 8,192, 32 nodes: 44 us.  A tile of 128 tokens and 64 rows is 5,800 warp
// instructions (1,450 issue slots of a scheduler), a quarter each for K, V, softmax,
// and waits and addresses, and takes 1,900 clocks.  That is the way of a softmax
// group through it, one thing after the other: 370 clocks until the logits are
// there, 540 to load them, 715 for the weights, 300 for the fence and the vote.
// K's and V's warps idle for half of that; the schedulers issue in two of three
// cycles, the ALU pipe is busy for 58%, the matrix unit for 25%, and memory gives a
// third of what it could.
#include <cfloat>

#include "sz_cache.cuh"
#include "sz_params.h"
#include "sz_tcgen.cuh"

namespace sz {
namespace {

constexpr uint32_t kTile = 128;  // tokens of a tile
// Tiles that an item's start and end count for in the split.  Measured with 4 / 5 /
// 6 / 8 / 10: a ragged batch of 16, 32 nodes: 48.3 / 46.6 / 43.6 / 46.7 / 47.9 us; 4
// sequences of 2,048, chains of 4: 16.7 / 17.0 / 17.2 / 17.6 / 17.0; 16 of 32,768, 8
// nodes: 128.7 / 129.0 / 128.9 / 130.9 / 130.8.  The dip of the first is where the
// cuts of that one list fall; by the others anything up to 6 will do.
constexpr uint32_t kItemCost = 6;
constexpr uint32_t kJoinThreads = 512;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kNone = -FLT_MAX;  // a row's reference before any
// A row's weights are 2^(x - reference), the reference at first 40 above the
// largest logit x and moved once a weight would pass 2^80, 2^120 times that one:
// as rarely as fp32 allows with sums over values up to 2^30.  What is lost below
// has less than 2^-86 of the largest weight, or of 1 where it is a weight times
// a value.  Rows whose references lie within 20 share one (20 to 40 above their
// largest logits), and rows whose queries' sizes lie within 2^12 a factor: the
// smallest of them has 2^2 or more as its largest fp16 value, whose steps end at
// 2^-24.
constexpr float kAbove = 40.f, kHigh = 80.f, kShare = 20.f;
constexpr int kShareExp = 12;
constexpr int kMinExp = -112;      // of a power of two that is taken out
constexpr uint32_t kMostScale = 0x7E117E11u;  // the largest bf16 number whose sevenfold is one, twice

template <int D, int N>
struct Shape {
    static constexpr int kGroups = N > 32 ? 2 : 1;     // of softmax warps
    static constexpr int kCols = N / kGroups;          // rows of a group
    static constexpr int kSoftmax = 4 * kGroups;       // warps
    // K and V: two sets of four warps each, for every other tile.
    static constexpr int kKWarp = kSoftmax, kVWarp = kKWarp + 8, kLoad = kVWarp + 8, kMma = kLoad + 1, kQuery = kLoad + 2;
    static constexpr int kQueries = 2;                 // warps
    static constexpr int kParts = 64 / N;              // their lanes of a row
    static constexpr int kThreads = 32 * (kLoad + 4);
    // Registers a thread: at launch, and of the warps of softmax, of K and V,
    // and of the others, which add up to as many.
    static constexpr int kRegs = kGroups == 2 ? 72 : 80, kSoftmaxRegs = kGroups == 2 ? 120 : 168, kCellRegs = kGroups == 2 ? 56 : 64,
                         kOtherRegs = kGroups == 2 ? 40 : 56;
    static_assert(4 * kGroups * kSoftmaxRegs + 16 * kCellRegs + 4 * kOtherRegs <= (4 * kGroups + 20) * kRegs, "registers of a block");
    static constexpr uint32_t kCell = Cell<D>::kBytes;
    static constexpr uint32_t kStageBytes = 8 * kCell;
    static constexpr uint32_t kQBytes = 2 * N * D, kPBytes = 2 * N * kTile;
    static constexpr uint32_t kRow = 2 * D + 16;  // bytes of a query row as it comes, padded against bank conflicts
    static constexpr uint32_t kP = 2 * kQBytes, kRows = kP + 2 * kPBytes, kRing = kRows + N * kRow;
    static constexpr uint32_t kTok = 4 * kMaxBatch, kCnt = kMaxBatch;
    static constexpr int kStages = (232448 - 16384 - kRing - kTok - kCnt) / kStageBytes < 16 ? (232448 - 16384 - kRing - kTok - kCnt) / kStageBytes : 16;
    static constexpr uint32_t kTokAt = kRing + kStages * kStageBytes, kCntAt = kTokAt + kTok, kBytes = kCntAt + kCnt;
    // Tensor memory columns.
    // Buffers for V, which runs ahead where there is room (4 sequences of 2,048,
    // chains of 4: 17.0 us, 17.7 with two).
    static constexpr uint32_t kV = D + 4 * 64 + 3 * N <= 512 ? 4 : 2;
    static constexpr uint32_t kKCol = 0, kVCol = D, kSCol = D + 64 * kV, kOCol = kSCol + 2 * N;
    static_assert(kOCol + N <= 512 && kStages >= 3, "tensor memory, ring");
    // The two sets of K's and of V's warps take every other tile, and each has to
    // see every phase of its stages and buffers: a parity tells neighbours only.
    static_assert(kStages % 2 == 0 && kV % 2 == 0, "stages of a set");
};

struct Bars {
    uint64_t raw_full[16], raw_free[16];
    uint64_t k_full[2], v_full[4], s_full[2], p_full[2], pv[4], q_full[2], q_free[2], q_raw[2];
    uint64_t o_full, o_free, end;
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
// Two fp32 numbers in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void fma2(float& a, float& b, uint64_t f, uint64_t c) {
    asm("{\n\t.reg .b64 x;\n\tmov.b64 x, {%0, %1};\n\tfma.rn.f32x2 x, x, %2, %3;\n\tmov.b64 {%0, %1}, x;\n\t}" : "+f"(a), "+f"(b) : "l"(f), "l"(c));
}
__device__ __forceinline__ void add2(float& a, float& b, float c, float d) {
    asm("{\n\t.reg .b64 x;\n\tmov.b64 x, {%0, %1};\n\tadd.rn.f32x2 x, x, %2;\n\tmov.b64 {%0, %1}, x;\n\t}" : "+f"(a), "+f"(b) : "l"(pair(c, d)));
}
// Both 16-bit halves.
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
// 2^e, e in -126 .. 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x, w[1] = v.y;
    }
}

// As mbar_try_wait, for up to kSuspend ns at a time: polls of warps that run ahead
// take issue slots from those that do not (16 x 32,768 tokens: 132.5 us, 134.5
// without the limit).
constexpr uint32_t kSuspend = 5000;
__device__ __forceinline__ bool mbar_rest(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"((uint32_t)__cvta_generic_to_shared(bar)), "r"(parity), "r"(kSuspend)
                 : "memory");
    return done;
}

// v[0 .. N) reduced over the warp's lanes: lane k gets value k % N.
template <int S, int N, typename Op>
__device__ __forceinline__ void halve_columns(float (&v)[N], uint32_t lane, Op op) {
    if constexpr (S > 0) {
        const bool up = lane & S;
#pragma unroll
        for (int k = 0; k < S; k++) {
            const float send = up ? v[k] : v[k + S], keep = up ? v[k + S] : v[k];
            v[k] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, send, S));
        }
        halve_columns<S / 2>(v, lane, op);
    }
}
template <int N, typename Op>
__device__ __forceinline__ float reduce_columns(float (&v)[N], uint32_t lane, Op op) {
    halve_columns<N / 2>(v, lane, op);
    return N == 16 ? op(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 16)) : v[0];
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// Registers a thread of this warpgroup from here on.
template <int R>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

__device__ __forceinline__ void group_sync(uint32_t id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool group_any(uint32_t id, bool x) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\tbar.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(id), "r"((uint32_t)x)
        : "memory");
    return any;
}

// A part of an item that a block has: tiles r0 .. r1 - 1 of its tokens.
struct Segment {
    uint32_t b, head, row0, rows;  // rows row0 .. row0 + rows - 1 of the sequence and kv head
    uint32_t r0, r1;
    uint32_t tokens, len;  // of the sequence: all, and its context
    uint32_t item, rest;   // tiles after r1
    bool starts, ends;
};

// The list: sequence, item (kv head and tile of rows) and entry of the item, of
// which the last kItemCost stand for its fixed cost.
template <int N>
struct Walk {
    uint32_t b, item, at, left;
    const uint32_t* tok;
    const uint8_t* cnt;
    uint32_t batch, heads, group;
    const Segment* first;  // the next one, where it has been found

    // Bit 7 of cnt: a sequence that has been reported, whose rows are zero.
    static __device__ __forceinline__ uint32_t nodes_of(uint32_t c) { return c & 0x80u ? 0u : c; }
    __device__ __forceinline__ uint32_t tiles(uint32_t b_) const { return (nodes_of(cnt[b_]) * group + N - 1) / N; }
    __device__ __forceinline__ uint32_t entries(uint32_t b_) const { return (tok[b_] + kTile - 1) / kTile + kItemCost; }
    __device__ __forceinline__ bool next(Segment& s) {
        if (first) {
            s = *first;
            first = nullptr;
            return true;
        }
        while (left) {
            while (item == heads * tiles(b)) b++, item = 0;  // the list has an entry yet
            const uint32_t cost = entries(b), units = cost - kItemCost, take = min(left, cost - at), to = at + take;
            s.r0 = min(at, units);
            s.r1 = min(to, units);
            const uint32_t t = tiles(b), count = nodes_of(cnt[b]);
            s.b = b;
            s.item = item;
            s.head = item / t;
            s.row0 = item % t * N;
            s.rows = min((uint32_t)N, count * group - s.row0);
            s.tokens = tok[b];
            s.len = tok[b] - count;
            s.starts = s.r0 == 0;
            s.ends = s.r1 == units;
            s.rest = units - s.r1;
            left -= take;
            at = to;
            if (at == cost) item++, at = 0;
            if (s.r0 != s.r1) return true;
        }
        return false;
    }
};

// Channel of a lane of O^T: V's warps take theirs in this order.
template <int D>
__device__ __forceinline__ uint32_t channel_of(uint32_t lane) {
    const uint32_t w = lane / 32, e = lane / 8 % 4, c = lane % 8;
    return D == 128 ? 32 * (c & 3) + 4 * (2 * w + (c >> 2)) + e : 32 * (c & 1) + 4 * (4 * w + (c >> 1)) + e;
}

template <int D, int N>
__global__ void __launch_bounds__(Shape<D, N>::kThreads, 1) tree_kernel(const TreeParams p) {
    using Sh = Shape<D, N>;
    using C = Cell<D>;
    constexpr int G = C::kGroups, NC = Sh::kCols, SG = Sh::kGroups, RS = Sh::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Bars bars;
    __shared__ uint32_t s_tmem, s_dead;
    __shared__ unsigned long long s_total, s_nan[8][2][4];  // [segment % 8][group][channels / 32]: nodes whose V is not finite
    __shared__ Segment s_first;                      // this block's first segment, and the walk after it
    __shared__ uint32_t s_after[4];
    __shared__ __align__(16) uint8_t s_valid[16][8];  // tokens of a stage's cells
    __shared__ float s_kf[4][kTile];                  // [tile % 4]: factor of a token, 0: not there
    __shared__ __align__(4) uint8_t s_absent[4][4];   // [tile % 4][warp]: whether any token is not there
    __shared__ __align__(16) float s_rf[4][N];        // [segment % 4]: factor of a row
    __shared__ float s_common[4][2];                  // of all rows of a group, or -1
    __shared__ __align__(16) float s_less[N], s_f[N];  // less the reference of a row; a factor
    __shared__ float s_one[2];                        // less the reference of all rows of a group, or infinity
    __shared__ float s_red[2][4][32];
    // [segment % 8][group]: the rows that see a node.  Queries are prepared while
    // softmax ends the fourth segment before.
    __shared__ uint32_t s_seen[8][Sh::kGroups][kMaxNodes];
    uint32_t* s_tok = reinterpret_cast<uint32_t*>(smem + Sh::kTokAt);
    uint8_t* s_cnt = smem + Sh::kCntAt;
    const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t heads = p.pool.heads, q_heads = heads * p.group, lg_page = p.pool.lg_page;

    if (tid == 0) {
        for (int k = 0; k < RS; k++) mbar_init(&bars.raw_full[k], 1), mbar_init(&bars.raw_free[k], 8);
        for (int k = 0; k < 2; k++) {
            mbar_init(&bars.k_full[k], 4);
            mbar_init(&bars.s_full[k], 2);
            mbar_init(&bars.p_full[k], Sh::kGroups);
            mbar_init(&bars.q_full[k], Sh::kQueries), mbar_init(&bars.q_free[k], 1), mbar_init(&bars.q_raw[k], 1);
        }
        for (uint32_t k = 0; k < Sh::kV; k++) mbar_init(&bars.v_full[k], 4), mbar_init(&bars.pv[k], 1);
        mbar_init(&bars.o_full, 2), mbar_init(&bars.o_free, Sh::kSoftmax), mbar_init(&bars.end, 1);
        fence_mbar_init();
        s_total = 0;
        s_dead = 0;
    }
    if (tid < 64) (&s_nan[0][0][0])[tid] = 0;
    if (warp == Sh::kMma) tmem_alloc(&s_tmem, 512);
    __syncthreads();
    wait_for_previous();

    // ---- the list, and this block's run of it ----
    using Wk = Walk<N>;
    Wk walk{0, 0, 0, 0, s_tok, s_cnt, p.batch, heads, p.group, nullptr};
    const uint64_t room = (uint64_t)p.table_width << lg_page;
    unsigned long long mine = 0;
    for (uint32_t b = tid; b < p.batch; b += Sh::kThreads) {
        const int32_t len = p.lens[b], count = p.counts ? p.counts[b] : (int32_t)p.nodes;
        const bool count_ok = count >= 0 && (uint32_t)count <= p.nodes;
        const bool ok = count_ok && len >= 0 && (uint64_t)len + (uint32_t)count <= room;
        if (!ok && p.status && blockIdx.x == 0) atomicMax(p.status, kStatusInvalid);
        s_tok[b] = ok ? (uint32_t)len + (uint32_t)count : 0u;
        s_cnt[b] = count_ok ? (uint8_t)(count | (ok ? 0 : 0x80)) : 0;
        mine += (unsigned long long)heads * walk.tiles(b) * walk.entries(b);
    }
    if (mine) atomicAdd(&s_total, mine);
    __syncthreads();
    const uint64_t total = s_total;
    const uint32_t share = total >> 31 ? (uint32_t)((total + gridDim.x - 1) / gridDim.x) : ((uint32_t)total + gridDim.x - 1) / gridDim.x;
    const uint64_t u0 = min((uint64_t)blockIdx.x * share, total);
    const uint32_t n_run = (uint32_t)(min(u0 + share, total) - u0);
    // Rows of sequences that cannot be served are zero.
    for (uint32_t b = blockIdx.x; b < p.batch; b += gridDim.x) {
        const uint32_t c = s_cnt[b];
        if (!(c & 0x80u)) continue;
        // A warp a row: there may be 2^28 of them, and 2^35 channels.
        for (uint32_t r = warp; r < (c & 0x7Fu) * q_heads; r += Sh::kThreads / 32) {
            const uint32_t node = r / q_heads, h = r % q_heads;
            uint16_t* out = p.out + (int64_t)b * p.out_seq + (int64_t)node * p.out_node + (int64_t)h * p.out_head;
            for (uint32_t k = lane; k < D; k += 32) out[k] = 0;
            if (p.lse && lane == 0) p.lse[((uint64_t)b * p.nodes + node) * q_heads + h] = kNegInf;
        }
    }
    if (tid == 0) p.meta[4 * blockIdx.x] = -1;
    if (warp == 0 && n_run) {
        uint64_t before = 0;
        for (uint32_t b0 = 0; b0 < p.batch; b0 += 32) {
            const uint64_t n = b0 + lane < p.batch ? (uint64_t)heads * walk.tiles(b0 + lane) * walk.entries(b0 + lane) : 0ull;
            uint64_t upto = n;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const uint64_t o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
                if (lane >= (uint32_t)d) upto += o;
            }
            const uint32_t past = __ballot_sync(0xFFFFFFFFu, before + upto > u0);
            if (past) {
                if (lane == (uint32_t)__ffs(past) - 1) {
                    const uint64_t at = u0 - (before + upto - n);
                    const uint32_t cost = walk.entries(b0 + lane);
                    Wk w = walk;
                    w.b = b0 + lane, w.left = n_run;
                    if (at >> 32)
                        w.item = (uint32_t)(at / cost), w.at = (uint32_t)(at % cost);
                    else
                        w.item = (uint32_t)at / cost, w.at = (uint32_t)at % cost;
                    if (!w.next(s_first)) s_first.r1 = s_first.r0 = 0;
                    s_after[0] = w.b, s_after[1] = w.item, s_after[2] = w.at, s_after[3] = w.left;
                }
                break;
            }
            before += __shfl_sync(0xFFFFFFFFu, upto, 31);
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (n_run && s_first.r0 != s_first.r1) {
        walk.first = &s_first;
        walk.b = s_after[0], walk.item = s_after[1], walk.at = s_after[2], walk.left = s_after[3];
    }
    const uint32_t tmem = s_tmem;

    // Waits for a phase; false once any wait of the block has given up.  The clock
    // is slow to read: not before many polls.
    volatile uint32_t* dead = &s_dead;
    auto wait_alone = [&](uint64_t* bar, uint32_t parity) {
        uint64_t t0 = 0;
        for (uint32_t k = 1; !mbar_rest(bar, parity); k++) {
            if (k % 64) continue;
            if (*dead) return false;
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > p.wait_limit_ns) {
                *dead = 1;
                return false;
            }
        }
        return true;
    };
    // The same for a warp, with one answer.
    auto wait = [&](uint64_t* bar, uint32_t parity) { return (bool)__all_sync(0xFFFFFFFFu, wait_alone(bar, parity)); };
    // On to the next stage of the ring.
    auto step = [](uint32_t& stage, uint32_t& phase) {
        if (++stage == (uint32_t)RS) stage = 0, phase ^= 1u;
    };
    // A warp's arrival, after what its lanes have written.
    auto arrive = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };

    if (warp < Sh::kSoftmax) {
        // ======== softmax: thread = token of a tile (row of S^T), and = channel of O^T ========
        more_registers<Sh::kSoftmaxRegs>();
        const uint32_t g = warp / 4, row = tid % kTile, col0 = g * NC, bar_id = 1 + g, at0 = (warp % 4) << 21;
        const uint32_t s_at = tmem + at0 + Sh::kSCol + col0, o_at = tmem + at0 + Sh::kOCol + col0;
        // Where this token's weights go: the order of V's columns.
        const uint32_t kpos = (row & ~15u) + 4 * (row >> 1 & 3u) + 2 * (row >> 3 & 1u) + (row & 1u);
        uint8_t* p_at = smem + Sh::kP + (col0 / 8) * (kTile * 16) + kpos * 16;
        // Its warps meet at barriers: once a wait has given up they go on to the
        // end without waiting, and what they write is written over.
        bool alive = true;
        auto attend_to = [&](uint64_t* bar, uint32_t parity) {
            if (alive) alive = wait(bar, parity);
        };
        {
            uint32_t n = 0, seg = 0;
            Segment s;
            for (Wk w = walk; w.next(s); seg++) {
                const bool used = col0 < s.rows;
                const uint32_t cols = used ? min((uint32_t)NC, s.rows - col0) : 0u;
                if (row < NC) s_less[col0 + row] = row < cols ? -kNone : 0.f;
                float l[NC];
#pragma unroll
                for (int j = 0; j < NC; j++) l[j] = 0.f;
                group_sync(bar_id);
                const float* rf = s_rf[seg & 3u] + col0;
                float one = 0.f, common = 0.f;
                bool shared = false;  // whether all rows share a reference and a factor
                float x[NC];
                auto ask = [&](uint32_t n) {
#pragma unroll
                    for (int j = 0; j < NC; j += 16) tmem_load16(s_at + (n & 1u) * N + j, x + j);
                };
                uint32_t t = s.r0;
                // Of a group without rows the first warp alone follows the tiles: a
                // warp that others do not wait for could fall two phases behind,
                // and a parity does not tell two from none.
                if (!used) {
                    for (uint32_t k = n; warp % 4 == 0 && k < n + (s.r1 - t); k++) {
                        attend_to(&bars.s_full[k & 1u], k >> 1 & 1u);
                        if (lane == 0) mbar_arrive(&bars.p_full[k & 1u]);
                    }
                    n += s.r1 - t, t = s.r1;
                }
                for (; t < s.r1; t++, n++) {
                    const uint32_t buf = n & 1u;
                    attend_to(&bars.s_full[buf], n >> 1 & 1u);
                    tmem_fence_after();
                    ask(n);
                    const float kf = s_kf[n & 3u][row];
                    const uint32_t token = t * kTile + row;
                    // Whether the tile has tokens that not every row sees, or that are not there.
                    const bool special = (t + 1) * kTile > s.len || *reinterpret_cast<const uint32_t*>(s_absent[n & 3u]) != 0;
                    uint32_t rows_seen = 0xFFFFFFFFu;
                    if (special) {
                        if (token >= s.len) rows_seen = s_seen[seg & 7u][g][token - s.len & 63u];
                        if (kf == 0.f) rows_seen = 0;
                    }
                    auto unseen = [&]() {
#pragma unroll
                        for (int j = 0; j < NC; j++) x[j] = rows_seen >> j & 1u ? x[j] : kNegInf;
                    };
                    bool move = t == s.r0;
                    for (int turn = 0; turn < 2; turn++) {
                        if (move) {
                            // ---- references: at first, and when a weight is too large ----
                            tmem_wait_loads();
#pragma unroll
                            for (int j = 0; j < NC; j++) x[j] *= rf[j] * kf;
                            if (special) unseen();
                            const float top = reduce_columns<NC>(x, lane, [](float a, float b) { return fmaxf(a, b); });
                            s_red[g][warp % 4][lane] = top;
                            group_sync(bar_id);
                            if (row < 32) {
                                float ref = 0.f;
                                if (row < NC) {
                                    const float old = -s_less[col0 + row];
                                    const float most = fmaxf(fmaxf(s_red[g][0][row], s_red[g][1][row]), fmaxf(s_red[g][2][row], s_red[g][3][row]));
                                    ref = most - old > kHigh ? most + kAbove : old;
                                    s_f[col0 + row] = exp2_fast(old - ref);
                                }
                                float above = row < cols ? ref : kNegInf, below = row < cols ? ref : -kNegInf;
#pragma unroll
                                for (int d = 16; d; d /= 2) {
                                    above = fmaxf(above, __shfl_xor_sync(0xFFFFFFFFu, above, d));
                                    below = fminf(below, __shfl_xor_sync(0xFFFFFFFFu, below, d));
                                }
                                // At the first tile only: there nothing has been added
                                // up.  Columns without a row have logits of 0.
                                const bool share = t == s.r0 && above - below <= kShare && (cols == NC || above >= kShare);
                                if (share) ref = above - kShare;
                                if (row < NC) s_less[col0 + row] = row < cols ? -ref : 0.f;
                                if (row == 0) s_one[g] = share ? -ref : -kNegInf;
                            }
                            group_sync(bar_id);
                            one = s_one[g];
                            common = s_common[seg & 3u][g];
                            shared = one != -kNegInf && common >= 0.f;
                            if (t > s.r0) {
#pragma unroll
                                for (int j = 0; j < NC; j++) l[j] *= s_f[col0 + j];
                                attend_to(&bars.pv[(n - 1) % Sh::kV], (n - 1) / Sh::kV & 1u);
                                tmem_fence_after();
#pragma unroll 1
                                for (int j = 0; j < NC; j += 16) {
                                    float o[16];
                                    tmem_load16(o_at + j, o);
                                    tmem_wait_loads();
#pragma unroll
                                    for (int k = 0; k < 16; k++) o[k] *= s_f[col0 + j + k];
                                    tmem_store16(o_at + j, o);
                                }
                                tmem_wait_stores();
                            }
                            ask(n);
                        }
                        // ---- weights ----
                        tmem_wait_loads();
                        if (shared) {
                            const uint64_t f = pair(common * kf, common * kf), less = pair(one, one);
#pragma unroll
                            for (int j = 0; j < NC; j += 2) fma2(x[j], x[j + 1], f, less);
                        } else {
#pragma unroll
                            for (int j = 0; j < NC; j += 4) {
                                const float4 f = *reinterpret_cast<const float4*>(rf + j), less = *reinterpret_cast<const float4*>(s_less + col0 + j);
                                x[j] = fmaf(x[j], f.x * kf, less.x), x[j + 1] = fmaf(x[j + 1], f.y * kf, less.y);
                                x[j + 2] = fmaf(x[j + 2], f.z * kf, less.z), x[j + 3] = fmaf(x[j + 3], f.w * kf, less.w);
                            }
                        }
                        if (special) unseen();
                        // O of tile n - 2, which read this buffer of weights, was
                        // issued before S of this tile, and so has ended.
                        float high = 0.f;
#pragma unroll
                        for (int j = 0; j < NC; j += 8) {
                            uint32_t v[4];
#pragma unroll
                            for (int k = 0; k < 4; k++) {
                                high = max3(high, x[j + 2 * k], x[j + 2 * k + 1]);
                                x[j + 2 * k] = exp2_fast(x[j + 2 * k]);
                                x[j + 2 * k + 1] = exp2_fast(x[j + 2 * k + 1]);
                                v[k] = pack_bf16(x[j + 2 * k], x[j + 2 * k + 1]);
                            }
                            *reinterpret_cast<uint4*>(p_at + buf * Sh::kPBytes + (j / 8) * (kTile * 16)) = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                        fence_async_smem();
                        tmem_fence_before();
                        // The group's weights are written, unless one is too large.
                        move = group_any(bar_id, high > kHigh);
                        if (!move) break;
                        ask(n);
                    }
                    if (row == 0) mbar_arrive(&bars.p_full[buf]);
#pragma unroll
                    for (int j = 0; j < NC; j += 2) add2(l[j], l[j + 1], x[j], x[j + 1]);
                }

                // ---- the item's rows, or a piece of them ----
                const bool direct = s.starts && s.ends;
                const uint32_t slot = 2 * blockIdx.x + (s.starts ? 1u : 0u);
                if (used) {
                    const float sum = reduce_columns<NC>(l, lane, [](float a, float b) { return a + b; });
                    s_red[g][warp % 4][lane] = sum;
                    group_sync(bar_id);
                    if (row < cols) {
                        const float all = (s_red[g][0][row] + s_red[g][1][row]) + (s_red[g][2][row] + s_red[g][3][row]);
                        const float m = -s_less[col0 + row];
                        s_f[col0 + row] = all == 0.f ? 0.f : 1.f / all;
                        if (direct) {
                            const uint32_t r = s.row0 + col0 + row;
                            if (p.lse)
                                p.lse[((uint64_t)s.b * p.nodes + r / p.group) * q_heads + s.head * p.group + r % p.group] =
                                    all == 0.f ? kNegInf : (m + log2f(all)) * 0.6931471805599453f;
                        } else {
                            *reinterpret_cast<float2*>(p.part_ml + ((uint64_t)slot * N + col0 + row) * 2) = make_float2(m, all);
                        }
                    }
                    group_sync(bar_id);
                }
                attend_to(&bars.o_full, seg & 1u);
                tmem_fence_after();
                float o[NC];
#pragma unroll
                for (int j = 0; j < NC; j += 16) tmem_load16(o_at + j, o + j);
                tmem_wait_loads();
                tmem_fence_before();
                arrive(&bars.o_free);
                // V's warps mark for both groups.  What is left here would be another
                // item's eight segments later.
                if (!used) {
                    if (row < 4) s_nan[seg & 7u][g][row] = 0;
                    continue;
                }
                const uint32_t ch = channel_of<D>(row);
                const uint64_t bad = row < D ? s_nan[seg & 7u][g][ch / 32] : 0ull;
                if (bad) {
                    uint32_t hit = 0;
                    for (uint64_t left = bad; left; left &= left - 1) hit |= s_seen[seg & 7u][g][__ffsll((long long)left) - 1];
#pragma unroll
                    for (int j = 0; j < NC; j++) o[j] = hit >> j & 1u ? __int_as_float(0x7FC00000) : o[j];
                }
                if (direct) {
                    // Through the first buffer of weights, this group's part of
                    // it, a row every 256 bytes.
                    uint8_t* stage = smem + Sh::kP + col0 * 256;
                    if (row < D) {
#pragma unroll
                        for (int j = 0; j < NC; j++)
                            *reinterpret_cast<uint16_t*>(stage + j * 256 + ch * 2) = (uint16_t)bf16_bits(o[j] * s_f[col0 + j]);
                    }
                    group_sync(bar_id);
                    for (uint32_t k = row; k < cols * (D / 8); k += kTile) {
                        const uint32_t j = k / (D / 8), c = 8 * (k % (D / 8)), r = s.row0 + col0 + j;
                        const uint4 v = *reinterpret_cast<const uint4*>(stage + j * 256 + c * 2);
                        uint16_t* dst = p.out + (int64_t)s.b * p.out_seq + (int64_t)(r / p.group) * p.out_node +
                                        (int64_t)(s.head * p.group + r % p.group) * p.out_head + c;
                        if (p.out_vec) {
                            *reinterpret_cast<uint4*>(dst) = v;
                        } else {
                            const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int e = 0; e < 4; e++) dst[2 * e] = (uint16_t)w4[e], dst[2 * e + 1] = (uint16_t)(w4[e] >> 16);
                        }
                    }
                } else {
                    float* dst = p.part_o + ((uint64_t)slot * N + col0) * kTile + row;
#pragma unroll
                    for (int j = 0; j < NC; j++)
                        if ((uint32_t)j < cols) dst[j * kTile] = o[j];
                    if (s.starts && g == 0 && row == 0) {
                        // The blocks after this one that hold the rest of the item.
                        p.meta[4 * blockIdx.x + 1] = (int32_t)s.item;
                        p.meta[4 * blockIdx.x + 2] = (int32_t)((s.rest + share - 1) / share);
                        p.meta[4 * blockIdx.x + 3] = (int32_t)(s.tokens - s.len);
                        p.meta[4 * blockIdx.x] = (int32_t)s.b;
                    }
                }
                group_sync(bar_id);
                if (row < 4) s_nan[seg & 7u][g][row] = 0;  // all have read it
            }
        }
    } else if (warp < Sh::kVWarp) {
        // ======== K: raw cells to the operand, two cells a warp and tile ========
        fewer_registers<Sh::kCellRegs>();
        const uint32_t w = warp % 4, set = (warp - Sh::kKWarp) / 4, x = lane % 4, t0 = lane / 4, half_sel = t0 & 1u ? 0x3244u : 0x1044u;  // scales come in pairs of tokens
        auto role = [&]() {
            uint32_t n = 0, stage = 0, phase = 0;
            Segment s;
            for (Wk wk = walk; wk.next(s);) {
                for (uint32_t t = s.r0; t < s.r1; t++, n++, step(stage, phase)) {
                    const uint32_t buf = n & 1u, par = n >> 1 & 1u;
                    if (buf != set) continue;
                    if (blockIdx.x == p.stalled_block) *dead = 1;
                    if (blockIdx.x == p.stalled_block || !wait(&bars.raw_full[stage], phase)) return;
                    if (!wait(&bars.s_full[buf], par ^ 1u)) return;
                    tmem_fence_after();
                    const uint8_t* raw = smem + Sh::kRing + stage * Sh::kStageBytes + 2 * w * Sh::kCell;
                    uint32_t missing = 32;
#pragma unroll 1
                    for (int cc = 0; cc < 2; cc++, raw += Sh::kCell) {
                        const uint32_t valid = s_valid[stage][2 * w + cc];
                        missing -= valid;
                        uint32_t words[2][G], mult[2][G];
#pragma unroll
                        for (int r = 0; r < 2; r++) {
                            const uint32_t tk = t0 + 8 * r;
                            // A lane has one of the token's scales, of which its four
                            // lanes find the largest.  One that is not finite makes
                            // values, and with them all logits of the token, that
                            // are not.
                            lds_words<G>(raw + (tk * 4 + x) * (4 * G), words[r]);
                            const uint32_t sc = *reinterpret_cast<const uint32_t*>(raw + 2 * C::kKScale + (tk >> 1) * (4 * G) + 4 * (x % G));
                            const float v = __uint_as_float(prmt(sc, 0u, half_sel));
                            float top = fabsf(v);
#pragma unroll
                            for (int d = 1; d < G; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                            const uint32_t e = max(__float_as_uint(top) & 0x7F800000u, (uint32_t)(kMinExp + 127) << 23);
                            const float unit = __uint_as_float(((127u + 15u + 127u) << 23) - e);
                            const uint32_t m = pack_f16(v * unit, v * unit);
#pragma unroll
                            for (int i = 0; i < G; i++) mult[r][i] = __shfl_sync(0xFFFFFFFFu, m, i, 4);
                            if (x == 0) s_kf[n & 3u][32 * w + 16 * cc + tk] = tk < valid ? __uint_as_float(e - (5u << 23)) : 0.f;
                        }
#pragma unroll
                        for (int i = 0; i < G; i++) {
                            uint32_t v[8];
#pragma unroll
                            for (int r = 0; r < 2; r++) {
                                // (code 2^-20 - 2^-17) * mult, mult below 2^16.
                                const uint32_t less = mul_f16x2(mult[r][i], 0x80808080u);
                                const uint32_t y = words[r][i];
                                v[2 * r] = fma_f16x2(y << 4 & 0x00F000F0u, mult[r][i], less);
                                v[2 * r + 1] = fma_f16x2(y & 0x00F000F0u, mult[r][i], less);
                                v[4 + 2 * r] = fma_f16x2(y >> 4 & 0x00F000F0u, mult[r][i], less);
                                v[4 + 2 * r + 1] = fma_f16x2(y >> 8 & 0x00F000F0u, mult[r][i], less);
                            }
                            tmem_store_fragments2(tmem + ((32 * w + 16 * cc) << 16) + Sh::kKCol + buf * (D / 2) + 16 * i, v);
                        }
                    }
                    if (lane == 0) s_absent[n & 3u][w] = (uint8_t)missing;
                    tmem_wait_stores();
                    tmem_fence_before();
                    arrive(&bars.k_full[buf]);
                    if (lane == 0) mbar_arrive(&bars.raw_free[stage]);
                }
            }
        };
        role();
    } else if (warp < Sh::kLoad) {
        // ======== V: the words of 32 channels, all cells ========
        fewer_registers<Sh::kCellRegs>();
        const uint32_t w = warp % 4, set = (warp - Sh::kVWarp) / 4, x = lane % 4, c8 = lane / 4;
        const uint32_t i = c8 % G, gg = D == 128 ? 2 * w + c8 / G : (4 * w + c8 / G) & 7u;
        const bool has = D == 128 || w < 2;
        auto role = [&]() {
            uint32_t n = 0, seg = 0, stage = 0, phase = 0;
            Segment s;
            for (Wk wk = walk; wk.next(s); seg++) {
                for (uint32_t t = s.r0; t < s.r1; t++, n++, step(stage, phase)) {
                    const uint32_t buf = n % Sh::kV, par = n / Sh::kV & 1u;
                    if ((n & 1u) != set) continue;
                    if (!wait(&bars.raw_full[stage], phase)) return;
                    if (!wait(&bars.pv[buf], par ^ 1u)) return;
                    tmem_fence_after();
                    const uint8_t* raw = smem + Sh::kRing + stage * Sh::kStageBytes;
                    // A tile that ends the sequence, or holds nodes or a page
                    // outside the pool, is looked at token by token.
                    const uint2 valid8 = *reinterpret_cast<const uint2*>(s_valid[stage]);
                    const bool plain = valid8.x == 0x10101010u && valid8.y == 0x10101010u && (t + 1) * kTile <= s.len;
                    if (has) {
                        const uint8_t* cell = raw + (x * G + i) * 4;
#pragma unroll 1
                        for (int c = 0; c < 8; c += 2, cell += 2 * Sh::kCell) {
                            uint32_t word[4], sc[4];  // cell c + k / 2, tokens 8 (k % 2) + 2 x and the next
#pragma unroll
                            for (int k = 0; k < 4; k++) {
                                const uint8_t* at = cell + (k >> 1) * Sh::kCell;
                                word[k] = *reinterpret_cast<const uint32_t*>(at + 2 * C::kV + ((k & 1) * 8 + gg) * (16 * G));
                                sc[k] = *reinterpret_cast<const uint32_t*>(at + 2 * C::kVScale + (k & 1) * (16 * G));
                            }
                            if (!plain) {
#pragma unroll 1
                                for (uint32_t h = 0; h < 8; h++) {
                                    const uint32_t k = h >> 1, tk = 8 * (k & 1) + 2 * x + (h & 1), cc = c + (k >> 1);
                                    const uint32_t token = t * kTile + 16 * cc + tk, half = 0xFFFFu << (16 * (h & 1));
                                    const uint32_t size = half & 0x7FFF7FFFu, inf = half & 0x7F807F80u, most = half & kMostScale;
                                    const uint32_t s0 = k == 0 ? sc[0] : k == 1 ? sc[1] : k == 2 ? sc[2] : sc[3];
                                    const bool there = tk < s_valid[stage][cc], off = there && token >= s.len && (s0 & size) > most;
                                    if (!there || off) {
                                        uint32_t now = s0 & ~half;
                                        if (off) {
                                            // Not finite: seen by some rows only, which get it at the end.
                                            // Finite, but not its sevenfold: the next smaller scale, as an
                                            // infinity would reach rows with a weight of 0.
                                            if ((s0 & size) < inf)
                                                now = (s0 & ~size) | most;
                                            else
                                                for (int q = 0; q < SG; q++) atomicOr(&s_nan[seg & 7u][q][i], 1ull << (token - s.len & 63u));
                                        }
#pragma unroll
                                        for (uint32_t y = 0; y < 4; y++)
                                            if (y == k) sc[y] = now;
                                    }
                                }
                            }
                            uint32_t lo[8], hi[8];
#pragma unroll
                            for (int k = 0; k < 4; k++) {
#pragma unroll
                                for (int e = 0; e < 4; e++) {
                                    // 128 + code is a bf16 number, less 136 exactly code - 8.
                                    (e < 2 ? lo : hi)[4 * (k >> 1) + 2 * (e & 1) + (k & 1)] =
                                        mul_bf16x2(sub_bf16x2((word[k] >> (4 * e) & 0x000F000Fu) | 0x43004300u, 0x43084308u), sc[k]);
                                }
                            }
                            const uint32_t at = tmem + (32 * w << 16) + Sh::kVCol + buf * 64 + 8 * c;
                            tmem_store_fragments2(at, lo);
                            tmem_store_fragments2(at + (16u << 16), hi);
                        }
                        tmem_wait_stores();
                    }
                    tmem_fence_before();
                    arrive(&bars.v_full[buf]);
                    if (lane == 0) mbar_arrive(&bars.raw_free[stage]);
                }
            }
        };
        role();
    } else {
        // One place for the warpgroup: its four warps have to come to the same instruction.
        fewer_registers<Sh::kOtherRegs>();
        if (warp == Sh::kLoad) {
            // ======== raw tiles into the ring: lane 8 k + j has cell j of tile k of four ========
            uint32_t n = 0;
            auto role = [&]() {
                Segment s;
                for (Wk wk = walk; wk.next(s);) {
                    auto page_of = [&](uint32_t t) {
                        const uint32_t tile = t + lane / 8, first = tile * kTile + lane % 8 * kCellTokens;
                        return tile < s.r1 && first < s.tokens ? p.table[(uint64_t)s.b * p.table_width + (first >> lg_page)] : 0;
                    };
                    int32_t page = page_of(s.r0);
                    for (uint32_t t4 = s.r0; t4 < s.r1; t4 += 4) {
                        const int32_t next_page = page_of(t4 + 4);
                        const uint32_t tile = t4 + lane / 8, first = tile * kTile + lane % 8 * kCellTokens;
                        uint32_t tokens = 0;
                        const uint8_t* src = nullptr;
                        if (tile < s.r1 && first < s.tokens) {
                            if ((uint32_t)page < p.pool.pages) {
                                tokens = min(s.tokens - first, kCellTokens);
                                src = p.pool.base + cell_offset<D>(p.pool, (uint32_t)page, s.head, first & ((1u << lg_page) - 1u));
                            } else if (p.status) {
                                atomicMax(p.status, kStatusInvalid);
                            }
                        }
                        const uint32_t held = __ballot_sync(0xFFFFFFFFu, tokens != 0);
                        for (uint32_t k = 0; k < 4 && t4 + k < s.r1; k++, n++) {
                            const uint32_t stage = n % RS;
                            if (!wait(&bars.raw_free[stage], (n / RS & 1u) ^ 1u)) return;
                            const bool my = lane / 8 == k;
                            if (my) s_valid[stage][lane % 8] = (uint8_t)tokens;
                            __syncwarp();
                            if (lane == 0) mbar_arrive_expect_tx(&bars.raw_full[stage], __popc(held >> (8 * k) & 0xFFu) * Sh::kCell);
                            __syncwarp();
                            if (my && tokens)
                                bulk_g2s(smem + Sh::kRing + stage * Sh::kStageBytes + lane % 8 * Sh::kCell, src, Sh::kCell, &bars.raw_full[stage]);
                        }
                        page = next_page;
                    }
                }
            };
            role();
            // Copies still under way must land before the block gives its shared
            // memory back.
            for (uint32_t k = n > RS ? n - RS : 0; k < n; k++) mbar_wait(&bars.raw_full[k % RS], k / RS & 1u, p.wait_limit_ns);
        } else if (warp == Sh::kMma) {
            // ======== matrix instructions: one thread waits and issues ========
            if (one_lane()) {
                auto role = [&]() {
                    uint32_t n = 0, seg = 0;
                    bool pending = false, first = false, last = false;  // O of the tile before
                    uint32_t p_seg = 0, p_shape = 0;
                    auto product = [&](uint32_t m) {
                        const uint32_t buf = m & 1u, v = m % Sh::kV;
                        if (!wait_alone(&bars.v_full[v], m / Sh::kV & 1u) || !wait_alone(&bars.p_full[buf], m >> 1 & 1u)) return false;
                        if (first && !wait_alone(&bars.o_free, (p_seg & 1u) ^ 1u)) return false;
                        tmem_fence_after();
                        const uint32_t a = tmem + Sh::kVCol + v * 64, d = tmem + Sh::kOCol;
                        const SmemOperand w(smem_u32(smem + Sh::kP) + buf * Sh::kPBytes, 128, kTile * 16);
                        if (first)
                            mma_tmem_smem<false>(d, a, w, 0, p_shape);
                        else
                            mma_tmem_smem<true>(d, a, w, 0, p_shape);
    #pragma unroll
                        for (int k = 1; k < 8; k++) mma_tmem_smem<true>(d, a + 8 * k, w, 256 * k, p_shape);
                        mma_commit(&bars.pv[v]);
                        if (last) {
                            mma_commit(&bars.o_full);
                            mbar_arrive(&bars.o_full);
                        }
                        return true;
                    };
                    Segment s;
                    for (Wk wk = walk; wk.next(s); seg++) {
                        const uint32_t cols = (s.rows + Sh::kCols - 1) / Sh::kCols * Sh::kCols;  // of whole groups
                        const uint32_t shape = mma_shape(false, false, cols);
                        if (!wait_alone(&bars.q_full[seg & 1u], seg >> 1 & 1u)) return;
                        const SmemOperand q_op(smem_u32(smem) + (seg & 1u) * Sh::kQBytes, N * 16, 128);
                        for (uint32_t t = s.r0; t < s.r1; t++, n++) {
                            const uint32_t buf = n & 1u;
                            // S of tile n - 2 has been read: O of that tile, issued
                            // before this, has waited for its weights.
                            if (!wait_alone(&bars.k_full[buf], n >> 1 & 1u)) return;
                            tmem_fence_after();
                            const uint32_t d = tmem + Sh::kSCol + buf * N, a = tmem + Sh::kKCol + buf * (D / 2);
                            mma_tmem_smem<false>(d, a, q_op, 0, shape);
    #pragma unroll
                            for (int k = 1; k < D / 16; k++) mma_tmem_smem<true>(d, a + 8 * k, q_op, 2 * k * (N * 16), shape);
                            mma_commit(&bars.s_full[buf]);
                            mbar_arrive(&bars.s_full[buf]);
                            if (t + 1 == s.r1) mma_commit(&bars.q_free[seg & 1u]);
                            if (pending && !product(n - 1)) return;
                            pending = true;
                            first = t == s.r0, last = t + 1 == s.r1;
                            p_seg = seg, p_shape = mma_shape(true, true, cols);
                        }
                    }
                    if (pending) product(n - 1);
                };
                role();
                // Nothing is under way when tensor memory is given back.
                mma_commit(&bars.end);
                mbar_wait(&bars.end, 0, p.wait_limit_ns);
            }
            __syncwarp();
        } else {
            // ======== queries: rows as they are into shared memory, then a lane a row,
            // or where there are fewer than 64 rows, kParts lanes of both warps ========
            const uint32_t wq = warp - Sh::kQuery, c = N == 64 ? 32 * wq + lane : lane % N;
            const uint32_t part = N == 64 ? 0u : N == 32 ? wq : 2 * wq + lane / 16;
            uint32_t seg = 0;
            bool asked = false;
            auto role = [&]() {
                Segment s;
                uint8_t* raw = smem + Sh::kRows + c * Sh::kRow;
                for (Wk wk = walk; wk.next(s); seg++) {
                    if (!wait(&bars.q_free[seg & 1u], (seg >> 1 & 1u) ^ 1u)) return;
                    // Both warps have read the rows of the segment before.
                    if (Sh::kParts > 1 && seg && !wait(&bars.q_full[(seg - 1) & 1u], (seg - 1) >> 1 & 1u)) return;
                    const bool there = c < s.rows;
                    const uint32_t r = s.row0 + c, node = there ? r / p.group : 0u;
                    const uint16_t* src = p.q + (int64_t)s.b * p.q_seq + (int64_t)node * p.q_node + (int64_t)(s.head * p.group + r - node * p.group) * p.q_head;
                    if (p.q_vec) {
                        const bool mine = there && (N == 64 || (lane < N && lane % 2 == wq));
                        const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, mine)) * (2 * D);
                        if (lane == 0) mbar_arrive_expect_tx(&bars.q_raw[wq], bytes);
                        __syncwarp();
                        asked = true;
                        if (mine) bulk_g2s(raw, src, 2 * D, &bars.q_raw[wq]);
                    } else if (there) {
    #pragma unroll 1
                        for (uint32_t k = 0; k < D; k++) reinterpret_cast<uint16_t*>(raw)[k] = src[k];
                    }
                    const bool sees = N == 64 || wq == 1;  // this warp's to find out
                    const uint64_t mask = there && sees ? p.mask[(uint64_t)s.b * p.nodes + node] : 0ull;
                    // Rows' bits of nodes into nodes' bits of rows, lane k the node k.
    #pragma unroll 1
                    for (uint32_t k0 = 0; sees && k0 < s.tokens - s.len; k0 += 32) {
                        const uint32_t bits = (uint32_t)(mask >> k0);
                        uint32_t mine = 0;
    #pragma unroll 8
                        for (uint32_t k = 0; k < 32; k++) {
                            const uint32_t seen = __ballot_sync(0xFFFFFFFFu, bits >> k & 1u);
                            mine = lane == k ? seen : mine;
                        }
                        s_seen[seg & 7u][N == 64 ? wq : 0u][k0 + lane] = mine;
                    }
                    if (p.q_vec && (!wait(&bars.q_raw[wq], seg & 1u) || (Sh::kParts > 1 && !wait(&bars.q_raw[wq ^ 1u], seg & 1u)))) return;
                    asked = false;
                    {
                        constexpr uint32_t kHalves = N == 16 ? 2 : 1;
                        uint32_t top = 0;
    #pragma unroll 4
                        for (uint32_t k = 0; k < D / 8 / kHalves; k++) {
                            if (!there) continue;
                            const uint4 v = *reinterpret_cast<const uint4*>(raw + 16 * (k + (kHalves == 2 ? lane / 16 * (D / 16) : 0u)));
                            const uint32_t m = max_u16x2(max_u16x2(v.x & 0x7F807F80u, v.y & 0x7F807F80u), max_u16x2(v.z & 0x7F807F80u, v.w & 0x7F807F80u));
                            top = max(top, max(m & 0xFFFFu, m >> 16));
                        }
                        if (kHalves == 2) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
                        const bool fine = top != 0x7F80u;
                        int up = max((int)(top >> 7) - 127, kMinExp);
                        const int most = (int)__reduce_max_sync(0xFFFFFFFFu, (uint32_t)(top && fine ? up + 128 : 0)) - 128;
                        const int least = (int)__reduce_min_sync(0xFFFFFFFFu, (uint32_t)(top && fine ? up + 128 : 1000)) - 128;
                        // Rows that are not finite have a factor of their own.
                        const bool common = __all_sync(0xFFFFFFFFu, fine) && most - least <= kShareExp;
                        if (common) up = max(most, kMinExp);
                        const float unit = copysignf(pow2(14 - up), p.scale_log2);
                        uint8_t* dst = smem + (seg & 1u) * Sh::kQBytes + c * 16;
    #pragma unroll 2
                        for (uint32_t k = part * (D / 8 / Sh::kParts); k < (part + 1) * (D / 8 / Sh::kParts); k++) {
                            const uint4 u = *reinterpret_cast<const uint4*>(raw + 16 * k);
                            const uint32_t v[4] = {u.x, u.y, u.z, u.w};
                            float f[8];
    #pragma unroll
                            for (int j = 0; j < 4; j++) {
                                f[2 * j] = there && fine ? __uint_as_float(v[j] << 16) * unit : 0.f;
                                f[2 * j + 1] = there && fine ? __uint_as_float(v[j] & 0xFFFF0000u) * unit : 0.f;
                            }
                            // Channels 32 i + 8 q + 4 h + e are k 32 i + 16 (e / 2) + 4 q + 2 (e % 2) + h.
                            uint8_t* to = dst + (4 * (k / 4) + k % 4 / 2) * (N * 16) + k % 2 * 8;
                            *reinterpret_cast<uint2*>(to) = make_uint2(pack_f16(f[0], f[4]), pack_f16(f[1], f[5]));
                            *reinterpret_cast<uint2*>(to + 2 * (N * 16)) = make_uint2(pack_f16(f[2], f[6]), pack_f16(f[3], f[7]));
                        }
                        const float rf = ldexpf(fabsf(p.scale_log2), up - 4);
                        if (part == 0) s_rf[seg & 3u][c] = !there ? 0.f : fine ? rf : __int_as_float(0x7FC00000);
                        if (lane == 0 && (N == 64 || wq == 0)) s_common[seg & 3u][N == 64 ? wq : 0u] = common ? rf : -1.f;
                    }
                    fence_async_smem();
                    arrive(&bars.q_full[seg & 1u]);
                }
            };
            if (wq < Sh::kQueries) role();
            // As with the ring.
            if (asked) mbar_wait(&bars.q_raw[wq], seg & 1u, p.wait_limit_ns);
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == Sh::kMma) tmem_free(tmem, 512);
    if (warp < Sh::kSoftmax && s_dead) {
        // Rows of all items that this block has a part of are NaN.
        if (tid == 0 && p.status) atomicMax(p.status, kStatusTimeout);
        const float nan = __int_as_float(0x7FC00000);
        Segment s;
        for (Wk w = walk; w.next(s);) {
            const uint32_t slot = 2 * blockIdx.x + (s.starts ? 1u : 0u);
            for (uint32_t k = tid; k < s.rows * kTile; k += 32 * Sh::kSoftmax) {
                const uint32_t c = k / kTile, ch = k % kTile, r = s.row0 + c, node = r / p.group, h = s.head * p.group + r % p.group;
                if (s.starts && s.ends) {
                    if (ch < D) p.out[(int64_t)s.b * p.out_seq + (int64_t)node * p.out_node + (int64_t)h * p.out_head + ch] = 0x7FC0;
                    if (ch == 0 && p.lse) p.lse[((uint64_t)s.b * p.nodes + node) * q_heads + h] = nan;
                } else {
                    p.part_o[((uint64_t)slot * N + c) * kTile + ch] = nan;
                    if (ch == 0) *reinterpret_cast<float2*>(p.part_ml + ((uint64_t)slot * N + c) * 2) = make_float2(0.f, nan);
                }
            }
            if (s.starts && !s.ends && tid == 0) {
                p.meta[4 * blockIdx.x + 1] = (int32_t)s.item;
                p.meta[4 * blockIdx.x + 2] = (int32_t)((s.rest + share - 1) / share);
                p.meta[4 * blockIdx.x + 3] = (int32_t)(s.tokens - s.len);
                p.meta[4 * blockIdx.x] = (int32_t)s.b;
            }
        }
    }
}

// Joins the partial sums of the item that block blockIdx.x of the first kernel
// started and did not end: its own, then those of the next blocks.  A warp has a
// row, a lane four of O^T's; all of a kernel's blocks run at once (4 sequences of
// 32,768 tokens, 64 nodes: 4.8 us; a thread for each channel 9.9).
template <int D, int N>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const TreeParams p) {
    wait_for_previous();
    const int4 meta = *reinterpret_cast<const int4*>(p.meta + 4 * blockIdx.x);
    const int32_t b = meta.x;
    if (b < 0) return;
    const uint32_t item = (uint32_t)meta.y, count = (uint32_t)meta.w;
    const int more = meta.z;
    const uint32_t tiles = (count * p.group + N - 1) / N, head = item / tiles, row0 = item % tiles * N;
    const uint32_t rows = min((uint32_t)N, count * p.group - row0), q_heads = p.pool.heads * p.group;
    const uint32_t lane = threadIdx.x % 32, c = blockIdx.y * (kJoinThreads / 32) + threadIdx.x / 32;
    if (c >= rows) return;
    auto slot = [&](int k) { return (uint64_t)(k == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + k)) * N + c; };
    // Each step's reference is the largest so far, so that the loads of all
    // steps are under way together.
    float top = kNone, l = 0.f, o[4] = {};
#pragma unroll 4
    for (int k = 0; k <= more; k++) {
        const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * slot(k));
        const float4 v = *reinterpret_cast<const float4*>(p.part_o + slot(k) * kTile + 4 * lane);
        const float to = fmaxf(top, ml.x), f = exp2_fast(top - to), f2 = exp2_fast(ml.x - to);
        l = fmaf(f2, ml.y, l * f);
        o[0] = fmaf(f2, v.x, o[0] * f), o[1] = fmaf(f2, v.y, o[1] * f);
        o[2] = fmaf(f2, v.z, o[2] * f), o[3] = fmaf(f2, v.w, o[3] * f);
        top = to;
    }
    const uint32_t r = row0 + c, node = r / p.group, h = head * p.group + r % p.group;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t* out = p.out + (int64_t)b * p.out_seq + (int64_t)node * p.out_node + (int64_t)h * p.out_head;
#pragma unroll
    for (uint32_t j = 0; j < 4; j++)
        if (4 * lane + j < D) out[channel_of<D>(4 * lane + j)] = (uint16_t)bf16_bits(o[j] * inv);
    if (lane == 0 && p.lse)
        p.lse[((uint64_t)b * p.nodes + node) * q_heads + h] = l == 0.f ? kNegInf : (top + log2f(l)) * 0.6931471805599453f;
}

template <int D, int N>
cudaError_t launch(const TreeParams& p, cudaStream_t s) {
    using Sh = Shape<D, N>;
    int sms = 0, per_sm = 0;
    cudaError_t err = kernel_fit(reinterpret_cast<const void*>(tree_kernel<D, N>), Sh::kThreads, Sh::kBytes, &sms, &per_sm);
    if (err != cudaSuccess) return err;
    // What the warps ask for beyond the registers of the launch would never come.
    static const int regs = [] {
        cudaFuncAttributes a{};
        return cudaFuncGetAttributes(&a, tree_kernel<D, N>) == cudaSuccess ? a.numRegs : 0;
    }();
    if (regs != Sh::kRegs) return cudaErrorLaunchOutOfResources;
    err = launch_dependent(tree_kernel<D, N>, dim3((uint32_t)sms), dim3(Sh::kThreads), Sh::kBytes, s, p);
    if (err != cudaSuccess) return err;
    return launch_dependent(tree_join_kernel<D, N>, dim3((uint32_t)sms, N * 32 / kJoinThreads), dim3(kJoinThreads), 0, s, p);
}

template <int D>
cudaError_t launch_dim(const TreeParams& p, cudaStream_t s) {
    switch (tree_item_rows((uint64_t)p.nodes * p.group)) {
        case 16:
            return launch<D, 16>(p, s);
        case 32:
            return launch<D, 32>(p, s);
        default:
            return launch<D, 64>(p, s);
    }
}

}  // namespace

// Rows of an item: of 64, 1,050 of a tile's 2,100 clocks were left with 16, so
// that fewer rows take the smaller kernels.  128 at once need softmax registers
// that are not there: 4 sequences of 32,768, 64 nodes took 229 us with them, 221
// with 64 at that time, the ragged batch 59 instead of 53.
uint32_t tree_item_rows(uint64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

cudaError_t launch_attend_tree(const TreeParams& p, cudaStream_t s) {
    return p.pool.dim == 64 ? launch_dim<64>(p, s) : launch_dim<128>(p, s);
}

}  // namespace sz
