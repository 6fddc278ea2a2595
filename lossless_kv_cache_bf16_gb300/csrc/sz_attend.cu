// sz_attend.cu -- attention of one query token per sequence over the 4-bit
// paged cache: o = sum_j p_j v_j / sum_j p_j, p_j = exp(scale q.k_j - max).
//
// What bounds it: each token and kv head costs 9 D / 8 bytes of cache and
// 4 D flops per query head, so with up to 16 query heads per kv head it is a
// stream of the cache from HBM as long as unpacking keeps up.
//
// Matrix instructions.  Both products use mma.sync m16n8k16 in bf16: with 8
// or 16 query heads per item the M = 128 rows of a tcgen05 tile would be at
// least 7/8 padding, and the legacy rate (measured: 970 instructions per SM
// and us) is twice what the stream needs.  Codes enter the matrix unit almost
// without conversion: a code q in the low mantissa bits of a bf16 word whose
// other bits are zero is the (subnormal or first normal) number q * 2^-133,
// and in the next four bits 16 q * 2^-133, so that one AND turns a word of
// eight codes into a pair of operands.  The powers of two are undone in fp32;
// queries are scaled to 2^120 and weights by 2^92 beforehand (exactly), which
// keeps products normal fp32 numbers.
//
//   S = K Q^T   A = K codes (row = token), B = queries (column = head).  Each
//               group of 32 channels sums into its own accumulator; -8 sum(q)
//               takes the codes' offset of 8 away, and the group's scale
//               multiplies the rest.
//   O = V^T P   A = V codes less 8 (one packed add, exact; row = channel),
//               B = weight times the group's scale, rounded to bf16 once
//               (column = head), turned from S's layout into B's by movmatrix.
//
// Work split.  The list of (sequence, kv head, unit of 32 tokens), with
// kItemCost more entries per (sequence, kv head) for its fixed cost, is cut
// into equal runs, one per warp, whatever the lengths.  A warp needs nobody
// else: it has its own ring of bulk copies, its own running maximum and sums,
// and writes the rows of an item that it holds whole.  Pieces of an item are
// joined once per block in shared memory, pieces over several blocks by a
// second kernel, both in list order: results do not depend on timing.  Few
// short sequences take one block per item and no second kernel (launch()).
//
// Measured: each 8 sequences of 32,768 tokens more (4 kv heads of 128, 28
// query heads, 151 MB) take 26 us, 5.7 TB/s or 85% of the copy rate, after
// 13 us that any such call takes (launch, lengths, first copies, joins).  About
// 650 instructions per 32 tokens and warp; 12 warps per SM with 168 registers
// are faster than 16 with 128 (62 against 64 us for 16 such sequences), and
// the scales' and codes' unpacking keeps the integer pipe half busy.
#include <cfloat>
#include <type_traits>

#include "sz_cache.cuh"
#include "sz_params.h"
#include "sz_pipeline.cuh"

namespace sz {
namespace {

constexpr int kPartHeads = 16;  // head rows of a partial result
constexpr float kNegInf = -__builtin_huge_valf();
// Weights are kept times 2^92: a weight (at most 2^8, see below) times a scale
// up to 2^26 is still finite, and a product down to 2^-85 still has all bits
// after the factor 2^-133 of the codes.
constexpr float kWeightShift = 92.f;
// Entries that stand for an item's fixed cost (its queries, its results).
// Main kernel on 64 ragged sequences up to 8,192 tokens: 32.5 us with 1, 28.0
// with 2, 29.6 with 3.
constexpr uint32_t kItemCost = 2;
// List entries of a warp, at least.  One sequence of 777 tokens cut into runs:
// 13.4 us with 4, 9.9 with 2, 8.4 with 1 (main kernel).
constexpr uint32_t kMinShare = 1;

template <int D, int NT>
struct Shape {
    // As many warps as their registers allow without spilling into the loop:
    // 168 each with 8 heads, 255 with 16.
    static constexpr int kWarps = NT == 1 ? 12 : 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kHeads = 8 * NT;
    static constexpr uint32_t kUnitBytes = 2 * Cell<D>::kBytes;
    // About 14 KB under way per warp, 166 KB per SM.
    static constexpr int kStages = (NT == 1 ? 3 : 4) * (D == 64 ? 2 : 1);
    static constexpr int kRow = D + 4;  // floats of a head's row of a piece, padded against bank conflicts
    static constexpr uint32_t kPieceBytes = 4 * kHeads * kRow + 8 * kHeads;
    static constexpr uint32_t kRingBytes = kStages * kUnitBytes;  // of a warp
    static constexpr uint32_t kPiece = kWarps * kRingBytes;
    static constexpr uint32_t kLen = kPiece + kWarps * kPieceBytes;
    static constexpr uint32_t kBar = kLen + 4u * kMaxBatch;
    static constexpr uint32_t kCount = kBar + 8u * kWarps * kStages;
    static constexpr uint32_t kBytes = kCount + 8u * kWarps * kStages;
    static_assert(kBytes + 1024 <= 232448, "shared memory of a block");
    static_assert(kPieceBytes <= kRingBytes, "a warp's last piece takes its ring's place");
};

// What a warp leaves for the join of its block.
struct Left {
    uint32_t first;       // bit 0: a piece that continues an item; bit 1: which ends it
    uint32_t last;        // 1: a piece that starts an item and does not end it
    uint32_t b, item;     // of the last piece
    uint32_t rest;        // list entries of that item after this warp's
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same into a fresh accumulator.
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Pairs of floats in one register pair: one instruction for two sums.
struct F2 {
    uint64_t v;
    __device__ __forceinline__ F2(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y)); }
    __device__ __forceinline__ void get(float& x, float& y) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
};
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(a.v) : "l"(a.v), "l"(b.v));
    return a;
}
// One of two packed bf16 as a float: sel is 0x1044 for the low one, 0x3244 for
// the high one.
__device__ __forceinline__ float scale_of(uint32_t w, uint32_t sel) { return __uint_as_float(prmt(w, 0u, sel)); }
// Transposes an 8 x 8 matrix of 16-bit values, of which lane 4 r + c holds
// columns 2 c and 2 c + 1 of row r.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// Codes less 8 in units of 2^-133 (low) and of 2^-129 (high nibbles).
__device__ __forceinline__ uint32_t low_less8(uint32_t w) { return add_bf16x2(w & 0x000F000Fu, 0x80088008u); }
__device__ __forceinline__ uint32_t high_less8(uint32_t w) { return add_bf16x2(w & 0x00F000F0u, 0x80808080u); }
// A reference to subtract from logits: 0 where there is no maximum yet.
__device__ __forceinline__ float or_zero(float m) { return m == kNegInf ? 0.f : m; }
// The factor that ends a row: 0 for a row without tokens (only those have the
// maximum -infinity), whose sums are 0.
__device__ __forceinline__ float inverse(float m, float l) { return m == kNegInf ? 0.f : 1.f / l; }

// N (2 or 4) consecutive words of shared memory.
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

// 64-bit division, in 32 bits where the numbers are that small.
__device__ __forceinline__ uint64_t divide(uint64_t a, uint64_t b) {
    return (a | b) >> 32 ? a / b : (uint32_t)a / (uint32_t)b;
}

// Entries of an item of a sequence of len tokens, 0 for an empty one.
__device__ __forceinline__ uint32_t entries(uint32_t len) {
    return len ? (len + kUnitTokens - 1) / kUnitTokens + kItemCost : 0u;
}

// A place in the list: sequence, item (kv head and tile of query heads) and
// entry of the item, of which the first kItemCost stand for its fixed cost;
// len[b] is sequence b's length.
struct Cursor {
    uint32_t b, item, at;
    __device__ __forceinline__ void next_item(uint32_t items, const uint32_t* len, uint32_t batch) {
        at = 0;
        if (++item == items) {
            item = 0;
            do {
                b++;
            } while (b < batch && len[b] == 0);
        }
    }
};

template <int D, int NT, bool LOGITS>
__global__ void __launch_bounds__(Shape<D, NT>::kThreads, 1) attend_kernel(const AttendParams p) {
    using Sh = Shape<D, NT>;
    using C = Cell<D>;
    constexpr int W = Sh::kWarps, kG = C::kGroups, kSteps = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    uint32_t* s_len = reinterpret_cast<uint32_t*>(smem + Sh::kLen);
    __shared__ uint64_t s_sum[W];
    __shared__ Left s_left[W];
    __shared__ uint32_t s_gave_up;
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u, g = lane >> 2, t = lane & 3u;
    const uint32_t items = p.pool.heads * p.tiles;
    const uint32_t lg_page = p.pool.lg_page;
    const uint64_t max_tokens = (uint64_t)p.table_width << lg_page;
    const uint32_t q_heads = p.pool.heads * p.group;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sh::kBar) + warp * Sh::kStages;
    uint32_t* counts = reinterpret_cast<uint32_t*>(smem + Sh::kCount) + warp * Sh::kStages * 2;
    uint8_t* ring = smem + warp * Sh::kRingBytes;
    if (lane == 0) {
        for (int k = 0; k < Sh::kStages; k++) mbar_init(&bars[k], 1);
        fence_mbar_init();
        s_left[warp] = Left{0, 0, 0, 0, 0};
        if (warp == 0) s_gave_up = 0;
    }
    wait_for_previous();

    // List entries of every sequence's items, and each warp's share of all.
    // A length outside [0, table width * page tokens] counts as 0.
    uint32_t mine = 0;
    for (uint32_t b = tid; b < p.batch; b += Sh::kThreads) {
        const int32_t len = p.lens[b];
        const bool ok = len >= 0 && (uint64_t)len <= max_tokens;
        if (!ok && p.status && blockIdx.x == 0) atomicMax(p.status, kStatusInvalid);
        s_len[b] = ok ? (uint32_t)len : 0u;
        mine += ok ? entries((uint32_t)len) : 0u;
    }
    // A thread's sum stays below 2^30 (at most 8 sequences of 2^26 units), a
    // warp's need not stay below 2^32: its halves are added up apart.
    const uint64_t of_warp = __reduce_add_sync(0xFFFFFFFFu, mine & 0xFFFFu) +
                             ((uint64_t)__reduce_add_sync(0xFFFFFFFFu, mine >> 16) << 16);
    if (lane == 0) s_sum[warp] = of_warp;
    __syncthreads();
    uint64_t total = 0;
    for (int w = 0; w < W; w++) total += s_sum[w];
    total *= items;
    const uint64_t workers = (uint64_t)gridDim.x * W;
    const uint32_t share = (uint32_t)max(divide(total + workers - 1, workers), (uint64_t)kMinShare);
    const uint64_t u0 = min(((uint64_t)blockIdx.x * W + warp) * share, total);
    uint32_t n_run = (uint32_t)(min(u0 + share, total) - u0);
    // Rows of empty sequences are zero, with a log-sum of -infinity.
    for (uint32_t b = blockIdx.x; b < p.batch; b += gridDim.x) {
        if (s_len[b]) continue;
        for (uint32_t x = tid; x < q_heads * D; x += Sh::kThreads)
            p.out[(int64_t)b * p.out_seq + (int64_t)(x / D) * p.out_head + x % D] = 0;
        for (uint32_t h = tid; h < q_heads; h += Sh::kThreads)
            if (p.lse) p.lse[(uint64_t)b * q_heads + h] = kNegInf;
    }
    if (tid == 0) p.meta[4 * blockIdx.x] = -1;

    // ---- where this warp's run starts ----
    Cursor cur{0, 0, 0};
    if (p.whole_items) {
        // One item a block: its units in equal runs.
        cur.b = blockIdx.x / items, cur.item = blockIdx.x % items;
        const uint32_t units = (s_len[cur.b] + kUnitTokens - 1) / kUnitTokens, per = (units + W - 1) / W;
        const uint32_t from = min(warp * per, units);
        cur.at = kItemCost + from;
        n_run = min(per, units - from);
    } else if (n_run) {
        // The lengths, 32 at a time.
        uint64_t before = 0;
        for (uint32_t b0 = 0; b0 < p.batch; b0 += 32) {
            const uint32_t n = b0 + lane < p.batch ? entries(s_len[b0 + lane]) : 0u;
            uint32_t upto = n;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
                if (lane >= (uint32_t)d) upto += o;
            }
            const uint64_t end = before + (uint64_t)upto * items;
            const uint32_t past = __ballot_sync(0xFFFFFFFFu, end > u0);
            if (past) {
                const int who = __ffs(past) - 1;
                const uint32_t nb = __shfl_sync(0xFFFFFFFFu, n, who);
                const uint64_t at = u0 - (__shfl_sync(0xFFFFFFFFu, end, who) - (uint64_t)nb * items);
                const uint32_t item = (uint32_t)divide(at, nb);
                cur = Cursor{b0 + (uint32_t)who, item, (uint32_t)(at - (uint64_t)item * nb)};
                break;
            }
            before = __shfl_sync(0xFFFFFFFFu, end, 31);
        }
    }

    // ---- this warp's ring of units ----
    Cursor nxt = cur;
    uint32_t nxt_left = n_run;  // list entries from nxt on
    // Moves nxt to the next entry that is a unit.
    auto settle = [&]() {
        while (nxt_left) {
            if (nxt.at < kItemCost) {
                const uint32_t skip = min(kItemCost - nxt.at, nxt_left);
                nxt.at += skip;
                nxt_left -= skip;
            } else if (nxt.at >= entries(s_len[nxt.b])) {
                nxt.next_item(items, s_len, p.batch);
            } else {
                break;
            }
        }
    };
    // Units are looked up 16 at a time, within an item: lane j holds the
    // address and the token count of cell j.
    const uint8_t* src = nullptr;
    uint32_t tokens = 0, batch_mask = 0, batch_units = 0, batch_at = 0;
    uint32_t in_flight = 0;  // stages issued and not yet waited for
    bool left_out = false;   // tokens of pages outside the pool: without any, no item is empty
    auto look_up = [&]() {
        batch_at = batch_units = 0;
        settle();
        if (!nxt_left) return;
        batch_units = min(min(nxt_left, entries(s_len[nxt.b]) - nxt.at), 16u);
        const uint32_t first = (nxt.at - kItemCost) * kUnitTokens + lane * kCellTokens;
        const uint32_t len = s_len[nxt.b];
        tokens = 0;
        const bool held = lane < 2 * batch_units && first < len;
        if (held) {
            const int32_t page = p.table[(uint64_t)nxt.b * p.table_width + (first >> lg_page)];
            if ((uint32_t)page < p.pool.pages) {
                tokens = min(len - first, kCellTokens);
                src = p.pool.base +
                      cell_offset<D>(p.pool, (uint32_t)page, nxt.item / p.tiles, first & ((1u << lg_page) - 1u));
            } else if (p.status) {
                atomicMax(p.status, kStatusInvalid);
            }
        }
        batch_mask = __ballot_sync(0xFFFFFFFFu, tokens != 0);
        left_out |= __any_sync(0xFFFFFFFFu, held && tokens == 0);
        nxt.at += batch_units;
        nxt_left -= batch_units;
    };
    auto issue = [&](uint32_t stage) {
        if (batch_at == batch_units) look_up();
        if (batch_units == 0) return;
        const bool mine = (lane >> 1) == batch_at;
        if (lane == 0) mbar_arrive_expect_tx(&bars[stage], __popc(batch_mask >> (2 * batch_at) & 3u) * C::kBytes);
        if (mine) counts[2 * stage + (lane & 1u)] = tokens;
        __syncwarp();
        if (mine && tokens)
            bulk_g2s(ring + stage * Sh::kUnitBytes + (lane & 1u) * C::kBytes, src, C::kBytes, &bars[stage]);
        in_flight++;
        batch_at++;
    };
    // The query values of the item at `at`, this thread's share: the first
    // item's are asked for before the ring's copies, behind which they would
    // queue.
    uint32_t q_raw[NT][kG][4];
    auto fetch_q = [&](const Cursor& at) {
        const uint32_t tile = at.item % p.tiles, first = at.item / p.tiles * p.group + tile * Sh::kHeads;
#pragma unroll
        for (int n = 0; n < NT; n++) {
            const uint32_t h = g + 8 * n;
            const uint16_t* q = p.q + (int64_t)at.b * p.q_seq + (int64_t)(first + h) * p.q_head + 8 * t;
            const bool in = tile * Sh::kHeads + h < p.group;
#pragma unroll
            for (int i = 0; i < kG; i++) {
#pragma unroll
                for (int j = 0; j < 4; j++) q_raw[n][i][j] = 0;
                if (in && p.q_vec) {
                    const uint4 v = *reinterpret_cast<const uint4*>(q + 32 * i);
                    q_raw[n][i][0] = v.x, q_raw[n][i][1] = v.y, q_raw[n][i][2] = v.z, q_raw[n][i][3] = v.w;
                } else if (in) {
#pragma unroll
                    for (int j = 0; j < 4; j++) q_raw[n][i][j] = q[32 * i + 2 * j] | (uint32_t)q[32 * i + 2 * j + 1] << 16;
                }
            }
        }
    };
    if (n_run) fetch_q(cur);
#pragma unroll 1
    for (int k = 0; k < Sh::kStages; k++) issue(k);
    const uint32_t half_sel = g & 1u ? 0x3244u : 0x1044u;  // scales come in pairs of tokens
    uint32_t stage = 0, phase = 0;
    // 0 once a wait has given up: the rest is left out.  -1: the first will.
    int alive = blockIdx.x == p.stalled_block ? -1 : 1;

    for (uint32_t left = n_run; left;) {
        const uint32_t cost = entries(s_len[cur.b]), take = min(left, cost - cur.at);
        const uint32_t r0 = max(cur.at, kItemCost) - kItemCost, r1 = max(cur.at + take, kItemCost) - kItemCost;
        const uint32_t seq = cur.b, item = cur.item;
        left -= take;
        cur.at += take;
        if (cur.at == cost) cur.next_item(items, s_len, p.batch);
        if (r0 == r1) {
            if (left) fetch_q(cur);
            continue;
        }
        const bool starts = r0 == 0, ends = r1 == cost - kItemCost;
        const uint32_t kv_head = item / p.tiles, tile = item % p.tiles;
        const uint32_t head0 = kv_head * p.group + tile * Sh::kHeads;
        const uint32_t heads = min((uint32_t)Sh::kHeads, p.group - tile * Sh::kHeads);

        // ---- query operands ----
        uint32_t qb[kSteps][NT][2];
        float bias[kG][NT][2], mult[NT][2];  // of heads 2t and 2t + 1
#pragma unroll
        for (int n = 0; n < NT; n++) {
            uint32_t(&x)[kG][4] = q_raw[n];
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < kG; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) top = max(top, max(x[i][j] & 0x7FFFu, (x[i][j] >> 16) & 0x7FFFu));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            // Scaled by 2^(120 - up): the largest query value's exponent, or
            // that of the smallest normal number where all are smaller,
            // becomes 120.  Exact; the factor in two steps, since it can be
            // above 2^127.  The softmax scale's sign goes with the queries, so
            // that the largest sum is the largest logit.
            const int up = (int)max(top >> 7, 1u) - 127;
            const float up1 = copysignf(__uint_as_float((uint32_t)(min(120 - up, 120) + 127) << 23), p.scale_log2);
            const float up2 = __uint_as_float((uint32_t)(max(-up, 0) + 127) << 23);
            const float factor = ldexpf(fabsf(p.scale_log2), 13 + up);
            mult[n][0] = __shfl_sync(0xFFFFFFFFu, factor, 8 * t);
            mult[n][1] = __shfl_sync(0xFFFFFFFFu, factor, 8 * t + 4);
#pragma unroll
            for (int i = 0; i < kG; i++) {
                float v[8], sum = 0.f;
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const uint32_t bits = (j & 1) ? x[i][j >> 1] & 0xFFFF0000u : x[i][j >> 1] << 16;
                    v[j] = __uint_as_float(bits) * up1 * up2;
                    sum += v[j];
                }
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
                sum *= -__uint_as_float(1u << 19);  // 8 * 2^-133
                bias[i][n][0] = __shfl_sync(0xFFFFFFFFu, sum, 8 * t);
                bias[i][n][1] = __shfl_sync(0xFFFFFFFFu, sum, 8 * t + 4);
                // Operand e: channels (e, 4 + e) of this thread's 8; odd e
                // meets codes times 16.
                qb[2 * i][n][0] = pack_bf16(v[0], v[4]);
                qb[2 * i][n][1] = pack_bf16(v[1] * 0.0625f, v[5] * 0.0625f);
                qb[2 * i + 1][n][0] = pack_bf16(v[2], v[6]);
                qb[2 * i + 1][n][1] = pack_bf16(v[3] * 0.0625f, v[7] * 0.0625f);
            }
        }

        float o[NT][2 * kG][4];
        float m[NT][2], l[NT][2];  // of heads 2t and 2t + 1; l: this thread's share of the sum of weights
#pragma unroll
        for (int n = 0; n < NT; n++) {
            m[n][0] = m[n][1] = kNegInf;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int j = 0; j < 2 * kG; j++)
#pragma unroll
                for (int k = 0; k < 4; k++) o[n][j][k] = 0.f;
        }

#pragma unroll 1
        for (uint32_t unit = r0; unit < r1; unit++) {
            if (alive) {
                alive = __all_sync(0xFFFFFFFFu, alive > 0 && mbar_wait(&bars[stage], phase, p.wait_limit_ns));
                if (!alive) {
                    // The copies still under way must land before the block
                    // gives its shared memory back.
                    if (lane == 0) {
                        s_gave_up = 1;
                        if (p.status) atomicMax(p.status, kStatusTimeout);
                    }
                    for (uint32_t k = 0, st = stage, ph = phase; k < in_flight; k++) {
                        mbar_wait(&bars[st], ph, p.wait_limit_ns);
                        if (++st == (uint32_t)Sh::kStages) st = 0, ph ^= 1u;
                    }
                }
            }
            if (!alive) break;
            const uint8_t* u = ring + stage * Sh::kUnitBytes;
            const uint2 held = *reinterpret_cast<const uint2*>(counts + 2 * stage);  // tokens of the two cells
            auto take_unit = [&](auto partial) {
                constexpr bool PARTIAL = decltype(partial)::value;
                // S: s[n][c][2 r + k] is token 16 c + 8 r + g, head 8 n + 2 t + k.
                float s[NT][2][4];
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    const uint8_t* cell = u + c * C::kBytes;
                    uint32_t k0[kG], k1[kG], s0[kG], s1[kG];
                    lds_words<kG>(cell + (4 * g + t) * (4 * kG), k0);
                    lds_words<kG>(cell + (32 + 4 * g + t) * (4 * kG), k1);
                    lds_words<kG>(cell + 2 * C::kKScale + (g >> 1) * (4 * kG), s0);
                    lds_words<kG>(cell + 2 * C::kKScale + (4 + (g >> 1)) * (4 * kG), s1);
#pragma unroll
                    for (int n = 0; n < NT; n++)
#pragma unroll
                        for (int k = 0; k < 4; k++) s[n][c][k] = 0.f;
#pragma unroll
                    for (int i = 0; i < kG; i++) {
                        const uint32_t x0 = k0[i] >> 8, x1 = k1[i] >> 8;
                        const uint32_t a0 = k0[i] & 0x000F000Fu, a1 = k1[i] & 0x000F000Fu;
                        const uint32_t a2 = k0[i] & 0x00F000F0u, a3 = k1[i] & 0x00F000F0u;
                        const uint32_t e0 = x0 & 0x000F000Fu, e1 = x1 & 0x000F000Fu;
                        const uint32_t e2 = x0 & 0x00F000F0u, e3 = x1 & 0x00F000F0u;
                        const float f0 = scale_of(s0[i], half_sel), f1 = scale_of(s1[i], half_sel);
#pragma unroll
                        for (int n = 0; n < NT; n++) {
                            float d[4];
                            mma_bf16_first(d, a0, a1, a2, a3, qb[2 * i][n][0], qb[2 * i][n][1]);
                            mma_bf16(d, e0, e1, e2, e3, qb[2 * i + 1][n][0], qb[2 * i + 1][n][1]);
                            const F2 off(bias[i][n][0], bias[i][n][1]);
                            add2(F2(d[0], d[1]), off).get(d[0], d[1]);
                            add2(F2(d[2], d[3]), off).get(d[2], d[3]);
                            s[n][c][0] = fmaf(d[0], f0, s[n][c][0]);
                            s[n][c][1] = fmaf(d[1], f0, s[n][c][1]);
                            s[n][c][2] = fmaf(d[2], f1, s[n][c][2]);
                            s[n][c][3] = fmaf(d[3], f1, s[n][c][3]);
                        }
                    }
                }
                if constexpr (PARTIAL) {
#pragma unroll
                    for (int n = 0; n < NT; n++)
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            if (8 * (k >> 1) + g >= held.x) s[n][0][k] = kNegInf;
                            if (8 * (k >> 1) + g >= held.y) s[n][1][k] = kNegInf;
                        }
                }
                if (LOGITS) {
#pragma unroll
                    for (int n = 0; n < NT; n++) {
                        const uint32_t h = 8 * n + 2 * t;
                        float* row = p.logits + ((uint64_t)seq * q_heads + head0 + h) * max_tokens + (uint64_t)unit * kUnitTokens + g;
                        const bool both = (uint64_t)unit * kUnitTokens + kCellTokens < max_tokens;
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            if (h + (k & 1) >= heads) continue;
                            float* dst = row + (k & 1) * max_tokens + 8 * (k >> 1);
                            dst[0] = s[n][0][k] * mult[n][k & 1];
                            if (both) dst[kCellTokens] = s[n][1][k] * mult[n][k & 1];
                        }
                    }
                }
                // Running maximum, moved only when a head outgrows it by 2^8:
                // weights stay at most 2^(92 + 8).
                float top[NT][2];
                bool grow = false;
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        top[n][k] = fmaxf(fmaxf(s[n][0][k], s[n][0][k + 2]), fmaxf(s[n][1][k], s[n][1][k + 2]));
                        grow |= top[n][k] * mult[n][k] > m[n][k] + 8.f;
                    }
                if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
                    for (int n = 0; n < NT; n++) {
                        float f[2];
#pragma unroll
                        for (int k = 0; k < 2; k++) {
                            float x = top[n][k];
                            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
                            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
                            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
                            x *= mult[n][k];
                            const float to = x > m[n][k] + 8.f ? x : m[n][k];
                            f[k] = exp2_fast(m[n][k] - or_zero(to));
                            m[n][k] = to;
                            l[n][k] *= f[k];
                        }
#pragma unroll
                        for (int j = 0; j < 2 * kG; j++) {
                            o[n][j][0] *= f[0], o[n][j][1] *= f[1];
                            o[n][j][2] *= f[0], o[n][j][3] *= f[1];
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        const float ref = kWeightShift - or_zero(m[n][k]);
#pragma unroll
                        for (int c = 0; c < 2; c++)
#pragma unroll
                            for (int r = 0; r < 2; r++) {
                                float& x = s[n][c][2 * r + k];
                                x = exp2_fast(fmaf(x, mult[n][k], ref));
                                // Minus infinity times a factor of 0 is no number.
                                if (PARTIAL && 8 * r + g >= (c ? held.y : held.x)) x = 0.f;
                                l[n][k] += x;
                            }
                    }
                // O += V^T P, 16 tokens (one cell) at a time.
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    const uint8_t* cell = u + c * C::kBytes;
                    uint32_t w0[kG], w1[kG], v0[kG], v1[kG];
                    lds_words<kG>(cell + 2 * C::kVScale + (g >> 1) * (4 * kG), v0);
                    lds_words<kG>(cell + 2 * C::kVScale + (4 + (g >> 1)) * (4 * kG), v1);
                    lds_words<kG>(cell + 2 * C::kV + (g * 4 + t) * (4 * kG), w0);
                    lds_words<kG>(cell + 2 * C::kV + (32 + g * 4 + t) * (4 * kG), w1);
                    if constexpr (PARTIAL) {
                        // Scales of slots that hold nothing may be anything: zero
                        // times infinity must not reach the sums.
                        const uint32_t n = c ? held.y : held.x;
#pragma unroll
                        for (int i = 0; i < kG; i++) v0[i] = g < n ? v0[i] : 0u, v1[i] = 8 + g < n ? v1[i] : 0u;
                    }
#pragma unroll
                    for (int i = 0; i < kG; i++) {
                        const uint32_t x0 = w0[i] >> 8, x1 = w1[i] >> 8;
                        const uint32_t a0 = low_less8(w0[i]), a1 = high_less8(w0[i]), a2 = low_less8(w1[i]), a3 = high_less8(w1[i]);
                        const uint32_t e0 = low_less8(x0), e1 = high_less8(x0), e2 = low_less8(x1), e3 = high_less8(x1);
                        const float f0 = scale_of(v0[i], half_sel), f1 = scale_of(v1[i], half_sel);
#pragma unroll
                        for (int n = 0; n < NT; n++) {
                            const uint32_t b0 = transpose8x8(pack_bf16(s[n][c][0] * f0, s[n][c][1] * f0));
                            const uint32_t b1 = transpose8x8(pack_bf16(s[n][c][2] * f1, s[n][c][3] * f1));
                            mma_bf16(o[n][2 * i], a0, a1, a2, a3, b0, b1);
                            mma_bf16(o[n][2 * i + 1], e0, e1, e2, e3, b0, b1);
                        }
                    }
                }
            };
            if (held.x == kCellTokens && held.y == kCellTokens)
                take_unit(std::false_type{});
            else
                take_unit(std::true_type{});
            in_flight--;
            __syncwarp();
            issue(stage);
            if (++stage == (uint32_t)Sh::kStages) stage = 0, phase ^= 1u;
        }

        // ---- the item's rows, or a piece of them ----
        // Sums of weights are in units of 2^-92, code sums times 2^-41 (odd
        // channels 2^-37).
        const bool first_piece = !starts;
        float* piece = reinterpret_cast<float*>(first_piece ? smem + Sh::kPiece + warp * Sh::kPieceBytes : ring);
        if (!starts || !ends) __syncwarp();
#pragma unroll
        for (int n = 0; n < NT; n++) {
#pragma unroll
            for (int k = 0; k < 2; k++) {
                l[n][k] += __shfl_xor_sync(0xFFFFFFFFu, l[n][k], 4);
                l[n][k] += __shfl_xor_sync(0xFFFFFFFFu, l[n][k], 8);
                l[n][k] += __shfl_xor_sync(0xFFFFFFFFu, l[n][k], 16);
                // A row that lacks tokens for a wait that gave up is NaN.
                l[n][k] = alive ? l[n][k] * 2.0194839173657902e-28f : __int_as_float(0x7FC00000);
                // A row without tokens keeps the maximum -infinity; one whose
                // logits are all -infinity does not.
                if (!left_out || l[n][k] != 0.f) m[n][k] = fmaxf(m[n][k], -FLT_MAX);
            }
#pragma unroll
            for (int j = 0; j < 2 * kG; j++) {
                o[n][j][0] *= 2199023255552.f, o[n][j][1] *= 2199023255552.f;
                o[n][j][2] *= 137438953472.f, o[n][j][3] *= 137438953472.f;
            }
            const uint32_t h = 8 * n + 2 * t;
            if (starts && ends) {
                const float i0 = inverse(m[n][0], l[n][0]), i1 = inverse(m[n][1], l[n][1]);
                uint16_t* dst = p.out + (int64_t)seq * p.out_seq + (int64_t)(head0 + h) * p.out_head + 4 * g;
#pragma unroll
                for (int i = 0; i < kG; i++) {
                    const float(&a)[4] = o[n][2 * i];
                    const float(&b)[4] = o[n][2 * i + 1];
                    const uint2 r[2] = {make_uint2(pack_bf16(a[0] * i0, a[2] * i0), pack_bf16(b[0] * i0, b[2] * i0)),
                                        make_uint2(pack_bf16(a[1] * i1, a[3] * i1), pack_bf16(b[1] * i1, b[3] * i1))};
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        if (h + k >= heads) continue;
                        uint16_t* d = dst + k * p.out_head + 32 * i;
                        if (p.out_vec) {
                            *reinterpret_cast<uint2*>(d) = r[k];
                        } else {
                            d[0] = (uint16_t)r[k].x, d[1] = (uint16_t)(r[k].x >> 16);
                            d[2] = (uint16_t)r[k].y, d[3] = (uint16_t)(r[k].y >> 16);
                        }
                    }
                }
                if (g < 2 && h + g < heads) {
                    const uint64_t row = (uint64_t)seq * q_heads + head0 + h + g;
                    const float lse2 = g ? m[n][1] + log2f(l[n][1]) : m[n][0] + log2f(l[n][0]);
                    if (p.lse) p.lse[row] = lse2 * 0.6931471805599453f;
                    if (LOGITS) p.lse2[row] = lse2;
                }
            } else {
                if (g < 2) {
                    float2* ml = reinterpret_cast<float2*>(piece + Sh::kHeads * Sh::kRow);
                    ml[h + g] = g ? make_float2(m[n][1], l[n][1]) : make_float2(m[n][0], l[n][0]);
                }
#pragma unroll
                for (int i = 0; i < kG; i++) {
                    const float(&a)[4] = o[n][2 * i];
                    const float(&b)[4] = o[n][2 * i + 1];
                    float* row = piece + h * Sh::kRow + 32 * i + 4 * g;
                    *reinterpret_cast<float4*>(row) = make_float4(a[0], a[2], b[0], b[2]);
                    *reinterpret_cast<float4*>(row + Sh::kRow) = make_float4(a[1], a[3], b[1], b[3]);
                }
            }
        }
        if (lane == 0) {
            if (first_piece) {
                s_left[warp].first = ends ? 3u : 1u;
            } else if (!ends) {
                s_left[warp].last = 1;
                s_left[warp].b = seq;
                s_left[warp].item = item;
                s_left[warp].rest = cost - kItemCost - r1;
            }
        }
        if (left) fetch_q(cur);
    }

    // ---- join the pieces of items that several warps of this block hold ----
    __syncthreads();
    if (tid == 0) p.meta[4 * blockIdx.x + 3] = (int32_t)s_gave_up;
    auto first_of = [&](int w) { return reinterpret_cast<const float*>(smem + Sh::kPiece + w * Sh::kPieceBytes); };
    for (int w0 = -1; w0 < W; w0++) {
        // w0 = -1: the item that the block before this one left; else the one
        // that warp w0 started.
        if (w0 < 0 ? !(s_left[0].first & 1u) : !s_left[w0].last) continue;
        int w1 = w0 + 1;  // one past the last warp with a piece
        bool ends = false;
        while (w1 < W && !ends) ends = (s_left[w1++].first & 2u) != 0;
        const uint32_t seq = w0 < 0 ? 0u : s_left[w0].b, item = w0 < 0 ? 0u : s_left[w0].item;
        const uint32_t kv_head = item / p.tiles, tile = item % p.tiles;
        const uint32_t head0 = kv_head * p.group + tile * Sh::kHeads;
        const uint32_t heads = w0 < 0 ? (uint32_t)Sh::kHeads : min((uint32_t)Sh::kHeads, p.group - tile * Sh::kHeads);
        auto piece_of = [&](int w) { return w == w0 ? reinterpret_cast<const float*>(smem + w * Sh::kRingBytes) : first_of(w); };
        const uint32_t slot = 2 * blockIdx.x + (w0 < 0 ? 0u : 1u);
        for (uint32_t x = tid; x < heads * (D / 4); x += Sh::kThreads) {
            const uint32_t h = x / (D / 4), c = 4 * (x % (D / 4));
            float top = kNegInf;
            for (int w = max(w0, 0); w < w1; w++)
                top = fmaxf(top, reinterpret_cast<const float2*>(piece_of(w) + Sh::kHeads * Sh::kRow)[h].x);
            const float ref = or_zero(top);
            float l = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
            for (int w = max(w0, 0); w < w1; w++) {
                const float* piece = piece_of(w);
                const float2 ml = reinterpret_cast<const float2*>(piece + Sh::kHeads * Sh::kRow)[h];
                const float4 v = *reinterpret_cast<const float4*>(piece + h * Sh::kRow + c);
                const float f = exp2_fast(ml.x - ref);
                l = fmaf(f, ml.y, l);
                a[0] = fmaf(f, v.x, a[0]), a[1] = fmaf(f, v.y, a[1]), a[2] = fmaf(f, v.z, a[2]), a[3] = fmaf(f, v.w, a[3]);
            }
            if (w0 >= 0 && ends) {
                const float inv = inverse(top, l);
                uint16_t* dst = p.out + (int64_t)seq * p.out_seq + (int64_t)(head0 + h) * p.out_head + c;
#pragma unroll
                for (int k = 0; k < 4; k++) dst[k] = (uint16_t)bf16_bits(a[k] * inv);
                if (c == 0) {
                    const uint64_t row = (uint64_t)seq * q_heads + head0 + h;
                    const float lse2 = top + log2f(l);
                    if (p.lse) p.lse[row] = lse2 * 0.6931471805599453f;
                    if (LOGITS) p.lse2[row] = lse2;
                }
            } else {
                if (c == 0) *reinterpret_cast<float2*>(p.part_ml + (slot * kPartHeads + h) * 2) = make_float2(top, l);
                *reinterpret_cast<float4*>(p.part_o + ((uint64_t)slot * kPartHeads + h) * D + c) =
                    make_float4(a[0], a[1], a[2], a[3]);
            }
        }
        if (w0 >= 0 && !ends && tid == 0) {
            // The blocks after this one that hold the rest of the item.
            const uint64_t here = (uint64_t)(W - 1 - w0) * share, run = (uint64_t)W * share;
            p.meta[4 * blockIdx.x + 1] = (int32_t)item;
            p.meta[4 * blockIdx.x + 2] = (int32_t)((s_left[w0].rest - here + run - 1) / run);
            p.meta[4 * blockIdx.x] = (int32_t)seq;
        }
    }
}

// Joins the partial sums of the item that block blockIdx.x of the first
// kernel started and did not end: its own, then those of the next blocks.
template <int D>
__global__ void __launch_bounds__(256) attend_join_kernel(const AttendParams p, const uint32_t item_heads) {
    wait_for_previous();
    const int32_t b = p.meta[4 * blockIdx.x];
    // Whether any block has given up, in the first one's place.  The list ends
    // in the last block or before, so that it never has an item to join.
    if (p.weight && blockIdx.x == gridDim.x - 1) {
        int gave_up = 0;
        for (uint32_t k = threadIdx.x; k < gridDim.x; k += 256) gave_up |= p.meta[4 * k + 3];
        gave_up = __syncthreads_or(gave_up);
        if (threadIdx.x == 0) p.meta[3] = gave_up;
    }
    if (b < 0) return;
    const uint32_t item = (uint32_t)p.meta[4 * blockIdx.x + 1];
    const int more = p.meta[4 * blockIdx.x + 2];
    const uint32_t kv_head = item / p.tiles, tile = item % p.tiles;
    const uint32_t head0 = kv_head * p.group + tile * item_heads;
    const uint32_t heads = min(item_heads, p.group - tile * item_heads);
    const uint32_t q_heads = p.pool.heads * p.group;
    for (uint32_t x = threadIdx.x; x < heads * (D / 4); x += 256) {
        const uint32_t h = x / (D / 4), c = 4 * (x % (D / 4));
        auto slot = [&](int k) { return (uint64_t)(k == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + k)) * kPartHeads + h; };
        float top = kNegInf;
#pragma unroll 4
        for (int k = 0; k <= more; k++) top = fmaxf(top, p.part_ml[2 * slot(k)]);
        const float ref = or_zero(top);
        float l = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int k = 0; k <= more; k++) {
            const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * slot(k));
            const float4 v = *reinterpret_cast<const float4*>(p.part_o + slot(k) * D + c);
            const float f = exp2_fast(ml.x - ref);
            l = fmaf(f, ml.y, l);
            a[0] = fmaf(f, v.x, a[0]), a[1] = fmaf(f, v.y, a[1]), a[2] = fmaf(f, v.z, a[2]), a[3] = fmaf(f, v.w, a[3]);
        }
        const float inv = inverse(top, l);
        uint16_t* dst = p.out + (int64_t)b * p.out_seq + (int64_t)(head0 + h) * p.out_head + c;
#pragma unroll
        for (int k = 0; k < 4; k++) dst[k] = (uint16_t)bf16_bits(a[k] * inv);
        if (c == 0) {
            const uint64_t row = (uint64_t)b * q_heads + head0 + h;
            const float lse2 = top + log2f(l);
            if (p.lse) p.lse[row] = lse2 * 0.6931471805599453f;
            if (p.weight) p.lse2[row] = lse2;
        }
    }
}

// weight[slot] += sum over the kv head's query heads of the step's attention
// weight, from the logits that the first kernel kept.  A slot gets one
// addition per call and sequence; atomic, for pages that two sequences share.
// Adds nothing where a block of the first kernel has given up: its logits are
// missing, and the call can be made again with the weights as they were.
// flags: how many of meta's blocks say so, 1 where the join has gathered them.
__global__ void __launch_bounds__(256) attend_weight_kernel(const AttendParams p, const uint32_t flags) {
    wait_for_previous();
    const uint32_t b = blockIdx.z, kv_head = blockIdx.y;
    const int32_t len = p.lens[b];
    // Looked at before the first addition only, behind the loads for it.
    int gave_up = p.meta[3];
    if (flags > 1) {
        for (uint32_t k = threadIdx.x % 32; k < flags; k += 32) gave_up |= p.meta[4 * k + 3];
        gave_up = __any_sync(0xFFFFFFFFu, gave_up);
    }
    const uint64_t max_tokens = (uint64_t)p.table_width << p.pool.lg_page;
    if (len <= 0 || (uint64_t)len > max_tokens) return;
    const uint32_t q_heads = p.pool.heads * p.group;
    const uint64_t row0 = (uint64_t)b * q_heads + (uint64_t)kv_head * p.group;
    const float* lse2 = p.lse2 + row0;
    for (uint32_t tok = (blockIdx.x * 256 + threadIdx.x) * 4; tok < (uint32_t)len; tok += gridDim.x * 1024) {
        const int32_t page = p.table[(uint64_t)b * p.table_width + (tok >> p.pool.lg_page)];
        if ((uint32_t)page >= p.pool.pages) continue;
        const float* s = p.logits + row0 * max_tokens + tok;
        float w[4] = {0.f, 0.f, 0.f, 0.f};
        for (uint32_t h0 = 0; h0 < p.group; h0 += 8) {
            float4 x[8];
            float ref[8];
#pragma unroll
            for (uint32_t k = 0; k < 8; k++)
                if (h0 + k < p.group) x[k] = *reinterpret_cast<const float4*>(s + (h0 + k) * max_tokens), ref[k] = lse2[h0 + k];
#pragma unroll
            for (uint32_t k = 0; k < 8; k++) {
                if (h0 + k >= p.group) continue;
                w[0] += exp2_fast(x[k].x - ref[k]), w[1] += exp2_fast(x[k].y - ref[k]);
                w[2] += exp2_fast(x[k].z - ref[k]), w[3] += exp2_fast(x[k].w - ref[k]);
            }
        }
        if (gave_up) return;
        float* dst = p.weight + ((((uint64_t)(uint32_t)page * p.pool.heads + kv_head) << p.pool.lg_page) +
                                 (tok & ((1u << p.pool.lg_page) - 1u)));
        if (p.weight_vec && tok + 4 <= (uint32_t)len) {
            asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(dst), "f"(w[0]), "f"(w[1]), "f"(w[2]), "f"(w[3])
                         : "memory");
        } else {
#pragma unroll
            for (uint32_t k = 0; k < 4; k++)
                if (tok + k < (uint32_t)len) atomicAdd(dst + k, w[k]);
        }
    }
}

template <int D, int NT, bool LOGITS>
cudaError_t launch(const AttendParams& p, cudaStream_t s) {
    using Sh = Shape<D, NT>;
    int sms = 0, per_sm = 0;
    cudaError_t err = kernel_fit(reinterpret_cast<const void*>(attend_kernel<D, NT, LOGITS>), Sh::kThreads, Sh::kBytes, &sms, &per_sm);
    if (err != cudaSuccess) return err;
    const uint64_t tokens = (uint64_t)p.table_width << p.pool.lg_page;
    // No more items than SMs, and a table with room for only 3 units a warp:
    // one item a block, and no join across blocks to launch.  With 8 items
    // (32 heads over 8 of 128 channels) of 384 tokens 7.5 us against 10.2 in
    // runs, of 768 tokens 8.9 against 10.5, of 1,152 (3 units a warp) 10.6
    // against 10.2; of 1,536 11.8 against 10.5, but 12.3 against 15.5 with 128
    // items, so that far only where the items fill half the SMs.
    const uint64_t items = (uint64_t)p.batch * p.pool.heads * p.tiles;
    const uint64_t unit_a_warp = (uint64_t)Sh::kWarps * kUnitTokens;
    AttendParams q = p;
    q.whole_items = items <= (uint64_t)sms && tokens <= (2 * items >= (uint64_t)sms ? 4 : 3) * unit_a_warp;
    const uint32_t first_blocks = q.whole_items ? (uint32_t)items : (uint32_t)sms;
    err = launch_dependent(attend_kernel<D, NT, LOGITS>, dim3(first_blocks), dim3(Sh::kThreads), Sh::kBytes, s, q);
    if (err != cudaSuccess) return err;
    if (!q.whole_items) err = launch_dependent(attend_join_kernel<D>, dim3((uint32_t)sms), dim3(256), 0, s, p, (uint32_t)Sh::kHeads);
    if (err != cudaSuccess || !LOGITS) return err;
    const uint32_t blocks = (uint32_t)((tokens + 1023) / 1024);
    return launch_dependent(attend_weight_kernel, dim3(blocks < 1024 ? blocks : 1024, p.pool.heads, p.batch), dim3(256), 0, s, p,
                            q.whole_items ? first_blocks : 1u);
}

template <int D>
cudaError_t launch_dim(const AttendParams& p, cudaStream_t s) {
    // More than 8 query heads per kv head: items of 16, so that the cache is read
    // once for all of them (12 heads, 16 sequences of 32,768 tokens: 88 us;
    // twice 61 us with items of 8).
    if (p.group <= 8) return p.weight ? launch<D, 1, true>(p, s) : launch<D, 1, false>(p, s);
    return p.weight ? launch<D, 2, true>(p, s) : launch<D, 2, false>(p, s);
}

}  // namespace

cudaError_t attend_shape(uint32_t group, uint32_t* item_heads, uint32_t* blocks) {
    *item_heads = group <= 8 ? 8 : 16;
    int dev = -1, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    *blocks = (uint32_t)sms;
    return err;
}

cudaError_t launch_attend(const AttendParams& p, cudaStream_t s) {
    return p.pool.dim == 64 ? launch_dim<64>(p, s) : launch_dim<128>(p, s);
}

}  // namespace sz
