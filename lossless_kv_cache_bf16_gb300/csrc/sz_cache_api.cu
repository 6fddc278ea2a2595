// sz_cache_api.cu -- the C ABI of the serving operators of splitzip.h:
// argument checks, workspace layout and launches.  Host code only.
#include <cmath>
#include <cstdint>

#include <nvtx3/nvToolsExt.h>

#include "splitzip.h"
#include "sz_cache.h"
#include "sz_params.h"
#include "sz_rows.h"

namespace {

using namespace sz;

constexpr uint64_t kWaitLimitNs = 1000000000ull;  // bounded in-kernel waits for asynchronous copies: 1 s
constexpr uint32_t kNoBlock = 0xFFFFFFFFu;

struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// Whether `bytes` from a on and from b on share memory.
bool ranges_overlap(const void* a, const void* b, uint64_t bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return (x > y ? x - y : y - x) < bytes;
}
uint64_t align256(uint64_t x) { return (x + 255) & ~255ull; }

sz_status from_cuda(cudaError_t e) {
    switch (e) {
        case cudaSuccess:
            return SZ_OK;
        case cudaErrorNoKernelImageForDevice:
        case cudaErrorNoDevice:
        case cudaErrorInsufficientDriver:
            return SZ_ERR_UNSUPPORTED;
        default:
            return SZ_ERR_CUDA;
    }
}

bool page_tokens_ok(size_t t) { return t >= 16 && t <= 4096 && (t & (t - 1)) == 0; }
bool dim_ok(size_t d) { return d == 64 || d == 128; }
bool heads_ok(size_t h) { return h >= 1 && h <= 4096; }

bool pool_for(const void* d_pool, size_t pages, size_t heads, size_t dim, size_t page_tokens, CachePool* c) {
    if (!d_pool || !aligned(d_pool, 16) || pages == 0 || pages >= (1ull << 31)) return false;
    if (!dim_ok(dim) || !heads_ok(heads) || !page_tokens_ok(page_tokens)) return false;
    c->base = static_cast<uint8_t*>(const_cast<void*>(d_pool));
    c->pages = (uint32_t)pages;
    c->heads = (uint32_t)heads;
    c->dim = (uint32_t)dim;
    c->lg_page = 0;
    while ((1ull << c->lg_page) < page_tokens) c->lg_page++;
    return true;
}

// A block table: rows of `width` page ids; at most 2^31 - 1 tokens a row.
bool table_ok(const int32_t* d_table, size_t width, size_t page_tokens) {
    return d_table && aligned(d_table, 4) && width >= 1 && width < (1ull << 31) && width * page_tokens < (1ull << 31);
}

bool multiple(int64_t a, int64_t b, int64_t m) { return a % m == 0 && b % m == 0; }

sz_status clear_status(int* d_status, cudaStream_t stream) {
    return d_status ? from_cuda(cudaMemsetAsync(d_status, 0, sizeof(int), stream)) : SZ_OK;
}

// Rows, slots and pool of append and read.
bool rows_for(const void* d_k, int64_t k_token, int64_t k_head, const void* d_v, int64_t v_token, int64_t v_head,
              const int64_t* d_slots, size_t tokens, int* d_status, AppendParams* p) {
    if (tokens >= (1ull << 31) || (d_status && !aligned(d_status, 4))) return false;
    if (tokens > 0 && (!d_k || !d_v || !aligned(d_k, 2) || !aligned(d_v, 2) || !d_slots || !aligned(d_slots, 8))) return false;
    p->rows[0] = static_cast<uint16_t*>(const_cast<void*>(d_k));
    p->rows[1] = static_cast<uint16_t*>(const_cast<void*>(d_v));
    p->token_stride[0] = k_token, p->head_stride[0] = k_head;
    p->token_stride[1] = v_token, p->head_stride[1] = v_head;
    p->slots = d_slots;
    p->tokens = (uint32_t)tokens;
    p->status = d_status;
    p->vec = aligned(d_k, 16) && aligned(d_v, 16) && multiple(k_token, k_head, 8) && multiple(v_token, v_head, 8);
    return true;
}

// Attention workspace sections (bytes), each 256-byte aligned: [i32 x 4 per
// block][2 x 16 (maximum, sum) per block][2 x 16 x D sums per block], and with
// weights [f32 log-sum per query row][f32 logits per query row].
struct AttendWs {
    uint64_t ml, o, lse2, logits, end;
};
AttendWs attend_ws(uint64_t blocks, uint64_t dim, uint64_t rows, uint64_t max_tokens, bool weights) {
    AttendWs w{};
    w.ml = align256(16 * blocks);
    w.o = w.ml + align256(blocks * 2 * 16 * 2 * 4);
    w.lse2 = w.o + align256(blocks * 2 * 16 * dim * 4);
    w.logits = w.lse2 + (weights ? align256(4 * rows) : 0);
    w.end = w.logits + (weights ? align256(4 * rows * max_tokens) : 0);
    return w;
}

bool attend_sizes_ok(size_t batch, size_t q_heads, size_t kv_heads, size_t dim, uint64_t max_tokens) {
    if (!dim_ok(dim) || !heads_ok(kv_heads) || batch > kMaxBatch || q_heads == 0 || q_heads % kv_heads) return false;
    if (q_heads / kv_heads > 1024 || max_tokens == 0 || max_tokens >= (1ull << 31)) return false;
    // The list of work units stays well below 2^40, a warp's run below 2^32.
    return (uint64_t)batch * q_heads * ((max_tokens + 31) / 32) < (1ull << 38);
}

uint64_t evict_max_moves(uint64_t max_tokens) { return (max_tokens + 1) / 2; }
uint64_t evict_pairs_offset(uint64_t lists) { return align256(4 * lists); }

sz_status attend(const char* name, uint32_t stalled_block, const void* d_q, int64_t q_seq_stride, int64_t q_head_stride,
                 size_t batch, size_t q_heads, const void* d_pool, size_t pool_pages, size_t kv_heads, size_t head_dim,
                 size_t page_tokens, const int32_t* d_table, size_t table_width, const int32_t* d_lens, float scale,
                 void* d_out, int64_t out_seq_stride, int64_t out_head_stride, float* d_lse, float* d_weight, int* d_status,
                 void* d_ws, size_t ws_bytes, cudaStream_t stream) {
    const NvtxRange range(name);
    AttendParams p{};
    if (!pool_for(d_pool, pool_pages, kv_heads, head_dim, page_tokens, &p.pool)) return SZ_ERR_INVALID_ARG;
    if (batch > 0 && !table_ok(d_table, table_width, page_tokens)) return SZ_ERR_INVALID_ARG;
    const uint64_t max_tokens = batch > 0 ? (uint64_t)table_width * page_tokens : page_tokens;
    if (!attend_sizes_ok(batch, q_heads, kv_heads, head_dim, max_tokens) || !std::isfinite(scale)) return SZ_ERR_INVALID_ARG;
    if ((d_status && !aligned(d_status, 4)) || (d_lse && !aligned(d_lse, 4)) || (d_weight && !aligned(d_weight, 4)))
        return SZ_ERR_INVALID_ARG;
    if (batch > 0 && (!d_q || !d_out || !aligned(d_q, 2) || !aligned(d_out, 2) || !d_lens || !aligned(d_lens, 4) || !d_ws ||
                      !aligned(d_ws, 256)))
        return SZ_ERR_INVALID_ARG;
    if (batch == 0) return clear_status(d_status, stream);
    if (rows_overlap({d_out, out_seq_stride, out_head_stride, batch, q_heads}, {d_q, q_seq_stride, q_head_stride, batch, q_heads},
                     head_dim))
        return SZ_ERR_INVALID_ARG;
    uint32_t item_heads = 0, blocks = 0;
    const uint32_t group = (uint32_t)(q_heads / kv_heads);
    const cudaError_t err = attend_shape(group, &item_heads, &blocks);
    if (err != cudaSuccess) return from_cuda(err);
    const AttendWs w = attend_ws(blocks, head_dim, batch * q_heads, max_tokens, d_weight != nullptr);
    if (ws_bytes < w.end) return SZ_ERR_CAPACITY;
    const sz_status st = clear_status(d_status, stream);
    if (st != SZ_OK) return st;
    uint8_t* ws = static_cast<uint8_t*>(d_ws);
    p.q = static_cast<const uint16_t*>(d_q);
    p.q_seq = q_seq_stride, p.q_head = q_head_stride;
    p.out = static_cast<uint16_t*>(d_out);
    p.out_seq = out_seq_stride, p.out_head = out_head_stride;
    p.table = d_table;
    p.table_width = (uint32_t)table_width;
    p.lens = d_lens;
    p.batch = (uint32_t)batch;
    p.group = group;
    p.tiles = (group + item_heads - 1) / item_heads;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    p.lse = d_lse;
    p.weight = d_weight;
    p.status = d_status;
    p.wait_limit_ns = kWaitLimitNs;
    p.stalled_block = stalled_block;
    p.q_vec = aligned(d_q, 16) && multiple(q_seq_stride, q_head_stride, 8);
    p.weight_vec = aligned(d_weight, 16);
    p.out_vec = aligned(d_out, 8) && multiple(out_seq_stride, out_head_stride, 4);
    p.meta = reinterpret_cast<int32_t*>(ws);
    p.part_ml = reinterpret_cast<float*>(ws + w.ml);
    p.part_o = reinterpret_cast<float*>(ws + w.o);
    p.lse2 = reinterpret_cast<float*>(ws + w.lse2);
    p.logits = reinterpret_cast<float*>(ws + w.logits);
    return from_cuda(launch_attend(p, stream));
}

}  // namespace

extern "C" {

size_t sz_cache_page_bytes(size_t head_dim, size_t kv_heads, size_t page_tokens) {
    if (!dim_ok(head_dim) || !heads_ok(kv_heads) || !page_tokens_ok(page_tokens)) return 0;
    return kv_heads * page_tokens * (head_dim + head_dim / 8);
}

sz_status sz_qk_norm_rope(const void* d_q, int64_t q_token_stride, int64_t q_head_stride, size_t q_heads,
                          const void* d_k, int64_t k_token_stride, int64_t k_head_stride, size_t kv_heads,
                          size_t tokens, size_t head_dim, const void* d_q_weight, const void* d_k_weight, float eps,
                          const float* d_inv_freq, size_t rot_dim, int interleaved, const int32_t* d_positions,
                          void* d_q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, void* d_k_out,
                          int64_t k_out_token_stride, int64_t k_out_head_stride, cudaStream_t stream) {
    const NvtxRange range("sz_qk_norm_rope");
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return SZ_ERR_INVALID_ARG;
    if (q_heads > 65536 || kv_heads > 65536 || q_heads + kv_heads == 0 || tokens >= (1ull << 31)) return SZ_ERR_INVALID_ARG;
    if (rot_dim > head_dim || rot_dim % 16 || !(eps >= 0.f) || std::isinf(eps)) return SZ_ERR_INVALID_ARG;
    if (tokens == 0) return SZ_OK;
    if (rot_dim && (!d_inv_freq || !aligned(d_inv_freq, 4))) return SZ_ERR_INVALID_ARG;
    if (!d_positions || !aligned(d_positions, 4)) return SZ_ERR_INVALID_ARG;
    NormRopeParams p{};
    const void* in[2] = {d_q, d_k};
    void* out[2] = {d_q_out, d_k_out};
    const void* weight[2] = {d_q_weight, d_k_weight};
    const int64_t strides[2][4] = {{q_token_stride, q_head_stride, q_out_token_stride, q_out_head_stride},
                                   {k_token_stride, k_head_stride, k_out_token_stride, k_out_head_stride}};
    const size_t heads[2] = {q_heads, kv_heads};
    p.vec = 1;
    for (int w = 0; w < 2; w++) {
        p.heads[w] = (uint32_t)heads[w];
        if (heads[w] == 0) continue;
        if (!in[w] || !out[w] || !aligned(in[w], 2) || !aligned(out[w], 2) || !aligned(weight[w], 2)) return SZ_ERR_INVALID_ARG;
        p.in[w] = static_cast<const uint16_t*>(in[w]);
        p.out[w] = static_cast<uint16_t*>(out[w]);
        p.weight[w] = static_cast<const uint16_t*>(weight[w]);
        p.in_token[w] = strides[w][0], p.in_head[w] = strides[w][1];
        p.out_token[w] = strides[w][2], p.out_head[w] = strides[w][3];
        p.vec &= aligned(in[w], 16) && aligned(out[w], 16) && aligned(weight[w], 16) &&
                 multiple(strides[w][0], strides[w][1], 8) && multiple(strides[w][2], strides[w][3], 8);
    }
    // An output may be its input; no other rows may share memory with one.
    RowSet src[2], dst[2];
    for (int w = 0; w < 2; w++) {
        src[w] = {in[w], strides[w][0], strides[w][1], tokens, heads[w]};
        dst[w] = {out[w], strides[w][2], strides[w][3], tokens, heads[w]};
    }
    for (int w = 0; w < 2; w++) {
        if (!same_rows(dst[w], src[w]) && rows_overlap(dst[w], src[w], head_dim)) return SZ_ERR_INVALID_ARG;
        if (rows_overlap(dst[w], src[1 - w], head_dim)) return SZ_ERR_INVALID_ARG;
    }
    if (rows_overlap(dst[0], dst[1], head_dim)) return SZ_ERR_INVALID_ARG;
    p.inv_freq = d_inv_freq;
    p.positions = d_positions;
    p.tokens = (uint32_t)tokens;
    p.dim = (uint32_t)head_dim;
    p.rot = (uint32_t)rot_dim;
    p.interleaved = interleaved != 0;
    p.eps = eps;
    return from_cuda(launch_norm_rope(p, stream));
}

sz_status sz_cache_append(const void* d_k, int64_t k_token_stride, int64_t k_head_stride, const void* d_v,
                          int64_t v_token_stride, int64_t v_head_stride, size_t tokens, const int64_t* d_slots,
                          const int32_t* d_positions, void* d_pool, size_t pool_pages, size_t kv_heads,
                          size_t head_dim, size_t page_tokens, float* d_weight, int32_t* d_pos, int* d_status,
                          cudaStream_t stream) {
    const NvtxRange range("sz_cache_append");
    AppendParams p{};
    if (!pool_for(d_pool, pool_pages, kv_heads, head_dim, page_tokens, &p.pool)) return SZ_ERR_INVALID_ARG;
    if (!rows_for(d_k, k_token_stride, k_head_stride, d_v, v_token_stride, v_head_stride, d_slots, tokens, d_status, &p))
        return SZ_ERR_INVALID_ARG;
    if ((d_weight && !aligned(d_weight, 4)) || (d_pos && (!aligned(d_pos, 4) || !d_positions || !aligned(d_positions, 4))))
        return SZ_ERR_INVALID_ARG;
    const sz_status st = clear_status(d_status, stream);
    if (st != SZ_OK || tokens == 0) return st;
    p.positions = d_positions;
    p.weight = d_weight;
    p.pos = d_pos;
    return from_cuda(launch_append(p, stream));
}

sz_status sz_cache_read(const void* d_pool, size_t pool_pages, size_t kv_heads, size_t head_dim, size_t page_tokens,
                        const int64_t* d_slots, size_t tokens, void* d_k, int64_t k_token_stride,
                        int64_t k_head_stride, void* d_v, int64_t v_token_stride, int64_t v_head_stride,
                        int* d_status, cudaStream_t stream) {
    const NvtxRange range("sz_cache_read");
    AppendParams p{};
    if (!pool_for(d_pool, pool_pages, kv_heads, head_dim, page_tokens, &p.pool)) return SZ_ERR_INVALID_ARG;
    if (!rows_for(d_k, k_token_stride, k_head_stride, d_v, v_token_stride, v_head_stride, d_slots, tokens, d_status, &p))
        return SZ_ERR_INVALID_ARG;
    if (rows_overlap({d_k, k_token_stride, k_head_stride, tokens, kv_heads}, {d_v, v_token_stride, v_head_stride, tokens, kv_heads},
                     head_dim))
        return SZ_ERR_INVALID_ARG;
    const sz_status st = clear_status(d_status, stream);
    if (st != SZ_OK || tokens == 0) return st;
    return from_cuda(launch_cache_read(p, stream));
}

size_t sz_cache_attend_workspace_size(size_t batch, size_t q_heads, size_t kv_heads, size_t head_dim,
                                      size_t max_tokens, int weights) {
    if (!attend_sizes_ok(batch, q_heads, kv_heads, head_dim, max_tokens)) return 0;
    uint32_t heads = 0, blocks = 0;
    if (attend_shape(1, &heads, &blocks) != cudaSuccess) {
        (void)cudaGetLastError();
        blocks = 152;
    }
    return attend_ws(blocks, head_dim, batch * q_heads, max_tokens, weights != 0).end;
}

sz_status sz_cache_attend(const void* d_q, int64_t q_seq_stride, int64_t q_head_stride, size_t batch, size_t q_heads,
                          const void* d_pool, size_t pool_pages, size_t kv_heads, size_t head_dim, size_t page_tokens,
                          const int32_t* d_table, size_t table_width, const int32_t* d_lens, float scale, void* d_out,
                          int64_t out_seq_stride, int64_t out_head_stride, float* d_lse, float* d_weight,
                          int* d_status, void* d_ws, size_t ws_bytes, cudaStream_t stream) {
    return attend("sz_cache_attend", kNoBlock, d_q, q_seq_stride, q_head_stride, batch, q_heads, d_pool, pool_pages, kv_heads,
                  head_dim, page_tokens, d_table, table_width, d_lens, scale, d_out, out_seq_stride, out_head_stride, d_lse,
                  d_weight, d_status, d_ws, ws_bytes, stream);
}

sz_status sz_debug_attend_stalled(const void* d_q, int64_t q_seq_stride, int64_t q_head_stride, size_t batch, size_t q_heads,
                                  const void* d_pool, size_t pool_pages, size_t kv_heads, size_t head_dim,
                                  size_t page_tokens, const int32_t* d_table, size_t table_width, const int32_t* d_lens,
                                  float scale, void* d_out, int64_t out_seq_stride, int64_t out_head_stride, float* d_lse,
                                  float* d_weight, int* d_status, void* d_ws, size_t ws_bytes, cudaStream_t stream) {
    if (!d_status) return SZ_ERR_INVALID_ARG;
    return attend("sz_debug_attend_stalled", 0, d_q, q_seq_stride, q_head_stride, batch, q_heads, d_pool, pool_pages, kv_heads,
                  head_dim, page_tokens, d_table, table_width, d_lens, scale, d_out, out_seq_stride, out_head_stride, d_lse,
                  d_weight, d_status, d_ws, ws_bytes, stream);
}

size_t sz_cache_evict_workspace_size(size_t batch, size_t kv_heads, size_t max_tokens) {
    if (batch > 65535 || !heads_ok(kv_heads) || max_tokens == 0 || max_tokens >= (1ull << 31)) return 0;
    const uint64_t lists = (uint64_t)batch * kv_heads;
    return evict_pairs_offset(lists) + 8 * lists * evict_max_moves(max_tokens);
}

sz_status sz_cache_evict(void* d_pool, size_t pool_pages, size_t kv_heads, size_t head_dim, size_t page_tokens,
                         const int32_t* d_table, size_t table_width, const int32_t* d_lens, const int32_t* d_next_pos,
                         size_t batch, size_t keep, size_t recent, float* d_weight, int32_t* d_pos,
                         int32_t* d_new_lens, int* d_status, void* d_ws, size_t ws_bytes, cudaStream_t stream) {
    const NvtxRange range("sz_cache_evict");
    EvictParams p{};
    if (!pool_for(d_pool, pool_pages, kv_heads, head_dim, page_tokens, &p.pool)) return SZ_ERR_INVALID_ARG;
    if ((batch > 0 && !table_ok(d_table, table_width, page_tokens)) || batch > 65535) return SZ_ERR_INVALID_ARG;
    if (keep == 0 || keep >= (1ull << 31) || recent >= (1ull << 31)) return SZ_ERR_INVALID_ARG;
    if (!d_weight || !aligned(d_weight, 4) || !d_pos || !aligned(d_pos, 4)) return SZ_ERR_INVALID_ARG;
    if (d_status && !aligned(d_status, 4)) return SZ_ERR_INVALID_ARG;
    if (batch == 0) return clear_status(d_status, stream);
    if (!d_ws || !aligned(d_ws, 256)) return SZ_ERR_INVALID_ARG;
    if (!d_lens || !aligned(d_lens, 4) || !d_next_pos || !aligned(d_next_pos, 4) || !d_new_lens || !aligned(d_new_lens, 4))
        return SZ_ERR_INVALID_ARG;
    // A list's blocks read the old lengths and positions while another's write the new lengths.
    if (ranges_overlap(d_new_lens, d_lens, 4 * batch) || ranges_overlap(d_new_lens, d_next_pos, 4 * batch)) return SZ_ERR_INVALID_ARG;
    const uint64_t max_tokens = (uint64_t)table_width * page_tokens;
    if (ws_bytes < sz_cache_evict_workspace_size(batch, kv_heads, max_tokens)) return SZ_ERR_CAPACITY;
    const sz_status st = clear_status(d_status, stream);
    if (st != SZ_OK) return st;
    p.table = d_table;
    p.table_width = (uint32_t)table_width;
    p.lens = d_lens;
    p.next_pos = d_next_pos;
    p.batch = (uint32_t)batch;
    p.keep = (uint32_t)keep;
    p.recent = (uint32_t)recent;
    p.weight = d_weight;
    p.pos = d_pos;
    p.new_lens = d_new_lens;
    p.status = d_status;
    p.moves = static_cast<uint32_t*>(d_ws);
    p.pairs = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(d_ws) + evict_pairs_offset((uint64_t)batch * kv_heads));
    p.max_moves = (uint32_t)evict_max_moves(max_tokens);
    return from_cuda(launch_evict(p, stream));
}

}  // extern "C"
