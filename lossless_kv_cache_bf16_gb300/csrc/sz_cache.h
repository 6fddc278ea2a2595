// sz_cache.h -- launch parameters of the serving operators around the 4-bit
// cache, shared by their kernels and the C ABI layer.  Not part of the public
// interface.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace sz {

constexpr uint32_t kCellTokens = 16;  // tokens of a cell
constexpr uint32_t kUnitTokens = 32;  // tokens that a warp of the attention takes at a time (two cells)
constexpr uint32_t kMaxBatch = 2048;  // sequences of one attention call (their lengths sit in shared memory)

// A pool of pages of the 4-bit cache: page p, kv head h, cell j of 16 tokens
// starts at byte ((p * heads + h) * cells of a page + j) * 18 D.
struct CachePool {
    uint8_t* base;
    uint32_t pages;
    uint32_t heads;
    uint32_t lg_page;  // log2 of the tokens of a page
    uint32_t dim;
};

struct NormRopeParams {
    const uint16_t* in[2];  // q, k (bf16 bits)
    uint16_t* out[2];
    int64_t in_token[2], in_head[2], out_token[2], out_head[2];  // strides in elements
    uint32_t heads[2];
    const uint16_t* weight[2];  // nullable: no norm
    const float* inv_freq;
    const int32_t* positions;
    uint32_t tokens, dim, rot;
    int interleaved;
    int vec;  // every row is 16-byte aligned
    float eps;
};

// Append, and read with `rows` as the outputs.
struct AppendParams {
    uint16_t* rows[2];  // k, v (bf16 bits)
    int64_t token_stride[2], head_stride[2];
    const int64_t* slots;
    const int32_t* positions;  // with pos
    uint32_t tokens;
    CachePool pool;
    float* weight;  // nullable
    int32_t* pos;   // nullable
    int* status;    // nullable
    int vec;        // rows are 16-byte aligned
};

struct AttendParams {
    const uint16_t* q;
    int64_t q_seq, q_head;
    uint16_t* out;
    int64_t out_seq, out_head;
    CachePool pool;
    const int32_t* table;
    uint32_t table_width;
    const int32_t* lens;
    uint32_t batch;
    uint32_t group;    // query heads per kv head
    uint32_t tiles;    // work items per kv head: ceil(group / heads of an item)
    float scale_log2;  // softmax scale * log2(e)
    float* lse;        // nullable [batch][q heads]
    float* weight;     // nullable
    int* status;       // nullable
    uint64_t wait_limit_ns;
    uint32_t stalled_block;  // test hook: its waits give up at once, though their copies land
    int whole_items;  // one item a block (set by the launch)
    int q_vec, out_vec, weight_vec;  // query rows are 16-byte, output rows 8-byte, weights 16-byte aligned
    // workspace
    int32_t* meta;   // [blocks][4]: the item that a block leaves to the join (sequence or -1, item, further blocks),
                     // whether a wait of the block gave up
    float* part_ml;  // [blocks][2][16][2]: maximum, sum of weights
    float* part_o;   // [blocks][2][16][dim]
    float* lse2;     // [batch][q heads], log2; with weight
    float* logits;   // [batch][q heads][max tokens], log2; with weight
};

struct EvictParams {
    CachePool pool;
    const int32_t* table;
    uint32_t table_width;
    const int32_t* lens;
    const int32_t* next_pos;
    uint32_t batch;
    uint32_t keep, recent;
    float* weight;
    int32_t* pos;
    int32_t* new_lens;
    int* status;  // nullable
    // workspace
    uint32_t* moves;  // [batch * heads]: moves of a (sequence, head)
    uint32_t* pairs;  // [batch * heads][2][max_moves]: target slots, source slots
    uint32_t max_moves;
};

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t s);
cudaError_t launch_append(const AppendParams& p, cudaStream_t s);
cudaError_t launch_cache_read(const AppendParams& p, cudaStream_t s);
// Query heads of one attention work item, and blocks of its launch on this device.
cudaError_t attend_shape(uint32_t group, uint32_t* item_heads, uint32_t* blocks);
cudaError_t launch_attend(const AttendParams& p, cudaStream_t s);
cudaError_t launch_evict(const EvictParams& p, cudaStream_t s);

}  // namespace sz
