// sz_append.cu -- K and V rows into the 4-bit cache, and back.
//
// A group of 32 channels shares s = bf16(max|x| / 7); a channel's code is
// 8 + round(x / s).  The quotient is correctly rounded (the product with the
// reciprocal, corrected by its remainder, which fma gives exactly), so that
// the codes are those of the definition: two bf16 significands have a
// quotient that is k + 1/2 or at least 2^-17 away from it, which fp32 tells
// apart.
//
// A lane takes 4 channels of a row, 8 lanes a group; each lane's 4 codes are
// one 16-bit word of the cell.
#include "sz_cache.cuh"
#include "sz_params.h"

namespace sz {
namespace {

constexpr uint32_t kThreads = 256;

__device__ __forceinline__ void load4(const uint16_t* p, bool vec, uint32_t (&x)[4]) {
    if (vec) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        x[0] = v.x & 0xFFFFu, x[1] = v.x >> 16, x[2] = v.y & 0xFFFFu, x[3] = v.y >> 16;
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++) x[j] = p[j];
    }
}

// The 4 codes of this lane's channels and, in every lane of the group, the
// scale's bf16 bits.  All 32 lanes take part.
__device__ __forceinline__ uint32_t quantise4(const uint32_t (&x)[4], uint32_t& scale) {
    uint32_t top = 0;  // |x| as bf16 bits compares like the value; above 0x7F7F: infinity or NaN
#pragma unroll
    for (int j = 0; j < 4; j++) top = max(top, x[j] & 0x7FFFu);
#pragma unroll
    for (uint32_t m = 1; m < 8; m *= 2) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
    scale = bf16_bits(__fdiv_rn(bf16_float(top), 7.f));
    if (scale < 0x0080u) scale = 0;      // below 2^-126
    if (top > 0x7F7Fu) scale = 0x7FC0u;  // NaN: the group reads as NaN
    if (scale == 0 || top > 0x7F7Fu) return 0x8888u;
    const float s = bf16_float(scale), inv = __frcp_rn(s);
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float v = bf16_float(x[j]);
        const float q0 = __fmul_rn(v, inv);
        const float q = __fmaf_rn(__fmaf_rn(-q0, s, v), inv, q0);
        const int c = max(-7, min(7, __float2int_rn(q)));
        w |= (uint32_t)(c + 8) << (4 * j);
    }
    return w;
}

// Where a slot lies, or false for one to leave out (-1, or outside the pool,
// which is reported).
__device__ __forceinline__ bool locate(const CachePool& c, int64_t slot, int* status, uint32_t& page, uint32_t& off) {
    const int64_t limit = (int64_t)c.pages << c.lg_page;
    if (slot < 0 || slot >= limit) {
        if (slot != -1 && status) atomicMax(status, kStatusInvalid);
        return false;
    }
    page = (uint32_t)(slot >> c.lg_page);
    off = (uint32_t)slot & ((1u << c.lg_page) - 1u);
    return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
    using C = Cell<D>;
    constexpr uint32_t kLanes = D / 4;  // lanes of a row
    wait_for_previous();
    const uint64_t rows = (uint64_t)p.tokens * p.pool.heads;
    const uint64_t step = (uint64_t)gridDim.x * (kThreads / kLanes);
    const uint32_t lr = threadIdx.x % kLanes, i = lr / 8, r = lr % 8;
    for (uint64_t row0 = (uint64_t)blockIdx.x * (kThreads / kLanes); row0 < rows; row0 += step) {
        const uint64_t row = row0 + threadIdx.x / kLanes;
        uint32_t token = 0, h = 0, page = 0, off = 0;
        bool live = row < rows;
        if (live) {
            token = (uint32_t)(row / p.pool.heads);
            h = (uint32_t)(row % p.pool.heads);
            live = locate(p.pool, p.slots[token], p.status, page, off);
        }
        uint32_t word[2], scale[2];
#pragma unroll
        for (int which = 0; which < 2; which++) {
            uint32_t x[4] = {0, 0, 0, 0};
            if (live)
                load4(p.rows[which] + (int64_t)token * p.token_stride[which] + (int64_t)h * p.head_stride[which] + 4 * lr,
                      p.vec, x);
            word[which] = quantise4(x, scale[which]);
        }
        if (!live) continue;
        uint16_t* cell = reinterpret_cast<uint16_t*>(p.pool.base + cell_offset<D>(p.pool, page, h, off));
        const uint32_t t = off & 15u;
        cell[C::k_word(t, i, r)] = (uint16_t)word[0];
        cell[C::v_word(t, i, r)] = (uint16_t)word[1];
        if (r == 0) {
            cell[C::scale_word(t, i)] = (uint16_t)scale[0];
            cell[C::scale_word(t, i) + D / 2] = (uint16_t)scale[1];
        }
        if (lr == 0) {
            const uint64_t at = (((uint64_t)page * p.pool.heads + h) << p.pool.lg_page) + off;
            if (p.weight) p.weight[at] = 0.f;
            if (p.pos) p.pos[at] = p.positions[token];
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const AppendParams p) {
    using C = Cell<D>;
    constexpr uint32_t kLanes = D / 4;
    wait_for_previous();
    const uint64_t rows = (uint64_t)p.tokens * p.pool.heads;
    const uint64_t step = (uint64_t)gridDim.x * (kThreads / kLanes);
    const uint32_t lr = threadIdx.x % kLanes, i = lr / 8, r = lr % 8;
    for (uint64_t row = (uint64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes; row < rows; row += step) {
        const uint32_t token = (uint32_t)(row / p.pool.heads), h = (uint32_t)(row % p.pool.heads);
        uint32_t page = 0, off = 0;
        uint32_t word[2] = {0x8888u, 0x8888u}, scale[2] = {0, 0};
        if (locate(p.pool, p.slots[token], p.status, page, off)) {
            const uint16_t* cell =
                reinterpret_cast<const uint16_t*>(p.pool.base + cell_offset<D>(p.pool, page, h, off));
            const uint32_t t = off & 15u;
            word[0] = cell[C::k_word(t, i, r)];
            word[1] = cell[C::v_word(t, i, r)];
            scale[0] = cell[C::scale_word(t, i)];
            scale[1] = cell[C::scale_word(t, i) + D / 2];
        }
#pragma unroll
        for (int which = 0; which < 2; which++) {
            uint16_t* out = p.rows[which] + (int64_t)token * p.token_stride[which] + (int64_t)h * p.head_stride[which] + 4 * lr;
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; j++)
                v[j] = (float)((int)((word[which] >> (4 * j)) & 15u) - 8) * bf16_float(scale[which]);
            if (p.vec) {
                *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++) out[j] = (uint16_t)bf16_bits(v[j]);
            }
        }
    }
}

cudaError_t launch(void (*kern)(AppendParams), const AppendParams& p, cudaStream_t s) {
    int sms = 0, per_sm = 0;
    const cudaError_t err = kernel_fit(reinterpret_cast<const void*>(kern), kThreads, 0, &sms, &per_sm);
    if (err != cudaSuccess) return err;
    const uint64_t per_block = kThreads / (p.pool.dim / 4);
    const uint64_t need = ((uint64_t)p.tokens * p.pool.heads + per_block - 1) / per_block;
    const uint64_t fit = (uint64_t)sms * per_sm;
    return launch_dependent(kern, dim3((uint32_t)(need < fit ? need : fit)), dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, cudaStream_t s) {
    return launch(p.pool.dim == 64 ? append_kernel<64> : append_kernel<128>, p, s);
}

cudaError_t launch_cache_read(const AppendParams& p, cudaStream_t s) {
    return launch(p.pool.dim == 64 ? read_kernel<64> : read_kernel<128>, p, s);
}

}  // namespace sz
