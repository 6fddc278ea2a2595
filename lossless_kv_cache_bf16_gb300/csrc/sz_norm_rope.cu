// sz_norm_rope.cu -- RMS norm of every query and key head and the position
// rotation, one read and one write of each value.
//
// y = x * rsqrt(mean(x^2) + eps) * w over a head's D channels, then for pair
// (a, b) number i of the first `rot` channels the rotation by
// position * inv_freq[i]: (a cos - b sin, b cos + a sin).  Everything is fp32
// with one rounding to bf16 at the end.
//
// Angles are kept in turns as 64-bit fractions: inv_freq / (2 pi) modulo 1
// times the position, modulo 1, is one integer product, exact but for the
// rounding of the factor (2^-53 of it, so that position 10^6 leaves the angle
// good to 10^-9), where fp32 would leave an error of 0.06.  Their top 32 bits
// go to sincospi.
//
// A block takes a few tokens at a time: their sines and cosines are computed
// once, in shared memory, for all heads.  D / 16 threads share a head's row,
// each with two vectors of 8 channels: channels [8c, 8c + 8) and their
// partners, so that a rotation never leaves a thread, and the sum of squares
// is a shuffle over a few lanes.  Bound by memory: 48 warps per SM with one
// row's loads each move more than 32 with two rows' (20,011 tokens of 28 and 4
// heads of 128: 56 against 62 us, 86% of the measured copy rate; 8,192 of 32
// and 8: 30 us, 81%).
#include "sz_cache.cuh"
#include "sz_params.h"

namespace sz {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kMaxRot = 256;
constexpr uint32_t kMaxTile = 16;  // tokens of a block at a time

template <bool VEC>
__device__ __forceinline__ void load8(const uint16_t* p, float (&x)[8]) {
    if constexpr (VEC) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; j++) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) x[j] = bf16_float(p[j]);
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
    if constexpr (VEC) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                                  pack_bf16(x[6], x[7]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) p[j] = (uint16_t)bf16_bits(x[j]);
    }
}

// One thread's share of a row.
struct Item {
    const uint16_t* src;
    uint16_t* dst;
    const uint16_t* weight;
    uint32_t turn;  // of the table
    bool live;
    float a[8], b[8];
};

template <int D, bool VEC>
__global__ void __launch_bounds__(kThreads, 6) norm_rope_kernel(const NormRopeParams p, const uint32_t tile) {
    constexpr uint32_t kPer = D / 16;              // threads of a row
    constexpr uint32_t kStep = kThreads / kPer;    // rows that the block takes at a time
    __shared__ float2 s_turn[kMaxTile * kMaxRot / 2];
    __shared__ uint64_t s_freq[kMaxRot / 2];
    const uint32_t half = p.rot / 2;
    // Pairs in a vector of 8 channels.  The table holds pair number j of every
    // vector side by side, so that a warp's lanes read neighbouring entries.
    const uint32_t vec = p.interleaved ? 4u : 8u;
    wait_for_previous();
    for (uint32_t i = threadIdx.x; i < half; i += kThreads) {
        const double f = (double)p.inv_freq[i] * 0.15915494309189535;  // 1 / (2 pi)
        s_freq[i] = (uint64_t)(int64_t)((f - rint(f)) * 18446744073709551616.0);
    }
    __syncthreads();
    const uint32_t rows = p.heads[0] + p.heads[1];
    // First channels of this thread's two vectors.
    const uint32_t c = threadIdx.x % kPer;
    const bool turn_halves = !p.interleaved && c < half / 8;
    uint32_t ca, cb;
    if (p.interleaved) {
        ca = 8 * c;
        cb = D / 2 + 8 * c;
    } else if (turn_halves) {
        ca = 8 * c;
        cb = half + 8 * c;
    } else {
        ca = p.rot + 16 * (c - half / 8);
        cb = ca + 8;
    }
    for (uint32_t token0 = blockIdx.x * tile; token0 < p.tokens; token0 += gridDim.x * tile) {
        const uint32_t n = min(tile, p.tokens - token0);
        for (uint32_t k = threadIdx.x; k < n * half; k += kThreads) {
            const uint32_t i = k % half;
            const uint64_t turns = s_freq[i] * (uint64_t)(int64_t)p.positions[token0 + k / half];
            float sn, cs;
            sincospif((float)(int32_t)(turns >> 32) * 4.656612873077393e-10f, &sn, &cs);  // 2^-31: half turns
            s_turn[k - i + (i % vec) * (half / vec) + i / vec] = make_float2(cs, sn);
        }
        __syncthreads();
        uint32_t row = threadIdx.x / kPer, token = 0;  // of the tile
        while (row >= rows) row -= rows, token++;
        auto next = [&](Item& it) {
            it.live = token < n;
            const uint32_t r = it.live ? row : 0u, at = token0 + (it.live ? token : 0u);
            const int which = r >= p.heads[0];
            const uint32_t h = r - (which ? p.heads[0] : 0);
            it.src = p.in[which] + (int64_t)at * p.in_token[which] + (int64_t)h * p.in_head[which];
            it.dst = p.out[which] + (int64_t)at * p.out_token[which] + (int64_t)h * p.out_head[which];
            it.weight = p.weight[which];
            it.turn = (it.live ? token : 0u) * half;
            load8<VEC>(it.src + ca, it.a);
            load8<VEC>(it.src + cb, it.b);
            row += kStep;
            while (row >= rows) row -= rows, token++;
        };
        auto finish = [&](Item& it) {
            float(&a)[8] = it.a;
            float(&b)[8] = it.b;
            // Every lane takes part in the sum: a warp can hold rows of both
            // tensors, and only one of them may have a norm.
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; j++) sum += a[j] * a[j] + b[j] * b[j];
#pragma unroll
            for (uint32_t m = 1; m < kPer; m *= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
            if (it.weight) {
                const float inv = rsqrtf(sum * (1.f / D) + p.eps);
                float wa[8], wb[8];
                load8<VEC>(it.weight + ca, wa);
                load8<VEC>(it.weight + cb, wb);
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    a[j] = a[j] * inv * wa[j];
                    b[j] = b[j] * inv * wb[j];
                }
            }
            const float2* turn = s_turn + it.turn;
            if (turn_halves) {
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float2 t = turn[j * (half / 8) + c];
                    const float u = a[j] * t.x - b[j] * t.y;
                    b[j] = b[j] * t.x + a[j] * t.y;
                    a[j] = u;
                }
            } else if (p.interleaved) {
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    if (ca + j < p.rot) {
                        const float2 t = turn[j / 2 * (half / 4) + ca / 8];
                        const float u = a[j] * t.x - a[j + 1] * t.y;
                        a[j + 1] = a[j + 1] * t.x + a[j] * t.y;
                        a[j] = u;
                    }
                    if (cb + j < p.rot) {
                        const float2 t = turn[j / 2 * (half / 4) + cb / 8];
                        const float u = b[j] * t.x - b[j + 1] * t.y;
                        b[j + 1] = b[j + 1] * t.x + b[j] * t.y;
                        b[j] = u;
                    }
                }
            }
            if (it.live) {
                store8<VEC>(it.dst + ca, a);
                store8<VEC>(it.dst + cb, b);
            }
        };
        for (uint32_t done = 0; done < n * rows; done += kStep) {
            Item x;
            next(x);
            finish(x);
        }
        __syncthreads();
    }
}

template <int D, bool VEC>
cudaError_t launch(const NormRopeParams& p, cudaStream_t s) {
    int sms = 0, per_sm = 0;
    const cudaError_t err = kernel_fit(reinterpret_cast<const void*>(norm_rope_kernel<D, VEC>), kThreads, 0, &sms, &per_sm);
    if (err != cudaSuccess) return err;
    // As many tokens at a time as leave every block the same number of times:
    // one token each while there are fewer tokens than blocks.
    const uint32_t fit = (uint32_t)sms * per_sm;
    const uint32_t times = (p.tokens + kMaxTile * fit - 1) / (kMaxTile * fit);
    const uint32_t tile = (p.tokens + times * fit - 1) / (times * fit);
    const uint32_t need = (p.tokens + tile - 1) / tile;
    return launch_dependent(norm_rope_kernel<D, VEC>, dim3(need < fit ? need : fit), dim3(kThreads), 0, s, p, tile);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t s) {
    if (p.dim == 64) return p.vec ? launch<64, true>(p, s) : launch<64, false>(p, s);
    if (p.dim == 128) return p.vec ? launch<128, true>(p, s) : launch<128, false>(p, s);
    return p.vec ? launch<256, true>(p, s) : launch<256, false>(p, s);
}

}  // namespace sz
