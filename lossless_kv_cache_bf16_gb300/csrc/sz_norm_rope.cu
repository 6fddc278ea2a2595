// sz_norm_rope.cu -- RMS norm of every query and key head and the position
// rotation, one read and one write of each value.
//
// y = x * rsqrt(mean(x^2) + eps) * w over a head's D channels, then for pair
// (a, b) number i of the first `rot` channels the rotation by
// position * inv_freq[i]: (a cos - b sin, b cos + a sin).  Everything is fp32
// with one rounding to bf16 at the end; the angle is formed and reduced to
// [-pi, pi] in double, since a position of 10^6 would leave fp32 an angle
// error of 0.06.
//
// A block takes one token: its rot / 2 sines and cosines are computed once,
// in shared memory, for all heads.  D / 16 threads share a head's row, each
// with two vectors of 8 channels: channels [8c, 8c + 8) and their partners,
// so that a rotation never leaves a thread, and the sum of squares is a
// shuffle over a few lanes.  Bound by memory.
#include "sz_cache.cuh"
#include "sz_params.h"

namespace sz {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kMaxRot = 256;

__device__ __forceinline__ void load8(const uint16_t* p, bool vec, float (&x)[8]) {
    if (vec) {
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

__device__ __forceinline__ void store8(uint16_t* p, bool vec, const float (&x)[8]) {
    if (vec) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                                  pack_bf16(x[6], x[7]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) p[j] = (uint16_t)bf16_bits(x[j]);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeParams p) {
    constexpr uint32_t kPer = D / 16;  // threads of a row
    __shared__ float2 s_turn[kMaxRot / 2];
    const uint32_t half = p.rot / 2;
    wait_for_previous();
    const uint32_t rows = p.heads[0] + p.heads[1];
    for (uint32_t token = blockIdx.x; token < p.tokens; token += gridDim.x) {
        const double position = (double)p.positions[token];
        for (uint32_t i = threadIdx.x; i < half; i += kThreads) {
            const double a = position * (double)p.inv_freq[i];
            const double turns = rint(a * 0.15915494309189535);  // 1 / (2 pi)
            // 2 pi as the sum of two doubles.
            const double r = fma(-turns, 2.4492935982947064e-16, fma(-turns, 6.283185307179586, a));
            float sn, cs;
            sincosf((float)r, &sn, &cs);
            s_turn[i] = make_float2(cs, sn);
        }
        __syncthreads();
        for (uint32_t item = threadIdx.x; item < ((rows * kPer + 31u) & ~31u); item += kThreads) {
            const bool live = item < rows * kPer;
            const uint32_t row = live ? item / kPer : 0, c = item % kPer;
            const int which = row >= p.heads[0];
            const uint32_t h = row - (which ? p.heads[0] : 0);
            // First channels of this thread's two vectors.
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
            const uint16_t* src = p.in[which] + (int64_t)token * p.in_token[which] + (int64_t)h * p.in_head[which];
            float a[8], b[8];
            load8(src + ca, p.vec, a);
            load8(src + cb, p.vec, b);
            // Every lane takes part in the sum: a warp can hold rows of both
            // tensors, and only one of them may have a norm.
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; j++) sum += a[j] * a[j] + b[j] * b[j];
#pragma unroll
            for (uint32_t m = 1; m < kPer; m *= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
            if (p.weight[which]) {
                const float inv = rsqrtf(sum * (1.f / D) + p.eps);
                float wa[8], wb[8];
                load8(p.weight[which] + ca, p.vec, wa);
                load8(p.weight[which] + cb, p.vec, wb);
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    a[j] = a[j] * inv * wa[j];
                    b[j] = b[j] * inv * wb[j];
                }
            }
            if (turn_halves) {
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float2 t = s_turn[8 * c + j];
                    const float u = a[j] * t.x - b[j] * t.y;
                    b[j] = b[j] * t.x + a[j] * t.y;
                    a[j] = u;
                }
            } else if (p.interleaved) {
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    if (ca + j < p.rot) {
                        const float2 t = s_turn[(ca + j) / 2];
                        const float u = a[j] * t.x - a[j + 1] * t.y;
                        a[j + 1] = a[j + 1] * t.x + a[j] * t.y;
                        a[j] = u;
                    }
                    if (cb + j < p.rot) {
                        const float2 t = s_turn[(cb + j) / 2];
                        const float u = b[j] * t.x - b[j + 1] * t.y;
                        b[j + 1] = b[j + 1] * t.x + b[j] * t.y;
                        b[j] = u;
                    }
                }
            }
            if (live) {
                uint16_t* dst = p.out[which] + (int64_t)token * p.out_token[which] + (int64_t)h * p.out_head[which];
                store8(dst + ca, p.vec, a);
                store8(dst + cb, p.vec, b);
            }
        }
        __syncthreads();
    }
}

template <int D>
cudaError_t launch(const NormRopeParams& p, cudaStream_t s) {
    int sms = 0, per_sm = 0;
    const cudaError_t err = kernel_fit(reinterpret_cast<const void*>(norm_rope_kernel<D>), kThreads, 0, &sms, &per_sm);
    if (err != cudaSuccess) return err;
    const uint64_t fit = (uint64_t)sms * per_sm;
    return launch_dependent(norm_rope_kernel<D>, dim3((uint32_t)(p.tokens < fit ? p.tokens : fit)), dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t s) {
    return p.dim == 64 ? launch<64>(p, s) : p.dim == 128 ? launch<128>(p, s) : launch<256>(p, s);
}

}  // namespace sz
