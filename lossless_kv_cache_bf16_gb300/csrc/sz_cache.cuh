// sz_cache.cuh -- device-side addressing of the 4-bit cache.
#pragma once

#include <cstdint>

#include "sz_cache.h"
#include "sz_device.cuh"

namespace sz {

// Waits for the kernels before this one in the stream (see launch_dependent).
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// 16-bit words of a cell: K codes at 0, V codes at 4 D, K scales at 8 D, V
// scales at 8.5 D; 9 D words in all.
template <int D>
struct Cell {
    static constexpr uint32_t kGroups = D / 32;
    static constexpr uint32_t kBytes = 18 * D;
    static constexpr uint32_t kV = 4 * D, kKScale = 8 * D, kVScale = 8 * D + D / 2;
    // Word of the four channels 32 i + 4 r .. + 3 of token t.
    static __device__ __forceinline__ uint32_t k_word(uint32_t t, uint32_t i, uint32_t r) {
        return ((t * 4 + (r >> 1)) * kGroups + i) * 2 + (r & 1);
    }
    static __device__ __forceinline__ uint32_t v_word(uint32_t t, uint32_t i, uint32_t r) {
        return kV + ((((t >> 3) * 8 + r) * 4 + ((t & 7) >> 1)) * kGroups + i) * 2 + (t & 1);
    }
    // Word of the scale of group i of token t (K; V is D / 2 further on).
    static __device__ __forceinline__ uint32_t scale_word(uint32_t t, uint32_t i) {
        return kKScale + ((t >> 1) * kGroups + i) * 2 + (t & 1);
    }
};

// Byte offset of the cell that holds token `off` of page `page` and head h.
template <int D>
__device__ __forceinline__ uint64_t cell_offset(const CachePool& c, uint32_t page, uint32_t h, uint32_t off) {
    const uint64_t run = (uint64_t)page * c.heads + h;
    return ((run << (c.lg_page - 4)) + (off >> 4)) * (uint64_t)Cell<D>::kBytes;
}

__device__ __forceinline__ float bf16_float(uint32_t bits) { return __uint_as_float(bits << 16); }

// Two floats to packed bf16, round to nearest even; `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ uint32_t bf16_bits(float x) { return pack_bf16(x, 0.f) & 0xFFFFu; }

}  // namespace sz
