// sz_append.cu -- K and V rows into the 4-bit cache, and back.
//
// A group of 32 channels shares s = bf16(max|x| / 7); a channel's code is
// 8 + round(x / s).  The quotient is the product with the reciprocal,
// corrected by its remainder, which fma gives exactly, so that
// the codes are those of the definition: two bf16 significands have a
// quotient that is k + 1/2 or at least 2^-17 away from it, which fp32 tells
// apart.  |x / s| stays below 7.03, so that no code needs clamping.
//
// 4 D bytes of rows and 9 D / 8 of cache per token and head; the integer and
// fp32 work per value keeps both kernels at 70 to 80% of the copy rate
// (32,768 tokens, 4 heads of 128, append and read: 33 us against 25 us).
// A warp takes 8 tokens of one head, and its lanes are laid out as the cell
// is, so that each moves whole 16-byte pieces of it (D = 128):
//   K  lane 4 g + q: token g, channels 32 i + 8 q .. + 7 of every group i;
//   V  lane 4 g + q: tokens 2 q and 2 q + 1, channels 32 i + 4 g .. + 3.
// Two neighbouring tokens share the words of V's codes and of all scales.
// Where their slots are not an even one and the next (scattered tokens, or a
// run that starts at an odd slot after the first), their 16-bit words are
// moved one by one.
#include "sz_cache.cuh"
#include "sz_params.h"

namespace sz {
namespace {

constexpr uint32_t kThreads = 128;
constexpr uint32_t kTaskTokens = 8;

// 2 N (4 or 8) bf16 values, two to a word.
template <int N>
__device__ __forceinline__ void load_row(const uint16_t* p, bool vec, uint32_t (&w)[N]) {
    if (vec) {
        if constexpr (N == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x, w[1] = v.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; j++) w[j] = p[2 * j] | (uint32_t)p[2 * j + 1] << 16;
    }
}

// N (2 or 4) words of packed bf16 to a row.
template <int N>
__device__ __forceinline__ void store_row(uint16_t* p, bool vec, const uint32_t (&w)[N]) {
    if (vec) {
        if constexpr (N == 4)
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int j = 0; j < N; j++) p[2 * j] = (uint16_t)w[j], p[2 * j + 1] = (uint16_t)(w[j] >> 16);
    }
}

__device__ __forceinline__ float reciprocal(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return r;
}
// a / b for inv = 1 / b within 2^-22: the product's remainder is exact, so
// that the sum has an error far below half a last place, and a quotient that
// fp32 holds comes out exactly.
__device__ __forceinline__ float quotient(float a, float b, float inv) {
    const float q = __fmul_rn(a, inv);
    return __fmaf_rn(__fmaf_rn(-q, b, a), inv, q);
}
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
// The bits of x / s + 1.5 * 2^23 + 8 for the two bf16 values of w, by the same
// steps on pairs of floats.  neg_s, inv: -s and 1 / s, twice each.
__device__ __forceinline__ void rounded_quotients(uint32_t w, uint64_t neg_s, uint64_t inv, uint32_t& lo, uint32_t& hi) {
    const uint64_t x = pair_of(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    asm("{\n\t.reg .b64 q, r;\n\t"
        "mul.rn.f32x2 q, %2, %4;\n\t"
        "fma.rn.f32x2 r, q, %3, %2;\n\t"
        "fma.rn.f32x2 q, r, %4, q;\n\t"
        "add.rn.f32x2 q, q, %5;\n\t"
        "mov.b64 {%0, %1}, q;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "l"(x), "l"(neg_s), "l"(inv), "l"(pair_of(12582920.f, 12582920.f)));
}

// The scale's bf16 bits of a group whose largest |x| has the bits `top`:
// 0 below 2^-126, a NaN for a group that holds an infinity or a NaN.
__device__ __forceinline__ uint32_t scale_bits(uint32_t top) {
    const uint32_t s = bf16_bits(quotient(bf16_float(top), 7.f, 1.f / 7.f));
    return top > 0x7F7Fu ? 0x7FC0u : s < 0x0080u ? 0u : s;
}

// Codes of the 2 N values of w, 4 bits each, the first lowest.  The bits of
// x / s + 1.5 * 2^23 + 8 are kMagic + code: they are added up as digits of 16,
// and the sum of the kMagic taken off at the end.
template <int N>
__device__ __forceinline__ uint32_t codes_of(const uint32_t (&w)[N], uint32_t scale) {
    constexpr uint32_t kMagic = 0x4B400000u;
    constexpr uint32_t kSum = N == 4 ? kMagic * 0x11111111u : kMagic * 0x1111u;
    const bool usable = scale - 1u < 0x7F7Fu;  // neither 0 nor a NaN
    const float s = usable ? bf16_float(scale) : 1.f, inv = reciprocal(s);
    const uint64_t neg_s = pair_of(-s, -s), inv2 = pair_of(inv, inv);
    uint32_t sum = 0;
#pragma unroll
    for (int j = N - 1; j >= 0; j--) {
        uint32_t lo, hi;
        rounded_quotients(w[j], neg_s, inv2, lo, hi);
        sum = (sum * 16u + hi) * 16u + lo;
    }
    return usable ? sum - kSum : 0x88888888u >> (32 - 8 * N);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// The largest |x| of w, as bf16 bits (which compare like the value), in the
// larger of the result's halves.
template <int N>
__device__ __forceinline__ uint32_t largest(const uint32_t (&w)[N]) {
    uint32_t top = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int j = 1; j < N; j++) top = max_u16x2(top, w[j] & 0x7FFF7FFFu);
    return top;
}
// The larger halves of a and of b, in the low and the high half.
__device__ __forceinline__ uint32_t larger_halves(uint32_t a, uint32_t b) {
    return max_u16x2(prmt(a, b, 0x5410u), prmt(a, b, 0x7632u));
}

// A token's place: its cell (null where the token is left out: slot -1, or one
// outside the pool, which is reported) and its number in the cell.
struct Place {
    uint16_t* cell;
    uint32_t t;
    uint64_t entry;  // of the tables beside the pool
};

template <int D>
__device__ __forceinline__ Place locate(const AppendParams& p, int64_t token, uint32_t h) {
    Place at{nullptr, 0, 0};
    if (token < 0 || token >= (int64_t)p.tokens) return at;
    const int64_t slot = p.slots[token];
    if (slot < 0 || slot >= (int64_t)p.pool.pages << p.pool.lg_page) {
        if (slot != -1 && p.status) atomicMax(p.status, kStatusInvalid);
        return at;
    }
    const uint32_t page = (uint32_t)(slot >> p.pool.lg_page), off = (uint32_t)slot & ((1u << p.pool.lg_page) - 1u);
    at.cell = reinterpret_cast<uint16_t*>(p.pool.base + cell_offset<D>(p.pool, page, h, off));
    at.t = off & 15u;
    at.entry = (((uint64_t)page * p.pool.heads + h) << p.pool.lg_page) + off;
    return at;
}

// Another lane's cell and token number.
__device__ __forceinline__ Place from_lane(const Place& a, uint32_t lane) {
    Place b;
    b.cell = reinterpret_cast<uint16_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(a.cell), lane));
    b.t = __shfl_sync(0xFFFFFFFFu, a.t, lane);
    b.entry = 0;
    return b;
}

// Whether two tokens' words lie side by side.
__device__ __forceinline__ bool side_by_side(const Place& a, const Place& b) {
    return a.cell && a.cell == b.cell && !(a.t & 1u) && b.t == a.t + 1;
}

// N (2 or 4) words to or from an 8 N / 2 byte aligned place.
template <int N>
__device__ __forceinline__ void put_words(uint16_t* p, const uint32_t (&w)[N]) {
    if constexpr (N == 4)
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
template <int N>
__device__ __forceinline__ void get_words(const uint16_t* p, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x, w[1] = v.y;
    }
}

// Tasks of the call: 8 tokens of a head each.  The first task starts one
// token early where the first slot is odd, so that pairs of a run are pairs
// of slots.
struct Task {
    int64_t token;
    uint32_t h;
    __device__ __forceinline__ Task(const AppendParams& p, uint64_t n) {
        h = (uint32_t)(n % p.pool.heads);
        token = (int64_t)(n / p.pool.heads) * kTaskTokens - (p.slots[0] & 1);
    }
};
__device__ __forceinline__ uint64_t tasks_of(const AppendParams& p) {
    return ((uint64_t)p.tokens + (p.slots[0] & 1) + kTaskTokens - 1) / kTaskTokens * p.pool.heads;
}

template <int D>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
    using C = Cell<D>;
    constexpr int kG = C::kGroups;
    const uint32_t lane = threadIdx.x & 31u, g = lane >> 2, q = lane & 3u;
    wait_for_previous();
    const uint64_t tasks = tasks_of(p);
    for (uint64_t n = (uint64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; n < tasks; n += (uint64_t)gridDim.x * (kThreads / 32)) {
        const Task task(p, n);
        const uint32_t h = task.h;
        // ---- loads of both, then K: token g of the task ----
        const int64_t token = task.token + g, va = task.token + 2 * q;
        const Place at = locate<D>(p, token, h);
        const Place place[2] = {from_lane(at, 8 * q), from_lane(at, 8 * q + 4)};  // of tokens 2 q and 2 q + 1
        uint32_t xk[kG][4], xv[2][kG][2];
        const uint16_t* row = p.rows[0] + token * p.token_stride[0] + (int64_t)h * p.head_stride[0] + 8 * q;
#pragma unroll
        for (int i = 0; i < kG; i++) {
#pragma unroll
            for (int j = 0; j < 4; j++) xk[i][j] = 0;
            if (at.cell) load_row<4>(row + 32 * i, p.vec, xk[i]);
        }
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const uint16_t* vrow = p.rows[1] + (va + e) * p.token_stride[1] + (int64_t)h * p.head_stride[1] + 4 * g;
#pragma unroll
            for (int i = 0; i < kG; i++) {
#pragma unroll
                for (int j = 0; j < 2; j++) xv[e][i][j] = 0;
                if (place[e].cell) load_row<2>(vrow + 32 * i, p.vec, xv[e][i]);
            }
        }
        // Two groups' maxima share a word while the lanes of a group compare theirs.
        uint32_t word[kG], scale[kG], both[kG];
#pragma unroll
        for (int i = 0; i < kG; i += 2) {
            uint32_t top = larger_halves(largest(xk[i]), largest(xk[i + 1]));
            top = max_u16x2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max_u16x2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            scale[i] = scale_bits(top & 0xFFFFu);
            scale[i + 1] = scale_bits(top >> 16);
        }
#pragma unroll
        for (int i = 0; i < kG; i++) {
            word[i] = codes_of<4>(xk[i], scale[i]);
            // Word q of a pair's scales: this token's and its neighbour's.
            both[i] = scale[i] | __shfl_xor_sync(0xFFFFFFFFu, scale[i], 4) << 16;
        }
        if (at.cell) {
            put_words<kG>(at.cell + C::k_word(at.t, 0, 2 * q), word);
            if (q == 0) {
                if (p.weight) p.weight[at.entry] = 0.f;
                if (p.pos) p.pos[at.entry] = p.positions[token];
            }
        }
        // Scales: the even token's lane stores the pair's words.  Its two
        // places are those of V's lane g / 2.
        const int cell_pair = __shfl_sync(0xFFFFFFFFu, (int)side_by_side(place[0], place[1]), g >> 1);
        if (q == 0 && at.cell) {
            if (cell_pair) {
                if (!(g & 1u)) put_words<kG>(at.cell + C::scale_word(at.t, 0), both);
            } else {
#pragma unroll
                for (int i = 0; i < kG; i++) at.cell[C::scale_word(at.t, i)] = (uint16_t)scale[i];
            }
        }

        // ---- V: tokens 2 q and 2 q + 1 ----
        uint32_t code[2][kG], sv[2][kG];
#pragma unroll
        for (int i = 0; i < kG; i++) {
            uint32_t top = larger_halves(largest(xv[0][i]), largest(xv[1][i]));
            top = max_u16x2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
            top = max_u16x2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
            top = max_u16x2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
            sv[0][i] = scale_bits(top & 0xFFFFu);
            sv[1][i] = scale_bits(top >> 16);
#pragma unroll
            for (int e = 0; e < 2; e++) code[e][i] = codes_of<2>(xv[e][i], sv[e][i]);
        }
        if (side_by_side(place[0], place[1])) {
#pragma unroll
            for (int i = 0; i < kG; i++) word[i] = code[0][i] | code[1][i] << 16, both[i] = sv[0][i] | sv[1][i] << 16;
            put_words<kG>(place[0].cell + C::v_word(place[0].t, 0, g), word);
            if (g == 0) put_words<kG>(place[0].cell + C::scale_word(place[0].t, 0) + D / 2, both);
        } else {
#pragma unroll
            for (int e = 0; e < 2; e++) {
                if (!place[e].cell) continue;
#pragma unroll
                for (int i = 0; i < kG; i++) {
                    place[e].cell[C::v_word(place[e].t, i, g)] = (uint16_t)code[e][i];
                    if (g == 0) place[e].cell[C::scale_word(place[e].t, i) + D / 2] = (uint16_t)sv[e][i];
                }
            }
        }
    }
}

// Values of the eight codes of w: nibble j of both halves, times the scale of
// their half, in r[j].  128 + code is a bf16 number (code in the mantissa's low
// bits), less 136 exactly code - 8, and its product with the scale is rounded
// once.
__device__ __forceinline__ void values_of(uint32_t w, uint32_t scales, uint32_t (&r)[4]) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const uint32_t code = (w >> (4 * j) & 0x000F000Fu) | 0x43004300u;
        asm("{\n\t.reg .b32 x;\n\tsub.rn.bf16x2 x, %1, %3;\n\tmul.rn.bf16x2 %0, x, %2;\n\t}"
            : "=r"(r[j])
            : "r"(code), "r"(scales), "r"(0x43084308u));
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const AppendParams p) {
    using C = Cell<D>;
    constexpr int kG = C::kGroups;
    const uint32_t lane = threadIdx.x & 31u, g = lane >> 2, q = lane & 3u;
    wait_for_previous();
    const uint64_t tasks = tasks_of(p);
    for (uint64_t n = (uint64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; n < tasks; n += (uint64_t)gridDim.x * (kThreads / 32)) {
        const Task task(p, n);
        const uint32_t h = task.h;
        const int64_t token = task.token + g, va = task.token + 2 * q;
        const Place at = locate<D>(p, token, h);
        const Place place[2] = {from_lane(at, 8 * q), from_lane(at, 8 * q + 4)};  // of tokens 2 q and 2 q + 1
        uint32_t kw[kG], ks[kG], vw[kG], vs[kG];  // V: both tokens, the even one in the low halves
#pragma unroll
        for (int i = 0; i < kG; i++) kw[i] = vw[i] = 0x88888888u, ks[i] = vs[i] = 0;
        if (at.cell) {
            get_words<kG>(at.cell + C::k_word(at.t, 0, 2 * q), kw);
            get_words<kG>(at.cell + C::scale_word(at.t & ~1u, 0), ks);  // of the pair
#pragma unroll
            for (int i = 0; i < kG; i++) ks[i] = prmt(ks[i], 0u, at.t & 1u ? 0x3232u : 0x1010u);
        }
        if (side_by_side(place[0], place[1])) {
            get_words<kG>(place[0].cell + C::v_word(place[0].t, 0, g), vw);
            get_words<kG>(place[0].cell + C::scale_word(place[0].t, 0) + D / 2, vs);
        } else {
#pragma unroll
            for (int e = 0; e < 2; e++) {
                if (!place[e].cell) continue;
                uint32_t w[kG], s[kG];
                get_words<kG>(place[e].cell + C::v_word(place[e].t & ~1u, 0, g), w);
                get_words<kG>(place[e].cell + C::scale_word(place[e].t & ~1u, 0) + D / 2, s);
                // This token's half into half e.
                const uint32_t from = place[e].t & 1u ? 0x32u : 0x10u, sel = e ? from << 8 | 0x54u : 0x7600u | from;
#pragma unroll
                for (int i = 0; i < kG; i++) vw[i] = prmt(w[i], vw[i], sel), vs[i] = prmt(s[i], vs[i], sel);
            }
        }
        if (token >= 0 && token < (int64_t)p.tokens) {
            uint16_t* row = p.rows[0] + token * p.token_stride[0] + (int64_t)h * p.head_stride[0] + 8 * q;
#pragma unroll
            for (int i = 0; i < kG; i++) {
                uint32_t r[4];
                values_of(kw[i], ks[i], r);
                const uint32_t v[4] = {prmt(r[0], r[1], 0x5410u), prmt(r[2], r[3], 0x5410u), prmt(r[0], r[1], 0x7632u),
                                       prmt(r[2], r[3], 0x7632u)};
                store_row<4>(row + 32 * i, p.vec, v);
            }
        }
        uint16_t* row = p.rows[1] + va * p.token_stride[1] + (int64_t)h * p.head_stride[1] + 4 * g;
        const bool in[2] = {va >= 0 && va < (int64_t)p.tokens, va + 1 >= 0 && va + 1 < (int64_t)p.tokens};
#pragma unroll
        for (int i = 0; i < kG; i++) {
            uint32_t r[4];
            values_of(vw[i], vs[i], r);
            const uint32_t even[2] = {prmt(r[0], r[1], 0x5410u), prmt(r[2], r[3], 0x5410u)};
            const uint32_t odd[2] = {prmt(r[0], r[1], 0x7632u), prmt(r[2], r[3], 0x7632u)};
            if (in[0]) store_row<2>(row + 32 * i, p.vec, even);
            if (in[1]) store_row<2>(row + p.token_stride[1] + 32 * i, p.vec, odd);
        }
    }
}

cudaError_t launch(void (*kern)(AppendParams), const AppendParams& p, cudaStream_t s) {
    int sms = 0, per_sm = 0;
    const cudaError_t err = kernel_fit(reinterpret_cast<const void*>(kern), kThreads, 0, &sms, &per_sm);
    if (err != cudaSuccess) return err;
    const uint64_t tasks = ((uint64_t)p.tokens + kTaskTokens) / kTaskTokens * p.pool.heads;
    const uint64_t need = (tasks + kThreads / 32 - 1) / (kThreads / 32);
    const uint64_t fit = (uint64_t)sms * per_sm;
    return launch_dependent(kern, dim3((uint32_t)(need < 16 * fit ? need : 16 * fit)), dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, cudaStream_t s) {
    return launch(p.pool.dim == 64 ? append_kernel<64> : append_kernel<128>, p, s);
}

cudaError_t launch_cache_read(const AppendParams& p, cudaStream_t s) {
    return launch(p.pool.dim == 64 ? read_kernel<64> : read_kernel<128>, p, s);
}

}  // namespace sz
