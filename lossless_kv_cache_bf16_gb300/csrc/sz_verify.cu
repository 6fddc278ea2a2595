// sz_verify.cu -- verification of a tree of drafted tokens against the target's
// probabilities, from given random numbers.
//
// One cluster of blocks per sequence walks down its tree: only the rows of
// nodes that the walk comes through are read.  At a node one pass over the row
// gives the sum of exponentials of all but the children's tokens, which are
// looked up one by one.  So without draft logits a node costs one reading of its
// row however many children it has, and nothing is taken out of a sum again: with W
// the sum over the other tokens and w_j the children's, child j is accepted if
// u_j (W + sum of w_i, i >= j) < w_j.  Where none is, a second pass over the
// row, which is in L1 by then, draws among the other tokens; noise is read there
// alone.  With draft logits the residual is max(a p - b q, 0), a and b two
// numbers that a rejection changes: max(r / s - q, 0) with s the sum of r gives
// a / s and (b + s) / s times s; a further pass over both rows gives each sum, one
// for every rejected child but the last.
//
// Sums.  exp(scale (l - m)) with m a largest logit, so that the difference is
// good to its own size.  A thread has its own m; maxima and sums are joined in
// one order, by shuffles, through shared memory and through the cluster's.
//
// The draw takes the largest log2 r(k) - log2 e(k).  Where another one is nearer
// to it than fp32 can tell (one draw in some ten thousand), a further pass
// compares those in fp64.  A residual a p - b q is a difference of fp32 numbers,
// good to 2^-20 of a p + b q: what it does not resolve is drawn from with that
// probability at most.
//
// What bounds it is the walk, not the rows: a level is one row from memory, then
// a join over the block and the cluster, about 4.5 us with 128 KB a block.  So
// the loads of a level are all under way at once as far as registers go, and a
// block holds what it needs of the tree.  Measured (GB300): one sequence of 5
// nodes, 32,000 fp32 logits, 3 accepted: 8 us.  16 sequences of 8, 131,072 bf16
// logits with draft logits, up to 8 accepted: 40 us.  64 trees of 32, 32,003 bf16
// logits: 25 us.  Greedy, 32 trees of 16, 131,072 fp32 logits, up to 9 accepted:
// 31 us.
#include <cstring>
#include <type_traits>

#include "sz_cache.cuh"
#include "sz_params.h"

namespace sz {
namespace {

constexpr uint32_t kThreads = 512, kWarps = kThreads / 32;
constexpr uint32_t kMaxCluster = 8;
constexpr uint32_t kFilter = 4096;  // bits of the filter for children's tokens
constexpr float kNegInf = -__builtin_huge_valf();

enum Mode { kGreedy, kCertain, kDraft };

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A word of this block's shared memory as block `rank` of the cluster holds it.
__device__ __forceinline__ uint32_t peer_word(const uint32_t* p, uint32_t rank) {
    uint32_t a, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float log2_fast(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T>
__device__ __forceinline__ float value_at(const T* p, uint32_t k) {
    if constexpr (sizeof(T) == 2)
        return bf16_float(p[k]);
    else
        return p[k];
}
// The values of 16 bytes of a row, as they are loaded.
template <typename T>
struct Row {
    static constexpr uint32_t kN = 16 / sizeof(T);
    uint32_t w[4];
    __device__ __forceinline__ void load(const T* p) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
    __device__ __forceinline__ void get(float (&x)[kN]) const {
#pragma unroll
        for (uint32_t j = 0; j < 4; j++) {
            if constexpr (sizeof(T) == 2)
                x[2 * j] = __uint_as_float(w[j] << 16), x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            else
                x[j] = __uint_as_float(w[j]);
        }
    }
};
// As many values of the noise.
template <uint32_t N>
__device__ __forceinline__ void load_noise(const float* p, float (&e)[N]) {
#pragma unroll
    for (uint32_t j = 0; j < N; j += 4) {
        const float4 n = *reinterpret_cast<const float4*>(p + j);
        e[j] = n.x, e[j + 1] = n.y, e[j + 2] = n.z, e[j + 3] = n.w;
    }
}
// Elements that p is behind a 16-byte boundary.
template <typename T>
__device__ __forceinline__ uint32_t behind(const T* p) {
    return (uint32_t)(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(T));
}

// What threads find out in a pass, and what is joined:
// the largest logit m and the sum of 2^(c (l - m)),
struct Sums {
    float m, sum;
};
struct Pair {  // the same of both rows,
    Sums p, q;
};
struct Draw {  // the largest score, its token (-1: none), and the largest of all others,
    float score;
    int32_t k;
    float runner;
};
struct Precise {  // and a draw in fp64.
    double value;
    int32_t k, pad;
};

__device__ __forceinline__ float or_zero(float m) { return m == kNegInf ? 0.f : m; }
__device__ __forceinline__ void add_sums(Sums& x, const Sums& y, float c) {
    const float top = fmaxf(x.m, y.m), ref = or_zero(top);
    x.sum = x.sum * exp2_fast((x.m - ref) * c) + y.sum * exp2_fast((y.m - ref) * c);
    x.m = top;
}
// Raises m to a larger `top`.
__device__ __forceinline__ void raise(Sums& x, float top, float c) {
    if (top > x.m) {
        x.sum *= exp2_fast((x.m - top) * c);
        x.m = top;
    }
}
__device__ __forceinline__ void offer(Draw& x, float score, int32_t k) {
    if (score > x.score) {
        x.runner = x.score;
        x.score = score;
        x.k = k;
    } else {
        x.runner = fmaxf(x.runner, score);
    }
}
// Equal scores leave a runner-up that is as good: they are compared again.
__device__ __forceinline__ void add_draw(Draw& x, const Draw& y) {
    const bool other = y.score > x.score;
    x.runner = fmaxf(fmaxf(x.runner, y.runner), other ? x.score : y.score);
    if (other) x.score = y.score, x.k = y.k;
}

// What a residual's value is made of.
template <typename T>
struct Residual {
    const T *p, *q;  // rows; q with DRAFT alone
    const float* noise;
    float c;              // scale * log2(e)
    float scale;
    float mp, mq, a, b;   // a 2^(c (l - mp)) - b 2^(c (d - mq)); mp the row's largest logit
    template <bool DRAFT>
    __device__ __forceinline__ float score(float l, float d, float e) const {
        if constexpr (DRAFT) {
            const float r = a * exp2_fast((l - mp) * c) - b * exp2_fast((d - mq) * c);
            return r > 0.f ? log2_fast(r) - log2_fast(e) : kNegInf;
        } else {
            // Less the row's largest logit, so that neither overflows nor takes
            // the noise's bits.
            return fmaf(l - mp, c, -log2_fast(e));
        }
    }
    // ln(r / e) in fp64.
    template <bool DRAFT>
    __device__ __noinline__ double value(uint32_t k) const {
        const double l = value_at(p, k), e = noise[k];
        if constexpr (DRAFT) {
            const double r = (double)a * exp((l - (double)mp) * (double)scale) -
                             (double)b * exp(((double)value_at(q, k) - (double)mq) * (double)scale);
            return log(r) - log(e);
        } else {
            return (l - (double)mp) * (double)scale - log(e);
        }
    }
    // Whether the winner of a draw is sure: lg2 is good to 2^-22 of numbers below
    // 150, the difference and the fma to 2^-24 of numbers below 150 + |s|.
    static __device__ __forceinline__ float doubt(float s) { return 1e-4f + 1e-6f * fabsf(s); }
};

template <typename T, Mode MODE>
__global__ void __launch_bounds__(kThreads, MODE == kDraft ? 1 : 2) verify_kernel(const VerifyParams p) {
    using R = Row<T>;
    constexpr uint32_t kN = R::kN;
    constexpr bool GREEDY = MODE == kGreedy;
    constexpr uint32_t kWords = 4;  // of what is joined, at most
    __shared__ uint32_t s_out[2][kWords];  // of this block's passes, in turn
    __shared__ uint32_t s_part[kWarps][kWords], s_all[kWords];
    __shared__ uint32_t s_filter[kFilter / 32];
    __shared__ int32_t s_child[kMaxNodes], s_token[kMaxNodes];
    __shared__ float s_w[kMaxNodes], s_q[kMaxNodes], s_uniform[kMaxNodes];
    __shared__ int32_t s_parent[kMaxNodes], s_drafted[kMaxNodes];
    __shared__ uint32_t s_first[2];
    const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t rank = cluster_rank(), ranks = cluster_size(), b = blockIdx.x / ranks;
    for (uint32_t k = tid; k < kFilter / 32; k += kThreads) s_filter[k] = 0;
    wait_for_previous();
    const int32_t given = p.counts ? p.counts[b] : (int32_t)p.nodes;
    const bool count_ok = given >= 0 && (uint32_t)given <= p.nodes;
    const uint32_t count = count_ok ? (uint32_t)given : 0u;
    int32_t* path = p.path + (uint64_t)b * p.nodes;
    if (tid < count) {
        s_parent[tid] = p.parents[(uint64_t)b * p.nodes + tid];
        s_drafted[tid] = p.tokens[(uint64_t)b * p.nodes + tid];
        s_uniform[tid] = GREEDY ? 0.f : p.uniforms[(uint64_t)b * p.nodes + tid];
    }
    __syncthreads();
    const bool writer = rank == 0 && tid == 0;
    const float c = p.scale * 1.4426950408889634f;
    const uint32_t stride = ranks * kThreads;
    uint32_t turn = 0, accepted = 0;
    int32_t next = -1;
    bool bad = !count_ok;  // to be reported

    // Joins every thread's part over the cluster, in one order; all threads get
    // the result.  into(x, y): y's part into x's.
    auto join = [&](auto x, const auto& into) {
        using P = decltype(x);
        constexpr int W = sizeof(P) / 4;
        static_assert(W <= (int)kWords && sizeof(P) % 4 == 0, "shared memory of a join");
        struct Raw {
            uint32_t w[W];
        };
        auto raw_of = [](const P& y) {
            Raw r;
            memcpy(&r, &y, sizeof(P));
            return r;
        };
        auto part_of = [](const Raw& r) {
            P y;
            memcpy(&y, &r, sizeof(P));
            return y;
        };
        auto across = [&](uint32_t from) {  // the warp's lanes, those from 2 `from` on apart
            for (uint32_t d = from; d; d /= 2) {
                Raw r = raw_of(x);
#pragma unroll
                for (int j = 0; j < W; j++) r.w[j] = __shfl_xor_sync(0xFFFFFFFFu, r.w[j], d);
                // The lower lane's first, on both sides.
                P low = lane & d ? part_of(r) : x;
                into(low, lane & d ? x : part_of(r));
                x = low;
            }
        };
        across(16);
        if (lane == 0) {
            const Raw r = raw_of(x);
#pragma unroll
            for (int j = 0; j < W; j++) s_part[warp][j] = r.w[j];
        }
        __syncthreads();
        if (warp == 0) {
            Raw r;
#pragma unroll
            for (int j = 0; j < W; j++) r.w[j] = s_part[lane % kWarps][j];
            x = part_of(r);
            across(kWarps / 2);
            r = raw_of(x);
            if (lane == 0) {
#pragma unroll
                for (int j = 0; j < W; j++) (ranks > 1 ? s_out[turn] : s_all)[j] = r.w[j];
            }
            __syncwarp();
        }
        if (ranks > 1) {
            cluster_sync();
            if (warp == 0) {
                Raw r;
#pragma unroll
                for (int j = 0; j < W; j++) r.w[j] = peer_word(&s_out[turn][j], lane % ranks);
                x = part_of(r);
                across(ranks / 2);
                r = raw_of(x);
                if (lane == 0) {
#pragma unroll
                    for (int j = 0; j < W; j++) s_all[j] = r.w[j];
                }
            }
        }
        __syncthreads();
        turn ^= 1;
        Raw r;
#pragma unroll
        for (int j = 0; j < W; j++) r.w[j] = s_all[j];
        return part_of(r);
    };
    // One pass over a row (or two, and the noise): visit(index of the first of
    // some neighbours, logits, draft's, noise).  Vectors begin where the row's
    // memory has its 16-byte boundaries, so that any row is read by them, and what
    // is in front of the first and behind the last is visited one by one; so is
    // everything where a draft row or the noise lies otherwise than the row.
    // Several loads are under way together, as many as registers hold.
    auto sweep = [&](const T* row, const T* row2, const float* noise, auto two, auto noisy, const auto& visit) {
        constexpr bool TWO = decltype(two)::value, NOISY = decltype(noisy)::value;
        // Words that are asked for together.  Measured: greedy, 131,072 fp32 logits,
        // 16 / 32 / 64 words: 39 / 31 / 55 us; certain, 32,003 bf16 logits, 16 / 24 /
        // 32: 26.5 / 26 / 29; draft, 131,072 bf16, 16 / 32 / 48: 44 / 39.5 / 41.
        constexpr uint32_t kWordsEach = (1 + TWO) * 4 + NOISY * kN;
        constexpr uint32_t kAhead = (MODE == kCertain ? 24 : 32) / kWordsEach;
        const uint32_t shift = behind(row), first = rank * kThreads + tid;
        const uint32_t head = min((kN - shift) % kN, p.vocab);
        const bool same = (!TWO || behind(row2) == shift) && (!NOISY || (behind(noise) - shift) % 4 == 0);
        const uint32_t vectors = same ? (p.vocab - head) / kN : 0u, singles = p.vocab - vectors * kN;
        struct Held {
            R x, y;
            float e[NOISY ? kN : 1];
        } held[kAhead];
        auto load = [&](Held& to, uint32_t v) {
            to = {};  // so that nothing older stays alive in its registers
            if (v >= vectors) return;
            const uint32_t k = head + v * kN;
            to.x.load(row + k);
            if constexpr (TWO) to.y.load(row2 + k);
            if constexpr (NOISY) load_noise(noise + k, to.e);
        };
#pragma unroll 1
        for (uint32_t v = first; v < vectors; v += kAhead * stride) {
#pragma unroll
            for (uint32_t u = 0; u < kAhead; u++) load(held[u], v + u * stride);
#pragma unroll
            for (uint32_t u = 0; u < kAhead; u++) {
                if (v + u * stride >= vectors) break;
                float l[kN], d[kN];
                held[u].x.get(l);
                if constexpr (TWO) held[u].y.get(d);
                visit((int32_t)(head + (v + u * stride) * kN), l, d, held[u].e);
            }
        }
        // Most often a few, so that these passes are short.
#pragma unroll 1
        for (uint32_t i = first; i < singles; i += 4 * stride) {
            float l[4][1] = {}, d[4][1] = {}, e[4][1] = {};
            auto at = [&](uint32_t u) { return i + u * stride < head || vectors == 0 ? i + u * stride : i + u * stride + vectors * kN; };
#pragma unroll
            for (uint32_t u = 0; u < 4; u++) {
                if (i + u * stride >= singles) break;
                l[u][0] = value_at(row, at(u));
                if constexpr (TWO) d[u][0] = value_at(row2, at(u));
                if constexpr (NOISY) e[u][0] = noise[at(u)];
            }
#pragma unroll
            for (uint32_t u = 0; u < 4; u++) {
                if (i + u * stride >= singles) break;
                visit((int32_t)at(u), l[u], d[u], e[u]);
            }
        }
    };
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    uint32_t children = 0;
    auto out_of_draw = [&](uint32_t k) {
        bool out = false;
        for (uint32_t j = 0; MODE == kCertain && j < children; j++) out |= (uint32_t)s_token[j] == k;
        return out;
    };
    auto into_sums = [&](Sums& x, const Sums& y) { add_sums(x, y, c); };
    // The token of a draw; where fp32 leaves it in doubt, after another pass.
    auto settle = [&](const Draw& d, const auto& res, auto draft, const T* row, const T* drow, const float* noise) {
        constexpr bool DRAFT = decltype(draft)::value;
        const float near = d.score - 2.f * res.doubt(d.score);
        if (d.k < 0 || d.runner < near) return d.k;
        Precise best{0.0, -1, 0};
#pragma unroll 1
        for (uint32_t k = rank * kThreads + tid; k < p.vocab; k += stride) {
            const float e = noise[k];
            if (!(e > 0.f) || !(res.template score<DRAFT>(value_at(row, k), DRAFT ? value_at(drow, k) : 0.f, e) >= near) || out_of_draw(k)) continue;
            const double value = res.template value<DRAFT>(k);
            if (best.k < 0 || value > best.value) best.value = value, best.k = (int32_t)k;
        }
        return join(best, [](Precise& x, const Precise& y) {
                   if (y.k >= 0 && (x.k < 0 || y.value > x.value || (y.value == x.value && y.k < x.k))) x = y;
               }).k;
    };

    for (uint32_t x = 0; count;) {
        if (writer) path[accepted] = (int32_t)x;
        accepted++;
        const T* row = static_cast<const T*>(p.logits) + (int64_t)b * p.seq + (int64_t)x * p.node;
        const T* drow = MODE == kDraft ? static_cast<const T*>(p.draft) + (int64_t)b * p.draft_seq + (int64_t)x * p.draft_node : nullptr;
        const float* noise = GREEDY ? nullptr : p.noise + (int64_t)b * p.noise_seq;
        auto vector_of = [&](int32_t t) { return ((uint32_t)t + behind(row)) / kN; };  // in a pass
        // ---- x's children, in order ----
        bool child = false;
        if (tid < kMaxNodes) child = tid > x && tid < count && s_parent[tid] == (int32_t)x;
        if (tid < kMaxNodes) {
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, child);
            if (lane == 0) s_first[warp] = who;
        }
        __syncthreads();
        const uint32_t low = s_first[0], high = s_first[1];
        children = __popc(low) + __popc(high);
        if (child) {
            const uint32_t at = tid < 32 ? __popc(low & ((1u << tid) - 1u)) : __popc(low) + __popc(high & ((1u << (tid - 32)) - 1u));
            const int32_t t = s_drafted[tid];
            s_child[at] = (int32_t)tid;
            s_token[at] = t;
            if (MODE == kCertain && (uint32_t)t < p.vocab) atomicOr(&s_filter[vector_of(t) % kFilter / 32], 1u << (vector_of(t) % 32));
        }
        __syncthreads();
        // Threads below `children` have a child each.
        const int32_t token = tid < children ? s_token[tid] : -1;
        const bool known = tid < children && (uint32_t)token < p.vocab;
        bad |= tid < children && !known;

        const bool leaf = children == 0;
        int32_t go = -1;  // the accepted child
        if constexpr (GREEDY) {
            Draw best{kNegInf, -1, 0.f};
            sweep(row, row, nullptr, no, no, [&](int32_t k, const auto& l, const auto&, const auto&) {
                constexpr uint32_t n = sizeof(l) / sizeof(float);
#pragma unroll
                for (uint32_t j = 0; j < n; j++) {
                    // A NaN or +infinity leaves a sum that is not 0.
                    best.runner += l[j] == kNegInf ? 0.f : l[j] * 0.f;
                    // Vectors come in ascending order, the single values in
                    // front of them last.
                    if (l[j] > best.score || (n == 1 && l[j] == best.score && k < best.k)) best.score = l[j], best.k = k + (int32_t)j;
                }
            });
            const Draw got = join(best, [](Draw& x, const Draw& y) {
                x.runner += y.runner;
                if (y.k >= 0 && (x.k < 0 || y.score > x.score || (y.score == x.score && y.k < x.k))) x.score = y.score, x.k = y.k;
            });
            const bool fine = got.runner == 0.f && got.k >= 0;
            bad |= !fine;
            next = fine ? got.k : -1;
            const uint32_t hit = tid < kMaxNodes ? __ballot_sync(0xFFFFFFFFu, known && fine && token == got.k) : 0u;
            if (lane == 0 && tid < kMaxNodes) s_first[warp] = hit;
            __syncthreads();
            const uint32_t first = s_first[0] ? __ffs(s_first[0]) - 1 : s_first[1] ? 31 + __ffs(s_first[1]) : children;
            if (first < children) go = s_child[first];
        } else if (MODE == kCertain || leaf) {
            Residual<T> res{row, nullptr, noise, c, p.scale, 0.f, 0.f, 1.f, 0.f};
            // Asked for now, looked at after the pass.
            const float l = known ? value_at(row, (uint32_t)token) : kNegInf;
            Sums got{kNegInf, 0.f};
            // A bit for each of a vector's values that is a child's token.
            auto excluded = [&](int32_t k, uint32_t n) {
                const uint32_t v = vector_of(k);
                uint32_t out = 0;
                if (MODE == kCertain && s_filter[v % kFilter / 32] >> (v % 32) & 1u)
                    for (uint32_t j = 0; j < children; j++)
                        if ((uint32_t)(s_token[j] - k) < n) out |= 1u << (s_token[j] - k);
                return out;
            };
            sweep(row, row, nullptr, no, no, [&](int32_t k, const auto& x, const auto&, const auto&) {
                constexpr uint32_t n = sizeof(x) / sizeof(float);
                float l[n];
#pragma unroll
                for (uint32_t j = 0; j < n; j++) l[j] = x[j];
                if (const uint32_t out = excluded(k, n)) {
#pragma unroll
                    for (uint32_t j = 0; j < n; j++)
                        if (out >> j & 1u) l[j] = kNegInf;
                }
                float top = l[0];
#pragma unroll
                for (uint32_t j = 1; j < n; j++) top = fmaxf(top, l[j]);
                raise(got, top, c);
                const float ref = or_zero(got.m);
#pragma unroll
                for (uint32_t j = 0; j < n; j++) got.sum += exp2_fast((l[j] - ref) * c);
            });
            got = join(got, into_sums);
            // ---- the children ----
            if (tid < kMaxNodes) {
                float top = l, nan = l != l ? 1.f : 0.f;
#pragma unroll
                for (uint32_t d = 16; d; d /= 2) {
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                    nan = fmaxf(nan, __shfl_xor_sync(0xFFFFFFFFu, nan, d));
                }
                if (lane == 0) s_part[warp][0] = __float_as_uint(top), s_part[warp][1] = __float_as_uint(nan);
            }
            __syncthreads();
            const float m = fmaxf(got.m, fmaxf(__uint_as_float(s_part[0][0]), __uint_as_float(s_part[1][0])));
            const bool fine = m > kNegInf && m < __builtin_huge_valf() && got.sum == got.sum && (s_part[0][1] | s_part[1][1]) == 0;
            if (tid < kMaxNodes) {
                bool again = false;  // an earlier child has the same token
                for (uint32_t j = 0; j < tid && j < children; j++) again |= s_token[j] == token;
                s_w[tid] = known && !again && fine ? exp2_fast((l - m) * c) : 0.f;
            }
            __syncthreads();
            if (tid < kMaxNodes) {
                float left = got.sum * exp2_fast((got.m - m) * c);
                for (uint32_t j = children; j > tid; j--) left += s_w[j - 1];
                const bool take = known && fine && s_uniform[s_child[tid]] * left < s_w[tid];
                const uint32_t hit = __ballot_sync(0xFFFFFFFFu, take);
                if (lane == 0) s_first[warp] = hit;
            }
            __syncthreads();
            const uint32_t first = s_first[0] ? __ffs(s_first[0]) - 1 : s_first[1] ? 31 + __ffs(s_first[1]) : children;
            if (first < children) go = s_child[first];
            next = -1;
            res.mp = m;
            if (go < 0 && fine) {
                Draw best{kNegInf, -1, kNegInf};
                sweep(row, row, noise, no, yes, [&](int32_t k, const auto& l, const auto&, const auto& e) {
                    constexpr uint32_t n = sizeof(l) / sizeof(float);
                    const uint32_t out = excluded(k, n);
#pragma unroll
                    for (uint32_t j = 0; j < n; j++)
                        offer(best, e[j] > 0.f && !(out >> j & 1u) ? res.template score<false>(l[j], 0.f, e[j]) : kNegInf, k + (int32_t)j);
                });
                next = settle(join(best, add_draw), res, no, row, row, noise);
            }
            bad |= !fine || (go < 0 && next < 0);
            __syncthreads();  // the filter has been read
            if (known && MODE == kCertain) s_filter[vector_of(token) % kFilter / 32] = 0;
        } else {
            // ---- draft logits: both rows' sums ----
            // The children's, asked for now, looked at after the pass.
            const float lp = known ? value_at(row, (uint32_t)token) : kNegInf, lq = known ? value_at(drow, (uint32_t)token) : kNegInf;
            Pair part{{kNegInf, 0.f}, {kNegInf, 0.f}};
            sweep(row, drow, nullptr, yes, no, [&](int32_t, const auto& l, const auto& d, const auto&) {
                constexpr uint32_t n = sizeof(l) / sizeof(float);
                float top = kNegInf, top2 = kNegInf;
#pragma unroll
                for (uint32_t j = 0; j < n; j++) top = fmaxf(top, l[j]), top2 = fmaxf(top2, d[j]);
                raise(part.p, top, c);
                raise(part.q, top2, c);
                const float ref = or_zero(part.p.m), ref2 = or_zero(part.q.m);
#pragma unroll
                for (uint32_t j = 0; j < n; j++) {
                    part.p.sum += exp2_fast((l[j] - ref) * c);
                    part.q.sum += exp2_fast((d[j] - ref2) * c);
                }
            });
            part = join(part, [&](Pair& x, const Pair& y) {
                add_sums(x.p, y.p, c);
                add_sums(x.q, y.q, c);
            });
            const Sums sp = part.p, sq = part.q;
            if (tid < children) s_w[tid] = lp, s_q[tid] = lq;
            __syncthreads();
            auto usable = [](const Sums& s) { return s.m > kNegInf && s.m < __builtin_huge_valf() && s.sum == s.sum; };
            const bool fine = usable(sp), both = fine && usable(sq);
            bad |= !both;
            Residual<T> res{row, drow, noise, c, p.scale, sp.m, sq.m, 1.f / sp.sum, 0.f};
            const float unit = both ? 1.f / sq.sum : 0.f;  // b is in units of 1 / q's sum
            float bq = 0.f;
            for (uint32_t j = 0; j < children && both && go < 0; j++) {
                const int32_t t = s_token[j];
                if ((uint32_t)t < p.vocab) {
                    // u q < r over q, from the logits' difference: neither
                    // underflows, and a q of 0 leaves an infinity where p is above 0.
                    // Their products with c may overflow one by one.
                    const float x = (s_w[j] - sp.m) - (s_q[j] - sq.m);
                    if (s_uniform[s_child[j]] + bq < res.a * sq.sum * exp2_fast(x * c)) {
                        go = s_child[j];
                        break;
                    }
                }
                if (j + 1 == children) break;
                // The next one's residual.
                Sums left{0.f, 0.f};
                sweep(row, drow, nullptr, yes, no, [&](int32_t, const auto& l, const auto& d, const auto&) {
                    constexpr uint32_t n = sizeof(l) / sizeof(float);
#pragma unroll
                    for (uint32_t i = 0; i < n; i++)
                        left.sum += fmaxf(res.a * exp2_fast((l[i] - sp.m) * c) - (bq + 1.f) * unit * exp2_fast((d[i] - sq.m) * c), 0.f);
                });
                const float s = join(left, into_sums).sum;
                if (s > 0.f) res.a /= s, bq = (bq + 1.f) / s;
            }
            next = -1;
            // With the last rejection, or without it where nothing is left.
            for (int last = both ? 1 : 0; last >= 0 && go < 0 && fine && next < 0; last--) {
                res.b = (bq + (float)last) * unit;
                Draw best{kNegInf, -1, kNegInf};
                if (res.b == 0.f) {
                    sweep(row, row, noise, no, yes, [&](int32_t k, const auto& l, const auto&, const auto& e) {
                        constexpr uint32_t n = sizeof(l) / sizeof(float);
#pragma unroll
                        for (uint32_t i = 0; i < n; i++)
                            offer(best, e[i] > 0.f ? res.template score<false>(l[i], 0.f, e[i]) : kNegInf, k + (int32_t)i);
                    });
                    next = settle(join(best, add_draw), res, no, row, row, noise);
                } else {
                    sweep(row, drow, noise, yes, yes, [&](int32_t k, const auto& l, const auto& d, const auto& e) {
                        constexpr uint32_t n = sizeof(l) / sizeof(float);
#pragma unroll
                        for (uint32_t i = 0; i < n; i++)
                            offer(best, e[i] > 0.f ? res.template score<true>(l[i], d[i], e[i]) : kNegInf, k + (int32_t)i);
                    });
                    next = settle(join(best, add_draw), res, yes, row, drow, noise);
                }
            }
            bad |= go < 0 && next < 0;
        }
        __syncthreads();  // what was read of this node is written for the next one
        if (go < 0) break;
        x = (uint32_t)go;
    }
    bad = __syncthreads_or(bad);
    if (rank == 0) {
        for (uint32_t k = accepted + tid; k < p.nodes; k += kThreads) path[k] = -1;
        if (tid == 0) {
            p.accepted[b] = (int32_t)accepted;
            p.next[b] = next;
            if (bad && p.status) atomicMax(p.status, kStatusInvalid);
        }
    }
    cluster_sync();  // no block ends while another reads its shared memory
}

template <typename T, Mode MODE>
cudaError_t launch(const VerifyParams& p, cudaStream_t s) {
    int sms = 0, per_sm = 0;
    const cudaError_t err = kernel_fit(reinterpret_cast<const void*>(verify_kernel<T, MODE>), kThreads, 0, &sms, &per_sm);
    if (err != cudaSuccess) return err;
    // As many blocks a sequence as run at once, with half a vector or more for
    // every thread: a level's time is that of a block's share (greedy, 32 trees of
    // 131,072 fp32 logits: 31 us with 8 blocks a sequence, 37 with 4; twice as many
    // as run at once: 37 to 44).  Two blocks fit on a processor but with draft
    // logits, where 64 registers a thread are too few.
    uint32_t ranks = kMaxCluster;
    while (ranks > 1 && ((uint64_t)p.batch * ranks > (uint64_t)sms * per_sm || (uint64_t)ranks * kThreads * Row<T>::kN >= 2ull * p.vocab)) ranks /= 2;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.batch * ranks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_kernel<T, MODE>, p);
}

template <typename T>
cudaError_t launch_type(const VerifyParams& p, cudaStream_t s) {
    if (!p.uniforms) return launch<T, kGreedy>(p, s);
    return p.draft ? launch<T, kDraft>(p, s) : launch<T, kCertain>(p, s);
}

}  // namespace

cudaError_t launch_verify_tree(const VerifyParams& p, cudaStream_t s) {
    return p.f32 ? launch_type<float>(p, s) : launch_type<uint16_t>(p, s);
}

}  // namespace sz
