// Log probabilities of given tokens, with their ranks, the rows' entropies and the best
// alternatives.  The definition is in include/mla_decode.h (mla_token_logprobs).
//
// One pass over a row.  With c = scale log2 e and a reference m, the maximum of xc so far, a thread keeps s = sum 2^(xc - m) and w = sum 2^(xc - m) (xc - m) of its
// share; when the reference moves by d = m - m', s becomes 2^d s and w becomes 2^d (w + d s).  Then
//   log p(x) = ln 2 (xc - m - log2 s),   H = ln 2 (log2 s - w / s):
// both terms of H are >= 0, so nothing cancels.  Sums and references are fp32.
//
// The best alternatives come out of the same pass: a thread's share of the row is a stripe of 16-byte
// units, and it keeps the stripe's maximum.  The k-th largest of those maxima is a lower bound of
// the k-th best logit, and only the batches of units that reach it - about k of them - are read again
// (from L2) for the tokens that reach it.  Rows where more than kCandidates do (many equal logits) take
// one pass for each alternative instead.
//
// A CTA takes a row after the other, the next one's first loads under the end of the present one; with few
// rows a cluster of up to eight CTAs shares one, its parts joined through distributed shared memory.
//
// 4,096 rows of 131,072 bf16 logits: 155 us for the sums alone (1.07 GB, a copy's rate), 176 with ranks of random
// tokens (159 where all are the best), 193 with the best alternative too, 201 with 20: issue slots are 60 % busy, and a
// row's end is a chain.  16-bit logits are therefore compared in pairs (bf16 ones clamped in pairs, too), and summed in
// packed fp32, and a batch is read while the one before is worked on (211 -> 201 us).  fp16, whose values are clamped one
// by one, as its range does not hold every limit: 186 us with ranks, 210 with 20 alternatives.  The same bytes in fp32:
// 159 and 177.  Few rows: 9 us, a chain of the loads, the joins and (with several CTAs) two cluster barriers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "sm103_ptx.cuh"
#include "tc_util.cuh"

namespace mla {
namespace {

constexpr int kLpSms = 152;          // a GB300's; only the grid's shape depends on it
constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
// 16-byte units of a thread in flight together, and CTAs per SM: 4,096 rows of 131,072 without and with 20 alternatives
// 176 and 201 us; 4 and 4: 184 and 213, 12 and 2: 203 and 258, 16 and 2: 187 and 243
constexpr int kLpBatch = 8;
constexpr int kLpCtas = 3;
constexpr int kLpMaxTop = 64;
constexpr int kCandidates = 1024;   // at least kLpMaxTop units' values
constexpr int kListed = 1024;       // batches that are read again
constexpr int kLpMaxCluster = 8;
constexpr int kLpShared = 2;        // CTAs per SM up to which rows are shared (see launch_logprobs)
constexpr unsigned kFull = 0xffffffffu;

struct LogprobArgs {
    const void *logits;
    int64_t row_stride;  // in elements
    int64_t N;
    int V, parts;        // parts: CTAs per row
    const int32_t *tokens;
    float scale, scale_log2;
    int top;
    float *logprob, *entropy;
    int32_t *rank, *top_tokens;
    float *top_logprobs;
    int *status;
};

// What the pass does with a 16-byte unit of each type: the largest of a batch's values; its values as
// packed fp32 pairs, those below `low` (whose weight is 0 in fp32) raised to it, so that -inf leaves the
// sums alone; and how many are above (or not below) a value.
struct Bf16 {
    using Raw = uint16_t;
    static constexpr int kUnit = 8;
    static constexpr uint32_t kMinusInf = 0xFF80FF80u;
    static __device__ __forceinline__ float value(Raw r) { return bf16_to_f32(r); }
    static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
    static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ float most(const uint4 *v, int n) {
        uint32_t m = kMinusInf;
#pragma unroll
        for (int q = 0; q < n; ++q) m = max2(m, max2(max2(v[q].x, v[q].y), max2(v[q].z, v[q].w)));
        return fmaxf(lo(m), hi(m));
    }
    // `low` rounded down to bf16 and doubled
    static __device__ __forceinline__ uint32_t floor2(float low) {
        const __nv_bfloat16 r = __float2bfloat16_rd(low);
        const uint32_t b = *reinterpret_cast<const uint16_t *>(&r);
        return b | b << 16;
    }
    using Low = uint32_t;
    static __device__ __forceinline__ Low low_of(float low) { return floor2(low); }
    static __device__ __forceinline__ void pairs(uint4 v, Low low, uint64_t (&f)[4]) {
        const uint32_t w[4] = {max2(v.x, low), max2(v.y, low), max2(v.z, low), max2(v.w, low)};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = pair(lo(w[i]), hi(w[i]));
    }
    static __device__ __forceinline__ void unpack(uint4 v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = lo(w[i]);
            f[2 * i + 1] = hi(w[i]);
        }
    }
    // (two counts of at most 4 n, exact in bf16)
    template <bool kEqual>
    static __device__ __forceinline__ float above(const uint4 *v, int n, float x) {
        const __nv_bfloat162 y = __float2bfloat162_rn(x);  // (exact: a logit)
        __nv_bfloat162 s = __float2bfloat162_rn(0.f);
#pragma unroll
        for (int q = 0; q < n; ++q) {
            const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 z = *reinterpret_cast<const __nv_bfloat162 *>(&w[i]);
                s = __hadd2(s, kEqual ? __hge2(z, y) : __hgt2(z, y));
            }
        }
        const uint32_t c = *reinterpret_cast<const uint32_t *>(&s);
        return lo(c) + hi(c);
    }
};
struct Fp16 {
    using Raw = uint16_t;
    static constexpr int kUnit = 8;
    static constexpr uint32_t kMinusInf = 0xFC00FC00u;
    static __device__ __forceinline__ float value(Raw r) { return __half2float(__ushort_as_half(r)); }
    static __device__ __forceinline__ float2 both(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ float most(const uint4 *v, int n) {
        uint32_t m = kMinusInf;
#pragma unroll
        for (int q = 0; q < n; ++q) m = max2(m, max2(max2(v[q].x, v[q].y), max2(v[q].z, v[q].w)));
        return fmaxf(both(m).x, both(m).y);
    }
    using Low = float;  // (beyond this type's range where the scale is small)
    static __device__ __forceinline__ Low low_of(float low) { return low; }
    static __device__ __forceinline__ void pairs(uint4 v, Low low, uint64_t (&f)[4]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = pair(fmaxf(both(w[i]).x, low), fmaxf(both(w[i]).y, low));
    }
    static __device__ __forceinline__ void unpack(uint4 v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = both(w[i]).x;
            f[2 * i + 1] = both(w[i]).y;
        }
    }
    template <bool kEqual>
    static __device__ __forceinline__ float above(const uint4 *v, int n, float x) {
        const __half2 y = __float2half2_rn(x);  // (exact: a logit)
        __half2 s = __float2half2_rn(0.f);
#pragma unroll
        for (int q = 0; q < n; ++q) {
            const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 z = *reinterpret_cast<const __half2 *>(&w[i]);
                s = __hadd2(s, kEqual ? __hge2(z, y) : __hgt2(z, y));
            }
        }
        const float2 c = __half22float2(s);
        return c.x + c.y;
    }
};
struct Fp32 {
    using Raw = float;
    static constexpr int kUnit = 4;
    static constexpr uint32_t kMinusInf = 0xFF800000u;
    static __device__ __forceinline__ float value(Raw r) { return r; }
    static __device__ __forceinline__ void unpack(uint4 v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ float most(const uint4 *v, int n) {
        float m = -INFINITY;
#pragma unroll
        for (int q = 0; q < n; ++q) {
            float f[4];
            unpack(v[q], f);
            m = max3(max3(m, f[0], f[1]), f[2], f[3]);
        }
        return m;
    }
    using Low = float;
    static __device__ __forceinline__ Low low_of(float low) { return low; }
    static __device__ __forceinline__ void pairs(uint4 v, Low low, uint64_t (&f)[2]) {
        float x[4];
        unpack(v, x);
        f[0] = pair(fmaxf(x[0], low), fmaxf(x[1], low));
        f[1] = pair(fmaxf(x[2], low), fmaxf(x[3], low));
    }
    template <bool kEqual>
    static __device__ __forceinline__ float above(const uint4 *v, int n, float x) {
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < n; ++q) {
            float f[4];
            unpack(v[q], f);
#pragma unroll
            for (int i = 0; i < 4; ++i) s += (kEqual ? f[i] >= x : f[i] > x) ? 1.f : 0.f;
        }
        return s;
    }
};

// A row as 16-byte units: unit u holds tokens first + u * kUnit ... (the first and the last unit may
// reach over the row's ends; what lies there is not read and counts as -inf).
template <typename T>
struct Row {
    const typename T::Raw *p;
    int first, V, units;

    __device__ __forceinline__ Row(const typename T::Raw *row, int v) : p(row), V(v) {
        const int past = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(typename T::Raw));
        first = -past;
        units = (int)(((int64_t)v + past + T::kUnit - 1) / T::kUnit);
    }
    __device__ __forceinline__ int token(int u) const { return first + u * T::kUnit; }
    // units that lie within the row: whole_begin() .. whole_end()
    __device__ __forceinline__ int whole_begin() const { return first < 0 ? 1 : 0; }
    __device__ __forceinline__ int whole_end() const { return (V - first) / T::kUnit; }
    __device__ __forceinline__ const uint4 *at(int u) const {
        return reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15)) + u;
    }
    __device__ __forceinline__ uint4 load(int u) const {
        const int e = token(u);
        if (e >= 0 && e <= V - T::kUnit) return *reinterpret_cast<const uint4 *>(p + e);
        uint4 v = make_uint4(T::kMinusInf, T::kMinusInf, T::kMinusInf, T::kMinusInf);
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < T::kUnit; ++i) {
            if (e + i < 0 || e + i >= V) continue;
            if constexpr (sizeof(typename T::Raw) == 4) {
                w[i] = __float_as_uint(p[e + i]);
            } else {
                const uint32_t r = p[e + i];
                w[i / 2] = i % 2 ? (w[i / 2] & 0xFFFFu) | r << 16 : (w[i / 2] & 0xFFFF0000u) | r;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Whole numbers in the order of the floats (-0 as +0), above 0 for every float but -inf and below.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
// A token's place among the alternatives: larger logits first, then lower tokens.
__device__ __forceinline__ uint64_t place_key(float x, int token) {
    return (uint64_t)ordered(x) << 32 | (uint32_t)~token;
}

struct Part {
    float m, s, w;  // the largest logit (-inf: nothing yet), sums
    int ahead;      // tokens before the given one in the order of place_key
};

// Two parts' sums under the larger of their maxima; c = scale log2 e.
__device__ __forceinline__ Part join(const Part &a, const Part &b, float c) {
    Part r;
    r.ahead = a.ahead + b.ahead;
    r.m = fmaxf(a.m, b.m);
    if (r.m == -INFINITY) {
        r.s = r.w = 0.f;
        return r;
    }
    const float da = fmaxf((a.m - r.m) * c, -200.f), db = fmaxf((b.m - r.m) * c, -200.f);  // (2^-200: 0 in fp32)
    const float fa = ptx::ex2_approx(da), fb = ptx::ex2_approx(db);
    r.s = a.s * fa + b.s * fb;
    r.w = fa * (a.w + a.s * da) + fb * (b.w + b.s * db);
    return r;
}

struct Shared {
    Part warp[kLpWarps];
    Part cta;                       // read by the cluster's first CTA
    uint32_t stripe[kLpThreads];    // each stripe's maximum, as ordered()
    uint32_t limit;
    int listed, candidates;
    int from[kListed];              // batches that reach the limit: their first units
    uint64_t key[kCandidates];
    uint64_t best[kLpMaxTop];       // this CTA's alternatives in order (0: none); read by the first CTA
    uint64_t warp_key[kLpWarps];
};

// Puts the `top` largest of the n keys (all different) into best, in order; 0 where there are fewer.
__device__ __forceinline__ void pick(const uint64_t *key, int n, uint64_t *best, int top) {
    for (int i = threadIdx.x; i < top; i += kLpThreads)
        if (i >= n) best[i] = 0;
    for (int i = threadIdx.x; i < n; i += kLpThreads) {
        const uint64_t k = key[i];
        int r = 0;
        for (int j = 0; j < n; ++j) r += key[j] > k;
        if (r < top) best[r] = k;
    }
}

// A thread's units u, u + kLpThreads, ... (-inf where there are none).
template <typename T>
__device__ __forceinline__ void load_batch(const Row<T> &row, int u, int u1, uint4 (&v)[kLpBatch]) {
    if (u >= row.whole_begin() && u + (kLpBatch - 1) * kLpThreads < min(u1, row.whole_end())) {
        const uint4 *from = row.at(u);
#pragma unroll
        for (int q = 0; q < kLpBatch; ++q) v[q] = from[q * kLpThreads];
        return;
    }
#pragma unroll
    for (int q = 0; q < kLpBatch; ++q) {
        v[q] = make_uint4(T::kMinusInf, T::kMinusInf, T::kMinusInf, T::kMinusInf);
        if (u + q * kLpThreads < u1) v[q] = row.load(u + q * kLpThreads);
    }
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads, kLpCtas) logprob_kernel(LogprobArgs a) {
    __shared__ Shared sh;
    grid_dep_wait();
    grid_dep_launch();
    constexpr int E = T::kUnit;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int parts = a.parts, part = blockIdx.x % parts;  // a row's CTAs are one cluster
    const float c = a.scale_log2, span = -160.f / c;
    const uint64_t c2 = pair(c, c);
    const int64_t rows_at_once = gridDim.x / parts;
    auto row_of = [&](int64_t n) {
        return Row<T>(reinterpret_cast<const typename T::Raw *>(a.logits) + n * a.row_stride, a.V);
    };
    auto part_of = [&](const Row<T> &row, int &u0, int &u1) {
        const int per = (row.units + parts - 1) / parts;
        u0 = part * per;
        u1 = min(row.units, u0 + per);
    };
    // The first batch of a row is on its way while the row before it is finished.
    uint4 v[kLpBatch];
    int64_t n = blockIdx.x / parts;
    {
        const Row<T> row = row_of(n);
        int u0, u1;
        part_of(row, u0, u1);
        load_batch(row, u0 + tid, u1, v);
    }
    for (; n < a.N; n += rows_at_once) {
        const Row<T> row = row_of(n);
        int u0, u1;
        part_of(row, u0, u1);
        const int token = a.tokens[n];
        const bool given = token >= 0 && token < a.V;
        const float mine = given ? T::value(row.p[token]) : INFINITY;
        const bool masked = mine == -INFINITY;  // all tokens below it are ahead, and those above it that are not masked
        const int own = given ? (token - row.first) / E : -1;  // the given token's unit

        // ---- the pass
        Part t{-INFINITY, 0.f, 0.f, 0};
        // the largest and the second largest of the stripe's batches, and where the largest one is
        float top = -INFINITY, second = -INFINITY;
        int top_at = u0 + tid;
        bool here = true;  // the batch is in v, or on its way
        for (int u = u0 + tid; u < u1; u += kLpBatch * kLpThreads) {
            if (!here) load_batch(row, u, u1, v);
            here = false;
            const float most = T::most(v, kLpBatch);
            // A whole batch is read while the one before it is worked on, each unit as soon as its place is free.
            const int un = u + kLpBatch * kLpThreads;
            const bool roll = un >= row.whole_begin() && un + (kLpBatch - 1) * kLpThreads < min(u1, row.whole_end());
            const uint4 *from = row.at(un);
            if (most == -INFINITY) continue;  // all masked
            if (most >= mine) {
                float ahead = 0.f;
                if (u > own) {
                    ahead = T::template above<false>(v, kLpBatch, mine);
                } else if (u + (kLpBatch - 1) * kLpThreads < own) {
                    if (!masked) ahead = T::template above<true>(v, kLpBatch, mine);
                } else {  // units on both sides of the token, or its own
#pragma unroll
                    for (int q = 0; q < kLpBatch; ++q) {
                        const int uq = u + q * kLpThreads, e = row.token(uq);
                        if (uq > own) {
                            ahead += T::template above<false>(&v[q], 1, mine);
                        } else if (uq < own) {
                            if (!masked) ahead += T::template above<true>(&v[q], 1, mine);
                        } else {
                            float f[E];
                            T::unpack(v[q], f);
#pragma unroll
                            for (int i = 0; i < E; ++i)
                                ahead += (f[i] > mine && (!masked || e + i > token)) ||
                                                 (f[i] == mine && !masked && e + i < token)
                                             ? 1.f
                                             : 0.f;
                        }
                    }
                }
                t.ahead += (int)ahead;
            }
            second = fmaxf(second, fminf(top, most));
            if (most > top) {
                top = most;
                top_at = u;
            }
            const float d = fmaxf((t.m - top) * c, -200.f), g = ptx::ex2_approx(d);
            // two chains of each sum
            uint64_t s2[2] = {pair(t.s * g, 0.f), 0}, w2[2] = {pair(g * (t.w + d * t.s), 0.f), 0};
            t.m = top;
            const uint64_t neg_m = pair(-top, -top);
            // 2^-160 is 0 in fp32.  (Rounded down, so that it stays below the maximum however large that is; at the
            // bottom of the range, where nothing does, masked tokens are told apart below.)
            const typename T::Low low = T::low_of(__fadd_rd(top, span));
            const bool bottom = top < -1e37f;
#pragma unroll
            for (int q = 0; q < kLpBatch; ++q) {
                if (bottom) break;
                uint64_t x[E / 2];
                T::pairs(v[q], low, x);
                if (roll) v[q] = from[q * kLpThreads];
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    const uint64_t y = mul2(add2(x[i], neg_m), c2);
                    const float2 e = halves(y);
                    const uint64_t p = pair(ptx::ex2_approx(e.x), ptx::ex2_approx(e.y));
                    s2[i & 1] = add2(s2[i & 1], p);
                    w2[i & 1] = fma2(p, y, w2[i & 1]);
                }
            }
            const float2 ss = halves(add2(s2[0], s2[1])), ww = halves(add2(w2[0], w2[1]));
            t.s = ss.x + ss.y;
            t.w = ww.x + ww.y;
            if (bottom) {
                for (int q = 0; q < kLpBatch; ++q) {
                    float f[E];
                    T::unpack(v[q], f);
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const float y = fmaxf((f[i] - top) * c, -200.f), e = ptx::ex2_approx(y);
                        t.s += e;
                        t.w = fmaf(e, y, t.w);
                    }
                }
            }
            here = roll && !bottom;
        }
        if (n + rows_at_once < a.N) {
            const Row<T> next = row_of(n + rows_at_once);
            int v0, v1;
            part_of(next, v0, v1);
            load_batch(next, v0 + tid, v1, v);
        }
        const uint32_t top_key = ordered(top);
        sh.stripe[tid] = top_key;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            Part b;
            b.m = __shfl_xor_sync(kFull, t.m, o);
            b.s = __shfl_xor_sync(kFull, t.s, o);
            b.w = __shfl_xor_sync(kFull, t.w, o);
            b.ahead = __shfl_xor_sync(kFull, t.ahead, o);
            t = join(t, b, c);
        }
        if (lane == 0) sh.warp[warp] = t;
        if (tid == 0) sh.listed = sh.candidates = 0;
        __syncthreads();
        if (tid == 32) {
            Part r = sh.warp[0];
            for (int i = 1; i < kLpWarps; ++i) r = join(r, sh.warp[i], c);
            sh.cta = r;
        }

        // ---- this CTA's alternatives
        if (a.top > 0) {
            if (warp == 0) {
                // the largest limit that `top` stripes reach, to 16 bits (rounded down); its upper bits are those
                // that all stripes have in common
                uint32_t k[kLpThreads / 32], least = ~0u, most = 0;
#pragma unroll
                for (int i = 0; i < kLpThreads / 32; ++i) {
                    k[i] = sh.stripe[lane + 32 * i];
                    least = min(least, k[i]);
                    most = max(most, k[i]);
                }
                least = __reduce_min_sync(kFull, least);
                most = __reduce_max_sync(kFull, most);
                int bit = least == most ? -1 : 31 - __clz(least ^ most);  // the first that differs
                uint32_t limit = bit < 0 ? most : most & ~(2u * (1u << bit) - 1u);
                for (; bit >= 16; --bit) {
                    const uint32_t l = limit | 1u << bit;
                    int cnt = 0;
#pragma unroll
                    for (int i = 0; i < kLpThreads / 32; ++i) cnt += k[i] >= l;
                    if (__reduce_add_sync(kFull, cnt) >= a.top) limit = l;
                }
                if (lane == 0) sh.limit = max(limit, ordered(-INFINITY) + 1);  // masked tokens are none
            }
            __syncthreads();
            const uint32_t limit = sh.limit;
            const float reach = unordered(limit);
            if (top_key >= limit) {
                // the batch with the stripe's maximum, or all of them where another one reaches the limit too
                const bool one = second < reach;
                const int batches = one ? 1 : (u1 - u0 - tid + kLpBatch * kLpThreads - 1) / (kLpBatch * kLpThreads);
                const int at = atomicAdd(&sh.listed, batches);
                for (int i = 0; i < batches && at + i < kListed; ++i)
                    sh.from[at + i] = one ? top_at : u0 + tid + i * kLpBatch * kLpThreads;
            }
            __syncthreads();
            const int listed = sh.listed;
            for (int i = tid; i < min(listed, kListed) * kLpBatch; i += kLpThreads) {
                const int u = sh.from[i / kLpBatch] + i % kLpBatch * kLpThreads;
                if (u >= u1) continue;
                const uint4 x = row.load(u);
                if (!(T::most(&x, 1) >= reach)) continue;
                float f[E];
                T::unpack(x, f);
                const int e = row.token(u);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    if (f[j] >= reach) {
                        const int at = atomicAdd(&sh.candidates, 1);
                        if (at < kCandidates) sh.key[at] = place_key(f[j], e + j);
                    }
                }
            }
            __syncthreads();
            const int found = sh.candidates;
            if (listed <= kListed && found <= kCandidates) {
                pick(sh.key, found, sh.best, a.top);
            } else {
                // one after the other: the largest key below the last one
                uint64_t last = ~0ull;
                for (int k = 0; k < a.top; ++k) {
                    uint64_t mx = 0;
                    for (int u = u0 + tid; u < u1; u += kLpThreads) {
                        float f[E];
                        T::unpack(row.load(u), f);
                        const int e = row.token(u);
#pragma unroll
                        for (int j = 0; j < E; ++j) {
                            const uint64_t key = place_key(f[j], e + j);
                            if (key < last && key > mx && f[j] >= reach) mx = key;
                        }
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(kFull, mx, o));
                    if (lane == 0) sh.warp_key[warp] = mx;
                    __syncthreads();
                    for (int i = 0; i < kLpWarps; ++i) mx = max(mx, sh.warp_key[i]);
                    if (tid == 0) sh.best[k] = mx;
                    last = mx;
                    __syncthreads();
                }
            }
        }
        __syncthreads();

        // ---- the row's
        Part r = sh.cta;
        if (parts > 1) {
            ptx::cluster_sync();
            if (part == 0) {
                const uint32_t here = ptx::smem_u32(&sh);
                auto peer = [&](int rank, const void *at) {
                    return ptx::mapa(here + (uint32_t)(reinterpret_cast<const char *>(at) - reinterpret_cast<const char *>(&sh)),
                                     rank);
                };
                auto ld32 = [](uint32_t at) {
                    uint32_t x;
                    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
                    return x;
                };
                auto ld64 = [](uint32_t at) {
                    uint64_t x;
                    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(x) : "r"(at) : "memory");
                    return x;
                };
                for (int q = 1; q < parts; ++q) {
                    const uint32_t at = peer(q, &sh.cta);
                    r = join(r,
                             Part{__uint_as_float(ld32(at)), __uint_as_float(ld32(at + 4)), __uint_as_float(ld32(at + 8)),
                                  (int)ld32(at + 12)},
                             c);
                }
                if (a.top > 0) {
                    // (the candidates' places are free by now)
                    if (tid == 0) sh.candidates = 0;
                    __syncthreads();
                    for (int i = tid; i < parts * a.top; i += kLpThreads) {
                        const uint64_t k = ld64(peer(i / a.top, &sh.best[i % a.top]));
                        if (k) sh.key[atomicAdd(&sh.candidates, 1)] = k;
                    }
                    __syncthreads();
                    pick(sh.key, sh.candidates, sh.best, a.top);
                    __syncthreads();
                }
            }
            ptx::cluster_sync();  // the first CTA has read the others' memory
        }
        if (part == 0) {
            const float log_s = log2f(r.s) * kLn2;
            const bool none = r.m == -INFINITY;  // every token masked
            if (tid == 0) {
                const float y = none || masked ? -INFINITY : (mine - r.m) * a.scale - log_s;
                a.logprob[n] = given ? y : token < 0 ? 0.f : NAN;
                if (a.entropy) a.entropy[n] = none ? 0.f : log_s - r.w / r.s * kLn2;
                if (a.rank) a.rank[n] = given ? r.ahead + (masked ? token : 0) : -1;
                if (token >= a.V && a.status) record_error(a.status, MLA_ERR_INDEX);
            }
            for (int i = tid; i < a.top; i += kLpThreads) {
                const uint64_t k = sh.best[i];
                a.top_tokens[n * a.top + i] = k ? (int32_t)~(uint32_t)k : -1;
                a.top_logprobs[n * a.top + i] =
                    k ? (unordered((uint32_t)(k >> 32)) - r.m) * a.scale - log_s : -INFINITY;
            }
        }
        __syncthreads();  // the shared memory is the next row's
    }
}

template <typename T>
mla_status launch_logprobs(LogprobArgs a, int64_t N, cudaStream_t stream) {
    // CTAs per row: twice as many while all rows' come to two per SM at most and each thread still has a batch of units.
    // Rows of 131,072 bf16 logits with 5 alternatives, us with 1, 2, 4 and 8 CTAs a row (* what the rule takes): 1 row 11.6,
    // 9.9, 8.7, 8.2*; 16 rows 11.9, 10.3, 9.1, 8.8*; 40 rows 12.0, 10.6, 10.0*, with three per SM 10.5; 100 rows 12.2, 13.0*,
    // with three per SM 12.7 for 4; 152 rows 15.4, 17.5*.  (Two a row cost 1 - 2 us where every SM has a row of its own.)
    const int64_t units = ((int64_t)a.V + T::kUnit - 1) / T::kUnit;
    int parts = 1;
    while (parts < kLpMaxCluster && N * parts * 2 <= kLpShared * kLpSms && units >= 2 * parts * kLpThreads * kLpBatch) parts *= 2;
    const int64_t rows = N * parts <= kLpSms * kLpCtas ? N : kLpSms * kLpCtas / parts;  // at once
    a.parts = parts;
    a.N = N;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * parts), 1, 1);
    cfg.blockDim = dim3(kLpThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = parts;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = parts > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, logprob_kernel<T>, a) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status mla_token_logprobs(const void *logits, mla_logits_dtype dtype, int64_t row_stride, int64_t N, int V,
                                         const int32_t *tokens, float scale, int top, float *logprob, float *entropy,
                                         int32_t *rank, int32_t *top_tokens, float *top_logprobs,
                                         int32_t *device_status, void *stream) {
    if (dtype != MLA_LOGITS_BF16 && dtype != MLA_LOGITS_FP16 && dtype != MLA_LOGITS_FP32) return MLA_ERR_INVALID_ARG;
    if (N < 0 || V < 1 || top < 0 || row_stride < 0) return MLA_ERR_INVALID_ARG;
    if (!(scale >= 1e-6f && scale <= 1e6f)) return MLA_ERR_INVALID_ARG;
    if (top > kLpMaxTop || V > (1 << 28) || N > (int64_t)1 << 30) return MLA_ERR_UNSUPPORTED;
    if (N == 0) return MLA_OK;
    if (!logits || !tokens || !logprob || (top > 0 && (!top_tokens || !top_logprobs))) return MLA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(logits) % (dtype == MLA_LOGITS_FP32 ? 4 : 2)) return MLA_ERR_INVALID_ARG;
    LogprobArgs a;
    a.logits = logits;
    a.row_stride = row_stride;
    a.V = V;
    a.tokens = tokens;
    a.scale = scale;
    a.scale_log2 = scale * kLog2e;
    a.top = top;
    a.logprob = logprob;
    a.entropy = entropy;
    a.rank = rank;
    a.top_tokens = top_tokens;
    a.top_logprobs = top_logprobs;
    a.status = (int *)device_status;
    cudaStream_t s = (cudaStream_t)stream;
    return dtype == MLA_LOGITS_BF16   ? launch_logprobs<Bf16>(a, N, s)
           : dtype == MLA_LOGITS_FP16 ? launch_logprobs<Fp16>(a, N, s)
                                      : launch_logprobs<Fp32>(a, N, s);
}
