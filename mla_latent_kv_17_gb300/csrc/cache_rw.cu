// Cache write and read of many tokens.  The definitions are in include/mla_decode.h
// (mla_cache_write, mla_cache_read).
//
// Both move every byte once.  A warp works on a token's latent at a time: lane l holds channels
// 16 l .. 16 l + 15, so the eight lanes of a 128-channel block find its maximum with three
// shuffles; keys are taken four tokens at a time.  The FP8 write is bound by its instructions
// (issue slots 63 % busy, half of them integer and logic), not by memory, hence packed fp32
// arithmetic and the Newton quotient; the others by memory.  65,536 tokens: write with norm and
// rotation into records 25 us, read of records 22 us (119 MB each: 0.70 and 0.79 of a copy's rate);
// 512 tokens into a 16-bit cache 2.8 us, 1,001 read back 2.0 us (the launch).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "common.cuh"
#include "rotary.cuh"
#include "tc_util.cuh"

namespace mla {
namespace {

constexpr int kRwWarps = 8;
constexpr int kWriteWarps = 32, kWriteMost = 16;  // see launch_rw
constexpr int kSms = 152;  // a GB300's; only the grids' shapes depend on it
constexpr unsigned kAll = 0xffffffffu;

struct RwArgs {
    unsigned char *cache;
    int64_t num_pages;
    const int32_t *block_table;
    int num_requests, max_pages;
    const int32_t *requests, *positions;
    uint16_t *rows;  // the tokens' rows: kv (write) or entries (read)
    int64_t stride;  // in elements
    int64_t N;
    const uint16_t *norm_weight;
    float norm_eps;
    const double *freqs;
    const int32_t *rope_positions;
    int interleaved;
    float mscale;
    int *status;
};

// The cache row of token n, or -1 if it is skipped (an index out of range is recorded).
__device__ __forceinline__ int64_t cache_row(const RwArgs &a, int64_t n) {
    const int32_t pos = a.positions[n];
    if (pos < 0) return -1;
    const int64_t r = a.requests ? (int64_t)a.requests[n] : n;
    const int32_t lp = pos / kPageRows;
    int64_t page = -1;
    if (r >= 0 && r < a.num_requests && lp < a.max_pages) page = a.block_table[r * a.max_pages + lp];
    if (page < 0 || page >= a.num_pages) {
        if (a.status) record_error(a.status, MLA_ERR_INDEX);
        return -1;
    }
    return page * kPageRows + pos % kPageRows;
}

__device__ __forceinline__ void unpack8(uint4 v, float *f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float *f) {
    return make_uint4(bf16x2_bits(f[0], f[1]), bf16x2_bits(f[2], f[3]), bf16x2_bits(f[4], f[5]),
                      bf16x2_bits(f[6], f[7]));
}
// e4m3 codes of two fp32 values (nearest, ties to even, saturated), the first in the low byte
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// Pairs of fp32 values in one 64-bit register pair, for the packed fp32 instructions.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 halves(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ void unpack_pairs(uint4 v, uint64_t *f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack_pairs(const uint64_t *f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = halves(f[i]);
        w[i] = bf16x2_bits(v.x, v.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two quotients x / s correctly rounded, given r = 1 / s correctly rounded and -s: one Newton
// step on the quotient (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  Exact while nothing under- or overflows on the way; the
// caller sees to that.  (A quotient of -0 comes out as +0.)
__device__ __forceinline__ float2 quotients(uint64_t x, uint64_t neg_s, uint64_t r) {
    const uint64_t q = mul2(x, r);
    return halves(fma2(fma2(q, neg_s, x), r, q));
}

// The keys of four tokens at a time: lane l holds values 8 (l % 8) .. + 7 of token l / 8, so that
// every lane works on a key, and the four angles a lane computes are the ones its pairs need.
// Interleaved: the pairs of its own values.  Half layout: lanes l and l ^ 4 hold the first and
// the second values of the same eight pairs; each computes four of their angles.
// turns: the 32 frequencies (shared memory).
__device__ __forceinline__ uint4 rotate_key(uint4 key, const uint64_t *turns, int32_t pos, float mscale, int lane,
                                            bool interleaved) {
    const int j = interleaved ? 4 * (lane & 7) : 8 * (lane & 3) + (lane & 4);
    float k[8];
    unpack8(key, k);
    float2 cs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) cs[i] = turn(pos, turns[j + i], mscale);
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float p = k[2 * i], q = k[2 * i + 1];
            k[2 * i] = p * cs[i].x - q * cs[i].y;
            k[2 * i + 1] = p * cs[i].y + q * cs[i].x;
        }
    } else {
        const bool second = lane & 4;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float c = __shfl_sync(kAll, cs[i & 3].x, (lane & ~4) | (i & 4));
            const float s = __shfl_sync(kAll, cs[i & 3].y, (lane & ~4) | (i & 4));
            const float other = __shfl_xor_sync(kAll, k[i], 4);
            k[i] = second ? other * s + k[i] * c : k[i] * c - other * s;
        }
    }
    return pack8(k);
}

struct Latent {
    uint4 v0, v1;  // lane l: channels 16 l .. 16 l + 15
};
__device__ __forceinline__ Latent load_latent(const uint16_t *src, int lane) {
    const uint4 *p = reinterpret_cast<const uint4 *>(src + 16 * lane);
    return Latent{p[0], p[1]};
}

// A warp takes `per` (<= 32) tokens in a row: lane i resolves the cache row of the i-th one, all
// at once, and the next token's latent is read while the present one is worked on, so that no
// token waits for the position -> page -> row chain.
template <bool kFp8, bool kNorm>
__global__ void __launch_bounds__(32 * kRwWarps, 4) write_kernel(RwArgs a, int per) {
    __shared__ uint64_t s_turns[32];
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const int64_t n0 = ((int64_t)blockIdx.x * kRwWarps + (threadIdx.x >> 5)) * per;
    const int cnt = (int)max((int64_t)0, min((int64_t)per, a.N - n0));
    const uint16_t *rows = a.rows + n0 * a.stride;
    Latent next{};
    if (cnt > 0) next = load_latent(rows, lane);
    int64_t row_l = -1;
    int32_t at_l = 0;
    if (lane < cnt) {
        row_l = cache_row(a, n0 + lane);
        if (a.freqs) at_l = (a.rope_positions ? a.rope_positions : a.positions)[n0 + lane];
    }
    const int64_t row_bytes = kFp8 ? kFp8RecordBytes : kDEntry * 2;
    if (a.freqs) {  // the same for the whole grid
        if (threadIdx.x < 32) s_turns[threadIdx.x] = turns_fixed(a.freqs[threadIdx.x]);
        __syncthreads();
    }
#pragma unroll 1
    for (int i0 = 0; i0 < cnt; i0 += 4) {
        {
            const int i = i0 + (lane >> 3);
            uint4 key = make_uint4(0u, 0u, 0u, 0u);
            if (i < cnt) key = reinterpret_cast<const uint4 *>(rows + i * a.stride + kDLatent)[lane & 7];
            const int64_t row = __shfl_sync(kAll, row_l, i & 31);
            if (a.freqs) key = rotate_key(key, s_turns, __shfl_sync(kAll, at_l, i & 31), a.mscale, lane, a.interleaved != 0);
            if (i < cnt && row >= 0)
                reinterpret_cast<uint4 *>(a.cache + row * row_bytes + (kFp8 ? kDLatent + 16 : kDLatent * 2))[lane & 7] = key;
        }
#pragma unroll 1
        for (int i = i0; i < min(cnt, i0 + 4); ++i) {
            Latent tk = next;
            if (i + 1 < cnt) next = load_latent(rows + (i + 1) * a.stride, lane);
            const int64_t row = __shfl_sync(kAll, row_l, i);
            if (row < 0) continue;  // the same in every lane
            unsigned char *dst = a.cache + row * row_bytes;
            if constexpr (!kFp8 && !kNorm) {
                reinterpret_cast<uint4 *>(dst)[2 * lane] = tk.v0;
                reinterpret_cast<uint4 *>(dst)[2 * lane + 1] = tk.v1;
                continue;
            }
            uint64_t x[8];
            unpack_pairs(tk.v0, x);
            unpack_pairs(tk.v1, x + 4);
            // y = x * weight * r: the products by the weight first, r (which scales the whole token) last
            float r = 1.f;
            if constexpr (kNorm) {
                uint64_t s2 = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) s2 = fma2(x[k], x[k], s2);
                float ss = halves(s2).x + halves(s2).y;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(kAll, ss, o);
                r = rsqrtf(ss * (1.f / kDLatent) + a.norm_eps);
                const uint4 *wp = reinterpret_cast<const uint4 *>(a.norm_weight + 16 * lane);  // (from L1)
                uint64_t w[8];
                unpack_pairs(__ldg(wp), w);
                unpack_pairs(__ldg(wp + 1), w + 4);
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = mul2(x[k], w[k]);
            }
            if constexpr (!kFp8) {
                const uint64_t r2 = pair(r, r);
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = mul2(x[k], r2);
                reinterpret_cast<uint4 *>(dst)[2 * lane] = pack_pairs(x);
                reinterpret_cast<uint4 *>(dst)[2 * lane + 1] = pack_pairs(x + 4);
            } else {
                // the codes are those of y / (max|y| / 448) = x / (max|x| / 448): r cancels
                float amax = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 v = halves(x[k]);
                    amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
                }
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
                // (products with a weight may be so small that amax / 448 is 0 in fp32: a zero block)
                float s = __fdiv_rn(amax, 448.f);
                const bool zero = !(s > 0.f);
                if (zero) s = 1.f;
                // Blocks of very small or large values are moved by a power of two first, which leaves
                // the quotients as they are and the remainders exact.  (What underflows on the way down
                // lies below 2^-40 of the scale: code 0.)
                float sq = s;
                if (!(s > 1e-25f && s < 1e25f)) {
                    const float f = s < 1.f ? 0x1p100f : 0x1p-60f;
                    sq = s * f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = mul2(x[k], pair(f, f));
                }
                const float rs = __frcp_rn(sq);
                const uint64_t neg_s2 = pair(-sq, -sq), rs2 = pair(rs, rs);
                const uint32_t w[8] = {tk.v0.x, tk.v0.y, tk.v0.z, tk.v0.w, tk.v1.x, tk.v1.y, tk.v1.z, tk.v1.w};
                uint32_t codes[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 lo = quotients(x[2 * k], neg_s2, rs2), hi = quotients(x[2 * k + 1], neg_s2, rs2);
                    codes[k] = e4m3x2_of(lo.x, lo.y) | e4m3x2_of(hi.x, hi.y) << 16;
                    // a value of -0 keeps its sign, as in the division
                    if constexpr (!kNorm) codes[k] |= __byte_perm(w[2 * k], w[2 * k + 1], 0x7531) & 0x80808080u;
                }
                reinterpret_cast<uint4 *>(dst)[lane] = make_uint4(codes[0], codes[1], codes[2], codes[3]);
                if ((lane & 7) == 0)
                    reinterpret_cast<float *>(dst + kDLatent)[lane >> 3] = kNorm && !zero ? s * r : s;
            }
        }
    }
}

// The read: a token per warp and step, 64 warps per SM.  (Runs of tokens per warp with two or four
// in flight, or the next token's row looked up ahead, cost registers and so warps, and ran
// slower: 24-28 us against 21 for 65,536 records.)
template <bool kFp8>
__global__ void __launch_bounds__(32 * kRwWarps, 8) read_kernel(RwArgs a) {
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const int64_t nw = (int64_t)gridDim.x * kRwWarps;
    for (int64_t n = (int64_t)blockIdx.x * kRwWarps + (threadIdx.x >> 5); n < a.N; n += nw) {
        const int64_t row = cache_row(a, n);
        if (row < 0) continue;  // the same in every lane
        uint4 *dst = reinterpret_cast<uint4 *>(a.rows + n * a.stride);
        uint4 key = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (!kFp8) {
            const uint4 *src = reinterpret_cast<const uint4 *>(a.cache + row * (kDEntry * 2));
            const uint4 v0 = src[lane], v1 = src[32 + lane];
            if (lane < 8) key = src[64 + lane];
            dst[lane] = v0;
            dst[32 + lane] = v1;
        } else {
            const unsigned char *rec = a.cache + row * kFp8RecordBytes;
            const uint4 codes = reinterpret_cast<const uint4 *>(rec)[lane];
            const float s = reinterpret_cast<const float *>(rec + kDLatent)[lane >> 3];
            if (lane < 8) key = reinterpret_cast<const uint4 *>(rec + kDLatent + 16)[lane];
            const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
            float x[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                    (__nv_fp8x2_storage_t)((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu), __NV_E4M3);
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                x[2 * i] = f.x * s;
                x[2 * i + 1] = f.y * s;
            }
            dst[2 * lane] = pack8(x);
            dst[2 * lane + 1] = pack8(x + 8);
        }
        if (lane < 8) dst[kDLatent * 2 / 16 + lane] = key;
    }
}

// Tokens per warp: one while that still gives every SM at most `warps` warps, then as many as
// keep them busy, up to `most`.
template <typename K>
mla_status launch_rw(K kernel, const RwArgs &a, int warps, int most, void *stream) {
    const int64_t want = (a.N + kSms * warps - 1) / (kSms * warps);
    const int per = (int)(want < 1 ? 1 : want > most ? most : want);
    const int64_t ctas = (a.N + (int64_t)per * kRwWarps - 1) / ((int64_t)per * kRwWarps);
    if (ctas > 0x7FFFFFFF) return MLA_ERR_UNSUPPORTED;
    return launch_pdl(kernel, (int)ctas, 32 * kRwWarps, 0, (cudaStream_t)stream, a, per) == cudaSuccess ? MLA_OK
                                                                                                       : MLA_ERR_CUDA;
}

// Arguments the write and the read share; fills `a` with them (where there are tokens).
mla_status check_rw(RwArgs *a, const void *cache, mla_kv_dtype kv_dtype, int64_t num_pages,
                    const int32_t *block_table, int num_requests, int max_pages, const int32_t *requests,
                    const int32_t *positions, const void *rows, int64_t stride, int64_t N, int32_t *device_status) {
    if (N < 0 || stride < kDEntry) return MLA_ERR_INVALID_ARG;
    if (kv_dtype != MLA_KV_BF16 && kv_dtype != MLA_KV_FP8_E4M3) return MLA_ERR_INVALID_ARG;
    if (N == 0) return MLA_OK;  // (the caller enqueues nothing; a batch may have no requests, then)
    if (num_requests < 1 || max_pages < 1 || num_pages < 1) return MLA_ERR_INVALID_ARG;
    if (!cache || !block_table || !positions || !rows) return MLA_ERR_INVALID_ARG;
    if (!requests && N > num_requests) return MLA_ERR_INVALID_ARG;
    if (!aligned16(cache) || !aligned16(rows) || stride % 8 != 0) return MLA_ERR_INVALID_ARG;
    a->cache = (unsigned char *)const_cast<void *>(cache);
    a->num_pages = num_pages;
    a->block_table = block_table;
    a->num_requests = num_requests;
    a->max_pages = max_pages;
    a->requests = requests;
    a->positions = positions;
    a->rows = (uint16_t *)const_cast<void *>(rows);
    a->stride = stride;
    a->N = N;
    a->norm_weight = nullptr;
    a->norm_eps = 0.f;
    a->freqs = nullptr;
    a->rope_positions = nullptr;
    a->interleaved = 0;
    a->mscale = 1.f;
    a->status = (int *)device_status;
    return MLA_OK;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status mla_cache_write(void *cache, mla_kv_dtype kv_dtype, int64_t num_pages,
                                      const int32_t *block_table, int num_requests, int max_pages,
                                      const int32_t *requests, const int32_t *positions, const void *kv,
                                      int64_t kv_stride, int64_t N, const void *norm_weight, float norm_eps,
                                      const double *freqs, const int32_t *rope_positions, mla_rope_layout layout,
                                      float mscale, int32_t *device_status, void *stream) {
    RwArgs a;
    const mla_status st = check_rw(&a, cache, kv_dtype, num_pages, block_table, num_requests, max_pages, requests,
                                   positions, kv, kv_stride, N, device_status);
    if (st != MLA_OK) return st;
    if (layout != MLA_ROPE_INTERLEAVED && layout != MLA_ROPE_HALF) return MLA_ERR_INVALID_ARG;
    if (norm_weight && (!aligned16(norm_weight) || !isfinite(norm_eps) || norm_eps < 0.f)) return MLA_ERR_INVALID_ARG;
    if (!isfinite(mscale)) return MLA_ERR_INVALID_ARG;
    if (N == 0) return MLA_OK;
    a.norm_weight = (const uint16_t *)norm_weight;
    a.norm_eps = norm_eps;
    a.freqs = freqs;
    a.rope_positions = rope_positions;
    a.interleaved = layout == MLA_ROPE_INTERLEAVED;
    a.mscale = mscale;
    const bool fp8 = kv_dtype == MLA_KV_FP8_E4M3;
    const auto kernel = norm_weight ? (fp8 ? write_kernel<true, true> : write_kernel<false, true>)
                                    : (fp8 ? write_kernel<true, false> : write_kernel<false, false>);
    return launch_rw(kernel, a, kWriteWarps, kWriteMost, stream);
}

extern "C" mla_status mla_cache_read(const void *cache, mla_kv_dtype kv_dtype, int64_t num_pages,
                                     const int32_t *block_table, int num_requests, int max_pages,
                                     const int32_t *requests, const int32_t *positions, int64_t N, void *entries,
                                     int64_t entries_stride, int32_t *device_status, void *stream) {
    RwArgs a;
    const mla_status st = check_rw(&a, cache, kv_dtype, num_pages, block_table, num_requests, max_pages, requests,
                                   positions, entries, entries_stride, N, device_status);
    if (st != MLA_OK) return st;
    if (N == 0) return MLA_OK;
    const int64_t ctas = (N + kRwWarps - 1) / kRwWarps, resident = kSms * 8;
    return launch_pdl(kv_dtype == MLA_KV_FP8_E4M3 ? read_kernel<true> : read_kernel<false>,
                      (int)(ctas < resident ? ctas : resident), 32 * kRwWarps, 0, (cudaStream_t)stream,
                      a) == cudaSuccess
               ? MLA_OK
               : MLA_ERR_CUDA;
}
