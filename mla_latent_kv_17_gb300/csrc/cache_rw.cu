// Cache write and read of many tokens.  The definitions are in include/mla_decode.h
// (mla_cache_write, mla_cache_read).
//
// Both move every byte once, so memory bounds them.  One warp per token: lane l holds latent
// channels 16 l .. 16 l + 15 (the eight lanes of a 128-channel block find its maximum with
// three shuffles) and, for l < 8, key values 8 l .. 8 l + 7; a lane also owns frequency l, so
// the 32 angles of a token are computed once, one per lane, and handed round by shuffles.
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
__device__ __forceinline__ int64_t cache_row(const RwArgs &a, int64_t n, int32_t pos) {
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

// Rotates the key values of lanes 0-7 (8 each; the other lanes hold zeros) by cs, the (cos,
// sin) of frequency `lane`.  Warp-collective.
__device__ __forceinline__ void rotate_key(float (&k)[8], float2 cs, int lane, bool interleaved) {
    if (interleaved) {
        // lane l: pairs 4 l .. 4 l + 3
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = (4 * lane + i) & 31;
            const float c = __shfl_sync(kAll, cs.x, j), s = __shfl_sync(kAll, cs.y, j);
            const float p = k[2 * i], q = k[2 * i + 1];
            k[2 * i] = p * c - q * s;
            k[2 * i + 1] = p * s + q * c;
        }
    } else {
        // lane l < 4: the first values of pairs 8 l .. 8 l + 7; lane l + 4 their second ones
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = (8 * (lane & 3) + i) & 31;
            const float c = __shfl_sync(kAll, cs.x, j), s = __shfl_sync(kAll, cs.y, j);
            const float other = __shfl_xor_sync(kAll, k[i], 4);
            k[i] = lane & 4 ? other * s + k[i] * c : k[i] * c - other * s;
        }
    }
}

template <bool kFp8>
__global__ void __launch_bounds__(32 * kRwWarps) write_kernel(RwArgs a) {
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const int64_t nw = (int64_t)gridDim.x * kRwWarps;
    const uint64_t turns = a.freqs ? turns_fixed(a.freqs[lane]) : 0;
    uint4 w0 = make_uint4(0u, 0u, 0u, 0u), w1 = w0;
    if (a.norm_weight) {
        const uint4 *w = reinterpret_cast<const uint4 *>(a.norm_weight + 16 * lane);
        w0 = w[0];
        w1 = w[1];
    }
    for (int64_t n = (int64_t)blockIdx.x * kRwWarps + (threadIdx.x >> 5); n < a.N; n += nw) {
        // the token's values are read together with its position, then the page id
        const uint16_t *src = a.rows + n * a.stride;
        const uint4 v0 = reinterpret_cast<const uint4 *>(src + 16 * lane)[0];
        const uint4 v1 = reinterpret_cast<const uint4 *>(src + 16 * lane)[1];
        uint4 kp = make_uint4(0u, 0u, 0u, 0u);
        if (lane < 8) kp = reinterpret_cast<const uint4 *>(src + kDLatent)[lane];
        const int32_t pos = a.positions[n];
        const int64_t row = cache_row(a, n, pos);
        if (row < 0) continue;  // the same in every lane
        float x[16];
        unpack8(v0, x);
        unpack8(v1, x + 8);
        if (a.norm_weight) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(kAll, ss, o);
            const float r = rsqrtf(ss * (1.f / kDLatent) + a.norm_eps);
            float w[16];
            unpack8(w0, w);
            unpack8(w1, w + 8);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = x[i] * r * w[i];
        }
        if (a.freqs) {
            float k[8];
            unpack8(kp, k);
            const int32_t at = a.rope_positions ? a.rope_positions[n] : pos;
            rotate_key(k, turn(at, turns, a.mscale), lane, a.interleaved != 0);
            kp = pack8(k);
        }
        if constexpr (!kFp8) {
            uint4 *dst = reinterpret_cast<uint4 *>(a.cache + row * (kDEntry * 2));
            dst[2 * lane] = pack8(x);
            dst[2 * lane + 1] = pack8(x + 8);
            if (lane < 8) dst[kDLatent * 2 / 16 + lane] = kp;
        } else {
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
            const float s = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
            uint32_t codes[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = fminf(fmaxf(__fdiv_rn(x[4 * k + i], s), -448.f), 448.f);
                codes[k] = e4m3x2_of(q[0], q[1]) | (e4m3x2_of(q[2], q[3]) << 16);
            }
            unsigned char *rec = a.cache + row * kFp8RecordBytes;
            reinterpret_cast<uint4 *>(rec)[lane] = make_uint4(codes[0], codes[1], codes[2], codes[3]);
            if ((lane & 7) == 0) reinterpret_cast<float *>(rec + kDLatent)[lane >> 3] = s;
            if (lane < 8) reinterpret_cast<uint4 *>(rec + kDLatent + 16)[lane] = kp;
        }
    }
}

template <bool kFp8>
__global__ void __launch_bounds__(32 * kRwWarps) read_kernel(RwArgs a) {
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const int64_t nw = (int64_t)gridDim.x * kRwWarps;
    for (int64_t n = (int64_t)blockIdx.x * kRwWarps + (threadIdx.x >> 5); n < a.N; n += nw) {
        const int64_t row = cache_row(a, n, a.positions[n]);
        if (row < 0) continue;
        uint4 *dst = reinterpret_cast<uint4 *>(a.rows + n * a.stride);
        if constexpr (!kFp8) {
            const uint4 *src = reinterpret_cast<const uint4 *>(a.cache + row * (kDEntry * 2));
            const uint4 v0 = src[lane], v1 = src[32 + lane];
            uint4 v2 = make_uint4(0u, 0u, 0u, 0u);
            if (lane < 8) v2 = src[64 + lane];
            dst[lane] = v0;
            dst[32 + lane] = v1;
            if (lane < 8) dst[64 + lane] = v2;
        } else {
            const unsigned char *rec = a.cache + row * kFp8RecordBytes;
            const uint4 codes = reinterpret_cast<const uint4 *>(rec)[lane];
            const float s = reinterpret_cast<const float *>(rec + kDLatent)[lane >> 3];
            uint4 kp = make_uint4(0u, 0u, 0u, 0u);
            if (lane < 8) kp = reinterpret_cast<const uint4 *>(rec + kDLatent + 16)[lane];
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
            if (lane < 8) dst[kDLatent * 2 / 16 + lane] = kp;
        }
    }
}

int rw_grid(int64_t N) {
    const int64_t ctas = (N + kRwWarps - 1) / kRwWarps;
    const int64_t most = 152 * 8;  // resident warps go on to the next tokens
    return (int)(ctas < most ? ctas : most);
}

// Arguments the write and the read share; fills `a` with them.
mla_status check_rw(RwArgs *a, const void *cache, mla_kv_dtype kv_dtype, int64_t num_pages,
                    const int32_t *block_table, int num_requests, int max_pages, const int32_t *requests,
                    const int32_t *positions, const void *rows, int64_t stride, int64_t N, int32_t *device_status) {
    if (N < 0 || num_requests < 1 || max_pages < 1 || num_pages < 1 || stride < kDEntry) return MLA_ERR_INVALID_ARG;
    if (kv_dtype != MLA_KV_BF16 && kv_dtype != MLA_KV_FP8_E4M3) return MLA_ERR_INVALID_ARG;
    if (!cache || !block_table) return MLA_ERR_INVALID_ARG;
    if (N > 0 && (!positions || !rows)) return MLA_ERR_INVALID_ARG;
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
    const auto kernel = kv_dtype == MLA_KV_FP8_E4M3 ? write_kernel<true> : write_kernel<false>;
    return launch_pdl(kernel, rw_grid(N), 32 * kRwWarps, 0, (cudaStream_t)stream, a) == cudaSuccess ? MLA_OK
                                                                                                    : MLA_ERR_CUDA;
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
    const auto kernel = kv_dtype == MLA_KV_FP8_E4M3 ? read_kernel<true> : read_kernel<false>;
    return launch_pdl(kernel, rw_grid(N), 32 * kRwWarps, 0, (cudaStream_t)stream, a) == cudaSuccess ? MLA_OK
                                                                                                    : MLA_ERR_CUDA;
}
