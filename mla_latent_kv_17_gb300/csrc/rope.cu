// Rotary positions of part of every head.  The definition is in include/mla_decode.h
// (mla_rope).
//
// Every value is read and written once, so memory bounds it.  A CTA takes a few tokens (or
// part of one token's heads) and first computes those tokens' cosines and sines once, into
// shared memory; then thread (u, y) owns unit u of a row - a vector of the passing part, or
// two vectors a, b whose values are the pairs of kVec (half layout) or 2 kVec values in a row
// (interleaved) - and walks the rows y, y + blockDim.y, ..., so that its cosines and sines
// stay in registers while it goes through a token's heads and no index is divided.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "common.cuh"
#include "rotary.cuh"
#include "tc_util.cuh"

namespace mla {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTableBytes = 16 * 1024;  // shared memory for the CTA's (cos, sin) pairs, at most

struct RopeArgs {
    const uint16_t *x;
    int64_t x_ts, x_hs;
    uint16_t *out_pass;  // null: the passing part is not copied
    int64_t p_ts, p_hs;
    uint16_t *out_rot;
    int64_t r_ts, r_hs;
    const int32_t *positions;
    const double *freqs;
    float mscale;
    int64_t N;
    int H, d_pass, d_rot, interleaved;
    int tokens;  // tokens per CTA
    int heads;   // heads per CTA (all of them when tokens > 1)
};

template <int kVec>
struct Vec;
template <>
struct Vec<8> {
    uint4 v;
    __device__ __forceinline__ void load(const uint16_t *p) { v = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(uint16_t *p) const { *reinterpret_cast<uint4 *>(p) = v; }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        v = make_uint4(bf16x2_bits(f[0], f[1]), bf16x2_bits(f[2], f[3]), bf16x2_bits(f[4], f[5]),
                       bf16x2_bits(f[6], f[7]));
    }
};
template <>
struct Vec<1> {
    uint16_t v;
    __device__ __forceinline__ void load(const uint16_t *p) { v = *p; }
    __device__ __forceinline__ void store(uint16_t *p) const { *p = v; }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = bf16_to_f32(v); }
    __device__ __forceinline__ void set(const float (&f)[1]) { v = bf16_bits(f[0]); }
};

// Rotates the kVec pairs of two vectors: pairs (a_i, b_i), or neighbours when interleaved.
template <int kVec>
__device__ __forceinline__ void rotate(Vec<kVec> &va, Vec<kVec> &vb, const float2 (&cs)[kVec], bool interleaved) {
    float a[kVec], b[kVec];
    va.get(a);
    vb.get(b);
    if (interleaved && kVec > 1) {
        // pair i: values 2i, 2i + 1 of the two vectors in a row
#pragma unroll
        for (int i = 0; i < kVec / 2; ++i) {
            const float p0 = a[2 * i], p1 = a[2 * i + 1], q0 = b[2 * i], q1 = b[2 * i + 1];
            const float2 c = cs[i], d = cs[kVec / 2 + i];
            a[2 * i] = p0 * c.x - p1 * c.y;
            a[2 * i + 1] = p0 * c.y + p1 * c.x;
            b[2 * i] = q0 * d.x - q1 * d.y;
            b[2 * i + 1] = q0 * d.y + q1 * d.x;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const float p0 = a[i], p1 = b[i];
            a[i] = p0 * cs[i].x - p1 * cs[i].y;
            b[i] = p0 * cs[i].y + p1 * cs[i].x;
        }
    }
    va.set(a);
    vb.set(b);
}

template <int kVec>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a) {
    extern __shared__ float2 s_cs[];  // [tokens][d_rot / 2]
    grid_dep_wait();
    grid_dep_launch();
    const int64_t n0 = (int64_t)blockIdx.x * a.tokens;
    const int nt = (int)min((int64_t)a.tokens, a.N - n0);
    const int h0 = (int)blockIdx.y * a.heads, nh = min(a.heads, a.H - h0);
    const int half = a.d_rot / 2;
    const int tid = threadIdx.y * blockDim.x + threadIdx.x, nthreads = blockDim.x * blockDim.y;
    for (int i = tid; i < nt * half; i += nthreads) {
        const int t = i / half;
        s_cs[i] = turn(a.positions[n0 + t], turns_fixed(a.freqs[i - t * half]), a.mscale);
    }
    __syncthreads();
    const int np = a.out_pass ? a.d_pass / kVec : 0;  // units that only pass
    const int units = np + half / kVec;
    for (int u = threadIdx.x; u < units; u += blockDim.x) {
        if (u < np) {
            int t = 0, h = threadIdx.y;
            while (h >= nh) {
                h -= nh;
                ++t;
            }
            while (t < nt) {
                // four rows in flight
                Vec<kVec> v[4];
                uint16_t *dst[4];
                int m = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (t < nt) {
                        v[k].load(a.x + (n0 + t) * a.x_ts + (int64_t)(h0 + h) * a.x_hs + u * kVec);
                        dst[k] = a.out_pass + (n0 + t) * a.p_ts + (int64_t)(h0 + h) * a.p_hs + u * kVec;
                        m = k + 1;
                        h += blockDim.y;
                        while (h >= nh) {
                            h -= nh;
                            ++t;
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < m) v[k].store(dst[k]);
            }
        } else {
            const int j = (u - np) * kVec;  // the unit's first pair
            const int offa = a.interleaved ? 2 * j : j, offb = a.interleaved ? 2 * j + kVec : j + half;
            int t = 0, h = threadIdx.y;
            while (h >= nh) {
                h -= nh;
                ++t;
            }
            int tcs = -1;
            float2 cs[kVec];
            while (t < nt) {
                if (t != tcs) {
#pragma unroll
                    for (int i = 0; i < kVec; ++i) cs[i] = s_cs[t * half + j + i];
                    tcs = t;
                }
                Vec<kVec> va[2], vb[2];
                uint16_t *dst[2];
                int m = 0;
                // two rows of the same token in flight
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (t == tcs && t < nt) {
                        const uint16_t *src = a.x + (n0 + t) * a.x_ts + (int64_t)(h0 + h) * a.x_hs + a.d_pass;
                        va[k].load(src + offa);
                        vb[k].load(src + offb);
                        dst[k] = a.out_rot + (n0 + t) * a.r_ts + (int64_t)(h0 + h) * a.r_hs;
                        m = k + 1;
                        h += blockDim.y;
                        while (h >= nh) {
                            h -= nh;
                            ++t;
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (k < m) {
                        rotate<kVec>(va[k], vb[k], cs, a.interleaved != 0);
                        va[k].store(dst[k] + offa);
                        vb[k].store(dst[k] + offb);
                    }
                }
            }
        }
    }
}

template <int kVec>
mla_status launch_rope(RopeArgs a, cudaStream_t stream) {
    const int units = (a.out_pass ? a.d_pass / kVec : 0) + a.d_rot / 2 / kVec;
    const int bx = units < kRopeThreads ? units : kRopeThreads;
    const int by = kRopeThreads / bx < 1 ? 1 : kRopeThreads / bx;
    // Rows per CTA: enough CTAs to fill the GPU several times over, and at most eight rows
    // per thread row; with many heads part of a token, with few several tokens.
    const int64_t rows = a.N * a.H;
    int64_t per = rows / (152 * 8);
    if (per < by) per = by;
    if (per > 8 * by) per = 8 * by;
    if (per >= a.H) {
        a.heads = a.H;
        a.tokens = (int)(per / a.H);
        const int most = kRopeTableBytes / ((a.d_rot / 2) * (int)sizeof(float2));
        if (a.tokens > most) a.tokens = most;
        if (a.tokens < 1) a.tokens = 1;
    } else {
        a.tokens = 1;
        const int groups = (int)((a.H + per - 1) / per);
        a.heads = (a.H + groups - 1) / groups;
    }
    const int64_t gx = (a.N + a.tokens - 1) / a.tokens;
    const int gy = (a.H + a.heads - 1) / a.heads;
    if (gx > 0x7FFFFFFF || gy > 65535) return MLA_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)gx, gy, 1);
    cfg.blockDim = dim3(bx, by, 1);
    cfg.dynamicSmemBytes = (size_t)a.tokens * (a.d_rot / 2) * sizeof(float2);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_kernel<kVec>, a) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status mla_rope(const void *x, int64_t x_token_stride, int64_t x_head_stride, int64_t N, int H,
                               int d_pass, int d_rot, mla_rope_layout layout, const int32_t *positions,
                               const double *freqs, float mscale, void *out_pass, int64_t pass_token_stride,
                               int64_t pass_head_stride, void *out_rot, int64_t rot_token_stride,
                               int64_t rot_head_stride, void *stream) {
    if (N < 0 || H < 1 || d_pass < 0 || d_rot < 2 || d_rot % 2 != 0) return MLA_ERR_INVALID_ARG;
    if (layout != MLA_ROPE_INTERLEAVED && layout != MLA_ROPE_HALF) return MLA_ERR_INVALID_ARG;
    if (!isfinite(mscale)) return MLA_ERR_INVALID_ARG;
    if (d_pass > 8192 || d_rot > 2048) return MLA_ERR_UNSUPPORTED;  // one token's cosines fit the CTA's table
    if (N == 0) return MLA_OK;
    if (!x || !positions || !freqs || !out_rot) return MLA_ERR_INVALID_ARG;
    RopeArgs a;
    a.x = (const uint16_t *)x;
    a.x_ts = x_token_stride;
    a.x_hs = x_head_stride;
    a.out_pass = d_pass > 0 ? (uint16_t *)out_pass : nullptr;
    a.p_ts = pass_token_stride;
    a.p_hs = pass_head_stride;
    a.out_rot = (uint16_t *)out_rot;
    a.r_ts = rot_token_stride;
    a.r_hs = rot_head_stride;
    a.positions = positions;
    a.freqs = freqs;
    a.mscale = mscale;
    a.N = N;
    a.H = H;
    a.d_pass = d_pass;
    a.d_rot = d_rot;
    a.interleaved = layout == MLA_ROPE_INTERLEAVED;
    a.tokens = a.heads = 0;
    // 16-byte accesses when every row of every tensor starts on a 16-byte boundary and the
    // parts are whole vectors; single values otherwise
    bool vec = aligned16(x) && aligned16(out_rot) && d_pass % 8 == 0 && d_rot % 16 == 0 &&
               (x_token_stride | x_head_stride | rot_token_stride | rot_head_stride) % 8 == 0;
    if (a.out_pass) vec = vec && aligned16(out_pass) && (pass_token_stride | pass_head_stride) % 8 == 0;
    return vec ? launch_rope<8>(a, (cudaStream_t)stream) : launch_rope<1>(a, (cudaStream_t)stream);
}
