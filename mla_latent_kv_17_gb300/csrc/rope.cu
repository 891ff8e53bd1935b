// Rotary positions of part of every head.  The definition is in include/mla_decode.h
// (mla_rope).
//
// Every value is read and written once, so memory bounds it: 4,096 tokens x 128 heads x 192 values
// (403 MB) take 62 us, 0.96 of a plain copy's rate; a few tokens take the launch, 3 us.  A CTA takes kRopeRows rows per
// thread row: part of a token's heads, or several tokens of few heads.  Thread (u, y) owns unit
// u of a row - two vectors of the passing part, or the two vectors whose values are the pairs -
// and rows y, y + blockDim.y, ...; it issues the loads of all its rows first, then the CTA
// computes its tokens' cosines and sines once into shared memory while they are in flight.
// (Angles first, then rows in turn, ran at 36 % of the memory's rate: the short CTAs waited for
// their angles with nothing in flight.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "common.cuh"
#include "rotary.cuh"
#include "tc_util.cuh"

namespace mla {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 4;                // rows per thread, in flight together
constexpr int kRopeCtas = 3;                // CTAs per SM (registers)
constexpr int kRopeTableBytes = 16 * 1024;  // shared memory for the CTA's (cos, sin) pairs, at most
constexpr int kMaxAxisPairs = 256;          // pairs of a head with several axes (their axes are a kernel parameter)

struct RopeArgs {
    const uint16_t *x;
    int64_t x_ts, x_hs;
    uint16_t *out_pass;  // null: the passing part is not copied
    int64_t p_ts, p_hs;
    uint16_t *out_rot;
    int64_t r_ts, r_hs;
    const double *freqs;
    float mscale;
    int64_t N;
    int H, d_pass, d_rot, interleaved;
    int tokens;  // tokens per CTA
    int heads;   // heads per CTA (all of them when tokens > 1)
};

// Where a token stands: one position for all pairs, or one per axis and an axis for each pair (4,096 tokens x 128
// heads x 192 values: 62 us with one axis or three).
struct OnePosition {
    const int32_t *p;
    __device__ __forceinline__ int32_t at(int64_t n, int) const { return p[n]; }
};
struct AxisPositions {
    const int32_t *p;
    int64_t token_stride, axis_stride;
    uint8_t axis[kMaxAxisPairs];
    __device__ __forceinline__ int32_t at(int64_t n, int pair) const { return p[n * token_stride + axis[pair] * axis_stride]; }
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
__device__ __forceinline__ void rotate(Vec<kVec> &va, Vec<kVec> &vb, const float2 *cs, bool interleaved) {
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

// kOne: the CTA's rows are heads of one token (rows at a fixed distance, no division).
template <int kVec, bool kOne, typename Positions>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(RopeArgs a, const __grid_constant__ Positions pos) {
    extern __shared__ float2 s_cs[];  // [tokens][d_rot / 2]
    grid_dep_wait();
    grid_dep_launch();
    const int64_t n0 = (int64_t)blockIdx.x * a.tokens;
    const int nt = kOne ? 1 : (int)min((int64_t)a.tokens, a.N - n0);
    const int h0 = (int)blockIdx.y * a.heads, nh = min(a.heads, a.H - h0);
    const int half = a.d_rot / 2;
    const int tid = threadIdx.y * blockDim.x + threadIdx.x, nthreads = blockDim.x * blockDim.y;
    const int pvec = a.out_pass ? a.d_pass / kVec : 0;  // vectors that only pass, two to a unit
    const int np = (pvec + 1) / 2, units = np + half / kVec;
    const int rows = nt * nh;
    const uint16_t *src0 = a.x + n0 * a.x_ts + (int64_t)h0 * a.x_hs;
    bool first = true;
    for (int u = threadIdx.x; u < units || first; u += blockDim.x) {
        const bool pass = u < np;
        const int j = (u - np) * kVec;  // a rotated unit's first pair
        const int offa = pass ? 2 * u * kVec : a.d_pass + (a.interleaved ? 2 * j : j);
        const int offb = pass ? offa + kVec : a.d_pass + (a.interleaved ? 2 * j + kVec : j + half);
        const bool has_b = !pass || 2 * u + 1 < pvec;
        for (int r0 = threadIdx.y; r0 < rows || first; r0 += kRopeRows * blockDim.y) {
            // this thread's rows of the unit, all loads in flight; the first ones before the
            // angles are computed
            Vec<kVec> va[kRopeRows], vb[kRopeRows];
#pragma unroll
            for (int k = 0; k < kRopeRows; ++k) {
                const int r = r0 + k * blockDim.y;
                if (u < units && r < rows) {
                    const int t = kOne ? 0 : r / nh, h = kOne ? r : r - t * nh;
                    const uint16_t *src = src0 + t * a.x_ts + h * a.x_hs;
                    va[k].load(src + offa);
                    if (has_b) vb[k].load(src + offb);
                }
            }
            if (first) {
                for (int i = tid; i < nt * half; i += nthreads) {
                    const int t = kOne ? 0 : i / half, p = i - t * half;
                    s_cs[i] = turn(pos.at(n0 + t, p), turns_fixed(a.freqs[p]), a.mscale);
                }
                __syncthreads();
                first = false;
            }
            if (u >= units) break;
            uint16_t *dst0 = pass ? a.out_pass + n0 * a.p_ts + (int64_t)h0 * a.p_hs + offa
                                  : a.out_rot + n0 * a.r_ts + (int64_t)h0 * a.r_hs + (offa - a.d_pass);
            const int64_t dts = pass ? a.p_ts : a.r_ts, dhs = pass ? a.p_hs : a.r_hs;
#pragma unroll
            for (int k = 0; k < kRopeRows; ++k) {
                const int r = r0 + k * (int)blockDim.y;
                if (r >= rows) break;
                const int t = kOne ? 0 : r / nh, h = kOne ? r : r - t * nh;
                if (!pass) rotate<kVec>(va[k], vb[k], s_cs + t * half + j, a.interleaved != 0);
                uint16_t *dst = dst0 + t * dts + h * dhs;
                va[k].store(dst);
                if (has_b) vb[k].store(dst + (offb - offa));
            }
        }
    }
}

template <int kVec, typename Positions>
mla_status launch_rope(RopeArgs a, const Positions &pos, cudaStream_t stream) {
    const int units = (a.out_pass ? (a.d_pass / kVec + 1) / 2 : 0) + a.d_rot / 2 / kVec;
    const int bx = units < kRopeThreads ? units : kRopeThreads;
    int by = 1;  // a power of two, like most head counts
    while (2 * by * bx <= kRopeThreads) by *= 2;
    // by * kRopeRows rows per CTA: part of a token's heads, or several tokens of few heads
    const int per = by * kRopeRows;
    if (per >= a.H) {
        a.heads = a.H;
        a.tokens = per / a.H;
        const int most = kRopeTableBytes / ((a.d_rot / 2) * (int)sizeof(float2));
        if (a.tokens > most) a.tokens = most;
    } else {
        a.tokens = 1;
        const int groups = (a.H + per - 1) / per;
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
    return cudaLaunchKernelEx(&cfg, a.tokens == 1 ? rope_kernel<kVec, true, Positions> : rope_kernel<kVec, false, Positions>,
                              a, pos) == cudaSuccess
               ? MLA_OK
               : MLA_ERR_CUDA;
}

// Checks the arguments that do not depend on where the positions stand, and launches.
template <typename Positions>
mla_status run_rope(const void *x, int64_t x_token_stride, int64_t x_head_stride, int64_t N, int H, int d_pass, int d_rot,
                    mla_rope_layout layout, const Positions &pos, const double *freqs, float mscale, void *out_pass,
                    int64_t pass_token_stride, int64_t pass_head_stride, void *out_rot, int64_t rot_token_stride,
                    int64_t rot_head_stride, void *stream) {

    if (N < 0 || H < 1 || d_pass < 0 || d_rot < 2 || d_rot % 2 != 0) return MLA_ERR_INVALID_ARG;
    if (layout != MLA_ROPE_INTERLEAVED && layout != MLA_ROPE_HALF) return MLA_ERR_INVALID_ARG;
    if (!isfinite(mscale)) return MLA_ERR_INVALID_ARG;
    if (d_pass > 8192 || d_rot > 2048) return MLA_ERR_UNSUPPORTED;  // one token's cosines fit the CTA's table
    if (N == 0) return MLA_OK;
    if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out_rot) | reinterpret_cast<uintptr_t>(out_pass)) % 2)
        return MLA_ERR_INVALID_ARG;  // no bf16 values
    if (!x || !pos.p || !freqs || !out_rot) return MLA_ERR_INVALID_ARG;
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
    return vec ? launch_rope<8>(a, pos, (cudaStream_t)stream) : launch_rope<1>(a, pos, (cudaStream_t)stream);
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status mla_rope(const void *x, int64_t x_token_stride, int64_t x_head_stride, int64_t N, int H,
                               int d_pass, int d_rot, mla_rope_layout layout, const int32_t *positions,
                               const double *freqs, float mscale, void *out_pass, int64_t pass_token_stride,
                               int64_t pass_head_stride, void *out_rot, int64_t rot_token_stride,
                               int64_t rot_head_stride, void *stream) {
    return run_rope(x, x_token_stride, x_head_stride, N, H, d_pass, d_rot, layout, OnePosition{positions}, freqs, mscale,
                    out_pass, pass_token_stride, pass_head_stride, out_rot, rot_token_stride, rot_head_stride, stream);
}

extern "C" mla_status mla_rope_axes(const void *x, int64_t x_token_stride, int64_t x_head_stride, int64_t N, int H,
                                    int d_pass, int d_rot, mla_rope_layout layout, const int32_t *positions,
                                    int64_t position_token_stride, int64_t position_axis_stride, int num_axes,
                                    const uint8_t *axes, const double *freqs, float mscale, void *out_pass,
                                    int64_t pass_token_stride, int64_t pass_head_stride, void *out_rot,
                                    int64_t rot_token_stride, int64_t rot_head_stride, void *stream) {
    if (d_rot < 2 || num_axes < 1 || !axes) return MLA_ERR_INVALID_ARG;
    if (num_axes > kMaxAxes || d_rot / 2 > kMaxAxisPairs) return MLA_ERR_UNSUPPORTED;
    AxisPositions pos;
    pos.p = positions;
    pos.token_stride = position_token_stride;
    pos.axis_stride = position_axis_stride;
    if (!copy_axes(pos.axis, axes, d_rot / 2, num_axes)) return MLA_ERR_INVALID_ARG;
    return run_rope(x, x_token_stride, x_head_stride, N, H, d_pass, d_rot, layout, pos, freqs, mscale, out_pass,
                    pass_token_stride, pass_head_stride, out_rot, rot_token_stride, rot_head_stride, stream);
}
