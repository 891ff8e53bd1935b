// Verification of a drafted tree against the target's probabilities.  The definition is in
// include/mla_decode.h (mla_verify_draft).
//
// What the walk needs of a token that is accepted is two probabilities; only where it stops
// are whole rows read: the target's row and the rows of the drafts rejected there.  One
// cluster of eight CTAs takes a request, each CTA an eighth of the vocabulary, so that a
// single request still streams its rows through eight SMs; memory bounds a large batch.
//
// All sums are 64-bit integers: a probability is cut to a multiple of 2^-58, which keeps every
// bit of a value of 2^-34 or more, the residual of a first rejection is an exact subtraction,
// and integer addition is exact in any order - so the chosen token does not depend on how the
// vocabulary is split.  (fp32 sums would move the borders between a vocabulary's tokens by
// about 1e-10 each, enough to change one draw in some ten thousand; fp64 additions run at 2
// per cycle and SM here.)
//
// Per stop the sum pass leaves a partial sum per warp (a contiguous chunk) and per CTA (a
// contiguous slice); the draw then finds its slice and chunk from those sums, and one warp
// searches its chunk again, from L2.
#include <cuda_runtime.h>
#include <math.h>

#include "common.cuh"
#include "sm103_ptx.cuh"
#include "tc_util.cuh"

namespace mla {
namespace {

constexpr int kVfCluster = 8;
constexpr int kVfThreads = 512;
constexpr int kVfWarps = kVfThreads / 32;
constexpr int kVfMaxT = 64;
constexpr float kVfOne = 288230376151711744.f;  // 2^58

struct VerifyArgs {
    const float *target, *draft;
    const int32_t *tokens, *parents, *tree_lens;
    const float *uniforms;
    int T, V;
    int32_t *num_accepted, *depths, *next_token;
    int *status;
};

// A probability as a multiple of 2^-58 (NaN and negative values: 0, above 1: 1).
__device__ __forceinline__ uint64_t fixed58(float p) {
    p = p > 0.f ? fminf(p, 1.f) : 0.f;
    return __float2ull_rz(p * kVfOne);
}

// What is left of the target's row after the rejected drafts rej[0 .. n): their masses are the
// sums left before each (the first: 1).
struct Residual {
    const float *p;        // the target's row
    const float *q;        // the draft's rows of this request, or null: certain of its token
    const int32_t *tokens;
    const int *rej;
    const double *mass;
    int n, V;

    __device__ __forceinline__ uint64_t minus(uint64_t left, int k, float qv) const {
        // the first draft is subtracted exactly; later ones are scaled by the mass left
        const uint64_t d = k == 0 ? fixed58(qv) : __double2ull_rz((double)(qv > 0.f ? fminf(qv, 1.f) : 0.f) * mass[k]);
        return left > d ? left - d : 0;
    }
    __device__ __forceinline__ uint64_t at(int v) const {
        uint64_t left = fixed58(p[v]);
        for (int k = 0; k < n; ++k) {
            if (q)
                left = minus(left, k, q[(int64_t)rej[k] * V + v]);
            else if (tokens[rej[k]] == v)
                left = 0;
        }
        return left;
    }
};

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__global__ void __cluster_dims__(kVfCluster, 1, 1) __launch_bounds__(kVfThreads) verify_kernel(VerifyArgs a) {
    __shared__ int32_t s_tok[kVfMaxT], s_par[kVfMaxT], s_depth[kVfMaxT];
    __shared__ float s_u[kVfMaxT + 1], s_p[kVfMaxT], s_q[kVfMaxT];
    __shared__ int s_rej[kVfMaxT];
    __shared__ double s_mass[kVfMaxT];
    __shared__ uint64_t s_warp[kVfWarps];         // sums of this CTA's chunks
    __shared__ uint64_t s_slice[2][kVfCluster];   // sums of all slices, written by every CTA (two turns)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const int b = blockIdx.x / kVfCluster;
    const int T = a.T, V = a.V;
    grid_dep_wait();
    grid_dep_launch();
    const float *target = a.target + (int64_t)b * (T + 1) * V;
    const float *draft = a.draft ? a.draft + (int64_t)b * T * V : nullptr;
    int len = a.tree_lens ? a.tree_lens[b] : T;
    if (len < 0 || len > T) {
        if (tid == 0 && rank == 0 && a.status) record_error(a.status, MLA_ERR_INDEX);
        len = min(max(len, 0), T);
    }
    // the tokens and the probabilities their first test needs, all at once
    if (tid < T) {
        const int32_t x = a.tokens[(int64_t)b * T + tid];
        const int32_t par = a.parents ? a.parents[(int64_t)b * T + tid] : tid - 1;
        const bool fine = x >= 0 && x < V && par >= -1 && par < tid;
        if (!fine && tid < len && rank == 0 && a.status) record_error(a.status, MLA_ERR_INDEX);
        s_tok[tid] = x >= 0 && x < V ? x : -1;
        s_par[tid] = par >= -1 && par < tid ? par : -2;  // -2: a parent that is never reached
        s_depth[tid] = -1;
        s_u[tid] = a.uniforms[(int64_t)b * (T + 1) + tid];
        s_p[tid] = fine ? target[(int64_t)(par + 1) * V + x] : 0.f;
        s_q[tid] = fine && draft ? draft[(int64_t)tid * V + x] : 1.f;
    }
    if (tid == 0) s_u[T] = a.uniforms[(int64_t)b * (T + 1) + T];
    __syncwarp();
    ptx::cluster_sync();  // and every CTA runs before another one writes into its s_slice

    // contiguous slices of whole 128-element groups, one per CTA, and chunks, one per warp
    const int slice = ((V + kVfCluster - 1) / kVfCluster + 127) & ~127;
    const int v0 = min(V, (int)rank * slice), v1 = min(V, v0 + slice);
    const int chunk = ((slice + kVfWarps - 1) / kVfWarps + 31) & ~31;
    const int c0 = min(v1, v0 + warp * chunk), c1 = min(v1, c0 + chunk);
    int turns = 0;

    // The sum of what is left, over the whole vocabulary; every thread of the cluster calls it.
    auto total_left = [&](const Residual &r) -> uint64_t {
        uint64_t sum = 0;
        if (r.n == 0 || (r.n == 1 && r.q)) {
            // the usual case: one or two rows, eight loads of each in flight
            const float *p = r.p, *q = r.n == 1 ? r.q + (int64_t)r.rej[0] * V : nullptr;
            for (int v = c0 + lane; v < c1; v += 32 * 8) {
                float pv[8], qv[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int w = v + 32 * i;
                    pv[i] = w < c1 ? p[w] : 0.f;
                    qv[i] = q && w < c1 ? q[w] : 0.f;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint64_t x = fixed58(pv[i]), y = fixed58(qv[i]);
                    sum += x > y ? x - y : 0;
                }
            }
        } else {
            for (int v = c0 + lane; v < c1; v += 32) sum += r.at(v);
        }
        sum = warp_sum(sum);
        if (lane == 0) s_warp[warp] = sum;
        __syncthreads();
        const int turn = turns & 1;
        if (warp == 0) {
            uint64_t t = lane < kVfWarps ? s_warp[lane] : 0;
            t = warp_sum(t);
            if (lane < kVfCluster) {
                const uint32_t dst = ptx::mapa(ptx::smem_u32(&s_slice[turn][rank]), (uint32_t)lane);
                asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(dst), "l"(t) : "memory");
            }
        }
        // two turns of s_slice: a CTA can be one turn ahead of a peer that still reads
        __syncwarp();
        ptx::cluster_sync();
        ++turns;
        uint64_t all = 0;
        for (int k = 0; k < kVfCluster; ++k) all += s_slice[turn][k];
        return all;
    };

    // the walk; every thread takes the same decisions
    int at = -1, depth = 0, nrej = 0;
    double mass = 1.0;
    Residual r{target, draft, s_tok, s_rej, s_mass, 0, V};
    for (int i = 0; i < len; ++i) {
        const int x = s_tok[i];
        if (s_par[i] != at || x < 0) continue;
        bool stands;
        if (nrej == 0) {
            stands = (double)s_u[i] * (double)s_q[i] < (double)s_p[i];  // 48-bit products: exact
        } else {
            stands = (double)s_u[i] * (double)s_q[i] * mass < (double)r.at(x);
        }
        if (stands) {
            if (tid == 0) s_depth[i] = depth;
            at = i;
            ++depth;
            nrej = 0;
            mass = 1.0;
            r.p = target + (int64_t)(i + 1) * V;
            r.n = 0;
            continue;
        }
        __syncthreads();  // the list below may still be read for an earlier test
        if (tid == 0) {
            s_rej[nrej] = i;
            s_mass[nrej] = mass;
        }
        __syncthreads();
        r.n = ++nrej;
        // the mass left is needed by a sibling's test (the draw sums again only if none came)
        bool sibling = false;
        for (int k = i + 1; k < len; ++k) sibling = sibling || (s_par[k] == at && s_tok[k] >= 0);
        if (sibling) mass = (double)total_left(r);
    }
    uint64_t all = total_left(r);
    if (all == 0 && nrej > 0) {  // nothing is left: the target's own row
        r.n = 0;
        all = total_left(r);
    }
    // the draw: the first v whose running sum exceeds u times the total
    if (all == 0) {
        if (rank == 0 && tid == 0) a.next_token[b] = -1;
    } else {
        const float u = s_u[T];
        uint64_t want = u > 0.f ? __double2ull_rz((double)u * (double)all) : 0;
        if (want >= all) want = all - 1;
        const int turn = (turns - 1) & 1;
        int owner = 0;
        while (owner < kVfCluster - 1 && want >= s_slice[turn][owner]) want -= s_slice[turn][owner++];
        if ((int)rank == owner) {
            int w = 0;
            while (w < kVfWarps - 1 && want >= s_warp[w]) want -= s_warp[w++];
            if (warp == w) {
                // each lane a contiguous run of the chunk; the lane whose run holds the place
                // searches it
                const int per = (c1 - c0 + 31) / 32;
                const int l0 = min(c1, c0 + lane * per), l1 = min(c1, l0 + per);
                uint64_t mine = 0;
#pragma unroll 4
                for (int v = l0; v < l1; ++v) mine += r.at(v);
                uint64_t upto = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += y;
                }
                const unsigned past = __ballot_sync(0xffffffffu, upto > want);
                if (past && lane == __ffs(past) - 1) {
                    uint64_t run = upto - mine;
                    int v = l0;
                    for (; v < l1 - 1; ++v) {
                        run += r.at(v);
                        if (run > want) break;
                    }
                    a.next_token[b] = v;
                } else if (!past && lane == 0) {
                    a.next_token[b] = min(c0, V - 1);  // sums that overflowed: rows far from adding up to 1
                }
            }
        }
    }
    if (rank == 0) {
        __syncthreads();  // s_depth
        if (tid == 0) a.num_accepted[b] = depth;
        if (tid < T) a.depths[(int64_t)b * T + tid] = s_depth[tid];
    }
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status mla_verify_draft(const float *target, const float *draft, const int32_t *tokens,
                                       const int32_t *parents, const int32_t *tree_lens, const float *uniforms, int B,
                                       int T, int V, int32_t *num_accepted, int32_t *depths, int32_t *next_token,
                                       int32_t *device_status, void *stream) {
    if (B < 0 || T < 1 || V < 1) return MLA_ERR_INVALID_ARG;
    if (T > kVfMaxT || V > (1 << 20) || B > 0x7FFFFFFF / kVfCluster) return MLA_ERR_UNSUPPORTED;
    if (B == 0) return MLA_OK;
    if (!target || !tokens || !uniforms || !num_accepted || !depths || !next_token) return MLA_ERR_INVALID_ARG;
    VerifyArgs a{target, draft, tokens, parents, tree_lens, uniforms, T, V, num_accepted, depths, next_token,
                 (int *)device_status};
    return launch_pdl(verify_kernel, B * kVfCluster, kVfThreads, 0, (cudaStream_t)stream, a) == cudaSuccess
               ? MLA_OK
               : MLA_ERR_CUDA;
}
