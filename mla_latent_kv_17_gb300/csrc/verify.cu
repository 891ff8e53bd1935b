// Verification of a drafted tree against the target's probabilities.  The definition is in
// include/mla_decode.h (mla_verify_draft).
//
// What the walk needs of a token that is accepted is two probabilities; only where it stops
// are whole rows read: the target's row and the rows of the drafts rejected there.  One
// cluster of eight CTAs takes a request, each CTA an eighth of the vocabulary, so that a
// single request still streams its rows through eight SMs; memory bounds a large batch (64
// requests x 131,072 tokens, one rejection each: 67 MB, 17.7 us - four CTAs per SM at most have
// their rows in flight, and the walk, the cluster's sum and the draw stand before and after).
//
// All sums are 64-bit integers: a probability is cut to a multiple of 2^-58, which keeps every
// bit of a value of 2^-34 or more, the residual of a first rejection is an exact subtraction,
// and integer addition is exact in any order - so the chosen token does not depend on how the
// vocabulary is split.  (fp32 sums would move the borders between a vocabulary's tokens by
// about 1e-10 each, enough to change one draw in some ten thousand; fp64 additions run at 2
// per cycle and SM here.)
//
// Per stop the sum pass leaves a partial sum per warp (a contiguous chunk) and per CTA (a
// contiguous slice); the draw then finds its slice and chunk from those sums, and the CTA that
// owns them searches the chunk again, from L2.
#include <cuda_runtime.h>
#include <math.h>

#include "common.cuh"
#include "sm103_ptx.cuh"
#include "tc_util.cuh"

namespace mla {
namespace {

constexpr int kVfCluster = 8;
constexpr int kVfThreads = 256;
constexpr int kVfWarps = kVfThreads / 32;
constexpr int kVfMaxT = 64;

struct VerifyArgs {
    const float *target, *draft;
    const int32_t *tokens, *parents, *tree_lens;
    const float *uniforms;
    int T, V;
    int32_t *num_accepted, *depths, *next_token;
    int *status;
};

// A probability as it counts (NaN and negative values: 0, above 1: 1).
__device__ __forceinline__ float counted(float p) { return fminf(fmaxf(p, 0.f), 1.f); }

// The same as a multiple of 2^-58: the significand at the top of a 64-bit word, shifted down by
// what the exponent lacks (shifts of 64 and more give 0).  The conversion instruction to 64-bit
// integers runs on the fp64 pipe, which it kept 75 % busy, for more than twice the whole call's time at 64 x 131,072.
__device__ __forceinline__ uint64_t fixed58(float p) {
    const uint32_t b = __float_as_uint(counted(p));
    const uint64_t m = (uint64_t)((b << 8) | 0x80000000u) << 32;  // 2^63 x 1.fraction
    uint64_t r;
    asm("shr.u64 %0, %1, %2;" : "=l"(r) : "l"(m), "r"(132u - (b >> 23)));
    return r;
}

// What is left of the target's row after the rejected drafts rej[0 .. n): their masses are the
// sums left before each (the first: 1).
struct Residual {
    const float *p;        // the target's row
    const float *q;        // the draft's rows of this request, or null: certain of its token
    const int32_t *tokens;
    const int *rej;
    const uint64_t *mass;  // multiples of 2^-58
    int n, V;

    __device__ __forceinline__ uint64_t minus(uint64_t left, int k, float qv) const {
        // the first draft is subtracted exactly; later ones are scaled by the mass left (q and the mass
        // as whole multiples of 2^-58, the product cut to one; fp64 units are few on this part)
        const uint64_t f = fixed58(qv), d = k == 0 ? f : __umul64hi(f, mass[k]) << 6 | (f * mass[k]) >> 58;
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

// What is left of tokens v, v + kStep, ..., v + 7 kStep (0 at `end` and beyond): the rows' loads in flight
// together.
template <int kStep>
__device__ __forceinline__ void left8(const Residual &r, int v, int end, uint64_t (&left)[8]) {
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = v + kStep * k < end ? r.p[v + kStep * k] : 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) left[k] = fixed58(x[k]);
    for (int j = 0; j < r.n; ++j) {
        if (r.q) {
            const float *q = r.q + (int64_t)r.rej[j] * r.V;
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = v + kStep * k < end ? q[v + kStep * k] : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) left[k] = r.minus(left[k], j, x[k]);
        } else {  // certain of its token
            const int d = r.tokens[r.rej[j]] - v;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (d == kStep * k) left[k] = 0;
        }
    }
}

__device__ __forceinline__ uint64_t left_of(float p, float q) {
    const uint64_t x = fixed58(p), y = fixed58(q);
    return x > y ? x - y : 0;
}

// A lane's part of the sum of max(p - q, 0) (or of p) over [c0, c1).  16-byte loads where both
// rows allow them (c0 is a multiple of 32), single values otherwise.
template <bool kQ>
__device__ __forceinline__ uint64_t sum_rows(const float *p, const float *q, int c0, int c1, int lane) {
    uint64_t sum = 0;
    int v = c0;
    if (((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & 15u) == 0) {
        for (; v + 512 <= c1; v += 512) {
            float4 pv[4], qv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                pv[i] = *reinterpret_cast<const float4 *>(p + v + 128 * i + 4 * lane);
                if constexpr (kQ) qv[i] = *reinterpret_cast<const float4 *>(q + v + 128 * i + 4 * lane);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (kQ)
                    sum += left_of(pv[i].x, qv[i].x) + left_of(pv[i].y, qv[i].y) + left_of(pv[i].z, qv[i].z) +
                           left_of(pv[i].w, qv[i].w);
                else
                    sum += fixed58(pv[i].x) + fixed58(pv[i].y) + fixed58(pv[i].z) + fixed58(pv[i].w);
            }
        }
    }
    for (; v < c1; v += 256) {
        float pv[8], qv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int w = v + 32 * i + lane;
            pv[i] = w < c1 ? p[w] : 0.f;
            if constexpr (kQ) qv[i] = w < c1 ? q[w] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += kQ ? left_of(pv[i], qv[i]) : fixed58(pv[i]);
    }
    return sum;
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__global__ void __cluster_dims__(kVfCluster, 1, 1) __launch_bounds__(kVfThreads, 4) verify_kernel(VerifyArgs a) {
    __shared__ int32_t s_tok[kVfMaxT], s_par[kVfMaxT], s_depth[kVfMaxT];
    __shared__ bool s_stands[kVfMaxT];            // would token i stand as the first one tried at its place?
    __shared__ bool s_answer;
    __shared__ int s_rej[kVfMaxT];
    __shared__ uint64_t s_mass[kVfMaxT];
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
    // every small load at once, then the probabilities the tokens' first tests need
    int32_t len = a.tree_lens ? a.tree_lens[b] : T;
    const float u_draw = a.uniforms[(int64_t)b * (T + 1) + T];
    int32_t x = -1, par = tid - 1;
    float u = 0.f;
    if (tid < T) {
        x = a.tokens[(int64_t)b * T + tid];
        if (a.parents) par = a.parents[(int64_t)b * T + tid];
        u = a.uniforms[(int64_t)b * (T + 1) + tid];
    }
    // (the cluster's CTAs all run before one writes into another's s_slice: waited for there)
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    bool wrong = len < 0 || len > T;
    len = min(max(len, 0), T);
    if (tid < T) {
        const bool fine = x >= 0 && x < V && par >= -1 && par < tid;
        wrong = wrong || (!fine && tid < len);
        s_tok[tid] = x >= 0 && x < V ? x : -1;
        s_par[tid] = par >= -1 && par < tid ? par : -2;  // -2: a parent that is never reached
        s_depth[tid] = -1;
        // (fp64: 48-bit products, exact; by the token's own thread only, since the units are few)
        const float p = fine ? target[(int64_t)(par + 1) * V + x] : 0.f;
        const float q = fine && draft ? draft[(int64_t)tid * V + x] : 1.f;
        s_stands[tid] = (double)u * (double)counted(q) < (double)counted(p);
        if (wrong && rank == 0 && a.status) record_error(a.status, MLA_ERR_INDEX);
    }
    __syncthreads();

    // contiguous slices of whole 128-element groups, one per CTA, and chunks, one per warp
    const int slice = ((V + kVfCluster - 1) / kVfCluster + 127) & ~127;
    const int v0 = min(V, (int)rank * slice), v1 = min(V, v0 + slice);
    const int chunk = ((slice + kVfWarps - 1) / kVfWarps + 31) & ~31;
    const int c0 = min(v1, v0 + warp * chunk), c1 = min(v1, c0 + chunk);
    int turns = 0;

    // The sum of what is left, over the whole vocabulary; every thread of the cluster calls it.
    auto total_left = [&](const Residual &r) -> uint64_t {
        uint64_t sum = 0;
        if (!r.q || r.n <= 1) {
            // the usual case: one or two rows, sixteen values of each in flight per lane
            const float *p = r.p, *q = r.q && r.n == 1 ? r.q + (int64_t)r.rej[0] * V : nullptr;
            sum = q ? sum_rows<true>(p, q, c0, c1, lane) : sum_rows<false>(p, p, c0, c1, lane);
            for (int j = lane; j < r.n && !r.q; j += 32) {  // certain drafts: their tokens are lost, each once
                const int x = r.tokens[r.rej[j]];
                bool lost = x >= c0 && x < c1;
                for (int i = 0; i < j; ++i) lost = lost && r.tokens[r.rej[i]] != x;
                if (lost) sum -= fixed58(p[x]);
            }
        } else {
            for (int v = c0 + lane; v < c1; v += 256) {
                uint64_t left[8];
                left8<32>(r, v, c1, left);
#pragma unroll
                for (int k = 0; k < 8; ++k) sum += left[k];
            }
        }
        sum = warp_sum(sum);
        if (lane == 0) s_warp[warp] = sum;
        __syncthreads();
        const int turn = turns & 1;
        if (turns == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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
    uint64_t mass = 0;  // what is left of the row's sum, where a sibling is tried after a rejection
    Residual r{target, draft, s_tok, s_rej, s_mass, 0, V};
    for (int i = 0; i < len; ++i) {
        const int x = s_tok[i];
        if (s_par[i] != at || x < 0) continue;
        bool stands = s_stands[i];
        if (nrej > 0) {
            if (tid == 0) {
                const double u = a.uniforms[(int64_t)b * (T + 1) + i];
                s_answer = u * (double)(draft ? counted(draft[(int64_t)i * V + x]) : 1.f) * (double)mass < (double)r.at(x);
            }
            __syncthreads();
            stands = s_answer;
        }
        if (stands) {
            if (tid == 0) s_depth[i] = depth;
            at = i;
            ++depth;
            nrej = 0;
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
        if (!sibling) continue;
        if (!draft && nrej > 1) {
            // certain drafts: only the token itself is lost (nothing, where it was lost before);
            // the first rejection's sum is the only pass a place needs
            r.n = nrej - 1;
            mass -= r.at(x);
            r.n = nrej;
        } else {
            mass = total_left(r);
        }
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
        // floor(u total), exact: u as a 64-bit fraction
        uint64_t want = u_draw < 1.f ? __umul64hi(fixed58(u_draw) << 6, all) : all - 1;
        const int turn = (turns - 1) & 1;
        int owner = 0;
        while (owner < kVfCluster - 1 && want >= s_slice[turn][owner]) want -= s_slice[turn][owner++];
        if ((int)rank == owner) {
            int w = 0;
            while (w < kVfWarps - 1 && want >= s_warp[w]) want -= s_warp[w++];
            // chunk w again, by the whole CTA, a piece of 8 values a thread at a time; the thread whose
            // values hold the place finds it among them (reading them again, one after another, took
            // 3 us of this call's end)
            const int k0 = min(v1, v0 + w * chunk), k1 = min(v1, k0 + chunk);
            // (sums that overflowed, of rows far from adding up to 1, may hold the place nowhere)
            if (tid == 0) a.next_token[b] = max(k1 - 1, 0);
            for (int c = k0; c < k1; c += 8 * kVfThreads) {
                const int v = c + 8 * tid;
                uint64_t left[8];
                left8<1>(r, v, k1, left);
                uint64_t mine = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) mine += left[k];
                uint64_t upto = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += y;
                }
                __syncthreads();  // s_warp has been read
                if (lane == 31) s_warp[warp] = upto;
                __syncthreads();
                uint64_t piece = 0;
                for (int k = 0; k < kVfWarps; ++k) {
                    if (k == warp) upto += piece;
                    piece += s_warp[k];
                }
                if (upto > want && upto - mine <= want) {  // one thread, unless they overflowed
                    uint64_t run = upto - mine;
                    int at_v = v + 7;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        run += left[k];
                        if (run > want && at_v == v + 7) at_v = v + k;
                    }
                    a.next_token[b] = min(at_v, k1 - 1);
                }
                if (want < piece) break;  // the same in every thread
                want -= piece;
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
