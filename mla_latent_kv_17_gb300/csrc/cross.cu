// Attention of a ragged batch of query runs to key runs of another length (an encoder's states, a
// cached prefix, a chunk over its prefix and itself).  The definition is in include/mla_decode.h
// (mla_cross_attention).
//
// cross_plan_kernel: one CTA cuts the batch into items - a tile of 128 or 256 query rows of a run
// with the key tiles (of 128) it sees - and, where whole items would leave SMs idle at the end, the
// longer ones into pieces: those of all heads, or of the last ones.  Items and pieces are ordered by
// falling length; the lists are the same for all their heads.  3 us (5 - 7 where keys are cut).
//
// cross_kernel: a persistent CTA per SM takes units (a piece and a head) from a counter, longest
// pieces first, groups of eight heads in turn so that the keys and values in use stay in L2.  Per
// unit, as in the causal prefill: S = Q K^T on tcgen05 into TMEM, online softmax with one thread per
// query row, P as bf16 over its scores in TMEM, O += P V.  The loads of the next unit run under the last
// tiles of the present one, its first scores under the epilogue.
//   P is rounded to bf16 because the MMA takes both operands in one type and the values are bf16 (fp16 would not hold
// them; P in two bf16 parts would double PV).  That is up to 2^-8 of each weight: with the result's own rounding to
// bf16 the error is 0.0022 - 0.0023 of the result (rms) where fp32 weights would give 0.0017.  The sum of weights is
// taken before the rounding, in fp32.
//   256 rows, for many long runs: two query tiles share the keys and take turns on the tensor pipe.  1,001 queries over 9,193 keys,
//   causal, 128 heads: 490 - 500 us with plan and joining, 0.75 of the measured bf16 rate (466 us, 0.80, by itself).  A key
//   tile takes 3,650 cycles where its MMAs take 2,560: the warp that issues them is the narrowest place (about 60
//   cycles an operation, and 120 a wait, even where there is nothing to wait for), then shared memory (8 KB of
//   operands in the 64 cycles of a score operation).
//   128 rows: one query tile with two score buffers and more of the shared memory for keys and values.  8 ragged
//   prompts of 200 - 1,024 queries over 256 - 2,048 keys, 32 heads: 116 us; 64 single tokens over 256 - 2,048 keys,
//   16 heads: 101 us, 0.88 of the copy rate.
// Keys and values go round one ring of 16-KB boxes in the order of their first use: with a key buffer twice and
// a value buffer once instead, the values came a load's latency late for the first of two query tiles (3,800
// cycles a key tile).  Two tiles ahead of their load they are brought into L2 where two query tiles share them
// (545 -> 531 us; where memory bounds the call it costs 3 %).
// The pieces of an item leave normalised partial results, which cross_merge_kernel joins (18 us by itself for 9 items
// of 128 rows in 26 parts x 16 heads, 40 MB: a chain of loads per 32 rows).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "launch.h"
#include "mla_decode.h"
#include "sm103_ptx.cuh"
#include "tc_util.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kCrDh = 128;
constexpr int kCrTile = 128;            // query rows of a tile (TMEM lanes), keys of a tile
constexpr int kCrHeadGroup = 8;
constexpr int kCrMinPiece = 4;          // key tiles
// An item longer than a third of an SM's share of the work is cut.  (4 x 256 - 512 queries over 1,024 - 8,192 keys x
// 16 heads with 2, 3, 4, 5: 110, 101, 104, 102 us; 2 x 2,048 causal queries over 4,096 x 16: 124, 123, 132, 144: parts
// cost a start, an end and their joining.)
constexpr int kCrShare = 3, kCrShareRest = 2;  // (at most kCrShare: see the layout)
constexpr int kCrJoin = 8;              // what the joining of parts costs, in key tiles
constexpr int kCrSms = 152;             // a GB300's (for the choice of the items' size alone)
constexpr float kCrPair = 1.77f;        // what a key tile takes with two query tiles, against one (3,600 cycles against 2,040)
constexpr float kCrAlike = 1.2f;        // items are much alike: the longest is at most this much longer than they are on average
constexpr int kCrAhead = 2;             // key tiles between the prefetch into L2 and the load
constexpr int kCrItemCost = 2;          // an item's start and end, in key tiles
// A role may wait as long as another one's unit takes, 3,600 cycles a key tile, so the limit of a wait grows with the
// keys: by twice that, and a little.
constexpr long long kCrWaitPerTile = 8000;
constexpr float kCrRescale = 8.f;       // the reference maximum moves when exceeded by 2^8
constexpr uint32_t kCrossMagic = 0x4D4C4158u;  // "MLAX"
// Beside the status word once a plan has been made: memory without them may hold anything where that word is.
constexpr uint32_t kCrossMarkY = 0x58535441u, kCrossMarkZ = 0x9E3779B9u, kCrossMarkW = 0xC2B2AE35u;

struct CrossHeader {
    uint32_t magic;
    int32_t B, H, total_q, total_k, causal, rows, sms, pieces, splits, groups, last;
    int32_t whole, items;  // heads whose items stay whole, and those (pieces: of the other heads)
    int32_t reserved[2];
};
static_assert(sizeof(CrossHeader) == 64, "plan header is 64 bytes");

// Key tiles [g0, g1) of the run's nk keys (from row k0 on) for query rows q0 .. q0 + nrows; a causal
// plan's row r sees the keys below see0 + r (0 and less: none), any other's all of them.
struct CrossPiece {
    int32_t q0, nrows, k0, nk, see0, g0, g1;
    int32_t row0;  // the piece's first partial row (-1: the item's only piece, its rows are the result)
    int32_t head;  // (filled in where a unit is taken)
    int32_t reserved[3];
};
// An item that is cut: its query rows, its parts' partial rows (part p: row0 + p nrows ..), and how many
// groups of kCrGroup rows the cut items before it have.
constexpr int kCrGroup = 32;
struct CrossSplit {
    int32_t q0, nrows, row0, parts, before;
};
// A part's results of one of the `heads` heads with cut items, rows row0 .. row0 + nrows of the partials: nrows
// log-sum-exps (log2 units), and 32 runs of nrows four-column pieces (a warp's 32 rows write and read 512 bytes in
// a row).
MLA_HD int64_t part_at(int row0, int nrows, int heads, int head) { return (int64_t)row0 * heads + (int64_t)head * nrows; }

struct CrossLayout {
    size_t pieces, order, splits, seqs, item_off, part_lse, part_o, total;
    int max_pieces, max_splits;
    int64_t max_parts;  // rows of partial results, of all heads
};

constexpr size_t kCrStatus = 128;    // device status word, where mla_decode_status looks for it, and three marks
constexpr size_t kCrCounters = 192;  // next unit, CTAs that are done

// Query rows per item: 256 (two query tiles that share each key tile's load) or 128.  Two share, where no more than
// a quarter of the tiles would be empty and the runs of keys are long (1,536 on average), if the keys and values of
// all heads do not stay in L2 (192 MB and more), or if their units, which are fewer and shorter per row, would end
// sooner: judged for runs of average length, and only where keys are three times the queries, since a causal run's
// items differ much where they are not.  Else smaller items balance better and overlap their ends.
// Measured, us with 128 and with 256 rows (runs x queries x keys x heads): 4 x 512 x 8,192 x 128 1,119 / 941,
// 8 x 1,024 x 2,048 x 32 290 / 254, 1 x 256 x 16,000 x 128 347 / 297; sooner: 2 x 2,048 x 16,384 x 8 305 / 234,
// 9 x 256 x 2,000 x 16 73 / 54, 2 x 1,024 x 6,000 x 32 209 / 187, 1 x 2,048 x 8,192 x 16 causal 134 / 126; not sooner:
// 1 x 512 x 4,096 x 40 61 / 88, 1 x 1,024 x 4,000 x 16 43 / 65; causal, keys twice the queries: 2 x 2,048 x 4,096 x 16
// 123 / 152; half-empty pairs: 8 x 300 x 4,000 x 64 451 / 467; short keys: 4 x 512 x 1,024 x 128 154 / 156,
// 8 x 1,024 x 1,024 x 32 152 / 147, 8 x 1,024 x 500 x 32 97 / 101, 8 x 1,024 x 200 x 32 68 / 73, 8 x 3,384 x 38 x 32
// 161 / 148, joined 8 x 1,750 x 13 x 64 277 / 297.  Where the average hides much, the other size may be better: 8 ragged
// causal runs of 200 - 1,024 queries over 1,024 - 2,048 keys x 32 heads 142 / 154 (256 rows, by the 192 MB), over
// 1,024 - 8,192 473 / 450.
// When this many units of this length would end, in key tiles: whole ones in rounds, or cut (see the plan).
MLA_HD float cross_end(int64_t units, float length) {
    const float rounds = (float)((units + kCrSms - 1) / kCrSms) * length, cut = 1.1f * units * length / kCrSms + kCrJoin;
    return rounds < cut ? rounds : cut;
}
MLA_HD int cross_rows(int B, int H, int64_t total_q, int64_t total_k) {
    const int64_t q = total_q / B, k = total_k / B, tiles = (q + kCrTile - 1) / kCrTile, pairs = (tiles + 1) / 2;
    if (tiles < 2 || 8 * pairs > 5 * tiles || k < 1536) return kCrTile;
    const bool far = (int64_t)H * total_k * (4 * kCrDh) >= ((int64_t)192 << 20);
    const float length = (float)k / kCrTile + kCrItemCost;
    const bool sooner = k >= 3 * q && 1.06f * kCrPair * cross_end(pairs * B * H, length) <= cross_end(tiles * B * H, length);
    return far || sooner ? 2 * kCrTile : kCrTile;
}

MLA_HD CrossLayout cross_layout(int B, int H, int64_t total_q, int sms) {
    CrossLayout L;
    // (room for items of either size)
    // An item of t tiles of a head is cut into n = ceil(t / target) > 1 pieces, and the target is at least the h
    // heads' cost / `cuts`: cuts / h items are cut at most, into 2 cuts / h pieces together and cuts / h + 1 each.
    const int64_t cuts = (int64_t)kCrShare * sms, items = total_q / kCrTile + B;
    L.max_pieces = (int)(2 * items + 4 + cuts);  // whole ones, then the others
    L.max_splits = (int)(items < cuts ? items : cuts);
    L.max_parts = (cuts + H) * (total_q < 4 * kCrTile ? total_q : 4 * kCrTile);
    size_t o = 256;
    L.pieces = o;
    o = align_up(o + sizeof(CrossPiece) * (size_t)L.max_pieces, 256);
    L.order = o;
    o = align_up(o + sizeof(int32_t) * (size_t)L.max_pieces, 256);
    L.splits = o;
    o = align_up(o + sizeof(CrossSplit) * (size_t)L.max_splits, 256);
    L.seqs = o;
    o = align_up(o + sizeof(int4) * (size_t)B, 256);
    L.item_off = o;
    o = align_up(o + sizeof(int32_t) * (size_t)(B + 1), 256);
    L.part_lse = o;
    o = align_up(o + sizeof(float) * (size_t)L.max_parts, 256);
    L.part_o = o;
    o = align_up(o + sizeof(float) * (size_t)L.max_parts * kCrDh, 256);
    L.total = o;
    return L;
}

// ------------------------------------------------------------------ the plan
constexpr int kCpThreads = 512;
constexpr int kCpWarps = kCpThreads / 32;
constexpr int kCpSort = 2048;  // pieces that are put in order (more of them even out by themselves)
constexpr int kCpKeep = 1024;  // runs whose starts stay in shared memory
constexpr int kCpFew = 8;      // pieces of an item that one thread writes

// Four values a thread, scanned together: sums, or maxima.
struct Four {
    int64_t v[4];
};
template <bool kMax>
__device__ __forceinline__ Four both(Four a, const Four &b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a.v[i] = kMax ? (a.v[i] > b.v[i] ? a.v[i] : b.v[i]) : a.v[i] + b.v[i];
    return a;
}
// Inclusive scan of the first kN of x over the block; *all receives the whole.  sh: kCpWarps places.
template <bool kMax, int kN>
__device__ Four block_scan(Four x, Four *all, Four *sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        Four y = x;
#pragma unroll
        for (int i = 0; i < kN; ++i) y.v[i] = __shfl_up_sync(0xffffffffu, x.v[i], o);
        if (lane >= o) x = both<kMax>(x, y);
    }
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    // (a lane per warp: every warp scans the warps' wholes for itself)
    Four t = sh[lane < kCpWarps ? lane : 0];
    if (lane >= kCpWarps) t = Four{};
#pragma unroll
    for (int o = 1; o < kCpWarps; o <<= 1) {
        Four y = t;
#pragma unroll
        for (int i = 0; i < kN; ++i) y.v[i] = __shfl_up_sync(0xffffffffu, t.v[i], o);
        if (lane >= o) t = both<kMax>(t, y);
    }
    Four before = x;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        before.v[i] = __shfl_sync(0xffffffffu, t.v[i], warp > 0 ? warp - 1 : 0);
        all->v[i] = __shfl_sync(0xffffffffu, t.v[i], kCpWarps - 1);
    }
    if (warp > 0) x = both<kMax>(x, before);
    __syncthreads();
    return x;
}

struct CrossPlanArgs {
    const int32_t *cu_q, *cu_k;
    int B, H, total_q, total_k, causal, rows, sms;
    unsigned char *ws;
    CrossLayout L;
};

// Keys that the rows up to `end` (of nq) see.
__device__ __forceinline__ int seen_by(int end, int nq, int nk, int causal) {
    if (!causal) return nk;
    const int s = nk - nq + end;
    return s < 0 ? 0 : s;
}
__device__ __forceinline__ int key_tiles(int keys) { return (keys + kCrTile - 1) / kCrTile; }

__global__ void __launch_bounds__(kCpThreads) cross_plan_kernel(const __grid_constant__ CrossPlanArgs a) {
    __shared__ Four s_scan[kCpWarps];
    __shared__ __align__(16) uint32_t s_key[kCpSort];
    __shared__ int4 s_seq[kCpKeep];
    __shared__ int32_t s_off[kCpKeep];
    __shared__ int s_last, s_longest;
    __shared__ uint4 s_state;
    if (threadIdx.x == 0) s_longest = 0;
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x;
    const bool keep = a.B <= kCpKeep;
    int4 *seqs = keep ? s_seq : reinterpret_cast<int4 *>(a.ws + a.L.seqs);
    int32_t *item_off = keep ? s_off : reinterpret_cast<int32_t *>(a.ws + a.L.item_off);
    CrossPiece *pieces = reinterpret_cast<CrossPiece *>(a.ws + a.L.pieces);
    CrossSplit *splits = reinterpret_cast<CrossSplit *>(a.ws + a.L.splits);
    int32_t *order = reinterpret_cast<int32_t *>(a.ws + a.L.order);
    uint4 *status = reinterpret_cast<uint4 *>(a.ws + kCrStatus);
    if (tid == kCpThreads - 1) s_state = *status;  // (used at the end; in a register the plan waits for it: +0.3 us)
    bool fell = false;                             // some run does not lie as it should

    // the runs: starts that fall or lie outside are moved up or in (and recorded), so that runs never
    // overlap and the items fit their places
    Four upto{}, all;  // ends of the queries and keys so far
    int64_t items = 0, cost = 0;
    for (int b0 = 0; b0 < a.B; b0 += kCpThreads) {
        const int b = b0 + tid;
        int qs = 0, qe = 0, ks = 0, ke = 0;
        bool bad = false;
        if (b < a.B) {
            const int32_t r[4] = {a.cu_q[b], a.cu_q[b + 1], a.cu_k[b], a.cu_k[b + 1]};
            qs = min(max(r[0], 0), a.total_q);
            qe = min(max(r[1], 0), a.total_q);
            ks = min(max(r[2], 0), a.total_k);
            ke = min(max(r[3], 0), a.total_k);
            bad = r[0] != qs || r[1] != qe || r[2] != ks || r[3] != ke || qs > qe || ks > ke;
        }
        bad = __syncthreads_or(bad);
        fell |= bad;
        if (bad || upto.v[1] > 0 || upto.v[3] > 0) {
            // a run starts no earlier than the largest start before it, and ends no earlier
            const Four x = block_scan<true, 4>(Four{{qs, max(qs, qe), ks, max(ks, ke)}}, &all, s_scan);
            qs = (int)max(upto.v[1], x.v[0]);
            qe = (int)max(upto.v[1], x.v[1]);
            ks = (int)max(upto.v[3], x.v[2]);
            ke = (int)max(upto.v[3], x.v[3]);
            upto = both<true>(upto, all);
        } else if (a.B > kCpThreads) {
            block_scan<true, 4>(Four{{qs, qe, ks, ke}}, &all, s_scan);
            upto = all;
        }
        const int nq = b < a.B ? qe - qs : 0, nk = b < a.B ? ke - ks : 0;
        const int tiles = (nq + a.rows - 1) / a.rows;
        int64_t c = 0;
        if (!a.causal) {
            c = (int64_t)tiles * (kCrItemCost + key_tiles(nk));
        } else {
            for (int j = 0; j < tiles; ++j)
                c += kCrItemCost + key_tiles(seen_by(min(nq, (j + 1) * a.rows), nq, nk, 1));
        }
        const Four x = block_scan<false, 2>(Four{{tiles, c, 0, 0}}, &all, s_scan);  // (a barrier: s_longest is set)
        if (tiles > 0) atomicMax(&s_longest, kCrItemCost + key_tiles(nk));
        if (b < a.B) {
            seqs[b] = make_int4(qs, nq, ks, nk);
            item_off[b] = (int32_t)(items + x.v[0] - tiles);
        }
        items += all.v[0];
        cost += all.v[1];
    }
    __syncthreads();

    // Items of more than a third of an SM's share are cut, where that pays: whole ones, longest first, end within
    // as many rounds of the longest as there are, and within the share and the longest; pieces end about half a
    // piece after the share, and are joined.  (Us whole and in pieces: 1,024 queries x 2,048 keys x 19 heads 29 / 41,
    // 256 x 8,192 x 128 causal 135 / 181, 256 x 32,000 x 128 490 / 538; 512 x 6,000 and 3,000 and 1,000 x 32 146 / 117.)
    // Where the items are much alike, those of the first heads stay whole, as many units as fill all SMs equally
    // often, and the other heads' are cut, more than half of an SM's share of them.  (Us before and so: 5 x 512 x
    // 3,000 x 32 heads 189 / 139, 512 x 4,096 x 40 74 / 62, 1,001 x 9,193 x 128 causal 532 / 497; by thirds 142, 62,
    // 502.  Where the longest is 1.8 times the mean, 30 x 1 x 50 - 8,750 x 16, 193 / 243: the last whole ones are long.)
    int whole = a.H, target = INT32_MAX;
    if (items > 0) {
        const uint32_t units = (uint32_t)items * a.H, rounds = (units + a.sms - 1) / a.sms;  // (fits: see the shapes)
        const float longest = s_longest, mean = (float)cost * a.H / a.sms;
        const bool alike = longest * items <= kCrAlike * cost;
        const int some = alike ? (int)((rounds - 1) * a.sms / (uint32_t)items) : 0;
        const int64_t shares = (int64_t)(some > 0 ? kCrShareRest : kCrShare) * a.sms;
        const int64_t share = (cost * (a.H - some) + shares - 1) / shares;
        const int least = (int)(share > kCrMinPiece ? share : kCrMinPiece);
        if (fminf(rounds * longest, mean + longest) > mean + 0.5f * least + kCrJoin) {
            whole = some;
            target = least;
        }
    }
    const int cut_heads = a.H - whole, cut_at = whole > 0 ? (int)(items + 3) & ~3 : 0;  // and their pieces' place
    auto key_of = [&](const CrossPiece &q, int i) {  // (one query tile takes about two thirds of two)
        const int length = (q.g1 - q.g0) * (q.nrows > kCrTile ? 3 : 2);
        return (uint32_t)(0xFFFF - min(length, 0xFFFF)) << 16 | (uint32_t)i;
    };
    Four done{};  // pieces, cut items, their partial rows, their groups of rows
    for (int i0 = 0; i0 < items; i0 += kCpThreads) {
        const int i = i0 + tid;
        int n = 0, tiles = 0;
        CrossPiece p = {};
        if (i < items) {
            int lo = 0, hi = a.B - 1;  // the last run that starts at or before item i (empty runs share a start)
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (item_off[mid] <= i)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int4 s = seqs[lo];
            const int r0 = (i - item_off[lo]) * a.rows;
            p.nrows = min(a.rows, s.y - r0);
            p.q0 = s.x + r0;
            p.k0 = s.z;
            p.nk = s.w;
            p.see0 = s.w - s.y + r0 + 1;
            tiles = key_tiles(seen_by(r0 + p.nrows, s.y, s.w, a.causal));
            n = tiles > target ? (tiles + target - 1) / target : 1;
        }
        if (whole > 0 && i < items) {
            CrossPiece q = p;
            q.g1 = tiles;
            q.row0 = -1;
            pieces[i] = q;
            if (i < kCpSort) s_key[i] = key_of(q, i);
        }
        if (cut_heads == 0) continue;
        int at = i;  // (nothing cut: each item is a piece)
        int64_t row0 = -1;
        if (__syncthreads_or(n > 1) || done.v[1] > 0) {
            const int cut = n > 1;
            const Four mine{{n, cut, cut ? (int64_t)n * p.nrows : 0, cut ? (p.nrows + kCrGroup - 1) / kCrGroup : 0}};
            const Four x = block_scan<false, 4>(mine, &all, s_scan);
            at = (int)(done.v[0] + x.v[0] - n);
            if (cut) {
                row0 = done.v[2] + x.v[2] - mine.v[2];
                splits[done.v[1] + x.v[1] - 1] = CrossSplit{p.q0, p.nrows, (int32_t)row0, n,
                                                            (int32_t)(done.v[3] + x.v[3] - mine.v[3])};
            }
            done = both<false>(done, all);
        } else {
            done.v[0] += min((int64_t)kCpThreads, items - i0);
        }
        auto emit = [&](CrossPiece q, int at, int64_t row0, int tiles, int k, int n) {
            q.g0 = (int)((int64_t)tiles * k / n);
            q.g1 = (int)((int64_t)tiles * (k + 1) / n);
            q.row0 = n > 1 ? (int)(row0 + (int64_t)k * q.nrows) : -1;
            pieces[cut_at + at + k] = q;
            if (cut_at + at + k < kCpSort) s_key[cut_at + at + k] = key_of(q, at + k);
        };
        if (n <= kCpFew)
            for (int k = 0; k < n; ++k) emit(p, at, row0, tiles, k, n);
        // many pieces of an item by its whole warp
        for (unsigned cut = __ballot_sync(0xffffffffu, n > kCpFew); cut; cut &= cut - 1) {
            const int from = __ffs(cut) - 1;
            auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, from); };
            CrossPiece q = {};
            q.q0 = of(p.q0);
            q.nrows = of(p.nrows);
            q.k0 = of(p.k0);
            q.nk = of(p.nk);
            q.see0 = of(p.see0);
            const int qn = of(n), qat = of(at), qtiles = of(tiles);
            const int64_t qrow0 = of((int)row0);
            for (int k = tid & 31; k < qn; k += 32) emit(q, qat, qrow0, qtiles, k, qn);
        }
    }
    __syncthreads();

    // Longest first: a piece's place is the number of smaller keys (all different).  Short ones (of half the
    // longest at most), as many as the longest unit takes on every SM, come last, for all heads: they fill what the
    // others leave.
    const int np = (int)done.v[0];
    if (tid == 0) s_last = 0;
    auto sort = [&](int from, int n, int heads, bool last) {
        const int rounded = (n + 3) & ~3;
        if (from + rounded > kCpSort) {
            for (int i = tid; i < n; i += kCpThreads) order[from + i] = from + i;
            return;
        }
        if (tid < rounded - n) s_key[from + n + tid] = 0xFFFFFFFFu;
        __syncthreads();
        for (int i = tid; i < n; i += kCpThreads) {
            const uint32_t key = s_key[from + i];
            int place = 0;
            uint32_t least = key;
            int64_t behind = 0;  // the lengths of this piece and of those behind it
            for (int j = 0; j < rounded; j += 4) {
                const uint4 q = *reinterpret_cast<const uint4 *>(s_key + from + j);
                const uint32_t k4[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    place += k4[k] < key;
                    least = min(least, k4[k]);
                    behind += k4[k] >= key ? 0xFFFF - (int)(k4[k] >> 16) : 0;
                }
            }
            order[from + place] = from + i;
            const int longest = 0xFFFF - (int)(least >> 16);
            if (last && behind * heads <= (int64_t)longest * a.sms && 2 * (0xFFFF - (int)(key >> 16)) <= longest)
                atomicAdd(&s_last, 1);
        }
    };
    __syncthreads();
    if (whole > 0) sort(0, (int)items, whole, cut_heads == 0);
    if (cut_heads > 0) sort(cut_at, np, cut_heads, true);
    __syncthreads();
    if (tid == 0) {
        int *counters = reinterpret_cast<int *>(a.ws + kCrCounters);
        counters[0] = counters[1] = 0;
        CrossHeader h = {};
        h.magic = kCrossMagic;
        h.B = a.B;
        h.H = a.H;
        h.total_q = a.total_q;
        h.total_k = a.total_k;
        h.causal = a.causal;
        h.rows = a.rows;
        h.sms = a.sms;
        h.pieces = np;
        h.splits = (int32_t)done.v[1];
        h.groups = (int32_t)done.v[3];
        h.last = s_last;
        h.whole = whole;
        h.items = whole > 0 ? (int32_t)items : 0;
        *reinterpret_cast<CrossHeader *>(a.ws) = h;
        // The first plan in this memory sets its status word up; a later one keeps an error that nobody has read yet.
        const uint4 state = s_state;
        if (state.y != kCrossMarkY || state.z != kCrossMarkZ || state.w != kCrossMarkW)
            *status = make_uint4(fell ? MLA_ERR_INDEX : MLA_OK, kCrossMarkY, kCrossMarkZ, kCrossMarkW);
        else if (fell)
            record_error(reinterpret_cast<int *>(status), MLA_ERR_INDEX);
    }
}

// ------------------------------------------------------------------ the attention
constexpr uint32_t kCrBox = 64 * kCrTile * 2;  // 64 columns x 128 rows, bf16

template <int kTiles>
struct Shape {
    static constexpr int kWarpsSoft = 4 * kTiles;
    static constexpr int kThreads = 32 * (kWarpsSoft + 4);  // + loads, MMAs, tails, units
    static constexpr int kRing = 14 - 3 * kTiles;           // boxes of keys and values
    static constexpr uint32_t kOffRing = 3 * kCrBox * kTiles, kOffBar = 14 * kCrBox;
    static constexpr uint32_t kSmem = kOffBar + 512 + 1024;
};

struct CrossArgs {
    unsigned char *ws;
    size_t ws_bytes;
    int B, H, total_q, total_k, rows;
    float scale_log2;
    int positions;
    long long wait_cycles;  // limit of a wait that may last as long as a unit
    int stall;              // tests: the MMA warp first waits for a barrier that nothing completes
    const float *before_out, *before_lse;
    float *out;       // one of the two
    uint16_t *out16;
    float *lse;       // or null
};

// The result's row: the new part (o, of sum e^{lse}) joined with an earlier one.
struct Share {
    float mine, before, lse;
};
__device__ __forceinline__ Share share_of(float lse, bool joined, float b) {
    Share s{1.f, 0.f, lse};
    if (joined) {
        const float m = fmaxf(lse, b);
        if (m == -INFINITY) return s;
        const float e0 = expf(b - m), e1 = expf(lse - m), sum = e0 + e1;
        s.mine = e1 / sum;
        s.before = e0 / sum;
        s.lse = m + logf(sum);
    }
    return s;
}
// 32 bytes at once (both directions; a row's thread then touches each sector once).
__device__ __forceinline__ void ld_global8(const float *p, float (&v)[8]) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void st_global8(void *p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// 32 values of the result's row from element `at` on.
__device__ __forceinline__ void store32(const CrossArgs &a, int64_t at, const float (&y)[32]) {
    if (a.out) {
#pragma unroll
        for (int c = 0; c < 32; c += 8) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(y[c + i]);
            st_global8(a.out + at + c, w);
        }
    } else {
#pragma unroll
        for (int c = 0; c < 32; c += 16) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = bf16x2_bits(y[c + 2 * i], y[c + 2 * i + 1]);
            st_global8(a.out16 + at + c, w);
        }
    }
}
// Four values, scaled already, and the earlier part's share.
__device__ __forceinline__ void store4(const CrossArgs &a, int64_t at, float4 o, float before) {
    if (before != 0.f) {
        const float4 b = *reinterpret_cast<const float4 *>(a.before_out + at);
        o = make_float4(fmaf(b.x, before, o.x), fmaf(b.y, before, o.y), fmaf(b.z, before, o.z), fmaf(b.w, before, o.w));
    }
    if (a.out)
        *reinterpret_cast<float4 *>(a.out + at) = o;
    else
        *reinterpret_cast<uint2 *>(a.out16 + at) = make_uint2(bf16x2_bits(o.x, o.y), bf16x2_bits(o.z, o.w));
}

// True when the workspace holds a plan made for this call.
__device__ __forceinline__ bool plan_fits(const CrossArgs &a, const CrossHeader *hd) {
    return hd->magic == kCrossMagic && hd->B == a.B && hd->H == a.H && hd->total_q == a.total_q &&
           hd->total_k == a.total_k && hd->rows == a.rows && hd->sms > 0 &&
           cross_layout(a.B, a.H, a.total_q, hd->sms).total <= a.ws_bytes;
}

// kJoined: with an earlier part's result.  (A kernel of its own: in one kernel for both, calls without an earlier part
// took 4 - 6 % longer where units are short; 8 x 3,384 queries x 38 keys x 32 heads take 161 us.)
template <int kTiles, bool kJoined>
__global__ void __launch_bounds__(Shape<kTiles>::kThreads, 1)
    cross_kernel(const __grid_constant__ CUtensorMap tm_qn, const __grid_constant__ CUtensorMap tm_qr,
                 const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_kr,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CrossArgs a) {
    using S = Shape<kTiles>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char *gbase = smem_raw + (base - raw);
    const uint32_t bars = base + S::kOffBar;
    // barriers: the ring's items (keys and values of a tile in turn, eight barriers each): full, empty, and
    // landed for the values of a run's last tile; per use of a score buffer s_full, p_full (one arrival per
    // softmax warp) and pv_done; per query tile o_free; per unit slot u_full, u_empty; the queries: q_full,
    // q_empty.  A score buffer has one set of barriers for two query tiles (0, 1) and another for one query
    // tile that uses both (2, 3): the second tile's warps take no part in such units, run ahead of them, and
    // would find a common barrier two phases back.  For the same reason pv_done is one per buffer: where one
    // query tile uses both, its scores say nothing about the PV before the last one.
    auto full = [&](int i) { return bars + 8u * (i & 7); };
    auto empty = [&](int i) { return bars + 64u + 8u * (i & 7); };
    auto landed = [&](int i) { return bars + 128u + 8u * (i & 3); };
    auto s_full = [&](int i) { return bars + 160u + 8u * i; };
    auto p_full = [&](int i) { return bars + 192u + 8u * i; };
    auto pv_done = [&](int i) { return bars + 224u + 8u * i; };
    auto o_free = [&](int x) { return bars + 256u + 8u * x; };
    auto u_full = [&](int j) { return bars + 272u + 8u * j; };
    auto u_empty = [&](int j) { return bars + 288u + 8u * j; };
    const uint32_t q_full = bars + 304, q_empty = bars + 312, never = bars + 432;
    CrossPiece *slots = reinterpret_cast<CrossPiece *>(gbase + S::kOffBar + 320);  // two of 48 bytes
    int *abort_flag = reinterpret_cast<int *>(gbase + S::kOffBar + 416);
    volatile uint32_t *tslot = reinterpret_cast<volatile uint32_t *>(gbase + S::kOffBar + 424);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 0) {
        if (lane == 0) {
            for (int i = 0; i < 8; ++i) {
                mbar_init(full(i), 1);
                mbar_init(empty(i), 1);
            }
            for (int i = 0; i < 4; ++i) {
                mbar_init(landed(i), 1);
                mbar_init(s_full(i), 1);
                mbar_init(p_full(i), 4);
                mbar_init(pv_done(i), 1);
            }
            for (int j = 0; j < 2; ++j) {
                mbar_init(o_free(j), 4);
                mbar_init(u_full(j), 1);
                mbar_init(u_empty(j), 3 + S::kWarpsSoft);
            }
            mbar_init(q_full, 1);
            mbar_init(q_empty, 1);
            mbar_init(never, 1);
            *abort_flag = 0;
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(smem_u32(const_cast<uint32_t *>(tslot)), 512);
        tmem_relinquish();
    }
    grid_dep_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    int *status = reinterpret_cast<int *>(a.ws + kCrStatus);
    int *counters = reinterpret_cast<int *>(a.ws + kCrCounters);
    CrossHeader *hd = reinterpret_cast<CrossHeader *>(a.ws);
    const bool match = plan_fits(a, hd);
    if (!match && threadIdx.x == 0) record_error(status, MLA_ERR_WORKSPACE);
    const int step = hd->causal ? 1 : 0;
    bool ok = true;
    // For the next unit, a slot for it, a unit's last values, and as the second of two query tiles, which has no rows in some
    // units, for its first scores, a role may wait as long as a unit takes.  (All waits with a limit that is no constant:
    // 1 % of short units.)
    auto wait = [&](uint32_t bar, uint32_t parity) { return wait_bounded(bar, parity, abort_flag); };
    auto wait_long = [&](uint32_t bar, uint32_t parity) { return wait_bounded(bar, parity, abort_flag, a.wait_cycles); };

    // The next unit's piece, from its slot (the whole warp); false: there is none, or a wait ran out.
    int taken = 0;
    CrossPiece p;
    auto next_unit = [&]() -> bool {
        if (!ok) return false;
        const int j = taken & 1;
        ok = __all_sync(0xffffffffu, wait_long(u_full(j), (taken >> 1) & 1));
        if (!ok) return false;
        p = slots[j];
        __syncwarp();
        if (lane == 0) mbar_arrive(u_empty(j));
        ++taken;
        return p.head >= 0;
    };
    // Keys that row r of the item sees, and key tiles of query tile x within the piece.
    auto seen = [&](int r) { return step ? min(p.nk, p.see0 + r) : p.nk; };
    auto tiles_of = [&](int x) -> int {
        const int rows = min(p.nrows - x * kCrTile, kCrTile);
        if (rows <= 0) return 0;
        const int keys = max(seen(x * kCrTile + rows - 1), 0);
        return max(min(p.g1, (keys + kCrTile - 1) / kCrTile) - p.g0, 0);
    };
    // (of two query tiles the second sees as many keys as the first, or more, where it has rows)
    auto tiles_loaded = [&]() -> int { return kTiles == 2 ? max(tiles_of(0), tiles_of(1)) : tiles_of(0); };
    // One query tile takes both score buffers in turn, so that the next scores are computed under its
    // softmax; two have one each.  use0 .. use3: how often each set of barriers has been used before the unit,
    // which says which phase is next, in every role that takes part.
    auto single = [&]() { return kTiles == 1 || p.nrows <= kCrTile; };
    int use0 = 0, use1 = 0, use2 = 0, use3 = 0;
    auto used = [&](int n0, int n1) {
        if (single()) {
            use2 += (n0 + 1) / 2;
            use3 += n0 / 2;
        } else {
            use0 += n0;
            use1 += n1;
        }
    };
    // The ring: key tile t (counted over the units) has `kw` boxes of 128 keys x 64 columns, and its values,
    // behind them, two of 64 keys x 128 columns (two column halves of 8 KB).
    const int kw = a.positions ? 3 : 2;
    auto box = [&](int t, int i) { return base + S::kOffRing + (uint32_t)((t * (kw + 2) + i) % S::kRing) * kCrBox; };
    const int w = warp - S::kWarpsSoft;

    if (!match) {
        // nothing to do
    } else if (w == 3) {
        // ---------------------------------------------------------------- units
        if (lane == 0) {
            const CrossLayout L = cross_layout(a.B, a.H, a.total_q, hd->sms);
            const CrossPiece *pieces = reinterpret_cast<const CrossPiece *>(a.ws + L.pieces);
            const int32_t *order = reinterpret_cast<const int32_t *>(a.ws + L.order);
            // whole items of the first heads, then the other heads' pieces; the last list's last ones for all its heads
            const int first = hd->items * hd->whole, cut_heads = a.H - hd->whole;
            const int total = first + hd->pieces * cut_heads;
            for (int i = 0; ok; ++i) {
                const int j = i & 1;
                if (i >= 2) ok = wait_long(u_empty(j), ((i >> 1) - 1) & 1);
                if (!ok) break;
                // (a CTA beyond the SMs that the plan is for takes none)
                const int u = (int)blockIdx.x < hd->sms ? atomicAdd(&counters[0], 1) : total;
                CrossPiece d;
                d.head = -1;
                if (u < total) {
                    const bool cut = u >= first;
                    int r = cut ? u - first : u;
                    const int from = cut && hd->whole > 0 ? (hd->items + 3) & ~3 : 0, heads = cut ? cut_heads : hd->whole;
                    const int n = (cut ? hd->pieces : hd->items) - (cut || cut_heads == 0 ? hd->last : 0);
                    int head;
                    if (r < n * heads) {
                        // a group of heads: each piece for all of them, in the pieces' order
                        const int h0 = r / (kCrHeadGroup * n) * kCrHeadGroup, hg = min(kCrHeadGroup, heads - h0);
                        r -= h0 * n;
                        d = pieces[order[from + r / hg]];
                        head = h0 + r % hg;
                    } else {
                        r -= n * heads;
                        d = pieces[order[from + n + r / heads]];
                        head = r % heads;
                    }
                    d.head = (cut ? hd->whole : 0) + head;
                }
                slots[j] = d;
                mbar_arrive(u_full(j));
                if (d.head < 0) break;
            }
        }
    } else if (w == 0) {
        // ---------------------------------------------------------------- loads
        // Keys and values go round the ring in the order of their first use; an item's boxes are free again
        // once the MMAs that read it have finished.
        int units = 0, t = 0, tails = 0;
        int freed = 0, freed_boxes = 0;  // items, and boxes up to them, that have been waited for
        auto room = [&](int boxes) -> bool {  // for the boxes up to this number
            while (ok && boxes - freed_boxes > S::kRing) {
                ok = wait(empty(freed), (freed >> 3) & 1);
                freed_boxes += freed & 1 ? 2 : kw;
                ++freed;
            }
            return ok;
        };
        while (next_unit()) {
            const int ntot = tiles_loaded();
            if (ntot == 0) continue;
            if (lane == 0) {
                const int nx = single() ? 1 : 2;
                if (units > 0) ok = wait(q_empty, (units - 1) & 1);
                if (ok) {
                    mbar_arrive_expect_tx(q_full, nx * kw * kCrBox);
                    for (int x = 0; x < nx; ++x) {
                        const uint32_t qd = base + 3 * kCrBox * x;
                        const int q0 = p.q0 + x * kCrTile;
                        tma_load_3d(qd, &tm_qn, 0, p.head, q0, q_full);
                        tma_load_3d(qd + kCrBox, &tm_qn, 64, p.head, q0, q_full);
                        if (a.positions) tma_load_3d(qd + 2 * kCrBox, &tm_qr, 0, p.head, q0, q_full);
                    }
                }
                for (int g = 0; g < ntot && ok; ++g, ++t) {
                    const int t0 = (p.g0 + g) * kCrTile, k0 = p.k0 + t0;
                    if (kTiles == 2 && g + kCrAhead < ntot) {  // on its way into L2
                        const int ka = k0 + kCrAhead * kCrTile;
                        tma_prefetch_3d(&tm_k, 0, ka, p.head);
                        tma_prefetch_3d(&tm_k, 64, ka, p.head);
                        if (a.positions) tma_prefetch_2d(&tm_kr, kDLatent, ka);
                        for (int i = 0; i < 2; ++i) {
                            tma_prefetch_3d(&tm_v, 0, ka + 64 * i, p.head);
                            tma_prefetch_3d(&tm_v, 64, ka + 64 * i, p.head);
                        }
                    }
                    if (!room(t * (kw + 2) + kw)) break;
                    mbar_arrive_expect_tx(full(2 * t), kw * kCrBox);
                    tma_load_3d(box(t, 0), &tm_k, 0, k0, p.head, full(2 * t));
                    tma_load_3d(box(t, 1), &tm_k, 64, k0, p.head, full(2 * t));
                    if (a.positions) tma_load_2d(box(t, 2), &tm_kr, kDLatent, k0, full(2 * t));
                    if (!room((t + 1) * (kw + 2))) break;
                    const uint32_t bar = p.nk - t0 < kCrTile ? landed(tails++) : full(2 * t + 1);
                    mbar_arrive_expect_tx(bar, 2 * kCrBox);
                    for (int i = 0; i < 2; ++i) {
                        tma_load_3d(box(t, kw + i), &tm_v, 0, k0 + 64 * i, p.head, bar);
                        tma_load_3d(box(t, kw + i) + kCrBox / 2, &tm_v, 64, k0 + 64 * i, p.head, bar);
                    }
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            ++units;
        }
    } else if (w == 2) {
        // ---------------------------------------------------------------- tails
        // What lies behind a run's last key is another run's, or anything: its weights are 0, but 0 x NaN is
        // not, so those values are zeroed before PV reads them.
        int t = 0, tails = 0;
        while (next_unit()) {
            const int ntot = tiles_loaded();
            t += ntot;
            const int valid = p.nk - (p.g0 + ntot - 1) * kCrTile;  // keys of the last tile
            if (ntot == 0 || valid >= kCrTile) continue;
            ok = __all_sync(0xffffffffu, wait_long(landed(tails), (tails >> 2) & 1));
            if (!ok) break;
            ++tails;
            for (int i = 0; i < 2; ++i) {
                const int from = min(max(valid - 64 * i, 0), 64), chunks = (64 - from) * 8;  // of 16 bytes
                uint4 *rows = reinterpret_cast<uint4 *>(gbase + (box(t - 1, kw + i) - base) + from * 128);
                for (int c = lane; c < chunks; c += 32) {
                    rows[c] = make_uint4(0u, 0u, 0u, 0u);
                    rows[kCrBox / 32 + c] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full(2 * t - 1));
        }
    } else if (w == 1) {
        // ---------------------------------------------------------------- MMAs
        // the whole warp runs the issue loop (its waits made warp-uniform); one elected lane issues
        auto wait_w = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, wait_quick(bar, parity, abort_flag));
        };
        constexpr uint32_t idesc_s = idesc_bf16_major(128, kCrTile, false, false);
        constexpr uint32_t idesc_o = idesc_bf16_major(128, kCrDh, false, true);
        // descriptors but for their addresses: keys and queries (K-major), values (MN-major)
        const uint64_t desc_k = smem_desc_sw128(0, 16u, 1024u), desc_v = smem_desc_sw128(0, kCrBox / 2, 1024u);
        int units = 0, t = 0, ou[2] = {0, 0};  // units with keys, their key tiles, units of each query tile
        if (a.stall) ok = __all_sync(0xffffffffu, wait_long(never, 0));
        while (next_unit()) {
            const int n0 = tiles_of(0), n1 = kTiles == 2 ? tiles_of(1) : 0, ntot = max(n0, n1);
            if (ntot == 0) continue;
            // Waits for the keys, or the values, of key tile g (once: for the first query tile that reads them).
            auto landed_k = [&](int x, int g) {
                return (x == 1 && g < n0) || wait_w(full(2 * (t + g)), (2 * (t + g) >> 3) & 1);
            };
            auto landed_v = [&](int x, int g) {
                return (x == 1 && g < n0) || wait_w(full(2 * (t + g) + 1), (2 * (t + g) >> 3) & 1);
            };
            // Scores of query tile x with key tile g into buffer j (barriers i); the keys' boxes go back after the
            // last query tile that reads them, the queries after the unit's last scores.
            auto qk = [&](int x, int j, int i, int g) -> bool {
                if (!landed_k(x, g)) return false;
                tc_fence_after();
                for (int c = 0; c < kw; ++c) {
                    const uint64_t kd = desc_k + (box(t + g, c) >> 4), qd = desc_k + ((base + (3 * x + c) * kCrBox) >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ss_warp(tmem + 256u * j, qd + 2u * k, kd + 2u * k, idesc_s, c + k > 0 ? 1u : 0u);
                }
                mma_commit_warp(s_full(i));
                if (x == (g < n1 ? 1 : 0)) {
                    mma_commit_warp(empty(2 * (t + g)));
                    if (g == ntot - 1) mma_commit_warp(q_empty);
                }
                return true;
            };
            // O_x += P(g) V(g), P in buffer j (use u of barriers i); the values' boxes go back after the last query
            // tile's.
            auto pv = [&](int x, int j, int i, int u, int g) -> bool {
                if (g == 0 && ou[x] > 0 && !wait_w(o_free(x), (ou[x] - 1) & 1)) return false;
                if (!landed_v(x, g) || !wait_w(p_full(i), u & 1)) return false;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint64_t vd = desc_v + (box(t + g, kw + c) >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ts_warp(tmem + 256u * x + 128u, tmem + 256u * j + 32u * c + 8u * k, vd + 128u * k, idesc_o,
                                    g + c + k > 0 ? 1u : 0u);
                }
                mma_commit_warp(pv_done(i));
                if (x == (g < n1 ? 1 : 0)) mma_commit_warp(empty(2 * (t + g) + 1));
                return true;
            };
            ok = wait_w(q_full, units & 1);
            if (single()) {
                ok = ok && qk(0, 0, 2, 0);
                for (int g = 0; g < ntot && ok; ++g) {
                    const int j = g & 1;
                    ok = (g + 1 >= ntot || qk(0, j ^ 1, 2 + (j ^ 1), g + 1)) &&
                         pv(0, j, 2 + j, (j ? use3 : use2) + (g >> 1), g);
                }
            } else {
                ok = ok && (n0 == 0 || qk(0, 0, 0, 0)) && (n1 == 0 || qk(1, 1, 1, 0));
                for (int g = 0; g < ntot && ok; ++g) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int n = x ? n1 : n0;
                        if (ok && g < n) ok = pv(x, x, x, (x ? use1 : use0) + g, g) && (g + 1 >= n || qk(x, x, x, g + 1));
                    }
                }
            }
            if (!ok) break;
            used(n0, n1);
            if (n0 > 0) ++ou[0];
            if (n1 > 0) ++ou[1];
            ++units;
            t += ntot;
        }
    } else {
        // ---------------------------------------------------------------- softmax
        // warps 4x .. 4x + 3: query tile x, rows 32 (w % 4) .. (its TMEM lanes), one thread per row
        const CrossLayout L = cross_layout(a.B, a.H, a.total_q, hd->sms);
        float *part_lse = reinterpret_cast<float *>(a.ws + L.part_lse);
        float *part_o = reinterpret_cast<float *>(a.ws + L.part_o);
        const int x = warp >> 2, quad = warp & 3;
        const int r = x * kCrTile + 32 * quad + lane;  // the item's row
        const uint32_t lane_base = (uint32_t)(32 * quad) << 16;
        const uint32_t cO = tmem + lane_base + 256u * x + 128u;
        // the score buffer of the unit's key tile g, its barriers, and which use of them that is
        auto buffer = [&](int g) { return single() ? g & 1 : x; };
        auto barriers = [&](int g) { return single() ? 2 + (g & 1) : x; };
        auto use_of = [&](int g) { return single() ? (g & 1 ? use3 : use2) + (g >> 1) : (x ? use1 : use0) + g; };
        auto wait_pv = [&](int g) { return wait(pv_done(barriers(g)), use_of(g) & 1); };
        while (next_unit()) {
            const int nt = tiles_of(x);
            // (rows past the item's compute something nobody reads)
            const int see = r < p.nrows ? seen(r) : p.nk;
            float m = -INFINITY, l = 0.f;  // reference maximum (log2 units), running sum
            const bool whole = p.row0 < 0, mine = r < p.nrows;
            const int64_t row = (int64_t)(p.q0 + r) * a.H + p.head;
            const float before = kJoined && whole && mine ? a.before_lse[row] : -INFINITY;
            for (int g = 0; g < nt; ++g) {
                ok = kTiles == 2 ? wait_long(s_full(barriers(g)), use_of(g) & 1) : wait(s_full(barriers(g)), use_of(g) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t cS = tmem + lane_base + 256u * buffer(g);
                float s[kCrTile];
                {
                    uint32_t v[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(cS + 32u * c, v[c]);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < kCrTile; ++c) s[c] = __uint_as_float(v[c / 32][c % 32]);
                }
                const int lim = see - (p.g0 + g) * kCrTile;  // columns c < lim are seen
                if (__any_sync(0xffffffffu, lim < kCrTile)) {
#pragma unroll
                    for (int c = 0; c < kCrTile; ++c) s[c] = c < lim ? s[c] : -INFINITY;
                }
                float mxs[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int c = 4; c + 8 <= kCrTile; c += 8) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) mxs[k] = max3(mxs[k], s[c + k], s[c + 4 + k]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) mxs[k] = fmaxf(mxs[k], s[kCrTile - 4 + k]);
                const float mx = fmaxf(m, a.scale_log2 * max3(mxs[0], mxs[1], fmaxf(mxs[2], mxs[3])));
                // the reference moves only when exceeded by 2^8 (probabilities stay <= 2^8), so most tiles leave
                // O alone; a row that has seen no key yet keeps -inf, probabilities of 0 and an O of 0
                const float mref = (m == -INFINITY || mx > m + kCrRescale) ? mx : m;
                const float alpha = m == -INFINITY ? 1.f : ex2_approx(m - mref);
                const float sub = mref == -INFINITY ? 0.f : -mref;
                const uint64_t c2 = pair(a.scale_log2, a.scale_log2), sub2 = pair(sub, sub);
                uint64_t sums[4] = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t pk[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float2 y = halves(fma2(pair(s[64 * c + 2 * i], s[64 * c + 2 * i + 1]), c2, sub2));
                        const float p0 = ex2_approx(y.x), p1 = ex2_approx(y.y);
                        sums[i & 3] = add2(sums[i & 3], pair(p0, p1));
                        pk[i] = bf16x2_bits(p0, p1);
                    }
                    tmem_st32(cS + 32u * c, pk);
                }
                const float2 sum = halves(add2(add2(sums[0], sums[1]), add2(sums[2], sums[3])));
                l = l * alpha + (sum.x + sum.y);
                m = mref;
                // O is rescaled (rarely) once the previous PV has finished; the next waits for this P
                if (g > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                    ok = wait_pv(g - 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < kCrDh / 32; ++c) {
                        uint32_t v[32];
                        tmem_ld32(cO + 32u * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
                        tmem_st32(cO + 32u * c, v);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(barriers(g)));
            }
            if (!ok) break;
            // the row's result, 32 columns at a time, normalised: the whole of it, or a piece's part
            const float lse2 = l == 0.f ? -INFINITY : m + log2f(l), inv = l == 0.f ? 0.f : 1.f / l;
            const int64_t part = whole ? 0 : part_at(p.row0, p.nrows, a.H - hd->whole, p.head - hd->whole);
            Share sh{1.f, 0.f, 0.f};
            if (whole && mine) sh = share_of(lse2 * kLn2, kJoined, before);
            auto finished = [&]() -> bool {  // the unit's last PV
                if (nt == 0) return true;
                ok = __all_sync(0xffffffffu, wait_pv(nt - 1));
                tc_fence_after();
                return ok;
            };
            auto output = [&](int c, uint32_t (&o)[32]) {
                if (nt > 0) {
                    tmem_ld32(cO + c, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0u;
                }
            };
            if (kJoined && kTiles == 1 && whole) {
                // the earlier part's row is on its way while PV finishes (what has no weight may hold anything; 8 x 1,750
                // queries x 13 keys x 64 heads 374 -> 318 us in fp32 without positions; in bf16 272, with positions 277)
                float e[kCrDh];
#pragma unroll
                for (int i = 0; i < kCrDh; ++i) e[i] = 0.f;
                if (sh.before != 0.f) {
#pragma unroll
                    for (int i = 0; i < kCrDh; i += 8)
                        ld_global8(a.before_out + row * kCrDh + i, *reinterpret_cast<float(*)[8]>(e + i));
                }
                if (finished()) {
#pragma unroll
                    for (int c = 0; c < kCrDh; c += 32) {
                        uint32_t o[32];
                        output(c, o);
                        float y[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            y[i] = fmaf(e[c + i], sh.before, __uint_as_float(o[i]) * (inv * sh.mine));
                        if (mine) store32(a, row * kCrDh + c, y);
                    }
                }
            } else if (finished()) {
#pragma unroll 1
                for (int c = 0; c < kCrDh; c += 32) {
                    uint32_t o[32];
                    output(c, o);
                    if (!mine) continue;
                    if (whole) {
                        float y[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(o[i]) * (inv * sh.mine);
                        if (kJoined && sh.before != 0.f) {  // (their registers leave no room for the whole row)
#pragma unroll
                            for (int k = 0; k < 32; k += 8) {
                                float e[8];
                                ld_global8(a.before_out + row * kCrDh + c + k, e);
#pragma unroll
                                for (int i = 0; i < 8; ++i) y[k + i] = fmaf(e[i], sh.before, y[k + i]);
                            }
                        }
                        store32(a, row * kCrDh + c, y);
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>(part_o + part * kCrDh) + r;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            dst[(c / 4 + k) * p.nrows] =
                                make_float4(__uint_as_float(o[4 * k]) * inv, __uint_as_float(o[4 * k + 1]) * inv,
                                            __uint_as_float(o[4 * k + 2]) * inv, __uint_as_float(o[4 * k + 3]) * inv);
                    }
                }
            }
            if (!ok) break;
            if (nt > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_free(x));
            }
            if (mine && whole && a.lse) a.lse[row] = sh.lse;
            if (mine && !whole) part_lse[part + r] = lse2;
            used(nt, nt);
        }
    }
    grid_dep_launch();
    if (!__syncthreads_and(ok ? 1 : 0)) {
        if (threadIdx.x == 0) {
            record_error(status, MLA_ERR_TIMEOUT);
            hd->magic = 0;  // units are where they were left: the plan has to be made again
        }
        drain_pause();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    // the last CTA to leave sets the unit counter back for the plan's next call
    if (match && threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(&counters[1], 1) == (int)gridDim.x - 1) counters[0] = counters[1] = 0;
    }
}

// The items that were cut: a CTA joins the parts of up to 32 rows of one head, in the parts' order.  Lane i
// of warp w has row i and columns 4 w .. 4 w + 3, 32 + 4 w .. and so on; the rows are then written a warp each.
constexpr int kCmThreads = 256;
// (two at once, the rest even out what the rows differ by; six cost calls without cut items 0.7 us more)
constexpr int kCmCtasPerSm = 4;
constexpr int kCmParts = 4;  // in flight together
__global__ void __launch_bounds__(kCmThreads, 2) cross_merge_kernel(const __grid_constant__ CrossArgs a) {
    __shared__ __align__(16) float s_o[kCrGroup][kCrDh + 4];
    __shared__ float s_before[kCrGroup];
    grid_dep_wait();
    grid_dep_launch();
    const CrossHeader *hd = reinterpret_cast<const CrossHeader *>(a.ws);
    if (!plan_fits(a, hd) || hd->splits == 0) return;
    const CrossLayout L = cross_layout(a.B, a.H, a.total_q, hd->sms);
    const CrossSplit *splits = reinterpret_cast<const CrossSplit *>(a.ws + L.splits);
    const float *part_lse = reinterpret_cast<const float *>(a.ws + L.part_lse);
    const float *part_o = reinterpret_cast<const float *>(a.ws + L.part_o);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_splits = hd->splits;
    const int heads = a.H - hd->whole;
    const int64_t tasks = (int64_t)hd->groups * heads;
    for (int64_t t = blockIdx.x; t < tasks; t += gridDim.x) {
        const int at = (int)(t / heads), h = (int)(t - (int64_t)at * heads);  // (of the heads with cut items)
        int lo = -1;  // the last cut item that starts at or before group `at`, 32 of them looked at together
        for (int i = lane; i - lane < n_splits; i += 32)
            lo += __popc(__ballot_sync(0xffffffffu, i < n_splits && splits[i].before <= at));
        const CrossSplit s = splits[lo];
        const int r0 = (at - s.before) * kCrGroup, rows = min(kCrGroup, s.nrows - r0);
        const int64_t first = part_at(s.row0, s.nrows, heads, h) + r0 + lane, pitch = (int64_t)s.nrows * heads;
        const int64_t row = (int64_t)(s.q0 + r0 + lane) * a.H + hd->whole + h;
        const bool mine = lane < rows;
        const float before = mine && a.before_lse ? a.before_lse[row] : -INFINITY;
        float top = -INFINITY, sum = 0.f;
        float4 acc[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = 0; k0 < s.parts; k0 += kCmParts) {
            float l[kCmParts];
            float4 v[kCmParts][4];
#pragma unroll
            for (int k = 0; k < kCmParts; ++k) {
                const bool is = mine && k0 + k < s.parts;
                const int64_t from = first + (k0 + k) * pitch;  // (of the log-sum-exps)
                l[k] = is ? part_lse[from] : -INFINITY;
                const float4 *o = reinterpret_cast<const float4 *>(part_o + (from - r0 - lane) * kCrDh) + r0 + lane;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    v[k][c] = is ? o[(8 * c + warp) * s.nrows] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float m = top;
#pragma unroll
            for (int k = 0; k < kCmParts; ++k) m = fmaxf(m, l[k]);
            if (m == -INFINITY) continue;  // no key seen so far
            const float f = ex2_approx(top - m);
            sum *= f;
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[c] = make_float4(acc[c].x * f, acc[c].y * f, acc[c].z * f, acc[c].w * f);
#pragma unroll
            for (int k = 0; k < kCmParts; ++k) {
                const float w = ex2_approx(l[k] - m);
                sum += w;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    acc[c] = make_float4(fmaf(w, v[k][c].x, acc[c].x), fmaf(w, v[k][c].y, acc[c].y),
                                         fmaf(w, v[k][c].z, acc[c].z), fmaf(w, v[k][c].w, acc[c].w));
            }
            top = m;
        }
        Share sh{0.f, 0.f, 0.f};
        if (mine) sh = share_of(sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2, a.before_lse != nullptr, before);
        const float f = sum == 0.f ? 0.f : sh.mine / sum;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            *reinterpret_cast<float4 *>(&s_o[lane][4 * (8 * c + warp)]) =
                make_float4(acc[c].x * f, acc[c].y * f, acc[c].z * f, acc[c].w * f);
        if (warp == 0) s_before[lane] = sh.before;
        __syncthreads();  // (and every warp has read before_lse, which may be lse itself)
        if (warp == 0 && mine && a.lse) a.lse[row] = sh.lse;
        for (int i = warp; i < rows; i += kCmThreads / 32)
            store4(a, (row + (int64_t)(i - lane) * a.H) * kCrDh + 4 * lane,
                   *reinterpret_cast<const float4 *>(&s_o[i][4 * lane]), s_before[i]);
        __syncthreads();
    }
}

bool tmap_bf16(CUtensorMap *m, const void *p, int rank, const uint64_t *d, const uint64_t *s, const uint32_t *b) {
    return tmap_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, rank, d, s, b);
}

template <typename K>
bool grant(K kernel, uint32_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
}
// SMs of the current device (0: none), its cross kernels' shared memory granted.
int cross_device() {
    static int sms[64] = {};
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (sms[dev] > 0) return sms[dev];
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        !grant(cross_kernel<1, false>, Shape<1>::kSmem) || !grant(cross_kernel<1, true>, Shape<1>::kSmem) ||
        !grant(cross_kernel<2, false>, Shape<2>::kSmem) || !grant(cross_kernel<2, true>, Shape<2>::kSmem)) {
        cudaGetLastError();
        return 0;
    }
    sms[dev] = n;
    return n;
}

int device_sms() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

// Units and partial rows fit 32 bits.
bool cross_shape_ok(int B, int H, int64_t total_q) {
    return B <= (1 << 20) && H <= kMaxHeads && total_q <= (1 << 24);
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" size_t mla_cross_workspace_size(int B, int H, int64_t total_q, int num_sms) {
    if (B < 1 || H < 1 || total_q < 0 || num_sms < 0 || num_sms > 4096 || !cross_shape_ok(B, H, total_q)) return 0;
    if (num_sms == 0) num_sms = device_sms();
    if (num_sms <= 0) return 0;
    return cross_layout(B, H, total_q, num_sms).total;
}

extern "C" mla_status mla_cross_plan(const int32_t *cu_q, const int32_t *cu_k, int B, int H, int64_t total_q,
                                     int64_t total_k, int causal, int num_sms, void *workspace, size_t ws_bytes,
                                     void *stream) {
    if (!workspace || !cu_q || !cu_k || B < 1 || H < 1 || total_q < 0 || total_k < 0 || num_sms < 0 || num_sms > 4096)
        return MLA_ERR_INVALID_ARG;
    if (!aligned16(workspace)) return MLA_ERR_INVALID_ARG;
    if (!cross_shape_ok(B, H, total_q) || total_k > INT32_MAX - kCrTile) return MLA_ERR_UNSUPPORTED;
    if (num_sms == 0) num_sms = device_sms();
    if (num_sms <= 0) return MLA_ERR_CUDA;
    CrossPlanArgs a;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.B = B;
    a.H = H;
    a.total_q = (int)total_q;
    a.total_k = (int)total_k;
    a.causal = causal ? 1 : 0;
    a.rows = cross_rows(B, H, total_q, total_k);
    a.sms = num_sms;
    a.ws = (unsigned char *)workspace;
    a.L = cross_layout(B, H, total_q, num_sms);
    if (ws_bytes < a.L.total) return MLA_ERR_WORKSPACE;
    return launch_pdl(cross_plan_kernel, 1, kCpThreads, 0, (cudaStream_t)stream, a) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

extern "C" mla_status mla_cross_attention(void *workspace, size_t ws_bytes, const void *q_nope, const void *q_rope,
                                          const void *entries, const void *k_nope, const void *v, int B, int H,
                                          int64_t total_q, int64_t total_k, float softmax_scale, const float *before_out,
                                          const float *before_lse, void *out, mla_out_dtype out_dtype, float *lse,
                                          void *stream) {
    if (!workspace || B < 1 || H < 1 || total_q < 0 || total_k < 0) return MLA_ERR_INVALID_ARG;
    if (out_dtype != MLA_OUT_FP32 && out_dtype != MLA_OUT_BF16) return MLA_ERR_INVALID_ARG;
    if (!(softmax_scale > 0.f) || softmax_scale == INFINITY) return MLA_ERR_INVALID_ARG;
    if ((q_rope == nullptr) != (entries == nullptr) && total_q > 0 && total_k > 0) return MLA_ERR_INVALID_ARG;
    if ((before_out == nullptr) != (before_lse == nullptr)) return MLA_ERR_INVALID_ARG;
    if (!aligned16(workspace) || !aligned16(q_nope) || !aligned16(q_rope) || !aligned16(entries) || !aligned16(k_nope) ||
        !aligned16(v) ||
        (reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(before_out)) % 32 != 0)
        return MLA_ERR_INVALID_ARG;
    if (!cross_shape_ok(B, H, total_q) || total_k > INT32_MAX - kCrTile) return MLA_ERR_UNSUPPORTED;
    if (total_q == 0) return MLA_OK;
    if (!q_nope || !out || (total_k > 0 && (!k_nope || !v))) return MLA_ERR_INVALID_ARG;
    if (ws_bytes < cross_layout(B, H, total_q, 1).total) return MLA_ERR_WORKSPACE;
    const int sms = cross_device();
    if (sms <= 0) return MLA_ERR_CUDA;
    // (without any key the maps stand for something that is never read)
    const uint64_t nk = total_k > 0 ? (uint64_t)total_k : 1;
    if (total_k == 0) k_nope = v = entries = q_rope = nullptr;
    if (!k_nope) k_nope = v = q_nope;
    const bool positions = q_rope != nullptr;
    CUtensorMap tqn, tqr, tk, tkr, tv;
    // q nope [total_q][H][128], q rope [total_q][H][64]: (cols, h, query); boxes of 64 columns x 128 queries
    const uint64_t dqn[3] = {kCrDh, (uint64_t)H, (uint64_t)total_q}, sqn[2] = {kCrDh * 2, (uint64_t)kCrDh * 2 * H};
    const uint64_t dqr[3] = {kDRope, (uint64_t)H, (uint64_t)total_q}, sqr[2] = {kDRope * 2, (uint64_t)kDRope * 2 * H};
    const uint32_t bq[3] = {64, 1, kCrTile};
    // k nope, v [H][total_k][128]: (cols, key, h); boxes of 64 columns x 128 keys, or 64 values
    const uint64_t dkv[3] = {kCrDh, nk, total_k > 0 ? (uint64_t)H : 1}, skv[2] = {kCrDh * 2, (uint64_t)kCrDh * 2 * nk};
    const uint32_t bk[3] = {64, kCrTile, 1}, bv[3] = {64, kCrTile / 2, 1};
    // RoPE keys: columns 512 .. 575 of the [total_k][576] entries
    const uint64_t de[2] = {kDEntry, nk}, se[1] = {kDEntry * 2};
    const uint32_t be[2] = {64, kCrTile};
    if (!tmap_bf16(&tqn, q_nope, 3, dqn, sqn, bq) || !tmap_bf16(&tk, k_nope, 3, dkv, skv, bk) ||
        !tmap_bf16(&tv, v, 3, dkv, skv, bv))
        return MLA_ERR_CUDA;
    tqr = tqn;
    tkr = tk;
    if (positions && (!tmap_bf16(&tqr, q_rope, 3, dqr, sqr, bq) || !tmap_bf16(&tkr, entries, 2, de, se, be)))
        return MLA_ERR_CUDA;
    CrossArgs a;
    a.ws = (unsigned char *)workspace;
    a.ws_bytes = ws_bytes;
    a.B = B;
    a.H = H;
    a.total_q = (int)total_q;
    a.total_k = (int)total_k;
    a.rows = cross_rows(B, H, total_q, total_k);
    a.scale_log2 = softmax_scale * kLog2e;
    a.positions = positions;
    const long long more = kCrWaitPerTile * ((total_k + kCrTile - 1) / kCrTile), limit = wait_limit();
    a.wait_cycles = limit < INT64_MAX - more ? limit + more : INT64_MAX;
    a.stall = stall_wanted();
    a.before_out = before_out;
    a.before_lse = before_lse;
    a.out = out_dtype == MLA_OUT_FP32 ? (float *)out : nullptr;
    a.out16 = out_dtype == MLA_OUT_BF16 ? (uint16_t *)out : nullptr;
    a.lse = lse;
    const auto one = before_out ? cross_kernel<1, true> : cross_kernel<1, false>;
    const auto two = before_out ? cross_kernel<2, true> : cross_kernel<2, false>;
    cudaError_t e = a.rows == kCrTile ? launch_pdl(one, sms, Shape<1>::kThreads, Shape<1>::kSmem, (cudaStream_t)stream, tqn,
                                                   tqr, tk, tkr, tv, a)
                                      : launch_pdl(two, sms, Shape<2>::kThreads, Shape<2>::kSmem, (cudaStream_t)stream, tqn,
                                                   tqr, tk, tkr, tv, a);
    // (no item has more key tiles than all keys together: short ones are never cut)
    if (e == cudaSuccess && total_k > kCrMinPiece * kCrTile)
        e = launch_pdl(cross_merge_kernel, kCmCtasPerSm * sms, kCmThreads, 0, (cudaStream_t)stream, a);
    return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
