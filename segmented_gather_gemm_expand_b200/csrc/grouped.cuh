// Large segmented products on the tensor cores: rows grouped by expert times
// the expert's weights, and a shared projection with low-rank adapters.
//
//     out[r, n] = (add ? out[r, n] : 0) + sum_k x[r, k] * W[e][n, k]          (r in a segment with index e)
//     out[r, n] = sum_k x[r, k] * W[n, k] + bias[n] + sum_j t[r, j] * B[a(r)][n, j]
//
// The product is computed turned round: the MMA's M axis are weight rows, its
// N axis are tokens.  M is fixed by the hardware (128, or 256 for a CTA pair),
// N is any multiple of 16 (32) up to 256, so a ragged segment costs only its
// own rows rounded up to that, and a decode batch streams its weights through
// the wide side of the MMA.  A segment of L rows is cut into ceil(L / tn)
// token tiles of equal size (rounded up), not into full tiles and a rest.
//
// Roles (320 threads per CTA, more with adapters): warp 0 loads with TMA (x rows
// in boxes of 16 to 128 rows, weights 128 rows, 64 columns of K per stage,
// 128-byte swizzle), warp 1 issues the MMAs into one of two TMEM accumulators,
// warps 2-9 read the other accumulator back (lane = weight row, column =
// token), finish the sums and store.  Producer and MMA roles are one elected
// thread each: run by a warp with a lane's branch inside, the MMAs' operands
// were rebuilt for every instruction (1120 TFLOP/s against 1390).
// Rows of a load past the segment's end are other segments' rows or zeros:
// they only reach accumulator columns that are not stored.
//
// Two forms, picked by a cost model on the host (choose_shape):
//   pair   CTA pairs (cta_group::2), 256 weight rows x up to 256 tokens.  Each
//          CTA loads its 128 weight rows and half of the tokens, so a stage
//          brings 64 MMA columns per KB instead of 43: compute-bound shapes.
//          16384 ragged rows over 8 experts, 4096 -> 11008, bf16: 1010-1023 us in a
//          single launch (1450 TFLOP/s), the tensor pipe 94 % busy at the 1.34-1.39 GHz
//          that the power limit leaves; 1200 us back to back.  Bound: power.
//   single one CTA, 128 weight rows x up to 128 tokens; with few tiles, the
//          CTAs of a cluster share one tile by cutting K, push their partial
//          sums into each other's shared memory (every CTA owns a part of the
//          tokens) and add them in rank order (deterministic): decode shapes.
//          96 rows over 64 experts, 2048 -> 1408: 59 us, 6.3 TB/s of weights.
//          Bound: memory, then the latency of the chain for the smallest calls.
//
// The low-rank part of a shared projection comes in one of two ways (LoraMode):
//   LORA_MMA   as further K steps of the same accumulator, for batches whose
//          segments are long enough to share an MMA: for every run of rows with
//          one adapter in a token tile and every 32 ranks, one stage holds B[a]'s
//          rows (TMA) and a buffer of t's rows, zero outside the run, which
//          warps of their own write some steps ahead of the MMAs.  t is fp32 and
//          enters as the sum of two bf16 parts (hi, and what is left of it, rounded),
//          three where out is fp32: two hold t to 2^-17 of itself (8 bits, and 8 of
//          the 16 left, which have a sign), against out's own rounding of 2^-8 (fp16:
//          2^-11); three hold fp32's 24 bits whole.  bf16 has fp32's range; fp16 parts
//          would lose what lies above 65504 or below 2^-24, which t does even where out
//          does not.  An fp16 B enters as two bf16 parts too, which hold its 11 bits
//          exactly: the warps that write t split its tiles in shared memory (37 mixed
//          segments of rank 24, fp16, 42.7 -> 44.7 us; 4520 rows of 118, 3680 -> 11867,
//          rank 64, 595 -> 617).
//          8764 rows of 16 prompts, 4096 -> 12288, rank 16: 1483 us with FMAs in the
//          epilogue, 690-720 with these steps (the kernel alone 574, the tensor pipe
//          91 % busy; power).
//          A B that TMA cannot read (a transposed view: the input gradient; ranks
//          that leave rows off the 16-byte boundaries) is laid out anew, per
//          segment or per adapter, where the workspace has room.
//   LORA_FMA   on the CUDA cores in fp32, by the epilogue's warps while the K loop
//          runs (they keep it in TMEM until the sums are there): single tokens
//          with an adapter each, or a B that TMA cannot read (without room).  Warp 10 copies
//          each token's 128 rows of B and its row of t into a ring.  256 tokens
//          of 256 adapters of rank 32, 5120 -> 5120: 56 us with the shrink before it
//          (169 with B read lane by lane after the sums); 37 of them here,
//          3.5 TB/s.  Bound: the bytes of W and B under way per SM.
//
// Every wait is bounded and reports a timeout through the device error word.
#pragma once

#include <cuda.h>

#include <mutex>

#include "common.cuh"
#include "plan_cache.cuh"
#include "tc_ptx.cuh"

namespace sgmv {
namespace grp {

using namespace sgmv::tc;

constexpr int BK = 64;                  // K columns per stage: 128-byte rows
constexpr int WROWS = 128;              // weight rows per CTA
constexpr int W_TILE = WROWS * BK * 2;  // 16 KB
constexpr int EPI_WARPS = 8;
constexpr int LORA_WARP = 2 + EPI_WARPS;   // first of the warps that write t (LORA_MMA only)
// LORA_MMA: warps that write t, each into a buffer of its own.  A single CTA's runs are short: four.
constexpr int lora_warps(int cg) { return cg == 2 ? 2 : 4; }
constexpr int MAX_T_BUFS = 4;
enum LoraMode { LORA_NONE = 0, LORA_FMA = 1, LORA_MMA = 2 };
constexpr int B_WARP = 2 + EPI_WARPS;      // loads B for LORA_FMA
constexpr int threads_of(int cg, int lora) {
    return 64 + 32 * EPI_WARPS + (lora == LORA_MMA ? 32 * lora_warps(cg) : lora == LORA_FMA ? 32 : 0);
}
constexpr int B_RING = 32 * 1024;          // LORA_FMA: buffered rows of B for each half of the epilogue's warps
constexpr int B_SLOTS = 8;                 // at most
constexpr int MAX_STAGES = 12;
// LORA_MMA with an fp16 B: barriers on which the tiles of B to be split arrive, one per step in turn.  A step's barrier
// is used again B_STEPS steps later, after the ring of stages has gone round, so its warp has seen the phase before.
constexpr int B_STEPS = 2 * B_SLOTS;
static_assert(B_STEPS >= MAX_STAGES && B_STEPS % 4 == 0, "a barrier belongs to one warp and never runs ahead of it");
constexpr int RING_MAX_RANK = 64;
constexpr int T_ROW = RING_MAX_RANK * 4;   // a slot's row of t, fp32
constexpr int NUM_XMAPS = 4;            // x boxes of 16, 32, 64, 128 rows
constexpr int MAX_SPLITS = 8;
constexpr int TURN = 2 * 8 * 64;        // shared memory in which an epilogue warp turns 8 x 32 halves round, twice
constexpr int BAND = 8;                 // token tiles walked together before the next weight tile
constexpr int SEG_CAP = 4096;           // most segments a launch takes
constexpr int SMEM_LIMIT = 232448 - 1024;

struct Seg {
    int32_t row0, rows, group;
    int32_t ts;       // tokens per tile (the last tile of the segment may own fewer rows)
    int32_t prefix;   // token tiles of earlier segments
};

struct Geo {
    int32_t nblk, kblocks;
    int32_t tn;           // most tokens per tile
    int32_t splits;       // CTAs that share a tile by cutting K (single form)
    int32_t stages, stage_bytes;
    int32_t b_slots, b_bytes;   // LORA_FMA: a ring of tokens' B and t per half of the epilogue (0 slots: read directly), bytes of B in a slot
    int32_t off_t, t_bytes, off_tr, off_out, off_red, off_seg, off_bar;
    int32_t out_vec;      // half output in 16-byte pieces
    int32_t acc_stride, tmem_cols;
    int32_t w_mn;         // the weights' N axis is the contiguous one
    int32_t dense_rows;   // >= 0: one segment of that many rows with group 0; -1: the call's segments
    int32_t dense_ts, dense_tiles;       // its tile height and token tiles
    int32_t off_runs, max_runs;          // LORA_MMA: runs, each token tile's first run, the call's segments
    int32_t early;        // the preceding kernel is the adapters' shrink, which writes neither x nor weights
    int32_t keep_w;       // weights are read by several token tiles: keep them in L2
};

struct XMaps {
    CUtensorMap m[NUM_XMAPS];
};

// Rows of one token tile that belong to one segment with an adapter.
struct Run {
    int32_t adapter, begin, end;   // B's matrix; rows [begin, end), counted from the tile's first
};

// The low-rank part and the bias of a shared projection.
struct Lora {
    const float* t;              // (rows, R) fp32: x A^T
    const int32_t* row_adapter;  // LORA_FMA, (rows): adapter, -1 for none
    MetaVec start, len, idx;     // LORA_MMA: the call's segments
    int32_t batches;
    int64_t adapters;
    const void* b;               // (adapters, N, R), the weights' dtype
    int64_t b_as, b_ns, b_ks;
    int32_t R;
    int32_t parts;               // LORA_MMA: bf16 parts of t (2 or 3)
    int32_t b_vec;               // rows of B can be read as 16-byte pieces
    int32_t by_seg;              // LORA_MMA: b is laid out anew with one matrix per segment, not per adapter
    const void* bias;            // (N) in the weights' dtype, or null
    int64_t bias_s;
};

struct Tile {
    int32_t row0, rows, ts, n0, group;
    int32_t tok;   // token tile within the segment
};

__host__ __device__ __forceinline__ void decode_tile(const Seg* segs, int32_t nseg, const Geo& g, int32_t id, int32_t wtile,
                                            Tile& t) {
    Seg s{0, g.dense_rows, 0, g.dense_ts, 0};
    if (g.dense_rows < 0) {
        const int32_t key = id / g.nblk;
        int lo = 0, hi = nseg - 1;   // last segment whose prefix <= key (empty ones share their successor's)
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (segs[mid].prefix <= key) lo = mid;
            else hi = mid - 1;
        }
        s = segs[lo];
    }
    const int32_t nt = (s.rows + s.ts - 1) / s.ts;
    // bands of BAND token tiles; within a band the token tile is fastest, so the
    // CTAs at work share few weight tiles and few x tiles
    const int32_t local = id - s.prefix * g.nblk;
    const int32_t band = local / (BAND * g.nblk);
    const int32_t in_band = min(BAND, nt - band * BAND);
    const int32_t r = local - band * BAND * g.nblk;
    const int32_t tok = band * BAND + r % in_band;
    t.n0 = (r / in_band) * wtile;
    t.row0 = s.row0 + tok * s.ts;
    t.rows = min(s.ts, s.rows - tok * s.ts);
    t.ts = s.ts;
    t.group = s.group;
    t.tok = tok;
}

// The runs of every token tile of a dense call, in segment order: `runs`, and
// first[i] .. first[i + 1] for tile i.  Built by warps 2 and up (they alone
// synchronise, on barrier 2) while the first loads are under way; overlapping
// segments may fill the list early (max_runs), the same way in every CTA.
template <int WARPS>
__device__ __forceinline__ void build_runs(const Geo& g, const Lora& lo, Run* runs, int32_t* first, Run* segs, int warp,
                                           int lane) {
    constexpr int THREADS = WARPS * 32;
    for (int32_t b = warp * 32 + lane; b < lo.batches; b += THREADS) {
        const Segment s =
            guard_segment(load_meta(lo.start, b), load_meta(lo.len, b), load_meta(lo.idx, b), g.dense_rows, lo.adapters);
        segs[b] = s.rows > 0 ? Run{lo.by_seg ? b : (int32_t)s.adapter, (int32_t)s.row0, (int32_t)(s.row0 + s.rows)}
                             : Run{-1, 0, 0};
    }
    bar_sync(2, THREADS);
    for (int pass = 0; pass < 2; ++pass) {
        for (int32_t i = warp; i < g.dense_tiles; i += WARPS) {
            const int32_t r0 = i * g.dense_ts, r1 = min(r0 + g.dense_ts, g.dense_rows);
            int32_t at = pass ? first[i] : 0;
            for (int32_t b0 = 0; b0 < lo.batches; b0 += 32) {
                const Run s = b0 + lane < lo.batches ? segs[b0 + lane] : Run{-1, 0, 0};
                const bool in = s.begin < r1 && s.end > r0;
                const unsigned mask = __ballot_sync(0xffffffffu, in);
                if (pass && in) {
                    const int32_t k = at + __popc(mask & ((1u << lane) - 1));
                    if (k < g.max_runs) runs[k] = Run{s.adapter, max(s.begin, r0) - r0, min(s.end, r1) - r0};
                }
                at += __popc(mask);
            }
            if (!pass && lane == 0) first[i + 1] = at;
        }
        bar_sync(2, THREADS);
        if (!pass) {
            if (warp == 0) {   // counts to places
                int32_t run = 0;
                for (int32_t i0 = 0; i0 < g.dense_tiles; i0 += 32) {
                    const int32_t i = i0 + lane, n = i < g.dense_tiles ? first[i + 1] : 0;
                    int32_t v = n;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int32_t u = __shfl_up_sync(0xffffffffu, v, o);
                        if (lane >= o) v += u;
                    }
                    if (i < g.dense_tiles) first[i + 1] = min(run + v, g.max_runs);
                    run += __shfl_sync(0xffffffffu, v, 31);
                }
                if (lane == 0) first[0] = 0;
            }
            bar_sync(2, THREADS);
        }
    }
}

// d[j] = sum_k t[row + j, k] * B[adapter of row + j][n, k] for j < valid, in
// fp32, 16 ranks at a time.  The B pieces of all eight tokens are requested
// before the first is used: decode batches have an adapter per token, and one
// after the other their latencies add up (48 tokens took 51 us so).
__device__ __forceinline__ void lora_delta(float (&d)[8], int64_t row, int valid, int64_t n, bool n_ok, const Lora& lo,
                                           bool bf16) {
    int a[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        d[j] = 0.f;
        a[j] = j < valid ? lo.row_adapter[row + j] : -1;
    }
    const uint16_t* b = static_cast<const uint16_t*>(lo.b) + n * lo.b_ns;
    const float* t = lo.t + row * lo.R;
    int r0 = 0;
    if (lo.b_vec && lo.R % 4 == 0) {
        for (; r0 + 16 <= lo.R; r0 += 16) {
            uint4 u[8][2];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool on = a[j] >= 0 && n_ok;
                const uint4* q = reinterpret_cast<const uint4*>(b + (int64_t)a[j] * lo.b_as + r0);
                u[j][0] = on ? __ldg(q) : make_uint4(0, 0, 0, 0);
                u[j][1] = on ? __ldg(q + 1) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (a[j] < 0) continue;
                const float4* tp = reinterpret_cast<const float4*>(t + j * lo.R + r0);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t w[4] = {u[j][h].x, u[j][h].y, u[j][h].z, u[j][h].w};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float4 f = tp[h * 2 + k];
                        const float2 b0 = unpack2(w[2 * k], bf16), b1 = unpack2(w[2 * k + 1], bf16);
                        d[j] = fmaf(f.x, b0.x, d[j]);
                        d[j] = fmaf(f.y, b0.y, d[j]);
                        d[j] = fmaf(f.z, b1.x, d[j]);
                        d[j] = fmaf(f.w, b1.y, d[j]);
                    }
                }
            }
        }
    }
    for (; r0 < lo.R; ++r0)   // the last ranks, and B in any other layout
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (a[j] >= 0 && n_ok)
                d[j] = fmaf(t[j * lo.R + r0],
                            half_bits_to_float(__ldg(b + (int64_t)a[j] * lo.b_as + r0 * lo.b_ks), bf16), d[j]);
}

// One token's low-rank sum over its buffered rows of B: row `row` of 128, R
// halves each, back to back.  Eight lanes read 16 bytes each at a time; rows of
// an even number of such pieces would meet in the same banks, so every lane
// starts at a piece of its own (`turn`, from lora_turn) and goes round.
__device__ __forceinline__ int lora_turn(int row, int R) {
    const int pieces = R / 8, g = pieces & 1 ? 1 : pieces & 2 ? 2 : pieces & 4 ? 4 : 8;   // gcd(pieces, 8)
    return (row * g / 8) % g;
}

__device__ __forceinline__ float lora_dot(const uint8_t* rows, int row, int R, int turn, const float* t, bool bf16) {
    const uint4* b = reinterpret_cast<const uint4*>(rows + row * R * 2);
    const float4* t4 = reinterpret_cast<const float4*>(t);
    const int pieces = R / 8;
    float d0 = 0.f, d1 = 0.f;
    int k = turn;
#pragma unroll 2
    for (int i = 0; i < pieces; ++i) {
        const float4 x = t4[2 * k], y = t4[2 * k + 1];
        const uint4 u = b[k];
        const float2 a = unpack2(u.x, bf16), c = unpack2(u.y, bf16), e = unpack2(u.z, bf16), f = unpack2(u.w, bf16);
        d0 = fmaf(x.x, a.x, d0);
        d1 = fmaf(x.y, a.y, d1);
        d0 = fmaf(x.z, c.x, d0);
        d1 = fmaf(x.w, c.y, d1);
        d0 = fmaf(y.x, e.x, d0);
        d1 = fmaf(y.y, e.y, d1);
        d0 = fmaf(y.z, f.x, d0);
        d1 = fmaf(y.w, f.y, d1);
        if (++k == pieces) k = 0;
    }
    return d0 + d1;
}

// LORA_FMA and shared tiles: the i-th token that a half of the epilogue's warps
// finishes, 8 of every 16.
__device__ __forceinline__ int half_token(int half, int i) { return (i >> 3) * 16 + half * 8 + (i & 7); }

// Adds the old output (add mode), rounds once and stores eight rows, row .. row +
// valid - 1, of column n (= the warp's first column + lane).  fp32: a warp's
// store is a row's 32 columns, 128 bytes.  Halves: the warp turns its 8 x 32
// piece round in shared memory (`turn`) and stores 16 bytes per lane; where the
// output's rows are not whole 16-byte pieces (vec false), element by element.
__device__ __forceinline__ void put8(float (&v)[8], int64_t row, int valid, int64_t n, const Problem& p, uint32_t* turn,
                                     bool vec) {
    if (valid <= 0) return;
    const int64_t base = row * p.H + n;
    if (p.out_dt == SGMV_F32) {
        if (n >= p.N) return;
        float* o = static_cast<float*>(p.out) + base;
        if (p.add) {
            float old[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) old[j] = j < valid ? o[j * p.H] : 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += old[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < valid) o[j * p.H] = v[j];
        return;
    }
    const bool ob = p.out_dt == SGMV_BF16;
    if (vec) {
        const int lane = threadIdx.x % 32, r = lane / 4, c = (lane % 4) * 8;
        const bool mine = r < valid && n - lane + c < p.N;   // this lane's row and 8 columns (N: a multiple of 8)
        uint16_t* o = static_cast<uint16_t*>(p.out) + (base - lane + r * p.H + c);
        uint16_t* halves = reinterpret_cast<uint16_t*>(turn);   // [token][32 columns]
        if (p.add) {
            if (mine) *reinterpret_cast<uint4*>(halves + r * 32 + c) = *reinterpret_cast<const uint4*>(o);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += half_bits_to_float(halves[j * 32 + lane], ob);   // rows past `valid` are not stored
            __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) halves[j * 32 + lane] = (uint16_t)float_to_half_bits(v[j], ob);
        __syncwarp();
        if (mine) *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(halves + r * 32 + c);
        __syncwarp();
        return;
    }
    if (n >= p.N) return;
    uint16_t* o = static_cast<uint16_t*>(p.out) + base;
    if (p.add) {
        uint16_t old[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) old[j] = j < valid ? o[j * p.H] : (uint16_t)0;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += half_bits_to_float(old[j], ob);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < valid) o[j * p.H] = (uint16_t)float_to_half_bits(v[j], ob);
}

// NaN where a value is no finite number, else z.
__device__ __forceinline__ float no_numbers(const float (&v)[8], float z) {
#pragma unroll
    for (int j = 0; j < 8; ++j) z = fmaf(v[j], 0.f, z);
    return z;
}

// LORA_MMA, where an accumulator was an infinity or NaN: rows outside a run take
// part in the run's MMA with t = 0, and 0 times an infinity in that adapter's B
// reaches other requests' rows.  Where a run of the tile has such a value in B's
// row n, the outputs of column n that are no finite numbers (of the tokens first_tok
// .. end_tok of the tile that this warp has stored, whose first row is row0) are
// computed again by the formula, in fp32; with a split B all such outputs of rows
// with an adapter, since an infinite t met the zeros that are left of B.  `runs`
// first .. last are the tile's.  The warp computes its 32 columns of eight tokens at
// once, after it has handed its accumulator back: with a warp per output and the
// accumulator held, a tile took up to 350 ms at K = 4096, which for K above 24000
// was more than the two seconds that the MMAs wait.  8192 rows of 16 segments, 4096 ->
// 4096, one adapter full of NaN: 352 ms then, 8 ms now (200 us without the NaN).
__device__ __forceinline__ void repair_outputs(int first_tok, int end_tok, int64_t row0, int64_t n, float bias, const Run* runs,
                                            int first, int last, const Problem& p, const Lora& lo) {
    const bool bf16 = p.w_dt == SGMV_BF16;
    const int64_t col = n < p.N ? n : p.N - 1;
    const uint16_t* b = static_cast<const uint16_t*>(lo.b) + col * lo.b_ns;
    float z = 0.f;   // NaN if a run's B is no finite number in this row
#pragma unroll 1
    for (int r = first; r < last; ++r)
#pragma unroll 4
        for (int k = 0; k < lo.R; ++k)
            z = fmaf(half_bits_to_float(__ldg(b + runs[r].adapter * lo.b_as + k * lo.b_ks), bf16), 0.f, z);
    // rows of x start on 16-byte boundaries, the weights' too where K is their contiguous axis
    const uint16_t* w = static_cast<const uint16_t*>(p.w) + col * p.w_ns;
    const bool w_vec = p.w_ks == 1 && (p.w_ns * 2) % 16 == 0;
    __syncwarp();   // the outputs were stored by other lanes
#pragma unroll 1
    for (int tok = first_tok; tok < end_tok; tok += 16) {
        const int64_t row = row0 + tok;
        unsigned bad = 0, in_run = 0;
        for (int j = 0; j < 8; ++j)
            if (tok + j < end_tok && n < p.N && fmaf(load_elem(p.out, p.out_dt, (row + j) * p.H + n), 0.f, 0.f) != 0.f)
                bad |= 1u << j;
        for (int r = first; r < last; ++r)
            for (int j = 0; j < 8; ++j) in_run |= (tok + j >= runs[r].begin && tok + j < runs[r].end ? 1u : 0u) << j;
        if (z == 0.f) bad &= bf16 ? 0u : in_run;
        const unsigned want = __reduce_or_sync(0xffffffffu, bad);
        if (!want) continue;
        const uint16_t* x[8];
        float s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {   // rows that nobody asks for may not exist
            x[j] = static_cast<const uint16_t*>(p.x) + (row + (want >> j & 1 ? j : __ffs(want) - 1)) * p.x_rs;
            s[j] = 0.f;
        }
        int64_t k = 0;
#pragma unroll 1
        for (; k + 8 <= p.K; k += 8) {
            uint4 u[8];
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = __ldg(reinterpret_cast<const uint4*>(x[j] + k));
            if (w_vec) {
                const uint4 q = __ldg(reinterpret_cast<const uint4*>(w + k));
                const uint32_t q4[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 c = unpack2(q4[i], bf16);
                    f[2 * i] = c.x;
                    f[2 * i + 1] = c.y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = half_bits_to_float(__ldg(w + (k + i) * p.w_ks), bf16);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t q4[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 c = unpack2(q4[i], bf16);
                    s[j] = fmaf(c.x, f[2 * i], s[j]);
                    s[j] = fmaf(c.y, f[2 * i + 1], s[j]);
                }
            }
        }
#pragma unroll 1
        for (; k < p.K; ++k) {
            const float f = half_bits_to_float(__ldg(w + k * p.w_ks), bf16);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = fmaf(half_bits_to_float(__ldg(x[j] + k), bf16), f, s[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (!(want >> j & 1)) continue;
#pragma unroll 1
            for (int r = first; r < last; ++r)
                if (tok + j >= runs[r].begin && tok + j < runs[r].end)
#pragma unroll 4
                    for (int i = 0; i < lo.R; ++i)
                        s[j] = fmaf(lo.t[(row + j) * lo.R + i],
                                    half_bits_to_float(__ldg(b + runs[r].adapter * lo.b_as + i * lo.b_ks), bf16), s[j]);
            if (bad >> j & 1) store_elem(p.out, p.out_dt, (row + j) * p.H + n, s[j] + bias);
        }
    }
}

// A warp's share of a tile from TMEM to memory: 8 of every 16 columns (tokens),
// from 8 * half on, two such pieces in turn, the next ones under way while these
// are stored (one piece at a time: 113 us instead of 104, on one GPU, for the weight
// gradient of 16 experts, whose tiles are short; the conversions and copies of a piece
// wait for one another).  Short loops on purpose: straight-line code for 32 tokens
// at a time spent its time fetching instructions.  `drained` runs once the last
// values are in registers.  With CHECK the result is NaN where a value was no
// finite number.
template <bool CHECK, class Drained>
__device__ __forceinline__ float drain(uint32_t taddr, int half, int ts, int64_t row0, int rows, int64_t n, float bias,
                                      const Problem& p, uint32_t* turn, bool vec, Drained&& drained) {
    const int lane = threadIdx.x % 32, r = lane / 4, c8 = (lane % 4) * 8;
    const bool ob = p.out_dt == SGMV_BF16;
    const bool fast = vec && !p.add;
    const bool c_ok = n - lane + c8 < p.N;                 // N: a multiple of 8 where vec
    const uint32_t pick = r & 1 ? 0x7632u : 0x5410u;
    uint16_t* o = static_cast<uint16_t*>(p.out) + ((row0 + half * 8 + r) * p.H + n - lane + c8);
    const int64_t step = 16 * p.H;
    uint32_t next[8], next2[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    float v[8], u[8];
    float z = 0.f;
    int c = half * 8;
    if (c >= rows) {
        drained();
        return z;
    }
    if (fast && rows >= 32) {
        tmem_ld8(taddr + (uint32_t)c, next);
        if (c + 16 < rows) tmem_ld8(taddr + (uint32_t)c + 16, next2);
#pragma unroll 1
        for (;; c += 32, o += 2 * step) {
            tmem_ld_wait(next);
            tmem_ld_wait(next2);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = __uint_as_float(next[j]);
                u[j] = __uint_as_float(next2[j]);
            }
            const bool more = c + 32 < rows;
            if (more) {
                tmem_ld8(taddr + (uint32_t)c + 32, next);
                if (c + 48 < rows) tmem_ld8(taddr + (uint32_t)c + 48, next2);
            } else drained();
            if (CHECK) z = no_numbers(u, no_numbers(v, z));
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                turn[j * 32 + lane] = pack2(v[2 * j] + bias, v[2 * j + 1] + bias, ob);
                turn[128 + j * 32 + lane] = pack2(u[2 * j] + bias, u[2 * j + 1] + bias, ob);
            }
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 x = *reinterpret_cast<const uint4*>(turn + h * 128 + (r >> 1) * 32 + c8);
                const uint4 y = *reinterpret_cast<const uint4*>(turn + h * 128 + (r >> 1) * 32 + c8 + 4);
                if (c_ok && c + 16 * h + r < rows)
                    *reinterpret_cast<uint4*>(o + h * step) = make_uint4(__byte_perm(x.x, x.y, pick), __byte_perm(x.z, x.w, pick),
                                                              __byte_perm(y.x, y.y, pick), __byte_perm(y.z, y.w, pick));
            }
            if (!more) break;
        }
        return z;
    }
    tmem_ld8(taddr + (uint32_t)c, next);
#pragma unroll 1
    for (;; c += 16, o += step) {
        tmem_ld_wait(next);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(next[j]);
        const bool more = c + 16 < rows;
        if (more) tmem_ld8(taddr + (uint32_t)c + 16, next);
        else drained();
        if (CHECK) z = no_numbers(v, z);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += bias;
        if (fast) {
            // pairs of tokens share a conversion and a word: [pair][32 columns], two buffers in turn
            uint32_t* s = turn + ((c >> 4) & 1) * 128;
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j * 32 + lane] = pack2(v[2 * j], v[2 * j + 1], ob);
            __syncwarp();
            const uint4 x = *reinterpret_cast<const uint4*>(s + (r >> 1) * 32 + c8);
            const uint4 y = *reinterpret_cast<const uint4*>(s + (r >> 1) * 32 + c8 + 4);
            if (c_ok && c + r < rows)
                *reinterpret_cast<uint4*>(o) = make_uint4(__byte_perm(x.x, x.y, pick), __byte_perm(x.z, x.w, pick),
                                                          __byte_perm(y.x, y.y, pick), __byte_perm(y.z, y.w, pick));
        } else {
            put8(v, row0 + c, min(8, rows - c), n, p, turn, vec);
        }
        if (!more) break;
    }
    return z;
}

// The bf16 part of (a, b): hi = rounded(v), and v - hi left for the next part.  A
// number above bf16's largest, or an infinity, leaves the largest, and the rest of it
// (an infinity) to the last part, which is rounded as it is.
__device__ __forceinline__ uint32_t next_part(float& a, float& b, bool last) {
    uint32_t bits;
    if (last) {
        bits = pack2(a, b, true);
    } else {
        asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(bits) : "f"(b), "f"(a));
        const float2 back = unpack2(bits, true);
        a -= back.x;
        b -= back.y;
    }
    return bits;
}

// An fp16 tile of B (128 rows of `cols` ranks, K-major, 128-byte swizzle) as two bf16
// tiles beside each other: the leading 8 of its 11 bits in place, the other three C
// columns on, both exact.  (An infinity leaves NaN beside it: repair_outputs sees to
// the outputs.)  One warp.
__device__ __forceinline__ void split_b(uint8_t* tile, int C, int cols, int lane) {
#pragma unroll 1
    for (int h = 0; h < cols / 8; ++h) {
#pragma unroll
        for (int i = 0; i < WROWS / 32; ++i) {
            const int row = lane + 32 * i;
            uint4* src = reinterpret_cast<uint4*>(tile + row * 128 + ((h ^ (row & 7)) << 4));
            const uint4 u = *src;
            const uint32_t in[4] = {u.x, u.y, u.z, u.w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 v = unpack2(in[k], false);
                const uint32_t a = __float_as_uint(v.x) & 0xffff0000u, b = __float_as_uint(v.y) & 0xffff0000u;
                hi[k] = __byte_perm(a, b, 0x7632);
                lo[k] = __byte_perm(__float_as_uint(v.x - __uint_as_float(a)), __float_as_uint(v.y - __uint_as_float(b)), 0x7632);
            }
            *src = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(tile + row * 128 + (((h + C / 8) ^ (row & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
}

// A low-rank step's t: up to 128 rows of t from row0 on, ranks [r, r + ranks), as
// a K-major tile with 128-byte swizzle: `parts` groups of C columns (C = 32 for
// two parts, 16 for three), zero outside the step's runs and past the last rank.
// One warp; a lane takes two rows at a time (i0 + lane, i0 + lane + 32), all
// their ranks requested at once.
struct TRows {
    float4 q[2][8];
};

__device__ __forceinline__ void load_t(TRows& x, int64_t row0, int i0, int begin, int end, int r, int ranks, const Lora& lo,
                                       int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int k0 = i0 + lane + 32 * i;
        const bool in = k0 >= begin && k0 < end;
        const float* src = lo.t + (row0 + k0) * lo.R + r;
        if (lo.R % 4 == 0) {   // r: a multiple of 16
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x.q[i][k] = in && 4 * k < ranks ? reinterpret_cast<const float4*>(src)[k] : make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
            const int n = in ? ranks : 0;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x.q[i][k] = make_float4(4 * k < n ? src[4 * k] : 0.f, 4 * k + 1 < n ? src[4 * k + 1] : 0.f,
                                        4 * k + 2 < n ? src[4 * k + 2] : 0.f, 4 * k + 3 < n ? src[4 * k + 3] : 0.f);
        }
    }
}

// Two runs at a time (ranks of 16 at most): a row's ranks enter columns 0 .. 15 if
// it belongs to run a, columns 16 .. 31 if to run b.
__device__ __forceinline__ void load_t2(TRows& x, int64_t row0, int i0, int base, const Run& a, const Run& b, const Lora& lo,
                                        int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int k0 = i0 + lane + 32 * i, at = base + k0;
        const bool in_a = at >= a.begin && at < a.end, in_b = at >= b.begin && at < b.end;
        const float* src = lo.t + (row0 + k0) * lo.R;
        const int n = in_a || in_b ? lo.R : 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float4 v;
            if (lo.R % 4 == 0)
                v = 4 * k < n ? reinterpret_cast<const float4*>(src)[k] : make_float4(0.f, 0.f, 0.f, 0.f);
            else
                v = make_float4(4 * k < n ? src[4 * k] : 0.f, 4 * k + 1 < n ? src[4 * k + 1] : 0.f,
                                4 * k + 2 < n ? src[4 * k + 2] : 0.f, 4 * k + 3 < n ? src[4 * k + 3] : 0.f);
            x.q[i][k] = in_a ? v : make_float4(0.f, 0.f, 0.f, 0.f);
            x.q[i][k + 4] = in_a ? make_float4(0.f, 0.f, 0.f, 0.f) : v;
        }
    }
}

// Rows of a buffer of t that are not zero: those of the runs (one or two) that
// its step holds.
struct TSpan {
    int b[2], e[2];
    __device__ __forceinline__ bool has(int row) const {
        return (row >= b[0] && row < e[0]) || (row >= b[1] && row < e[1]);
    }
    __device__ __forceinline__ bool meets(int from, int to) const {
        return max(b[0], from) < min(e[0], to) || max(b[1], from) < min(e[1], to);
    }
};

// Writes the rows of `now` and zeroes those of `before`; all others are zero already
// (2048 rows of 64 segments, rank 32: 96 us; 110 with every row written every time).
__device__ __forceinline__ void store_t(uint8_t* dst, TRows& x, int i0, const TSpan& now, const TSpan& before, int parts,
                                        int lane) {
    const int C = parts == 2 ? 32 : 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = i0 + lane + 32 * i;
        if (!now.has(row) && !before.has(row)) continue;
        for (int part = 0; part < parts; ++part) {
            const bool last = part + 1 == parts;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                if (h >= C / 8) continue;
                float4 &a = x.q[i][2 * h], &b = x.q[i][2 * h + 1];
                const uint32_t w0 = next_part(a.x, a.y, last), w1 = next_part(a.z, a.w, last);
                const uint32_t w2 = next_part(b.x, b.y, last), w3 = next_part(b.z, b.w, last);
                const int chunk = part * C / 8 + h;
                *reinterpret_cast<uint4*>(dst + row * 128 + ((chunk ^ (row & 7)) << 4)) = make_uint4(w0, w1, w2, w3);
            }
        }
    }
}

// The token columns of a run's MMA: the whole tile for a CTA pair, whose second
// half of the columns is the other CTA's; the 16-column groups that the run
// touches for a single CTA.
template <int CG>
__device__ __forceinline__ void run_columns(const Run& run, int32_t ts, int32_t& off, int32_t& cols) {
    off = CG == 2 ? 0 : run.begin & ~15;
    cols = CG == 2 ? ts : min(ts, (run.end + 15) & ~15) - off;
}

// Runs that share a buffer of t: in a CTA pair two where their ranks fit into 32
// columns, since writing a buffer takes longer than its MMAs (2048 rows of 64
// segments, 4096 -> 4096, rank 16: 98 us with one, 87 with two).  A single CTA's
// buffers are its run's rows alone, and twice as many: 81 us against 86.
template <int CG>
__device__ __forceinline__ int runs_per_step(const Lora& lo) {
    return CG == 2 && lo.parts == 2 && lo.R <= 16 ? 2 : 1;
}

// The next box of x (16 << level rows) for `rows` more rows, a positive multiple of
// 16: the smallest that holds them all if the stage has `room` for it (every
// further box costs the producer time: 1230 us instead of 1176 for the experts'
// prefill with exact boxes), else the largest within them.
__device__ __forceinline__ int x_box(int rows, int room) {
    const int up = rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : 3;
    if ((16 << up) <= room) return up;
    return rows >= 128 ? 3 : rows >= 64 ? 2 : rows >= 32 ? 1 : 0;
}

// LORA_FMA is held to 128 registers a thread (as for 512 threads): a CTA of the
// shrink before it then fits beside it, and the weights stream while the shrink runs.
template <int CG, int LORA>
__global__ void __launch_bounds__(LORA == LORA_FMA ? 512 : threads_of(CG, LORA), 1)
gemm_kernel(const __grid_constant__ XMaps xmaps, const __grid_constant__ CUtensorMap wmap,
            const __grid_constant__ CUtensorMap bmap, const __grid_constant__ Problem p, const Geo g,
            const __grid_constant__ Lora lo) {
    constexpr int THREADS = threads_of(CG, LORA), LORA_WARPS = lora_warps(CG);
    constexpr bool EARLY = LORA != LORA_NONE;   // producer and MMAs may run while the shrink still does
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ int s_abort;
    __shared__ uint32_t s_tmem_base;
    __shared__ int32_t s_token_tiles;

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t csize = CG == 2 ? 2u : (uint32_t)g.splits;
    const uint32_t crank = csize > 1 ? cluster_rank() : 0u;
    const int32_t cid = (int32_t)(blockIdx.x / csize), ncl = (int32_t)(gridDim.x / csize);
    const uint32_t S = (uint32_t)g.stages;
    Seg* segs = reinterpret_cast<Seg*>(smem + g.off_seg);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + g.off_bar);
    uint64_t* empty = full + S;
    uint64_t* acc_full = empty + S;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* red_full = acc_empty + 2;
    uint64_t* red_free = red_full + 1;
    uint64_t* t_full = red_free + 1;   // LORA_MMA: buffers of t besides the stages
    uint64_t* t_empty = t_full + MAX_T_BUFS;
    uint64_t* b_full = t_empty + MAX_T_BUFS;    // LORA_FMA: [half][slot]; LORA_MMA: [step % B_STEPS]
    uint64_t* b_empty = b_full + 2 * B_SLOTS;

    // The table of runs (LORA_MMA) and its barrier.
    uint64_t* runs_ready = b_empty + 2 * B_SLOTS;
    Run* runs = reinterpret_cast<Run*>(smem + g.off_runs);
    int32_t* first_run = reinterpret_cast<int32_t*>(runs + g.max_runs);
    const bool dense = LORA != LORA_NONE || g.dense_rows >= 0;

    if (warp == 0) {
        if (lane == 0) {
            s_abort = 0;
            for (uint32_t i = 0; i < S; ++i) {
                mbar_init(smem_u32(&full[i]), 1);   // the first CTA of a pair announces the bytes of both
                mbar_init(smem_u32(&empty[i]), 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(smem_u32(&acc_full[i]), 1);
                mbar_init(smem_u32(&acc_empty[i]), CG * EPI_WARPS);
            }
            for (int i = 0; i < MAX_T_BUFS; ++i) {
                mbar_init(smem_u32(&t_full[i]), CG);
                mbar_init(smem_u32(&t_empty[i]), 1);
            }
            for (int i = 0; LORA != LORA_NONE && i < 2 * B_SLOTS; ++i) {
                mbar_init(smem_u32(&b_full[i]), 1);
                mbar_init(smem_u32(&b_empty[i]), EPI_WARPS / 2);
            }
            mbar_init(smem_u32(red_full), 1);   // the expected bytes, then the stores' own counts
            mbar_init(smem_u32(red_free), csize * EPI_WARPS);
            mbar_init(smem_u32(runs_ready), 1);
            fence_barrier_init();
        }
        __syncwarp();
    } else if (warp == 1) {
        if (CG == 2) tmem_alloc_pair(smem_u32(&s_tmem_base), (uint32_t)g.tmem_cols);
        else tmem_alloc(smem_u32(&s_tmem_base), (uint32_t)g.tmem_cols);
    } else if (warp == 2 && lane == 0) {
        prefetch_tmap(&wmap);
        for (int k = 0; k < NUM_XMAPS; ++k) prefetch_tmap(&xmaps.m[k]);
        if (LORA == LORA_MMA) prefetch_tmap(&bmap);
    }

    // Everything below may read memory written by the preceding kernel, unless
    // that is the adapters' shrink: then only what reads t waits for it.
    if (!g.early) {
        grid_dependency_wait();
        grid_dependents_launch();
    }

    const int32_t nseg = dense ? 1 : (int32_t)p.batches;
    if (!dense) {
        // Segment table (guards of sgmv.h applied), tile size and tiles of earlier segments.
        constexpr int32_t STEP = 16 * CG;
        for (int32_t b = tid; b < nseg; b += THREADS) {
            const Segment s = load_segment(p, b);
            const int32_t rows = (int32_t)s.rows;
            const int32_t nt = (rows + g.tn - 1) / g.tn;
            const int32_t ts = nt > 0 ? ((rows + nt - 1) / nt + STEP - 1) / STEP * STEP : STEP;
            segs[b] = Seg{(int32_t)s.row0, rows, (int32_t)s.adapter, ts, 0};
        }
        __syncthreads();
        if (warp == 0) {
            int32_t run = 0;
            for (int32_t base = 0; base < nseg; base += 32) {
                const int32_t b = base + lane;
                const int32_t nt = b < nseg ? (segs[b].rows + segs[b].ts - 1) / segs[b].ts : 0;
                int32_t v = nt;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int32_t t = __shfl_up_sync(0xffffffffu, v, o);
                    if (lane >= o) v += t;
                }
                if (b < nseg) segs[b].prefix = run + v - nt;
                run += __shfl_sync(0xffffffffu, v, 31);
            }
            if (lane == 0) s_token_tiles = run;
        }
    }
    // A single CTA's producer needs nothing of the others for a dense call: it
    // starts at once (the other roles would hold the first loads up by a
    // microsecond).  The CTAs of a cluster meet before their first exchange, a
    // pair before its first load.
    const bool ahead = CG == 1 && dense && warp == 0;
    tc_fence_before();
    if (csize > 1) cluster_arrive();
    if (CG == 1 && dense) {
        if (warp == 0) bar_arrive(1, THREADS);
        else bar_sync(1, THREADS);
    } else {
        __syncthreads();
    }
    if (CG == 2) cluster_wait();
    if (CG == 1 && csize > 1 && warp >= 2) cluster_wait();
    tc_fence_after();

    const uint32_t tmem_base = ahead ? 0u : s_tmem_base;
    const int32_t total = (dense ? g.dense_tiles : s_token_tiles) * g.nblk;
    volatile int* abort_flag = &s_abort;
    const bool bf16 = p.w_dt == SGMV_BF16;
    constexpr int32_t WT = WROWS * CG;
    const int32_t kb0 = CG == 2 ? 0 : (int32_t)((int64_t)g.kblocks * crank / csize);
    const int32_t kb1 = CG == 2 ? g.kblocks : (int32_t)((int64_t)g.kblocks * (crank + 1) / csize);
    const bool lora_here = CG == 2 || crank == 0;   // of CTAs that share a tile, the first adds the low-rank part
    const int32_t t_ranks = lo.parts == 2 ? 32 : 16;
    const bool split = LORA == LORA_MMA && !bf16;   // B's tiles are split before the MMAs see them
    Tile t;
    if (LORA == LORA_MMA && warp >= 2) {
        constexpr int WARPS = EPI_WARPS + LORA_WARPS;
        build_runs<WARPS>(g, lo, runs, first_run, reinterpret_cast<Run*>(first_run + g.dense_tiles + 1), warp - 2, lane);
        if (warp == 2 && lane == 0) mbar_arrive(smem_u32(runs_ready));
    }

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (elect_one()) {
            const uint64_t pol_x = policy_evict_normal();
            const uint64_t pol_w = g.keep_w ? policy_evict_normal() : policy_evict_first();
            uint32_t s = 0, phase = 1, m = 0;
            bool ok = true;
            for (int32_t id = cid; ok && id < total; id += ncl) {
                decode_tile(segs, nseg, g, id, WT, t);
                const int32_t hs = t.ts / CG;   // token rows of this CTA
                const int room = g.tn / CG;
                int x_rows = 0;                 // rows that the boxes bring
                while (x_rows < hs) x_rows += 16 << x_box(hs - x_rows, room - x_rows);
                const uint32_t bytes = W_TILE + (uint32_t)x_rows * 128u;
                const int lvl0 = x_box(hs, room), rows0 = 16 << lvl0;   // the first box, nearly always the only one
                const CUtensorMap* x0 = &xmaps.m[lvl0];
                const int32_t xr = t.row0 + (CG == 2 ? (int32_t)crank * hs : 0);
                const int32_t n0 = t.n0 + (CG == 2 ? (int32_t)crank * WROWS : 0);
                for (int32_t kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait<EARLY>(smem_u32(&empty[s]), phase, abort_flag, DEVERR_TIMEOUT_PRODUCER)) {
                        ok = false;
                        break;
                    }
                    const uint32_t ws = smem_u32(smem + s * g.stage_bytes), xs = ws + W_TILE;
                    if (CG == 2) {
                        // both CTAs' loads count at the first one's barrier; it alone announces them: a remote
                        // arrival with release semantics costs a memory barrier per stage (1640 cycles a stage
                        // instead of 512).  The second CTA cannot run a phase ahead, since it waits for `empty`.
                        const uint32_t bar = map_to_rank(smem_u32(&full[s]), 0);
                        if (crank == 0) mbar_expect_tx(smem_u32(&full[s]), 2 * bytes);
                        if (g.w_mn) {
                            tma_load_3d_pair(ws, &wmap, n0, kb * BK, t.group, bar, pol_w);
                            tma_load_3d_pair(ws + W_TILE / 2, &wmap, n0 + 64, kb * BK, t.group, bar, pol_w);
                        } else {
                            tma_load_3d_pair(ws, &wmap, kb * BK, n0, t.group, bar, pol_w);
                        }
                        tma_load_2d_pair(xs, x0, kb * BK, xr, bar, pol_x);
                        for (int r = rows0; r < hs;) {
                            const int lvl = x_box(hs - r, room - r);
                            tma_load_2d_pair(xs + r * 128, &xmaps.m[lvl], kb * BK, xr + r, bar, pol_x);
                            r += 16 << lvl;
                        }
                    } else {
                        const uint32_t bar = smem_u32(&full[s]);
                        mbar_expect_tx(bar, bytes);
                        if (g.w_mn) {
                            tma_load_3d(ws, &wmap, n0, kb * BK, t.group, bar, pol_w);
                            tma_load_3d(ws + W_TILE / 2, &wmap, n0 + 64, kb * BK, t.group, bar, pol_w);
                        } else {
                            tma_load_3d(ws, &wmap, kb * BK, n0, t.group, bar, pol_w);
                        }
                        tma_load_2d(xs, x0, kb * BK, xr, bar, pol_x);
                        for (int r = rows0; r < hs;) {
                            const int lvl = x_box(hs - r, room - r);
                            tma_load_2d(xs + r * 128, &xmaps.m[lvl], kb * BK, xr + r, bar, pol_x);
                            r += 16 << lvl;
                        }
                    }
                    if (++s == S) {
                        s = 0;
                        phase ^= 1;
                    }
                }
                if (LORA == LORA_MMA && ok && lora_here) {
                    ok = mbar_wait<EARLY>(smem_u32(runs_ready), 0, abort_flag, DEVERR_TIMEOUT_PRODUCER);
                    const int32_t last = ok ? first_run[t.tok + 1] : 0;
                    const int per_step = runs_per_step<CG>(lo);
                    for (int32_t r = ok ? first_run[t.tok] : 0; ok && r < last; r += per_step) {
                        const int n_runs = CG == 2 ? min(per_step, last - r) : 1;
                        for (int32_t r0 = 0; ok && r0 < lo.R; r0 += t_ranks, ++m) {
                            for (int i = 0; i < n_runs; ++i) {
                                if (!mbar_wait<EARLY>(smem_u32(&empty[s]), phase, abort_flag, DEVERR_TIMEOUT_PRODUCER)) {
                                    ok = false;
                                    break;
                                }
                                const int32_t a = runs[r + i].adapter;
                                const uint32_t ws = smem_u32(smem + s * g.stage_bytes);
                                uint32_t bar = smem_u32(&full[s]);
                                if (split) {
                                    // the bytes arrive at this CTA's own barrier of the step; the stage's phase
                                    // passes, and what the MMAs wait for is t's barrier, after the split
                                    if (CG == 1 || crank == 0) mbar_arrive(bar);
                                    bar = smem_u32(&b_full[m % B_STEPS]);
                                    if (i == 0) mbar_expect_tx(bar, (uint32_t)n_runs * W_TILE);
                                } else if (CG == 2) {
                                    if (crank == 0) mbar_expect_tx(bar, 2 * W_TILE);
                                    bar = map_to_rank(bar, 0);
                                } else {
                                    mbar_expect_tx(bar, W_TILE);
                                }
                                if (CG == 2) tma_load_3d_pair(ws, &bmap, r0, n0, a, bar, pol_x);
                                else tma_load_3d(ws, &bmap, r0, n0, a, bar, pol_x);
                                if (++s == S) {
                                    s = 0;
                                    phase ^= 1;
                                }
                            }
                        }
                    }
                }
            }
            // the commits of the other CTA's MMAs arrive here: none may be under way when this CTA ends
            for (uint32_t i = 0; CG == 2 && ok && i < S; ++i) {
                ok = mbar_wait<EARLY>(smem_u32(&empty[s]), phase, abort_flag, DEVERR_TIMEOUT_PRODUCER);
                if (++s == S) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        __syncwarp();
    } else if (LORA == LORA_MMA && warp >= LORA_WARP) {
        // ------------------------------------------------------------ t, ahead of the MMAs by up to a few low-rank steps
        // The warps take the steps in turn, each with its own buffer.
        if (g.early) grid_dependency_wait();
        const uint32_t buf = (uint32_t)(warp - LORA_WARP);
        uint8_t* dst = smem + g.off_t + buf * g.t_bytes;
        uint32_t m = 0, mine = 0, st = 0;   // st: the step's first stage, followed where B is split
        const int per_step = runs_per_step<CG>(lo);
        for (int o = lane * 16; o < g.t_bytes; o += 512) *reinterpret_cast<uint4*>(dst + o) = make_uint4(0, 0, 0, 0);
        __syncwarp();
        TSpan before{{0, 0}, {0, 0}};
        bool ok = true;
        for (int32_t id = cid; ok && lora_here && id < total; id += ncl) {
            decode_tile(segs, nseg, g, id, WT, t);
            const int32_t last = first_run[t.tok + 1];
            if (split) st = (st + (uint32_t)(kb1 - kb0)) % S;
            for (int32_t r = first_run[t.tok]; ok && r < last; r += per_step) {
                const int n = CG == 2 ? min(per_step, last - r) : 1;
                const Run run = runs[r], next = n == 2 ? runs[r + 1] : Run{0, 0, 0};
                int32_t off, cols;
                run_columns<CG>(run, t.ts, off, cols);
                // the rows of t that this CTA's columns are: all of a single CTA's, a half of a pair's
                const int32_t base = CG == 2 ? (int32_t)crank * (t.ts / 2) : off, rows = CG == 2 ? t.ts / 2 : cols;
                for (int32_t r0 = 0; ok && r0 < lo.R; r0 += t_ranks, ++m) {
                    const uint32_t at = st;
                    if (split) st = st + n >= S ? st + n - S : st + n;
                    if (m % LORA_WARPS != buf) continue;
                    const int ranks = n == 2 ? 32 : min(t_ranks, lo.R - r0);
                    TRows v;
                    const auto load = [&](int i0) {
                        if (CG == 2 && per_step == 2) load_t2(v, (int64_t)t.row0 + base, i0, base, run, next, lo, lane);
                        else load_t(v, (int64_t)t.row0 + base, i0, run.begin - base, run.end - base, r0, ranks, lo, lane);
                    };
                    const TSpan now{{max(run.begin - base, 0), max(next.begin - base, 0)},
                                    {min(run.end - base, rows), min(next.end - base, rows)}};
                    const bool low = now.meets(0, 64) || before.meets(0, 64), high = now.meets(64, 128) || before.meets(64, 128);
                    const int i0 = low ? 0 : 64;
                    if (low || high) load(i0);
                    // A pair's warps fall behind its MMAs, so they split B while t is on its way (642 us against
                    // 658 on 4520 rows of 118 segments); a single CTA's have t ready long before B arrives (37 mixed
                    // segments 45.8 against 48.3).
                    const auto split_step = [&] {
                        ok = warp_wait(smem_u32(&b_full[m % B_STEPS]), (m / B_STEPS) & 1, abort_flag, DEVERR_TIMEOUT_CONVERT);
                        const int width = (min(t_ranks, lo.R - r0) + 15) & ~15;
                        for (int i = 0; ok && i < n; ++i)
                            split_b(smem + (at + i >= S ? at + i - S : at + i) * g.stage_bytes, t_ranks, width, lane);
                        return ok;
                    };
                    if (CG == 2 && split && !split_step()) break;
                    ok = warp_wait(smem_u32(&t_empty[buf]), (mine & 1) ^ 1, abort_flag, DEVERR_TIMEOUT_CONVERT);
                    if (!ok) break;
                    ++mine;
                    if (low || high) store_t(dst, v, i0, now, before, lo.parts, lane);
                    if (low && high) {
                        load(64);
                        store_t(dst, v, 64, now, before, lo.parts, lane);
                    }
                    before = now;
                    if (CG == 1 && split && !split_step()) break;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (CG == 2 && crank != 0) mbar_arrive_cluster(map_to_rank(smem_u32(&t_full[buf]), 0));
                        else mbar_arrive(smem_u32(&t_full[buf]));
                    }
                }
            }
        }
        // the commits of the other CTA's MMAs free the buffers: none may be under way when this CTA ends
        if (CG == 2 && ok) warp_wait(smem_u32(&t_empty[buf]), (mine & 1) ^ 1, abort_flag, DEVERR_TIMEOUT_CONVERT);
    } else if (LORA == LORA_FMA && warp == B_WARP) {
        // ------------------------------------------------------------ B and t of the tokens that this CTA finishes
        if (g.early) grid_dependency_wait();
        if (g.b_slots > 0) {
            const uint64_t pol = policy_evict_first();
            const bool one = elect_one();
            uint32_t slot[2] = {0, 0}, phase[2] = {1, 1};
            bool ok = true;
            for (int32_t id = cid; ok && id < total; id += ncl) {
                decode_tile(segs, nseg, g, id, WT, t);
                const int tw = csize > 1 ? ((t.ts + (int)csize - 1) / (int)csize + 3) & ~3 : t.ts;
                const int t0 = (int)crank * tw, cnt = min(tw, t.rows - t0);
                for (int i0 = 0; ok && half_token(0, i0) < cnt; i0 += 32) {
                    int32_t mine[2];   // adapters of 32 tokens of each half, one per lane
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int tok = half_token(h, i0 + lane);
                        mine[h] = tok < cnt ? lo.row_adapter[t.row0 + t0 + tok] : -1;
                    }
                    for (int i = 0; ok && i < 64; ++i) {
                        const int h = i & 1;
                        const int32_t a = __shfl_sync(0xffffffffu, h ? mine[1] : mine[0], i >> 1);
                        if (a < 0) continue;
                        const int64_t row = (int64_t)t.row0 + t0 + half_token(h, i0 + (i >> 1));
                        const uint32_t sl = h ? slot[1] : slot[0], ph = h ? phase[1] : phase[0];
                        const uint32_t bar = smem_u32(&b_full[h * B_SLOTS + sl]), q = (uint32_t)(h * g.b_slots) + sl;
                        ok = warp_wait(smem_u32(&b_empty[h * B_SLOTS + sl]), ph, abort_flag, DEVERR_TIMEOUT_PRODUCER);
                        if (ok && one) {
                            // B's rows are contiguous (lora_b.b_ns == R): one copy of 128 rows, fewer at N's end
                            const uint32_t bytes = (uint32_t)min((int64_t)WROWS, p.N - t.n0) * (uint32_t)lo.R * 2u;
                            const uint32_t tb = (uint32_t)lo.R * 4u;
                            mbar_expect_tx(bar, bytes + tb);
                            bulk_load(smem_u32(smem + g.off_t) + q * g.b_bytes,
                                      static_cast<const uint16_t*>(lo.b) + (int64_t)a * lo.b_as + (int64_t)t.n0 * lo.R, bytes,
                                      bar, pol);
                            bulk_load(smem_u32(smem + g.off_tr) + q * T_ROW, lo.t + row * lo.R, tb, bar, pol);
                        }
                        const bool wrap = sl + 1 == (uint32_t)g.b_slots;
                        if (h) {
                            slot[1] = wrap ? 0 : sl + 1;
                            phase[1] ^= wrap;
                        } else {
                            slot[0] = wrap ? 0 : sl + 1;
                            phase[0] ^= wrap;
                        }
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA (the pair's first CTA)
        if ((CG == 1 || crank == 0) && elect_one()) {
            uint32_t s = 0, phase = 0, n = 0, m = 0;
            bool ok = true;
            // K step of 16 inside a stage: 32 bytes along a K-major row, 16 rows of an N-major tile
            const uint64_t w_step = (uint64_t)((g.w_mn ? 16 * 128 : 32) >> 4);
            const uint64_t ad0 = smem_desc(smem_u32(smem), g.w_mn ? W_TILE / 2 : 16, 1024, 2);
            const uint64_t bd0 = smem_desc(smem_u32(smem) + W_TILE, 16, 1024, 2);
            const uint64_t stage_step = (uint64_t)(g.stage_bytes >> 4);
            for (int32_t id = cid; ok && id < total; id += ncl, ++n) {
                decode_tile(segs, nseg, g, id, WT, t);
                const uint32_t acc = n & 1;
                const uint32_t idesc = instr_desc_mn(bf16, WT, t.ts) | (g.w_mn ? IDESC_A_MN : 0u);
                const uint32_t d = tmem_base + acc * (uint32_t)g.acc_stride;
                if (!mbar_wait<EARLY>(smem_u32(&acc_empty[acc]), ((n >> 1) & 1) ^ 1, abort_flag, DEVERR_TIMEOUT_MMA)) break;
                tc_fence_after();
                for (int32_t kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait<EARLY>(smem_u32(&full[s]), phase, abort_flag, DEVERR_TIMEOUT_MMA)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = ad0 + s * stage_step, bd = bd0 + s * stage_step;
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk) {
                        const uint32_t more = (kk > 0 || kb > kb0) ? 1u : 0u;
                        if (CG == 2) tc_mma_pair(d, ad + kk * w_step, bd + kk * 2, idesc, more);
                        else tc_mma(d, ad + kk * w_step, bd + kk * 2, idesc, more);
                    }
                    if (CG == 2) tc_commit_pair(smem_u32(&empty[s]));
                    else tc_commit(smem_u32(&empty[s]));
                    if (++s == S) {
                        s = 0;
                        phase ^= 1;
                    }
                }
                if (LORA == LORA_MMA && ok && lora_here) {
                    ok = mbar_wait<EARLY>(smem_u32(runs_ready), 0, abort_flag, DEVERR_TIMEOUT_MMA);
                    const uint64_t bk0 = smem_desc(smem_u32(smem), 16, 1024, 2);   // B's rows are K-major
                    const int32_t last = ok ? first_run[t.tok + 1] : 0;
                    const int per_step = runs_per_step<CG>(lo);
                    for (int32_t r = ok ? first_run[t.tok] : 0; ok && r < last; r += per_step) {
                        const int n_runs = CG == 2 ? min(per_step, last - r) : 1;
                        int32_t off, cols;
                        run_columns<CG>(runs[r], t.ts, off, cols);   // a pair's: the whole tile for every run
                        const uint32_t idesc_t = instr_desc_mn(true, WT, cols), dt = d + (uint32_t)off;   // t and B in bf16
                        for (int32_t r0 = 0; ok && r0 < lo.R; r0 += t_ranks, ++m) {
                            const uint32_t buf = m % LORA_WARPS;
                            // a pair's second CTA writes its half of t (and splits its rows of B) itself
                            const uint32_t tb = smem_u32(&t_full[buf]), tp = (m / LORA_WARPS) & 1;
                            ok = CG == 2 ? mbar_wait_cluster<EARLY>(tb, tp, abort_flag, DEVERR_TIMEOUT_MMA)
                                         : mbar_wait<EARLY>(tb, tp, abort_flag, DEVERR_TIMEOUT_MMA);
                            if (!ok) break;
                            const uint64_t bd = smem_desc(smem_u32(smem + g.off_t + buf * g.t_bytes), 16, 1024, 2);
                            const int steps = (min(t_ranks, lo.R - r0) + 15) / 16;
                            for (int i = 0; i < n_runs; ++i) {
                                if (!mbar_wait<EARLY>(smem_u32(&full[s]), phase, abort_flag, DEVERR_TIMEOUT_MMA)) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
                                const uint64_t ad = bk0 + s * stage_step;
                                for (int q = 0; q < (split ? 2 : 1); ++q)
                                    for (int part = 0; part < lo.parts; ++part)
                                        for (int kk = 0; kk < steps; ++kk) {
                                            const uint64_t bq = ad + (uint64_t)((q * t_ranks) / 8 + kk * 2);
                                            const uint64_t td = bd + (uint64_t)((part * t_ranks) / 8 + (kk + i) * 2);
                                            if (CG == 2) tc_mma_pair(dt, bq, td, idesc_t, 1u);
                                            else tc_mma(dt, bq, td, idesc_t, 1u);
                                        }
                                if (CG == 2) tc_commit_pair(smem_u32(&empty[s]));
                                else tc_commit(smem_u32(&empty[s]));
                                if (++s == S) {
                                    s = 0;
                                    phase ^= 1;
                                }
                            }
                            if (!ok) break;
                            if (CG == 2) tc_commit_pair(smem_u32(&t_empty[buf]));
                            else tc_commit(smem_u32(&t_empty[buf]));
                        }
                    }
                }
                if (!ok) break;
                if (CG == 2) tc_commit_pair(smem_u32(&acc_full[acc]));
                else tc_commit(smem_u32(&acc_full[acc]));
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        if (g.early) {
            grid_dependency_wait();   // t and the rows' adapters; nothing was written before
            grid_dependents_launch();
        }
        const int quad = warp % 4, half = (warp - 2) / 4;
        const int nl = quad * 32 + lane;
        uint32_t* stage = reinterpret_cast<uint32_t*>(smem + g.off_out + (warp - 2) * TURN);
        uint32_t b_slot = 0, b_phase = 0;
        const int turn = LORA == LORA_FMA ? lora_turn(nl, lo.R) : 0;
        uint32_t n = 0, reds = 0;   // reds: exchanges in which this CTA owned tokens
        for (int32_t id = cid; id < total; id += ncl, ++n) {
            decode_tile(segs, nseg, g, id, WT, t);
            const uint32_t acc = n & 1;
            const int64_t col = t.n0 + (CG == 2 ? (int32_t)crank * WROWS : 0) + nl;
            const bool n_ok = col < p.N;
            float bias = 0.f;
            if (lo.bias && n_ok) bias = half_bits_to_float(static_cast<const uint16_t*>(lo.bias)[col * lo.bias_s], bf16);
            const int tw = csize > 1 && CG == 1 ? ((t.ts + (int)csize - 1) / (int)csize + 3) & ~3 : t.ts;
            const int t0 = CG == 1 ? (int)crank * tw : 0, cnt = min(tw, t.rows - t0);   // tokens this CTA finishes
            const uint32_t lanes = (uint32_t)(quad * 32) << 16;
            const uint32_t delta = tmem_base + 2 * (uint32_t)g.acc_stride + lanes;   // LORA_FMA: a TMEM column per token
            if (LORA == LORA_FMA) {
                // while the K loop runs: the low-rank part of the tokens that this warp will store
                if (g.b_slots > 0) {
                    bool ok = true;
                    for (int i0 = 0; ok && half_token(half, i0) < cnt; i0 += 32) {
                        const int mine = half_token(half, i0 + lane);
                        const unsigned on = __ballot_sync(
                            0xffffffffu, mine < cnt && lo.row_adapter[(int64_t)t.row0 + t0 + min(mine, cnt - 1)] >= 0);
                        for (int i = 0; ok && i < 32; ++i) {
                            const int tok = half_token(half, i0 + i);
                            if (tok >= cnt) break;
                            float d = 0.f;
                            if ((on >> i) & 1) {
                                const uint32_t at = (uint32_t)half * B_SLOTS + b_slot, q = (uint32_t)(half * g.b_slots) + b_slot;
                                ok = warp_wait(smem_u32(&b_full[at]), b_phase, abort_flag, DEVERR_TIMEOUT_EPILOGUE);
                                if (!ok) break;
                                d = lora_dot(smem + g.off_t + q * g.b_bytes, nl, lo.R, turn,
                                             reinterpret_cast<const float*>(smem + g.off_tr + q * T_ROW), bf16);
                                __syncwarp();
                                if (lane == 0) mbar_arrive(smem_u32(&b_empty[at]));
                                if (++b_slot == (uint32_t)g.b_slots) {
                                    b_slot = 0;
                                    b_phase ^= 1;
                                }
                            }
                            tmem_st1(delta + (uint32_t)tok, __float_as_uint(d));
                        }
                    }
                    if (!ok) break;
                } else {
                    for (int i = 0; half_token(half, i) < cnt; i += 8) {
                        const int j0 = half_token(half, i);
                        float d[8];
                        lora_delta(d, (int64_t)t.row0 + t0 + j0, cnt - j0, col, n_ok, lo, bf16);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            tmem_st1(delta + (uint32_t)(j0 + j), __float_as_uint(d[j]));
                    }
                }
                tmem_st_wait();
            }
            if (!warp_wait(smem_u32(&acc_full[acc]), (n >> 1) & 1, abort_flag, DEVERR_TIMEOUT_EPILOGUE)) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + acc * (uint32_t)g.acc_stride + lanes;
            if (LORA == LORA_FMA && csize == 1) {
                for (int j0 = half * 8; j0 < cnt; j0 += 16) {
                    uint32_t a[8], b[8];
                    tmem_ld8(taddr + (uint32_t)j0, a);
                    tmem_ld8(delta + (uint32_t)j0, b);
                    tmem_ld_wait(a, b);
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(a[j]) + __uint_as_float(b[j]) + bias;
                    put8(v, (int64_t)t.row0 + j0, min(8, cnt - j0), col, p, stage, g.out_vec);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && id + 2 * ncl < total) mbar_arrive(smem_u32(&acc_empty[acc]));
            } else if (CG == 2 || csize == 1) {
                const float z = drain<LORA == LORA_MMA>(
                    taddr, half, t.ts, t.row0, t.rows, col, bias, p, stage, g.out_vec, [&] {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0 && id + 2 * ncl < total) {   // somebody waits for it
                            if (CG == 2) mbar_arrive_remote(map_to_rank(smem_u32(&acc_empty[acc]), 0));
                            else mbar_arrive(smem_u32(&acc_empty[acc]));
                        }
                    });
                if (LORA == LORA_MMA && __any_sync(0xffffffffu, z != 0.f))
                    repair_outputs(half * 8, t.rows, t.row0, col, bias, runs, first_run[t.tok], first_run[t.tok + 1], p, lo);
            } else {
                // Partial sums go to the CTA that owns the token, four tokens of a weight row
                // (16 bytes) at a time: red[source][token / 4][weight row][token % 4].  The
                // stores count themselves at the owner's barrier, so nobody fences.
                const uint32_t red = smem_u32(smem + g.off_red) + (crank * (tw / 4) * WROWS + nl) * 16;
                if (cnt > 0 && warp == 2 && lane == 0)
                    mbar_expect_tx(smem_u32(red_full), csize * (uint32_t)((cnt + 3) / 4) * WROWS * 16u);
                if (n > 0 && !warp_wait_cluster(smem_u32(red_free), (n & 1) ^ 1, abort_flag, DEVERR_TIMEOUT_EPILOGUE))
                    break;
                for (int c = half * 32; c < t.rows; c += 64) {
                    float v[32];
                    tmem_ld32(taddr + (uint32_t)c, reinterpret_cast<uint32_t(&)[32]>(v));
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const int tok = c + j;
                        if (tok < t.rows) {
                            const uint32_t owner = (uint32_t)(tok / tw);
                            st_async_v4(map_to_rank(red + ((tok - (int)owner * tw) / 4) * (WROWS * 16), owner),
                                        map_to_rank(smem_u32(red_full), owner), v[j], v[j + 1], v[j + 2], v[j + 3]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&acc_empty[acc]));
                if (cnt > 0) {
                    if (!warp_wait_cluster(smem_u32(red_full), reds & 1, abort_flag, DEVERR_TIMEOUT_EPILOGUE)) break;
                    ++reds;
                    const float4* rp = reinterpret_cast<const float4*>(smem + g.off_red) + nl;
                    float z = 0.f;
                    for (int j0 = half * 8; j0 < cnt; j0 += 16) {
                        float v[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = 0.f;
                        if (LORA == LORA_FMA) {
                            uint32_t b[8];
                            tmem_ld8(delta + (uint32_t)j0, b);
                            tmem_ld_wait(b);
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[j] += __uint_as_float(b[j]);
                        }
                        for (int src = 0; src < (int)csize; ++src)
#pragma unroll
                            for (int j = 0; j < 8; j += 4)
                                if (j0 + j < cnt) {
                                    const float4 f = rp[(src * (tw / 4) + (j0 + j) / 4) * WROWS];
                                    v[j] += f.x;
                                    v[j + 1] += f.y;
                                    v[j + 2] += f.z;
                                    v[j + 3] += f.w;
                                }
                        if (LORA == LORA_MMA) z = no_numbers(v, z);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] += bias;
                        put8(v, (int64_t)t.row0 + t0 + j0, min(8, cnt - j0), col, p, stage, g.out_vec);
                    }
                    if (LORA == LORA_MMA && __any_sync(0xffffffffu, z != 0.f))
                        repair_outputs(t0 + half * 8, t0 + cnt, t.row0, col, bias, runs, first_run[t.tok], first_run[t.tok + 1],
                                       p, lo);
                }
                __syncwarp();
                if (lane < (int)csize && id + ncl < total) mbar_arrive_remote(map_to_rank(smem_u32(red_free), (uint32_t)lane));
            }
        }
    }

    if (CG == 1 && csize > 1 && warp < 2) cluster_wait();   // the meeting at the start
    tc_fence_before();
    __syncthreads();
    outlast_copies(abort_flag);
    if (csize > 1) cluster_sync();   // no CTA leaves while another may still signal it
    tc_fence_after();
    if (warp == 1) {
        if (CG == 2) tmem_dealloc_pair(tmem_base, (uint32_t)g.tmem_cols);
        else tmem_dealloc(tmem_base, (uint32_t)g.tmem_cols);
    }
}

// ====================================================================== host side

struct Plan {
    Geo geo;
    XMaps xm;
    CUtensorMap wm;
    int cg;
    int smem_bytes;
    int grid;
};

// The tensor-core kernels take x and weights of one half dtype whose rows
// (along K, or along N for the weights) are contiguous and start on 16-byte
// boundaries.
inline bool supports(const Problem& p) {
    if (p.x_dt != p.w_dt || p.K < 1 || p.N < 1) return false;
    if (p.x_cs != 1 || (p.x_rs * 2) % 16 || p.x_rs < p.K || (reinterpret_cast<uintptr_t>(p.x) & 15)) return false;
    if (reinterpret_cast<uintptr_t>(p.w) & 15) return false;
    const bool k_major = p.w_ks == 1 && (p.w_ns * 2) % 16 == 0 && p.w_ns >= p.K;
    const bool n_major = p.w_ns == 1 && (p.w_ks * 2) % 16 == 0 && p.w_ks >= p.N;
    if (!k_major && !n_major) return false;
    const int64_t span = k_major ? p.N * p.w_ns : p.K * p.w_ks;
    if (p.lora_num > 1 && ((p.w_as * 2) % 16 || p.w_as + (k_major ? p.w_ns - p.K : p.w_ks - p.N) < span)) return false;
    const int64_t lim = int64_t(1) << 31;
    if (p.K >= lim || p.N >= lim || p.x_rows >= lim || p.out_rows >= lim || p.lora_num >= lim) return false;
    if (p.x_rs >= (int64_t(1) << 38) || p.w_ns >= (int64_t(1) << 38) || p.w_ks >= (int64_t(1) << 38) ||
        p.w_as >= (int64_t(1) << 38))
        return false;
    // tile numbers are 32-bit
    const int64_t rows = p.x_rows < p.out_rows ? p.x_rows : p.out_rows;
    if ((rows / 16 + p.batches + 1) * ((p.N + WROWS - 1) / WROWS) >= lim) return false;
    return p.batches <= SEG_CAP;
}

// Half output rows can be written as 16-byte pieces.
inline bool out_vec_ok(const Problem& p) {
    return p.out_dt != SGMV_F32 && (reinterpret_cast<uintptr_t>(p.out) & 15) == 0 && p.H % 8 == 0 && p.N % 8 == 0;
}

struct Shape {
    int cg, tn, splits;
};

// What a plan is made for, besides the problem.
struct Want {
    bool dense;      // one segment of all rows
    bool early;
    int lora;        // LoraMode
    int R;
    int ring;        // LORA_FMA: B's rows can be copied into a ring
    int segs;        // LORA_MMA: the call's segments
    int sm_count;
    int clusters[MAX_SPLITS]; // clusters of 1, 2, .. 8 CTAs that fit on the device at a time
    int forced_cg;   // 0: the cost model chooses
};

// Shared memory of a form besides the stages and the segment table.
struct Extra {
    int t, b_bytes, b_slots, out, red;
    int t_bufs;
    int total() const { return t_bufs * t + 2 * b_slots * (b_bytes + T_ROW) + out + red; }
};

inline Extra extra_of(const Shape& sh, const Want& w) {
    Extra e;
    const int own = ((sh.tn + sh.splits - 1) / sh.splits + 3) & ~3;   // tokens a CTA finishes
    e.t_bufs = lora_warps(sh.cg);
    e.t = w.lora == LORA_MMA ? (sh.tn / sh.cg < 64 ? 64 : sh.tn / sh.cg) * 128 : 0;
    e.b_bytes = w.lora == LORA_FMA && w.ring ? w.R * WROWS * 2 : 0;
    e.b_slots = 0;
    if (e.b_bytes) {
        e.b_slots = B_RING / e.b_bytes;
        e.b_slots = e.b_slots > B_SLOTS ? B_SLOTS : e.b_slots < 2 ? 2 : e.b_slots;
    }
    e.out = EPI_WARPS * TURN;
    e.red = sh.splits > 1 ? sh.splits * own * WROWS * 4 : 0;
    return e;
}

inline int stage_bytes(const Shape& sh) { return W_TILE + sh.tn / sh.cg * 128; }

// Token tiles of a dense call, and their height.
struct DenseTiles {
    int32_t ts, count;
    DenseTiles(int64_t rows, const Shape& sh) {
        const int64_t step = 16 * sh.cg, nt = (rows + sh.tn - 1) / sh.tn;
        ts = (int32_t)(nt > 0 ? ((rows + nt - 1) / nt + step - 1) / step * step : step);
        count = (int32_t)((rows + ts - 1) / ts);
    }
};

// Bytes of the segment table, and of the table of runs (LORA_MMA: segments that do not overlap leave at most segs +
// tiles runs, beside which stand each tile's first run and the call's segments).
inline int64_t seg_table(const Problem& p, const Want& w) { return w.dense ? 0 : p.batches * (int64_t)sizeof(Seg); }
inline int64_t run_table(int64_t tiles, const Want& w) {
    return w.lora == LORA_MMA ? (2 * (int64_t)w.segs + tiles) * (int64_t)sizeof(Run) + (tiles + 1) * 4 : 0;
}

// The form with the least estimated time, in SM cycles.  A tile takes the
// longest of: its loads at 64 bytes a cycle (weights, x, and B for LORA_FMA),
// its MMAs (2 cycles per token column for 128 weight rows and 64 of K),
// LORA_FMA's arithmetic, and the loads' latency over the stages under way;
// plus a fixed cost, and for a shared tile the exchange of the partial sums.
// The whole takes at least as long as memory needs for the weights (3500 bytes
// a cycle).  Segments are taken as equally long, since their lengths are on the
// device.
inline Shape choose_shape(const Problem& p, const Want& w) {
    const int64_t rows = p.x_rows < p.out_rows ? p.x_rows : p.out_rows;
    const int64_t segs = w.dense ? 1 : (p.batches < rows ? p.batches : rows);
    const int64_t mean = segs > 0 ? (rows + segs - 1) / segs : 1;
    const int64_t kblocks = (p.K + BK - 1) / BK;
    const double experts = w.dense ? 1 : (double)(segs < p.lora_num ? segs : p.lora_num);
    const double bytes = experts * (double)p.N * p.K * 2.0;
    Shape best{1, 32, 1};
    double best_cost = -1;
    const int tns[2][5] = {{32, 48, 64, 96, 128}, {64, 96, 128, 192, 256}};
    for (int cg = 1; cg <= 2; ++cg) {
        if (w.lora == LORA_FMA ? cg == 2 : w.forced_cg && cg != w.forced_cg) continue;
        for (int ti = 0; ti < 5; ++ti) {
            const int tn = tns[cg - 1][ti];
            const int64_t nt = (mean + tn - 1) / tn;
            const int64_t ts = ((mean + nt - 1) / nt + 16 * cg - 1) / (16 * cg) * (16 * cg);
            const int64_t tiles = segs * nt * ((p.N + WROWS * cg - 1) / (WROWS * cg));
            for (int sp = 1; sp <= (cg == 1 ? MAX_SPLITS : 1); sp *= 2) {   // clusters of 3 measured slower than both 2 and 4
                if (sp > 1 && kblocks < 4 * sp) break;
                const Shape sh{cg, tn, sp};
                const Extra e = extra_of(sh, w);
                // tables, barriers and alignment
                const int64_t tables = seg_table(p, w) + run_table(w.dense ? DenseTiles(rows, sh).count : 0, w) + 1664;
                const int stages = (int)((SMEM_LIMIT - (tables > 4096 ? tables : 4096) - e.total()) / stage_bytes(sh));
                if (stages < 2) continue;
                const int64_t workers = w.clusters[cg == 2 ? 1 : sp - 1];
                if (workers < 1) continue;
                const int64_t waves = (tiles + workers - 1) / workers;
                const double kb = (double)((kblocks + sp - 1) / sp);
                const double own = (double)((ts + sp - 1) / sp);   // tokens a CTA finishes
                const double load = (kb * (W_TILE + ts / cg * 128.0) + own * e.b_bytes) / 64.0;
                const double mma = kb * 2.0 * ts;
                const double alu = w.lora != LORA_FMA ? 0.0 : own * w.R * (w.ring ? 4.0 : 30.0) + 1000.0;
                const double late = kb * 1500.0 / stages;
                double body = load > mma ? load : mma;
                if (body < alu) body = alu;
                if (body < late) body = late;
                // LORA_MMA: a step per run of a segment and 32 ranks, its t written by a warp of its own
                const double runs = (double)ts * w.segs / (rows > 0 ? rows : 1) + 1.0;
                const double steps = w.lora == LORA_MMA ? runs * ((w.R + 31) / 32) * (cg == 2 ? 2500.0 : 500.0) : 0.0;
                if (body < steps) body = steps;
                const double exchange = sp > 1 ? 3000.0 + 32.0 * ts : 0.0;
                const double path = waves * (body + exchange + 600.0) + 16.0 * own;
                // memory: 3500 bytes a cycle, or the weights' stages under way over a latency of 2800 cycles
                const double active = (double)(tiles < workers ? tiles : workers) * sp * cg;
                const double under_way = active * stages * W_TILE / 2800.0;
                const double memory = bytes / (under_way < 3500.0 ? under_way : 3500.0);
                const double cost = (path > memory ? path : memory) + 0.1 * path;
                if (best_cost < 0 || cost < best_cost * 0.97) {
                    best_cost = cost;
                    best = sh;
                }
            }
        }
    }
    return best;
}

inline bool make_plan(const Problem& p, const Want& w, EncodeTiledFn enc, Plan* out) {
    if (!supports(p) || !enc) return false;
    const bool dense = w.dense;
    const Shape sh = choose_shape(p, w);
    Geo& g = out->geo;
    const int64_t rows = p.x_rows < p.out_rows ? p.x_rows : p.out_rows;
    out->cg = sh.cg;
    g.tn = sh.tn;
    g.splits = sh.splits;
    g.nblk = (int32_t)((p.N + WROWS * sh.cg - 1) / (WROWS * sh.cg));
    g.kblocks = (int32_t)((p.K + BK - 1) / BK);
    g.w_mn = !(p.w_ks == 1 && (p.w_ns * 2) % 16 == 0 && p.w_ns >= p.K);
    g.dense_rows = dense ? (int32_t)rows : -1;
    g.early = w.early ? 1 : 0;
    g.out_vec = out_vec_ok(p);
    const int64_t segs = dense ? 1 : p.batches;
    g.keep_w = rows > (int64_t)sh.tn * segs ? 1 : 0;
    g.acc_stride = sh.tn < 32 ? 32 : sh.tn;
    g.tmem_cols = 32;
    while (g.tmem_cols < 2 * g.acc_stride + (w.lora == LORA_FMA ? (sh.tn + 31) / 32 * 32 : 0)) g.tmem_cols *= 2;
    g.stage_bytes = stage_bytes(sh);
    const Extra e = extra_of(sh, w);
    g.t_bytes = e.t;
    g.b_slots = e.b_slots;
    g.b_bytes = e.b_bytes;
    const DenseTiles tiles_of(dense ? rows : 0, sh);
    g.dense_ts = tiles_of.ts;
    g.dense_tiles = tiles_of.count;
    g.max_runs = w.lora == LORA_MMA ? w.segs + g.dense_tiles : 0;
    if (seg_table(p, w) + run_table(g.dense_tiles, w) > SMEM_LIMIT) return false;
    const int table = (int)run_table(g.dense_tiles, w);
    for (g.stages = MAX_STAGES; g.stages >= 2; --g.stages) {
        g.off_t = g.stages * g.stage_bytes;                       // t or B (1024-byte aligned: swizzled)
        g.off_tr = g.off_t + e.t_bufs * e.t + 2 * e.b_slots * g.b_bytes;
        g.off_out = g.off_tr + 2 * e.b_slots * T_ROW;
        g.off_red = g.off_out + e.out;
        g.off_seg = g.off_red + e.red;
        g.off_runs = (g.off_seg + (int)seg_table(p, w) + 15) & ~15;
        g.off_bar = (g.off_runs + table + 15) & ~15;
        out->smem_bytes = g.off_bar + 8 * (2 * g.stages + 7 + 2 * MAX_T_BUFS + 4 * B_SLOTS) + 1024;
        if (out->smem_bytes <= SMEM_LIMIT) break;
    }
    if (g.stages < 2) return false;

    const cuuint32_t ones[3] = {1, 1, 1};
    for (int k = 0; k < NUM_XMAPS; ++k) {
        const cuuint64_t dims[2] = {(cuuint64_t)p.K, (cuuint64_t)p.x_rows};
        const cuuint64_t strides[1] = {(cuuint64_t)(p.x_rs * 2)};
        const cuuint32_t box[2] = {(cuuint32_t)BK, (cuuint32_t)(16 << k)};
        if (enc(&out->xm.m[k], CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(p.x), dims, strides, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    }
    const int64_t in = g.w_mn ? p.N : p.K, mid = g.w_mn ? p.K : p.N, pitch = g.w_mn ? p.w_ks : p.w_ns;
    const cuuint64_t dims[3] = {(cuuint64_t)in, (cuuint64_t)mid, (cuuint64_t)p.lora_num};
    cuuint64_t e_stride = (cuuint64_t)(p.w_as * 2);
    if (p.lora_num == 1) e_stride = (cuuint64_t)((mid * pitch * 2 + 15) / 16 * 16);
    const cuuint64_t strides[2] = {(cuuint64_t)(pitch * 2), e_stride};
    const cuuint32_t box[3] = {64, (cuuint32_t)(g.w_mn ? BK : WROWS), 1};
    if (enc(&out->wm, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(p.w), dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return false;
    // most tiles the call can have: every segment may end in a partial one
    const int64_t most_segs = segs < rows ? segs : rows;
    const int64_t tiles = (rows / sh.tn + most_segs + 1) * g.nblk;
    const int csize = sh.cg == 2 ? 2 : sh.splits;
    int64_t clusters = w.clusters[csize - 1];
    if (tiles < clusters) clusters = tiles;
    out->grid = (int)(clusters < 1 ? 1 : clusters) * csize;
    return true;
}

struct PlanKey {
    Problem p;
    Want w;
    int32_t device;
};

// Clusters of 1 to 8 CTAs (one per SM) that the current device holds at a time:
// a GPC whose SM count the size does not divide leaves some idle.  0: unknown.
inline bool cluster_capacity(int device, int sm_count, int (&out)[MAX_SPLITS]) {
    static std::mutex mu;
    static int known[64][MAX_SPLITS];
    std::lock_guard<std::mutex> lk(mu);
    if (device < 0 || device >= 64) return false;
    if (!known[device][0]) {
        auto kern = gemm_kernel<1, LORA_NONE>;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_LIMIT) != cudaSuccess) return false;
        int got[MAX_SPLITS] = {sm_count};
        for (int size = 2; size <= MAX_SPLITS; ++size) {
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = (unsigned)size;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)(sm_count / size * size));
            cfg.blockDim = dim3(threads_of(1, LORA_NONE));
            cfg.dynamicSmemBytes = SMEM_LIMIT;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&got[size - 1], kern, &cfg) != cudaSuccess) {
                (void)cudaGetLastError();
                got[size - 1] = 0;
            }
        }
        if (got[1] < 1) return false;
        for (int i = 0; i < MAX_SPLITS; ++i) known[device][i] = got[i];
    }
    for (int i = 0; i < MAX_SPLITS; ++i) out[i] = known[device][i];
    return true;
}

// The driver's call that points a tensor map at another address; sizes, strides
// and boxes stay.
typedef CUresult (*ReplaceAddressFn)(CUtensorMap*, void*);
inline ReplaceAddressFn replace_address_fn() {
    static ReplaceAddressFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapReplaceAddress", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<ReplaceAddressFn>(ptr);
    });
    return fn;
}

// The problem as a plan's key: sizes, strides, types and alignments; of the
// addresses only what is left over 16 bytes.
inline void keyed_problem(const Problem& p, Problem* key) {
    const auto rest = [](const void* a) { return reinterpret_cast<void*>(reinterpret_cast<uintptr_t>(a) & 15); };
    std::memcpy(key, &p, sizeof(Problem));
    key->x = rest(p.x);
    key->w = rest(p.w);
    key->out = rest(p.out);
    key->start.ptr = key->len.ptr = key->idx.ptr = nullptr;
}

// Points a plan's maps at this call's x and weights.
inline bool point(CUtensorMap* x, int n, CUtensorMap* w, const Problem& p) {
    const ReplaceAddressFn put = replace_address_fn();
    if (!put) return false;
    for (int i = 0; i < n; ++i)
        if (put(&x[i], const_cast<void*>(p.x)) != CUDA_SUCCESS) return false;
    return put(w, const_cast<void*>(p.w)) == CUDA_SUCCESS;
}

// Plans of recent calls, keyed by the problem but for its addresses, the wishes and the device.
inline bool cached_plan(const Problem& p, bool dense, bool early, int lora, int R, bool ring, int segs, int sm_count, int forced_cg,
                        EncodeTiledFn enc, Plan* out) {
    static PlanCache<PlanKey, Plan> cache;
    PlanKey key;
    std::memset(&key, 0, sizeof(key));
    keyed_problem(p, &key.p);
    key.w.dense = dense;
    key.w.early = early;
    key.w.lora = lora;
    key.w.R = R;
    key.w.ring = ring;
    key.w.segs = segs;
    key.w.sm_count = sm_count;
    key.w.forced_cg = forced_cg;
    if (cudaGetDevice(&key.device) != cudaSuccess || !cluster_capacity(key.device, sm_count, key.w.clusters)) return false;
    return cache.get(key, out, [&](Plan* pl) { return make_plan(p, key.w, enc, pl); }) &&
           point(out->xm.m, NUM_XMAPS, &out->wm, p);
}

template <int CG, int LORA>
int launch_kernel(const Plan& pl, const CUtensorMap& bm, const Problem& p, const Lora& lo, cudaStream_t stream) {
    auto kern = gemm_kernel<CG, LORA>;
    static std::atomic<uint64_t> configured{0};
    if (!set_smem_limit_once(kern, SMEM_LIMIT, configured)) return SGMV_ERR_CUDA;
    const int csize = CG == 2 ? 2 : pl.geo.splits;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)csize;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)pl.grid);
    cfg.blockDim = dim3(threads_of(CG, LORA));
    cfg.dynamicSmemBytes = (size_t)pl.smem_bytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = csize > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, pl.xm, pl.wm, bm, p, pl.geo, lo) == cudaSuccess ? SGMV_OK : SGMV_ERR_LAUNCH;
}

template <int LORA>
int launch(const Plan& pl, const CUtensorMap& bm, const Problem& p, const Lora& lo, cudaStream_t stream) {
    return pl.cg == 2 ? launch_kernel<2, LORA>(pl, bm, p, lo, stream) : launch_kernel<1, LORA>(pl, bm, p, lo, stream);
}

// LORA_FMA: a token's 128 rows of B and its row of t are copies of whole 16-byte pieces.
inline bool ring_ok(const Lora& lo) { return lo.b_vec && lo.R % 8 == 0 && lo.R <= RING_MAX_RANK && lo.b_ns == lo.R; }

// Tensor map of lora_b (adapters, N, R) for LORA_MMA; false where TMA cannot read it.
inline bool encode_b(const Lora& lo, int64_t N, int64_t adapters, EncodeTiledFn enc, CUtensorMap* out) {
    if (!enc || !lo.b_vec || lo.b_ns < lo.R || adapters >= (int64_t(1) << 31)) return false;
    if (lo.b_ns >= (int64_t(1) << 38) || lo.b_as >= (int64_t(1) << 38)) return false;
    if (adapters > 1 && lo.b_as < (N - 1) * lo.b_ns + lo.R) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)lo.R, (cuuint64_t)N, (cuuint64_t)adapters};
    const cuuint64_t strides[2] = {(cuuint64_t)(lo.b_ns * 2),
                                   (cuuint64_t)(adapters > 1 ? lo.b_as * 2 : (N * lo.b_ns * 2 + 15) / 16 * 16)};
    const cuuint32_t box[3] = {64, WROWS, 1}, ones[3] = {1, 1, 1};
    return enc(out, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(lo.b), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace grp
}  // namespace sgmv
