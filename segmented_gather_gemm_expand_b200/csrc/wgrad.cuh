// Weight gradient of the segmented products on the tensor cores:
//
//     dW[e][n, k] = (add ? dW[e][n, k] : 0) + sum over the rows r of index e of dY[r, n] * X[r, k]
//
// The reduction runs over tokens, so both operands are read along their
// contiguous axis (the MMA's "MN-major" form): no transposed copy is made.
// M = X's columns (256 per CTA pair), N = dY's columns (up to 256), 64 tokens
// per stage.  Lanes of the accumulator are k, so 32 lanes store 32 neighbouring
// elements of a row of dW, and a short N (an adapter's rank) costs only itself.
//
// A segment may start and end anywhere.  Its last block issues only the K=16
// steps that hold rows, and the rows past the end in the last of them, which
// belong to another segment (or are anything at all: 0 x NaN is NaN), are
// zeroed in shared memory in both operands by warps of their own (10 to 12, by
// stage) before the MMA sees the stage.
//
// Several segments of one index add up in segment order in one accumulator.
// Indexes without rows get zeros (or keep dW in add mode).  The tiles of long and
// short indexes take turns (longest, shortest, second longest, ...), so that the
// stores of short ones, whose tiles are all epilogue, meet the MMAs of long ones.
//
// Measured: 16384 ragged rows of 8 experts, 4096 x 11008, bf16: 1200-1250 us
// back to back (1200 TFLOP/s, the power limit).  8192 rows of 16 experts, 2048 x
// 2816: 118-124 us by GPU, where the flops alone would take 57.  In an earlier build of
// 104 us on one GPU, 89 were left with no epilogue at all (8 K steps per tile on
// average; the longest cluster has 20 % more than the mean); the other 15 were the
// stores, which share the shared memory's bandwidth with the MMAs' operands and TMA's writes.  18 indexes of 888 x 1528 of
// which one has rows: 22 us, of which the zeros are most (36 by way of the
// epilogue's 64-byte pieces).
#pragma once

#include "grouped.cuh"

namespace sgmv {
namespace wgr {

using namespace sgmv::tc;
using grp::BAND;
using grp::EPI_WARPS;
using grp::TURN;

constexpr int BT = 64;                     // tokens per stage
constexpr int HALF = 64 * BT * 2;          // one box of 64 columns: 8 KB
constexpr int STAGE = 4 * HALF;            // two boxes of X, two of dY
constexpr int FIX_WARP = 2 + EPI_WARPS;
constexpr int FIX_WARPS = 3;
constexpr int WARPS = FIX_WARP + FIX_WARPS;
constexpr int THREADS = 32 * WARPS;
constexpr int SMEM_LIMIT = grp::SMEM_LIMIT;

struct Geo {
    int32_t kblk, nblk, ts;     // tiles along K and N; columns of dY per tile (multiple of 32)
    int32_t stages;
    int32_t off_out, off_seg, off_exp, off_bar;
    int32_t out_vec;            // half dW in 16-byte pieces
    int32_t acc_stride, tmem_cols;
    int64_t rows_per_group;     // rows of dW between two indexes
};

struct Seg {
    int32_t row0, rows, index;  // index -1: nothing to add
    int32_t next;               // next segment of the same index, -1 at the end
};

struct Exp {
    int32_t first;              // first segment, -1 for none
    int32_t rows;               // tokens in all
    int32_t order;              // place in the deal -> index
};

// p: x = X, w = dY (w_ns its row stride), lora_num = number of indexes, out = dW with row stride H and N = X's columns.
__global__ void __launch_bounds__(THREADS, 1)
wgrad_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap ymap, const Problem p, const Geo g) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ int s_abort;
    __shared__ uint32_t s_tmem_base;

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t crank = cluster_rank();
    const int32_t cid = (int32_t)(blockIdx.x / 2), ncl = (int32_t)(gridDim.x / 2);
    const uint32_t S = (uint32_t)g.stages;
    Seg* segs = reinterpret_cast<Seg*>(smem + g.off_seg);
    Exp* exps = reinterpret_cast<Exp*>(smem + g.off_exp);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + g.off_bar);
    uint64_t* empty = full + S;
    uint64_t* part = empty + S;       // a stage whose last rows have to be zeroed has arrived in this CTA
    uint64_t* acc_full = part + S;
    uint64_t* acc_empty = acc_full + 2;

    if (tid == 0) {
        s_abort = 0;
        for (uint32_t i = 0; i < S; ++i) {
            mbar_init(smem_u32(&full[i]), 2);   // two arrivals of the first CTA's producer, or one of each CTA's zeroing warp
            mbar_init(smem_u32(&empty[i]), 1);
            mbar_init(smem_u32(&part[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&acc_full[i]), 1);
            mbar_init(smem_u32(&acc_empty[i]), 2 * EPI_WARPS);
        }
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&xmap);
        prefetch_tmap(&ymap);
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(&s_tmem_base), (uint32_t)g.tmem_cols);

    grid_dependency_wait();
    grid_dependents_launch();

    const int32_t nseg = (int32_t)p.batches, nexp = (int32_t)p.lora_num;
    for (int32_t b = tid; b < nseg; b += THREADS) {
        const Segment s = load_segment(p, b);
        segs[b] = Seg{(int32_t)s.row0, (int32_t)s.rows, s.rows > 0 ? (int32_t)s.adapter : -1, -1};
    }
    __syncthreads();
    // each index's segments as a list, and its rows: a warp per index, a lane per segment
    for (int32_t e = warp; e < nexp; e += WARPS) {
        int32_t first = -1, last = -1, rows = 0;
        for (int32_t b0 = 0; b0 < nseg; b0 += 32) {
            const int32_t b = b0 + lane;
            const bool in = b < nseg && segs[b].index == e;
            const unsigned mask = __ballot_sync(0xffffffffu, in);
            if (!mask) continue;
            rows += __reduce_add_sync(0xffffffffu, in ? segs[b].rows : 0);
            const unsigned after = mask & ~((2u << lane) - 1);
            if (in && after) segs[b].next = b0 + __ffs(after) - 1;
            if (lane == 0 && last >= 0) segs[last].next = b0 + __ffs(mask) - 1;
            if (first < 0) first = b0 + __ffs(mask) - 1;
            last = b0 + 31 - __clz(mask);
        }
        if (lane == 0) {
            exps[e].first = first;
            exps[e].rows = rows;
        }
    }
    __syncthreads();
    for (int32_t e = warp; e < nexp; e += WARPS) {
        const int32_t mine = exps[e].rows;
        int32_t place = 0;   // in descending order of rows
        for (int32_t o0 = 0; o0 < nexp; o0 += 32) {
            const int32_t o = o0 + lane, r = o < nexp ? exps[o].rows : -1;
            place += __popc(__ballot_sync(0xffffffffu, r > mine || (r == mine && o < e)));
        }
        if (lane == 0) exps[2 * place < nexp ? 2 * place : 2 * (nexp - 1 - place) + 1].order = e;
    }
    tc_fence_before();
    cluster_sync();
    __syncthreads();
    tc_fence_after();

    const uint32_t tmem_base = s_tmem_base;
    const int32_t per = g.kblk * g.nblk, total = nexp * per;
    volatile int* abort_flag = &s_abort;
    const bool bf16 = p.w_dt == SGMV_BF16;
    const uint32_t hs = (uint32_t)g.ts / 2;   // dY columns of this CTA

    // tile id -> index, first column of X, first column of dY
    auto decode = [&](int32_t id, int32_t& e, int32_t& k0, int32_t& n0) {
        const int32_t o = id / per, local = id - o * per;
        e = exps[o].order;
        const int32_t band = local / (BAND * g.kblk), in_band = min(BAND, g.nblk - band * BAND);
        const int32_t r = local - band * BAND * g.kblk;
        n0 = (band * BAND + r % in_band) * g.ts;
        k0 = (r / in_band) * 256;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (elect_one()) {
            const uint64_t pol = policy_evict_normal();
            const int nybox = hs > 64 ? 2 : 1;
            const uint32_t bytes = (uint32_t)(2 + nybox) * HALF;
            uint32_t s = 0, phase = 1;
            bool ok = true;
            for (int32_t id = cid; ok && id < total; id += ncl) {
                int32_t e, k0, n0;
                decode(id, e, k0, n0);
                k0 += (int32_t)crank * 128;
                n0 += (int32_t)(crank * hs);
                for (int32_t b = exps[e].first; ok && b >= 0; b = segs[b].next) {
                    const Seg sg = segs[b];
                    for (int32_t r = 0; r < sg.rows; r += BT) {
                        if (!mbar_wait(smem_u32(&empty[s]), phase, abort_flag, DEVERR_TIMEOUT_PRODUCER)) {
                            ok = false;
                            break;
                        }
                        const uint32_t xs = smem_u32(smem + s * STAGE), ys = xs + 2 * HALF;
                        const bool partial = sg.rows - r < BT && (sg.rows - r) % 16 != 0;
                        // a stage to be zeroed first arrives at this CTA's own barrier
                        uint32_t bar = smem_u32(&part[s]);
                        if (partial) {
                            mbar_expect_tx(bar, bytes);
                        } else {
                            bar = map_to_rank(smem_u32(&full[s]), 0);
                            if (crank == 0) {
                                mbar_expect_tx(smem_u32(&full[s]), 2 * bytes);
                                mbar_arrive(smem_u32(&full[s]));
                            }
                        }
                        for (int i = 0; i < 2; ++i)
                            tma_load_2d_pair(xs + i * HALF, &xmap, k0 + i * 64, sg.row0 + r, bar, pol);
                        for (int i = 0; i < nybox; ++i)
                            tma_load_2d_pair(ys + i * HALF, &ymap, n0 + i * 64, sg.row0 + r, bar, pol);
                        if (++s == S) {
                            s = 0;
                            phase ^= 1;
                        }
                    }
                }
            }
            // the commits of the other CTA's MMAs arrive here: none may be under way when this CTA ends
            for (uint32_t i = 0; ok && i < S; ++i) {
                ok = mbar_wait(smem_u32(&empty[s]), phase, abort_flag, DEVERR_TIMEOUT_PRODUCER);
                if (++s == S) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA (the pair's first CTA)
        if (crank == 0 && elect_one()) {
            const uint32_t idesc = instr_desc_mn(bf16, 256, g.ts) | IDESC_A_MN | IDESC_B_MN;
            // 64-column boxes are HALF apart, 8-token groups 1024 bytes; a K step is 16 tokens
            const uint64_t ad0 = smem_desc(smem_u32(smem), HALF, 1024, 2);
            const uint64_t bd0 = smem_desc(smem_u32(smem) + 2 * HALF, HALF, 1024, 2);
            uint32_t s = 0, phase = 0, n = 0;
            bool ok = true;
            for (int32_t id = cid; ok && id < total; id += ncl, ++n) {
                int32_t e, k0, n0;
                decode(id, e, k0, n0);
                const uint32_t acc = n & 1;
                const uint32_t d = tmem_base + acc * (uint32_t)g.acc_stride;
                if (!mbar_wait(smem_u32(&acc_empty[acc]), ((n >> 1) & 1) ^ 1, abort_flag, DEVERR_TIMEOUT_MMA)) break;
                tc_fence_after();
                uint32_t more = 0;
                for (int32_t b = exps[e].first; ok && b >= 0; b = segs[b].next) {
                    const int32_t rows = segs[b].rows;
                    for (int32_t r = 0; r < rows; r += BT) {
                        // a segment's end: the other CTA's warps have zeroed rows of this stage
                        const bool zeroed = rows - r < BT && (rows - r) % 16 != 0;
                        ok = zeroed ? mbar_wait_cluster(smem_u32(&full[s]), phase, abort_flag, DEVERR_TIMEOUT_MMA)
                                    : mbar_wait(smem_u32(&full[s]), phase, abort_flag, DEVERR_TIMEOUT_MMA);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t ad = ad0 + s * (uint64_t)(STAGE >> 4), bd = bd0 + s * (uint64_t)(STAGE >> 4);
                        const int steps = (rows - r + 15) / 16;   // K steps that hold rows
#pragma unroll
                        for (int kk = 0; kk < BT / 16; ++kk) {
                            if (kk < steps) tc_mma_pair(d, ad + kk * 128, bd + kk * 128, idesc, more);
                            more = 1;
                        }
                        tc_commit_pair(smem_u32(&empty[s]));
                        if (++s == S) {
                            s = 0;
                            phase ^= 1;
                        }
                    }
                }
                if (!ok) break;
                tc_commit_pair(smem_u32(&acc_full[acc]));
            }
        }
        __syncwarp();
    } else if (warp >= FIX_WARP) {
        // ------------------------------------------------------------ rows past a segment's end
        uint32_t q = 0, phase = 0;   // phase: one bit per stage (at most 32 stages)
        bool ok = true;
        for (int32_t id = cid; ok && id < total; id += ncl) {
            int32_t e, k0, n0;
            decode(id, e, k0, n0);
            for (int32_t b = exps[e].first; ok && b >= 0; b = segs[b].next) {
                const int32_t rows = segs[b].rows, blocks = (rows + BT - 1) / BT;
                const int32_t rem = rows - (blocks - 1) * BT;
                q += (uint32_t)blocks;
                if (rem % 16 == 0) continue;   // whole K steps (or a whole block)
                const uint32_t s = (q - 1) % S;
                if (s % FIX_WARPS != (uint32_t)(warp - FIX_WARP)) continue;   // a stage has one warp: it sees every phase
                if (!warp_wait(smem_u32(&part[s]), (phase >> s) & 1, abort_flag, DEVERR_TIMEOUT_CONVERT)) {
                    ok = false;
                    break;
                }
                phase ^= 1u << s;
                const int32_t bytes = ((rem + 15) / 16 * 16 - rem) * 128;
                for (int i = 0; i < (hs > 64 ? 4 : 3); ++i)
                    for (int32_t o = lane * 16; o < bytes; o += 512)
                        *reinterpret_cast<uint4*>(smem + s * STAGE + i * HALF + rem * 128 + o) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (crank == 0) mbar_arrive(smem_u32(&full[s]));
                    else mbar_arrive_cluster(map_to_rank(smem_u32(&full[s]), 0));
                }
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int quad = warp % 4, half = (warp - 2) / 4;
        uint32_t* stage = reinterpret_cast<uint32_t*>(smem + g.off_out + (warp - 2) * TURN);
        uint32_t n = 0;
        for (int32_t id = cid; id < total; id += ncl, ++n) {
            int32_t e, k0, n0;
            decode(id, e, k0, n0);
            const uint32_t acc = n & 1;
            const int64_t col = k0 + (int32_t)crank * 128 + quad * 32 + lane;
            const bool any = exps[e].first >= 0;
            const int32_t valid = min(g.ts, (int32_t)p.K - n0);   // p.K: dY's columns
            if (!warp_wait(smem_u32(&acc_full[acc]), (n >> 1) & 1, abort_flag, DEVERR_TIMEOUT_EPILOGUE)) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + acc * (uint32_t)g.acc_stride + ((uint32_t)(quad * 32) << 16);
            const auto drained = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && id + 2 * ncl < total) mbar_arrive_remote(map_to_rank(smem_u32(&acc_empty[acc]), 0));
            };
            const int64_t row0 = (int64_t)e * g.rows_per_group + n0;
            if (any) {
                grp::drain<false>(taddr, half, g.ts, row0, valid, col, 0.f, p, stage, g.out_vec, drained);
            } else {
                drained();
                if (g.out_vec && !p.add) {
                    // zeros: 16 lanes write a row's 128 columns, a warp two rows at a time
                    const int64_t k = k0 + (int32_t)crank * 128 + lane % 16 * 8;
                    uint16_t* o = static_cast<uint16_t*>(p.out) + row0 * p.H + k;
                    if (k < p.N)
#pragma unroll 4
                        for (int c = (warp - 2) * 2 + lane / 16; c < valid; c += 2 * EPI_WARPS)
                            *reinterpret_cast<uint4*>(o + c * p.H) = make_uint4(0, 0, 0, 0);
                } else {
#pragma unroll 1
                    for (int c = half * 8; c < valid && !p.add; c += 16) {
                        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                        grp::put8(v, row0 + c, min(8, valid - c), col, p, stage, g.out_vec);
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    outlast_copies(abort_flag);
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem_base, (uint32_t)g.tmem_cols);
}

// Generic form on the CUDA cores: any strides, alignment and dtypes.  A CTA
// owns 32 x 64 elements of one index's dW and adds the rows in segment order.
constexpr int SIMT_N = 32, SIMT_K = 64;
__global__ void __launch_bounds__(256) wgrad_simt_kernel(Problem p, int64_t y_cs, int64_t out_gs, int64_t out_cs) {
    const int64_t k = (int64_t)blockIdx.x * SIMT_K + threadIdx.x % SIMT_K;
    const int64_t n0 = (int64_t)blockIdx.y * SIMT_N + threadIdx.x / SIMT_K;
    for (int64_t e = blockIdx.z; e < p.lora_num; e += gridDim.z) {
        float acc[SIMT_N / 4];
#pragma unroll
        for (int i = 0; i < SIMT_N / 4; ++i) acc[i] = 0.f;
        bool any = false;
        for (int64_t b = 0; b < p.batches; ++b) {
            const Segment s = load_segment(p, b);
            if (s.rows == 0 || s.adapter != e) continue;
            any = true;
            for (int64_t r = s.row0; r < s.row0 + s.rows; ++r) {
                const float xv = k < p.N ? load_elem(p.x, p.x_dt, r * p.x_rs + k * p.x_cs) : 0.f;
#pragma unroll
                for (int i = 0; i < SIMT_N / 4; ++i)
                    if (n0 + 4 * i < p.K)
                        acc[i] = fmaf(load_elem(p.w, p.w_dt, r * p.w_ns + (n0 + 4 * i) * y_cs), xv, acc[i]);
            }
        }
        if (k >= p.N || (p.add && !any)) continue;
#pragma unroll
        for (int i = 0; i < SIMT_N / 4; ++i) {
            if (n0 + 4 * i >= p.K) continue;
            const int64_t at = e * out_gs + (n0 + 4 * i) * p.H + k * out_cs;
            store_elem(p.out, p.out_dt, at, p.add ? load_elem(p.out, p.out_dt, at) + acc[i] : acc[i]);
        }
    }
}

// ====================================================================== host side

struct Plan {
    Geo geo;
    CUtensorMap xm, ym;
    int smem_bytes;
    int grid;
};

inline bool supports(const Problem& p, int64_t y_cs, int64_t out_gs, int64_t out_cs) {
    if (p.x_dt != p.w_dt || p.x_dt == SGMV_F32 || p.K < 1 || p.N < 1) return false;
    if (p.x_cs != 1 || y_cs != 1 || out_cs != 1) return false;
    if ((p.x_rs * 2) % 16 || (p.w_ns * 2) % 16 || p.x_rs < p.N || p.w_ns < p.K) return false;
    if ((reinterpret_cast<uintptr_t>(p.x) & 15) || (reinterpret_cast<uintptr_t>(p.w) & 15)) return false;
    if (p.lora_num > 1 && out_gs % p.H) return false;
    const int64_t lim = int64_t(1) << 31;
    if (p.K >= lim || p.N >= lim || p.x_rows >= lim || p.out_rows >= lim || p.x_rows < 1 || p.out_rows < 1) return false;
    if (p.x_rs >= (int64_t(1) << 38) || p.w_ns >= (int64_t(1) << 38)) return false;
    if (p.batches > grp::SEG_CAP || p.lora_num > grp::SEG_CAP) return false;
    return p.lora_num * ((p.N + 255) / 256) * ((p.K + 31) / 32 + 1) < lim;
}

inline bool make_plan(const Problem& p, int64_t y_cs, int64_t out_gs, int64_t out_cs, int sm_count, EncodeTiledFn enc,
                      Plan* out) {
    if (!supports(p, y_cs, out_gs, out_cs) || !enc) return false;
    Geo& g = out->geo;
    g.kblk = (int32_t)((p.N + 255) / 256);
    const int64_t nt = (p.K + 255) / 256;
    g.ts = (int32_t)(((p.K + nt - 1) / nt + 31) / 32 * 32);
    g.nblk = (int32_t)((p.K + g.ts - 1) / g.ts);
    g.rows_per_group = p.lora_num > 1 ? out_gs / p.H : 0;
    g.out_vec = grp::out_vec_ok(p);
    g.acc_stride = g.ts;
    g.tmem_cols = 32;
    while (g.tmem_cols < 2 * g.acc_stride) g.tmem_cols *= 2;
    for (g.stages = 7; g.stages >= 2; --g.stages) {
        g.off_out = g.stages * STAGE;
        g.off_seg = g.off_out + EPI_WARPS * TURN;
        g.off_exp = g.off_seg + (int)p.batches * (int)sizeof(Seg);
        g.off_bar = (g.off_exp + (int)p.lora_num * (int)sizeof(Exp) + 15) & ~15;
        out->smem_bytes = g.off_bar + 8 * (3 * g.stages + 4) + 1024;
        if (out->smem_bytes <= SMEM_LIMIT) break;
    }
    if (g.stages < 2) return false;
    const cuuint32_t ones[2] = {1, 1};
    const cuuint32_t box[2] = {64, BT};
    const cuuint64_t xd[2] = {(cuuint64_t)p.N, (cuuint64_t)p.x_rows}, yd[2] = {(cuuint64_t)p.K, (cuuint64_t)p.out_rows};
    const cuuint64_t xs[1] = {(cuuint64_t)(p.x_rs * 2)}, ys[1] = {(cuuint64_t)(p.w_ns * 2)};
    if (enc(&out->xm, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(p.x), xd, xs, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return false;
    if (enc(&out->ym, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(p.w), yd, ys, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return false;
    const int64_t tiles = p.lora_num * g.kblk * g.nblk;
    int64_t clusters = sm_count / 2;
    if (tiles < clusters) clusters = tiles;
    out->grid = (int)(clusters < 1 ? 1 : clusters) * 2;
    return true;
}

struct PlanKey {
    Problem p;
    int64_t y_cs, out_gs, out_cs;
    int32_t device, sm_count;
};

inline bool cached_plan(const Problem& p, int64_t y_cs, int64_t out_gs, int64_t out_cs, int sm_count, EncodeTiledFn enc,
                        Plan* out) {
    static PlanCache<PlanKey, Plan> cache;
    PlanKey key;
    std::memset(&key, 0, sizeof(key));
    grp::keyed_problem(p, &key.p);
    key.y_cs = y_cs;
    key.out_gs = out_gs;
    key.out_cs = out_cs;
    key.sm_count = sm_count;
    if (cudaGetDevice(&key.device) != cudaSuccess) return false;
    return cache.get(key, out, [&](Plan* pl) { return make_plan(p, y_cs, out_gs, out_cs, sm_count, enc, pl); }) &&
           grp::point(&out->xm, 1, &out->ym, p);
}

inline int launch(const Plan& pl, const Problem& p, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    if (!set_smem_limit_once(wgrad_kernel, SMEM_LIMIT, configured)) return SGMV_ERR_CUDA;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)pl.grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = (size_t)pl.smem_bytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, wgrad_kernel, pl.xm, pl.ym, p, pl.geo) == cudaSuccess ? SGMV_OK : SGMV_ERR_LAUNCH;
}

inline int launch_simt(const Problem& p, int64_t y_cs, int64_t out_gs, int64_t out_cs, cudaStream_t stream) {
    const int64_t gx = (p.N + SIMT_K - 1) / SIMT_K, gy = (p.K + SIMT_N - 1) / SIMT_N;
    if (gx > 0x7fffffff || gy > 65535) return SGMV_ERR_TOO_LARGE;
    dim3 grid((unsigned)gx, (unsigned)gy, (unsigned)(p.lora_num < 65535 ? p.lora_num : 65535));
    wgrad_simt_kernel<<<grid, 256, 0, stream>>>(p, y_cs, out_gs, out_cs);
    return cudaGetLastError() == cudaSuccess ? SGMV_OK : SGMV_ERR_LAUNCH;
}

}  // namespace wgr
}  // namespace sgmv
