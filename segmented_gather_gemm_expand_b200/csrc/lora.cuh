// The small kernels beside a shared projection with adapters: which adapter a
// row has, its low-rank input t = x A^T for few rows, and the generic form of
// the whole projection.
#pragma once

#include "common.cuh"
#include "grouped.cuh"
#include "tc_ptx.cuh"

namespace sgmv {
namespace lora {

// Adapter of `row` (-1: none), found by the whole block; segments do not overlap.
__device__ __forceinline__ int32_t block_adapter(const Problem& p, int64_t row, int64_t rows, int32_t* s_adapter) {
    // a decode batch has one token per segment, in order: look there first
    if (row < p.batches) {
        const Segment s = load_segment(p, row);
        if (s.rows > 0 && row >= s.row0 && row < s.row0 + s.rows) return (int32_t)s.adapter;
    }
    // else around the place that segments of one length would give it, then everywhere
    if (threadIdx.x == 0) *s_adapter = -1;
    __syncthreads();
    int64_t b = threadIdx.x;
    if (p.batches > blockDim.x) b += row * p.batches / rows - (int64_t)(blockDim.x / 2);
    if (b < 0) b += p.batches;
    for (int64_t left = p.batches; left > 0; left -= blockDim.x, b += blockDim.x) {
        if (b >= p.batches) b -= p.batches;
        bool found = false;
        if (threadIdx.x < left) {
            const Segment s = load_segment(p, b);
            found = s.rows > 0 && row >= s.row0 && row < s.row0 + s.rows;
            if (found) *s_adapter = (int32_t)s.adapter;
        }
        if (__syncthreads_or(found)) break;
    }
    const int32_t a = *s_adapter;
    __syncthreads();   // read by all before the next row's search
    return a;
}

// The adapter of every row: one thread per row scans the segments, which the
// block stages in shared memory 256 at a time.
constexpr int ROWS_THREADS = 256;
__global__ void __launch_bounds__(ROWS_THREADS) row_adapter_kernel(Problem p, int32_t* row_adapter, int64_t rows) {
    __shared__ Segment s_seg[ROWS_THREADS];
    tc::grid_dependency_wait();
    tc::grid_dependents_launch();
    const int tid = threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x * ROWS_THREADS + tid;
    int32_t a = -1;
    for (int64_t base = 0; base < p.batches; base += ROWS_THREADS) {
        __syncthreads();
        if (base + tid < p.batches) s_seg[tid] = load_segment(p, base + tid);
        __syncthreads();
        const int n = (int)min((int64_t)ROWS_THREADS, p.batches - base);
        for (int i = 0; i < n; ++i)
            if (row >= s_seg[i].row0 && row < s_seg[i].row0 + s_seg[i].rows) a = (int32_t)s_seg[i].adapter;
    }
    if (row < rows) row_adapter[row] = a;
}

// t[row, j] = sum_k x^[row, k] * A[a][j, k] in fp32 for four ranks per block;
// also writes row_adapter.  Bound by A's bytes (a decode batch uses each
// adapter once; 256 rows x 32 ranks x 5120: 84 MB in 21 us) and, for one row, by
// latency (3 us): the block's threads cover 2048 columns at once, so the loads of
// a 4096-wide row are all in flight together.  A warp per two ranks without
// blocks took 28 us for the 256 rows.
// p: x, w = A (N = rank), the call's segments.
constexpr int SHRINK_THREADS = 256;
constexpr int SHRINK_RANKS = 4;
template <bool VEC>
__global__ void __launch_bounds__(SHRINK_THREADS) row_shrink_kernel(Problem p, float* t, int32_t* row_adapter, int64_t rows) {
    __shared__ int32_t s_adapter;
    __shared__ float s_sum[SHRINK_THREADS / 32][SHRINK_RANKS];
    tc::grid_dependency_wait();
    tc::grid_dependents_launch();
    const int tid = threadIdx.x;
    const int64_t j0 = (int64_t)blockIdx.x * SHRINK_RANKS;
    const bool bf16 = p.w_dt == SGMV_BF16;
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const int32_t a = block_adapter(p, row, rows, &s_adapter);
        if (blockIdx.x == 0 && tid == 0) row_adapter[row] = a;
        if (a >= 0) {
            float acc[SHRINK_RANKS] = {0.f, 0.f, 0.f, 0.f};
            const int64_t wbase = (int64_t)a * p.w_as;
            if (VEC) {
                const uint16_t* xr = static_cast<const uint16_t*>(p.x) + row * p.x_rs;
                const uint16_t* ar = static_cast<const uint16_t*>(p.w) + wbase + j0 * p.w_ns;
#pragma unroll 2
                for (int64_t k = (int64_t)tid * 8; k < p.K; k += SHRINK_THREADS * 8) {
                    const uint4 xu = *reinterpret_cast<const uint4*>(xr + k);
                    uint4 au[SHRINK_RANKS];
#pragma unroll
                    for (int j = 0; j < SHRINK_RANKS; ++j)
                        au[j] = j0 + j < p.N ? __ldg(reinterpret_cast<const uint4*>(ar + j * p.w_ns + k))
                                             : make_uint4(0, 0, 0, 0);
                    const uint32_t xw[4] = {xu.x, xu.y, xu.z, xu.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 xf = tc::unpack2(xw[i], bf16);
#pragma unroll
                        for (int j = 0; j < SHRINK_RANKS; ++j) {
                            const uint32_t aw = i == 0 ? au[j].x : i == 1 ? au[j].y : i == 2 ? au[j].z : au[j].w;
                            const float2 af = tc::unpack2(aw, bf16);
                            acc[j] = fmaf(xf.x, af.x, acc[j]);
                            acc[j] = fmaf(xf.y, af.y, acc[j]);
                        }
                    }
                }
            } else {
                for (int64_t k = tid; k < p.K; k += SHRINK_THREADS) {
                    const float xv = round_to(load_elem(p.x, p.x_dt, row * p.x_rs + k * p.x_cs), p.w_dt);
#pragma unroll
                    for (int j = 0; j < SHRINK_RANKS; ++j)
                        if (j0 + j < p.N)
                            acc[j] = fmaf(xv, load_elem(p.w, p.w_dt, wbase + (j0 + j) * p.w_ns + k * p.w_ks), acc[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < SHRINK_RANKS; ++j) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
                if (tid % 32 == 0) s_sum[tid / 32][j] = acc[j];
            }
            __syncthreads();
            if (tid < SHRINK_RANKS && j0 + tid < p.N) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < SHRINK_THREADS / 32; ++w) v += s_sum[w][tid];
                t[row * p.N + j0 + tid] = v;
            }
        }
        __syncthreads();   // s_adapter and s_sum are free for the next row
    }
}

inline bool row_shrink_vec(const Problem& p) {
    return p.x_dt == p.w_dt && p.x_cs == 1 && p.w_ks == 1 && p.K % 8 == 0 && (p.x_rs * 2) % 16 == 0 &&
           (p.w_ns * 2) % 16 == 0 && (p.lora_num <= 1 || (p.w_as * 2) % 16 == 0) &&
           (reinterpret_cast<uintptr_t>(p.x) & 15) == 0 && (reinterpret_cast<uintptr_t>(p.w) & 15) == 0;
}

// B with its ranks contiguous, rows padded to whole 16-byte pieces: out[i][n][j],
// j < pitch.  i: a segment, whose adapter's B it is (by_seg), or an adapter,
// whichever are fewer.  A thread takes a row of B, eight ranks at a time;
// neighbouring threads take neighbouring rows, which is how a transposed view
// lies in memory.  Segments without rows and adapters without segments are left out.
constexpr int PACK_THREADS = 256;
__global__ void __launch_bounds__(PACK_THREADS) pack_b_kernel(Problem p, grp::Lora lo, uint16_t* out, int64_t N, int32_t pitch,
                                                              bool by_seg) {
    tc::grid_dependency_wait();
    tc::grid_dependents_launch();
    int64_t adapter = blockIdx.y;
    bool used = false;
    if (by_seg) {
        const Segment s = load_segment(p, blockIdx.y);
        used = s.rows > 0;
        adapter = s.adapter;
    } else {
        for (int64_t b = threadIdx.x; b < p.batches && !used; b += PACK_THREADS) {
            const Segment s = load_segment(p, b);
            used = s.rows > 0 && s.adapter == adapter;
        }
        used = __syncthreads_or(used);
    }
    const int64_t n = (int64_t)blockIdx.x * PACK_THREADS + threadIdx.x;
    if (!used || n >= N) return;
    const uint16_t* b = static_cast<const uint16_t*>(lo.b) + adapter * lo.b_as + n * lo.b_ns;
    uint16_t* o = out + ((int64_t)blockIdx.y * N + n) * pitch;
    for (int32_t j0 = 0; j0 < pitch; j0 += 8) {
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j0 + j < lo.R ? b[(j0 + j) * lo.b_ks] : 0u;
        *reinterpret_cast<uint4*>(o + j0) = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
}

// Generic form of the whole projection on the CUDA cores: any strides, rank,
// alignment and dtypes.  Tiling as in the generic expand: a CTA of 256 threads
// owns 128 columns and 32 rows at a time, x and W staged as fp32 in chunks of
// 32 along K; the low-rank part is added from t per element.
constexpr int ST = 256, SN = 128, SR = 32, SK = 32;
__global__ void __launch_bounds__(ST) lora_linear_simt_kernel(Problem p, grp::Lora lo, int64_t rows) {
    __shared__ float sW[SK][SN];
    __shared__ float sX[SR][SK + 1];
    const int tid = threadIdx.x, col = tid % SN, phase = tid / SN;
    const int64_t n0 = (int64_t)blockIdx.x * SN, n = n0 + col;
    for (int64_t c0 = (int64_t)blockIdx.y * SR; c0 < rows; c0 += (int64_t)gridDim.y * SR) {
        const int here = (int)min((int64_t)SR, rows - c0);
        float acc[SR / 2];
#pragma unroll
        for (int i = 0; i < SR / 2; ++i) acc[i] = 0.f;
        for (int64_t kc = 0; kc < p.K; kc += SK) {
            __syncthreads();
            for (int i = tid; i < SK * SN; i += ST) {
                const int kk = i / SN, nn = i % SN;
                sW[kk][nn] = kc + kk < p.K && n0 + nn < p.N
                                 ? load_elem(p.w, p.w_dt, (n0 + nn) * p.w_ns + (kc + kk) * p.w_ks)
                                 : 0.f;
            }
            for (int i = tid; i < SR * SK; i += ST) {
                const int rr = i / SK, kk = i % SK;
                sX[rr][kk] = rr < here && kc + kk < p.K
                                 ? round_to(load_elem(p.x, p.x_dt, (c0 + rr) * p.x_rs + (kc + kk) * p.x_cs), p.w_dt)
                                 : 0.f;
            }
            __syncthreads();
            const int kmax = (int)min((int64_t)SK, p.K - kc);
            for (int kk = 0; kk < kmax; ++kk) {
                const float wv = sW[kk][col];
#pragma unroll
                for (int i = 0; i < SR / 2; ++i) acc[i] = fmaf(sX[phase + 2 * i][kk], wv, acc[i]);
            }
        }
        if (n < p.N) {
            const float bias = lo.bias ? load_elem(lo.bias, p.w_dt, n * lo.bias_s) : 0.f;
#pragma unroll
            for (int i = 0; i < SR / 2; ++i) {
                const int rr = phase + 2 * i;
                if (rr >= here) continue;
                const int64_t r = c0 + rr;
                float v = 0.f;
                const int32_t a = lo.R > 0 ? lo.row_adapter[r] : -1;
                if (a >= 0)
                    for (int j = 0; j < lo.R; ++j)
                        v = fmaf(lo.t[r * lo.R + j],
                                 load_elem(lo.b, p.w_dt, (int64_t)a * lo.b_as + n * lo.b_ns + j * lo.b_ks), v);
                store_elem(p.out, p.out_dt, r * p.H + n, acc[i] + v + bias);
            }
        }
    }
}

template <class... KArgs, class... Args>
int launch_dependent(void (*kern)(KArgs...), dim3 grid, int threads, cudaStream_t stream, Args... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, KArgs(args)...) == cudaSuccess ? SGMV_OK : SGMV_ERR_LAUNCH;
}

inline int launch_row_adapter(const Problem& p, int32_t* row_adapter, int64_t rows, cudaStream_t stream) {
    const int64_t blocks = (rows + ROWS_THREADS - 1) / ROWS_THREADS;
    return launch_dependent(row_adapter_kernel, dim3((unsigned)blocks), ROWS_THREADS, stream, p, row_adapter, rows);
}

inline int launch_row_shrink(const Problem& p, float* t, int32_t* row_adapter, int64_t rows, cudaStream_t stream) {
    const int64_t gx = (p.N + SHRINK_RANKS - 1) / SHRINK_RANKS;
    if (gx > 0x7fffffff) return SGMV_ERR_TOO_LARGE;
    const dim3 grid((unsigned)gx, (unsigned)(rows < 65535 ? rows : 65535));
    return row_shrink_vec(p)
               ? launch_dependent(row_shrink_kernel<true>, grid, SHRINK_THREADS, stream, p, t, row_adapter, rows)
               : launch_dependent(row_shrink_kernel<false>, grid, SHRINK_THREADS, stream, p, t, row_adapter, rows);
}

// The caller's lora_b (`given`) into the place and layout of `packed`.
inline int launch_pack_b(const Problem& p, const grp::Lora& given, const grp::Lora& packed, int64_t N, cudaStream_t stream) {
    const int64_t gx = (N + PACK_THREADS - 1) / PACK_THREADS;
    return launch_dependent(pack_b_kernel, dim3((unsigned)gx, (unsigned)(packed.by_seg ? p.batches : p.lora_num)), PACK_THREADS,
                            stream, p, given, const_cast<uint16_t*>(static_cast<const uint16_t*>(packed.b)), N,
                            (int32_t)packed.b_ns, packed.by_seg != 0);
}

inline int launch_lora_simt(const Problem& p, const grp::Lora& lo, int64_t rows, cudaStream_t stream) {
    const int64_t gx = (p.N + SN - 1) / SN, gy = (rows + SR - 1) / SR;
    if (gx > 0x7fffffff) return SGMV_ERR_TOO_LARGE;
    lora_linear_simt_kernel<<<dim3((unsigned)gx, (unsigned)(gy < 65535 ? gy : 65535)), ST, 0, stream>>>(p, lo, rows);
    return cudaGetLastError() == cudaSuccess ? SGMV_OK : SGMV_ERR_LAUNCH;
}

}  // namespace lora
}  // namespace sgmv
