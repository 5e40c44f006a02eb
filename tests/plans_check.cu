// Host check (no GPU needed) that the large products' plans exist for every count of rows and segments that the
// tensor-core forms take: up to 4096 segments from four rows a segment on, and millions of rows.  Prints "ok" or a reason.
#include <cuda.h>

#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <random>

#include "common.cuh"

namespace sgmv {
__device__ void raise_device_error(int32_t) {}
namespace tc {
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                  const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
}
}  // namespace sgmv

#include "grouped.cuh"

using namespace sgmv;

static CUresult any_map(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                        const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                        CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    return CUDA_SUCCESS;
}

static bool plan(long rows, long segs, long K, long N, long R, int lora, int out_dt, int forced_cg, grp::Plan* pl) {
    Problem p;
    std::memset(&p, 0, sizeof p);
    grp::Want w;
    std::memset(&w, 0, sizeof w);
    p.x_dt = p.w_dt = SGMV_F16;
    p.out_dt = out_dt;
    p.K = p.x_rs = p.w_ns = K;
    p.N = p.H = N;
    p.x_cs = p.w_ks = 1;
    p.w_as = K * N;
    p.x_rows = p.out_rows = rows;
    p.x = p.w = p.out = reinterpret_cast<void*>(uintptr_t(4096));
    w.dense = lora >= 0;
    w.early = w.dense;
    p.lora_num = w.dense ? 1 : 8;
    p.batches = w.dense ? 0 : segs;
    w.lora = lora < 0 ? (int)grp::LORA_NONE : lora;
    w.R = (int)R;
    w.ring = R % 8 == 0 && R <= grp::RING_MAX_RANK;
    w.segs = w.dense ? (int)segs : 0;
    w.sm_count = 148;
    const int caps[grp::MAX_SPLITS] = {148, 74, 48, 33, 27, 22, 18, 15};
    std::memcpy(w.clusters, caps, sizeof caps);
    w.forced_cg = forced_cg;
    std::memset(pl, 0, sizeof *pl);
    return grp::make_plan(p, w, any_map, pl);
}

#define CHECK(c)                                                                                                      \
    do {                                                                                                              \
        if (!(c)) {                                                                                                   \
            std::printf("line %d: %s: rows %ld segs %ld K %ld N %ld R %ld form %d\n", __LINE__, #c, rows, segs, K, N, \
                        R, pl.cg);                                                                                    \
            return 1;                                                                                                 \
        }                                                                                                             \
    } while (0)

int main() {
    std::mt19937 rng(11);
    auto spread = [&](double lo, double hi) { return (long)(lo * std::pow(hi / lo, rng() / 4294967295.0)); };
    grp::Plan pl;
    for (int it = 0; it < 6000; ++it) {
        const long rows = it % 4 == 0 ? 4 * spread(1024, 4096) : spread(1, 3e6);
        const long most = rows / 4 < 4096 ? rows / 4 : 4096;
        const long segs = it % 4 == 0 ? rows / 4 : most < 1 ? 1 : it % 3 ? spread(1, most) : most;
        const long K = 8 * spread(1, 2048), N = spread(1, 16384), R = 8 * spread(1, 32);
        const int out_dt = it % 2 ? SGMV_F16 : SGMV_F32, forced = it % 5 == 0 ? 2 : 0;
        const bool mma = plan(rows, segs, K, N, R, grp::LORA_MMA, out_dt, forced, &pl);
        // the table of runs: 24 bytes a segment, 16 a token tile
        if (rows <= 400000) CHECK(mma);
        if (mma) {
            CHECK(pl.geo.stages >= 2 && pl.geo.stages <= grp::MAX_STAGES && pl.smem_bytes <= grp::SMEM_LIMIT);
            CHECK(pl.geo.max_runs >= segs + pl.geo.dense_tiles && pl.geo.off_runs >= pl.geo.off_seg);
            CHECK((int64_t)pl.geo.off_bar >= pl.geo.off_runs + (pl.geo.max_runs + segs) * (int64_t)sizeof(grp::Run) +
                                                 (pl.geo.dense_tiles + 1) * 4);
        }
        CHECK(plan(rows, segs, K, N, R, grp::LORA_FMA, out_dt, forced, &pl));   // what such a call runs instead
        CHECK(plan(rows, segs, K, N, 0, -1, out_dt, forced, &pl));
    }
    std::printf("ok\n");
    return 0;
}
