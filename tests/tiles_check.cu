// Host check of the large products' tiling (grouped.cuh, no GPU needed): for
// random segment tables the tiles cover every row and column of every segment
// exactly once, and every plan that the cost model can pick fits the device:
// shared memory in order and within the limit, TMEM columns, box and MMA sizes,
// and the MMA's reads inside the CTA's shared memory.  Prints "ok" or a reason.
#include <cuda.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <atomic>
#include <random>
#include <vector>

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

static const char* g_bad = nullptr;
static CUresult check_map(CUtensorMap*, CUtensorMapDataType, cuuint32_t rank, void* base, const cuuint64_t* dims,
                          const cuuint64_t* strides, const cuuint32_t* box, const cuuint32_t*, CUtensorMapInterleave,
                          CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    if ((uintptr_t)base % 16) g_bad = "map base";
    for (cuuint32_t i = 0; i < rank; ++i) {
        if (dims[i] < 1 || dims[i] > (cuuint64_t(1) << 32)) g_bad = "map extent";
        if (box[i] < 1 || box[i] > 256) g_bad = "map box";
    }
    for (cuuint32_t i = 0; i + 1 < rank; ++i)
        if (strides[i] % 16 || strides[i] >= (cuuint64_t(1) << 40)) g_bad = "map stride";
    if (box[0] * 2 != 128) g_bad = "map box width";
    return CUDA_SUCCESS;
}

#define CHECK(c)                                          \
    do {                                                  \
        if (!(c)) {                                       \
            std::printf("line %d: %s\n", __LINE__, #c);   \
            return 1;                                     \
        }                                                 \
    } while (0)

int main() {
    std::mt19937 rng(7);
    auto pick = [&](long lo, long hi) { return lo + (long)(rng() % (unsigned long)(hi - lo + 1)); };
    const int caps[grp::MAX_SPLITS] = {148, 74, 48, 33, 27, 22, 18, 15};
    for (int it = 0; it < 4000; ++it) {
        Problem p;
        std::memset(&p, 0, sizeof p);
        grp::Want w;
        std::memset(&w, 0, sizeof w);
        const bool dense = it % 2;
        p.x_dt = p.w_dt = SGMV_BF16;
        p.out_dt = it % 3 ? SGMV_BF16 : SGMV_F32;
        p.K = 8 * pick(1, it % 5 ? 700 : 8);
        p.N = it % 7 ? pick(1, 13000) : pick(1, 40);
        p.H = p.N;
        p.x_cs = 1;
        p.x_rs = p.K;
        const bool turned = !dense && p.N % 8 == 0 && it % 4 == 0;
        p.w_ks = turned ? p.N : 1;
        p.w_ns = turned ? 1 : p.K;
        p.w_as = p.K * p.N;
        p.lora_num = dense ? 1 : pick(1, 64);
        if (p.lora_num > 1 && (p.w_as * 2) % 16) continue;
        p.x_rows = p.out_rows = it % 3 == 0 ? pick(1, 300) : pick(1, 20000);
        p.batches = dense ? 0 : pick(1, it % 11 ? 300 : 4096);
        p.x = p.w = p.out = reinterpret_cast<void*>(uintptr_t(4096));
        w.dense = dense;
        w.early = dense;
        w.lora = dense ? (int)pick(0, 2) : (int)grp::LORA_NONE;
        w.R = w.lora == grp::LORA_NONE ? 0 : 8 * (int)pick(1, 16);
        w.ring = w.R > 0 && w.R <= grp::RING_MAX_RANK;
        w.segs = w.lora == grp::LORA_MMA ? (int)(p.x_rows / 16 < 1 ? 1 : p.x_rows / 16 > 4096 ? 4096 : p.x_rows / 16) : 0;
        w.sm_count = 148;
        std::memcpy(w.clusters, caps, sizeof caps);
        w.forced_cg = it % 9 == 0 ? 2 : 0;
        grp::Plan pl;
        std::memset(&pl, 0, sizeof pl);
        g_bad = nullptr;
        CHECK(grp::make_plan(p, w, check_map, &pl));
        if (g_bad) {
            std::printf("%s\n", g_bad);
            return 1;
        }
        const grp::Geo& g = pl.geo;
        CHECK(pl.smem_bytes <= grp::SMEM_LIMIT && g.stages >= 2 && g.stages <= 32);
        CHECK(g.stage_bytes % 1024 == 0 && g.off_t == g.stages * g.stage_bytes && g.off_t <= g.off_out && g.off_out <= g.off_red &&
              g.off_red <= g.off_seg && g.off_seg <= g.off_runs && g.off_runs <= g.off_bar && g.off_bar % 8 == 0);
        CHECK(g.tn / pl.cg * 128 + grp::W_TILE == g.stage_bytes);
        CHECK(g.tmem_cols <= 512 && 2 * g.acc_stride + (w.lora == grp::LORA_FMA ? g.tn : 0) <= g.tmem_cols);
        CHECK(pl.grid % (pl.cg == 2 ? 2 : g.splits) == 0 && g.splits <= g.kblocks);
        // tiles
        std::vector<grp::Seg> segs;
        std::vector<int> owner((size_t)p.x_rows, -1);
        const int step = 16 * pl.cg;
        int prefix = 0;
        if (!dense) {
            long at = 0;
            for (long b = 0; b < p.batches; ++b) {
                at += pick(0, 2);
                long rows = b % 6 == 0 ? 0 : pick(0, 2 * p.x_rows / p.batches + 2);
                if (at + rows > p.x_rows) rows = at < p.x_rows ? p.x_rows - at : 0;
                const int nt = (int)((rows + g.tn - 1) / g.tn);
                const int ts = nt > 0 ? (int)(((rows + nt - 1) / nt + step - 1) / step * step) : step;
                segs.push_back(grp::Seg{(int32_t)at, (int32_t)rows, (int32_t)b, ts, prefix});
                prefix += (int)((rows + ts - 1) / ts);
                for (long r = at; r < at + rows; ++r) owner[(size_t)r] = (int)b;
                at += rows;
            }
        } else {
            prefix = g.dense_tiles;
            for (auto& o : owner) o = 0;
        }
        std::vector<int> hit((size_t)p.x_rows, 0);
        const int total = prefix * g.nblk;
        if (total > 400000) continue;
        for (int id = 0; id < total; ++id) {
            grp::Tile t;
            grp::decode_tile(segs.data(), dense ? 1 : (int)segs.size(), g, id, grp::WROWS * pl.cg, t);
            CHECK(t.ts >= step && t.ts <= g.tn && t.ts % step == 0 && t.rows >= 1 && t.rows <= t.ts);
            CHECK(t.n0 >= 0 && t.n0 < p.N && t.n0 % (grp::WROWS * pl.cg) == 0 && t.row0 >= 0 && t.row0 + t.rows <= p.x_rows);
            for (int r = t.row0; r < t.row0 + t.rows; ++r) {
                CHECK(owner[(size_t)r] == (dense ? 0 : t.group));
                ++hit[(size_t)r];
            }
        }
        for (size_t r = 0; r < hit.size(); ++r) CHECK(hit[r] == (owner[r] < 0 ? 0 : g.nblk));
    }
    std::printf("ok\n");
    return 0;
}
