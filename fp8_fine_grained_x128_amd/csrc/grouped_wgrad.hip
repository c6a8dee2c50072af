// grouped_wgrad.hip -- the weight gradients of all experts:
//   dW_g[n][k] (=|+=) sum over the 128-token chunks t of group g
//                     s_a(t, n) * s_b(t, k) * sum_{token in t} dec(A[n][token]) * dec(B[k][token])
// A = dY^T and B = X^T in the layout of groups.hpp (every group takes whole
// chunks of its own), one scale per row and chunk, so a tile of a group's
// gradient is the row-scaled product of gemm_tile.hpp over that group's chunks.
#include "gemm_tile.hpp"
#include "groups.hpp"

namespace fp8q {

constexpr int kMaxWgradGroups = 1024;

template <int BM, int BN, int WM, int WN, int OUT, bool ACC, int MMA>
__global__ __launch_bounds__(64 * WM * WN, 1) void grouped_wgrad_kernel(GemmParams p, int64_t c_group_stride) {
    using Cfg = GemmCfg<BM, BN, WM, WN, 1>;
    // one LDS object (see grouped_gemm_kernel): the tile stages, then the first chunk of every group
    __shared__ __align__(1024) uint8_t lds[2 * Cfg::kStageBytes + 4 * (kMaxWgradGroups + 1)];
    int32_t* first = reinterpret_cast<int32_t*>(lds + 2 * Cfg::kStageBytes);
    const int G = p.groups;
    if (p.K == 0) {  // no rows, perhaps no offsets either
        for (int g = threadIdx.x; g <= G; g += 64 * WM * WN) first[g] = 0;
    } else if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        int mine = 0;
        for_groups_of_lane(p.offsets, G, (int)p.K, lane, [&](int, int lo, int hi) { mine += (hi - lo + 127) >> 7; });
        int at = wave_scan_sum(mine) - mine;
        for_groups_of_lane(p.offsets, G, (int)p.K, lane, [&](int g, int lo, int hi) {
            first[g] = at;
            at += (hi - lo + 127) >> 7;
            first[g + 1] = at;
        });
    }
    __syncthreads();
    const int64_t tiles = p.tiles_m * p.tiles_n;
    const int64_t total = tiles * G;
    const int64_t nwg = gridDim.x;
    const int64_t slot = nwg % 8 == 0 ? (int64_t)(blockIdx.x % 8) * (nwg / 8) + blockIdx.x / 8 : blockIdx.x;
    for (int64_t w = slot; w < total; w += nwg) {
        const int g = __builtin_amdgcn_readfirstlane((int)(w / tiles));
        const int64_t in_g = w % tiles;
        TileCoord tc;
        tc.group = g;
        tc.m0 = uniform64(in_g / p.tiles_n * BM);
        tc.n0 = uniform64(in_g % p.tiles_n * BN);
        tc.m_end = p.M;
        const int64_t kb0 = __builtin_amdgcn_readfirstlane(first[g]), kb1 = __builtin_amdgcn_readfirstlane(first[g + 1]);
        GemmParams q = p;
        q.c = static_cast<uint8_t*>(p.c) + g * c_group_stride * (OUT == kDtypeF32 ? 4 : 2);
        if (kb0 < kb1) {
            gemm_tile<BM, BN, WM, WN, 1, OUT, ACC, MMA, -2, true>(q, tc, p.b, p.sb, lds, kb0, kb1);
            __syncthreads();
        } else if (!ACC) {  // no tokens: a zero gradient
            const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
            const v4f zero[Cfg::MT][Cfg::NT] = {};
            store_tile<Cfg, OUT, false>(zero, q.c, p.ldc, tc, p.N, wave / WN, wave % WN, lane);
        }
    }
}

namespace {

template <int MMA>
void launch_wgrad_mma(const GemmArgs& g, const GemmParams& p, int64_t grid, int64_t c_group_stride, hipStream_t st) {
    const dim3 gr((unsigned)grid), bl(512);
    if (g.c_dtype == kDtypeBF16)
        hipLaunchKernelGGL((grouped_wgrad_kernel<256, 256, 2, 4, kDtypeBF16, false, MMA>), gr, bl, 0, st, p, c_group_stride);
    else if (g.accumulate)
        hipLaunchKernelGGL((grouped_wgrad_kernel<256, 256, 2, 4, kDtypeF32, true, MMA>), gr, bl, 0, st, p, c_group_stride);
    else
        hipLaunchKernelGGL((grouped_wgrad_kernel<256, 256, 2, 4, kDtypeF32, false, MMA>), gr, bl, 0, st, p, c_group_stride);
}

}  // namespace

int64_t grouped_wgrad_bytes(int64_t, int, int64_t, int64_t) { return 0; }

hipError_t launch_grouped_wgrad(const GemmArgs& g, int64_t c_group_stride, hipStream_t st) {
    GemmParams p{};
    p.a = g.a; p.lda = g.lda; p.sa = g.sa; p.ldsa = g.ldsa;
    p.b = g.b; p.ldb = g.ldb; p.sb = g.sb; p.ldsb = g.ldsb;
    p.offsets = g.offsets; p.groups = g.groups;
    p.M = g.M; p.N = g.N; p.K = g.K; p.c = g.c; p.ldc = g.ldc;
    p.tiles_m = (g.M + 255) / 256;
    p.tiles_n = (g.N + 255) / 256;
    const int64_t el = g.c_dtype == kDtypeF32 ? 4 : 2;
    p.vec_store = (reinterpret_cast<uintptr_t>(g.c) % 16 == 0) && ((g.ldc * el) % 16 == 0) &&
                  ((c_group_stride * el) % 16 == 0);
    const int64_t work = p.tiles_m * p.tiles_n * g.groups, cus = compute_units();
    const int64_t grid = work < cus ? work : cus;
    switch (g.mma) {
        case kMmaFp8: launch_wgrad_mma<kMmaFp8>(g, p, grid, c_group_stride, st); break;
        case kMmaBf16Fold: launch_wgrad_mma<kMmaBf16Fold>(g, p, grid, c_group_stride, st); break;
        case kMmaFp8Scaled: launch_wgrad_mma<kMmaFp8Scaled>(g, p, grid, c_group_stride, st); break;
        default: launch_wgrad_mma<kMmaF16>(g, p, grid, c_group_stride, st); break;
    }
    return hipGetLastError();
}

}  // namespace fp8q
