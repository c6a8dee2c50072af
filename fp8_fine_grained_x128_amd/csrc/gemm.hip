// gemm.hip -- block-scaled FP8 GEMM (plain and grouped) for gfx950.
//
//   C[m][n] = sum_kb  s_a(m, kb) * s_b(n, kb) * P_kb(m, n),
//   P_kb(m, n) = sum_{k in 128-wide chunk kb} dec(A[m][k]) * dec(B[n][k])
//
// Method: the matrix cores form each chunk's partial product P_kb in FP32
// and the partial is then multiplied by its two scales and added to an FP32
// running total held in vector registers (one "promotion" per 128-wide K
// interval).  Page 3 (why-be.why-be.co.kr, wr_id=55081) describes promoting
// the limited-precision matrix-unit partials to FP32 registers at a fixed K
// interval (Figure 7(b)); page 2 (xn--jj0bz6z98ct0a29q.com, wr_id=362465)
// folds dequantization into that step.  The Wgrad form (one scale per row of
// both operands per chunk) follows page 4 (sunipension.com, wr_id=314414),
// passage on Figure 6 and on 128x1 tiles.
//
// gfx950 mapping:
//   - a work-group (8 waves, 2 x 4) owns a 256x256 output tile, or a 256x448
//     strip (256x256 + 256x192 tiles) when that balances the CUs better; a
//     wave owns 128 rows x 64 columns (64 x 96 in the strip's second tile);
//   - A/B chunk tiles are copied global -> LDS with buffer_load_dwordx4 ...
//     lds (no register staging) through one buffer descriptor per operand
//     whose record count ends at the tile's last valid row, so rows past the
//     matrix read zeros with no clamping code; double-buffered, in 128-byte
//     rows whose 16-byte units are XOR-swizzled by swz(row) (below) so that
//     the fragment reads are free of LDS bank conflicts; the chunk's scales
//     travel as 4-byte direct copies (one fp32 per lane) into a small array
//     next to the tiles;
//   - default datapath: each wave converts its fragments exactly to f16 and
//     forms P_kb of every 16x16 subtile with a dependent chain of four
//     v_mfma_f32_16x16x32_f16; the promotion of a subtile's partial (four
//     FP32 FMAs per lane) is issued under the next subtile's MFMAs (the CDNA
//     analogue of the pages' two-warpgroup overlap); the codes of the next
//     row subtile are read from LDS while the current one is multiplied.
//     The FP8 and power-of-two datapaths (kMma* below) change only this
//     inner loop;
//   - the finished tile goes out through LDS as 16-byte row segments.
//
// MFMA lane layouts, checked on the hardware:
//   16x16x128 (8-bit operands): A: lane l holds row (l % 16), K bytes
//     32*(l/16) .. +32; B: lane l holds column (l % 16), the same K bytes;
//   16x16x32 (f16/bf16 operands): lane l holds row/column (l % 16), 8 values
//     of one 32-wide K step (which 8 is a free choice as long as A and B
//     agree: here K-step s of a chunk takes bytes 8s .. 8s+7 of the lane's 32);
//   D (both): lane l, element r is row 4*(l/16) + r, column (l % 16).
#include "gemm_tile.hpp"

namespace fp8q {

// Plain GEMM: one work-group per output tile.  Work-group ids are dealt to
// the 8 XCDs round-robin; the remap gives each XCD a contiguous run of the
// logical tile order, and the logical order walks groups of kGroupM row tiles
// column by column, so an XCD's run is a compact block of output tiles (8 x 7
// at 4096 x 7168 with 256 x 256 tiles): its L2 then serves each A and B chunk
// to several concurrently running tiles.
constexpr int kGroupM = 8;

__device__ __forceinline__ void tile_of(int64_t logical, int64_t tiles_m, int64_t tiles_n, int64_t& tm,
                                        int64_t& tn) {
    const int64_t group = (int64_t)kGroupM * tiles_n;
    const int64_t first_m = (logical / group) * kGroupM;
    const int64_t gm = tiles_m - first_m < kGroupM ? tiles_m - first_m : kGroupM;
    const int64_t in_group = logical % group;
    tm = first_m + in_group % gm;
    tn = in_group / gm;
}

template <int BM, int BN, int WM, int WN, int BMODE, int OUT, bool ACC, int MMA>
__global__ __launch_bounds__(64 * WM * WN, 1) void gemm_kernel(GemmParams p) {
    using Cfg = GemmCfg<BM, BN, WM, WN, BMODE>;
    __shared__ __align__(1024) uint8_t lds[2 * Cfg::kStageBytes];

    const int64_t tiles = p.tiles_m * p.tiles_n;
    const int64_t bid = blockIdx.x;
    const int64_t per_xcd = (tiles + 7) / 8;
    const int64_t xcd = bid % 8, local = bid / 8;
    const int64_t logical = xcd * per_xcd + local;
    if (logical >= tiles) return;
    int64_t tm, tn;
    tile_of(logical, p.tiles_m, p.tiles_n, tm, tn);
    TileCoord tc;
    tc.m0 = tm * BM;
    tc.n0 = tn * BN;
    tc.m_end = p.M;
    tc.group = 0;
    gemm_tile<BM, BN, WM, WN, BMODE, OUT, ACC, MMA>(p, tc, p.b, p.sb, lds);
}

// Split-K GEMM: work-group (tile, slice) runs chunks [slice * kb_split, ...)
// of one 256x256 output tile and writes the slice's FP32 partial tile to the
// workspace; splitk_reduce_kernel adds the slices in order.  For shapes whose
// tiles alone leave most CUs idle (1024 x 1024 x 65536: 16 tiles on 256
// CUs).  Slice-major order: the tiles of one slice read the same K range of
// A and B, so an XCD's run shares its L2 between them.
template <int BM, int BN, int WM, int WN, int BMODE, int MMA>
__global__ __launch_bounds__(64 * WM * WN, 1) void gemm_splitk_kernel(GemmParams p) {
    using Cfg = GemmCfg<BM, BN, WM, WN, BMODE>;
    __shared__ __align__(1024) uint8_t lds[2 * Cfg::kStageBytes];

    const int64_t tiles = p.tiles_m * p.tiles_n;
    const int64_t work = tiles * p.splits;
    const int64_t bid = blockIdx.x;
    const int64_t per_xcd = (work + 7) / 8;
    const int64_t logical = (bid % 8) * per_xcd + bid / 8;
    if (logical >= work) return;
    const int64_t slice = logical / tiles;
    int64_t tm, tn;
    tile_of(logical % tiles, p.tiles_m, p.tiles_n, tm, tn);
    TileCoord tc;
    tc.m0 = tm * BM;
    tc.n0 = tn * BN;
    tc.m_end = p.M;
    tc.group = 0;
    const int64_t nk = p.K / 128;
    const int64_t kb0 = slice * p.kb_split;
    const int64_t kb1 = kb0 + p.kb_split < nk ? kb0 + p.kb_split : nk;
    gemm_tile<BM, BN, WM, WN, BMODE, kDtypeF32, false, MMA>(p, tc, p.b, p.sb, lds, kb0, kb1,
                                                            p.ws + slice * p.ws_stride, p.ldws);
}

// C = sum over slices s = 0 .. S-1 (in that order) of the FP32 partials, then
// the output conversion (bf16, fp32, or fp32 added to C).  Each thread owns 4
// consecutive columns of one row; the partials are read as 16-byte vectors.
template <int OUT, bool ACC>
__global__ __launch_bounds__(256) void splitk_reduce_kernel(const float* __restrict__ ws, int64_t ldws,
                                                            int64_t ws_stride, int splits, int64_t M,
                                                            int64_t N, void* __restrict__ c, int64_t ldc,
                                                            int vec_store) {
    const int64_t quads = (N + 3) / 4;
    const int64_t total = M * quads;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t m = i / quads;
        const int64_t n = 4 * (i % quads);
        const float* src = ws + m * ldws + n;
        float4 acc = *reinterpret_cast<const float4*>(src);
        for (int sl = 1; sl < splits; ++sl) {
            const float4 v = *reinterpret_cast<const float4*>(src + sl * ws_stride);
            acc.x += v.x;
            acc.y += v.y;
            acc.z += v.z;
            acc.w += v.w;
        }
        const float r[4] = {acc.x, acc.y, acc.z, acc.w};
        if constexpr (OUT == kDtypeF32) {
            float* dst = static_cast<float*>(c) + m * ldc + n;
            if (vec_store && n + 4 <= N) {
                float4 o = acc;
                if constexpr (ACC) {
                    const float4 old = *reinterpret_cast<const float4*>(dst);
                    o.x = old.x + acc.x;
                    o.y = old.y + acc.y;
                    o.z = old.z + acc.z;
                    o.w = old.w + acc.w;
                }
                *reinterpret_cast<float4*>(dst) = o;
            } else {
                for (int e = 0; e < 4 && n + e < N; ++e) dst[e] = ACC ? dst[e] + r[e] : r[e];
            }
        } else {
            uint16_t* dst = static_cast<uint16_t*>(c) + m * ldc + n;
            if (vec_store && n + 4 <= N) {
                uint2 o;
                o.x = (uint32_t)f32_to_bf16(r[0]) | ((uint32_t)f32_to_bf16(r[1]) << 16);
                o.y = (uint32_t)f32_to_bf16(r[2]) | ((uint32_t)f32_to_bf16(r[3]) << 16);
                *reinterpret_cast<uint2*>(dst) = o;
            } else {
                for (int e = 0; e < 4 && n + e < N; ++e) dst[e] = f32_to_bf16(r[e]);
            }
        }
    }
}

// Strip GEMM: one work-group per 256 x 448 strip, computed as a 256x256 tile
// and then a 256x192 tile.  For shapes whose 256x256 tile count leaves the
// last round of work-groups partly empty (4096 x 7168: 448 tiles on 256
// CUs, a second round of 192), 448-wide strips give one equal unit of work
// per CU instead (256 strips of 1.75 tiles).  The host picks the layout.
// The second tile's waves are laid out 4 x 2 (64 x 96 wave tiles): a wave
// then issues 160 conversions per 96 MFMAs per chunk instead of 176 with
// 128 x 48 wave tiles.
constexpr int kStripN = 448;

template <int WM, int WN, int BMODE, int OUT, bool ACC, int MMA>
__global__ __launch_bounds__(64 * WM * WN, 1) void gemm_strip_kernel(GemmParams p) {
    using Cfg1 = GemmCfg<256, 256, WM, WN, BMODE>;
    using Cfg2 = GemmCfg<256, kStripN - 256, 4, 2, BMODE>;
    static_assert(Cfg2::kStageBytes <= Cfg1::kStageBytes, "the second tile reuses the first one's LDS");
    __shared__ __align__(1024) uint8_t lds[2 * Cfg1::kStageBytes];

    const int64_t strips = p.tiles_m * p.tiles_n;  // tiles_n counts strips here
    const int64_t bid = blockIdx.x;
    const int64_t per_xcd = (strips + 7) / 8;
    const int64_t logical = (bid % 8) * per_xcd + bid / 8;
    if (logical >= strips) return;
    int64_t tm, ts;
    tile_of(logical, p.tiles_m, p.tiles_n, tm, ts);
    TileCoord tc;
    tc.m0 = tm * 256;
    tc.n0 = ts * kStripN;
    tc.m_end = p.M;
    tc.group = 0;
    gemm_tile<256, 256, WM, WN, BMODE, OUT, ACC, MMA>(p, tc, p.b, p.sb, lds);
    tc.n0 += 256;
    if (tc.n0 < p.N) {
        __syncthreads();  // every wave is done with the first tile's LDS stages
        static_assert(kStripN % 64 == 0 && Cfg2::TN == 96, "crossing points below assume these");
        if constexpr (BMODE == 0 && MMA == kMmaF16 && Cfg2::kSbPerJ) {
            // Strips start at multiples of 448 columns, so a 96-column wave
            // of this tile starts 0, 32, 64 or 96 columns into a 128-column
            // weight block and crosses into the next block at subtile 4, 2
            // or not at all.  Each wave runs the K loop specialised for its
            // crossing point (same copies and barriers in every variant), so
            // its promotion factors are formed once per row subtile.
            const int ncol = (int)(tc.n0 & 127) + (__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % 2) * Cfg2::TN;
            const int js = (128 - (ncol & 127)) / 16;
            if (js == 2)
                gemm_tile<256, kStripN - 256, 4, 2, BMODE, OUT, ACC, MMA, 2>(p, tc, p.b, p.sb, lds);
            else if (js == 4)
                gemm_tile<256, kStripN - 256, 4, 2, BMODE, OUT, ACC, MMA, 4>(p, tc, p.b, p.sb, lds);
            else  // js = 6 or 8: inside one block
                gemm_tile<256, kStripN - 256, 4, 2, BMODE, OUT, ACC, MMA, Cfg2::NT>(p, tc, p.b, p.sb, lds);
        } else {
            gemm_tile<256, kStripN - 256, 4, 2, BMODE, OUT, ACC, MMA>(p, tc, p.b, p.sb, lds);
        }
    }
}

// Grouped GEMM: persistent work-groups walk a device-side tile list built from
// the group offsets (no host synchronization after routing).  An expert's rows
// are covered by 256-row tiles, except that its last row tile, when it holds
// at most 192, 128 or 64 rows, runs as a tile of that height (with Zipf expert
// sizes this cuts the padded rows from 24 % of the work, all tiles 256 high,
// to 6 %).  The list holds the tiles class by class in decreasing height
// (each class expert-major, then row tile, then column tile), so the final
// round of every work-group is a short one.
constexpr int kMaxGroups = 1024;
constexpr int kTileClasses = 4;  // 256-, 192-, 128- and 64-row tiles

// Height class of an expert's last row tile: 0 (256 rows), 1 (192), 2 (128)
// or 3 (64) for `last` = 1..256 rows in it.
__device__ __forceinline__ int last_tile_class(int64_t last) {
    return last > 192 ? 0 : last > 128 ? 1 : last > 64 ? 2 : 3;
}

template <int BM, int BN, int WM, int WN, int OUT, int MMA>
__global__ __launch_bounds__(64 * WM * WN, 1) void grouped_gemm_kernel(GemmParams p) {
    using Cfg = GemmCfg<BM, BN, WM, WN, 0>;
    static_assert(BM == 256, "tile classes are 256, 192, 128 and 64 rows");
    // One LDS object: the two tile stages, then the tile tables and the
    // checked offsets.  (With the tables in a second __shared__ array the
    // compiler no longer tells the copies into one stage from the fragment
    // reads of the other, and waits for each chunk's copies before computing
    // it.)
    constexpr int kTables = 4 * kTileClasses * (kMaxGroups + 1);
    __shared__ __align__(1024) uint8_t lds[2 * Cfg::kStageBytes + kTables + 4 * (kMaxGroups + 1)];
    int32_t* start = reinterpret_cast<int32_t*>(lds + 2 * Cfg::kStageBytes);  // [class][G + 1]
    int32_t* off = start + kTileClasses * (kMaxGroups + 1);                     // [G + 1]

    const int G = p.groups;
    const int64_t tiles_n = (p.N + BN - 1) / BN;
    if (threadIdx.x == 0) {
        // Offsets as the kernel uses them: clamped to [0, M] and made
        // non-decreasing, so a routing step that produced out-of-range or
        // decreasing offsets cannot send a tile outside A, its scales or C.
        int64_t prev = p.offsets[0];
        prev = prev < 0 ? 0 : prev > p.M ? p.M : prev;
        off[0] = (int32_t)prev;
        int64_t n[kTileClasses] = {0, 0, 0, 0};
        for (int g = 0; g < G; ++g) {
            int64_t hi = p.offsets[g + 1];
            hi = hi < prev ? prev : hi > p.M ? p.M : hi;
            off[g + 1] = (int32_t)hi;
            const int64_t cnt = hi - prev;
            prev = hi;
#pragma unroll
            for (int c = 0; c < kTileClasses; ++c) start[c * (kMaxGroups + 1) + g] = (int32_t)n[c];
            const int64_t rows_tiles = (cnt + BM - 1) / BM;
            if (rows_tiles > 0) {
                const int cl = last_tile_class(cnt - (rows_tiles - 1) * BM);
                n[0] += (rows_tiles - 1) * tiles_n;
                n[cl] += tiles_n;
            }
        }
#pragma unroll
        for (int c = 0; c < kTileClasses; ++c) start[c * (kMaxGroups + 1) + G] = (int32_t)n[c];
    }
    __syncthreads();
    int64_t first[kTileClasses + 1];  // first list index of each class
    first[0] = 0;
#pragma unroll
    for (int c = 0; c < kTileClasses; ++c) first[c + 1] = uniform64(first[c] + start[c * (kMaxGroups + 1) + G]);
    const int64_t total = first[kTileClasses];
    // Work-groups are dealt to the 8 XCDs round-robin.  Each round of gridDim
    // tiles is split into 8 contiguous runs, one per XCD, so that an XCD's L2
    // holds whole row tiles (all their column tiles run there) instead of
    // every XCD fetching every A row tile.
    const int64_t nwg = gridDim.x;
    const int64_t slot = nwg % 8 == 0 ? (int64_t)(blockIdx.x % 8) * (nwg / 8) + blockIdx.x / 8 : blockIdx.x;
    for (int64_t tile = slot; tile < total; tile += nwg) {
        const int cl = __builtin_amdgcn_readfirstlane(tile < first[1] ? 0 : tile < first[2] ? 1 : tile < first[3] ? 2 : 3);
        const int32_t* st = start + cl * (kMaxGroups + 1);
        const int64_t local = tile - first[cl];
        const int g = find_group(st, G, local);
        const int64_t in_g = local - st[g];
        const int64_t lo = off[g], hi = off[g + 1];
        TileCoord tc;
        tc.group = g;
        // full tiles: row tile in_g / tiles_n of the expert; a short tile is
        // the expert's last row tile
        tc.m0 = uniform64(lo + (cl == 0 ? (in_g / tiles_n) * BM : ((hi - lo + BM - 1) / BM - 1) * BM));
        tc.n0 = uniform64((in_g % tiles_n) * BN);
        tc.m_end = uniform64(hi);
        const uint8_t* b = p.b + g * p.b_group_stride;
        const float* sb = p.sb + g * p.sb_group_stride;
        if (cl == 0)
            gemm_tile<BM, BN, WM, WN, 0, OUT, false, MMA, -2, true>(p, tc, b, sb, lds);
        else if (cl == 1)
            gemm_tile<BM * 3 / 4, BN, WM, WN, 0, OUT, false, MMA, -2, true>(p, tc, b, sb, lds);
        else if (cl == 2)
            gemm_tile<BM / 2, BN, WM, WN, 0, OUT, false, MMA, -2, true>(p, tc, b, sb, lds);
        else
            gemm_tile<BM / 4, BN, WM, WN, 0, OUT, false, MMA, -2, true>(p, tc, b, sb, lds);
        __syncthreads();
    }
}

// ----------------------------------------------------------------------------
// Launchers
// ----------------------------------------------------------------------------
namespace {

constexpr int kBM = 256, kBN = 256, kWM = 2, kWN = 4;

int cu_count();

GemmParams to_params(const GemmArgs& g) {
    GemmParams p;
    p.a = g.a; p.lda = g.lda; p.sa = g.sa; p.ldsa = g.ldsa;
    p.b = g.b; p.ldb = g.ldb; p.b_group_stride = g.b_group_stride;
    p.sb = g.sb; p.ldsb = g.ldsb; p.sb_group_stride = g.sb_group_stride;
    p.offsets = g.offsets; p.groups = g.groups;
    p.M = g.M; p.N = g.N; p.K = g.K; p.c = g.c; p.ldc = g.ldc;
    p.tiles_m = (g.M + kBM - 1) / kBM;
    p.tiles_n = (g.N + kBN - 1) / kBN;
    const int64_t el = g.c_dtype == kDtypeF32 ? 4 : 2;
    p.vec_store = (reinterpret_cast<uintptr_t>(g.c) % 16 == 0) && ((g.ldc * el) % 16 == 0);
    p.splits = 1;
    p.kb_split = g.K / 128;
    p.ws = nullptr;
    p.ldws = 0;
    p.ws_stride = 0;
    return p;
}

int cu_count() {
    int dev = 0, cus = 256;
    if (hipGetDevice(&dev) == hipSuccess) {
        int v = 0;
        if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && v > 0) cus = v;
    }
    return cus;
}

// Strips when they finish in fewer 64-column units of work per CU: a round of
// 256x256 tiles costs 4 units, a round of 256x448 strips 7.
bool use_strips(const GemmArgs& g) {
    const int64_t cus = cu_count();
    const int64_t tiles_m = (g.M + kBM - 1) / kBM;
    const int64_t t1 = tiles_m * ((g.N + kBN - 1) / kBN);
    const int64_t t2 = tiles_m * ((g.N + kStripN - 1) / kStripN);
    return ((t2 + cus - 1) / cus) * 7 < ((t1 + cus - 1) / cus) * 4;
}

template <int BMODE, int OUT, bool ACC, int MMA>
void launch_plain(const GemmArgs& g, GemmParams p, hipStream_t st) {
    if (use_strips(g)) {
        p.tiles_n = (g.N + kStripN - 1) / kStripN;
        const int64_t per_xcd = (p.tiles_m * p.tiles_n + 7) / 8;
        hipLaunchKernelGGL((gemm_strip_kernel<kWM, kWN, BMODE, OUT, ACC, MMA>), dim3((unsigned)(per_xcd * 8)),
                           dim3(64 * kWM * kWN), 0, st, p);
        return;
    }
    const int64_t tiles = p.tiles_m * p.tiles_n;
    const int64_t per_xcd = (tiles + 7) / 8;
    hipLaunchKernelGGL((gemm_kernel<kBM, kBN, kWM, kWN, BMODE, OUT, ACC, MMA>), dim3((unsigned)(per_xcd * 8)),
                       dim3(64 * kWM * kWN), 0, st, p);
}

template <int BMODE, int MMA>
void launch_split(const GemmArgs& g, const GemmParams& p, hipStream_t st) {
    const int64_t work = p.tiles_m * p.tiles_n * p.splits;
    const int64_t per_xcd = (work + 7) / 8;
    hipLaunchKernelGGL((gemm_splitk_kernel<kBM, kBN, kWM, kWN, BMODE, MMA>), dim3((unsigned)(per_xcd * 8)),
                       dim3(64 * kWM * kWN), 0, st, p);
    const int64_t quads = g.M * ((g.N + 3) / 4);
    const int64_t blocks = (quads + 255) / 256 < 4096 ? (quads + 255) / 256 : 4096;
    const uintptr_t ca = reinterpret_cast<uintptr_t>(g.c);
    const int vec = g.c_dtype == kDtypeF32 ? (ca % 16 == 0 && g.ldc % 4 == 0) : (ca % 8 == 0 && g.ldc % 4 == 0);
    if (g.c_dtype == kDtypeBF16)
        hipLaunchKernelGGL((splitk_reduce_kernel<kDtypeBF16, false>), dim3((unsigned)blocks), dim3(256), 0, st,
                           p.ws, p.ldws, p.ws_stride, p.splits, g.M, g.N, g.c, g.ldc, vec);
    else if (g.accumulate)
        hipLaunchKernelGGL((splitk_reduce_kernel<kDtypeF32, true>), dim3((unsigned)blocks), dim3(256), 0, st,
                           p.ws, p.ldws, p.ws_stride, p.splits, g.M, g.N, g.c, g.ldc, vec);
    else
        hipLaunchKernelGGL((splitk_reduce_kernel<kDtypeF32, false>), dim3((unsigned)blocks), dim3(256), 0, st,
                           p.ws, p.ldws, p.ws_stride, p.splits, g.M, g.N, g.c, g.ldc, vec);
}

template <int MMA>
void launch_plain_mma(const GemmArgs& g, const GemmParams& p, hipStream_t st) {
    if (p.splits > 1) {
        if (g.bscale == 0)
            launch_split<0, MMA>(g, p, st);
        else
            launch_split<1, MMA>(g, p, st);
        return;
    }
    if (g.bscale == 0) {
        if (g.c_dtype == kDtypeBF16) launch_plain<0, kDtypeBF16, false, MMA>(g, p, st);
        else if (g.accumulate) launch_plain<0, kDtypeF32, true, MMA>(g, p, st);
        else launch_plain<0, kDtypeF32, false, MMA>(g, p, st);
    } else {
        if (g.c_dtype == kDtypeBF16) launch_plain<1, kDtypeBF16, false, MMA>(g, p, st);
        else if (g.accumulate) launch_plain<1, kDtypeF32, true, MMA>(g, p, st);
        else launch_plain<1, kDtypeF32, false, MMA>(g, p, st);
    }
}

template <int MMA>
void launch_grouped_mma(const GemmArgs& g, const GemmParams& p, int64_t grid, hipStream_t st) {
    if (g.c_dtype == kDtypeBF16)
        hipLaunchKernelGGL((grouped_gemm_kernel<kBM, kBN, kWM, kWN, kDtypeBF16, MMA>), dim3((unsigned)grid),
                           dim3(64 * kWM * kWN), 0, st, p);
    else
        hipLaunchKernelGGL((grouped_gemm_kernel<kBM, kBN, kWM, kWN, kDtypeF32, MMA>), dim3((unsigned)grid),
                           dim3(64 * kWM * kWN), 0, st, p);
}

}  // namespace

// Split K when the 256x256 tiles fill at most half of the CUs: as many
// slices as fit the CUs, each at least 4 chunks (512 K) long.
SplitPlan plan_splitk(int64_t M, int64_t N, int64_t K) {
    SplitPlan sp{1, K / 128, 0, 0};
    const int64_t cus = cu_count();
    const int64_t tiles = ((M + kBM - 1) / kBM) * ((N + kBN - 1) / kBN);
    const int64_t nk = K / 128;
    if (tiles <= 0 || nk <= 0 || 2 * tiles > cus) return sp;
    int64_t s = cus / tiles;
    if (s > nk / 4) s = nk / 4;
    if (s < 2) return sp;
    sp.kb_split = (nk + s - 1) / s;
    sp.slices = (int)((nk + sp.kb_split - 1) / sp.kb_split);
    if (sp.slices < 2) return SplitPlan{1, nk, 0, 0};
    sp.ldws = (N + 3) / 4 * 4;
    sp.bytes = (int64_t)sp.slices * M * sp.ldws * 4;
    return sp;
}

hipError_t launch_gemm(const GemmArgs& g, hipStream_t st) {
    GemmParams p = to_params(g);
    if (g.workspace) {
        const SplitPlan sp = plan_splitk(g.M, g.N, g.K);
        if (sp.slices > 1 && sp.bytes <= g.workspace_bytes) {
            p.splits = sp.slices;
            p.kb_split = sp.kb_split;
            p.ws = static_cast<float*>(g.workspace);
            p.ldws = sp.ldws;
            p.ws_stride = g.M * sp.ldws;
        }
    }
    switch (g.mma) {
        case kMmaFp8: launch_plain_mma<kMmaFp8>(g, p, st); break;
        case kMmaBf16Fold: launch_plain_mma<kMmaBf16Fold>(g, p, st); break;
        case kMmaFp8Scaled: launch_plain_mma<kMmaFp8Scaled>(g, p, st); break;
        default: launch_plain_mma<kMmaF16>(g, p, st); break;
    }
    return hipGetLastError();
}

hipError_t launch_grouped_gemm(const GemmArgs& g, hipStream_t st) {
    const GemmParams p = to_params(g);
    const int cus = cu_count();
    // upper bound of the tile count without reading the offsets
    const int64_t tiles_n = (g.N + kBN - 1) / kBN;
    const int64_t bound = ((g.M + kBM - 1) / kBM + g.groups) * tiles_n;
    const int64_t grid = bound < cus ? (bound > 0 ? bound : 1) : cus;
    switch (g.mma) {
        case kMmaFp8: launch_grouped_mma<kMmaFp8>(g, p, grid, st); break;
        case kMmaBf16Fold: launch_grouped_mma<kMmaBf16Fold>(g, p, grid, st); break;
        case kMmaFp8Scaled: launch_grouped_mma<kMmaFp8Scaled>(g, p, grid, st); break;
        default: launch_grouped_mma<kMmaF16>(g, p, grid, st); break;
    }
    return hipGetLastError();
}

}  // namespace fp8q
