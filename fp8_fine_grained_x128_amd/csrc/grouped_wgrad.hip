// grouped_wgrad.hip -- the weight gradients of all experts:
//   dW_g[n][k] (=|+=) sum over the 128-token chunks c of group g
//                     s_dy(c, n) * s_x(c, k) * sum_{i in c} dec(dY^T[n][i]) * dec(X^T[k][i])
// Both operands lie transposed in the layout of groups.hpp (every group takes
// whole chunks of its own), one scale per channel and chunk, so a tile of a
// group's gradient is the row-scaled product of gemm_tile.hpp over that
// group's chunks.
//
// Contractions are short (a few chunks) and gradients large, so what counts is
// that a tile's stores, its next tile's loads and the products run together.  A
// work-group walks many tiles as one stream of chunks: under the last chunk of
// a tile the first one of the next is copied, and a tile's stores go on under
// the next one's first chunk.  64 experts of 2048x7168 over 32768 rows, fp32:
// 1255 to 1330 us, by card.  The products alone take 853 (equal groups) to 970
// (Zipf), the 3.8 GB of stores alone, in these pieces, 670 (5.6 TB/s).  What
// does not overlap is the time for which a tile's 256 KB queue at the memory: copies that
// are issued behind them arrive late, whichever wave issues them, and there is
// room for one chunk ahead.  (Half the waves copying and the other half
// storing, so that only the copies are waited for: 1234 : 1205 of equal groups;
// 128x128 tiles, two work-groups a compute unit: 1021 without the stores, 1323
// with, the same 300 more; stores between the last chunk's products:
// 1347 : 1199.)  Few large experts are bound by the products (4 of 4096x7168,
// 16384 rows, added: 890 to 957, of which the products alone are 740 to 796).
#include <cmath>
#include <type_traits>

#include "gemm_tile.hpp"
#include "groups.hpp"
#include "tile_io.hpp"

namespace fp8q {

namespace {

constexpr int kSortedGroups = 256;  // up to so many can be taken by size (each is ranked against all)

// 4-byte buffer copy to LDS: lane i's dword (or 0 past the record count) lands at lds + 4 * i.
__device__ __forceinline__ void buffer_copy4_to_lds(__amdgpu_buffer_rsrc_t r, uint32_t voffset, void* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)lds, 4, voffset, 0, 0, 0);
#else
    (void)r;
    (void)voffset;
    (void)lds;
#endif
}

// A is X^T (rows k), B is dY^T (rows n): an accumulator's four elements of a
// lane are then four consecutive k of one row of dW.
struct WgradParams {
    const uint8_t* a;
    const uint8_t* b;
    const float* sa;
    const float* sb;
    uint32_t lda, ldb;  // 256 rows stay below 2^32
    int64_t ldsa, ldsb;
    const int32_t* offsets;
    int groups;
    int rows;
    int M, N;  // channels of X, channels of dY
    void* c;
    int64_t ldc, c_group_stride;
    int tiles_m, tiles_n;
    int vec;    // c and its strides allow stores of four elements
    int sorted;  // groups are taken by size
    int slice;   // chunks of a slice: groups of 1.5 or more are split, their slices' tiles go to ws
    float* ws;  // [slice][N][ldws]
    int64_t ldws;
};

// Slices of a group of `chunks`, of about `slice` each; 0: one part, stored to
// dW at once.
__device__ __forceinline__ int split_slices(int chunks, int slice) {
    const int n = (chunks + (slice >> 1)) / slice;
    return n > 1 ? n : 0;
}

struct Job {
    int kb, kb1;  // chunks
    int m0, n0;
    void* c;      // nullptr: no more jobs
    int64_t ldc;
    bool partial;  // fp32 slice in ws
};

// Four consecutive values of a row, the first at p; `count` of them exist.
template <int OUT, bool ACC>
__device__ __forceinline__ void store4(void* row, int64_t k, int count, const v4f& v, bool vec) {
    if constexpr (OUT == kDtypeF32) {
        float* p = static_cast<float*>(row) + k;
        if (vec && count >= 4) {
            v4f w = v;
            if constexpr (ACC) w += *reinterpret_cast<const v4f*>(p);
            *reinterpret_cast<v4f*>(p) = w;
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < count) p[r] = ACC ? p[r] + v[r] : v[r];
        }
    } else {
        uint16_t* p = static_cast<uint16_t*>(row) + k;
        uint16_t h[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = f32_to_bf16(v[r]);
        if (vec && count >= 4) {
            *reinterpret_cast<uint2*>(p) = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < count) p[r] = h[r];
        }
    }
}

// A wave's tile that lies inside dW's columns, 16 rows at a time through its
// LDS region: a store instruction writes two 512-byte (bf16: four 256-byte)
// pieces of rows, through a buffer descriptor whose record count ends at dW's
// last row (rows past it are dropped by the range check).  kStores of them.
// They are marked as streaming: 64 experts of 2048x7168, 1312 -> 1277 us.
[[maybe_unused]] constexpr int kStreaming = 2;
template <class Cfg, int OUT>
struct Rows {
    static constexpr int kEl = OUT == kDtypeF32 ? 4 : 2;
    static constexpr int kBytes = Cfg::TM * kEl, kPitch = kBytes + 16, kUnits = kBytes / 16;
    static constexpr int kAtOnce = 64 / kUnits;  // rows of one store
    static constexpr int kStores = Cfg::NT * 16 / kAtOnce;
    static_assert(16 * kPitch * Cfg::kWaves <= Cfg::kStageBytes, "the regions of all waves in one stage");
};
// Rows 16j .. 16j+15 of a wave's tile into its LDS region.
template <class Cfg, int OUT>
__device__ __forceinline__ void stage_rows(const v4f (&acc)[Cfg::MT][Cfg::NT], int j, uint8_t* region, int lane) {
    using R = Rows<Cfg, OUT>;
    uint8_t* to = region + (lane & 15) * R::kPitch + 4 * (lane >> 4) * R::kEl;
    if (j > 0) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the last rows are read
#pragma unroll
    for (int i = 0; i < Cfg::MT; ++i) {
        if constexpr (OUT == kDtypeF32)
            *reinterpret_cast<v4f*>(to + 16 * i * R::kEl) = acc[i][j];
        else
            *reinterpret_cast<uint2*>(to + 16 * i * R::kEl) =
                make_uint2(pack_bf16(acc[i][j][0], acc[i][j][1]), pack_bf16(acc[i][j][2], acc[i][j][3]));
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // written
}

template <class Cfg, int OUT, bool ACC>
__device__ __forceinline__ void store_rows(const v4f (&acc)[Cfg::MT][Cfg::NT], __amdgpu_buffer_rsrc_t rc,
                                           uint32_t row_bytes, int wm, int wn, int lane, uint8_t* region) {
#if defined(__HIP_DEVICE_COMPILE__)
    using R = Rows<Cfg, OUT>;
    const uint8_t* from = region + lane / R::kUnits * R::kPitch + lane % R::kUnits * 16;
    const uint32_t off = (wn * Cfg::TN + lane / R::kUnits) * row_bytes + wm * R::kBytes + lane % R::kUnits * 16;
    constexpr int kN = 16 / R::kAtOnce;
    // the values to add to are read one pass ahead
    v4f old[2][ACC ? kN : 1];
    auto read_old = [&](int j) __attribute__((always_inline)) {
        if constexpr (ACC) {
#pragma unroll
            for (int u = 0; u < kN; ++u)
                old[j & 1][u] = __builtin_bit_cast(
                    v4f, __builtin_amdgcn_raw_buffer_load_b128(rc, off + (16 * j + u * R::kAtOnce) * row_bytes, 0, 0));
        }
    };
    read_old(0);
#pragma unroll
    for (int j = 0; j < Cfg::NT; ++j) {
        if (j + 1 < Cfg::NT) read_old(j + 1);
        stage_rows<Cfg, OUT>(acc, j, region, lane);
        u32x4 v[kN];
#pragma unroll
        for (int u = 0; u < kN; ++u) v[u] = *reinterpret_cast<const u32x4*>(from + u * R::kAtOnce * R::kPitch);
#pragma unroll
        for (int u = 0; u < kN; ++u) {
            if constexpr (ACC) v[u] = __builtin_bit_cast(u32x4, old[j & 1][u] + __builtin_bit_cast(v4f, v[u]));
            __builtin_amdgcn_raw_buffer_store_b128(v[u], rc, off + (16 * j + u * R::kAtOnce) * row_bytes, 0, kStreaming);
        }
    }
#endif
}

// The same for a tile at dW's last columns, or rows that do not lie on 16
// bytes: 64 consecutive elements of a row by one instruction.  (Elements
// stored from the accumulators, 16 rows by one instruction: 16 experts of
// 333x1111 in bf16 27 us.)
template <class Cfg, int OUT, bool ACC>
__device__ __forceinline__ void store_elements(const v4f (&acc)[Cfg::MT][Cfg::NT], void* c, int64_t ldc, int m0, int n0,
                                               int M, int N, int wm, int wn, int lane, uint8_t* region) {
    using R = Rows<Cfg, OUT>;
    using T = typename std::conditional<OUT == kDtypeF32, float, uint16_t>::type;
    constexpr int kRows = 4;  // rows under way at once
    const int k0 = m0 + wm * Cfg::TM + lane;
#pragma unroll
    for (int j = 0; j < Cfg::NT; ++j) {
        stage_rows<Cfg, OUT>(acc, j, region, lane);
        const int nj = n0 + wn * Cfg::TN + 16 * j;
#pragma unroll 1
        for (int r0 = 0; r0 < 16 && nj + r0 < N; r0 += kRows) {
            T* const row = static_cast<T*>(c) + (int64_t)(nj + r0) * ldc + k0;
            const uint8_t* from = region + r0 * R::kPitch + lane * R::kEl;
            const int rows = N - nj - r0;
#pragma unroll
            for (int h = 0; h < Cfg::TM / 64; ++h) {
                if (k0 + 64 * h >= M) continue;
                T v[kRows];
                T old[kRows];
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    v[r] = *reinterpret_cast<const T*>(from + r * R::kPitch + 64 * h * R::kEl);
                    old[r] = ACC && r < rows ? row[r * ldc + 64 * h] : T(0);
                }
#pragma unroll
                for (int r = 0; r < kRows; ++r)
                    if (r < rows) row[r * ldc + 64 * h] = ACC ? T(old[r] + v[r]) : v[r];
            }
        }
    }
}

// This lane's number, formed where it stands: what is derived from it is then
// not held (and spilled) across the loops around.
__device__ __forceinline__ int lane_now() {
#if defined(__HIP_DEVICE_COMPILE__)
    int v = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    asm volatile("" : "+v"(v));
    return v;
#else
    return 0;
#endif
}

// Where a job's operands come from: descriptors of its rows of codes (as in
// gemm_tile.hpp: rows past the matrix read zeros) and of the scales of one
// 64-channel run a wave, which move by a row of scales from chunk to chunk.
struct Source {
    __amdgpu_buffer_rsrc_t ra, rb;
    const float* s;  // this wave's run in chunk 0
    uint32_t s_bytes;
};

// The asynchronous copies of chunk kb into a stage, in gemm_tile.hpp's layout:
// part `it` of a wave is 8 rows of codes, and with part 0 goes its run of scales.
template <class Cfg, int BM>
struct Copies {
    uint32_t off_a, off_b;
    __device__ __forceinline__ Copies(const WgradParams& p, int wave) {
        const int lane = lane_now(), lrow = lane >> 3, unit = (lane & 7) ^ swz(lrow);
        off_a = (uint32_t)(8 * wave + lrow) * p.lda + 16 * unit;
        off_b = (uint32_t)(8 * wave + lrow) * p.ldb + 16 * unit;
    }
    __device__ __forceinline__ void issue(uint8_t* stage, const Source& src, const WgradParams& p, int kb, int wave,
                                          int it) const {
        constexpr int kRows = 8 * Cfg::kWaves;  // rows of one part of all waves
        const bool is_a = kRows * it < BM;
        const uint32_t step = is_a ? (uint32_t)(kRows * it) * p.lda : (uint32_t)(kRows * it - BM) * p.ldb;
        uint32_t voff;
        asm volatile("v_add_u32 %0, %1, %2" : "=v"(voff) : "s"(step), "v"(is_a ? off_a : off_b));
        buffer_copy16_to_lds(is_a ? src.ra : src.rb, voff, (uint32_t)kb * 128u, stage + 1024 * (wave + Cfg::kWaves * it));
        if (it == 0 && wave < Cfg::kScaleCopies) {
            const __amdgpu_buffer_rsrc_t rs =
                make_rsrc(src.s + (int64_t)kb * (wave < BM / 64 ? p.ldsa : p.ldsb), src.s_bytes);
            buffer_copy4_to_lds(rs, 4u * lane_now(), stage + Cfg::kTileBytes + 256 * wave);
        }
    }
};

// One chunk's products from stage `cur` while the next one's operands are
// copied into stage `nxt`.  (The stages are told apart by the parameters'
// __restrict__: without it the compiler lets every fragment read wait for all
// copies under way, 1.4 times the time of the whole kernel.)
template <class Cfg, int BM, int MMA>
__device__ __forceinline__ void chunk_step(const uint8_t* __restrict__ cur, uint8_t* __restrict__ nxt, const Source& src,
                                           const WgradParams& p, int kb_next, v4f (&acc)[Cfg::MT][Cfg::NT], int wave,
                                           int wm, int wn, int lane) {
    const Copies<Cfg, BM> copies(p, wave);
    auto issue = [&](int part) __attribute__((always_inline)) { copies.issue(nxt, src, p, kb_next, wave, part); };
    compute_chunk<Cfg, BM, 1, MMA>(cur, reinterpret_cast<const float*>(cur + Cfg::kTileBytes), acc, wm, wn, lane, 0,
                                   issue);
}

template <int BM, int BN, int WM, int WN, int OUT, bool ACC, int MMA>
__global__ __launch_bounds__(64 * WM * WN, 2) void grouped_wgrad_kernel(WgradParams p) {
    using Cfg = GemmCfg<BM, BN, WM, WN, 1>;
    // One LDS object (see grouped_gemm_kernel): the tile stages, then tables of
    // the groups: their first chunks and the slices before them in ws, the
    // parts (one a slice) before each in the order that they are taken in (the
    // longest parts first, or as they come), the lengths of their parts and
    // that order.
    constexpr int kThreads = 64 * WM * WN;
    __shared__ __align__(1024) uint8_t lds[2 * Cfg::kStageBytes + 12 * (kMostGroups + 4) + 6 * kSortedGroups];
    int32_t* first = reinterpret_cast<int32_t*>(lds + 2 * Cfg::kStageBytes);
    int32_t* slices = first + kMostGroups + 4;
    int32_t* parts = slices + kMostGroups + 4;
    int32_t* length = parts + kMostGroups + 4;
    uint16_t* by_size = reinterpret_cast<uint16_t*>(length + kSortedGroups);
    const int G = p.groups;
    const int lane = threadIdx.x & 63;
    if (p.rows == 0) {  // perhaps no offsets either
        for (int g = threadIdx.x; g <= G; g += kThreads) first[g] = slices[g] = 0;
    } else if (threadIdx.x < 64) {
        for_group_count(G, [&](auto per) __attribute__((always_inline)) {
            constexpr int PER = decltype(per)::value;
            const LaneGroups<PER> l(p.offsets, G, p.rows, lane);
            int n_chunks = 0, n_slices = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j) n_chunks += l.chunks(j), n_slices += split_slices(l.chunks(j), p.slice);
            int c0 = wave_scan_sum(n_chunks) - n_chunks, s0 = wave_scan_sum(n_slices) - n_slices;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                if (PER * lane + j <= G) first[PER * lane + j] = c0, slices[PER * lane + j] = s0;
                c0 += l.chunks(j), s0 += split_slices(l.chunks(j), p.slice);
            }
            if (lane == 63) first[G] = c0, slices[G] = s0;  // of all: groups past G are empty
        });
    }
    __syncthreads();
    if (p.sorted) {
        for (int g = threadIdx.x; g < G; g += kThreads) {
            const int n = max(1, slices[g + 1] - slices[g]);
            length[g] = (first[g + 1] - first[g] + n - 1) / n;
        }
        __syncthreads();
        // a group's place: how many are longer, or as long and before it
        for (int g = threadIdx.x; g < G; g += kThreads) {
            const int mine = length[g];
            int place = 0;
            for (int h = 0; h < G; ++h) place += length[h] > mine || (length[h] == mine && h < g);
            by_size[place] = (uint16_t)g;
        }
    }
    auto group_at = [&](int order) __attribute__((always_inline)) { return p.sorted ? by_size[order] : order; };
    __syncthreads();
    if (threadIdx.x < 64) {  // parts in that order
        const int per = (G + 63) / 64;
        int n_parts = 0;
        for (int i = lane * per; i < G && i < (lane + 1) * per; ++i) {
            const int g = group_at(i);
            n_parts += max(1, slices[g + 1] - slices[g]);
        }
        int p0 = wave_scan_sum(n_parts) - n_parts;
        for (int i = lane * per; i < G && i < (lane + 1) * per; ++i) {
            const int g = group_at(i);
            parts[i] = p0;
            p0 += max(1, slices[g + 1] - slices[g]);
            parts[i + 1] = p0;
        }
    }
    __syncthreads();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    // The jobs are the tiles of the parts, one part after the other, dealt in
    // rounds to the work-groups; by size every other round in reverse, so that
    // who has a longer job in a round has a shorter one in the next.
    const uint32_t tiles = (uint32_t)p.tiles_m * p.tiles_n, nwg = gridDim.x;
    const uint32_t slot = nwg % 8 == 0 ? blockIdx.x % 8 * (nwg / 8) + blockIdx.x / 8 : blockIdx.x;
    uint32_t in = slot, step = p.sorted ? 2 * (nwg - 1 - slot) + 1 : nwg;  // to the next round; 2 nwg - step from there
    int part = 0, order = 0;
    const int n_parts = __builtin_amdgcn_readfirstlane(parts[G]);
    constexpr int kEl = OUT == kDtypeF32 ? 4 : 2;

    // The next job; gradients of groups without rows are written on the way.
    auto next_job = [&]() __attribute__((always_inline)) {
        Job job;
        job.c = nullptr;
        for (;; in += step, step = 2 * nwg - step) {
            while (in >= tiles) in -= tiles, ++part;
            if (part >= n_parts) return job;
            while (__builtin_amdgcn_readfirstlane(parts[order + 1]) <= part) ++order;
            const int g = __builtin_amdgcn_readfirstlane(group_at(order));
            const int c0 = __builtin_amdgcn_readfirstlane(first[g]), c1 = __builtin_amdgcn_readfirstlane(first[g + 1]);
            // eight tiles of k by all of n, then the next eight: concurrent tiles share their operands in L2
            const uint32_t band = 8 * p.tiles_n, b0 = in / band * 8, in_band = in % band;
            const uint32_t height = p.tiles_m - b0 < 8 ? p.tiles_m - b0 : 8;
            job.m0 = (int)(b0 + in_band % height) * BM;
            job.n0 = (int)(in_band / height) * BN;
            uint8_t* c = static_cast<uint8_t*>(p.c) + g * p.c_group_stride * kEl;
            const int s0 = __builtin_amdgcn_readfirstlane(slices[g]), n = __builtin_amdgcn_readfirstlane(slices[g + 1]) - s0;
            job.partial = n > 0;
            if (job.partial) {
                const int sl = part - __builtin_amdgcn_readfirstlane(parts[order]);
                const int each = (c1 - c0) / n, more = (c1 - c0) % n;
                job.kb = c0 + sl * each + min(sl, more);
                job.kb1 = job.kb + each + (sl < more);
                job.ldc = p.ldws;
                job.c = p.ws + (int64_t)(s0 + sl) * p.N * p.ldws;
                return job;
            }
            if (c0 < c1) {
                job.kb = c0, job.kb1 = c1, job.ldc = p.ldc;
                job.c = c;
                return job;
            }
            if constexpr (!ACC) {
                const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
                for (int e = 64 * wave + lane_now(); e < BN * BM / 4; e += 64 * WM * WN) {
                    const int n = job.n0 + e / (BM / 4), k = job.m0 + e % (BM / 4) * 4;
                    if (n < p.N && k < p.M)
                        store4<OUT, false>(c + n * p.ldc * kEl, k, p.M - k > 4 ? 4 : p.M - k, zero, p.vec);
                }
            }
        }
    };

    auto source_of = [&](const Job& job) __attribute__((always_inline)) {
        Source s;
        s.ra = make_rsrc(p.a + (int64_t)job.m0 * p.lda, (int64_t)(p.M - job.m0) * p.lda);
        s.rb = make_rsrc(p.b + (int64_t)job.n0 * p.ldb, (int64_t)(p.N - job.n0) * p.ldb);
        const int of_a = job.m0 + 64 * wave, of_b = job.n0 + 64 * (wave - BM / 64);
        const int left = wave < BM / 64 ? p.M - of_a : p.N - of_b;
        s.s = wave < BM / 64 ? p.sa + of_a : p.sb + of_b;
        s.s_bytes = left <= 0 ? 0u : left >= 64 ? 256u : 4u * left;
        return s;
    };

    Job job = next_job();
    if (!job.c) return;
    Source src = source_of(job);
    int stage = 0;
    bool behind = false;  // at least Rows::kStores stores were issued after the last copies
    {
        const Copies<Cfg, BM> copies(p, wave);
#pragma unroll
        for (int it = 0; it < Cfg::kLoadsPerWave; ++it) copies.issue(lds, src, p, job.kb, wave, it);
    }
    // Waits for the copies of the chunk that comes next.  Memory operations
    // complete in order: a job's first chunk was copied before the last job's
    // stores, which go on under it.
    auto arrive = [&]() __attribute__((always_inline)) {
        if (behind) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(Rows<Cfg, OUT>::kStores) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        behind = false;
        lds_barrier();  // (__syncthreads would wait for the stores)
    };
    constexpr int kRegion = Cfg::kStageBytes / Cfg::kWaves & ~15;
    for (;;) {
        v4f acc[Cfg::MT][Cfg::NT];
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
            for (int j = 0; j < Cfg::NT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        in += step, step = 2 * nwg - step;
        const Job next = next_job();
        // under a chunk's products the next one of this job is copied, or the
        // first one of the next job (after the last of all, this one again,
        // into the stage that is not read any more)
        auto next_chunk = [&](int kb) __attribute__((always_inline)) {
            if (kb + 1 < job.kb1) return kb + 1;
            if (!next.c) return kb;
            src = source_of(next);
            return next.kb;
        };
        const bool inside = (job.partial || p.vec) && job.m0 + BM <= p.M;
        const uint32_t el = job.partial ? 4 : kEl, row_bytes = (uint32_t)job.ldc * el;
        const int rows = p.N - job.n0 < BN ? p.N - job.n0 : BN;
        const __amdgpu_buffer_rsrc_t rc =
            make_rsrc(static_cast<uint8_t*>(job.c) + job.n0 * (int64_t)row_bytes + (int64_t)job.m0 * el,
                      (int64_t)(rows - 1) * row_bytes + BM * el);
        int kb = job.kb;
        for (; kb < job.kb1; ++kb) {
            arrive();
            const int kb_next = next_chunk(kb);
            chunk_step<Cfg, BM, MMA>(lds + stage * Cfg::kStageBytes, lds + (stage ^ 1) * Cfg::kStageBytes, src, p, kb_next,
                                     acc, wave, wm, wn, lane_now());
            stage ^= 1;
        }
        const int ln = lane_now();
        lds_barrier();  // every wave is done with the stage just read
        uint8_t* region = lds + (stage ^ 1) * Cfg::kStageBytes + wave * kRegion;
        if (inside) {
            if (job.partial) store_rows<Cfg, kDtypeF32, false>(acc, rc, row_bytes, wm, wn, ln, region);
            else store_rows<Cfg, OUT, ACC>(acc, rc, row_bytes, wm, wn, ln, region);
            behind = true;
        } else if (job.partial) {
            store_elements<Cfg, kDtypeF32, false>(acc, job.c, job.ldc, job.m0, job.n0, p.M, p.N, wm, wn, ln, region);
        } else {
            store_elements<Cfg, OUT, ACC>(acc, job.c, job.ldc, job.m0, job.n0, p.M, p.N, wm, wn, ln, region);
        }
        if (!next.c) break;
        job = next;
    }
}

// dW of the groups that were split: the sum of their slices, in order.  Each
// thread owns four consecutive k of a row.
template <int OUT, bool ACC>
__global__ __launch_bounds__(256) void wgrad_join_kernel(WgradParams p) {
    const int g = blockIdx.y, lane = threadIdx.x & 63;
    int before = 0, count = 0;
    for_group_count(p.groups, [&](auto per) __attribute__((always_inline)) {
        constexpr int PER = decltype(per)::value;
        const LaneGroups<PER> l(p.offsets, p.groups, p.rows, lane);
        int mine = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int sl = split_slices(l.chunks(j), p.slice);
            if (PER * lane + j < g) before += sl;
            if (PER * lane + j == g) count = sl;
            mine += sl;
        }
        before += wave_scan_sum(mine) - mine;  // of the lanes below
        count = __builtin_amdgcn_readlane(count, g / PER);
        before = __builtin_amdgcn_readlane(before, g / PER);
    });
    if (count == 0) return;
    const int64_t quads = (p.M + 3) / 4, total = p.N * quads, stride = p.N * p.ldws;
    constexpr int kEl = OUT == kDtypeF32 ? 4 : 2;
    constexpr int kAtOnce = 8;  // slices loaded at once
    const float* first = p.ws + before * stride;
    uint8_t* c = static_cast<uint8_t*>(p.c) + g * p.c_group_stride * kEl;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
        const int64_t n = e / quads;
        const int k = 4 * (int)(e - n * quads);
        const float* q = first + n * p.ldws + k;
        v4f sum = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int s0 = 0; s0 < count; s0 += kAtOnce) {
            v4f v[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) v[u] = *reinterpret_cast<const v4f*>(q + min(s0 + u, count - 1) * stride);
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u)
                if (s0 + u < count) sum += v[u];
        }
        store4<OUT, ACC>(c + n * p.ldc * kEl, k, p.M - k > 4 ? 4 : p.M - k, sum, p.vec);
    }
}

// How a product is cut.  A compute unit holds one work-group of 8 waves with
// 256x256 tiles, or two of 4 waves with 128x128.  Times are in us, for fp32
// gradients and groups of Zipf sizes.
// Tiles: 256x256 halves the operands' way through the LDS, so it wins where a
// round of work-groups stays within one or two groups, from half as many such
// tiles a group as there are compute units (large : small for 64 experts of
// 2048x7168 1256 : 1432, 4 of 7168x4096 1600 : 1944, 8 of 4096x4096 502 : 577,
// 8 of 4096x2048 279 : 297), unless a quarter of the rounds would be empty.
// Where a round spans many groups it waits for the largest one, with fewer and
// longer jobs to even that out (8 of 2048x2048 117 : 103, 32 of 1024x1024 76 :
// 62, 64 of 2048x2048 407 : 403).
// Slices: where 128x128 tiles of a long group leave the card waiting for it,
// groups are split into even slices of about as many chunks as one job a
// work-group makes them, kMinSlice or more (groups below 1.5 of that are left
// whole).  How long the longest group is the host does not know: it is taken as
// sizes that fall as 1 / rank have it, 1 / (1 + ln G) of all.  A split has to
// save kSavedChunks against it (the join's launch, 5 us) and one chunk's time
// for every kChunkBytes of slices, which are written and read again; and the
// longest group has to be two slices, else hardly any is cut.
// Without : with, Zipf sizes (equal sizes in brackets), for 32 groups of
// 512x512, 32768 rows 100 : 44 (28 : 34), 8 of 1024x1024, 65536 rows 399 : 202
// (153 : 148), 9 of 128x640, 8014 rows 37 : 17 (15 : 17), 4 of 384x512, 8192
// rows 47 : 23 (26 : 23), 3 of 256x4288, 17908 rows 107 : 66 (68 : 66), 1 of
// 428x2239, 24782 rows 249 : 76; and where the rule leaves them whole, 1 of
// 2048x2048, 2048 rows 29 : 41, 4 of 512x1536, 2048 rows 18 : 24 (14 : 23), 4 of
// 768x2304, 4096 rows 42 : 36 (25 : 29), 16 of 640x640, 4096 rows 24 : 23 (13 :
// 19), 32 of 1024x1024, 8192 rows 61 : 68 (37 : 51), 4 of 1408x1408, 8192 rows
// 59 : 57 (43 : 45).  (Slices of equal length with a remainder, in the groups'
// order: 3 of 256x4288 81, 4 of 1408x1408 86.)
// Order: work-groups that get few jobs each (under kFewJobs) take the largest
// groups first (as they come : by size for 64 of 2048x2048, 32 jobs each, 442 :
// 403; 32 of 1024x2048 152 : 135).  Many jobs even out by themselves, and
// groups bound by their stores then run beside others bound by their products
// (64 of 2048x7168 1256 : 1286).
struct WgradPlan {
    bool large;
    int slice;  // chunks; INT32_MAX: no split
    int64_t ldws, bytes;
};

constexpr int kMinSlice = 4, kSavedChunks = 6, kFewJobs = 48;
constexpr double kChunkBytes = 5.3e6;

WgradPlan plan_wgrad(int64_t rows, int64_t G, int64_t N, int64_t K) {
    const int64_t cus = compute_units(), groups = G < rows ? G : rows;
    const int64_t large = ((N + 255) / 256) * ((K + 255) / 256), rounds = (large * groups + cus - 1) / cus;
    WgradPlan plan{true, INT32_MAX, 0, 0};
    if (rounds == 0 || (2 * large >= cus && 100 * groups * N * K >= 75 * rounds * cus * 65536)) return plan;
    plan.large = false;
    const int64_t tiles = ((N + 127) / 128) * ((K + 127) / 128), slots = 2 * cus;
    const int64_t chunks = rows / 128 + (groups + 1) / 2;  // about as many
    int64_t slice = (chunks * tiles + slots - 1) / slots;
    slice = slice < kMinSlice ? kMinSlice : slice;
    plan.ldws = (K + 3) / 4 * 4;
    const double longest = (double)chunks / (1.0 + std::log((double)groups));
    const double cost = kSavedChunks + longest / slice * N * plan.ldws * 4 / kChunkBytes;
    if (longest < 2.0 * slice || longest < slice + cost || plan.ldws * 4 >= (int64_t(1) << 24)) return plan;
    plan.slice = (int)slice;
    // a split group of c chunks has at most c / slice + 1/2 slices, and c >= 1.5 slice
    plan.bytes = 4 * group_chunks(rows, G) / (3 * slice) * N * plan.ldws * 4;
    return plan;
}

template <int OUT, bool ACC, int MMA>
void launch_wgrad_typed(const WgradParams& p, const WgradPlan& plan, int64_t grid, hipStream_t st) {
    const dim3 gr((unsigned)grid);
    if (plan.large)
        hipLaunchKernelGGL((grouped_wgrad_kernel<256, 256, 2, 4, OUT, ACC, MMA>), gr, dim3(512), 0, st, p);
    else
        hipLaunchKernelGGL((grouped_wgrad_kernel<128, 128, 2, 2, OUT, ACC, MMA>), gr, dim3(256), 0, st, p);
    if (plan.slice == INT32_MAX) return;
    const int64_t quads = (int64_t)p.N * ((p.M + 3) / 4);
    const int64_t blocks = (quads + 255) / 256;
    hipLaunchKernelGGL((wgrad_join_kernel<OUT, ACC>), dim3((unsigned)(blocks < 1024 ? blocks : 1024), p.groups), dim3(256),
                       0, st, p);
}

template <int MMA>
void launch_wgrad_mma(const GemmArgs& g, const WgradParams& p, const WgradPlan& plan, int64_t grid, hipStream_t st) {
    if (g.c_dtype == kDtypeBF16) launch_wgrad_typed<kDtypeBF16, false, MMA>(p, plan, grid, st);
    else if (g.accumulate) launch_wgrad_typed<kDtypeF32, true, MMA>(p, plan, grid, st);
    else launch_wgrad_typed<kDtypeF32, false, MMA>(p, plan, grid, st);
}

}  // namespace

int64_t grouped_wgrad_bytes(int64_t rows, int groups, int64_t M, int64_t N) {
    return plan_wgrad(rows, groups, M, N).bytes;
}

hipError_t launch_grouped_wgrad(const GemmArgs& g, int64_t c_group_stride, hipStream_t st) {
    const WgradPlan plan = plan_wgrad(g.K, g.groups, g.M, g.N);
    WgradParams p{};
    p.a = g.b; p.lda = (uint32_t)g.ldb; p.sa = g.sb; p.ldsa = g.ldsb;
    p.b = g.a; p.ldb = (uint32_t)g.lda; p.sb = g.sa; p.ldsb = g.ldsa;
    p.offsets = g.offsets; p.groups = g.groups; p.rows = (int)g.K;
    p.M = (int)g.N; p.N = (int)g.M; p.c = g.c; p.ldc = g.ldc; p.c_group_stride = c_group_stride;
    const int tile = plan.large ? 256 : 128;
    p.tiles_m = (p.M + tile - 1) / tile;
    p.tiles_n = (p.N + tile - 1) / tile;
    const int64_t el = g.c_dtype == kDtypeF32 ? 4 : 2;
    p.vec = reinterpret_cast<uintptr_t>(g.c) % 16 == 0 && g.ldc * el % 16 == 0 && c_group_stride * el % 16 == 0 &&
            g.ldc * el < (int64_t(1) << 24);  // 256 rows within 32-bit offsets
    p.slice = plan.slice;
    p.ws = static_cast<float*>(g.workspace);
    p.ldws = plan.ldws;
    // work-groups: as many as there are jobs, or as fit at once
    const int64_t split = plan.slice == INT32_MAX ? 0 : 4 * group_chunks(g.K, g.groups) / (3 * plan.slice);
    const int64_t jobs = (int64_t)p.tiles_m * p.tiles_n * (g.groups + split);
    const int64_t slots = (plan.large ? 1 : 2) * (int64_t)compute_units();
    const int64_t grid = jobs < slots ? jobs : slots;
    p.sorted = g.groups <= kSortedGroups && jobs > slots && jobs < kFewJobs * slots;
    switch (g.mma) {
        case kMmaFp8: launch_wgrad_mma<kMmaFp8>(g, p, plan, grid, st); break;
        case kMmaBf16Fold: launch_wgrad_mma<kMmaBf16Fold>(g, p, plan, grid, st); break;
        case kMmaFp8Scaled: launch_wgrad_mma<kMmaFp8Scaled>(g, p, plan, grid, st); break;
        default: launch_wgrad_mma<kMmaF16>(g, p, plan, grid, st); break;
    }
    return hipGetLastError();
}

}  // namespace fp8q
