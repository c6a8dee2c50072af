// groups.hpp -- rows grouped by expert, laid out in whole 128-token chunks.
//
// Rows [off[g], off[g+1]) belong to group g.  The weight gradients contract
// over them in 128-wide chunks that may not cross groups (a chunk has one
// scale per channel), so in the transposed operands every group takes
// ceil(n_g / 128) chunks of its own, one group after the other; the last one's
// missing tokens are zeros.  The offsets stay on the device: the kernels find
// their chunks themselves, with the offsets taken as
//   off'[0] = clamp(off[0], 0, M),  off'[g+1] = clamp(off[g+1], off'[g], M)
// (a running maximum of the clamped values), so that no offsets, however wrong,
// lead outside the arrays.
#pragma once

#include <type_traits>

#include "device_common.hpp"

namespace fp8q {

// Chunks that any G groups of M rows together fit into: each of the at most
// min(G, M) groups with rows adds less than one partly filled chunk.
inline int64_t group_chunks(int64_t M, int64_t G) { return (M + 127 * (G < M ? G : M)) / 128; }

// Inclusive scans over the 64 lanes of non-negative values (the identity of
// both is the 0 that lanes without a source read).  Steps inside a 16-lane row
// by row shifts, then the last lane of a row to the next row, and of the lower
// half to the upper one.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_or_zero(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
template <class Op>
__device__ __forceinline__ int wave_scan(int v, Op op) {
    v = op(v, dpp_or_zero<0x111, 0xf>(v));
    v = op(v, dpp_or_zero<0x112, 0xf>(v));
    v = op(v, dpp_or_zero<0x114, 0xf>(v));
    v = op(v, dpp_or_zero<0x118, 0xf>(v));
    v = op(v, dpp_or_zero<0x142, 0xa>(v));
    v = op(v, dpp_or_zero<0x143, 0xc>(v));
    return v;
}
__device__ __forceinline__ int wave_scan_sum(int v) {
    return wave_scan(v, [](int a, int b) { return a + b; });
}
__device__ __forceinline__ int wave_scan_max(int v) {
    return wave_scan(v, [](int a, int b) { return a > b ? a : b; });
}
// The value one lane below; 0 in lane 0.
__device__ __forceinline__ int from_lane_below(int v) { return dpp_or_zero<0x138, 0xf>(v); }

__device__ __forceinline__ int clamp_offset(int32_t v, int M) { return v < 0 ? 0 : v > M ? M : v; }

constexpr int kMostGroups = 1024;

// The rows of groups PER * lane .. PER * lane + PER - 1 (64 * PER >= G; those
// past G are empty): group j of the lane's has rows [edge[j], edge[j + 1]).
// All offsets are loaded at once (one after the other, as a loop that carries
// the running maximum loads them, 2048x2048 of 256 groups took 53 us, not 35).
template <int PER>
struct LaneGroups {
    int edge[PER + 1];
    // Needs the whole wave.
    __device__ __forceinline__ LaneGroups(const int32_t* __restrict__ off, int G, int M, int lane) {
        int32_t v[PER + 1];
#pragma unroll
        for (int j = 0; j <= PER; ++j) v[j] = off[min(PER * lane + j, G)];
        int top = clamp_offset(v[0], M);
#pragma unroll
        for (int j = 1; j <= PER; ++j) top = max(top, clamp_offset(v[j], M));
        edge[0] = max(clamp_offset(v[0], M), from_lane_below(wave_scan_max(top)));
#pragma unroll
        for (int j = 1; j <= PER; ++j) edge[j] = max(edge[j - 1], clamp_offset(v[j], M));
    }
    __device__ __forceinline__ int chunks(int j) const { return (edge[j + 1] - edge[j] + 127) >> 7; }
};

// f(std::integral_constant<int, PER>) with a PER for G groups.
template <class F>
__device__ __forceinline__ void for_group_count(int G, F&& f) {
    if (G <= 64) f(std::integral_constant<int, 1>());
    else if (G <= 256) f(std::integral_constant<int, 4>());
    else f(std::integral_constant<int, kMostGroups / 64>());
}

struct GroupChunk {
    int row0;     // first row of the chunk
    int row_end;  // one past the last row of its group
    bool live;    // false: past the last group's chunks
};

// The rows of chunk c, the same in every lane of the wave.
template <int PER>
__device__ __forceinline__ GroupChunk find_chunk(const int32_t* __restrict__ off, int G, int M, int c) {
    const int lane = threadIdx.x & 63;
    const LaneGroups<PER> l(off, G, M, lane);
    int n = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) n += l.chunks(j);
    const int end = wave_scan_sum(n), start = end - n;
    int row0 = 0, row_end = 0, at = start;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int next = at + l.chunks(j);
        if (c >= at && c < next) {
            row0 = l.edge[j] + 128 * (c - at);
            row_end = l.edge[j + 1];
        }
        at = next;
    }
    GroupChunk r;
    const uint64_t holds = __ballot(c >= start && c < end);
    r.live = holds != 0;
    const int src = r.live ? __builtin_ctzll(holds) : 0;
    r.row0 = __builtin_amdgcn_readlane(row0, src);
    r.row_end = __builtin_amdgcn_readlane(row_end, src);
    return r;
}

}  // namespace fp8q
