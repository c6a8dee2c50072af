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

// Walks the groups of this lane, [lane * per, lane * per + per) of G with per =
// ceil(G / 64): f(g, lo, hi) with the offsets as above.  Needs the whole wave.
template <class F>
__device__ __forceinline__ void for_groups_of_lane(const int32_t* __restrict__ off, int G, int M, int lane, F&& f) {
    const int per = (G + 63) / 64;
    const int g0 = lane * per < G ? lane * per : G, g1 = g0 + per < G ? g0 + per : G;
    int top = lane == 0 ? clamp_offset(off[0], M) : 0;
    for (int g = g0; g < g1; ++g) {
        const int hi = clamp_offset(off[g + 1], M);
        top = hi > top ? hi : top;
    }
    int lo = from_lane_below(wave_scan_max(top));
    if (lane == 0) lo = clamp_offset(off[0], M);
    for (int g = g0; g < g1; ++g) {
        int hi = clamp_offset(off[g + 1], M);
        hi = hi > lo ? hi : lo;
        f(g, lo, hi);
        lo = hi;
    }
}

struct GroupChunk {
    int row0;     // first row of the chunk
    int row_end;  // one past the last row of its group
    bool live;    // false: past the last group's chunks
};

// The rows of chunk c, the same in every lane of the wave.
__device__ __forceinline__ GroupChunk find_chunk(const int32_t* __restrict__ off, int G, int M, int c) {
    const int lane = threadIdx.x & 63;
    GroupChunk r;
    int row0 = 0, row_end = 0, start, end;
    if (G <= 64) {  // a group a lane
        int lo = clamp_offset(off[lane < G ? lane : G], M);
        const int hi = wave_scan_max(max(lo, clamp_offset(off[lane < G ? lane + 1 : G], M)));
        lo = max(lo, from_lane_below(hi));
        const int n = (hi - lo + 127) >> 7;
        end = wave_scan_sum(n);
        start = end - n;
        row0 = lo + 128 * (c - start);
        row_end = hi;
    } else {
        int mine = 0;
        for_groups_of_lane(off, G, M, lane, [&](int, int lo, int hi) { mine += (hi - lo + 127) >> 7; });
        end = wave_scan_sum(mine);
        start = end - mine;
        int at = start;
        for_groups_of_lane(off, G, M, lane, [&](int, int lo, int hi) {
            const int n = (hi - lo + 127) >> 7;
            if (c >= at && c < at + n) {
                row0 = lo + 128 * (c - at);
                row_end = hi;
            }
            at += n;
        });
    }
    const uint64_t holds = __ballot(c >= start && c < end);
    r.live = holds != 0;
    const int src = r.live ? __builtin_ctzll(holds) : 0;
    r.row0 = __builtin_amdgcn_readlane(row0, src);
    r.row_end = __builtin_amdgcn_readlane(row_end, src);
    return r;
}

}  // namespace fp8q
