// norm.hip -- layer norm (and RMS norm) in front of an FP8 GEMM, forward into
// 1x128 codes and backward with the reduction of the weights' gradients.
//
//   mu = mean x, r = 1/sqrt(mean (x-mu)^2 + eps)        (RMS: mu = 0)
//   y  = (x-mu) r gamma + beta
//   backward, with xh = (x-mu) r and w = dy gamma, over one row:
//   dx = r (w - xh mean(w xh) - mean(w)) + skip          (RMS: no mean(w))
//   and over all rows: dgamma = sum dy xh, dbeta = sum dy
//
// The pages keep normalization in higher precision (page 1,
// why-be.why-be.co.kr wr_id=65900, passage on the operators that stay in
// BF16/FP32) and cache the activations that feed the Linear operators in FP8
// (same page, passage on FP8-cached activations): the norm's result leaves
// this kernel as those codes.  Every sum is fp32 (of squares fp64, where eps
// is too small to hide what fp32 loses).
//
// A row is read once and stays in registers, so the mean, the sum of squared
// deviations (a second pass over registers: no cancellation) and the result
// come from one read.
#include <algorithm>
#include <type_traits>

#include "launch.hpp"
#include "tile_io.hpp"

namespace fp8q {

namespace {

// Eight weights at column c (zero beyond `cols`; `dflt` where there are none).
__device__ __forceinline__ void load_weights8(const void* w, int dtype, int64_t c, int64_t cols, float dflt,
                                              float v[8]) {
    if (w == nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = dflt;
    } else if (dtype == kDtypeBF16) {
        Raw8<uint16_t> r;
        load_row8<uint16_t, false>(r, static_cast<const uint16_t*>(w), c, cols, false);
        r.values(v);
    } else {
        Raw8<float> r;
        load_row8<float, false>(r, static_cast<const float*>(w), c, cols, false);
        r.values(v);
    }
}

// Sum over the work-group's W waves; every thread receives it.  `red` may be
// used again after the next barrier that follows the return.
template <int W, typename S>
__device__ __forceinline__ S block_sum(S v, S* red) {
    v = wave_sum(v);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < W; ++w) v += red[w];
    }
    return v;
}

}  // namespace

// ----------------------------------------------------------------------------
// Forward.  A row belongs to N lanes (16, a wave, or whole waves): lane t of
// them has columns 8*(t + N*i) .. +7 for i < I, so 16 neighbouring lanes hold
// one 128-column tile and a tile maximum is a DPP row maximum.
// ----------------------------------------------------------------------------

// Makes the compiler decode a row's stored values again instead of keeping
// them as fp32 from pass to pass (twice the registers for bf16).
template <int I>
__device__ __forceinline__ void forget(Raw8<uint16_t> (&raw)[I]) {
#pragma unroll
    for (int i = 0; i < I; ++i) {
        opaque(raw[i].d.x);
        opaque(raw[i].d.y);
        opaque(raw[i].d.z);
        opaque(raw[i].d.w);
    }
}
template <int I>
__device__ __forceinline__ void forget(Raw8<float> (&)[I]) {}

// Sum of a row's deviations from `mean`, squared, in the type S: in fp32 times
// shrink^2 (shrink is a power of two: one rounding, that of the difference).
// Zeros beyond the row's end stay out.  WHOLE: the row is whole groups of
// eight columns.
template <typename S, typename T, int N, int I, bool WHOLE>
__device__ __forceinline__ S sum_squares(const Raw8<T> (&raw)[I], int t, int64_t cols, float mean, float shrink) {
    const float shift = -mean * shrink;
    auto deviation = [&](float v) -> S {
        if constexpr (sizeof(S) == 8) return v - mean;
        return __builtin_fmaf(v, shrink, shift);
    };
    S sq = 0;
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int64_t c = 8 * (t + N * i);
        float v[8];
        raw[i].values(v);
        if (WHOLE ? c < cols : c + 8 <= cols) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const S d = deviation(v[k]);
                sq = __builtin_elementwise_fma(d, d, sq);
            }
        } else if (!WHOLE) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const S d = c + k < cols ? deviation(v[k]) : 0;
                sq = __builtin_elementwise_fma(d, d, sq);
            }
        }
    }
    return sq;
}

// 1 / sqrt(variance + eps) from sum_squares().
__device__ __forceinline__ float rstd_of(const LayernormArgs& a, float sq) {
    return 1.0f / sqrtf(sq / ((float)a.cols * a.shrink * a.shrink) + a.eps);
}
__device__ __forceinline__ float rstd_of(const LayernormArgs& a, double sq) {
    return (float)(1.0 / sqrt(sq / (double)a.cols + (double)a.eps));
}

// Results of G groups of a row: y from the row's statistics, its values and
// codes to memory.  One lane per tile computes the scale (lane i of a DPP row
// for group i).  weights(i, gm, bt) gives the weights of group i.
template <typename T, int N, int G, bool POW2, bool NT, bool WHOLE, typename Weights>
__device__ __forceinline__ void finish_groups(const LayernormArgs& a, const Raw8<T>* raw, int i0, int t, int64_t row,
                                              float mean, float rstd, const Weights& weights) {
    const int sub = t & 15;
    float v[G][8];
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < G; ++i) {
        const int64_t c = 8 * (t + N * (i0 + i));
        if (!WHOLE || c < a.cols) {
            float gm[8], bt[8];
            weights(i0 + i, gm, bt);
            raw[i].values(v[i]);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[i][k] = __builtin_fmaf((v[i][k] - mean) * rstd, gm[k], bt[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[i][k] = 0.0f;
        }
        if (!WHOLE && c + 8 > a.cols) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[i][k] = c + k < a.cols ? v[i][k] : 0.0f;
        }
        if (a.y && c < a.cols) {
            const int64_t valid = WHOLE ? c + 8 : a.cols;
            if (a.y_dtype == kDtypeBF16)
                store_values8<NT>(static_cast<uint16_t*>(a.y) + row * a.ldy, c, valid, v[i]);
            else
                store_values8(static_cast<float*>(a.y) + row * a.ldy, c, valid, v[i]);
        }
        if (a.q) {
            const uint32_t m = row_max_u32(amax8(v[i]));
            mine = sub == i ? m : mine;
        }
    }
    if (!a.q) return;
    const TileScale ts = make_scale_mode<POW2>(mine);
    if (sub < G) {
        const int64_t tile = (N / 16) * (int64_t)(i0 + sub) + (t >> 4);
        if (tile * 128 < a.cols) a.s[tile * a.lds + row] = ts.s;
    }
    const bool fast = wave_all(sub >= G || ts.fast);
    float s[G], r[G];
    row_broadcast(std::make_integer_sequence<int, G>{}, ts.s, s);
    row_broadcast(std::make_integer_sequence<int, G>{}, ts.r, r);
    uint8_t* q = a.q + row * a.ldq;
#pragma unroll
    for (int i = 0; i < G; ++i) {
        const int64_t c = 8 * (t + N * (i0 + i));
        if (fast && (WHOLE ? c < a.cols : c + 8 <= a.cols)) {
            *reinterpret_cast<uint2*>(q + c) =
                make_uint2(encode4_sr<POW2>(v[i][0], v[i][1], v[i][2], v[i][3], s[i], r[i]),
                           encode4_sr<POW2>(v[i][4], v[i][5], v[i][6], v[i][7], s[i], r[i]));
        } else if (c < a.cols) {
            const TileScale tt = scale_from(s[i], r[i]);
            store8(q, c, WHOLE ? c + 8 : a.cols, encode4_any<POW2>(v[i][0], v[i][1], v[i][2], v[i][3], tt),
                   encode4_any<POW2>(v[i][4], v[i][5], v[i][6], v[i][7], tt));
        }
    }
}

// One row per work-group of W waves: few rows, and rows too wide for a team.
// A row of 7168 takes 3.5 us, which is a launch, one read from memory and two
// sums over 16 waves; 1001 rows of 1000 fp32 columns 5.8 us.
template <typename S, typename T, int W, int I, bool LAYER, bool POW2>
__global__ __launch_bounds__(64 * W) void layernorm_row_kernel(LayernormArgs a) {
    __shared__ float s_sum[16];
    __shared__ S s_squares[16];
    const int64_t cols = a.cols, row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (row >= a.rows) return;
    const int t = threadIdx.x;
    const float n = (float)cols;
    Raw8<T> raw[I];
#pragma unroll
    for (int i = 0; i < I; ++i)
        load_row8(raw[i], static_cast<const T*>(a.x) + row * a.ldx, 8 * (t + 64 * W * i), cols, false);
    float mean = 0.0f;
    if constexpr (LAYER) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            float v[8];
            raw[i].values(v);
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += v[k];
        }
        mean = block_sum<W>(sum, s_sum) / n;
    }
    const float rstd = rstd_of(a, block_sum<W>(sum_squares<S, T, 64 * W, I, false>(raw, t, cols, mean, a.shrink), s_squares));
    if (t == 0) {
        if (LAYER && a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    finish_groups<T, 64 * W, I, POW2, false, false>(a, raw, 0, t, row, mean, rstd, [&](int i, float gm[8], float bt[8]) {
        load_weights8(a.gamma, a.w_dtype, 8 * (t + 64 * W * i), cols, 1.0f, gm);
        load_weights8(a.beta, a.w_dtype, 8 * (t + 64 * W * i), cols, 0.0f, bt);
    });
}

// Weights in LDS: the two halves of every group of eight lie in two runs, so
// that neighbouring lanes read neighbouring 16 bytes.
template <int N>  // columns
struct LdsWeights {
    float4 half[2][N / 8];
    __device__ __forceinline__ void put(int c, const float v[8]) {
        half[0][c >> 3] = make_float4(v[0], v[1], v[2], v[3]);
        half[1][c >> 3] = make_float4(v[4], v[5], v[6], v[7]);
    }
    __device__ __forceinline__ void get(int c, float v[8]) const {
        *reinterpret_cast<float4*>(v) = half[0][c >> 3];
        *reinterpret_cast<float4*>(v + 4) = half[1][c >> 3];
    }
};

// Fills the weights' LDS copy with all threads of the work-group.
template <int N>
__device__ __forceinline__ void fill_weights(LdsWeights<N>& to, const void* w, int dtype, int64_t cols, float dflt) {
    for (int c = 8 * threadIdx.x; c < cols; c += 8 * blockDim.x) {
        float v[8];
        load_weights8(w, dtype, c, cols, dflt, v);
        to.put(c, v);
    }
}

// Teams of N lanes with a row each, 512/N teams per work-group, which share
// the weights in LDS; a team loads its next row before it works on the current
// one.  A work-group's rows are consecutive, so the scales that it writes fill
// whole lines.  Many rows, or narrow ones.  G work-groups are meant to share a
// compute unit.  (8192x7168: RMS norm in bf16 with codes and values 56 us (5.3
// TB/s), codes alone 40, layer norm 58 and 46; fp32 100 and 64.  Non-temporal
// stores of y are worth 7 us in bf16 and cost 19 in fp32.  A wave per row
// needs over 200 registers there and took 85, a work-group per row reads the
// weights again for every row, 88.  Bound by memory with values, by vector
// instructions and the wait for two sums with codes alone.)
constexpr int kTeamThreads = 512;

template <typename S, typename T, int N, int I, int G, bool LAYER, bool POW2, bool WHOLE>
__global__ __launch_bounds__(kTeamThreads, 2 * G) void layernorm_team_kernel(LayernormArgs a, int rows_per_group) {
    constexpr int kTeams = kTeamThreads / N, W = N / 64;
    // Through the caches, narrow rows come faster (20000x1024 bf16, codes and
    // values: 22 us, 26 non-temporal) and wide ones slower
    // (8192x7168 fp32: 102 against 96).
    constexpr bool kNT = N >= 256;
    __shared__ LdsWeights<8 * N * I> s_gamma, s_beta;
    __shared__ S s_red[2][kTeams][W > 1 ? W : 1];
    const int64_t cols = a.cols;
    const int team = threadIdx.x / N, t = threadIdx.x % N;
    const int64_t first = (int64_t)blockIdx.x * rows_per_group, end = min(first + rows_per_group, a.rows);
    const float n = (float)cols;
    auto load = [&](Raw8<T> (&raw)[I], int64_t row) {
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int64_t c = 8 * (t + N * i);
            const T* x = row < end ? static_cast<const T*>(a.x) + row * a.ldx : nullptr;
            if (!WHOLE) load_row8_ahead<T, kNT>(raw[i], x, c, cols);
            else if (x != nullptr && c < cols) raw[i].template load_full<kNT>(x + c);
        }
    };
    auto team_sum = [&](auto v, int phase) {
        if constexpr (N == 16) return row_sum(v);
        v = wave_sum(v);
        if constexpr (W > 1) {
            if ((t & 63) == 0) s_red[phase][team][t >> 6] = v;
            lds_barrier();
            v = s_red[phase][team][0];
#pragma unroll
            for (int w = 1; w < W; ++w) v += s_red[phase][team][w];
        }
        return v;
    };
    Raw8<T> raw[I], next[I];
#pragma unroll
    for (int i = 0; i < I; ++i) next[i].zero();
    load(next, first + team);
    fill_weights(s_gamma, a.gamma, a.w_dtype, cols, 1.0f);
    fill_weights(s_beta, a.beta, a.w_dtype, cols, 0.0f);
    __syncthreads();
    int phase = 0;
    for (int64_t r = first; r < end; r += kTeams) {  // the same trips for all teams: the barriers are the work-group's
        const int64_t row = r + team;
#pragma unroll
        for (int i = 0; i < I; ++i) raw[i] = next[i];
        load(next, row + kTeams);
        float mean = 0.0f;
        if constexpr (LAYER) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < I; ++i) {
                float v[8];
                raw[i].values(v);
#pragma unroll
                for (int k = 0; k < 8; ++k) sum += v[k];
            }
            mean = team_sum(sum, 0) / n;
            forget(raw);
        }
        // a layer norm's two sums have a buffer each, an RMS norm's sums take turns
        const S sq = team_sum(sum_squares<S, T, N, I, WHOLE>(raw, t, cols, mean, a.shrink), LAYER ? 1 : phase);
        phase ^= 1;
        forget(raw);
        const float rstd = rstd_of(a, sq);
        if (row >= end) continue;
        if (t == 0) {
            if (LAYER && a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        finish_groups<T, N, I, POW2, true, WHOLE>(a, raw, 0, t, row, mean, rstd, [&](int i, float gm[8], float bt[8]) {
            s_gamma.get(8 * (t + N * i), gm);
            s_beta.get(8 * (t + N * i), bt);
        });
    }
}

// ----------------------------------------------------------------------------
// Backward.  A work-group of 1024 threads works on 1024/N rows at a time, one
// per team of N lanes, with columns as in the forward pass; the sums over
// its rows stay in registers.  At the end the teams' sums are added in LDS and
// go to part[group][gamma|beta][cols]; layernorm_parts_kernel adds the P
// partial sums in order, so repeated calls give the same bits.  Where
// registers allow (I == 1) a team's next row is on its way while a row is
// worked on; the only wait inside a row is the join of its two sums.
//   One work-group per compute unit: 8192x7168 bf16 with skip takes 87 us
// (5.4 TB/s), 94 with two, 116 with work-groups of eight waves, whose twice as
// many sums per thread leave no registers for the next row.
// ----------------------------------------------------------------------------
template <typename T, int N, int I, bool LAYER>
__global__ __launch_bounds__(1024, 4) void layernorm_backward_kernel(LayernormBackwardArgs a) {
    constexpr int kTeams = 1024 / N, kCols = 8 * N * I, W = N / 64;
    constexpr bool kAhead = I == 1;
    constexpr bool kNT = sizeof(T) == 2 && N == 1024;  // as in the forward pass (30000x331 bf16: 37 us, 48 non-temporal)
    __shared__ LdsWeights<kCols> s_gamma;
    __shared__ float s_red[2][2][16];
    __shared__ float s_team[kTeams > 1 ? kTeams : 1][kTeams > 1 ? kCols : 1];
    const int64_t cols = a.cols;
    const int wave = threadIdx.x >> 6, team = threadIdx.x / N, t = threadIdx.x % N;
    const float inv_n = 1.0f / (float)cols;
    auto load = [&](Raw8<T> (&raw)[I], const void* p, int64_t ld, int64_t row) {
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const T* from = row < a.rows ? static_cast<const T*>(p) + row * ld : nullptr;
            load_row8_ahead<T, kNT>(raw[i], from, 8 * (t + N * i), cols);
        }
    };
    float dgamma[I][8], dbeta[I][8];
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) dgamma[i][k] = dbeta[i][k] = 0.0f;
    Raw8<T> x[I], dy[I], skip[I], nx[I], ndy[I];
    const int64_t step = (int64_t)gridDim.x * kTeams;
    int64_t base = (int64_t)blockIdx.x * kTeams;  // the work-group's rows are base .. base + kTeams - 1
    auto statistic = [&](const float* p, int64_t row) { return row < a.rows ? p[row] : 0.0f; };
    float n_mean = LAYER ? statistic(a.mean, base + team) : 0.0f, n_rstd = statistic(a.rstd, base + team);
    if (kAhead) {
        load(nx, a.x, a.ldx, base + team);
        load(ndy, a.dy, a.lddy, base + team);
    }
    fill_weights(s_gamma, a.gamma, a.w_dtype, cols, 1.0f);
    __syncthreads();
    for (int phase = 0; base < a.rows; base += step, phase ^= 1) {
        const int64_t row = base + team;
        const float mean = n_mean, rstd = n_rstd;
        if (kAhead) {
#pragma unroll
            for (int i = 0; i < I; ++i) {
                x[i] = nx[i];
                dy[i] = ndy[i];
            }
        } else {
            load(x, a.x, a.ldx, row);
            load(dy, a.dy, a.lddy, row);
        }
        if (a.skip) {
            load(skip, a.skip, a.ldskip, row);
        } else {
#pragma unroll
            for (int i = 0; i < I; ++i) skip[i].zero();
        }
        if (kAhead) {
            load(nx, a.x, a.ldx, row + step);
            load(ndy, a.dy, a.lddy, row + step);
        }
        if (LAYER) n_mean = statistic(a.mean, row + step);
        n_rstd = statistic(a.rstd, row + step);
        float xh[I][8], w[I][8];
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            float gm[8];
            s_gamma.get(8 * (t + N * i), gm);
            x[i].values(xh[i]);
            dy[i].values(w[i]);  // dy, zero beyond the row's end
            if (8 * (t + N * i) >= cols) {
#pragma unroll
                for (int k = 0; k < 8; ++k) gm[k] = 0.0f;  // LDS holds nothing there
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                xh[i][k] = (xh[i][k] - mean) * rstd;
                dgamma[i][k] = __builtin_fmaf(w[i][k], xh[i][k], dgamma[i][k]);
                dbeta[i][k] += w[i][k];
                w[i][k] *= gm[k];
                s0 = __builtin_fmaf(w[i][k], xh[i][k], s0);
                s1 += w[i][k];
            }
        }
        s0 = N == 16 ? row_sum(s0) : wave_sum(s0);
        if (LAYER) s1 = N == 16 ? row_sum(s1) : wave_sum(s1);
        if constexpr (W > 1) {
            if ((t & 63) == 0) {
                s_red[phase][0][wave] = s0;
                if (LAYER) s_red[phase][1][wave] = s1;
            }
            lds_barrier();
            s0 = s1 = 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                s0 += s_red[phase][0][W * team + k];
                if (LAYER) s1 += s_red[phase][1][W * team + k];
            }
        }
        if (row >= a.rows) continue;
        const float c2 = s0 * inv_n, c1 = LAYER ? s1 * inv_n : 0.0f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            float add[8];
            skip[i].values(add);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                w[i][k] = __builtin_fmaf(__builtin_fmaf(-xh[i][k], c2, w[i][k]) - c1, rstd, add[k]);
            store_values8(static_cast<T*>(a.dx) + row * a.lddx, 8 * (t + N * i), cols, w[i]);
        }
    }
    if (a.parts == nullptr) return;
    float* out = a.parts + (int64_t)blockIdx.x * 2 * a.ldparts;
    if constexpr (kTeams == 1) {
#pragma unroll
        for (int i = 0; i < I; ++i) {
            store_values8(out, 8 * (t + N * i), cols, dgamma[i]);
            store_values8(out + a.ldparts, 8 * (t + N * i), cols, dbeta[i]);
        }
    } else {
        static_assert(I == 1, "a column group per thread");
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            __syncthreads();
            store_values8(s_team[team], 8 * t, kCols, m == 0 ? dgamma[0] : dbeta[0]);
            __syncthreads();
            for (int c = threadIdx.x; c < cols; c += 1024) {
                float v = 0.0f;
#pragma unroll
                for (int k = 0; k < kTeams; ++k) v += s_team[k][c];
                out[m * a.ldparts + c] = v;
            }
        }
    }
}

// Sum of the P partial rows: 64 columns per work-group, 16 waves that take
// every 16th partial, joined in order.  blockIdx.y: 0 gamma, 1 beta.
// (256 partials of 7168 columns: 5 us; 512 with four waves took 38.)
__global__ __launch_bounds__(1024) void layernorm_parts_kernel(const float* __restrict__ parts, int64_t ldparts, int P,
                                                               int64_t cols, float* dgamma, float* dbeta,
                                                               int accumulate) {
    __shared__ float s_sum[16][64];
    float* out = blockIdx.y == 0 ? dgamma : dbeta;
    if (out == nullptr) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float v = 0.0f;
    if (c < cols) {
        const float* from = parts + blockIdx.y * ldparts + c;
#pragma unroll 8
        for (int p = wave; p < P; p += 16) v += from[(int64_t)p * 2 * ldparts];
    }
    s_sum[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && c < cols) {
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < 16; ++w) v += s_sum[w][lane];
        out[c] = accumulate ? out[c] + v : v;
    }
}

// ----------------------------------------------------------------------------
// Launchers (arguments already validated by the API layer).
// ----------------------------------------------------------------------------
namespace {

constexpr int kMaxParts = 256;  // work-groups (and partial sums) of a backward pass

// The power of two 2^-ceil(log2(n)/2): deviations are scaled by it before they
// are squared, so the sum of n squares overflows only where their mean does.
float shrink_of(int64_t n) {
    float c = 1.0f;
    for (int64_t m = 1; m < n; m *= 4) c *= 0.5f;
    return c;
}

// Below this eps the squares of small deviations are summed in fp64.  (In fp32
// a square that is no normal number is off by up to 2^-150, which the scaling
// makes 2^-136 of the mean square: nothing next to a larger eps.)
constexpr float kTinyEps = 0x1p-100f;

template <typename S, typename T, int W, int I>
void launch_row(const LayernormArgs& a, hipStream_t st) {
    const int64_t x = std::min<int64_t>(a.rows, 1 << 20);  // a grid has fewer than 2^32 threads along x
    const dim3 grid((unsigned)x, (unsigned)((a.rows + x - 1) / x)), block(64 * W);
    if (a.layer && a.pow2) hipLaunchKernelGGL((layernorm_row_kernel<S, T, W, I, true, true>), grid, block, 0, st, a);
    else if (a.layer) hipLaunchKernelGGL((layernorm_row_kernel<S, T, W, I, true, false>), grid, block, 0, st, a);
    else if (a.pow2) hipLaunchKernelGGL((layernorm_row_kernel<S, T, W, I, false, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((layernorm_row_kernel<S, T, W, I, false, false>), grid, block, 0, st, a);
}

template <typename S, typename T, int N, int I, int G>
void launch_teams(const LayernormArgs& a, hipStream_t st) {
    constexpr int64_t kTeams = kTeamThreads / N;
    const int64_t groups = G * (int64_t)compute_units();
    const int64_t per = ((a.rows + groups - 1) / groups + kTeams - 1) / kTeams * kTeams;
    const dim3 grid((unsigned)((a.rows + per - 1) / per)), block(kTeamThreads);
    const int n = (int)per;
    // Rows of whole groups of eight columns go without the masks of a partial
    // one, which pay from four groups per lane on (8192x7168 bf16, codes: 50
    // against 61 us; with one or two groups the time is the same).
    auto launch = [&](auto whole) {
        constexpr bool kWhole = decltype(whole)::value;
        if (a.layer && a.pow2)
            hipLaunchKernelGGL((layernorm_team_kernel<S, T, N, I, G, true, true, kWhole>), grid, block, 0, st, a, n);
        else if (a.layer)
            hipLaunchKernelGGL((layernorm_team_kernel<S, T, N, I, G, true, false, kWhole>), grid, block, 0, st, a, n);
        else if (a.pow2)
            hipLaunchKernelGGL((layernorm_team_kernel<S, T, N, I, G, false, true, kWhole>), grid, block, 0, st, a, n);
        else
            hipLaunchKernelGGL((layernorm_team_kernel<S, T, N, I, G, false, false, kWhole>), grid, block, 0, st, a, n);
    };
    if constexpr (I >= 4 && sizeof(S) == 4) {
        if (a.cols % 8 == 0) return launch(std::true_type{});
    }
    launch(std::false_type{});
}

// Rows per compute unit from which teams are faster than a work-group per row.
// (bf16 with values, then fp32 layer norm into codes, teams against work-groups
// in us, at 1300 and 1800 rows on 256 compute units: 1024 columns 4.4 and 4.6,
// 4.5 and 5.5; 4.5 and 5.0, 4.6 and 5.6; 2048 columns 5.5 and 5.2, 6.0 and 6.4;
// 6.7 and 5.8, 7.5 and 7.0; 4096 columns 8.6 and 12.2, 9.6 and 15.5; 10.2 and
// 13.7, 11.2 and 17.8; 8192 columns 16.1 and 16.1, 18.5 and 20.2; 21.4 and 20.0,
// 22.4 and 25.7.  512x4096: 5.8 and 5.6; 6.4 and 6.1.)
int rows_for_teams(int64_t cols) { return cols <= 1024 ? 5 : cols <= 2048 ? 8 : cols <= 4096 ? 4 : 6; }

// Many rows, and narrow ones, go to teams; few wide rows get a work-group
// each.  Four groups per lane carry a row's fixed work best (16384x4096 bf16,
// codes: 51 us with 128 lanes a row, 56 with 256 lanes of two groups).
// Registers and LDS decide how many work-groups share a compute unit.
template <typename T>
void launch_forward_for(const LayernormArgs& a, hipStream_t st) {
    constexpr int kShare = sizeof(T) == 2 ? 3 : 2;
    const bool many = a.rows >= rows_for_teams(a.cols) * (int64_t)compute_units();
    if (a.cols <= 128) launch_teams<float, T, 16, 1, 4>(a, st);
    else if (a.cols <= 512) launch_teams<float, T, 64, 1, 4>(a, st);
    else if (a.cols <= 1024 && many) launch_teams<float, T, 64, 2, kShare>(a, st);
    else if (a.cols <= 2048 && many) launch_teams<float, T, 64, 4, 2>(a, st);
    else if (a.cols <= 2048) launch_row<float, T, 4, 1>(a, st);
    else if (a.cols <= 4096 && many) launch_teams<float, T, 128, 4, 2>(a, st);
    else if (a.cols <= 8192 && many) launch_teams<float, T, 256, 4, 2>(a, st);
    else if (a.cols <= 8192) launch_row<float, T, 16, 1>(a, st);
    else launch_row<float, T, 16, 2>(a, st);
}

// With the sums of squares in fp64 (8192x7168 bf16: RMS norm with values 65 us
// against 56, layer norm into codes 60 against 45).  Fewer layouts: a tiny eps
// is rare.
template <typename T>
void launch_forward_tiny_eps(const LayernormArgs& a, hipStream_t st) {
    if (a.cols <= 128) launch_teams<double, T, 16, 1, 4>(a, st);
    else if (a.cols <= 512) launch_teams<double, T, 64, 1, 4>(a, st);
    else if (a.cols <= 2048) launch_teams<double, T, 64, 4, 2>(a, st);
    else if (a.cols <= 8192) launch_teams<double, T, 256, 4, 2>(a, st);
    else launch_row<double, T, 16, 2>(a, st);
}

template <typename T, int N, int I>
void launch_backward(const LayernormBackwardArgs& a, int parts, hipStream_t st) {
    if (a.layer)
        hipLaunchKernelGGL((layernorm_backward_kernel<T, N, I, true>), dim3((unsigned)parts), dim3(1024), 0, st, a);
    else
        hipLaunchKernelGGL((layernorm_backward_kernel<T, N, I, false>), dim3((unsigned)parts), dim3(1024), 0, st, a);
}

// Lanes of a row in the backward pass.
int backward_lanes(int64_t cols) {
    int n = 64;
    while (n < 1024 && 8 * n < cols) n *= 2;
    return cols <= 128 ? 16 : n;
}

template <typename T>
void launch_backward_for(const LayernormBackwardArgs& a, int parts, hipStream_t st) {
    switch (backward_lanes(a.cols)) {
        case 16: launch_backward<T, 16, 1>(a, parts, st); break;
        case 64: launch_backward<T, 64, 1>(a, parts, st); break;
        case 128: launch_backward<T, 128, 1>(a, parts, st); break;
        case 256: launch_backward<T, 256, 1>(a, parts, st); break;
        case 512: launch_backward<T, 512, 1>(a, parts, st); break;
        default:
            if (a.cols <= 8192) launch_backward<T, 1024, 1>(a, parts, st);
            else launch_backward<T, 1024, 2>(a, parts, st);
    }
}

// Work-groups of a backward pass: one per compute unit of an MI355X, fewer
// where the rows do not go round.
int backward_parts(int64_t rows, int64_t cols) {
    const int64_t teams = 1024 / backward_lanes(cols);
    return (int)std::min<int64_t>((rows + teams - 1) / teams, kMaxParts);
}
int64_t parts_ld(int64_t cols) { return (cols + 7) / 8 * 8; }

}  // namespace

int64_t layernorm_backward_bytes(int64_t rows, int64_t cols) {
    return (int64_t)backward_parts(rows, cols) * 2 * parts_ld(cols) * 4;
}

hipError_t launch_layernorm(LayernormArgs a, hipStream_t st) {
    a.shrink = shrink_of(a.cols);
    if (a.x_dtype == kDtypeBF16) {
        if (a.eps < kTinyEps) launch_forward_tiny_eps<uint16_t>(a, st);
        else launch_forward_for<uint16_t>(a, st);
    } else {
        if (a.eps < kTinyEps) launch_forward_tiny_eps<float>(a, st);
        else launch_forward_for<float>(a, st);
    }
    return hipGetLastError();
}

hipError_t launch_layernorm_backward(LayernormBackwardArgs a, void* workspace, hipStream_t st) {
    const int parts = backward_parts(a.rows, a.cols);  // 0 rows: only the sums of nothing are written
    const bool weights = a.dgamma || a.dbeta;
    a.parts = weights ? static_cast<float*>(workspace) : nullptr;
    a.ldparts = parts_ld(a.cols);
    if (parts > 0) {
        if (a.dtype == kDtypeBF16) launch_backward_for<uint16_t>(a, parts, st);
        else launch_backward_for<float>(a, parts, st);
    }
    if (weights)
        hipLaunchKernelGGL(layernorm_parts_kernel, dim3((unsigned)((a.cols + 63) / 64), 2), dim3(1024), 0, st, a.parts,
                           a.ldparts, parts, a.cols, a.dgamma, a.dbeta, a.accumulate);
    return hipGetLastError();
}

}  // namespace fp8q
