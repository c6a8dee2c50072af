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
// this kernel as those codes.  Every sum is fp32.
//
// One work-group owns a row and holds it in registers, so the mean, the sum
// of squared deviations (a second pass, over registers: no cancellation) and
// the result come from one read of the row.
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

// Sums of N values over the work-group's W waves; every thread receives them.
// `red` may be used again after the next barrier that follows the return.
template <int W, int N>
__device__ __forceinline__ void block_sum(float v[N], float (*red)[16]) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = wave_sum(v[k]);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int k = 0; k < N; ++k) red[k][threadIdx.x >> 6] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            v[k] = red[k][0];
#pragma unroll
            for (int w = 1; w < W; ++w) v[k] += red[k][w];
        }
    }
}

}  // namespace

// ----------------------------------------------------------------------------
// Forward.  W waves hold I groups of eight columns per thread: thread t has
// columns 8*(t + 64*W*i) .. +7, so 16 neighbouring lanes hold one 128-column
// tile and a tile maximum is a DPP row maximum.
// ----------------------------------------------------------------------------
template <typename T, int W, int I, bool LAYER, bool POW2>
__global__ __launch_bounds__(64 * W) void layernorm_kernel(LayernormArgs a) {
    __shared__ float s_red[2][1][16];
    const int64_t cols = a.cols;
    const float n = (float)cols;
    int parity = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float v[I][8];
        float sum[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < I; ++i) {
            Raw8<T> raw;
            load_row8(raw, static_cast<const T*>(a.x) + row * a.ldx, 8 * (threadIdx.x + 64 * W * i), cols, false);
            raw.values(v[i]);
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[0] += v[i][k];
        }
        float mean = 0.0f;
        if constexpr (LAYER) {
            block_sum<W, 1>(sum, s_red[0]);
            mean = sum[0] / n;
        }
        float sq[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < I; ++i) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int64_t c = 8 * (threadIdx.x + 64 * W * i) + k;
                v[i][k] = c < cols ? v[i][k] - mean : 0.0f;
                sq[0] += (v[i][k] * a.shrink) * (v[i][k] * a.shrink);
            }
        }
        block_sum<W, 1>(sq, s_red[LAYER ? 1 : parity]);
        parity ^= 1;
        const float rstd = 1.0f / sqrtf(sq[0] / (n * a.shrink * a.shrink) + a.eps);
        if (threadIdx.x == 0) {
            if (LAYER && a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int64_t c = 8 * (threadIdx.x + 64 * W * i);
            float gm[8], bt[8];
            load_weights8(a.gamma, a.w_dtype, c, cols, 1.0f, gm);
            load_weights8(a.beta, a.w_dtype, c, cols, 0.0f, bt);
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[i][k] = v[i][k] * rstd * gm[k] + bt[k];
                if (c + k < cols) m = max(m, abs_bits(v[i][k]));
            }
            if (a.y) {
                if (a.y_dtype == kDtypeBF16)
                    store_values8(static_cast<uint16_t*>(a.y) + row * a.ldy, c, cols, v[i]);
                else
                    store_values8(static_cast<float*>(a.y) + row * a.ldy, c, cols, v[i]);
            }
            if (a.q) {
                const TileScale t = make_scale_mode<POW2>(row_max_u32(m));
                if (c < cols) {
                    if ((threadIdx.x & 15) == 0) a.s[(c >> 7) * a.lds + row] = t.s;
                    const uint32_t w0 = encode4_any<POW2>(v[i][0], v[i][1], v[i][2], v[i][3], t);
                    const uint32_t w1 = encode4_any<POW2>(v[i][4], v[i][5], v[i][6], v[i][7], t);
                    store8(a.q + row * a.ldq, c, cols, w0, w1);
                }
            }
        }
    }
}

// ----------------------------------------------------------------------------
// Backward.  Work-group p of P handles rows p, p+P, ...: thread columns as in
// the forward pass, so the sums over rows stay in registers until the end,
// where they go to part[p][gamma|beta][cols]; layernorm_parts_kernel adds the
// P partial sums in order, so repeated calls give the same bits.
// ----------------------------------------------------------------------------
template <typename T, int W, int I, bool LAYER>
__global__ __launch_bounds__(64 * W) void layernorm_backward_kernel(LayernormBackwardArgs a) {
    __shared__ float s_red[2][2][16];
    const int64_t cols = a.cols;
    const float inv_n = 1.0f / (float)cols;
    float dgamma[I][8], dbeta[I][8];
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) dgamma[i][k] = dbeta[i][k] = 0.0f;
    int parity = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float mean = LAYER ? a.mean[row] : 0.0f;
        const float rstd = a.rstd[row];
        float xh[I][8], w[I][8];
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int64_t c = 8 * (threadIdx.x + 64 * W * i);
            Raw8<T> raw;
            float gm[8];
            load_row8(raw, static_cast<const T*>(a.x) + row * a.ldx, c, cols, false);
            raw.values(xh[i]);
            load_row8(raw, static_cast<const T*>(a.dy) + row * a.lddy, c, cols, false);
            raw.values(w[i]);  // dy, zero beyond the row's end
            load_weights8(a.gamma, a.w_dtype, c, cols, 1.0f, gm);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                xh[i][k] = (xh[i][k] - mean) * rstd;
                dgamma[i][k] += w[i][k] * xh[i][k];
                dbeta[i][k] += w[i][k];
                w[i][k] *= gm[k];
                sum[0] += w[i][k] * xh[i][k];
                sum[1] += w[i][k];
            }
        }
        block_sum<W, 2>(sum, s_red[parity]);
        parity ^= 1;
        const float c2 = sum[0] * inv_n, c1 = LAYER ? sum[1] * inv_n : 0.0f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int64_t c = 8 * (threadIdx.x + 64 * W * i);
            float add[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (a.skip) {
                Raw8<T> raw;
                load_row8(raw, static_cast<const T*>(a.skip) + row * a.ldskip, c, cols, false);
                raw.values(add);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) w[i][k] = (w[i][k] - xh[i][k] * c2 - c1) * rstd + add[k];
            store_values8(static_cast<T*>(a.dx) + row * a.lddx, c, cols, w[i]);
        }
    }
    if (a.parts == nullptr) return;
    float* out = a.parts + (int64_t)blockIdx.x * 2 * a.ldparts;
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int64_t c = 8 * (threadIdx.x + 64 * W * i);
        store_values8(out, c, cols, dgamma[i]);
        store_values8(out + a.ldparts, c, cols, dbeta[i]);
    }
}

// Sum of the P partial rows: 64 columns per work-group, 4 waves that take
// every fourth partial, joined in order.  blockIdx.y: 0 gamma, 1 beta.
__global__ __launch_bounds__(256) void layernorm_parts_kernel(const float* __restrict__ parts, int64_t ldparts, int P,
                                                              int64_t cols, float* dgamma, float* dbeta,
                                                              int accumulate) {
    __shared__ float s_sum[4][64];
    float* out = blockIdx.y == 0 ? dgamma : dbeta;
    if (out == nullptr) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float v = 0.0f;
    if (c < cols)
        for (int p = wave; p < P; p += 4) v += parts[((int64_t)p * 2 + blockIdx.y) * ldparts + c];
    s_sum[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && c < cols) {
        v = (s_sum[0][lane] + s_sum[1][lane]) + (s_sum[2][lane] + s_sum[3][lane]);
        out[c] = accumulate ? out[c] + v : v;
    }
}

// ----------------------------------------------------------------------------
// Launchers (arguments already validated by the API layer).
// ----------------------------------------------------------------------------
namespace {

constexpr int kMaxParts = 512;  // work-groups (and partial sums) of a backward pass

// The power of two 2^-ceil(log2(n)/2): deviations are scaled by it before they
// are squared, so the sum of n squares overflows only where their mean does.
float shrink_of(int64_t n) {
    float c = 1.0f;
    for (int64_t m = 1; m < n; m *= 4) c *= 0.5f;
    return c;
}

template <typename T, int W, int I>
void launch_forward(const LayernormArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)std::min<int64_t>(a.rows, 1 << 20)), block(64 * W);
    if (a.layer && a.pow2)
        hipLaunchKernelGGL((layernorm_kernel<T, W, I, true, true>), grid, block, 0, st, a);
    else if (a.layer)
        hipLaunchKernelGGL((layernorm_kernel<T, W, I, true, false>), grid, block, 0, st, a);
    else if (a.pow2)
        hipLaunchKernelGGL((layernorm_kernel<T, W, I, false, true>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((layernorm_kernel<T, W, I, false, false>), grid, block, 0, st, a);
}

template <typename T>
void launch_forward_for(const LayernormArgs& a, hipStream_t st) {
    if (a.cols <= 512)
        launch_forward<T, 1, 1>(a, st);
    else if (a.cols <= 2048)
        launch_forward<T, 4, 1>(a, st);
    else if (a.cols <= 8192)
        launch_forward<T, 4, 4>(a, st);
    else
        launch_forward<T, 16, 2>(a, st);
}

template <typename T, int W, int I>
void launch_backward(const LayernormBackwardArgs& a, int parts, hipStream_t st) {
    if (a.layer)
        hipLaunchKernelGGL((layernorm_backward_kernel<T, W, I, true>), dim3((unsigned)parts), dim3(64 * W), 0, st, a);
    else
        hipLaunchKernelGGL((layernorm_backward_kernel<T, W, I, false>), dim3((unsigned)parts), dim3(64 * W), 0, st, a);
}

template <typename T>
void launch_backward_for(const LayernormBackwardArgs& a, int parts, hipStream_t st) {
    if (a.cols <= 512)
        launch_backward<T, 1, 1>(a, parts, st);
    else if (a.cols <= 2048)
        launch_backward<T, 4, 1>(a, parts, st);
    else if (a.cols <= 8192)
        launch_backward<T, 4, 4>(a, parts, st);
    else
        launch_backward<T, 16, 2>(a, parts, st);
}

int backward_parts(int64_t rows) { return (int)std::min<int64_t>(rows, kMaxParts); }
int64_t parts_ld(int64_t cols) { return (cols + 7) / 8 * 8; }

}  // namespace

int64_t layernorm_backward_bytes(int64_t rows, int64_t cols) {
    return (int64_t)backward_parts(rows) * 2 * parts_ld(cols) * 4;
}

hipError_t launch_layernorm(LayernormArgs a, hipStream_t st) {
    a.shrink = shrink_of(a.cols);
    if (a.x_dtype == kDtypeBF16) launch_forward_for<uint16_t>(a, st);
    else launch_forward_for<float>(a, st);
    return hipGetLastError();
}

hipError_t launch_layernorm_backward(LayernormBackwardArgs a, void* workspace, hipStream_t st) {
    const int parts = backward_parts(a.rows);  // 0 rows: only the sums of nothing are written
    const bool weights = a.dgamma || a.dbeta;
    a.parts = weights ? static_cast<float*>(workspace) : nullptr;
    a.ldparts = parts_ld(a.cols);
    if (parts > 0) {
        if (a.dtype == kDtypeBF16) launch_backward_for<uint16_t>(a, parts, st);
        else launch_backward_for<float>(a, parts, st);
    }
    if (weights)
        hipLaunchKernelGGL(layernorm_parts_kernel, dim3((unsigned)((a.cols + 63) / 64), 2), dim3(256), 0, st, a.parts,
                           a.ldparts, parts, a.cols, a.dgamma, a.dbeta, a.accumulate);
    return hipGetLastError();
}

}  // namespace fp8q
