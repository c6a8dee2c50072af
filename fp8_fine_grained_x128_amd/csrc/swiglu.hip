// swiglu.hip -- SwiGLU between the two FP8 GEMMs of a feed-forward block,
// with its inputs kept as 8-bit checkpoints, and its backward pass from them.
//
//   h  = g sigma(g) u,  sigma(x) = 1 / (1 + exp(-x))
//   du = dh g sigma(g)
//   dg = dh u sigma(g) (1 + g (1 - sigma(g)))
//
// The pages cache the SwiGLU's inputs (in FP8) and recompute its output in
// the backward pass (page 1, why-be.why-be.co.kr wr_id=65900, passage on
// caching the inputs of the SwiGLU operator; same page, FP8-cached
// activations).  The checkpoint is codes with 1x128 scales, the layout of the
// activation quantizer; the backward kernels work on the checkpoint's values
// fl32(dec(q) * s), so they differentiate the function at those values.
//
// All arithmetic between the stored types is fp32, each value rounded once
// when it is encoded or stored.
#include <algorithm>
#include <type_traits>

#include "launch.hpp"
#include "tile_io.hpp"

namespace fp8q {

namespace {

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

struct SwigluPoint {
    float h, dg, du;
};

// The three results at one element.
__device__ __forceinline__ SwigluPoint swiglu_point(float g, float u, float dh) {
    const float sg = sigmoid(g);
    const float a = g * sg;  // silu(g)
    SwigluPoint p;
    p.h = a * u;
    p.du = dh * a;
    p.dg = dh * u * sg * (1.0f + g * (1.0f - sg));
    return p;
}

// Eight checkpoint values at column c of a row: codes times the row's scale.
__device__ __forceinline__ uint2 load_codes8(const uint8_t* row, int64_t c, int64_t cols) {
    if (c + 8 <= cols) return *reinterpret_cast<const uint2*>(row + c);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int b = 0; b < 8; ++b)
        if (c + b < cols) w[b >> 2] |= (uint32_t)row[c + b] << (8 * (b & 3));
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void decode8(uint2 w, float s, float v[8]) {
    decode4(w.x, v);
    decode4(w.y, v + 4);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= s;
}

__device__ __forceinline__ uint32_t amax8(const float v[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, abs_bits(v[k]));
    return m;
}

// One 1x128 tile of 16 lanes with eight values each: scale and codes of row
// `row`, columns c .. c+7 of this lane.
template <bool POW2>
__device__ __forceinline__ void put_tile(const float v[8], int64_t row, int64_t c, int64_t cols, uint8_t* q,
                                         int64_t ldq, float* s, int64_t lds) {
    const TileScale t = make_scale_mode<POW2>(row_max_u32(amax8(v)));
    if (c >= cols) return;
    if ((threadIdx.x & 15) == 0) s[(c >> 7) * lds + row] = t.s;
    const uint32_t w0 = encode4_any<POW2>(v[0], v[1], v[2], v[3], t);
    const uint32_t w1 = encode4_any<POW2>(v[4], v[5], v[6], v[7], t);
    store8(q + row * ldq, c, cols, w0, w1);
}

}  // namespace

// ----------------------------------------------------------------------------
// Forward: a wave per row and 512 columns, eight columns per lane.
// ----------------------------------------------------------------------------
template <typename T, bool POW2, bool KEEP>
__global__ __launch_bounds__(256) void swiglu_quantize_kernel(SwigluArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t row = ((int64_t)blockIdx.z * 65535 + blockIdx.y) * 4 + (threadIdx.x >> 6);
    if (row >= a.rows) return;
    const int64_t c = (int64_t)blockIdx.x * 512 + 8 * lane;
    Raw8<T> raw;
    float g[8], u[8], h[8];
    load_row8(raw, static_cast<const T*>(a.g) + row * a.ldgu, c, a.cols, false);
    raw.values(g);
    load_row8(raw, static_cast<const T*>(a.u) + row * a.ldgu, c, a.cols, false);
    raw.values(u);
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = g[k] * sigmoid(g[k]) * u[k];
    put_tile<POW2>(h, row, c, a.cols, a.qh, a.ldqh, a.sh, a.ldsh);
    if constexpr (KEEP) {
        put_tile<POW2>(g, row, c, a.cols, a.qg, a.ldq, a.sg, a.lds);
        put_tile<POW2>(u, row, c, a.cols, a.qu, a.ldq, a.su, a.lds);
    }
}

// ----------------------------------------------------------------------------
// Backward into plain gradients.
// ----------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(256) void swiglu_backward_kernel(SwigluBackwardArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t row = ((int64_t)blockIdx.z * 65535 + blockIdx.y) * 4 + (threadIdx.x >> 6);
    if (row >= a.rows) return;
    const int64_t c = (int64_t)blockIdx.x * 512 + 8 * lane;
    if (c >= a.cols) return;
    float g[8], u[8], dh[8], dg[8], du[8];
    Raw8<T> raw;
    load_row8(raw, static_cast<const T*>(a.dh) + row * a.lddh, c, a.cols, false);
    raw.values(dh);
    decode8(load_codes8(a.qg + row * a.ldq, c, a.cols), a.sg[(c >> 7) * a.lds + row], g);
    decode8(load_codes8(a.qu + row * a.ldq, c, a.cols), a.su[(c >> 7) * a.lds + row], u);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const SwigluPoint p = swiglu_point(g[k], u[k], dh[k]);
        dg[k] = p.dg;
        du[k] = p.du;
    }
    store_values8(static_cast<T*>(a.dg) + row * a.ldd, c, a.cols, dg);
    store_values8(static_cast<T*>(a.du) + row * a.ldd, c, a.cols, du);
}

// ----------------------------------------------------------------------------
// Backward into FP8 operands: dg and du in 1x128 tiles (the Dgrad operand)
// and, transposed, in 128x1 tiles (the Wgrad operand of the gate and up
// projections), and the recomputed h, transposed, in 128x1 tiles (the Wgrad
// operand of the down projection).
// A work-group of 8 waves takes 128 rows x 128 columns: thread t has columns
// 8*(t%16) .. +7 of rows 4*(t/16) .. +3, so a row's tile maximum is a DPP row
// maximum and a column's goes across the lanes of a wave and then through
// LDS.  The codes of the 128x1 tiles are transposed in LDS, whose 16-byte
// units are XOR-swizzled by ((column >> 3) & 7).
// ----------------------------------------------------------------------------
template <typename T, bool POW2>
__global__ __launch_bounds__(512) void swiglu_backward_quantize_kernel(SwigluBackwardArgs a) {
    __shared__ uint32_t s_part[3][8][128];
    __shared__ float2 s_sr[3][128];
    __shared__ __align__(16) uint8_t s_tile[3][128 * 128];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int cg = t & 15, rg = t >> 4;
    const int64_t r0 = (int64_t)blockIdx.y * 128, c0 = (int64_t)blockIdx.x * 128;
    const int64_t c = c0 + 8 * cg;

    float v[3][4][8];  // dg, du, h
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + 4 * rg + i;
        float g[8], u[8], dh[8];
        if (r < a.rows && c < a.cols) {
            Raw8<T> raw;
            load_row8(raw, static_cast<const T*>(a.dh) + r * a.lddh, c, a.cols, false);
            raw.values(dh);
            decode8(load_codes8(a.qg + r * a.ldq, c, a.cols), a.sg[(c >> 7) * a.lds + r], g);
            decode8(load_codes8(a.qu + r * a.ldq, c, a.cols), a.su[(c >> 7) * a.lds + r], u);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) g[k] = u[k] = dh[k] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const SwigluPoint p = swiglu_point(g[k], u[k], dh[k]);
            v[0][i][k] = p.dg;
            v[1][i][k] = p.du;
            v[2][i][k] = p.h;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + 4 * rg + i;
        if (r < a.rows) {  // uniform over the 16 lanes of the tile
            put_tile<POW2>(v[0][i], r, c, a.cols, a.qdg, a.ldqd, a.sdg, a.ldsd);
            put_tile<POW2>(v[1][i], r, c, a.cols, a.qdu, a.ldqd, a.sdu, a.ldsd);
        }
    }
#pragma unroll
    for (int m = 0; m < 3; ++m) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t x = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) x = max(x, abs_bits(v[m][i][k]));
            x = max(x, (uint32_t)__shfl_xor((int)x, 16));
            x = max(x, (uint32_t)__shfl_xor((int)x, 32));
            if (lane < 16) s_part[m][wave][8 * cg + k] = x;
        }
    }
    __syncthreads();
    if (t < 384) {
        const int m = t >> 7, ch = t & 127;
        uint32_t x = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) x = max(x, s_part[m][w][ch]);
        const TileScale ts = make_scale_mode<POW2>(x);
        s_sr[m][ch] = make_float2(ts.s, ts.r);
        float* st = m == 0 ? a.sdgt : m == 1 ? a.sdut : a.sht;
        const int64_t ldst = m == 2 ? a.ldsht : a.ldst;
        if (c0 + ch < a.cols) st[(r0 >> 7) * ldst + c0 + ch] = ts.s;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 3; ++m) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int ch = 8 * cg + k;
            const float2 sr = s_sr[m][ch];
            const uint32_t w = encode4_any<POW2>(v[m][0][k], v[m][1][k], v[m][2][k], v[m][3][k], scale_from(sr.x, sr.y));
            const int unit = (rg >> 2) ^ (cg & 7);
            *reinterpret_cast<uint32_t*>(s_tile[m] + ch * 128 + 16 * unit + 4 * (rg & 3)) = w;
        }
    }
    __syncthreads();
    // thread t: column 64*j + t/8, 16 tokens of physical unit t%8
#pragma unroll
    for (int m = 0; m < 3; ++m) {
        uint8_t* qt = m == 0 ? a.qdgt : m == 1 ? a.qdut : a.qht;
        const int64_t ldqt = m == 2 ? a.ldqht : a.ldqt;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int ch = 64 * j + (t >> 3), unit = t & 7;
            const uint4 val = *reinterpret_cast<const uint4*>(s_tile[m] + ch * 128 + 16 * unit);
            const int64_t tok = r0 + 16 * (unit ^ ((ch >> 3) & 7));
            if (c0 + ch >= a.cols) continue;
            uint8_t* dst = qt + (c0 + ch) * ldqt + tok;
            if (tok + 16 <= a.rows) {
                *reinterpret_cast<uint4*>(dst) = val;
            } else {
                const uint32_t wv[4] = {val.x, val.y, val.z, val.w};
#pragma unroll
                for (int b = 0; b < 16; ++b)
                    if (tok + b < a.rows) dst[b] = (uint8_t)((wv[b >> 2] >> (8 * (b & 3))) & 0xffu);
            }
        }
    }
}

// ----------------------------------------------------------------------------
// Launchers (arguments already validated by the API layer).
// ----------------------------------------------------------------------------
namespace {

dim3 row_grid(int64_t rows, int64_t cols) {
    const int64_t groups = (rows + 3) / 4;
    return dim3((unsigned)((cols + 511) / 512), (unsigned)std::min<int64_t>(groups, 65535),
                (unsigned)((groups + 65534) / 65535));
}

template <typename T, bool POW2>
void launch_forward(const SwigluArgs& a, hipStream_t st) {
    if (a.qg)
        hipLaunchKernelGGL((swiglu_quantize_kernel<T, POW2, true>), row_grid(a.rows, a.cols), dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((swiglu_quantize_kernel<T, POW2, false>), row_grid(a.rows, a.cols), dim3(256), 0, st, a);
}

template <typename T>
void launch_backward_quantize(const SwigluBackwardArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)((a.cols + 127) / 128), (unsigned)((a.rows + 127) / 128));
    if (a.pow2)
        hipLaunchKernelGGL((swiglu_backward_quantize_kernel<T, true>), grid, dim3(512), 0, st, a);
    else
        hipLaunchKernelGGL((swiglu_backward_quantize_kernel<T, false>), grid, dim3(512), 0, st, a);
}

}  // namespace

hipError_t launch_swiglu_quantize(const SwigluArgs& a, hipStream_t st) {
    if (a.dtype == kDtypeBF16) {
        if (a.pow2) launch_forward<uint16_t, true>(a, st);
        else launch_forward<uint16_t, false>(a, st);
    } else {
        if (a.pow2) launch_forward<float, true>(a, st);
        else launch_forward<float, false>(a, st);
    }
    return hipGetLastError();
}

hipError_t launch_swiglu_backward(const SwigluBackwardArgs& a, hipStream_t st) {
    const dim3 grid = row_grid(a.rows, a.cols);
    if (a.dtype == kDtypeBF16)
        hipLaunchKernelGGL((swiglu_backward_kernel<uint16_t>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((swiglu_backward_kernel<float>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_swiglu_backward_quantize(const SwigluBackwardArgs& a, hipStream_t st) {
    if (a.dtype == kDtypeBF16) launch_backward_quantize<uint16_t>(a, st);
    else launch_backward_quantize<float>(a, st);
    return hipGetLastError();
}

}  // namespace fp8q
