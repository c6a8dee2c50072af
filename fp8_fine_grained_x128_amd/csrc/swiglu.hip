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

// Up to here exp(x) and exp(-x) and their reciprocals are normal numbers.
constexpr float kNear = 87.0f;

// w with w * w = exp(x) for x < 0.  The two factors keep exp(x) and x exp(x)
// down to the subnormal numbers, where 2^p itself is flushed to zero.
__device__ __forceinline__ float root_exp(float x) { return __builtin_amdgcn_exp2f(x * 0x1.715476p-1f); }

// 1 / (1 + exp(-x)) for x >= -kNear from the hardware's 2^p and reciprocal,
// each good to a unit in the last place; with the rounding of p = -x log2(e),
// which the sum with 1 weighs down, the relative error stays below
// (5 + 1.3 |x| (1 - sigma)) 2^-24: 6 2^-24 of the sigmoid for open gates, and
// never more than that of 1.  Both backward forms use it, so that the codes of
// one are the quantizer's codes of the other's gradients bit for bit.  (Against
// expf and a division, or a corrected p and a Newton step: 7 to 25
// instructions fewer per element, in kernels that issue 35 to 55; the form
// into FP8 operands takes 6 % longer with them, the gradients themselves are of
// inputs that 8 bits hold.)
__device__ __forceinline__ float sigmoid_near(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -0x1.715476p+0f));
}

// For any x, with the bits of sigmoid_near where that holds.
__device__ __forceinline__ float sigmoid(float x) {
    const float w = root_exp(x), s = sigmoid_near(x);
    return x < -kNear ? w * w : s;
}

// x / (1 + exp(-x)) for |x| <= kNear, with the quotient corrected from its
// remainder, which leaves about the error of a division.  (The forward pass
// has room for the two instructions; feeding p's rounding back too would cost
// 4 %.)
__device__ __forceinline__ float silu_near(float x) {
    const float d = 1.0f + __builtin_amdgcn_exp2f(x * -0x1.715476p+0f);
    const float r = __builtin_amdgcn_rcpf(d), q = x * r;
    return __builtin_fmaf(__builtin_fmaf(-d, q, x), r, q);
}

// For any x, with the bits of silu_near where that holds: beyond, the
// denominator (of x exp(x) / (1 + exp(x)) for x < 0) is 1.
__device__ __forceinline__ float silu(float x) {
    const float w = root_exp(x), q = silu_near(x);
    return x < -kNear ? x * w * w : x > kNear ? x : q;
}

struct SwigluPoint {
    float h, dg, du;
};

// The three results at one element.  NEAR: |g| <= kNear.
template <bool NEAR>
__device__ __forceinline__ SwigluPoint swiglu_point(float g, float u, float dh) {
    const float sg = NEAR ? sigmoid_near(g) : sigmoid(g);
    const float a = g * sg;  // silu(g)
    SwigluPoint p;
    p.h = a * u;
    p.du = dh * a;
    p.dg = dh * u * sg * __builtin_fmaf(g, 1.0f - sg, 1.0f);
    return p;
}

// Whether all checkpoint values of a tile with this scale are within kNear.
__device__ __forceinline__ bool near_scale(float s) { return s * kE4M3Max <= kNear; }

// Hides a wave-uniform pointer's value from the optimizer.
template <typename P>
__device__ __forceinline__ void opaque_uniform(P& p) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+s"(p));
#endif
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

// Codes of eight values of a row at q[c .. c+7], clipped to `cols`.  `fast`:
// the scale allows the reciprocal quotient.
template <bool POW2>
__device__ __forceinline__ void put_codes8(uint8_t* q, int64_t c, int64_t cols, bool fast, const float v[8], float2 sr) {
    if (fast) {
        store8(q, c, cols, encode4_sr<POW2>(v[0], v[1], v[2], v[3], sr.x, sr.y),
               encode4_sr<POW2>(v[4], v[5], v[6], v[7], sr.x, sr.y));
    } else {
        const TileScale t = scale_from(sr.x, sr.y);
        store8(q, c, cols, encode4_any<POW2>(v[0], v[1], v[2], v[3], t), encode4_any<POW2>(v[4], v[5], v[6], v[7], t));
    }
}

// Byte of 16-token unit `unit` of column `ch` in a transposed 128x128 tile of
// codes.  Units are XOR-ed with the column's group of eight, and the columns
// of the upper half trade places with their neighbours, so that the 16 column
// groups that a wave writes at once fall into different LDS banks.
__device__ __forceinline__ int tile_place(int ch, int unit) {
    return 128 * (ch ^ (ch >> 6)) + 16 * (unit ^ ((ch >> 3) & 7));
}

}  // namespace

// ----------------------------------------------------------------------------
// Forward.  A work-group takes a 512-column segment of W*R rows, a wave R of
// them, a lane eight columns of each, so a 16-lane DPP row holds one tile of
// h, g and u for every row.  One lane computes a tile's scale and passes it
// to the others through LDS.  Segments of one group of rows are dispatched
// back to back (whole rows stream).
//   Bound by memory: 8192x7168 bf16 with the checkpoint, 417 MB, takes 74 us
// (5.6 TB/s); fp32, 652 MB, 120 us.
// ----------------------------------------------------------------------------
template <typename T, int W, int R, bool POW2, bool KEEP>
__global__ __launch_bounds__(64 * W) void swiglu_quantize_kernel(SwigluArgs a) {
    constexpr int M = KEEP ? 3 : 1;  // h, and g and u
    static_assert(M * R <= 16, "a lane of the DPP row for each tile");
    __shared__ __align__(16) float2 s_sr[W][4][M * R];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane & 15;
    const int64_t row0 = (((int64_t)blockIdx.z * 65535 + blockIdx.y) * W + wave) * R;
    if (row0 >= a.rows) return;
    const int64_t seg = (int64_t)blockIdx.x * 512, c = seg + 8 * lane;
    const bool full = seg + 512 <= a.cols && row0 + R <= a.rows;
    const T* gp = static_cast<const T*>(a.g) + row0 * a.ldgu;
    const T* up = static_cast<const T*>(a.u) + row0 * a.ldgu;
    Raw8<T> rg[R], ru[R];
    if (full) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            rg[i].load_full(gp + i * a.ldgu + c);
            ru[i].load_full(up + i * a.ldgu + c);
        }
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            rg[i].zero();
            ru[i].zero();
            if (row0 + i < a.rows) {
                load_row8(rg[i], gp + i * a.ldgu, c, a.cols, false);
                load_row8(ru[i], up + i * a.ldgu, c, a.cols, false);
            }
        }
    }
    float h[R][8];
    uint32_t mine = 0;  // lane R*m + i of the DPP row: maximum of row i of h, g or u
#pragma unroll
    for (int i = 0; i < R; ++i) {
        float g[8], u[8];
        rg[i].values(g);
        ru[i].values(u);
        const uint32_t amax_g = rg[i].amax_bits();
        // gates beyond kNear are rare: without them twelve instructions an
        // element are eight (8192x7168 bf16: 73 us, 80 otherwise)
        if (wave_all(amax_g <= __float_as_uint(kNear))) {
#pragma unroll
            for (int k = 0; k < 8; ++k) h[i][k] = silu_near(g[k]) * u[k];
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) h[i][k] = silu(g[k]) * u[k];
        }
        const uint32_t amax[3] = {amax8(h[i]), amax_g, ru[i].amax_bits()};
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const uint32_t x = row_max_u32(amax[m]);
            mine = sub == R * m + i ? x : mine;
        }
    }
    bool my_fast = true;
    if (sub < M * R) {
        const TileScale t = make_scale_mode<POW2>(mine);
        s_sr[wave][lane >> 4][sub] = make_float2(t.s, t.r);
        my_fast = t.fast;
        const int64_t chunk = 4 * (int64_t)blockIdx.x + (lane >> 4), row = row0 + sub % R;
        if (row < a.rows && chunk * 128 < a.cols) {
            if (!KEEP || sub < R) a.sh[chunk * a.ldsh + row] = t.s;
            else (sub < 2 * R ? a.sg : a.su)[chunk * a.lds + row] = t.s;
        }
    }
    wave_lds_sync();
    const bool fast = wave_all(my_fast);
    if (c >= a.cols) return;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        uint8_t* q = m == 0 ? a.qh : m == 1 ? a.qg : a.qu;
        const int64_t ldq = m == 0 ? a.ldqh : a.ldq;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float v[8];
            if (m == 0) {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = h[i][k];
            } else {
                (m == 1 ? rg[i] : ru[i]).values(v);
            }
            if (full || row0 + i < a.rows)
                put_codes8<POW2>(q + (row0 + i) * ldq, c, a.cols, fast, v, s_sr[wave][lane >> 4][R * m + i]);
        }
    }
}

// ----------------------------------------------------------------------------
// Backward into plain gradients: a lane has eight columns of a row, nothing
// is shared.  Bound by memory: 8192x7168 takes 80 us in bf16 (473 MB, 5.9
// TB/s), 153 us in fp32.
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
    load_row8<T, sizeof(T) == 2>(raw, static_cast<const T*>(a.dh) + row * a.lddh, c, a.cols, false);
    raw.values(dh);
    const float sg = a.sg[(c >> 7) * a.lds + row];
    decode8(load_codes8(a.qg + row * a.ldq, c, a.cols), sg, g);
    decode8(load_codes8(a.qu + row * a.ldq, c, a.cols), a.su[(c >> 7) * a.lds + row], u);
    auto points = [&](auto near) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const SwigluPoint p = swiglu_point<decltype(near)::value>(g[k], u[k], dh[k]);
            dg[k] = p.dg;
            du[k] = p.du;
        }
    };
    if (wave_all(near_scale(sg))) points(std::true_type{});
    else points(std::false_type{});
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
// maximum and a column's goes through LDS.  The codes of the 128x1 tiles are
// transposed in LDS (tile_place).
//   8192x7168 bf16 moves 541 MB, the bytes it cannot do without, in 105 to
// 120 us (4.5 to 5.1 TB/s, run by run), with power-of-two scales in 95; fp32
// 659 MB in 140.  Memory and arithmetic share the
// bound: 48 instructions per element keep the vector units busy for two
// thirds of that, and 128 registers hold 16 waves on a compute unit.
// ----------------------------------------------------------------------------
template <typename T, bool POW2>
__global__ __launch_bounds__(512, 4) void swiglu_backward_quantize_kernel(SwigluBackwardArgs a) {
    constexpr int kRows = 4;                                   // rows per thread
    __shared__ __align__(16) float2 s_row[8][4][2 * kRows];    // [wave][row group][dg rows, du rows]: s, 1/s
    __shared__ __align__(16) float2 s_col[3][8][16];           // [column % 8][column / 8]
    __shared__ int s_slow;                                     // some column's scale needs the exact division
    // first the column maxima [3][row group][column], then the transposed codes
    __shared__ __align__(16) uint8_t s_tile[3][128 * 128];
    uint32_t(*s_part)[32][128] = reinterpret_cast<uint32_t(*)[32][128]>(&s_tile[0][0]);
    static_assert(sizeof(s_tile) == 3 * 32 * 128 * 4, "the maxima fill the tiles");
    const int t = threadIdx.x, wave = t >> 6;
    const int cg = t & 15, rg = t >> 4;
    // Eight row tiles of a column tile one after the other: both the rows and
    // the transposed rows are then written in runs (7 % faster at 8192x7168
    // than whole rows of tiles or whole columns).
    const uint32_t band = blockIdx.y / 8, height = min(8u, gridDim.y - 8 * band);
    const uint32_t in_band = blockIdx.y % 8 * gridDim.x + blockIdx.x;
    const uint32_t tile_c = in_band / height, tile_r = 8 * band + in_band % height;
    const uint32_t r0 = tile_r * 128, c0 = tile_c * 128;  // below 2^31: 32 bits spare registers here
    const uint32_t c = c0 + 8 * cg, row = r0 + kRows * rg;
    const bool full = r0 + 128 <= a.rows && c0 + 128 <= a.cols;

    Raw8<T> raw[kRows];
    uint2 qg[kRows], qu[kRows];
    float sg[kRows], su[kRows];
    if (full) {  // every load goes out before any arithmetic
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            qg[i] = load8_nt(a.qg + (row + i) * a.ldq + c);
            qu[i] = load8_nt(a.qu + (row + i) * a.ldq + c);
            raw[i].load_full(static_cast<const T*>(a.dh) + (row + i) * a.lddh + c);
            sg[i] = a.sg[tile_c * a.lds + row + i];
            su[i] = a.su[tile_c * a.lds + row + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (row + i < a.rows && c < a.cols) {
                qg[i] = load_codes8(a.qg + (row + i) * a.ldq, c, a.cols);
                qu[i] = load_codes8(a.qu + (row + i) * a.ldq, c, a.cols);
                load_row8(raw[i], static_cast<const T*>(a.dh) + (row + i) * a.lddh, c, a.cols, false);
                sg[i] = a.sg[tile_c * a.lds + row + i];
                su[i] = a.su[tile_c * a.lds + row + i];
            } else {
                qg[i] = qu[i] = make_uint2(0, 0);
                raw[i].zero();
                sg[i] = su[i] = 0.0f;
            }
        }
    }
    float v[3][kRows][8];  // dg, du, h
    bool my_near = true;
    auto points = [&](auto near, int i, uint2 qg, uint2 qu, float sg, float su, const Raw8<T>& raw) {
        float g[8], u[8], dh[8];
        decode8(qg, sg, g);
        decode8(qu, su, u);
        raw.values(dh);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const SwigluPoint p = swiglu_point<decltype(near)::value>(g[k], u[k], dh[k]);
            v[0][i][k] = p.dg;
            v[1][i][k] = p.du;
            v[2][i][k] = p.h;
        }
    };
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        points(std::true_type{}, i, qg[i], qu[i], sg[i], su[i], raw[i]);
        my_near = my_near && near_scale(sg[i]);
    }
    if (!wave_all(my_near)) {
        // Rare.  The inputs are loaded again: held until here, or a choice of
        // two ways in the loop above, they would be spilled registers (200 us
        // against 105 at 8192x7168 bf16; a sigmoid for any gate 111).
        SwigluBackwardArgs b = a;
        opaque_uniform(b.qg);
        opaque_uniform(b.qu);
        opaque_uniform(b.sg);
        opaque_uniform(b.su);
        opaque_uniform(b.dh);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (row + i >= a.rows || c >= a.cols) continue;
            Raw8<T> d;
            load_row8(d, static_cast<const T*>(b.dh) + (row + i) * a.lddh, c, a.cols, false);
            points(std::false_type{}, i, load_codes8(b.qg + (row + i) * a.ldq, c, a.cols),
                   load_codes8(b.qu + (row + i) * a.ldq, c, a.cols), b.sg[tile_c * a.lds + row + i],
                   b.su[tile_c * a.lds + row + i], d);
        }
    }
    uint32_t mine = 0;  // lane 4*m + i of a row group: maximum of row i of dg (m = 0) or du
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const uint32_t x = row_max_u32(amax8(v[m][i]));
            mine = cg == kRows * m + i ? x : mine;
        }
#pragma unroll
    for (int m = 0; m < 3; ++m) {
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] = max_abs3(max_abs2(v[m][0][k], v[m][1][k]), v[m][2][k], v[m][3][k]);
        float4* part = reinterpret_cast<float4*>(&s_part[m][rg][8 * cg]);
        part[0] = make_float4(x[0], x[1], x[2], x[3]);
        part[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
    if (t == 0) s_slow = 0;
    // 1x128 tiles: scales by one lane each, then the codes
    bool my_fast = true;
    if (cg < 2 * kRows) {
        const TileScale ts = make_scale_mode<POW2>(mine);
        s_row[wave][rg & 3][cg] = make_float2(ts.s, ts.r);
        my_fast = ts.fast;
        const uint32_t r = row + (cg & (kRows - 1));
        if (r < a.rows) (cg < kRows ? a.sdg : a.sdu)[tile_c * a.ldsd + r] = ts.s;
    }
    wave_lds_sync();
    const bool fast_rows = wave_all(my_fast);
    if (full && fast_rows) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            uint8_t* q = (m == 0 ? a.qdg : a.qdu) + row * a.ldqd + c;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const float2 sr = s_row[wave][rg & 3][kRows * m + i];
                const float* x = v[m][i];
                *reinterpret_cast<uint2*>(q + i * a.ldqd) = make_uint2(
                    encode4_sr<POW2>(x[0], x[1], x[2], x[3], sr.x, sr.y), encode4_sr<POW2>(x[4], x[5], x[6], x[7], sr.x, sr.y));
            }
        }
    } else if (c < a.cols) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            uint8_t* q = (m == 0 ? a.qdg : a.qdu) + row * a.ldqd;
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                if (row + i < a.rows)
                    put_codes8<POW2>(q + i * a.ldqd, c, a.cols, fast_rows, v[m][i], s_row[wave][rg & 3][kRows * m + i]);
        }
    }
    __syncthreads();
    if (t < 384) {
        const int m = t >> 7, ch = t & 127;
        uint32_t x = 0;
#pragma unroll
        for (int g = 0; g < 32; ++g) x = max(x, s_part[m][g][ch]);
        const TileScale ts = make_scale_mode<POW2>(x);
        s_col[m][ch & 7][ch >> 3] = make_float2(ts.s, ts.r);
        if (!ts.fast) s_slow = 1;
        float* st = m == 0 ? a.sdgt : m == 1 ? a.sdut : a.sht;
        const int64_t ldst = m == 2 ? a.ldsht : a.ldst;
        if (c0 + ch < a.cols) st[tile_r * ldst + c0 + ch] = ts.s;
    }
    __syncthreads();
    const bool fast = s_slow == 0;
#pragma unroll
    for (int m = 0; m < 3; ++m) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 sr = s_col[m][k][cg];
            const uint32_t w =
                fast ? encode4_sr<POW2>(v[m][0][k], v[m][1][k], v[m][2][k], v[m][3][k], sr.x, sr.y)
                     : encode4_any<POW2>(v[m][0][k], v[m][1][k], v[m][2][k], v[m][3][k], scale_from(sr.x, sr.y));
            *reinterpret_cast<uint32_t*>(s_tile[m] + tile_place(8 * cg + k, rg >> 2) + 4 * (rg & 3)) = w;
        }
    }
    __syncthreads();
    // thread t: columns t/8 and t/8 + 64, tokens 16*(t%8) .. +15 of the tile
    const int unit = t & 7;
    const uint32_t tok = r0 + 16 * unit;
#pragma unroll
    for (int m = 0; m < 3; ++m) {
        uint8_t* qt = m == 0 ? a.qdgt : m == 1 ? a.qdut : a.qht;
        const int64_t ldqt = m == 2 ? a.ldqht : a.ldqt;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int ch = 64 * j + (t >> 3);
            const uint4 val = *reinterpret_cast<const uint4*>(s_tile[m] + tile_place(ch, unit));
            uint8_t* dst = qt + (c0 + ch) * ldqt + tok;
            if (full || (c0 + ch < a.cols && tok + 16 <= a.rows)) {
                store16_nt(dst, val);
            } else if (c0 + ch < a.cols) {
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

dim3 row_grid(int64_t rows, int64_t cols, int rows_per_group) {
    const int64_t groups = (rows + rows_per_group - 1) / rows_per_group;
    return dim3((unsigned)((cols + 511) / 512), (unsigned)std::min<int64_t>(groups, 65535),
                (unsigned)((groups + 65534) / 65535));
}

template <typename T, bool POW2>
void launch_forward(const SwigluArgs& a, hipStream_t st) {
    constexpr int W = 4, R = 2;  // 8 x 2 and 4 x 4 run alike, one row per wave 10 % slower
    const dim3 grid = row_grid(a.rows, a.cols, W * R);
    if (a.qg)
        hipLaunchKernelGGL((swiglu_quantize_kernel<T, W, R, POW2, true>), grid, dim3(64 * W), 0, st, a);
    else
        hipLaunchKernelGGL((swiglu_quantize_kernel<T, W, R, POW2, false>), grid, dim3(64 * W), 0, st, a);
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
    const dim3 grid = row_grid(a.rows, a.cols, 4);
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
