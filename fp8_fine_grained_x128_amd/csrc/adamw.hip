// adamw.hip -- one AdamW step over many tensors, with the FP8 codes of the new
// weights.  For every element, in fp32, every product and sum of 8-bit moments
// rounded (so that their codes can be reproduced bit for bit), the sums of fp32
// moments fused:
//   m' = beta1 m + (1 - beta1) g,  v' = beta2 v + (1 - beta2) g^2,
//   p' = p (1 - lr decay) - lr / (1 - beta1^t) * m' / (sqrt(v' / (1 - beta2^t)) + eps)
// Moments of 32 bits are m and v.  Moments of 8 bits are E4M3 codes of m and of
// sqrt(v), one fp32 scale of amax for 128 consecutive elements (16 lanes of 8
// elements, so a tile's maximum takes four row rotations):
//   - sqrt(v), not v: both moments then span the gradient's range, which E4M3's
//     18 binades hold; those of v would be twice as many;
//   - rounded to the neighbour above with a probability of the way to it: a
//     moving average changes by less than half a step of a 4-bit significand
//     almost always, and rounded to nearest it would never move;
//     (What it does not bias is sqrt(v).  v, the square, gets the rounding's
//     variance: 2.4 % in the mean at beta2 = 0.95, 5.5 % at 0.999, where a
//     step's change is a small part of the grid's step and so is its variance.)
//   - sqrt(v) of a positive v rounds to one step of the smallest codes at least:
//     with a zero there the next step would divide m by eps alone.
// The step itself takes the moments before they are rounded.
//
// Both kernels are bound by memory: every byte moves once (per element fp32 28,
// with 8-bit moments and bf16 gradients 14; the codes add one byte each).  16
// experts of 2048x7168 with 8-bit moments and both codes, 4.26 GB: 854 us, 5.0
// TB/s, where a large copy reaches 4.7; 29 million weights with fp32 moments
// and both codes, 881 MB: 193 us, 4.6 TB/s.  With 8-bit moments the rounding's
// instructions come close to the time of the bytes: the shorter forms that a
// wave's values allow, below, took 932 us to 901.
#include <cmath>

#include "../../include/fp8q.h"
#include "launch.hpp"
#include "tile_io.hpp"

namespace fp8q {

namespace {

// Two rounds of xor-shift and multiplication: 32 bits that each depend on all
// of x's.  Shifts and factors are those of a published 32-bit integer hash,
// searched for there so that every input bit flips every output bit half the
// time.  The same function on the host (keys) and on the device.
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
    x ^= x >> 16;
    x *= 0x7feb352du;
    x ^= x >> 15;
    x *= 0x846ca68bu;
    return x ^ (x >> 16);
}

// b^t by squaring.  Every squaring doubles the relative error of b's power, so
// the result is within about t 2^-53.  What counts is 1 - b^t, whose relative
// error is t b^t / (1 - b^t) 2^-53, at most 2^-53 / (1 - b): 2^-26 up to b =
// 1 - 2^-27.
__host__ __device__ inline double power(double b, int64_t t) {
    double r = 1.0;
    for (; t > 0; t >>= 1) {
        if (t & 1) r *= b;
        b *= b;
    }
    return r;
}

struct Step {
    float beta1, rest1, beta2, rest2, eps;
    float keep;   // 1 - lr * decay
    float rate;   // lr / (1 - beta1^t)
    float root;   // 1 / sqrt(1 - beta2^t)
    float grad;   // factor of the gradient
    uint32_t time;  // low bits of t, for the random numbers
};

struct StepArgs {
    Step s;  // of the host's lr and t
    double beta1, beta2, lr, decay;
    const float* lr_dev;
    const int64_t* step_dev;
    const float* grad_scale;
    int64_t t;
};

__host__ __device__ inline void set_time(Step& s, double beta1, double beta2, double lr, double decay, int64_t t) {
    s.keep = (float)(1.0 - lr * decay);
    s.rate = (float)(lr / (1.0 - power(beta1, t)));
    s.root = (float)(1.0 / sqrt(1.0 - power(beta2, t)));
    s.time = (uint32_t)t;
}

__device__ __forceinline__ Step step_of(const StepArgs& a) {
    Step s = a.s;
    if (a.lr_dev || a.step_dev)
        set_time(s, a.beta1, a.beta2, a.lr_dev ? (double)*a.lr_dev : a.lr, a.decay, a.step_dev ? *a.step_dev : a.t);
    if (a.grad_scale) s.grad = *a.grad_scale;
    return s;
}

// y >= 0 (up to 448 and its rounding error) on the E4M3 grid, `unit` = 2^k the
// grid's step at y: unit * floor(fl32(y / unit + u)), at most 448, with u =
// (r + 1/2) / 2^16 of a 16-bit number r.
__device__ __forceinline__ float round_up_by(float y, uint32_t r) {
    const int k = max(__builtin_amdgcn_frexp_expf(y), -5) - 4;  // y in [2^(k+3), 2^(k+4)), or below 2^-6 with k = -9
    const float t = __builtin_amdgcn_ldexpf(y, -k) + __builtin_fmaf((float)r, 0x1p-16f, 0x1p-17f);
    return fminf(__builtin_amdgcn_ldexpf(__builtin_floorf(t), k), kE4M3Max);
}

// The same for y = 0 or y >= 2^-6, four instructions instead of eleven: there
// y / unit lies in [8, 16) with 20 bits behind the point, the last 20 of y's, so
// adding u to them carries into the four bits that stay.  (Where the sum
// reaches 16 it may be rounded up to 17 units of y; the grid's step is two there
// and the code is that of 16 either way.)
__device__ __forceinline__ float round_normal_up_by(float y, uint32_t r20) {
    return fminf(__uint_as_float((__float_as_uint(y) + r20) & 0xfff00000u), kE4M3Max);
}

// Square root rounded to nearest of v in [2^-90, 2^90]: the reciprocal root
// (within an ulp), one step of Goldschmidt's iteration for the root and half its
// reciprocal, and the root's remainder (all 2^24 significands of two binades,
// at both ends of the range too, give sqrtf's root).  11 issue slots; sqrtf,
// which takes any v, has 19.
__device__ __forceinline__ float sqrt_in_range(float v) {
    const float y = __builtin_amdgcn_rsqf(v);
    float s = v * y, h = 0.5f * y;
    const float e = __builtin_fmaf(-h, s, 0.5f);
    h = __builtin_fmaf(h, e, h);
    s = __builtin_fmaf(s, e, s);
    return __builtin_fmaf(__builtin_fmaf(-s, s, v), h, s);
}

// 1 / d rounded to nearest of d in [2^-45, 2^91]: the hardware's reciprocal
// (within an ulp) and one step.  (Every significand gives the IEEE quotient.)
__device__ __forceinline__ float reciprocal_in_range(float d) {
    const float y = __builtin_amdgcn_rcpf(d);
    return __builtin_fmaf(__builtin_fmaf(-d, y, 1.0f), y, y);
}

// A tensor as the kernels see it: 64 bytes, and 120 with codes.
struct FlatTensor {
    float* p;
    const void* g;
    void* m;
    void* v;
    float* sm;
    float* sv;
    int64_t n;
    uint32_t first;  // its first work unit
    uint32_t key;    // of its random numbers
};
struct CodedTensor : FlatTensor {
    uint8_t* q;
    float* s;
    uint8_t* qt;  // nullptr: no transposed codes
    float* st;
    int64_t N, K;  // n / (N K) matrices
    uint32_t units;
};

// Scale of a tile of moments: fl32(amax * fl32(1 / 448)), a product where
// make_scale divides: every lane forms two of them per eight elements.  That is
// one rounding more; the scale is the header's definition of what is held, and
// what it multiplies is rounded to four bits.  (The largest quotient may then
// be an ulp above 448, and is held at 448.)
__device__ __forceinline__ TileScale moment_scale(uint32_t amax_bits) {
    TileScale t;
    t.s = __uint_as_float(amax_bits) * (1.0f / kE4M3Max);
    t.fast = t.s >= kFastScaleMin;
    t.r = t.fast ? 1.0f / t.s : 0.0f;
    return t;
}

template <int BITS>
struct Moments;

template <>
struct Moments<32> {
    Raw8<float> m, v;
};
template <>
struct Moments<8> {
    uint2 m, v;
    float sm, sv;
};

// Eight elements of one tensor from element e on; `valid` of them exist.
template <typename GT, int BITS>
struct Eight {
    Raw8<float> p;
    Raw8<GT> g;
    Moments<BITS> mo;

    __device__ __forceinline__ void load(const FlatTensor& t, int64_t e, int64_t valid) {
        if (valid >= 8) {
            p.template load_full<false>(t.p + e);
            g.template load_full<sizeof(GT) == 2>(static_cast<const GT*>(t.g) + e);
            if constexpr (BITS == 32) {
                mo.m.template load_full<false>(static_cast<const float*>(t.m) + e);
                mo.v.template load_full<false>(static_cast<const float*>(t.v) + e);
            } else {
                mo.m = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + e);
                mo.v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + e);
                mo.sm = t.sm[e >> 7];
                mo.sv = t.sv[e >> 7];
            }
            return;
        }
        p.zero();
        g.zero();
        if constexpr (BITS == 32) {
            mo.m.zero();
            mo.v.zero();
        } else {
            mo.m = mo.v = make_uint2(0, 0);
            mo.sm = mo.sv = 0.0f;
        }
        if (valid <= 0) return;
        p.load_partial(t.p + e, valid);
        g.load_partial(static_cast<const GT*>(t.g) + e, valid);
        if constexpr (BITS == 32) {
            mo.m.load_partial(static_cast<const float*>(t.m) + e, valid);
            mo.v.load_partial(static_cast<const float*>(t.v) + e, valid);
        } else {
            const uint8_t* qm = static_cast<const uint8_t*>(t.m) + e;
            const uint8_t* qv = static_cast<const uint8_t*>(t.v) + e;
            uint32_t a[2] = {0, 0}, b[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < valid) {
                    a[i >> 2] |= (uint32_t)qm[i] << (8 * (i & 3));
                    b[i >> 2] |= (uint32_t)qv[i] << (8 * (i & 3));
                }
            mo.m = make_uint2(a[0], a[1]);
            mo.v = make_uint2(b[0], b[1]);
            mo.sm = t.sm[e >> 7];
            mo.sv = t.sv[e >> 7];
        }
    }

    // The step: writes p, m and v, leaves the new p in `out`.  The 16 lanes of
    // a DPP row hold one tile of 128 elements (those that do not exist are
    // zeros and stay zeros).
    __device__ __forceinline__ void step(const FlatTensor& t, const Step& s, uint32_t key, int64_t e, int64_t valid,
                                         float (&out)[8]) {
        float gr[8], m[8], v[8];
        p.values(out);
        g.values(gr);
        if constexpr (BITS == 32) {
            mo.m.values(m);
            mo.v.values(v);
        } else {
            decode4(mo.m.x, m);
            decode4(mo.m.y, m + 4);
            decode4(mo.v.x, v);
            decode4(mo.v.y, v + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m[i] *= mo.sm;
                v[i] *= mo.sv;
                v[i] *= v[i];
            }
        }
        float r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = gr[i] * s.grad;
            if constexpr (BITS == 32) {  // one rounding less than 8-bit moments are defined with
                m[i] = __builtin_fmaf(x, s.rest1, m[i] * s.beta1);
                v[i] = __builtin_fmaf(x * x, s.rest2, v[i] * s.beta2);
            } else {
                m[i] = m[i] * s.beta1 + x * s.rest1;
                v[i] = v[i] * s.beta2 + x * x * s.rest2;
            }
        }
        // Where every second moment of the wave is far from the ends of the
        // range root and quotient take fewer instructions.  They are those of
        // the other branch (the quotient's residual is exact from |m| = 2^-102
        // on), so that an element does not depend on its neighbours.  An IEEE
        // division in both: 13 tensors of 8.5 million elements with 8-bit
        // moments 26.6 us, so 25.9; the reciprocal alone, two ulp off, 25.6.
        float least = v[0], most = v[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) least = fminf(least, v[i]), most = fmaxf(most, v[i]);
        if (wave_all(least >= 0x1p-90f && most <= 0x1p90f) && s.eps <= 0x1p90f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                r[i] = sqrt_in_range(v[i]);
                const float d = r[i] * s.root + s.eps;
                out[i] = __builtin_fmaf(-s.rate, quotient_fast(m[i], d, reciprocal_in_range(d)), out[i] * s.keep);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                r[i] = sqrtf(v[i]);
                out[i] = __builtin_fmaf(-s.rate, m[i] / (r[i] * s.root + s.eps), out[i] * s.keep);
            }
        }
        store_values8(t.p, e, e + valid, out);
        if constexpr (BITS == 32) {
            store_values8(static_cast<float*>(t.m), e, e + valid, m);
            store_values8(static_cast<float*>(t.v), e, e + valid, v);
        } else {
            const uint32_t am = row_max_u32(amax8(m)), ar = row_max_u32(amax8(r));
            const TileScale tm = moment_scale(am), tv = moment_scale(ar);
            float cm[8], cv[8];
            if (wave_all(tm.fast && tv.fast)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    cm[i] = quotient_fast(__builtin_fabsf(m[i]), tm.s, tm.r);
                    cv[i] = quotient_fast(r[i], tv.s, tv.r);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    cm[i] = quotient(__builtin_fabsf(m[i]), tm);
                    cv[i] = quotient(r[i], tv);
                }
            }
            // any value with 0 < y < 2^-6?  (a zero becomes the largest number here)
            uint32_t low = 0xffffffffu;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                low = min(low, min(__float_as_uint(cm[i]) - 1u, __float_as_uint(cv[i]) - 1u));
            // (2^-6 in bits, less one; and no quotient of a positive root that is zero)
            const bool normal = wave_all(low >= 0x3c7fffffu && tv.s <= 0x1p60f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t h = mix32((uint32_t)(e + i) ^ key);
                if (normal) {
                    cm[i] = round_normal_up_by(cm[i], (h << 4 & 0xffff0u) | 8u);
                    cv[i] = round_normal_up_by(cv[i], (h >> 12 & 0xffff0u) | 8u);
                } else {
                    cm[i] = round_up_by(cm[i], h & 0xffffu);
                    cv[i] = round_up_by(cv[i], h >> 16);
                    cv[i] = r[i] > 0.0f ? fmaxf(cv[i], 0x1p-9f) : cv[i];
                }
                cm[i] = __builtin_copysignf(cm[i], m[i]);
            }
            uint32_t a = cvt2_in_range<false>(cm[0], cm[1], 0), b = cvt2_in_range<false>(cm[4], cm[5], 0);
            a = cvt2_in_range<true>(cm[2], cm[3], a);
            b = cvt2_in_range<true>(cm[6], cm[7], b);
            store8(static_cast<uint8_t*>(t.m), e, e + valid, a, b);
            a = cvt2_in_range<false>(cv[0], cv[1], 0), b = cvt2_in_range<false>(cv[4], cv[5], 0);
            a = cvt2_in_range<true>(cv[2], cv[3], a);
            b = cvt2_in_range<true>(cv[6], cv[7], b);
            store8(static_cast<uint8_t*>(t.v), e, e + valid, a, b);
            if (valid > 0 && (threadIdx.x & 15) == 0) {
                t.sm[e >> 7] = tm.s;
                t.sv[e >> 7] = tv.s;
            }
        }
    }
};

// The tensors travel as kernel arguments, of which a launch has 4 KB at most.
template <class Tensor, int COUNT>
struct Batch {
    Tensor t[COUNT];
    StepArgs step;
    int count;
    int pow2;
};
using FlatBatch = Batch<FlatTensor, 60>;
using CodedBatch = Batch<CodedTensor, 33>;
static_assert(sizeof(FlatBatch) <= 4096 && sizeof(CodedBatch) <= 4096, "kernel arguments");

// Work unit u of the launch belongs to the last tensor whose first unit is <= u.
template <class B>
__device__ __forceinline__ int tensor_of(const B& b, uint32_t u) {
    int lo = 0, hi = b.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (b.t[mid].first <= u) lo = mid;
        else hi = mid;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

constexpr int kFlatThreads = 256;
constexpr int kFlatUnit = 8 * kFlatThreads;

template <typename GT, int BITS>
__global__ __launch_bounds__(kFlatThreads) void adamw_flat_kernel(FlatBatch b) {
    const FlatTensor& t = b.t[tensor_of(b, blockIdx.x)];
    const Step s = step_of(b.step);
    const uint32_t key = mix32(t.key + s.time);
    const int64_t e = (int64_t)(blockIdx.x - t.first) * kFlatUnit + 8 * threadIdx.x;
    Eight<GT, BITS> x;
    x.load(t, e, t.n - e);
    float out[8];
    x.step(t, s, key, e, t.n - e, out);
}

// A 128x128 block of a weight: the step, then the block's codes from the new
// values in registers, and their transpose through LDS.
// Work-groups go to the eight XCDs in turn.  Where rows are wide (from 2048
// columns) each XCD takes a contiguous run of a tensor's blocks, so that the
// blocks it works on at a time lie in few bands of rows (16 experts 2048x7168
// with 8-bit moments 901 -> 854 us); in narrow tensors the blocks at a time
// are contiguous memory as they are (56 experts 2048x1024: 620 us, 664 so).
__device__ __forceinline__ uint32_t unit_of(uint32_t id, uint32_t units) {
    const uint32_t xcd = id & 7, per = units >> 3, more = units & 7;
    return xcd * per + (xcd < more ? xcd : more) + (id >> 3);
}

template <typename GT, int BITS>
__global__ __launch_bounds__(512, 4) void adamw_codes_kernel(CodedBatch b) {
    __shared__ uint32_t s_max[8];
    __shared__ __align__(16) uint8_t s_tile[128 * 128];  // [column][row], 16-byte units swizzled
    const CodedTensor& t = b.t[tensor_of(b, blockIdx.x)];
    const Step s = step_of(b.step);
    const uint32_t key = mix32(t.key + s.time);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t kb = (uint32_t)(t.K >> 7), nb = (uint32_t)((t.N + 127) >> 7);
    uint32_t u = blockIdx.x - t.first;
    if (t.K >= 2048) u = unit_of(u, t.units);
    const uint32_t bj = u % kb;
    u /= kb;
    const uint32_t bi = u % nb, mat = u / nb;
    const int64_t r0 = (int64_t)bi * 128, c0 = (int64_t)bj * 128;
    const int cg = tid & 15, rg = tid >> 4;
    const int64_t row = r0 + 4 * rg, col = c0 + 8 * cg;
    const int64_t e0 = ((int64_t)mat * t.N + row) * t.K + col;
    float w[4][8];
    constexpr int kAhead = 2;  // rows loaded before the first of them is worked on
    uint32_t am = 0;
#pragma unroll
    for (int k0 = 0; k0 < 4; k0 += kAhead) {
        Eight<GT, BITS> x[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) x[k].load(t, e0 + (k0 + k) * t.K, row + k0 + k < t.N ? 8 : 0);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const bool exists = row + k0 + k < t.N;
            x[k].step(t, s, key, e0 + (k0 + k) * t.K, exists ? 8 : 0, w[k0 + k]);
            // (rows past N step on zeros: 0 / 0 where eps is zero)
            am = max(am, exists ? amax8(w[k0 + k]) : 0u);
        }
    }
    am = row_max_u32(am);
    am = max(am, (uint32_t)__shfl_xor((int)am, 16));
    am = max(am, (uint32_t)__shfl_xor((int)am, 32));
    if (lane == 0) s_max[wave] = am;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) am = max(am, s_max[k]);
    const TileScale ts = b.pow2 ? make_scale_pow2(am) : make_scale(am);
    if (tid == 0) {
        t.s[((int64_t)mat * nb + bi) * kb + bj] = ts.s;
        if (t.st) t.st[((int64_t)mat * kb + bj) * nb + bi] = ts.s;
    }
    const bool fast = wave_all(ts.s >= kFastScaleMin);
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        lo[k] = fast ? encode4_fast(w[k][0], w[k][1], w[k][2], w[k][3], ts.s, ts.r)
                     : encode4(w[k][0], w[k][1], w[k][2], w[k][3], ts);
        hi[k] = fast ? encode4_fast(w[k][4], w[k][5], w[k][6], w[k][7], ts.s, ts.r)
                     : encode4(w[k][4], w[k][5], w[k][6], w[k][7], ts);
        if (row + k < t.N) *reinterpret_cast<uint2*>(t.q + e0 + k * t.K) = make_uint2(lo[k], hi[k]);
    }
    if (!t.qt) return;
    uint32_t tr[8];
    transpose4x4(lo, tr);
    transpose4x4(hi, tr + 4);
    const int tok = 4 * rg;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int ch = 8 * cg + k;
        *reinterpret_cast<uint32_t*>(s_tile + ch * 128 + 16 * ((tok >> 4) ^ (cg & 7)) + (tok & 15)) = tr[k];
    }
    __syncthreads();
    const int64_t ldqt = (t.N + 15) / 16 * 16;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int ch = 64 * j + (tid >> 3), unit = tid & 7;
        const uint4 val = *reinterpret_cast<const uint4*>(s_tile + ch * 128 + 16 * unit);
        const int64_t n = r0 + 16 * (unit ^ ((ch >> 3) & 7));
        uint8_t* dst = t.qt + ((int64_t)mat * t.K + c0 + ch) * ldqt + n;
        if (n + 16 <= t.N) {
            *reinterpret_cast<uint4*>(dst) = val;
        } else {
            const uint32_t wv[4] = {val.x, val.y, val.z, val.w};
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (n + k < t.N) dst[k] = (uint8_t)(wv[k >> 2] >> (8 * (k & 3)));
        }
    }
}

// Collects tensors into launches: a full batch, or one whose grid would grow
// past kMaxUnits work-groups, is sent off.
constexpr int64_t kMaxUnits = int64_t(1) << 22;

template <class B, class Launch>
struct Sender {
    B b;
    int64_t units = 0;
    Launch launch;
    Sender(const StepArgs& step, int pow2, Launch l) : launch(l) {
        b.step = step;
        b.count = 0;
        b.pow2 = pow2;
    }
    template <class Tensor>
    void add(Tensor t, int64_t n_units) {
        if (b.count == (int)(sizeof(b.t) / sizeof(b.t[0])) || units + n_units > kMaxUnits) send();
        t.first = (uint32_t)units;
        b.t[b.count++] = t;
        units += n_units;
    }
    void send() {
        if (b.count) launch(b, (unsigned)units);
        b.count = 0;
        units = 0;
    }
};

template <typename GT, int BITS>
void launch_typed(const fp8q_adamw_tensor* tensors, int count, const StepArgs& step, uint32_t seed, int pow2,
                  hipStream_t st) {
    auto flat_launch = [st](const FlatBatch& b, unsigned units) {
        hipLaunchKernelGGL((adamw_flat_kernel<GT, BITS>), dim3(units), dim3(kFlatThreads), 0, st, b);
    };
    auto coded_launch = [st](const CodedBatch& b, unsigned units) {
        hipLaunchKernelGGL((adamw_codes_kernel<GT, BITS>), dim3(units), dim3(512), 0, st, b);
    };
    Sender<FlatBatch, decltype(flat_launch)> flat(step, pow2, flat_launch);
    Sender<CodedBatch, decltype(coded_launch)> coded(step, pow2, coded_launch);
    for (int i = 0; i < count; ++i) {
        const fp8q_adamw_tensor& a = tensors[i];
        if (a.n == 0) continue;
        CodedTensor t{};
        t.p = a.p; t.g = a.g; t.m = a.m; t.v = a.v; t.sm = a.sm; t.sv = a.sv; t.n = a.n;
        t.key = mix32(seed + (uint32_t)i * 0x9e3779b9u);
        if (!a.q) {
            flat.add(static_cast<const FlatTensor&>(t), (a.n + kFlatUnit - 1) / kFlatUnit);
            continue;
        }
        t.q = a.q; t.s = a.s; t.qt = a.qt; t.st = a.st; t.N = a.N; t.K = a.K;
        t.units = (uint32_t)(a.n / (a.N * a.K) * ((a.N + 127) / 128) * (a.K / 128));
        coded.add(t, t.units);
    }
    coded.send();
    flat.send();
}

}  // namespace

hipError_t launch_adamw(const fp8q_adamw_tensor* tensors, int count, int g_dtype, int bits,
                        const fp8q_adamw_config& c, int pow2, hipStream_t st) {
    StepArgs a{};
    a.s.beta1 = (float)c.beta1;
    a.s.rest1 = (float)(1.0 - c.beta1);
    a.s.beta2 = (float)c.beta2;
    a.s.rest2 = (float)(1.0 - c.beta2);
    a.s.eps = c.eps > 0.0 ? fmaxf((float)c.eps, 0x1p-149f) : 0.0f;  // never from positive to zero: 0 / eps is 0
    a.s.grad = 1.0f;
    a.beta1 = c.beta1; a.beta2 = c.beta2; a.lr = c.lr; a.decay = c.weight_decay;
    a.lr_dev = c.lr_dev; a.step_dev = c.step_dev; a.grad_scale = c.grad_scale;
    a.t = c.step;
    set_time(a.s, a.beta1, a.beta2, a.lr, a.decay, a.t);
    if (g_dtype == kDtypeBF16) {
        if (bits == 8) launch_typed<uint16_t, 8>(tensors, count, a, c.seed, pow2, st);
        else launch_typed<uint16_t, 32>(tensors, count, a, c.seed, pow2, st);
    } else {
        if (bits == 8) launch_typed<float, 8>(tensors, count, a, c.seed, pow2, st);
        else launch_typed<float, 32>(tensors, count, a, c.seed, pow2, st);
    }
    return hipGetLastError();
}

}  // namespace fp8q
