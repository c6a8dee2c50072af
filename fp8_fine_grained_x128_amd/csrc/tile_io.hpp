// tile_io.hpp -- loading, encoding and storing of rows in groups of eight
// elements, shared by the kernels that read or write 1x128 and 128x1 tiles.
#pragma once

#include <utility>

#include "device_common.hpp"

namespace fp8q {

typedef unsigned short us2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 16-byte load, marked non-temporal when NT: a quantizer that reads each
// input byte once need not let its input displace cached data (such as the
// codes a GEMM is about to read); measured 3-6 % faster at the step's sizes.
// A gather reads repeated source rows and keeps the normal (cached) load.
template <bool NT>
__device__ __forceinline__ uint4 load16(const void* p) {
    if constexpr (NT) {
        const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
        return make_uint4(v[0], v[1], v[2], v[3]);
    } else {
        return *reinterpret_cast<const uint4*>(p);
    }
}

// 8-byte load and 16-byte store, marked non-temporal.
__device__ __forceinline__ uint2 load8_nt(const void* p) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
    return make_uint2(v[0], v[1]);
}

__device__ __forceinline__ void store16_nt(void* p, uint4 v) {
    const u32x4 w = {v.x, v.y, v.z, v.w};
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(p));
}

// Orders LDS traffic between the lanes of one wave: a wave's LDS operations
// execute in program order, the fences keep the compiler from reordering them.
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Work-group barrier that orders LDS traffic and leaves global loads and
// stores in flight.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

__device__ __forceinline__ bool wave_all(bool p) { return __all((int)p) != 0; }

// fl32(x/s) by the reciprocal path (valid when s >= kFastScaleMin).
__device__ __forceinline__ float quotient_fast(float x, float s, float r) {
    const float y = x * r;
    const float e = __builtin_fmaf(y, s, -x);
    return __builtin_fmaf(-e, r, y);
}

__device__ __forceinline__ uint32_t encode4_fast(float v0, float v1, float v2, float v3, float s, float r) {
    const uint32_t w = cvt2_in_range<false>(quotient_fast(v0, s, r), quotient_fast(v1, s, r), 0u);
    return cvt2_in_range<true>(quotient_fast(v2, s, r), quotient_fast(v3, s, r), w);
}

// General-path encoder of either scale rule.
template <bool POW2>
__device__ __forceinline__ uint32_t encode4_any(float v0, float v1, float v2, float v3, const TileScale& t) {
    if constexpr (POW2)
        return encode4_mul(v0, v1, v2, v3, t.r);
    else
        return encode4(v0, v1, v2, v3, t);
}

// Fast-path encoder of either scale rule (s, r of a tile whose quotient may
// take the reciprocal path).
template <bool POW2>
__device__ __forceinline__ uint32_t encode4_sr(float v0, float v1, float v2, float v3, float s, float r) {
    if constexpr (POW2)
        return encode4_mul(v0, v1, v2, v3, r);
    else
        return encode4_fast(v0, v1, v2, v3, s, r);
}

__device__ __forceinline__ TileScale scale_from(float s, float r) {
    TileScale t;
    t.s = s;
    t.r = r;
    t.fast = s >= kFastScaleMin;
    return t;
}

// Hides a register's value from the optimizer: values derived from it are
// recomputed after this point instead of being kept live across it.
template <typename V>
__device__ __forceinline__ void opaque(V& x) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+v"(x));
#endif
}

// Eight consecutive input elements of one row, kept in their storage form.
template <typename T>
struct Raw8;

template <>
struct Raw8<uint16_t> {  // bf16 bit patterns, two per dword
    uint4 d;
    __device__ void zero() { d = make_uint4(0, 0, 0, 0); }
    template <bool NT = true>
    __device__ void load_full(const uint16_t* p) { d = load16<NT>(p); }
    __device__ void load_partial(const uint16_t* p, int64_t n) {  // n < 8 valid elements
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
        d = make_uint4(w[0], w[1], w[2], w[3]);
    }
    // The first n < 8 elements, n the same for all lanes; the others stay.
    // Every load has registers of its own.
    __device__ void load_tail(const uint16_t* p, int n) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(p);
        switch (n) {
            case 1: d.x = p[0]; break;
            case 2: d.x = w[0]; break;
            case 3: d.x = w[0], d.y = p[2]; break;
            case 4: d.x = w[0], d.y = w[1]; break;
            case 5: d.x = w[0], d.y = w[1], d.z = p[4]; break;
            case 6: d.x = w[0], d.y = w[1], d.z = w[2]; break;
            case 7: d.x = w[0], d.y = w[1], d.z = w[2], d.w = p[6]; break;
        }
    }
    __device__ uint32_t amax_bits() const {  // fp32 bits of max |x|
        const us2 m0 = __builtin_bit_cast(us2, d.x & 0x7fff7fffu);
        const us2 m1 = __builtin_bit_cast(us2, d.y & 0x7fff7fffu);
        const us2 m2 = __builtin_bit_cast(us2, d.z & 0x7fff7fffu);
        const us2 m3 = __builtin_bit_cast(us2, d.w & 0x7fff7fffu);
        const us2 m = __builtin_elementwise_max(__builtin_elementwise_max(m0, m1),
                                                __builtin_elementwise_max(m2, m3));
        const uint32_t mm = m[0] > m[1] ? m[0] : m[1];
        return mm << 16;
    }
    __device__ void values(float v[8]) const {
        v[0] = bf16_lo(d.x); v[1] = bf16_hi(d.x);
        v[2] = bf16_lo(d.y); v[3] = bf16_hi(d.y);
        v[4] = bf16_lo(d.z); v[5] = bf16_hi(d.z);
        v[6] = bf16_lo(d.w); v[7] = bf16_hi(d.w);
    }
};

template <>
struct Raw8<float> {
    float4 a, b;
    __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    template <bool NT = true>
    __device__ void load_full(const float* p) {
        const uint4 u = load16<NT>(p), v = load16<NT>(p + 4);
        a = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
        b = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
    }
    __device__ void load_partial(const float* p, int64_t n) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
        a = make_float4(v[0], v[1], v[2], v[3]);
        b = make_float4(v[4], v[5], v[6], v[7]);
    }
    __device__ void load_tail(const float* p, int n) {
        if (n > 0) a.x = p[0];
        if (n > 1) a.y = p[1];
        if (n > 2) a.z = p[2];
        if (n > 3) a.w = p[3];
        if (n > 4) b.x = p[4];
        if (n > 5) b.y = p[5];
        if (n > 6) b.z = p[6];
    }
    __device__ uint32_t amax_bits() const {
        uint32_t m = max(max(abs_bits(a.x), abs_bits(a.y)), max(abs_bits(a.z), abs_bits(a.w)));
        return max(m, max(max(abs_bits(b.x), abs_bits(b.y)), max(abs_bits(b.z), abs_bits(b.w))));
    }
    __device__ void values(float v[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};

// Loads x[c .. c+8) of a row; elements at or beyond `valid` read as 0.
// `full` (wave-uniform) says that all 8 are valid.  NT marks the loads
// non-temporal: right for a lane's 8 bf16 values, one load whose neighbours
// complete the line; 8 fp32 values are two loads of half a line's bytes each,
// and where such a kernel waits for memory alone the caches serve the second
// (layer-norm backward 179 us against 189, SwiGLU backward 153 against 159,
// both 8192x7168 fp32; the forward kernels are as fast or slower with it).
template <typename T, bool NT = true>
__device__ __forceinline__ void load_row8(Raw8<T>& r, const T* row, int64_t c, int64_t valid, bool full) {
    if (full || c + 8 <= valid)
        r.template load_full<NT>(row + c);
    else if (c < valid)
        r.load_partial(row + c, valid - c);
    else
        r.zero();
}

__device__ __forceinline__ void opaque_raw(Raw8<uint16_t>& r) {
    opaque(r.d.x);
    opaque(r.d.y);
    opaque(r.d.z);
    opaque(r.d.w);
}
__device__ __forceinline__ void opaque_raw(Raw8<float>& r) {
    float* const v[8] = {&r.a.x, &r.a.y, &r.a.z, &r.a.w, &r.b.x, &r.b.y, &r.b.z, &r.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) opaque(*v[i]);
}

// load_row8 (c a multiple of 8, `valid` the same for all lanes, `row` null for
// no row) for loads that stay under way while others are worked on.  The zeros
// are written first and the compiler may not move them into the other branch:
// there a wave that crosses the row's end would wait for its loads before it
// can write them (norm backward in bf16: 8192x7104 93 us against 120, 8192x7001
// 121 against 138, 30000x331 27 against 36).
template <typename T, bool NT>
__device__ __forceinline__ void load_row8_ahead(Raw8<T>& r, const T* row, int64_t c, int64_t valid) {
    r.zero();
    opaque_raw(r);
    if (row != nullptr && c + 8 <= valid) r.template load_full<NT>(row + c);
    if (row != nullptr && c < valid && c + 8 > valid) r.load_tail(row + c, (int)(valid & 7));
}

// Stores 8 codes (two dwords) at q[c .. c+8), clipped to `valid`.
__device__ __forceinline__ void store8(uint8_t* q, int64_t c, int64_t valid, uint32_t w0, uint32_t w1) {
    if (c + 8 <= valid) {
        *reinterpret_cast<uint2*>(q + c) = make_uint2(w0, w1);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < valid) q[c + i] = (uint8_t)(((i < 4 ? w0 : w1) >> (8 * (i & 3))) & 0xffu);
    }
}

// Two fp32 values -> packed bf16, round to nearest even (one instruction).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    const f2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf2));
}

// Stores 8 values of a row at p[c .. c+8), clipped to `valid`; bf16 rows get
// the nearest-even rounding.  NT marks the store non-temporal (a lane's fp32
// values are two stores, each of half the bytes of every line: those go
// through the caches).
__device__ __forceinline__ void store_values8(float* p, int64_t c, int64_t valid, const float v[8]) {
    if (c + 8 <= valid) {
        *reinterpret_cast<float4*>(p + c) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < valid) p[c + i] = v[i];
    }
}

template <bool NT = false>
__device__ __forceinline__ void store_values8(uint16_t* p, int64_t c, int64_t valid, const float v[8]) {
    const uint32_t w[4] = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    if (c + 8 <= valid) {
        const uint4 v4 = make_uint4(w[0], w[1], w[2], w[3]);
        if constexpr (NT) store16_nt(p + c, v4);
        else *reinterpret_cast<uint4*>(p + c) = v4;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < valid) p[c + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
}

// v_perm_b32: byte i of the result is byte sel[i] of the 8-byte value hi:lo.
__device__ __forceinline__ uint32_t perm(uint32_t hi, uint32_t lo, uint32_t sel) {
    return __builtin_amdgcn_perm(hi, lo, sel);
}

// Transpose of a 4x4 byte matrix held as 4 dwords (dword r = row r, byte c =
// column c): out[c] = column c.
__device__ __forceinline__ void transpose4x4(const uint32_t a[4], uint32_t out[4]) {
    const uint32_t x0 = perm(a[1], a[0], 0x06020400u);  // a0.0 a1.0 a0.2 a1.2
    const uint32_t x1 = perm(a[1], a[0], 0x07030501u);  // a0.1 a1.1 a0.3 a1.3
    const uint32_t x2 = perm(a[3], a[2], 0x06020400u);
    const uint32_t x3 = perm(a[3], a[2], 0x07030501u);
    out[0] = perm(x2, x0, 0x05040100u);
    out[1] = perm(x3, x1, 0x05040100u);
    out[2] = perm(x2, x0, 0x07060302u);
    out[3] = perm(x3, x1, 0x07060302u);
}

// Lane n of each 16-lane DPP row to all 16 of them, for n = 0 .. N-1.
template <int... N>
__device__ __forceinline__ void row_broadcast(std::integer_sequence<int, N...>, float v, float (&out)[sizeof...(N)]) {
    ((out[N] = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x150 + N, 0xf, 0xf, false))), ...);
}

// Magnitude maxima: the absolute value is an operand modifier and three
// operands go into one maximum.  The bits of the result order like the number.
// A NaN operand gives NaN (IEEE 754-2019 maximum), whose bits are the largest:
// a tile that holds one has a NaN scale, as in the quantizers.
__device__ __forceinline__ float max_abs2(float a, float b) {
    return __builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b));
}
__device__ __forceinline__ float max_abs3(float m, float a, float b) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, __builtin_fabsf(a)), __builtin_fabsf(b));
}

__device__ __forceinline__ uint32_t amax8(const float v[8]) {
    float m = max_abs2(v[0], v[1]);
#pragma unroll
    for (int k = 2; k < 8; k += 2) m = max_abs3(m, v[k], v[k + 1]);
    return __float_as_uint(m);
}

// Sum over the 16 lanes of a DPP row, and over the 64 lanes of a wave; every
// lane receives the same bits (each step adds a pair of equal-length partial
// sums, so the order within a pair does not matter).
__device__ __forceinline__ float row_sum(float v) {
    v += __uint_as_float(row_ror<8>(__float_as_uint(v)));
    v += __uint_as_float(row_ror<4>(__float_as_uint(v)));
    v += __uint_as_float(row_ror<2>(__float_as_uint(v)));
    v += __uint_as_float(row_ror<1>(__float_as_uint(v)));
    return v;
}

__device__ __forceinline__ double row_sum(double v) {
    for (int off = 8; off; off >>= 1) v += __shfl_xor(v, off);
    return v;
}

template <typename S>
__device__ __forceinline__ S wave_sum(S v) {
    v = row_sum(v);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

}  // namespace fp8q
