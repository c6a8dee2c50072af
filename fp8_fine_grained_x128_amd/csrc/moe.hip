// moe.hip -- a whole mixture-of-experts layer for the few tokens of a decode
// step (up to 64), on FP8 weights with 128x128 block scales.
//
//   S_t  = the top_k largest router logits of token t (ties: lower expert
//          first; -inf is never chosen), p_te = their softmax
//   h_te = p_te * silu(Wg_e x_t) * (Wu_e x_t)
//   y_t  = sum_{e in S_t} Wd_e h_te
//
// The pages keep gating in higher precision and run the experts' GEMMs in FP8
// with 128x128 weight blocks (page 1, why-be.why-be.co.kr wr_id=65900,
// passage on the operators that stay in BF16/FP32; page 4, sunipension.com
// wr_id=314414, passage on Figure 7(a)).  At these token counts the layer is
// bound by reading the chosen experts' weights once.
//
// Numerics: codes are converted to bf16 (exact) and multiplied by bf16
// activations on the matrix cores, products exact and sums fp32; each
// 128-wide chunk's sum is multiplied by its block scale into an fp32 total.
// h is held as two bf16 numbers hi + lo (16 significant bits), so the second
// product sees it with a relative error below 2^-16.
//
// MFMA 16x16x32 (bf16): A: lane l holds row l%16, 8 values of the K step;
// B: column l%16, the same 8; D: lane l, element r is row 4*(l/16) + r,
// column l%16.  A holds weight rows, B tokens.
#include <algorithm>

#include "launch.hpp"
#include "tile_io.hpp"

namespace fp8q {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int kMaxTokens = 64;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;

// Where the pieces of the workspace lie (bytes from its start).
struct MoeLayout {
    int slots;          // active experts at most
    int64_t pairs;      // (token, expert) pairs at most
    int64_t experts, base, mask, token, prob, hi, lo, parts, total;
    int splits;         // partial sums of the down projection (1: none)
};

// Routing's result in the workspace.
struct MoePlan {
    int active;         // number of active experts
    int pad;
    uint64_t nan_mask;  // tokens whose logits hold NaN or +inf: their rows are NaN
};

__device__ __forceinline__ v8bf bf16_of_codes(uint32_t w0, uint32_t w1) {
    v8bf r;
    const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
    const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
    const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
    const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
    r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1];
    r[4] = c[0]; r[5] = c[1]; r[6] = d[0]; r[7] = d[1];
    return r;
}

__device__ __forceinline__ v4f mfma(v8bf a, v8bf b, v4f c) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
#else
    return c;
#endif
}

__device__ __forceinline__ int rank_below(uint64_t mask, int t) { return __popcll(mask & ((1ull << t) - 1)); }

}  // namespace

// ----------------------------------------------------------------------------
// Routing: one work-group, a wave per token at a time.  Logits become
// order-preserving keys (-0 counts as 0); the k-th largest key is found bit
// by bit with wave ballots, then ties at that key go to the lowest indices.
// ----------------------------------------------------------------------------
constexpr int kRouteWaves = 16;

__global__ __launch_bounds__(64 * kRouteWaves) void moe_route_kernel(MoeArgs a, MoeLayout L) {
    __shared__ uint64_t s_mask[kMaxExperts];
    __shared__ uint64_t s_nan;
    __shared__ int s_base[kMaxExperts];
    __shared__ int s_id[kMaxTokens][kMaxTopK];
    __shared__ float s_p[kMaxTokens][kMaxTopK];
    __shared__ int s_n[kMaxTokens];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) s_mask[e] = 0;
    if (threadIdx.x == 0) s_nan = 0;
    __syncthreads();
    const int per_lane = (a.experts + 63) / 64;
    for (int t = wave; t < a.tokens; t += kRouteWaves) {
        const float* row = a.logits + (int64_t)t * a.ldl;
        constexpr uint32_t kNone = 0x007fffffu;  // key of -inf; keys up to it are no candidates
        uint32_t key[kMaxExperts / 64];
        float top = -__builtin_inff();
        bool bad = false;
#pragma unroll
        for (int j = 0; j < kMaxExperts / 64; ++j) {
            key[j] = 0;
            if (j < per_lane && lane + 64 * j < a.experts) {
                const float l = row[lane + 64 * j] + 0.0f;
                const uint32_t b = __float_as_uint(l);
                key[j] = b & 0x80000000u ? ~b : b | 0x80000000u;
                bad = bad || !(l < __builtin_inff());
                top = fmaxf(top, l);
            }
        }
        if (__any((int)bad)) {
            if (lane == 0) {
                atomicOr((unsigned long long*)&s_nan, 1ull << t);
                s_n[t] = 0;
            }
            continue;
        }
#pragma unroll
        for (int off = 32; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
        uint32_t kth = 0;
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t cand = kth | (1u << bit);
            int n = 0;
#pragma unroll
            for (int j = 0; j < kMaxExperts / 64; ++j)
                if (j < per_lane) n += __popcll(__ballot(key[j] >= cand));
            if (n >= a.top_k) kth = cand;
        }
        kth = max(kth, kNone);  // fewer candidates than top_k: all of them
        int above = 0;
        float total = 0.0f;
#pragma unroll
        for (int j = 0; j < kMaxExperts / 64; ++j)
            if (j < per_lane) above += __popcll(__ballot(key[j] > kth));
        int ties = kth > kNone ? a.top_k - above : 0, n = 0;
        const uint64_t below = (1ull << lane) - 1;
#pragma unroll
        for (int j = 0; j < kMaxExperts / 64; ++j) {
            if (j < per_lane) {
                const uint64_t tie = __ballot(key[j] == kth);
                const bool in = key[j] > kth || (key[j] == kth && __popcll(tie & below) < ties);
                const uint64_t chosen = __ballot(in);
                ties -= min(ties, (int)__popcll(tie));
                const int e = lane + 64 * j;
                const float p = key[j] > kNone ? expf(row[e < a.experts ? e : 0] - top) : 0.0f;
                if (in) {
                    const int at = n + __popcll(chosen & below);
                    s_id[t][at] = e;
                    s_p[t][at] = p;
                    atomicOr((unsigned long long*)&s_mask[e], 1ull << t);
                }
                n += __popcll(chosen);
                total += a.renormalize ? (in ? p : 0.0f) : p;
            }
        }
        total = wave_sum(total);
        wave_lds_sync();
        if (lane < n) s_p[t][lane] /= total;
        if (lane == 0) s_n[t] = n;
    }
    __syncthreads();
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    if (wave == 0) {  // active experts in ascending order, with their first pair
        int active = 0, pairs = 0;
        for (int j = 0; j < per_lane; ++j) {
            const int e = lane + 64 * j;
            const uint64_t m = e < a.experts ? s_mask[e] : 0;
            const uint64_t live = __ballot(m != 0);
            const int cnt = __popcll(m);
            int before = cnt;  // inclusive prefix sum over the lanes
            for (int off = 1; off < 64; off <<= 1) {
                const int o = __shfl_up(before, off);
                if (lane >= off) before += o;
            }
            if (m) {
                const int idx = active + rank_below(live, lane);
                const int first = pairs + before - cnt;
                s_base[e] = first;
                reinterpret_cast<int*>(ws + L.experts)[idx] = e;
                reinterpret_cast<int*>(ws + L.base)[idx] = first;
                reinterpret_cast<uint64_t*>(ws + L.mask)[idx] = m;
            }
            active += __popcll(live);
            pairs += __shfl(before, 63);
        }
        if (lane == 0) {
            MoePlan* plan = reinterpret_cast<MoePlan*>(ws);
            plan->active = active;
            plan->nan_mask = s_nan;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.tokens * kMaxTopK; i += blockDim.x) {
        const int t = i / kMaxTopK, at = i % kMaxTopK;
        if (at >= s_n[t]) continue;
        const int e = s_id[t][at];
        const int pair = s_base[e] + rank_below(s_mask[e], t);
        reinterpret_cast<int*>(ws + L.token)[pair] = t;
        reinterpret_cast<float*>(ws + L.prob)[pair] = s_p[t][at];
    }
}

// ----------------------------------------------------------------------------
// Gate and up projections with the SwiGLU: 16 gate rows and the 16 up rows
// beside them, one active expert, 16 of its tokens at a time.  The four waves
// take every fourth 128-wide chunk of the hidden size and join their sums in
// LDS.
// ----------------------------------------------------------------------------
__global__ __launch_bounds__(256) void moe_up_kernel(MoeArgs a, MoeLayout L) {
    __shared__ float s_acc[2][4][256];
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    const int idx = blockIdx.y;
    if (idx >= reinterpret_cast<const MoePlan*>(ws)->active) return;
    const int e = reinterpret_cast<const int*>(ws + L.experts)[idx];
    const int base = reinterpret_cast<const int*>(ws + L.base)[idx];
    const int count = __popcll(reinterpret_cast<const uint64_t*>(ws + L.mask)[idx]);
    const int* token = reinterpret_cast<const int*>(ws + L.token) + base;
    const float* prob = reinterpret_cast<const float*>(ws + L.prob) + base;
    uint16_t* hi = reinterpret_cast<uint16_t*>(ws + L.hi);
    uint16_t* lo = reinterpret_cast<uint16_t*>(ws + L.lo);

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, kq = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.x * 16;
    const uint8_t* wg = a.w_gu + e * a.w_gu_stride + (row0 + r) * a.ldw_gu + 16 * kq;
    const uint8_t* wu = wg + a.inner * a.ldw_gu;
    const float* sg = a.s_gu + e * a.s_gu_stride + (row0 >> 7) * a.lds_gu;
    const float* su = sg + (a.inner >> 7) * a.lds_gu;
    const int chunks = (int)(a.hidden >> 7);

    for (int t0 = 0; t0 < count; t0 += 16) {
        const bool live = t0 + r < count;
        const uint16_t* x = a.x + (live ? token[t0 + r] : 0) * a.ldx + 16 * kq;
        v4f ag = {0.f, 0.f, 0.f, 0.f}, au = {0.f, 0.f, 0.f, 0.f};
        for (int kb = wave; kb < chunks; kb += 4) {
            v4f pg = {0.f, 0.f, 0.f, 0.f}, pu = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int64_t k = 128 * (int64_t)kb + 64 * j;
                const uint4 g = *reinterpret_cast<const uint4*>(wg + k);
                const uint4 u = *reinterpret_cast<const uint4*>(wu + k);
                uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
                if (live) {
                    x0 = *reinterpret_cast<const uint4*>(x + k);
                    x1 = *reinterpret_cast<const uint4*>(x + k + 8);
                }
                pg = mfma(bf16_of_codes(g.x, g.y), __builtin_bit_cast(v8bf, x0), pg);
                pg = mfma(bf16_of_codes(g.z, g.w), __builtin_bit_cast(v8bf, x1), pg);
                pu = mfma(bf16_of_codes(u.x, u.y), __builtin_bit_cast(v8bf, x0), pu);
                pu = mfma(bf16_of_codes(u.z, u.w), __builtin_bit_cast(v8bf, x1), pu);
            }
            ag += pg * sg[kb];
            au += pu * su[kb];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s_acc[0][wave][r * 16 + 4 * kq + i] = ag[i];
            s_acc[1][wave][r * 16 + 4 * kq + i] = au[i];
        }
        __syncthreads();
        const int tok = threadIdx.x >> 4, wr = threadIdx.x & 15;  // token and weight row of this thread
        if (t0 + tok < count) {
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                g += s_acc[0][w][threadIdx.x];
                u += s_acc[1][w][threadIdx.x];
            }
            const float h = g / (1.0f + expf(-g)) * u * prob[t0 + tok];
            const uint16_t h0 = (uint16_t)pack_bf16(h, 0.0f);
            const int64_t at = (int64_t)(base + t0 + tok) * a.inner + row0 + wr;
            hi[at] = h0;
            lo[at] = (uint16_t)pack_bf16(h - bf16_bits_to_f32(h0), 0.0f);
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------------------------
// Down projection: 16 rows of the hidden size, the active experts split,
// split+S, ... of S splits, all tokens as matrix columns (a token that did
// not choose the expert multiplies zeros).  The waves share the (expert,
// chunk) pairs and join their sums in LDS.
// ----------------------------------------------------------------------------
template <int NT>
__global__ __launch_bounds__(256) void moe_down_kernel(MoeArgs a, MoeLayout L) {
    __shared__ float s_acc[4][NT][256];
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    const MoePlan* plan = reinterpret_cast<const MoePlan*>(ws);
    const int active = plan->active;
    const uint16_t* hi = reinterpret_cast<const uint16_t*>(ws + L.hi);
    const uint16_t* lo = reinterpret_cast<const uint16_t*>(ws + L.lo);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, kq = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.x * 16;
    const int chunks = (int)(a.inner >> 7);

    v4f acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = v4f{0.f, 0.f, 0.f, 0.f};
    int item = wave;  // over (expert of this split, chunk)
    for (int idx = blockIdx.y; idx < active; idx += L.splits) {
        const int e = reinterpret_cast<const int*>(ws + L.experts)[idx];
        const int base = reinterpret_cast<const int*>(ws + L.base)[idx];
        const uint64_t mask = reinterpret_cast<const uint64_t*>(ws + L.mask)[idx];
        const uint8_t* w = a.w_down + e * a.w_down_stride + (row0 + r) * a.ldw_down + 16 * kq;
        const float* s = a.s_down + e * a.s_down_stride + (row0 >> 7) * a.lds_down;
        for (; item < chunks; item += 4) {
            v8bf f[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint4 c = *reinterpret_cast<const uint4*>(w + 128 * (int64_t)item + 64 * j);
                f[2 * j] = bf16_of_codes(c.x, c.y);
                f[2 * j + 1] = bf16_of_codes(c.z, c.w);
            }
            const float scale = s[item];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (((mask >> (16 * n)) & 0xffff) == 0) continue;
                const int t = 16 * n + r;
                const bool live = (mask >> t) & 1;
                const int64_t at = (int64_t)(base + (live ? rank_below(mask, t) : 0)) * a.inner + 128 * item + 16 * kq;
                v4f p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint4 h = make_uint4(0, 0, 0, 0), l = h;
                    if (live) {
                        h = *reinterpret_cast<const uint4*>(hi + at + 64 * (j >> 1) + 8 * (j & 1));
                        l = *reinterpret_cast<const uint4*>(lo + at + 64 * (j >> 1) + 8 * (j & 1));
                    }
                    p = mfma(f[j], __builtin_bit_cast(v8bf, l), p);
                    p = mfma(f[j], __builtin_bit_cast(v8bf, h), p);
                }
                acc[n] += p * scale;
            }
        }
        item -= chunks;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s_acc[wave][n][r * 16 + 4 * kq + i] = acc[n][i];
    __syncthreads();
    const int wr = threadIdx.x & 15;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t = 16 * n + (threadIdx.x >> 4);
        if (t >= a.tokens) continue;
        float v = (s_acc[0][n][threadIdx.x] + s_acc[1][n][threadIdx.x]) +
                  (s_acc[2][n][threadIdx.x] + s_acc[3][n][threadIdx.x]);
        if (L.splits > 1) {
            float* parts = reinterpret_cast<float*>(ws + L.parts);
            parts[((int64_t)blockIdx.y * a.tokens + t) * a.hidden + row0 + wr] = v;
            continue;
        }
        if ((plan->nan_mask >> t) & 1) v = __builtin_nanf("");
        if (a.y_dtype == kDtypeBF16)
            static_cast<uint16_t*>(a.y)[t * a.ldy + row0 + wr] = (uint16_t)pack_bf16(v, 0.0f);
        else
            static_cast<float*>(a.y)[t * a.ldy + row0 + wr] = v;
    }
}

// Sum of the splits' partial results, in order.
__global__ __launch_bounds__(256) void moe_join_kernel(MoeArgs a, MoeLayout L) {
    const uint8_t* ws = static_cast<const uint8_t*>(a.workspace);
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int t = blockIdx.y;
    if (c >= a.hidden) return;
    const float* parts = reinterpret_cast<const float*>(ws + L.parts) + (int64_t)t * a.hidden + c;
    float v = 0.0f;
    for (int s = 0; s < L.splits; ++s) v += parts[(int64_t)s * a.tokens * a.hidden];
    if ((reinterpret_cast<const MoePlan*>(ws)->nan_mask >> t) & 1) v = __builtin_nanf("");
    if (a.y_dtype == kDtypeBF16)
        static_cast<uint16_t*>(a.y)[t * a.ldy + c] = (uint16_t)pack_bf16(v, 0.0f);
    else
        static_cast<float*>(a.y)[t * a.ldy + c] = v;
}

// ----------------------------------------------------------------------------
// Workspace and launcher (arguments already validated by the API layer).
// ----------------------------------------------------------------------------
namespace {

// Splits of the down projection: as many as bring its work-groups (16 rows of
// the hidden size each) to about 1024, four for each of 256 compute units, as
// long as every split has an expert.
int down_splits(int64_t hidden, int slots) {
    const int64_t want = (1024 * 16 + hidden - 1) / hidden;
    return (int)std::max<int64_t>(1, std::min<int64_t>(want, slots));
}

MoeLayout moe_layout(int64_t tokens, int64_t hidden, int64_t inner, int experts, int top_k) {
    MoeLayout L;
    const int64_t k = std::min(top_k, experts);
    L.pairs = tokens * k;
    L.slots = (int)std::min<int64_t>(experts, L.pairs);
    L.splits = down_splits(hidden, L.slots);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    take(sizeof(MoePlan));
    L.experts = take(4 * (int64_t)L.slots);
    L.base = take(4 * (int64_t)L.slots);
    L.mask = take(8 * (int64_t)L.slots);
    L.token = take(4 * L.pairs);
    L.prob = take(4 * L.pairs);
    L.hi = take(2 * L.pairs * inner);
    L.lo = take(2 * L.pairs * inner);
    L.parts = take(L.splits > 1 ? 4 * L.splits * tokens * hidden : 0);
    L.total = at;
    return L;
}

}  // namespace

int64_t moe_decode_bytes(int64_t tokens, int64_t hidden, int64_t inner, int experts, int top_k) {
    return moe_layout(tokens, hidden, inner, experts, top_k).total;
}

hipError_t launch_moe_decode(const MoeArgs& a, hipStream_t st) {
    const MoeLayout L = moe_layout(a.tokens, a.hidden, a.inner, a.experts, a.top_k);
    hipLaunchKernelGGL(moe_route_kernel, dim3(1), dim3(64 * kRouteWaves), 0, st, a, L);
    hipLaunchKernelGGL(moe_up_kernel, dim3((unsigned)(a.inner / 16), (unsigned)L.slots), dim3(256), 0, st, a, L);
    const dim3 down((unsigned)(a.hidden / 16), (unsigned)L.splits);
    if (a.tokens <= 16)
        hipLaunchKernelGGL(moe_down_kernel<1>, down, dim3(256), 0, st, a, L);
    else if (a.tokens <= 32)
        hipLaunchKernelGGL(moe_down_kernel<2>, down, dim3(256), 0, st, a, L);
    else
        hipLaunchKernelGGL(moe_down_kernel<4>, down, dim3(256), 0, st, a, L);
    if (L.splits > 1)
        hipLaunchKernelGGL(moe_join_kernel, dim3((unsigned)((a.hidden + 255) / 256), (unsigned)a.tokens), dim3(256), 0,
                           st, a, L);
    return hipGetLastError();
}

}  // namespace fp8q
