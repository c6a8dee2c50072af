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
    int slots;      // active experts at most
    int64_t pairs;  // (token, expert) pairs at most
    int64_t experts, base, mask, prob, pair, hi, lo, parts, total;
};

// Routing's result in the workspace.  Pairs are numbered expert by expert
// (ascending), a pair's place among its expert's is its token's rank in the
// expert's mask.
struct MoePlan {
    int active;         // number of active experts
    int pad;
    uint64_t nan_mask;  // tokens whose logits hold NaN or +inf: their rows are NaN
    int count[kMaxTokens];
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

template <int PL>  // experts per lane
__global__ __launch_bounds__(64 * kRouteWaves) void moe_route_kernel(MoeArgs a, MoeLayout L) {
    __shared__ uint64_t s_mask[64 * PL];
    __shared__ uint64_t s_nan;
    __shared__ int s_base[64 * PL];
    __shared__ int s_id[kMaxTokens][kMaxTopK];
    __shared__ float s_p[kMaxTokens][kMaxTopK];
    __shared__ int s_n[kMaxTokens];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int e = threadIdx.x; e < 64 * PL; e += blockDim.x) s_mask[e] = 0;
    if (threadIdx.x == 0) s_nan = 0;
    __syncthreads();
    constexpr uint32_t kNone = 0x007fffffu;  // key of -inf; keys up to it are no candidates
    const uint64_t below = (1ull << lane) - 1;
    for (int t = wave; t < a.tokens; t += blockDim.x / 64) {
        const float* row = a.logits + (int64_t)t * a.ldl;
        float l[PL];
        uint32_t key[PL];
        float top = -__builtin_inff();
        bool bad = false;
#pragma unroll
        for (int j = 0; j < PL; ++j) {
            const int e = lane + 64 * j;
            l[j] = e < a.experts ? row[e] + 0.0f : -__builtin_inff();
        }
#pragma unroll
        for (int j = 0; j < PL; ++j) {
            const uint32_t b = __float_as_uint(l[j]);
            key[j] = b & 0x80000000u ? ~b : b | 0x80000000u;
            bad = bad || !(l[j] < __builtin_inff());
            top = fmaxf(top, l[j]);
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
#pragma unroll
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t cand = kth | (1u << bit);
            int n = 0;
#pragma unroll
            for (int j = 0; j < PL; ++j) n += __popcll(__ballot(key[j] >= cand));
            if (n >= a.top_k) kth = cand;
        }
        kth = max(kth, kNone);  // fewer candidates than top_k: all of them
        int above = 0;
#pragma unroll
        for (int j = 0; j < PL; ++j) above += __popcll(__ballot(key[j] > kth));
        int ties = kth > kNone ? a.top_k - above : 0, n = 0;
        float p[PL], total = 0.0f;
        int at[PL];  // place among the token's choices, or -1
#pragma unroll
        for (int j = 0; j < PL; ++j) {
            const uint64_t tie = __ballot(key[j] == kth);
            const bool in = key[j] > kth || (key[j] == kth && __popcll(tie & below) < ties);
            const uint64_t in_mask = __ballot(in);
            ties -= min(ties, (int)__popcll(tie));
            p[j] = key[j] > kNone ? expf(l[j] - top) : 0.0f;
            at[j] = in ? n + (int)__popcll(in_mask & below) : -1;
            n += __popcll(in_mask);
            total += in || !a.renormalize ? p[j] : 0.0f;
        }
        total = wave_sum(total);
#pragma unroll
        for (int j = 0; j < PL; ++j) {
            if (at[j] < 0) continue;
            s_id[t][at[j]] = lane + 64 * j;
            s_p[t][at[j]] = p[j] / total;
            atomicOr((unsigned long long*)&s_mask[lane + 64 * j], 1ull << t);
        }
        if (lane == 0) s_n[t] = n;
    }
    __syncthreads();
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    if (wave == 0) {  // active experts in ascending order, with their first pair
        int active = 0, pairs = 0;
#pragma unroll
        for (int j = 0; j < PL; ++j) {
            const int e = lane + 64 * j;
            const uint64_t m = s_mask[e];
            const uint64_t live = __ballot(m != 0);
            const int cnt = __popcll(m);
            int before = cnt;  // inclusive prefix sum over the lanes
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const int o = __shfl_up(before, off);
                if (lane >= off) before += o;
            }
            if (m) {
                const int idx = active + (int)__popcll(live & below);
                const int first = pairs + before - cnt;
                s_base[e] = first;
                reinterpret_cast<int*>(ws + L.experts)[idx] = e;
                reinterpret_cast<int*>(ws + L.base)[idx] = first;
                reinterpret_cast<uint64_t*>(ws + L.mask)[idx] = m;
            }
            active += __popcll(live);
            pairs += __shfl(before, 63);
        }
        MoePlan* plan = reinterpret_cast<MoePlan*>(ws);
        if (lane == 0) {
            plan->active = active;
            plan->nan_mask = s_nan;
        }
        if (lane < a.tokens) plan->count[lane] = s_n[lane];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.tokens * kMaxTopK; i += blockDim.x) {
        const int t = i / kMaxTopK, at = i % kMaxTopK;
        if (at >= s_n[t]) continue;
        const int e = s_id[t][at];
        const int pair = s_base[e] + rank_below(s_mask[e], t);
        reinterpret_cast<float*>(ws + L.prob)[pair] = s_p[t][at];
        reinterpret_cast<int*>(ws + L.pair)[i] = pair;
    }
}

// ----------------------------------------------------------------------------
// Both projections: a work-group of four waves takes 64 weight rows (four row
// tiles) of one active expert and 16 of its tokens at a time.  The waves take
// every fourth 128-wide chunk of the contraction and join their sums in LDS;
// a wave loads its next chunk while it multiplies the current one.  Weights
// go straight from memory to the matrix operand (16 rows of 64 contiguous
// bytes a load: the same rate as whole lines), each one read once; 64 rows
// share one read of the tokens, so those cost at most (tokens x 2 or 4)/64 of
// the weights' bytes, from the caches.
// A lane whose column has no token repeats the first one's reads; its results
// are dropped.
// ----------------------------------------------------------------------------
constexpr int kTiles = 4;  // row tiles of 16 in a work-group

// NB: activation arrays whose sum is multiplied (x, or hi and lo).
template <int NB>
struct Chunk {
    uint4 w[kTiles][2];
    uint4 b[NB][4];
};

template <int NB>
__device__ __forceinline__ void load_chunk(Chunk<NB>& c, const uint8_t* const (&w)[kTiles],
                                           const uint16_t* const (&b)[NB], int kb) {
    const int64_t k = 128 * (int64_t)kb;
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) c.w[t][j] = *reinterpret_cast<const uint4*>(w[t] + k + 64 * j);
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c.b[n][j] = *reinterpret_cast<const uint4*>(b[n] + k + 64 * (j >> 1) + 8 * (j & 1));
}

template <int NB>
__device__ __forceinline__ void multiply_chunk(v4f (&acc)[kTiles], const Chunk<NB>& c, float s01, float s23) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        v4f p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const v8bf w0 = bf16_of_codes(c.w[t][j].x, c.w[t][j].y), w1 = bf16_of_codes(c.w[t][j].z, c.w[t][j].w);
#pragma unroll
            for (int n = NB - 1; n >= 0; --n) {
                p = mfma(w0, __builtin_bit_cast(v8bf, c.b[n][2 * j]), p);
                p = mfma(w1, __builtin_bit_cast(v8bf, c.b[n][2 * j + 1]), p);
            }
        }
        const float s = t < kTiles / 2 ? s01 : s23;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(p[i], s, acc[t][i]);
    }
}

// Sums over the chunks wave, wave+4, ... ; s01 and s23 are the block scales'
// rows of the first and last two row tiles.
template <int NB>
__device__ __forceinline__ void multiply(v4f (&acc)[kTiles], const uint8_t* const (&w)[kTiles],
                                         const uint16_t* const (&b)[NB], const float* s01, const float* s23,
                                         int chunks, int wave) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
    Chunk<NB> c0, c1;
    int kb = wave;
    if (kb >= chunks) return;
    load_chunk<NB>(c0, w, b, kb);
    for (;;) {
        if (kb + 4 < chunks) load_chunk<NB>(c1, w, b, kb + 4);
        multiply_chunk<NB>(acc, c0, s01[kb], s23[kb]);
        kb += 4;
        if (kb >= chunks) return;
        if (kb + 4 < chunks) load_chunk<NB>(c0, w, b, kb + 4);
        multiply_chunk<NB>(acc, c1, s01[kb], s23[kb]);
        kb += 4;
        if (kb >= chunks) return;
    }
}

// The lane's token among the expert's (the (t0 + r)-th bit of the mask); the
// first one's for a lane without.
__device__ __forceinline__ int token_of(uint64_t mask, int t0, int r) {
    int mine = __builtin_ctzll(mask);
    for (int i = 0; mask != 0; ++i, mask &= mask - 1)
        if (i == t0 + r) mine = __builtin_ctzll(mask);
    return mine;
}

// Writes the waves' sums to LDS: element (token column, row) of tile t.
__device__ __forceinline__ void put_sums(float (*s_acc)[kTiles][256], const v4f (&acc)[kTiles], int wave, int r, int kq) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t) *reinterpret_cast<v4f*>(&s_acc[wave][t][r * 16 + 4 * kq]) = acc[t];
}

__device__ __forceinline__ float sum_waves(const float (*s_acc)[kTiles][256], int t, int at) {
    return (s_acc[0][t][at] + s_acc[1][t][at]) + (s_acc[2][t][at] + s_acc[3][t][at]);
}

// Gate and up projections with the SwiGLU: 32 gate rows and the 32 up rows
// that belong to them.
__global__ __launch_bounds__(256) void moe_up_kernel(MoeArgs a, MoeLayout L) {
    __shared__ __align__(16) float s_acc[4][kTiles][256];
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    const int idx = blockIdx.y;
    if (idx >= reinterpret_cast<const MoePlan*>(ws)->active) return;
    const int e = reinterpret_cast<const int*>(ws + L.experts)[idx];
    const int base = reinterpret_cast<const int*>(ws + L.base)[idx];
    const uint64_t mask = reinterpret_cast<const uint64_t*>(ws + L.mask)[idx];
    const int count = __popcll(mask);
    const float* prob = reinterpret_cast<const float*>(ws + L.prob) + base;

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, kq = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.x * 32;
    const uint8_t* wg = a.w_gu + e * a.w_gu_stride + (row0 + r) * a.ldw_gu + 16 * kq;
    const uint8_t* wu = wg + a.inner * a.ldw_gu;
    const uint8_t* w[kTiles] = {wg, wg + 16 * a.ldw_gu, wu, wu + 16 * a.ldw_gu};
    const float* sg = a.s_gu + e * a.s_gu_stride + (row0 >> 7) * a.lds_gu;
    const float* su = sg + (a.inner >> 7) * a.lds_gu;

    for (int t0 = 0; t0 < count; t0 += 16) {
        const uint16_t* x[1] = {a.x + token_of(mask, t0, r) * a.ldx + 16 * kq};
        v4f acc[kTiles];
        multiply<1>(acc, w, x, sg, su, (int)(a.hidden >> 7), wave);
        put_sums(s_acc, acc, wave, r, kq);
        __syncthreads();
        const int tok = threadIdx.x >> 4, c = 2 * (threadIdx.x & 15);  // two neighbouring columns of h
        if (t0 + tok < count) {
            float h[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = tok * 16 + (c & 15) + i;
                const float g = sum_waves(s_acc, c >> 4, at), u = sum_waves(s_acc, 2 + (c >> 4), at);
                h[i] = g / (1.0f + expf(-g)) * u * prob[t0 + tok];
            }
            const uint32_t hi = pack_bf16(h[0], h[1]);
            const int64_t at = (int64_t)(base + t0 + tok) * a.inner + row0 + c;
            *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(ws + L.hi) + at) = hi;
            *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(ws + L.lo) + at) =
                pack_bf16(h[0] - bf16_lo(hi), h[1] - bf16_hi(hi));
        }
        __syncthreads();
    }
}

// Down projection: 64 rows of the hidden size, one fp32 row of it per pair.
__global__ __launch_bounds__(256) void moe_down_kernel(MoeArgs a, MoeLayout L) {
    __shared__ __align__(16) float s_acc[4][kTiles][256];
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    const int idx = blockIdx.y;
    if (idx >= reinterpret_cast<const MoePlan*>(ws)->active) return;
    const int e = reinterpret_cast<const int*>(ws + L.experts)[idx];
    const int base = reinterpret_cast<const int*>(ws + L.base)[idx];
    const int count = __popcll(reinterpret_cast<const uint64_t*>(ws + L.mask)[idx]);

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, kq = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.x * 64;
    const uint8_t* w0 = a.w_down + e * a.w_down_stride + (row0 + r) * a.ldw_down + 16 * kq;
    const uint8_t* w[kTiles] = {w0, w0 + 16 * a.ldw_down, w0 + 32 * a.ldw_down, w0 + 48 * a.ldw_down};
    const float* s = a.s_down + e * a.s_down_stride + (row0 >> 7) * a.lds_down;

    for (int t0 = 0; t0 < count; t0 += 16) {
        const int64_t from = (int64_t)(base + t0 + (t0 + r < count ? r : 0)) * a.inner + 16 * kq;
        const uint16_t* h[2] = {reinterpret_cast<const uint16_t*>(ws + L.hi) + from,
                                reinterpret_cast<const uint16_t*>(ws + L.lo) + from};
        v4f acc[kTiles];
        multiply<2>(acc, w, h, s, s, (int)(a.inner >> 7), wave);
        put_sums(s_acc, acc, wave, r, kq);
        __syncthreads();
        const int c = threadIdx.x & 63;  // row of the hidden size
        for (int tok = threadIdx.x >> 6; tok < 16 && t0 + tok < count; tok += 4) {
            const float v = sum_waves(s_acc, c >> 4, tok * 16 + (c & 15));
            reinterpret_cast<float*>(ws + L.parts)[(int64_t)(base + t0 + tok) * a.hidden + row0 + c] = v;
        }
        __syncthreads();
    }
}

// A token's pairs added in the order of their experts.
__global__ __launch_bounds__(256) void moe_join_kernel(MoeArgs a, MoeLayout L) {
    const uint8_t* ws = static_cast<const uint8_t*>(a.workspace);
    const MoePlan* plan = reinterpret_cast<const MoePlan*>(ws);
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int t = blockIdx.y;
    if (c >= a.hidden) return;
    const int* pair = reinterpret_cast<const int*>(ws + L.pair) + t * kMaxTopK;
    const float* parts = reinterpret_cast<const float*>(ws + L.parts) + c;
    const int n = plan->count[t];
    float v = 0.0f;
    for (int i = 0; i < n; ++i) v += parts[pair[i] * a.hidden];
    if ((plan->nan_mask >> t) & 1) v = __builtin_nanf("");
    if (a.y_dtype == kDtypeBF16)
        static_cast<uint16_t*>(a.y)[t * a.ldy + c] = (uint16_t)pack_bf16(v, 0.0f);
    else
        static_cast<float*>(a.y)[t * a.ldy + c] = v;
}

// ----------------------------------------------------------------------------
// Workspace and launcher (arguments already validated by the API layer).
// ----------------------------------------------------------------------------
namespace {

MoeLayout moe_layout(int64_t tokens, int64_t hidden, int64_t inner, int experts, int top_k) {
    MoeLayout L;
    L.pairs = tokens * std::min(top_k, experts);
    L.slots = (int)std::min<int64_t>(experts, L.pairs);
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
    L.prob = take(4 * L.pairs);
    L.pair = take(4 * tokens * kMaxTopK);
    L.hi = take(2 * L.pairs * inner);
    L.lo = take(2 * L.pairs * inner);
    L.parts = take(4 * L.pairs * hidden);
    L.total = at;
    return L;
}

template <int PL>
void launch_route(const MoeArgs& a, const MoeLayout& L, hipStream_t st) {
    hipLaunchKernelGGL(moe_route_kernel<PL>, dim3(1), dim3(64 * std::min(kRouteWaves, a.tokens)), 0, st, a, L);
}

}  // namespace

int64_t moe_decode_bytes(int64_t tokens, int64_t hidden, int64_t inner, int experts, int top_k) {
    return moe_layout(tokens, hidden, inner, experts, top_k).total;
}

hipError_t launch_moe_decode(const MoeArgs& a, hipStream_t st) {
    const MoeLayout L = moe_layout(a.tokens, a.hidden, a.inner, a.experts, a.top_k);
    if (a.experts <= 64) launch_route<1>(a, L, st);
    else if (a.experts <= 256) launch_route<4>(a, L, st);
    else launch_route<kMaxExperts / 64>(a, L, st);
    hipLaunchKernelGGL(moe_up_kernel, dim3((unsigned)(a.inner / 32), (unsigned)L.slots), dim3(256), 0, st, a, L);
    hipLaunchKernelGGL(moe_down_kernel, dim3((unsigned)(a.hidden / 64), (unsigned)L.slots), dim3(256), 0, st, a, L);
    hipLaunchKernelGGL(moe_join_kernel, dim3((unsigned)((a.hidden + 255) / 256), (unsigned)a.tokens), dim3(256), 0, st,
                       a, L);
    return hipGetLastError();
}

}  // namespace fp8q
