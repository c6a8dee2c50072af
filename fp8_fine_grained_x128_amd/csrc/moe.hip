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
// h is held as a sum of bf16 numbers: for a bf16 result two, hi + lo (16
// significant bits: a relative error below 2^-16, the result's own rounding is
// 2^-9), for an fp32 result three, hi + lo + rest, which hold all of its 24.
//
// MFMA 16x16x32 (bf16): A: lane l holds row l%16, 8 values of the K step;
// B: column l%16, the same 8; D: lane l, element r is row 4*(l/16) + r,
// column l%16.  A holds weight rows, B tokens.
#include <algorithm>

#include "../../include/fp8q.h"
#include "launch.hpp"
#include "tile_io.hpp"

namespace fp8q {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int kMaxTokens = 64;
constexpr int kMaxExperts = 1024;
constexpr int kFusedTokens = 16;  // tokens that the gate and up projections may route themselves
constexpr int kFewTokens = 8;     // tokens whose two halves of h share a matrix operand

// Where the pieces of the workspace lie (bytes from its start).  Token t's
// pairs are t*top_k, t*top_k + 1, ..., one for each of its experts in
// ascending order.
struct MoeLayout {
    int slots;      // active experts at most
    int words;      // 64-bit words of a token's expert set
    int64_t sets;   // uint64[tokens][words]
    int64_t count;  // int[tokens]: experts of the token; -1: its logits hold NaN or +inf
    int64_t prob;   // float[pairs]
    int64_t hi, lo;  // bf16[pairs][inner], and a third, as far on, for rest: h
    int64_t parts;  // float[pairs][hidden]
    int64_t total;
};

__device__ __forceinline__ int64_t rest_of(const MoeLayout& L) { return 2 * L.lo - L.hi; }

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

// Bitwise or over the lanes of a wave, the same in all of them.
__device__ __forceinline__ uint32_t wave_or(uint32_t v) {
    v |= row_ror<8>(v);
    v |= row_ror<4>(v);
    v |= row_ror<2>(v);
    v |= row_ror<1>(v);
    return __builtin_amdgcn_readlane(v, 0) | __builtin_amdgcn_readlane(v, 16) | __builtin_amdgcn_readlane(v, 32) |
           __builtin_amdgcn_readlane(v, 48);
}

}  // namespace

// ----------------------------------------------------------------------------
// Routing: a wave per token.  Logits become order-preserving keys (-0 counts
// as 0); the k-th largest key is found bit by bit with wave ballots, ending
// early where exactly top_k keys lie at or above the prefix found so far;
// ties at the k-th key go to the lowest indices.
//   Only sets of experts are written, so tokens need nothing of each other
// and every token has a compute unit of its own (64 tokens: 4.5 us, which is
// a launch and one wave's dependent steps; one work-group for all tokens was
// bound by its scalar unit, 10 us).
// ----------------------------------------------------------------------------
template <int PL>  // experts per lane
__device__ __forceinline__ void route_token(const MoeArgs& a, const MoeLayout& L, int t, uint64_t* set, int* count,
                                            float* prob) {
    const int lane = threadIdx.x & 63;
    constexpr uint32_t kNone = 0x007fffffu;  // key of -inf; keys up to it are no candidates
    const uint64_t below = (1ull << lane) - 1;
    const float* row = a.logits + (int64_t)t * a.ldl;

    float l[PL], top = -__builtin_inff();
    uint32_t key[PL];
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
        if (lane < L.words) set[lane] = 0;
        if (lane == 0) *count = -1;
        return;
    }
#pragma unroll
    for (int off = 32; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    uint32_t kth = 0;
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t cand = kth | (1u << bit);
        int n = 0;
#pragma unroll
        for (int j = 0; j < PL; ++j) n += __popcll(__ballot(key[j] >= cand));
        if (n >= a.top_k) kth = cand;
        if (n == a.top_k) break;
    }
    kth = max(kth, kNone + 1);  // fewer candidates than top_k: all of them
    int above = 0;
#pragma unroll
    for (int j = 0; j < PL; ++j) above += __popcll(__ballot(key[j] > kth));
    int ties = a.top_k - above, n = 0;
    float p[PL], total = 0.0f;
    int at[PL];  // place among the token's choices, or -1
#pragma unroll
    for (int j = 0; j < PL; ++j) {
        // the search may end at a prefix below the k-th key: then exactly
        // top_k keys are at or above it, and all "ties" are in
        const uint64_t tie = __ballot(key[j] == kth);
        const bool in = key[j] > kth || (key[j] == kth && __popcll(tie & below) < ties);
        const uint64_t in_mask = __ballot(in);
        ties -= min(ties, (int)__popcll(tie));
        p[j] = key[j] >= kNone + 1 ? expf(l[j] - top) : 0.0f;
        at[j] = in ? n + (int)__popcll(in_mask & below) : -1;
        n += __popcll(in_mask);
        total += in || !a.renormalize ? p[j] : 0.0f;
        if (lane == 0 && j < L.words) set[j] = in_mask;
    }
    total = wave_sum(total);
#pragma unroll
    for (int j = 0; j < PL; ++j)
        if (at[j] >= 0) prob[at[j]] = p[j] / total;
    if (lane == 0) *count = n;
}

// Where routing leaves its result for the other kernels.
__device__ __forceinline__ uint64_t* sets_of(const MoeArgs& a, const MoeLayout& L) {
    return reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(a.workspace) + L.sets);
}
__device__ __forceinline__ int* counts_of(const MoeArgs& a, const MoeLayout& L) {
    return reinterpret_cast<int*>(static_cast<uint8_t*>(a.workspace) + L.count);
}
__device__ __forceinline__ float* probs_of(const MoeArgs& a, const MoeLayout& L) {
    return reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + L.prob);
}

template <int PL>
__global__ __launch_bounds__(64) void moe_route_kernel(MoeArgs a, MoeLayout L) {
    const int t = blockIdx.x;
    route_token<PL>(a, L, t, sets_of(a, L) + (int64_t)t * L.words, counts_of(a, L) + t, probs_of(a, L) + t * a.top_k);
}

// ----------------------------------------------------------------------------
// Both projections.  A work-group takes TILES row tiles of 16 weight rows of
// one active expert: rows of the hidden size, or as many tiles of gate rows as
// of the up rows that belong to them.  Its four waves take every fourth
// 128-wide chunk of the contraction, for NG groups of 16 of the expert's
// tokens at a time, and join their sums in LDS.
//   Weights go straight from memory to the matrix operand (16 rows of 64
// contiguous bytes a load), each one read once.  The row tiles share one read
// of the tokens, which comes from the caches; lanes of a column without a
// token read nothing and their results are dropped.
//   Bound by reading the weights: 64 tokens on 64 experts of 7168/2048 take
// 313 us for the 1.88 GB of gate and up rows and 175 us for the 0.94 GB of down
// rows (whose tokens are two halves, and whose pairs leave as fp32 rows); bare
// reads in the same pattern take 300 and 148, and reads of whole lines or
// copies into LDS no less.  Not faster: a chunk loaded ahead in registers,
// work-groups that run through the items with the next one's first chunk under
// way, an expert's work-groups on one XCD (2 % slower), tokens in LDS for waves
// that share the chunks and split the rows (a barrier per chunk: 60 % slower).
//   Row tiles and groups trade registers (work-groups per compute unit) for
// reads of the tokens and of the weights; expert_variant() chooses.
// ----------------------------------------------------------------------------

// A 128-wide chunk of TILES row tiles.
template <int TILES>
struct Weights {
    uint4 w[TILES][2];
    float s[2];  // block scales of the first and of the last half of the row tiles
};

// The same chunk of a lane's token.  NB: activation arrays whose sum is
// multiplied (x, or hi and lo, or hi, lo and rest).
template <int NB>
struct Tokens {
    uint4 b[NB][4];
};

// Where a work-group's chunks come from.
template <int TILES, int NG>
struct Operands {
    const uint8_t* w[TILES];
    const float* s[2];
    uint32_t row_offset;    // of the lane in a row tile
    const uint16_t* b[NG];  // the lane's token in every group; null: none
    int64_t lo;             // elements from one activation array to the next
};

template <int TILES, int NG>
__device__ __forceinline__ void load_weights(Weights<TILES>& c, const Operands<TILES, NG>& o, int kb) {
    const int64_t k = 128 * (int64_t)kb;
    c.s[0] = o.s[0][kb];
    c.s[1] = o.s[1][kb];
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) c.w[t][j] = *reinterpret_cast<const uint4*>(o.w[t] + k + 64 * j + o.row_offset);
}

// Keeps the codes and not the bf16 values made of them, which take twice the
// registers, from one group of tokens to the next.
template <int TILES>
__device__ __forceinline__ void forget(Weights<TILES>& c) {
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            opaque(c.w[t][j].x);
            opaque(c.w[t][j].y);
            opaque(c.w[t][j].z);
            opaque(c.w[t][j].w);
        }
}

template <int NB>
__device__ __forceinline__ void load_tokens(Tokens<NB>& c, const uint16_t* b, int64_t lo, int kb) {
    if (b == nullptr) return;
    const int64_t k = 128 * (int64_t)kb;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c.b[n][j] = *reinterpret_cast<const uint4*>(b + n * lo + k + (NB > 1 ? 32 * j : 64 * (j >> 1) + 8 * (j & 1)));
}

template <int NB, int TILES>
__device__ __forceinline__ void multiply_chunk(v4f (&acc)[TILES], const Weights<TILES>& c, const Tokens<NB>& x) {
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
        v4f p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const v8bf w0 = bf16_of_codes(c.w[t][j].x, c.w[t][j].y), w1 = bf16_of_codes(c.w[t][j].z, c.w[t][j].w);
#pragma unroll
            for (int n = NB - 1; n >= 0; --n) {
                p = mfma(w0, __builtin_bit_cast(v8bf, x.b[n][2 * j]), p);
                p = mfma(w1, __builtin_bit_cast(v8bf, x.b[n][2 * j + 1]), p);
            }
        }
        const float s = c.s[2 * t / TILES];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(p[i], s, acc[t][i]);
    }
}

// Sums of a wave over its chunks wave, wave+4, ..., for the first `groups`
// groups of 16 tokens.
template <int NB, int TILES, int NG>
__device__ __forceinline__ void multiply(v4f (&acc)[NG][TILES], const Operands<TILES, NG>& o, int chunks, int wave,
                                         int groups) {
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int t = 0; t < TILES; ++t) acc[g][t] = v4f{0.f, 0.f, 0.f, 0.f};
    Weights<TILES> w;
    Tokens<NB> x;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) x.b[n][j] = make_uint4(0, 0, 0, 0);
    for (int kb = wave; kb < chunks; kb += 4) {
        load_weights(w, o, kb);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (g > 0 && g >= groups) continue;
            load_tokens<NB>(x, o.b[g], o.lo, kb);
            multiply_chunk<NB>(acc[g], w, x);
            if (g + 1 < NG) forget(w);
        }
    }
}

// Joins the waves' sums of a group in LDS: [wave][row tile][token column * 16 + row].
template <int TILES>
__device__ __forceinline__ void join_waves(float (*sums)[TILES][256], const v4f (&acc)[TILES], int wave) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int t = 0; t < TILES; ++t) *reinterpret_cast<v4f*>(&sums[wave][t][16 * (lane & 15) + 4 * (lane >> 4)]) = acc[t];
    __syncthreads();
}

template <int TILES>
__device__ __forceinline__ float sum_waves(const float (*s)[TILES][256], int t, int at) {
    return (s[0][t][at] + s[1][t][at]) + (s[2][t][at] + s[3][t][at]);
}

// Waves per SIMD that the registers of a variant leave.
constexpr int waves_of(int tiles, int groups) { return tiles * groups <= 4 ? 4 : tiles * groups <= 8 ? 3 : 2; }

// Where column k of h is stored in its row: inside each 128-wide chunk, column
// 64*j + 16*kq + 8*i + n (the bytes of a 16-byte load of the weights) lies at
// 64*j + 32*i + 8*kq + n, so that a load instruction of the down projection
// reads 64 contiguous bytes of every token.
__device__ __forceinline__ int64_t h_place(int64_t k) {
    return (k & ~int64_t(0x3f)) | ((k & 8) << 2) | ((k & 0x30) >> 1) | (k & 7);
}

// The work-group's expert, its tokens and their pairs, from the tokens' sets:
// lane t of every wave looks at token t.
struct Chosen {
    int expert;  // -1: there are not that many active experts
    int count;   // tokens
};

__device__ __forceinline__ Chosen choose(const MoeArgs& a, const MoeLayout& L, const uint64_t* sets, int idx, int* tokens,
                                         int* pairs) {
    const int t = threadIdx.x & 63;
    const uint64_t* set = sets + t * L.words;
    int rank = 0;  // the token's experts below
    for (int w0 = 0; w0 < L.words; w0 += 4) {
        uint64_t m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = t < a.tokens && w0 + i < L.words ? set[w0 + i] : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint64_t any = wave_or((uint32_t)m[i]) | (uint64_t)wave_or((uint32_t)(m[i] >> 32)) << 32;
            const int n = __popcll(any);
            if (idx >= n) {
                idx -= n;
                rank += __popcll(m[i]);
                continue;
            }
            for (; idx > 0; --idx) any &= any - 1;
            const int bit = __builtin_ctzll(any);
            const bool mine = (m[i] >> bit) & 1;
            const uint64_t users = __ballot(mine);
            if (mine && threadIdx.x < 64) {
                const int at = __popcll(users & ((1ull << t) - 1));
                tokens[at] = t;
                pairs[at] = t * a.top_k + rank + (int)__popcll(m[i] & ((1ull << bit) - 1));
            }
            return {64 * (w0 + i) + bit, (int)__popcll(users)};
        }
    }
    return {-1, 0};
}

// Gate and up projections with the SwiGLU.  PL > 0: every work-group routes
// the (few) tokens for itself, and the first one leaves the result for the
// kernels that follow; PL == 0: routing has run.
template <int PL, int TILES, int NG>
__global__ __launch_bounds__(256, waves_of(TILES, NG)) void moe_up_kernel(MoeArgs a, MoeLayout L) {
    __shared__ __align__(16) float s_sums[4][TILES][256];
    __shared__ int s_token[kMaxTokens], s_pair[kMaxTokens];
    __shared__ uint64_t s_sets[PL > 0 ? kFusedTokens * PL : 1];
    __shared__ int s_count[kFusedTokens];
    __shared__ float s_prob[PL > 0 ? kFusedTokens * FP8Q_MOE_MAX_TOP_K : 1];
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    const float* prob = probs_of(a, L);
    Chosen e;
    if constexpr (PL > 0) {
        for (int t = threadIdx.x >> 6; t < a.tokens; t += 4)
            route_token<PL>(a, L, t, s_sets + t * L.words, s_count + t, s_prob + t * a.top_k);
        __syncthreads();
        if (blockIdx.x == 0 && blockIdx.y == 0) {
            for (int i = threadIdx.x; i < a.tokens * L.words; i += 256) sets_of(a, L)[i] = s_sets[i];
            if ((int)threadIdx.x < a.tokens) counts_of(a, L)[threadIdx.x] = s_count[threadIdx.x];
        }
        e = choose(a, L, s_sets, blockIdx.y, s_token, s_pair);
        prob = s_prob;
    } else {
        e = choose(a, L, sets_of(a, L), blockIdx.y, s_token, s_pair);
    }
    if (e.expert < 0) return;
    __syncthreads();
    int y_dtype = __builtin_amdgcn_readfirstlane(a.y_dtype);
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+s"(y_dtype));  // loaded here: where it is used its load would be waited for (0.2 us)
#endif
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, kq = lane >> 4;
    constexpr int kCols = 8 * TILES;  // columns of h
    const int64_t row0 = (int64_t)blockIdx.x * kCols;
    Operands<TILES, NG> o;
    const uint8_t* w = a.w_gu + e.expert * a.w_gu_stride + row0 * a.ldw_gu;
#pragma unroll
    for (int t = 0; t < TILES / 2; ++t) {
        o.w[t] = w + 16 * t * a.ldw_gu;
        o.w[TILES / 2 + t] = w + (a.inner + 16 * t) * a.ldw_gu;
    }
    o.row_offset = (uint32_t)(r * a.ldw_gu) + 16 * kq;
    o.s[0] = a.s_gu + e.expert * a.s_gu_stride + (row0 >> 7) * a.lds_gu;
    o.s[1] = o.s[0] + (a.inner >> 7) * a.lds_gu;
    o.lo = 0;
    for (int t0 = 0; t0 < e.count; t0 += 16 * NG) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int t = t0 + 16 * g + r;
            o.b[g] = t < e.count ? a.x + s_token[t] * a.ldx + 16 * kq : nullptr;
        }
        const int groups = min(NG, (e.count - t0 + 15) / 16);
        v4f acc[NG][TILES];
        multiply<1>(acc, o, (int)(a.hidden >> 7), wave, groups);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (g >= groups) continue;
            join_waves(s_sums, acc[g], wave);
            constexpr int kPer = TILES / 2;  // columns of a thread
            const int tok = threadIdx.x >> 4, c = kPer * (threadIdx.x & 15);
            if (t0 + 16 * g + tok < e.count) {
                const int64_t pair = s_pair[t0 + 16 * g + tok];
                const float p = prob[pair];
                const int64_t at = pair * a.inner + h_place(row0 + c);
                float rest[kPer];
                uint16_t hi[kPer], lo[kPer];
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int in = tok * 16 + (c & 15) + i;
                    const float gate = sum_waves(s_sums, c >> 4, in), up = sum_waves(s_sums, TILES / 2 + (c >> 4), in);
                    const float h = gate / (1.0f + expf(-gate)) * up * p;
                    hi[i] = (uint16_t)pack_bf16(h, 0.0f);
                    // both differences are exact; an infinite h has none
                    const float l = (hi[i] & 0x7f80u) == 0x7f80u ? 0.0f : h - bf16_bits_to_f32(hi[i]);
                    lo[i] = (uint16_t)pack_bf16(l, 0.0f);
                    rest[i] = l - bf16_bits_to_f32(lo[i]);
                }
                uint16_t* to_hi = reinterpret_cast<uint16_t*>(ws + L.hi) + at;
                uint16_t* to_lo = reinterpret_cast<uint16_t*>(ws + L.lo) + at;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    to_hi[i] = hi[i];
                    to_lo[i] = lo[i];
                }
                if (y_dtype == kDtypeF32) {
                    uint16_t* to_rest = reinterpret_cast<uint16_t*>(ws + rest_of(L)) + at;
#pragma unroll
                    for (int i = 0; i < kPer; ++i) to_rest[i] = (uint16_t)pack_bf16(rest[i], 0.0f);
                }
            }
            __syncthreads();
        }
    }
}

// Down projection: one fp32 row of the hidden size per pair.  NB: arrays whose
// sum is h.
template <int NB, int TILES, int NG>
__global__ __launch_bounds__(256, waves_of(TILES, NG)) void moe_down_kernel(MoeArgs a, MoeLayout L) {
    __shared__ __align__(16) float s_sums[4][TILES][256];
    __shared__ int s_token[kMaxTokens], s_pair[kMaxTokens];
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    const Chosen e = choose(a, L, sets_of(a, L), blockIdx.y, s_token, s_pair);
    if (e.expert < 0) return;
    __syncthreads();
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, kq = lane >> 4;
    constexpr int kRows = 16 * TILES;
    const int64_t row0 = (int64_t)blockIdx.x * kRows;
    Operands<TILES, NG> o;
    const uint8_t* w = a.w_down + e.expert * a.w_down_stride + row0 * a.ldw_down;
#pragma unroll
    for (int t = 0; t < TILES; ++t) o.w[t] = w + 16 * t * a.ldw_down;
    o.row_offset = (uint32_t)(r * a.ldw_down) + 16 * kq;
    o.s[0] = o.s[1] = a.s_down + e.expert * a.s_down_stride + (row0 >> 7) * a.lds_down;
    o.lo = (L.lo - L.hi) / 2;
    for (int t0 = 0; t0 < e.count; t0 += 16 * NG) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int t = t0 + 16 * g + r;
            o.b[g] = t < e.count ? reinterpret_cast<const uint16_t*>(ws + L.hi) + s_pair[t] * a.inner + 8 * kq : nullptr;
        }
        const int groups = min(NG, (e.count - t0 + 15) / 16);
        v4f acc[NG][TILES];
        multiply<NB>(acc, o, (int)(a.inner >> 7), wave, groups);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (g >= groups) continue;
            join_waves(s_sums, acc[g], wave);
            const int c = threadIdx.x % kRows, first = t0 + 16 * g;
            for (int tok = threadIdx.x / kRows; tok < 16 && first + tok < e.count; tok += 256 / kRows)
                reinterpret_cast<float*>(ws + L.parts)[s_pair[first + tok] * a.hidden + row0 + c] =
                    sum_waves(s_sums, c >> 4, tok * 16 + (c & 15));
            __syncthreads();
        }
    }
}

// Down projection and weighted sum of at most eight tokens: a work-group takes
// 16 rows of the hidden size and all active experts, so y needs no partial
// results.  Matrix columns 0..7 are the tokens' hi halves of h, columns 8..15
// their lo halves (half the loads and products of separate operands); an fp32
// result's rests are a second operand; a token that did not choose the expert
// takes nothing of it (its NaN neither).  The
// eight waves share the (expert, chunk) pairs; weights are loaded three of
// them ahead, h one ahead.
//   One token of 8 experts of 7168/2048 (117 MB): 28 us, of which 19 are the
// reads at the rate of the general kernel's probe and the rest the start (the
// experts' sets come before the first weights) and 448 work-groups on 256
// compute units.
constexpr int kFewWaves = 8;

template <bool REST>
__global__ __launch_bounds__(64 * kFewWaves, 4) void moe_down_few_kernel(MoeArgs a, MoeLayout L) {
    constexpr int kSlots = kFewTokens * FP8Q_MOE_MAX_TOP_K;
    __shared__ __align__(16) float s_sums[kFewWaves][256];
    __shared__ int s_expert[kSlots];
    __shared__ int s_pair[kSlots][kFewTokens];  // the token's pair with the expert, or -1
    const uint8_t* ws = static_cast<const uint8_t*>(a.workspace);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, kq = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.x * 16;
    const int chunks = (int)(a.inner >> 7);

    int active = 0, rank = 0;  // experts so far; the lane's token's experts so far
    for (int w = 0; w < L.words; ++w) {
        const uint64_t m = lane < a.tokens ? sets_of(a, L)[lane * L.words + w] : 0;
        uint64_t any = wave_or((uint32_t)m) | (uint64_t)wave_or((uint32_t)(m >> 32)) << 32;
        for (; any != 0; any &= any - 1, ++active) {
            const int bit = __builtin_ctzll(any);
            if (active % kFewWaves != wave) continue;
            if (lane < kFewTokens)
                s_pair[active][lane] =
                    (m >> bit) & 1 ? lane * a.top_k + rank + (int)__popcll(m & ((1ull << bit) - 1)) : -1;
            if (lane == 0) s_expert[active] = 64 * w + bit;
        }
        rank += __popcll(m);
    }
    __syncthreads();

    struct Item {  // an (expert, chunk) pair of this wave
        int idx, kb;
    };
    auto advance = [&](Item& i) {
        i.kb += kFewWaves;
        while (i.kb >= chunks) {
            i.kb -= chunks;
            ++i.idx;
        }
    };
    const uint8_t* w_rows = a.w_down + row0 * a.ldw_down;
    const uint32_t row_offset = (uint32_t)(r * a.ldw_down) + 16 * kq;
    const float* s_rows = a.s_down + (row0 >> 7) * a.lds_down;
    const uint16_t* half = reinterpret_cast<const uint16_t*>(ws + (r < kFewTokens ? L.hi : L.lo));
    const uint16_t* rests = reinterpret_cast<const uint16_t*>(ws + rest_of(L));
    uint4 w[4][2], h[2][4], rest[2][REST ? 4 : 1];
    float scale[4];
    bool takes[2];  // the lane's token chose the expert
    auto load_w = [&](const Item& i, int slot) {
        if (i.idx >= active) return;
        const int e = __builtin_amdgcn_readfirstlane(s_expert[i.idx]);
        const uint8_t* p = w_rows + e * a.w_down_stride + 128 * (int64_t)i.kb;
        w[slot][0] = *reinterpret_cast<const uint4*>(p + row_offset);
        w[slot][1] = *reinterpret_cast<const uint4*>(p + 64 + row_offset);
        scale[slot] = s_rows[e * a.s_down_stride + i.kb];
    };
    auto load_h = [&](const Item& i, int slot) {
        const int pair = i.idx < active ? s_pair[i.idx][r % kFewTokens] : -1;
        takes[slot] = pair >= 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) h[slot][j] = make_uint4(0, 0, 0, 0);
        if constexpr (REST) {
#pragma unroll
            for (int j = 0; j < 4; ++j) rest[slot][j] = make_uint4(0, 0, 0, 0);
        }
        if (pair < 0) return;
        const int64_t at = (int64_t)pair * a.inner + 128 * (int64_t)i.kb + 8 * kq;
#pragma unroll
        for (int j = 0; j < 4; ++j) h[slot][j] = *reinterpret_cast<const uint4*>(half + at + 32 * j);
        if constexpr (REST) {
            if (r >= kFewTokens) return;
#pragma unroll
            for (int j = 0; j < 4; ++j) rest[slot][j] = *reinterpret_cast<const uint4*>(rests + at + 32 * j);
        }
    };
    Item now{0, wave - kFewWaves}, next_h, next_w;
    advance(now);
    next_h = next_w = now;
#pragma unroll
    for (int u = 0; u < 3; ++u) {
        load_w(next_w, u);
        advance(next_w);
    }
    load_h(next_h, 0);
    advance(next_h);
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    while (now.idx < active) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (now.idx >= active) break;
            load_w(next_w, (u + 3) & 3);
            advance(next_w);
            load_h(next_h, (u + 1) & 1);
            advance(next_h);
            v4f p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const v8bf w0 = bf16_of_codes(w[u][j].x, w[u][j].y), w1 = bf16_of_codes(w[u][j].z, w[u][j].w);
                if constexpr (REST) {
                    p = mfma(w0, __builtin_bit_cast(v8bf, rest[u & 1][2 * j]), p);
                    p = mfma(w1, __builtin_bit_cast(v8bf, rest[u & 1][2 * j + 1]), p);
                }
                p = mfma(w0, __builtin_bit_cast(v8bf, h[u & 1][2 * j]), p);
                p = mfma(w1, __builtin_bit_cast(v8bf, h[u & 1][2 * j + 1]), p);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = takes[u & 1] ? __builtin_fmaf(p[i], scale[u], acc[i]) : acc[i];
            advance(now);
        }
    }
    *reinterpret_cast<v4f*>(&s_sums[wave][16 * r + 4 * kq]) = acc;
    __syncthreads();
    const int t = threadIdx.x >> 4, c = threadIdx.x & 15;  // token and row
    if (t >= a.tokens) return;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kFewWaves; ++k) v += s_sums[k][16 * t + c] + s_sums[k][16 * (t + kFewTokens) + c];
    if (counts_of(a, L)[t] < 0) v = __builtin_nanf("");
    if (a.y_dtype == kDtypeBF16)
        static_cast<uint16_t*>(a.y)[t * a.ldy + row0 + c] = (uint16_t)pack_bf16(v, 0.0f);
    else
        static_cast<float*>(a.y)[t * a.ldy + row0 + c] = v;
}

// A token's pairs added in the order of their experts (64 tokens of 8 experts,
// 7168 columns: 6 us for 15 MB from the caches).
__global__ __launch_bounds__(256) void moe_join_kernel(MoeArgs a, MoeLayout L) {
    const uint8_t* ws = static_cast<const uint8_t*>(a.workspace);
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int t = blockIdx.y;
    if (c >= a.hidden) return;
    const float* parts = reinterpret_cast<const float*>(ws + L.parts) + (int64_t)t * a.top_k * a.hidden + c;
    const int n = reinterpret_cast<const int*>(ws + L.count)[t];
    float v = n < 0 ? __builtin_nanf("") : 0.0f;
    for (int i = 0; i < n; ++i) v += parts[i * a.hidden];
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
    const int64_t pairs = tokens * top_k;
    L.slots = (int)std::min<int64_t>(experts, pairs);
    L.words = (experts + 63) / 64;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    L.sets = take(8 * tokens * L.words);
    L.count = take(4 * tokens);
    L.prob = take(4 * pairs);
    L.hi = take(2 * pairs * inner);
    L.lo = take(2 * pairs * inner);
    take(2 * pairs * inner);
    L.parts = take(4 * pairs * hidden);
    L.total = at;
    return L;
}

// Row tiles and token groups of the projections, for the mean number of
// tokens of an expert.
struct Variant {
    int tiles, groups;
};

// `tiles`: row tiles of an expert.
//   Groups: with more tokens than one group of 16 holds, a second group saves
// reading the weights again (64 tokens, 8 of 24 experts 7168/2048: 246 us,
// 375 without), where an expert has few it only costs registers (8 of 64: 505
// against 500; 8 of 64 experts 2048/512: 58 against 56).  Four groups pay where
// nearly all tokens share the experts (8 of 8 experts 7168/2048: 174, two groups
// of eight tiles 179; 8 of 24: 286 against 246).
//   Eight tiles halve the reads of the tokens, which matter from about four
// tokens per expert (64 tokens, 8 of 64 experts 7168/2048: 500 us against 528,
// 16 tokens: 430 against 425), if there are still two work-groups for every
// compute unit (8 of 8 experts 2048/1024, half a work-group: 65 against 49).
// Two tiles where four give less than one (12 tokens, 2 experts 4096/14336: 96
// us, 108 with four; 16 tokens, 4 experts 2048/8192: 61 and 68; with enough of
// them they are slower: 16 tokens, 8 of 64 experts 7168/2048, 452 against 427).
Variant expert_variant(const MoeArgs& a, const MoeLayout& L, int64_t tiles) {
    const int64_t pairs = a.tokens * a.top_k;
    if (pairs >= 32 * L.slots) return {4, 4};
    const int cus = compute_units(), groups = pairs > 8 * L.slots && a.tokens > 16 ? 2 : 1;
    if (pairs >= 4 * L.slots && tiles / 8 * L.slots >= 2 * cus) return {8, groups};
    return {groups == 1 && tiles / 4 * L.slots < cus ? 2 : 4, groups};
}

template <int TILES, int NG>
void launch_up(const MoeArgs& a, const MoeLayout& L, hipStream_t st) {
    hipLaunchKernelGGL((moe_up_kernel<0, TILES, NG>), dim3((unsigned)(a.inner / (8 * TILES)), (unsigned)L.slots),
                       dim3(256), 0, st, a, L);
}

template <int TILES, int NG>
void launch_down(const MoeArgs& a, const MoeLayout& L, hipStream_t st) {
    const dim3 grid((unsigned)(a.hidden / (16 * TILES)), (unsigned)L.slots);
    if (a.y_dtype == kDtypeF32) hipLaunchKernelGGL((moe_down_kernel<3, TILES, NG>), grid, dim3(256), 0, st, a, L);
    else hipLaunchKernelGGL((moe_down_kernel<2, TILES, NG>), grid, dim3(256), 0, st, a, L);
}

void launch_up(const MoeArgs& a, const MoeLayout& L, hipStream_t st) {
    const Variant v = expert_variant(a, L, a.inner / 8);  // gate and up tiles
    if (v.groups == 4) launch_up<4, 4>(a, L, st);
    else if (v.tiles == 8) v.groups == 2 ? launch_up<8, 2>(a, L, st) : launch_up<8, 1>(a, L, st);
    else if (v.groups == 2) launch_up<4, 2>(a, L, st);
    else v.tiles == 4 ? launch_up<4, 1>(a, L, st) : launch_up<2, 1>(a, L, st);
}

void launch_down(const MoeArgs& a, const MoeLayout& L, hipStream_t st) {
    const Variant v = expert_variant(a, L, a.hidden / 16);
    if (v.groups == 4) launch_down<4, 4>(a, L, st);
    else if (v.tiles == 8) v.groups == 2 ? launch_down<8, 2>(a, L, st) : launch_down<8, 1>(a, L, st);
    else if (v.groups == 2) launch_down<4, 2>(a, L, st);
    else v.tiles == 4 ? launch_down<4, 1>(a, L, st) : launch_down<2, 1>(a, L, st);
}

// Routing, alone or (fused) in the gate and up projections.
template <int PL>
void launch_route(const MoeArgs& a, const MoeLayout& L, bool fused, hipStream_t st) {
    if (fused)
        hipLaunchKernelGGL((moe_up_kernel<PL, 4, 1>), dim3((unsigned)(a.inner / 32), (unsigned)L.slots), dim3(256), 0,
                           st, a, L);
    else
        hipLaunchKernelGGL(moe_route_kernel<PL>, dim3((unsigned)a.tokens), dim3(64), 0, st, a, L);
}

}  // namespace

int64_t moe_decode_bytes(int64_t tokens, int64_t hidden, int64_t inner, int experts, int top_k) {
    return moe_layout(tokens, hidden, inner, experts, top_k).total;
}

hipError_t launch_moe_decode(const MoeArgs& a, hipStream_t st) {
    const MoeLayout L = moe_layout(a.tokens, a.hidden, a.inner, a.experts, a.top_k);
    const int cus = compute_units();
    // A kernel of its own for routing costs 5 us; done by every work-group of
    // the gate and up projections it costs each about 1 us for four tokens.
    const bool fused = a.tokens <= 4 || (a.tokens <= kFusedTokens && a.inner / 32 * L.slots <= 4 * cus);
    if (a.experts <= 64) launch_route<1>(a, L, fused, st);
    else if (a.experts <= 256) launch_route<4>(a, L, fused, st);
    else launch_route<kMaxExperts / 64>(a, L, fused, st);
    if (!fused) launch_up(a, L, st);
    // All experts in one work-group where they are little to read, or few for
    // few tokens.  A kernel less is worth 2 to 3 us to a caller that waits for
    // its launches and 1 to 10 us of the kernels' own time; but each expert
    // costs its start there, and there are only hidden / 16 work-groups.  (This
    // kernel against the general one and its join, kernels' time.  Hidden 2048,
    // half a work-group for each compute unit: one token on 8 of 64 experts
    // 2048/512 16.6 and 18.9 us, two 20.6 and 21.2, four 30.1 and 27.3, eight on
    // 2 of 8 experts 2048/8192 104 and 84; one token on 7 experts 1280/1408 20.4
    // and 20.9, five on 8 experts 512/1280 21.8 and 18.6.  Hidden 4096 and 7168: one token on
    // 8 of 64 experts 7168/2048 76.3 and 76.7, on 2 of 8 experts 4096/14336 82
    // and 87; four on 8 experts 195 and 205; two on 8 of 64 experts 7168/2048
    // 139 and 132; eight on 2 of 8 experts 4096/2048 51 and 54, 4096/14336 261
    // and 254.  A call of three tokens on 4 of 24 experts 1024/512: 19.9 and
    // 22.3.  With the rests of an fp32 result: one token on 8 of 64 experts
    // 2048/512 19.3 and 21.4, 7168/2048 85 and 76; four on 2 of 16 experts
    // 2048/1024 22.9 and 21.0.)
    const int64_t bytes = L.slots * 16 * a.inner;
    const bool wide = a.hidden / 16 >= cus, light = a.tokens <= 4 && L.slots <= 8;
    const bool few = a.y_dtype == kDtypeF32 ? bytes <= 1 << 16
                                            : bytes <= (wide || light ? 1 << 18 : 1 << 17) || (wide && light);
    if (a.tokens <= kFewTokens && few) {
        const dim3 grid((unsigned)(a.hidden / 16)), block(64 * kFewWaves);
        if (a.y_dtype == kDtypeF32) hipLaunchKernelGGL(moe_down_few_kernel<true>, grid, block, 0, st, a, L);
        else hipLaunchKernelGGL(moe_down_few_kernel<false>, grid, block, 0, st, a, L);
    } else {
        launch_down(a, L, st);
        hipLaunchKernelGGL(moe_join_kernel, dim3((unsigned)((a.hidden + 255) / 256), (unsigned)a.tokens), dim3(256), 0,
                           st, a, L);
    }
    return hipGetLastError();
}

}  // namespace fp8q
