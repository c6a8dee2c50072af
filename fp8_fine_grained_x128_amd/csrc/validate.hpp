// validate.hpp -- host-side argument checks of the C ABI (include/fp8q.h).
//
// Plain C++ with no HIP dependency (so that it can also be built and run
// under the host sanitizers).  Every function returns kLaunch when the call
// is valid and has work to enqueue, FP8Q_OK when it is valid and empty
// (nothing is launched), or the fp8q_status error to return.  Nothing here
// dereferences a pointer: pointers are only tested for null and alignment.
#pragma once

#include <stdint.h>

#include "../../include/fp8q.h"

namespace fp8q {
namespace check {

constexpr int kLaunch = -1;

// Grid-dimension limit of the quantizer launches (y / x extents).
constexpr int64_t kMaxGridY = 65535;
constexpr int kMaxGroups = 1024;
// The GEMM reads a tile's operand rows through a buffer descriptor with 32-bit
// offsets and a 32-bit record count: 256 rows * ld must stay below 2^32.
constexpr int64_t kMaxOperandLd = (int64_t(1) << 24) - 1;
// Leading dimensions beyond 2^32 elements are refused before any size
// arithmetic, so that the products formed below (a leading dimension times
// an element size, a row count or a block count) stay far inside int64.
constexpr int64_t kMaxLd = int64_t(1) << 32;
// Expert strides of the grouped GEMM (elements); the kernels multiply them by
// an expert index below 1024.
constexpr int64_t kMaxGroupStride = int64_t(1) << 50;
constexpr unsigned kKnownGemmFlags = FP8Q_GEMM_MMA_FP8 | FP8Q_GEMM_POW2_SCALES;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int elem_bytes(int dtype) { return dtype == FP8Q_BF16 ? 2 : 4; }
inline bool valid_dtype(int d) { return d == FP8Q_F32 || d == FP8Q_BF16; }
inline bool valid_scale_mode(int m) { return m == FP8Q_SCALE_FP32 || m == FP8Q_SCALE_POW2; }
inline bool ld_ok(int64_t ld) { return ld >= 0 && ld <= kMaxLd; }

inline int quantize_act(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, int tile,
                        const void* q, int64_t ldq, const void* s, int64_t lds, int scale_mode) {
    if (!valid_dtype(x_dtype) || (tile != FP8Q_TILE_1x128 && tile != FP8Q_TILE_128x1)) return FP8Q_EINVAL;
    if (!valid_scale_mode(scale_mode)) return FP8Q_EINVAL;
    if (rows < 0 || cols < 0 || !ld_ok(ldx) || !ld_ok(ldq) || !ld_ok(lds)) return FP8Q_ESHAPE;
    if (ldx < cols) return FP8Q_ESHAPE;
    if (tile == FP8Q_TILE_1x128) {
        if (ldq < cols || lds < rows) return FP8Q_ESHAPE;
    } else {
        if (ldq < rows || lds < cols) return FP8Q_ESHAPE;
    }
    if (rows == 0 || cols == 0) return FP8Q_OK;
    if (!x || !q || !s) return FP8Q_EINVAL;
    if (!aligned(x, 16) || (ldx * elem_bytes(x_dtype)) % 16 != 0 || !aligned(q, 16) || ldq % 16 != 0 ||
        !aligned(s, 4))
        return FP8Q_EALIGN;
    if (tile == FP8Q_TILE_1x128 ? cdiv(cols, 512) > kMaxGridY : cdiv(rows, 128) > kMaxGridY)
        return FP8Q_EUNSUPPORTED;
    return kLaunch;
}

inline int gather_quantize_act(const void* x, int x_dtype, int64_t rows_in, int64_t cols, int64_t ldx,
                               const void* row_index, int64_t rows_out, const void* q, int64_t ldq,
                               const void* s, int64_t lds, int scale_mode) {
    if (!valid_dtype(x_dtype) || !valid_scale_mode(scale_mode)) return FP8Q_EINVAL;
    if (!ld_ok(ldx) || !ld_ok(ldq) || !ld_ok(lds)) return FP8Q_ESHAPE;
    if (rows_in < 0 || rows_out < 0 || cols < 0 || ldx < cols || ldq < cols || lds < rows_out) return FP8Q_ESHAPE;
    if (rows_out == 0 || cols == 0) return FP8Q_OK;
    if (!row_index || !q || !s || (rows_in > 0 && !x)) return FP8Q_EINVAL;
    if ((rows_in > 0 && !aligned(x, 16)) || (ldx * elem_bytes(x_dtype)) % 16 != 0 || !aligned(q, 16) ||
        ldq % 16 != 0 || !aligned(s, 4) || !aligned(row_index, 4))
        return FP8Q_EALIGN;
    if (cdiv(cols, 512) > kMaxGridY) return FP8Q_EUNSUPPORTED;
    return kLaunch;
}

inline int quantize_weight(const void* w, int w_dtype, int64_t N, int64_t K, int64_t ldw, const void* q,
                           int64_t ldq, const void* s, int64_t lds, int scale_mode) {
    if (!valid_dtype(w_dtype) || !valid_scale_mode(scale_mode)) return FP8Q_EINVAL;
    if (!ld_ok(ldw) || !ld_ok(ldq) || !ld_ok(lds)) return FP8Q_ESHAPE;
    if (N < 0 || K < 0 || ldw < K || ldq < K || lds < cdiv(K, 128)) return FP8Q_ESHAPE;
    if (N == 0 || K == 0) return FP8Q_OK;
    if (!w || !q || !s) return FP8Q_EINVAL;
    if (!aligned(w, 16) || (ldw * elem_bytes(w_dtype)) % 16 != 0 || !aligned(q, 16) || ldq % 16 != 0 ||
        !aligned(s, 4))
        return FP8Q_EALIGN;
    if (cdiv(N, 128) > kMaxGridY) return FP8Q_EUNSUPPORTED;
    return kLaunch;
}

inline int requant(const void* q, int64_t rows, int64_t cols, int64_t ldq, const void* s, int64_t lds,
                   const void* qt, int64_t ldqt, const void* st, int64_t ldst, int scale_mode) {
    if (!valid_scale_mode(scale_mode)) return FP8Q_EINVAL;
    if (!ld_ok(ldq) || !ld_ok(lds) || !ld_ok(ldqt) || !ld_ok(ldst)) return FP8Q_ESHAPE;
    if (rows < 0 || cols < 0 || ldq < cols || lds < rows || ldqt < rows || ldst < cols) return FP8Q_ESHAPE;
    if (rows == 0 || cols == 0) return FP8Q_OK;
    if (!q || !s || !qt || !st) return FP8Q_EINVAL;
    if (!aligned(q, 16) || ldq % 16 != 0 || !aligned(qt, 16) || ldqt % 16 != 0 || !aligned(s, 4) ||
        !aligned(st, 4))
        return FP8Q_EALIGN;
    if (cdiv(rows, 128) > kMaxGridY) return FP8Q_EUNSUPPORTED;
    return kLaunch;
}

inline int transpose_weight(const void* q, int64_t N, int64_t K, int64_t ldq, const void* s, int64_t lds,
                            const void* qt, int64_t ldqt, const void* st, int64_t ldst) {
    if (!ld_ok(ldq) || !ld_ok(lds) || !ld_ok(ldqt) || !ld_ok(ldst)) return FP8Q_ESHAPE;
    if (N < 0 || K < 0 || ldq < K || ldqt < N || lds < cdiv(K, 128) || ldst < cdiv(N, 128)) return FP8Q_ESHAPE;
    if (N == 0 || K == 0) return FP8Q_OK;
    if (!q || !s || !qt || !st) return FP8Q_EINVAL;
    if (!aligned(q, 16) || ldq % 16 != 0 || !aligned(qt, 16) || ldqt % 16 != 0 || !aligned(s, 4) ||
        !aligned(st, 4))
        return FP8Q_EALIGN;
    if (cdiv(N, 128) > kMaxGridY) return FP8Q_EUNSUPPORTED;
    return kLaunch;
}

// Checks shared by the plain and the grouped GEMM.
inline int gemm_common(const void* a, int64_t lda, const void* sa, const void* b, int64_t ldb, const void* sb,
                       int64_t M, int64_t N, int64_t K, const void* c, int c_dtype, int64_t ldc, unsigned flags) {
    if (!valid_dtype(c_dtype) || (flags & ~kKnownGemmFlags) != 0u) return FP8Q_EINVAL;
    if (!ld_ok(lda) || !ld_ok(ldb) || !ld_ok(ldc)) return FP8Q_ESHAPE;
    if (M < 0 || N < 0 || K < 0 || K % 128 != 0) return FP8Q_ESHAPE;
    if (lda < K || ldb < K || ldc < N) return FP8Q_ESHAPE;
    if (lda > kMaxOperandLd || ldb > kMaxOperandLd) return FP8Q_EUNSUPPORTED;
    if (M == 0 || N == 0) return FP8Q_OK;
    if (K == 0) return FP8Q_ESHAPE;  // an empty contraction is not a GEMM this library runs
    if (!a || !sa || !b || !sb || !c) return FP8Q_EINVAL;
    if (!aligned(a, 16) || lda % 16 != 0 || !aligned(b, 16) || ldb % 16 != 0 || !aligned(sa, 4) ||
        !aligned(sb, 4) || !aligned(c, (uintptr_t)elem_bytes(c_dtype)))
        return FP8Q_EALIGN;
    return kLaunch;
}

inline int gemm(const void* a, int64_t lda, const void* sa, int64_t ldsa, const void* b, int64_t ldb,
                const void* sb, int64_t ldsb, int bscale, int64_t M, int64_t N, int64_t K, const void* c,
                int c_dtype, int64_t ldc, int accumulate, unsigned flags) {
    if (bscale != FP8Q_BSCALE_BLOCK128 && bscale != FP8Q_BSCALE_ROW) return FP8Q_EINVAL;
    if ((flags & ~kKnownGemmFlags) != 0u) return FP8Q_EINVAL;
    if (accumulate && c_dtype != FP8Q_F32) return FP8Q_EUNSUPPORTED;
    const int rc = gemm_common(a, lda, sa, b, ldb, sb, M, N, K, c, c_dtype, ldc, flags);
    if (rc != kLaunch) return rc;
    if (ldsa < M) return FP8Q_ESHAPE;
    if (bscale == FP8Q_BSCALE_BLOCK128 ? ldsb < K / 128 : ldsb < N) return FP8Q_ESHAPE;
    return kLaunch;
}

// Split-K workspace (need: the plan's bytes, 0 when the shape does not split).
inline int splitk_workspace(int64_t need, const void* workspace, int64_t workspace_bytes) {
    if (workspace_bytes < 0) return FP8Q_ESHAPE;
    if (need > 0) {
        if (!workspace) return FP8Q_EINVAL;
        if (workspace_bytes < need) return FP8Q_ESHAPE;
        if (!aligned(workspace, 256)) return FP8Q_EALIGN;
    }
    return kLaunch;
}

inline int grouped(const void* a, int64_t lda, const void* sa, int64_t ldsa, const void* b, int64_t ldb,
                   int64_t b_group_stride, const void* sb, int64_t ldsb, int64_t sb_group_stride,
                   const void* group_offsets, int G, int64_t M_total, int64_t N, int64_t K, const void* c,
                   int c_dtype, int64_t ldc, unsigned flags) {
    if ((flags & ~kKnownGemmFlags) != 0u) return FP8Q_EINVAL;
    if (G < 1 || G > kMaxGroups) return FP8Q_ESHAPE;
    const int rc = gemm_common(a, lda, sa, b, ldb, sb, M_total, N, K, c, c_dtype, ldc, flags);
    if (rc != kLaunch) return rc;
    if (!group_offsets) return FP8Q_EINVAL;
    if (!aligned(group_offsets, 4)) return FP8Q_EALIGN;
    if (M_total > INT32_MAX) return FP8Q_EUNSUPPORTED;
    if (!ld_ok(ldsa) || !ld_ok(ldsb) || b_group_stride < 0 || b_group_stride > kMaxGroupStride ||
        sb_group_stride < 0 || sb_group_stride > kMaxGroupStride)
        return FP8Q_ESHAPE;
    if (ldsa < M_total || ldsb < K / 128) return FP8Q_ESHAPE;
    // N <= ldc <= 2^32 and ldb < 2^24, ldsb <= 2^32: both products stay below 2^57
    if (b_group_stride < (N - 1) * ldb + K || sb_group_stride < (cdiv(N, 128) - 1) * ldsb + K / 128)
        return FP8Q_ESHAPE;
    if (b_group_stride % 16 != 0) return FP8Q_EALIGN;
    return kLaunch;
}

inline int clock_probe(const void* out, int64_t ticks) {
    if (!out) return FP8Q_EINVAL;
    if (!aligned(out, 8)) return FP8Q_EALIGN;
    if (ticks <= 0 || ticks > 100000000) return FP8Q_ESHAPE;
    return kLaunch;
}

// ---- feed-forward operators around the GEMMs

// Widths a work-group holds in registers.
constexpr int64_t kMaxNormCols = FP8Q_NORM_MAX_COLS;

inline bool row_aligned(const void* p, int64_t ld, int dtype) {
    return aligned(p, 16) && (ld * elem_bytes(dtype)) % 16 == 0;
}

inline int layernorm(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, const void* gamma,
                     const void* beta, int w_dtype, float eps, int kind, const void* y, int y_dtype, int64_t ldy,
                     const void* q, int64_t ldq, const void* s, int64_t lds, int scale_mode, const void* mean,
                     const void* rstd) {
    if (!valid_dtype(x_dtype) || !valid_dtype(w_dtype) || !valid_scale_mode(scale_mode)) return FP8Q_EINVAL;
    if (kind != FP8Q_NORM_LAYER && kind != FP8Q_NORM_RMS) return FP8Q_EINVAL;
    if (!(eps >= 0.0f)) return FP8Q_EINVAL;  // NaN too
    if (rows < 0 || cols < 0 || !ld_ok(ldx) || ldx < cols) return FP8Q_ESHAPE;
    if ((y != nullptr) && (!valid_dtype(y_dtype))) return FP8Q_EINVAL;
    if (y && (!ld_ok(ldy) || ldy < cols)) return FP8Q_ESHAPE;
    if (q && (!ld_ok(ldq) || !ld_ok(lds) || ldq < cols || lds < rows)) return FP8Q_ESHAPE;
    if (rows == 0 || cols == 0) return FP8Q_OK;
    if (!x || (!y && !q) || (q != nullptr) != (s != nullptr)) return FP8Q_EINVAL;
    if (!row_aligned(x, ldx, x_dtype) || (y && !row_aligned(y, ldy, y_dtype)) ||
        (q && (!aligned(q, 16) || ldq % 16 != 0 || !aligned(s, 4))) || !aligned(gamma, 16) || !aligned(beta, 16) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return FP8Q_EALIGN;
    if (cols > kMaxNormCols) return FP8Q_EUNSUPPORTED;
    return kLaunch;
}

// `need`: the bytes the partial sums of this shape take.  rows == 0 launches
// when there is a weight gradient to set to zero.
inline int layernorm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, int dtype, int64_t rows,
                              int64_t cols, const void* gamma, int w_dtype, const void* mean, const void* rstd,
                              int kind, const void* skip, int64_t ldskip, const void* dx, int64_t lddx,
                              const void* dgamma, const void* dbeta, int accumulate, int64_t need,
                              const void* workspace, int64_t workspace_bytes) {
    if (!valid_dtype(dtype) || !valid_dtype(w_dtype)) return FP8Q_EINVAL;
    if (kind != FP8Q_NORM_LAYER && kind != FP8Q_NORM_RMS) return FP8Q_EINVAL;
    if (rows < 0 || cols < 0 || !ld_ok(lddy) || !ld_ok(ldx) || !ld_ok(lddx) || lddy < cols || ldx < cols ||
        lddx < cols || workspace_bytes < 0)
        return FP8Q_ESHAPE;
    if (skip && (!ld_ok(ldskip) || ldskip < cols)) return FP8Q_ESHAPE;
    if (cols == 0) return FP8Q_OK;
    const bool weights = dgamma || dbeta;
    if (!aligned(dgamma, 4) || !aligned(dbeta, 4)) return FP8Q_EALIGN;
    if (rows == 0) return weights && !accumulate ? kLaunch : FP8Q_OK;
    if (!dy || !x || !rstd || !dx || (kind == FP8Q_NORM_LAYER && !mean)) return FP8Q_EINVAL;
    if (cols > kMaxNormCols) return FP8Q_EUNSUPPORTED;  // no workspace holds its sums: `need` is 0
    if (weights && !workspace) return FP8Q_EINVAL;
    if (weights && workspace_bytes < need) return FP8Q_ESHAPE;
    if (!row_aligned(dy, lddy, dtype) || !row_aligned(x, ldx, dtype) || !row_aligned(dx, lddx, dtype) ||
        (skip && !row_aligned(skip, ldskip, dtype)) || !aligned(gamma, 16) || !aligned(mean, 4) ||
        !aligned(rstd, 4) || (weights && !aligned(workspace, 256)))
        return FP8Q_EALIGN;
    return kLaunch;
}

inline int swiglu_quantize(const void* g, const void* u, int dtype, int64_t ldgu, int64_t rows, int64_t cols,
                           const void* qh, int64_t ldqh, const void* sh, int64_t ldsh, const void* qg,
                           const void* qu, int64_t ldq, const void* sg, const void* su, int64_t lds,
                           int scale_mode) {
    if (!valid_dtype(dtype) || !valid_scale_mode(scale_mode)) return FP8Q_EINVAL;
    const int kept = (qg ? 1 : 0) + (qu ? 1 : 0) + (sg ? 1 : 0) + (su ? 1 : 0);
    if (rows < 0 || cols < 0 || !ld_ok(ldgu) || !ld_ok(ldqh) || !ld_ok(ldsh) || ldgu < cols || ldqh < cols ||
        ldsh < rows)
        return FP8Q_ESHAPE;
    if (kept && (!ld_ok(ldq) || !ld_ok(lds) || ldq < cols || lds < rows)) return FP8Q_ESHAPE;
    if (rows == 0 || cols == 0) return FP8Q_OK;
    if (!g || !u || !qh || !sh || (kept != 0 && kept != 4)) return FP8Q_EINVAL;
    if (!row_aligned(g, ldgu, dtype) || !row_aligned(u, ldgu, dtype) || !aligned(qh, 16) || ldqh % 16 != 0 ||
        !aligned(sh, 4))
        return FP8Q_EALIGN;
    if (kept && (!aligned(qg, 16) || !aligned(qu, 16) || ldq % 16 != 0 || !aligned(sg, 4) || !aligned(su, 4)))
        return FP8Q_EALIGN;
    if (cdiv(rows, 4) > kMaxGridY * 65535 || cols > (int64_t(1) << 31)) return FP8Q_EUNSUPPORTED;
    return kLaunch;
}

// The checkpoint and the incoming gradient, shared by both backward forms.
inline int swiglu_backward_inputs(const void* qg, const void* qu, int64_t ldq, const void* sg, const void* su,
                                  int64_t lds, const void* dh, int dtype, int64_t lddh, int64_t rows, int64_t cols) {
    if (!valid_dtype(dtype)) return FP8Q_EINVAL;
    if (rows < 0 || cols < 0 || !ld_ok(ldq) || !ld_ok(lds) || !ld_ok(lddh) || ldq < cols || lds < rows ||
        lddh < cols)
        return FP8Q_ESHAPE;
    if (rows == 0 || cols == 0) return FP8Q_OK;
    if (!qg || !qu || !sg || !su || !dh) return FP8Q_EINVAL;
    if (!aligned(qg, 16) || !aligned(qu, 16) || ldq % 16 != 0 || !aligned(sg, 4) || !aligned(su, 4) ||
        !row_aligned(dh, lddh, dtype))
        return FP8Q_EALIGN;
    if (cdiv(rows, 4) > kMaxGridY * 65535 || cols > (int64_t(1) << 31)) return FP8Q_EUNSUPPORTED;
    return kLaunch;
}

inline int swiglu_backward(const void* qg, const void* qu, int64_t ldq, const void* sg, const void* su, int64_t lds,
                           const void* dh, int dtype, int64_t lddh, int64_t rows, int64_t cols, const void* dg,
                           const void* du, int64_t ldd) {
    if (!ld_ok(ldd) || ldd < cols) return FP8Q_ESHAPE;
    const int rc = swiglu_backward_inputs(qg, qu, ldq, sg, su, lds, dh, dtype, lddh, rows, cols);
    if (rc != kLaunch) return rc;
    if (!dg || !du) return FP8Q_EINVAL;
    if (!row_aligned(dg, ldd, dtype) || !row_aligned(du, ldd, dtype)) return FP8Q_EALIGN;
    return kLaunch;
}

inline int swiglu_backward_quantize(const void* qg, const void* qu, int64_t ldq, const void* sg, const void* su,
                                    int64_t lds, const void* dh, int dtype, int64_t lddh, int64_t rows, int64_t cols,
                                    const void* qdg, const void* qdu, int64_t ldqd, const void* sdg, const void* sdu,
                                    int64_t ldsd, const void* qdgt, const void* qdut, int64_t ldqt, const void* sdgt,
                                    const void* sdut, int64_t ldst, const void* qht, int64_t ldqht, const void* sht,
                                    int64_t ldsht, int scale_mode) {
    if (!valid_scale_mode(scale_mode)) return FP8Q_EINVAL;
    if (!ld_ok(ldqd) || !ld_ok(ldsd) || !ld_ok(ldqt) || !ld_ok(ldst) || !ld_ok(ldqht) || !ld_ok(ldsht) ||
        ldqd < cols || ldsd < rows || ldqt < rows || ldst < cols || ldqht < rows || ldsht < cols)
        return FP8Q_ESHAPE;
    const int rc = swiglu_backward_inputs(qg, qu, ldq, sg, su, lds, dh, dtype, lddh, rows, cols);
    if (rc != kLaunch) return rc;
    if (!qdg || !qdu || !sdg || !sdu || !qdgt || !qdut || !sdgt || !sdut || !qht || !sht) return FP8Q_EINVAL;
    if (!aligned(qdg, 16) || !aligned(qdu, 16) || ldqd % 16 != 0 || !aligned(qdgt, 16) || !aligned(qdut, 16) ||
        ldqt % 16 != 0 || !aligned(qht, 16) || ldqht % 16 != 0 || !aligned(sdg, 4) || !aligned(sdu, 4) ||
        !aligned(sdgt, 4) || !aligned(sdut, 4) || !aligned(sht, 4))
        return FP8Q_EALIGN;
    if (cdiv(rows, 128) > kMaxGridY || cols >= (int64_t(1) << 30)) return FP8Q_EUNSUPPORTED;  // 2^32 threads along x
    return kLaunch;
}

// Sizes of the mixture-of-experts layer: FP8Q_ESHAPE or FP8Q_EUNSUPPORTED
// where there is no such layer, kLaunch otherwise.
inline int moe_sizes(int64_t tokens, int64_t hidden, int64_t inner, int experts, int top_k) {
    if (tokens < 0 || hidden <= 0 || inner <= 0 || hidden % 128 != 0 || inner % 128 != 0 || experts < 1 || top_k < 1)
        return FP8Q_ESHAPE;
    if (tokens > FP8Q_MOE_MAX_TOKENS || experts > kMaxGroups || top_k > FP8Q_MOE_MAX_TOP_K ||
        hidden > kMaxOperandLd || inner > kMaxOperandLd)
        return FP8Q_EUNSUPPORTED;
    return kLaunch;
}

inline int moe_weight(const void* w, int64_t ldw, int64_t stride, const void* s, int64_t lds, int64_t s_stride,
                      int64_t rows, int64_t cols) {
    if (!ld_ok(ldw) || !ld_ok(lds) || ldw < cols || lds < cols / 128 || stride < 0 || stride > kMaxGroupStride ||
        s_stride < 0 || s_stride > kMaxGroupStride)
        return FP8Q_ESHAPE;
    if (ldw > kMaxOperandLd) return FP8Q_EUNSUPPORTED;
    if (stride < (rows - 1) * ldw + cols || s_stride < (rows / 128 - 1) * lds + cols / 128) return FP8Q_ESHAPE;
    if (!w || !s) return FP8Q_EINVAL;
    if (!aligned(w, 16) || ldw % 16 != 0 || stride % 16 != 0 || !aligned(s, 4)) return FP8Q_EALIGN;
    return kLaunch;
}

inline int moe_decode(const void* x, int64_t ldx, int64_t tokens, int64_t hidden, const void* logits, int64_t ldl,
                      int experts, int top_k, int64_t inner, const void* w_gu, int64_t ldw_gu, int64_t w_gu_stride,
                      const void* s_gu, int64_t lds_gu, int64_t s_gu_stride, const void* w_down, int64_t ldw_down,
                      int64_t w_down_stride, const void* s_down, int64_t lds_down, int64_t s_down_stride,
                      const void* y, int y_dtype, int64_t ldy, int64_t need, const void* workspace,
                      int64_t workspace_bytes) {
    if (!valid_dtype(y_dtype)) return FP8Q_EINVAL;
    int rc = moe_sizes(tokens, hidden, inner, experts, top_k);
    if (rc != kLaunch) return rc;
    if (!ld_ok(ldx) || !ld_ok(ldl) || !ld_ok(ldy) || ldx < hidden || ldl < experts || ldy < hidden ||
        workspace_bytes < 0)
        return FP8Q_ESHAPE;
    if (tokens == 0) return FP8Q_OK;
    rc = moe_weight(w_gu, ldw_gu, w_gu_stride, s_gu, lds_gu, s_gu_stride, 2 * inner, hidden);
    if (rc != kLaunch) return rc;
    rc = moe_weight(w_down, ldw_down, w_down_stride, s_down, lds_down, s_down_stride, hidden, inner);
    if (rc != kLaunch) return rc;
    if (!x || !logits || !y || !workspace) return FP8Q_EINVAL;
    if (workspace_bytes < need) return FP8Q_ESHAPE;
    if (!row_aligned(x, ldx, FP8Q_BF16) || !row_aligned(y, ldy, y_dtype) || !aligned(logits, 4) ||
        !aligned(workspace, 256))
        return FP8Q_EALIGN;
    return kLaunch;
}

// ---- weight gradients of groups of rows, AdamW

// Columns of the padded layout (groups.hpp): chunks of all groups at most.
inline int64_t padded_rows(int64_t rows, int64_t G) { return (rows + 127 * (G < rows ? G : rows)) / 128 * 128; }

inline int groups(int64_t rows, int64_t cols, const void* group_offsets, int G, const void* qt, int64_t ldqt,
                  const void* st, int64_t ldst, int scale_mode) {
    if (!valid_scale_mode(scale_mode)) return FP8Q_EINVAL;
    if (G < 1 || G > kMaxGroups || rows < 0 || cols < 0 || !ld_ok(ldqt) || !ld_ok(ldst)) return FP8Q_ESHAPE;
    if (rows > INT32_MAX) return FP8Q_EUNSUPPORTED;
    if (ldqt < padded_rows(rows, G) || ldst < cols) return FP8Q_ESHAPE;
    if (rows == 0 || cols == 0) return FP8Q_OK;
    if (!group_offsets || !qt || !st) return FP8Q_EINVAL;
    if (!aligned(group_offsets, 4) || !aligned(qt, 16) || ldqt % 16 != 0 || !aligned(st, 4)) return FP8Q_EALIGN;
    if (padded_rows(rows, G) / 128 > kMaxGridY) return FP8Q_EUNSUPPORTED;
    return kLaunch;
}

inline int grouped_quantize_act(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx,
                                const void* group_offsets, int G, const void* qt, int64_t ldqt, const void* st,
                                int64_t ldst, int scale_mode) {
    if (!valid_dtype(x_dtype)) return FP8Q_EINVAL;
    if (!ld_ok(ldx) || ldx < cols) return FP8Q_ESHAPE;
    const int rc = groups(rows, cols, group_offsets, G, qt, ldqt, st, ldst, scale_mode);
    if (rc != kLaunch) return rc;
    if (!x) return FP8Q_EINVAL;
    return row_aligned(x, ldx, x_dtype) ? kLaunch : FP8Q_EALIGN;
}

inline int grouped_requant(const void* q, int64_t rows, int64_t cols, int64_t ldq, const void* s, int64_t lds,
                           const void* group_offsets, int G, const void* qt, int64_t ldqt, const void* st,
                           int64_t ldst, int scale_mode) {
    if (!ld_ok(ldq) || !ld_ok(lds) || ldq < cols || lds < rows) return FP8Q_ESHAPE;
    const int rc = groups(rows, cols, group_offsets, G, qt, ldqt, st, ldst, scale_mode);
    if (rc != kLaunch) return rc;
    if (!q || !s) return FP8Q_EINVAL;
    return aligned(q, 16) && ldq % 16 == 0 && aligned(s, 4) ? kLaunch : FP8Q_EALIGN;
}

constexpr int64_t kMaxWgradChannels = int64_t(1) << 30;
constexpr int64_t kMaxWgradTiles = int64_t(1) << 30;

// Sizes of the weight gradients: FP8Q_ESHAPE or FP8Q_EUNSUPPORTED where there
// are none.
inline int wgrad_sizes(int64_t rows, int G, int64_t N, int64_t K) {
    if (G < 1 || G > kMaxGroups || rows < 0 || N < 0 || K < 0) return FP8Q_ESHAPE;
    if (rows > INT32_MAX || padded_rows(rows, G) > kMaxOperandLd) return FP8Q_EUNSUPPORTED;
    // channels and 128x128 tiles of all groups are counted in 32 bits
    if (N > kMaxWgradChannels || K > kMaxWgradChannels || cdiv(N, 128) * cdiv(K, 128) > kMaxWgradTiles / G)
        return FP8Q_EUNSUPPORTED;
    return kLaunch;
}

// `need`: the bytes that the split of this shape takes.  rows == 0 launches:
// the gradients are set to zero.
inline int grouped_wgrad(const void* a, int64_t lda, const void* sa, int64_t ldsa, const void* b, int64_t ldb,
                         const void* sb, int64_t ldsb, const void* group_offsets, int G, int64_t rows, int64_t N,
                         int64_t K, const void* dw, int dw_dtype, int64_t lddw, int64_t dw_group_stride,
                         int accumulate, unsigned flags, int64_t need, const void* workspace,
                         int64_t workspace_bytes) {
    if (!valid_dtype(dw_dtype) || (flags & ~kKnownGemmFlags) != 0u) return FP8Q_EINVAL;
    if (accumulate && dw_dtype != FP8Q_F32) return FP8Q_EUNSUPPORTED;
    if (!ld_ok(lda) || !ld_ok(ldb) || !ld_ok(ldsa) || !ld_ok(ldsb) || !ld_ok(lddw) || dw_group_stride < 0 ||
        dw_group_stride > kMaxGroupStride || workspace_bytes < 0)
        return FP8Q_ESHAPE;
    const int rc = wgrad_sizes(rows, G, N, K);
    if (rc != kLaunch) return rc;
    if (lda < padded_rows(rows, G) || ldb < padded_rows(rows, G) || ldsa < N || ldsb < K || lddw < K)
        return FP8Q_ESHAPE;
    if (lda > kMaxOperandLd || ldb > kMaxOperandLd) return FP8Q_EUNSUPPORTED;
    if (N == 0 || K == 0) return FP8Q_OK;
    if (G > 1 && dw_group_stride < (N - 1) * lddw + K) return FP8Q_ESHAPE;
    if (!dw) return FP8Q_EINVAL;
    if (!aligned(dw, (uintptr_t)elem_bytes(dw_dtype))) return FP8Q_EALIGN;
    if (rows == 0) return accumulate ? FP8Q_OK : kLaunch;
    if (!a || !sa || !b || !sb || !group_offsets) return FP8Q_EINVAL;
    if (!aligned(a, 16) || lda % 16 != 0 || !aligned(b, 16) || ldb % 16 != 0 || !aligned(sa, 4) || !aligned(sb, 4) ||
        !aligned(group_offsets, 4))
        return FP8Q_EALIGN;
    return splitk_workspace(need, workspace, workspace_bytes);
}

constexpr int64_t kMaxAdamwElements = int64_t(1) << 33;
constexpr int64_t kMaxAdamwBlocks = int64_t(1) << 22;

inline int adamw_tensor(const fp8q_adamw_tensor& t, int bits) {
    if (t.n < 0) return FP8Q_ESHAPE;
    if (t.n == 0) return FP8Q_OK;
    if (!t.p || !t.g || !t.m || !t.v || (bits == 8 && (!t.sm || !t.sv))) return FP8Q_EINVAL;
    if (!t.q != !t.s || !t.qt != !t.st || (t.qt && !t.q)) return FP8Q_EINVAL;
    if (!aligned(t.p, 16) || !aligned(t.g, 16) || !aligned(t.m, 16) || !aligned(t.v, 16) ||
        (bits == 8 && (!aligned(t.sm, 4) || !aligned(t.sv, 4))))
        return FP8Q_EALIGN;
    if (t.n > kMaxAdamwElements) return FP8Q_EUNSUPPORTED;
    if (!t.q) return kLaunch;
    if (t.N < 1 || t.K < 1 || t.K % 128 != 0 || t.N > t.n || t.K > t.n || t.n % t.N != 0 || t.n / t.N % t.K != 0)
        return FP8Q_ESHAPE;
    if (!aligned(t.q, 16) || !aligned(t.s, 4) || !aligned(t.qt, 16) || !aligned(t.st, 4)) return FP8Q_EALIGN;
    if (t.n / (t.N * t.K) * cdiv(t.N, 128) * (t.K / 128) > kMaxAdamwBlocks) return FP8Q_EUNSUPPORTED;
    return kLaunch;
}

// The first tensor that is refused gives the status; nothing is launched then.
inline int adamw(const fp8q_adamw_tensor* tensors, int count, int g_dtype, int bits, const fp8q_adamw_config* c,
                 int scale_mode) {
    if (!valid_dtype(g_dtype) || (bits != 8 && bits != 32) || !valid_scale_mode(scale_mode) || !c) return FP8Q_EINVAL;
    if (count < 0) return FP8Q_ESHAPE;
    if (!(c->beta1 >= 0.0 && c->beta1 < 1.0 && c->beta2 >= 0.0 && c->beta2 < 1.0 && c->eps >= 0.0)) return FP8Q_EINVAL;
    if (!(c->weight_decay >= 0.0) || (!c->lr_dev && !(c->lr >= 0.0)) || (!c->step_dev && c->step < 1)) return FP8Q_EINVAL;
    if (count == 0) return FP8Q_OK;
    if (!tensors) return FP8Q_EINVAL;
    if (!aligned(c->lr_dev, 4) || !aligned(c->step_dev, 8) || !aligned(c->grad_scale, 4)) return FP8Q_EALIGN;
    int all = FP8Q_OK;
    for (int i = 0; i < count; ++i) {
        const int rc = adamw_tensor(tensors[i], bits);
        if (rc == kLaunch) all = kLaunch;
        else if (rc != FP8Q_OK) return rc;
    }
    return all;
}

}  // namespace check
}  // namespace fp8q
