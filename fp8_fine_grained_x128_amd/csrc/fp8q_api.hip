// fp8q_api.hip -- C ABI (include/fp8q.h): host-side validation
// (validate.hpp), then the kernel launches on the caller's stream.  No
// allocation, no synchronization; the only state is the per-device address
// of the split-K scratch array below, looked up once per device.
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "../../include/fp8q.h"
#include "launch.hpp"
#include "validate.hpp"

// Device scratch of fp8q_gemm_splitk_noalloc: the split-K partials live here
// instead of in a caller workspace.  Each device that runs the library holds
// its own copy until the process ends.  Host code never passes `scratch`
// itself to a kernel (on the host it is only a stand-in for the symbol); it
// uses the device address that hipGetSymbolAddress returns for the current
// device (scratch_ptr below).
static __device__ __align__(256) uint8_t scratch[FP8Q_SPLITK_SCRATCH_BYTES];

namespace {

using fp8q::check::kLaunch;

inline int status_of(hipError_t e) { return e == hipSuccess ? FP8Q_OK : FP8Q_EHIP; }

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mutex;
void* g_scratch_ptr[kMaxDevices] = {};

// This device's address of `scratch`, looked up once per device (with that
// device current) on the first call; nullptr if the lookup fails.
void* scratch_ptr() {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lock(g_scratch_mutex);
    if (!g_scratch_ptr[dev]) {
        void* p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess) {
            (void)hipGetLastError();  // do not leave the error for the next call to report
            return nullptr;
        }
        g_scratch_ptr[dev] = p;
    }
    return g_scratch_ptr[dev];
}

inline int datapath_of(unsigned flags) {
    const bool fp8 = (flags & FP8Q_GEMM_MMA_FP8) != 0u;
    if (flags & FP8Q_GEMM_POW2_SCALES) return fp8 ? fp8q::kMmaFp8Scaled : fp8q::kMmaBf16Fold;
    return fp8 ? fp8q::kMmaFp8 : fp8q::kMmaF16;
}

int quantize_act_impl(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, int tile, uint8_t* q,
                      int64_t ldq, float* s, int64_t lds, int scale_mode, void* stream) {
    const int rc = fp8q::check::quantize_act(x, x_dtype, rows, cols, ldx, tile, q, ldq, s, lds, scale_mode);
    if (rc != kLaunch) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int pow2 = scale_mode == FP8Q_SCALE_POW2;
    if (tile == FP8Q_TILE_1x128)
        return status_of(fp8q::launch_quantize_1x128(x, x_dtype, rows, cols, ldx, q, ldq, s, lds, pow2, st));
    const int kind = x_dtype == FP8Q_BF16 ? 1 : 0;
    return status_of(fp8q::launch_quantize_128x1(x, kind, rows, cols, ldx, nullptr, 0, q, ldq, s, lds, pow2, st));
}

int quantize_weight_impl(const void* w, int w_dtype, int64_t N, int64_t K, int64_t ldw, uint8_t* q, int64_t ldq,
                         float* s, int64_t lds, int scale_mode, void* stream) {
    const int rc = fp8q::check::quantize_weight(w, w_dtype, N, K, ldw, q, ldq, s, lds, scale_mode);
    if (rc != kLaunch) return rc;
    return status_of(fp8q::launch_quantize_128x128(w, w_dtype, N, K, ldw, q, ldq, s, lds,
                                                   scale_mode == FP8Q_SCALE_POW2, static_cast<hipStream_t>(stream)));
}

int requant_impl(const uint8_t* q, int64_t rows, int64_t cols, int64_t ldq, const float* s, int64_t lds,
                 uint8_t* qt, int64_t ldqt, float* st, int64_t ldst, int scale_mode, void* stream) {
    const int rc = fp8q::check::requant(q, rows, cols, ldq, s, lds, qt, ldqt, st, ldst, scale_mode);
    if (rc != kLaunch) return rc;
    return status_of(fp8q::launch_quantize_128x1(q, 2, rows, cols, ldq, s, lds, qt, ldqt, st, ldst,
                                                 scale_mode == FP8Q_SCALE_POW2, static_cast<hipStream_t>(stream)));
}

// The plain GEMM after validation; `workspace` holds the split-K partials
// when the shape splits (nullptr: no split).
int gemm_launch(const uint8_t* a, int64_t lda, const float* sa, int64_t ldsa, const uint8_t* b, int64_t ldb,
                const float* sb, int64_t ldsb, int bscale, int64_t M, int64_t N, int64_t K, void* c, int c_dtype,
                int64_t ldc, int accumulate, unsigned flags, void* workspace, int64_t workspace_bytes,
                void* stream) {
    fp8q::GemmArgs g{};
    g.a = a; g.lda = lda; g.sa = sa; g.ldsa = ldsa;
    g.b = b; g.ldb = ldb; g.b_group_stride = 0;
    g.sb = sb; g.ldsb = ldsb; g.sb_group_stride = 0;
    g.offsets = nullptr; g.groups = 1;
    g.M = M; g.N = N; g.K = K; g.c = c; g.ldc = ldc;
    g.bscale = bscale; g.c_dtype = c_dtype; g.accumulate = accumulate ? 1 : 0;
    g.mma = datapath_of(flags);
    g.workspace = workspace;
    g.workspace_bytes = workspace_bytes;
    return status_of(fp8q::launch_gemm(g, static_cast<hipStream_t>(stream)));
}

int grouped_impl(const uint8_t* a, int64_t lda, const float* sa, int64_t ldsa, const uint8_t* b, int64_t ldb,
                 int64_t b_group_stride, const float* sb, int64_t ldsb, int64_t sb_group_stride,
                 const int32_t* group_offsets, int G, int64_t M_total, int64_t N, int64_t K, void* c,
                 int c_dtype, int64_t ldc, unsigned flags, void* stream) {
    const int rc = fp8q::check::grouped(a, lda, sa, ldsa, b, ldb, b_group_stride, sb, ldsb, sb_group_stride,
                                        group_offsets, G, M_total, N, K, c, c_dtype, ldc, flags);
    if (rc != kLaunch) return rc;
    fp8q::GemmArgs g{};
    g.a = a; g.lda = lda; g.sa = sa; g.ldsa = ldsa;
    g.b = b; g.ldb = ldb; g.b_group_stride = b_group_stride;
    g.sb = sb; g.ldsb = ldsb; g.sb_group_stride = sb_group_stride;
    g.offsets = group_offsets; g.groups = G;
    g.M = M_total; g.N = N; g.K = K; g.c = c; g.ldc = ldc;
    g.bscale = FP8Q_BSCALE_BLOCK128; g.c_dtype = c_dtype; g.accumulate = 0;
    g.mma = datapath_of(flags);
    return status_of(fp8q::launch_grouped_gemm(g, static_cast<hipStream_t>(stream)));
}

// The checkpoint and incoming gradient of a SwiGLU backward call.
fp8q::SwigluBackwardArgs swiglu_inputs(const uint8_t* qg, const uint8_t* qu, int64_t ldq, const float* sg,
                                       const float* su, int64_t lds, const void* dh, int dtype, int64_t lddh,
                                       int64_t rows, int64_t cols) {
    fp8q::SwigluBackwardArgs a{};
    a.qg = qg; a.qu = qu; a.ldq = ldq; a.sg = sg; a.su = su; a.lds = lds;
    a.dh = dh; a.dtype = dtype; a.lddh = lddh; a.rows = rows; a.cols = cols;
    return a;
}

}  // namespace

extern "C" {

const char* fp8q_strerror(int status) {
    switch (status) {
        case FP8Q_OK: return "ok";
        case FP8Q_EINVAL: return "invalid argument (null pointer or unknown enum value)";
        case FP8Q_ESHAPE: return "invalid shape or leading dimension";
        case FP8Q_EALIGN: return "misaligned pointer or leading dimension";
        case FP8Q_EUNSUPPORTED: return "unsupported request";
        case FP8Q_EHIP: return "HIP launch error";
        default: return "unknown status";
    }
}

int fp8q_version(void) { return 300; }

int fp8q_quantize_act(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, int tile,
                      uint8_t* q, int64_t ldq, float* s, int64_t lds, void* stream) {
    return quantize_act_impl(x, x_dtype, rows, cols, ldx, tile, q, ldq, s, lds, FP8Q_SCALE_FP32, stream);
}

int fp8q_quantize_act_ex(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, int tile,
                         uint8_t* q, int64_t ldq, float* s, int64_t lds, int scale_mode, void* stream) {
    return quantize_act_impl(x, x_dtype, rows, cols, ldx, tile, q, ldq, s, lds, scale_mode, stream);
}

int fp8q_gather_quantize_act(const void* x, int x_dtype, int64_t rows_in, int64_t cols, int64_t ldx,
                             const int32_t* row_index, int64_t rows_out, uint8_t* q, int64_t ldq, float* s,
                             int64_t lds, int scale_mode, void* stream) {
    const int rc = fp8q::check::gather_quantize_act(x, x_dtype, rows_in, cols, ldx, row_index, rows_out, q, ldq,
                                                    s, lds, scale_mode);
    if (rc != kLaunch) return rc;
    return status_of(fp8q::launch_gather_quantize_1x128(x, x_dtype, rows_in, cols, ldx, row_index, rows_out, q,
                                                        ldq, s, lds, scale_mode == FP8Q_SCALE_POW2,
                                                        static_cast<hipStream_t>(stream)));
}

int fp8q_quantize_weight(const void* w, int w_dtype, int64_t N, int64_t K, int64_t ldw, uint8_t* q,
                         int64_t ldq, float* s, int64_t lds, void* stream) {
    return quantize_weight_impl(w, w_dtype, N, K, ldw, q, ldq, s, lds, FP8Q_SCALE_FP32, stream);
}

int fp8q_quantize_weight_ex(const void* w, int w_dtype, int64_t N, int64_t K, int64_t ldw, uint8_t* q,
                            int64_t ldq, float* s, int64_t lds, int scale_mode, void* stream) {
    return quantize_weight_impl(w, w_dtype, N, K, ldw, q, ldq, s, lds, scale_mode, stream);
}

int fp8q_requant_transpose(const uint8_t* q, int64_t rows, int64_t cols, int64_t ldq, const float* s,
                           int64_t lds, uint8_t* qt, int64_t ldqt, float* st, int64_t ldst, void* stream) {
    return requant_impl(q, rows, cols, ldq, s, lds, qt, ldqt, st, ldst, FP8Q_SCALE_FP32, stream);
}

int fp8q_requant_transpose_ex(const uint8_t* q, int64_t rows, int64_t cols, int64_t ldq, const float* s,
                              int64_t lds, uint8_t* qt, int64_t ldqt, float* st, int64_t ldst, int scale_mode,
                              void* stream) {
    return requant_impl(q, rows, cols, ldq, s, lds, qt, ldqt, st, ldst, scale_mode, stream);
}

int fp8q_transpose_weight(const uint8_t* q, int64_t N, int64_t K, int64_t ldq, const float* s, int64_t lds,
                          uint8_t* qt, int64_t ldqt, float* st, int64_t ldst, void* stream) {
    const int rc = fp8q::check::transpose_weight(q, N, K, ldq, s, lds, qt, ldqt, st, ldst);
    if (rc != kLaunch) return rc;
    return status_of(fp8q::launch_transpose_weight(q, N, K, ldq, s, lds, qt, ldqt, st, ldst,
                                                   static_cast<hipStream_t>(stream)));
}

int fp8q_gemm(const uint8_t* a, int64_t lda, const float* sa, int64_t ldsa, const uint8_t* b, int64_t ldb,
              const float* sb, int64_t ldsb, int bscale, int64_t M, int64_t N, int64_t K, void* c,
              int c_dtype, int64_t ldc, int accumulate, void* stream) {
    const int rc = fp8q::check::gemm(a, lda, sa, ldsa, b, ldb, sb, ldsb, bscale, M, N, K, c, c_dtype, ldc,
                                     accumulate, 0u);
    if (rc != kLaunch) return rc;
    return gemm_launch(a, lda, sa, ldsa, b, ldb, sb, ldsb, bscale, M, N, K, c, c_dtype, ldc, accumulate, 0u,
                       nullptr, 0, stream);
}

int fp8q_gemm_ex(const uint8_t* a, int64_t lda, const float* sa, int64_t ldsa, const uint8_t* b,
                 int64_t ldb, const float* sb, int64_t ldsb, int bscale, int64_t M, int64_t N, int64_t K,
                 void* c, int c_dtype, int64_t ldc, int accumulate, unsigned flags, void* stream) {
    const int rc = fp8q::check::gemm(a, lda, sa, ldsa, b, ldb, sb, ldsb, bscale, M, N, K, c, c_dtype, ldc,
                                     accumulate, flags);
    if (rc != kLaunch) return rc;
    return gemm_launch(a, lda, sa, ldsa, b, ldb, sb, ldsb, bscale, M, N, K, c, c_dtype, ldc, accumulate, flags,
                       nullptr, 0, stream);
}

int64_t fp8q_gemm_splitk_workspace(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0 || K % 128 != 0) return 0;
    return fp8q::plan_splitk(M, N, K).bytes;
}

int fp8q_gemm_splitk(const uint8_t* a, int64_t lda, const float* sa, int64_t ldsa, const uint8_t* b,
                     int64_t ldb, const float* sb, int64_t ldsb, int bscale, int64_t M, int64_t N, int64_t K,
                     void* c, int c_dtype, int64_t ldc, int accumulate, unsigned flags, void* workspace,
                     int64_t workspace_bytes, void* stream) {
    const int64_t need = fp8q_gemm_splitk_workspace(M, N, K);
    int rc = fp8q::check::splitk_workspace(need, workspace, workspace_bytes);
    if (rc != kLaunch) return rc;
    rc = fp8q::check::gemm(a, lda, sa, ldsa, b, ldb, sb, ldsb, bscale, M, N, K, c, c_dtype, ldc, accumulate,
                           flags);
    if (rc != kLaunch) return rc;
    return gemm_launch(a, lda, sa, ldsa, b, ldb, sb, ldsb, bscale, M, N, K, c, c_dtype, ldc, accumulate, flags,
                       need > 0 ? workspace : nullptr, need, stream);
}

int fp8q_gemm_splitk_noalloc(const uint8_t* a, int64_t lda, const float* sa, int64_t ldsa, const uint8_t* b,
                             int64_t ldb, const float* sb, int64_t ldsb, int bscale, int64_t M, int64_t N,
                             int64_t K, void* c, int c_dtype, int64_t ldc, int accumulate, unsigned flags,
                             void* stream) {
    const int rc = fp8q::check::gemm(a, lda, sa, ldsa, b, ldb, sb, ldsb, bscale, M, N, K, c, c_dtype, ldc,
                                     accumulate, flags);
    if (rc != kLaunch) return rc;
    const int64_t need = fp8q_gemm_splitk_workspace(M, N, K);
    if (need > (int64_t)FP8Q_SPLITK_SCRATCH_BYTES) return FP8Q_EUNSUPPORTED;
    void* ws = nullptr;
    if (need > 0) {
        ws = scratch_ptr();
        if (!ws) return FP8Q_EHIP;
    }
    return gemm_launch(a, lda, sa, ldsa, b, ldb, sb, ldsb, bscale, M, N, K, c, c_dtype, ldc, accumulate, flags, ws,
                       need, stream);
}

int fp8q_clock_probe(uint64_t* out, int64_t ticks, void* stream) {
    const int rc = fp8q::check::clock_probe(out, ticks);
    if (rc != kLaunch) return rc;
    return status_of(fp8q::launch_clock_probe(out, ticks, static_cast<hipStream_t>(stream)));
}

int fp8q_grouped_gemm(const uint8_t* a, int64_t lda, const float* sa, int64_t ldsa, const uint8_t* b,
                      int64_t ldb, int64_t b_group_stride, const float* sb, int64_t ldsb,
                      int64_t sb_group_stride, const int32_t* group_offsets, int G, int64_t M_total,
                      int64_t N, int64_t K, void* c, int c_dtype, int64_t ldc, void* stream) {
    return grouped_impl(a, lda, sa, ldsa, b, ldb, b_group_stride, sb, ldsb, sb_group_stride, group_offsets, G,
                        M_total, N, K, c, c_dtype, ldc, 0u, stream);
}

int fp8q_grouped_gemm_ex(const uint8_t* a, int64_t lda, const float* sa, int64_t ldsa, const uint8_t* b,
                         int64_t ldb, int64_t b_group_stride, const float* sb, int64_t ldsb,
                         int64_t sb_group_stride, const int32_t* group_offsets, int G, int64_t M_total,
                         int64_t N, int64_t K, void* c, int c_dtype, int64_t ldc, unsigned flags,
                         void* stream) {
    return grouped_impl(a, lda, sa, ldsa, b, ldb, b_group_stride, sb, ldsb, sb_group_stride, group_offsets, G,
                        M_total, N, K, c, c_dtype, ldc, flags, stream);
}

int fp8q_layernorm(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, const void* gamma,
                   const void* beta, int w_dtype, float eps, int kind, void* y, int y_dtype, int64_t ldy, uint8_t* q,
                   int64_t ldq, float* s, int64_t lds, int scale_mode, float* mean, float* rstd, void* stream) {
    const int rc = fp8q::check::layernorm(x, x_dtype, rows, cols, ldx, gamma, beta, w_dtype, eps, kind, y, y_dtype,
                                          ldy, q, ldq, s, lds, scale_mode, mean, rstd);
    if (rc != kLaunch) return rc;
    fp8q::LayernormArgs a{};
    a.x = x; a.x_dtype = x_dtype; a.rows = rows; a.cols = cols; a.ldx = ldx;
    a.gamma = gamma; a.beta = beta; a.w_dtype = w_dtype; a.eps = eps;
    a.layer = kind == FP8Q_NORM_LAYER;
    a.y = y; a.y_dtype = y_dtype; a.ldy = ldy;
    a.q = q; a.ldq = ldq; a.s = s; a.lds = lds; a.pow2 = scale_mode == FP8Q_SCALE_POW2;
    a.mean = mean; a.rstd = rstd;
    return status_of(fp8q::launch_layernorm(a, static_cast<hipStream_t>(stream)));
}

int64_t fp8q_layernorm_backward_workspace(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0 || cols > FP8Q_NORM_MAX_COLS) return 0;
    return fp8q::layernorm_backward_bytes(rows, cols);
}

int fp8q_layernorm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, int dtype, int64_t rows,
                            int64_t cols, const void* gamma, int w_dtype, const float* mean, const float* rstd,
                            int kind, const void* skip, int64_t ldskip, void* dx, int64_t lddx, float* dgamma,
                            float* dbeta, int accumulate, void* workspace, int64_t workspace_bytes, void* stream) {
    const int64_t need = fp8q_layernorm_backward_workspace(rows, cols);
    const int rc = fp8q::check::layernorm_backward(dy, lddy, x, ldx, dtype, rows, cols, gamma, w_dtype, mean, rstd,
                                                   kind, skip, ldskip, dx, lddx, dgamma, dbeta, accumulate, need,
                                                   workspace, workspace_bytes);
    if (rc != kLaunch) return rc;
    fp8q::LayernormBackwardArgs a{};
    a.dy = dy; a.lddy = lddy; a.x = x; a.ldx = ldx; a.dtype = dtype; a.rows = rows; a.cols = cols;
    a.gamma = gamma; a.w_dtype = w_dtype; a.mean = mean; a.rstd = rstd;
    a.layer = kind == FP8Q_NORM_LAYER;
    a.skip = skip; a.ldskip = ldskip; a.dx = dx; a.lddx = lddx;
    a.dgamma = dgamma; a.dbeta = dbeta; a.accumulate = accumulate ? 1 : 0;
    return status_of(fp8q::launch_layernorm_backward(a, workspace, static_cast<hipStream_t>(stream)));
}

int fp8q_swiglu_quantize(const void* g, const void* u, int dtype, int64_t ldgu, int64_t rows, int64_t cols,
                         uint8_t* qh, int64_t ldqh, float* sh, int64_t ldsh, uint8_t* qg, uint8_t* qu, int64_t ldq,
                         float* sg, float* su, int64_t lds, int scale_mode, void* stream) {
    const int rc = fp8q::check::swiglu_quantize(g, u, dtype, ldgu, rows, cols, qh, ldqh, sh, ldsh, qg, qu, ldq, sg,
                                                su, lds, scale_mode);
    if (rc != kLaunch) return rc;
    fp8q::SwigluArgs a{};
    a.g = g; a.u = u; a.dtype = dtype; a.ldgu = ldgu; a.rows = rows; a.cols = cols;
    a.qh = qh; a.ldqh = ldqh; a.sh = sh; a.ldsh = ldsh;
    a.qg = qg; a.qu = qu; a.ldq = ldq; a.sg = sg; a.su = su; a.lds = lds;
    a.pow2 = scale_mode == FP8Q_SCALE_POW2;
    return status_of(fp8q::launch_swiglu_quantize(a, static_cast<hipStream_t>(stream)));
}

int fp8q_swiglu_backward(const uint8_t* qg, const uint8_t* qu, int64_t ldq, const float* sg, const float* su,
                         int64_t lds, const void* dh, int dtype, int64_t lddh, int64_t rows, int64_t cols, void* dg,
                         void* du, int64_t ldd, void* stream) {
    const int rc = fp8q::check::swiglu_backward(qg, qu, ldq, sg, su, lds, dh, dtype, lddh, rows, cols, dg, du, ldd);
    if (rc != kLaunch) return rc;
    fp8q::SwigluBackwardArgs a = swiglu_inputs(qg, qu, ldq, sg, su, lds, dh, dtype, lddh, rows, cols);
    a.dg = dg; a.du = du; a.ldd = ldd;
    return status_of(fp8q::launch_swiglu_backward(a, static_cast<hipStream_t>(stream)));
}

int fp8q_swiglu_backward_quantize(const uint8_t* qg, const uint8_t* qu, int64_t ldq, const float* sg,
                                  const float* su, int64_t lds, const void* dh, int dtype, int64_t lddh, int64_t rows,
                                  int64_t cols, uint8_t* qdg, uint8_t* qdu, int64_t ldqd, float* sdg, float* sdu,
                                  int64_t ldsd, uint8_t* qdgt, uint8_t* qdut, int64_t ldqt, float* sdgt, float* sdut,
                                  int64_t ldst, uint8_t* qht, int64_t ldqht, float* sht, int64_t ldsht,
                                  int scale_mode, void* stream) {
    const int rc = fp8q::check::swiglu_backward_quantize(qg, qu, ldq, sg, su, lds, dh, dtype, lddh, rows, cols, qdg,
                                                         qdu, ldqd, sdg, sdu, ldsd, qdgt, qdut, ldqt, sdgt, sdut,
                                                         ldst, qht, ldqht, sht, ldsht, scale_mode);
    if (rc != kLaunch) return rc;
    fp8q::SwigluBackwardArgs a = swiglu_inputs(qg, qu, ldq, sg, su, lds, dh, dtype, lddh, rows, cols);
    a.qdg = qdg; a.qdu = qdu; a.ldqd = ldqd; a.sdg = sdg; a.sdu = sdu; a.ldsd = ldsd;
    a.qdgt = qdgt; a.qdut = qdut; a.ldqt = ldqt; a.sdgt = sdgt; a.sdut = sdut; a.ldst = ldst;
    a.qht = qht; a.ldqht = ldqht; a.sht = sht; a.ldsht = ldsht;
    a.pow2 = scale_mode == FP8Q_SCALE_POW2;
    return status_of(fp8q::launch_swiglu_backward_quantize(a, static_cast<hipStream_t>(stream)));
}

int64_t fp8q_moe_decode_workspace(int64_t tokens, int64_t hidden, int64_t inner, int experts, int top_k) {
    if (tokens == 0 || fp8q::check::moe_sizes(tokens, hidden, inner, experts, top_k) != kLaunch) return 0;
    return fp8q::moe_decode_bytes(tokens, hidden, inner, experts, std::min(top_k, experts));
}

int fp8q_moe_decode(const void* x, int64_t ldx, int64_t tokens, int64_t hidden, const float* logits, int64_t ldl,
                    int experts, int top_k, int renormalize, int64_t inner, const uint8_t* w_gu, int64_t ldw_gu,
                    int64_t w_gu_stride, const float* s_gu, int64_t lds_gu, int64_t s_gu_stride,
                    const uint8_t* w_down, int64_t ldw_down, int64_t w_down_stride, const float* s_down,
                    int64_t lds_down, int64_t s_down_stride, void* y, int y_dtype, int64_t ldy, void* workspace,
                    int64_t workspace_bytes, void* stream) {
    const int64_t need = fp8q_moe_decode_workspace(tokens, hidden, inner, experts, top_k);
    const int rc = fp8q::check::moe_decode(x, ldx, tokens, hidden, logits, ldl, experts, top_k, inner, w_gu, ldw_gu,
                                           w_gu_stride, s_gu, lds_gu, s_gu_stride, w_down, ldw_down, w_down_stride,
                                           s_down, lds_down, s_down_stride, y, y_dtype, ldy, need, workspace,
                                           workspace_bytes);
    if (rc != kLaunch) return rc;
    fp8q::MoeArgs a{};
    a.x = static_cast<const uint16_t*>(x); a.ldx = ldx;
    a.tokens = (int)tokens; a.hidden = hidden; a.inner = inner;
    a.logits = logits; a.ldl = ldl; a.experts = experts; a.top_k = std::min(top_k, experts); a.renormalize = renormalize ? 1 : 0;
    a.w_gu = w_gu; a.ldw_gu = ldw_gu; a.w_gu_stride = w_gu_stride;
    a.s_gu = s_gu; a.lds_gu = lds_gu; a.s_gu_stride = s_gu_stride;
    a.w_down = w_down; a.ldw_down = ldw_down; a.w_down_stride = w_down_stride;
    a.s_down = s_down; a.lds_down = lds_down; a.s_down_stride = s_down_stride;
    a.y = y; a.y_dtype = y_dtype; a.ldy = ldy; a.workspace = workspace;
    return status_of(fp8q::launch_moe_decode(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
