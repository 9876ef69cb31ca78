// capi_encoder.cpp -- the C ABI declared in include/maxsim_encoder.h: host-side
// argument validation (no HIP call before it passes), then the kernel launchers.
#include "maxsim_encoder.h"

#include <hip/hip_runtime_api.h>

#include <cmath>

#include "encoder.h"

namespace {

using maxsim::ceil_div;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool is_float(int32_t dt) { return dt == MAXSIM_F16 || dt == MAXSIM_BF16 || dt == MAXSIM_F32; }
uintptr_t elem(int32_t dt) { return dt == MAXSIM_F32 ? 4 : dt == MAXSIM_F16 || dt == MAXSIM_BF16 ? 2 : 1; }
int hip_status(hipError_t e) { return e == hipSuccess ? MAXSIM_OK : MAXSIM_ERR_HIP; }

// A pitch of at least `width`, with every offset of `rows` of them far inside 64 bits.
bool pitch_ok(int64_t ld, int64_t width) { return ld >= width && ld <= (int64_t)1 << 31; }

}  // namespace

extern "C" {

int maxsim_rmsnorm_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                       int32_t weight_dtype, int32_t R, int32_t H, int32_t dtype, float eps, int32_t out_dtype,
                       void* y, int64_t ldy, float* scale, void* sum, int64_t lds, float* rstd, void* stream) {
    if (R < 0 || H < 1 || !(eps >= 0.f)) return MAXSIM_ERR_SHAPE;
    if (H > maxsim::kMaxNormWidth || !is_float(dtype)) return MAXSIM_ERR_UNSUPPORTED;
    if (weight && weight_dtype != dtype && weight_dtype != MAXSIM_F32) return MAXSIM_ERR_UNSUPPORTED;
    const bool eight = out_dtype == MAXSIM_I8 || out_dtype == MAXSIM_E4M3;
    if (!eight && !is_float(out_dtype)) return MAXSIM_ERR_UNSUPPORTED;
    if (!pitch_ok(ldx, H) || !pitch_ok(ldy, H) || (residual && !pitch_ok(ldr, H)) || (sum && !pitch_ok(lds, H)))
        return MAXSIM_ERR_SHAPE;
    if (R == 0) return MAXSIM_OK;
    if (!x || !y || (eight && !scale)) return MAXSIM_ERR_NULL;
    const uintptr_t e = elem(dtype);
    if (!aligned(x, e) || !aligned(residual, e) || !aligned(sum, e) || !aligned(y, elem(out_dtype)) ||
        !aligned(weight, elem(weight_dtype)) || !aligned(scale, 4) || !aligned(rstd, 4))
        return MAXSIM_ERR_ALIGN;
    maxsim::NormArgs a{};
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.y = y;
    a.scale = scale;
    a.sum = sum;
    a.rstd = rstd;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldy = ldy;
    a.lds = lds;
    a.R = R;
    a.H = H;
    a.dtype = dtype;
    a.weight_f32 = weight_dtype == MAXSIM_F32;
    a.out_dtype = out_dtype;
    a.eps = eps;
    return hip_status(maxsim::launch_rmsnorm_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t maxsim_rmsnorm_bwd_workspace_bytes(int32_t R, int32_t H) {
    if (R < 0 || H < 1 || H > maxsim::kMaxNormWidth || maxsim::norm_bwd_small(R, H)) return 0;
    return (size_t)maxsim::norm_bwd_groups(R, H) * (size_t)H * sizeof(float);
}

int maxsim_rmsnorm_bwd(const void* dy, int64_t lddy, const void* h, int64_t ldh, const float* rstd,
                       const void* weight, int32_t weight_dtype, const void* dsum, int64_t ldds, int32_t R, int32_t H,
                       int32_t dtype, void* dx, int64_t lddx, float* dweight, void* workspace,
                       size_t workspace_bytes, void* stream) {
    if (R < 0 || H < 1) return MAXSIM_ERR_SHAPE;
    if (H > maxsim::kMaxNormWidth || !is_float(dtype)) return MAXSIM_ERR_UNSUPPORTED;
    if (weight && weight_dtype != dtype && weight_dtype != MAXSIM_F32) return MAXSIM_ERR_UNSUPPORTED;
    if (!pitch_ok(lddy, H) || !pitch_ok(ldh, H) || !pitch_ok(lddx, H) || (dsum && !pitch_ok(ldds, H)))
        return MAXSIM_ERR_SHAPE;
    if (R == 0 && !dweight) return MAXSIM_OK;
    const size_t need = dweight ? maxsim_rmsnorm_bwd_workspace_bytes(R, H) : 0;
    if (R > 0 && (!dy || !h || !rstd || !dx || (need > 0 && !workspace))) return MAXSIM_ERR_NULL;
    const uintptr_t e = elem(dtype);
    if (!aligned(dy, e) || !aligned(h, e) || !aligned(dsum, e) || !aligned(dx, e) || !aligned(rstd, 4) ||
        !aligned(weight, elem(weight_dtype)) || !aligned(dweight, 4) || !aligned(workspace, 16))
        return MAXSIM_ERR_ALIGN;
    if (workspace_bytes < need) return MAXSIM_ERR_WORKSPACE;
    maxsim::NormBwdArgs a{};
    a.dy = dy;
    a.h = h;
    a.rstd = rstd;
    a.weight = weight;
    a.dsum = dsum;
    a.dx = dx;
    a.dweight = dweight;
    a.partial = static_cast<float*>(workspace);
    a.lddy = lddy;
    a.ldh = ldh;
    a.ldds = ldds;
    a.lddx = lddx;
    a.R = R;
    a.H = H;
    a.dtype = dtype;
    a.weight_f32 = weight_dtype == MAXSIM_F32;
    return hip_status(maxsim::launch_rmsnorm_bwd(a, static_cast<hipStream_t>(stream)));
}

int maxsim_quant_fp8(const void* x, int64_t ldx, int32_t R, int32_t C, int32_t dtype, int32_t block_rows, void* q,
                     int64_t ldq, float* scale, void* qt, int64_t ldqt, float* scale_t, void* stream) {
    if (R < 0 || C < 0) return MAXSIM_ERR_SHAPE;
    if (!is_float(dtype) || (block_rows != 1 && block_rows != MAXSIM_QBLOCK)) return MAXSIM_ERR_UNSUPPORTED;
    if (!pitch_ok(ldx, C) || (q && !pitch_ok(ldq, C)) || (qt && !pitch_ok(ldqt, R))) return MAXSIM_ERR_SHAPE;
    // one workgroup to 128 x 128 values; a launch holds fewer than 2^32 threads
    if (ceil_div(R, MAXSIM_QBLOCK) * ceil_div(C, MAXSIM_QBLOCK) >= (int64_t)1 << 24) return MAXSIM_ERR_SHAPE;
    if (R == 0 || C == 0) return MAXSIM_OK;
    if (!x || (!q && !qt) || (q && !scale) || (qt && !scale_t)) return MAXSIM_ERR_NULL;
    if (!aligned(x, elem(dtype)) || !aligned(scale, 4) || !aligned(scale_t, 4)) return MAXSIM_ERR_ALIGN;
    maxsim::QuantArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.R = R;
    a.C = C;
    a.dtype = dtype;
    a.square = block_rows != 1;
    a.q = static_cast<uint8_t*>(q);
    a.ldq = ldq;
    a.scale = scale;
    a.qt = static_cast<uint8_t*>(qt);
    a.ldqt = ldqt;
    a.scale_t = scale_t;
    return hip_status(maxsim::launch_quant_fp8(a, static_cast<hipStream_t>(stream)));
}

size_t maxsim_gemm_fp8_workspace_bytes(int32_t M, int32_t N, int32_t K) {
    if (M <= 0 || N <= 0 || K <= 0 || K > 1 << 22) return 0;
    return maxsim::gemm_fp8_workspace_bytes(M, N, K);
}

int maxsim_gemm_fp8(const void* A, int64_t lda, const float* a_scale, const void* B, int64_t ldb,
                    const float* b_scale, int32_t b_block_rows, int32_t M, int32_t N, int32_t K, int32_t out_dtype,
                    void* c, int64_t ldc, void* workspace, size_t workspace_bytes, void* stream) {
    if (M < 0 || N < 0 || K < 0) return MAXSIM_ERR_SHAPE;
    if (!is_float(out_dtype) || (b_block_rows != 1 && b_block_rows != MAXSIM_QBLOCK)) return MAXSIM_ERR_UNSUPPORTED;
    const int64_t most = (int64_t)1 << 22;  // a tile's rows stay within 32-bit byte offsets
    if (K > most || lda > most || ldb > most) return MAXSIM_ERR_UNSUPPORTED;
    const int64_t k16 = ceil_div(K, 16) * 16;
    if (lda < k16 || ldb < k16 || !pitch_ok(ldc, N)) return MAXSIM_ERR_SHAPE;
    if (ceil_div(M, 128) * ceil_div(N, 128) >= (int64_t)1 << 22) return MAXSIM_ERR_SHAPE;
    if (M == 0 || N == 0) return MAXSIM_OK;
    if (!c || (K > 0 && (!A || !B || !a_scale || !b_scale))) return MAXSIM_ERR_NULL;
    if (!aligned(A, 16) || !aligned(B, 16) || lda % 16 != 0 || ldb % 16 != 0 || !aligned(a_scale, 4) ||
        !aligned(b_scale, 4) || !aligned(c, elem(out_dtype)) || !aligned(workspace, 16))
        return MAXSIM_ERR_ALIGN;
    const size_t need = maxsim_gemm_fp8_workspace_bytes(M, N, K);
    if (need > 0 && !workspace) return MAXSIM_ERR_NULL;
    if (workspace_bytes < need) return MAXSIM_ERR_WORKSPACE;
    maxsim::GemmArgs a{};
    a.A = static_cast<const uint8_t*>(A);
    a.B = static_cast<const uint8_t*>(B);
    a.a_scale = a_scale;
    a.b_scale = b_scale;
    a.c = c;
    a.partial = static_cast<float*>(workspace);
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = ldc;
    a.M = M;
    a.N = N;
    a.K = K;
    a.b_block_rows = b_block_rows;
    a.out_dtype = out_dtype;
    return hip_status(maxsim::launch_gemm_fp8(a, static_cast<hipStream_t>(stream)));
}

int maxsim_adamw(const maxsim_adamw_tensor* tensors, int32_t count, int32_t param_dtype, int32_t grad_dtype,
                 int32_t state_dtype, double lr, double beta1, double beta2, double eps, double weight_decay,
                 int32_t step, const int32_t* step_dev, void* stream) {
    if (count < 0 || (!step_dev && step < 1)) return MAXSIM_ERR_SHAPE;
    if (!(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) || !(eps >= 0)) return MAXSIM_ERR_SHAPE;
    if (!std::isfinite(lr) || !std::isfinite(weight_decay)) return MAXSIM_ERR_SHAPE;
    if (!is_float(param_dtype) || !is_float(grad_dtype)) return MAXSIM_ERR_UNSUPPORTED;
    if (state_dtype != MAXSIM_F32 && state_dtype != MAXSIM_E4M3) return MAXSIM_ERR_UNSUPPORTED;
    if (count == 0) return MAXSIM_OK;
    if (!tensors) return MAXSIM_ERR_NULL;
    if (!aligned(step_dev, 4)) return MAXSIM_ERR_ALIGN;
    const bool packed = state_dtype == MAXSIM_E4M3;
    for (int32_t i = 0; i < count; ++i) {
        const maxsim_adamw_tensor& t = tensors[i];
        if (t.n < 0 || t.n > (int64_t)1 << 40) return MAXSIM_ERR_SHAPE;
        if (t.n == 0) continue;
        if (!t.param || !t.grad || !t.m || !t.v || (packed && (!t.m_scale || !t.v_scale))) return MAXSIM_ERR_NULL;
        if (t.master && param_dtype == MAXSIM_F32) return MAXSIM_ERR_UNSUPPORTED;
        const uintptr_t s = packed ? 1 : 4;
        if (!aligned(t.param, elem(param_dtype)) || !aligned(t.grad, elem(grad_dtype)) || !aligned(t.master, 4) ||
            !aligned(t.m, s) || !aligned(t.v, s) || !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))
            return MAXSIM_ERR_ALIGN;
    }
    maxsim::AdamWHyper hp{lr, beta1, beta2, eps, weight_decay, step, step_dev};
    return hip_status(maxsim::launch_adamw(tensors, count, param_dtype, grad_dtype, state_dtype, hp,
                                           static_cast<hipStream_t>(stream)));
}

}  // extern "C"
