// encoder.h -- host-side interface between the C ABI of the embedding head's
// operators (capi_encoder.cpp) and their kernel launchers (rmsnorm.hip,
// quant.hip, gemm_fp8.hip, adamw.hip).  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "maxsim_encoder.h"

namespace maxsim {

constexpr int kQBlock = MAXSIM_QBLOCK;
constexpr int kMaxNormWidth = 32768;  // 1024 threads x 4 vectors of 8 values hold one row

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct NormArgs {
    const void* x;
    const void* residual;
    const void* weight;
    void* y;
    float* scale;
    void* sum;
    float* rstd;
    int64_t ldx, ldr, ldy, lds;
    int R, H;
    int dtype, weight_f32, out_dtype;
    float eps;
};
hipError_t launch_rmsnorm_fwd(const NormArgs& a, hipStream_t stream);

struct NormBwdArgs {
    const void* dy;
    const void* h;
    const float* rstd;
    const void* weight;
    const void* dsum;
    void* dx;
    float* dweight;  // or nullptr
    float* partial;  // [norm_bwd_groups][H] (workspace)
    int64_t lddy, ldh, ldds, lddx;
    int R, H;
    int dtype, weight_f32;
};
bool norm_bwd_small(int R, int H);  // one launch and no partial sums
int norm_bwd_groups(int R, int H);  // workgroups of the row pass = partial sums of dweight
hipError_t launch_rmsnorm_bwd(const NormBwdArgs& a, hipStream_t stream);

struct QuantArgs {
    const void* x;
    int64_t ldx;
    int R, C, dtype;
    bool square;  // one scale for 128 x 128 values
    uint8_t* q;
    int64_t ldq;
    float* scale;
    uint8_t* qt;
    int64_t ldqt;
    float* scale_t;
};
hipError_t launch_quant_fp8(const QuantArgs& a, hipStream_t stream);

struct GemmArgs {
    const uint8_t* A;
    const uint8_t* B;
    const float* a_scale;
    const float* b_scale;
    void* c;
    float* partial;  // [splits][M][N] (workspace)
    int64_t lda, ldb, ldc;
    int M, N, K;
    int b_block_rows, out_dtype;
};
size_t gemm_fp8_workspace_bytes(int M, int N, int K);
hipError_t launch_gemm_fp8(const GemmArgs& a, hipStream_t stream);

struct AdamWHyper {
    double lr, beta1, beta2, eps, decay;
    int step;
    const int32_t* step_dev;
};
hipError_t launch_adamw(const maxsim_adamw_tensor* t, int count, int param_dtype, int grad_dtype, int state_dtype,
                        const AdamWHyper& hp, hipStream_t stream);

}  // namespace maxsim
