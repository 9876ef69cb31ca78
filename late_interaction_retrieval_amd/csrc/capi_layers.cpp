// capi_layers.cpp -- the C ABI declared in include/maxsim_layers.h: host-side
// argument validation (no HIP call before it passes), then the kernel launchers.
#include "maxsim_layers.h"

#include <hip/hip_runtime_api.h>

#include <cmath>

#include "layers.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool is_float(int32_t dt) { return dt == MAXSIM_F16 || dt == MAXSIM_BF16 || dt == MAXSIM_F32; }
uintptr_t elem(int32_t dt) { return dt == MAXSIM_F32 ? 4 : 2; }
int hip_status(hipError_t e) { return e == hipSuccess ? MAXSIM_OK : MAXSIM_ERR_HIP; }

// A factor of scores that leaves their exponents, and its own square, inside fp32.
bool factor_ok(float f) { return f >= 0x1p-60f && f <= 0x1p60f; }

// Steps whose multiples stay far inside 64 bits.
bool steps_ok(const maxsim_view& v) {
    const int64_t most = (int64_t)1 << 40;
    return v.batch >= 0 && v.batch <= most && v.token >= 0 && v.token <= most && v.head >= 0 && v.head <= most;
}
// Rows of D values of which no two overlap along one dimension.
bool apart(const maxsim_view& v, int32_t D, int32_t H, int64_t L, int32_t B) {
    return (H <= 1 || v.head >= D) && (L <= 1 || v.token >= D) && (B <= 1 || v.batch >= D);
}

int64_t rows_q(const maxsim_attn& a) { return a.cu_q ? a.rows_q : (int64_t)a.B * a.max_q; }
int64_t rows_k(const maxsim_attn& a) { return a.cu_k ? a.rows_k : (int64_t)a.B * a.max_k; }

// Sizes and the window (what the workspaces go by too).
int attn_sizes(const maxsim_attn& a) {
    if (a.B < 0 || a.max_q < 0 || a.max_k < 0 || a.Hq < 1 || a.Hk < 1 || a.Hq % a.Hk != 0 || a.sinks < 0 || !factor_ok(a.scale))
        return MAXSIM_ERR_SHAPE;
    if (a.D < 8 || a.D > 128 || a.D % 8 != 0 || (a.dtype != MAXSIM_F16 && a.dtype != MAXSIM_BF16)) return MAXSIM_ERR_UNSUPPORTED;
    if (a.lse_step < 1 || (a.lse_step > 1 && a.lse_step < 1 + a.D / 2)) return MAXSIM_ERR_SHAPE;
    const int64_t most = (int64_t)1 << 29;
    if ((int64_t)a.max_q * (a.Hq / a.Hk) >= most || a.max_k >= most) return MAXSIM_ERR_SHAPE;
    if ((a.cu_q && (a.rows_q < 0 || a.rows_q > INT32_MAX)) || (a.cu_k && (a.rows_k < 0 || a.rows_k > INT32_MAX)))
        return MAXSIM_ERR_SHAPE;
    return maxsim::attn_grid_ok(a) ? MAXSIM_OK : MAXSIM_ERR_SHAPE;
}
// A view of 16-bit rows that tiles are loaded from, or rows stored to.
int attn_view(const maxsim_attn& a, const maxsim_view& v, bool keys, bool written) {
    if (!steps_ok(v) || v.token < a.D || v.token > (int64_t)1 << 20) return MAXSIM_ERR_SHAPE;
    const bool packed = keys ? a.cu_k != nullptr : a.cu_q != nullptr;
    if (written && !apart(v, a.D, keys ? a.Hk : a.Hq, 1, packed ? 1 : a.B)) return MAXSIM_ERR_SHAPE;
    if ((keys ? rows_k(a) : rows_q(a)) > 0 && !v.data) return MAXSIM_ERR_NULL;
    if (!aligned(v.data, 16) || v.token % 8 || v.head % 8 || v.batch % 8) return MAXSIM_ERR_ALIGN;
    return MAXSIM_OK;
}
int attn_pointers(const maxsim_attn& a) {
    return aligned(a.cu_q, 4) && aligned(a.cu_k, 4) && aligned(a.q_lens, 4) && aligned(a.k_lens, 4) ? MAXSIM_OK : MAXSIM_ERR_ALIGN;
}

}  // namespace

extern "C" {

int maxsim_rope(const maxsim_view* x, const maxsim_view* y, int32_t B, int32_t L, int32_t H, int32_t D, int32_t rotary,
                int32_t layout, int32_t dtype, const double* inv_freq, const int32_t* positions, const int32_t* offsets,
                float scale, int32_t inverse, void* stream) {
    if (B < 0 || L < 0 || H < 1 || D < 1 || rotary < 2 || rotary % 2 != 0 || rotary > D || !std::isfinite(scale))
        return MAXSIM_ERR_SHAPE;
    if (D > 1024 || !is_float(dtype) || (layout != MAXSIM_ROPE_HALF && layout != MAXSIM_ROPE_INTERLEAVED))
        return MAXSIM_ERR_UNSUPPORTED;
    if ((int64_t)B * L >= (int64_t)1 << 25 || (positions && offsets)) return MAXSIM_ERR_SHAPE;
    if (!x || !y) return MAXSIM_ERR_NULL;
    if (!steps_ok(*x) || !steps_ok(*y) || !apart(*y, D, H, L, B)) return MAXSIM_ERR_SHAPE;
    if (B == 0 || L == 0) return MAXSIM_OK;
    if (!x->data || !y->data || !inv_freq) return MAXSIM_ERR_NULL;
    if (x->data == y->data && (x->batch != y->batch || x->token != y->token || x->head != y->head)) return MAXSIM_ERR_SHAPE;
    if (!aligned(x->data, elem(dtype)) || !aligned(y->data, elem(dtype)) || !aligned(inv_freq, 8) || !aligned(positions, 4) ||
        !aligned(offsets, 4))
        return MAXSIM_ERR_ALIGN;
    maxsim::RopeArgs a{};
    a.x = *x;
    a.y = *y;
    a.B = B;
    a.L = L;
    a.H = H;
    a.D = D;
    a.rotary = rotary;
    a.interleaved = layout == MAXSIM_ROPE_INTERLEAVED;
    a.dtype = dtype;
    a.inverse = inverse != 0;
    a.scale = scale;
    a.inv_freq = inv_freq;
    a.positions = positions;
    a.offsets = offsets;
    return hip_status(maxsim::launch_rope(a, static_cast<hipStream_t>(stream)));
}

size_t maxsim_attn_fwd_workspace_bytes(const maxsim_attn* a) {
    return a && a->B > 0 && attn_sizes(*a) == MAXSIM_OK ? maxsim::attn_fwd_workspace_bytes(*a) : 0;
}
size_t maxsim_attn_bwd_workspace_bytes(const maxsim_attn* a) {
    return a && a->B > 0 && attn_sizes(*a) == MAXSIM_OK ? maxsim::attn_bwd_workspace_bytes(*a) : 0;
}

int maxsim_attn_fwd(const maxsim_attn* a, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    if (!a) return MAXSIM_ERR_NULL;
    int st = attn_sizes(*a);
    if (st == MAXSIM_OK) st = attn_view(*a, a->q, false, false);
    if (st == MAXSIM_OK) st = attn_view(*a, a->k, true, false);
    if (st == MAXSIM_OK) st = attn_view(*a, a->v, true, false);
    if (st == MAXSIM_OK) st = attn_view(*a, a->out, false, true);
    if (st == MAXSIM_OK) st = attn_pointers(*a);
    if (st != MAXSIM_OK) return st;
    if (!aligned(lse, 4) || !aligned(workspace, 16)) return MAXSIM_ERR_ALIGN;
    if (a->B == 0) return MAXSIM_OK;
    const size_t need = maxsim::attn_fwd_workspace_bytes(*a);
    if (need > 0 && !workspace) return MAXSIM_ERR_NULL;
    if (workspace_bytes < need) return MAXSIM_ERR_WORKSPACE;
    return hip_status(maxsim::launch_attn_fwd(*a, lse, workspace, static_cast<hipStream_t>(stream)));
}

int maxsim_attn_bwd(const maxsim_attn* a, const float* lse, const maxsim_view* dout, const maxsim_view* dq,
                    const maxsim_view* dk, const maxsim_view* dv, void* workspace, size_t workspace_bytes, void* stream) {
    if (!a || !dout || !dq || !dk || !dv) return MAXSIM_ERR_NULL;
    int st = attn_sizes(*a);
    if (st == MAXSIM_OK) st = attn_view(*a, a->q, false, false);
    if (st == MAXSIM_OK) st = attn_view(*a, a->k, true, false);
    if (st == MAXSIM_OK) st = attn_view(*a, a->v, true, false);
    if (st == MAXSIM_OK) st = attn_view(*a, a->out, false, false);
    if (st == MAXSIM_OK) st = attn_view(*a, *dout, false, false);
    if (st == MAXSIM_OK) st = attn_view(*a, *dq, false, true);
    if (st == MAXSIM_OK) st = attn_view(*a, *dk, true, true);
    if (st == MAXSIM_OK) st = attn_view(*a, *dv, true, true);
    if (st == MAXSIM_OK) st = attn_pointers(*a);
    if (st != MAXSIM_OK) return st;
    if (!aligned(lse, 4) || !aligned(workspace, 16)) return MAXSIM_ERR_ALIGN;
    if (a->B == 0) return MAXSIM_OK;
    if (rows_q(*a) > 0 && !lse) return MAXSIM_ERR_NULL;
    const size_t need = maxsim::attn_bwd_workspace_bytes(*a);
    if (need > 0 && !workspace) return MAXSIM_ERR_NULL;
    if (workspace_bytes < need) return MAXSIM_ERR_WORKSPACE;
    return hip_status(maxsim::launch_attn_bwd(*a, lse, *dout, *dq, *dk, *dv, workspace, static_cast<hipStream_t>(stream)));
}

static int distill_sizes(int32_t N, int32_t V, int32_t K, int32_t dtype, float temperature, int64_t ld) {
    if (N < 0 || V < 0 || K < 0 || !factor_ok(temperature)) return MAXSIM_ERR_SHAPE;
    if (K > 1024 || !is_float(dtype)) return MAXSIM_ERR_UNSUPPORTED;
    if (N >= 1 << 24 || V >= 1 << 30 || ld < V || ld > (int64_t)1 << 31) return MAXSIM_ERR_SHAPE;
    return MAXSIM_OK;
}

size_t maxsim_distill_workspace_bytes(int32_t N, int32_t V) {
    return distill_sizes(N, V, 0, MAXSIM_F32, 1.f, V) == MAXSIM_OK ? maxsim::distill_workspace_bytes(N, V) : 0;
}

int maxsim_distill_fwd(const void* scores, int64_t ld, const int32_t* index, const float* teacher, int32_t N, int32_t V,
                       int32_t K, int32_t dtype, float temperature, float* loss, float* stat, void* workspace,
                       size_t workspace_bytes, void* stream) {
    const int st = distill_sizes(N, V, K, dtype, temperature, ld);
    if (st != MAXSIM_OK) return st;
    if (N == 0) return MAXSIM_OK;
    if ((V > 0 && !scores) || (K > 0 && (!index || !teacher)) || !loss || !stat) return MAXSIM_ERR_NULL;
    if (!aligned(scores, elem(dtype)) || !aligned(index, 4) || !aligned(teacher, 4) || !aligned(loss, 4) || !aligned(stat, 4) ||
        !aligned(workspace, 16))
        return MAXSIM_ERR_ALIGN;
    const size_t need = maxsim::distill_workspace_bytes(N, V);
    if (need > 0 && !workspace) return MAXSIM_ERR_NULL;
    if (workspace_bytes < need) return MAXSIM_ERR_WORKSPACE;
    maxsim::DistillArgs a{};
    a.scores = scores;
    a.index = index;
    a.teacher = teacher;
    a.loss = loss;
    a.stat = stat;
    a.partial = static_cast<float*>(workspace);
    a.ld = ld;
    a.N = N;
    a.V = V;
    a.K = K;
    a.dtype = dtype;
    a.temperature = temperature;
    return hip_status(maxsim::launch_distill_fwd(a, static_cast<hipStream_t>(stream)));
}

int maxsim_distill_bwd(const float* dloss, const void* scores, int64_t ld, const float* stat, const int32_t* index,
                       const float* teacher, int32_t N, int32_t V, int32_t K, int32_t dtype, float temperature,
                       void* dscores, int64_t ldd, void* stream) {
    const int st = distill_sizes(N, V, K, dtype, temperature, ld);
    if (st != MAXSIM_OK) return st;
    if (ldd < V || ldd > (int64_t)1 << 31 || (scores && scores == dscores && ld != ldd)) return MAXSIM_ERR_SHAPE;
    if (N == 0 || V == 0) return MAXSIM_OK;
    if (!dloss || !scores || !stat || (K > 0 && (!index || !teacher)) || !dscores) return MAXSIM_ERR_NULL;
    if (!aligned(scores, elem(dtype)) || !aligned(dscores, elem(dtype)) || !aligned(index, 4) || !aligned(teacher, 4) ||
        !aligned(dloss, 4) || !aligned(stat, 4))
        return MAXSIM_ERR_ALIGN;
    maxsim::DistillArgs a{};
    a.scores = scores;
    a.index = index;
    a.teacher = teacher;
    a.dloss = dloss;
    a.dscores = dscores;
    a.stat = const_cast<float*>(stat);
    a.ld = ld;
    a.ldd = ldd;
    a.N = N;
    a.V = V;
    a.K = K;
    a.dtype = dtype;
    a.temperature = temperature;
    return hip_status(maxsim::launch_distill_bwd(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
