// adamw.hip -- one AdamW step over many tensors at once, states in fp32 or in
// 8 bits, for gfx950 (MI355X).
//
//     m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//     p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// The moments are formed in the order of the elementary steps (m times b1, then g times
// 1 - b1 added; v times b2, then g g times 1 - b2 added), each rounded once, so they equal
// the plain fp32 form's bit for bit.  In another order they differ by a unit in the last
// place, which is nothing in fp32 but, held in 8 bits, carried 160 of 67 M codes over a
// tie in each step; where such a code became its block's largest, the block's
// scale parted from the plain form's by 2 to 6 % a step later.
//
// HBM-bound: every value is read and written once (28 bytes with fp32 weights,
// gradients and states).  The tensors' table travels in the kernel's arguments,
// 56 to a launch, so there is nothing to copy or keep on the device and a
// captured launch holds its own table.  Workgroups of 2048 values are dealt to the
// tensors in order; each finds its tensor by a search over the first workgroups.
//
// 8-bit states: 16 lanes hold a block of 128 values, whose scale is a 16-lane
// maximum.  The first moment is e4m3 times the scale.  The second is held as its
// square root, which halves the exponents that the 4 bits have to span, and a
// root above 0 is rounded up to the smallest value at least: read as 0 it would
// leave m / eps.
//
// Measured: 67,108,864 values in 100 tensors, bf16 weights and gradients, fp32
// masters, 8-bit states, 206 us in two launches (1.08 GB, 5.2 TB/s: HBM);
// 132,224 fp32 values in 3 tensors 4.2 us (a launch).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "encoder_dev.h"

namespace maxsim {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = kThreads * kVec;  // values of one workgroup
constexpr int kTensors = 56;             // entries of one launch's table

struct Table {
    maxsim_adamw_tensor t[kTensors];
    uint32_t first[kTensors + 1];  // first workgroup of each tensor
    int count;
};
struct Step {
    float beta1, beta2, eps, keep;  // keep = 1 - lr * decay
    float one_minus_beta1, one_minus_beta2;
    float rate;      // lr / (1 - beta1^t)
    float inv_root;  // 1 / sqrt(1 - beta2^t)
    double lr, log_beta1, log_beta2;  // for a step number on the device
    const int32_t* step_dev;
};
static_assert(sizeof(Table) + sizeof(Step) <= 4096, "kernel arguments");

// lr / (1 - beta1^t) and 1 / sqrt(1 - beta2^t), without the cancellation that 1 - pow has at small t
__host__ __device__ inline void corrections(double lr, double log_beta1, double log_beta2, int t, float* rate,
                                            float* inv_root) {
    *rate = (float)(lr / -expm1(t * log_beta1));
    *inv_root = (float)(1.0 / sqrt(-expm1(t * log_beta2)));
}

template <typename T>
__device__ __forceinline__ void load_f(const void* base, int64_t at, int n, float* f) {
    const auto v = load8<T>((const T*)base + at, 0, n);
#pragma unroll
    for (int i = 0; i < kVec; ++i) f[i] = (float)v[i];
}

__device__ __forceinline__ void load_e4m3(const void* base, int64_t at, int n, float scale, float* f) {
    const uint8_t* row = (const uint8_t*)base + at;
    u8x8 v;
    if (n >= kVec) {
        v = *reinterpret_cast<const u8x8*>(row);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = i < n ? row[i] : (uint8_t)0;
    }
    const u32x2 b = __builtin_bit_cast(u32x2, v);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        f[4 * w + 0] = __builtin_amdgcn_cvt_f32_fp8((int)b[w], 0) * scale;
        f[4 * w + 1] = __builtin_amdgcn_cvt_f32_fp8((int)b[w], 1) * scale;
        f[4 * w + 2] = __builtin_amdgcn_cvt_f32_fp8((int)b[w], 2) * scale;
        f[4 * w + 3] = __builtin_amdgcn_cvt_f32_fp8((int)b[w], 3) * scale;
    }
}

template <typename PT, typename GT, bool PACKED>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const Table tab, const Step st) {
    typedef typename PT::type P;
    typedef typename GT::type G;
    int lo = 0, hi = tab.count;  // the last tensor whose first workgroup is not past this one
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tab.first[mid] <= blockIdx.x)
            lo = mid;
        else
            hi = mid;
    }
    const maxsim_adamw_tensor& t = tab.t[lo];
    float rate = st.rate, inv_root = st.inv_root;
    if (st.step_dev != nullptr) {
        __shared__ float both[2];
        if (threadIdx.x == 0) corrections(st.lr, st.log_beta1, st.log_beta2, *st.step_dev, &both[0], &both[1]);
        __syncthreads();
        rate = both[0];
        inv_root = both[1];
    }
    const int64_t at = (int64_t)(blockIdx.x - tab.first[lo]) * kChunk + threadIdx.x * kVec;
    const int64_t left = t.n - at;
    // lanes past the end hold zeros: they add nothing to a block's scale
    const int n = left >= kVec ? kVec : left > 0 ? (int)left : 0;
    float p[kVec], g[kVec], m[kVec], v[kVec];
    load_f<G>(t.grad, at, n, g);
    if (!std::is_same<PT, F32>::value && t.master != nullptr)
        load_f<float>(t.master, at, n, p);
    else
        load_f<P>(t.param, at, n, p);
    if constexpr (PACKED) {
        const bool any = n > 0;
        load_e4m3(t.m, at, n, any ? t.m_scale[at / kQBlock] : 0.f, m);
        load_e4m3(t.v, at, n, any ? t.v_scale[at / kQBlock] : 0.f, v);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {  // a root that is not 0 has a square that is not 0, below 2^-75 too
            const float sq = v[i] * v[i];
            v[i] = sq == 0.f && v[i] != 0.f ? __FLT_DENORM_MIN__ : sq;
        }
    } else {
        load_f<float>(t.m, at, n, m);
        load_f<float>(t.v, at, n, v);
    }
    float root[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        m[i] = __builtin_fmaf(st.one_minus_beta1, g[i], st.beta1 * m[i]);
        v[i] = __builtin_fmaf(st.one_minus_beta2, g[i] * g[i], st.beta2 * v[i]);
        root[i] = __builtin_sqrtf(v[i]);
        p[i] = __builtin_fmaf(p[i], st.keep, -rate * (m[i] / __builtin_fmaf(root[i], inv_root, st.eps)));
    }
    if (!std::is_same<PT, F32>::value && t.master != nullptr) store8<float>(t.master + at, 0, n, p);
    store8<P>((P*)t.param + at, 0, n, p);
    if constexpr (PACKED) {
        uint32_t top_m = 0, top_v = 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            top_m = umax(top_m, mag(m[i]));
            top_v = umax(top_v, mag(root[i]));
        }
        const Scale km = block_scale(max16(top_m), 448.f);
        const Scale kv = block_scale(max16(top_v), 448.f);
        u32x2 qv = to_e4m3(root, kv);
        if (!kv.zeros) {
#pragma unroll
            for (int i = 0; i < kVec; ++i)  // the code 1 is the smallest value
                if (root[i] > 0.f && ((qv[i >> 2] >> (8 * (i & 3))) & 255u) == 0u) qv[i >> 2] |= 1u << (8 * (i & 3));
        }
        if (n > 0) {
            store8_bytes((uint8_t*)t.m + at, 0, n, to_e4m3(m, km));
            store8_bytes((uint8_t*)t.v + at, 0, n, qv);
            if (at % kQBlock == 0) {
                t.m_scale[at / kQBlock] = km.s;
                t.v_scale[at / kQBlock] = kv.s;
            }
        }
    } else {
        store8<float>((float*)t.m + at, 0, n, m);
        store8<float>((float*)t.v + at, 0, n, v);
    }
}

template <typename PT, typename GT>
void launch(const Table& tab, const Step& st, bool packed, unsigned grid, hipStream_t stream) {
    if (packed)
        adamw_kernel<PT, GT, true><<<grid, kThreads, 0, stream>>>(tab, st);
    else
        adamw_kernel<PT, GT, false><<<grid, kThreads, 0, stream>>>(tab, st);
}
template <typename PT>
void launch_by_grad(int grad_dtype, const Table& tab, const Step& st, bool packed, unsigned grid, hipStream_t stream) {
    if (grad_dtype == MAXSIM_F16)
        launch<PT, F16>(tab, st, packed, grid, stream);
    else if (grad_dtype == MAXSIM_BF16)
        launch<PT, BF16>(tab, st, packed, grid, stream);
    else
        launch<PT, F32>(tab, st, packed, grid, stream);
}

}  // namespace

hipError_t launch_adamw(const maxsim_adamw_tensor* t, int count, int param_dtype, int grad_dtype, int state_dtype,
                        const AdamWHyper& hp, hipStream_t stream) {
    // An error that an earlier call of the program left unread is not this step's: reported
    // after the launches it would make a step that ran look like one that did not.
    (void)hipGetLastError();
    Step st{};
    // doubles up to here: 1 - 0.999 in fp32 is off by 1e-5 of itself
    st.beta1 = (float)hp.beta1;
    st.beta2 = (float)hp.beta2;
    st.one_minus_beta1 = (float)(1.0 - hp.beta1);
    st.one_minus_beta2 = (float)(1.0 - hp.beta2);
    st.eps = (float)hp.eps;
    st.keep = (float)(1.0 - hp.lr * hp.decay);
    st.lr = hp.lr;
    st.log_beta1 = std::log(hp.beta1);
    st.log_beta2 = std::log(hp.beta2);
    st.step_dev = hp.step_dev;
    if (hp.step_dev == nullptr) corrections(hp.lr, st.log_beta1, st.log_beta2, hp.step, &st.rate, &st.inv_root);
    // a launch holds fewer than 2^32 threads: at most this many workgroups of a tensor at a time
    constexpr int64_t kMost = (int64_t)1 << 22;
    Table tab{};
    uint32_t blocks = 0;
    auto flush = [&]() {
        if (tab.count == 0) return hipSuccess;
        tab.first[tab.count] = blocks;
        const bool packed = state_dtype == MAXSIM_E4M3;
        if (param_dtype == MAXSIM_F16)
            launch_by_grad<F16>(grad_dtype, tab, st, packed, blocks, stream);
        else if (param_dtype == MAXSIM_BF16)
            launch_by_grad<BF16>(grad_dtype, tab, st, packed, blocks, stream);
        else
            launch_by_grad<F32>(grad_dtype, tab, st, packed, blocks, stream);
        tab.count = 0;
        blocks = 0;
        return hipGetLastError();
    };
    const int64_t elem[3] = {2, 2, 4};
    const int64_t state = state_dtype == MAXSIM_E4M3 ? 1 : 4;
    for (int i = 0; i < count; ++i) {
        for (int64_t from = 0; from < t[i].n; from += kMost * kChunk) {  // a part of the tensor
            maxsim_adamw_tensor e = t[i];
            e.n = std::min(t[i].n - from, kMost * kChunk);
            e.param = (char*)e.param + from * elem[param_dtype];
            e.grad = (const char*)e.grad + from * elem[grad_dtype];
            e.m = (char*)e.m + from * state;
            e.v = (char*)e.v + from * state;
            if (e.master != nullptr) e.master += from;
            if (e.m_scale != nullptr) e.m_scale += from / kQBlock;
            if (e.v_scale != nullptr) e.v_scale += from / kQBlock;
            const int64_t need = ceil_div(e.n, kChunk);
            if (tab.count == kTensors || blocks + need > kMost) {
                const hipError_t err = flush();
                if (err != hipSuccess) return err;
            }
            tab.t[tab.count] = e;
            tab.first[tab.count++] = blocks;
            blocks += (uint32_t)need;
        }
    }
    return flush();
}

}  // namespace maxsim
