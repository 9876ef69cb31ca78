// distill.hip -- distillation from a teacher's top scores, forward and backward,
// for gfx950 (MI355X).
//
//     q = softmax(teacher / T) over a row's entries;  p = softmax(z / T) over its columns
//     loss = T^2 sum_k q_k (log q_k - log p_{i_k});  dz_v = dloss T (p_v - sum_{k: i_k = v} q_k)
//
// Bound by HBM: the forward reads z once, with a running maximum and sum in each thread; the
// backward reads it once and writes dz.  The entries touch a few columns only: the backward first writes
// dloss T p over the whole row and then the entries' columns again.  Few long rows are split over
// workgroups.  Differences z - max are formed before they are multiplied by 1 / T, and the backward gets
// the maximum and the sum's logarithm apart, so that large scores at a low temperature lose nothing.
//
// Measured, the kernels alone: 8192 x 32768 bf16 forward 120 - 131 us (537 MB at 4.1 - 4.5 TB/s), backward 207 - 215 (1.07 GB at
// 5.0 - 5.2); 10393 x 2887 fp32 36 and 48; 32 x 200003 fp32 forward 7.2 + 4.4 (the parts' join), backward 11.9; 64 x 64 4.4 and 5.5, a launch each.
#include <algorithm>

#include "encoder_dev.h"
#include "layers.h"

namespace maxsim {
namespace {

constexpr int kMostEntries = 1024;
constexpr size_t kLastCache = (size_t)256 << 20;  // bytes
constexpr int kThreads = 256;
// Columns that one wave takes by itself.  Forward (us with a wave to a row, and with four; 16 entries, scores in the last cache): many rows, up to 4096 columns:
// 10393 x 2887 fp32 24, 36; 4096 x 4096 bf16 9.8, 15; 1024 x 4096 bf16 5.1, 5.9; 1024 x 512 fp32 3.6, 5.1 (but 600 x 6000 bf16 7.7,
// 7.4; 16384 x 8192 bf16 91, 87).  Rows that leave a CU few waves (kFewRows), up to 2048: 256 x 512 fp32 3.6, 4.1; 16 x 1500 fp32 4.0, 4.1, with
// 100 entries 4.4, 4.2; but 64 x 2887 fp32 4.8, 4.4; 256 x 4096 bf16 5.0, 4.4, with 100 entries 5.6, 4.5.  Backward, whose four waves share
// the entries: 10393 x 2887 fp32 53, 49; 512 x 2887 fp32 9.9, 6.6; 128 x 1500 fp32 6.7, 4.8; 16384 x 1500 bf16 28, 33.
constexpr int kShortForward = 4096, kShortFew = 2048, kFewRows = 512, kShortRow = 1024;
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

// The largest z and the sum of exp((z - largest) / T).
struct Soft {
    float top, sum;
};
__device__ __forceinline__ Soft join(Soft a, Soft b, float c) {
    const float top = fmaxf(a.top, b.top), at = top == -INFINITY ? 0.f : top;
    return {top, a.sum * __builtin_amdgcn_exp2f((a.top - at) * c) + b.sum * __builtin_amdgcn_exp2f((b.top - at) * c)};
}
__device__ __forceinline__ Soft join64(Soft s, float c) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) s = join(s, {__shfl_xor(s.top, d), __shfl_xor(s.sum, d)}, c);
    return s;
}
// Over TPR threads of a row: a wave, or the workgroup, whose waves meet in `part`.
template <int TPR>
__device__ __forceinline__ Soft join_row(Soft s, float c, Soft* part) {
    s = join64(s, c);
    if constexpr (TPR > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
        __syncthreads();
        s = part[0];
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i) s = join(s, part[i], c);
    }
    return s;
}
template <int TPR>
__device__ __forceinline__ float add_row(float v, float* part) {
    v = sum64(v);
    if constexpr (TPR > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = part[0];
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i) v += part[i];
    }
    return v;
}

// Vectors that pass the caches by (STREAM) or not.
template <typename T, bool STREAM>
__device__ __forceinline__ typename Pack8<T>::V load_vec(const T* row, int c, int n) {
    if (STREAM && c + kVec <= n) return __builtin_nontemporal_load(reinterpret_cast<const typename Pack8<T>::V*>(row + c));
    return load8<T>(row, c, n);
}
template <typename T, bool STREAM>
__device__ __forceinline__ void store_vec(T* row, int c, int n, const float* f) {
    if (STREAM && c + kVec <= n) {
        typename Pack8<T>::V v;
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = (T)f[i];
        __builtin_nontemporal_store(v, reinterpret_cast<typename Pack8<T>::V*>(row + c));
    } else {
        store8<T>(row, c, n, f);
    }
}

// A row's threads have read and written what comes before: one wave's, or the workgroup's.
template <int TPR>
__device__ __forceinline__ void row_sync() {
    if constexpr (TPR > 64) {
        __syncthreads();
    } else {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0): the row's stores are made
        asm volatile("" ::: "memory");
    }
}

// A row's columns [from, to) by its threads; the next ones are on their way while these are worked on.
template <typename T, int TPR>
__device__ __forceinline__ Soft soft_of(const T* z, int from, int to, int lane, float c) {
    constexpr int AHEAD = 4;
    Soft s = {-INFINITY, 0.f};
    typename Pack8<T>::V v[AHEAD], next[AHEAD];
    const auto load = [&](int first, typename Pack8<T>::V* to_) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
            if (first + a * TPR * kVec < to) to_[a] = load8<T>(z, first + a * TPR * kVec, to);
    };
    int at = from + lane * kVec;
    load(at, v);
    while (at < to) {
        load(at + AHEAD * TPR * kVec, next);
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const int col = at + a * TPR * kVec;
            if (col >= to) continue;
            float f[kVec], top = s.top;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                f[i] = col + i < to ? (float)v[a][i] : -INFINITY;
                top = fmaxf(top, f[i]);
            }
            const float base = top == -INFINITY ? 0.f : top;
            s.sum *= __builtin_amdgcn_exp2f((s.top - base) * c);
            s.top = top;
#pragma unroll
            for (int i = 0; i < kVec; ++i) s.sum += __builtin_amdgcn_exp2f((f[i] - base) * c);
        }
        at += AHEAD * TPR * kVec;
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) v[a] = next[a];
    }
    return s;
}

// One of a row's entries: its column (-1: none), the teacher's score and the row's.
struct Entry {
    int col;
    float teacher, score;
};
template <typename T>
__device__ __forceinline__ Entry entry_of(const DistillArgs& p, int64_t row, int k) {
    if (k >= p.K) return {-1, 0.f, 0.f};
    const int v = p.index[row * p.K + k];
    if ((uint32_t)v >= (uint32_t)p.V) return {-1, 0.f, 0.f};
    return {v, p.teacher[row * p.K + k], (float)((const T*)p.scores)[row * p.ld + v]};
}

// A row's loss from its largest score and the logarithm of its sum.  mine: this thread's first entry, which was read before
// the row was (10393 x 2887 fp32: 39 -> 36 us).
template <typename T, int TPR>
__device__ __forceinline__ void finish(const DistillArgs& p, int64_t row, Soft z, Entry mine, int lane, float c, Soft* part,
                                       float* parts) {
    const float log_sum = __builtin_amdgcn_logf(z.sum) * kLn2, t = p.temperature;
    // the teacher's softmax: the largest score and the sum, 0 where there are no entries
    Soft q = {-INFINITY, 0.f};
    for (int k = lane; k < p.K; k += TPR) {
        const Entry e = k < TPR ? mine : entry_of<T>(p, row, k);
        if (e.col >= 0) q = join(q, {e.teacher, e.teacher == -INFINITY ? 0.f : 1.f}, c);
    }
    q = join_row<TPR>(q, c, part);
    float loss = 0.f;
    if (q.sum != 0.f) {
        const float log_q = __builtin_amdgcn_logf(q.sum) * kLn2, inv = 1.f / t;
        for (int k = lane; k < p.K; k += TPR) {
            const Entry e = k < TPR ? mine : entry_of<T>(p, row, k);
            if (e.col < 0) continue;
            const float lq = (e.teacher - q.top) * inv - log_q, w = __builtin_amdgcn_exp2f(lq * kLog2e);
            const float lp = e.score == -INFINITY ? -INFINITY : (e.score - z.top) * inv - log_sum;
            if (w != 0.f) loss += w * (lq - lp);
        }
    }
    loss = add_row<TPR>(loss, parts);
    if (lane == 0) {
        p.loss[row] = loss * (t * t);
        const f32x4 stat = {z.top, log_sum, q.sum == 0.f ? 0.f : q.top, q.sum == 0.f ? INFINITY : __builtin_amdgcn_logf(q.sum) * kLn2};
        *reinterpret_cast<f32x4_any*>(p.stat + 4 * row) = stat;
    }
}

template <typename TT, int TPR>
__global__ __launch_bounds__(kThreads) void distill_fwd_kernel(DistillArgs p) {
    typedef typename TT::type T;
    __shared__ Soft part[kThreads / 64];
    __shared__ float parts[kThreads / 64];
    const int lane = threadIdx.x % TPR;
    const float c = kLog2e / p.temperature;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
    if (row >= p.N) return;  // whole waves, and whole workgroups where they meet
    const Entry mine = entry_of<T>(p, row, lane);
    const Soft z = join_row<TPR>(soft_of<T, TPR>((const T*)p.scores + row * p.ld, 0, p.V, lane, c), c, part);
    finish<T, TPR>(p, row, z, mine, lane, c, part, parts);
}

// Split rows: a part of a row to a workgroup, and the rest of the work when all are there.
template <typename TT>
__global__ __launch_bounds__(kThreads) void distill_part_kernel(DistillArgs p, int splits, int width) {
    typedef typename TT::type T;
    __shared__ Soft part[kThreads / 64];
    const int64_t row = blockIdx.x / splits;
    const int n = blockIdx.x % splits, from = n * width, to = min(p.V, from + width);
    const float c = kLog2e / p.temperature;
    const Soft z =
        join_row<kThreads>(soft_of<T, kThreads>((const T*)p.scores + row * p.ld, from, to, threadIdx.x, c), c, part);
    if (threadIdx.x == 0) {
        p.partial[2 * blockIdx.x] = z.top;
        p.partial[2 * blockIdx.x + 1] = z.sum;
    }
}
template <typename TT>
__global__ __launch_bounds__(64) void distill_finish_kernel(DistillArgs p, int splits) {
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x;
    const float c = kLog2e / p.temperature;
    const Entry mine = entry_of<typename TT::type>(p, row, lane);
    Soft z = {-INFINITY, 0.f};
    for (int i = lane; i < splits; i += 64)
        z = join(z, {p.partial[2 * (row * splits + i)], p.partial[2 * (row * splits + i) + 1]}, c);
    finish<typename TT::type, 64>(p, row, join64(z, c), mine, lane, c, nullptr, nullptr);
}

// dz over columns [from, to) of a row by TPR threads, and the entries among them.  The first columns are on their way
// while the entries are looked at.  STREAM: scores past what the last cache holds (256 MB), which would only push each other out of it
// (8192 x 32768 bf16: 225 -> 213 us, and the next forward 158 -> 123).
template <typename TT, int TPR, bool STREAM>
__global__ __launch_bounds__(kThreads) void distill_bwd_kernel(DistillArgs p, int splits, int width) {
    typedef typename TT::type T;
    constexpr int PER = kThreads / TPR, AHEAD = 4;
    extern __shared__ __align__(16) float entries[];  // for each row: the entries' columns and q, in fours
    const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int64_t row = (int64_t)(blockIdx.x / splits) * PER + sub;
    const int from = (int)(blockIdx.x % splits) * width, to = min(p.V, from + width);
    if (row >= p.N) return;  // whole waves, and whole workgroups where they meet
    const int fours = (p.K + 3) / 4 * 4;
    int* col = (int*)entries + sub * 2 * fours;
    float* q = (float*)col + fours;
    const T* z = (const T*)p.scores + row * p.ld;
    T* dz = (T*)p.dscores + row * p.ldd;
    const int32_t* index = p.index + row * p.K;
    typename Pack8<T>::V v[AHEAD];
    int at = from + lane * kVec;
    const auto load = [&](int first) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
            if (first + a * TPR * kVec < to) v[a] = load_vec<T, STREAM>(z, first + a * TPR * kVec, to);
    };
    load(at);
    const f32x4 stat = *reinterpret_cast<const f32x4_any*>(p.stat + 4 * row);
    const float c = kLog2e / p.temperature, top = stat[0] == -INFINITY ? 0.f : stat[0], log_sum = stat[1] * kLog2e;
    const bool nothing = stat[0] == -INFINITY;   // no column is there: p = 0
    const float k = stat[3] == INFINITY ? 0.f : p.dloss[row] * p.temperature;  // no entries: no gradient
    const auto p_of = [&](float s) {
        return nothing ? 0.f : __builtin_amdgcn_exp2f(__builtin_fmaf(s - top, c, -log_sum));
    };
    // this thread's first entry; the score is read before anything of the row is written, which may be in its place
    const bool in_place = p.scores == p.dscores;
    const int mine = lane < p.K ? index[lane] : -1;
    float score = 0.f;
    if (mine >= from && mine < to) score = (float)z[mine];
    for (int i = lane; i < fours; i += TPR) {
        const int n = i < p.K ? index[i] : -1;
        const bool there = (uint32_t)n < (uint32_t)p.V;
        col[i] = there ? n : -1;
        q[i] = !there || stat[3] == INFINITY ? 0.f
                                             : __builtin_amdgcn_exp2f(__builtin_fmaf(p.teacher[row * p.K + i] - stat[2], c, -stat[3] * kLog2e));
    }
    float more[kMostEntries / TPR - 1];  // with more entries than threads: the other ones' scores
#pragma unroll
    for (int r = 1; r < kMostEntries / TPR; ++r) {
        more[r - 1] = 0.f;
        const int i = lane + r * TPR, n = i < p.K ? index[i] : -1;
        if (n >= from && n < to) more[r - 1] = (float)z[n];
    }
    if (in_place) row_sync<TPR>();
    while (at < to) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const int cl = at + a * TPR * kVec;
            if (cl >= to) continue;
            float f[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) f[i] = k == 0.f ? 0.f : p_of((float)v[a][i]) * k;
            store_vec<T, STREAM>(dz, cl, to, f);
        }
        at += AHEAD * TPR * kVec;
        load(at);
    }
    row_sync<TPR>();  // the row is written: its entries' columns come after
#pragma unroll
    for (int r = 0; r < kMostEntries / TPR; ++r) {
        const int i = lane + r * TPR;
        if (i >= p.K) break;
        const int n = col[i];
        if (n < from || n >= to) continue;
        f32x4 all = {0.f, 0.f, 0.f, 0.f};  // a column may be listed more than once: the same value from each
#pragma unroll 4
        for (int j = 0; j < fours; j += 4) {
            const i32x4 cs = *reinterpret_cast<const i32x4*>(col + j);
            const f32x4 qs = *reinterpret_cast<const f32x4*>(q + j);
#pragma unroll
            for (int e = 0; e < 4; ++e) all[e] += cs[e] == n ? qs[e] : 0.f;
        }
        dz[n] = (T)(k == 0.f ? 0.f : (p_of(r == 0 ? score : more[r > 0 ? r - 1 : 0]) - ((all[0] + all[1]) + (all[2] + all[3]))) * k);
    }
}

struct DistillPlan {
    int splits, width;
};
// Rows over workgroups while there are fewer than 4 for each CU, a part of at least 4096 columns; `from` is the
// row's length from which that pays.  The backward takes no launch more for it: always (8 x 9210 bf16: 6.0 -> 5.3 us).  The forward
// takes one: 64 x 16384 6.6 us whole and 7.2 in parts, 64 x 32768 8.7 and 7.5.
DistillPlan plan_of(int N, int V, int from) {
    DistillPlan d{1, V};
    if (N <= 0 || V <= from) return d;
    const int64_t splits = std::min<int64_t>(1024 / N, V / 4096);
    if (splits <= 1) return d;
    d.width = (int)(ceil_div(ceil_div(V, splits), 64) * 64);
    d.splits = (int)ceil_div(V, d.width);
    return d;
}
DistillPlan forward_plan(int N, int V) { return plan_of(N, V, 24576); }
DistillPlan backward_plan(int N, int V) { return plan_of(N, V, kShortRow); }

template <typename TT>
hipError_t fwd(const DistillArgs& a, hipStream_t stream) {
    const DistillPlan d = forward_plan(a.N, a.V);
    (void)hipGetLastError();  // an error that an earlier call left unread is not this one's
    if (d.splits > 1) {
        distill_part_kernel<TT><<<(unsigned)(a.N * d.splits), kThreads, 0, stream>>>(a, d.splits, d.width);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        distill_finish_kernel<TT><<<(unsigned)a.N, 64, 0, stream>>>(a, d.splits);
    } else if (a.V <= (a.N < kFewRows ? kShortFew : kShortForward)) {
        distill_fwd_kernel<TT, 64><<<(unsigned)ceil_div(a.N, kThreads / 64), kThreads, 0, stream>>>(a);
    } else {
        distill_fwd_kernel<TT, kThreads><<<(unsigned)a.N, kThreads, 0, stream>>>(a);
    }
    return hipGetLastError();
}
template <typename TT>
hipError_t bwd(const DistillArgs& a, hipStream_t stream) {
    const DistillPlan d = backward_plan(a.N, a.V);
    (void)hipGetLastError();
    const size_t lds = (size_t)((a.K + 3) / 4 * 4) * 8;
    const size_t bytes = (size_t)a.N * a.V * (a.dtype == MAXSIM_F32 ? 4 : 2);
    if (a.V <= kShortRow)
        distill_bwd_kernel<TT, 64, false>
            <<<(unsigned)ceil_div(a.N, kThreads / 64), kThreads, lds * (kThreads / 64), stream>>>(a, 1, a.V);
    else if (bytes <= kLastCache)
        distill_bwd_kernel<TT, kThreads, false><<<(unsigned)(a.N * d.splits), kThreads, lds, stream>>>(a, d.splits, d.width);
    else
        distill_bwd_kernel<TT, kThreads, true><<<(unsigned)(a.N * d.splits), kThreads, lds, stream>>>(a, d.splits, d.width);
    return hipGetLastError();
}

}  // namespace

size_t distill_workspace_bytes(int N, int V) {
    const DistillPlan d = forward_plan(N, V);
    return d.splits > 1 ? (size_t)N * d.splits * 2 * sizeof(float) : 0;
}
hipError_t launch_distill_fwd(const DistillArgs& a, hipStream_t stream) {
    return a.dtype == MAXSIM_F32 ? fwd<F32>(a, stream) : a.dtype == MAXSIM_BF16 ? fwd<BF16>(a, stream) : fwd<F16>(a, stream);
}
hipError_t launch_distill_bwd(const DistillArgs& a, hipStream_t stream) {
    return a.dtype == MAXSIM_F32 ? bwd<F32>(a, stream) : a.dtype == MAXSIM_BF16 ? bwd<BF16>(a, stream) : bwd<F16>(a, stream);
}

}  // namespace maxsim
