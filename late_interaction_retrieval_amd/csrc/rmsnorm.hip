// rmsnorm.hip -- RMS norm of rows with the residual's addition, 16-bit or
// 8-bit output, and its backward, for gfx950 (MI355X).
//
//     h = x + residual;  r = 1 / sqrt(mean(h^2) + eps);  y = h r w
//     g = dy w;  xh = h r;  dx = r (g - xh mean(g xh)) + dsum;  dw = sum_rows dy xh
//
// Both are bound by HBM (a few operations per byte), so the design is one pass:
// a row is read once into the registers of 16 lanes to a whole workgroup, its
// sum goes over the lanes by DPP (and over waves through LDS), and everything
// that depends on it is formed from those registers.  A lane holds vectors of
// 8 neighbouring columns, so 16 lanes hold exactly one block of 128 columns and
// an e4m3 block's scale is a 16-lane maximum.
//
// Measured (bf16, the times of the kernels alone): forward 32768 x 2048 with a
// residual, its sum and e4m3 out 92-100 us, 472 MB at 4.7-5.1 TB/s; backward 16384 x
// 2048 with a gradient of the sum 54 us + 5 us for the gains, 268 MB at 4.6
// TB/s; a copy of 1 GiB reaches 5.2.  32 x 128 fp32 to int8 2.7 us, a launch.  1003 x 769
// fp16 backward 7.7 us, inputs in cache 6.1: dx alone is 4.1 there, as for 64 rows, the rest
// the dweight workgroups' way over the rows.
#include <algorithm>
#include <type_traits>

#include "encoder_dev.h"

namespace maxsim {
namespace {

// TPR threads hold a row, NV vectors of 8 columns each: column
// (v * TPR + lane) * 8.  Rows of 16 or 64 threads share a workgroup of 256;
// wider rows (TPR 0 here) have one of as many waves as their columns ask for.
constexpr int kWide = 0;
constexpr int kMostWaves = 8;  // of a row: leaves a thread 256 registers
template <int TPR>
struct Rows {
    static constexpr int threads = TPR == kWide ? 64 * kMostWaves : 256;
    static constexpr int per_group = TPR == kWide ? 1 : 256 / TPR;
    __device__ static __forceinline__ int wide() { return TPR == kWide ? (int)blockDim.x : TPR; }
};

// Sum (or maximum) over a row's threads, the same in each of them.  The waves of
// a wide row meet in `part` (one word each), which each call uses anew.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
    if constexpr (TPR == 16) return sum16(v);
    v = sum64(v);
    if constexpr (TPR == kWide) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = part[0];
        for (int w = 1; w < (int)blockDim.x >> 6; ++w) v += part[w];
    }
    return v;
}
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* part) {
    if constexpr (TPR == 16) return max16(v);
    v = max64(v);
    if constexpr (TPR == kWide) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = part[0];
        for (int w = 1; w < (int)blockDim.x >> 6; ++w) v = umax(v, part[w]);
    }
    return v;
}

// The gain of 8 columns in fp32.
template <typename T>
__device__ __forceinline__ void load_gain(const void* weight, int f32, int c, int n, float* w) {
    if (weight == nullptr) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) w[i] = 1.f;
    } else if (f32) {
        auto v = near8<float>((const float*)weight, c, n);
        fit8<float>(v, c, n);
#pragma unroll
        for (int i = 0; i < kVec; ++i) w[i] = v[i];
    } else {
        auto v = near8<T>((const T*)weight, c, n);
        fit8<T>(v, c, n);
#pragma unroll
        for (int i = 0; i < kVec; ++i) w[i] = (float)v[i];
    }
}

template <typename TT, int TPR, int NV>
__global__ __launch_bounds__(Rows<TPR>::threads) void rmsnorm_fwd_kernel(NormArgs p) {
    typedef typename TT::type T;
    constexpr int PER = Rows<TPR>::per_group;
    constexpr bool TOGETHER = NV <= 2;
    __shared__ float part_sum[2][kMostWaves];
    __shared__ uint32_t part_max[2][kMostWaves];
    const int tpr = Rows<TPR>::wide();
    const int lane = TPR == kWide ? threadIdx.x : threadIdx.x % tpr;
    int turn = 0;  // two sets of words in LDS in turn: a wave may be a row ahead of another's read
    // a row that all its threads leave together: rows of up to 64 threads meet no barrier
    for (int64_t row = (int64_t)blockIdx.x * PER + (TPR == kWide ? 0 : threadIdx.x / tpr); row < p.R;
         row += (int64_t)gridDim.x * PER, turn ^= 1) {
        const T* x = (const T*)p.x + row * p.ldx;
        float h[NV][kVec];
        typename Pack8<T>::V in[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) in[v] = near8<T, TOGETHER>(x, (v * tpr + lane) * kVec, p.H);
        if (p.residual != nullptr) {
            const T* res = (const T*)p.residual + row * p.ldr;
            typename Pack8<T>::V also[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v) also[v] = near8<T, TOGETHER>(res, (v * tpr + lane) * kVec, p.H);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                fit8<T, TOGETHER>(in[v], (v * tpr + lane) * kVec, p.H);
                fit8<T, TOGETHER>(also[v], (v * tpr + lane) * kVec, p.H);
#pragma unroll
                for (int i = 0; i < kVec; ++i) h[v][i] = (float)in[v][i] + (float)also[v][i];
            }
        } else {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                fit8<T, TOGETHER>(in[v], (v * tpr + lane) * kVec, p.H);
#pragma unroll
                for (int i = 0; i < kVec; ++i) h[v][i] = (float)in[v][i];
            }
        }
        float ss = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < kVec; ++i) ss = __builtin_fmaf(h[v][i], h[v][i], ss);
        if (p.sum != nullptr) {
            T* sum = (T*)p.sum + row * p.lds;
#pragma unroll
            for (int v = 0; v < NV; ++v) store8<T>(sum, (v * tpr + lane) * kVec, p.H, h[v]);
        }
        ss = row_sum<TPR>(ss, part_sum[turn]);
        const float r = 1.f / __builtin_sqrtf(ss / (float)p.H + p.eps);
        if (p.rstd != nullptr && lane == 0) p.rstd[row] = r;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float w[kVec];
            load_gain<T>(p.weight, p.weight_f32, (v * tpr + lane) * kVec, p.H, w);
#pragma unroll
            for (int i = 0; i < kVec; ++i) h[v][i] = h[v][i] * r * w[i];
        }
        if (p.out_dtype == MAXSIM_E4M3) {
            const int64_t blocks = (p.H + kQBlock - 1) / kQBlock;
            uint8_t* y = (uint8_t*)p.y + row * p.ldy;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < kVec; ++i) top = umax(top, mag(h[v][i]));
                const Scale k = block_scale(max16(top), 448.f);
                const int c = (v * tpr + lane) * kVec;
                if (c < p.H) {
                    store8_bytes(y, c, p.H, to_e4m3(h[v], k));
                    if (c % kQBlock == 0) p.scale[row * blocks + c / kQBlock] = k.s;
                }
            }
        } else if (p.out_dtype == MAXSIM_I8) {
            uint32_t top = 0;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < kVec; ++i) top = umax(top, mag(h[v][i]));
            const Scale k = block_scale(row_max<TPR>(top, part_max[turn]), 127.f);
            if (lane == 0) p.scale[row] = k.s;
            uint8_t* y = (uint8_t*)p.y + row * p.ldy;
#pragma unroll
            for (int v = 0; v < NV; ++v) store8_bytes(y, (v * tpr + lane) * kVec, p.H, to_i8(h[v], k));
        } else if (p.out_dtype == MAXSIM_F32) {
            float* y = (float*)p.y + row * p.ldy;
#pragma unroll
            for (int v = 0; v < NV; ++v) store8<float>(y, (v * tpr + lane) * kVec, p.H, h[v]);
        } else if (p.out_dtype == MAXSIM_BF16) {
            __bf16* y = (__bf16*)p.y + row * p.ldy;
#pragma unroll
            for (int v = 0; v < NV; ++v) store8<__bf16>(y, (v * tpr + lane) * kVec, p.H, h[v]);
        } else {
            _Float16* y = (_Float16*)p.y + row * p.ldy;
#pragma unroll
            for (int v = 0; v < NV; ++v) store8<_Float16>(y, (v * tpr + lane) * kVec, p.H, h[v]);
        }
    }
}

// Rows in turn, a workgroup's every gridDim-th; each thread keeps its columns'
// share of dw in registers over all of them and the workgroup writes one
// partial row at the end.
template <typename TT, int TPR, int NV>
__global__ __launch_bounds__(Rows<TPR>::threads) void rmsnorm_bwd_kernel(NormBwdArgs p) {
    typedef typename TT::type T;
    constexpr int PER = Rows<TPR>::per_group;
    constexpr bool TOGETHER = NV <= 4;
    __shared__ float part[2][kMostWaves];
    __shared__ float share[PER][PER > 1 ? TPR * kVec : 1];
    const int tpr = Rows<TPR>::wide();
    const int lane = TPR == kWide ? threadIdx.x : threadIdx.x % tpr;
    const int sub = TPR == kWide ? 0 : threadIdx.x / tpr;
    // the gain stays in registers, or, where a row takes too many, comes from L2 for each row
    constexpr bool KEEP = NV <= 4;
    float w[KEEP ? NV : 1][kVec], dw[NV][kVec];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if constexpr (KEEP) load_gain<T>(p.weight, p.weight_f32, (v * tpr + lane) * kVec, p.H, w[v]);
#pragma unroll
        for (int i = 0; i < kVec; ++i) dw[v][i] = 0.f;
    }
    const float inv_h = 1.f / (float)p.H;
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * PER + sub; row < p.R; row += (int64_t)gridDim.x * PER, turn ^= 1) {
        const T* dyr = (const T*)p.dy + row * p.lddy;
        const T* hr = (const T*)p.h + row * p.ldh;
        typename Pack8<T>::V dy[NV], h[NV], ds[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            dy[v] = near8<T, TOGETHER>(dyr, (v * tpr + lane) * kVec, p.H);
            h[v] = near8<T, TOGETHER>(hr, (v * tpr + lane) * kVec, p.H);
        }
        if (NV < 8 && p.dsum != nullptr) {  // 8 vectors have no registers for it before dx
            const T* dsr = (const T*)p.dsum + row * p.ldds;
#pragma unroll
            for (int v = 0; v < NV; ++v) ds[v] = near8<T, TOGETHER>(dsr, (v * tpr + lane) * kVec, p.H);
        }
        const float r = p.rstd[row];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int at = (v * tpr + lane) * kVec;
            fit8<T, TOGETHER>(dy[v], at, p.H);
            fit8<T, TOGETHER>(h[v], at, p.H);
            if (NV < 8 && p.dsum != nullptr) fit8<T, TOGETHER>(ds[v], at, p.H);
        }
        float c = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if constexpr (!KEEP) load_gain<T>(p.weight, p.weight_f32, (v * tpr + lane) * kVec, p.H, w[0]);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const float t = (float)dy[v][i] * ((float)h[v][i] * r);
                dw[v][i] += t;
                c = __builtin_fmaf(t, w[KEEP ? v : 0][i], c);
            }
        }
        // two words of LDS in turn: a wave may be a row ahead of another's read
        c = row_sum<TPR>(c, part[turn]) * inv_h;
        T* dxr = (T*)p.dx + row * p.lddx;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float dx[kVec];
            if constexpr (!KEEP) load_gain<T>(p.weight, p.weight_f32, (v * tpr + lane) * kVec, p.H, w[0]);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const float g = (float)dy[v][i] * w[KEEP ? v : 0][i];
                dx[i] = r * (g - (float)h[v][i] * r * c);
            }
            if (p.dsum != nullptr) {
                if constexpr (NV >= 8) {
                    ds[v] = near8<T, TOGETHER>((const T*)p.dsum + row * p.ldds, (v * tpr + lane) * kVec, p.H);
                    fit8<T, TOGETHER>(ds[v], (v * tpr + lane) * kVec, p.H);
                }
#pragma unroll
                for (int i = 0; i < kVec; ++i) dx[i] += (float)ds[v][i];
            }
            store8<T>(dxr, (v * tpr + lane) * kVec, p.H, dx);
        }
    }
    if (p.dweight == nullptr) return;
    float* out = p.partial + (int64_t)blockIdx.x * p.H;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * tpr + lane) * kVec;
        if constexpr (PER > 1) {  // the workgroup's rows, added in order
            if (v > 0) __syncthreads();
#pragma unroll
            for (int i = 0; i < kVec; ++i) share[sub][lane * kVec + i] = dw[v][i];
            __syncthreads();
            for (int k = threadIdx.x; k < TPR * kVec; k += Rows<TPR>::threads) {
                float s = share[0][k];
                for (int q = 1; q < PER; ++q) s += share[q][k];
                if (v * TPR * kVec + k < p.H) out[v * TPR * kVec + k] = s;
            }
        } else {
            store8<float>(out, c, p.H, dw[v]);
        }
    }
}

// dweight = the partial rows, added in a fixed order: a workgroup takes 32
// columns (one line of each row), its 32 runs of 32 threads every 32nd row, so
// that a few hundred rows are on their way at once.
constexpr int kReduceCols = 32, kReduceRuns = 32;
__global__ __launch_bounds__(kReduceCols * kReduceRuns) void rmsnorm_dweight_kernel(const float* partial, int groups,
                                                                                   int H, float* dw) {
    __shared__ float run[kReduceRuns][kReduceCols];
    const int col = threadIdx.x % kReduceCols, part = threadIdx.x / kReduceCols;
    const int c = blockIdx.x * kReduceCols + col;
    float s = 0.f;
    if (c < H) {
#pragma unroll 8
        for (int g = part; g < groups; g += kReduceRuns) s += partial[(int64_t)g * H + c];
    }
    run[part][col] = s;
    __syncthreads();
    if (part == 0 && c < H) {
#pragma unroll
        for (int q = 1; q < kReduceRuns; ++q) s += run[q][col];
        dw[c] = s;
    }
}

// Few values: dx and dweight in one launch.  dweight does not need the rows'
// means, so workgroups past those of the rows take 32 columns each over all
// rows (read a second time, from L2) and no partial sums go to memory.
constexpr int kSmallThreads = 1024;
template <typename TT, int TPR, int NV>
__global__ __launch_bounds__(kSmallThreads) void rmsnorm_bwd_small_kernel(NormBwdArgs p, int row_groups) {
    typedef typename TT::type T;
    constexpr int PER = kSmallThreads / TPR;
    __shared__ float run[kReduceRuns][kReduceCols];
    if ((int)blockIdx.x >= row_groups) {
        const int col = threadIdx.x % kReduceCols, part = threadIdx.x / kReduceCols;
        const int c = ((int)blockIdx.x - row_groups) * kReduceCols + col;
        float s = 0.f;
        if (c < p.H) {
#pragma unroll 8
            for (int r = part; r < p.R; r += kReduceRuns)
                s += (float)((const T*)p.dy)[r * p.lddy + c] * ((float)((const T*)p.h)[r * p.ldh + c] * p.rstd[r]);
        }
        run[part][col] = s;
        __syncthreads();
        if (part == 0 && c < p.H) {
#pragma unroll
            for (int q = 1; q < kReduceRuns; ++q) s += run[q][col];
            p.dweight[c] = s;
        }
        return;
    }
    const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int64_t row = (int64_t)blockIdx.x * PER + sub;
    const bool on = row < p.R;
    typename Pack8<T>::V dy[NV], h[NV];
    float w[NV][kVec];
    float c = 0.f, r = 0.f;
    if (on) {
        r = p.rstd[row];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            dy[v] = load8<T>((const T*)p.dy + row * p.lddy, (v * TPR + lane) * kVec, p.H);
            h[v] = load8<T>((const T*)p.h + row * p.ldh, (v * TPR + lane) * kVec, p.H);
            load_gain<T>(p.weight, p.weight_f32, (v * TPR + lane) * kVec, p.H, w[v]);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < kVec; ++i) c = __builtin_fmaf((float)dy[v][i] * ((float)h[v][i] * r), w[v][i], c);
    }
    if constexpr (TPR == 16) {
        c = sum16(c);
    } else {
        c = sum64(c);
        if constexpr (TPR > 64) {  // the row's waves, in order
            constexpr int W = TPR / 64;
            if ((threadIdx.x & 63) == 0) run[0][threadIdx.x >> 6] = c;
            __syncthreads();
            c = run[0][sub * W];
#pragma unroll
            for (int q = 1; q < W; ++q) c += run[0][sub * W + q];
        }
    }
    if (!on) return;
    c *= 1.f / (float)p.H;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        float dx[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) dx[i] = r * ((float)dy[v][i] * w[v][i] - (float)h[v][i] * r * c);
        if (p.dsum != nullptr) {
            const auto ds = load8<T>((const T*)p.dsum + row * p.ldds, (v * TPR + lane) * kVec, p.H);
#pragma unroll
            for (int i = 0; i < kVec; ++i) dx[i] += (float)ds[i];
        }
        store8<T>((T*)p.dx + row * p.lddx, (v * TPR + lane) * kVec, p.H, dx);
    }
}

// Threads to a row: 16 or 64 for narrow ones; else as many waves as its columns
// fill with one vector a thread, two past 2560 columns, and so on.  Go is
// called with (threads to a row or kWide, vectors a thread, threads of a workgroup).
template <typename Go>
void by_width(int H, Go&& go) {
    typedef std::integral_constant<int, kWide> wide;
    const auto waves = [&](int nv) { return 64 * (int)ceil_div(H, 64 * kVec * nv); };
    if (H <= 128) return go(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{}, 256);
    if (H <= 512) return go(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{}, 256);
    if (H <= 1024) return go(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{}, 256);
    if (H <= 2560) return go(wide{}, std::integral_constant<int, 1>{}, waves(1));
    if (H <= 8192) return go(wide{}, std::integral_constant<int, 2>{}, waves(2));
    if (H <= 16384) return go(wide{}, std::integral_constant<int, 4>{}, waves(4));
    return go(wide{}, std::integral_constant<int, 8>{}, waves(8));
}
// The one-launch backward has 1024 threads whatever the width.
template <typename Go>
void by_width_small(int H, Go&& go) {
    if (H <= 128) return go(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
    if (H <= 512) return go(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    if (H <= 1024) return go(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
    if (H <= 2048) return go(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
    if (H <= 4096) return go(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
    if (H <= 8192) return go(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
    if (H <= 16384) return go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
    return go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
}
template <typename F>
void by_type(int dtype, F&& go) {
    if (dtype == MAXSIM_F16) return go(F16{});
    if (dtype == MAXSIM_BF16) return go(BF16{});
    return go(F32{});
}

}  // namespace

hipError_t launch_rmsnorm_fwd(const NormArgs& a, hipStream_t stream) {
    by_type(a.dtype, [&](auto t) {
        by_width(a.H, [&](auto tpr, auto nv, int threads) {
            constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
            // at most 2^22 workgroups (a launch holds fewer than 2^32 threads); more rows go round
            const int grid = (int)std::min<int64_t>(ceil_div(a.R, Rows<TPR>::per_group), 1 << 22);
            rmsnorm_fwd_kernel<decltype(t), TPR, NV><<<grid, threads, 0, stream>>>(a);
        });
    });
    return hipGetLastError();
}

// Us in one launch and in two: 1 x 128 3.3, 5.4; 1003 x 769 7.9, 9.9; 200 x 2048
// 4.1, 7.9; 64 x 8192 6.3, 8.7; but 3000 x 128 11.7, 7.0; 1000 x 2048 10.9, 9.8.
bool norm_bwd_small(int R, int H) { return R <= 512 || (R <= 1024 && H <= 1024); }

int norm_bwd_groups(int R, int H) {
    // fewer than four rows each do not pay for a workgroup's partial row, once there are enough of them
    if (H > 1024) return std::min({R, 512, std::max(256, R / 4)});
    return (int)std::min<int64_t>(ceil_div(R, H <= 128 ? 16 : 4), 512);
}

hipError_t launch_rmsnorm_bwd(const NormBwdArgs& a, hipStream_t stream) {
    if (a.dweight != nullptr && a.R > 0 && norm_bwd_small(a.R, a.H)) {
        by_type(a.dtype, [&](auto t) {
            by_width_small(a.H, [&](auto tpr, auto nv) {
                constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
                const int rows = (int)ceil_div(a.R, kSmallThreads / TPR), cols = (int)ceil_div(a.H, kReduceCols);
                auto go = [&](int grid, int row_groups) {
                    rmsnorm_bwd_small_kernel<decltype(t), TPR, NV><<<grid, kSmallThreads, 0, stream>>>(a, row_groups);
                };
                if (a.dx == a.dy || a.dx == a.h) {  // in place: the columns read what the rows overwrite
                    go(cols, 0);
                    go(rows, rows);
                } else {
                    go(rows + cols, rows);
                }
            });
        });
        return hipGetLastError();
    }
    const int groups = norm_bwd_groups(a.R, a.H);
    if (groups > 0) {
        by_type(a.dtype, [&](auto t) {
            by_width(a.H, [&](auto tpr, auto nv, int threads) {
                constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
                rmsnorm_bwd_kernel<decltype(t), TPR, NV><<<groups, threads, 0, stream>>>(a);
            });
        });
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.dweight != nullptr)
        rmsnorm_dweight_kernel<<<(a.H + kReduceCols - 1) / kReduceCols, kReduceCols * kReduceRuns, 0, stream>>>(
            a.partial, groups, a.H, a.dweight);
    return hipGetLastError();
}

}  // namespace maxsim
