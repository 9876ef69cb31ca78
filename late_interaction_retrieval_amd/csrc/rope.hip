// rope.hip -- rotary positions for gfx950 (MI355X).
//
//     (u, w) -> scale * (u cos a - w sin a, w cos a + u sin a),   a = position * inv_freq[pair]
//
// Bound by HBM: a read and a write of each value.  A workgroup takes some tokens: it forms their
// sines and cosines once, into LDS (an angle serves all heads), and then streams their heads' rows, 8 columns of a
// row (8 of either half) to a thread.
//
// The angle is a product in fp64 in turns, whose whole part is dropped before it becomes fp32: at position 2^20 a
// product in fp32 would be off by up to 0.06 radians.
//
// Measured, the kernel alone: 32768 tokens, 20 heads of 128, bf16 63.5 us, 336 MB at 5.3 TB/s (a copy of 1 GiB: 5.1);
// 5003 tokens, 7 heads of 80, 48 turned, fp32 6.3 - 7.2, 22 MB in cache; 8 next tokens 3.4, a launch.
#include <algorithm>

#include "encoder_dev.h"
#include "layers.h"

namespace maxsim {
namespace {

constexpr int kThreads = 256;
constexpr int kTable = 2048;  // angles of a workgroup at most, 16 KB of LDS

struct RopePlan {
    int tokens;     // of a workgroup
    int heads;      // of a workgroup; the others in further ones
    int splits;     // of the heads
    int turn_units, units;  // pieces of a row: of the turned columns, and in all
    int pitch;      // angles of a token in the table
};

// 8 values of a row, read past the caches (STREAM) or not.
template <typename T, bool STREAM>
__device__ __forceinline__ typename Pack8<T>::V load_vec(const T* row, int c, int n) {
    if (STREAM && c + kVec <= n) return __builtin_nontemporal_load(reinterpret_cast<const typename Pack8<T>::V*>(row + c));
    return load8<T>(row, c, n);
}

// STREAM: rows that the last cache (256 MB) does not hold beside the result, which is what will be read next (335 MB in all:
// 69 -> 63.5 us; 22 MB in cache took 9.2 us for 6.8).
template <typename TT, bool STREAM>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs p, RopePlan plan) {
    typedef typename TT::type T;
    __shared__ __align__(16) float cosine[kTable], sine[kTable];
    const int half = p.rotary / 2;
    const int t0 = (int)(blockIdx.x / plan.splits) * plan.tokens;  // B * L < 2^25
    const int h0 = (int)(blockIdx.x % plan.splits) * plan.heads;
    const int tokens = min(plan.tokens, p.B * p.L - t0), heads = min(plan.heads, p.H - h0);
    for (int e = threadIdx.x; e < tokens * plan.pitch; e += kThreads) {
        const int k = e / plan.pitch, i = e - k * plan.pitch;
        const int t = t0 + k, b = t / p.L, l = t - b * p.L;
        const double at = p.positions ? (double)p.positions[t] : (double)l + (p.offsets ? (double)p.offsets[b] : 0.0);
        const double turns = i < half ? at * (p.inv_freq[i] * 0.15915494309189533577) : 0.0;
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        cosine[e] = c * p.scale;
        sine[e] = (p.inverse ? -s : s) * p.scale;
    }
    __syncthreads();
    const int rows = kThreads / plan.units, unit = (int)threadIdx.x % plan.units;
    if ((int)threadIdx.x >= rows * plan.units) return;
    const bool turned = unit < plan.turn_units, in_place = p.x.data == p.y.data;
    if (!turned && in_place) return;
    const int c = (turned ? unit : unit - plan.turn_units) * kVec;
    int k = 0, h = (int)threadIdx.x / plan.units;
    while (h >= heads) h -= heads, ++k;
    for (; k < tokens;) {
        const int t = t0 + k, b = t / p.L, l = t - b * p.L;
        const T* x = (const T*)p.x.data + b * p.x.batch + l * p.x.token + (int64_t)(h0 + h) * p.x.head;
        T* y = (T*)p.y.data + b * p.y.batch + l * p.y.token + (int64_t)(h0 + h) * p.y.head;
        const float *cs = cosine + k * plan.pitch, *sn = sine + k * plan.pitch;
        if (!turned) {
            put8<T>(y + p.rotary, c, p.D - p.rotary, load_vec<T, STREAM>(x + p.rotary, c, p.D - p.rotary));
        } else if (p.interleaved) {
            const auto v = load_vec<T, STREAM>(x, c, p.rotary);
            float f[kVec];
#pragma unroll
            for (int i = 0; i < kVec; i += 2) {
                const float u = (float)v[i], w = (float)v[i + 1], co = cs[(c + i) >> 1], si = sn[(c + i) >> 1];
                f[i] = __builtin_fmaf(u, co, -(w * si));
                f[i + 1] = __builtin_fmaf(w, co, u * si);
            }
            store8<T>(y, c, p.rotary, f);
        } else {
            const auto a = load_vec<T, STREAM>(x, c, half), d = load_vec<T, STREAM>(x + half, c, half);
            float f[kVec], g[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const float u = (float)a[i], w = (float)d[i], co = cs[c + i], si = sn[c + i];
                f[i] = __builtin_fmaf(u, co, -(w * si));
                g[i] = __builtin_fmaf(w, co, u * si);
            }
            store8<T>(y, c, half, f);
            store8<T>(y + half, c, half, g);
        }
        h += rows;
        while (h >= heads) h -= heads, ++k;
    }
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream) {
    RopePlan plan;
    const int half = a.rotary / 2, rest = a.D - a.rotary;
    plan.turn_units = a.interleaved ? (int)ceil_div(a.rotary, kVec) : (int)ceil_div(half, kVec);
    plan.units = plan.turn_units + (int)ceil_div(rest, kVec);
    plan.pitch = (int)ceil_div(half, kVec) * kVec;
    const int64_t all = (int64_t)a.B * a.L;
    // 4 tokens to a workgroup (32768 tokens x 20 heads of 128: 16 took 82 us, 8 73, 4 69, 2 76), fewer where that leaves
    // CUs without work; then fewer heads
    plan.tokens = (int)std::max<int64_t>(1, std::min<int64_t>({kTable / plan.pitch, 4, all / 1024}));
    const int64_t groups = ceil_div(all, plan.tokens);
    const int per_pass = std::max(1, kThreads / plan.units);
    plan.splits = (int)std::max<int64_t>(1, std::min<int64_t>(ceil_div(a.H, per_pass), 1024 / std::max<int64_t>(1, groups)));
    plan.heads = (int)ceil_div(a.H, plan.splits);
    plan.splits = (int)ceil_div(a.H, plan.heads);
    const unsigned blocks = (unsigned)(groups * plan.splits);
    const int64_t bytes = 2 * all * a.H * a.D * (a.dtype == MAXSIM_F32 ? 4 : 2);
    const bool stream_past = bytes > (int64_t)256 << 20 && a.x.data != a.y.data;
    const auto kernel = a.dtype == MAXSIM_F32    ? (stream_past ? rope_kernel<F32, true> : rope_kernel<F32, false>)
                        : a.dtype == MAXSIM_BF16 ? (stream_past ? rope_kernel<BF16, true> : rope_kernel<BF16, false>)
                                                 : (stream_past ? rope_kernel<F16, true> : rope_kernel<F16, false>);
    (void)hipGetLastError();  // an error that an earlier call left unread is not this one's
    kernel<<<blocks, kThreads, 0, stream>>>(a, plan);
    return hipGetLastError();
}

}  // namespace maxsim
