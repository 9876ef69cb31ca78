// attn_bwd.hip -- attention's backward for gfx950 (MI355X), in two launches without atomics.
//
//     P = exp(S - lse);  dP = dO V^T;  delta = rowsum(dO * out);  dS = P * (dP - delta)
//     dQ = scale dS K;  dK = scale dS^T Q;  dV = P^T dO
//
// The first goes over the keys for each tile of queries (dQ, and what the second needs of a row), the
// second over the queries for each tile of keys (dK and dV, summed over the query heads of the key
// head).  Each makes S and dP anew: 7 products of a pair for the 5 of a single pass, whose dQ would have to be
// added up in memory by all workgroups in an order of chance.
#include "attn_dev.h"

namespace maxsim {
namespace {

constexpr int kWaves = 4;
constexpr int kRows = 32 * kWaves;  // rows (dQ) or keys (dK, dV) of a workgroup, 32 of a wave
constexpr int kTile = 64;           // keys (dQ) or rows (dK, dV) of a tile

template <typename T>
constexpr bool is_f16() {
    return std::is_same<T, _Float16>::value;
}
// fp16 holds P and dS for their products only if they are brought into its range by powers of 2, which are
// exact: P (at most 1, 1 / keys where attention is flat) times 2^8; dS by the size of its row's dO.
constexpr float kLiftP = 8.f;  // log2
// The power of 2 that brings a row of dO with the largest magnitude `top` into [1, 2); 1 for a row of zeros.
__device__ __forceinline__ float lift_of(float top) {
    const int e = (int)((fbits(top) >> 23) & 255u);
    return e == 0 || e == 255 ? 1.f : __uint_as_float((uint32_t)(254 - e) << 23);
}

template <typename TT, int DP>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_dq_kernel(AttnArgs p, int tiles) {
    typedef typename TT::type T;
    typedef typename Vec8<T>::V V8;
    constexpr int KS = DP / 16, DB = DP / 32, BYTES = kTile * Tile<DP>::ROW;
    __shared__ __align__(16) uint8_t k_0[BYTES], v_0[BYTES], k_1[BYTES], v_1[BYTES];
    const maxsim_attn& a = p.a;
    int id = item_of_block();
    const int item = id, tile = tiles - 1 - id % tiles;
    id /= tiles;
    const int h = id % a.Hk, b = id / a.Hk;
    const Seq s = sequence(a, b);
    const int G = p.group, D = a.D, rows = s.lq * G;
    if (a.zero_rest)
        zero_rest<T>(p.dq, nullptr, 1, a.cu_q, a.B, a.rows_q, b, s.q0, s.lq, s.all_q, a.Hq, D, h * tiles + tile, a.Hk * tiles, item,
                     (int)gridDim.x);
    const int r0 = tile * kRows;
    if (r0 >= rows) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int shift = s.lk - s.lq;
    const Span span = span_of(a, s.lk, r0 / G + shift, (min(r0 + kRows, rows) - 1) / G + shift, kTile);
    const int wr = r0 + wave * 32;
    const int r = min(wr + (lane & 31), rows - 1), token = r / G, head = h * G + r % G;
    const bool mine = wr + (lane & 31) < rows;
    const bool packed = a.cu_q != nullptr;

    // the row's q and dO as operands, delta, and lse in powers of 2: a row that sees nothing has P = 0
    V8 q[KS], g[KS];
    const T* qr = first<T>(a.q, packed, b, s.q0, 0) + (int64_t)token * a.q.token + (int64_t)head * a.q.head;
    const T* gr = first<T>(p.dout, packed, b, s.q0, 0) + (int64_t)token * p.dout.token + (int64_t)head * p.dout.head;
    const T* orow = first<T>(a.out, packed, b, s.q0, 0) + (int64_t)token * a.out.token + (int64_t)head * a.out.head;
    const int64_t at = first_row(a, s, b) + token;
    const T* rest = rest_of<T>(p, at * a.Hq + head);
    float delta = 0.f, top = 0.f;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
        const int c = 16 * kk + 8 * (lane >> 5);
        q[kk] = row8<T>(qr, c, D);
        g[kk] = row8<T>(gr, c, D);
        const V8 o = row8<T>(orow, c, D);
        typename Pack8<T>::V off;
#pragma unroll
        for (int i = 0; i < 8; ++i) off[i] = (T)0.f;
        if (rest && c < D) off = *reinterpret_cast<const typename Pack8<T>::V*>(rest + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            delta = __builtin_fmaf((float)g[kk][i], (float)o[i] + (float)off[i], delta);
            if (is_f16<T>()) top = fmaxf(top, __builtin_fabsf((float)g[kk][i]));
        }
    }
    delta = swap_sum(delta);
    top = is_f16<T>() ? swap_max(top) : 0.f;
    float lse = p.lse[(at * a.Hq + head) * a.lse_step] * kLog2e;
    if (lse == -INFINITY) lse = INFINITY;
    if (mine && lane < 32) {
        float* stat = p.row_stat + (int64_t)head * p.rows + at;
        stat[0] = is_f16<T>() ? lse - kLiftP : lse;
        stat[p.rows * a.Hq] = delta;
        if (is_f16<T>()) stat[2 * p.rows * a.Hq] = top;
    }
    const float lift = is_f16<T>() ? lift_of(top) : 1.f;

    const int p_lo = min(wr, rows - 1) / G + shift, p_hi = min(wr + 31, rows - 1) / G + shift, pos = token + shift;
    const int lo = pos - a.left, hi = min(pos + a.right, s.lk - 1);
    const float c = a.scale * kLog2e;
    f32x16 acc[DB];
#pragma unroll
    for (int db = 0; db < DB; ++db) acc[db] = zero16();

    const T* ks = first<T>(a.k, a.cu_k != nullptr, b, s.k0, h);
    const T* vs = first<T>(a.v, a.cu_k != nullptr, b, s.k0, h);
    Loader<DP, kTile, kWaves> lk, lv;
    lk.init(wave, lane, a.k.token, D);
    lv.init(wave, lane, a.v.token, D);
    const auto load = [&](int t, uint8_t* kt, uint8_t* vt) {
        const int j = span.at(t, kTile);
        lk.load(ks + (int64_t)j * a.k.token, s.lk - j, a.k.token, D, kt, wave);
        lv.load(vs + (int64_t)j * a.v.token, s.lk - j, a.v.token, D, vt, wave);
    };
    const auto work = [&](int t, const uint8_t* kt, const uint8_t* vt) {
        const int j0 = span.at(t, kTile), end = span.end(t), j_last = j0 + kTile - 1;
        if (wr >= rows || j0 > p_hi + a.right || (j_last < p_lo - a.left && j0 >= a.sinks)) return;
        const bool whole = j_last < end && j_last <= min(p_lo + a.right, s.lk - 1) && (j0 >= p_hi - a.left || j_last < a.sinks);
#pragma unroll
        for (int nb = 0; nb < kTile / 32; ++nb) {
            const uint8_t *kb = kt + nb * 32 * Tile<DP>::ROW, *vb = vt + nb * 32 * Tile<DP>::ROW;
            f32x16 x = zero16(), dp = zero16();
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) x = mma<T>(rows_at<T, DP>(kb, lane, kk), q[kk], x);
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) dp = mma<T>(rows_at<T, DP>(vb, lane, kk), g[kk], dp);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], c, -lse));
            if (!whole) {
                const int j = j0 + 32 * nb + 4 * (lane >> 5);
                const int upto = min(hi, end - 1) - j, low = lo - j, sink = a.sinks - j;
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = slot(i) <= upto && (slot(i) >= low || slot(i) < sink) ? x[i] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] *= (dp[i] - delta) * lift;
#pragma unroll
            for (int t2 = 0; t2 < 2; ++t2) {
                const V8 ds = pack8<T>(x, 8 * t2);
#pragma unroll
                for (int db = 0; db < DB; ++db) acc[db] = mma<T>(cols_at<T, DP>(kb, lane, t2, db), ds, acc[db]);
            }
        }
    };
    if (span.tiles > 0) load(0, k_0, v_0);
    for (int t = 0; t < span.tiles; t += 2) {
        tile_ready();
        if (t + 1 < span.tiles) load(t + 1, k_1, v_1);
        work(t, k_0, v_0);
        if (t + 1 >= span.tiles) break;
        tile_ready();
        if (t + 2 < span.tiles) load(t + 2, k_0, v_0);
        work(t + 1, k_1, v_1);
    }
    T* out = first<T>(p.dq, packed, b, s.q0, 0) + (int64_t)token * p.dq.token + (int64_t)head * p.dq.head;
    store_row<T, DB>(out, mine, acc, a.scale / lift, lane, D);
}

// A workgroup's 128 keys of one key head; the query heads that share it one after the other, 64 tokens at a
// time.  The queries are the rows of S here, the keys its columns, so P and dS are the B operands of dV^T = dO^T P and
// dK^T = Q^T dS, and a lane's two result rows stay in registers.
template <typename TT, int DP>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_dkv_kernel(AttnArgs p, int tiles) {
    typedef typename TT::type T;
    typedef typename Vec8<T>::V V8;
    constexpr int KS = DP / 16, DB = DP / 32, BYTES = kTile * Tile<DP>::ROW, STATS = is_f16<T>() ? 3 : 2;
    __shared__ __align__(16) uint8_t q_0[BYTES], g_0[BYTES], q_1[BYTES], g_1[BYTES];
    __shared__ __align__(16) float stat_0[4 * 64], stat_1[4 * 64];
    const maxsim_attn& a = p.a;
    int id = item_of_block();
    const int item = id, tile = id % tiles;
    id /= tiles;
    const int h = id % a.Hk, b = id / a.Hk;
    const Seq s = sequence(a, b);
    const int G = p.group, D = a.D;
    if (a.zero_rest) {
        zero_rest<T>(p.dk, nullptr, 1, a.cu_k, a.B, a.rows_k, b, s.k0, s.lk, s.all_k, a.Hk, D, h * tiles + tile, a.Hk * tiles, item,
                     (int)gridDim.x);
        zero_rest<T>(p.dv, nullptr, 1, a.cu_k, a.B, a.rows_k, b, s.k0, s.lk, s.all_k, a.Hk, D, h * tiles + tile, a.Hk * tiles, item,
                     (int)gridDim.x);
    }
    const int j0 = tile * kRows;
    if (j0 >= s.lk) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int shift = s.lk - s.lq;
    // tokens that see any of the keys
    const int i_lo = max(0, j0 - a.right - shift);
    const int i_hi = j0 < a.sinks ? s.lq : min(s.lq, min(j0 + kRows, s.lk) - 1 + a.left - shift + 1);
    const int steps = (max(i_hi - i_lo, 0) + kTile - 1) / kTile, total = steps * G;

    const int wj = j0 + wave * 32, j = min(wj + (lane & 31), s.lk - 1);
    const bool mine = wj + (lane & 31) < s.lk, packed = a.cu_k != nullptr;
    V8 k[KS], v[KS];
    const T* kr = first<T>(a.k, packed, b, s.k0, h) + (int64_t)j * a.k.token;
    const T* vr = first<T>(a.v, packed, b, s.k0, h) + (int64_t)j * a.v.token;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
        k[kk] = row8<T>(kr, 16 * kk + 8 * (lane >> 5), D);
        v[kk] = row8<T>(vr, 16 * kk + 8 * (lane >> 5), D);
    }
    // the lane's key is seen by tokens [lo, hi]
    const int lo = j - a.right - shift, hi = j < a.sinks ? s.lq - 1 : min(s.lq - 1, j + a.left - shift);
    const int j_hi = min(wj + 31, s.lk - 1);  // the wave's last key
    const float c = a.scale * kLog2e;
    f32x16 dk[DB], dv[DB];
#pragma unroll
    for (int db = 0; db < DB; ++db) dk[db] = dv[db] = zero16();
    float lift = 0.f;  // of what dk holds (fp16): the smallest of the rows' so far; 0: nothing yet

    const T* qs = first<T>(a.q, a.cu_q != nullptr, b, s.q0, h * G);
    const T* gs = first<T>(p.dout, a.cu_q != nullptr, b, s.q0, h * G);
    const int64_t row0 = first_row(a, s, b);
    Loader<DP, kTile, kWaves> lq, lg;
    lq.init(wave, lane, a.q.token, D);
    lg.init(wave, lane, p.dout.token, D);
    const auto load = [&](int t, uint8_t* qt, uint8_t* gt, float* stat) {
        const int g = t / steps, i = i_lo + (t - g * steps) * kTile;
        lq.load(qs + (int64_t)g * a.q.head + (int64_t)i * a.q.token, s.lq - i, a.q.token, D, qt, wave);
        lg.load(gs + (int64_t)g * p.dout.head + (int64_t)i * p.dout.token, s.lq - i, p.dout.token, D, gt, wave);
        if (wave < STATS) {  // 64 rows' values of one kind; zeros past the last row, whose q and dO are zeros too
            const uint64_t at = (uint64_t)(p.row_stat + ((int64_t)wave * a.Hq + h * G + g) * p.rows + row0 + i);
            const uint32_t first_ = __builtin_amdgcn_readfirstlane((uint32_t)at), second = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32));
            const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
                (void*)(((uint64_t)second << 32) | first_), (short)0, min(s.lq - i, kTile) * 4, 0x00020000);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lptr_t)(stat + wave * 64), 4, lane * 4, 0, 0, 0);
        }
    };
    const auto work = [&](int t, const uint8_t* qt, const uint8_t* gt, const float* stat) {
        const int i0 = i_lo + (t % steps) * kTile;
        if (wj >= s.lk) return;
        float f = 1.f;
        if constexpr (is_f16<T>()) {
            // rows in the scale of the largest dO seen so far, what is there already brought to it
            const float now = lift_of(fmaxf(__uint_as_float(max64(fbits(stat[128 + lane]))), 0.f));
            const bool any = max64(fbits(stat[128 + lane])) != 0;
            if (any && (lift == 0.f || now < lift)) {
                const float down = lift == 0.f ? 1.f : now / lift;
#pragma unroll
                for (int db = 0; db < DB; ++db)
#pragma unroll
                    for (int i = 0; i < 16; ++i) dk[db][i] *= down;
                lift = now;
            }
            f = lift == 0.f ? 1.f : lift;
        }
#pragma unroll
        for (int nb = 0; nb < kTile / 32; ++nb) {
            const int ib = i0 + 32 * nb;
            // all of the block's tokens before, or behind, those that see the wave's keys
            if (ib > (wj < a.sinks ? s.lq - 1 : j_hi + a.left - shift) || ib + 31 < wj - a.right - shift || ib >= s.lq) continue;
            const bool whole = ib >= j_hi - a.right - shift && ib + 31 < s.lq && (j_hi < a.sinks || ib + 31 <= wj + a.left - shift);
            const uint8_t *qb = qt + nb * 32 * Tile<DP>::ROW, *gb = gt + nb * 32 * Tile<DP>::ROW;
            f32x16 x = zero16(), dp = zero16();
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) x = mma<T>(rows_at<T, DP>(qb, lane, kk), k[kk], x);
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) dp = mma<T>(rows_at<T, DP>(gb, lane, kk), v[kk], dp);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 l = *reinterpret_cast<const f32x4*>(stat + 32 * nb + 8 * q + 4 * (lane >> 5));
#pragma unroll
                for (int i = 0; i < 4; ++i) x[4 * q + i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[4 * q + i], c, -l[i]));
            }
            if (!whole) {
                const int i = ib + 4 * (lane >> 5);
                const int low = lo - i, upto = hi - i;
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = slot(e) >= low && slot(e) <= upto ? x[e] : 0.f;
            }
#pragma unroll
            for (int t2 = 0; t2 < 2; ++t2) {
                const V8 pt = pack8<T>(x, 8 * t2);
#pragma unroll
                for (int db = 0; db < DB; ++db) dv[db] = mma<T>(cols_at<T, DP>(gb, lane, t2, db), pt, dv[db]);
            }
            if constexpr (is_f16<T>()) f *= 1.f / 256.f;  // P is lifted by 2^8
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 d = *reinterpret_cast<const f32x4*>(stat + 64 + 32 * nb + 8 * q + 4 * (lane >> 5));
#pragma unroll
                for (int i = 0; i < 4; ++i) x[4 * q + i] *= is_f16<T>() ? (dp[4 * q + i] - d[i]) * f : dp[4 * q + i] - d[i];
            }
            if constexpr (is_f16<T>()) f *= 256.f;
#pragma unroll
            for (int t2 = 0; t2 < 2; ++t2) {
                const V8 ds = pack8<T>(x, 8 * t2);
#pragma unroll
                for (int db = 0; db < DB; ++db) dk[db] = mma<T>(cols_at<T, DP>(qb, lane, t2, db), ds, dk[db]);
            }
        }
    };
    if (total > 0) load(0, q_0, g_0, stat_0);
    for (int t = 0; t < total; t += 2) {
        tile_ready();
        if (t + 1 < total) load(t + 1, q_1, g_1, stat_1);
        work(t, q_0, g_0, stat_0);
        if (t + 1 >= total) break;
        tile_ready();
        if (t + 2 < total) load(t + 2, q_0, g_0, stat_0);
        work(t + 1, q_1, g_1, stat_1);
    }
    T* dkr = first<T>(p.dk, packed, b, s.k0, h) + (int64_t)j * p.dk.token;
    T* dvr = first<T>(p.dv, packed, b, s.k0, h) + (int64_t)j * p.dv.token;
    store_row<T, DB>(dkr, mine, dk, is_f16<T>() && lift != 0.f ? a.scale / lift : a.scale, lane, D);
    store_row<T, DB>(dvr, mine, dv, is_f16<T>() ? 1.f / 256.f : 1.f, lane, D);
}

template <typename TT, int DP>
hipError_t launch(const AttnArgs& p, hipStream_t stream) {
    const maxsim_attn& a = p.a;
    const int64_t q_tiles = ((int64_t)a.max_q * p.group + kRows - 1) / kRows, k_tiles = ((int64_t)a.max_k + kRows - 1) / kRows;
    // (of no queries, or no keys, the rows of no sequence are still to be made 0)
    const int q_blocks = (int)(q_tiles > 0 ? q_tiles : 1), k_blocks = (int)(k_tiles > 0 ? k_tiles : 1);
    attn_dq_kernel<TT, DP><<<(unsigned)(q_blocks * a.Hk * a.B), 64 * kWaves, 0, stream>>>(p, q_blocks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    attn_dkv_kernel<TT, DP><<<(unsigned)(k_blocks * a.Hk * a.B), 64 * kWaves, 0, stream>>>(p, k_blocks);
    return hipGetLastError();
}

int64_t rows_in_memory(const maxsim_attn& a) { return a.cu_q ? a.rows_q : (int64_t)a.B * a.max_q; }

}  // namespace

size_t attn_bwd_workspace_bytes(const maxsim_attn& a) {
    return (size_t)(a.dtype == MAXSIM_F16 ? 3 : 2) * (size_t)rows_in_memory(a) * a.Hq * sizeof(float);
}

hipError_t launch_attn_bwd(const maxsim_attn& a, const float* lse, const maxsim_view& dout, const maxsim_view& dq,
                           const maxsim_view& dk, const maxsim_view& dv, void* workspace, hipStream_t stream) {
    AttnArgs p{};
    p.a = a;
    if (a.left < 0 || a.left > kNoBound) p.a.left = kNoBound;
    if (a.right < 0 || a.right > kNoBound) p.a.right = kNoBound;
    p.lse = const_cast<float*>(lse);
    p.dout = dout;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.group = a.Hq / a.Hk;
    p.splits = 1;
    p.rows = rows_in_memory(a);
    p.row_stat = static_cast<float*>(workspace);
    const bool half = a.dtype == MAXSIM_F16;
    if (a.D <= 64) return half ? launch<F16, 64>(p, stream) : launch<BF16, 64>(p, stream);
    return half ? launch<F16, 128>(p, stream) : launch<BF16, 128>(p, stream);
}

}  // namespace maxsim
