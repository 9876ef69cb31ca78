// attn_bwd.hip -- attention's backward for gfx950 (MI355X), in two launches without atomics.
//
//     P = exp(S - lse);  dP = dO V^T;  delta = rowsum(dO * out);  dS = P * (dP - delta)
//     dQ = scale dS K;  dK = scale dS^T Q;  dV = P^T dO
//
// The first goes over the keys for each tile of queries (dQ, and what the second needs of a row), the
// second over the queries for each tile of keys (dK and dV, summed over the query heads of the key
// head).  Each makes S and dP anew: 7 products of a pair for the 5 of a single pass, whose dQ would have to be
// added up in memory by all workgroups in an order of chance.
//
// P and dS are rounded to T for their products, as P is in the forward: the matrix instruction takes both operands in one
// type.  Each is held to half a step of T (fp16: brought into its range first, below), which averages out over many keys: the
// gradients' error is 0.0024 of their norm in bf16 and 0.0003 in fp16, where their own rounding makes 0.0017 and 0.0002.
//
// Bound as the forward is.  Measured, the kernels alone once the clocks have settled (bf16):
//     2 x 4096 tokens, 16 / 4 heads of 128, all pairs     dQ 376 us (1.10 PFLOP/s of its three products), dK and dV 506 + 14 (1.09 of four)
//     2 x 4096 tokens, 32 heads of 64, all pairs          dQ 415, dK and dV 535
//     16 documents of 700 to 1024 tokens, 16 / 4 heads of 128    dQ 182, dK and dV 216 (matrix pipes 39 % and 47 % of their cycles)
//     9 sequences of up to 601 tokens, 100 back and the first 3, 6 / 2 heads of 80, fp16    dQ 15.5, dK and dV 24.2 + 6.3: the way of a
//                                                         few tiles through one wave (of it the largest dS of each block 1 and 1)
// Tried and slower: 64 keys to a wave (its 512 registers move through the accumulator half: 340 us for 247); k's operands in
// registers beside two waves to a SIMD (memory takes what does not fit, and waits for the next tile's loads: 494).
#include <algorithm>

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
// Half a step of a value of 1.
template <typename T>
constexpr float kHalfStep = is_f16<T>() ? 0x1p-11f : 0x1p-8f;
// fp16 holds P and dS for their products only if they are brought into its range by powers of 2, which are
// exact: P (at most 1, 1 / keys where attention is flat) times 2^8; dS by the largest that the row of the result has met so far.
constexpr float kLiftP = 8.f;  // log2
// The factor of dS (fp16) of one row of the result, which the sum at hand holds too: it brought the largest magnitude at the time
// it was set to [2^7, 2^8), and stays until one passes 2^15.  So a value is held to fp16's half step or to 2^-32 of the
// largest one of the same sum, whichever is more, whatever the rows' dO, v and P are.
struct Lift {
    uint32_t bits;  // of the factor, a power of 2
    __device__ __forceinline__ void start() { bits = 221u << 23; }  // 2^94: nothing met yet
    __device__ __forceinline__ float factor() const { return __uint_as_float(bits); }
    __device__ __forceinline__ float inverse() const { return __uint_as_float((254u << 23) - bits); }
    // Takes in a block's largest magnitude; true where some lane's sums are to be multiplied by 2^shift first.
    __device__ __forceinline__ bool take(float m, int& shift) {
        const bool past = m > __uint_as_float((269u << 23) - bits);  // 2^15 / factor
        shift = 0;
        if (!__any(past)) return false;
        const int e = min(max((int)(fbits(m) >> 23), 40), 246);
        const uint32_t now = past ? (uint32_t)(261 - e) << 23 : bits;
        shift = (int)(now - bits) >> 23;
        bits = now;
        return true;
    }
};

// A block of dS, 16 values in either lane of a pair, by that factor, with the sums brought to it where it changes.
template <int DB>
__device__ __forceinline__ void lifted(f32x16& x, f32x16* sums, Lift& lift) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = larger(m, __builtin_fabsf(x[i]));
    int shift;
    if (lift.take(swap_max(m), shift)) {
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) sums[db][i] = __builtin_ldexpf(sums[db][i], shift);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= lift.factor();
}

// The first token past the window of all of a key tile's keys.
__device__ __forceinline__ int far_from(const maxsim_attn& a, const Seq& s, int j0) {
    return max(0, min(s.lq, min(j0 + kRows, s.lk) + a.left - (s.lk - s.lq)));
}
__device__ __forceinline__ float* part_row(const AttnArgs& p, int b, int h, int tile, int slot, int row) {
    const int64_t block = (((int64_t)b * p.a.Hk + h) * p.part_tiles + tile) * ((p.far_chunks + 1) * p.head_splits) + slot;
    return p.part + (block * 2 * p.part_rows + row) * p.a.D;
}

template <typename TT, int DP>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_dq_kernel(AttnArgs p, int tiles) {
    typedef typename TT::type T;
    typedef typename Vec8<T>::V V8;
    constexpr int KS = DP / 16, DB = DP / 32, BYTES = kTile * Tile<DP>::ROW;
    __shared__ __align__(16) uint8_t k_0[BYTES], v_0[BYTES], k_1[BYTES], v_1[BYTES];
    const maxsim_attn& a = p.a;
    Work w;
    if (!work_of(w, a.B, a.Hk, tiles)) return;
    const int b = w.b, h = w.h, tile = tiles - 1 - w.part;
    const Seq s = sequence(a, b);
    const int G = p.group, D = a.D, rows = s.lq * G;
    if (a.zero_rest)
        zero_rest<T>(p.dq, nullptr, 1, a.cu_q, a.B, a.rows_q, b, s.q0, s.lq, s.all_q, a.Hq, D, h * tiles + tile, a.Hk * tiles,
                     w.item(tiles, a.Hk), w.items);
    const int r0 = tile * kRows;
    if (r0 >= rows) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int shift = s.lk - s.lq;
    const Span span = span_of(a, s.lk, r0 / G + shift, (min(r0 + kRows, rows) - 1) / G + shift, kTile);
    const int wr = r0 + wave * 32;
    const int r = min(wr + (lane & 31), rows - 1), token = r / G, head = h * G + r % G;
    const bool mine = wr + (lane & 31) < rows;
    const bool packed = a.cu_q != nullptr;

    const T* ks = first<T>(a.k, a.cu_k != nullptr, b, s.k0, h);
    const T* vs = first<T>(a.v, a.cu_k != nullptr, b, s.k0, h);
    Loader<DP, kTile, kWaves> lk, lv;
    lk.init(wave, lane, a.k.token, D);
    lv.init(wave, lane, a.v.token, D);
    Walk<T> next;
    next.start(span, 0, kTile, ks, vs, a.k.token, a.v.token);
    const auto load = [&](uint8_t* kt, uint8_t* vt) {
        const int left = span.end(next.t) - next.j;
        lk.load(next.k, left, a.k.token, D, kt, wave);
        lv.load(next.v, left, a.v.token, D, vt, wave);
        next.next(span, kTile, ks, vs, a.k.token, a.v.token);
    };
    if (span.tiles > 0) load(k_0, v_0);  // on its way while the rows are read

    // the row's q and dO as operands, delta, and lse in powers of 2: a row that sees nothing has P = 0
    V8 q[KS], g[KS];
    const T* qr = first<T>(a.q, packed, b, s.q0, 0) + (int64_t)token * a.q.token + (int64_t)head * a.q.head;
    const T* gr = first<T>(p.dout, packed, b, s.q0, 0) + (int64_t)token * p.dout.token + (int64_t)head * p.dout.head;
    const T* orow = first<T>(a.out, packed, b, s.q0, 0) + (int64_t)token * a.out.token + (int64_t)head * a.out.head;
    const int64_t at = first_row(a, s, b) + token;
    const T* rest = rest_of<T>(p, at * a.Hq + head);
    float delta = 0.f;
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
            // what rounding left off out is half a step of it at most (of fp16's subnormal values nothing, which is 0 as T): more
            // than that, or a NaN, is something else that lies behind the caller's lse, and left out
            const float x = (float)o[i], left = (float)off[i];
            const float more = __builtin_fabsf(left) <= __builtin_fabsf(x) * kHalfStep<T> ? left : 0.f;
            delta = __builtin_fmaf((float)g[kk][i], x + more, delta);
        }
    }
    delta = swap_sum(delta);
    float lse = p.lse[(at * a.Hq + head) * a.lse_step] * kLog2e;
    if (lse == -INFINITY) lse = INFINITY;
    if (mine && lane < 32) {
        float* stat = p.row_stat + (int64_t)head * p.rows + at;
        stat[0] = is_f16<T>() ? lse - kLiftP : lse;
        stat[p.rows * a.Hq] = delta;
    }
    Lift lift;  // of what acc holds (fp16)
    lift.start();
    const Place place = place_of<DP>(lane);

    const int p_lo = min(wr, rows - 1) / G + shift, p_hi = min(wr + 31, rows - 1) / G + shift, pos = token + shift;
    const int lo = pos - a.left, hi = min(pos + a.right, s.lk - 1);
    const float c = a.scale * kLog2e;
    f32x16 acc[DB];
#pragma unroll
    for (int db = 0; db < DB; ++db) acc[db] = zero16();

    const auto work = [&](int t, const uint8_t* kt, const uint8_t* vt) {
        const int j0 = span.at(t, kTile), end = span.end(t);
        if (wr >= rows) return;
#pragma unroll
        for (int nb = 0; nb < kTile / 32; ++nb) {
            const int jb = j0 + 32 * nb;
            if (jb >= end || jb > p_hi + a.right || (jb + 31 < p_lo - a.left && jb >= a.sinks)) continue;  // no row sees any
            const bool whole = jb + 32 <= end && jb + 31 <= min(p_lo + a.right, s.lk - 1) && (jb >= p_hi - a.left || jb + 32 <= a.sinks);
            const uint8_t *kb = kt + nb * 32 * Tile<DP>::ROW, *vb = vt + nb * 32 * Tile<DP>::ROW;
            f32x16 x = zero16(), dp = zero16();
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) x = mma<T>(rows_at<T, DP>(kb, place, kk), q[kk], x);
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) dp = mma<T>(rows_at<T, DP>(vb, place, kk), g[kk], dp);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], c, -lse));
            if (!whole) {
                const int j = jb + 4 * (lane >> 5);
                const uint32_t bits = slots_seen(lo - j, min(hi, end - 1) - j, a.sinks - j);
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = keep(bits, i, x[i], 0u);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] *= dp[i] - delta;
            if constexpr (is_f16<T>()) lifted<DB>(x, acc, lift);
#pragma unroll
            for (int t2 = 0; t2 < 2; ++t2) {
                const V8 ds = pack8<T>(x, 8 * t2);
#pragma unroll
                for (int db = 0; db < DB; ++db) acc[db] = mma<T>(cols_at<T, DP>(kb, place, t2, db), ds, acc[db]);
            }
        }
    };
    for (int t = 0; t < span.tiles; t += 2) {
        tile_ready();
        if (t + 1 < span.tiles) load(k_1, v_1);
        work(t, k_0, v_0);
        if (t + 1 >= span.tiles) break;
        tile_ready();
        if (t + 2 < span.tiles) load(k_0, v_0);
        work(t + 1, k_1, v_1);
    }
    T* out = first<T>(p.dq, packed, b, s.q0, 0) + (int64_t)token * p.dq.token + (int64_t)head * p.dq.head;
    store_row<T, DB>(out, mine, acc, is_f16<T>() ? a.scale * lift.inverse() : a.scale, lane, D);
}

// A workgroup's 128 keys of one key head, 32 of a wave; the query heads that share it one after the other, TR tokens
// at a time.  The queries are the rows of S here, the keys its columns, so P and dS are the B operands of dV^T = dO^T P and
// dK^T = Q^T dS, and a lane's result rows stay in registers.  WAVES to a SIMD: two leave a wave 256 registers, which do
// not hold k's operands beside the sums at a width of 128 (they stay in LDS), one leaves 512.
template <typename TT, int DP, int WAVES>
__global__ __launch_bounds__(64 * kWaves, DP == 64 ? 3 : WAVES) void attn_dkv_kernel(AttnArgs p, int tiles) {
    typedef typename TT::type T;
    typedef typename Vec8<T>::V V8;
    constexpr int TR = DP == 128 && WAVES == 2 ? 32 : 64;
    constexpr bool K_IN_LDS = DP == 128 && WAVES == 2;
    constexpr int KS = DP / 16, DB = DP / 32, BYTES = TR * Tile<DP>::ROW, STATS = 2;
    __shared__ __align__(16) uint8_t q_0[BYTES], g_0[BYTES], q_1[BYTES], g_1[BYTES];
    __shared__ __align__(16) float stat_0[STATS * 64], stat_1[STATS * 64];
    __shared__ __align__(16) uint8_t k_lds[K_IN_LDS ? kWaves * KS * 1024 : 16];  // 64 lanes x 16 bytes for each step
    const maxsim_attn& a = p.a;
    Work w;
    const int fars = p.far_tiles * p.far_chunks;
    if (!work_of(w, a.B, a.Hk, (tiles + fars) * p.head_splits)) return;
    const int b = w.b, h = w.h, heads = w.part % p.head_splits, unit = w.part / p.head_splits;
    const bool far = unit < fars;
    const int tile = far ? unit / p.far_chunks : unit - fars, chunk = far ? unit % p.far_chunks : 0;
    const Seq s = sequence(a, b);
    const int G = p.group, D = a.D, g0 = G * heads / p.head_splits, g1 = G * (heads + 1) / p.head_splits;
    if (a.zero_rest && !far && heads == 0) {
        const int part = h * tiles + tile, parts = a.Hk * tiles, item = (b * a.Hk + h) * tiles + tile, items = a.B * a.Hk * tiles;
        zero_rest<T>(p.dk, nullptr, 1, a.cu_k, a.B, a.rows_k, b, s.k0, s.lk, s.all_k, a.Hk, D, part, parts, item, items);
        zero_rest<T>(p.dv, nullptr, 1, a.cu_k, a.B, a.rows_k, b, s.k0, s.lk, s.all_k, a.Hk, D, part, parts, item, items);
    }
    const int j0 = tile * kRows;
    if (j0 >= s.lk) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int shift = s.lk - s.lq;
    // tokens [i_lo, i_hi) see any of the keys; where first tokens' keys are worked on apart, those past the window do not count
    const bool apart = tile < p.far_tiles;
    const int i_far = far_from(a, s, j0);
    int i_lo = max(0, j0 - a.right - shift), i_hi = j0 < a.sinks && !apart ? s.lq : i_far;
    if (far) {
        i_lo = i_far + chunk * p.far_tokens;
        i_hi = min(s.lq, i_lo + p.far_tokens);
        if (i_lo >= i_hi) return;
    }
    const int steps = (max(i_hi - i_lo, 0) + TR - 1) / TR, total = steps * (g1 - g0);

    const T* qs = first<T>(a.q, a.cu_q != nullptr, b, s.q0, h * G);
    const T* gs = first<T>(p.dout, a.cu_q != nullptr, b, s.q0, h * G);
    const int64_t row0 = first_row(a, s, b);
    Loader<DP, TR, kWaves> lq, lg;
    lq.init(wave, lane, a.q.token, D);
    lg.init(wave, lane, p.dout.token, D);
    // the token that the next tile starts with, and where q, dO and the rows' values lie there
    int i_next = i_lo;
    const T* q_next = qs + (int64_t)g0 * a.q.head + (int64_t)i_lo * a.q.token;
    const T* g_next = gs + (int64_t)g0 * p.dout.head + (int64_t)i_lo * p.dout.token;
    const float* stat_next = p.row_stat + ((int64_t)wave * a.Hq + h * G + g0) * p.rows + row0 + i_lo;
    const int64_t q_back = a.q.head - (int64_t)steps * TR * a.q.token, g_back = p.dout.head - (int64_t)steps * TR * p.dout.token;
    const int64_t stat_back = p.rows - (int64_t)steps * TR;
    const auto load = [&](uint8_t* qt, uint8_t* gt, float* stat) {
        lq.load(q_next, i_hi - i_next, a.q.token, D, qt, wave);
        lg.load(g_next, i_hi - i_next, p.dout.token, D, gt, wave);
        if (wave < STATS) {  // the rows' values of one kind; zeros past the last row, whose q and dO are zeros too
            const uint64_t at = (uint64_t)stat_next;
            const uint32_t low = __builtin_amdgcn_readfirstlane((uint32_t)at), high = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32));
            const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
                (void*)(((uint64_t)high << 32) | low), (short)0, min(i_hi - i_next, TR) * 4, 0x00020000);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lptr_t)(stat + wave * 64), 4, lane * 4, 0, 0, 0);
        }
        i_next += TR;
        q_next += TR * a.q.token;
        g_next += TR * p.dout.token;
        stat_next += TR;
        if (i_next >= i_hi) {  // on to the next head
            i_next = i_lo;
            q_next += q_back;
            g_next += g_back;
            stat_next += stat_back;
        }
    };
    if (total > 0) load(q_0, g_0, stat_0);  // on its way while the keys' rows are read

    const int wj = j0 + wave * 32, j_hi = min(wj + 31, s.lk - 1);  // the wave's keys
    const int j = min(wj + (lane & 31), s.lk - 1);
    const bool mine = wj + (lane & 31) < s.lk, packed = a.cu_k != nullptr;
    V8 k[K_IN_LDS ? 1 : KS], v[KS];
    const int k_at = wave * KS * 1024 + lane * 16;
    const Place place = place_of<DP>(lane);
    // the lane's key is seen by tokens [lo, hi] of these; one that none of them sees is zeros, whatever it holds
    const int hi_first = i_hi - 1, hi_plain = far ? -1 : min(i_hi - 1, j + a.left - shift);
    const int lo = max(i_lo, j - a.right - shift), hi = j < a.sinks ? hi_first : hi_plain;
    const T* kr = first<T>(a.k, packed, b, s.k0, h) + (int64_t)j * a.k.token;
    const T* vr = first<T>(a.v, packed, b, s.k0, h) + (int64_t)j * a.v.token;
    const int columns = lo <= hi ? D : 0;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
        const V8 x = row8<T>(kr, 16 * kk + 8 * (lane >> 5), columns);
        if constexpr (K_IN_LDS) *reinterpret_cast<V8*>(k_lds + k_at + kk * 1024) = x;
        else k[kk] = x;
        v[kk] = row8<T>(vr, 16 * kk + 8 * (lane >> 5), columns);
    }
    // all of the wave's keys by tokens [all_lo, all_hi], any of them by [any_lo, any_hi]
    const int all_lo = max(i_lo, j_hi - a.right - shift), any_lo = max(i_lo, wj - a.right - shift);
    const int all_hi = j_hi < a.sinks ? hi_first : far ? -1 : min(i_hi - 1, wj + a.left - shift);
    const int any_hi = wj < a.sinks ? hi_first : far ? -1 : min(i_hi - 1, j_hi + a.left - shift);
    const float c = a.scale * kLog2e;
    f32x16 dk[DB], dv[DB];
#pragma unroll
    for (int db = 0; db < DB; ++db) dk[db] = dv[db] = zero16();
    Lift lift;  // of what dk holds (fp16)
    lift.start();

    int i_now = i_lo;  // the token that the tile at hand starts with
    const auto work = [&](const uint8_t* qt, const uint8_t* gt, const float* stat) {
        const int at = i_now;
        i_now = i_now + TR >= i_hi ? i_lo : i_now + TR;
        if (wj >= s.lk) return;
#pragma unroll
        for (int nb = 0; nb < TR / 32; ++nb) {
            const int ib = at + 32 * nb;
            if (ib > any_hi || ib + 31 < any_lo) continue;
            const bool whole = ib >= all_lo && ib + 31 <= all_hi;
            const uint8_t *qb = qt + nb * 32 * Tile<DP>::ROW, *gb = gt + nb * 32 * Tile<DP>::ROW;
            // (the compiler is not to see that these places are the same in each step: it would keep all that follows from them,
            // and k's operands, in registers that the sums need)
            int ka = k_at;
            Place at_ = place;
            if constexpr (WAVES == 2) asm volatile("" : "+v"(ka), "+v"(at_.rows), "+v"(at_.cols));
            f32x16 x = zero16(), dp = zero16();
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
                V8 kx;
                if constexpr (K_IN_LDS) kx = *reinterpret_cast<const V8*>(k_lds + ka + kk * 1024);
                else kx = k[kk];
                x = mma<T>(rows_at<T, DP>(qb, at_, kk), kx, x);
            }
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) dp = mma<T>(rows_at<T, DP>(gb, at_, kk), v[kk], dp);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 l = *reinterpret_cast<const f32x4*>(stat + 32 * nb + 8 * q + 4 * (lane >> 5));
#pragma unroll
                for (int i = 0; i < 4; ++i) x[4 * q + i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[4 * q + i], c, -l[i]));
            }
            if (!whole) {
                const int i = ib + 4 * (lane >> 5);
                const uint32_t bits = slots_seen(lo - i, hi - i, 0);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = keep(bits, e, x[e], 0u);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const V8 pt = pack8<T>(x, 8 * t);
#pragma unroll
                for (int db = 0; db < DB; ++db) dv[db] = mma<T>(cols_at<T, DP>(gb, at_, t, db), pt, dv[db]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 d = *reinterpret_cast<const f32x4*>(stat + 64 + 32 * nb + 8 * q + 4 * (lane >> 5));
#pragma unroll
                for (int i = 0; i < 4; ++i) x[4 * q + i] *= dp[4 * q + i] - d[i];
            }
            if constexpr (is_f16<T>()) lifted<DB>(x, dk, lift);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const V8 ds = pack8<T>(x, 8 * t);
#pragma unroll
                for (int db = 0; db < DB; ++db) dk[db] = mma<T>(cols_at<T, DP>(qb, at_, t, db), ds, dk[db]);
            }
        }
    };
    for (int t = 0; t < total; t += 2) {
        tile_ready();
        if (t + 1 < total) load(q_1, g_1, stat_1);
        work(q_0, g_0, stat_0);
        if (t + 1 >= total) break;
        tile_ready();
        if (t + 2 < total) load(q_0, g_0, stat_0);
        work(q_1, g_1, stat_1);
    }
    const float vf = is_f16<T>() ? 1.f / 256.f : 1.f, kf = is_f16<T>() ? a.scale * (lift.inverse() * vf) : a.scale;  // P is lifted by 2^8
    const bool part = p.head_splits > 1 || (apart && j < a.sinks);
    if (!far && p.head_splits == 1) {
        T* dkr = first<T>(p.dk, packed, b, s.k0, h) + (int64_t)j * p.dk.token;
        T* dvr = first<T>(p.dv, packed, b, s.k0, h) + (int64_t)j * p.dv.token;
        store_row<T, DB>(dkr, mine && !part, dk, kf, lane, D);
        store_row<T, DB>(dvr, mine && !part, dv, vf, lane, D);
    }
    if (part && mine && (!far || j < a.sinks)) {
        float* to = part_row(p, b, h, tile, (far ? chunk + 1 : 0) * p.head_splits + heads, j - j0);
        const int64_t other = (int64_t)p.part_rows * D;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int d = 32 * db + 8 * q + 4 * (lane >> 5);
                if (d >= D) continue;
                f32x4 x, y;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = dk[db][4 * q + i] * kf;
                    y[i] = dv[db][4 * q + i] * vf;
                }
                *reinterpret_cast<f32x4*>(to + d) = x;
                *reinterpret_cast<f32x4*>(to + other + d) = y;
            }
    }
}

// The rows of dK and dV that more than one workgroup adds to: their parts, added in order.  32 threads to a row, 4 columns each.
template <typename TT>
__global__ __launch_bounds__(64) void attn_parts_kernel(AttnArgs p, int keys) {
    typedef typename TT::type T;
    typedef T V4 __attribute__((ext_vector_type(4)));
    const maxsim_attn& a = p.a;
    const int j = blockIdx.x % keys, pair = blockIdx.x / keys, h = pair % a.Hk, b = pair / a.Hk;
    const Seq s = sequence(a, b);
    const int d = (threadIdx.x & 31) * 4, tile = j / kRows, j0 = tile * kRows;
    if (j >= s.lk || d >= a.D) return;
    const bool of_v = threadIdx.x >= 32;
    int slots = p.head_splits;
    if (tile < p.far_tiles && j < a.sinks)
        slots += (max(s.lq - far_from(a, s, j0), 0) + p.far_tokens - 1) / p.far_tokens * p.head_splits;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int n = 0; n < slots; ++n)
        sum += *reinterpret_cast<const f32x4*>(part_row(p, b, h, tile, n, j - j0) + (of_v ? (int64_t)p.part_rows * a.D : 0) + d);
    const maxsim_view& out = of_v ? p.dv : p.dk;
    V4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = (T)sum[i];
    *reinterpret_cast<V4*>(first<T>(out, a.cu_k != nullptr, b, s.k0, h) + (int64_t)j * out.token + d) = y;
}

int key_tiles(const maxsim_attn& a) { return std::max(1, (a.max_k + kRows - 1) / kRows); }

// How the work on dK and dV is shared out.  Where first tokens stay visible past the window, their key tile would go
// over all queries and the others over a window's worth: with more than two such stretches of queries the far ones get workgroups
// of their own (8192 tokens, a window of 2048 and 4 first tokens, 32 / 8 heads: 1542 -> 686 us).  Up to 256
// workgroups: several for the query heads of a key head (9 sequences of up to 601 tokens, 6 / 2 heads: 46 -> 37 us; 2 x 4096
// tokens, 16 / 4 heads: 687 -> 561).
void plan_parts(const maxsim_attn& a, AttnArgs& p) {
    p.far_tiles = p.far_chunks = p.far_tokens = p.part_tiles = p.part_rows = 0;
    p.head_splits = 1;
    if (a.max_k == 0) return;
    const int keys = std::min(a.sinks, a.max_k);
    if (a.sinks > 0 && a.left >= 0 && a.sinks <= 2 * kRows) {
        const int64_t right = a.right < 0 ? 0 : a.right, stretch = ((int64_t)kRows + a.left + right + 63) / 64 * 64;
        // (a launch of a wave for each of their rows holds fewer than 2^32 threads)
        if (a.max_q > 2 * stretch && (int64_t)a.B * a.Hk * keys < (int64_t)1 << 25) {
            // (64 chunks at most, which bounds the parts' memory: narrow windows over long sequences)
            p.far_tokens = (int)std::max<int64_t>(stretch, ((int64_t)a.max_q + 63) / 64);
            p.far_chunks = (a.max_q + p.far_tokens - 1) / p.far_tokens;
            p.far_tiles = (keys + kRows - 1) / kRows;
        }
    }
    const int64_t items = (int64_t)a.B * a.Hk * (key_tiles(a) + p.far_tiles * p.far_chunks);
    if (items <= 256) p.head_splits = (int)std::min<int64_t>(a.Hq / a.Hk, 512 / items);
    p.part_tiles = p.head_splits > 1 ? key_tiles(a) : p.far_tiles;
    p.part_rows = p.head_splits > 1 ? kRows : std::min(keys, kRows);
}
int64_t part_floats(const maxsim_attn& a, const AttnArgs& p) {
    return (int64_t)a.B * a.Hk * p.part_tiles * (p.far_chunks + 1) * p.head_splits * 2 * p.part_rows * a.D;
}

template <typename TT, int DP>
hipError_t launch(const AttnArgs& p, hipStream_t stream) {
    const maxsim_attn& a = p.a;
    const int64_t pairs = (int64_t)a.B * a.Hk;
    // (of no queries, or no keys, the rows of no sequence are still to be made 0)
    const int q_tiles = (int)std::max<int64_t>(1, ((int64_t)a.max_q * p.group + kRows - 1) / kRows);
    const int k_tiles = key_tiles(a), each = (k_tiles + p.far_tiles * p.far_chunks) * p.head_splits;
    attn_dq_kernel<TT, DP><<<(unsigned)blocks_for(pairs, q_tiles), 64 * kWaves, 0, stream>>>(p, q_tiles);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t blocks = blocks_for(pairs, each);
    // a width of 128: two workgroups to a CU where there are so many (4096 tokens, 8 heads, 256 workgroups: one to a CU
    // 185 us, two 221; 16 x 1024 tokens, 512: 320 and 247)
    const auto dkv = DP == 128 && blocks <= 256 ? attn_dkv_kernel<TT, DP, DP == 128 ? 1 : 2> : attn_dkv_kernel<TT, DP, 2>;
    dkv<<<(unsigned)blocks, 64 * kWaves, 0, stream>>>(p, k_tiles);
    e = hipGetLastError();
    if (e != hipSuccess || p.part_tiles == 0) return e;
    const int keys = p.head_splits > 1 ? a.max_k : std::min(a.sinks, a.max_k);
    attn_parts_kernel<TT><<<(unsigned)(pairs * keys), 64, 0, stream>>>(p, keys);
    return hipGetLastError();
}

int64_t rows_in_memory(const maxsim_attn& a) { return a.cu_q ? a.rows_q : (int64_t)a.B * a.max_q; }
int64_t stat_floats(const maxsim_attn& a) {  // the parts after them start at a multiple of 16 bytes
    return (2 * rows_in_memory(a) * a.Hq + 3) / 4 * 4;
}

}  // namespace

size_t attn_bwd_workspace_bytes(const maxsim_attn& a) {
    AttnArgs p{};
    plan_parts(a, p);
    return (size_t)(stat_floats(a) + part_floats(a, p)) * sizeof(float);
}

hipError_t launch_attn_bwd(const maxsim_attn& a, const float* lse, const maxsim_view& dout, const maxsim_view& dq,
                           const maxsim_view& dk, const maxsim_view& dv, void* workspace, hipStream_t stream) {
    AttnArgs p{};
    plan_parts(a, p);
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
    p.part = p.row_stat + stat_floats(a);
    const bool half = a.dtype == MAXSIM_F16;
    (void)hipGetLastError();  // an error that an earlier call left unread is not this one's
    if (a.D <= 64) return half ? launch<F16, 64>(p, stream) : launch<BF16, 64>(p, stream);
    return half ? launch<F16, 128>(p, stream) : launch<BF16, 128>(p, stream);
}

}  // namespace maxsim
