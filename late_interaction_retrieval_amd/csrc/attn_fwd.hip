// attn_fwd.hip -- attention with a sliding window and first tokens that stay
// visible, forward, for gfx950 (MI355X).
//
//     S = scale q k^T over the keys a query sees;  P = softmax(S);  out = P v;  lse = log sum exp S
//
// One pass over the keys with the running maximum and sum.  The products run with the
// queries as columns: S^T = K Q^T leaves a query's scores in one lane pair, so its maximum
// and sum need one exchange between lanes and the factors of a new maximum are the lane's own; P^T goes
// from the registers it was made in to out^T = V^T P^T as it stands.
//
// What bounds it: with many keys the matrix pipes and the exponentials together (a 64 x 32 tile at a width of 128 is
// 1024 cycles of matrix instructions and about 900 of the vector unit, half of them exponentials at a quarter of its rate);
// two waves to a SIMD overlap them to 52 % of the matrix pipes' cycles and 48 % of the vector unit's.  LDS has no bank conflicts.  A next
// token is bound by the cache's bytes.  Measured, the kernels alone once the clocks have settled (the first 40 to 100 passes after other work
// take 10 to 18 % longer; a library product of 8192^3 reaches 1.39 PFLOP/s then):
//     8192 tokens, causal, 2048 back and the first 4, 32 / 8 heads of 128, bf16     251 - 271 us over cards, 0.89 - 0.96 PFLOP/s of the pairs that
//                                                                            see each other
//     2 x 4096 tokens, 16 / 4 heads of 128, all pairs                        276 us, 1.00 PFLOP/s
//     2 x 4096 tokens, 32 heads of 64, all pairs                             310 us, 0.89 PFLOP/s
//     64 packed documents of 32 to 1024 tokens, 128 to each side and the first, 16 heads of 64    80 - 81 us: the vector unit (56 % of its
//                                              cycles, the matrix pipes 20 %; 3 waves to a SIMD on average), 3616 workgroups in 3.5 rounds, 4576
//                                              that find nothing
//     16 next tokens, caches of 8192 to 32768 keys, 8 key heads of 128       267 us + 6.5 the join, 1.45 GB at 5.4 TB/s
// Tried and slower: the next tile's scores made beside this one's softmax (through the branches between them the compiler
// moves the accumulators to memory: 8 times the time); leaving out hidden blocks of 32 keys, or their exponentials, by
// branches (89 -> 98 and 117 us); first tokens in blocks of 32 before the window's tiles (no difference).
#include <algorithm>

#include "attn_dev.h"

namespace maxsim {
namespace {

constexpr int kWaves = 4;
constexpr int kRowsWave = 32;                  // rows (a token's query head each) of a wave
constexpr int kRows = kWaves * kRowsWave;      // of a workgroup
constexpr int kKeys = 64;                      // of a tile
constexpr int kKeysFew = 32;                   // of a wave's own tile, with few rows

// A wave's state for its 32 rows: out^T and, for the lane's row, the reference of the exponents in
// units of the scores and the sum of this lane's keys.  out^T and the sum hold P times 2^LIFT, a power of 2 that costs nothing: in fp16 a
// weight then keeps a step of 2^-31 of the largest one's instead of 2^-24, which 65536 keys of 2^-25.5 behind a first
// token would fall below together, 1 / 700 of the row.
template <typename T, int DP>
struct Rows {
    static constexpr int KS = DP / 16, DB = DP / 32;
    static constexpr float LIFT = std::is_same<T, _Float16>::value ? 7.f : 0.f;  // log2
    typename Vec8<T>::V q[KS];
    f32x16 o[DB];
    float ref, sum;
    Place at;
    int lo, hi;  // the lane's row sees keys [lo, hi] (and those below `sinks` that are at most hi)

    __device__ __forceinline__ void start(const T* row, int lane, int D, int pos, int lk, const maxsim_attn& a) {
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) q[kk] = row8<T>(row, 16 * kk + 8 * (lane >> 5), D);
#pragma unroll
        for (int db = 0; db < DB; ++db) o[db] = zero16();
        at = place_of<DP>(lane);
        ref = -INFINITY;
        sum = 0.f;
        lo = pos - a.left;
        hi = min(pos + a.right, lk - 1);
    }

    // The exponent, in powers of 2, that the sum is in units of; `none` of a row that has seen nothing.
    __device__ __forceinline__ float top(float c, float none) const { return ref == -INFINITY ? none : ref * c - LIFT; }

    // Which of a block's keys from j0 on, before `end`, the lane's row sees.
    __device__ __forceinline__ uint32_t bits(int j0, int end, int sinks, int lane) const {
        const int j = j0 + 4 * (lane >> 5);
        return slots_seen(lo - j, min(hi, end - 1) - j, sinks - j);
    }

    // NB blocks of 32 keys.  all: every row sees all of them; else bits[nb] are the lane's.
    // The reference stays while the maximum passes it by less than 2^8: P grows to 256 at most (2^15 with LIFT), which both
    // types hold, and relative to the row's sum nothing is lost.  P is rounded to T for its product: the matrix instruction
    // takes both operands in one type, and v comes in T.  (That
    // takes out's error from the 0.0017 of its norm that its own rounding makes in bf16 to 0.0022 - 0.0023, in fp16 from 0.00020 to 0.00024;
    // P in two halves would take the product twice.)
    template <int NB>
    __device__ __forceinline__ void step(const uint8_t* kt, const uint8_t* vt, bool all, const uint32_t* bits, float c, float slack) {
        f32x16 s[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            s[nb] = zero16();
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) s[nb] = mma<T>(rows_at<T, DP>(kt + nb * 32 * Tile<DP>::ROW, at, kk), q[kk], s[nb]);
        }
        if (!all) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[nb][i] = keep(bits[nb], i, s[nb][i], kMinusInfinity);
        }
        float m = s[0][0];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 16; ++i) m = larger(m, s[nb][i]);
        m = swap_max(m);
        if (__any(!(m <= ref + slack))) {  // -infinity + slack is -infinity; a NaN becomes the reference, and with it the row
            const float now = larger(ref, m);
            const float f = ref == now ? 1.f : __builtin_amdgcn_exp2f((ref - now) * c);
            ref = now;
            sum *= f;
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[db][i] *= f;
        }
        const float base = ref == -INFINITY ? 0.f : LIFT - ref * c;  // a row that has seen nothing yet
        float part[4] = {0.f, 0.f, 0.f, 0.f};  // chains that do not wait for each other
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[nb][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[nb][i], c, base));
                part[i & 3] += s[nb][i];
            }
        sum += (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const typename Vec8<T>::V p = pack8<T>(s[nb], 8 * t);
#pragma unroll
                for (int db = 0; db < DB; ++db) o[db] = mma<T>(cols_at<T, DP>(vt, at, 2 * nb + t, db), p, o[db]);
            }
        }
    }
};

// Row r of a sequence and key head: query token r / group, head r % group of those that share the key head.
template <typename TT, int DP>
__global__ __launch_bounds__(64 * kWaves, DP == 64 ? 4 : 2) void attn_fwd_kernel(AttnArgs p, int tiles) {
    typedef typename TT::type T;
    typedef Rows<T, DP> R;
    constexpr int BYTES = kKeys * Tile<DP>::ROW;
    // separate arrays: the compiler then sees that a tile's reads and the next one's loads touch different memory
    __shared__ __align__(16) uint8_t k_0[BYTES], v_0[BYTES], k_1[BYTES], v_1[BYTES];
    const maxsim_attn& a = p.a;
    Work w;
    if (!work_of(w, a.B, a.Hk, tiles * p.splits)) return;
    // with a causal bound the last rows see the most keys: first
    const int split = w.part / tiles, tile = tiles - 1 - w.part % tiles;
    const Seq s = sequence(a, w.b);
    const int G = p.group, D = a.D, rows = s.lq * G;
    if (a.zero_rest && p.splits == 1)
        zero_rest<T>(a.out, p.lse, a.lse_step, a.cu_q, a.B, a.rows_q, w.b, s.q0, s.lq, s.all_q, a.Hq, D, w.h * tiles + tile,
                     a.Hk * tiles, w.item(tiles, a.Hk), w.items);
    const int r0 = tile * kRows;
    if (r0 >= rows) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int shift = s.lk - s.lq;
    const int last = min(r0 + kRows, rows) - 1;
    const Span span = span_of(a, s.lk, r0 / G + shift, last / G + shift, kKeys);
    const int t0 = (int)((int64_t)span.tiles * split / p.splits), t1 = (int)((int64_t)span.tiles * (split + 1) / p.splits);

    const T* ks = first<T>(a.k, a.cu_k != nullptr, w.b, s.k0, w.h);
    const T* vs = first<T>(a.v, a.cu_k != nullptr, w.b, s.k0, w.h);
    Loader<DP, kKeys, kWaves> lk, lv;
    lk.init(wave, lane, a.k.token, D);
    lv.init(wave, lane, a.v.token, D);
    Walk<T> next;
    next.start(span, t0, kKeys, ks, vs, a.k.token, a.v.token);
    const auto load = [&](uint8_t* kt, uint8_t* vt) {
        const int left = span.end(next.t) - next.j;
        lk.load(next.k, left, a.k.token, D, kt, wave);
        lv.load(next.v, left, a.v.token, D, vt, wave);
        next.next(span, kKeys, ks, vs, a.k.token, a.v.token);
    };
    if (t0 < t1) load(k_0, v_0);  // on its way while the queries are read

    const int wr = r0 + wave * kRowsWave;
    const int r = min(wr + (lane & 31), rows - 1), token = r / G, head = w.h * G + r % G;
    const T* qs = first<T>(a.q, a.cu_q != nullptr, w.b, s.q0, 0);
    R row;
    row.start(qs + (int64_t)token * a.q.token + (int64_t)head * a.q.head, lane, D, token + shift, s.lk, a);
    // the wave's rows: the positions between which they lie
    const int p_lo = min(wr, rows - 1) / G + shift, p_hi = min(wr + kRowsWave - 1, rows - 1) / G + shift;
    const float c = a.scale * kLog2e, slack = 8.f / c;

    const auto all_see = [&](int j, int end) {
        return j + kKeys <= end && j + kKeys - 1 <= min(p_lo + a.right, s.lk - 1) && (j >= p_hi - a.left || j + kKeys <= a.sinks);
    };

    const auto work = [&](int t, const uint8_t* kt, const uint8_t* vt) {
        const int j = span.at(t, kKeys), end = span.end(t);
        if (wr >= rows) return;
        if (j > p_hi + a.right || (j + kKeys - 1 < p_lo - a.left && j >= a.sinks)) return;  // none sees any
        const bool all = all_see(j, end);
        uint32_t bits[kKeys / 32] = {};
        if (!all) {
#pragma unroll
            for (int nb = 0; nb < kKeys / 32; ++nb) bits[nb] = row.bits(j + 32 * nb, end, a.sinks, lane);
        }
        row.template step<kKeys / 32>(kt, vt, all, bits, c, slack);
    };
    for (int t = t0; t < t1; t += 2) {
        tile_ready();
        if (t + 1 < t1) load(k_1, v_1);
        work(t, k_0, v_0);
        if (t + 1 >= t1) break;
        tile_ready();
        if (t + 2 < t1) load(k_0, v_0);
        work(t + 1, k_1, v_1);
    }

    const float sum = swap_sum(row.sum), top = row.top(c, 0.f);
    const bool mine = wr + (lane & 31) < rows;
    const int64_t at = (first_row(a, s, w.b) + token) * a.Hq + head;
    if (p.splits == 1) {
        T* out = first<T>(a.out, a.cu_q != nullptr, w.b, s.q0, 0) + (int64_t)token * a.out.token + (int64_t)head * a.out.head;
        const float inv = is_zero(sum) ? 0.f : 1.f / sum;
        store_row<T, R::DB>(out, mine, row.o, inv, lane, D);
        if (p.lse && a.lse_step > 1) store_row<T, R::DB, true>(rest_of<T>(p, at), mine, row.o, inv, lane, D);
        if (p.lse && mine && lane < 32)
            p.lse[at * a.lse_step] = is_zero(sum) ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
    } else if (mine) {
        const int64_t part = (int64_t)split * p.rows * a.Hq + at;
        if (lane < 32) {
            p.part_ml[2 * part] = top;
            p.part_ml[2 * part + 1] = sum;
        }
        float* o = p.part_o + part * D;
#pragma unroll
        for (int db = 0; db < R::DB; ++db)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int d = 32 * db + 8 * q + 4 * (lane >> 5);
                if (d < D) {
                    f32x4 v = {row.o[db][4 * q], row.o[db][4 * q + 1], row.o[db][4 * q + 2], row.o[db][4 * q + 3]};
                    *reinterpret_cast<f32x4*>(o + d) = v;
                }
            }
    }
}

// Few rows of a key head (32 at most: a sequence's next token, a short query): the four waves take the same rows
// and every fourth tile of 32 keys each, in buffers of their own that no barrier orders; they are joined in LDS at the end.
template <typename TT, int DP>
__global__ __launch_bounds__(64 * kWaves, 1) void attn_fwd_few_kernel(AttnArgs p) {
    typedef typename TT::type T;
    typedef Rows<T, DP> R;
    constexpr int BYTES = kKeysFew * Tile<DP>::ROW;
    __shared__ __align__(16) uint8_t k_0[kWaves * BYTES], v_0[kWaves * BYTES], k_1[kWaves * BYTES], v_1[kWaves * BYTES];
    __shared__ __align__(16) float joined[kWaves][32][2];
    const maxsim_attn& a = p.a;
    Work w;
    if (!work_of(w, a.B, a.Hk, p.splits)) return;
    const int split = w.part;
    const Seq s = sequence(a, w.b);
    const int G = p.group, D = a.D, rows = s.lq * G;
    if (a.zero_rest && p.splits == 1)
        zero_rest<T>(a.out, p.lse, a.lse_step, a.cu_q, a.B, a.rows_q, w.b, s.q0, s.lq, s.all_q, a.Hq, D, w.h, a.Hk, w.item(1, a.Hk), w.items);
    if (rows <= 0) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int shift = s.lk - s.lq;
    const int p_lo = shift, p_hi = (rows - 1) / G + shift;
    const Span span = span_of(a, s.lk, p_lo, p_hi, kKeysFew);
    const int t0 = (int)((int64_t)span.tiles * split / p.splits), t1 = (int)((int64_t)span.tiles * (split + 1) / p.splits);
    const int r = min(lane & 31, rows - 1), token = r / G, head = w.h * G + r % G;
    R row;
    row.start(first<T>(a.q, a.cu_q != nullptr, w.b, s.q0, 0) + (int64_t)token * a.q.token + (int64_t)head * a.q.head, lane, D,
              token + shift, s.lk, a);
    const float c = a.scale * kLog2e, slack = 8.f / c;
    const T* ks = first<T>(a.k, a.cu_k != nullptr, w.b, s.k0, w.h);
    const T* vs = first<T>(a.v, a.cu_k != nullptr, w.b, s.k0, w.h);
    Loader<DP, kKeysFew, 1> lk, lv;
    lk.init(0, lane, a.k.token, D);
    lv.init(0, lane, a.v.token, D);
    constexpr int LOADS = 2 * Loader<DP, kKeysFew, 1>::N;  // on their way for the next tile
    const auto load = [&](int t, uint8_t* kt, uint8_t* vt) {
        // the reads of what these loads overwrite are done, not only on their way
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        asm volatile("" ::: "memory");
        const int j = span.at(t, kKeysFew), left = span.end(t) - j;
        lk.load(ks + (int64_t)j * a.k.token, left, a.k.token, D, kt + wave * BYTES, 0);
        lv.load(vs + (int64_t)j * a.v.token, left, a.v.token, D, vt + wave * BYTES, 0);
    };
    const auto work = [&](int t, const uint8_t* kt, const uint8_t* vt) {
        const int j = span.at(t, kKeysFew), end = span.end(t);
        const bool whole = j + 32 <= end && j + 31 <= min(p_lo + a.right, s.lk - 1) && (j >= p_hi - a.left || j + 32 <= a.sinks);
        const uint32_t bits = whole ? 0u : row.bits(j, end, a.sinks, lane);
        row.template step<1>(kt + wave * BYTES, vt + wave * BYTES, whole, &bits, c, slack);
    };
    const auto landed = [&](bool ahead) {  // the tile's loads; those of the next one may stay on their way
        asm volatile("" ::: "memory");
        if (ahead) __builtin_amdgcn_s_waitcnt((LOADS & 15) | ((LOADS >> 4) << 14) | 0x0F70);
        else __builtin_amdgcn_s_waitcnt(0x0F70);
        asm volatile("" ::: "memory");
    };
    int t = t0 + wave;
    if (t < t1) load(t, k_0, v_0);
    for (; t < t1; t += 2 * kWaves) {
        const bool one = t + kWaves < t1, two = t + 2 * kWaves < t1;
        if (one) load(t + kWaves, k_1, v_1);
        landed(one);
        work(t, k_0, v_0);
        if (!one) break;
        if (two) load(t + 2 * kWaves, k_0, v_0);
        landed(two);
        work(t + kWaves, k_1, v_1);
    }

    // the waves' parts: references and sums first, then out^T, scaled to the largest reference, added in order
    const float sum = swap_sum(row.sum), top = row.top(c, -INFINITY);
    if (lane < 32) {
        joined[wave][lane][0] = top;
        joined[wave][lane][1] = sum;
    }
    __syncthreads();  // all tiles are read: their memory takes the parts
    float most = -INFINITY, total = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) most = larger(most, joined[i][lane & 31][0]);
    const float f = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(top - most);
#pragma unroll
    for (int i = 0; i < kWaves; ++i)
        total += joined[i][lane & 31][0] == -INFINITY ? 0.f : joined[i][lane & 31][1] * __builtin_amdgcn_exp2f(joined[i][lane & 31][0] - most);
    constexpr int BLOCK = 16 * 64 * 4;  // bytes of a block of 32 columns: register by register, 64 lanes each
    // wave i's part in array i
    uint8_t* const mem = wave == 0 ? k_0 : wave == 1 ? v_0 : wave == 2 ? k_1 : v_1;
    static_assert(R::DB * BLOCK <= kWaves * BYTES, "a wave's part fits an array");
#pragma unroll
    for (int db = 0; db < R::DB; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) reinterpret_cast<float*>(mem)[(db * 16 + i) * 64 + lane] = row.o[db][i] * f;
    __syncthreads();
    // each wave sums DB / 4 blocks: registers of 8 columns at a time are spread over the waves
    const bool mine = (lane & 31) < rows;
    const int64_t at = (first_row(a, s, w.b) + token) * a.Hq + head;
    if (wave == 0 && mine && lane < 32) {
        if (p.splits == 1) {
            if (p.lse) p.lse[at * a.lse_step] = is_zero(total) ? -INFINITY : (most + __builtin_amdgcn_logf(total)) * kLn2;
        } else {
            const int64_t part = (int64_t)split * p.rows * a.Hq + at;
            p.part_ml[2 * part] = most == -INFINITY ? 0.f : most;
            p.part_ml[2 * part + 1] = total;
        }
    }
    const float inv = is_zero(total) ? 0.f : 1.f / total;
    for (int q = wave; q < R::DB * 4; q += kWaves) {  // 4 registers: columns 8 q + 4 (l / 32) on
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = (4 * q + i) * 64 + lane;
            v[i] = ((reinterpret_cast<const float*>(k_0)[e] + reinterpret_cast<const float*>(v_0)[e]) +
                    reinterpret_cast<const float*>(k_1)[e]) + reinterpret_cast<const float*>(v_1)[e];
        }
        const int d = 8 * q + 4 * (lane >> 5);
        if (!mine || d >= D) continue;
        if (p.splits == 1) {
            v *= inv;
            T* rest = rest_of<T>(p, at);
            store4<T>(first<T>(a.out, a.cu_q != nullptr, w.b, s.q0, 0) + (int64_t)token * a.out.token +
                          (int64_t)head * a.out.head + d,
                      rest ? rest + d : nullptr, v);
        } else {
            *reinterpret_cast<f32x4*>(p.part_o + ((int64_t)split * p.rows * a.Hq + at) * D + d) = v;
        }
    }
}

// Rows whose keys were split: their parts, joined in order.  GROUPS groups of 32 threads to a row (of one head), each thread 4
// columns of every GROUPS-th part, all of them on their way at once; the parts' references and sums are a lane's each.
// (One thread after the other over the parts took 30 us for 64; 8 groups 35 us for two parts of 8192 rows and 28 for 16 of 4096, where
// two groups take 8.4 for 16 of 2048.)
constexpr int kMostSplits = 64;
template <typename TT, int GROUPS>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs p, int row_groups) {
    typedef typename TT::type T;
    constexpr int ROWS = 8 / GROUPS, EACH = 8;
    static_assert(EACH * 8 == kMostSplits, "8 groups take all parts");
    __shared__ float factor[ROWS][kMostSplits];
    __shared__ __align__(16) f32x4 share[ROWS][GROUPS][32];
    const maxsim_attn& a = p.a;
    const int b = blockIdx.x / row_groups, g = blockIdx.x % row_groups;
    const Seq s = sequence(a, b);
    if (a.zero_rest)
        zero_rest<T>(a.out, p.lse, a.lse_step, a.cu_q, a.B, a.rows_q, b, s.q0, s.lq, s.all_q, a.Hq, a.D, g, row_groups,
                     (int)blockIdx.x, (int)gridDim.x);
    const int lane = threadIdx.x & 31, group = (threadIdx.x >> 5) % GROUPS, sub = (threadIdx.x >> 5) / GROUPS;
    const int r = min(g * ROWS + sub, s.lq * a.Hq - 1), d = lane * 4;
    if (g * ROWS >= s.lq * a.Hq) return;
    const bool mine = g * ROWS + sub < s.lq * a.Hq && d < a.D;
    const int token = r / a.Hq, head = r % a.Hq;
    const int64_t at = (first_row(a, s, b) + token) * a.Hq + head, step = p.rows * a.Hq;
    f32x4 part[EACH];
    const float* o = p.part_o + at * a.D + d;
#pragma unroll
    for (int n = 0; n < EACH; ++n) {
        const int i = group + GROUPS * n;
        part[n] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (i < p.splits && mine) part[n] = *reinterpret_cast<const f32x4*>(o + i * step * a.D);
    }
    // every wave makes its rows' factors for itself: of one row with up to 64 parts, or of two with up to 8
    constexpr int WIDE = GROUPS == 1 ? 32 : 64;
    const int i = threadIdx.x & (WIDE - 1);
    float top = -INFINITY, l = 0.f;
    if (i < p.splits) {
        l = p.part_ml[2 * (at + i * step) + 1];
        top = is_zero(l) ? -INFINITY : p.part_ml[2 * (at + i * step)];
    }
    float most = top;
#pragma unroll
    for (int x = 1; x < WIDE; x <<= 1) most = larger(most, __shfl_xor(most, x));
    const float f = is_zero(l) ? -1.f : __builtin_amdgcn_exp2f(top - most);  // -1: a part in which the row sees nothing
    float total = is_zero(l) ? 0.f : l * f;
#pragma unroll
    for (int x = 1; x < WIDE; x <<= 1) total += __shfl_xor(total, x);
    if (GROUPS <= 2 || threadIdx.x < 64) factor[sub][i] = f;
    __syncthreads();
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < EACH; ++n) {
        const int k = group + GROUPS * n;
        // (a factor that fell to 0 counts, as its product with a value that is not finite does; NaN too)
        if (k < p.splits && !(factor[sub][k] < 0.f)) sum += part[n] * factor[sub][k];
    }
    if constexpr (GROUPS > 1) {
        share[sub][group][lane] = sum;
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int k = 1; k < GROUPS; ++k) sum += share[sub][k][lane];
    }
    if (mine) {
        sum *= is_zero(total) ? 0.f : 1.f / total;
        T* rest = rest_of<T>(p, at);
        store4<T>(first<T>(a.out, a.cu_q != nullptr, b, s.q0, 0) + (int64_t)token * a.out.token + (int64_t)head * a.out.head + d,
                  rest ? rest + d : nullptr, sum);
        if (p.lse && lane == 0) p.lse[at * a.lse_step] = is_zero(total) ? -INFINITY : (most + __builtin_amdgcn_logf(total)) * kLn2;
    }
}

struct Plan {
    bool few;
    int tiles, splits;
    int64_t blocks;
};
int64_t rows_in_memory(const maxsim_attn& a) { return a.cu_q ? a.rows_q : (int64_t)a.B * a.max_q; }

// Keys are split where the rows alone do not fill the chip and the second launch, which joins the parts, costs less
// than what it spares.  Measured (us, one key head's worth of rows to a workgroup):
//     a next token, 16 / 2 heads of 128:  500 keys 10.4 whole, 11.6 in parts; 852 13.1, 11.7; 8192 65.9, 13.6; 32768 250, 19
//     512 tokens, 16 / 4 heads of 64:     768 keys 15.5 whole, 20.2 in parts; 1536 26.0, 23.8; 8192 117, 46
// As many workgroups as there are CUs (4 x next token, 32 / 8 heads, 8192 keys: 28.7, twice as many 33.1).  Twice as
// many for long keys where that makes no more than 8 parts, which one kind of join takes (16 / 4 heads of 128, 512 tokens,
// 32768 keys: 203 and 167, 8192: 66 and 63; 2 x 493 tokens, 12 / 6 heads, 12770 keys: 150 and 111; but 8 x 64 tokens, 8 / 2 heads, 8192
// keys, 16 parts: 41 and 62; 1024 tokens, 2048 keys: 53 and 59), and for a next token over long caches of
// lengths that differ (16 x 8192 to 32768 keys, 32 / 8 heads of 128: 292 and 274; of one length 367 and 370).
Plan plan_of(const maxsim_attn& a) {
    Plan p;
    const int64_t group = a.Hq / a.Hk, rows = (int64_t)a.max_q * group;
    p.few = rows <= kRowsWave;
    p.tiles = p.few ? 1 : (int)((rows + kRows - 1) / kRows);
    const int64_t base = (int64_t)p.tiles * a.Hk * a.B;
    // keys that a workgroup's rows may see
    int64_t keys = a.max_k;
    if (a.left >= 0 && a.right >= 0)
        keys = std::min<int64_t>(keys, (int64_t)a.left + a.right + std::min<int64_t>(rows, kRows) / group + 2 + a.sinks);
    const int64_t from = p.few ? 640 : 1024, least = p.few && keys < 4096 ? 128 : 256;  // keys to be split; of a part
    const bool ragged = a.k_lens || a.cu_k;
    const int64_t wanted = keys >= 8192 && (p.few ? ragged : 512 <= 8 * base) ? 512 : 256;
    p.splits = 1;
    // (of no rows, those of no sequence are still to be made 0, by the one kernel: the join has nothing to join)
    if (base > 0 && rows > 0 && keys >= from) p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({wanted / base, keys / least, kMostSplits}));
    p.blocks = blocks_for((int64_t)a.Hk * a.B, (int64_t)p.tiles * p.splits);
    return p;
}

template <typename TT, int DP>
void launch(const AttnArgs& p, const Plan& plan, hipStream_t stream) {
    if (plan.few)
        attn_fwd_few_kernel<TT, DP><<<(unsigned)plan.blocks, 64 * kWaves, 0, stream>>>(p);
    else
        attn_fwd_kernel<TT, DP><<<(unsigned)plan.blocks, 64 * kWaves, 0, stream>>>(p, plan.tiles);
}

}  // namespace

size_t attn_fwd_workspace_bytes(const maxsim_attn& a) {
    const Plan plan = plan_of(a);
    if (plan.splits == 1) return 0;
    return (size_t)plan.splits * (size_t)rows_in_memory(a) * a.Hq * (a.D + 2) * sizeof(float);
}

bool attn_grid_ok(const maxsim_attn& a) {
    const int64_t most = (int64_t)1 << 21, pairs = (int64_t)a.Hk * a.B;
    const int64_t q_tiles = ((int64_t)a.max_q * (a.Hq / a.Hk) + kRows - 1) / kRows, k_tiles = ((int64_t)a.max_k + kRows - 1) / kRows;
    return pairs < most && (std::max(q_tiles, k_tiles) + 1) * pairs < most;
}

hipError_t launch_attn_fwd(const maxsim_attn& a, float* lse, void* workspace, hipStream_t stream) {
    const Plan plan = plan_of(a);
    AttnArgs p{};
    p.a = a;
    if (a.left < 0 || a.left > kNoBound) p.a.left = kNoBound;
    if (a.right < 0 || a.right > kNoBound) p.a.right = kNoBound;
    p.lse = lse;
    p.group = a.Hq / a.Hk;
    p.splits = plan.splits;
    p.rows = rows_in_memory(a);
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = p.part_o + (size_t)plan.splits * p.rows * a.Hq * a.D;
    const bool half = a.dtype == MAXSIM_F16;
    (void)hipGetLastError();  // an error that an earlier call left unread is not this one's
    if (a.D <= 64) half ? launch<F16, 64>(p, plan, stream) : launch<BF16, 64>(p, plan, stream);
    else half ? launch<F16, 128>(p, plan, stream) : launch<BF16, 128>(p, plan, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || plan.splits == 1) return e;
    // the rows are few, or the parts are
    const int each = plan.splits <= 8 ? 8 : plan.splits <= 16 ? 4 : 1;  // rows of a workgroup
    const int groups = (a.max_q * a.Hq + each - 1) / each;
    const auto join = each == 8   ? (half ? attn_join_kernel<F16, 1> : attn_join_kernel<BF16, 1>)
                      : each == 4 ? (half ? attn_join_kernel<F16, 2> : attn_join_kernel<BF16, 2>)
                                  : (half ? attn_join_kernel<F16, 8> : attn_join_kernel<BF16, 8>);
    join<<<(unsigned)groups * a.B, 256, 0, stream>>>(p, groups);
    return hipGetLastError();
}

}  // namespace maxsim
