// attn_dev.h -- device code shared by attention's forward and backward: where a
// sequence lies, tiles of rows in LDS that are read both as rows and transposed,
// and which keys a query sees.
//
// Everything is built on the 32x32x16 matrix instruction D = A B + C.  A lane
// gives row l % 32 of A and column l % 32 of B, 8 values along the sum from
// 8 * (l / 32) on; of D it holds column l % 32 and the 16 rows
// slot(l / 32, i) = 8 (i / 4) + 4 (l / 32) + i % 4.  So what one product leaves in
// registers (keys x queries) is the B operand of the next (whose sum runs over the keys),
// provided that product's A operand takes the keys in the slots' order: the
// transposing LDS read gives 4 rows that follow each other to a lane, which is that order.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "encoder_dev.h"
#include "layers.h"

namespace maxsim {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef __attribute__((address_space(3))) void* lptr_t;
typedef __attribute__((address_space(3))) s16x4* ltr_t;
typedef const __attribute__((address_space(4))) int32_t* cint_ptr;  // read-only for the kernel: scalar loads

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <typename T>
struct Vec8 {
    typedef T V __attribute__((ext_vector_type(8)));
};

template <typename T>
__device__ __forceinline__ f32x16 mma(typename Vec8<T>::V a, typename Vec8<T>::V b, f32x16 c) {
    if constexpr (std::is_same<T, _Float16>::value) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    } else {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
}
__device__ __forceinline__ f32x16 zero16() {
    f32x16 z;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.f;
    return z;
}
// The row of D in register i, without the lane's 4 * (l / 32).
__device__ __forceinline__ constexpr int slot(int i) { return 8 * (i >> 2) + (i & 3); }

// The larger one; NaN if either is (fmaxf would drop it, and costs an instruction more for each value whose NaN may be of
// the signalling kind).
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float swap_max(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(fbits(v), fbits(v), false, false);
    return larger(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float swap_sum(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(fbits(v), fbits(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Whether a sum of exponentials is 0: no key was seen.
__device__ __forceinline__ bool is_zero(float v) { return (fbits(v) << 1) == 0; }

// One sequence: its rows' places, lengths, and how far queries' positions are shifted.
struct Seq {
    int64_t q0, k0;  // first rows, where packed
    int lq, lk;
    int64_t all_q, all_k;  // rows up to the next sequence
};
__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }
__device__ __forceinline__ Seq sequence(const maxsim_attn& a, int b) {
    Seq s;
    if (a.cu_q) {
        s.q0 = clamp64(((cint_ptr)a.cu_q)[b], 0, a.rows_q);
        s.all_q = clamp64(clamp64(((cint_ptr)a.cu_q)[b + 1], 0, a.rows_q) - s.q0, 0, a.rows_q);
        s.lq = (int)clamp64(s.all_q, 0, a.max_q);
    } else {
        s.q0 = 0;
        s.all_q = a.max_q;
        s.lq = a.q_lens ? (int)clamp64(((cint_ptr)a.q_lens)[b], 0, a.max_q) : a.max_q;
    }
    if (a.cu_k) {
        s.k0 = clamp64(((cint_ptr)a.cu_k)[b], 0, a.rows_k);
        s.all_k = clamp64(clamp64(((cint_ptr)a.cu_k)[b + 1], 0, a.rows_k) - s.k0, 0, a.rows_k);
        s.lk = (int)clamp64(s.all_k, 0, a.max_k);
    } else {
        s.k0 = 0;
        s.all_k = a.max_k;
        s.lk = a.k_lens ? (int)clamp64(((cint_ptr)a.k_lens)[b], 0, a.max_k) : a.max_k;
    }
    return s;
}
// A sequence's first row of head h.
template <typename T>
__device__ __forceinline__ T* first(const maxsim_view& v, bool packed, int b, int64_t row0, int h) {
    return (T*)v.data + (packed ? row0 * v.token : (int64_t)b * v.batch) + (int64_t)h * v.head;
}
// The same row among all rows of q (of lse, row_stat and the parts).
__device__ __forceinline__ int64_t first_row(const maxsim_attn& a, const Seq& s, int b) {
    return a.cu_q ? s.q0 : (int64_t)b * a.max_q;
}

// The keys that a workgroup's rows see, cut into tiles: `first` tiles over the keys [0, sinks) that lie
// before the window, then [lo, hi).  What none of the rows sees is in no tile and is not read: entries that were
// dropped from a cache may hold anything, and 0 times a NaN is not 0.
struct Span {
    int lo, hi, sink_end, first, tiles;
    __device__ __forceinline__ int at(int t, int step) const { return t < first ? t * step : lo + (t - first) * step; }
    __device__ __forceinline__ int end(int t) const { return t < first ? sink_end : hi; }
};
__device__ __forceinline__ Span span_of(const maxsim_attn& a, int lk, int p_lo, int p_hi, int step) {
    Span s;
    s.lo = max(0, p_lo - a.left);
    s.hi = max(min(lk, p_hi + a.right + 1), 0);
    if (s.lo <= a.sinks) s.lo = 0;  // first tokens that reach into the window: no tiles of their own
    s.sink_end = min(min(a.sinks, s.lo), lk);
    s.first = (s.sink_end + step - 1) / step;
    s.tiles = s.first + (max(s.hi - s.lo, 0) + step - 1) / step;
    return s;
}

// The tiles of a span one after the other, from tile t0 on: the key that the next one starts with, and where k and v lie
// there.
template <typename T>
struct Walk {
    const T *k, *v;
    int j, t;
    __device__ __forceinline__ void start(const Span& s, int t0, int step, const T* k0, const T* v0, int64_t kt, int64_t vt) {
        t = t0;
        j = s.at(t0, step);
        k = k0 + (int64_t)j * kt;
        v = v0 + (int64_t)j * vt;
    }
    __device__ __forceinline__ void next(const Span& s, int step, const T* k0, const T* v0, int64_t kt, int64_t vt) {
        ++t;
        if (t == s.first) {  // on to the window
            j = s.lo;
            k = k0 + (int64_t)j * kt;
            v = v0 + (int64_t)j * vt;
        } else {
            j += step;
            k += step * kt;
            v += step * vt;
        }
    }
};

// What a block works on: sequence b, key head h, and one of the `each` parts of their work.  Blocks go round-robin over
// the 8 XCDs; the parts of one (b, h) read the same keys and go to one XCD, whose L2 holds them.  Many (b, h), of
// lengths that differ, are dealt out in turn; few of them in runs, which leave no XCD without work (16 sequences of
// 700 to 1024 tokens and 4 key heads: the forward 165 us in runs, 146 dealt out).
struct Work {
    int b, h, part;
    int items;  // in all: B * Hk * each
    __device__ __forceinline__ int item(int each, int Hk) const { return (b * Hk + h) * each + part; }
};
inline __host__ __device__ bool dealt(int64_t pairs) { return pairs % 8 == 0 || pairs >= 64; }
// Blocks to launch for that.
inline int64_t blocks_for(int64_t pairs, int64_t each) { return (dealt(pairs) ? ceil_div(pairs, 8) * 8 : pairs) * each; }
// False: nothing for this block.
__device__ __forceinline__ bool work_of(Work& w, int B, int Hk, int each) {
    const int pairs = B * Hk, xcd = blockIdx.x & 7, at = (int)(blockIdx.x >> 3);
    int pair;
    if (dealt(pairs)) {
        pair = at / each * 8 + xcd;
        w.part = at % each;
    } else {
        const int total = gridDim.x, run = total >> 3, more = total & 7;
        const int id = xcd * run + min(xcd, more) + at;
        pair = id / each;
        w.part = id % each;
    }
    w.b = pair / Hk;
    w.h = pair % Hk;
    w.items = pairs * each;
    return pair < pairs;
}

// A lane's values of a block of 32 keys (or rows), in the slots' order, as bits: those from `low` up to `top`, and those
// below `sink`, all counted from the lane's first slot.
__device__ __forceinline__ uint32_t slots_below(int n) {  // n slots' worth of bits below place n
    n = max(0, min(n, 32));
    const uint32_t count = 4 * (n >> 3) + min(n & 7, 4);
    return (1u << count) - 1;  // 16 at most
}
__device__ __forceinline__ uint32_t slots_seen(int low, int top, int sink) {
    return slots_below(top + 1) & (~slots_below(low) | slots_below(sink));
}
__device__ __forceinline__ float keep(uint32_t bits, int i, float v, uint32_t other) {
    const uint32_t m = (uint32_t)((int)(bits << (31 - i)) >> 31);
    return __uint_as_float((fbits(v) & m) | (other & ~m));
}
constexpr uint32_t kMinusInfinity = 0xff800000u;

// A tile in LDS: rows of DP values (DP * 2 bytes = NCH chunks of 16 bytes), chunk c of row r at
// place c ^ turn(r) of its row.  16 rows that follow each other, read at one chunk, lie in 16 different
// 16-byte columns of LDS's 256; so do the 4 rows x 64 bytes that a transposing read of 32 lanes takes.
template <int DP>
struct Tile {
    static constexpr int NCH = DP / 8, ROW = DP * 2;
    static __device__ __forceinline__ int turn(int r) {
        if constexpr (NCH == 16) return ((r & 3) << 2) | ((r >> 2) & 3);
        else return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
    }
};

// This wave's part of a tile's direct HBM -> LDS loads: 64 lanes x 16 bytes each.  A lane's slot is fixed
// by the instruction, so the lane that fills chunk place s of row r fetches chunk s ^ turn(r).
template <int DP, int ROWS, int WAVES>
struct Loader {
    typedef Tile<DP> TL;
    static constexpr int N = ROWS * TL::NCH / 64 / WAVES, PER = 64 / TL::NCH;  // loads; rows to a load
    uint32_t off[N];
    __device__ __forceinline__ void init(int wave, int lane, int64_t token, int D) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int row = (wave * N + n) * PER + lane / TL::NCH;
            const int c = (lane % TL::NCH) ^ TL::turn(row);
            off[n] = c * 8 < D ? (uint32_t)(row * (int)(token * 2) + c * 16) : 0xFFFFFFF0u;
        }
    }
    // rows [0, left) of the tile at `base`; the others (and columns past D) become zeros
    __device__ __forceinline__ void load(const void* base, int left, int64_t token, int D, uint8_t* lds, int wave) const {
        left = min(left, ROWS);
        const uint32_t bytes = left > 0 ? (uint32_t)((left - 1) * (int)(token * 2) + D * 2) : 0u;
        const uint64_t a = (uint64_t)base;
        const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
        const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            (void*)(((uint64_t)hi << 32) | lo), (short)0, (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000);
#pragma unroll
        for (int n = 0; n < N; ++n)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lptr_t)(lds + (wave * N + n) * 1024), 16, (int)off[n], 0, 0, 0);
    }
};

// Where a lane reads: its first place of either kind, from which the others differ by an exclusive or (a place's turn does
// not reach beyond its row).
struct Place {
    int rows, cols;
};
template <int DP>
__device__ __forceinline__ Place place_of(int lane) {
    const int r = lane & 31, k = 4 * (lane >> 5) + ((lane & 15) >> 2), c = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    return {r * Tile<DP>::ROW + (((lane >> 5) ^ Tile<DP>::turn(r)) << 4),
            k * Tile<DP>::ROW + ((c ^ Tile<DP>::turn(k)) << 4) + ((lane & 1) << 3)};
}
// A operand from a tile's rows: row l % 32 of a block of 32, values 16 kk + 8 (l / 32) on.
template <typename T, int DP>
__device__ __forceinline__ typename Vec8<T>::V rows_at(const uint8_t* block, const Place& at, int kk) {
    return *reinterpret_cast<const typename Vec8<T>::V*>(block + (at.rows ^ (kk << 5)));
}
// A operand from a tile transposed: column 32 db + l % 32 of its rows slot(l / 32, 0 .. 7) from row 16 t of `block` on.
// (8 rows further the turn differs by 2.)
template <typename T, int DP>
__device__ __forceinline__ typename Vec8<T>::V cols_at(const uint8_t* block, const Place& at, int t, int db) {
    const uint8_t* from = block + 16 * t * Tile<DP>::ROW;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ltr_t)(from + (at.cols ^ (db << 6))));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ltr_t)(from + 8 * Tile<DP>::ROW + (at.cols ^ (db << 6) ^ 32)));
    return __builtin_bit_cast(typename Vec8<T>::V, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
// B operand from memory: 8 values of a row from column c on, zeros from column D on.
template <typename T>
__device__ __forceinline__ typename Vec8<T>::V row8(const T* row, int c, int D) {
    typename Vec8<T>::V v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (T)0.f;
    if (c < D) v = *reinterpret_cast<const typename Vec8<T>::V*>(row + c);
    return v;
}
// 8 registers of D as the B operand of the next product.
template <typename T>
__device__ __forceinline__ typename Vec8<T>::V pack8(const f32x16& d, int at) {
    typename Vec8<T>::V v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (T)d[at + i];
    return v;
}

// This wave's direct loads have landed; then the workgroup's barrier (__syncthreads would also wait for
// what was loaded ahead).
__device__ __forceinline__ void tile_ready() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// D^T in registers (DB blocks of 32 columns x this lane's row) times k to a row of T: the lane halves trade
// 4 values so that each lane stores 16 bytes.  REST: what the values' rounding to T leaves off, in their place (rows
// of 4-byte alignment).  Every lane takes part; `row` is used where `mine`.
template <typename T, int DB, bool REST = false>
__device__ __forceinline__ void store_row(T* row, bool mine, const f32x16* o, float k, int lane, int D) {
    typedef T V4 __attribute__((ext_vector_type(4)));
    typedef typename std::conditional<REST, u32x4_any, u32x4>::type U4;
#pragma unroll
    for (int db = 0; db < DB; ++db) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            V4 a, b;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = o[db][8 * h + i] * k, y = o[db][8 * h + 4 + i] * k;
                a[i] = (T)x;
                b[i] = (T)y;
                if (REST) {
                    a[i] = (T)(x - (float)a[i]);
                    b[i] = (T)(y - (float)b[i]);
                }
            }
            const u32x2 ua = __builtin_bit_cast(u32x2, a), ub = __builtin_bit_cast(u32x2, b);
            const auto s0 = __builtin_amdgcn_permlane32_swap(ua[0], ub[0], false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(ua[1], ub[1], false, false);
            const u32x4 v = {s0[0], s1[0], s0[1], s1[1]};
            const int c = 32 * db + 16 * h + 8 * (lane >> 5);
            if (mine && c < D) *reinterpret_cast<U4*>(row + c) = v;
        }
    }
}
// 4 values in fp32 to a row of T, and what their rounding leaves off to another (or nullptr).
template <typename T>
__device__ __forceinline__ void store4(T* row, T* rest, f32x4 v) {
    typedef T V4 __attribute__((ext_vector_type(4)));
    typedef T R4 __attribute__((ext_vector_type(4), aligned(4)));
    V4 y;
    R4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[i] = (T)v[i];
        r[i] = (T)(v[i] - (float)y[i]);
    }
    *reinterpret_cast<V4*>(row) = y;
    if (rest) *reinterpret_cast<R4*>(rest) = r;
}
// Where a row's rest is kept, behind its lse; nullptr where it is not.
template <typename T>
__device__ __forceinline__ T* rest_of(const AttnArgs& p, int64_t at) {
    return p.lse && p.a.lse_step > 1 ? reinterpret_cast<T*>(p.lse + at * p.a.lse_step + 1) : nullptr;
}

// Rows from, from + step, .. before `to` of a view become 0 (and the same rows of lse, where there is one).
template <typename T>
__device__ __forceinline__ void zero_rows(T* row0, int64_t token, int64_t head, float* lse, int lse_step, int64_t from,
                                          int64_t to, int64_t step, int heads, int D) {
    const int each = D / 8;
    for (int64_t t = from; t < to; t += step) {
        for (int i = threadIdx.x; i < heads * each; i += blockDim.x) {
            const int h = i / each;
            *reinterpret_cast<u32x4*>(row0 + t * token + (int64_t)h * head + (i - h * each) * 8) = u32x4{0, 0, 0, 0};
        }
        if (lse)
            for (int i = threadIdx.x; i < heads; i += blockDim.x) lse[(t * heads + i) * lse_step] = 0.f;
    }
}
// The rows that belong to no sequence: [len, all) of sequence b, shared out over `parts` workgroups, and of
// packed rows those before the first sequence and past the last, over all `items`.
template <typename T>
__device__ __forceinline__ void zero_rest(const maxsim_view& v, float* lse, int lse_step, const int32_t* cu, int B, int64_t rows, int b,
                                          int64_t row0, int len, int64_t all, int heads, int D, int part, int parts,
                                          int item, int items) {
    const int64_t at = cu ? row0 : (int64_t)b * all;  // of lse
    zero_rows<T>(first<T>(v, cu != nullptr, b, row0, 0), v.token, v.head, lse ? lse + at * heads * lse_step : nullptr, lse_step,
                 (int64_t)len + part, all, parts, heads, D);
    if (!cu) return;
    int64_t low = clamp64(((cint_ptr)cu)[0], 0, rows), high = clamp64(((cint_ptr)cu)[B], 0, rows);
    // Some workgroups do it, 16 rows each and more: should the starts not be in order, another one's sequence may lie there, and each
    // looks through all of them first (4096 sequences of 32 and 1000 rows behind: 841 us forward and backward where every workgroup did
    // that, 468 so, 461 where none does).
    items = (int)min((int64_t)items, 64 + (low + rows - high) / 16);
    if (item >= items) return;
    if (low > 0 || high < rows) {
        int least = INT32_MAX, most = 0;
#pragma unroll 8
        for (int i = threadIdx.x & 63; i < B; i += 64) {
            const int from = cu[i], to = cu[i + 1];
            if (from >= to) continue;
            least = min(least, from);
            most = max(most, to);
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            least = min(least, __shfl_xor(least, d));
            most = max(most, __shfl_xor(most, d));
        }
        low = clamp64(least, 0, rows);  // (of no rows at all in any sequence, all)
        high = max(clamp64(most, 0, rows), low);
    }
    zero_rows<T>((T*)v.data, v.token, v.head, lse, lse_step, item, low, items, heads, D);
    zero_rows<T>((T*)v.data, v.token, v.head, lse, lse_step, high + item, rows, items, heads, D);
}

}  // namespace
}  // namespace maxsim
