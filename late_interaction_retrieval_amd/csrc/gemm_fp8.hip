// gemm_fp8.hip -- product of two e4m3 matrices with a scale for each 128 along
// K, for gfx950 (MI355X).
//
//     c[m, n] = sum_kb sa[m, kb] sb[n or n / 128, kb] sum_{k in kb} A[m, k] B[n, k]
//
// One v_mfma_f32_16x16x128_f8f6f4 contracts exactly one block of 128, so its
// result, started from 0, is the block's unscaled sum, and one fused multiply-add a value
// (4 for 65,536 flop) adds it, scaled, to the fp32 accumulator: a quarter of
// an MFMA's cycles each, on the VALU beside the matrix pipe.
//   * Rows of B are the MFMA's rows and rows of A its columns: a lane then holds
//     values of one row of A, whose scale is one register, and neighbouring
//     columns of c, which leave in 16-byte stores.
//   * Tiles go HBM -> LDS by direct loads into two buffers, 128 bytes of K a
//     step; 16-byte chunks are XOR-swizzled so that operand reads hit all banks.
//   * Workgroups that share rows of A or B follow each other on one XCD.
//   * Where tiles are few, K is split over workgroups whose fp32 partial sums
//     a second launch adds in order.
//   * Up to 64 rows of A (single queries) take a kernel bound by the bytes of B:
//     operands go straight to registers and a workgroup's waves split K.
#include <algorithm>
#include <type_traits>

#include "encoder_dev.h"

namespace maxsim {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lptr_t;

constexpr int kStep = kQBlock;  // bytes of K a step
constexpr uint32_t kOutside = 0xF0000000u;  // an offset past any buffer: reads zeros

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// An operand of one MFMA block: a lane's 32 bytes, or their 32 values in fp16
// (which holds every e4m3 value).
template <bool FINE>
struct Operand {
    i32x8 v;
};
template <>
struct Operand<true> {
    f16x8 v[4];
};
template <bool FINE>
__device__ __forceinline__ Operand<FINE> operand_of(i32x8 bytes) {
    Operand<FINE> o;
    if constexpr (FINE) {
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((unsigned)bytes[w], 1.f, false);
            const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((unsigned)bytes[w], 1.f, true);
            o.v[w >> 1][(w & 1) * 4 + 0] = lo[0];
            o.v[w >> 1][(w & 1) * 4 + 1] = lo[1];
            o.v[w >> 1][(w & 1) * 4 + 2] = hi[0];
            o.v[w >> 1][(w & 1) * 4 + 3] = hi[1];
        }
    } else {
        o.v = bytes;
    }
    return o;
}

// The unscaled sum of one block of 128.  The 8-bit instruction aligns a block's
// products to the largest and keeps about 13 bits below it (measured against
// exact sums of normal values: 1.4e-5 relative, at most 2^-13.4 of the largest product; 2 bits
// fewer than a 16-bit result needs).  An fp32 result takes the values through fp16, whose
// products and sums are exact to fp32 (1.2e-8), at half the rate.
template <bool FINE>
__device__ __forceinline__ f32x4 mfma(const Operand<FINE>& b, const Operand<FINE>& a) {
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
    if constexpr (FINE) {
#pragma unroll
        for (int q = 0; q < 4; ++q) d = __builtin_amdgcn_mfma_f32_16x16x32_f16(b.v[q], a.v[q], d, 0, 0, 0);
    } else {
        // both scale operands 0: the compiler emits the instruction without scales
        d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a.v, d, 0, 0, 0, 0, 0, 0);
    }
    return d;
}
__device__ __forceinline__ i32x8 join(u32x4 lo, u32x4 hi) {
    return __builtin_bit_cast(i32x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Direct HBM -> LDS load of `size` (4 or 16) bytes a lane: lane l's bytes at
// base + voff land at lds + l * size; bytes past nbytes read as zero without a
// memory access.  base and nbytes are wave-uniform.
template <int SIZE>
__device__ __forceinline__ void load_lds(const void* base, uint32_t nbytes, uint32_t voff, lptr_t lds) {
    const uint64_t a = (uint64_t)base;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
    const uint32_t n = __builtin_amdgcn_readfirstlane(nbytes);
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc((void*)(((uint64_t)hi << 32) | lo), (short)0, (int)n, 0x00020000);
    if constexpr (SIZE == 16)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds, 16, (int)voff, 0, 0, 0);
    else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds, 4, (int)voff, 0, 0, 0);
}

// Every direct load of this wave has landed; then the workgroup's barrier, for
// LDS only (__syncthreads would not keep the next tile's loads in flight).
__device__ __forceinline__ void tile_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// 4 (a vector) neighbouring values of a row of c, rounded once.
__device__ __forceinline__ void store4(const GemmArgs& p, int64_t row, int n, f32x4 v) {
    typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
    typedef __bf16 bf16x4u __attribute__((ext_vector_type(4), aligned(2)));
    typedef _Float16 f16x4u __attribute__((ext_vector_type(4), aligned(2)));
    if (n >= p.N) return;
    const int64_t at = row * p.ldc + n;
    const int left = p.N - n;
    if (p.out_dtype == MAXSIM_F32) {
        float* c = (float*)p.c + at;
        if (left >= 4)
            *reinterpret_cast<f32x4u*>(c) = v;
        else
            for (int i = 0; i < left; ++i) c[i] = v[i];
    } else if (p.out_dtype == MAXSIM_BF16) {
        __bf16* c = (__bf16*)p.c + at;
        bf16x4u w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (__bf16)v[i];
        if (left >= 4)
            *reinterpret_cast<bf16x4u*>(c) = w;
        else
            for (int i = 0; i < left; ++i) c[i] = w[i];
    } else {
        _Float16* c = (_Float16*)p.c + at;
        f16x4u w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (_Float16)v[i];
        if (left >= 4)
            *reinterpret_cast<f16x4u*>(c) = w;
        else
            for (int i = 0; i < left; ++i) c[i] = w[i];
    }
}

struct TilePlan {
    int tiles_m, tiles_n, splits;
    int steps;      // of K in all
    int per_split;  // of K in a split (the last may have fewer)
};

// A workgroup of WGM x WGN waves makes a tile of TM rows of A x TN rows of B; a
// wave makes (TM / WGM) x (TN / WGN), which lies within 128 rows of B.
// ROWS: b_scale by the row; FINE: products in fp16
template <int TM, int TN, int WGM, int WGN, bool ROWS, bool FINE>
__global__ __launch_bounds__(64 * WGM * WGN) void gemm_tile_kernel(GemmArgs p, TilePlan plan) {
    constexpr int WAVES = WGM * WGN;
    constexpr int NI = TM / WGM / 16, NJ = TN / WGN / 16;
    constexpr int LA = TM / 8 / WAVES, LB = TN / 8 / WAVES;  // a wave's direct loads of 8 rows
    constexpr int SCALES = TM + (ROWS ? TN : 0);
    static_assert(LA * 8 * WAVES == TM && LB * 8 * WAVES == TN && TN / WGN <= kQBlock, "tile");
    __shared__ __align__(16) uint8_t tile[2][(TM + TN) * kStep];
    __shared__ __align__(16) float scale[2][SCALES];
    const int tid = threadIdx.x;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // Workgroups go round-robin over the 8 XCDs: give each XCD a run of
    // neighbouring tiles, in columns of 8 tiles of A, that share operands in its L2.
    const int total = plan.tiles_m * plan.tiles_n * plan.splits;
    const int xcd = blockIdx.x & 7, each = total >> 3, more = total & 7;
    int id = xcd * each + min(xcd, more) + (blockIdx.x >> 3);
    const int per_z = plan.tiles_m * plan.tiles_n;
    const int z = id / per_z;
    id -= z * per_z;
    const int band = id / (8 * plan.tiles_n);
    const int high = min(8, plan.tiles_m - 8 * band);
    const int rest = id - band * 8 * plan.tiles_n;
    const int m0 = (band * 8 + rest % high) * TM, n0 = (rest / high) * TN;
    const int k_begin = z * plan.per_split, k_end = min(plan.steps, k_begin + plan.per_split);

    const int rows_a = min(TM, p.M - m0), rows_b = min(TN, p.N - n0);
    const uint32_t k16 = ((uint32_t)p.K + 15u) & ~15u;  // readable bytes of a row that are used
    const uint8_t* base_a = p.A + (int64_t)m0 * p.lda;
    const uint8_t* base_b = p.B + (int64_t)n0 * p.ldb;
    const uint32_t bytes_a = (uint32_t)(rows_a - 1) * (uint32_t)p.lda + k16;
    const uint32_t bytes_b = (uint32_t)(rows_b - 1) * (uint32_t)p.ldb + k16;

    // LDS row r holds its 16-byte chunk c at position c ^ swizzle(r).  The
    // 16 rows a wave reads at once are neighbours in A; in B they are 4 runs of 4
    // rows, 4 * NJ apart, so that a lane's NJ results are neighbouring columns of c.
    auto swz_a = [](int r) { return (r >> 1) & 7; };
    auto swz_b = [](int r) { return ((r >> 1) & 1) | (((r / (4 * NJ)) & 3) << 1); };

    // this lane's part of each direct load: row (group * 8 + lane / 8), position lane % 8
    uint32_t off_a[LA], off_b[LB];
    uint32_t chunk_a[LA], chunk_b[LB];
#pragma unroll
    for (int j = 0; j < LA; ++j) {
        const int r = (wave * LA + j) * 8 + (lane >> 3);
        chunk_a[j] = (uint32_t)((lane & 7) ^ swz_a(r)) * 16;
        off_a[j] = r < rows_a ? (uint32_t)r * (uint32_t)p.lda : kOutside;
    }
#pragma unroll
    for (int j = 0; j < LB; ++j) {
        const int r = (wave * LB + j) * 8 + (lane >> 3);
        chunk_b[j] = (uint32_t)((lane & 7) ^ swz_b(r)) * 16;
        off_b[j] = r < rows_b ? (uint32_t)r * (uint32_t)p.ldb : kOutside;
    }
    const float* sa = p.a_scale + (int64_t)m0 * plan.steps;
    const float* sb = p.b_scale + (int64_t)(ROWS ? n0 : n0 / kQBlock) * plan.steps;

    auto load = [&](int kb, int buf) {
        const uint32_t at = (uint32_t)kb * kStep;
#pragma unroll
        for (int j = 0; j < LA; ++j) {
            const uint32_t k = at + chunk_a[j];
            load_lds<16>(base_a, bytes_a, k < k16 ? off_a[j] + k : kOutside,
                         (lptr_t)&tile[buf][(wave * LA + j) * 8 * kStep]);
        }
#pragma unroll
        for (int j = 0; j < LB; ++j) {
            const uint32_t k = at + chunk_b[j];
            load_lds<16>(base_b, bytes_b, k < k16 ? off_b[j] + k : kOutside,
                         (lptr_t)&tile[buf][(TM + (wave * LB + j) * 8) * kStep]);
        }
        // scales: 64 rows a wave; rows past the end read 0
#pragma unroll
        for (int q = 0; q < SCALES / 64; ++q) {
            if (q % WAVES != wave) continue;
            const bool is_a = q < TM / 64;
            const int r = (is_a ? q : q - TM / 64) * 64 + lane;
            const int rows = is_a ? rows_a : rows_b;
            load_lds<4>(is_a ? sa : sb, (uint32_t)rows * (uint32_t)plan.steps * 4u,
                        r < rows ? ((uint32_t)r * (uint32_t)plan.steps + (uint32_t)kb) * 4u : kOutside,
                        (lptr_t)&scale[buf][q * 64]);
        }
    };

    const int wm = wave / WGN * (TM / WGM), wn = wave % WGN * (TN / WGN);
    const int col = lane & 15, grp = lane >> 4;
    const int row_b = wn + (col >> 2) * (4 * NJ) + (col & 3);  // + 4 j
    f32x4 acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (k_begin < k_end) load(k_begin, 0);
    for (int kb = k_begin; kb < k_end; ++kb) {
        const int buf = (kb - k_begin) & 1;
        float s_block = 1.f;
        if constexpr (!ROWS) {
            const int b = min(wn, rows_b - 1) / kQBlock;  // a wave past the last row: any scale
            s_block = sb[(int64_t)b * plan.steps + kb];
        }
        tile_barrier();
        if (kb + 1 < k_end) load(kb + 1, buf ^ 1);
        if (kb == plan.steps - 1 && (p.K & 15) != 0) {  // clear what follows K in its last chunk
            const int last = (p.K & (kStep - 1)) >> 4, keep = p.K & 15;
            for (int r = tid; r < TM + TN; r += 64 * WAVES) {
                const int s = r < TM ? swz_a(r) : swz_b(r - TM);
                uint32_t* w = reinterpret_cast<uint32_t*>(&tile[buf][r * kStep + (last ^ s) * 16]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int left = keep - 4 * i;
                    if (left < 4) w[i] = left <= 0 ? 0u : w[i] & ((1u << (8 * left)) - 1u);
                }
            }
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
        }
        auto operand = [&](int r, int s) {
            const uint8_t* w = &tile[buf][r * kStep];
            return join(*reinterpret_cast<const u32x4*>(w + ((2 * grp) ^ s) * 16),
                        *reinterpret_cast<const u32x4*>(w + ((2 * grp + 1) ^ s) * 16));
        };
        Operand<FINE> a[NI];
        float s[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int r = wm + i * 16 + col;
            a[i] = operand_of<FINE>(operand(r, swz_a(r)));
            s[i] = scale[buf][r] * s_block;
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int r = row_b + 4 * j;
            const Operand<FINE> b = operand_of<FINE>(operand(TM + r, swz_b(r)));
            f32x4 t = {1.f, 1.f, 1.f, 1.f};
            if constexpr (ROWS)
                t = *reinterpret_cast<const f32x4*>(&scale[buf][TM + wn + grp * (4 * NJ) + 4 * j]);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const f32x4 d = mfma<FINE>(b, a[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][j][e] = __builtin_fmaf(ROWS ? d[e] * t[e] : d[e], s[i], acc[i][j][e]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int m = m0 + wm + i * 16 + col;
        if (m >= p.M) continue;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int n = n0 + wn + grp * (4 * NJ) + 4 * j;
            if (plan.splits == 1) {
                store4(p, m, n, acc[i][j]);
            } else {  // N4 = N rounded up to 4: whole vectors
                const int64_t n4 = (p.N + 3) & ~3;
                if (n < p.N) *reinterpret_cast<f32x4*>(p.partial + ((int64_t)z * p.M + m) * n4 + n) = acc[i][j];
            }
        }
    }
}

// c = the splits' partial sums, added in order.
__global__ __launch_bounds__(256) void gemm_join_kernel(GemmArgs p, int splits) {
    const int n4 = (p.N + 3) >> 2;
    const int64_t each = (int64_t)p.M * n4;
    const f32x4* part = reinterpret_cast<const f32x4*>(p.partial);
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < each; k += (int64_t)gridDim.x * 256) {
        f32x4 v = part[k];
        for (int z = 1; z < splits; ++z) v += part[z * each + k];
        const int64_t row = k / n4;
        store4(p, row, (int)(k - row * n4) * 4, v);
    }
}

// Few rows of A (at most 16 * NI): a workgroup takes 16 rows of B, its 8 waves
// every 8th block of K each, operands straight from memory to registers.
template <int NI, bool ROWS, bool FINE>
__global__ __launch_bounds__(512) void gemm_rows_kernel(GemmArgs p, int steps) {
    __shared__ f32x4 part[8][NI][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, grp = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int rb = min(n0 + col, p.N - 1);  // rows past the end repeat the last one
    const uint8_t* b = p.B + (int64_t)rb * p.ldb + grp * 32;
    const uint8_t* a[NI];
    const float* sa[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int ra = min(i * 16 + col, p.M - 1);
        a[i] = p.A + (int64_t)ra * p.lda + grp * 32;
        sa[i] = p.a_scale + (int64_t)ra * steps;
    }
    const float* sb[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)  // results 4 grp + e of the 16 rows
        sb[e] = p.b_scale + (int64_t)(ROWS ? min(n0 + 4 * grp + e, p.N - 1) : n0 / kQBlock) * steps;
    f32x4 acc[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto fold = [&](int kb, i32x8 b_bytes, const i32x8* a_bytes) {
        const Operand<FINE> bv = operand_of<FINE>(b_bytes);
        f32x4 t;
        if constexpr (ROWS) {
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] = sb[e][kb];
        } else {
            const float s = sb[0][kb];
            t = f32x4{s, s, s, s};
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const f32x4 d = mfma<FINE>(bv, operand_of<FINE>(a_bytes[i]));
            const float s = sa[i][kb];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = __builtin_fmaf(d[e] * t[e], s, acc[i][e]);
        }
    };
    auto whole = [](const uint8_t* row) {
        return join(*reinterpret_cast<const u32x4*>(row), *reinterpret_cast<const u32x4*>(row + 16));
    };
    const int full = p.K / kStep;  // blocks without an end in them
    for (int kb = wave; kb < full; kb += 8) {
        const int64_t at = (int64_t)kb * kStep;
        i32x8 av[NI];
        const i32x8 bv = whole(b + at);
#pragma unroll
        for (int i = 0; i < NI; ++i) av[i] = whole(a[i] + at);
        fold(kb, bv, av);
    }
    if (full < steps && full % 8 == wave) {  // the last block: bytes from K on are 0
        const int64_t at = (int64_t)full * kStep;
        const int keep = p.K - (int)at - grp * 32;  // of this lane's 32 bytes
        auto tail = [&](const uint8_t* row) {
            u32x4 h[2] = {u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}};
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (keep > 16 * q) h[q] = *reinterpret_cast<const u32x4*>(row + 16 * q);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int left = keep - 16 * q - 4 * w;
                    if (left < 4) h[q][w] = left <= 0 ? 0u : h[q][w] & ((1u << (8 * left)) - 1u);
                }
            }
            return join(h[0], h[1]);
        };
        i32x8 av[NI];
        const i32x8 bv = tail(b + at);
#pragma unroll
        for (int i = 0; i < NI; ++i) av[i] = tail(a[i] + at);
        fold(full, bv, av);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    if (wave < NI) {  // wave i adds the 16 rows from 16 i on
        f32x4 v = part[0][wave][lane];
#pragma unroll
        for (int w = 1; w < 8; ++w) v += part[w][wave][lane];
        const int m = wave * 16 + col;
        if (m < p.M) store4(p, m, n0 + 4 * grp, v);
    }
}

constexpr int kFewRows = 64;
constexpr int kCUs = 256;

TilePlan plan_tiles(int M, int N, int K, int tm, int tn) {
    TilePlan t;
    t.tiles_m = (int)ceil_div(M, tm);
    t.tiles_n = (int)ceil_div(N, tn);
    t.steps = (int)ceil_div(K, kStep);
    const int64_t tiles = (int64_t)t.tiles_m * t.tiles_n;
    // fewer tiles than half the CUs: split K, at least 8 steps to a split
    int s = tiles * 2 > kCUs ? 1 : (int)(kCUs / tiles);
    s = std::max(1, std::min(s, t.steps / 8));
    t.per_split = (int)ceil_div(t.steps, s);
    t.splits = t.per_split ? (int)ceil_div(t.steps, t.per_split) : 1;
    t.splits = std::max(1, t.splits);
    return t;
}

// 256 x 256 tiles where they still give every CU one; else 128 x 128.
bool big_tiles(int M, int N) { return ceil_div(M, 256) * ceil_div(N, 256) >= kCUs / 2; }

template <typename F>
void by_kind(const GemmArgs& a, F&& go) {
    const bool rows = a.b_block_rows == 1, fine = a.out_dtype == MAXSIM_F32;
    if (rows && fine) return go(std::true_type{}, std::true_type{});
    if (rows) return go(std::true_type{}, std::false_type{});
    if (fine) return go(std::false_type{}, std::true_type{});
    return go(std::false_type{}, std::false_type{});
}

template <int TM, int TN, int WGM, int WGN>
void launch_tiles(const GemmArgs& a, const TilePlan& t, hipStream_t stream) {
    const unsigned grid = (unsigned)(t.tiles_m * t.tiles_n * t.splits);
    by_kind(a, [&](auto rows, auto fine) {
        gemm_tile_kernel<TM, TN, WGM, WGN, decltype(rows)::value, decltype(fine)::value>
            <<<grid, 64 * WGM * WGN, 0, stream>>>(a, t);
    });
}

template <int NI>
void launch_rows(const GemmArgs& a, hipStream_t stream) {
    const unsigned grid = (unsigned)ceil_div(a.N, 16);
    const int steps = (int)ceil_div(a.K, kStep);
    by_kind(a, [&](auto rows, auto fine) {
        gemm_rows_kernel<NI, decltype(rows)::value, decltype(fine)::value><<<grid, 512, 0, stream>>>(a, steps);
    });
}

}  // namespace

size_t gemm_fp8_workspace_bytes(int M, int N, int K) {
    if (M <= kFewRows || big_tiles(M, N)) return 0;
    const TilePlan t = plan_tiles(M, N, K, 128, 128);
    return t.splits == 1 ? 0 : (size_t)t.splits * M * (size_t)((N + 3) & ~3) * sizeof(float);
}

hipError_t launch_gemm_fp8(const GemmArgs& a, hipStream_t stream) {
    if (a.M <= kFewRows) {
        const int ni = (a.M + 15) / 16;
        if (ni == 1)
            launch_rows<1>(a, stream);
        else if (ni == 2)
            launch_rows<2>(a, stream);
        else if (ni == 3)
            launch_rows<3>(a, stream);
        else
            launch_rows<4>(a, stream);
        return hipGetLastError();
    }
    if (big_tiles(a.M, a.N)) {
        TilePlan t = plan_tiles(a.M, a.N, a.K, 256, 256);
        t.splits = 1;
        t.per_split = t.steps;
        launch_tiles<256, 256, 4, 2>(a, t, stream);
        return hipGetLastError();
    }
    const TilePlan t = plan_tiles(a.M, a.N, a.K, 128, 128);
    launch_tiles<128, 128, 2, 2>(a, t, stream);
    if (t.splits > 1) {
        const int64_t vecs = (int64_t)a.M * ((a.N + 3) / 4);
        gemm_join_kernel<<<(unsigned)std::min<int64_t>(ceil_div(vecs, 256), 4096), 256, 0, stream>>>(a, t.splits);
    }
    return hipGetLastError();
}

}  // namespace maxsim
