// gemm_fp8.hip -- product of two e4m3 matrices with a scale for each 128 along
// K, for gfx950 (MI355X).
//
//     c[m, n] = sum_kb sa[m, kb] sb[n or n / 128, kb] sum_{k in kb} A[m, k] B[n, k]
//
// Two v_mfma_f32_32x32x64_f8f6f4 (one 16x16x128 for few rows) contract exactly
// one block of 128, so their result, started from 0, is the block's unscaled
// sum, and one fused multiply-add a value adds it, scaled, to the fp32
// accumulator, on the VALU beside the matrix pipe.
//   * Rows of B are the MFMA's rows and rows of A its columns: a lane then holds
//     values of one row of A, whose scale is one register, and neighbouring
//     columns of c, which leave in 16-byte stores.
//   * Tiles go HBM -> LDS by direct loads into two buffers, 128 bytes of K a
//     step; 16-byte chunks are XOR-swizzled so that operand reads hit all banks.
//   * Workgroups that share rows of A or B follow each other on one XCD.
//   * Where tiles are few, K is split over workgroups whose fp32 partial sums
//     a second launch adds in order.
//   * Few rows of A (a query) take a kernel bound by the bytes of B: operands go
//     straight to registers and a workgroup's waves split K.
//
// Measured (bf16 results, scales of 128 x 128 for B): 16384 x 8192 x 4096
// 505-553 us, 2.0-2.2 PFLOP/s; the matrix pipes are busy 54 % of the cycles at
// the 1.9 GHz that the card holds under this load, and what they wait for is
// the scaling (16 multiply-adds beside two MFMAs of 64 cycles), the issue of
// the direct loads, and 9 us a tile before its first product and after its last.
// 65536 x 128 x 2048 37.6 us (153 MB, 4.1 TB/s: HBM); 32 x 2048 x 2048 6.1 us
// (latency); 1024 x 2048 x 20001 with fp32 results 97 + 8 us (0.87 PFLOP/s
// in fp16 products, bound by their conversions).
#include <algorithm>
#include <type_traits>

#include "encoder_dev.h"

namespace maxsim {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lptr_t;

constexpr int kStep = kQBlock;  // bytes of K a step
constexpr uint32_t kOutside = 0xF0000000u;  // an offset past any buffer: reads zeros

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// A lane's part of a block of 128 along K: 32 bytes for an operand of 16 rows, two times 32
// for one of 32 rows; or the values in fp16, which holds every e4m3 value.  Which of the 128
// a lane holds is the same for both operands, and does not matter otherwise.
__device__ __forceinline__ void to_f16(i32x8 bytes, f16x8* v) {
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((unsigned)bytes[w], 1.f, false);
        const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((unsigned)bytes[w], 1.f, true);
        v[w >> 1][(w & 1) * 4 + 0] = lo[0];
        v[w >> 1][(w & 1) * 4 + 1] = lo[1];
        v[w >> 1][(w & 1) * 4 + 2] = hi[0];
        v[w >> 1][(w & 1) * 4 + 3] = hi[1];
    }
}
template <bool FINE>
struct Operand {
    i32x8 v[2];
};
template <>
struct Operand<true> {
    f16x8 v[8];
};
template <bool FINE>
__device__ __forceinline__ Operand<FINE> operand_of(i32x8 lo, i32x8 hi) {
    Operand<FINE> o;
    if constexpr (FINE) {
        to_f16(lo, o.v);
        to_f16(hi, o.v + 4);
    } else {
        o.v[0] = lo;
        o.v[1] = hi;
    }
    return o;
}

__device__ __forceinline__ f32x16 zero16() {
    f32x16 z;
#pragma unroll
    for (int e = 0; e < 16; ++e) z[e] = 0.f;
    return z;
}

// The unscaled sum of one block of 128, for 16 x 16 or 32 x 32 results.  The
// 8-bit instructions add eight products that follow each other along K at a time, each cut
// toward 0 to a multiple of 2^(e - 13), e the largest sum of two values' exponents
// among the eight (at least -6 a value; products with a zero do not count): measured by single small
// products beside a large one.  On values of normal distribution the losses cancel to 1.4e-5 of the
// result's norm, on one sign they add up to 8.5e-4 of the sum at most, a fifth of half a
// step of bf16 and up to twice half a step of fp16.  An fp32
// result takes the values through fp16, whose products and sums are exact to
// fp32 (1.2e-8), at half the rate.  Both scale operands 0: the compiler emits the 8-bit instruction without scales.
template <bool FINE>
__device__ __forceinline__ f32x4 mfma16(i32x8 b, i32x8 a) {
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
    if constexpr (FINE) {
        f16x8 x[4], y[4];
        to_f16(b, x);
        to_f16(a, y);
#pragma unroll
        for (int q = 0; q < 4; ++q) d = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[q], y[q], d, 0, 0, 0);
    } else {
        d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, d, 0, 0, 0, 0, 0, 0);
    }
    return d;
}
template <bool FINE>
__device__ __forceinline__ f32x16 mfma32(const Operand<FINE>& b, const Operand<FINE>& a) {
    f32x16 d = zero16();
    if constexpr (FINE) {
#pragma unroll
        for (int q = 0; q < 8; ++q) d = __builtin_amdgcn_mfma_f32_32x32x16_f16(b.v[q], a.v[q], d, 0, 0, 0);
    } else {
#pragma unroll
        for (int q = 0; q < 2; ++q)
            d = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b.v[q], a.v[q], d, 0, 0, 0, 0, 0, 0);
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

// This wave's direct loads have landed (LANDED) and its LDS accesses are done;
// then the workgroup's barrier (__syncthreads would not keep the next tile's loads in flight).
template <bool LANDED>
__device__ __forceinline__ void tile_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(LANDED ? 0x0070 : 0xC07F);  // vmcnt(0) lgkmcnt(0), or lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// N neighbouring values of a row of c, rounded once.
template <typename T, int N>
__device__ __forceinline__ void store_n(T* c, int left, const float* v) {
    typedef T VN __attribute__((ext_vector_type(N), aligned(sizeof(T))));
    VN w;
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = (T)v[i];
    if (left >= N) {
        *reinterpret_cast<VN*>(c) = w;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < left) c[i] = w[i];
    }
}
__device__ __forceinline__ void store4(const GemmArgs& p, int64_t row, int n, f32x4 v) {
    const int64_t at = row * p.ldc + n;
    const float f[4] = {v[0], v[1], v[2], v[3]};
    if (p.out_dtype == MAXSIM_F32)
        store_n<float, 4>((float*)p.c + at, p.N - n, f);
    else if (p.out_dtype == MAXSIM_BF16)
        store_n<__bf16, 4>((__bf16*)p.c + at, p.N - n, f);
    else
        store_n<_Float16, 4>((_Float16*)p.c + at, p.N - n, f);
}

struct TilePlan {
    int tiles_m, tiles_n, splits;
    int steps;      // of K in all
    int per_split;  // of K in a split (the last may have fewer)
};

// A workgroup of WGM x WGN waves makes a tile of TM rows of A x TN rows of B; a
// wave makes (TM / WGM) x (TN / WGN), which lies within 128 rows of B, in
// blocks of 32 x 32 (the 32x32x64 instruction ran 1.22x the rate of 16x16x128).
// ROWS: b_scale by the row; FINE: products in fp16
template <int TM, int TN, int WGM, int WGN, bool ROWS, bool FINE>
__global__ __launch_bounds__(64 * WGM * WGN) void gemm_tile_kernel(GemmArgs p, TilePlan plan) {
    constexpr int WAVES = WGM * WGN;
    constexpr int NI = TM / WGM / 32, NJ = TN / WGN / 32;
    // Issuing a tile's direct loads holds a wave up for about as long as a SIMD
    // works on a step, so with two waves on each SIMD the first issues all of them and the
    // second keeps the matrix pipe busy.
    constexpr int LOADERS = WAVES == 8 ? 4 : WAVES;
    constexpr int LA = TM / 8 / LOADERS, LB = TN / 8 / LOADERS;  // a loading wave's direct loads of 8 rows
    constexpr int SA = TM, SB = ROWS ? TN : 64;  // scales of a step: of each row, or of 128 rows of B in 64 words
    static_assert(LA * 8 * LOADERS == TM && LB * 8 * LOADERS == TN && TN / WGN <= kQBlock && LA % 2 == 0 && LB % 4 == 0,
                  "tile");
    constexpr int LS = ((SA + SB) / 64 + LOADERS - 1) / LOADERS;  // a loading wave's loads of 64 scales
    // Two arrays and a loop unrolled by two, not one array indexed by the step:
    // the compiler then sees that a step's reads and the next tile's direct
    // loads touch different memory, and does not make the reads wait for them.
    // (A third buffer was slower: 256 x 128 tiles 37 -> 40 us, 97 -> 108 us.)
    constexpr int TILE = (TM + TN) * kStep, SCALES = LS * LOADERS * 64;
    __shared__ __align__(16) uint8_t tile_0[TILE], tile_1[TILE];
    __shared__ __align__(16) float scale_0[SCALES], scale_1[SCALES];
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
    // LDS row r holds its 16-byte chunk c at position c ^ swizzle(r), so that the
    // 16 rows of a quarter wave's read fall on all 64 banks.  They are neighbours
    // in A.  In B a block's row rr is row rr / 8 * 4 + rr / 4 % 2 * 16 + rr % 4 of
    // its 32, so that a lane's 16 results are neighbouring columns of c.
    auto swz_a = [](int r) { return (r >> 1) & 7; };
    auto swz_b = [](int r) { return ((r >> 1) & 3) | (((r >> 4) & 1) << 2); };

    // Direct loads: 8 rows each, row lane / 8 at position lane % 8 a lane.  A's
    // swizzle changes with every group of 8 rows and B's with every second one,
    // both between two values, so a lane's offsets are 4 in all.
    uint32_t off_a[2], off_b[2], chunk_a[2], chunk_b[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        chunk_a[j] = (uint32_t)((lane & 7) ^ swz_a((wave * LA + j) * 8 + (lane >> 3))) * 16;
        chunk_b[j] = (uint32_t)((lane & 7) ^ swz_b((wave * LB + 2 * j) * 8 + (lane >> 3))) * 16;
        off_a[j] = (uint32_t)(lane >> 3) * (uint32_t)p.lda + chunk_a[j];
        off_b[j] = (uint32_t)(lane >> 3) * (uint32_t)p.ldb + chunk_b[j];
    }
    const float* sa = p.a_scale + (int64_t)m0 * plan.steps;
    const float* sb = p.b_scale + (int64_t)(ROWS ? n0 : n0 / kQBlock) * plan.steps;
    const int scales_b = ROWS ? rows_b : (rows_b + kQBlock - 1) / kQBlock;

    // Step `at` takes block `at` of K; or, where each row of A is read once (one
    // column of tiles), the blocks turned by the tile: workgroups all at the same
    // distance from their rows' starts would press on a few of HBM's channels.
    constexpr bool TURN = TM > TN;
    const int count = k_end - k_begin, turn = TURN && plan.tiles_n == 1 && count > 0 ? (int)((m0 / TM) % count) : 0;
    auto block_of = [&](int at) {
        if constexpr (!TURN) return at;
        const int kb = at + turn;
        return at >= k_end ? k_end : kb >= k_end ? kb - count : kb;
    };

    // One operand's part of tile kb: rows [first, first + 8 * L) of the `rows` of the tile.
    auto load_rows = [&](const uint8_t* base, int64_t ld, int first, int rows, const uint32_t* off, const uint32_t* chunk,
                         int kb, uint8_t* to, auto count, auto period) {
        constexpr int L = decltype(count)::value, P = decltype(period)::value;
        const uint32_t left = kb < k_end ? k16 - (uint32_t)kb * kStep : 0u;  // bytes of K from this step on
        const uint8_t* at = base + (int64_t)first * ld + (int64_t)kb * kStep;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int n = min(8, rows - first - j * 8);  // rows of this load; none: reads zeros
            const uint32_t bytes = n > 0 && left > 0 ? (uint32_t)(n - 1) * (uint32_t)ld + left : 0u;
            const uint32_t o = chunk[j / P & 1] < left ? off[j / P & 1] : kOutside;
            load_lds<16>(at, bytes, o, (lptr_t)(to + j * 8 * kStep));
            at += 8 * ld;
        }
    };
    auto load = [&](int at, uint8_t* tile, float* scale) {
        if (wave >= LOADERS) return;
        const int kb = block_of(at);
        load_rows(p.A + (int64_t)m0 * p.lda, p.lda, wave * LA * 8, rows_a, off_a, chunk_a, kb, tile + wave * LA * 8 * kStep,
                  std::integral_constant<int, LA>{}, std::integral_constant<int, 1>{});
        load_rows(p.B + (int64_t)n0 * p.ldb, p.ldb, wave * LB * 8, rows_b, off_b, chunk_b, kb,
                  tile + (TM + wave * LB * 8) * kStep, std::integral_constant<int, LB>{}, std::integral_constant<int, 2>{});
        // scales, 64 to a load; those past the end read 0, as do the loads of waves that have none left
#pragma unroll
        for (int u = 0; u < LS; ++u) {
            const int q = u * LOADERS + wave;
            const bool is_a = q < SA / 64;
            const int r = (is_a ? q : q - SA / 64) * 64 + lane;
            const int rows = kb < k_end ? is_a ? rows_a : scales_b : 0;
            load_lds<4>((is_a ? sa : sb) + kb, rows > 0 ? ((uint32_t)rows * (uint32_t)plan.steps - (uint32_t)kb) * 4u : 0u,
                        r < rows ? (uint32_t)r * (uint32_t)plan.steps * 4u : kOutside, (lptr_t)&scale[q * 64]);
        }
    };

    const int wm = wave / WGN * (TM / WGM), wn = wave % WGN * (TN / WGN);
    const int col = lane & 31, half = lane >> 5;
    const int row_b = wn + (col >> 3) * 4 + ((col >> 2) & 1) * 16 + (col & 3);
    uint32_t lds_a = (uint32_t)((wm + col) * kStep + (((2 * half) ^ swz_a(wm + col)) << 4));
    uint32_t lds_b = (uint32_t)((TM + row_b) * kStep + (((2 * half) ^ swz_b(row_b)) << 4));
    f32x16 acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = zero16();

    // LAG: a block is added while the next one is on the matrix pipe, and a
    // step's last block while the next step's first is.  Scales by the row and
    // fp16 operands leave no registers for a second block; there the other
    // wave of the SIMD fills the pipe.
    constexpr bool LAG = !ROWS && !FINE;
    constexpr bool AHEAD = LAG || NI * NJ < 8;  // the next rows of B are read while these are multiplied
    f32x16 d_last = zero16();
    float s_last = 0.f;
    auto add = [&](f32x16& c, const f32x16& d, const f32x4* t, float s) {
#pragma unroll
        for (int e = 0; e < 16; ++e) c[e] = __builtin_fmaf(ROWS ? d[e] * t[e >> 2][e & 3] : d[e], s, c[e]);
        asm volatile("" : "+v"(c));  // here, and not sunk to a later block that reads c
    };
    // K ends inside a chunk: clear what follows it there
    auto end_of_k = [&](int at, uint8_t* tile) {
        if (block_of(at) != plan.steps - 1 || (p.K & 15) == 0) return;
        const int last = (p.K & (kStep - 1)) >> 4, keep = p.K & 15;
        for (int r = tid; r < TM + TN; r += 64 * WAVES) {
            const int s = r < TM ? swz_a(r) : swz_b(r - TM);
            uint32_t* w = reinterpret_cast<uint32_t*>(tile + r * kStep + (last ^ s) * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int left = keep - 4 * i;
                if (left < 4) w[i] = left <= 0 ? 0u : w[i] & ((1u << (8 * left)) - 1u);
            }
        }
        tile_barrier<false>();
    };
    auto step = [&](int kb, uint8_t* tile, const float* scale, uint8_t* next, float* next_scale) {
        tile_barrier<true>();
        end_of_k(kb, tile);
        load(kb + 1, next, next_scale);
        // Half `half` of the wave holds chunks 2 half, 2 half + 1 of each 64 of K; blocks of 32 rows share a lane's
        // swizzle.  The compiler may not keep all these addresses over the loop: registers are short, adds are not.
        asm volatile("" : "+v"(lds_a), "+v"(lds_b));
        auto operand = [&](uint32_t at, int block) {
            auto chunk = [&](uint32_t flip) {
                return *reinterpret_cast<const u32x4*>(tile + (at ^ flip) + block * 32 * kStep);
            };
            return operand_of<FINE>(join(chunk(0), chunk(16)), join(chunk(64), chunk(80)));
        };
        const float s_block = ROWS ? 1.f : scale[SA + wn / kQBlock];
        Operand<FINE> a[NI];
        float s[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            a[i] = operand(lds_a, i);
            s[i] = scale[wm + i * 32 + col] * s_block;
        }
        Operand<FINE> b;
        if (AHEAD) b = operand(lds_b, 0);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            f32x4 t[4];
            if constexpr (ROWS) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    t[q] = *reinterpret_cast<const f32x4*>(&scale[SA + wn + 32 * j + 16 * half + 4 * q]);
            }
            if (!AHEAD) b = operand(lds_b, j);
            Operand<FINE> b_next = b;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const f32x16 d = mfma32<FINE>(b, a[i]);
                if (AHEAD && i == 0 && j + 1 < NJ) b_next = operand(lds_b, j + 1);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (LAG) {
                    add(i > 0 ? acc[i - 1][j] : acc[NI - 1][j > 0 ? j - 1 : NJ - 1], d_last, t, s_last);
                    d_last = d;
                    s_last = s[i];
                } else {
                    add(acc[i][j], d, t, s[i]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            b = b_next;
        }
    };
    if (k_begin < k_end) {
        load(k_begin, tile_0, scale_0);
        // an odd number of steps: the last one adds zeros
        for (int kb = k_begin; kb < k_end; kb += 2) {
            step(kb, tile_0, scale_0, tile_1, scale_1);
            step(kb + 1, tile_1, scale_1, tile_0, scale_0);
        }
        if constexpr (LAG) add(acc[NI - 1][NJ - 1], d_last, nullptr, s_last);
    }
    // Results leave through LDS, 32 rows of each row of waves at a time, so that
    // neighbouring lanes store neighbouring 16 bytes: straight from the accumulators a
    // store would put 8 bytes each into 64 cache lines (41 us a tile of 256 x 256).
    // 16-byte chunks are XOR-swizzled by the row.
    auto leave = [&](auto type, auto* c, int64_t ld, int width) {
        typedef decltype(type) T;
        constexpr int V = 16 / sizeof(T), CH = TN / V;  // values of a chunk, chunks of a row
        // rows of waves at a time
        constexpr int FIT = TILE / (32 * TN * (int)sizeof(T)), NOW = FIT >= WGM ? WGM : FIT >= WGM / 2 ? WGM / 2 : WGM / 4;
        static_assert(NOW >= 1 && NOW * 32 * TN * sizeof(T) <= TILE && CH >= 16, "LDS");
        typedef T VT __attribute__((ext_vector_type(V)));
        VT* box = reinterpret_cast<VT*>(tile_0);
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int g = 0; g < WGM; g += NOW) {
                __syncthreads();
                if (wave / WGN >= g && wave / WGN < g + NOW) {
                    const int r = (wave / WGN - g) * 32 + col;
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
#pragma unroll
                        for (int q = 0; q < 16 / V; ++q) {
                            VT v;
#pragma unroll
                            for (int e = 0; e < V; ++e) v[e] = (T)acc[i][j][q * V + e];
                            box[r * CH + (((wn + 32 * j + 16 * half) / V + q) ^ (r & (CH - 1)))] = v;
                        }
                }
                __syncthreads();
#pragma unroll 4
                for (int k = tid; k < NOW * 32 * CH; k += 64 * WAVES) {
                    const int r = k / CH, ch = k % CH;
                    const int m = m0 + (g + r / 32) * (TM / WGM) + i * 32 + r % 32, n = n0 + ch * V;
                    if (m >= p.M || n >= width) continue;
                    const VT v = box[r * CH + (ch ^ (r & (CH - 1)))];
                    T* to = c + (int64_t)m * ld + n;
                    typedef T VU __attribute__((ext_vector_type(V), aligned(sizeof(T))));
                    if (n + V <= width) {
                        *reinterpret_cast<VU*>(to) = v;
                    } else {
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            if (n + e < width) to[e] = v[e];
                    }
                }
            }
    };
    if constexpr (TN <= 128) {  // tiles that split K, or have fp32 results
        if (plan.splits > 1) {  // rows of N rounded up to 4: the join reads whole vectors
            const int64_t n4 = (p.N + 3) & ~3;
            return leave(0.f, p.partial + (int64_t)z * p.M * n4, n4, (int)n4);
        }
        if constexpr (FINE) return leave(0.f, (float*)p.c, p.ldc, p.N);
    }
    if constexpr (!FINE) {
        if (p.out_dtype == MAXSIM_BF16)
            leave((__bf16)0.f, (__bf16*)p.c, p.ldc, p.N);
        else
            leave((_Float16)0.f, (_Float16*)p.c, p.ldc, p.N);
    }
}

// c = the splits' partial sums, added in order.
__global__ __launch_bounds__(256) void gemm_join_kernel(GemmArgs p, int splits) {
    const int n4 = (p.N + 3) >> 2;
    const int64_t each = (int64_t)p.M * n4;
    const f32x4* part = reinterpret_cast<const f32x4*>(p.partial);
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < each; k += (int64_t)gridDim.x * 256) {
        f32x4 v = part[k];
#pragma unroll 8
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

    auto fold = [&](int kb, i32x8 bv, const i32x8* av) {
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
            const f32x4 d = mfma16<FINE>(bv, av[i]);
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

constexpr int kCUs = 256;

// Few rows: each lane's share of A comes from memory as often as B's, so long
// rows of more than a few tokens are better shared through LDS.  Us by
// this kernel and by tiles (N x K): 32 rows 2048 x 2048 5.6, 8.0; 4096 x 4096 9.3, 11.3;
// 8192 x 8192 30, 18; 16 rows of it 20, 17; 1 row of it 12.4, 16.5.  (Its 512
// threads to 16 rows of B pass a launch's 2^32 near N = 2^27; the tiles' do not.)
bool few_rows(int M, int N, int K) { return (M <= 4 || (M <= 32 && K <= 4096)) && N <= 1 << 26; }

// How a product is cut up: by 256 x 256 tiles where they give every other CU
// one; by 256 x 128 where they give every CU one (or, for fp32 results, where K
// split does); else by 128 x 128, or 64 x 128 where those are too few.
// Us by 128 x 128 and 64 x 128: 512 x 2048 x 2048 14.6, 12.8; 100 x 2048 x 2048
// 11.7, 9.3; by 128 x 128 and 256 x 128, 65536 x 128 x 2048: 43, 37.
enum TileKind { kBig, kTall, kSmall, kLow };
struct Cut {
    TileKind kind;
    TilePlan plan;
};
Cut cut(int M, int N, int K, bool fine) {
    const int64_t tall = ceil_div(M, 256) * ceil_div(N, 128), steps = ceil_div(K, kStep);
    Cut c;
    if (!fine && N > 128 && ceil_div(M, 256) * ceil_div(N, 256) >= kCUs / 2)
        c.kind = kBig;
    else if (tall >= kCUs || (fine && tall * (steps / 8) >= kCUs))
        c.kind = kTall;
    else
        c.kind = ceil_div(M, 128) * ceil_div(N, 128) > kCUs / 2 ? kSmall : kLow;
    TilePlan& t = c.plan;
    t.tiles_m = (int)ceil_div(M, c.kind == kLow ? 64 : c.kind == kSmall ? 128 : 256);
    t.tiles_n = (int)ceil_div(N, c.kind == kBig ? 256 : 128);
    t.steps = (int)steps;
    // Split K while it pays: a step costs about this, the second launch 4 us
    // and the partial sums' way to memory and back.
    const double step_us = c.kind == kTall ? (fine ? 2.2 : 1.3) : c.kind == kSmall ? 0.9 : 0.75;
    const double sums_us = (double)M * N * 8 / 4e6;
    const int64_t tiles = (int64_t)t.tiles_m * t.tiles_n;
    // (two workgroups of the low tiles share a CU: 274 x 2822 x 12036 48.3 -> 36.5 us; fp16 operands need its registers alone)
    const int64_t groups = c.kind == kLow && !fine ? 2 * kCUs : kCUs;
    const int64_t most = c.kind == kBig ? 1 : std::min<int64_t>({groups / tiles, steps / 4, 32});
    int best = 1;
    double best_us = steps * step_us;
    for (int s = 2; s <= most; ++s) {
        const double us = (double)ceil_div(steps, s) * step_us + 4 + s * sums_us;
        if (us < best_us) best = s, best_us = us;
    }
    t.per_split = (int)ceil_div(steps, best);
    t.splits = t.per_split ? (int)ceil_div(steps, t.per_split) : 1;
    return c;
}

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
        constexpr bool ROWS = decltype(rows)::value, FINE = decltype(fine)::value;
        if constexpr (!FINE || TN <= 128)  // fp16 operands of a larger tile do not fit the registers
            gemm_tile_kernel<TM, TN, WGM, WGN, ROWS, FINE><<<grid, 64 * WGM * WGN, 0, stream>>>(a, t);
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
    if (few_rows(M, N, K)) return 0;
    const size_t partial = (size_t)M * (size_t)((N + 3) & ~3) * sizeof(float);
    const int s = std::max(cut(M, N, K, false).plan.splits, cut(M, N, K, true).plan.splits);
    return s > 1 ? s * partial : 0;  // enough for every type of result
}

hipError_t launch_gemm_fp8(const GemmArgs& a, hipStream_t stream) {
    if (few_rows(a.M, a.N, a.K)) {
        if (a.M <= 16)
            launch_rows<1>(a, stream);
        else
            launch_rows<2>(a, stream);
        return hipGetLastError();
    }
    const Cut c = cut(a.M, a.N, a.K, a.out_dtype == MAXSIM_F32);
    if (c.kind == kBig)
        launch_tiles<256, 256, 4, 2>(a, c.plan, stream);
    else if (c.kind == kTall)
        launch_tiles<256, 128, 4, 2>(a, c.plan, stream);
    else if (c.kind == kSmall)
        launch_tiles<128, 128, 4, 2>(a, c.plan, stream);
    else
        launch_tiles<64, 128, 2, 4>(a, c.plan, stream);
    if (c.plan.splits > 1) {
        const int64_t vecs = (int64_t)a.M * ((a.N + 3) / 4);
        gemm_join_kernel<<<(unsigned)std::min<int64_t>(ceil_div(vecs, 256), 4096), 256, 0, stream>>>(a, c.plan.splits);
    }
    return hipGetLastError();
}

}  // namespace maxsim
