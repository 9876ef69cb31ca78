// quant.hip -- rows in 8-bit floating point with a scale for each 128 values,
// as rows, transposed, or both from one read, for gfx950 (MI355X).
//
// A workgroup takes one tile of 128 x 128 values, whose row blocks, column
// blocks and square block all lie inside it, so each kind of scale is a maximum
// over registers of the tile and x is read once.  A thread holds 8 x 8
// neighbouring values: a row block's maximum goes over 16 lanes by DPP, a
// column block's over the thread's 8 rows, the lane groups and, through LDS,
// the 4 waves.  HBM-bound: 2 (bf16) + 1 + 1 bytes a value.  Measured: 16384 x
// 4096 bf16 both ways, scales by 128 values, 55 us where the outputs' memory is
// written again and again, 62 where it is not (273 MB, 5.0 and 4.4 TB/s; square
// blocks, without the scales' 4 bytes into a line each, 46); 128 x 2048 in square
// blocks 5.4 us, a launch and one tile's way through.
#include "encoder_dev.h"

namespace maxsim {
namespace {

template <typename TT, bool SQUARE>
__global__ __launch_bounds__(256) void quant_kernel(QuantArgs p) {
    typedef typename TT::type T;
    __shared__ uint32_t col_top[4][kQBlock];     // per wave: column maxima (or, square, one word)
    __shared__ u32x2 bytes_t[kQBlock][16 + 1];   // the transposed tile: row = column of x, 8 bytes a word
    const int tid = threadIdx.x, wave = tid >> 6;
    const int lane_c = tid & 15, lane_r = tid >> 4;  // 8 columns x 8 rows of the tile
    const int64_t row_blocks = (p.C + kQBlock - 1) / kQBlock;  // scales of a row of q
    const int64_t col_blocks = (p.R + kQBlock - 1) / kQBlock;  // scales of a row of qt
    // A row's scales share cache lines.  Where they are few, or all that is written
    // besides q, bands of 128 rows go to the XCDs in turn, so that such a line
    // fills in one L2 (else each 4 bytes went to memory alone): 16384 x 4096 rows
    // alone 37.9 -> 36.3 us, 65536 x 1024 38.3 -> 36.3, 30001 x 1000 both ways
    // 32.3 -> 28.5; but 16384 x 2048 both ways 31.2 -> 32.0, x 4096 54.8 -> 57.4.
    uint32_t bc = blockIdx.x % (uint32_t)row_blocks, br = blockIdx.x / (uint32_t)row_blocks;
    if (p.qt == nullptr || row_blocks <= 8) {
        const uint32_t eight = br >> 3, rest = blockIdx.x - eight * 8 * (uint32_t)row_blocks;
        if (8 * (eight + 1) <= (uint32_t)col_blocks) {
            bc = rest >> 3;
            br = 8 * eight + (rest & 7);
        }
    }
    const int c0 = (int)bc * kQBlock, r0 = (int)br * kQBlock;
    const int c = c0 + lane_c * kVec, r = r0 + lane_r * kVec;
    // All 8 rows' loads are on their way together: rows past the end read the last
    // one again, and what is not the tile's becomes 0 afterwards.  (With a branch at
    // each load they waited for each other: 16384 x 4096 both ways 61.4 -> 55.3 us,
    // 128 x 128 blocks 55.0 -> 46.0; 128 x 2048 6.4 -> 5.6.)
    typename Pack8<T>::V in[kVec];
    const T* rows[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) rows[j] = (const T*)p.x + (int64_t)min(r + j, p.R - 1) * p.ldx;
    if (p.C >= kVec) {
        const int at = min(c, p.C - kVec);
#pragma unroll
        for (int j = 0; j < kVec; ++j) in[j] = *reinterpret_cast<const typename Pack8<T>::V*>(rows[j] + at);
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) in[j] = load8<T>(rows[j], c, p.C);
    }
    float x[kVec][kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        fit8<T>(in[j], c, p.C);
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[j][i] = (float)in[j][i];
    }
    if (r0 + kQBlock > p.R) {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
#pragma unroll
            for (int i = 0; i < kVec; ++i) x[j][i] = r + j < p.R ? x[j][i] : 0.f;
    }
    Scale whole;
    if constexpr (SQUARE) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < kVec; ++j)
#pragma unroll
            for (int i = 0; i < kVec; ++i) top = umax(top, mag(x[j][i]));
        top = max64(top);
        if ((tid & 63) == 0) col_top[wave][0] = top;
        __syncthreads();
        top = umax(umax(col_top[0][0], col_top[1][0]), umax(col_top[2][0], col_top[3][0]));
        whole = block_scale(top, 448.f);
        if (tid == 0) {
            if (p.q != nullptr) p.scale[br * row_blocks + bc] = whole.s;
            if (p.qt != nullptr) p.scale_t[bc * col_blocks + br] = whole.s;
        }
    }
    if (p.q != nullptr) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            Scale k;
            if constexpr (SQUARE) {
                k = whole;
            } else {
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < kVec; ++i) top = umax(top, mag(x[j][i]));
                k = block_scale(max16(top), 448.f);
            }
            if (r + j < p.R && c < p.C) {
                store8_bytes(p.q + (int64_t)(r + j) * p.ldq, c, p.C, to_e4m3(x[j], k));
                if (!SQUARE && lane_c == 0) p.scale[(int64_t)(r + j) * row_blocks + bc] = k.s;
            }
        }
    }
    if (p.qt == nullptr) return;
    if constexpr (!SQUARE) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < kVec; ++j) top = umax(top, mag(x[j][i]));
            auto s = __builtin_amdgcn_permlane16_swap(top, top, false, false);
            top = umax(s[0], s[1]);
            s = __builtin_amdgcn_permlane32_swap(top, top, false, false);
            top = umax(s[0], s[1]);
            if ((tid & 63) < 16) col_top[wave][lane_c * kVec + i] = top;
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int cc = lane_c * kVec + i;
        Scale k;
        if constexpr (SQUARE) {
            k = whole;
        } else {
            k = block_scale(umax(umax(col_top[0][cc], col_top[1][cc]), umax(col_top[2][cc], col_top[3][cc])), 448.f);
            if (lane_r == 0 && c0 + cc < p.C) p.scale_t[(int64_t)(c0 + cc) * col_blocks + br] = k.s;
        }
        float t[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) t[j] = x[j][i];
        bytes_t[cc][lane_r] = to_e4m3(t, k);
    }
    __syncthreads();
    // 16 lanes write one row of 128 bytes
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const int cc = j * 16 + lane_r;
        if (c0 + cc < p.C) store8_bytes(p.qt + (int64_t)(c0 + cc) * p.ldqt, r0 + lane_c * kVec, p.R, bytes_t[cc][lane_c]);
    }
}

template <typename TT>
void launch(const QuantArgs& a, hipStream_t stream) {
    const unsigned grid = (unsigned)(ceil_div(a.C, kQBlock) * ceil_div(a.R, kQBlock));
    if (a.square)
        quant_kernel<TT, true><<<grid, 256, 0, stream>>>(a);
    else
        quant_kernel<TT, false><<<grid, 256, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_quant_fp8(const QuantArgs& a, hipStream_t stream) {
    if (a.dtype == MAXSIM_F16)
        launch<F16>(a, stream);
    else if (a.dtype == MAXSIM_BF16)
        launch<BF16>(a, stream);
    else
        launch<F32>(a, stream);
    return hipGetLastError();
}

}  // namespace maxsim
