// layers.h -- host-side interface between the C ABI of the attention layer's
// operators (capi_layers.cpp) and their kernel launchers (rope.hip, attn_fwd.hip,
// attn_bwd.hip, distill.hip).  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "maxsim_layers.h"

namespace maxsim {

struct RopeArgs {
    maxsim_view x, y;
    int B, L, H, D, rotary;
    int interleaved, dtype, inverse;
    float scale;
    const double* inv_freq;
    const int32_t* positions;
    const int32_t* offsets;
};
hipError_t launch_rope(const RopeArgs& a, hipStream_t stream);

// maxsim_attn with what the kernels derive from it.
struct AttnArgs {
    maxsim_attn a;   // left, right: INT32_MAX / 2 where there is no bound
    float* lse;
    maxsim_view dout, dq, dk, dv;
    int group;       // query heads of a key head
    int splits;      // of the keys; above 1 the forward's parts go through part_o, part_ml
    float* part_o;   // [splits][rows][Hq][D]
    float* part_ml;  // [splits][rows][Hq][2]
    int64_t rows;    // of q in memory
    float* row_stat; // backward: [2][Hq][rows]: lse in powers of 2 (+infinity where it is -infinity), rowsum(dO * out)
    // Backward, dK and dV.  Queries past the window see the first tokens' keys alone: of the first far_tiles key tiles they
    // are worked on apart, far_tokens at a time.  Where key tiles are few, the query heads of a key head are shared out too,
    // over head_splits workgroups.  What more than one workgroup adds to goes through parts:
    // part [B * Hk][part_tiles][(far_chunks + 1) * head_splits][dk, dv][part_rows][D].
    int far_tiles, far_chunks, far_tokens, head_splits, part_tiles, part_rows;
    float* part;
};
constexpr int kNoBound = 1 << 29;  // past every position

size_t attn_fwd_workspace_bytes(const maxsim_attn& a);
size_t attn_bwd_workspace_bytes(const maxsim_attn& a);
bool attn_grid_ok(const maxsim_attn& a);  // the launches stay below 2^32 threads
hipError_t launch_attn_fwd(const maxsim_attn& a, float* lse, void* workspace, hipStream_t stream);
hipError_t launch_attn_bwd(const maxsim_attn& a, const float* lse, const maxsim_view& dout, const maxsim_view& dq,
                           const maxsim_view& dk, const maxsim_view& dv, void* workspace, hipStream_t stream);

struct DistillArgs {
    const void* scores;
    const int32_t* index;
    const float* teacher;
    const float* dloss;  // backward
    void* dscores;
    float* loss;
    float* stat;     // [N][4]
    float* partial;  // [N][parts][2] (workspace), where a row is split
    int64_t ld, ldd;
    int N, V, K, dtype;
    float temperature;
};
size_t distill_workspace_bytes(int N, int V);
hipError_t launch_distill_fwd(const DistillArgs& a, hipStream_t stream);
hipError_t launch_distill_bwd(const DistillArgs& a, hipStream_t stream);

}  // namespace maxsim
