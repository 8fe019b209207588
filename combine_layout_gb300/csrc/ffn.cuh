// Launch arguments of the experts' feed-forward kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moeep {

// Products of the receive rows with their expert's weights.
enum RowsEpilogue {
    kRowsGateUp = 0,   // weights [E][2F][H]: out[row][F] = act(gate) * up, keep[row][2F] (may be null)
    kRowsStore = 1,    // weights [E][M][K]: out[row][M]
    kRowsDownBwd = 2,  // weights [E][K][M], M = F: out[row][2F] = d gate, d up; keep[row][F] = act(gate) * up
    kRowsStoreT = 3    // weights [E][K][M]: out[row][M]
};

struct RowsArgs {
    const int32_t* cnt;  // [E] rows of each expert
    const int32_t* off;  // [E] first row of each expert (HT)
    int E, S, mode;
    int M, K, F;
    int mt;   // m tiles, set by the launch
    int act;  // moe_ep_act_t
    __nv_bfloat16* out;
    __nv_bfloat16* keep;
    const __nv_bfloat16* gate_up;
    unsigned* err;
};

// The rows' tensor maps, boxes of 128, 64, 32 and 16 rows: a tile's rows are
// loaded in the boxes that add up to their number.
constexpr int kRowBoxes = 4;
struct RowMaps {
    CUtensorMap box[kRowBoxes];
};

// rows_in: bf16 [nrows][K]; max_rows: an upper bound of the defined rows.
cudaError_t launch_rows_product(int epi, const void* rows_in, int64_t nrows, const void* weights,
                                RowsArgs a, int64_t max_rows, int sm_count, cudaStream_t s);

// Weight gradients dw[e][M][N] = sum over e's rows of a_row b_row^T, bf16 or fp32.
struct GradArgs {
    const int32_t* cnt;
    const int32_t* off;
    int E, S, mode;
    int M, N;
    int mt, nt;  // tiles, set by the launch
    int accumulate;
    void* dw;
    unsigned* err;
};
cudaError_t launch_weight_grad(const void* arows, const void* brows, int64_t nrows, int f32, GradArgs a,
                               int sm_count, cudaStream_t s);

}  // namespace moeep
