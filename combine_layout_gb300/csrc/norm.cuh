// Launch arguments of the norms around a block.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moeep {

// Widest row the norms take: four vectors of 8 for each of 512 threads.
constexpr int kMaxNormWidth = 16384;

struct NormArgs {
    const uint4* o;       // bf16 [T][H] (may be null)
    const uint4* res;     // bf16 [T][H] (may be null)
    const float* w_post;  // [H] (may be null)
    const float* gate;    // [H], or [T] with per_token (may be null)
    const float* w_pre;   // [H]
    uint4* res_out;       // bf16 [T][H] (may be null)
    uint4* y;             // bf16 [T][H] (may be null)
    int H, per_token;
    float scale, eps, inv_h;
};
cudaError_t launch_norm(const NormArgs& a, int T, int sm_count, cudaStream_t s);

struct NormBwdArgs {
    NormArgs f;        // the forward pass's inputs
    const uint4* dr;   // (may be null)
    const uint4* dy;   // (may be null)
    uint4* d_o;        // (may be null)
    uint4* dres;       // (may be null)
    float* dgate;      // [T]: the per-token gate's gradient (may be null)
    float* work;       // [CTAs][2][H]
    int T;
    unsigned* err;
};
cudaError_t launch_norm_bwd(const NormBwdArgs& b, float* dw_pre, float* dw_post, float* dgate_channel,
                            int sm_count, cudaStream_t s);

}  // namespace moeep
