// Backward pass of the weighted combine out[t] = sum_j w[t][j] y[row(t, j)]:
//   dy[row(t, j)] = bf16_rn(w[t][j] dout[t]),   dw[t][j] = <dout[t], y[row(t, j)]>
// (fp32 sums; dw is 0 for a pair without a row).  Memory-bound: every row of y
// is read and every row of dy written once, dout once; a CTA takes one token,
// each thread holding its vector of dout while it walks the token's rows.
// 4096 x 7168, k = 8: 153 us, 6.5 TB/s of the 998.6 MB it cannot do without.
#include "bf16x8.cuh"
#include "common.cuh"

namespace moeep {
namespace {

constexpr int kThreads = 128;

template <int KMAX>
__global__ void __launch_bounds__(kThreads, KMAX <= 8 ? 8 : 4)
    combine_bwd_kernel(const uint4* __restrict__ dout, const uint4* __restrict__ y, int k, int nvec,
                       const int32_t* __restrict__ row, const float* __restrict__ w,
                       uint4* __restrict__ dy, float* __restrict__ dw)
{
    griddep_wait();
    __shared__ float s_sum[kThreads / 32][KMAX];
    const size_t t = blockIdx.x;
    int r[KMAX];
    float wj[KMAX], sum[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
        r[j] = j < k ? __ldg(row + t * k + j) : -1;
        wj[j] = j < k ? __ldg(w + t * k + j) : 0.f;
        sum[j] = 0.f;
    }
    for (int v = threadIdx.x; v < nvec; v += kThreads) {
        const uint4 dv = __ldg(dout + t * nvec + v);
        uint4 val[KMAX];
#pragma unroll
        for (int j = 0; j < KMAX; ++j)
            if (r[j] >= 0) val[j] = __ldcs(y + (size_t)r[j] * nvec + v);
        const uint32_t du[4] = {dv.x, dv.y, dv.z, dv.w};
        float d[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d[2 * i] = __uint_as_float(du[i] << 16);
            d[2 * i + 1] = __uint_as_float(du[i] & 0xffff0000u);
        }
#pragma unroll
        for (int j = 0; j < KMAX; ++j) {
            if (r[j] < 0) continue;
            const uint32_t yu[4] = {val[j].x, val[j].y, val[j].z, val[j].w};
            float g[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum[j] = fmaf(d[2 * i], __uint_as_float(yu[i] << 16), sum[j]);
                sum[j] = fmaf(d[2 * i + 1], __uint_as_float(yu[i] & 0xffff0000u), sum[j]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = wj[j] * d[i];
            dy[(size_t)r[j] * nvec + v] = pack8(g);
        }
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
        if (lane == 0) s_sum[warp][j] = sum[j];
    }
    __syncthreads();
    if (threadIdx.x < k) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) x += s_sum[i][threadIdx.x];
        dw[t * k + threadIdx.x] = x;
    }
}

}  // namespace

cudaError_t launch_combine_bwd(const void* dout, const void* y, int T, int H, int k, const int32_t* row,
                               const float* w, void* dy, float* dw, cudaStream_t s)
{
    if (T <= 0) return cudaSuccess;
#define MOEEP_COMBINE_BWD(KM)                                                                  \
    return launch_pdl(combine_bwd_kernel<KM>, dim3(T), dim3(kThreads), s, (const uint4*)dout,  \
                      (const uint4*)y, k, H / 8, row, w, (uint4*)dy, dw)
    if (k <= 1) MOEEP_COMBINE_BWD(1);
    if (k <= 2) MOEEP_COMBINE_BWD(2);
    if (k <= 4) MOEEP_COMBINE_BWD(4);
    if (k <= 8) MOEEP_COMBINE_BWD(8);
    if (k <= 16) MOEEP_COMBINE_BWD(16);
    MOEEP_COMBINE_BWD(32);
#undef MOEEP_COMBINE_BWD
}

}  // namespace moeep
