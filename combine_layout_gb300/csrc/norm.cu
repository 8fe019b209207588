// The norms after and before a block, fused with the block's gate and residual
// scale, forward and backward.
//
//   u = w_post o rstd(o)                 (u = o without w_post)
//   r = s res + gate u                   (gate per channel, per token, or 1)
//   y = w_pre r rstd(r)                  rstd(v) = 1 / sqrt(mean(v^2) + eps)
//
// Backward, with D the whole gradient of r:
//   n = r rstd(r), v = w_pre dy:   D = dr + rstd(r) (v - n mean(v n))
//   dres = s D, dw_pre = sum_t dy n, dgate = sum D u (over tokens or channels)
//   m = o rstd(o), z = w_post gate D:  do = rstd(o) (z - m mean(z m)),
//   dw_post = sum_t gate D m
//
// The mean of squares is summed as v (v / H), so that it overflows only where
// the mean itself does.  All sums and values between the loads and the stores are fp32; res_out, y,
// do and dres are rounded once, to bf16.
#include "bf16x8.cuh"
#include "common.cuh"
#include "norm.cuh"

namespace moeep {
namespace {

__device__ __forceinline__ void unpack8(float (&f)[8], const uint4& v)
{
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void load8(float (&f)[8], const float* __restrict__ p)
{
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// Sums of N values over the CTA, in a fixed order; `part` is the caller's own
// [N][32] piece of shared memory, not in use by another sum since the last
// barrier.  One barrier.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*part)[32])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (nw == 1) return;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) part[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane < nw ? part[i][lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// One CTA per token, its row in registers (VPT vectors of 8 per thread).
template <int VPT>
__global__ void __launch_bounds__(256, VPT <= 2 ? 4 : VPT == 4 ? 3 : 1) norm_kernel(const NormArgs a)
{
    griddep_wait();
    __shared__ float part[2][1][32];
    const int nvec = a.H / 8, nt = blockDim.x;
    const size_t t = blockIdx.x;
    const uint4* o = a.o ? a.o + t * nvec : nullptr;
    const uint4* res = a.res ? a.res + t * nvec : nullptr;
    float u[VPT][8], r[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * nt;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        unpack8(u[i], o && v < nvec ? __ldcs(o + v) : zero);
        unpack8(r[i], res && v < nvec ? __ldcs(res + v) : zero);
    }
    if (a.w_post) {
        float ss[1] = {0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss[0] = fmaf(u[i][j] * a.inv_h, u[i][j], ss[0]);
        block_sum<1>(ss, part[0]);
        const float p = rsqrtf(ss[0] + a.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = threadIdx.x + i * nt;
            if (v < nvec) {
                float w[8];
                load8(w, a.w_post + v * 8);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[i][j] = w[j] * (u[i][j] * p);
            }
        }
    }
    const float gt = a.gate && a.per_token ? __ldg(a.gate + t) : 1.f;
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * nt;
        if (v < nvec) {
            float g[8];
            if (a.gate && !a.per_token) {
                load8(g, a.gate + v * 8);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = gt;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                r[i][j] = fmaf(g[j], u[i][j], a.scale * r[i][j]);
                ss[0] = fmaf(r[i][j] * a.inv_h, r[i][j], ss[0]);
            }
            if (a.res_out) a.res_out[t * nvec + v] = pack8(r[i]);
        }
    }
    if (!a.y) return;
    block_sum<1>(ss, part[1]);
    const float q = rsqrtf(ss[0] + a.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * nt;
        if (v < nvec) {
            float w[8];
            load8(w, a.w_pre + v * 8);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] = w[j] * (r[i][j] * q);
            a.y[t * nvec + v] = pack8(r[i]);
        }
    }
}

// Backward: persistent CTAs take tokens in grid-stride order; a thread keeps
// its columns' weight gradients in registers over all the CTA's tokens and
// writes them to the CTA's row of the workspace, which norm_columns_kernel
// adds up in a fixed order (no atomics: the result does not depend on
// scheduling).
template <int VPT>
__global__ void __launch_bounds__(1024, 1) norm_bwd_kernel(const NormBwdArgs b)
{
    griddep_wait();
    __shared__ float part[5][2][32];
    const NormArgs& a = b.f;
    const int nvec = a.H / 8, nt = blockDim.x;
    float c_pre[VPT][8] = {}, c_post[VPT][8] = {}, c_gate[VPT][8] = {};
    for (int t = blockIdx.x; t < b.T; t += gridDim.x) {
        const size_t base = (size_t)t * nvec;
        float o[VPT][8], u[VPT][8], r[VPT][8], d[VPT][8];
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = threadIdx.x + i * nt;
            unpack8(o[i], a.o && v < nvec ? __ldcs(a.o + base + v) : zero);
            unpack8(r[i], a.res && v < nvec ? __ldcs(a.res + base + v) : zero);
            unpack8(d[i], b.dr && v < nvec ? __ldcs(b.dr + base + v) : zero);
        }
        float p = 0.f;
        if (a.w_post) {
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) s[0] = fmaf(o[i][j] * a.inv_h, o[i][j], s[0]);
            block_sum<1>(s, part[0]);
            p = rsqrtf(s[0] + a.eps);
        }
        const float gt = a.gate && a.per_token ? __ldg(a.gate + t) : 1.f;
        float s2[2] = {0.f, 0.f};
        float dy[VPT][8];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = threadIdx.x + i * nt;
            float w[8], g[8];
            unpack8(dy[i], b.dy && v < nvec ? __ldcs(b.dy + base + v) : zero);
            if (a.w_post && v < nvec) load8(w, a.w_post + v * 8);
            if (a.gate && !a.per_token && v < nvec) load8(g, a.gate + v * 8);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                u[i][j] = a.w_post ? (v < nvec ? w[j] * (o[i][j] * p) : 0.f) : o[i][j];
                const float gj = a.gate && !a.per_token ? (v < nvec ? g[j] : 0.f) : gt;
                r[i][j] = fmaf(gj, u[i][j], a.scale * r[i][j]);
            }
            if (b.dy && v < nvec) {
                load8(w, a.w_pre + v * 8);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s2[0] = fmaf(r[i][j] * a.inv_h, r[i][j], s2[0]);
                    s2[1] = fmaf(r[i][j], w[j] * dy[i][j], s2[1]);
                }
            }
        }
        if (b.dy) {
            block_sum<2>(s2, part[1]);
            const float q = rsqrtf(s2[0] + a.eps);
            const float k = s2[1] * q * a.inv_h;  // mean(v n)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int v = threadIdx.x + i * nt;
                if (v < nvec) {
                    float w[8];
                    load8(w, a.w_pre + v * 8);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float n = r[i][j] * q;
                        c_pre[i][j] = fmaf(dy[i][j], n, c_pre[i][j]);
                        d[i][j] = fmaf(q, w[j] * dy[i][j] - n * k, d[i][j]);
                    }
                }
            }
        }
        // gradients of the gate and, with w_post, of the norm after the block
        s2[0] = s2[1] = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = threadIdx.x + i * nt;
            if (v < nvec) {
                if (b.dres) {
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = a.scale * d[i][j];
                    b.dres[base + v] = pack8(x);
                }
                float w[8], g[8];
                if (a.w_post) load8(w, a.w_post + v * 8);
                if (a.gate && !a.per_token) load8(g, a.gate + v * 8);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float du = d[i][j] * u[i][j];
                    s2[0] += du;
                    c_gate[i][j] += du;
                    d[i][j] *= a.gate && !a.per_token ? g[j] : gt;
                    if (a.w_post) {
                        const float m = o[i][j] * p;
                        c_post[i][j] = fmaf(d[i][j], m, c_post[i][j]);
                        d[i][j] *= w[j];
                        s2[1] = fmaf(d[i][j], m, s2[1]);
                    }
                }
            }
        }
        const bool token_gate = b.dgate && a.per_token;
        if (a.w_post || token_gate) {
            block_sum<2>(s2, part[3]);
            if (token_gate && threadIdx.x == 0) b.dgate[t] = s2[0];
        }
        if (b.d_o) {
            const float k = s2[1] * a.inv_h;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int v = threadIdx.x + i * nt;
                if (v < nvec) {
                    if (a.w_post)
#pragma unroll
                        for (int j = 0; j < 8; ++j) d[i][j] = p * (d[i][j] - (o[i][j] * p) * k);
                    b.d_o[base + v] = pack8(d[i]);
                }
            }
        }
        __syncthreads();  // the sums' shared memory before the next token
    }
    float* row = b.work + (size_t)blockIdx.x * 3 * a.H;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * nt;
        if (v < nvec) {
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                *reinterpret_cast<float4*>(row + v * 8 + j) =
                    make_float4(c_pre[i][j], c_pre[i][j + 1], c_pre[i][j + 2], c_pre[i][j + 3]);
                *reinterpret_cast<float4*>(row + a.H + v * 8 + j) =
                    make_float4(c_post[i][j], c_post[i][j + 1], c_post[i][j + 2], c_post[i][j + 3]);
                *reinterpret_cast<float4*>(row + 2 * a.H + v * 8 + j) =
                    make_float4(c_gate[i][j], c_gate[i][j + 1], c_gate[i][j + 2], c_gate[i][j + 3]);
            }
        }
    }
}

// Sums the CTAs' column gradients; blockIdx.y picks the output.
__global__ void __launch_bounds__(256) norm_columns_kernel(const float* __restrict__ work, int rows, int H,
                                                           float* dw_pre, float* dw_post, float* dgate)
{
    griddep_wait();
    float* out = blockIdx.y == 0 ? dw_pre : blockIdx.y == 1 ? dw_post : dgate;
    if (!out) return;
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < H)
        for (int i = part; i < rows; i += 8) v += work[((size_t)i * 3 + blockIdx.y) * H + c];
    s[part][lane] = v;
    __syncthreads();
    if (part == 0 && c < H) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += s[i][lane];
        out[c] = v;
    }
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int T, cudaStream_t s)
{
    if (T <= 0) return cudaSuccess;
    const int nvec = a.H / 8;
    // four CTAs of 256 threads per SM hold more rows in flight than one of 1024
    const int vpt = nvec <= 256 ? 1 : nvec <= 512 ? 2 : nvec <= 1024 ? 4 : 8;
    int threads = ((nvec + vpt - 1) / vpt + 31) & ~31;
    if (vpt == 1) return launch_pdl(norm_kernel<1>, dim3(T), dim3(threads), s, a);
    if (vpt == 2) return launch_pdl(norm_kernel<2>, dim3(T), dim3(threads), s, a);
    if (vpt == 4) return launch_pdl(norm_kernel<4>, dim3(T), dim3(threads), s, a);
    return launch_pdl(norm_kernel<8>, dim3(T), dim3(threads), s, a);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& b, float* dw_pre, float* dw_post, float* dgate_channel,
                            int sm_count, cudaStream_t s)
{
    const int H = b.f.H, nvec = H / 8;
    const int grid = b.T < sm_count ? b.T : sm_count;
    if (grid > 0) {
        const int vpt = nvec <= 1024 ? 1 : 2;
        const int threads = ((nvec + vpt - 1) / vpt + 31) & ~31;
        cudaError_t e = vpt == 1 ? launch_pdl(norm_bwd_kernel<1>, dim3(grid), dim3(threads), s, b)
                                 : launch_pdl(norm_bwd_kernel<2>, dim3(grid), dim3(threads), s, b);
        if (e != cudaSuccess) return e;
    }
    if (!dw_pre && !dw_post && !dgate_channel) return cudaSuccess;
    return launch_pdl(norm_columns_kernel, dim3((H + 31) / 32, 3), dim3(256), s, (const float*)b.work, grid, H,
                      dw_pre, dw_post, dgate_channel);
}

}  // namespace moeep
