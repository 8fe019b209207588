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
#include "tc.cuh"

namespace moeep {
namespace {

using f2 = unsigned long long;  // two fp32 values

__device__ __forceinline__ f2 pack(float a, float b)
{
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack(f2 v, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b)
{
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c)
{
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum2(f2 v)
{
    float a, b;
    unpack(v, a, b);
    return a + b;
}

// Eight bf16 values as four pairs, and back (rounded to nearest even).
struct Vec {
    f2 v[4];
};
__device__ __forceinline__ Vec widen(const uint4& x)
{
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
    Vec r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = pack(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    return r;
}
__device__ __forceinline__ uint4 narrow(const Vec& x)
{
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        unpack(x.v[i], a, b);
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        o[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ Vec vec_of(const float* p)
{
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(p), b = *reinterpret_cast<const ulonglong2*>(p + 4);
    Vec r;
    r.v[0] = a.x; r.v[1] = a.y; r.v[2] = b.x; r.v[3] = b.y;
    return r;
}

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

// Forward: one CTA per token, its row in registers (VPT vectors per thread);
// the weights come from L1.  Rows are independent, so what hides the two sums'
// latency is more CTAs per SM.
template <int VPT>
__global__ void __launch_bounds__(256, VPT <= 4 ? 4 : 2) norm_kernel(const NormArgs a)
{
    griddep_wait();
    __shared__ float part[2][1][32];
    const int nvec = a.H / 8, nt = blockDim.x;
    const size_t t = blockIdx.x;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    uint4 o[VPT];
    Vec r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * nt;
        o[i] = a.o && v < nvec ? __ldcs(a.o + t * nvec + v) : zero;
    }
    uint4 res[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * nt;
        res[i] = a.res && v < nvec ? __ldcs(a.res + t * nvec + v) : zero;
    }
    const f2 inv = pack(a.inv_h, a.inv_h), sc = pack(a.scale, a.scale);
    float gt = a.gate && a.per_token ? __ldg(a.gate + t) : 1.f;
    if (a.w_post) {
        f2 s2 = pack(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const Vec x = widen(o[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) s2 = fma2(mul2(x.v[j], inv), x.v[j], s2);
        }
        float ss[1] = {sum2(s2)};
        block_sum<1>(ss, part[0]);
        gt *= rsqrtf(ss[0] + a.eps);
    }
    const f2 gg = pack(gt, gt);  // the token's gate times rstd(o)
    f2 s2 = pack(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * nt;
        if (v >= nvec) continue;
        Vec u = widen(o[i]);
        const Vec x = widen(res[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) u.v[j] = mul2(u.v[j], gg);
        if (a.w_post) {
            const Vec w = vec_of(a.w_post + v * 8);
#pragma unroll
            for (int j = 0; j < 4; ++j) u.v[j] = mul2(u.v[j], w.v[j]);
        }
        if (a.gate && !a.per_token) {
            const Vec w = vec_of(a.gate + v * 8);
#pragma unroll
            for (int j = 0; j < 4; ++j) u.v[j] = mul2(u.v[j], w.v[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r[i].v[j] = fma2(sc, x.v[j], u.v[j]);
            s2 = fma2(mul2(r[i].v[j], inv), r[i].v[j], s2);
        }
        if (a.res_out) a.res_out[t * nvec + v] = narrow(r[i]);
    }
    if (!a.y) return;
    float ss[1] = {sum2(s2)};
    block_sum<1>(ss, part[1]);
    const float q = rsqrtf(ss[0] + a.eps);
    const f2 qq = pack(q, q);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * nt;
        if (v >= nvec) continue;
        const Vec w = vec_of(a.w_pre + v * 8);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[i].v[j] = mul2(w.v[j], mul2(r[i].v[j], qq));
        a.y[t * nvec + v] = narrow(r[i]);
    }
}

// Backward, rows wider than the pipelined form below takes: persistent CTAs
// take tokens in grid-stride order; a thread keeps its columns' gradients in registers over all the CTA's tokens and
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
    float c_pre[VPT][8] = {}, c_dm[VPT][8] = {};
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
                    const float m = a.w_post ? o[i][j] * p : o[i][j];
                    s2[0] = fmaf(d[i][j], u[i][j], s2[0]);
                    c_dm[i][j] = fmaf(gt * d[i][j], m, c_dm[i][j]);
                    d[i][j] *= a.gate && !a.per_token ? g[j] : gt;
                    if (a.w_post) {
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
    float* row = b.work + (size_t)blockIdx.x * 2 * a.H;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * nt;
        if (v < nvec) {
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                *reinterpret_cast<float4*>(row + v * 8 + j) =
                    make_float4(c_pre[i][j], c_pre[i][j + 1], c_pre[i][j + 2], c_pre[i][j + 3]);
                *reinterpret_cast<float4*>(row + a.H + v * 8 + j) =
                    make_float4(c_dm[i][j], c_dm[i][j + 1], c_dm[i][j + 2], c_dm[i][j + 3]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Sums of 8 values over the CTA in a fixed order, every thread getting all;
// one barrier.  In a warp the values are halved at each step (4 + 2 + 1 + 1 +
// 1 exchanges instead of 40); part is [2][8][32], used in turn.
__device__ __forceinline__ void block_sum8(float (&v)[8], float (*part)[32])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int n = 4, o = 16; n >= 1; n >>= 1, o >>= 1) {
        const bool hi = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = hi ? v[i] : v[i + n], keep = hi ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
    // lane holds value (lane >> 4) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1) = lane >> 2
    if ((lane & 3) == 0) part[lane >> 2][warp] = v[0];
    __syncthreads();
    float x = 0.f;
    const int which = lane >> 2;
    for (int i = lane & 3; i < nw; i += 4) x += part[which][i];
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    x += __shfl_xor_sync(0xffffffffu, x, 1);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __shfl_sync(0xffffffffu, x, i * 4);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Backward, pipelined (H <= 8192).  Persistent CTAs take tokens in grid-stride
// order, a thread owning two vectors of 8 columns; one thread copies the rows
// of the tokens ahead into a ring in shared memory (cp.async.bulk).
//
// All sums over a token's row follow from r, v = w_pre dy and u once rstd(o) is
// known:  sum D u = sum u dr + q sum u v - q^2 k sum u r   (q = rstd(r), k =
// mean(v n)), and mean(z m) is that sum over H (with the gate), so no sum needs
// the gradient D itself.  That leaves one barrier per token, between which a
// thread works on three tokens: the outputs of token i, the sums of token i + 1
// and mean(o^2) of token i + 2.
//
// The gradients of w_post and of the channel gate are both column sums of D m
// (times the other weight), so two column accumulators serve all three; they
// stay in registers and end in the CTA's row of the workspace, which
// norm_columns_kernel adds up in a fixed order (no atomics: the result does not
// depend on scheduling).
constexpr int kRowVecs = 2;       // vectors of a thread
constexpr int kRowThreads = 512;  // at most
constexpr int kRows = 3;          // tokens in the ring
constexpr int kNormSmem = 227 * 1024 - 2560;  // dynamic shared memory of a CTA, less the static part

template <bool WS>
__global__ void __launch_bounds__(kRowThreads, 1) norm_bwd_rows_kernel(const NormBwdArgs b)
{
    const NormArgs& a = b.f;
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ float part[2][8][32];
    __shared__ uint64_t bar_o[kRows], bar_r[kRows];
    __shared__ volatile int dead;
    const int H = a.H, nvec = H / 8, nt = blockDim.x;
    const uint32_t rb = (uint32_t)H * 2;
    uint4* ring = reinterpret_cast<uint4*>(dyn);                  // [kRows][4][nvec]: o, res, dr, dy
    float* sw = reinterpret_cast<float*>(ring + kRows * 4 * nvec);  // [2][H]: w_post gate, w_pre
    const bool chan = a.gate && !a.per_token, post = a.w_post != nullptr;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRows; ++i) {
            mbar_init(smem_u32(&bar_o[i]), 1);
            mbar_init(smem_u32(&bar_r[i]), 1);
        }
        dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    griddep_wait();
    // inputs that are absent read as zero
    if (!a.o || !a.res || !b.dr || !b.dy)
        for (int v = threadIdx.x; v < kRows * 4 * nvec; v += nt) ring[v] = make_uint4(0u, 0u, 0u, 0u);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();

    const int first = blockIdx.x, step = gridDim.x;
    const int count = first < b.T ? (b.T - first + step - 1) / step : 0;
    int issued = 0;  // thread 0: tokens whose copies were started
    auto load = [&](int i) {  // the CTA's i-th token
        if (i >= count) return;
        issued = i + 1;
        const size_t at = (size_t)(first + i * step) * nvec;
        uint4* d = ring + (i % kRows) * 4 * nvec;
        uint32_t bar = smem_u32(&bar_o[i % kRows]);
        if (a.o) {
            mbar_expect_tx(bar, rb);
            bulk_load(smem_u32(d), a.o + at, rb, bar);
        }
        bar = smem_u32(&bar_r[i % kRows]);
        mbar_expect_tx(bar, rb * ((a.res ? 1 : 0) + (b.dr ? 1 : 0) + (b.dy ? 1 : 0)));
        if (a.res) bulk_load(smem_u32(d + nvec), a.res + at, rb, bar);
        if (b.dr) bulk_load(smem_u32(d + 2 * nvec), b.dr + at, rb, bar);
        if (b.dy) bulk_load(smem_u32(d + 3 * nvec), b.dy + at, rb, bar);
    };
    if (threadIdx.x == 0)
        for (int i = 0; i < kRows; ++i) load(i);

    // w_post gate (channel), and w_pre; absent ones count as 1
    auto fetch = [&](int which, int v) {
        Vec w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w.v[j] = pack(1.f, 1.f);
        if (which == 1) return a.w_pre ? vec_of(a.w_pre + v * 8) : w;
        if (post) w = vec_of(a.w_post + v * 8);
        if (chan) {
            const Vec g = vec_of(a.gate + v * 8);
#pragma unroll
            for (int j = 0; j < 4; ++j) w.v[j] = mul2(w.v[j], g.v[j]);
        }
        return w;
    };
    if (WS) {
        // a thread stages the columns that it alone reads: no barrier
#pragma unroll
        for (int x = 0; x < kRowVecs; ++x) {
            const int v = threadIdx.x + x * nt;
            if (v >= nvec) continue;
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                const Vec w = fetch(which, v);
                ulonglong2* d = reinterpret_cast<ulonglong2*>(sw + which * H + v * 8);
                d[0] = make_ulonglong2(w.v[0], w.v[1]);
                d[1] = make_ulonglong2(w.v[2], w.v[3]);
            }
        }
    }
    auto weight = [&](int which, int v) { return WS ? vec_of(sw + which * H + v * 8) : fetch(which, v); };

    Vec c_pre[kRowVecs], c_dm[kRowVecs];
#pragma unroll
    for (int x = 0; x < kRowVecs; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) c_pre[x].v[j] = c_dm[x].v[j] = pack(0.f, 0.f);
    const f2 inv = pack(a.inv_h, a.inv_h), sc = pack(a.scale, a.scale);

    // Bounded waits for a token's rows; every thread waits for itself, and a
    // thread that gives up takes the whole CTA with it at the next barrier.
    auto wait = [&](uint64_t* bars, int i) {
        if (!mbar_wait(smem_u32(&bars[i % kRows]), (i / kRows) & 1, &dead)) dead = 1;
    };
    auto token_gate = [&](int i) { return a.gate && a.per_token ? __ldg(a.gate + first + i * step) : 1.f; };
    // s[5] = this thread's part of mean(o^2) of token i
    auto mean_o = [&](int i, float (&s)[8]) {
        if (i >= count || !a.o) return;
        wait(bar_o, i);
        if (!post) return;
        f2 acc = pack(0.f, 0.f);
#pragma unroll
        for (int x = 0; x < kRowVecs; ++x) {
            const int v = threadIdx.x + x * nt;
            if (v >= nvec) continue;
            const Vec o = widen(ring[(i % kRows) * 4 * nvec + v]);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc = fma2(mul2(o.v[j], inv), o.v[j], acc);
        }
        s[5] = sum2(acc);
    };
    // mean(r^2), mean(r v), and the sums of u (times the channel gate) with dr, v and r of token i
    auto sums = [&](int i, float p, float gt, float (&s)[8]) {
        if (i >= count) return;
        wait(bar_r, i);
        const uint4* row = ring + (i % kRows) * 4 * nvec;
        const f2 pp = pack(p, p), gg = pack(gt, gt);
        f2 s0 = pack(0.f, 0.f), s1 = s0, s2 = s0, s3 = s0, s4 = s0;
#pragma unroll
        for (int x = 0; x < kRowVecs; ++x) {
            const int v = threadIdx.x + x * nt;
            if (v >= nvec) continue;
            const Vec o = widen(row[v]), res = widen(row[nvec + v]), dr = widen(row[2 * nvec + v]),
                      dy = widen(row[3 * nvec + v]);
            const Vec wg = weight(0, v), wq = weight(1, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f2 u = mul2(wg.v[j], mul2(o.v[j], pp));
                const f2 r = fma2(sc, res.v[j], mul2(u, gg));
                const f2 vv = mul2(wq.v[j], dy.v[j]), ri = mul2(r, inv);
                s0 = fma2(ri, r, s0);
                s1 = fma2(ri, vv, s1);
                s2 = fma2(u, dr.v[j], s2);
                s3 = fma2(u, vv, s3);
                s4 = fma2(u, r, s4);
            }
        }
        s[0] = sum2(s0);
        s[1] = sum2(s1);
        s[2] = sum2(s2);
        s[3] = sum2(s3);
        s[4] = sum2(s4);
    };
    // the outputs of token i from its sums
    auto outputs = [&](int i, float p, float gt, const float (&s)[8]) {
        const size_t base = (size_t)(first + i * step) * nvec;
        const uint4* row = ring + (i % kRows) * 4 * nvec;
        const float q = b.dy ? rsqrtf(s[0] + a.eps) : 0.f;
        const float k = s[1] * q;                                    // mean(v n)
        const float du = s[2] + q * s[3] - q * q * k * s[4];         // sum of D u
        if (b.dgate && threadIdx.x == 0) b.dgate[first + i * step] = du;
        const float kz = du * gt * a.inv_h;                          // mean(z m)
        const f2 pp = pack(p, p), gg = pack(gt, gt), qq = pack(q, q), kq = pack(-k * q, -k * q), nz = pack(-kz, -kz);
#pragma unroll
        for (int x = 0; x < kRowVecs; ++x) {
            const int v = threadIdx.x + x * nt;
            if (v >= nvec) continue;
            const Vec o = widen(row[v]), res = widen(row[nvec + v]), dr = widen(row[2 * nvec + v]),
                      dy = widen(row[3 * nvec + v]);
            const Vec wg = weight(0, v), wq = weight(1, v);
            Vec ds, dz;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f2 m = mul2(o.v[j], pp);
                const f2 r = fma2(sc, res.v[j], mul2(mul2(wg.v[j], m), gg));
                const f2 n = mul2(r, qq);
                c_pre[x].v[j] = fma2(dy.v[j], n, c_pre[x].v[j]);
                f2 d = fma2(mul2(wq.v[j], dy.v[j]), qq, dr.v[j]);
                d = fma2(n, kq, d);
                ds.v[j] = mul2(sc, d);
                d = mul2(d, gg);
                c_dm[x].v[j] = fma2(d, m, c_dm[x].v[j]);
                dz.v[j] = mul2(wg.v[j], d);
                if (post) dz.v[j] = mul2(pp, fma2(m, nz, dz.v[j]));
            }
            if (b.dres) b.dres[base + v] = narrow(ds);
            if (b.d_o) b.d_o[base + v] = narrow(dz);
        }
    };

    float s[8] = {};
    mean_o(0, s);
    block_sum8(s, part[0]);
    float p = post ? rsqrtf(s[5] + a.eps) : 1.f, gt = count > 0 ? token_gate(0) : 1.f;
    float st[8] = {};  // sums of the token whose outputs come next
    sums(0, p, gt, st);
    mean_o(1, st);
    st[6] = (float)dead;
    block_sum8(st, part[1]);
    float p1 = post ? rsqrtf(st[5] + a.eps) : 1.f;
    for (int i = 0; i < count && st[6] == 0.f; ++i) {
        float nx[8] = {};
        const float gt1 = i + 1 < count ? token_gate(i + 1) : 1.f;
        sums(i + 1, p1, gt1, nx);
        outputs(i, p, gt, st);
        mean_o(i + 2, nx);
        nx[6] = (float)dead;
        block_sum8(nx, part[i & 1]);
        // every thread is done with token i: its place in the ring is free
        if (threadIdx.x == 0) load(i + kRows);
        p = p1;
        gt = gt1;
        p1 = post ? rsqrtf(nx[5] + a.eps) : 1.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) st[j] = nx[j];
    }
    if (st[6] != 0.f) {
        if (threadIdx.x == 0) {
            *(volatile unsigned*)(b.err + kErrTimeout) = 1u;
            // copies still in flight land in this CTA's shared memory
            volatile int go_on = 0;
            for (int i = max(0, issued - kRows); i < issued; ++i) {
                if (a.o) mbar_wait(smem_u32(&bar_o[i % kRows]), (i / kRows) & 1, &go_on);
                mbar_wait(smem_u32(&bar_r[i % kRows]), (i / kRows) & 1, &go_on);
            }
        }
        __syncthreads();
    }
    float* row = b.work + (size_t)blockIdx.x * 2 * H;
#pragma unroll
    for (int x = 0; x < kRowVecs; ++x) {
        const int v = threadIdx.x + x * nt;
        if (v >= nvec) continue;
        ulonglong2* d0 = reinterpret_cast<ulonglong2*>(row + v * 8);
        ulonglong2* d1 = reinterpret_cast<ulonglong2*>(row + H + v * 8);
        d0[0] = make_ulonglong2(c_pre[x].v[0], c_pre[x].v[1]);
        d0[1] = make_ulonglong2(c_pre[x].v[2], c_pre[x].v[3]);
        d1[0] = make_ulonglong2(c_dm[x].v[0], c_dm[x].v[1]);
        d1[1] = make_ulonglong2(c_dm[x].v[2], c_dm[x].v[3]);
    }
}

// Adds up the CTAs' column sums: dw_pre, and from the sums of D m the gradients
// of w_post (times the channel gate) and of the channel gate (times w_post).
__global__ void __launch_bounds__(256) norm_columns_kernel(const float* __restrict__ work, int rows, int H,
                                                           const float* w_post, const float* gate, float* dw_pre,
                                                           float* dw_post, float* dgate)
{
    griddep_wait();
    if (blockIdx.y == 0 ? !dw_pre : !dw_post && !dgate) return;
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < H)
        for (int i = part; i < rows; i += 8) v += work[((size_t)i * 2 + blockIdx.y) * H + c];
    s[part][lane] = v;
    __syncthreads();
    if (part != 0 || c >= H) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][lane];
    if (blockIdx.y == 0) {
        dw_pre[c] = v;
    } else {
        if (dw_post) dw_post[c] = gate ? v * __ldg(gate + c) : v;
        if (dgate) dgate[c] = w_post ? v * __ldg(w_post + c) : v;
    }
}

template <typename... KArgs, typename... Args>
cudaError_t launch_smem(void (*k)(KArgs...), int grid, int threads, int smem, cudaStream_t s, Args... args)
{
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl_smem(k, dim3(grid), dim3(threads), smem, s, args...);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int T, cudaStream_t s)
{
    if (T <= 0) return cudaSuccess;
    const int nvec = a.H / 8;
    const int vpt = nvec <= 256 ? 1 : nvec <= 512 ? 2 : nvec <= 1024 ? 4 : 8;
    const int threads = ((nvec + vpt - 1) / vpt + 31) & ~31;
    if (vpt == 1) return launch_pdl(norm_kernel<1>, dim3(T), dim3(threads), s, a);
    if (vpt == 2) return launch_pdl(norm_kernel<2>, dim3(T), dim3(threads), s, a);
    if (vpt == 4) return launch_pdl(norm_kernel<4>, dim3(T), dim3(threads), s, a);
    return launch_pdl(norm_kernel<8>, dim3(T), dim3(threads), s, a);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& b, float* dw_pre, float* dw_post, float* dgate_channel,
                            int sm_count, cudaStream_t s)
{
    const int H = b.f.H, nvec = H / 8;
    const int most = sm_count * norm_ctas(H), grid = b.T < most ? b.T : most;
    if (grid > 0) {
        const int ring = kRows * 4 * 2 * H, weights = 8 * H;
        cudaError_t e;
        if (nvec <= kRowVecs * kRowThreads) {
            const int threads = ((nvec + kRowVecs - 1) / kRowVecs + 31) & ~31;
            const bool ws = ring + weights <= kNormSmem;
            e = ws ? launch_smem(norm_bwd_rows_kernel<true>, grid, threads, ring + weights, s, b)
                   : launch_smem(norm_bwd_rows_kernel<false>, grid, threads, ring, s, b);
        } else {
            const int threads = ((nvec + 1) / 2 + 31) & ~31;
            e = launch_pdl(norm_bwd_kernel<2>, dim3(grid), dim3(threads), s, b);
        }
        if (e != cudaSuccess) return e;
    }
    if (!dw_pre && !dw_post && !dgate_channel) return cudaSuccess;
    const float* gate = b.f.per_token ? nullptr : b.f.gate;
    return launch_pdl(norm_columns_kernel, dim3((H + 31) / 32, 2), dim3(256), s, (const float*)b.work, grid, H,
                      b.f.w_post, gate, dw_pre, dw_post, dgate_channel);
}

}  // namespace moeep
