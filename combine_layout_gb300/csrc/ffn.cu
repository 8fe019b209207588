// The experts' gated feed-forward over the receive rows, forward and backward,
// on the fifth-generation tensor cores: products of the rows with their
// expert's weights, the activation fused into the product that feeds it.
//
// Orientation.  A tile is 256 weight rows (features) x up to 256 receive rows
// of one expert, shared by a pair of CTAs (cta_group::2): the weights are the
// tensor core's fixed operand of 2 x 128 rows and the tokens its n dimension,
// which any multiple of 32 up to 256 serves.  An
// expert's share of a batch is ragged and often small (a decoding step gives
// an expert a handful of rows), so the ragged dimension goes where the
// instruction takes it; with tokens on the 128-row side an expert with 5 rows
// would cost as much as one with 128.  The pair halves what a CTA stages of the tokens: 32 KB for
// 128 x 256 x 64 products per CTA where a CTA alone stages 48 KB.
//
// Roles of a CTA (192 threads): one thread loads its operand tiles by TMA into a
// ring of shared-memory stages, one thread of the pair's first CTA issues the
// products, four warps read the fp32 accumulators from tensor memory, apply the activation and
// store bf16.  The accumulators are double-buffered, so a tile's epilogue runs
// under the next tile's products.  CTAs are persistent; the tile list is
// derived on the device from the layout's counts (no host synchronisation).
#include <cuda_bf16.h>

#include "common.cuh"
#include "ffn.cuh"
#include "tc.cuh"

namespace moeep {
namespace {

constexpr int kThreads = 192;
constexpr int kKB = 64;      // contraction elements per stage (128 bytes of bf16)
constexpr int kTileM = 128;  // weight rows per CTA, 256 per pair
constexpr int kTileN = 256;  // receive rows per tile, at most
constexpr int kStages = 6;
constexpr int kBand = 8;     // n tiles that share the weights of one pass over an expert

// Shared-memory control block of a CTA.
template <int STAGES>
struct Control {
    uint64_t full[STAGES], empty[STAGES], ready[STAGES];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem;
    volatile int dead;  // a bounded wait gave up
    int part[kThreads / 32];
    int cnt[kMaxExperts];
    int pre[kMaxExperts + 1];  // n tiles before each expert
};

// One whole 32-byte sector.
__device__ __forceinline__ void store32(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e,
                                        uint32_t f, uint32_t g, uint32_t h)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a), "r"(b), "r"(c),
                 "r"(d), "r"(e), "r"(f), "r"(g), "r"(h)
                 : "memory");
}

__device__ __forceinline__ void give_up(volatile int* dead, unsigned* err)
{
    *dead = 1;
    *(volatile unsigned*)(err + kErrTimeout) = 1u;
}

// Counts and the exclusive prefix of the experts' n tiles (rows / nt, rounded
// up); all threads of the CTA.
__device__ __forceinline__ void tile_prefix(const int32_t* __restrict__ cnt, int E, int nt, int* s_cnt,
                                            int* s_pre, int* s_part)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (E + kThreads - 1) / kThreads;
    const int lo = min(tid * per, E), hi = min(lo + per, E);
    int sum = 0;
    for (int e = lo; e < hi; ++e) {
        const int c = __ldg(cnt + e);
        s_cnt[e] = c;
        sum += (c + nt - 1) / nt;
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
    }
    if (lane == 31) s_part[warp] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < warp; ++w) run += s_part[w];
    if (tid == kThreads - 1) s_pre[E] = run + sum;
    for (int e = lo; e < hi; ++e) {
        s_pre[e] = run;
        run += (s_cnt[e] + nt - 1) / nt;
    }
    __syncthreads();
}

// The i-th tile of the list: expert by expert; within an expert bands of
// kBand n tiles, and in a band the n tiles of one m tile before the next m
// tile, so CTAs that run together share weights and rows in L2.
struct Tile {
    int e = 0;     // expert
    int m;         // m tile
    int row;       // first receive row
    int rows;      // valid rows
    int n;         // rows of the product (a multiple of 32)

    __device__ __forceinline__ void find(int i, const int* cnt, const int* pre, int mt, const RowsArgs& a)
    {
        while (pre[e + 1] * mt <= i) ++e;
        const int nt = pre[e + 1] - pre[e], c = cnt[e];
        const int r = i - pre[e] * mt;
        const int b = r / (kBand * mt);
        const int nb = min(kBand, nt - b * kBand);
        const int q = r - b * kBand * mt;
        m = q / nb;
        const int j = b * kBand + (q - m * nb);
        // equal tiles, in steps of the instruction's n granularity
        const int w = ((c + nt - 1) / nt + 31) & ~31;
        rows = min(w, c - j * w);
        n = (rows + 31) & ~31;
        row = (a.mode == MOE_EP_HT ? __ldg(a.off + e) : e * a.S) + j * w;
    }
};

__device__ __forceinline__ float sigmoid(float g) { return 1.f / (1.f + __expf(-g)); }

// act(g) and its derivative.
template <bool GRAD>
__device__ __forceinline__ float act(float g, int kind, float& slope)
{
    if (kind == MOE_EP_ACT_SILU) {
        const float s = sigmoid(g);
        if (GRAD) slope = s * (1.f + g * (1.f - s));
        return g * s;
    }
    const float cdf = 0.5f * (1.f + erff(g * 0.70710678f));
    if (GRAD) slope = cdf + g * 0.39894228f * __expf(-0.5f * g * g);
    return g * cdf;
}

// Epilogues: sixteen accumulator columns (receive rows r0 + c0 ..) of the
// warp's 32 tile rows.
__device__ __forceinline__ void epi_store(const float (&v)[16], const RowsArgs& a, size_t row, int left,
                                          int m)
{
    if (m >= a.M) return;
    __nv_bfloat16* p = a.out + row * a.M + m;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < left) p[(size_t)i * a.M] = __float2bfloat16_rn(v[i]);
}

// Tile rows alternate 8 gate and 8 up features, so a feature's gate and up
// values sit 8 lanes apart: of two neighbouring columns the gate lane takes
// the first and the up lane the second, after one exchange.
__device__ __forceinline__ void epi_gate_up(const float (&v)[16], const RowsArgs& a, size_t row, int left,
                                            int f, int up)
{
    const bool ok = f < a.F;
    if (a.keep && ok) {
        __nv_bfloat16* p = a.keep + row * 2 * a.F + (up ? a.F : 0) + f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < left) p[(size_t)i * 2 * a.F] = __float2bfloat16_rn(v[i]);
    }
    __nv_bfloat16* h = a.out + (row + up) * a.F + f;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const float got = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 1], 8);
        const float g = up ? got : v[i], u = up ? v[i + 1] : got;
        float slope;
        const float r = act<false>(g, a.act, slope) * u;
        if (ok && i + up < left) h[(size_t)i * a.F] = __float2bfloat16_rn(r);
    }
}

// d hid (the accumulators) to d gate, d up, and the product of the forward
// pass again.
__device__ __forceinline__ void epi_down_bwd(const float (&v)[16], const RowsArgs& a, size_t row, int left,
                                             int f)
{
    if (f >= a.F) return;
    const __nv_bfloat16* gp = a.gate_up + row * 2 * a.F + f;
    __nv_bfloat16* dp = a.out + row * 2 * a.F + f;
    __nv_bfloat16 g[16], u[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < left) {
            g[i] = gp[(size_t)i * 2 * a.F];
            u[i] = gp[(size_t)i * 2 * a.F + a.F];
        }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < left) {
            const float gf = __bfloat162float(g[i]), uf = __bfloat162float(u[i]);
            float slope;
            const float av = act<true>(gf, a.act, slope);
            dp[(size_t)i * 2 * a.F] = __float2bfloat16_rn(v[i] * uf * slope);
            dp[(size_t)i * 2 * a.F + a.F] = __float2bfloat16_rn(v[i] * av);
            if (a.keep) a.keep[(row + i) * a.F + f] = __float2bfloat16_rn(av * uf);
        }
}

// Barriers, tensor memory and the pair; every thread of both CTAs.
template <int STAGES>
__device__ __forceinline__ void start_pair(Control<STAGES>& c, int warp)
{
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(smem_u32(&c.full[i]), 1);
            mbar_init(smem_u32(&c.empty[i]), 1);
            mbar_init(smem_u32(&c.ready[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&c.acc_full[i]), 1);
            mbar_init(smem_u32(&c.acc_empty[i]), 8);  // the epilogue warps of both CTAs
        }
        mbar_init(smem_u32(&c.drain), 1);
        c.dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc(smem_u32(&c.tmem), 512);
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
}

// Nothing may still arrive at a CTA that has left: both leave together.
template <int STAGES>
__device__ __forceinline__ void end_pair(Control<STAGES>& c, int warp)
{
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_free(c.tmem, 512);
}

// A producer that gave up waits (with a limit) for the copies in flight: they
// land in the pair's shared memory.
template <int STAGES>
__device__ __forceinline__ void drain_copies(Control<STAGES>& c, uint32_t issued, unsigned* err)
{
    give_up(&c.dead, err);
    volatile int go_on = 0;
    for (uint32_t j = issued < STAGES ? 0 : issued - STAGES; j < issued; ++j)
        mbar_wait(smem_u32(&c.full[j % STAGES]), (j / STAGES) & 1u, &go_on);
}
// ... and an issuer for its products, which read that memory.
template <int STAGES>
__device__ __forceinline__ void drain_products(Control<STAGES>& c, unsigned* err)
{
    give_up(&c.dead, err);
    volatile int go_on = 0;
    tc_commit(smem_u32(&c.drain));
    mbar_wait(smem_u32(&c.drain), 0, &go_on);
}

template <int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    rows_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ RowMaps rmap,
                const RowsArgs a)
{
    constexpr bool A_MN = EPI == kRowsDownBwd || EPI == kRowsStoreT;
    constexpr int STAGES = kStages;
    constexpr int kABytes = kTileM * kKB * 2, kStageBytes = kABytes + kTileN / 2 * kKB * 2;
    extern __shared__ uint8_t dyn[];
    __shared__ Control<STAGES> c;
    const int warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_rank();
    const uint32_t ring = (smem_u32(dyn) + 1023u) & ~1023u;

    start_pair(c, warp);
    griddep_wait();
    tile_prefix(a.cnt, a.E, kTileN, c.cnt, c.pre, c.part);
    const int total = c.pre[a.E] * a.mt, first = blockIdx.x >> 1, step = gridDim.x >> 1;
    const int kblocks = (a.K + kKB - 1) / kKB;

    if (warp == 0) {
        if (elect_one()) {
            uint32_t it = 0;  // k blocks loaded
            Tile t;
            bool ok = true;
            for (int i = first; i < total && ok; i += step) {
                t.find(i, c.cnt, c.pre, a.mt, a);
                const int m = t.m * 2 + (int)rank, half = t.n / 2, row = t.row + (int)rank * half;
                for (int kb = 0; kb < kblocks; ++kb, ++it) {
                    const uint32_t s = it % STAGES, ph = (it / STAGES) & 1u;
                    if (!mbar_wait(smem_u32(&c.empty[s]), ph ^ 1u, &c.dead)) {
                        ok = false;
                        break;
                    }
                    // both CTAs' bytes are counted on the first one's barrier
                    const uint32_t bar = in_cta(smem_u32(&c.full[s]), 0);
                    const uint32_t sa = ring + s * kStageBytes, sb = sa + kABytes;
                    if (rank == 0) mbar_expect_tx(smem_u32(&c.full[s]), 2 * kABytes + t.n * kKB * 2);
                    const int k0 = kb * kKB;
                    if (EPI == kRowsGateUp) {
                        // [expert][f / 8][gate, up][f % 8][H]: 8 gate and 8 up rows in turn
                        tma_load(sa, &wmap, bar, k0, 0, 0, m * (kTileM / 16), t.e);
                    } else if (A_MN) {
                        tma_load(sa, &wmap, bar, m * kTileM, k0, t.e);
                        tma_load(sa + kABytes / 2, &wmap, bar, m * kTileM + 64, k0, t.e);
                    } else {
                        tma_load(sa, &wmap, bar, k0, m * kTileM, t.e);
                    }
                    for (int b = 0, r = 0; b < kRowBoxes; ++b) {
                        const int h = 128 >> b;
                        for (; half - r >= h; r += h) tma_load(sb + r * 128, &rmap.box[b], bar, k0, row + r);
                    }
                }
            }
            if (!ok) drain_copies(c, rank == 0 ? it : 0, a.err);
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            uint32_t it = 0, tile = 0;
            Tile t;
            bool ok = true;
            for (int i = first; i < total && ok; i += step, ++tile) {
                t.find(i, c.cnt, c.pre, a.mt, a);
                const uint32_t acc = tile & 1u;
                if (!mbar_wait(smem_u32(&c.acc_empty[acc]), ((tile >> 1) & 1u) ^ 1u, &c.dead)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = c.tmem + acc * kTileN;
                const uint32_t idesc = tc_idesc(2 * kTileM, t.n, A_MN, 0);
                for (int kb = 0; kb < kblocks; ++kb, ++it) {
                    const uint32_t s = it % STAGES, ph = (it / STAGES) & 1u;
                    if (!mbar_wait(smem_u32(&c.full[s]), ph, &c.dead)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = ring + s * kStageBytes, sb = sa + kABytes;
                    // past the end of the contraction the tiles hold zeros
                    const int steps = min(kKB / 16, (a.K - kb * kKB + 15) / 16);
                    for (int k = 0; k < steps; ++k)
                        tc_mma(d, tc_desc(sa + k * (A_MN ? 2048 : 32), A_MN ? kABytes / 2 : 16),
                               tc_desc(sb + k * 32, 16), idesc, (kb | k) != 0);
                    tc_commit(smem_u32(&c.empty[s]));
                }
                if (ok) tc_commit(smem_u32(&c.acc_full[acc]));
            }
            if (!ok) drain_products(c, a.err);
        }
    } else {
        const int lane = threadIdx.x & 31, quarter = warp & 3;  // tensor-memory lanes of this warp
        uint32_t tile = 0;
        Tile t;
        for (int i = first; i < total; i += step, ++tile) {
            t.find(i, c.cnt, c.pre, a.mt, a);
            const uint32_t acc = tile & 1u;
            if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&c.acc_full[acc]), (tile >> 1) & 1u, &c.dead))) {
                if (lane == 0) give_up(&c.dead, a.err);
                break;
            }
            tc_fence_after();
            const uint32_t src = c.tmem + acc * kTileN + ((uint32_t)(quarter * 32) << 16);
            const int r = (t.m * 2 + (int)rank) * kTileM + quarter * 32 + lane;  // weight row
            for (int c0 = 0; c0 < t.n; c0 += 16) {
                float v[16];
                tmem_ld16(src + c0, v);
                const size_t row = (size_t)(t.row + c0);
                const int left = t.rows - c0;
                if (EPI == kRowsGateUp)
                    epi_gate_up(v, a, row, left, (r >> 4) * 8 + (r & 7), (r >> 3) & 1);
                else if (EPI == kRowsDownBwd)
                    epi_down_bwd(v, a, row, left, r);
                else
                    epi_store(v, a, row, left, r);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(in_cta(smem_u32(&c.acc_empty[acc]), 0));
        }
    }
    end_pair(c, warp);
}

// ---------------------------------------------------------------------------
// Weight gradients: dW[e] = sum over the expert's rows of a_row b_row^T.  Both
// operands are read with their features contiguous (rows are the contraction);
// a tile is 256 x 256 of one expert's gradient, 128 x 256 in each CTA.  The last
// block of an expert's rows may reach into rows that are not its own (the next
// expert's, or slots that were never written): those rows of both operands are
// cleared in shared memory before the product, because 0 x NaN would not be 0.
// For that each CTA's copies are counted on its own barrier; the second CTA's
// issuing warp clears its rows and passes the block on to the first one's
// (`ready`), which clears its own and issues.
template <bool F32>
__device__ __forceinline__ void store_grad(const float (&v)[16], const GradArgs& a, size_t at, int n, bool wide)
{
    if (F32) {
        float* p = (float*)a.dw + at;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = v[i];
        if (a.accumulate) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                if (i < n) {
                    const float4 o = *reinterpret_cast<const float4*>(p + i);
                    x[i] += o.x; x[i + 1] += o.y; x[i + 2] += o.z; x[i + 3] += o.w;
                }
        }
#pragma unroll
        for (int i = 0; i < 16; i += 8)
            if (i < n) {
                if (wide) {
                    store32(p + i, __float_as_uint(x[i]), __float_as_uint(x[i + 1]), __float_as_uint(x[i + 2]),
                            __float_as_uint(x[i + 3]), __float_as_uint(x[i + 4]), __float_as_uint(x[i + 5]),
                            __float_as_uint(x[i + 6]), __float_as_uint(x[i + 7]));
                } else {
                    *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                    *reinterpret_cast<float4*>(p + i + 4) = make_float4(x[i + 4], x[i + 5], x[i + 6], x[i + 7]);
                }
            }
    } else {
        __nv_bfloat16* p = (__nv_bfloat16*)a.dw + at;
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            o[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        if (wide && n >= 16) {
            store32(p, o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7]);
        } else {
            *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
            if (n >= 16) *reinterpret_cast<uint4*>(p + 8) = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

template <bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    grad_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                const GradArgs a)
{
    constexpr int STAGES = kStages;
    constexpr int kABytes = kTileM * kKB * 2, kStageBytes = 2 * kABytes;
    constexpr int kBlock = 64 * kKB * 2;  // 64 features x 64 rows
    extern __shared__ uint8_t dyn[];
    __shared__ Control<STAGES> c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t ring = (smem_u32(dyn) + 1023u) & ~1023u;
    start_pair(c, warp);
    griddep_wait();
    const int per = a.mt * a.nt;
    const int64_t total = (int64_t)per * a.E, first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (warp == 0) {
        if (elect_one()) {
            uint32_t it = 0;
            bool ok = true;
            for (int64_t i = first; i < total && ok; i += step) {
                const int e = (int)(i / per), q = (int)(i - (int64_t)e * per);
                const int m0 = ((q / a.nt) * 2 + (int)rank) * kTileM;
                const int n0 = (q % a.nt) * kTileN + (int)rank * (kTileN / 2);
                const int rows = __ldg(a.cnt + e), base = a.mode == MOE_EP_HT ? __ldg(a.off + e) : e * a.S;
                for (int r = 0; r < rows; r += kKB, ++it) {
                    const uint32_t s = it % STAGES, ph = (it / STAGES) & 1u;
                    if (!mbar_wait(smem_u32(&c.empty[s]), ph ^ 1u, &c.dead)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = smem_u32(&c.full[s]);
                    const uint32_t sa = ring + s * kStageBytes, sb = sa + kABytes;
                    mbar_expect_tx(bar, kStageBytes);
                    for (int b = 0; b < 2; ++b) {
                        tma_load(sa + b * kBlock, &amap, bar, m0 + b * 64, base + r);
                        tma_load(sb + b * kBlock, &bmap, bar, n0 + b * 64, base + r);
                    }
                }
            }
            if (!ok) drain_copies(c, it, a.err);
        }
    } else if (warp == 1) {
        uint32_t it = 0, tile = 0;
        bool ok = true;
        const uint32_t idesc = tc_idesc(2 * kTileM, kTileN, 1, 1);
        for (int64_t i = first; i < total && ok; i += step) {
            const int rows = __ldg(a.cnt + (int)(i / per));
            if (rows == 0) continue;
            const uint32_t acc = tile & 1u;
            if (rank == 0) {
                ok = __all_sync(0xffffffffu,
                                mbar_wait(smem_u32(&c.acc_empty[acc]), ((tile >> 1) & 1u) ^ 1u, &c.dead));
                if (!ok) break;
                tc_fence_after();
            }
            const uint32_t d = c.tmem + acc * kTileN;
            for (int r = 0; r < rows; r += kKB, ++it) {
                const uint32_t s = it % STAGES, ph = (it / STAGES) & 1u;
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&c.full[s]), ph, &c.dead));
                if (!ok) break;
                const uint32_t sa = ring + s * kStageBytes, sb = sa + kABytes;
                const int left = min(rows - r, kKB), steps = (left + 15) / 16;
                if (left < steps * 16) {
                    // rows left .. steps * 16 of every 64-feature block (the
                    // swizzle moves 16-byte units within a row's 128 bytes only)
                    const int units = (steps * 16 - left) * 8;
                    for (int b = 0; b < kStageBytes / kBlock; ++b)
                        for (int x = lane; x < units; x += 32)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             sa + b * kBlock + left * 128 + x * 16),
                                         "r"(0)
                                         : "memory");
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                if (rank != 0) {
                    if (lane == 0) mbar_arrive_cluster(in_cta(smem_u32(&c.ready[s]), 0));
                    continue;
                }
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&c.ready[s]), ph, &c.dead));
                if (!ok) break;
                tc_fence_after();
                if (lane == 0) {
                    for (int k = 0; k < steps; ++k)
                        tc_mma(d, tc_desc(sa + k * 2048, kBlock), tc_desc(sb + k * 2048, kBlock), idesc,
                               (r | k) != 0);
                    tc_commit(smem_u32(&c.empty[s]));
                }
                __syncwarp();
            }
            if (ok && rank == 0 && lane == 0) tc_commit(smem_u32(&c.acc_full[acc]));
            __syncwarp();
            ++tile;
        }
        if (!ok && lane == 0) {
            if (rank == 0)
                drain_products(c, a.err);
            else
                give_up(&c.dead, a.err);
        }
    } else {
        const int quarter = warp & 3;
        // 32-byte stores need rows that start on 32 bytes
        const bool wide = a.N % 16 == 0 && ((uintptr_t)a.dw & 31u) == 0;
        uint32_t tile = 0;
        for (int64_t i = first; i < total; i += step) {
            const int e = (int)(i / per), q = (int)(i - (int64_t)e * per);
            const int m = ((q / a.nt) * 2 + (int)rank) * kTileM + quarter * 32 + lane, n0 = (q % a.nt) * kTileN;
            const bool some = __ldg(a.cnt + e) > 0;
            if (!some && a.accumulate) continue;
            const uint32_t acc = tile & 1u;
            if (some) {
                if (!__all_sync(0xffffffffu,
                                mbar_wait(smem_u32(&c.acc_full[acc]), (tile >> 1) & 1u, &c.dead))) {
                    if (lane == 0) give_up(&c.dead, a.err);
                    break;
                }
                tc_fence_after();
            }
            const uint32_t src = c.tmem + acc * kTileN + ((uint32_t)(quarter * 32) << 16);
            const size_t at = ((size_t)e * a.M + m) * a.N + n0;
            const int cols = min(kTileN, a.N - n0);
            for (int c0 = 0; c0 < cols; c0 += 16) {
                float v[16];
                if (some) {
                    tmem_ld16(src + c0, v);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = 0.f;
                }
                if (m < a.M) store_grad<F32>(v, a, at + c0, cols - c0, wide);
            }
            if (some) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(in_cta(smem_u32(&c.acc_empty[acc]), 0));
                ++tile;
            }
        }
    }
    end_pair(c, warp);
}

constexpr int kSmem = kStages * 2 * kTileM * kKB * 2 + 1024;

template <typename... KArgs, typename... Args>
cudaError_t launch_pairs(void (*k)(KArgs...), int64_t pairs, int sm_count, cudaStream_t s, const Args&... args)
{
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const int most = sm_count / 2;
    const int n = (int)(pairs < most ? pairs : most);
    return launch_pdl_smem(k, dim3(2 * n), dim3(kThreads), kSmem, s, args...);
}

}  // namespace

cudaError_t launch_rows_product(int epi, const void* rows_in, int64_t nrows, const void* weights,
                                RowsArgs a, int64_t max_rows, int sm_count, cudaStream_t s)
{
    CUtensorMap wmap;
    RowMaps rmap;
    cudaError_t e;
    const uint64_t K = (uint64_t)a.K, M = (uint64_t)a.M, F = (uint64_t)a.F, E = (uint64_t)a.E;
    if (epi == kRowsGateUp) {
        const uint64_t dims[5] = {K, 8, 2, F / 8, E};
        const uint64_t str[4] = {K * 2, F * K * 2, 8 * K * 2, 2 * F * K * 2};
        const uint32_t box[5] = {kKB, 8, 2, kTileM / 16, 1};
        e = encode_tiles(&wmap, weights, 5, dims, str, box);
    } else if (epi == kRowsStore) {
        const uint64_t dims[3] = {K, M, E}, str[2] = {K * 2, M * K * 2};
        const uint32_t box[3] = {kKB, kTileM, 1};
        e = encode_tiles(&wmap, weights, 3, dims, str, box);
    } else {
        const uint64_t dims[3] = {M, K, E}, str[2] = {M * 2, M * K * 2};
        const uint32_t box[3] = {64, kKB, 1};
        e = encode_tiles(&wmap, weights, 3, dims, str, box);
    }
    if (e != cudaSuccess) return e;
    for (int b = 0; b < kRowBoxes; ++b) {
        const uint64_t dims[2] = {K, (uint64_t)nrows}, str[1] = {K * 2};
        const uint32_t box[2] = {kKB, 128u >> b};
        e = encode_tiles(&rmap.box[b], rows_in, 2, dims, str, box);
        if (e != cudaSuccess) return e;
    }
    a.mt = (int)(((epi == kRowsGateUp ? 2 * F : M) + 2 * kTileM - 1) / (2 * kTileM));
    // an upper bound of the tiles: every expert with rows ends in a partial tile
    const int64_t bound = (int64_t)a.mt * ((max_rows < a.E ? max_rows : a.E) + max_rows / kTileN);
    if (bound > INT32_MAX) return cudaErrorInvalidValue;  // tiles are counted in 32 bits
    switch (epi) {
        case kRowsGateUp: return launch_pairs(rows_kernel<kRowsGateUp>, bound, sm_count, s, wmap, rmap, a);
        case kRowsStore: return launch_pairs(rows_kernel<kRowsStore>, bound, sm_count, s, wmap, rmap, a);
        case kRowsDownBwd: return launch_pairs(rows_kernel<kRowsDownBwd>, bound, sm_count, s, wmap, rmap, a);
        default: return launch_pairs(rows_kernel<kRowsStoreT>, bound, sm_count, s, wmap, rmap, a);
    }
}

cudaError_t launch_weight_grad(const void* arows, const void* brows, int64_t nrows, int f32, GradArgs a,
                               int sm_count, cudaStream_t s)
{
    CUtensorMap amap, bmap;
    const uint32_t box[2] = {64, kKB};
    const uint64_t ad[2] = {(uint64_t)a.M, (uint64_t)nrows}, as[1] = {(uint64_t)a.M * 2};
    const uint64_t bd[2] = {(uint64_t)a.N, (uint64_t)nrows}, bs[1] = {(uint64_t)a.N * 2};
    cudaError_t e = encode_tiles(&amap, arows, 2, ad, as, box);
    if (e == cudaSuccess) e = encode_tiles(&bmap, brows, 2, bd, bs, box);
    if (e != cudaSuccess) return e;
    a.mt = (a.M + 2 * kTileM - 1) / (2 * kTileM);
    a.nt = (a.N + kTileN - 1) / kTileN;
    const int64_t total = (int64_t)a.mt * a.nt * a.E;
    return f32 ? launch_pairs(grad_kernel<true>, total, sm_count, s, amap, bmap, a)
               : launch_pairs(grad_kernel<false>, total, sm_count, s, amap, bmap, a);
}

cudaError_t encode_tiles(CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
                         const uint64_t* strides, const uint32_t* box)
{
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (Encode)p;
    }();
    if (!encode) return cudaErrorNotSupported;
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base),
                              reinterpret_cast<const cuuint64_t*>(dims),
                              reinterpret_cast<const cuuint64_t*>(strides), box, one,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace moeep
