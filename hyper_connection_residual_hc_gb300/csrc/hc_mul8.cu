// Products of 8-bit rows with 8-bit weights, both with a scale for each 128 values along k, for few rows: plain, or the gate and
// up projections at once with the activation, the product and its quantisation behind them. Formulas and format: include/hc.h.
//
//   out[t, f] = sum over blocks b of  xs[t, b] * ws[f / 128, b] * sum over i in b of  x[t, i] * w[f, i]
//
// The inner sums run on tcgen05.mma (fp32 accumulators in tensor memory, 4 instructions of K = 32 to a block); as the scales are
// any fp32 numbers, each block's sums leave tensor memory and are added up in fp32 registers with the two scales' product.
//
// The weights are the MMA's M: a CTA takes 128 features (tensor memory lanes) by up to 128 tokens (columns), so that a single
// token wastes columns, which cost nothing, rather than rows of weights, which have to be read anyway. With few tokens the
// weights' bytes are what counts: the blocks of k of a feature tile are cut over a cluster of up to 8 CTAs, so that all SMs
// read, and the partial sums meet through distributed shared memory in the order of the ranks. No workspace, no atomics: the result
// does not depend on timing.
//
// Warps: one issues TMA loads (a ring of k blocks: 128 x 128 bytes of weights, the tokens' block), one the MMAs, 4 or 8 add up.
//
// Measured: one token by 20,480 x 5,120 20 us (16 of it reading, at 6.6 TB/s; the rest is launch, set-up and the join), by 5,120 x 5,120 5.8
// in a graph, 33 tokens by 5,120 x 100,003 87 us (89% of the copy rate); gated, one token by 5,120 x 20,480 35 us. With more than 128
// tokens, or gated more than 64, hc_mul8_tiles.cu is faster nearly always: its adding warps have one factor a thread, these have one
// a column, from shared memory. launch_mul8 compares the two kernels' estimated times.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "hc_attn.h"
#include "hc_ffn.h"
#include "hc_mul8_dev.cuh"
#include "hc_mul8_host.h"

namespace hc {
namespace {

__device__ unsigned int g_hc_mul8_error = 0;
std::atomic<bool> g_launched{false};

constexpr int kTile = 128;    // features of a CTA
constexpr int kGroup = 8;     // k blocks whose scales are staged together
constexpr int kMostCluster = 8;

// kN: tokens of a tile; kGated: gate and up; kPerSm: CTAs that share an SM
template <int kN, bool kGated, int kPerSm>
struct Plan {
    static constexpr int kMats = kGated ? 2 : 1;
    static constexpr int kSets = kN > 64 ? 2 : 1;             // sets of 4 warps that share the tokens
    static constexpr int kCols = kN / kSets;                  // of a thread
    static constexpr int kAddWarps = 4 * kSets;
    static constexpr int kAhead = kMats * kCols < 128 ? 1 : 0;  // loads of 16 columns ahead of their use, where registers allow it
    static constexpr int kThreads = 32 * (kAddWarps + 2);
    static constexpr int kW = kTile * kBlock8;                // bytes
    static constexpr int kX = kN * kBlock8;
    static constexpr int kStage = kMats * kW + kX;
    static constexpr int kScaleBytes = 2 * kGroup * kMats * kN * 4;
    static constexpr int kBarBytes = 256;
    static constexpr int kRoom = (kPerSm == 2 ? 113 : 227) * 1024 - 1024 - kScaleBytes - kBarBytes;
    static constexpr int kStages = kRoom / kStage < 8 ? kRoom / kStage : 8;
    static_assert(kStages >= 2, "a ring");
    static_assert(kN * kTile * 4 * kMats <= kStages * kStage, "the partial sums take the ring's place");
    static constexpr int kScales = kStages * kStage;
    static constexpr int kBars = kScales + kScaleBytes;
    static constexpr int kSmem = kBars + kBarBytes + 1024;    // + alignment
    static constexpr uint32_t kBuffer = kMats * kN;           // tensor memory columns of a block's sums
    static constexpr uint32_t kColumns = 2 * kBuffer < 32 ? 32 : 2 * kBuffer;
    static_assert((2 * kStages + 4) * 8 + 16 <= kBarBytes, "barriers");
};

struct Params {
    Mul8Args a;
    int k_blocks, token_tiles, ctas;
};

template <int kN, bool kGated, int kPerSm>
__global__ void __launch_bounds__(Plan<kN, kGated, kPerSm>::kThreads, kPerSm)
mul8_rows_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_up,
                 const __grid_constant__ Params p) {
    using P = Plan<kN, kGated, kPerSm>;
    extern __shared__ unsigned char raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t bars = base + P::kBars;
    const uint32_t full = bars, empty = full + 8 * P::kStages, acc_full = empty + 8 * P::kStages, acc_empty = acc_full + 16, slot = acc_empty + 16;
    unsigned char* at = raw + (base - smem_u32(raw));
    volatile uint32_t* abort_word = reinterpret_cast<volatile uint32_t*>(at + (slot + 4 - base));
    const Wait8 wait{abort_word, &g_hc_mul8_error};

    const int rank = static_cast<int>(blockIdx.x) % p.ctas, unit = static_cast<int>(blockIdx.x) / p.ctas;
    const int ft = unit / p.token_tiles, tt = unit % p.token_tiles;
    const long long t0 = static_cast<long long>(tt) * kN;
    const int tokens = static_cast<int>(min(static_cast<long long>(kN), p.a.n - t0));
    const int b0 = static_cast<int>(static_cast<long long>(p.k_blocks) * rank / p.ctas);
    const int b1 = static_cast<int>(static_cast<long long>(p.k_blocks) * (rank + 1) / p.ctas);

    if (warp == P::kAddWarps + 1) {
        tmem_alloc(slot, P::kColumns);
        tmem_relinquish();
        // The kernel behind sets itself up as SMs get free. It may hold tensor memory while it waits for this grid's end, so that it must
        // not come before this CTA has its own.
        griddep_launch_dependents();
    }
    if (tid == 0) {
        for (int i = 0; i < P::kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, P::kAddWarps);
        }
        *abort_word = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(at + (slot - base));
    griddep_wait();  // what the kernels ahead write and read

    if (warp == P::kAddWarps) {  // ---- loads
        if (lane == 0) {
            const uint64_t once = policy_evict_normal(), again = policy_evict_last();
            for (int b = b0; b < b1; ++b) {
                const int i = b - b0, s = i % P::kStages;
                if (i >= P::kStages) wait(empty + 8 * s, (i / P::kStages - 1) & 1);
                const uint32_t st = base + s * P::kStage;
                mbar_arrive_expect_tx(full + 8 * s, P::kStage);
                tma_load_2d(st, &tm_w, full + 8 * s, b * kBlock8, ft * kTile, once);
                if constexpr (kGated) tma_load_2d(st + P::kW, &tm_up, full + 8 * s, b * kBlock8, ft * kTile, once);
                tma_load_2d(st + P::kMats * P::kW, &tm_x, full + 8 * s, b * kBlock8, static_cast<int>(t0), again);
            }
            // no copy is in flight when the CTA ends, whatever happened
            for (int i = max(b1 - b0 - P::kStages, 0); i < b1 - b0; ++i) wait.drain(full + 8 * (i % P::kStages), (i / P::kStages) & 1);
        }
        __syncwarp();
    } else if (warp == P::kAddWarps + 1) {  // ---- MMAs
        const uint32_t lead = elect_one();
        constexpr uint32_t idesc = idesc8(kTile, kN);
        for (int i = 0; i < b1 - b0; ++i) {
            const int s = i % P::kStages, u = i & 1;
            if (i >= 2) wait(acc_empty + 8 * u, (i / 2 - 1) & 1);
            wait(full + 8 * s, (i / P::kStages) & 1);
            tc_fence_after();
            const uint32_t st = base + s * P::kStage, d = tmem + u * P::kBuffer;
            const uint64_t x = sdesc8(st + P::kMats * P::kW);
#pragma unroll
            for (int m = 0; m < P::kMats; ++m) {
                const uint64_t w = sdesc8(st + m * P::kW);
#pragma unroll
                for (int q = 0; q < 4; ++q) mma8(lead, d + m * kN, w + 2 * q, x + 2 * q, idesc, q > 0);
            }
            if (i + P::kStages < b1 - b0) commit8(lead, empty + 8 * s);  // (an arrival that nothing waited for could come when the CTA has ended)
            commit8(lead, acc_full + 8 * u);
        }
        if (b1 > b0) wait.drain(acc_full + 8 * ((b1 - b0 - 1) & 1), ((b1 - b0 - 1) / 2) & 1);
    } else {  // ---- sums
        constexpr int kAdders = 32 * P::kAddWarps, kEach = kGroup * kN / kAdders;
        static_assert(kEach >= 1, "every thread stages scales");
        float* scales = reinterpret_cast<float*>(at + P::kScales);  // [2][kMats][kGroup][kN]
        float next[kEach][P::kMats];
        // the products of the tokens' scales and the feature tile's, for the k blocks of a group
        auto fetch = [&](int group) {
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int i = tid + e * kAdders, t = i / kGroup, b = b0 + group * kGroup + i % kGroup;
                const bool in = t < tokens && b < b1;
                const float xs = in ? p.a.x_scales[(t0 + t) * p.k_blocks + b] : 0.f;
                const long long w = static_cast<long long>(ft) * p.k_blocks + b;
                next[e][0] = in ? xs * p.a.w_scales[w] : 0.f;
                if constexpr (kGated) next[e][1] = in ? xs * p.a.up_scales[w] : 0.f;
            }
        };
        auto put = [&](int group) {
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int i = tid + e * kAdders, t = i / kGroup, b = i % kGroup;
#pragma unroll
                for (int m = 0; m < P::kMats; ++m) scales[(((group & 1) * P::kMats + m) * kGroup + b) * kN + t] = next[e][m];
            }
            asm volatile("bar.sync 1, %0;" ::"n"(kAdders) : "memory");
        };
        const int set = warp / 4;
        uint64_t acc[P::kMats][P::kCols / 2];
#pragma unroll
        for (int m = 0; m < P::kMats; ++m)
#pragma unroll
            for (int j = 0; j < P::kCols / 2; ++j) acc[m][j] = 0;
        if (b1 > b0) {
            fetch(0);
            put(0);
        }
        for (int i = 0; i < b1 - b0; ++i) {
            const int u = i & 1, group = i / kGroup;
            if (i % kGroup == 0 && i + kGroup < b1 - b0) fetch(group + 1);
            wait(acc_full + 8 * u, (i / 2) & 1);
            tc_fence_after();
            const uint32_t from = tmem + (static_cast<uint32_t>(32 * (warp % 4)) << 16) + u * P::kBuffer + set * P::kCols;
            const float* f = scales + ((group & 1) * P::kMats * kGroup + i % kGroup) * kN + set * P::kCols;
            constexpr int kParts = P::kCols / 16;
            float v[P::kAhead + 1][16];
            if constexpr (P::kAhead) tmem_start16(from, v[0]);
#pragma unroll
            for (int q = 0; q < kParts * P::kMats; ++q) {
                const int m = q / kParts, c = q % kParts;
                if constexpr (P::kAhead) {
                    tmem_wait();
                    if (q + 1 < kParts * P::kMats) tmem_start16(from + ((q + 1) / kParts) * kN + 16 * ((q + 1) % kParts), v[(q + 1) % 2]);
                } else {
                    tmem_start16(from + m * kN + 16 * c, v[0]);
                    tmem_wait();
                }
                const float(&w)[16] = v[P::kAhead ? q % 2 : 0];
                const float4* g = reinterpret_cast<const float4*>(f + m * kGroup * kN + 16 * c);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 s = g[j];
                    add_scaled(acc[m][8 * c + 2 * j], w[4 * j], w[4 * j + 1], pair8(s.x, s.y));
                    add_scaled(acc[m][8 * c + 2 * j + 1], w[4 * j + 2], w[4 * j + 3], pair8(s.z, s.w));
                }
            }
            tc_fence_before();
            if (lane == 0) mbar_arrive(acc_empty + 8 * u);
            if (i % kGroup == kGroup - 1 && i + 1 < b1 - b0) put(group + 1);
        }
        // The partial sums go over the ring: [kMats][token][feature]. (The last block's MMAs are done, so all copies are.)
        asm volatile("bar.sync 1, %0;" ::"n"(kAdders) : "memory");
        float* part = reinterpret_cast<float*>(at);
        const int feature = 32 * (warp % 4) + lane;
#pragma unroll
        for (int m = 0; m < P::kMats; ++m)
#pragma unroll
            for (int j = 0; j < P::kCols / 2; ++j) {
                float a, b;
                unpair8(acc[m][j], a, b);
                part[(m * kN + set * P::kCols + 2 * j) * kTile + feature] = a;
                part[(m * kN + set * P::kCols + 2 * j + 1) * kTile + feature] = b;
            }
    }
    tc_fence_before();
    if (p.ctas > 1)
        cluster_sync8();
    else
        __syncthreads();

    // Tokens rank, rank + ctas, ... of the tile, one to a warp: a lane has 4 features and adds the ranks' sums in their order.
    const int f0 = ft * kTile + 4 * lane, left = p.a.features - f0;  // features from this lane's first on
    for (int t = rank + p.ctas * warp; t < tokens; t += p.ctas * (P::kThreads / 32)) {
        float s[P::kMats][4];
#pragma unroll
        for (int m = 0; m < P::kMats; ++m) {
            const uint32_t mine = base + static_cast<uint32_t>(((m * kN + t) * kTile + 4 * lane) * 4);
            s[m][0] = s[m][1] = s[m][2] = s[m][3] = 0.f;
            for (int r = 0; r < p.ctas; ++r) {
                const float4 v = ld_cluster_f4(mapa8(mine, static_cast<uint32_t>(r)));
                s[m][0] += v.x;
                s[m][1] += v.y;
                s[m][2] += v.z;
                s[m][3] += v.w;
            }
        }
        const long long row = t0 + t;
        if constexpr (kGated) {
#pragma unroll
            for (int j = 0; j < 4; ++j) s[0][j] = activate8(s[0][j], p.a.act) * s[1][j];
        }
        if (kGated && p.a.out_type == kOutE4m3) {
            float top = 0.f;
            if (left > 0)
#pragma unroll
                for (int j = 0; j < 4; ++j) top = max_nan(top, fabsf(s[0][j]));
#pragma unroll
            for (int o = 16; o; o /= 2) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            top = max_nan(top, kLeastTop8);
            const float up = kTop8 / top;
            if (left > 0)
                *reinterpret_cast<uint32_t*>(static_cast<unsigned char*>(p.a.out) + row * p.a.out_stride + f0) =
                    e4m3x4(s[0][0] * up, s[0][1] * up, s[0][2] * up, s[0][3] * up);
            if (lane == 0) p.a.out_scales[row * blocks8(p.a.features) + ft] = top / kTop8;
        } else if (p.a.out_type == kOutF32) {
            float* o = static_cast<float*>(p.a.out) + row * p.a.out_stride + f0;
            if (left >= 4)
                *reinterpret_cast<float4*>(o) = make_float4(s[0][0], s[0][1], s[0][2], s[0][3]);
            else
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    if (j < left) o[j] = s[0][j];
        } else {
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.a.out) + row * p.a.out_stride + f0;
            const __nv_bfloat162 lo = __floats2bfloat162_rn(s[0][0], s[0][1]), hi = __floats2bfloat162_rn(s[0][2], s[0][3]);
            if (left >= 4) {
                *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            } else {
                if (left > 0) o[0] = __low2bfloat16(lo);
                if (left > 1) o[1] = __high2bfloat16(lo);
                if (left > 2) o[2] = __low2bfloat16(hi);
            }
        }
    }
    if (p.ctas > 1)
        cluster_sync8();  // the other CTAs' sums stay until they have been read
    else
        __syncthreads();
    if (warp == P::kAddWarps + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, P::kColumns);
    }
}

// CTAs of a cluster: as many as let all clusters run at once, at least 2 blocks of k for each. One more and some clusters wait for others to
// end, which costs more than fewer readers do: 20,480 x 5,120 weights (40 tiles) and one token 20.2 us in clusters of 3, 19.7 of 4, 19.4 of
// 5, 25.2 of 7; gate and up of 5,120 x 20,480 (160 tiles) 35.8 us in clusters of 1, 42.3 of 2. `fit`: clusters of each size that run
// at once, as the runtime tells; it counts one CTA an SM for a kernel with tensor memory, though two of the smaller ones share
// one, so that it leaves something over.
int cluster_ctas(long long units, int k_blocks, const std::atomic<int>* fit) {
    int c = 1;
    for (int more = 2; more <= kMostCluster && 2 * more <= k_blocks; ++more)
        if (units <= fit[more].load(std::memory_order_relaxed)) c = more;
    return c;
}

// How a call would run with tiles of kN tokens, and about how long it would take, in ns: the weights' bytes, or the busiest SM's tiles
// with their blocks (kBlockNs each) and their ends (kEndNs: out of registers, joined, written), a launch, and the join of a cluster's
// parts. Measured (us, model in brackets): 128 tokens by 20,480 x 5,120 27.4 (28), by 5,120 x 5,120 11.2 (12), 715 tokens by 320 x
// 19,728 39 (32); gated, 64 tokens by 5,120 x 20,480 50.8 (52), 344 tokens by 176 x 6,720 24.6 (22).
struct RowsPlan {
    long long token_tiles, units;
    int ctas;
    long long ns;
};
template <int kN, bool kGated>
constexpr int kBlockNs = kGated ? (kN == 128 ? 1000 : kN == 64 ? 550 : 250) : (kN == 128 ? 400 : 200);
template <int kN, bool kGated>
constexpr int kEndNs = kGated ? (kN == 128 ? 7500 : kN == 64 ? 3000 : 1500) : (kN == 128 ? 3000 : 1500);

template <int kN, bool kGated, int kPerSm>
struct Rows {
    using P = Plan<kN, kGated, kPerSm>;

    // Clusters of each size that run at once, found once per device; null if that failed.
    static const std::atomic<int>* fit() {
        static std::atomic<bool> ready[kMul8Devices];
        static std::atomic<int> fits[kMul8Devices][kMostCluster + 1];
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMul8Devices) return nullptr;
        if (!ready[dev].load(std::memory_order_acquire)) {
            const auto kernel = &mul8_rows_kernel<kN, kGated, kPerSm>;
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kSmem) != cudaSuccess) return nullptr;
            for (int c = 2; c <= kMostCluster; ++c) {
                const int n = mul8_clusters(reinterpret_cast<const void*>(kernel), c, P::kThreads, P::kSmem);
                if (n < 0) return nullptr;
                fits[dev][c].store(n, std::memory_order_relaxed);
            }
            ready[dev].store(true, std::memory_order_release);
        }
        return fits[dev];
    }

    static bool plan(const Mul8Args& a, int sms, RowsPlan* r) {
        const std::atomic<int>* f = fit();
        if (!f) return false;
        const int k_blocks = blocks8(a.k);
        r->token_tiles = (a.n + kN - 1) / kN;
        r->units = r->token_tiles * blocks8(a.features);
        r->ctas = cluster_ctas(r->units, k_blocks, f);
        const long long turns = (r->units * r->ctas + sms - 1) / sms, end = kEndNs<kN, kGated>;
        const long long bytes_ns = static_cast<long long>(P::kMats) * a.features * a.k / 6200 + end;
        const long long tiles_ns = turns * ((k_blocks + r->ctas - 1) / r->ctas * kBlockNs<kN, kGated> + end);
        r->ns = 2500 + (bytes_ns > tiles_ns ? bytes_ns : tiles_ns) + (r->ctas > 1 ? 7 * kN * P::kMats : 0);
        return true;
    }

    static int run(const Mul8Args& a, const RowsPlan& r, cudaStream_t stream) {
        if (r.units * r.ctas > 0x7FFFFFFFLL) return -7;
        Params p;
        p.a = a;
        p.k_blocks = blocks8(a.k);
        p.token_tiles = static_cast<int>(r.token_tiles);
        p.ctas = r.ctas;
        CUtensorMap tm_x, tm_w, tm_up;
        if (!mul8_map(&tm_x, a.x, a.k, a.n, a.x_stride, kN) || !mul8_map(&tm_w, a.w, a.k, a.features, a.w_stride, kTile)) return -7;
        tm_up = tm_w;
        if (kGated && !mul8_map(&tm_up, a.up, a.k, a.features, a.w_stride, kTile)) return -7;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(r.units * r.ctas));
        cfg.blockDim = dim3(P::kThreads);
        cfg.dynamicSmemBytes = P::kSmem;
        cfg.stream = stream;
        cudaLaunchAttribute attrs[2];
        attrs[0].id = cudaLaunchAttributeClusterDimension;
        attrs[0].val.clusterDim.x = static_cast<unsigned>(r.ctas);
        attrs[0].val.clusterDim.y = attrs[0].val.clusterDim.z = 1;
        cfg.attrs = attrs;
        cfg.numAttrs = 1 + static_cast<unsigned>(programmatic_launch(r.ns, true, stream, attrs + 1));
        g_launched.store(true, std::memory_order_relaxed);
        return cudaLaunchKernelEx(&cfg, &mul8_rows_kernel<kN, kGated, kPerSm>, tm_x, tm_w, tm_up, p) == cudaSuccess ? 0 : -7;
    }

    // The shorter of this and the pairs' kernel.
    static int choose(const Mul8Args& a, int sms, cudaStream_t stream) {
        RowsPlan r;
        if (!plan(a, sms, &r)) return -7;
        if (a.n > 32) {
            const long long pairs = mul8_tiles_ns(a);
            if (mul8_by_pairs(pairs, r.ns)) return launch_mul8_tiles(a, stream);
            if (pairs < 0) cudaGetLastError();  // (what refused the plan is not this call's error)
        }
        return run(a, r, stream);
    }
};

}  // namespace

PFN_cuTensorMapEncodeTiled_v12000 mul8_encode() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, []() {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

bool mul8_map(CUtensorMap* m, const void* base, long long cols, long long rows, long long stride, int box_rows) {
    const auto fn = mul8_encode();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)}, strides[1] = {static_cast<cuuint64_t>(stride)};
    const cuuint32_t box[2] = {kBlock8, static_cast<cuuint32_t>(box_rows)}, ones[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int mul8_clusters(const void* kernel, int ctas, int threads, int smem) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(ctas);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n : -1;
}

int launch_mul8(const Mul8Args& a, cudaStream_t stream) {
    const int sms = attn_sm_count();
    if (sms < 1) return -7;
    if (a.up) {
        if (a.n <= 16) return Rows<16, true, 2>::choose(a, sms, stream);
        if (a.n <= 32) return Rows<32, true, 2>::choose(a, sms, stream);
        if (a.n <= 64) return Rows<64, true, 2>::choose(a, sms, stream);
        return Rows<128, true, 1>::choose(a, sms, stream);
    }
    if (a.n <= 16) return Rows<16, false, 2>::choose(a, sms, stream);
    if (a.n <= 32) return Rows<32, false, 2>::choose(a, sms, stream);
    if (a.n <= 64) return Rows<64, false, 2>::choose(a, sms, stream);
    return Rows<128, false, 1>::choose(a, sms, stream);
}

int read_mul8_error(unsigned int* word, int clear, cudaStream_t stream) {
    unsigned int v = 0;
    if (read_mul8_tiles_error(word, clear, stream) != 0) return -7;
    if (!g_launched.load(std::memory_order_relaxed)) return 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_hc_mul8_error, sizeof(v), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return -7;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return -7;
    *word |= v;
    if (clear && v != 0) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbolAsync(g_hc_mul8_error, &z, sizeof(z), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess) return -7;
        if (cudaStreamSynchronize(stream) != cudaSuccess) return -7;
    }
    return 0;
}

}  // namespace hc
