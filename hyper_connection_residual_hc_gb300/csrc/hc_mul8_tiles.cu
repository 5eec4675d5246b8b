// Products of 8-bit rows with 8-bit weights for many rows (formulas and format: include/hc.h; few rows: hc_mul8.cu).
//
// A pair of CTAs (a cluster of 2) takes 256 tokens by 256 rows of weights with tcgen05.mma of cta_group::2: each CTA holds its 128
// tokens and half of the weights in shared memory and the sums of its tokens, 128 lanes by 256 columns, in tensor memory. The 256
// rows of weights are 256 features of a plain product, or 128 of the gate and 128 of the up projection.
//
// Scales are any fp32 numbers, one for each 128 values of k, so a block's sums (4 instructions of K = 32) leave tensor memory and
// are added up in registers: acc += (token's scale * weights' scale) * sums. A token is a lane, so the factor is one number a
// thread. The columns go in two halves of 128, each with two buffers in tensor memory and four adding warps of its own: while one
// half is added up the other is multiplied, and the next block's MMAs run under this one's additions. (One MMA of 256 columns a step, both
// halves released together: 67 us where halves take 54, though a step of 128 columns reads the tokens' tile again.)
//
// Measured: 16,384 tokens by 20,480 x 5,120 1,040 us in a graph, 3,300 TFLOP/s, 1,220 us when the card is at its power limit; cuBLAS'
// product with one scale a tensor takes 981. A block of k takes about 590 cycles of the 512 that its MMAs need. What it was before: 1.3
// us a block with a release at cluster scope at each arrival (a fence of all memory), 0.42 with scales loaded by the adding warps (a
// register that is copied waits for its load) and 0.31 now; an accumulator that crosses more than one loop body is copied about by
// the compiler, twice as slow. 256 tokens by 20,480 x 5,120 29 us, gated by 5,120 x 20,480 54; 4,099 gated tokens 566 us, 3,040
// TFLOP/s, of which a tile's end (activation and stores, 2 us of 15) is the part that no MMA runs under.
//
// Warps: 8 add up (4 for each half of the columns; a gated product's two halves are columns 0..63 and 64..127 of gate and up, so that a
// thread has both), 1 issues TMA loads, 1 (of the first CTA) the MMAs. Registers move from the last 4 warps to the first 8.
// Results leave through shared memory by TMA stores, 64 bytes of 32 rows at a time, which also cut off rows and columns
// outside the output.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <initializer_list>

#include "hc_ffn.h"
#include "hc_mul8_dev.cuh"
#include "hc_mul8_host.h"

namespace hc {
namespace {

__device__ unsigned int g_hc_mul8_tiles_error = 0;
std::atomic<bool> g_launched{false};

constexpr int kTokens = 256;                     // of a pair
constexpr int kRowsW = 256;                      // rows of weights of a pair
constexpr int kHalf = 128;
constexpr int kStages = 5;
constexpr int kOperand = kHalf * kBlock8;        // bytes: 128 rows of one operand
constexpr int kStage = 2 * kOperand;
constexpr int kAddWarps = 8, kLoadWarp = 8, kMmaWarp = 9, kScaleWarps = 2;  // in this order
constexpr int kThreads = 384;
constexpr int kOutWarp = 4096;                   // two buffers of 32 rows of 64 bytes
constexpr int kOut = kStages * kStage;
constexpr int kBatch = 8;                        // blocks of k whose scales are handed over together
constexpr int kScales = kOut + kAddWarps * kOutWarp;  // [2][kBatch][2][128] factors
constexpr int kTops = kScales + 2 * kBatch * 2 * kHalf * 4;  // [2][kAddWarps][32] largest magnitudes
constexpr int kBars = kTops + 2 * kAddWarps * 32 * 4;
constexpr int kSmem = kBars + 256 + 1024;        // + alignment
static_assert(kSmem <= 227 * 1024, "fits");
constexpr int kMostPairs = 4;                    // that share a tile
constexpr int kBand = 8;                         // token tiles that go through the weights together

struct Params {
    Mul8Args a;
    int k_blocks, token_tiles, feature_tiles;
    int pairs;   // of the grid, which take tiles in turn; with kSplit the pairs of a cluster, which share one tile's blocks of k
    int stored;  // features that TMA stores: whole 16 bytes of a row
    long long first, until;  // tiles
};

__device__ __forceinline__ void tmem_alloc2(uint32_t dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish2() { asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void mma8_pair(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
// Arrives on the barrier at this offset in both CTAs of the pair (`both`: their bits).
__device__ __forceinline__ void commit8_pair(uint32_t lead, uint32_t bar, uint16_t both) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n\t}" ::"r"(bar),
        "r"(lead), "h"(both)
        : "memory");
}
// Into this CTA's shared memory, completing on a barrier of either CTA (`bar`: an address in the cluster's window).
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
// One lane's arrival without a branch around it, in this CTA.
__device__ __forceinline__ void arrive_if(uint32_t bar, bool lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"(static_cast<uint32_t>(lead))
        : "memory");
}
// Without release: what the arrival stands for is tensor memory reads, which tcgen05.fence orders; a release at cluster scope would
// wait for all of the thread's memory operations.
__device__ __forceinline__ void arrive_cluster(uint32_t bar, bool lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"(static_cast<uint32_t>(lead))
        : "memory");
}
// 64 consecutive columns of this thread's lane (see tmem_start16).
__device__ __forceinline__ void tmem_start64(uint32_t addr, float (&v)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]),
          "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]),
          "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]),
          "=f"(v[48]), "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]),
          "=f"(v[56]), "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
}

struct Tile {
    int tokens, features;  // tile numbers
};
// Bands of kBand token tiles; within a band the token tiles of one feature tile come first, so that what runs at the same time
// shares both operands in L2.
__device__ __forceinline__ Tile tile_at(const Params& p, long long i) {
    const long long band = i / (static_cast<long long>(kBand) * p.feature_tiles);
    const int first = static_cast<int>(band) * kBand, rows = min(kBand, p.token_tiles - first);
    const int r = static_cast<int>(i - band * kBand * p.feature_tiles);
    return {first + r % rows, r / rows};
}

__device__ __forceinline__ float ld_cluster_f1(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// With kSplit, by the adding warps of all pairs of the cluster: their sums of a tile are added up in the order of the pairs. Each
// thread puts its columns into shared memory, over the ring (the last block's MMAs of both halves are done, so all copies are), 4 at a time:
// [column / 4][token][4]. Then the columns are dealt out 16 at a time: a pair takes every p.pairs-th of each half (of a gated
// product 16 features with their 16 columns of up), reads them from all pairs and writes the result.
template <bool kGated>
__device__ __forceinline__ void join_parts(const Params& p, const Tile& t, const uint64_t (&acc)[64], uint32_t base, unsigned char* at, int half, int in_cta,
                                           int rank, int pair) {
    float4* part = reinterpret_cast<float4*>(at) + half * kHalf * kHalf / 4 + in_cta;
    static_assert(2 * kHalf * kHalf * 4 + 2 * kHalf * 4 <= kStages * kStage, "the sums and the largest magnitudes take the ring's place");
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        float4 v;
        unpair8(acc[2 * j], v.x, v.y);
        unpair8(acc[2 * j + 1], v.z, v.w);
        part[j * kHalf] = v;
    }
    cluster_sync8();
    const long long row = static_cast<long long>(t.tokens) * kTokens + rank * kHalf + in_cta;
    const bool has = row < p.a.n;
    // the sums of columns c .. c + 15 of this half
    auto columns = [&](int c, float (&s)[16]) {
        const uint32_t mine = base + static_cast<uint32_t>(((half * kHalf + c) / 4 * kHalf + in_cta) * 16);
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = 0.f;
        float4 v[kMostPairs][4];  // all loads at once: one by one they took as long as 10 blocks
#pragma unroll
        for (int r = 0; r < kMostPairs; ++r) {
            if (r >= p.pairs) break;
            const uint32_t from = mapa8(mine, static_cast<uint32_t>(2 * r + rank));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (r == pair)
                    v[r][e] = *reinterpret_cast<const float4*>(at + (mine - base) + e * kHalf * 16);
                else
                    v[r][e] = ld_cluster_f4(from + static_cast<uint32_t>(e * kHalf * 16));
            }
        }
#pragma unroll
        for (int r = 0; r < kMostPairs; ++r) {
            if (r >= p.pairs) break;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[4 * e] += v[r][e].x;
                s[4 * e + 1] += v[r][e].y;
                s[4 * e + 2] += v[r][e].z;
                s[4 * e + 3] += v[r][e].w;
            }
        }
    };
    if constexpr (kGated) {
        float h[4][16];
        float top = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (c % p.pairs != pair) continue;
            float g[16], u[16];
            columns(16 * c, g);
            columns(64 + 16 * c, u);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                h[c][e] = activate8(g[e], p.a.act) * u[e];
                top = max_nan(top, fabsf(h[c][e]));  // (features past the last are 0)
            }
        }
        const bool codes = p.a.out_type == kOutE4m3;
        float up = 1.f;
        if (codes) {  // the token's largest of all 128 features
            const uint32_t tops = 2 * kHalf * kHalf * 4;
            *reinterpret_cast<float*>(at + tops + (half * kHalf + in_cta) * 4) = top;
            cluster_sync8();
            top = kLeastTop8;
            for (int r = 0; r < p.pairs; ++r)
#pragma unroll
                for (int g = 0; g < 2; ++g) top = max_nan(top, ld_cluster_f1(mapa8(base + tops + static_cast<uint32_t>((g * kHalf + in_cta) * 4), static_cast<uint32_t>(2 * r + rank))));
            up = kTop8 / top;
            if (pair == 0 && half == 0 && has) p.a.out_scales[row * p.feature_tiles + t.features] = top / kTop8;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int f = t.features * kHalf + 64 * half + 16 * c;
            if (c % p.pairs != pair || f >= p.a.features || !has) continue;
            if (codes) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = e4m3x4(h[c][4 * e] * up, h[c][4 * e + 1] * up, h[c][4 * e + 2] * up, h[c][4 * e + 3] * up);
                *reinterpret_cast<uint4*>(static_cast<unsigned char*>(p.a.out) + row * p.a.out_stride + f) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = bf16x2(h[c][2 * e], h[c][2 * e + 1]);
                uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.out) + row * p.a.out_stride + f);
                o[0] = make_uint4(w[0], w[1], w[2], w[3]);
                o[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
        }
    } else {
        for (int c = pair; c < 8; c += p.pairs) {
            const int f = t.features * kRowsW + kHalf * half + 16 * c, left = p.a.features - f;
            if (left <= 0) break;
            float s[16];
            columns(16 * c, s);
            if (!has) continue;
            const long long o = row * p.a.out_stride + f;
            if (p.a.out_type == kOutF32) {
                float* to = static_cast<float*>(p.a.out) + o;
                if (left >= 16) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) reinterpret_cast<float4*>(to)[e] = make_float4(s[4 * e], s[4 * e + 1], s[4 * e + 2], s[4 * e + 3]);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (e < left) to[e] = s[e];
                }
            } else {
                __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.a.out) + o;
                if (left >= 16) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        reinterpret_cast<uint4*>(to)[e] = make_uint4(bf16x2(s[8 * e], s[8 * e + 1]), bf16x2(s[8 * e + 2], s[8 * e + 3]),
                                                                     bf16x2(s[8 * e + 4], s[8 * e + 5]), bf16x2(s[8 * e + 6], s[8 * e + 7]));
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (e < left) to[e] = __float2bfloat16_rn(s[e]);
                }
            }
        }
    }
}

template <bool kGated, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
mul8_tiles_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_up,
                  const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ Params p) {
    extern __shared__ unsigned char raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    unsigned char* at = raw + (base - smem_u32(raw));
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t full = base + kBars, empty = full + 8 * kStages, acc_full = empty + 8 * kStages, acc_empty = acc_full + 32, sc_full = acc_empty + 32, sc_empty = sc_full + 16, slot = sc_empty + 16;
    volatile uint32_t* abort_word = reinterpret_cast<volatile uint32_t*>(at + (slot + 4 - base));
    const Wait8 wait{abort_word, &g_hc_mul8_tiles_error};
    const uint32_t in_cluster = cluster_ctarank8(), rank = in_cluster & 1, leader = in_cluster & ~1u;
    const int pair = kSplit ? static_cast<int>(in_cluster) / 2 : 0;  // of those that share a tile
    // tiles n0, n0 + step, ...; blocks k0 .. k1 - 1 of each
    const long long n0 = p.first + (kSplit ? blockIdx.x / (2 * p.pairs) : blockIdx.x / 2), step = kSplit ? p.until : p.pairs;
    const int k0 = kSplit ? p.k_blocks * pair / p.pairs : 0, k1 = kSplit ? p.k_blocks * (pair + 1) / p.pairs : p.k_blocks;

    if (warp == kLoadWarp && lane == 0) {
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(kGated && rank ? &tm_up : &tm_w);
    }
    if (warp == kMmaWarp) {
        tmem_alloc2(slot, 512);
        tmem_relinquish2();
    }
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, kAddWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sc_full + 8 * i, kScaleWarps);
            mbar_init(sc_empty + 8 * i, kAddWarps);
        }
        *abort_word = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    cluster_sync8();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(at + (slot - base));
    // What the kernels ahead write and read. (A call's second launch could take its tiles beside the first's last ones, 1 to 3% sooner, but
    // that what the kernels before the first wrote is visible to it is only promised behind a wait of its own.)
    griddep_wait();
    griddep_launch_dependents();

    if (warp >= kAddWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == kLoadWarp && lane == 0) {  // ---- loads
            const uint32_t first_full = mapa8(full, leader);
            int i = 0;  // blocks so far
            for (long long n = n0; n < p.until; n += step) {
                const Tile t = tile_at(p, n);
                const int token = t.tokens * kTokens + static_cast<int>(rank) * kHalf;
                const int row = kGated ? t.features * kHalf : t.features * kRowsW + static_cast<int>(rank) * 64, next = kGated ? 64 : kHalf;
                const CUtensorMap* w = kGated && rank ? &tm_up : &tm_w;
                for (int b = k0; b < k1; ++b, ++i) {
                    const int s = i % kStages;
                    if (i >= kStages) wait(empty + 8 * s, (i / kStages - 1) & 1);
                    if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, 2 * kStage);
                    const uint32_t st = base + s * kStage;
                    tma_load_pair(st, &tm_x, first_full + 8 * s, b * kBlock8, token);
                    tma_load_pair(st + kOperand, w, first_full + 8 * s, b * kBlock8, row);
                    tma_load_pair(st + kOperand + kOperand / 2, w, first_full + 8 * s, b * kBlock8, row + next);
                }
            }
            // No copy of either CTA is in flight when the pair ends, whatever happened, and no arrival of a commit, which come to both CTAs by
            // themselves: nothing else waits for the last ones on `empty`.
            if (rank == 0)
                for (int j = max(i - kStages, 0); j < i; ++j) wait.drain(full + 8 * (j % kStages), (j / kStages) & 1);
            for (int j = max(i - kStages, 0); j < i; ++j) wait.drain(empty + 8 * (j % kStages), (j / kStages) & 1);
            for (int j = max(i - 2, 0); j < i; ++j)
                for (int h = 0; h < 2; ++h) wait.drain(acc_full + 16 * (j & 1) + 8 * h, (j / 2) & 1);
        } else if (warp == kMmaWarp && rank == 0) {  // ---- MMAs
            const uint32_t lead = elect_one();
            const uint16_t both = static_cast<uint16_t>(3u << leader);
            constexpr uint32_t idesc = idesc8(256, 128);
            int i = 0;
            for (long long n = n0; n < p.until; n += step) {
                for (int b = k0; b < k1; ++b, ++i) {
                    const int s = i % kStages, u = i & 1;
                    wait(full + 8 * s, (i / kStages) & 1);
                    const uint32_t st = base + s * kStage;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (i >= 2) wait(acc_empty + 16 * u + 8 * h, (i / 2 - 1) & 1);
                        tc_fence_after();
                        const uint32_t d = tmem + u * 256 + h * 128;
                        const uint64_t x = sdesc8(st), w = sdesc8(st + kOperand + h * (kOperand / 2));
#pragma unroll
                        for (int q = 0; q < 4; ++q) mma8_pair(lead, d, x + 2 * q, w + 2 * q, idesc, q > 0);
                        commit8_pair(lead, acc_full + 16 * u + 8 * h, both);
                    }
                    commit8_pair(lead, empty + 8 * s, both);
                }
            }
            if (i > 0) wait.drain(acc_full + 16 * ((i - 1) & 1) + 8, ((i - 1) / 2) & 1);
        } else if (warp > kMmaWarp) {  // ---- scales
            // The factors of the CTA's 128 tokens, 2 to a lane, with the weights of either half of the columns (gate and up). Tokens and
            // features outside the matrices take the last ones inside (their sums are not stored).
            int batch = 0;
            for (long long n = n0; n < p.until; n += step) {
                const Tile t = tile_at(p, n);
                const int in_cta = 64 * (warp - kMmaWarp - 1) + lane;
                const long long token = static_cast<long long>(t.tokens) * kTokens + rank * kHalf + in_cta;
                const float* x0 = p.a.x_scales + min(token, p.a.n - 1) * p.k_blocks;
                const float* x1 = p.a.x_scales + min(token + 32, p.a.n - 1) * p.k_blocks;
                const int most = blocks8(p.a.features) - 1;
                const float* w0 = p.a.w_scales + static_cast<long long>(min(kGated ? t.features : 2 * t.features, most)) * p.k_blocks;
                const float* w1 = kGated ? p.a.up_scales + static_cast<long long>(t.features) * p.k_blocks
                                         : p.a.w_scales + static_cast<long long>(min(2 * t.features + 1, most)) * p.k_blocks;
                for (int b = k0; b < k1; b += kBatch, ++batch) {
                    if (batch >= 2) wait(sc_empty + 8 * (batch & 1), (batch / 2 - 1) & 1);
                    float* o = reinterpret_cast<float*>(at + kScales) + (batch & 1) * kBatch * 2 * kHalf + in_cta;
                    float x[2][kBatch], w[2][kBatch];  // (all loads at once: the first ones are waited for)
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        const int from = min(b + j, k1 - 1);
                        x[0][j] = __ldg(x0 + from);
                        x[1][j] = __ldg(x1 + from);
                        w[0][j] = __ldg(w0 + from);
                        w[1][j] = __ldg(w1 + from);
                    }
#pragma unroll
                    for (int j = 0; j < kBatch; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) o[(j * 2 + r / 2) * kHalf + r % 2 * 32] = x[r % 2][j] * w[r / 2][j];
                    __syncwarp();
                    arrive_if(sc_full + 8 * (batch & 1), lane == 0);
                }
            }
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int half = warp / 4, quarter = warp % 4;
        const int in_cta = 32 * quarter + lane;  // token
        const uint32_t mine = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
        const uint32_t released = mapa8(acc_empty, leader);
        const uint32_t out_smem = base + kOut + warp * kOutWarp;
        const float* factors = reinterpret_cast<const float*>(at + kScales) + (kGated ? 0 : half * kHalf) + in_cta;
        int i = 0, batch = 0, turn = 0, stores = 0;
        for (long long n = n0; n < p.until; n += step, ++turn) {
            uint64_t acc[64];  // pairs of columns: 128 features, or 64 of the gate and 64 of up
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[j] = 0;
#pragma unroll 1
            for (int b = k0; b < k1; b += kBatch, ++batch) {
                wait(sc_full + 8 * (batch & 1), (batch / 2) & 1);
                const float* g = factors + (batch & 1) * kBatch * 2 * kHalf;
                const int until = i + min(kBatch, k1 - b);
#pragma unroll 1
                for (; i < until; ++i, g += 2 * kHalf) {
                    const float factor[2] = {g[0], kGated ? g[kHalf] : g[0]};
                    const int u = i & 1;
                    wait(acc_full + 16 * u + 8 * half, (i / 2) & 1);
                    tc_fence_after();
                    const uint32_t from = mine + u * 256 + half * 128;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float v[64];
                        tmem_start64(from + q * 64, v);
                        tmem_wait();
                        if (q == 1) {
                            tc_fence_before();
                            arrive_cluster(released + 16 * u + 8 * half, lane == 0);
                        }
                        const uint64_t f = pair8(factor[q], factor[q]);
#pragma unroll
                        for (int e = 0; e < 32; ++e) add_scaled(acc[32 * q + e], v[2 * e], v[2 * e + 1], f);
                    }
                }
                __syncwarp();
                arrive_if(sc_empty + 8 * (batch & 1), lane == 0);
            }
            const Tile t = tile_at(p, n);
            const int token0 = t.tokens * kTokens + static_cast<int>(rank) * kHalf + 32 * quarter;  // of the warp
            if constexpr (kSplit) {
                // The ring is free when the other half's last MMAs have read it too.
                wait(acc_full + 16 * ((i - 1) & 1) + 8 * (1 - half), ((i - 1) / 2) & 1);
                join_parts<kGated>(p, t, acc, base, at, half, in_cta, static_cast<int>(rank), pair);
                break;
            }
            // Stages 64 bytes of each of the warp's 32 rows (a lane's words w, 16 bytes at a time, swizzled as the map says) and stores them
            // at column x, in one of two buffers by turns: the store before this one is read out meanwhile.
            auto store = [&](const uint32_t (&w)[16], int x) {
                const uint32_t to = out_smem + (stores++ & 1) * (kOutWarp / 2) + static_cast<uint32_t>(lane * 64);
                const int mask = (lane >> 1) & 3;
                if (lane == 0) bulk_wait_read<1>();
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 4; ++c) st_smem_v4(to + (c ^ mask) * 16, make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (token0 < p.a.n && x < p.stored) tma_store_2d(&tm_out, to, x, token0);
                    bulk_commit();
                }
                if constexpr (!kGated) {
                    // A TMA store writes whole 16 bytes; the features past the last of those go one by one.
                    const int size = p.a.out_type == kOutF32 ? 4 : 2, rest = p.a.features - p.stored, off = (p.stored - x) * size;
                    if (rest > 0 && off >= 0 && off < 64 && token0 + lane < p.a.n) {
                        const uint4 q = ld_smem_v4(to + ((off / 16) ^ mask) * 16);
                        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
                        const long long o = (static_cast<long long>(token0) + lane) * p.a.out_stride + p.stored;
#pragma unroll
                        for (int e = 0; e < 7; ++e) {
                            if (e >= rest) break;
                            if (size == 4)
                                static_cast<uint32_t*>(p.a.out)[o + e] = u[e % 4];
                            else
                                static_cast<uint16_t*>(p.a.out)[o + e] = static_cast<uint16_t>(u[e / 2] >> (e % 2 * 16));
                        }
                    }
                }
            };
            if constexpr (kGated) {
                float h[64];
                auto gate = [&](int act) {  // (an activation known at compile time: 2,000 tokens by 1,024 x 8,192 47.5 -> 44 us)
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float g0, g1, u0, u1;
                        unpair8(acc[e], g0, g1);
                        unpair8(acc[32 + e], u0, u1);
                        h[2 * e] = activate8(g0, act) * u0;
                        h[2 * e + 1] = activate8(g1, act) * u1;
                    }
                };
                if (p.a.act == kActGelu)
                    gate(kActGelu);
                else
                    gate(kActSilu);
                const int x = t.features * kHalf + 64 * half;
                if (p.a.out_type == kOutE4m3) {
                    float top = 0.f;
#pragma unroll
                    for (int e = 0; e < 64; ++e) top = max_nan(top, fabsf(h[e]));  // (features past the last are 0)
                    // the other 64 features' is with the warp of the other half
                    float* tops = reinterpret_cast<float*>(at + kTops) + (turn & 1) * 32 * kAddWarps + lane;
                    tops[warp * 32] = top;
                    asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
                    top = max_nan(max_nan(top, tops[(warp ^ 4) * 32]), kLeastTop8);
                    const float up = kTop8 / top;
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = e4m3x4(h[4 * e] * up, h[4 * e + 1] * up, h[4 * e + 2] * up, h[4 * e + 3] * up);
                    store(w, x);
                    const long long row = static_cast<long long>(token0) + lane;
                    if (half == 0 && row < p.a.n) p.a.out_scales[row * p.feature_tiles + t.features] = top / kTop8;
                } else {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = bf16x2(h[32 * c + 2 * e], h[32 * c + 2 * e + 1]);
                        store(w, x + 32 * c);
                    }
                }
            } else {
                const int x = t.features * kRowsW + kHalf * half;
                if (p.a.out_type == kOutF32) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float a, b;
                            unpair8(acc[8 * c + e], a, b);
                            w[2 * e] = __float_as_uint(a);
                            w[2 * e + 1] = __float_as_uint(b);
                        }
                        store(w, x + 16 * c);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float a, b;
                            unpair8(acc[16 * c + e], a, b);
                            w[e] = bf16x2(a, b);
                        }
                        store(w, x + 32 * c);
                    }
                }
            }
        }
        if constexpr (!kSplit) {
            if (lane == 0) bulk_wait<0>();
            __syncwarp();
        }
    }
    if (kSplit && warp >= kAddWarps) {  // (the other warps' barriers are in join_parts)
        cluster_sync8();
        if (kGated && p.a.out_type == kOutE4m3) cluster_sync8();
    }
    tc_fence_before();
    cluster_sync8();  // nothing of this pair is in flight any more
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc2(tmem, 512);
    }
}

bool out_map(CUtensorMap* m, const Mul8Args& a, int stored) {
    const auto fn = mul8_encode();
    if (!fn) return false;
    const int size = a.out_type == kOutF32 ? 4 : a.out_type == kOutE4m3 ? 1 : 2;
    const CUtensorMapDataType type = a.out_type == kOutF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : a.out_type == kOutE4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(stored > 0 ? stored : 8), static_cast<cuuint64_t>(a.n)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.out_stride) * static_cast<cuuint64_t>(size)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(64 / size), 32}, ones[2] = {1, 1};
    return fn(m, type, 2, a.out, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How the tiles go to pairs: as many as fill all pairs a whole number of times are taken whole, and so are the others unless sharing
// each of them between the pairs of a cluster is shorter (they are few then: the clusters run at once). In blocks of k: a tile's
// start and end cost about as much as kEnds, joining kJoin more, another launch kLaunch. `fit`: clusters of 1 to 4 pairs that run at once.
constexpr int kEnds = 6, kJoin = 11, kLaunch = 20;
struct Schedule {
    long long whole;  // tiles
    int split;        // pairs that share each of the others; 1: none are left
};
Schedule schedule(long long tiles, int k_blocks, const std::atomic<int>* fit) {
    const int pairs = fit[1].load(std::memory_order_relaxed);
    const long long whole = tiles / pairs * pairs, rest = tiles - whole;
    Schedule best = {tiles, 1};
    int least = k_blocks + kEnds;  // of another turn
    for (int s = 2; s <= kMostPairs && 2 * s <= k_blocks && rest > 0; ++s) {
        const int cost = (k_blocks + s - 1) / s + kEnds + kJoin + (whole > 0 ? kLaunch : 0);
        if (rest <= fit[s].load(std::memory_order_relaxed) && cost < least) {
            least = cost;
            best = {whole, s};
        }
    }
    return best;
}

struct Maps {
    CUtensorMap x, w, up, out;
};

template <bool kGated, bool kSplit>
cudaError_t start(const Maps& m, const Params& p, unsigned ctas, int cluster, long long ns, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeClusterDimension;
    attrs[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attrs[0].val.clusterDim.y = attrs[0].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 1 + static_cast<unsigned>(programmatic_launch(ns, true, stream, attrs + 1));
    return cudaLaunchKernelEx(&cfg, &mul8_tiles_kernel<kGated, kSplit>, m.x, m.w, m.up, m.out, p);
}

// Clusters of 1 to kMostPairs pairs that run at once, found once per device; null if that failed.
template <bool kGated>
const std::atomic<int>* fits() {
    static std::atomic<bool> ready[kMul8Devices];
    static std::atomic<int> fit[kMul8Devices][kMostPairs + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMul8Devices) return nullptr;
    if (!ready[dev].load(std::memory_order_acquire)) {
        const void* const whole = reinterpret_cast<const void*>(&mul8_tiles_kernel<kGated, false>);
        const void* const shared = reinterpret_cast<const void*>(&mul8_tiles_kernel<kGated, true>);
        for (const void* k : {whole, shared})
            if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) return nullptr;
        for (int c = 1; c <= kMostPairs; ++c) {
            const int n = mul8_clusters(c == 1 ? whole : shared, 2 * c, kThreads, kSmem);
            if (n < (c == 1 ? 1 : 0)) return nullptr;
            fit[dev][c].store(n, std::memory_order_relaxed);
        }
        ready[dev].store(true, std::memory_order_release);
    }
    return fit[dev];
}

struct Shape {
    int token_tiles, feature_tiles;
    long long tiles;
};
Shape shape_of(const Mul8Args& a) {
    Shape s;
    const int wide = a.up ? kHalf : kRowsW;
    s.token_tiles = static_cast<int>((a.n + kTokens - 1) / kTokens);
    s.feature_tiles = (a.features + wide - 1) / wide;
    s.tiles = static_cast<long long>(s.token_tiles) * s.feature_tiles;
    return s;
}

template <bool kGated>
int start(const Mul8Args& a, cudaStream_t stream) {
    const std::atomic<int>* fit = fits<kGated>();
    if (!fit) return -7;
    Params p;
    p.a = a;
    p.k_blocks = blocks8(a.k);
    const Shape shape = shape_of(a);
    p.token_tiles = shape.token_tiles;
    p.feature_tiles = shape.feature_tiles;
    const int unit = a.out_type == kOutF32 ? 4 : a.out_type == kOutE4m3 ? 16 : 8;
    p.stored = a.features / unit * unit;
    Maps m;
    if (!mul8_map(&m.x, a.x, a.k, a.n, a.x_stride, kHalf) || !mul8_map(&m.w, a.w, a.k, a.features, a.w_stride, kHalf / 2) || !out_map(&m.out, a, p.stored))
        return -7;
    m.up = m.w;
    if (kGated && !mul8_map(&m.up, a.up, a.k, a.features, a.w_stride, kHalf / 2)) return -7;
    const long long tiles = shape.tiles;
    const Schedule plan = schedule(tiles, p.k_blocks, fit);
    const long long ns = mul8_tiles_ns(a);
    g_launched.store(true, std::memory_order_relaxed);
    if (plan.whole > 0) {
        p.first = 0;
        p.until = plan.whole;
        const long long pairs = fit[1].load(std::memory_order_relaxed);
        p.pairs = static_cast<int>(plan.whole < pairs ? plan.whole : pairs);
        if (start<kGated, false>(m, p, static_cast<unsigned>(2 * p.pairs), 2, ns, stream) != cudaSuccess) return -7;
    }
    if (plan.whole < tiles) {
        p.first = plan.whole;
        p.until = tiles;
        p.pairs = plan.split;
        if (start<kGated, true>(m, p, static_cast<unsigned>((tiles - plan.whole) * 2 * plan.split), 2 * plan.split, ns, stream) != cudaSuccess) return -7;
    }
    return 0;
}

}  // namespace

// In blocks of kBlockNs; with one token tile what runs at once reads weights of its own, and the more of it the longer a block takes.
// Measured (us, model in brackets): 256 tokens by 20,480 x 5,120 30.8 (29), by 5,120 x 5,120 14.8 (14), 715 tokens by 320 x 19,728 14.4
// (15), 4,096 tokens by 20,480 x 5,120 280 (263); gated, 256 tokens by 5,120 x 20,480 55 (62), 128 tokens by 1,024 x 512 8.1 (8).
long long mul8_tiles_ns(const Mul8Args& a) {
    constexpr long long kBlockNs = 300, kStartNs = 5500;
    const std::atomic<int>* fit = a.up ? fits<true>() : fits<false>();
    if (!fit) return -1;
    const Shape shape = shape_of(a);
    const int k_blocks = blocks8(a.k);
    const Schedule plan = schedule(shape.tiles, k_blocks, fit);
    const long long pairs = fit[1].load(std::memory_order_relaxed), at_once = plan.split > 1 && plan.whole == 0 ? shape.tiles * plan.split : shape.tiles < pairs ? shape.tiles : pairs;
    const long long block = kBlockNs + (shape.token_tiles == 1 ? at_once * 6 / 5 : 0);
    const long long turns = (plan.whole + pairs - 1) / pairs;
    long long ns = kStartNs + turns * k_blocks * block + (turns > 1 ? turns - 1 : 0) * kEnds * kBlockNs;
    if (plan.whole < shape.tiles) ns += (k_blocks + plan.split - 1) / plan.split * block + kJoin * kBlockNs + (plan.whole > 0 ? kLaunch * kBlockNs : 0);
    return ns;
}

int launch_mul8_tiles(const Mul8Args& a, cudaStream_t stream) {
    return a.up ? start<true>(a, stream) : start<false>(a, stream);
}

int read_mul8_tiles_error(unsigned int* word, int clear, cudaStream_t stream) {
    *word = 0;
    if (!g_launched.load(std::memory_order_relaxed)) return 0;
    if (cudaMemcpyFromSymbolAsync(word, g_hc_mul8_tiles_error, sizeof(*word), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return -7;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return -7;
    if (clear && *word != 0) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbolAsync(g_hc_mul8_tiles_error, &z, sizeof(z), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess) return -7;
        if (cudaStreamSynchronize(stream) != cudaSuccess) return -7;
    }
    return 0;
}

}  // namespace hc
