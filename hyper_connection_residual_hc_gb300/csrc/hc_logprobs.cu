// Log probabilities of given tokens, the entropy and the most likely alternatives of rows of logits, in one pass over them.
// Formulas and edge cases: include/hc.h.
//
// A row is cut into equal segments for a cluster of 1, 2, 4 or 8 CTAs. A CTA takes its segment in chunks of 256 threads x 8
// vectors of 16 bytes, held in registers. Each thread keeps, for z = scale * logit in units of log 2 below its own running
// maximum m: S = sum 2^t and W = sum t 2^t, t = (x - m) * scale * log2(e); joined over threads, warps and the cluster
// (shared memory of the other CTAs), log sum e^z = m * scale + ln S and the entropy is ln S - ln 2 * W / S.
//
// The alternatives ride along as a sorted list of 64-bit keys: the logit's bits as a number that rises with it, then the index
// backwards, so that keys differ and of two equal logits the lower index is the greater key. A chunk is looked at again (in
// registers) only if some thread's largest logit exceeds the last key of a full list. For the first chunk, the q-th
// largest of each warp's 32 thread maxima, q * warps >= top, bounds the list's last key from below. What passes goes to a buffer
// in any order and is ranked there by counting, so the result does not depend on it. Should more pass than the buffer holds
// (many equal logits), the top-th largest of the threads' own first keys takes the bound's place: exactly `top` threads then have
// candidates, whose 64 values each fit.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "hc_attn.h"
#include "hc_attn_dev.cuh"
#include "hc_ffn.h"
#include "hc_ptx.cuh"

namespace hc {
namespace {

__device__ unsigned int g_hc_logprob_error = 0;
std::atomic<bool> g_launched{false};

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kVecs = 8;                                // vectors of a thread in a chunk
constexpr int kMostEach = kVecs * 8;                    // values of a thread in a chunk (bf16)
constexpr int kCandidates = kMostTop * kMostEach;       // see above: `top` threads' values always fit
constexpr int kChunk = kThreads * kVecs;
constexpr float kFar = -256.f;                          // 2^t is 0 in fp32 from -150 on; keeps t 2^t from being -inf * 0

struct Sums {
    float m, s, w;  // s == 0: nothing yet, m means nothing
};
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.f : m; }
// What s and w of a become below the larger reference m
__device__ __forceinline__ void lower_to(Sums& a, float m, float c) {
    if (a.s != 0.f) {
        const float d = fmaxf((a.m - m) * c, kFar);
        const float f = ex2(d);
        a.w = f * fmaf(d, a.s, a.w);
        a.s *= f;
    }
    a.m = m;
}
__device__ __forceinline__ Sums join(Sums a, Sums b, float c) {
    if (b.s == 0.f) return a;
    if (a.s == 0.f) return b;
    const float m = fmaxf(a.m, b.m);
    lower_to(a, m, c);
    lower_to(b, m, c);
    return {m, a.s + b.s, a.w + b.w};
}

// A number that rises with x; NaN below everything, never 0
__device__ __forceinline__ uint32_t rising(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return x != x ? 1u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float falling(uint32_t r) {
    return r == 1u ? __uint_as_float(0x7FC00000u) : __uint_as_float((r & 0x80000000u) ? r & 0x7FFFFFFFu : ~r);
}
__device__ __forceinline__ unsigned long long make_key(uint32_t r, int index) {
    return static_cast<unsigned long long>(r) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(index));
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ unsigned long long ld_cluster_u64(uint32_t addr) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

struct Shared {
    unsigned long long candidates[kCandidates + kMostTop];
    unsigned long long list[2][kMostTop];
    unsigned long long keys[kThreads];
    unsigned long long bound;
    uint32_t of_warp[kWarps];
    int count;
    float warp_sums[kWarps][3];
    float total[3];
    int list_n;  // of the list that counts, for the cluster's first CTA
    int list_at;
};

template <bool kWide>
struct Chunk {
    static constexpr int kEach = kWide ? 4 : 8;
    uint4 v[kVecs];
    __device__ __forceinline__ float at(int i) const {  // (i known at compile time)
        const uint4& q = v[i / kEach];
        const int e = i % kEach;
        if constexpr (kWide) {
            return __uint_as_float(e == 0 ? q.x : e == 1 ? q.y : e == 2 ? q.z : q.w);
        } else {
            const uint32_t u = e / 2 == 0 ? q.x : e / 2 == 1 ? q.y : e / 2 == 2 ? q.z : q.w;
            return __uint_as_float(e % 2 ? u & 0xFFFF0000u : u << 16);
        }
    }
    __device__ __forceinline__ float largest() const {  // of the numbers among them
        if constexpr (kWide) {
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < kVecs * kEach; ++i) m = fmaxf(m, at(i));
            return m;
        } else {
            __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&v[0].x);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&v[i].x));
                m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&v[i].y));
                m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&v[i].z));
                m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&v[i].w));
            }
            return fmaxf(__low2float(m), __high2float(m));
        }
    }
};

template <bool kWide>
__device__ __forceinline__ float logit(const LogprobArgs& p, long long row, int i) {
    const long long at = row * p.stride + i;
    if constexpr (kWide) return static_cast<const float*>(p.logits)[at];
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[at]);
}

// Ranks the `total` candidates by counting and puts the first `top` in order into list.
__device__ __forceinline__ void rank_candidates(const unsigned long long* candidates, int total, int top, unsigned long long* list) {
    for (int i = threadIdx.x; i < total; i += kThreads) {
        const unsigned long long mine = candidates[i];
        int above = 0;
        for (int j = 0; j < total; ++j) above += candidates[j] > mine;
        if (above < top) list[above] = mine;
    }
}

template <bool kWide>
__global__ void __launch_bounds__(kThreads) logprob_kernel(const LogprobArgs p, int ctas) {
    using C = Chunk<kWide>;
    constexpr int kEach = C::kEach, kValues = kVecs * kEach;
    __shared__ __align__(16) Shared sh;
    const int t = threadIdx.x, warp = t / 32, lane = t % 32;
    const int rank = ctas > 1 ? static_cast<int>(cluster_rank()) : 0;
    const long long row = blockIdx.x / static_cast<unsigned>(ctas);
    const char* base = static_cast<const char*>(p.logits) + row * p.stride * (kWide ? 4 : 2);
    const int vecs = (p.vocab + kEach - 1) / kEach, whole = p.vocab / kEach;
    const int each = (vecs + ctas - 1) / ctas;
    const int v0 = min(rank * each, vecs), v1 = min(v0 + each, vecs);
    const float c = p.scale * kLog2e;
    Sums sum = {0.f, 0.f, 0.f};
    unsigned long long bound = 0;  // the list's last key once it is full
    int list_n = 0, cur = 0;

    for (int b = v0; b < v1; b += kChunk) {
        C x;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int i = b + j * kThreads + t;
            constexpr uint32_t kNone = kWide ? 0xFF800000u : 0xFF80FF80u;  // minus infinity
            x.v[j] = make_uint4(kNone, kNone, kNone, kNone);
            if (i < v1) {
                if (i < whole) {
                    x.v[j] = __ldcs(reinterpret_cast<const uint4*>(base) + i);
                } else {  // the row's last values
                    uint32_t* u = &x.v[j].x;
#pragma unroll
                    for (int e = 0; e < kEach; ++e) {
                        if (i * kEach + e >= p.vocab) break;
                        if constexpr (kWide) {
                            u[e] = reinterpret_cast<const uint32_t*>(base)[i * kEach + e];
                        } else {
                            const uint32_t h = reinterpret_cast<const uint16_t*>(base)[i * kEach + e];
                            u[e / 2] = e % 2 ? (u[e / 2] & 0xFFFFu) | h << 16 : (u[e / 2] & 0xFFFF0000u) | h;
                        }
                    }
                }
            }
        }
        const float most = x.largest();
        {
            const float m = reference(fmaxf(sum.s != 0.f ? sum.m : -INFINITY, most));
            lower_to(sum, m, c);
            float s = 0.f, w = 0.f;
#pragma unroll
            for (int i = 0; i < kValues; ++i) {
                const float d = (x.at(i) - m) * c;
                const float e = ex2(d);
                s += e;
                w = fmaf(e, fmaxf(d, kFar), w);
            }
            sum.s += s;
            sum.w += w;
        }
        if (p.top == 0) continue;
        const uint32_t mine = rising(most);
        // (the barrier also keeps the buffers of the last chunk until all have read them)
        if (!__syncthreads_or(mine > static_cast<uint32_t>(bound >> 32))) continue;
        uint32_t least = static_cast<uint32_t>(bound >> 32) + 1;  // equal logits further on rank behind
        const int full = min(v1 - b, kThreads) / 32;             // warps whose every thread has a vector at least
        if (t == 0) sh.count = 0;
        if (bound == 0) {
            if (full > 0) {
                const int q = (p.top + full - 1) / full;
                uint32_t left = most > -INFINITY ? mine : 1u, w = 0;  // (padding counts as minus infinity, and is none)
                for (int i = 0; i < q; ++i) {
                    w = __reduce_max_sync(0xFFFFFFFFu, left);
                    const uint32_t who = __ballot_sync(0xFFFFFFFFu, left == w);
                    if (lane == __ffs(static_cast<int>(who)) - 1) left = 0;
                }
                if (lane == 0) sh.of_warp[warp] = w;
            }
            __syncthreads();
            least = full > 0 ? sh.of_warp[0] : 0;
            for (int i = 1; i < full; ++i) least = min(least, sh.of_warp[i]);
            if (list_n > 0) least = 0;  // (a list that a short first chunk left unfilled)
        } else {
            __syncthreads();
        }
        const int first = b + t;
        auto index = [&](int i) { return (first + i / kEach * kThreads) * kEach + i % kEach; };
        if (mine >= least) {
#pragma unroll
            for (int i = 0; i < kValues; ++i) {
                const uint32_t r = rising(x.at(i));
                if (r >= least && first + i / kEach * kThreads < v1 && index(i) < p.vocab) {
                    const int at = atomicAdd(&sh.count, 1);
                    if (at < kCandidates) sh.candidates[at] = make_key(r, index(i));
                }
            }
        }
        __syncthreads();
        int count = sh.count;
        if (count > kCandidates) {
            unsigned long long key = 0;  // this thread's greatest
            if (mine >= least) {
#pragma unroll
                for (int i = 0; i < kValues; ++i)
                    if (first + i / kEach * kThreads < v1 && index(i) < p.vocab) key = max(key, make_key(rising(x.at(i)), index(i)));
            }
            sh.keys[t] = key;
            __syncthreads();
            if (t == 0) sh.count = 0;
            int above = 0;
            for (int i = 0; i < kThreads; ++i) above += sh.keys[i] > key;
            if (key != 0 && above == p.top - 1) sh.bound = key;
            __syncthreads();
            const unsigned long long from = sh.bound;
            if (key >= from) {
#pragma unroll
                for (int i = 0; i < kValues; ++i) {
                    const unsigned long long k = make_key(rising(x.at(i)), index(i));
                    if (k >= from && first + i / kEach * kThreads < v1 && index(i) < p.vocab) {
                        const int at = atomicAdd(&sh.count, 1);
                        if (at < kCandidates) sh.candidates[at] = k;
                    }
                }
            }
            __syncthreads();
            count = min(sh.count, kCandidates);
        }
        if (t < list_n) sh.candidates[count + t] = sh.list[cur][t];
        __syncthreads();
        cur ^= 1;
        rank_candidates(sh.candidates, count + list_n, p.top, sh.list[cur]);
        list_n = min(count + list_n, p.top);
        __syncthreads();
        bound = list_n == p.top ? sh.list[cur][p.top - 1] : 0;
    }

    // the CTA's sums
#pragma unroll
    for (int o = 16; o; o /= 2) {
        const Sums other = {__shfl_xor_sync(0xFFFFFFFFu, sum.m, o), __shfl_xor_sync(0xFFFFFFFFu, sum.s, o), __shfl_xor_sync(0xFFFFFFFFu, sum.w, o)};
        sum = lane & o ? join(other, sum, c) : join(sum, other, c);
    }
    if (lane == 0) {
        sh.warp_sums[warp][0] = sum.m;
        sh.warp_sums[warp][1] = sum.s;
        sh.warp_sums[warp][2] = sum.w;
    }
    __syncthreads();
    sum = {sh.warp_sums[0][0], sh.warp_sums[0][1], sh.warp_sums[0][2]};
    for (int i = 1; i < kWarps; ++i) sum = join(sum, {sh.warp_sums[i][0], sh.warp_sums[i][1], sh.warp_sums[i][2]}, c);

    if (ctas > 1) {
        if (t == 0) {
            sh.total[0] = sum.m;
            sh.total[1] = sum.s;
            sh.total[2] = sum.w;
            sh.list_n = list_n;
            sh.list_at = cur;
        }
        cluster_sync();
        if (rank == 0) {
            int total = 0;
            for (int r = 1; r < ctas; ++r) {
                const uint32_t from = in_cta(smem_u32(&sh), static_cast<uint32_t>(r));
                const uint32_t tot = from + static_cast<uint32_t>(offsetof(Shared, total));
                sum = join(sum, {__uint_as_float(ld_cluster_u32(tot)), __uint_as_float(ld_cluster_u32(tot + 4)), __uint_as_float(ld_cluster_u32(tot + 8))}, c);
            }
            if (p.top > 0) {
                for (int r = 0; r < ctas; ++r) {
                    const uint32_t from = in_cta(smem_u32(&sh), static_cast<uint32_t>(r));
                    const int have = static_cast<int>(ld_cluster_u32(from + static_cast<uint32_t>(offsetof(Shared, list_n))));
                    const int at = static_cast<int>(ld_cluster_u32(from + static_cast<uint32_t>(offsetof(Shared, list_at))));
                    if (t < have) sh.candidates[total + t] = ld_cluster_u64(from + static_cast<uint32_t>(offsetof(Shared, list)) + static_cast<uint32_t>((at * kMostTop + t) * 8));
                    total += have;
                }
                __syncthreads();
                rank_candidates(sh.candidates, total, p.top, sh.list[cur ^ 1]);
                cur ^= 1;
                __syncthreads();
            }
        }
        cluster_sync();  // the other CTAs' shared memory stays until it has been read
        if (rank != 0) return;
    }

    const bool none = sum.s == 0.f;  // every logit is minus infinity
    const float log_s = logf(sum.s);
    auto log_probability = [&](float x) { return none ? -INFINITY : (x - sum.m) * p.scale - log_s; };
    if (t == 0) {
        if (p.logprob) {
            const long long token = p.tokens[row];
            float lp = 0.f;
            if (token >= 0 && token < p.vocab)
                lp = log_probability(logit<kWide>(p, row, static_cast<int>(token)));
            else if (token >= 0)
                atomicOr(&g_hc_logprob_error, kErrToken);
            p.logprob[row] = lp;
        }
        if (p.entropy) {
            const float h = none ? 0.f : log_s - sum.w / sum.s * kLn2;
            p.entropy[row] = h < 0.f ? 0.f : h;
        }
    }
    if (t < p.top) {
        const unsigned long long key = sh.list[cur][t];
        p.top_logprob[row * p.top + t] = log_probability(falling(static_cast<uint32_t>(key >> 32)));
        p.top_token[row * p.top + t] = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(key));
    }
}

template <bool kWide>
cudaError_t start(const LogprobArgs& a, int ctas, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.n * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(ctas);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = ctas > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, logprob_kernel<kWide>, a, ctas);
}

}  // namespace

int launch_logprobs(const LogprobArgs& a, cudaStream_t stream) {
    const int sms = attn_sm_count();
    if (sms < 1) return -7;
    const int vecs = (a.vocab + (a.wide ? 3 : 7)) / (a.wide ? 4 : 8);
    int ctas = 1;
    while (ctas < 8 && a.n * ctas < 2LL * sms && vecs >= 2 * ctas * kThreads) ctas *= 2;
    g_launched.store(true, std::memory_order_relaxed);
    return (a.wide ? start<true>(a, ctas, stream) : start<false>(a, ctas, stream)) == cudaSuccess ? 0 : -7;
}

int read_logprob_error(unsigned int* word, int clear, cudaStream_t stream) {
    *word = 0;
    if (!g_launched.load(std::memory_order_relaxed)) return 0;
    if (cudaMemcpyFromSymbolAsync(word, g_hc_logprob_error, sizeof(*word), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return -7;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return -7;
    if (clear && *word != 0) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbolAsync(g_hc_logprob_error, &z, sizeof(z), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess) return -7;
        if (cudaStreamSynchronize(stream) != cudaSuccess) return -7;
    }
    return 0;
}

}  // namespace hc
