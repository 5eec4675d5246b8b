// Log probabilities of given tokens, the entropy and the most likely alternatives of rows of logits, in one pass over them.
// Formulas and edge cases: include/hc.h.
//
// A row is cut into equal segments for a cluster of 1, 2, 4 or 8 CTAs. A CTA takes its segment in chunks of 256 threads x 4 vectors of
// 16 bytes; two chunks are on their way into shared memory while one is worked on (with one on its way, into registers, fp32 rows of
// 100,003 took 16% longer). Each thread keeps, for z = scale * logit in units of log 2 below its own running maximum m: S = sum 2^t
// and W = sum t 2^t, t = (x - m) * scale * log2(e); joined over threads, warps and the cluster (shared memory of the other CTAs),
// log sum e^z = m * scale + ln S and the entropy is ln S - ln 2 * W / S. Logits far below m are raised to where 2^t is still 0, so
// that minus infinity does not make t 2^t a NaN; a NaN stays one.
//
// The alternatives are 64-bit keys: the logit's bits as a number that rises with it, then the index backwards, so that keys differ
// and of two equal logits the lower index is the greater key. They are looked for once the segment has gone by. On the way a lane keeps
// only the largest logit of each of up to 12 groups of chunks. Then each warp posts the 4 largest of its 32 lanes' maxima; the top-th
// largest of the 32 posted numbers is no larger than the CTA's top-th logit, and of normal logits 1.1 top reach it. Lanes with such a
// logit in a group take the group's vectors once more, from shared memory or L2: 1% of a segment. (Collecting candidates on the way,
// against a bound that rises, took 27 us instead of 20 for 256 rows of 131,072 with 20: it doubles the instructions.) A warp whose
// buffer is full ranks it by counting and keeps the first `top`, of which the last is a bound of its own (many equal logits get there).
// The warps' candidates are ranked together, and the lists of a cluster's CTAs once more; the result does not depend on the order in
// which candidates came.

// Measured: 256 rows of 131,072 (bf16) with 20 alternatives 20 us, 14.4 without alternatives (4,650 GB/s: 9 instructions a value, 56% of
// the issue slots with 20, and 512 CTAs are 3 on some SMs and 4 on others), 18 with one; 4,097 rows of 100,003 (fp32) with 5 239 to 243 us,
// 6,700 to 6,800 GB/s, the copy rate; 8 rows of 131,072 with 20 8 us. A row takes a whole chunk (8,192 bf16 or 4,096 fp32 values) at
// least, however short: 4,000 rows of 500 (bf16) 28 us, of 2,000 19, of 8,192 20; with 5 alternatives 43, 35 and 36.

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
constexpr int kDevices = 64;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kVecs = 4;                                // vectors of a thread in a chunk
constexpr int kPosted = 4;                              // numbers that a warp posts
static_assert(kWarps * kPosted == 32 && kMostTop <= 32, "a lane for each");
constexpr int kBuffer = 96;                             // candidates of a warp
static_assert(kBuffer % 32 == 0 && kBuffer >= 2 * kMostTop + 32 - 1, "room for one of each lane behind a ranked list");
constexpr int kGroups = 12;                             // of chunks, whose largest logits are kept
constexpr int kChunk = kThreads * kVecs;
constexpr int kSlots = 3;                               // chunks in shared memory: one in work, two on their way
constexpr float kFar = -256.f;                          // 2^t is 0 in fp32 from -150 on

static_assert(kGroups * 32 * sizeof(uint16_t) == kBuffer * sizeof(unsigned long long), "a warp's own part of the same memory");

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

__device__ __forceinline__ unsigned long long pair(float a, float b) { unsigned long long r; asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b)); return r; }
__device__ __forceinline__ void unpair(unsigned long long v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) { unsigned long long r; asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c)); return r; }
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) { unsigned long long r; asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b)); return r; }

struct Shared {
    union {
        uint4 ring[kSlots][kVecs][kThreads];  // a thread's vectors are its own
        unsigned long long candidates[kWarps * kBuffer + 2];  // once the last chunk is done with
    };
    union {
        uint16_t most[kWarps][kGroups][32];  // the largest of a lane's logits in a group of chunks, or the next bf16 above
        __align__(16) unsigned long long buffer[kWarps][kBuffer];  // a warp's candidates, once it has been through its `most`
    };
    unsigned long long list[kMostTop];
    unsigned long long last[kMostTop];  // the list of a cluster's CTA, 0 where there is none
    float total[3];                     // its sums
    float warp_sums[kWarps][3];
    __align__(16) uint32_t posted[kWarps * kPosted];
    int count;
    uint32_t given;  // the given token's logit, or the word that holds it
    __align__(8) long long token;
};

// 16 bytes of global memory to shared memory, behind the thread's back.
__device__ __forceinline__ void copy_ahead(uint4* to, const uint4* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits for all but the last n groups of copies.
template <int n>
__device__ __forceinline__ void wait_copies() {
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

static_assert(4 * (sizeof(Shared) + 1024) <= 228 * 1024, "four CTAs an SM");

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t not_below2(uint32_t a, uint32_t b) {  // all ones in the halves where a is not below b
    return __hgeu2_mask(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
}
__device__ __forceinline__ float low_half(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float high_half(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

template <bool kWide>
struct Chunk {
    static constexpr int kEach = kWide ? 4 : 8;
    uint4 v[kVecs];
    __device__ __forceinline__ uint32_t word(int j, int i) const { return i == 0 ? v[j].x : i == 1 ? v[j].y : i == 2 ? v[j].z : v[j].w; }
    __device__ __forceinline__ float at(int j, int e) const {  // value e of vector j (both known at compile time)
        if constexpr (kWide) return __uint_as_float(word(j, e));
        return e % 2 ? high_half(word(j, e / 2)) : low_half(word(j, e / 2));
    }
    __device__ __forceinline__ float largest() const {  // of the numbers
        if constexpr (kWide) {
            float m = at(0, 0);
#pragma unroll
            for (int k = 1; k < kVecs * 4; ++k) m = fmaxf(m, at(k / 4, k % 4));
            return m;
        } else {
            auto h = [](const uint32_t& u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
            __nv_bfloat162 m = h(v[0].x);
#pragma unroll
            for (int k = 1; k < kVecs * 4; ++k) {
                const uint32_t u = word(k / 4, k % 4);
                m = __hmax2(m, h(u));
            }
            return fmaxf(__low2float(m), __high2float(m));
        }
    }
    static constexpr uint32_t kNone = kWide ? 0xFF800000u : 0xFF80FF80u;  // minus infinity
};

template <bool kWide>
__device__ __forceinline__ float logit(const LogprobArgs& p, long long row, int i) {
    const long long at = row * p.stride + i;
    if constexpr (kWide) return static_cast<const float*>(p.logits)[at];
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[at]);
}

// How many of `total` keys are above `mine`
__device__ __forceinline__ int keys_above(const unsigned long long* keys, int total, unsigned long long mine) {
    const ulonglong2* pairs = reinterpret_cast<const ulonglong2*>(keys);
    int above = 0;
#pragma unroll 8
    for (int j = 0; j < total / 2; ++j) {
        const ulonglong2 k = pairs[j];
        above += (k.x > mine) + (k.y > mine);
    }
    if (total % 2) above += keys[total - 1] > mine;
    return above;
}

// The first `top` of the CTA's candidates, in order, as `list`. Zeros are none.
__device__ __forceinline__ void rank_candidates(unsigned long long* candidates, int total, int top, unsigned long long* list) {
    for (int i = threadIdx.x; i < total; i += kThreads) {
        const unsigned long long mine = candidates[i];
        if (mine == 0) continue;
        const int above = keys_above(candidates, total, mine);
        if (above < top) list[above] = mine;
    }
}

// The same of a warp's own buffer, in place; returns how many there are then.
__device__ __forceinline__ int rank_buffer(unsigned long long* buffer, int count, int top) {
    const int lane = threadIdx.x % 32;
    unsigned long long mine[kBuffer / 32];
    int above[kBuffer / 32];
#pragma unroll
    for (int i = 0; i < kBuffer / 32; ++i) {
        mine[i] = lane + 32 * i < count ? buffer[lane + 32 * i] : 0;
        above[i] = mine[i] ? keys_above(buffer, count, mine[i]) : top;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kBuffer / 32; ++i)
        if (above[i] < top) buffer[above[i]] = mine[i];
    __syncwarp();
    return min(count, top);
}

// Four CTAs an SM: their loads and barriers cover each other.
template <bool kWide>
__global__ void __launch_bounds__(kThreads, 4) logprob_kernel(const LogprobArgs p, int ctas) {
    using C = Chunk<kWide>;
    constexpr int kEach = C::kEach;
    extern __shared__ __align__(16) unsigned char smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    griddep_launch_dependents();
    griddep_wait();
    const int t = threadIdx.x, warp = t / 32, lane = t % 32;
    const int rank = ctas > 1 ? static_cast<int>(cluster_rank()) : 0;
    const long long row = blockIdx.x / static_cast<unsigned>(ctas);
    const char* base = static_cast<const char*>(p.logits) + row * p.stride * (kWide ? 4 : 2);
    const int whole = p.vocab / kEach;  // vectors; the values behind them are a chunk of their own, of the last CTA's first thread
    const int each = (whole + ctas - 1) / ctas;
    const int v0 = min(rank * each, whole), v1 = min(v0 + each, whole);
    const int chunks = (v1 - v0 + kChunk - 1) / kChunk, all_chunks = chunks + (rank == ctas - 1 && whole * kEach < p.vocab ? 1 : 0);
    const float c = p.scale * kLog2e;
    Sums sum = {0.f, 0.f, 0.f};
    const float range = kFar / c;
    float far = range;  // logits below sum.m + range count as that: 2^t is 0
    uint32_t far2 = 0;  // the same as a pair of bf16
    auto refer_to = [&](float m) {
        lower_to(sum, m, c);
        far = m + range;  // or the next number below m, where the sum is m itself; that is far enough then
        if constexpr (kWide) {
            if (far >= m) far = falling(rising(m) - 1u);
        } else {
            uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rd(far));
            if (!(low_half(h) < m)) h = __float_as_uint(falling(rising(m) - 0x10000u)) >> 16;
            far2 = h | h << 16;
        }
    };
    refer_to(0.f);
    // candidates
    float lane_best = -INFINITY;                            // of all chunks so far
    float group_best = -INFINITY;                           // of the group's chunks so far
    const int group = (chunks + kGroups - 1) / kGroups;     // chunks
    int in_group = 0;
    uint16_t* to_most = &sh.most[warp][0][lane];
    if (t == 0) sh.count = 0;

    // Chunk i on its way to a slot; minus infinity in the place of what is not there.
    const uint4* ahead = reinterpret_cast<const uint4*>(base) + v0 + t;
    C x;
    auto load = [&](int i, int slot) {
        uint4* const to = &sh.ring[slot][0][t];
        if (v0 + (i + 1) * kChunk <= v1) {
#pragma unroll
            for (int j = 0; j < kVecs; ++j) copy_ahead(to + j * kThreads, ahead + j * kThreads);
        } else if (i < all_chunks) {
            const uint4 nothing = make_uint4(C::kNone, C::kNone, C::kNone, C::kNone);
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                if (i < chunks && v0 + i * kChunk + j * kThreads + t < v1)
                    copy_ahead(to + j * kThreads, ahead + j * kThreads);
                else
                    to[j * kThreads] = nothing;
            }
            if (i == chunks && t == 0) {  // the values behind the whole vectors, shifted in from below
                uint4 v = nothing;
#pragma unroll 1
                for (int e = p.vocab - 1; e >= whole * kEach; --e) {
                    if constexpr (kWide)
                        v = make_uint4(reinterpret_cast<const uint32_t*>(base)[e], v.x, v.y, v.z);
                    else
                        v = make_uint4(v.x << 16 | reinterpret_cast<const uint16_t*>(base)[e], v.y << 16 | v.x >> 16, v.z << 16 | v.y >> 16, v.w << 16 | v.z >> 16);
                }
                to[0] = v;
            }
        }
        ahead += kChunk;
        copies_end();
    };
    static_assert(kSlots == 3, "two chunks ahead");
    // The given token and its logit come on the way, as at the end they would be waited for one after the other.
    const bool gives = t == 0 && rank == 0 && p.logprob;
    if (gives) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(&sh.token)), "l"(p.tokens + row) : "memory");
    load(0, 0);
    load(1, 1);
    int slot = 0;
#pragma unroll 1
    for (int i = 0; i < all_chunks; ++i, slot = slot == kSlots - 1 ? 0 : slot + 1) {
        wait_copies<kSlots - 2>();
        const uint4* const here = &sh.ring[slot][0][t];
#pragma unroll
        for (int j = 0; j < kVecs; ++j) x.v[j] = here[j * kThreads];
        if (i == 0 && gives && sh.token >= 0 && (kWide ? sh.token : sh.token | 1) < p.vocab)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&sh.given)), "l"(base + (kWide ? sh.token * 4 : sh.token / 2 * 4)) : "memory");
        load(i + kSlots - 1, slot == 0 ? kSlots - 1 : slot - 1);
        const float most = x.largest();
        if (most > (sum.s != 0.f ? sum.m : -INFINITY)) refer_to(most);
        if (p.top > 0 && i < chunks) {
            lane_best = fmaxf(lane_best, most);
            group_best = fmaxf(group_best, most);
            if (++in_group == group || i + 1 == chunks) {
                *to_most = kWide ? __bfloat16_as_ushort(__float2bfloat16_ru(group_best)) : static_cast<uint16_t>(__float_as_uint(group_best) >> 16);
                to_most += 32;
                in_group = 0;
                group_best = -INFINITY;
            }
        }
        // t = x c - m c by one FMA with m c rounded; what that rounding is off by goes back into the sums. Two values an instruction,
        // but for the unpacking and 2^t.
        const float mc = sum.m * c;
        float s, w;
        if (fabsf(mc) < 1e6f) {
            unsigned long long s2 = 0, w2 = 0;
            const unsigned long long c2 = pair(c, c), mc2 = pair(-mc, -mc);
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
#pragma unroll
                for (int e = 0; e < kEach; e += 2) {
                    float d0, d1;
                    if constexpr (kWide) {
                        d0 = max_nan(x.at(j, e), far);
                        d1 = max_nan(x.at(j, e + 1), far);
                    } else {
                        const uint32_t u = max_nan2(x.word(j, e / 2), far2);
                        d0 = low_half(u);
                        d1 = high_half(u);
                    }
                    const unsigned long long d = fma2(pair(d0, d1), c2, mc2);
                    unpair(d, d0, d1);
                    const unsigned long long f = pair(ex2(d0), ex2(d1));
                    s2 = add2(s2, f);
                    w2 = fma2(f, d, w2);
                }
            }
            float s0, s1, w0, w1;
            unpair(s2, s0, s1);
            unpair(w2, w0, w1);
            const float off = -fmaf(sum.m, c, -mc), f = ex2(off);
            s = (s0 + s1) * f;
            w = fmaf(s, off, (w0 + w1) * f);
        } else {  // so far out that the rounding would be whole doublings
            s = w = 0.f;
#pragma unroll 1
            for (int k = 0; k < kVecs * kEach; ++k) {
                const uint4* v = here + k / kEach * kThreads;
                const float u = kWide ? reinterpret_cast<const float*>(v)[k % kEach]
                                      : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(v)[k % kEach]) << 16);
                const float d = (u - sum.m) * c, f = ex2(d);
                s += f;
                if (f != 0.f) w = fmaf(f, d, w);  // (below the lowest number there is minus infinity)
            }
        }
        sum.s += s;
        sum.w += w;
    }
    wait_copies<0>();
    if (p.top > 0) {
        // the warp's largest numbers for the others
        {
            uint32_t mine = lane_best > -INFINITY ? rising(lane_best) : 1u, w = 0;  // (what is not there is minus infinity too)
#pragma unroll
            for (int k = 0; k < kPosted; ++k) {
                w = __reduce_max_sync(0xFFFFFFFFu, mine);
                const uint32_t who = __ballot_sync(0xFFFFFFFFu, mine == w);
                if (lane == __ffs(static_cast<int>(who)) - 1) mine = 0;
                if (lane == 0) sh.posted[warp * kPosted + k] = w;
            }
        }
        __syncthreads();
        uint32_t least = 0;  // logits below are not wanted: the top-th largest of what is posted
        {
            const uint32_t mine = sh.posted[lane];
            int above = 0;
#pragma unroll
            for (int k = 0; k < kWarps * kPosted; k += 4) {
                const uint4 u = *reinterpret_cast<const uint4*>(&sh.posted[k]);
                above += (u.x > mine) + (u.y > mine) + (u.z > mine) + (u.w > mine);
            }
            least = __reduce_min_sync(0xFFFFFFFFu, above < p.top ? mine : 0xFFFFFFFFu);
        }
        const float from = least <= 1 ? -INFINITY : falling(least);  // what is not below is looked at, NaN too
        uint32_t groups = 0;
        for (int g = 0; g * group < chunks; ++g) groups |= (__uint_as_float(static_cast<uint32_t>(sh.most[warp][g][lane]) << 16) < from ? 0u : 1u) << g;
        __syncwarp();
        unsigned long long own = 0;  // keys up to this one are not among the first `top`
        int count = 0;               // in the warp's buffer
        // A value of each lane (0 bits: none) becomes a candidate.
        auto collect = [&](unsigned long long key) {
            if (key <= own || static_cast<uint32_t>(key >> 32) < least) key = 0;
            uint32_t who = __ballot_sync(0xFFFFFFFFu, key != 0);
            if (count + __popc(who) > kBuffer) {
                count = rank_buffer(sh.buffer[warp], count, p.top);
                own = sh.buffer[warp][p.top - 1];  // (the buffer held more than kMostTop)
                if (key <= own) key = 0;
                who = __ballot_sync(0xFFFFFFFFu, key != 0);
            }
            if (key != 0) sh.buffer[warp][count + __popc(who & ((1u << lane) - 1u))] = key;
            count += __popc(who);
            __syncwarp();
        };
        int i = 0, until = 0;  // chunks to look at
        while (true) {
            if (i == until && groups != 0) {
                const int g = __ffs(static_cast<int>(groups)) - 1;
                groups &= groups - 1;
                i = g * group;
                until = min(i + group, chunks);
            }
            if (!__any_sync(0xFFFFFFFFu, i < until)) break;
            uint32_t mask = 0;  // a bit for each value
            const int vec = v0 + i * kChunk + t;
            if (i < until) {
                // Behind the bound's own index only greater logits are wanted: rows of many equal ones, masked ones above all, would
                // go through the ranking for nothing (256 rows of 131,072 with 16 of them not minus infinity: 167 us without this).
                float wanted = from;
                if (own != 0) {
                    uint32_t u = static_cast<uint32_t>(own >> 32);
                    if (static_cast<uint32_t>(vec) * kEach > 0xFFFFFFFFu - static_cast<uint32_t>(own)) u += kWide ? 1u : 0x10000u;
                    if (u > 1 && u <= 0xFF800000u) wanted = falling(u);  // (up to infinity)
                }
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    if (i >= all_chunks - kSlots)
                        x.v[j] = sh.ring[i % kSlots][j][t];
                    else
                        x.v[j] = reinterpret_cast<const uint4*>(base)[vec + j * kThreads];  // (all of such a chunk is there)
                }
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    uint32_t bits = 0;
                    if constexpr (kWide) {
#pragma unroll
                        for (int e = 0; e < kEach; ++e) bits |= (x.at(j, e) < wanted ? 0u : 1u) << e;
                    } else {  // the even values' bits first
                        const uint32_t f = __float_as_uint(wanted), pair_wanted = __byte_perm(f, f, 0x3232);
#pragma unroll
                        for (int k = 0; k < 4; ++k) bits |= not_below2(x.word(j, k), pair_wanted) & 0x00010001u << k;
                        bits = (bits | bits >> 12) & 0xFFu;
                    }
                    if (vec + j * kThreads < v1) mask |= bits << (j * kEach);
                }
                ++i;
            }
            while (__any_sync(0xFFFFFFFFu, mask != 0)) {  // one value of each lane
                unsigned long long key = 0;
                if (mask) {
                    const int bit = __ffs(static_cast<int>(mask)) - 1, j = bit / kEach;
                    mask &= mask - 1;
                    uint4 v = j & 2 ? (j & 1 ? x.v[3] : x.v[2]) : (j & 1 ? x.v[1] : x.v[0]);
                    const int k = bit % 4;
                    const uint32_t u = k & 2 ? (k & 1 ? v.w : v.z) : (k & 1 ? v.y : v.x);
                    const int e = kWide ? k : 2 * k + bit / 4 % 2;
                    key = make_key(rising(kWide ? __uint_as_float(u) : e % 2 ? high_half(u) : low_half(u)), (vec + j * kThreads) * kEach + e);
                }
                collect(key);
            }
        }
        if (rank == ctas - 1 && warp == 0 && whole * kEach < p.vocab) {  // the values behind the whole vectors
            const int index = whole * kEach + lane;
            collect(index < p.vocab ? make_key(rising(logit<kWide>(p, row, index)), index) : 0);
        }
        int at = 0;
        if (lane == 0) at = atomicAdd(&sh.count, count);
        at = __shfl_sync(0xFFFFFFFFu, at, 0);
        __syncthreads();  // the ring is done with
        for (int k = lane; k < count; k += 32) sh.candidates[at + k] = sh.buffer[warp][k];
        __syncthreads();
        rank_candidates(sh.candidates, sh.count, p.top, sh.list);
    }

    // The CTA's sums: all lanes refer to the largest maximum, then sums add up.
    auto gather = [&](int lanes) {
        float m = sum.s != 0.f ? sum.m : -INFINITY;
#pragma unroll
        for (int o = 16; o; o /= 2)
            if (o < lanes) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        lower_to(sum, reference(m), c);
#pragma unroll
        for (int o = 16; o; o /= 2) {
            if (o < lanes) {
                sum.s += __shfl_xor_sync(0xFFFFFFFFu, sum.s, o);
                sum.w += __shfl_xor_sync(0xFFFFFFFFu, sum.w, o);
            }
        }
    };
    gather(32);
    if (lane == 0) {
        sh.warp_sums[warp][0] = sum.m;
        sh.warp_sums[warp][1] = sum.s;
        sh.warp_sums[warp][2] = sum.w;
    }
    __syncthreads();
    sum = {sh.warp_sums[lane % kWarps][0], sh.warp_sums[lane % kWarps][1], sh.warp_sums[lane % kWarps][2]};
    gather(kWarps);

    if (ctas > 1) {
        if (t == 0) {
            sh.total[0] = sum.m;
            sh.total[1] = sum.s;
            sh.total[2] = sum.w;
        }
        if (t < p.top) sh.last[t] = t < sh.count ? sh.list[t] : 0;
        cluster_sync();
        if (rank == 0) {
            const uint32_t own_smem = smem_u32(&sh);
            sum = {0.f, 0.f, 0.f};
            if (lane % 8 < ctas) {
                const uint32_t from = in_cta(own_smem + static_cast<uint32_t>(offsetof(Shared, total)), static_cast<uint32_t>(lane % 8));
                sum.m = __uint_as_float(ld_cluster_u32(from));
                sum.s = __uint_as_float(ld_cluster_u32(from + 4));
                sum.w = __uint_as_float(ld_cluster_u32(from + 8));
            }
            gather(8);
            if (p.top > 0) {
                static_assert(kThreads == 8 * kMostTop, "a thread for each key");
                if (t < ctas * p.top)
                    sh.candidates[t] = ld_cluster_u64(in_cta(own_smem + static_cast<uint32_t>(offsetof(Shared, last) + t % p.top * 8), static_cast<uint32_t>(t / p.top)));
                __syncthreads();
                rank_candidates(sh.candidates, ctas * p.top, p.top, sh.list);
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
            const long long token = sh.token;
            float lp = 0.f;
            if (token >= 0 && (kWide ? token : token | 1) < p.vocab)
                lp = log_probability(kWide ? __uint_as_float(sh.given) : token % 2 ? high_half(sh.given) : low_half(sh.given));
            else if (token >= 0 && token < p.vocab)  // (the last of an odd number)
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
        const unsigned long long key = sh.list[t];
        p.top_logprob[row * p.top + t] = log_probability(falling(static_cast<uint32_t>(key >> 32)));
        p.top_token[row * p.top + t] = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(key));
    }
}

template <bool kWide>
cudaError_t start(const LogprobArgs& a, int ctas, cudaStream_t stream) {
    static std::atomic<bool> ready[kDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    if (!ready[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(logprob_kernel<kWide>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared));
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.n * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    unsigned more = 0;
    if (ctas > 1) {
        attrs[0].id = cudaLaunchAttributeClusterDimension;
        attrs[0].val.clusterDim.x = static_cast<unsigned>(ctas);
        attrs[0].val.clusterDim.y = attrs[0].val.clusterDim.z = 1;
        more = 1;
    }
    more += static_cast<unsigned>(programmatic_launch(a.n * a.vocab / 600, false, stream, attrs + more));  // (0.5 to 1.5 values a ps)
    cfg.attrs = attrs;
    cfg.numAttrs = more;
    return cudaLaunchKernelEx(&cfg, logprob_kernel<kWide>, a, ctas);
}

}  // namespace

int launch_logprobs(const LogprobArgs& a, cudaStream_t stream) {
    const int sms = attn_sm_count();
    if (sms < 1) return -7;
    const int vecs = (a.vocab + (a.wide ? 3 : 7)) / (a.wide ? 4 : 8);
    int ctas = 1;
    // CTAs a row: until there are 2 an SM, or a segment would be less than 2 chunks, as a cluster's join takes 1.5 us or more. 256 rows of
    // 131,072 (bf16, 20 alternatives): 1 CTA a row 27 us, 2 20, 4 26. 160 rows of 16,384: 1 5.6, 2 7.3. 64 rows of 8,192 (fp32): 1
    // 5.1, 4 8.9. One row of 32,768 (bf16) is the other way round: 2 6.2, 4 5.7.
    while (ctas < 8 && a.n * ctas < 2LL * sms && vecs >= 4 * ctas * kChunk) ctas *= 2;
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
