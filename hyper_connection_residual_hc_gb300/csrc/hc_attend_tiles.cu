// Attention over the 4-bit cache for many queries of a sequence (prefill, chunk by chunk), on the tensor cores'
// tcgen05.mma with accumulators in tensor memory. Formulas, masks and format: include/hc.h; the kernel for few
// queries (hc_attend.cu) shares the definitions of rows and masks.
//
// A CTA takes 256 rows of one (sequence, kv head): row = query * group + head in the group, two tiles of 128 (the
// MMA's M). It walks the keys in tiles of 128 tokens:
//   4 dequantising warps turn the tile's 8 cache blocks into fp16 (exact) in shared memory, once for both row
//     tiles: keys and values as rows of 64 columns (128 bytes, 128-byte swizzle), one row a token. As the B operand of
//     S = Q K^T that is K-major; as the B operand of O += P V the same layout reads as MN-major.
//   1 warp issues the MMAs: S_a = Q_a K^T (128 x 128 x D) and O_a += P_a V (128 x D x 128), the two row tiles in turn,
//     so that one tile's softmax runs under the other tile's products.
//   2 x 4 softmax warps, one thread a row (a tensor-memory lane): scores to registers, the running maximum, weights to
//     fp16 back into tensor memory over the scores, where the second MMA reads them as its A operand.
// The maximum is raised only when a score exceeds it by more than 2^8 (as in hc_attend.cu, with weights as large as fp16
// allows: kLift), so the outputs in tensor memory are rarely rescaled. S_a of the next tile is issued behind P_a V of this
// one: a thread that sees its scores knows that its outputs are complete.
//
// Row tiles that would leave SMs idle (few of them, or the last of many) have their key tiles cut into slices, one CTA
// each, joined in their order by the CTA that finishes last.
//
// Measured: 2 sequences of 2,048 queries behind 4,096 to 6,144 cached keys, 40 query and 8 kv heads of 128: 418 us, 1,233
// TFLOP/s, 63% of the measured cuBLAS rate (the first form, with separate score and value steps by 17 warps of 96 registers,
// took 1,806 us). A key tile takes about 1.75 us; in an earlier form (541 us) the call's MMAs alone took 302 us,
// dequantising alone 278, the softmax alone with its barriers 444 and its barriers alone 283: the round trip scores -> weights ->
// scores is what bounds it, with two row tiles to overlap and no tensor memory left for a second set of scores. About 14 us a
// CTA are its start and end; they were 27 before the queries were loaded and the outputs written by whole rows, beside
// the first keys, and before divisions became products. Tried and slower, against 560 to 577 us then: 16 softmax warps with
// half a row each (604 us), an MMA warp that polls for whichever row tile is ready (704 us: its polling takes issue slots), 8
// dequantising warps (630 us); against 428 us: an eighth of the exponentials by a polynomial instead of the special
// function unit (444 us). Heads of 64, 64 query and 8 kv heads, the same lengths: 568 us, 725 TFLOP/s.
//
// Every wait is bounded: on expiry the kernel sets a bit of the device error word, stops waiting, lets its MMAs end
// and frees its tensor memory.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "hc_attn.h"
#include "hc_attn_dev.cuh"
#include "hc_kv.cuh"
#include "hc_ptx.cuh"

namespace hc {
namespace {

__device__ unsigned int g_hc_tiles_error = 0;
std::atomic<bool> g_launched{false};  // whether the word above can be set at all (reading it costs a copy and a wait)

constexpr int kRowTile = 128;   // rows of an MMA
constexpr int kRows = 2 * kRowTile;
constexpr int kKeys = 128;      // keys of a tile
constexpr int kSoftmaxWarps = 8, kDequantWarps = 4;
static_assert(kDequantWarps == 4, "a word of notes");
constexpr int kBlocksPerWarp = kKeys / 16 / kDequantWarps;  // cache blocks of a key tile that a dequantising warp takes
constexpr int kMmaWarp = kSoftmaxWarps + kDequantWarps;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kLeastSlice = 8;  // key tiles of a slice at least: joining costs as much as a few
constexpr int kNotes = 8;       // key tiles whose notes (absent blocks, NaN values) are kept
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kMaxDevices = 64;

template <int D>
struct TilePlan {
    static constexpr int kHalf = kKeys * 128;              // bytes of 128 rows of 64 columns
    static constexpr int kTile = kHalf * (D / 64);         // one operand tile
    static constexpr int kQ = 0;                           // two row tiles of Q
    static constexpr int kK = kQ + 2 * kTile;              // two stages
    static constexpr int kV = kK + 2 * kTile;
    static constexpr int kNan = kV + 2 * kTile;            // [kNotes][kKeys] bits: 16-column groups whose scale is NaN
    static constexpr int kBars = kNan + kNotes * kKeys * 2;
    static constexpr int kSmem = kBars + 16 * 8 + 16 + 1024;  // + alignment
    static constexpr int kO = 256;                         // tensor memory: S_0, S_1, O_0, O_1
    static constexpr uint32_t kColumns = 512;
    static constexpr int kPartFloats = kRows * (D + 2);    // a slice's result in the workspace
};

struct Wait {
    volatile uint32_t* abort;
    __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity) const {
        if (mbar_sleep(bar, parity)) return;
        const uint64_t t0 = global_timer_ns();
        while (true) {
            if (mbar_sleep(bar, parity)) return;
            if (*abort) return;
            if (global_timer_ns() - t0 > kWaitNs) {
                *abort = 1u;
                atomicOr(&g_hc_tiles_error, kErrTile);
                return;
            }
        }
    }
    // at exit: lets MMAs in flight end whatever was aborted
    __device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) const {
        const uint64_t t0 = global_timer_ns();
        while (!mbar_test(bar, parity)) {
            if (global_timer_ns() - t0 > kWaitNs) {
                atomicOr(&g_hc_tiles_error, kErrTile);
                return;
            }
        }
    }
};

// Shared-memory descriptor of an operand stored as rows of 128 bytes with the 128-byte swizzle, 8-row groups 1,024
// bytes apart; `leading`: bytes between blocks of 64 columns (read by MN-major operands only). Fields as in
// sdesc_kmajor_sw64; swizzle mode 2 = 128 bytes.
__device__ __forceinline__ uint64_t sdesc_sw128(uint32_t saddr, uint32_t leading) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(leading >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}
// kind::f16, fp16 operands, fp32 accumulator; bit 16: B is MN-major
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// The whole warp comes here with the same arguments (so that they stay in uniform registers); `lead` is 1 in one lane,
// which issues.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t lead;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(lead));
    return lead;
}
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(lead)
        : "memory");
}
// 32 consecutive columns of this thread's lane; the values are there after tmem_ld_wait, which waits for all loads so far.
__device__ __forceinline__ void tmem_ld32_start(uint32_t addr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(addr)
        : "memory");
}
// The wait names the registers it waits for, so that no use of them moves above it.
__device__ __forceinline__ void tmem_ld_wait(float (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]),
                   "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]),
                   "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]),
                   "+f"(v[28]), "+f"(v[29]), "+f"(v[30])
                 :
                 : "memory");
    asm volatile("" : "+f"(v[31])::"memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&v)[32]) {
    tmem_ld32_start(addr, v);
    tmem_ld_wait(v);
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const float (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]),
        "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]),
        "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// Pairs of fp32 in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Columns [from, upto) without the blocks in `gone`, as bits of columns 32 q .. 32 q + 31.
__device__ __forceinline__ uint32_t seen_columns(int q, int from, int upto, uint32_t gone) {
    const int a = min(max(from - 32 * q, 0), 32), b = min(max(upto - 32 * q, 0), 32);
    uint32_t seen = b > a ? (0xFFFFFFFFu >> (32 - (b - a))) << a : 0u;
    if (gone >> (2 * q) & 1) seen &= 0xFFFF0000u;
    if (gone >> (2 * q + 1) & 1) seen &= 0x0000FFFFu;
    return seen;
}

// The largest of a row's scores in tensor memory. kMask: of the columns in seen[].
template <bool kMask>
__device__ __forceinline__ float largest(uint32_t ts, const uint32_t* seen) {
    float top0 = -INFINITY, top1 = -INFINITY;
    float v[2][32];
    tmem_ld32_start(ts, v[0]);
#pragma unroll
    for (int q = 0; q < kKeys / 32; ++q) {
        tmem_ld_wait(v[q % 2]);
        if (q + 1 < kKeys / 32) tmem_ld32_start(ts + static_cast<uint32_t>(32 * (q + 1)), v[(q + 1) % 2]);
        if constexpr (kMask) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (!(seen[q] >> i & 1)) v[q % 2][i] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            top0 = fmaxf(top0, fmaxf(v[q % 2][i], v[q % 2][i + 1]));
            top1 = fmaxf(top1, fmaxf(v[q % 2][i + 2], v[q % 2][i + 3]));
        }
    }
    return fmaxf(top0, top1);
}

// The weights 2^(score * f + shift) of half a row of scores in tensor memory, as fp16 pairs over the scores' first columns
// (of which nothing is needed any more), and added to `sum` (in fp32, before the rounding).
template <bool kMask>
__device__ __forceinline__ void weights(uint32_t ts, int half, float f, float shift, const uint32_t* seen, uint64_t& sum) {
    uint64_t s0 = pair(0.f, 0.f);
    const uint64_t ff = pair(f, f), sh = pair(shift, shift);
    float v[2][32];
    tmem_ld32_start(ts + static_cast<uint32_t>(64 * half), v[0]);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        tmem_ld_wait(v[q]);
        if (q == 0) tmem_ld32_start(ts + static_cast<uint32_t>(64 * half + 32), v[1]);
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            float a, b, c, d;
            unpair(fma2(pair(v[q][i], v[q][i + 1]), ff, sh), a, b);
            unpair(fma2(pair(v[q][i + 2], v[q][i + 3]), ff, sh), c, d);
            if constexpr (kMask) {
                a = seen[2 * half + q] >> i & 1 ? a : -INFINITY;
                b = seen[2 * half + q] >> (i + 1) & 1 ? b : -INFINITY;
                c = seen[2 * half + q] >> (i + 2) & 1 ? c : -INFINITY;
                d = seen[2 * half + q] >> (i + 3) & 1 ? d : -INFINITY;
            }
            a = ex2(a);
            b = ex2(b);
            c = ex2(c);
            d = ex2(d);
            sum = add2(sum, pair(a, b));
            s0 = add2(s0, pair(c, d));
            w[i / 2] = pack_f16(a, b);
            w[i / 2 + 1] = pack_f16(c, d);
        }
        tmem_st16(ts + static_cast<uint32_t>(32 * half + 16 * q), w);
    }
    sum = add2(sum, s0);
}

__device__ __forceinline__ void store32(__nv_bfloat16* dst, const float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(v[i + 2 * e], v[i + 2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&t);
        }
        *reinterpret_cast<uint4*>(dst + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// What a CTA works on: one slice of the keys of one row tile of a sequence and a kv head. seq is -1 for CTAs without work;
// `rest` counts the sliced row tiles.
struct Found {
    int seq, tile, head, rest, slice, slices;
};
struct FindScratch {
    int part[2][16];  // of the warps, for one sum and the next
    int seq, tile;
};
// By all threads. CTAs start in turn as SMs get free, so the row tiles with the most key tiles come first, and the last ones to
// start are short: 2 fresh prompts of 2,048 tokens, 143 us in this order, 152 us one sequence after the other. (With more
// than 32 sequences the latter: the search would take barriers, and the order matters less: 64 of 10 queries, 111 and 104 us.)
// As many row tiles as fill the SMs a whole number of times are taken whole; those left, if they fill half of the SMs at
// most, are cut into slices that fill them: 1,024 queries behind 32,768 keys 1,024 us whole, 604 us cut.
__device__ __forceinline__ Found find_tile(const AttArgs& p, int cta, const Divider& sms, const Divider& heads, int tid, FindScratch& f) {
    const int warp = tid / 32, lane = tid % 32, group = p.group.by;
    struct Seq {
        long long behind;  // rows of (queries - keys) queries
        int rows, tiles, kvl;
    };
    auto load = [&](int b) {
        Seq q = {};
        if (b < p.seqs) {
            const SeqRows s = load_seq(p, b, cta == 0 ? &g_hc_tiles_error : nullptr);
            q.rows = s.ql * group;
            q.tiles = static_cast<int>((static_cast<unsigned int>(q.rows) + kRows - 1) / kRows);
            q.kvl = s.kvl;
            q.behind = static_cast<long long>(s.ql - s.kvl) * group;
        }
        return q;
    };
    // Up to 32 sequences: each warp does it all, one sequence a lane, without barriers.
    const bool few = p.seqs <= 32;
    const int me = few ? lane : tid;
    const Seq own = load(me);
    int tiles = own.tiles;
    if (!few)
        for (int b = me + kThreads; b < p.seqs; b += kThreads) tiles += load(b).tiles;
    tiles = __reduce_add_sync(0xFFFFFFFFu, tiles);
    if (!few) {
        if (tid == 0) f.seq = -1;
        if (lane == 0) f.part[0][warp] = tiles;
        __syncthreads();
        tiles = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) tiles += f.part[0][w];
    }
    // More than tiles_bound come from starts that decrease, and so claim rows again, only. The grid has no CTAs for them, and a
    // row tile that got some of its slices would leave its counter in the workspace: nothing is done.
    const long long all = static_cast<long long>(static_cast<unsigned int>(tiles)) * heads.by;
    const int items = all > static_cast<long long>(gridDim.x) - sms.by ? 0 : static_cast<int>(all);
    const int whole = divide(items, sms) * sms.by, left = items - whole;
    Found r = {-1, 0, 0, 0, 0, 1};
    int item = cta;
    if (cta >= whole && left > 0) {
        r.slices = max(1, min(sms.by, kAttMaxSlices) / left);
        r.rest = (cta - whole) / r.slices;
        r.slice = cta - whole - r.rest * r.slices;
        item = whole + r.rest;
    }
    if (item >= items) return r;  // the same in every thread
    const int want = divide(item, heads);  // in the order
    r.head = item - want * heads.by;
    auto scan = [&](int v) {  // inclusive, over the warp
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, v, o);
            if (lane >= o) v += y;
        }
        return v;
    };
    if (few) {
        // how many of the lane's row tiles (the last ones) have more than x key tiles, where there is no window
        auto above = [&](int x) {
            if (x < 0) return own.tiles;
            const int keys = kKeys * x;  // a row must see more
            if (!p.causal) return own.kvl > keys ? own.tiles : 0;
            const long long r0 = own.behind + static_cast<long long>(keys) * group;  // the first row that does
            return r0 <= 0 ? own.tiles : r0 >= own.rows ? 0 : own.tiles - static_cast<int>(static_cast<unsigned int>(r0) / kRows);
        };
        // the least number of key tiles that no more than `want` row tiles exceed, and how many do
        int lo = 0, hi = __reduce_max_sync(0xFFFFFFFFu, own.tiles > 0 ? (own.kvl + kKeys - 1) / kKeys : 0), exceed = 0;
        while (lo < hi) {
            const int x = (lo + hi) / 2, n = __reduce_add_sync(0xFFFFFFFFu, above(x));
            if (n <= want) {
                hi = x;
                exceed = n;
            } else {
                lo = x + 1;
            }
        }
        const int n0 = above(lo), n = above(lo - 1) - n0, x = exceed + scan(n);
        const int src = __ffs(static_cast<int>(__ballot_sync(0xFFFFFFFFu, x > want))) - 1;
        if (src >= 0) {
            r.seq = src;
            r.tile = __shfl_sync(0xFFFFFFFFu, own.tiles - n0 - n + want - (x - n), src);
        }
        return r;
    }
    int before = 0;
    for (int b0 = 0; b0 < p.seqs && before <= want; b0 += kThreads) {
        const int n = b0 == 0 ? own.tiles : load(b0 + tid).tiles;
        int x = before + scan(n);
        int* part = f.part[1 - b0 / kThreads % 2];
        if (lane == 31) part[warp] = x - before;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) x += part[w];
            before += part[w];
        }
        if (x > want && x - n <= want) {
            f.seq = b0 + tid;
            f.tile = want - (x - n);
        }
    }
    __syncthreads();
    r.seq = f.seq;
    r.tile = f.tile;
    return r;
}

// One lane's part of a cache block in registers.
template <int D>
struct BlockRegs {
    uint4 k[D / 64], v[D / 64];
    uint32_t ks, vs;  // D / 32 key scales, 4 value scales
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attend_tiles_kernel(const AttArgs p, const Divider sms, const Divider kv_heads) {
    using T = TilePlan<D>;
    constexpr int kSteps = D / 16;       // MMAs of S
    constexpr int kLanes = D / 8, kSide = 32 / kLanes;  // lanes to a row in memory, 16 bytes each, and rows side by side
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ FindScratch find_scratch;
    __shared__ bool last_flag;
    __shared__ __align__(4) uint8_t absent[kNotes][kDequantWarps];  // per key tile and warp: bits of its blocks that are not there
    __shared__ uint32_t nan_any[kNotes];                // per key tile: some value's scale is NaN
    const uint32_t sbase = smem_u32(smem);
    const int tid = static_cast<int>(threadIdx.x), warp = tid / 32, lane = tid % 32;
    const int group = p.group.by;

    const uint32_t bars = sbase + T::kBars;
    auto k_full = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
    auto k_empty = [&](int i) { return bars + 8u * static_cast<uint32_t>(2 + i); };
    auto v_full = [&](int i) { return bars + 8u * static_cast<uint32_t>(4 + i); };
    auto v_empty = [&](int i) { return bars + 8u * static_cast<uint32_t>(6 + i); };
    auto s_full = [&](int a) { return bars + 8u * static_cast<uint32_t>(8 + a); };
    auto p_full = [&](int a, int half) { return bars + 8u * static_cast<uint32_t>(10 + 2 * a + half); };
    const uint32_t o_full = bars + 8u * 14u, q_full = bars + 8u * 15u;
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(smem + T::kBars + 16 * 8);
    volatile uint32_t* abort_flag = tmem_ptr + 1;
    const Wait wait{abort_flag};
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(k_full(i), kDequantWarps);
            mbar_init(k_empty(i), 1);
            mbar_init(v_full(i), kDequantWarps);
            mbar_init(v_empty(i), 1);
            mbar_init(s_full(i), 1);
            mbar_init(p_full(i, 0), 4);
            mbar_init(p_full(i, 1), 4);
        }
        mbar_init(o_full, 1);
        mbar_init(q_full, kSoftmaxWarps);
        for (int i = 0; i < kNotes; ++i) nan_any[i] = 0;
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_ptr), T::kColumns);
        tmem_relinquish();
    }

    // ---- which rows and keys -------------------------------------------------------------------------------
    const Found found = find_tile(p, static_cast<int>(blockIdx.x), sms, kv_heads, tid, find_scratch);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_ptr);
    auto leave = [&]() {
        griddep_wait();  // the call has ended when both kernels have
        if (warp == kMmaWarp) tmem_dealloc(tmem, T::kColumns);
    };
    if (found.seq < 0) return leave();  // more CTAs than tiles and slices
    const int b = found.seq, tile = found.tile, h = found.head, rest = found.rest;
    const SeqRows s = load_seq(p, b, nullptr);
    const int rows = s.ql * group, row0 = tile * kRows;
    const bool two = rows - row0 > kRowTile;  // the second row tile has rows
    const TileBounds g = tile_bounds(p, s, row0, min(row0 + kRows, rows) - 1);
    // this CTA's slice of the key tiles: cache blocks from block0 on, `tiles` tiles of 8
    int block0 = g.lo / 16;
    const int block_end = (g.hi + 15) / 16;
    int tiles = block_end > block0 ? (block_end - block0 + 7) / 8 : 0;
    const int slices = min(found.slices, max(1, tiles / kLeastSlice)), slice = found.slice;
    if (slice >= slices) return leave();
    {
        const int t0 = static_cast<int>(static_cast<long long>(tiles) * slice / slices);
        tiles = static_cast<int>(static_cast<long long>(tiles) * (slice + 1) / slices) - t0;
        block0 += 8 * t0;
    }

    float m = -INFINITY, l = 0.f;  // the row's running maximum less kLift (log2 units) and sum
    float f = 0.f;
    int see = 0;
    const bool softmax = warp < kSoftmaxWarps;
    const int row = row0 + tid;
    const bool real = softmax && row < rows;
    auto lse_at = [&]() {
        const int query = divide(row, p.group);
        return static_cast<long long>(s.qs + query) * p.q_heads + h * group + row - query * group;
    };
    // the slices' results in the workspace: of each [column, maximum, sum][row]
    auto parts_of = [&](int sliced) {
        return reinterpret_cast<float*>(static_cast<unsigned char*>(p.workspace) + kAttCounterBytes) +
               static_cast<size_t>(sliced) * found.slices * T::kPartFloats;
    };

    if (warp == kMmaWarp) {
        // ===== MMAs =======================================================================================
        constexpr uint32_t id_s = idesc_f16(kRowTile, kKeys, false), id_o = idesc_f16(kRowTile, D, true);
        const int na = two ? 2 : 1;
        const uint32_t lead = elect_lane();
        // the descriptors of each operand's start; a step adds to the address field (16-byte units) only
        const uint64_t qd = sdesc_sw128(sbase + T::kQ, 16), kd = sdesc_sw128(sbase + T::kK, 16), vd = sdesc_sw128(sbase + T::kV, T::kHalf);
        auto scores = [&](int a, int j) {
            const uint64_t q = qd + static_cast<uint64_t>(a * (T::kTile / 16)), k = kd + static_cast<uint64_t>(j % 2 * (T::kTile / 16));
            const uint32_t d = tmem + static_cast<uint32_t>(a * kKeys);
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
                const uint64_t off = static_cast<uint64_t>((st / 4 * T::kHalf + st % 4 * 32) / 16);
                mma_ss(lead, d, q + off, k + off, id_s, st != 0 ? 1u : 0u);
            }
            commit(lead, s_full(a));
        };
        auto outputs = [&](int a, int j, int half) {
            const uint64_t v = vd + static_cast<uint64_t>(j % 2 * (T::kTile / 16) + half * (64 * 128 / 16));
            const uint32_t d = tmem + static_cast<uint32_t>(T::kO + a * D), w = tmem + static_cast<uint32_t>(a * kKeys + half * 32);
            mma_ts(lead, d, w, v, id_o, j != 0 || half != 0 ? 1u : 0u);
#pragma unroll
            for (int st = 1; st < kKeys / 32; ++st)
                mma_ts(lead, d, w + static_cast<uint32_t>(st * 8), v + static_cast<uint64_t>(st * 2048 / 16), id_o, 1u);
        };
        // Keys and values are waited for right after the scores have been issued, ahead of their use: a wait takes a hundred
        // cycles even where nothing is waited for, and between the weights' arrival and their product it would show.
        if (tiles > 0) {
            wait(q_full, 0);
            wait(k_full(0), 0);
            tc_fence_after();
            for (int a = 0; a < na; ++a) scores(a, 0);
            commit(lead, k_empty(0));
            wait(v_full(0), 0);
            if (tiles > 1) wait(k_full(1), 0);
        }
        for (int j = 0; j < tiles; ++j) {
            for (int a = 0; a < na; ++a) {
                wait(p_full(a, 0), j & 1);
                __syncwarp();
                tc_fence_after();
                outputs(a, j, 0);
                wait(p_full(a, 1), j & 1);
                __syncwarp();
                tc_fence_after();
                outputs(a, j, 1);
                if (a == na - 1) commit(lead, v_empty(j % 2));
                if (j + 1 < tiles) {
                    scores(a, j + 1);
                    if (a == na - 1) commit(lead, k_empty((j + 1) % 2));
                }
            }
            if (j + 1 < tiles) wait(v_full((j + 1) % 2), (j + 1) / 2 & 1);
            if (j + 2 < tiles) wait(k_full(j % 2), (j + 2) / 2 & 1);
        }
        commit(lead, o_full);
        if (lead) wait.drain(o_full, 0);
        __syncwarp();
    } else if (!softmax) {
        // ===== dequantising: warp w takes blocks 2w and 2w + 1 of each key tile ============================
        const int w = warp - kSoftmaxWarps, r = lane / 4, c = lane % 4;
        const int* table = p.page_table + static_cast<long long>(b) * p.max_pages;
        const unsigned char* src[kBlocksPerWarp];  // of the tile whose words are being loaded; null: nothing there
        bool there[kBlocksPerWarp];
        int pages[kBlocksPerWarp];  // lane i: the page entries of tile 32 k + i; -2: behind the last block
        BlockRegs<D> x[kBlocksPerWarp] = {};
        auto place = [&](int j) {  // in order of j
            if (j % 32 == 0) {
                // 32 tiles' entries at once: a load a tile would wait, with its tile, for the codes that are on their way
#pragma unroll
                for (int i = 0; i < kBlocksPerWarp; ++i) {
                    const int blk = block0 + 8 * (j + lane) + kBlocksPerWarp * w + i;
                    pages[i] = j + lane < tiles && blk < block_end ? __ldg(table + (blk * 16 >> p.s.page_shift)) : -2;
                }
            }
#pragma unroll
            for (int i = 0; i < kBlocksPerWarp; ++i) {
                src[i] = nullptr;
                const int page = __shfl_sync(0xFFFFFFFFu, pages[i], j % 32);
                if (page == -2) continue;
                if (page < 0 || page >= p.s.pages) {
                    if (lane == 0) atomicOr(&g_hc_tiles_error, kErrPage);
                    continue;
                }
                const int tok = (block0 + 8 * j + kBlocksPerWarp * w + i) * 16;
                src[i] = p.cache + (((static_cast<long long>(page) * kv_heads.by + h) << (p.s.page_shift - 4)) +
                                    ((tok & ((1 << p.s.page_shift) - 1)) >> 4)) * kv_block_bytes(D);
            }
        };
        auto fetch_keys = [&]() {
#pragma unroll
            for (int i = 0; i < kBlocksPerWarp; ++i) {
                if (!src[i]) {  // zeros: codes of 0 with the scale 0
#pragma unroll
                    for (int q = 0; q < D / 64; ++q) x[i].k[q] = make_uint4(0, 0, 0, 0);
                    x[i].ks = 0;
                    continue;
                }
#pragma unroll
                for (int q = 0; q < D / 64; ++q) x[i].k[q] = *reinterpret_cast<const uint4*>(src[i] + q * 512 + lane * 16);
                if constexpr (D == 64) x[i].ks = *reinterpret_cast<const uint16_t*>(src[i] + KvPlace<D>::kKeyScales + lane * 2);
                else x[i].ks = *reinterpret_cast<const uint32_t*>(src[i] + KvPlace<D>::kKeyScales + lane * 4);
            }
        };
        auto fetch_values = [&]() {
#pragma unroll
            for (int i = 0; i < kBlocksPerWarp; ++i) {
                if (!src[i]) {
#pragma unroll
                    for (int q = 0; q < D / 64; ++q) x[i].v[q] = make_uint4(0, 0, 0, 0);
                    x[i].vs = 0;
                    continue;
                }
#pragma unroll
                for (int q = 0; q < D / 64; ++q)
                    x[i].v[q] = *reinterpret_cast<const uint4*>(src[i] + KvPlace<D>::kValueCodes + q * 512 + lane * 16);
                x[i].vs = *reinterpret_cast<const uint32_t*>(src[i] + KvPlace<D>::kValueScales + (r * (D / 8) / 16 * 4 + c) * 4);
            }
        };
        place(0);
        fetch_keys();
        fetch_values();
        for (int j = 0; j < tiles; ++j) {
            const int st = j % 2, note = j % kNotes;
            const uint32_t parity = static_cast<uint32_t>((j / 2 & 1) ^ 1);
            const int tok0 = (block0 + 8 * j) * 16;
            const bool whole = tok0 >= g.all_lo && tok0 + kKeys <= g.all_hi;
#pragma unroll
            for (int i = 0; i < kBlocksPerWarp; ++i) there[i] = src[i] != nullptr;
            place(j + 1);
            // keys: tokens r and r + 8, columns [c D/4, (c+1) D/4): 16-byte chunks of 8 columns
            if (j >= 2) wait(k_empty(st), parity);
#pragma unroll
            for (int i = 0; i < kBlocksPerWarp; ++i) {
                // 16-byte chunk e of the lane's columns goes to chunk (c D/32 + e) ^ r of its row. The two 64-column halves lie in
                // the same banks: lanes of the second take each pair of chunks (two words of codes each) the other way round.
                const bool swap = D > 64 && c >= 2;
                const uint32_t base = sbase + T::kK + static_cast<uint32_t>(st * T::kTile + (16 * (kBlocksPerWarp * w + i) + r) * 128 +
                                                                            c * (D / 32) / 8 * T::kHalf);
                const uint32_t at = static_cast<uint32_t>((c * (D / 32) % 8 ^ r ^ (swap ? 1 : 0)) << 4);
                const uint32_t h0 = e4m3x2_to_f16(x[i].ks & 0xFFFFu), h1 = D == 64 ? h0 : e4m3x2_to_f16(x[i].ks >> 16);
#pragma unroll
                for (int q = 0; q < D / 64; ++q) {
                    const uint4 k = x[i].k[q];
                    const uint32_t wd[4] = {swap ? k.z : k.x, swap ? k.w : k.y, swap ? k.x : k.z, swap ? k.y : k.w};
                    const int i0 = D == 64 ? 0 : q, i1 = D == 64 ? 1 : q;
                    const uint32_t s0 = __byte_perm(h0, 0, i0 ? 0x3232 : 0x1010), s1 = __byte_perm(h1, 0, i1 ? 0x3232 : 0x1010);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t t[8];
                        e2m1_word_to_f16(wd[2 * e], t[0], t[1], t[4], t[5]);
                        e2m1_word_to_f16(wd[2 * e + 1], t[2], t[3], t[6], t[7]);
                        const uint32_t to = base + (at ^ static_cast<uint32_t>((2 * q + e) << 4));
                        st_smem_v4(to, make_uint4(mul_f16x2(t[0], s0), mul_f16x2(t[1], s0), mul_f16x2(t[2], s0), mul_f16x2(t[3], s0)));
                        st_smem_v4(to + 1024, make_uint4(mul_f16x2(t[4], s1), mul_f16x2(t[5], s1), mul_f16x2(t[6], s1), mul_f16x2(t[7], s1)));
                    }
                }
            }
            fetch_keys();  // tile j + 1's
            if (lane == 0) {
                // tile j + 2's note, which no warp can write before this one arrives below, and whose last reader was
                // tile j + 2 - kNotes: scores of tile j - 2 are done, so every softmax up to tile j - 3 is
                if (w == 0) nan_any[(j + 2) % kNotes] = 0;
                uint32_t off = 0;
#pragma unroll
                for (int i = 0; i < kBlocksPerWarp; ++i) off |= there[i] ? 0u : 1u << i;
                absent[note][w] = static_cast<uint8_t>(off);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(k_full(st));
            // values: tokens 2c, 2c+1, 2c+8, 2c+9, columns [r D/8, (r+1) D/8)
            if (j >= 2) wait(v_empty(st), parity);
#pragma unroll
            for (int i = 0; i < kBlocksPerWarp; ++i) {
                const int blk = kBlocksPerWarp * w + i;
                uint32_t s4 = x[i].vs;
                if (!whole) {
                    // a NaN scale must not reach rows that do not see the token: 0 here, noted for the rows that do
                    uint16_t* notes = reinterpret_cast<uint16_t*>(smem + T::kNan) + note * kKeys + 16 * blk;
                    uint32_t bad = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (there[i] && (s4 >> (8 * e) & 0x7Fu) == 0x7Fu) {
                            bad |= 1u << e;
                            s4 &= ~(0xFFu << (8 * e));
                        }
                    if (lane < 16) notes[lane] = 0;
                    __syncwarp();
                    if (__any_sync(0xFFFFFFFFu, bad != 0)) {
                        const int kb = r * (D / 8) / 16;
                        // lanes of one c hold the groups of the same tokens, in turn
                        for (int y = 0; y < 8; ++y) {
                            if (r == y && bad)
                                for (int e = 0; e < 4; ++e)
                                    if (bad >> e & 1) notes[2 * c + e % 2 + 8 * (e / 2)] |= static_cast<uint16_t>(1u << kb);
                            __syncwarp();
                        }
                        if (lane == 0) nan_any[note] = 1;
                    }
                }
                // chunk q of the lane's columns goes to chunk (r D/64 + q) ^ (token % 8) of the token's row; odd r take their two
                // chunks the other way round, or they would meet r ^ 1 in the banks
                const bool swap = D > 64 && r % 2 != 0;
                const uint32_t base = sbase + T::kV + static_cast<uint32_t>(st * T::kTile + 16 * blk * 128 + r * (D / 64) / 8 * T::kHalf);
                const uint32_t at = static_cast<uint32_t>((r * (D / 64) % 8 ^ (swap ? 1 : 0)) << 4);
                const uint32_t sp0 = e4m3x2_to_f16(s4 & 0xFFFFu), sp1 = e4m3x2_to_f16(s4 >> 16);
                const uint32_t sc[4] = {__byte_perm(sp0, 0, 0x1010), __byte_perm(sp0, 0, 0x3232), __byte_perm(sp1, 0, 0x1010),
                                        __byte_perm(sp1, 0, 0x3232)};
#pragma unroll
                for (int q = 0; q < D / 64; ++q) {
                    const uint4 k0 = x[i].v[q], k1 = x[i].v[D > 64 ? q ^ 1 : q];
                    const uint32_t wd[4] = {swap ? k1.x : k0.x, swap ? k1.y : k0.y, swap ? k1.z : k0.z, swap ? k1.w : k0.w};
                    uint32_t y[4][4];  // [token][pairs of columns]
#pragma unroll
                    for (int m = 0; m < 4; ++m) e2m1_word_to_f16(wd[m], y[0][m], y[1][m], y[2][m], y[3][m]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = 2 * c + e % 2 + 8 * (e / 2);
                        st_smem_v4(base + static_cast<uint32_t>(t * 128) + (at ^ static_cast<uint32_t>((q ^ t % 8) << 4)),
                                   make_uint4(mul_f16x2(y[e][0], sc[e]), mul_f16x2(y[e][1], sc[e]), mul_f16x2(y[e][2], sc[e]),
                                              mul_f16x2(y[e][3], sc[e])));
                    }
                }
            }
            fetch_values();  // tile j + 1's
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(v_full(st));
        }
    } else {
        // ===== softmax ========================================================================================
        {
            // the warp's 32 rows of queries, kLanes lanes a row; thread i takes row i afterwards
            const int e = lane % kLanes;  // 16-byte chunk of the row
            const uint32_t base = sbase + T::kQ + static_cast<uint32_t>(warp / 4 * T::kTile + e / 8 * T::kHalf);
            uint4 x[kLanes];
#pragma unroll
            for (int k = 0; k < kLanes; ++k) {
                const int y = row0 + 32 * warp + k * kSide + lane / kLanes, i = divide(y, p.group);
                x[k] = make_uint4(0, 0, 0, 0);
                if (y < rows)
                    x[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + static_cast<long long>(s.qs + i) * p.q_stride +
                                                                static_cast<long long>(h * group + y - i * group) * D) + e);
            }
#pragma unroll
            for (int k = 0; k < kLanes; ++k) {
                uint32_t big = __vmaxu2(__vmaxu2(x[k].x & 0x7FFF7FFFu, x[k].y & 0x7FFF7FFFu), __vmaxu2(x[k].z & 0x7FFF7FFFu, x[k].w & 0x7FFF7FFFu));
                big = max(big & 0xFFFFu, big >> 16);
#pragma unroll
                for (int o = 1; o < kLanes; o *= 2) big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, o));
                float up, down;
                row_scale(big, up, down);
                const float fr = __shfl_sync(0xFFFFFFFFu, down, lane % kSide * kLanes);  // of row lane % kSide of these
                if (lane / kSide == k) f = p.scale * kLog2e * p.s.k_unit * fr;
                const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                uint32_t o[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) o[y] = pack_f16(__uint_as_float(w[y] << 16) * up, __uint_as_float(w[y] & 0xFFFF0000u) * up);
                const int i = 32 * (warp % 4) + k * kSide + lane / kLanes;  // row of the row tile
                st_smem_v4(base + static_cast<uint32_t>(i * 128 + ((e % 8 ^ i % 8) << 4)), make_uint4(o[0], o[1], o[2], o[3]));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
            see = p.causal ? (real ? max(s.kvl - s.ql + divide(row, p.group) + 1, 0) : 0) : s.kvl;
        }
        const int a = warp / 4;
        if (a == 0 || two) {
            const uint32_t quad = tmem + (static_cast<uint32_t>(warp % 4 * 32) << 16);
            const uint32_t ts = quad + static_cast<uint32_t>(a * kKeys), to = quad + static_cast<uint32_t>(T::kO + a * D);
            uint32_t nan_groups = 0;
            const int low = p.window > 0 ? see - p.window : 0, high = min(see, s.kvl);
            for (int j = 0; j < tiles; ++j) {
                wait(s_full(a), j & 1);
                tc_fence_after();
                const int tok0 = (block0 + 8 * j) * 16;
                uint32_t gone = *reinterpret_cast<volatile uint32_t*>(&absent[j % kNotes]);  // the four warps' bytes, two bits each
                if (gone) gone = (gone & 3u) | (gone >> 6 & 12u) | (gone >> 12 & 48u) | (gone >> 18 & 192u);
                const bool whole = tok0 >= g.all_lo && tok0 + kKeys <= g.all_hi && gone == 0;
                // this row sees columns [from, upto) of the tile, but for blocks that are not there
                const int from = low - tok0, upto = high - tok0;
                uint32_t seen[kKeys / 32] = {};
                float top;
                if (whole) {
                    top = largest<false>(ts, seen);
                } else {
#pragma unroll
                    for (int q = 0; q < kKeys / 32; ++q) seen[q] = seen_columns(q, from, upto, gone);
                    top = largest<true>(ts, seen);
                }
                top = top == -INFINITY ? top : top * f;  // (f may be 0)
                if (__any_sync(0xFFFFFFFFu, top > m + kSlack)) {
                    const float m2 = fmaxf(m, top - kLift);
                    const float fade = m2 == -INFINITY ? 1.f : ex2(m - m2);
                    m = m2;
                    l *= fade;
                    if (j > 0) {
                        float v[32];
#pragma unroll
                        for (int q = 0; q < D / 32; ++q) {
                            tmem_ld32(to + static_cast<uint32_t>(32 * q), v);
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] *= fade;
                            tmem_st32(to + static_cast<uint32_t>(32 * q), v);
                        }
                    }
                }
                if (!whole) {
                    // The notes are complete with the tile's values, which may come after its scores. (Before the weights are handed
                    // over: after that the values' stage may be filled anew, and its barrier go on to another phase.)
                    wait(v_full(j % 2), j / 2 & 1);
                    if (*reinterpret_cast<volatile uint32_t*>(&nan_any[j % kNotes])) {
                        const uint16_t* notes = reinterpret_cast<const uint16_t*>(smem + T::kNan) + j % kNotes * kKeys;
                        for (int n = max(from, 0); n < min(upto, kKeys); ++n) nan_groups |= notes[n];
                    }
                }
                const float shift = m == -INFINITY ? 0.f : -m;
                uint64_t sum = pair(0.f, 0.f);
                // half by half: the second product of the first 64 keys starts while the weights of the others are made
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (whole) weights<false>(ts, half, f, shift, seen, sum);
                    else weights<true>(ts, half, f, shift, seen, sum);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full(a, half));
                }
                float x, y;
                unpair(sum, x, y);
                l += x + y;
            }
            // ---- results -----------------------------------------------------------------------------------
            float* mine = parts_of(rest) + static_cast<size_t>(slice) * T::kPartFloats;
            if (tiles > 0) wait(o_full, 0);
            tc_fence_after();
            if (slices > 1) griddep_wait();  // the kernel ahead may use the workspace
            const bool nan_row = __any_sync(0xFFFFFFFFu, nan_groups != 0);
            const float scale = slices > 1 ? 1.f : l == 0.f ? 0.f : p.s.v_unit / l;
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
                float v[32];
                if (tiles > 0) {
                    tmem_ld32(to + static_cast<uint32_t>(32 * q), v);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= scale;  // a row that sees nothing has zeros here and the scale 0
                if (nan_row) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (nan_groups >> (2 * q + i / 16) & 1) v[i] = __uint_as_float(0x7FC00000u);
                }
                if (slices == 1) {
                    // to where the row's queries were (all MMAs that read them are done), to be written by whole rows
                    const int i = tid % kRowTile;
                    const uint32_t to_row = sbase + T::kQ + static_cast<uint32_t>(a * T::kTile + q / 2 * T::kHalf + i * 128);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        uint32_t w[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const __nv_bfloat162 t = __floats2bfloat162_rn(v[8 * y + 2 * z], v[8 * y + 2 * z + 1]);
                            w[z] = *reinterpret_cast<const uint32_t*>(&t);
                        }
                        st_smem_v4(to_row + static_cast<uint32_t>((q % 2 * 4 + y ^ i % 8) << 4), make_uint4(w[0], w[1], w[2], w[3]));
                    }
                } else if (real) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) mine[(32 * q + i) * kRows + tid] = v[i];
                }
            }
            if (slices == 1) {
                __syncwarp();
                const int e = lane % kLanes;
                const uint32_t from = sbase + T::kQ + static_cast<uint32_t>(a * T::kTile + e / 8 * T::kHalf);
#pragma unroll
                for (int k = 0; k < kLanes; ++k) {
                    const int in = k * kSide + lane / kLanes, i = 32 * (warp % 4) + in, y = row0 + 32 * warp + in, j = divide(y, p.group);
                    if (y >= rows) continue;
                    const uint4 w = ld_smem_v4(from + static_cast<uint32_t>(i * 128 + ((e % 8 ^ i % 8) << 4)));
                    reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + static_cast<long long>(s.qs + j) * p.out_stride +
                                             static_cast<long long>(h * group + y - j * group) * D)[e] = w;
                }
            }
            if (real && slices == 1 && p.lse) p.lse[lse_at()] = log_sum_exp(m, l);
            if (real && slices > 1) {
                mine[D * kRows + tid] = m;
                mine[(D + 1) * kRows + tid] = l;
            }
        }
    }
    if (slices > 1) {
        // The slices of a row tile are joined by the CTA that finishes last, in their order.
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            unsigned int* counter = static_cast<unsigned int*>(p.workspace) + rest;
            last_flag = atomicAdd(counter, 1u) + 1 == static_cast<unsigned int>(slices);
            if (last_flag) *counter = 0;
            __threadfence();
        }
        __syncthreads();
        if (last_flag && real) {
            const float* from = parts_of(rest) + tid;
            const int query = divide(row, p.group);
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + static_cast<long long>(s.qs + query) * p.out_stride +
                                 static_cast<long long>(h * group + row - query * group) * D;
            float top = -INFINITY;
#pragma unroll 4
            for (int x = 0; x < slices; ++x) top = fmaxf(top, __ldcg(from + x * static_cast<size_t>(T::kPartFloats) + D * kRows));
            const float base = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
#pragma unroll 4
            for (int x = 0; x < slices; ++x) {
                const float* part = from + x * static_cast<size_t>(T::kPartFloats);
                sum = fmaf(__ldcg(part + (D + 1) * kRows), ex2(__ldcg(part + D * kRows) - base), sum);
            }
            const float scale = sum == 0.f ? 0.f : p.s.v_unit / sum;
            for (int q = 0; q < D / 32; ++q) {
                float v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0.f;
#pragma unroll 2
                for (int x = 0; x < slices; ++x) {
                    const float* part = from + x * static_cast<size_t>(T::kPartFloats);
                    const float w = ex2(__ldcg(part + D * kRows) - base);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = fmaf(w, __ldcg(part + (32 * q + i) * kRows), v[i]);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= scale;
                store32(dst + 32 * q, v);
            }
            if (p.lse) p.lse[lse_at()] = log_sum_exp(top, sum);
        }
    }
    griddep_wait();  // the call has ended when both kernels have
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, T::kColumns);
    }
}

// CTAs that a call's row tiles need at most: each of its sequences may end inside one.
long long tiles_bound(const AttArgs& a) {
    const long long most = a.q_min > 1 ? a.n / a.q_min : a.n;
    return (a.n * (a.q_heads / a.s.heads) / kRows + (a.seqs < most ? a.seqs : most)) * a.s.heads;
}

template <int D>
int launch_tiles(const AttArgs& a, cudaStream_t stream) {
    using T = TilePlan<D>;
    static std::mutex mu;
    static bool done[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -7;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!done[dev]) {
            if (cudaFuncSetAttribute(attend_tiles_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem) != cudaSuccess) return -7;
            done[dev] = true;
        }
    }
    static_assert(static_cast<size_t>(T::kPartFloats) * kAttMaxSlices <= kAttPartFloatsTotal, "the slices' results fit the workspace");
    const long long grid = tiles_bound(a);
    if (grid == 0) return 0;  // no sequence can have q_min queries
    const int sms = attn_sm_count();
    if (sms == 0) return -7;
    // Behind a launch for the sequences of few queries this kernel may start before that one has ended: it reads
    // nothing of it, and waits for it before it touches the workspace.
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid + sms));  // slices take fewer than sms more
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = T::kSmem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = a.q_min > 0 ? 1 : 0;
    g_launched.store(true, std::memory_order_relaxed);
    return cudaLaunchKernelEx(&cfg, attend_tiles_kernel<D>, a, make_divider(sms), make_divider(a.s.heads)) == cudaSuccess ? 0 : -7;
}

}  // namespace

bool attention_tiles_take(const AttArgs& a) { return a.s.dim <= 128 && tiles_bound(a) <= 0x7FFF0000LL; }

int launch_attention_tiles(const AttArgs& a, cudaStream_t stream) {
    return a.s.dim == 64 ? launch_tiles<64>(a, stream) : launch_tiles<128>(a, stream);
}

int read_tiles_error(unsigned int* word, int clear, cudaStream_t stream) {
    unsigned int v = 0;
    *word = 0;
    if (!g_launched.load(std::memory_order_relaxed)) return 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_hc_tiles_error, sizeof(v), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return -7;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return -7;
    if (clear && v != 0) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbolAsync(g_hc_tiles_error, &z, sizeof(z), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess) return -7;
        if (cudaStreamSynchronize(stream) != cudaSuccess) return -7;
    }
    *word = v;
    return 0;
}

}  // namespace hc
