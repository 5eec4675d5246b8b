// Softmax attention of ragged queries over the 4-bit cache (formulas, masks and format: include/hc.h).
//
// The rows of a sequence and a kv head are its queries times the group of query heads that share the kv head
// (row = query * group + head in the group): they read the same keys, so a tile takes R = 8 kNT of them at once
// and the products go to mma.sync.m16n8k16 with the cache as the A operand (16 tokens, or 16 columns, by 16)
// and the rows as the 8 columns of B: a tile of few rows wastes nothing, and A comes straight from registers.
// The tensor memory path (tcgen05) would have to write every dequantised block to shared memory first, 8 times
// the bytes that the cache has; this kernel's bound is the dequantisation and HBM, not the products.
//
// Measured: 256 sequences of 2,050 to 4,096 keys, 40 query and 8 kv heads of 128 (912 MB): 202 us, 4.5 TB/s, 67% of the
// measured copy rate; 3 sequences of up to 131,072 keys: 84 us, 67%; 8 of up to 509 keys: 8.1 us. With few rows nothing is
// full: a unit of 32 keys of a head takes about 600 instructions (128 conversions from 4 bits, about as many products with
// scales, 32 MMAs) in a chain of scores, maximum, weights and values whose fixed latencies 16 warps an SM cover in part:
// issue slots about 60% busy, no pipe above half. In an earlier form that took 215 us, leaving out the keys' scale products
// saved 7 us; two warps a unit took 258 us, blocks of 4 warps 255 us. Heads of 256 come here for prefills too, 16 rows a
// tile, which dequantises the keys for each of them: 2 x 2,048 queries behind 4,096 to 6,144 keys, 40 and 8 heads, 4,850 us,
// nine times their products at the measured cuBLAS rate. More rows cost more of everything: five queries of 4
// heads each, 64 sequences, window of 1,024 keys (81 MB): 54 us.
//
// A cache block (16 tokens, one head) is laid out in A-fragment order: lane (r, c) = (lane / 4, lane % 4) finds
// in its own 32-bit words the codes of keys r and r + 8, columns [c D/4, (c+1) D/4) (the contraction index of
// the product may run in any order, so a lane takes whole 16-column groups and needs few scales), and of values
// 2c, 2c+1, 2c+8, 2c+9, columns [r D/8, (r+1) D/8). A word becomes four fp16 pairs (cvt from e2m1x2), times its
// scale (exact in fp16). S^T = K Q^T leaves lane (r, c) the scores of tokens r, r + 8 and rows 2c, 2c + 1; the
// weights, rounded to fp16, are turned into the second product's B fragment by movmatrix.
//
// The softmax keeps a running maximum (less a constant: kLift) and sum per row. The maximum is raised only when a score
// exceeds it by more than 2^8 (weights then stay below 2^15, inside fp16), so that most steps need no exchange between
// lanes and no rescaling of the sums. Sums, maxima and outputs are fp32; the weights are rounded to fp16: by 2^-11 of
// themselves at most down to 2^-21 of the row's largest, by 2^-32 of the largest below, well below the bf16 rounding of
// the result.
//
// Work. All the (sequence, kv head, tile of rows) segments of a call, each so many units of 32 tokens, are laid
// end to end and cut into equal ranges, one a CTA, whatever the lengths. The warps of a CTA take its units in
// turn, each with a ring of cache blocks of its own, filled by bulk copies that the warp issues ahead; they join
// at the end of a segment. A segment cut between CTAs leaves partial results in the workspace, and the CTA that
// finishes last joins them in their order: the result does not depend on timing. Where a cut would cost more than it
// evens out, segments stay whole (kJoinSteps).

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

__device__ unsigned int g_hc_attention_error = 0;
std::atomic<bool> g_launched{false};  // whether the word above can be set at all (reading it costs a copy and a wait)

constexpr uint64_t kWaitNs = 1000000000ull;   // 1 s
constexpr int kUnit = 32;                     // tokens a warp takes at a time: two cache blocks
// What it costs a CTA to have segments cut, in steps of its teams: left whole, they may take so many steps longer. 64 sequences
// of 5 queries with a window of 1,024 keys, 18 steps whole, 14 cut: 56 us whole, 63 us cut; 128 of up to 1,000 keys: 49 and
// 53 us; 128 of up to 509: 34 and 42 us. At 11, 40 sequences with that window (18 and 8 steps): 55 us whole, 42 us cut.
constexpr int kJoinSteps = 9;
constexpr int kMaxDevices = 64;
// Rows of the longest sequence from which hc_attend_tiles.cu takes a call: more than this kernel's largest tile of rows
// reads and dequantises the keys twice. 64 sequences of up to 4,096 keys, 28 rows: 143 us here, 195 us there; 64 of up to
// 1,000 keys, 40 rows: 104 against 80 us; 32 of up to 4,096 keys, 96 rows: 107 against 62 us. (One sequence alone would be
// better off here for longer: 40 rows over 32,768 keys, 54 against 80 us.)
constexpr long long kTilesFromRows = 33;

// The shape of a CTA. A team of kSplit warps takes a unit at a time: alone (kSplit = 1), or two warps that share it, each
// the scores of one of its two blocks and then half the output columns for both, the weights exchanged through
// shared memory. Two halve the registers of the outputs, so that 16 warps an SM still fit with more rows or columns.
template <int D, int kNT, int kSplit_>
struct Plan {
    static constexpr int kSplit = kSplit_;
    static constexpr int kWarps = D == 256 ? 4 : 8;
    static constexpr int kTeams = kWarps / kSplit;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kCtas = D == 256 ? (kSplit == 1 ? 2 : 3) : 2;
    static constexpr int kLogStages = D == 64 ? 2 : 1;  // of a team's ring, one unit each
    static constexpr int kStages = 1 << kLogStages;
    static constexpr int kStage = kUnit / 16 * kv_block_bytes(D);
    static constexpr int kRing = kTeams * kStages * kStage;
    static constexpr int kTiles = D / 16 / kSplit;              // 16-column tiles of the output a warp
    // The outputs are joined in so many passes, so that shared memory holds two CTAs an SM or more, and the L1 cache gets a part
    // of it: with kTiles * kNT = 12, 58.2 us in one pass, 55.7 us in two (5 queries of 4 heads, 64 sequences, window of 1,024
    // keys); with 8, 209.7 us in one, 213.3 us in two (one query of 5 heads, 256 sequences of up to 4,096 keys).
    static constexpr int kPasses = kTiles * kNT >= 12 ? 2 : 1;
    static constexpr int kPassTiles = kTiles / kPasses;
    static constexpr int kStateFloats = kPassTiles * kNT * 4 * 32;  // a warp's outputs of a pass
    static constexpr int kMl = 2 * 8 * kNT;                         // its maxima and sums
    static constexpr int kMerge = kWarps * (kStateFloats + kMl) * 4;
    static constexpr int kQ = kSplit == 1 ? 0 : kNT * (D / 16) * 32 * 8;            // the queries as B fragments
    static constexpr int kWeights = kSplit == 1 ? 0 : kTeams * 2 * 2 * kNT * 2 * 128;  // [team][step parity][block][fragment]
    static constexpr int kRows = kSplit == 1 ? 0 : (2 + 2 * kTeams) * 8 * kNT * 4;  // score factors; ends of what rows see; a team's exchange of maxima
    static constexpr int kBars = kTeams * kStages * 8;
    static constexpr int kSmem = kRing + kMerge + kQ + kWeights + kRows + kBars;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// (a.low * s.low, b.low * t.high), where s.high and t.low are 0: two pairs of columns of two tokens become a pair of
// tokens of one column, scaled. A permutation and a product would do as well, but permutations share their pipe with
// the conversions, which is the fuller one (exact either way: one term of the sum is 0).
__device__ __forceinline__ uint32_t weave(__half2 a, uint32_t s, __half2 b, uint32_t t) {
    const __half2 r = __hfma2(a, *reinterpret_cast<const __half2*>(&s), __hmul2(b, *reinterpret_cast<const __half2*>(&t)));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t weave_low(uint32_t a, uint32_t s, uint32_t b, uint32_t t) {
    return weave(__low2half2(*reinterpret_cast<const __half2*>(&a)), s, __low2half2(*reinterpret_cast<const __half2*>(&b)), t);
}
__device__ __forceinline__ uint32_t weave_high(uint32_t a, uint32_t s, uint32_t b, uint32_t t) {
    return weave(__high2half2(*reinterpret_cast<const __half2*>(&a)), s, __high2half2(*reinterpret_cast<const __half2*>(&b)), t);
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void lds64(uint32_t a, uint32_t& x, uint32_t& y) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(a) : "memory");
}
// Barriers of a team's two warps (named barrier `id`).
__device__ __forceinline__ void pair_sync(int id) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool pair_any(int id, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %2, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(static_cast<uint32_t>(x))
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void wait_copy(uint32_t bar, uint32_t parity) {
    if (mbar_sleep(bar, parity)) return;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (mbar_sleep(bar, parity)) return;
        if (global_timer_ns() - t0 > kWaitNs) {
            atomicOr(&g_hc_attention_error, kErrCopy);
            return;
        }
    }
}

// ---- sequences and their work -----------------------------------------------------------------------

template <int R>
struct Work {
    int tiles, units;  // tiles of rows, units of each tile
    __device__ __forceinline__ Work(const AttArgs& p, const SeqRows& s, int group) {
        const long long rows = static_cast<long long>(s.ql) * group;
        tiles = static_cast<int>((rows + R - 1) / R);
        units = (s.kvl + kUnit - 1) / kUnit;
        if (p.window > 0) {
            // a tile's queries span so many positions at most; its first unit may begin up to 31 tokens early
            const int span = min(s.ql, (R - 1) / group + 2);
            const long long most = (static_cast<long long>(p.window) + span - 1 + 2 * (kUnit - 1)) / kUnit;
            if (most < units) units = static_cast<int>(most);
        }
        if (units < 1) units = 1;  // a tile without keys still writes its zeros
    }
    __device__ __forceinline__ long long total(int heads) const { return static_cast<long long>(tiles) * heads * units; }
};

// A CTA's part of one segment.
struct Segment {
    int b, h, tile, u0, u1, units;
    SeqRows s;
    int lo, hi, all_lo, all_hi;  // TileBounds
    int first_block, end_block;  // this part's cache blocks
};

template <int D, int kNT, int kSplit>
__global__ void __launch_bounds__(Plan<D, kNT, kSplit>::kThreads, Plan<D, kNT, kSplit>::kCtas) attend_rows_kernel(const AttArgs p) {
    using P = Plan<D, kNT, kSplit>;
    constexpr int kWarps = P::kWarps, kThreads = P::kThreads, kTeams = P::kTeams, kTiles = P::kTiles;
    constexpr int kOwn = 2 / kSplit;        // blocks of a unit whose scores a warp takes
    constexpr int R = 8 * kNT;
    constexpr int kKeySteps = D / 16;  // MMAs over a key's columns; also the 16-column tiles of the output
    constexpr int kBlock = kv_block_bytes(D);
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long scan[kWarps + 1];
    __shared__ int longest[kWarps];
    __shared__ long long found_at;
    __shared__ int found_seq;
    __shared__ int last_flag;
    const int tid = static_cast<int>(threadIdx.x), warp = tid / 32, lane = tid % 32;
    const int r = lane / 4, c = lane % 4;
    const int heads = p.s.heads, group = p.group.by;
    const int team = warp / kSplit, part = warp % kSplit;
    const uint32_t ring = smem_u32(smem) + static_cast<uint32_t>(team * P::kStages * P::kStage);
    float* merge = reinterpret_cast<float*>(smem + P::kRing);
    const uint32_t queries = smem_u32(smem) + P::kRing + P::kMerge;
    const uint32_t exchanged = queries + P::kQ + static_cast<uint32_t>(team * (P::kWeights / kTeams));
    float* factors = reinterpret_cast<float*>(smem + P::kRing + P::kMerge + P::kQ + P::kWeights);
    float* shared_rows = factors + 2 * R + team * 2 * R;  // [part][row]
    const uint32_t bars = smem_u32(smem) + P::kSmem - P::kBars + static_cast<uint32_t>(team * P::kStages * 8);
    if (part == 0 && lane < P::kStages) mbar_init(bars + 8u * static_cast<uint32_t>(lane), 1);
    fence_mbar_init();
    auto team_sync = [&]() {
        if constexpr (kSplit == 1) __syncwarp();
        else pair_sync(1 + team);
    };

    // ---- this CTA's range of the call's units ----------------------------------------------------------
    auto block_scan = [&](long long v, long long& sum) {  // inclusive, over the block's threads
        long long x = v;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = x;
        __syncthreads();
        sum = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) x += scan[w];
            sum += scan[w];
        }
        return x;
    };
    // The tiles' kernel comes behind this one (launch_attention): its CTAs may move in as soon as SMs are free.
    if (p.q_max != kAnyQueries) griddep_launch_dependents();
    // A sequence's segments, and its units where segments may be cut.
    long long segments = 0, units = 0;
    int most = 0;  // units of the longest segment
    for (int b = tid; b < p.seqs; b += kThreads) {
        const Work<R> w(p, load_seq(p, b, blockIdx.x == 0 ? &g_hc_attention_error : nullptr), group);
        segments += static_cast<long long>(w.tiles) * heads;
        units += w.total(heads);
        if (w.tiles > 0) most = max(most, w.units);
    }
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (lane == 0) longest[warp] = most;
    long long all_units, all_segments;
    const long long xs = block_scan(segments, all_segments), xu = block_scan(units, all_units);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) most = max(most, longest[w]);
    // Segments are left whole, one after the other, where joining their parts would cost more than uneven shares.
    const long long grid = gridDim.x;
    const bool whole_ones = (all_segments + grid - 1) / grid * ((most + kTeams - 1) / kTeams) <= all_units / (grid * kTeams) + kJoinSteps;
    const long long total = whole_ones ? all_segments : all_units, x = whole_ones ? xs : xu;
    const long long least = whole_ones ? 1 : kTeams;  // a CTA's smallest share: one unit a team
    const long long want = (total + least - 1) / least;
    // More segments than the call's rows can have come from starts that decrease, and so claim rows again, only: nothing is
    // done (the units of so many might not even be counted in 64 bits).
    const long long ctas = want < grid ? want : grid;
    if (static_cast<long long>(blockIdx.x) >= ctas || all_segments > p.most_segments) return;
    long long at = total * blockIdx.x / ctas;
    const long long end = total * (blockIdx.x + 1) / ctas;
    if (p.seqs <= kThreads) {
        const long long v = whole_ones ? segments : units;
        if (x > at && x - v <= at) {
            found_seq = tid;
            found_at = at - (x - v);
        }
    } else {
        // the sequence that holds unit `at`, a scan of kThreads sequences at a time
        long long before = 0;
        for (int b0 = 0; b0 < p.seqs; b0 += kThreads) {
            const int b = b0 + tid;
            long long v = 0, sum;
            if (b < p.seqs) {
                const Work<R> w(p, load_seq(p, b, nullptr), group);
                v = whole_ones ? static_cast<long long>(w.tiles) * heads : w.total(heads);
            }
            const long long y = block_scan(v, sum) + before;
            if (y > at && y - v <= at) {
                found_seq = b;
                found_at = at - (y - v);
            }
            before += sum;
            if (before > at) break;  // the same in every thread
        }
    }
    __syncthreads();

    Segment g = {};
    // the tile's bounds, from g.s, g.tile, g.u0 and g.u1
    auto place = [&]() {
        const TileBounds t = tile_bounds(p, g.s, g.tile * R, min(g.tile * R + R, g.s.ql * group) - 1);
        g.lo = t.lo;
        g.hi = t.hi;
        g.all_lo = t.all_lo;
        g.all_hi = t.all_hi;
        const int base = g.lo / kUnit * kUnit;
        g.first_block = base / 16 + 2 * g.u0;
        g.end_block = min(base / 16 + 2 * g.u1, (g.hi + 15) / 16);
    };
    {
        g.b = found_seq;
        const long long in = found_at;
        g.s = load_seq(p, g.b, nullptr);
        const Work<R> w(p, g.s, group);
        g.units = w.units;
        const long long k = whole_ones ? in : in / w.units;
        g.u0 = whole_ones ? 0 : static_cast<int>(in - k * w.units);
        g.h = static_cast<int>(k / w.tiles);
        g.tile = static_cast<int>(k - static_cast<long long>(g.h) * w.tiles);
        g.u1 = whole_ones ? w.units : static_cast<int>(min(static_cast<long long>(w.units), g.u0 + (end - at)));
        place();
    }

    // ---- the team's stream of units ----------------------------------------------------------------------
    // Step k of a segment takes unit team + kTeams k of the CTA's part: two cache blocks, one stage of the ring. The lanes look
    // up the blocks of 16 steps at a time (page and address), lane j block j % 2 of step j / 2, and each issues its copy
    // when its step's turn comes (those of the team's first warp; the other warp keeps the same account).
    uint32_t uses = 0;                     // units before this segment's first: step k is use `uses` + k of the ring
    uint32_t there = 0;                    // of the 16 steps looked up: bit j: block j is there
    uint32_t staged = 0;                   // of the units in the ring: bits 2 st, 2 st + 1: the unit's blocks are there
    const unsigned char* where = nullptr;
    int steps = 0, issued = 0;
    auto look_up = [&](int k0) {
        const int blk = g.first_block + 2 * (team + kTeams * (k0 + lane / 2)) + lane % 2;
        where = nullptr;
        if (blk < g.end_block && blk * 16 + 16 > g.lo) {
            const int tok = blk * 16;
            const int page = p.page_table[static_cast<long long>(g.b) * p.max_pages + (tok >> p.s.page_shift)];
            if (page >= 0 && page < p.s.pages)
                where = p.cache + (((static_cast<long long>(page) * heads + g.h) << (p.s.page_shift - 4)) +
                                   ((tok & ((1 << p.s.page_shift) - 1)) >> 4)) * kBlock;
            else
                atomicOr(&g_hc_attention_error, kErrPage);
        }
        there = __ballot_sync(0xFFFFFFFFu, where != nullptr);
    };
    auto issue = [&](int k) {  // in order of k
        if (k % 16 == 0) look_up(k);
        const uint32_t st = (uses + static_cast<uint32_t>(k)) % P::kStages;
        const uint32_t here = there >> (2 * (k % 16)) & 3u;
        staged = (staged & ~(3u << (2 * st))) | here << (2 * st);
        if (part == 0 && lane / 2 == k % 16) {
            const uint32_t bar = bars + 8 * st;
            if (lane % 2 == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(here) * kBlock));
            if (where) bulk_copy(ring + st * P::kStage + static_cast<uint32_t>(lane % 2 * kBlock), where, kBlock, bar);
        }
    };
    auto open = [&]() {  // start the copies of a new segment
        const int units_here = (g.end_block - g.first_block + 1) / 2;
        steps = units_here > team ? (units_here - team + kTeams - 1) / kTeams : 0;
        for (issued = 0; issued < steps && issued < P::kStages; ++issued) issue(issued);
    };
    __syncthreads();  // barriers ready
    open();

    while (true) {
        // ---- the tile's queries ----------------------------------------------------------------------------
        const int rows = g.s.ql * group, row0 = g.tile * R;
        const int pos0 = g.s.kvl - g.s.ql;
        uint32_t qf[kSplit == 1 ? kNT : 1][kKeySteps][2];  // (kSplit = 2: in shared memory)
        float f[kNT][2];   // score factor (log2 units) of rows 2c, 2c + 1 (kSplit = 2: loaded when needed)
        // keys below this position are seen (causal)
        auto sees = [&](int row) { return p.causal ? (row < rows ? max(pos0 + divide(row, p.group) + 1, 0) : 0x7FFFFFFF) : g.s.kvl; };
        auto see = [&](int t, int j) {
            if constexpr (kSplit == 1) return sees(row0 + 8 * t + 2 * c + j);
            else return static_cast<int>(lds32(smem_u32(factors) + static_cast<uint32_t>((R + 8 * t + 2 * c + j) * 4)));
        };
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
            if (kSplit == 2 && t % kWarps != warp) continue;  // one warp makes a tile's fragments for all
            const int row = row0 + 8 * t + r;
            const bool real = row < rows;
            const int query = real ? divide(row, p.group) : 0;
            uint4 x[D / 32];
            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) +
                                       static_cast<long long>(g.s.qs + query) * p.q_stride +
                                       static_cast<long long>(g.h * group + (real ? row - query * group : 0)) * D + c * (D / 4);
#pragma unroll
            for (int e = 0; e < D / 32; ++e) x[e] = real ? __ldg(reinterpret_cast<const uint4*>(src) + e) : make_uint4(0, 0, 0, 0);
            uint32_t big = 0;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                big = __vmaxu2(big, __vmaxu2(__vmaxu2(x[e].x & 0x7FFF7FFFu, x[e].y & 0x7FFF7FFFu),
                                             __vmaxu2(x[e].z & 0x7FFF7FFFu, x[e].w & 0x7FFF7FFFu)));
            }
            big = max(big & 0xFFFFu, big >> 16);
            big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
            big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
            float up, down;
            row_scale(big, up, down);
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                const uint32_t w[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) h[k] = pack_f16(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xFFFF0000u) * up);
                if constexpr (kSplit == 1) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) qf[t][2 * e + k / 2][k % 2] = h[k];
                } else {
#pragma unroll
                    for (int k = 0; k < 4; k += 2)
                        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(queries + static_cast<uint32_t>(((t * kKeySteps + 2 * e + k / 2) * 32 + lane) * 8)),
                                     "r"(h[k]), "r"(h[k + 1])
                                     : "memory");
                }
            }
            const float fr = p.scale * kLog2e * p.s.k_unit * down;
            if constexpr (kSplit == 1) {
#pragma unroll
                for (int j = 0; j < 2; ++j) f[t][j] = __shfl_sync(0xFFFFFFFFu, fr, 4 * (2 * c + j));
            } else {
                if (c == 0) factors[8 * t + r] = fr;
                if (c == 1) factors[R + 8 * t + r] = __int_as_float(sees(row));
            }
        }
        if constexpr (kSplit == 2) __syncthreads();
        float m[kNT][2], l[kNT][2], o[kTiles][kNT][4];
#pragma unroll
        for (int t = 0; t < kNT; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m[t][j] = -INFINITY;
                l[t][j] = 0.f;
            }
#pragma unroll
        for (int k = 0; k < kTiles; ++k)
#pragma unroll
            for (int t = 0; t < kNT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[k][t][e] = 0.f;

        for (int k = 0; k < steps; ++k) {
            const uint32_t use = uses + static_cast<uint32_t>(k), st = use % P::kStages;
            const int blk0 = g.first_block + 2 * (team + kTeams * k);
            const uint32_t slot = ring + st * P::kStage;
            const uint32_t have = staged >> (2 * st) & 3u;
            wait_copy(bars + 8 * st, use >> P::kLogStages & 1);
            // ---- scores of the unit's blocks (kSplit = 2: of block `part`) -------------------------------------
            float z[kOwn][kNT][4];
            uint32_t ks[kOwn][2];  // key scales: tokens r, then r + 8, D / 64 each
            const uint32_t own = slot + static_cast<uint32_t>(kSplit == 1 ? 0 : part * kBlock);
#pragma unroll
            for (int n = 0; n < kOwn; ++n) {
#pragma unroll
                for (int t = 0; t < kNT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[n][t][e] = 0.f;
                const uint32_t at_ = own + static_cast<uint32_t>(n * kBlock + KvPlace<D>::kKeyScales + lane * (D / 32));
                if constexpr (D == 64) {
                    ks[n][0] = lds32(at_ & ~3u) >> (8 * (at_ & 2u)) & 0xFFFFu;
                    ks[n][1] = 0;
                } else {
                    ks[n][0] = lds32(at_);
                    ks[n][1] = D == 256 ? lds32(at_ + 4) : 0;
                }
            }
#pragma unroll
            for (int quad = 0; quad < D / 64; ++quad) {
                uint32_t w[kOwn][4], s0[kOwn], s1[kOwn];
#pragma unroll
                for (int n = 0; n < kOwn; ++n) {
                    const uint4 v = ld_smem_v4(own + static_cast<uint32_t>(n * kBlock + quad * 512 + lane * 16));
                    w[n][0] = v.x;
                    w[n][1] = v.y;
                    w[n][2] = v.z;
                    w[n][3] = v.w;
                    const int i0 = quad, i1 = D / 64 + quad;
                    const uint32_t h0 = e4m3x2_to_f16(ks[n][i0 / 4] >> (16 * (i0 % 4 / 2)) & 0xFFFFu);
                    const uint32_t h1 = e4m3x2_to_f16(ks[n][i1 / 4] >> (16 * (i1 % 4 / 2)) & 0xFFFFu);
                    s0[n] = __byte_perm(h0, 0, i0 % 2 ? 0x3232 : 0x1010);
                    s1[n] = __byte_perm(h1, 0, i1 % 2 ? 0x3232 : 0x1010);
                }
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int n = 0; n < kOwn; ++n) {
                        uint32_t x0, x1, x2, x3;
                        e2m1_word_to_f16(w[n][s], x0, x1, x2, x3);
                        const uint32_t a0 = mul_f16x2(x0, s0[n]), a2 = mul_f16x2(x1, s0[n]), a1 = mul_f16x2(x2, s1[n]), a3 = mul_f16x2(x3, s1[n]);
#pragma unroll
                        for (int t = 0; t < kNT; ++t) {
                            uint32_t b0, b1;
                            if constexpr (kSplit == 1) {
                                b0 = qf[t][quad * 4 + s][0];
                                b1 = qf[t][quad * 4 + s][1];
                            } else {
                                lds64(queries + static_cast<uint32_t>(((t * kKeySteps + quad * 4 + s) * 32 + lane) * 8), b0, b1);
                            }
                            mma_f16(z[n][t], a0, a1, a2, a3, b0, b1);
                        }
                    }
            }
            // ---- masks, running maximum, weights ------------------------------------------------------------
            if constexpr (kSplit == 2) {
#pragma unroll
                for (int t = 0; t < kNT; ++t) {
                    uint32_t x, y;
                    lds64(smem_u32(factors) + static_cast<uint32_t>((8 * t + 2 * c) * 4), x, y);
                    f[t][0] = __uint_as_float(x);
                    f[t][1] = __uint_as_float(y);
                }
            }
            const bool whole = have == 3u && blk0 * 16 >= g.all_lo && blk0 * 16 + kUnit <= g.all_hi;
            if (!whole) {  // scores to their final scale here, so that a masked one stays -infinity whatever the factor
#pragma unroll
                for (int t = 0; t < kNT; ++t)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int upto = see(t, j), hi = min(upto, g.s.kvl), lo = p.window > 0 ? upto - p.window : 0;
#pragma unroll
                        for (int n = 0; n < kOwn; ++n)
#pragma unroll
                            for (int e = j; e < 4; e += 2) {
                                const int in_unit = kSplit == 1 ? n : part;
                                const int pos = (blk0 + in_unit) * 16 + r + 8 * (e / 2);
                                z[n][t][e] = (have >> in_unit & 1) && pos < hi && pos >= lo ? z[n][t][e] * f[t][j] : -INFINITY;
                            }
                    }
            }
            float top[kNT][2];
            bool raise = false;
#pragma unroll
            for (int t = 0; t < kNT; ++t)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = fmaxf(z[0][t][j], z[0][t][2 + j]);
                    if constexpr (kSplit == 1) x = fmaxf(x, fmaxf(z[kOwn - 1][t][j], z[kOwn - 1][t][2 + j]));
                    top[t][j] = x * (whole ? f[t][j] : 1.f);
                    raise |= top[t][j] > m[t][j] + kSlack;
                }
            if constexpr (kSplit == 1) {
                raise = __any_sync(0xFFFFFFFFu, raise);
            } else {
                raise = pair_any(1 + team, raise);
                if (k > 0 && issued < steps) issue(issued++);  // both warps are done with the last step's stage
            }
            if (raise) {
#pragma unroll
                for (int t = 0; t < kNT; ++t)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
#pragma unroll
                        for (int x = 4; x < 32; x *= 2) top[t][j] = fmaxf(top[t][j], __shfl_xor_sync(0xFFFFFFFFu, top[t][j], x));
                        if constexpr (kSplit == 2) {
                            if (r == 0) shared_rows[part * R + 8 * t + 2 * c + j] = top[t][j];
                        }
                    }
                if constexpr (kSplit == 2) {
                    team_sync();
#pragma unroll
                    for (int t = 0; t < kNT; ++t)
#pragma unroll
                        for (int j = 0; j < 2; ++j) top[t][j] = fmaxf(top[t][j], shared_rows[(part ^ 1) * R + 8 * t + 2 * c + j]);
                }
#pragma unroll
                for (int t = 0; t < kNT; ++t)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float m2 = fmaxf(m[t][j], top[t][j] - kLift);
                        const float fade = m2 == -INFINITY ? 1.f : ex2(m[t][j] - m2);
                        m[t][j] = m2;
                        l[t][j] *= fade;
#pragma unroll
                        for (int q = 0; q < kTiles; ++q) {
                            o[q][t][j] *= fade;
                            o[q][t][2 + j] *= fade;
                        }
                    }
            }
            uint32_t pb[2][kNT][2];
#pragma unroll
            for (int t = 0; t < kNT; ++t) {
                const float b0 = m[t][0] == -INFINITY ? 0.f : -m[t][0], b1 = m[t][1] == -INFINITY ? 0.f : -m[t][1];
                const float f0 = whole ? f[t][0] : 1.f, f1 = whole ? f[t][1] : 1.f;
#pragma unroll
                for (int n = 0; n < kOwn; ++n) {
                    const float w0 = ex2(fmaf(z[n][t][0], f0, b0)), w1 = ex2(fmaf(z[n][t][1], f1, b1));
                    const float w2 = ex2(fmaf(z[n][t][2], f0, b0)), w3 = ex2(fmaf(z[n][t][3], f1, b1));
                    l[t][0] += w0 + w2;
                    l[t][1] += w1 + w3;
                    pb[n][t][0] = transpose_8x8(pack_f16(w0, w1));
                    pb[n][t][1] = transpose_8x8(pack_f16(w2, w3));
                }
            }
            if constexpr (kSplit == 2) {
                // this block's fragments to the other warp, its block's from there (two buffers in turn: the next step's
                // writes pass no reads of this step's, which end before the other warp's next pair_any)
                const uint32_t buf = exchanged + static_cast<uint32_t>(k % 2 * (2 * kNT * 2 * 128) + lane * 4);
#pragma unroll
                for (int t = 0; t < kNT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(buf + static_cast<uint32_t>((part * kNT * 2 + t * 2 + i) * 128)), "r"(pb[0][t][i])
                                     : "memory");
                team_sync();
#pragma unroll
                for (int t = 0; t < kNT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t mine = pb[0][t][i], theirs = lds32(buf + static_cast<uint32_t>(((part ^ 1) * kNT * 2 + t * 2 + i) * 128));
                        pb[0][t][i] = part == 0 ? mine : theirs;
                        pb[1][t][i] = part == 0 ? theirs : mine;
                    }
            }
            // ---- weighted values: the warp's output tiles, both blocks ------------------------------------------
            constexpr int kGroups = (kTiles + 7) / 8, kPer = kTiles / kGroups;  // 16-column groups of a lane; tiles of each
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                uint32_t nan16[kGroups] = {};  // tokens of the block whose scale is NaN
#pragma unroll
                for (int x = 0; x < kGroups; ++x) {
                    const int group16 = (r * (D / 8) + 2 * part * kTiles + 16 * x) / 16;
                    uint32_t s4 = lds32(slot + static_cast<uint32_t>(n * kBlock + KvPlace<D>::kValueScales + (group16 * 4 + c) * 4));
                    if (!whole) {
                        // a token that some row does not see must not reach that row through 0 * NaN: its NaN scale becomes 0
                        // here and is put into the rows that do see it below
                        uint32_t bad = 0;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if ((s4 >> (8 * j) & 0x7Fu) == 0x7Fu) {
                                bad |= 1u << (2 * c + j % 2 + 8 * (j / 2));
                                s4 &= ~(0xFFu << (8 * j));
                            }
                        bad |= __shfl_xor_sync(0xFFFFFFFFu, bad, 1);
                        bad |= __shfl_xor_sync(0xFFFFFFFFu, bad, 2);
                        nan16[x] |= have >> n & 1 ? bad : 0u;
                    }
                    const uint32_t sp0 = e4m3x2_to_f16(s4 & 0xFFFFu), sp1 = e4m3x2_to_f16(s4 >> 16);
                    const uint32_t e0 = sp0 & 0xFFFFu, o0 = sp0 & 0xFFFF0000u, e1 = sp1 & 0xFFFFu, o1 = sp1 & 0xFFFF0000u;
                    constexpr int kWords = kPer < 4 ? kPer : 4;  // codes of so many tiles at a time
#pragma unroll
                    for (int q = x * kPer; q < (x + 1) * kPer; q += kWords) {
                        const int tile = part * kTiles + q;
                        const uint32_t from = slot + static_cast<uint32_t>(n * kBlock + KvPlace<D>::kValueCodes + tile / 4 * 512 + lane * 16 + tile % 4 * 4);
                        uint32_t w[4];
                        if constexpr (kWords == 4) {
                            const uint4 v = ld_smem_v4(from);
                            w[0] = v.x;
                            w[1] = v.y;
                            w[2] = v.z;
                            w[3] = v.w;
                        } else {
                            lds64(from, w[0], w[1]);
                        }
#pragma unroll
                        for (int mm = 0; mm < kWords; ++mm) {
                            uint32_t x0, x1, x2, x3;  // tokens 2c, 2c + 1, 2c + 8, 2c + 9; a pair of columns each
                            e2m1_word_to_f16(w[mm], x0, x1, x2, x3);
                            const uint32_t a0 = weave_low(x0, e0, x1, o0), a1 = weave_high(x0, e0, x1, o0);
                            const uint32_t a2 = weave_low(x2, e1, x3, o1), a3 = weave_high(x2, e1, x3, o1);
#pragma unroll
                            for (int t = 0; t < kNT; ++t) mma_f16(o[q + mm][t], a0, a1, a2, a3, pb[n][t][0], pb[n][t][1]);
                        }
                    }
                }
                if (!whole) {
#pragma unroll
                    for (int x = 0; x < kGroups; ++x) {
                        if (nan16[x] == 0) continue;
#pragma unroll
                        for (int t = 0; t < kNT; ++t)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int upto = see(t, j), lo = p.window > 0 ? upto - p.window : 0, hi = min(upto, g.s.kvl);
                                const int b0 = (blk0 + n) * 16;
                                const int from = min(max(lo - b0, 0), 16), to = min(max(hi - b0, 0), 16);
                                const uint32_t vis = to > from ? ((1u << to) - 1u) & ~((1u << from) - 1u) : 0u;
                                if (nan16[x] & vis) {
#pragma unroll
                                    for (int q = x * kPer; q < (x + 1) * kPer; ++q) o[q][t][j] = o[q][t][2 + j] = __uint_as_float(0x7FC00000u);
                                }
                            }
                    }
                }
            }
            if constexpr (kSplit == 1) {
                __syncwarp();
                if (issued < steps) issue(issued++);  // into the stage that is free now
            }
        }
        uses += static_cast<uint32_t>(steps);
        if constexpr (kSplit == 2) team_sync();  // the ring is free

        // ---- the next part's copies start before this one is joined ---------------------------------------
        const Segment done = g;
        at += whole_ones ? 1 : g.u1 - g.u0;
        const bool more = at < end;
        if (more) {
            g.u0 = 0;
            const Work<R> w(p, g.s, group);
            if (++g.tile == w.tiles) {
                g.tile = 0;
                ++g.h;
            }
            if (g.h == heads) {
                g.h = 0;
                while (true) {  // `at` < `end` <= total: a sequence with work follows
                    g.s = load_seq(p, ++g.b, nullptr);
                    if (g.s.ql > 0) break;
                }
            }
            g.units = Work<R>(p, g.s, group).units;
            g.u1 = whole_ones ? g.units : static_cast<int>(min(static_cast<long long>(g.units), end - at));
            place();
            open();
        }

        // ---- join the warps' results --------------------------------------------------------------------------
        // Each warp leaves its own in shared memory; then an item of four columns (two output tiles of the fragments' layout) of
        // the rows 8 t + 2 c + j goes to one warp, which adds up what the teams have of it.
#pragma unroll
        for (int t = 0; t < kNT; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int x = 4; x < 32; x *= 2) l[t][j] += __shfl_xor_sync(0xFFFFFFFFu, l[t][j], x);
        constexpr int kPairs = kSplit * P::kPassTiles / 2, kItems = kPairs * 2 * kNT;
        static_assert(P::kPassTiles % 2 == 0, "whole items");
        constexpr int kWarpFloats = P::kStateFloats + P::kMl;
        auto leave = [&](int pass) {
            float* ml = merge + warp * kWarpFloats;
            if (pass == 0 && r == 0) {
#pragma unroll
                for (int t = 0; t < kNT; ++t)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        ml[8 * t + 2 * c + j] = m[t][j];
                        ml[8 * kNT + 8 * t + 2 * c + j] = l[t][j];
                    }
            }
#pragma unroll
            for (int k = 0; k < P::kPassTiles; ++k)
#pragma unroll
                for (int t = 0; t < kNT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        ml[P::kMl + ((k * kNT + t) * 4 + e) * 32 + lane] = o[pass * P::kPassTiles + k][t][e];
        };
        // one item's sum over the segment's keys to the outputs
        const int drows = done.s.ql * group, drow0 = done.tile * R;
        auto put = [&](int pass, int item, const float (&v)[4], float top, float sum) {
            const int pr = item % kPairs, tj = item / kPairs;
            const int row = drow0 + 8 * (tj / 2) + 2 * c + tj % 2;
            if (row >= drows) return;
            const float scale = sum == 0.f ? 0.f : p.s.v_unit / sum;
            const int query = divide(row, p.group), head = done.h * group + row - query * group;
            const long long token = done.s.qs + query;
            const int tile = 2 * pr / P::kPassTiles * kTiles + pass * P::kPassTiles + 2 * pr % P::kPassTiles;
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + token * p.out_stride + static_cast<long long>(head) * D + r * (D / 8) + 2 * tile;
            const __nv_bfloat162 x = __floats2bfloat162_rn(v[0] * scale, v[1] * scale), y = __floats2bfloat162_rn(v[2] * scale, v[3] * scale);
            *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
            if (p.lse && r == 0 && pr == 0 && pass == 0) p.lse[token * p.q_heads + head] = log_sum_exp(top, sum);
        };
        const bool all = done.u0 == 0 && done.u1 == done.units;
        // a part of a segment: units [done.u0, done.u1) of it; the segment's first unit is `at` - done.u1 of the call
        const long long seg0 = at - done.u1, seg1 = seg0 + done.units - 1;
        auto cta_of = [&](long long x) { return static_cast<int>(((x + 1) * ctas - 1) / total); };
        const int c0 = all ? 0 : cta_of(seg0), c1 = all ? 0 : cta_of(seg1);
        // in the workspace: rows' maxima and sums, then the items. A CTA's second slot is for the segment that begins in it, the
        // first for one that began before.
        auto part_of = [&](int cta) {
            return reinterpret_cast<float*>(static_cast<unsigned char*>(p.workspace) + kAttCounterBytes) +
                   static_cast<long long>(2 * cta + (cta == c0 ? 1 : 0)) * kAttPartFloats;
        };
#pragma unroll
        for (int pass = 0; pass < P::kPasses; ++pass) {
            if (pass > 0) __syncthreads();
            leave(pass);
            __syncthreads();
            // all of the warp's items at once, so that their loads overlap
            constexpr int kMine = (kItems + kWarps - 1) / kWarps;
            float top[kMine], sum[kMine], v[kMine][4];
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int item = min(warp + i * kWarps, kItems - 1), pr = item % kPairs, tj = item / kPairs, t = tj / 2, j = tj % 2;
                const float* ml = merge + 8 * t + 2 * c + j;
                const float* words = merge + 2 * pr / P::kPassTiles * kWarpFloats + P::kMl + ((2 * pr % P::kPassTiles * kNT + t) * 4 + j) * 32 + lane;
                top[i] = -INFINITY;
#pragma unroll
                for (int w = 0; w < kTeams; ++w) top[i] = fmaxf(top[i], ml[w * kSplit * kWarpFloats]);
                const float base = top[i] == -INFINITY ? 0.f : top[i];
                sum[i] = v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
#pragma unroll
                for (int w = 0; w < kTeams; ++w) {
                    const float* x = ml + w * kSplit * kWarpFloats;
                    const float fade = ex2(x[0] - base);
                    sum[i] = fmaf(fade, kSplit == 1 ? x[8 * kNT] : x[8 * kNT] + x[8 * kNT + kWarpFloats], sum[i]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[i][e] = fmaf(fade, words[w * kSplit * kWarpFloats + (e / 2 * kNT * 4 + e % 2 * 2) * 32], v[i][e]);
                }
            }
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int item = warp + i * kWarps, tj = item / kPairs, col = 8 * (tj / 2) + 2 * c + tj % 2;
                if (item >= kItems) break;
                if (all) {
                    put(pass, item, v[i], top[i], sum[i]);
                } else {
                    float* mine = part_of(static_cast<int>(blockIdx.x));
                    if (pass == 0 && item % kPairs == 0 && r == 0) {
                        mine[col] = top[i];
                        mine[8 * kNT + col] = sum[i];
                    }
                    *reinterpret_cast<float4*>(mine + P::kMl + ((pass * kItems + item) * 32 + lane) * 4) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
                }
            }
        }
        if (!all) {
            __syncthreads();
            if (tid == 0) {
                unsigned int* counter = static_cast<unsigned int*>(p.workspace) + c0;
                __threadfence();
                const bool last = atomicAdd(counter, 1u) + 1 == static_cast<unsigned int>(c1 - c0 + 1);
                if (last) *counter = 0;
                last_flag = last ? 1 : 0;
                __threadfence();
            }
            __syncthreads();
            if (last_flag) {  // the parts in their order (other SMs' writes: from L2)
                constexpr int kMine = (P::kPasses * kItems + kWarps - 1) / kWarps;
                float top[kMine], sum[kMine], v[kMine][4];
                int col[kMine], x[kMine];
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    x[i] = min(warp + i * kWarps, P::kPasses * kItems - 1);
                    const int tj = x[i] % kItems / kPairs;
                    col[i] = 8 * (tj / 2) + 2 * c + tj % 2;
                    top[i] = -INFINITY;
                    sum[i] = v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
                }
#pragma unroll 4
                for (int w = c0; w <= c1; ++w) {
                    const float* from = part_of(w);
#pragma unroll
                    for (int i = 0; i < kMine; ++i) top[i] = fmaxf(top[i], __ldcg(from + col[i]));
                }
#pragma unroll 2
                for (int w = c0; w <= c1; ++w) {
                    const float* from = part_of(w);
#pragma unroll
                    for (int i = 0; i < kMine; ++i) {
                        const float fade = ex2(__ldcg(from + col[i]) - (top[i] == -INFINITY ? 0.f : top[i]));
                        const float4 y = __ldcg(reinterpret_cast<const float4*>(from + P::kMl) + x[i] * 32 + lane);
                        sum[i] = fmaf(fade, __ldcg(from + 8 * kNT + col[i]), sum[i]);
                        v[i][0] = fmaf(fade, y.x, v[i][0]);
                        v[i][1] = fmaf(fade, y.y, v[i][1]);
                        v[i][2] = fmaf(fade, y.z, v[i][2]);
                        v[i][3] = fmaf(fade, y.w, v[i][3]);
                    }
                }
#pragma unroll
                for (int i = 0; i < kMine; ++i)
                    if (warp + i * kWarps < P::kPasses * kItems) put(x[i] / kItems, x[i] % kItems, v[i], top[i], sum[i]);
            }
        }
        if (!more) break;
        __syncthreads();  // last_flag and the merge buffers are free again
    }
}

template <int D, int kNT, int kSplit>
int launch_rows(const AttArgs& args, cudaStream_t stream) {
    using P = Plan<D, kNT, kSplit>;
    AttArgs a = args;
    a.most_segments = (a.n * a.group.by / (8 * kNT) + (a.seqs < a.n ? a.seqs : a.n)) * a.s.heads;  // each sequence may end inside a tile
    static_assert(8 * kNT * (D + 2) <= kAttPartFloats, "a partial result fits its place in the workspace");
    static std::mutex mu;
    static int ctas[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -7;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (ctas[dev] == 0) {
            int sms = 0, per_sm = 0;
            if (cudaFuncSetAttribute(attend_rows_kernel<D, kNT, kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kSmem) != cudaSuccess ||
                cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
                cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, attend_rows_kernel<D, kNT, kSplit>, P::kThreads, P::kSmem) != cudaSuccess ||
                sms < 1 || per_sm < 1)
                return -7;
            ctas[dev] = sms * per_sm < kAttMaxCtas ? sms * per_sm : kAttMaxCtas;
        }
    }
    g_launched.store(true, std::memory_order_relaxed);
    attend_rows_kernel<D, kNT, kSplit><<<static_cast<unsigned>(ctas[dev]), P::kThreads, P::kSmem, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? 0 : -7;
}

// `rows`: of the sequences that the call's tiles are made for
int launch_rows_for(long long rows, const AttArgs& a, cudaStream_t stream) {
    switch (a.s.dim) {
        case 64:
            if (rows <= 8) return launch_rows<64, 1, 1>(a, stream);
            if (rows <= 16) return launch_rows<64, 2, 2>(a, stream);
            return launch_rows<64, 4, 2>(a, stream);
        case 128:
            if (rows <= 8) return launch_rows<128, 1, 1>(a, stream);
            if (rows <= 16) return launch_rows<128, 2, 2>(a, stream);
            if (rows <= 24) return launch_rows<128, 3, 2>(a, stream);
            return launch_rows<128, 4, 2>(a, stream);
        default:
            if (rows <= 8) return launch_rows<256, 1, 2>(a, stream);
            return launch_rows<256, 2, 2>(a, stream);
    }
}

}  // namespace

int launch_attention(const AttArgs& args, cudaStream_t stream) {
    AttArgs a = args;
    a.q_min = 0;
    a.q_max = kAnyQueries;
    if (a.max_q_len > a.n) a.max_q_len = static_cast<int>(a.n);  // n is at most 2^31 - 1
    const int group = a.group.by;
    const long long rows = static_cast<long long>(a.max_q_len) * group;
    if (rows < kTilesFromRows || !attention_tiles_take(a)) return launch_rows_for(rows, a, stream);
    // Sequences of a single query, or so few that they fit the same tile of rows, among longer ones (chunks of a prefill in
    // a batch that decodes) get a launch of their own. 255 single queries over 2,050 to 4,096 keys and one chunk of 2,305,
    // 40 and 8 heads of 128: 434 us, 922 us where the tiles' kernel takes all; with a chunk of 513, 283 us. Where no
    // sequence is short the launch costs 8 us or more, so n = seqs * max_q_len (none is) goes without.
    const int few = group <= 32 ? (group + 7) / 8 * 8 / group : 0;
    if (few > 0 && a.n != static_cast<long long>(a.seqs) * a.max_q_len) {
        a.q_max = few;
        const int st = launch_rows_for(static_cast<long long>(few) * group, a, stream);
        if (st != 0) return st;
        a.q_min = few + 1;
        a.q_max = kAnyQueries;
    }
    return launch_attention_tiles(a, stream);
}

int read_attention_error(unsigned int* word, int clear, cudaStream_t stream) {
    unsigned int v = 0, tiles = 0;
    if (read_tiles_error(&tiles, clear, stream) != 0) return -7;
    *word = tiles;
    if (!g_launched.load(std::memory_order_relaxed)) return 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_hc_attention_error, sizeof(v), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess)
        return -7;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return -7;
    if (clear && v != 0) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbolAsync(g_hc_attention_error, &z, sizeof(z), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess)
            return -7;
        if (cudaStreamSynchronize(stream) != cudaSuccess) return -7;
    }
    *word = v | tiles;
    return 0;
}

}  // namespace hc
