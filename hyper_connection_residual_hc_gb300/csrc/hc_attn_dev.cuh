// Device code that the two attention kernels (hc_attend.cu, hc_attend_tiles.cu) share: sequences, masks and small
// instructions.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "hc_attn.h"

namespace hc {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A weight is 2^(score - m), where m is raised to kLift below a score that exceeds it by more than kSlack: the largest is
// 2^7 or more and none is above 2^15, inside fp16's range (65,504), so that its normal numbers, 11 bits, reach down to 2^-21 of
// the row's largest weight and its least steps to 2^-31. With m at the maximum itself, weights below 2^-25 of the largest
// were 0 while the sums counted them: 2^17 keys 26 doublings behind one lost all that they add to the output.
constexpr float kLift = 7.f;
constexpr float kUnlift = 1.f / 128.f;
constexpr float kSlack = 15.f;
// log of the sum of e^z of a row with the sum l of such weights
__device__ __forceinline__ float log_sum_exp(float m, float l) {
    return l == 0.f ? -INFINITY : (m + kLift + log2f(l * kUnlift)) * kLn2;
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A probe of an mbarrier's phase that lets the warp sleep for up to a millisecond while the phase is not complete: a
// warp that polls instead takes issue slots from those it waits for.
__device__ __forceinline__ bool mbar_sleep(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(1000000u)
        : "memory");
    return ok != 0;
}

// The power of two that brings a query row whose largest magnitude has the bf16 bits m to [2^7, 2^8): bf16's 8 bits
// are then exact in fp16 down to 2^-14, and sums stay far below fp32's range. NaN and infinity stay what they are.
__device__ __forceinline__ void row_scale(uint32_t m, float& up, float& down) {
    const uint32_t e = m >= 0x7F80u ? 134u : max(m >> 7, 27u);
    up = __uint_as_float((261u - e) << 23);
    down = __uint_as_float((e - 7u) << 23);
}

__device__ __forceinline__ int divide(int n, const Divider& d) {
    return static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned int>(n)) * d.factor) >> d.shift);
}

struct SeqRows {
    int qs, ql, kvl;  // first row of q, queries (0: another kernel takes the sequence), keys
};

// `tell`: the error word to note clamped bounds in, or null
__device__ __forceinline__ SeqRows load_seq(const AttArgs& p, int b, unsigned int* tell) {
    const int n = static_cast<int>(p.n);
    const int q0 = p.q_start[b], q1 = p.q_start[b + 1], kv = p.kv_len[b];
    const int most = p.max_pages << p.s.page_shift;
    SeqRows s;
    s.qs = min(max(q0, 0), n);
    const int qe = min(max(q1, s.qs), n);
    s.ql = qe - s.qs;
    s.kvl = min(max(kv, 0), most);
    if (tell && (s.qs != q0 || qe != q1 || s.kvl != kv)) atomicOr(tell, kErrSeq);
    if (s.ql < p.q_min || s.ql > p.q_max) s.ql = 0;
    return s;
}

// Keys of the rows row0..row1 of a sequence (row = query * group + head of the group): some row sees [lo, hi), every
// row sees [all_lo, all_hi).
struct TileBounds {
    int lo, hi, all_lo, all_hi;
};
__device__ __forceinline__ TileBounds tile_bounds(const AttArgs& p, const SeqRows& s, int row0, int row1) {
    TileBounds g;
    if (p.causal) {
        const int pos0 = s.kvl - s.ql;
        const int first = pos0 + divide(row0, p.group), last = pos0 + divide(row1, p.group);
        g.hi = min(max(last + 1, 0), s.kvl);
        g.all_hi = first + 1;
        // (positions are negative where a sequence has more queries than keys; a window is as large as an int)
        g.lo = p.window > 0 ? max(0, max(first + 1, 0) - p.window) : 0;
        g.all_lo = p.window > 0 ? max(0, max(last + 1, 0) - p.window) : 0;
    } else {
        g.hi = g.all_hi = s.kvl;
        g.lo = g.all_lo = 0;
    }
    return g;
}

}  // namespace hc
