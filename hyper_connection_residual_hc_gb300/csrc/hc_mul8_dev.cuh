// Device code that the kernels of the 8-bit products share: bounded waits, descriptors and instructions of tcgen05.mma with 8-bit
// operands, clusters.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "hc_attn_dev.cuh"
#include "hc_ffn.h"
#include "hc_ptx.cuh"

namespace hc {

// A bounded wait: on expiry it notes so in the error word and in the CTA's `abort`, after which no wait of the CTA lasts.
struct Wait8 {
    volatile uint32_t* abort;
    unsigned int* error;
    static constexpr uint64_t kNs = 1000000000ull;
    __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity) const {
        if (mbar_test(bar, parity)) return;
        slow(bar, parity);
    }
    __device__ __forceinline__ void slow(uint32_t bar, uint32_t parity) const {
        const uint64_t t0 = global_timer_ns();
        while (true) {
            for (int i = 0; i < 64; ++i)
                if (mbar_test(bar, parity)) return;
            if (*abort) return;
            if (global_timer_ns() - t0 > kNs) {
                *abort = 1u;
                atomicOr(error, kErrMul8);
                return;
            }
        }
    }
    // At the end, whatever was aborted: waits for what is in flight.
    __device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) const {
        const uint64_t t0 = global_timer_ns();
        while (!mbar_sleep(bar, parity)) {
            if (global_timer_ns() - t0 > kNs) {
                atomicOr(error, kErrMul8);
                return;
            }
        }
    }
};

// Shared-memory descriptor of a K-major operand stored as rows of 128 bytes with the 128-byte swizzle, 8-row groups 1,024 bytes
// apart (fields as in sdesc_kmajor_sw64; swizzle mode 2 = 128 bytes).
__device__ __forceinline__ uint64_t sdesc8(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(1u) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}
// kind::f8f6f4, both operands e4m3 (format 0) and K-major, fp32 accumulator
__host__ __device__ constexpr uint32_t idesc8(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t elect_one() {
    uint32_t lead;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(lead));
    return lead;
}
// The whole warp comes here with the same arguments; `lead` is 1 in the lane that issues.
__device__ __forceinline__ void mma8(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void commit8(uint32_t lead, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(lead)
        : "memory");
}

// 16 consecutive columns of this thread's lane; the values are there after tmem_wait, which waits for all loads so far. What uses
// them has to be volatile (add_scaled), so that it stays behind the wait: naming the registers there instead made the compiler
// move them about.
__device__ __forceinline__ void tmem_start16(uint32_t addr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Pairs of fp32 in one instruction.
__device__ __forceinline__ uint64_t pair8(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair8(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
// acc += {a, b} * scale, for values that came by tmem_start16
__device__ __forceinline__ void add_scaled(uint64_t& acc, float a, float b, uint64_t scale) {
    asm volatile(
        "{\n\t.reg .b64 t;\n\t"
        "mov.b64 t, {%1, %2};\n\t"
        "fma.rn.f32x2 %0, t, %3, %0;\n\t}"
        : "+l"(acc)
        : "f"(a), "f"(b), "l"(scale));
}

__device__ __forceinline__ uint32_t cluster_ctarank8() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync8() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t mapa8(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// NaN wins.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// The gate's activation. Both forms are x times a logistic function, 1 / (1 + e^-y), in which e^-y overflows to infinity for a
// large negative y and the quotient is 0, as it should be; GELU is its form with tanh, (1 + tanh z) / 2 = 1 / (1 + e^-2z). By the
// special function unit's 2^t and 1/t, each within 2^-22 or so of the exact value for its argument; that of 2^t is rounded before, which
// adds |y| 2^-24 to the relative error, and where 1/t falls below fp32's normal numbers it is 0 (SILU below about -87, GELU
// below -10, where the results are below 2^-119). A full exponential and a division took as long as 4 blocks of k a tile.
__device__ __forceinline__ float activate8(float x, int act) {
    float y = -kLog2e * x;
    if (act == kActGelu) y *= 1.5957691216057308f * fmaf(0.044715f * x, x, 1.f);
    return x * rcp_approx(1.f + ex2(y));
}

}  // namespace hc
