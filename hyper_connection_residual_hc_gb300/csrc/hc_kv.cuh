// The 4-bit cache's conversions and byte places (format and layout: include/hc.h), for the kernels
// that write it, read it back and attend over it.
#pragma once

#include <cstdint>

namespace hc {

// Four code bytes of one 32-bit word as four fp16 pairs: lo half = low nibble. e2m1 is exact in fp16.
__device__ __forceinline__ void e2m1_word_to_f16(uint32_t w, uint32_t& p0, uint32_t& p1, uint32_t& p2, uint32_t& p3) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(p0), "=r"(p1), "=r"(p2), "=r"(p3)
        : "r"(w));
}

// Two scale bytes (the low 16 bits) as an fp16 pair, lo half = low byte. e4m3 is exact in fp16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\t"
        "cvt.u16.u32 h, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
        : "=r"(r)
        : "r"(two));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Byte places inside a block of 16 tokens (t) for column i: i is a multiple of 8 for the codes.
template <int D>
struct KvPlace {
    static constexpr int kKeyScales = 8 * D, kValueCodes = 9 * D, kValueScales = 17 * D;
    // the first two of the eight columns' four code bytes; the other two lie 4 bytes on
    static __device__ __forceinline__ int key_code(int t, int i) {
        const int x = i % (D / 4);
        return x / 16 * 512 + (t % 8) * 64 + i / (D / 4) * 16 + x / 4 % 4 * 4 + t / 8 * 2;
    }
    static __device__ __forceinline__ int key_scale(int t, int i) {
        return kKeyScales + (t % 8) * (D / 8) + i / (D / 4) * (D / 32) + t / 8 * (D / 64) + i % (D / 4) / 16;
    }
    // the first of the eight columns' four code bytes; they lie 4 bytes apart
    static __device__ __forceinline__ int value_code(int t, int i) {
        const int x = i % (D / 8);
        return kValueCodes + x / 8 * 512 + i / (D / 8) * 64 + t % 8 / 2 * 16 + t / 8 * 2 + t % 2;
    }
    static __device__ __forceinline__ int value_scale(int t, int i) {
        return kValueScales + i / 16 * 16 + t % 8 / 2 * 4 + t / 8 * 2 + t % 2;
    }
};

}  // namespace hc
