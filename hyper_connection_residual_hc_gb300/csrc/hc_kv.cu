// The 4-bit key/value cache: quantising tokens as they are written, and reading them back (format and
// byte layout: include/hc.h).
//
// Each 16 columns of a token's head share the scale s = e4m3(amax / (6 unit)), and a code is
// e2m1(x / (s unit)). Both are decided exactly.
//   The code: borders b between two codes are 0.25, 0.75, 1.25, 1.75, 2.5, 3.5 and 5. x has 8 significant bits and
//   b s at most 7, so |x - b s| is 0 or at least x / 256, and the quotient q = x / s is a border exactly or at least
//   2^-10 away from one. x * (1/s) with the hardware's reciprocal (1 ulp) is off by less than 2^-19 for q up to 8; adding
//   and taking away 1.5 * 2^11 rounds it to a multiple of 2^-12, which puts a border on itself and leaves the others on
//   their side. (Above 8 all is the largest code.) The sign is put back from x, for the zeros.
//   The scale: amax / 6 is taken as amax * (1/6) and one residual step (v + (a - 6 v) / 6, the classical correction of
//   a quotient by its remainder), exact where the quotient has few bits, so that ties between two scales are seen as ties.
//
// The layout is the one that the attention's matrix instructions read, so the bytes of one token are
// scattered in 1- and 2-byte pieces over its block of 16 tokens. A warp takes 16 tokens of the call and the keys or
// the values of one head, and looks for a run among their slots: 16 consecutive tokens on the 16 slots of one cache block. A run
// (prefill) goes block-wise: each lane takes the tokens and columns that it has in the layout, so that it
// holds whole 16-column groups and whole words, and every store is 16 bytes wide. Other tokens (decode,
// ragged ends) go token-wise, 8 columns a lane. Both give the same bytes.
//
// Bound: HBM, (4 + 1.125) bytes for a column of a key and a value; at these rates the instructions that decide and
// place the codes come close behind (the ALU pipe is 64% busy while writing). 16,384 tokens of 8 heads of 128, 86 MB:
// written in 22.2 us (3.9 TB/s, 57% of the measured copy rate), read back in 21.8 us (4.0 TB/s), 41.8 us one after the
// other (the read finds part of the cache in L2); 256 single tokens on as many pages in 3.8 and 3.1 us. Keys and values by
// separate warps balance the few waves of such a call (reading 28.9 to 21.5 us); runs found by ballot in independent warps
// instead of by a loop in shared memory: 69 to 49 us for both.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "hc_attn.h"
#include "hc_kv.cuh"
#include "hc_ptx.cuh"

namespace hc {
namespace {

__device__ unsigned int g_hc_kv_error = 0;
std::atomic<bool> g_launched{false};  // whether the word above can be set at all (reading it costs a copy and a wait)

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroup = 16;                 // tokens of the call per block
constexpr int kWindow = 3 * kGroup - 2;    // slots looked at: 15 before the group, 15 after it

// the bits of the largest magnitude of bf16 pairs; a NaN's (above infinity's) if there is one
__device__ __forceinline__ uint32_t amax_bits(const uint32_t* w, int words) {
    uint32_t m = 0;
    for (int i = 0; i < words; ++i) {
        uint32_t x;
        asm("abs.bf16x2 %0, %1;" : "=r"(x) : "r"(w[i]));
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(x));
    }
    return max(m & 0x7FFFu, m >> 16 & 0x7FFFu);
}

__device__ __forceinline__ uint32_t scale_byte(uint32_t amax, float inv_unit) {
    if (amax >= 0x7F80u) return 0x7Fu;  // NaN or infinity in the group
    const float a = __uint_as_float(amax << 16) * inv_unit;
    constexpr float kSixth = 1.0f / 6.0f;
    float q = a * kSixth;
    q = fmaf(fmaf(-6.0f, q, a), kSixth, q);
    if (!(a < 1e30f)) q = a;  // far above the largest scale; infinity has no remainder
    uint16_t two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.0f), "f"(q));
    return two & 0xFFu;
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
    const uint32_t h = e4m3x2_to_f16(byte);
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}

// 1 / (s unit), 0 for the scale 0
__device__ __forceinline__ float recip_or_zero(float s, float inv_unit) { return s > 0.f ? rcp_approx(s) * inv_unit : 0.f; }

// four bf16 pairs (the even column in the low half) -> four bytes of two codes
__device__ __forceinline__ uint32_t code_word(const uint32_t* w, float rs) {
    constexpr float kGrid = 0x1.8p11f;
    float v[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a = __uint_as_float(w[e] << 16), b = __uint_as_float(w[e] & 0xFFFF0000u);
        const float u = fmaf(fabsf(a), rs, kGrid) - kGrid, t = fmaf(fabsf(b), rs, kGrid) - kGrid;
        v[2 * e] = copysignf(u, a);
        v[2 * e + 1] = copysignf(t, b);
    }
    uint32_t r;
    asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c3, %8, %7;\n\t"
        "mov.b32 %0, {c0, c1, c2, c3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// ---- eight columns of one token a lane (token-wise) -----------------------------------------------
// 32 / (D / 8) tokens side by side in a warp; all lanes come here (the scale is exchanged between two).

template <int D, bool kKeys>
__device__ __forceinline__ void write_token(const KvArgs& p, bool active, long long i, int h, unsigned char* block, int t, int lane) {
    const int col = 8 * (lane % (D / 8));
    uint4 x = make_uint4(0, 0, 0, 0);
    if (active) {
        const __nv_bfloat16* src = kKeys ? static_cast<const __nv_bfloat16*>(p.k_in) + i * p.k_stride
                                         : static_cast<const __nv_bfloat16*>(p.v_in) + i * p.v_stride;
        x = __ldcs(reinterpret_cast<const uint4*>(src + static_cast<long long>(h) * D + col));
    }
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = amax_bits(w, 4);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    const float inv_unit = 1.0f / (kKeys ? p.s.k_unit : p.s.v_unit);  // exact: a power of two
    const uint32_t sb = scale_byte(m, inv_unit);
    const uint32_t codes = code_word(w, recip_or_zero(scale_value(sb), inv_unit));
    if (!active) return;
    if constexpr (kKeys) {
        unsigned char* dst = block + KvPlace<D>::key_code(t, col);
        *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(codes);
        *reinterpret_cast<uint16_t*>(dst + 4) = static_cast<uint16_t>(codes >> 16);
        if (lane % 2 == 0) block[KvPlace<D>::key_scale(t, col)] = static_cast<unsigned char>(sb);
    } else {
        unsigned char* dst = block + KvPlace<D>::value_code(t, col);
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[4 * e] = static_cast<unsigned char>(codes >> (8 * e));
        if (lane % 2 == 0) block[KvPlace<D>::value_scale(t, col)] = static_cast<unsigned char>(sb);
    }
}

// a pair of fp16 values times the unit, as a bf16 pair (exact)
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t v, float unit) {
    const __half2 h = *reinterpret_cast<const __half2*>(&v);
    const float2 f = __half22float2(h);
    const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * unit, f.y * unit);
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t both(uint32_t scale_byte_) { return e4m3x2_to_f16(scale_byte_ | scale_byte_ << 8); }

// block null: zeros
template <int D, bool kKeys>
__device__ __forceinline__ void read_token(const KvArgs& p, long long i, int h, const unsigned char* block, int t, int lane) {
    const int col = 8 * (lane % (D / 8));
    uint4 o = make_uint4(0, 0, 0, 0);
    if (block) {
        uint32_t w, s;
        if constexpr (kKeys) {
            const unsigned char* src = block + KvPlace<D>::key_code(t, col);
            w = *reinterpret_cast<const uint16_t*>(src) | static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(src + 4)) << 16;
            s = both(block[KvPlace<D>::key_scale(t, col)]);
        } else {
            const unsigned char* src = block + KvPlace<D>::value_code(t, col);
            w = src[0] | src[4] << 8 | src[8] << 16 | static_cast<uint32_t>(src[12]) << 24;
            s = both(block[KvPlace<D>::value_scale(t, col)]);
        }
        uint32_t x[4];
        e2m1_word_to_f16(w, x[0], x[1], x[2], x[3]);
        const float unit = kKeys ? p.s.k_unit : p.s.v_unit;
        o = make_uint4(f16x2_to_bf16x2(mul_f16x2(x[0], s), unit), f16x2_to_bf16x2(mul_f16x2(x[1], s), unit),
                       f16x2_to_bf16x2(mul_f16x2(x[2], s), unit), f16x2_to_bf16x2(mul_f16x2(x[3], s), unit));
    }
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(kKeys ? p.k_out : p.v_out) + i * (kKeys ? p.k_stride : p.v_stride);
    __stcs(reinterpret_cast<uint4*>(dst + static_cast<long long>(h) * D + col), o);
}

// ---- a whole block of 16 tokens (block-wise) ------------------------------------------------------
// Lane (r, c) = (lane / 4, lane % 4). Keys: tokens r and r + 8, columns [c D/4, (c+1) D/4). Values: tokens
// 2c, 2c+1, 2c+8, 2c+9, columns [r D/8, (r+1) D/8).

template <int D>
__device__ __forceinline__ void write_key_block(const KvArgs& p, long long i, int h, unsigned char* block, int lane) {
    constexpr int kN = D / 4;  // columns a lane
    const int r = lane / 4, c = lane % 4;
    const float inv_unit = 1.0f / p.s.k_unit;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.k_in) + i * p.k_stride + static_cast<long long>(h) * D + c * kN;
    uint4 x[2][kN / 8];
#pragma unroll
    for (int hw = 0; hw < 2; ++hw)
#pragma unroll
        for (int e = 0; e < kN / 8; ++e) x[hw][e] = __ldcs(reinterpret_cast<const uint4*>(src + (r + 8 * hw) * p.k_stride) + e);
    uint32_t codes[2][kN / 8];  // per token, 8 columns a word
    uint32_t scales[2] = {};
#pragma unroll
    for (int hw = 0; hw < 2; ++hw)
#pragma unroll
        for (int g = 0; g < kN / 16; ++g) {
            const uint32_t w[8] = {x[hw][2 * g].x, x[hw][2 * g].y, x[hw][2 * g].z, x[hw][2 * g].w,
                                   x[hw][2 * g + 1].x, x[hw][2 * g + 1].y, x[hw][2 * g + 1].z, x[hw][2 * g + 1].w};
            const uint32_t sb = scale_byte(amax_bits(w, 8), inv_unit);
            const float rs = recip_or_zero(scale_value(sb), inv_unit);
            const int at = hw * (kN / 16) + g;  // place among the lane's scale bytes
            scales[at / 4] |= sb << (8 * (at % 4));
            codes[hw][2 * g] = code_word(w, rs);
            codes[hw][2 * g + 1] = code_word(w + 4, rs);
        }
#pragma unroll
    for (int quad = 0; quad < D / 64; ++quad) {
        // word s of the quad: four columns of token r (low half), the same of token r + 8
        uint32_t o[4];
#pragma unroll
        for (int s = 0; s < 4; ++s)
            o[s] = __byte_perm(codes[0][2 * quad + s / 2], codes[1][2 * quad + s / 2], s % 2 ? 0x7632 : 0x5410);
        *reinterpret_cast<uint4*>(block + quad * 512 + lane * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    unsigned char* sc = block + KvPlace<D>::kKeyScales + lane * (D / 32);
    if constexpr (D == 64) *reinterpret_cast<uint16_t*>(sc) = static_cast<uint16_t>(scales[0]);
    else if constexpr (D == 128) *reinterpret_cast<uint32_t*>(sc) = scales[0];
    else *reinterpret_cast<uint2*>(sc) = make_uint2(scales[0], scales[1]);
}

template <int D>
__device__ __forceinline__ void write_value_block(const KvArgs& p, long long i, int h, unsigned char* block, int lane) {
    constexpr int kN = D / 8;
    constexpr int kG = (kN + 15) / 16;  // groups a lane (D = 64: half a group)
    const int r = lane / 4, c = lane % 4;
    const float inv_unit = 1.0f / p.s.v_unit;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.v_in) + i * p.v_stride + static_cast<long long>(h) * D + r * kN;
    uint4 x[4][kN / 8];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < kN / 8; ++e)
            x[j][e] = __ldcs(reinterpret_cast<const uint4*>(src + (2 * c + j % 2 + 8 * (j / 2)) * p.v_stride) + e);
    uint32_t codes[4][kN / 8];
    uint32_t scales[kG] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int g = 0; g < kG; ++g) {
            constexpr int kWords = kN < 16 ? 4 : 8;
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < kWords / 4; ++e) {
                w[4 * e] = x[j][2 * g + e].x;
                w[4 * e + 1] = x[j][2 * g + e].y;
                w[4 * e + 2] = x[j][2 * g + e].z;
                w[4 * e + 3] = x[j][2 * g + e].w;
            }
            uint32_t m = amax_bits(w, kWords);
            if constexpr (D == 64) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));  // the group is shared by r and r ^ 1
            const uint32_t sb = scale_byte(m, inv_unit);
            const float rs = recip_or_zero(scale_value(sb), inv_unit);
            scales[g] |= sb << (8 * j);
#pragma unroll
            for (int e = 0; e < kWords / 4; ++e) codes[j][2 * g + e] = code_word(w + 4 * e, rs);
        }
#pragma unroll
    for (int quad = 0; quad < D / 64; ++quad) {
        // word m: byte j holds columns 2m, 2m + 1 of token j
        uint32_t o[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const uint32_t lo = __byte_perm(codes[0][quad], codes[1][quad], m | (m + 4) << 4);
            const uint32_t hi = __byte_perm(codes[2][quad], codes[3][quad], m | (m + 4) << 4);
            o[m] = __byte_perm(lo, hi, 0x5410);
        }
        *reinterpret_cast<uint4*>(block + KvPlace<D>::kValueCodes + quad * 512 + lane * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    unsigned char* sc = block + KvPlace<D>::kValueScales;
    if constexpr (D == 64) {
        if (r % 2 == 0) *reinterpret_cast<uint32_t*>(sc + (r / 2 * 4 + c) * 4) = scales[0];
    } else {
#pragma unroll
        for (int g = 0; g < kG; ++g) *reinterpret_cast<uint32_t*>(sc + ((r * kG + g) * 4 + c) * 4) = scales[g];
    }
}

template <int D>
__device__ __forceinline__ void read_key_block(const KvArgs& p, long long i, int h, const unsigned char* block, int lane) {
    constexpr int kN = D / 4;
    const int r = lane / 4, c = lane % 4;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.k_out) + i * p.k_stride + static_cast<long long>(h) * D + c * kN;
    const unsigned char* sc = block + KvPlace<D>::kKeyScales + lane * (D / 32);
    uint4 v[D / 64];
    uint32_t s0[D / 64], s1[D / 64];
#pragma unroll
    for (int quad = 0; quad < D / 64; ++quad) {
        v[quad] = __ldcs(reinterpret_cast<const uint4*>(block + quad * 512 + lane * 16));
        s0[quad] = sc[quad];
        s1[quad] = sc[D / 64 + quad];
    }
#pragma unroll
    for (int quad = 0; quad < D / 64; ++quad) {
        const uint32_t w[4] = {v[quad].x, v[quad].y, v[quad].z, v[quad].w};
        const uint32_t f0 = both(s0[quad]), f1 = both(s1[quad]);
        uint32_t a[8], b[8];  // 16 columns of tokens r and r + 8
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            uint32_t x0, x1, x2, x3;
            e2m1_word_to_f16(w[s], x0, x1, x2, x3);
            a[2 * s] = f16x2_to_bf16x2(mul_f16x2(x0, f0), p.s.k_unit);
            a[2 * s + 1] = f16x2_to_bf16x2(mul_f16x2(x1, f0), p.s.k_unit);
            b[2 * s] = f16x2_to_bf16x2(mul_f16x2(x2, f1), p.s.k_unit);
            b[2 * s + 1] = f16x2_to_bf16x2(mul_f16x2(x3, f1), p.s.k_unit);
        }
        uint4* ra = reinterpret_cast<uint4*>(dst + r * p.k_stride + quad * 16);
        uint4* rb = reinterpret_cast<uint4*>(dst + (r + 8) * p.k_stride + quad * 16);
        __stcs(ra, make_uint4(a[0], a[1], a[2], a[3]));
        __stcs(ra + 1, make_uint4(a[4], a[5], a[6], a[7]));
        __stcs(rb, make_uint4(b[0], b[1], b[2], b[3]));
        __stcs(rb + 1, make_uint4(b[4], b[5], b[6], b[7]));
    }
}

template <int D>
__device__ __forceinline__ void read_value_block(const KvArgs& p, long long i, int h, const unsigned char* block, int lane) {
    constexpr int kN = D / 8;
    const int r = lane / 4, c = lane % 4;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.v_out) + i * p.v_stride + static_cast<long long>(h) * D + r * kN;
    const unsigned char* sc = block + KvPlace<D>::kValueScales;
    uint4 v[D / 64];
    uint32_t s4[D / 64];
#pragma unroll
    for (int quad = 0; quad < D / 64; ++quad) {
        v[quad] = __ldcs(reinterpret_cast<const uint4*>(block + KvPlace<D>::kValueCodes + quad * 512 + lane * 16));
        s4[quad] = *reinterpret_cast<const uint32_t*>(sc + ((r * kN + quad * 8) / 16 * 4 + c) * 4);
    }
#pragma unroll
    for (int quad = 0; quad < D / 64; ++quad) {
        const uint32_t w[4] = {v[quad].x, v[quad].y, v[quad].z, v[quad].w};
        uint32_t o[4][4];  // token j, 8 columns
#pragma unroll
        for (int m = 0; m < 4; ++m) e2m1_word_to_f16(w[m], o[0][m], o[1][m], o[2][m], o[3][m]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t s = both(s4[quad] >> (8 * j) & 0xFFu);
#pragma unroll
            for (int m = 0; m < 4; ++m) o[j][m] = f16x2_to_bf16x2(mul_f16x2(o[j][m], s), p.s.v_unit);
            const int t = 2 * c + j % 2 + 8 * (j / 2);
            __stcs(reinterpret_cast<uint4*>(dst + t * p.v_stride + quad * 8), make_uint4(o[j][0], o[j][1], o[j][2], o[j][3]));
        }
    }
}

// One warp takes 16 tokens of the call and the keys or the values of one head; gridDim.y parts share a group's tokens when there are few
// groups. Warps are independent: each reads the slots of its group and of the 15 tokens on either side, lane j
// those at j and j + 32 of this window (token i0 - 15 + j).
template <int D, bool kRead>
__global__ void __launch_bounds__(kThreads) kv_move_kernel(const KvArgs p) {
    const int lane = static_cast<int>(threadIdx.x) % 32;
    const int heads = p.s.heads;
    const long long item = static_cast<long long>(blockIdx.x) * kWarps + threadIdx.x / 32;
    const bool keys = (item & 1) == 0;
    const long long group = item / 2 / heads;
    const int h = static_cast<int>(item / 2 - group * heads);
    const long long i0 = group * kGroup;
    if (i0 >= p.n) return;
    if (kRead && !(keys ? p.k_out : p.v_out)) return;
    const long long cap = static_cast<long long>(p.s.pages) << p.s.page_shift;
    long long s[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int j = lane + 32 * x;
        const long long i = i0 - (kGroup - 1) + j;
        s[x] = -1;
        if (j < kWindow && i >= 0 && i < p.n) {
            s[x] = __ldg(p.slots + i);
            if (s[x] >= cap) {
                if (h == 0 && blockIdx.y == 0 && j >= kGroup - 1 && j < 2 * kGroup - 1) atomicOr(&g_hc_kv_error, kErrPage);
                s[x] = -1;
            }
        }
    }
    // bit j: token j + 1 of the window lies on the slot behind token j's
    const long long after0 = __shfl_down_sync(0xFFFFFFFFu, s[0], 1), first1 = __shfl_sync(0xFFFFFFFFu, s[1], 0);
    const long long after1 = __shfl_down_sync(0xFFFFFFFFu, s[1], 1);
    const unsigned long long next =
        __ballot_sync(0xFFFFFFFFu, s[0] >= 0 && (lane < 31 ? after0 : first1) == s[0] + 1) |
        static_cast<unsigned long long>(__ballot_sync(0xFFFFFFFFu, lane < 31 && s[1] >= 0 && after1 == s[1] + 1)) << 32;
    // bit j: a run of 16 tokens on one cache block begins at token j (they begin at 0..30: 15 tokens must follow)
    const unsigned int run = __ballot_sync(0xFFFFFFFFu, lane < 2 * kGroup - 1 && s[0] >= 0 && s[0] % kGroup == 0 &&
                                                             (next >> lane & 0x7FFFu) == 0x7FFFu);
    auto block_of = [&](long long slot) {
        const long long page = slot >> p.s.page_shift;
        const int in_page = static_cast<int>(slot & ((1LL << p.s.page_shift) - 1));
        return p.cache + (((page * heads + h) << (p.s.page_shift - 4)) + in_page / kGroup) * kv_block_bytes(D);
    };
    // the run that begins in this group, if any (runs begin 16 tokens apart at least)
    const unsigned int here = run >> (kGroup - 1);
    if (here != 0 && blockIdx.y == 0) {
        const int j = kGroup - 1 + __ffs(here) - 1;
        const long long slot = __shfl_sync(0xFFFFFFFFu, s[0], j);  // j <= 30
        const long long i = i0 + j - (kGroup - 1);
        unsigned char* block = block_of(slot);
        if constexpr (kRead) {
            if (keys) read_key_block<D>(p, i, h, block, lane);
            else read_value_block<D>(p, i, h, block, lane);
        } else {
            if (keys) write_key_block<D>(p, i, h, block, lane);
            else write_value_block<D>(p, i, h, block, lane);
        }
    }
    // the tokens of this group that no run has, kSide of them at a time
    constexpr int kSide = 32 / (D / 8);
    for (int x0 = static_cast<int>(blockIdx.y) * kSide; x0 < kGroup; x0 += static_cast<int>(gridDim.y) * kSide) {
        const int x = x0 + lane / (D / 8), j = kGroup - 1 + x;
        const long long slot = __shfl_sync(0xFFFFFFFFu, s[0], j);
        const int t = slot < 0 ? 0 : static_cast<int>(slot % kGroup);
        const bool mine = i0 + x < p.n && !(slot >= 0 && (run >> (j - t) & 1u));
        if (!__any_sync(0xFFFFFFFFu, mine)) continue;
        if constexpr (kRead) {
            if (!mine) continue;
            const unsigned char* block = slot < 0 ? nullptr : block_of(slot);
            if (keys) read_token<D, true>(p, i0 + x, h, block, t, lane);
            else read_token<D, false>(p, i0 + x, h, block, t, lane);
        } else {
            const bool active = mine && slot >= 0;
            unsigned char* block = active ? block_of(slot) : nullptr;
            if (keys) write_token<D, true>(p, active, i0 + x, h, block, t, lane);
            else write_token<D, false>(p, active, i0 + x, h, block, t, lane);
        }
    }
}

template <bool kRead>
int launch_move(const KvArgs& a, cudaStream_t stream) {
    if (a.n <= 0) return 0;
    const int sms = attn_sm_count();
    if (sms == 0) return -7;
    const long long items = (a.n + kGroup - 1) / kGroup * a.s.heads * 2;
    const long long blocks = (items + kWarps - 1) / kWarps;
    if (blocks > 0x7FFFFFFFLL) return -7;
    // few groups (decode, short prompts): spread the tokens of each, down to as many as a warp takes side by side
    long long parts = (2LL * sms + blocks - 1) / blocks;
    const long long most = kGroup * a.s.dim / 256;
    if (parts > most) parts = most;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(parts));
    g_launched.store(true, std::memory_order_relaxed);
    switch (a.s.dim) {
        case 64: kv_move_kernel<64, kRead><<<grid, kThreads, 0, stream>>>(a); break;
        case 128: kv_move_kernel<128, kRead><<<grid, kThreads, 0, stream>>>(a); break;
        default: kv_move_kernel<256, kRead><<<grid, kThreads, 0, stream>>>(a); break;
    }
    return cudaGetLastError() == cudaSuccess ? 0 : -7;
}

}  // namespace

int launch_kv_write(const KvArgs& a, cudaStream_t stream) { return launch_move<false>(a, stream); }
int launch_kv_read(const KvArgs& a, cudaStream_t stream) { return launch_move<true>(a, stream); }

int read_kv_error(unsigned int* word, int clear, cudaStream_t stream) {
    unsigned int v = 0;
    *word = 0;
    if (!g_launched.load(std::memory_order_relaxed)) return 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_hc_kv_error, sizeof(v), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return -7;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return -7;
    if (clear && v != 0) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbolAsync(g_hc_kv_error, &z, sizeof(z), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess) return -7;
        if (cudaStreamSynchronize(stream) != cudaSuccess) return -7;
    }
    *word = v;
    return 0;
}

}  // namespace hc
