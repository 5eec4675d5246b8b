// Softmax attention of ragged queries over the 4-bit cache (formulas, masks and format: include/hc.h).
//
// One warp takes one query row of one head and walks its keys in cache blocks of 16 tokens with a running
// maximum and sum. Lane (r, c) = (lane / 4, lane % 4) holds the tokens and columns of a block that the
// layout gives it: keys r and r + 8, columns [c D/4, (c+1) D/4); values 2c, 2c+1, 2c+8, 2c+9, columns
// [r D/8, (r+1) D/8).

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "hc_attn.h"
#include "hc_kv.cuh"

namespace hc {
namespace {

__device__ unsigned int g_hc_attention_error = 0;

constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

template <int D>
__global__ void __launch_bounds__(32 * kWarps) attend_kernel(const AttArgs p) {
    const int lane = static_cast<int>(threadIdx.x) % 32, warp = static_cast<int>(threadIdx.x) / 32;
    const int r = lane / 4, c = lane % 4;
    const long long item = static_cast<long long>(blockIdx.x) * kWarps + warp;
    if (item >= p.n * p.q_heads) return;
    const long long row = item / p.q_heads;
    const int head = static_cast<int>(item % p.q_heads);
    const int h = head / (p.q_heads / p.s.heads);
    // the row's sequence: the last one that starts at or before it
    int b = -1;
    for (int i = 0; i < p.seqs; ++i)
        if (p.q_start[i] <= row && row < p.q_start[i + 1]) b = i;
    if (b < 0) return;
    const long long qs = p.q_start[b], qe = p.q_start[b + 1];
    if ((qs < 0 || qe > p.n) && lane == 0) atomicOr(&g_hc_attention_error, kErrSeq);
    const long long most = static_cast<long long>(p.max_pages) << p.s.page_shift;
    long long kvl = p.kv_len[b];
    if (kvl < 0 || kvl > most) {
        if (lane == 0) atomicOr(&g_hc_attention_error, kErrSeq);
        kvl = kvl < 0 ? 0 : most;
    }
    const long long pos = kvl - qe + row;
    const long long hi = p.causal ? (pos + 1 < kvl ? pos + 1 : kvl) : kvl;
    const long long lo = p.window > 0 && pos - p.window + 1 > 0 ? pos - p.window + 1 : 0;
    const float f = p.scale * kLog2e * p.s.k_unit;

    float q[D / 4];
    const __nv_bfloat16* qrow = static_cast<const __nv_bfloat16*>(p.q) + row * p.q_stride + static_cast<long long>(head) * D + c * (D / 4);
#pragma unroll
    for (int e = 0; e < D / 4; ++e) q[e] = __bfloat162float(qrow[e]) * f;
    float m = -INFINITY, l = 0.f, acc[D / 8];
#pragma unroll
    for (int e = 0; e < D / 8; ++e) acc[e] = 0.f;

    for (long long t0 = lo / 16 * 16; t0 < hi; t0 += 16) {
        const int page = p.page_table[static_cast<long long>(b) * p.max_pages + (t0 >> p.s.page_shift)];
        if (page < 0 || page >= p.s.pages) {
            if (lane == 0) atomicOr(&g_hc_attention_error, kErrPage);
            continue;
        }
        const long long in_page = t0 & ((1LL << p.s.page_shift) - 1);
        const unsigned char* block = p.cache + (((static_cast<long long>(page) * p.s.heads + h) << (p.s.page_shift - 4)) + in_page / 16) * kv_block_bytes(D);
        float z[2] = {0.f, 0.f};  // tokens r and r + 8
#pragma unroll
        for (int quad = 0; quad < D / 64; ++quad) {
            const uint4 v = *reinterpret_cast<const uint4*>(block + quad * 512 + lane * 16);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            const unsigned char* sc = block + KvPlace<D>::kKeyScales + lane * (D / 32);
            const float s0 = f16x2_to_float2(e4m3x2_to_f16(sc[quad])).x, s1 = f16x2_to_float2(e4m3x2_to_f16(sc[D / 64 + quad])).x;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                uint32_t x[4];
                e2m1_word_to_f16(w[s], x[0], x[1], x[2], x[3]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 a = f16x2_to_float2(x[e]), d = f16x2_to_float2(x[2 + e]);
                    const int i = quad * 16 + s * 4 + e * 2;
                    z[0] = fmaf(q[i], a.x * s0, fmaf(q[i + 1], a.y * s0, z[0]));
                    z[1] = fmaf(q[i], d.x * s1, fmaf(q[i + 1], d.y * s1, z[1]));
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            z[j] += __shfl_xor_sync(0xFFFFFFFFu, z[j], 1);
            z[j] += __shfl_xor_sync(0xFFFFFFFFu, z[j], 2);
            const long long t = t0 + r + 8 * j;
            if (t < lo || t >= hi) z[j] = -INFINITY;
        }
        float top = fmaxf(z[0], z[1]);
#pragma unroll
        for (int o = 4; o < 32; o *= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const float m2 = fmaxf(m, top);
        const float base = m2 == -INFINITY ? 0.f : m2;
        const float w0 = exp2f(z[0] - base), w1 = exp2f(z[1] - base), fade = exp2f(m - base);
        m = m2;
        l = l * fade + (c == 0 ? w0 + w1 : 0.f);
#pragma unroll
        for (int e = 0; e < D / 8; ++e) acc[e] *= fade;
        float wt[4];  // weights of tokens 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
        for (int j = 0; j < 4; ++j) wt[j] = __shfl_sync(0xFFFFFFFFu, j < 2 ? w0 : w1, 4 * (2 * c + j % 2));
#pragma unroll
        for (int quad = 0; quad < D / 64; ++quad) {
            const uint4 v = *reinterpret_cast<const uint4*>(block + KvPlace<D>::kValueCodes + quad * 512 + lane * 16);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            const uint32_t s4 = *reinterpret_cast<const uint32_t*>(block + KvPlace<D>::kValueScales + ((r * (D / 8) + quad * 8) / 16 * 4 + c) * 4);
            float s[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[j] = f16x2_to_float2(e4m3x2_to_f16(s4 >> (8 * j) & 0xFFu)).x * wt[j];
                const long long t = t0 + 2 * c + j % 2 + 8 * (j / 2);
                if (t < lo || t >= hi) s[j] = 0.f;  // not seen: whatever the cache holds there
            }
#pragma unroll
            for (int mm = 0; mm < 4; ++mm) {
                uint32_t x[4];
                e2m1_word_to_f16(w[mm], x[0], x[1], x[2], x[3]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 a = f16x2_to_float2(x[j]);
                    acc[quad * 8 + 2 * mm] = fmaf(s[j], a.x, acc[quad * 8 + 2 * mm]);
                    acc[quad * 8 + 2 * mm + 1] = fmaf(s[j], a.y, acc[quad * 8 + 2 * mm + 1]);
                }
            }
        }
    }
#pragma unroll
    for (int o = 1; o < 32; o *= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    const float g = l == 0.f ? 0.f : p.s.v_unit / l;
#pragma unroll
    for (int e = 0; e < D / 8; ++e) {
        acc[e] += __shfl_xor_sync(0xFFFFFFFFu, acc[e], 1);
        acc[e] += __shfl_xor_sync(0xFFFFFFFFu, acc[e], 2);
    }
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + row * p.out_stride + static_cast<long long>(head) * D + r * (D / 8);
    if (c == 0) {
#pragma unroll
        for (int e = 0; e < D / 8; ++e) o[e] = __float2bfloat16_rn(acc[e] * g);
    }
    if (p.lse && lane == 0) p.lse[item] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

int launch_attention(const AttArgs& a, cudaStream_t stream) {
    const long long items = a.n * a.q_heads;
    const unsigned grid = static_cast<unsigned>((items + kWarps - 1) / kWarps);
    switch (a.s.dim) {
        case 64: attend_kernel<64><<<grid, 32 * kWarps, 0, stream>>>(a); break;
        case 128: attend_kernel<128><<<grid, 32 * kWarps, 0, stream>>>(a); break;
        default: attend_kernel<256><<<grid, 32 * kWarps, 0, stream>>>(a); break;
    }
    return cudaGetLastError() == cudaSuccess ? 0 : -7;
}

int read_attention_error(unsigned int* word, int clear, cudaStream_t stream) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_hc_attention_error, sizeof(v), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess)
        return -7;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return -7;
    if (clear && v != 0) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbolAsync(g_hc_attention_error, &z, sizeof(z), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess)
            return -7;
        if (cudaStreamSynchronize(stream) != cudaSuccess) return -7;
    }
    *word = v;
    return 0;
}

}  // namespace hc
