// Residual addition, RMSNorm and quantisation of rows to 8 bits with a scale for each 128 columns, in one pass over the row.
// Formulas and format: include/hc.h.
//
// A row stays in the registers of the threads that load it, 8 columns (16 bytes) at a time: 16 neighbouring lanes hold the 128
// columns of a block, so that a block's largest magnitude takes four exchanges within half a warp. The norm needs one sum
// over the whole row before that; without it the blocks are independent. Rows of up to 512 columns go to one warp each, longer
// ones to as many threads as hold 4 vectors each (8 above 32,768 columns).
//
// Measured: 16,384 rows of 5,120, residual added, summed, normed and quantised: 88 us, 6,690 GB/s, 98% of the measured copy rate. 64 rows of
// 5,120 quantised only: 2.2 us, which is a launch and one chain of latencies.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "hc_ffn.h"
#include "hc_mul8_dev.cuh"

namespace hc {
namespace {

__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// The sum or the largest of a row's threads, the same in all of them; `part` is one call's own.
template <bool kMax>
__device__ __forceinline__ float over_row(float v, int row_threads, float* part) {
    auto over_warp = [](float u) {
#pragma unroll
        for (int m = 16; m; m /= 2) {
            const float o = __shfl_xor_sync(0xFFFFFFFFu, u, m);
            u = kMax ? fmaxf(u, o) : u + o;
        }
        return u;
    };
    v = over_warp(v);
    if (row_threads > 32) {
        const int lane = threadIdx.x % 32;
        if (lane == 0) part[threadIdx.x / 32] = v;
        __syncthreads();
        v = over_warp(lane < row_threads / 32 ? part[lane] : 0.f);
    }
    return v;
}

// row_threads: threads that share a row (a multiple of 32); kVecs: 16-byte vectors of it that each holds, so that all of the row
// is in registers.
template <int kVecs, bool kResidual>
__global__ void __launch_bounds__(kVecs < 4 ? 128 : 1024) quant8_kernel(const Quant8Args p, int row_threads) {
    __shared__ float part[3][32];
    griddep_launch_dependents();
    griddep_wait();
    const int t = threadIdx.x % row_threads, lane = threadIdx.x % 32;
    const long long row = static_cast<long long>(blockIdx.x) * (blockDim.x / row_threads) + threadIdx.x / row_threads;
    if (row >= p.n) return;  // (whole warps; a block of several rows has no barrier)
    const int vecs = p.d / 8;
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) + row * p.x_stride);
    uint4 v[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int c = t + i * row_threads;
        v[i] = c < vecs ? x[c] : make_uint4(0, 0, 0, 0);
    }
    float f[8];
    if constexpr (kResidual) {
        const uint4* r = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.residual) + row * p.residual_stride);
        uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.sum_out) + row * p.sum_stride);
        uint4 w[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int c = t + i * row_threads;
            w[i] = c < vecs ? r[c] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            float g[8];
            unpack(v[i], f);
            unpack(w[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] += g[j];
            v[i] = pack(f);
            const int c = t + i * row_threads;
            if (p.sum_out && c < vecs) o[c] = v[i];
        }
    }
    float inv = 1.f;
    if (p.norm) {
        auto squares = [&]() {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                unpack(v[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
            }
            return sum;
        };
        float mean = over_row<false>(squares(), row_threads, part[0]) / static_cast<float>(p.d) + p.eps;
        // bf16 has fp32's range, squares twice that. Where their mean overflowed, or (with an eps that allows it) came near the subnormal
        // numbers, the row is taken times a power of two that brings the larger of its largest value and sqrt(eps) to 1 .. 4; the result
        // does not change with it. What falls below bf16's least number by that is 2^-126 of the largest. All threads of a row agree.
        if (mean > FLT_MAX || mean < 0x1p-100f) {
            uint32_t pairs = 0;
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                pairs = __vmaxu2(__vmaxu2(pairs, __vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu)), __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
            float most = fmaxf(fmaxf(__uint_as_float(pairs << 16), __uint_as_float(pairs & 0xFFFF0000u)), sqrtf(p.eps));
            most = over_row<true>(most, row_threads, part[1]);
            if (most > 0.f && most <= FLT_MAX) {  // (an infinity stays one)
                const int e = min(max(static_cast<int>(__float_as_uint(most) >> 23), 1), 253);
                const float by = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
                const __nv_bfloat162 by2 = __float2bfloat162_rn(by);
                auto times = [&](uint32_t& u) {
                    const __nv_bfloat162 t = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&u), by2);
                    u = *reinterpret_cast<const uint32_t*>(&t);
                };
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    times(v[i].x);
                    times(v[i].y);
                    times(v[i].z);
                    times(v[i].w);
                }
                mean = over_row<false>(squares(), row_threads, part[2]) / static_cast<float>(p.d) + p.eps * by * by;
            }
        }
        inv = rsqrtf(mean);
    }
    unsigned char* codes = p.codes + row * p.codes_stride;
    float* scales = p.scales + row * blocks8(p.d);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int c = t + i * row_threads;
        unpack(v[i], f);
        if (p.norm) {
            float4 a = make_float4(1.f, 1.f, 1.f, 1.f), b = a;
            if (p.w && c < vecs) {
                a = reinterpret_cast<const float4*>(p.w)[2 * c];
                b = reinterpret_cast<const float4*>(p.w)[2 * c + 1];
            }
            f[0] *= inv * a.x; f[1] *= inv * a.y; f[2] *= inv * a.z; f[3] *= inv * a.w;
            f[4] *= inv * b.x; f[5] *= inv * b.y; f[6] *= inv * b.z; f[7] *= inv * b.w;
        }
        float top = fabsf(f[0]);
#pragma unroll
        for (int j = 1; j < 8; ++j) top = max_nan(top, fabsf(f[j]));
#pragma unroll
        for (int m = 8; m; m /= 2) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
        top = max_nan(top, kLeastTop8);
        if (c < vecs) {
            const float up = kTop8 / top;
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= up;
            *reinterpret_cast<uint2*>(codes + 8 * static_cast<long long>(c)) =
                make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
            if (lane % 16 == 0) scales[c / 16] = top / kTop8;
        }
    }
}

template <int kVecs>
cudaError_t start(const Quant8Args& a, int row_threads, int rows, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.n + rows - 1) / rows));
    cfg.blockDim = dim3(static_cast<unsigned>(row_threads * rows));
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    cfg.attrs = &attr;
    cfg.numAttrs = static_cast<unsigned>(programmatic_launch(a.n * a.d * (a.residual ? 7 : 3) / 6500, false, stream, &attr));
    return cudaLaunchKernelEx(&cfg, a.residual ? quant8_kernel<kVecs, true> : quant8_kernel<kVecs, false>, a, row_threads);
}

}  // namespace

int launch_norm_quant8(const Quant8Args& a, cudaStream_t stream) {
    const int vecs = a.d / 8;
    cudaError_t e;
    if (vecs <= 32)
        e = start<1>(a, 32, 4, stream);
    else if (vecs <= 64)
        e = start<2>(a, 32, 4, stream);
    else if (vecs <= 1024 * 4)
        e = start<4>(a, (vecs + 4 * 32 - 1) / (4 * 32) * 32, 1, stream);
    else
        e = start<8>(a, (vecs + 8 * 32 - 1) / (8 * 32) * 32, 1, stream);
    return e == cudaSuccess ? 0 : -7;
}

}  // namespace hc
