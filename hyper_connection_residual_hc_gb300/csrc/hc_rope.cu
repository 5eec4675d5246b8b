// Per-head RMSNorm of queries and keys and the position rotation, in one pass.
//
// For a head's row x of `dim` values with gain w: u_i = w_i x_i / sqrt(mean(x^2) + eps) ("Final
// RMSNorm" page, RMSNorm excerpt, applied per head); then frequency j turns the pair (a, b) of u by
// phi = position * f_j: a' = a cos phi - b sin phi, b' = b cos phi + a sin phi.
//
// The angle. A position times a frequency is taken modulo one turn in 64-bit fixed point: the table
// holds round(f / 2 pi * 2^64) mod 2^64, the product with the position wraps modulo 2^64, and the
// wrapped product, read as a signed integer, is the angle in (-1/2, 1/2] turns. Nothing is lost for
// far positions, where an fp32 product would be off by radians; sincospif then takes an argument in
// (-1, 1].
//
// Layout. One block takes one token: its first rot/2 threads make the (cos, sin) pairs once, for all
// heads, while the rows' loads are in flight; then each row is 8 values a lane on a group of kLanes
// lanes (dim / 8 rounded up to a power of two). The sum of squares is a shuffle tree over the group;
// in the half style the partner columns sit rot/16 lanes away and come by shuffle too.
//
// Bound: HBM (4 bytes a value). 40 + 8 heads of 128: see the table of measurements in the design notes.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "hc_attn.h"

namespace hc {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 3;  // rows per lane group whose loads are in flight together

__global__ void prepare_rope_kernel(const __grid_constant__ RopeTable t, int freqs, RopeEntry* out) {
    const int j = static_cast<int>(threadIdx.x);
    if (j < freqs) out[j] = t.e[j];
}

__device__ __forceinline__ float lo16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi16(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pk(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <int kLanes>
__global__ void __launch_bounds__(kThreads, 4) norm_rope_kernel(const RopeArgs p) {
    __shared__ float2 cs[kRopeMaxFreqs];
    const int lane = static_cast<int>(threadIdx.x) % kLanes;
    const int group = static_cast<int>(threadIdx.x) / kLanes;
    constexpr int kGroups = kThreads / kLanes;
    const long long t = blockIdx.x;
    const int rows = p.q_heads + p.k_heads;
    const int col = 8 * lane;
    const bool in = col < p.dim;
    const float inv_dim = 1.0f / static_cast<float>(p.dim);

    const uint4* qrow = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + t * p.q_stride + col);
    const uint4* krow = p.k_heads ? reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.k) + t * p.k_stride + col)
                                  : nullptr;
    const int pitch = p.dim / 8;  // uint4 per row
    uint4 v[kRows];
    auto load = [&](int r0) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * kGroups;
            v[i] = make_uint4(0, 0, 0, 0);
            if (in && r < rows)
                v[i] = r < p.q_heads ? __ldcs(qrow + static_cast<long long>(r) * pitch)
                                     : __ldcs(krow + static_cast<long long>(r - p.q_heads) * pitch);
        }
    };
    load(group);

    if (static_cast<int>(threadIdx.x) < p.rot / 2) {
        const int j = static_cast<int>(threadIdx.x);
        const RopeEntry e = p.table[j];
        // an axis outside `axes` can only come from a table made for other axes
        const int axis = e.axis < p.axes && e.axis >= 0 ? e.axis : 0;
        const unsigned long long ph = static_cast<unsigned long long>(p.positions[axis * p.n + t]) * e.turns;
        // signed 2^-64 turns to half turns
        const float half_turns = static_cast<float>(static_cast<long long>(ph)) * 1.0842021724855044e-19f;  // 2^-63
        float s, c;
        sincospif(half_turns, &s, &c);
        cs[j] = make_float2(c, s);
    }
    __syncthreads();

    // this lane's eight columns: cos and signed sin of each, the lane of its partner columns (half style)
    const int x = col - p.start;
    const bool turned = in && x >= 0 && x < p.rot;
    const int half = p.rot / 2;
    const int away = p.rot / 16;  // lanes between partners
    float c[8], s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        c[e] = 1.f;
        s[e] = 0.f;
    }
    int partner = lane;
    if (turned) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            int j;
            bool first;
            if (p.pairs) {
                j = (x + e) / 2;
                first = (e & 1) == 0;
            } else {
                first = x < half;
                j = first ? x + e : x - half + e;
            }
            const float2 f = cs[j];
            c[e] = f.x;
            s[e] = first ? -f.y : f.y;
        }
        partner = p.pairs ? lane : x < half ? lane + away : lane - away;
    }

    for (int r0 = group; r0 < rows + group; r0 += kRows * kGroups) {  // the same trip count in every group
        if (r0 != group) load(r0);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * kGroups;
            if (r0 - group + i * kGroups >= rows) break;  // no group has a row here
            float u[8] = {lo16(v[i].x), hi16(v[i].x), lo16(v[i].y), hi16(v[i].y),
                          lo16(v[i].z), hi16(v[i].z), lo16(v[i].w), hi16(v[i].w)};
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(u[e], u[e], ss);
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o, 32);
            const float rs = rsqrtf(fmaf(ss, inv_dim, p.eps));
            const bool is_q = r < p.q_heads;
            const float* w = is_q ? p.q_w : p.k_w;
            if (in && r < rows && w) {
                w += col + (p.gain_per_head ? static_cast<long long>(is_q ? r : r - p.q_heads) * p.dim : 0);
                const float4 g0 = __ldg(reinterpret_cast<const float4*>(w));
                const float4 g1 = __ldg(reinterpret_cast<const float4*>(w) + 1);
                u[0] *= rs * g0.x; u[1] *= rs * g0.y; u[2] *= rs * g0.z; u[3] *= rs * g0.w;
                u[4] *= rs * g1.x; u[5] *= rs * g1.y; u[6] *= rs * g1.z; u[7] *= rs * g1.w;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] *= rs;
            }
            float o[8];
            if (p.pairs) {
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = fmaf(u[e ^ 1], s[e], u[e] * c[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = fmaf(__shfl_sync(0xFFFFFFFFu, u[e], partner, kLanes), s[e], u[e] * c[e]);
            }
            if (!turned) {  // outside the rotated columns the value itself (a NaN partner must not reach it)
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = u[e];
            }
            if (in && r < rows) {
                __nv_bfloat16* dst = is_q ? static_cast<__nv_bfloat16*>(p.q_out) + t * p.q_out_stride + static_cast<long long>(r) * p.dim
                                          : static_cast<__nv_bfloat16*>(p.k_out) + t * p.k_out_stride +
                                                static_cast<long long>(r - p.q_heads) * p.dim;
                *reinterpret_cast<uint4*>(dst + col) =
                    make_uint4(pk(o[0], o[1]), pk(o[2], o[3]), pk(o[4], o[5]), pk(o[6], o[7]));
            }
        }
    }
}

}  // namespace

int launch_prepare_rope(const RopeTable& t, int freqs, void* table, cudaStream_t stream) {
    prepare_rope_kernel<<<1, kRopeMaxFreqs, 0, stream>>>(t, freqs, static_cast<RopeEntry*>(table));
    return cudaGetLastError() == cudaSuccess ? 0 : -7;
}

int launch_norm_rope(const RopeArgs& a, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(a.n);
    const int lanes = a.dim / 8;
    if (lanes <= 1) norm_rope_kernel<1><<<grid, kThreads, 0, stream>>>(a);
    else if (lanes <= 2) norm_rope_kernel<2><<<grid, kThreads, 0, stream>>>(a);
    else if (lanes <= 4) norm_rope_kernel<4><<<grid, kThreads, 0, stream>>>(a);
    else if (lanes <= 8) norm_rope_kernel<8><<<grid, kThreads, 0, stream>>>(a);
    else if (lanes <= 16) norm_rope_kernel<16><<<grid, kThreads, 0, stream>>>(a);
    else norm_rope_kernel<32><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? 0 : -7;
}

}  // namespace hc
