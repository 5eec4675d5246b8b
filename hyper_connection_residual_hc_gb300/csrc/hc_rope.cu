// Per-head RMSNorm of queries and keys and the position rotation, in one pass.
//
// For a head's row x of `dim` values with gain w: u_i = w_i x_i / sqrt(mean(x^2) + eps) ("Final
// RMSNorm" page, RMSNorm excerpt, applied per head); then frequency j turns the pair (a, b) of u by
// phi = position * f_j: a' = a cos phi - b sin phi, b' = b cos phi + a sin phi.
//
// The angle. A position times a frequency is taken modulo one turn in 64-bit fixed point: the table
// holds round(f / 2 pi * 2^64) mod 2^64, the product with the position wraps modulo 2^64, and the
// wrapped product's upper 32 bits, read as a signed integer, are the angle in [-1/2, 1/2) turns. Nothing is
// lost for far positions, where an fp32 product would be off by radians; sincospif then takes an argument
// in [-1, 1).
//
// Layout. A block takes one token at a time: its first rot/2 threads make cosine and sine once, for all heads,
// a token ahead, and leave them in shared memory multiplied with the gains, so that a row needs one product
// and one FMA a value; each row is 8 values a lane on a group of kLanes lanes (dim / 8 rounded up to
// a power of two). The sum of squares is a shuffle tree over the group; in the half style the partner
// columns sit rot/16 lanes away and come by shuffle too. The grid is what is resident, and a register
// is refilled with the next token's row as soon as it has been unpacked, so loads never pause.
//
// Bound: HBM (4 bytes a value). 40 + 8 heads of 128: 67.5 us at 16,384 tokens (403 MB, 5.97 TB/s, 88% of the
// measured copy rate), 3.4 us at 64. What brought it there: the next row in flight in the register of the last (loads
// alone did not bound it: 122 us with and without), gains and rotation from a per-token table instead of registers
// and per-row loads of the gains (120 to 88 us: 239 to 130 instructions a row), packed fp32 and a table without bank
// conflicts (88 to 71 us), 5 blocks an SM at 48 registers instead of 4 at 64 (71 to 67.5 us). A row of 80 columns leaves
// 6 of 16 lanes idle: 15.2 us for 4,097 tokens of 32 such rows (42 MB).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "hc_attn.h"

namespace hc {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 3;         // rows per lane group whose loads are in flight together
constexpr int kBlocksPerSm = 5;
constexpr int kMaxDim = 256;

__global__ void prepare_rope_kernel(const __grid_constant__ RopeTable t, int freqs, RopeEntry* out) {
    const int j = static_cast<int>(threadIdx.x);
    if (j < freqs) out[j] = t.e[j];
}

__device__ __forceinline__ float lo16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi16(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
// pairs of fp32 in one instruction
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 split(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint32_t pk(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// What a token's rows are multiplied with, per column: out = r (x direct + x_partner cross), the gains and the
// rotation in one. [q or k][place of the column]: the first four of each lane's eight columns, then the other four, so that
// 16-byte loads of neighbouring lanes lie side by side.
struct Turn {
    float direct[2][kMaxDim];
    float cross[2][kMaxDim];
};
__device__ __forceinline__ int place(int col) { return col % 8 / 4 * (kMaxDim / 2) + col / 8 * 4 + col % 4; }

// kOne: all rows of a token fit the block's registers at once
template <int kLanes, bool kOne>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) norm_rope_kernel(const RopeArgs p) {
    __shared__ __align__(16) Turn turns[2];  // of this token and of the next
    const int tid = static_cast<int>(threadIdx.x);
    const int lane = tid % kLanes, group = tid / kLanes;
    constexpr int kGroups = kThreads / kLanes;
    const int rows = p.q_heads + p.k_heads;
    const int chunks = kOne ? 1 : (rows + kRows * kGroups - 1) / (kRows * kGroups);
    const int col = 8 * lane;
    const bool in = col < p.dim;
    const float inv_dim = 1.0f / static_cast<float>(p.dim);
    const long long step = gridDim.x;
    const float* gains[2] = {p.gain_per_head ? nullptr : p.q_w, p.gain_per_head ? nullptr : p.k_w};  // per-head ones apply to x
    auto gain = [&](int kind, int i) { return gains[kind] ? __ldg(gains[kind] + i) : 1.f; };

    auto load = [&](long long t, int r) {  // row r of token t; zeros where there is none
        if (!in || r >= rows || t >= p.n) return make_uint4(0, 0, 0, 0);
        const bool is_q = r < p.q_heads;
        const __nv_bfloat16* x = is_q ? static_cast<const __nv_bfloat16*>(p.q) + t * p.q_stride
                                      : static_cast<const __nv_bfloat16*>(p.k) + t * p.k_stride;
        return __ldcs(reinterpret_cast<const uint4*>(x + ((is_q ? r : r - p.q_heads) * p.dim + col)));
    };

    long long t = blockIdx.x;
    uint4 v[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) v[i] = load(t, group + i * kGroups);

    for (int i = tid; i < p.dim; i += kThreads)  // the columns that are not turned keep these
        for (int kind = 0; kind < 2; ++kind)
            for (int buf = 0; buf < 2; ++buf) {
                turns[buf].direct[kind][place(i)] = gain(kind, i);
                turns[buf].cross[kind][place(i)] = 0.f;
            }
    // the thread's own frequency, if it makes one, and its two columns
    const bool turns_one = tid < p.rot / 2;
    const int ca = p.start + (p.pairs ? 2 * tid : tid), cb = ca + (p.pairs ? 1 : p.rot / 2);
    const int pa = place(ca), pb = place(cb);
    RopeEntry entry = {};
    float ga[2], gb[2];
    if (turns_one) {
        entry = p.table[tid];
        // an axis outside `axes` can only come from a table made for other axes
        if (entry.axis >= p.axes || entry.axis < 0) entry.axis = 0;
        for (int kind = 0; kind < 2; ++kind) {
            ga[kind] = gain(kind, ca);
            gb[kind] = gain(kind, cb);
        }
    }
    auto position = [&](long long tok) { return turns_one && tok < p.n ? __ldg(p.positions + entry.axis * p.n + tok) : 0; };
    auto turn = [&](long long pos, Turn& to) {
        const unsigned long long ph = static_cast<unsigned long long>(pos) * entry.turns;
        // the upper 32 bits: the angle to 2^-32 turns, as a signed number of half turns
        const float half_turns = static_cast<float>(static_cast<int>(ph >> 32)) * 4.6566128730773926e-10f;  // 2^-31
        float s, c;
        sincospif(half_turns, &s, &c);
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            to.direct[kind][pa] = ga[kind] * c;
            to.cross[kind][pa] = -gb[kind] * s;
            to.direct[kind][pb] = gb[kind] * c;
            to.cross[kind][pb] = ga[kind] * s;
        }
    };
    __syncthreads();
    long long pos = position(t);
    if (turns_one) turn(pos, turns[0]);
    pos = position(t + step);

    const int x = col - p.start;
    const bool turned = in && x >= 0 && x < p.rot;
    const int away = p.rot / 16;  // lanes between partners (half style)
    const int partner = turned && !p.pairs ? (x < p.rot / 2 ? lane + away : lane - away) : lane;

    for (int buf = 0; t < p.n; t += step, buf ^= 1) {
        __syncthreads();  // turns[buf] is there; turns[buf ^ 1] has been read
        if (turns_one) {
            turn(pos, turns[buf ^ 1]);
            pos = position(t + 2 * step);
        }
        const Turn& now = turns[buf];
        for (int k = 0; k < chunks; ++k) {
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int r = (k * kRows + i) * kGroups + group;
                const uint32_t w4[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                uint64_t u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) u[e] = pair(lo16(w4[e]), hi16(w4[e]));
                // the row that follows in this register: of the next chunk, or of the next token's first
                v[i] = k + 1 < chunks ? load(t, r + kRows * kGroups) : load(t + step, group + i * kGroups);
                if (r - group >= rows) continue;  // no group has a row here
                uint64_t sq = mul2(u[0], u[0]);
#pragma unroll
                for (int e = 1; e < 4; ++e) sq = fma2(u[e], u[e], sq);
                const float2 sq2 = split(sq);
                float ss = sq2.x + sq2.y;
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o, 32);
                const float rs = rsqrtf(fmaf(ss, inv_dim, p.eps));
                const bool is_q = r < p.q_heads;
                const int at = (is_q ? r : r - p.q_heads) * p.dim + col;
                if (p.gain_per_head) {
                    const float* w = is_q ? p.q_w : p.k_w;
                    if (in && r < rows && w) {
                        const float4 g0 = __ldg(reinterpret_cast<const float4*>(w + at));
                        const float4 g1 = __ldg(reinterpret_cast<const float4*>(w + at) + 1);
                        u[0] = mul2(u[0], pair(g0.x, g0.y));
                        u[1] = mul2(u[1], pair(g0.z, g0.w));
                        u[2] = mul2(u[2], pair(g1.x, g1.y));
                        u[3] = mul2(u[3], pair(g1.z, g1.w));
                    }
                }
                const int kind = is_q ? 0 : 1;
                const uint64_t rr = pair(rs, rs);
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // the partner columns; where nothing turns, zeros in the pairs style (cross is 0, but 0 * infinity is not)
                    const float2 x2 = split(u[e]);
                    const uint64_t q = p.pairs ? pair(turned ? x2.y : 0.f, turned ? x2.x : 0.f)
                                               : pair(__shfl_sync(0xFFFFFFFFu, x2.x, partner, kLanes), __shfl_sync(0xFFFFFFFFu, x2.y, partner, kLanes));
                    const int from = e / 2 * (kMaxDim / 2) + lane * 4 + e % 2 * 2;
                    const uint64_t d = *reinterpret_cast<const uint64_t*>(&now.direct[kind][from]);
                    const uint64_t c = *reinterpret_cast<const uint64_t*>(&now.cross[kind][from]);
                    const float2 y = split(mul2(rr, fma2(q, c, mul2(u[e], d))));
                    o[e] = pk(y.x, y.y);
                }
                if (in && r < rows) {
                    __nv_bfloat16* dst = is_q ? static_cast<__nv_bfloat16*>(p.q_out) + t * p.q_out_stride
                                              : static_cast<__nv_bfloat16*>(p.k_out) + t * p.k_out_stride;
                    __stcs(reinterpret_cast<uint4*>(dst + at), make_uint4(o[0], o[1], o[2], o[3]));
                }
            }
        }
    }
}

template <int kLanes>
int launch(const RopeArgs& a, cudaStream_t stream) {
    const int sms = attn_sm_count();
    if (sms == 0) return -7;
    const long long resident = static_cast<long long>(kBlocksPerSm) * sms;
    const unsigned grid = static_cast<unsigned>(a.n < resident ? a.n : resident);
    if (a.q_heads + a.k_heads <= kRows * (kThreads / kLanes)) norm_rope_kernel<kLanes, true><<<grid, kThreads, 0, stream>>>(a);
    else norm_rope_kernel<kLanes, false><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? 0 : -7;
}

}  // namespace

int launch_prepare_rope(const RopeTable& t, int freqs, void* table, cudaStream_t stream) {
    prepare_rope_kernel<<<1, kRopeMaxFreqs, 0, stream>>>(t, freqs, static_cast<RopeEntry*>(table));
    return cudaGetLastError() == cudaSuccess ? 0 : -7;
}

int launch_norm_rope(const RopeArgs& a, cudaStream_t stream) {
    const int lanes = a.dim / 8;
    if (lanes <= 1) return launch<1>(a, stream);
    if (lanes <= 2) return launch<2>(a, stream);
    if (lanes <= 4) return launch<4>(a, stream);
    if (lanes <= 8) return launch<8>(a, stream);
    if (lanes <= 16) return launch<16>(a, stream);
    return launch<32>(a, stream);
}

}  // namespace hc
