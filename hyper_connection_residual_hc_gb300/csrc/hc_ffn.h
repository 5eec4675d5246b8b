// Declarations shared by the translation units of the 8-bit operators of the feed-forward sublayer and the head (hc_quant8.cu,
// hc_mul8.cu, hc_logprobs.cu and their entry points in hc_ffn_api.cu); not part of the C ABI. The launchers take arguments that
// the entry points have checked and return 0 or -7 (CUDA failure).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace hc {

// bits of the device error word set by these operators
enum : unsigned int {
    kErrToken = 1u << 24,  // a token outside the vocabulary
    kErrMul8 = 1u << 25,   // a bounded wait of a product's kernel ran out
};

constexpr int kBlock8 = 128;  // values that share a scale along a row; a weight's scale is for 128 x 128
__host__ __device__ constexpr int blocks8(int n) { return (n + kBlock8 - 1) / kBlock8; }

// 8-bit scales: the largest magnitude of a block stands for 448, e4m3's largest number. A block of zeros (or of values too
// small to matter) keeps a normal scale.
constexpr float kTop8 = 448.f;
constexpr float kLeastTop8 = 0x1p-64f;

// The kernels may start under the end of the kernel ahead on their stream (they wait for it before they touch memory): 256 tokens by
// 20,480 x 5,120 30.4 -> 28.8 us in a graph, 32.9 -> 30.1 called one by one. Such a launch takes the host 1 us longer, which counts
// where the host is what one waits for (64 rows of 5,120 quantised: 11.7 us a call, 12.5 so launched), so that short kernels are
// launched plainly; `in_graphs`: unless they go into a graph. That is for the products, whose CTAs have much to set up (one token by
// 5,120 x 5,120 6.5 -> 5.8 us); many small CTAs that only wait are slower (1,027 rows of 2,000 quantised 4.3 -> 5.5 us). `ns`: about how
// long the kernel takes.
inline int programmatic_launch(long long ns, bool in_graphs, cudaStream_t stream, cudaLaunchAttribute* a) {
    if (ns < 12000) {
        if (!in_graphs) return 0;
        cudaStreamCaptureStatus s = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(stream, &s) != cudaSuccess) {
            cudaGetLastError();  // (another stream's capture forbids the question, and the launch will tell)
            return 0;
        }
        if (s != cudaStreamCaptureStatusActive) return 0;
    }
    a->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a->val.programmaticStreamSerializationAllowed = 1;
    return 1;
}

// ---- norm and quantisation (hc_quant8.cu) ----------------------------------------------------------
struct Quant8Args {
    const void* x;         // bf16
    const void* residual;  // bf16 or null
    const float* w;        // gains or null
    void* sum_out;         // bf16 or null
    unsigned char* codes;
    float* scales;         // [n, blocks8(d)]
    long long x_stride, residual_stride, sum_stride, codes_stride;  // elements
    long long n;
    int d, norm;
    float eps;
};
int launch_norm_quant8(const Quant8Args& a, cudaStream_t stream);

// ---- 8-bit products (hc_mul8.cu) -------------------------------------------------------------------
enum Out8 : int { kOutBf16 = 0, kOutF32 = 1, kOutE4m3 = 2 };
enum Act8 : int { kActSilu = 0, kActGelu = 1 };
struct Mul8Args {
    const unsigned char* x;   // e4m3 [n, k]
    const float* x_scales;    // [n, blocks8(k)]
    const unsigned char* w;   // e4m3 [features, k]; the gate's weights of a gated product
    const float* w_scales;    // [blocks8(features), blocks8(k)]
    const unsigned char* up;  // null: a plain product
    const float* up_scales;
    long long x_stride, w_stride, out_stride;
    long long n;
    int features, k;
    int act;  // Act8
    int out_type;  // Out8
    void* out;
    float* out_scales;  // with kOutE4m3: [n, blocks8(features)]
};
int launch_mul8(const Mul8Args& a, cudaStream_t stream);
int read_mul8_error(unsigned int* word, int clear, cudaStream_t stream);
// many rows (hc_mul8_tiles.cu)
int launch_mul8_tiles(const Mul8Args& a, cudaStream_t stream);
long long mul8_tiles_ns(const Mul8Args& a);  // about how long it would take; negative if it cannot run
int read_mul8_tiles_error(unsigned int* word, int clear, cudaStream_t stream);

// ---- log probabilities (hc_logprobs.cu) ------------------------------------------------------------
constexpr int kMostTop = 32;
struct LogprobArgs {
    const void* logits;
    long long stride;
    const long long* tokens;  // null with logprob null
    float* logprob;           // [n] or null
    float* entropy;           // [n] or null
    float* top_logprob;       // [n, top]
    int* top_token;           // [n, top]
    long long n;
    int vocab, top, wide;     // wide: fp32 logits, else bf16
    float scale;
};
int launch_logprobs(const LogprobArgs& a, cudaStream_t stream);
int read_logprob_error(unsigned int* word, int clear, cudaStream_t stream);

}  // namespace hc
