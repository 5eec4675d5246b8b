// C ABI of the 8-bit operators of the feed-forward sublayer and the head (declared in include/hc.h): host-side argument checks and
// dispatch to the kernels in hc_quant8.cu, hc_mul8.cu, hc_mul8_tiles.cu and hc_logprobs.cu.

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/hc.h"
#include "hc_ffn.h"

namespace hc {
namespace {

constexpr int64_t kMaxRows = 0x7FFFFFFFLL;
constexpr int64_t kMaxStride = 1LL << 37;  // (a tensor map's strides are below 2^40 bytes)

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// n rows of `width` bytes, `stride` bytes apart; nothing if p is null
struct Rows {
    const void* p;
    size_t n, stride, width;
    Rows(const void* p_, int64_t n_, int64_t stride_, int64_t width_, int64_t size = 1)
        : p(p_), n(static_cast<size_t>(n_)), stride(static_cast<size_t>(stride_ * size)), width(static_cast<size_t>(width_ * size)) {}
    size_t extent() const { return !p || n == 0 || width == 0 ? 0 : (n - 1) * stride + width; }
};
Rows flat(const void* p, int64_t count, int64_t size) { return Rows(p, 1, count, count, size); }

// Rows of one stride may interleave (columns of one buffer); rows of two strides are taken to overlap when their extents do.
bool overlap(const Rows& a, const Rows& b) {
    const size_t na = a.extent(), nb = b.extent();
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    if (!na || !nb || x >= y + nb || y >= x + na) return false;
    if (a.stride != b.stride || a.n == 1 || b.n == 1) return true;
    const size_t s = a.stride;
    const size_t off = y >= x ? (y - x) % s : (s - (x - y) % s) % s;  // b's rows after a's, modulo the stride
    return !(off >= a.width && off + b.width <= s);
}
bool overlap_any(const Rows& out, std::initializer_list<Rows> others) {
    for (const Rows& r : others)
        if (overlap(out, r)) return true;
    return false;
}

// multiple: of elements
bool good_stride(int64_t stride, int64_t width, int multiple) { return stride >= width && stride % multiple == 0 && stride <= kMaxStride; }

int status(int internal) { return internal == 0 ? HC_OK : HC_ERR_CUDA; }

int check_mul(const void* x, int64_t x_stride, const void* x_scales, const void* w, int64_t w_stride, const void* w_scales, int64_t n, int features, int k) {
    if (n < 0 || n > kMaxRows || features < 1 || features > (1 << 24) || k < 16 || k > (1 << 20) || k % 16 != 0) return HC_ERR_SHAPE;
    if (!good_stride(x_stride, k, 16) || !good_stride(w_stride, k, 16)) return HC_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4)) return HC_ERR_ALIGN;
    return HC_OK;
}

}  // namespace
}  // namespace hc

using namespace hc;

extern "C" {

int hc_norm_quant8(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride, const float* norm_w, hc_quant8_t q,
                   void* sum_out, int64_t sum_stride, void* codes, int64_t codes_stride, float* scales, hc_stream_t stream) {
    if (!x || !codes || !scales || (sum_out && !residual)) return HC_ERR_NULL;
    if (q.n < 0 || q.n > kMaxRows || q.d < 16 || q.d > 65536 || q.d % 16 != 0) return HC_ERR_SHAPE;
    if (!good_stride(x_stride, q.d, 8) || !good_stride(codes_stride, q.d, 16) || (residual && !good_stride(residual_stride, q.d, 8)) ||
        (sum_out && !good_stride(sum_stride, q.d, 8)))
        return HC_ERR_SHAPE;
    if (!std::isfinite(q.norm_eps) || q.norm_eps < 0.f) return HC_ERR_ARG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(norm_w, 16) || !aligned(sum_out, 16) || !aligned(codes, 16) || !aligned(scales, 4))
        return HC_ERR_ALIGN;
    const Rows xr(x, q.n, x_stride, q.d, 2), rr(residual, q.n, residual_stride, q.d, 2), so(sum_out, q.n, sum_stride, q.d, 2);
    const Rows co(codes, q.n, codes_stride, q.d), sc = flat(scales, q.n * blocks8(q.d), 4), gw = flat(q.norm ? norm_w : nullptr, q.d, 4);
    if (overlap_any(co, {xr, rr, so, sc, gw}) || overlap_any(sc, {xr, rr, so, gw}) || overlap(so, gw)) return HC_ERR_ALIAS;
    if (!(sum_out == x && sum_stride == x_stride) && overlap(so, xr)) return HC_ERR_ALIAS;
    if (!(sum_out == residual && sum_stride == residual_stride) && overlap(so, rr)) return HC_ERR_ALIAS;
    if (q.n == 0) return HC_OK;
    Quant8Args a = {};
    a.x = x;
    a.residual = residual;
    a.w = q.norm ? norm_w : nullptr;
    a.sum_out = sum_out;
    a.codes = static_cast<unsigned char*>(codes);
    a.scales = scales;
    a.x_stride = x_stride;
    a.residual_stride = residual_stride;
    a.sum_stride = sum_stride;
    a.codes_stride = codes_stride;
    a.n = q.n;
    a.d = q.d;
    a.norm = q.norm ? 1 : 0;
    a.eps = q.norm_eps;
    return status(launch_norm_quant8(a, reinterpret_cast<cudaStream_t>(stream)));
}

int hc_mul8(const void* x, int64_t x_stride, const float* x_scales, const void* w, int64_t w_stride, const float* w_scales, int64_t n,
            hc_mul8_t s, void* out, int64_t out_stride, hc_stream_t stream) {
    if (!x || !x_scales || !w || !w_scales || !out) return HC_ERR_NULL;
    const int st = check_mul(x, x_stride, x_scales, w, w_stride, w_scales, n, s.features, s.k);
    if (st != HC_OK) return st;
    if (s.out_type != HC_BF16 && s.out_type != HC_F32) return HC_ERR_ARG;
    if (!good_stride(out_stride, s.features, 8)) return HC_ERR_SHAPE;
    if (!aligned(out, 16)) return HC_ERR_ALIGN;
    const Rows o(out, n, out_stride, s.features, s.out_type == HC_F32 ? 4 : 2);
    const int64_t kb = blocks8(s.k), fb = blocks8(s.features);
    if (overlap_any(o, {Rows(x, n, x_stride, s.k), flat(x_scales, n * kb, 4), Rows(w, s.features, w_stride, s.k), flat(w_scales, fb * kb, 4)}))
        return HC_ERR_ALIAS;
    if (n == 0) return HC_OK;
    Mul8Args a = {};
    a.x = static_cast<const unsigned char*>(x);
    a.x_scales = x_scales;
    a.w = static_cast<const unsigned char*>(w);
    a.w_scales = w_scales;
    a.x_stride = x_stride;
    a.w_stride = w_stride;
    a.out_stride = out_stride;
    a.n = n;
    a.features = s.features;
    a.k = s.k;
    a.out_type = s.out_type == HC_F32 ? kOutF32 : kOutBf16;
    a.out = out;
    return status(launch_mul8(a, reinterpret_cast<cudaStream_t>(stream)));
}

int hc_gated_mul8(const void* x, int64_t x_stride, const float* x_scales, const void* w_gate, const float* gate_scales, const void* w_up,
                  const float* up_scales, int64_t w_stride, int64_t n, hc_gated8_t s, void* out, int64_t out_stride, float* out_scales,
                  hc_stream_t stream) {
    const bool codes = s.out_type == HC_E4M3;
    if (!x || !x_scales || !w_gate || !gate_scales || !w_up || !up_scales || !out || (codes && !out_scales)) return HC_ERR_NULL;
    int st = check_mul(x, x_stride, x_scales, w_gate, w_stride, gate_scales, n, s.features, s.k);
    if (st != HC_OK) return st;
    if (s.features % 16 != 0) return HC_ERR_SHAPE;
    if (s.out_type != HC_BF16 && s.out_type != HC_E4M3) return HC_ERR_ARG;
    if (s.act != HC_ACT_SILU && s.act != HC_ACT_GELU) return HC_ERR_ARG;
    if (!good_stride(out_stride, s.features, codes ? 16 : 8)) return HC_ERR_SHAPE;
    if (!aligned(w_up, 16) || !aligned(up_scales, 4) || !aligned(out, 16) || (codes && !aligned(out_scales, 4))) return HC_ERR_ALIGN;
    const Rows o(out, n, out_stride, s.features, codes ? 1 : 2);
    const int64_t kb = blocks8(s.k), fb = blocks8(s.features);
    const Rows os = flat(codes ? out_scales : nullptr, n * fb, 4);
    const std::initializer_list<Rows> in = {Rows(x, n, x_stride, s.k),           flat(x_scales, n * kb, 4),
                                            Rows(w_gate, s.features, w_stride, s.k), flat(gate_scales, fb * kb, 4),
                                            Rows(w_up, s.features, w_stride, s.k),   flat(up_scales, fb * kb, 4)};
    if (overlap_any(o, in) || overlap_any(os, in) || overlap(o, os)) return HC_ERR_ALIAS;
    if (n == 0) return HC_OK;
    Mul8Args a = {};
    a.x = static_cast<const unsigned char*>(x);
    a.x_scales = x_scales;
    a.w = static_cast<const unsigned char*>(w_gate);
    a.w_scales = gate_scales;
    a.up = static_cast<const unsigned char*>(w_up);
    a.up_scales = up_scales;
    a.x_stride = x_stride;
    a.w_stride = w_stride;
    a.out_stride = out_stride;
    a.n = n;
    a.features = s.features;
    a.k = s.k;
    a.act = s.act == HC_ACT_GELU ? kActGelu : kActSilu;
    a.out_type = codes ? kOutE4m3 : kOutBf16;
    a.out = out;
    a.out_scales = out_scales;
    return status(launch_mul8(a, reinterpret_cast<cudaStream_t>(stream)));
}

int hc_token_logprobs(const void* logits, int64_t stride, const int64_t* tokens, hc_logprobs_t s, float* logprob, float* entropy,
                      float* top_logprob, int* top_token, hc_stream_t stream) {
    if (!logits || (!logprob && !entropy && s.top == 0) || (logprob && !tokens) || (s.top > 0 && (!top_logprob || !top_token))) return HC_ERR_NULL;
    if (s.n < 0 || s.n > kMaxRows || s.vocab < 1 || s.vocab > (1 << 30) || s.top < 0 || s.top > s.vocab) return HC_ERR_SHAPE;
    if (s.top > kMostTop) return HC_ERR_UNSUPPORTED;
    if (!good_stride(stride, s.vocab, 8)) return HC_ERR_SHAPE;
    if (!(s.scale >= 0x1p-64f && s.scale <= 0x1p64f) || (s.type != HC_BF16 && s.type != HC_F32)) return HC_ERR_ARG;
    if (!aligned(logits, 16) || !aligned(tokens, 8) || !aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(top_logprob, 4) || !aligned(top_token, 4))
        return HC_ERR_ALIGN;
    const Rows z(logits, s.n, stride, s.vocab, s.type == HC_F32 ? 4 : 2), tk = flat(logprob ? tokens : nullptr, s.n, 8);
    const Rows outs[4] = {flat(logprob, s.n, 4), flat(entropy, s.n, 4), flat(s.top ? top_logprob : nullptr, s.n * s.top, 4),
                          flat(s.top ? top_token : nullptr, s.n * s.top, 4)};
    for (int i = 0; i < 4; ++i) {
        if (overlap_any(outs[i], {z, tk})) return HC_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return HC_ERR_ALIAS;
    }
    if (s.n == 0) return HC_OK;
    LogprobArgs a = {};
    a.logits = logits;
    a.stride = stride;
    a.tokens = reinterpret_cast<const long long*>(tokens);
    a.logprob = logprob;
    a.entropy = entropy;
    a.top_logprob = top_logprob;
    a.top_token = top_token;
    a.n = s.n;
    a.vocab = s.vocab;
    a.top = s.top;
    a.wide = s.type == HC_F32 ? 1 : 0;
    a.scale = s.scale;
    return status(launch_logprobs(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
