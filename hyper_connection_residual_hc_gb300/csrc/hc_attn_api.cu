// C ABI of the attention sublayer's operators (declared in include/hc.h): host-side argument checks and
// dispatch to the kernels in hc_rope.cu, hc_kv.cu and hc_attend.cu.

#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/hc.h"
#include "hc_attn.h"

namespace hc {
namespace {

constexpr int64_t kMaxRows = 0x7FFFFFFFLL;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

// n rows of `width` bytes, `stride` bytes apart
struct Rows {
    const void* p;
    size_t n, stride, width;
    Rows(const void* p_, int64_t n_, int64_t stride_elements, int64_t width_elements)
        : p(p_), n(static_cast<size_t>(n_)), stride(static_cast<size_t>(stride_elements) * 2),
          width(static_cast<size_t>(width_elements) * 2) {}
    size_t extent() const { return !p || n == 0 || width == 0 ? 0 : (n - 1) * stride + width; }
};

// Rows of one stride may interleave (columns of one buffer); rows of two strides are taken to overlap when
// their extents do.
bool overlap(const Rows& a, const Rows& b) {
    if (!overlap(a.p, a.extent(), b.p, b.extent())) return false;
    if (a.stride != b.stride) return true;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    const size_t s = a.stride;
    const size_t off = y >= x ? (y - x) % s : (s - (x - y) % s) % s;  // b's rows after a's, modulo the stride
    return !(off >= a.width && off + b.width <= s);
}
bool overlap(const Rows& a, const void* b, size_t nb) { return overlap(a.p, a.extent(), b, nb); }

bool good_stride(int64_t stride, int64_t width) { return stride >= width && stride % 8 == 0 && stride <= (1LL << 40); }

bool power_of_two(float x) {
    if (!(x >= 0x1p-40f && x <= 0x1p40f)) return false;
    uint32_t bits;
    std::memcpy(&bits, &x, 4);
    return (bits & 0x7FFFFFu) == 0;
}

int check_kv_shape(const hc_kv_shape_t& s, KvShape* out) {
    if (s.pages < 1 || s.page_size < 16 || s.page_size > 1024 || (s.page_size & (s.page_size - 1)) != 0) return HC_ERR_SHAPE;
    if (s.heads < 1 || s.heads > 1024 || s.dim < 1) return HC_ERR_SHAPE;
    if (s.dim != 64 && s.dim != 128 && s.dim != 256) return HC_ERR_UNSUPPORTED;
    if (!power_of_two(s.k_scale) || !power_of_two(s.v_scale)) return HC_ERR_ARG;
    out->pages = s.pages;
    out->page_shift = __builtin_ctz(static_cast<unsigned>(s.page_size));
    out->heads = s.heads;
    out->dim = s.dim;
    out->k_unit = s.k_scale;
    out->v_unit = s.v_scale;
    return HC_OK;
}

int status(int internal) { return internal == 0 ? HC_OK : HC_ERR_CUDA; }

}  // namespace

int attn_sm_count() {
    static std::atomic<int> count[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = count[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 0;
        count[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

}  // namespace hc

using namespace hc;

extern "C" {

int hc_rope_table_size(int rot, size_t* bytes) {
    if (!bytes) return HC_ERR_NULL;
    if (rot < 0 || rot > 2 * kRopeMaxFreqs || rot % 16 != 0) return HC_ERR_SHAPE;
    *bytes = static_cast<size_t>(rot / 2) * sizeof(RopeEntry);
    return HC_OK;
}

int hc_prepare_rope(const double* inv_freq, const int* axis, int rot, int axes, void* table, hc_stream_t stream) {
    if (!inv_freq || !table) return HC_ERR_NULL;
    if (rot < 16 || rot > 2 * kRopeMaxFreqs || rot % 16 != 0 || axes < 1 || axes > 4) return HC_ERR_SHAPE;
    if (!aligned(table, 16)) return HC_ERR_ALIGN;
    RopeTable t = {};
    for (int j = 0; j < rot / 2; ++j) {
        const int a = axis ? axis[j] : 0;
        if (a < 0 || a >= axes || !std::isfinite(inv_freq[j])) return HC_ERR_ARG;
        // The magnitude's fraction of a turn and its product with 2^64 are exact in fp64 and, below 1, far from 2^64; the
        // sign is put back in integers, where 1 - a small fraction loses nothing.
        double turns = std::fabs(inv_freq[j]) / 6.283185307179586476925286766559;
        turns -= std::floor(turns);
        const unsigned long long fixed = static_cast<unsigned long long>(std::nearbyint(turns * 0x1p64));
        t.e[j].turns = inv_freq[j] < 0.0 ? 0ull - fixed : fixed;
        t.e[j].axis = a;
    }
    return status(launch_prepare_rope(t, rot / 2, table, reinterpret_cast<cudaStream_t>(stream)));
}

int hc_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const float* q_w, const float* k_w,
                    const int64_t* positions, hc_rope_t r, int64_t n, hc_heads_t s, void* q_out, int64_t q_out_stride,
                    void* k_out, int64_t k_out_stride, hc_stream_t stream) {
    const bool has_k = s.k_heads != 0;
    if (!q || !q_out || (has_k && (!k || !k_out)) || (r.rot != 0 && (!r.table || !positions))) return HC_ERR_NULL;
    if (n < 0 || n > kMaxRows || s.q_heads < 1 || s.k_heads < 0 || s.q_heads > 65536 || s.k_heads > 65536 || s.dim < 8 ||
        s.dim % 8 != 0)
        return HC_ERR_SHAPE;
    if (s.dim > 256) return HC_ERR_UNSUPPORTED;
    const int64_t qw = static_cast<int64_t>(s.q_heads) * s.dim, kw = static_cast<int64_t>(s.k_heads) * s.dim;
    if (!good_stride(q_stride, qw) || !good_stride(q_out_stride, qw)) return HC_ERR_SHAPE;
    if (has_k && (!good_stride(k_stride, kw) || !good_stride(k_out_stride, kw))) return HC_ERR_SHAPE;
    if (r.rot < 0 || r.rot % 16 != 0) return HC_ERR_SHAPE;
    if (r.rot != 0) {
        if (r.start < 0 || r.start % 8 != 0 || r.start > s.dim || r.rot > s.dim - r.start || r.axes < 1 || r.axes > 4)
            return HC_ERR_SHAPE;
        if (r.style != HC_ROPE_HALF && r.style != HC_ROPE_PAIRS) return HC_ERR_ARG;
        if (!aligned(r.table, 16) || !aligned(positions, 8)) return HC_ERR_ALIGN;
    }
    if (!std::isfinite(s.norm_eps) || s.norm_eps < 0.f) return HC_ERR_ARG;
    if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(q_w, 16)) return HC_ERR_ALIGN;
    if (has_k && (!aligned(k, 16) || !aligned(k_out, 16) || !aligned(k_w, 16))) return HC_ERR_ALIGN;
    const Rows qi(q, n, q_stride, qw), qo(q_out, n, q_out_stride, qw);
    const Rows ki(has_k ? k : nullptr, n, k_stride, kw), ko(has_k ? k_out : nullptr, n, k_out_stride, kw);
    if (!(q_out == q && q_out_stride == q_stride) && overlap(qo, qi)) return HC_ERR_ALIAS;
    if (has_k && !(k_out == k && k_out_stride == k_stride) && overlap(ko, ki)) return HC_ERR_ALIAS;
    if (has_k && (overlap(qo, ki) || overlap(ko, qi) || overlap(qo, ko))) return HC_ERR_ALIAS;
    const size_t gq = static_cast<size_t>(s.gain_per_head ? qw : s.dim) * 4;
    const size_t gk = static_cast<size_t>(s.gain_per_head ? kw : s.dim) * 4;
    const size_t pos = r.rot ? static_cast<size_t>(n) * static_cast<size_t>(r.axes) * 8 : 0;
    const size_t tab = static_cast<size_t>(r.rot / 2) * sizeof(RopeEntry);
    for (const Rows* o : {&qo, &ko}) {
        if (o->extent() == 0) continue;
        if ((q_w && overlap(*o, q_w, gq)) || (has_k && k_w && overlap(*o, k_w, gk)) || overlap(*o, positions, pos) ||
            overlap(*o, r.table, tab))
            return HC_ERR_ALIAS;
    }
    if (n == 0) return HC_OK;
    RopeArgs a = {};
    a.q = q;
    a.k = k;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.q_w = q_w;
    a.k_w = k_w;
    a.positions = reinterpret_cast<const long long*>(positions);
    a.table = static_cast<const RopeEntry*>(r.table);
    a.rot = r.rot;
    a.start = r.rot ? r.start : 0;
    a.axes = r.axes;
    a.pairs = r.style == HC_ROPE_PAIRS ? 1 : 0;
    a.n = n;
    a.q_heads = s.q_heads;
    a.k_heads = s.k_heads;
    a.dim = s.dim;
    a.gain_per_head = s.gain_per_head ? 1 : 0;
    a.eps = s.norm_eps;
    a.q_out = q_out;
    a.k_out = k_out;
    a.q_out_stride = q_out_stride;
    a.k_out_stride = k_out_stride;
    return status(launch_norm_rope(a, reinterpret_cast<cudaStream_t>(stream)));
}

int hc_kv_cache_size(hc_kv_shape_t s, size_t* bytes) {
    if (!bytes) return HC_ERR_NULL;
    KvShape k;
    const int st = check_kv_shape(s, &k);
    if (st != HC_OK) return st;
    *bytes = kv_cache_bytes(k);
    return HC_OK;
}

int hc_kv_write(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const int64_t* slots, int64_t n,
                hc_kv_shape_t s, void* cache, hc_stream_t stream) {
    if (!k || !v || !slots || !cache) return HC_ERR_NULL;
    KvArgs a = {};
    const int st = check_kv_shape(s, &a.s);
    if (st != HC_OK) return st;
    const int64_t w = static_cast<int64_t>(s.heads) * s.dim;
    if (n < 0 || n > kMaxRows || !good_stride(k_stride, w) || !good_stride(v_stride, w)) return HC_ERR_SHAPE;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cache, 16) || !aligned(slots, 8)) return HC_ERR_ALIGN;
    const size_t cb = kv_cache_bytes(a.s);
    if (overlap(Rows(k, n, k_stride, w), cache, cb) || overlap(Rows(v, n, v_stride, w), cache, cb) ||
        overlap(slots, static_cast<size_t>(n) * 8, cache, cb))
        return HC_ERR_ALIAS;
    if (n == 0) return HC_OK;
    a.k_in = k;
    a.v_in = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.slots = reinterpret_cast<const long long*>(slots);
    a.n = n;
    a.cache = static_cast<unsigned char*>(cache);
    return status(launch_kv_write(a, reinterpret_cast<cudaStream_t>(stream)));
}

int hc_kv_read(const void* cache, const int64_t* slots, int64_t n, hc_kv_shape_t s, void* k_out, int64_t k_stride,
               void* v_out, int64_t v_stride, hc_stream_t stream) {
    if (!cache || !slots || (!k_out && !v_out)) return HC_ERR_NULL;
    KvArgs a = {};
    const int st = check_kv_shape(s, &a.s);
    if (st != HC_OK) return st;
    const int64_t w = static_cast<int64_t>(s.heads) * s.dim;
    if (n < 0 || n > kMaxRows || (k_out && !good_stride(k_stride, w)) || (v_out && !good_stride(v_stride, w)))
        return HC_ERR_SHAPE;
    if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(cache, 16) || !aligned(slots, 8)) return HC_ERR_ALIGN;
    const size_t cb = kv_cache_bytes(a.s);
    const Rows ko(k_out, n, k_stride, w), vo(v_out, n, v_stride, w);
    if (overlap(ko, cache, cb) || overlap(vo, cache, cb) || overlap(ko, slots, static_cast<size_t>(n) * 8) ||
        overlap(vo, slots, static_cast<size_t>(n) * 8) || (k_out && v_out && overlap(ko, vo)))
        return HC_ERR_ALIAS;
    if (n == 0) return HC_OK;
    a.k_out = k_out;
    a.v_out = v_out;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.slots = reinterpret_cast<const long long*>(slots);
    a.n = n;
    a.cache = static_cast<unsigned char*>(const_cast<void*>(cache));
    return status(launch_kv_read(a, reinterpret_cast<cudaStream_t>(stream)));
}

int hc_kv_workspace_size(size_t* bytes) {
    if (!bytes) return HC_ERR_NULL;
    *bytes = kAttWorkspaceBytes;
    return HC_OK;
}

int hc_kv_attention(const void* q, int64_t q_stride, const int* q_start, const int* kv_len, const int* page_table,
                    const void* cache, hc_attention_t a, hc_kv_shape_t s, void* out, int64_t out_stride, float* lse,
                    void* workspace, hc_stream_t stream) {
    if (!q || !q_start || !kv_len || !page_table || !cache || !out || !workspace) return HC_ERR_NULL;
    AttArgs g = {};
    const int st = check_kv_shape(s, &g.s);
    if (st != HC_OK) return st;
    if (a.n < 0 || a.n > kMaxRows || a.seqs < 0 || a.max_q_len < 0 || a.max_pages < 1) return HC_ERR_SHAPE;
    // positions are 32-bit, with room for what the kernels add to them; so are the sequences' numbers
    if (static_cast<int64_t>(a.max_pages) * s.page_size > (1LL << 30) || a.seqs > 1 << 24) return HC_ERR_SHAPE;
    if (a.q_heads < 1 || a.q_heads % s.heads != 0 || a.q_heads / s.heads > 128) return HC_ERR_SHAPE;
    if (a.n * (a.q_heads / s.heads) > kMaxRows) return HC_ERR_SHAPE;  // rows are counted in 32 bits
    const int64_t w = static_cast<int64_t>(a.q_heads) * s.dim;
    if (!good_stride(q_stride, w) || !good_stride(out_stride, w)) return HC_ERR_SHAPE;
    if (!std::isfinite(a.scale) || a.scale < 0.f || a.window < 0 || (a.window > 0 && !a.causal)) return HC_ERR_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cache, 16) || !aligned(workspace, 16) || !aligned(q_start, 4) ||
        !aligned(kv_len, 4) || !aligned(page_table, 4) || !aligned(lse, 4))
        return HC_ERR_ALIGN;
    const Rows qi(q, a.n, q_stride, w), oo(out, a.n, out_stride, w);
    const size_t B = static_cast<size_t>(a.seqs);
    const void* plain[4] = {cache, q_start, kv_len, page_table};
    const size_t bytes[4] = {kv_cache_bytes(g.s), (B + 1) * 4, B * 4, B * static_cast<size_t>(a.max_pages) * 4};
    const size_t lb = lse ? static_cast<size_t>(a.n) * static_cast<size_t>(a.q_heads) * 4 : 0;
    if (overlap(oo, qi) || overlap(oo, workspace, kAttWorkspaceBytes) || overlap(oo, lse, lb) || overlap(qi, lse, lb) ||
        overlap(qi, workspace, kAttWorkspaceBytes) || overlap(lse, lb, workspace, kAttWorkspaceBytes))
        return HC_ERR_ALIAS;
    for (int i = 0; i < 4; ++i)
        if (overlap(oo, plain[i], bytes[i]) || overlap(lse, lb, plain[i], bytes[i]) ||
            overlap(workspace, kAttWorkspaceBytes, plain[i], bytes[i]))
            return HC_ERR_ALIAS;
    if (a.n == 0 || a.seqs == 0) return HC_OK;
    g.q = q;
    g.q_stride = q_stride;
    g.q_start = q_start;
    g.kv_len = kv_len;
    g.page_table = page_table;
    g.cache = static_cast<const unsigned char*>(cache);
    g.n = a.n;
    g.seqs = a.seqs;
    g.max_q_len = a.max_q_len;
    g.max_pages = a.max_pages;
    g.q_heads = a.q_heads;
    g.causal = a.causal ? 1 : 0;
    g.window = a.window;
    g.scale = a.scale;
    g.out = out;
    g.out_stride = out_stride;
    g.lse = lse;
    g.workspace = workspace;
    g.group = make_divider(a.q_heads / s.heads);
    return status(launch_attention(g, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
