// Declarations shared by the translation units of the attention sublayer's operators (hc_rope.cu,
// hc_kv.cu, hc_attend.cu and their entry points in hc_attn_api.cu); not part of the C ABI. The
// launchers take arguments that the entry points have checked and return 0 or -7 (CUDA failure).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace hc {

// bits of the device error word set by these operators
enum : unsigned int {
    kErrPage = 1u << 20,   // a slot or a page outside the cache
    kErrSeq = 1u << 21,    // a sequence's bounds outside the arrays
    kErrCopy = 1u << 22,   // a bounded wait for a copy of cache blocks ran out
    kErrTile = 1u << 23,   // a bounded wait between the warps of a tile ran out
};

// SMs of the current device, found once per device; 0 if that failed
int attn_sm_count();

// ---- norms and rotation (hc_rope.cu) -------------------------------------------------------------
constexpr int kRopeMaxFreqs = 128;
struct RopeEntry {
    unsigned long long turns;  // turns per position, modulo 1, as a fraction of 2^64
    int axis;
    int pad;
};
static_assert(sizeof(RopeEntry) == 16, "one table entry per 16 bytes");
struct RopeTable {
    RopeEntry e[kRopeMaxFreqs];
};
struct RopeArgs {
    const void* q;
    const void* k;
    long long q_stride, k_stride;  // elements
    const float* q_w;
    const float* k_w;
    const long long* positions;
    const RopeEntry* table;
    int rot, start, axes, pairs;
    long long n;
    int q_heads, k_heads, dim, gain_per_head;
    float eps;
    void* q_out;
    void* k_out;
    long long q_out_stride, k_out_stride;
};
int launch_prepare_rope(const RopeTable& t, int freqs, void* table, cudaStream_t stream);
int launch_norm_rope(const RopeArgs& a, cudaStream_t stream);

// ---- the 4-bit cache (hc_kv.cu) ------------------------------------------------------------------
struct KvShape {
    int pages, page_shift, heads, dim;  // page_size = 1 << page_shift
    float k_unit, v_unit;
};
// bytes of 16 tokens of one head
__host__ __device__ constexpr int kv_block_bytes(int dim) { return 18 * dim; }
inline size_t kv_cache_bytes(const KvShape& s) {
    return (static_cast<size_t>(s.pages) << (s.page_shift - 4)) * static_cast<size_t>(s.heads) *
           static_cast<size_t>(kv_block_bytes(s.dim));
}
struct KvArgs {
    const void* k_in;   // bf16 (write)
    const void* v_in;
    void* k_out;        // bf16 (read; either may be null)
    void* v_out;
    long long k_stride, v_stride;
    const long long* slots;
    long long n;
    KvShape s;
    unsigned char* cache;
};
int launch_kv_write(const KvArgs& a, cudaStream_t stream);
int launch_kv_read(const KvArgs& a, cudaStream_t stream);
int read_kv_error(unsigned int* word, int clear, cudaStream_t stream);

// ---- attention (hc_attend.cu) --------------------------------------------------------------------
// Workspace: counters, then the partial results of either kernel: 2 of each of up to 512 CTAs of hc_attend.cu, or the
// slices of hc_attend_tiles.cu, 256 at most.
constexpr int kAttMaxCtas = 512;
constexpr int kAttPartFloats = 32 * (128 + 2);  // of hc_attend.cu, any variant: rows x (dim + maximum + sum)
constexpr int kAttMaxSlices = 256;
constexpr size_t kAttPartFloatsTotal = size_t(kAttMaxSlices) * 256 * (128 + 2);
static_assert(size_t(2) * kAttMaxCtas * kAttPartFloats <= kAttPartFloatsTotal, "both fit");
constexpr size_t kAttCounterBytes = kAttMaxCtas * 4;
constexpr size_t kAttWorkspaceBytes = kAttCounterBytes + kAttPartFloatsTotal * 4;
constexpr int kAnyQueries = 0x7FFFFFFF;
// Division of 0..2^31 - 1 by a number that the host knows: n * ceil(2^(31 + s) / d) / 2^(31 + s) with 2^s >= d is off
// by less than 1 / d, so its integer part is exact. One product and a shift, where a division takes a few tens of
// instructions in a row.
struct Divider {
    int by;
    unsigned int factor, shift;
};
inline Divider make_divider(int by) {
    unsigned int s = 0;
    while ((1ull << s) < static_cast<unsigned long long>(by)) ++s;
    return {by, static_cast<unsigned int>(((1ull << (31 + s)) + static_cast<unsigned long long>(by) - 1) / static_cast<unsigned long long>(by)), 31 + s};
}
struct AttArgs {
    const void* q;
    long long q_stride;
    const int* q_start;
    const int* kv_len;
    const int* page_table;
    const unsigned char* cache;
    long long n;
    int seqs, max_q_len, max_pages, q_heads, causal, window;
    float scale;
    KvShape s;
    void* out;
    long long out_stride;
    float* lse;
    void* workspace;
    Divider group;     // query heads that share a kv head
    long long most_segments;  // of the rows' kernel: (sequence, kv head, tile of rows)
    int q_min, q_max;  // a kernel takes the sequences with so many queries and leaves the others to the other kernel
};
int launch_attention(const AttArgs& a, cudaStream_t stream);
int read_attention_error(unsigned int* word, int clear, cudaStream_t stream);
// many queries a sequence (hc_attend_tiles.cu), dim 64 or 128
bool attention_tiles_take(const AttArgs& a);
int launch_attention_tiles(const AttArgs& a, cudaStream_t stream);
int read_tiles_error(unsigned int* word, int clear, cudaStream_t stream);

}  // namespace hc
