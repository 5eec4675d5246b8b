// Host helpers that the launchers of the 8-bit products share.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

namespace hc {

constexpr int kMul8Devices = 64;

// Whether a call goes to the pairs' kernel, by both kernels' estimated times. A negative one: that kernel cannot run here (the pairs'
// needs two SMs next to each other, with nearly all of their shared memory), and the other takes the call.
constexpr bool mul8_by_pairs(long long pairs_ns, long long rows_ns) { return pairs_ns >= 0 && pairs_ns < rows_ns; }

// The driver's encoder of tensor maps; null if it has none.
PFN_cuTensorMapEncodeTiled_v12000 mul8_encode();

// A tensor map of 8-bit rows (`cols` bytes, `stride` bytes apart) whose box is 128 columns by box_rows, 128-byte swizzle, zeros outside.
bool mul8_map(CUtensorMap* m, const void* base, long long cols, long long rows, long long stride, int box_rows);

// Clusters of `ctas` CTAs of a kernel that run at once on the current device; -1 if that cannot be told.
int mul8_clusters(const void* kernel, int ctas, int threads, int smem);

}  // namespace hc
