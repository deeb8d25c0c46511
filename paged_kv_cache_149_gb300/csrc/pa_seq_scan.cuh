// Block-wide prefix sums over the sequences of a batch, for kernels whose every CTA plans
// its own share of the batch: thread u owns the sequences [u * per, (u + 1) * per), and a
// work item's owner is found by a binary search over the threads' prefix sums.
#pragma once

#include <cstdint>

namespace pa {

constexpr int kScanThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;

struct SeqScan {
  unsigned long long warp_sum[kScanWarps];
  unsigned long long pre[kScanThreads + 1];  // pre[u]: sum over the threads before u
};

// Exclusive prefix sums of every thread's `mine` into s.pre (s.pre[kScanThreads]: the
// total).  Called by all kScanThreads threads; the caller synchronises before reading.
__device__ __forceinline__ void seq_scan(SeqScan& s, unsigned long long mine) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s.warp_sum[warp] = incl;
  __syncthreads();
  unsigned long long before = 0;
#pragma unroll
  for (int w = 0; w < kScanWarps; ++w)
    if (w < warp) before += s.warp_sum[w];
  s.pre[threadIdx.x] = before + incl - mine;
  if (threadIdx.x == kScanThreads - 1) s.pre[kScanThreads] = before + incl;
}

// The thread whose share holds item x: the u with pre[u] <= x < pre[u + 1].  x is below
// the total.
__device__ __forceinline__ int seq_owner(const SeqScan& s, unsigned long long x) {
  int u = 0;
#pragma unroll
  for (int step = kScanThreads / 2; step > 0; step >>= 1)
    if (s.pre[u + step] <= x) u += step;
  return u;
}

}  // namespace pa
