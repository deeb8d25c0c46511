// Arrival counters of the decode kernel's split-KV merge, written for host and device so
// that the protocol can be driven on the CPU as well.
//
// A pair cut between CTAs leaves one piece per CTA; each piece is counted in at the pair's
// counter, and the arrival that completes the count merges the pieces.  A counter holds
// tag << 24 | count, the tag being 40 bits that differ from call to call.  A counter with
// another tag (an earlier call's, or workspace never written) counts as zero.  The
// arrival that completes a pair stores tag << 24 (count zero) in place of the full count,
// so the counter is zero again when the call ends: a later call with the same tag (a
// captured CUDA graph replayed) starts from zero as well.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define PA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define PA_HOST_DEVICE inline
#endif

namespace pa {

constexpr int kArriveTries = 1 << 20;
constexpr unsigned long long kArriveCountMask = 0xffffffull;

// Count one piece in at *ctr for a pair of n pieces.  cas(ptr, expected, desired) is an
// atomic compare-and-swap returning the old value; load(ptr) reads the counter.  Returns
// the count this arrival makes (1 .. n; n means it completed the pair), or -1 when `tries`
// compare-and-swaps in a row found the counter changed (the caller flags the pair).
#if defined(__CUDACC__)
#pragma nv_exec_check_disable
#endif
template <class Cas, class Load>
PA_HOST_DEVICE int arrive_count(unsigned long long* ctr, unsigned long long tag, int n, Cas cas,
                                Load load, int tries = kArriveTries) {
  unsigned long long cur = load(ctr);
  for (int t = 0; t < tries; ++t) {
    const unsigned long long base = (cur >> 24) == tag ? cur : (tag << 24);
    const int count = static_cast<int>(base & kArriveCountMask) + 1;
    const unsigned long long want = count >= n ? (tag << 24) : base + 1;
    const unsigned long long prev = cas(ctr, cur, want);
    if (prev == cur) return count;
    cur = prev;
  }
  return -1;
}

// The same with an atomic add once the counter carries this call's tag, which only arrivals
// of the pair's own pieces put there.  Compare-and-swaps that many arrivals make at once fail
// for all but one, a round trip to the L2 for each; adds all succeed.  One sequence of 512
// tokens with 8 kv heads, whose 16 pieces a head all end together: 67 us with swaps alone.
// A counter that turns out to hold a third call's tag is left to the loop above.
// add(ptr) adds one and returns the old value; store(ptr, value) writes the counter.
#if defined(__CUDACC__)
#pragma nv_exec_check_disable
#endif
template <class Cas, class Load, class Add, class Store>
PA_HOST_DEVICE int arrive_add(unsigned long long* ctr, unsigned long long tag, int n, Cas cas,
                              Load load, Add add, Store store) {
  unsigned long long cur = load(ctr);
  if ((cur >> 24) != tag) {
    const unsigned long long prev = cas(ctr, cur, n > 1 ? (tag << 24) + 1 : tag << 24);
    if (prev == cur) return 1;
    if ((prev >> 24) != tag) return arrive_count(ctr, tag, n, cas, load);
  }
  const int count = static_cast<int>(add(ctr) & kArriveCountMask) + 1;
  if (count < n) return count;
  store(ctr, tag << 24);
  return n;
}

}  // namespace pa
