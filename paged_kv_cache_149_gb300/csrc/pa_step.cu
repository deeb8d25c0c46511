// The bookkeeping of one serving step on the GPU: block tables and slots from request
// lengths (pa_build_step).
//
// A request with c tokens of context, q of them new, holds ceil((c - q) / B) blocks and
// needs ceil(c / B) (horeb.top "vLLM PagedAttention：大模型推理的显存管理革命", section
// 分配策略; aiqz.cc "vLLM PagedAttention engine", section 分页存储设计); the new blocks come
// from the head of the free list in request order, and token p of the request goes to slot
// table[p / B] * B + p % B.
//
// What bounds it is latency, not bytes (64 requests with one new token each: 2.3 KB): a
// launch, one round of loads, a scan, one dependent round of loads.  So there is one launch
// and no CTA waits for another: every CTA scans all requests by itself (one per thread up
// to 256 of them; the lengths come from L2), then fills its own stretch of slots.  A table
// entry is written by the token that opens its block: every block a step adds holds exactly
// one new token at row 0.  Measured on GB300 (device time): 64 requests with one token each
// 2.5 us; 256 requests with up to 2048 each (127 K of them) 4.5 us, of which 0.2 are bytes.
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_seq_scan.cuh"

namespace pa {
namespace {

constexpr int kSlotsPerThread = 4;

struct StepParams {
  const int32_t* query_lens;
  const int32_t* context_lens;
  const int32_t* free_blocks;
  const int32_t* free_start;
  int32_t* block_tables;
  int64_t* slot_mapping;
  int32_t* query_start;
  int32_t* free_next;
  int num_seqs, num_free, max_blocks_per_seq, log2_block, num_blocks, num_slots;
  unsigned* err;
};

// A request as the step sees it.  An impossible one (negative counts, more new tokens than
// context, a context beyond the table) keeps its place in the token order (q) and gets no
// blocks.
struct Request {
  long long q;  // new tokens, at least 0
  int have, need;
  int c;
  bool ok;
};

__device__ __forceinline__ Request request_of(const StepParams& p, int s) {
  const int q = __ldg(p.query_lens + s), c = __ldg(p.context_lens + s);
  Request r;
  r.q = q > 0 ? q : 0;
  r.c = c;
  r.ok = q >= 0 && c >= q &&
         c <= (static_cast<long long>(p.max_blocks_per_seq) << p.log2_block);
  const long long up = (1ll << p.log2_block) - 1;
  r.have = r.ok ? static_cast<int>((c - q + up) >> p.log2_block) : 0;
  r.need = r.ok ? static_cast<int>((c + up) >> p.log2_block) - r.have : 0;
  return r;
}

__global__ void __launch_bounds__(kScanThreads) build_step_kernel(const StepParams p) {
  __shared__ SeqScan tok, blk;
  const int tid = threadIdx.x;
  const int per = (p.num_seqs + kScanThreads - 1) / kScanThreads;
  const int sa = min(p.num_seqs, tid * per), sb = min(p.num_seqs, sa + per);
  const int start = __ldg(p.free_start);
  unsigned long long tokens = 0, need = 0;
  bool bad = false;
  for (int s = sa; s < sb; ++s) {
    const Request r = request_of(p, s);
    tokens += r.q;
    need += r.need;
    bad = bad || !r.ok;
  }
  seq_scan(tok, tokens);
  seq_scan(blk, need);
  __syncthreads();
  const unsigned long long total = tok.pre[kScanThreads], want = blk.pre[kScanThreads];
  // all or nothing: a step that lacks blocks, or slots for its tokens, assigns none
  const bool enough = start >= 0 && start <= p.num_free &&
                      want <= static_cast<unsigned long long>(p.num_free - start);
  const bool fits = total <= static_cast<unsigned long long>(p.num_slots);
  const bool go = enough && fits;
  if (blockIdx.x == 0) {
    unsigned long long at = tok.pre[tid];
    auto clip = [](unsigned long long x) {
      return static_cast<int32_t>(x < 0x7fffffffull ? x : 0x7fffffffull);
    };
    for (int s = sa; s < sb; ++s) {
      p.query_start[s] = clip(at);
      const int q = __ldg(p.query_lens + s);
      at += q > 0 ? q : 0;
    }
    if (tid == 0) {
      p.query_start[p.num_seqs] = clip(total);
      *p.free_next = go ? start + static_cast<int>(want) : start;
      const unsigned e = (enough ? 0u : kErrNoBlocks) | (fits ? 0u : kErrBadSlot);
      if (e) atomicOr(p.err, e);
    }
    if (bad) atomicOr(p.err, kErrBadContext);
  }
  const int bmask = (1 << p.log2_block) - 1;
  bool bad_block = false;
  for (long long t = static_cast<long long>(blockIdx.x) * kScanThreads + tid; t < p.num_slots;
       t += static_cast<long long>(gridDim.x) * kScanThreads) {
    int64_t slot = -1;
    if (go && static_cast<unsigned long long>(t) < total) {
      const int u = seq_owner(tok, t);
      unsigned long long at = tok.pre[u], nb = blk.pre[u];
      int s = u * per;
      Request r = request_of(p, s);
      while (static_cast<unsigned long long>(t) >= at + r.q) {  // (ends inside the thread's share)
        at += r.q;
        nb += r.need;
        r = request_of(p, ++s);
      }
      if (r.ok) {
        const int pos = r.c - static_cast<int>(r.q) + static_cast<int>(t - at);
        const int j = pos >> p.log2_block, row = pos & bmask;
        int32_t* entry = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq + j;
        const int b = j < r.have ? *entry
                                 : __ldg(p.free_blocks + start + static_cast<int>(nb) + (j - r.have));
        if (b >= 0 && b < p.num_blocks) {
          slot = (static_cast<int64_t>(b) << p.log2_block) + row;
          if (j >= r.have && row == 0) *entry = b;
        } else {
          bad_block = true;
        }
      }
    }
    p.slot_mapping[t] = slot;
  }
  if (bad_block) atomicOr(p.err, kErrBadBlock);
}

}  // namespace

int build_step_launch(const int32_t* query_lens, const int32_t* context_lens, int num_seqs,
                      const int32_t* free_blocks, int num_free, const int32_t* free_start,
                      int32_t* block_tables, int max_blocks_per_seq, int block_size,
                      int num_blocks, int64_t* slot_mapping, int num_slots, int32_t* query_start,
                      int32_t* free_next, int sm_count, unsigned* err, cudaStream_t stream) {
  StepParams p;
  p.query_lens = query_lens;
  p.context_lens = context_lens;
  p.free_blocks = free_blocks;
  p.free_start = free_start;
  p.block_tables = block_tables;
  p.slot_mapping = slot_mapping;
  p.query_start = query_start;
  p.free_next = free_next;
  p.num_seqs = num_seqs;
  p.num_free = num_free;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.log2_block = block_size == 8 ? 3 : (block_size == 16 ? 4 : 5);
  p.num_blocks = num_blocks;
  p.num_slots = num_slots;
  p.err = err;
  const int per_cta = kScanThreads * kSlotsPerThread;
  int grid = num_slots / per_cta + (num_slots % per_cta != 0);
  if (grid > 4 * sm_count) grid = 4 * sm_count;
  if (grid < 1) grid = 1;
  // Launched plainly, and it lets no dependent start early: it writes block tables, which
  // the decode kernels read while the kernel before them drains.
  build_step_kernel<<<grid, kScanThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

}  // namespace pa
