// Rotary positions of a step's new tokens, with or without the cache write.
//
// The row of sequence s at place i of its q_len new ones has position p = context_lens[s] - q_len +
// i.  Pair j of the first rotary_dim values of each head, (x_j, x_{j + rotary_dim / 2}) or
// (x_{2j}, x_{2j+1}), is turned by the angle p f_j:
//   a' = (a cos - b sin) A,   b' = (b cos + a sin) A
// and the rest of the head is copied.  The turned keys and the values go through the block table
// into the cache, row p % B of block table[p / B].
//
// Angles are exact however far the position: f_j comes as turns per token in units of 2^-64, so
// p f_j is a 64-bit product whose overflow drops whole turns.  What is left, as a signed number of
// half turns, goes into sincospif: no table of cosines is read, and a position of a million is as
// good as one of ten.  (p times f_j in fp32 would be off by 0.06 radians there.)
//
// What bounds it: bytes, 4 d (Hq + 2 Hkv) a token, each read and written once; for single tokens a
// launch and three dependent loads (the row's sequence, its lengths, its block).  A CTA takes one
// token: its threads have their first loads of q, k and v under way before they look for the
// sequence, the angles are computed once for all heads, and a thread's unit is a pair of 16-byte
// chunks that holds both values of eight pairs.
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 3;  // units whose loads a thread starts before it knows the position

struct RotaryParams {
  const uint8_t* q;
  const uint8_t* key;
  const uint8_t* value;  // with the cache write only
  uint8_t* q_out;
  uint8_t* key_out;  // without it: rows as key's
  uint8_t* k_cache;  // with it
  uint8_t* v_cache;
  long long q_stride, key_stride, value_stride, q_out_stride, key_out_stride;  // bytes from row to row
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  const unsigned long long* freqs;  // [rotary_dim / 2] turns per token, 2^-64 each
  int num_seqs, num_tokens, num_q_heads, num_kv_heads, max_blocks_per_seq, log2_block, num_blocks;
  int turned;  // units (pairs of chunks) of a head that are turned: rotary_dim / 16
  float amplitude;
  unsigned* err;
};

// D: head size; PAIRS: neighbours are pairs (else the halves of the turned part); CACHE: k and v go
// into the cache.
template <typename T, int D, bool PAIRS, bool CACHE>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  constexpr int UN = D / 16;  // units of a head
  __shared__ float2 turn[D / 2];  // (cos, sin) A
  pdl_wait_primary();
  pdl_launch_dependents();
  const int tid = threadIdx.x, tok = blockIdx.x;
  const int rows = p.num_q_heads + (CACHE ? 2 : 1) * p.num_kv_heads, units = rows * UN;
  // unit u: of head u / UN (q's heads, k's, v's), its two chunks
  auto chunks = [&](int u, int* a, int* b) {
    const int c = u % UN;
    const bool v = CACHE && u / UN >= p.num_q_heads + p.num_kv_heads;
    if (!PAIRS && c < p.turned && !v) {
      *a = c;
      *b = c + p.turned;
    } else {
      *a = 2 * c;
      *b = 2 * c + 1;
    }
  };
  auto source = [&](int u) -> const uint4* {
    const int h = u / UN, hk = h - p.num_q_heads, hv = hk - p.num_kv_heads;
    const uint8_t* at = hk < 0 ? p.q + tok * p.q_stride + h * (D * 2)
                      : !CACHE || hv < 0 ? p.key + tok * p.key_stride + hk * (D * 2)
                                         : p.value + tok * p.value_stride + hv * (D * 2);
    return reinterpret_cast<const uint4*>(at);
  };
  uint4 xa[kAhead], xb[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int u = tid + k * kThreads;
    if (u < units) {
      int a, b;
      chunks(u, &a, &b);
      xa[k] = source(u)[a];
      xb[k] = source(u)[b];
    }
  }
  // the row's sequence: the first one with a possible span that holds it.  (Counting the spans that end at or
  // before it reads half as much, but beside a decreasing span finds one that does not hold it.)
  int found = p.num_seqs;
  bool wrong = false;
  for (int s = tid; s < p.num_seqs; s += kThreads) {
    const int qs = p.query_start[s], qe = p.query_start[s + 1];
    const bool span = qs >= 0 && qe >= qs && qe <= p.num_tokens;
    if (span && qs <= tok && tok < qe) found = min(found, s);
    wrong = wrong || !span;
  }
  if (wrong && tok == 0) atomicOr(p.err, kErrBadContext);  // (one CTA tells of impossible spans)
  found = __reduce_min_sync(0xffffffffu, found);
  __shared__ int part[kThreads / 32];
  if ((tid & 31) == 0) part[tid >> 5] = found;
  __syncthreads();
  int s = p.num_seqs;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s = min(s, part[w]);
  if (s >= p.num_seqs) return;  // of no sequence
  const int qs = p.query_start[s], qe = p.query_start[s + 1], ctx = p.context_lens[s];
  const long long cap = CACHE ? static_cast<long long>(p.max_blocks_per_seq) << p.log2_block : 0x7fffffffll;
  if (qe - qs > ctx || ctx > cap) {
    if (tid == 0) atomicOr(p.err, kErrBadContext);
    return;
  }
  const int pos = ctx - qe + tok;
  int block = 0;
  if (CACHE) block = p.block_tables[static_cast<size_t>(s) * p.max_blocks_per_seq + (pos >> p.log2_block)];
  for (int j = tid; j < p.turned * 8; j += kThreads) {
    // turns of this position, less the whole ones, in half turns: [-1, 1]
    const long long left = static_cast<long long>(p.freqs[j] * static_cast<unsigned long long>(pos));
    float sn, cs;
    sincospif(__ll2float_rn(left) * 0x1p-63f, &sn, &cs);
    turn[j] = make_float2(cs * p.amplitude, sn * p.amplitude);
  }
  const bool there = !CACHE || (block >= 0 && block < p.num_blocks);
  if (!there && tid == 0) atomicOr(p.err, kErrBadBlock);
  __syncthreads();
  const int row = pos & ((1 << p.log2_block) - 1);
  auto one = [&](int u, uint4 a, uint4 b) {
    const int h = u / UN, c = u % UN, hk = h - p.num_q_heads, hv = hk - p.num_kv_heads;
    if (c < p.turned && !(CACHE && hv >= 0)) {
      uint32_t* wa = reinterpret_cast<uint32_t*>(&a);
      uint32_t* wb = reinterpret_cast<uint32_t*>(&b);
      const float2* t = turn + 8 * c;
      if (PAIRS) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t& w = i < 4 ? wa[i] : wb[i - 4];
          const float2 x = unpack2<T>(w), r = t[i];
          w = pack2<T>(x.x * r.x - x.y * r.y, x.y * r.x + x.x * r.y);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = unpack2<T>(wa[i]), y = unpack2<T>(wb[i]), r = t[2 * i], z = t[2 * i + 1];
          wa[i] = pack2<T>(x.x * r.x - y.x * r.y, x.y * z.x - y.y * z.y);
          wb[i] = pack2<T>(y.x * r.x + x.x * r.y, y.y * z.x + x.y * z.y);
        }
      }
    }
    uint8_t* at;
    if (hk < 0) {
      at = p.q_out + tok * p.q_out_stride + h * (D * 2);
    } else if (!CACHE) {
      at = p.key_out + tok * p.key_out_stride + hk * (D * 2);
    } else {
      if (!there) return;
      const size_t r = ((static_cast<size_t>(block) * p.num_kv_heads + (hv < 0 ? hk : hv)) << p.log2_block) + row;
      at = (hv < 0 ? p.k_cache : p.v_cache) + r * (D * 2);
    }
    int ca, cb;
    chunks(u, &ca, &cb);
    reinterpret_cast<uint4*>(at)[ca] = a;
    reinterpret_cast<uint4*>(at)[cb] = b;
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int u = tid + k * kThreads;
    if (u < units) one(u, xa[k], xb[k]);
  }
  for (int u = tid + kAhead * kThreads; u < units; u += kThreads) {
    int a, b;
    chunks(u, &a, &b);
    const uint4 x = source(u)[a], y = source(u)[b];
    one(u, x, y);
  }
}

}  // namespace

int rotary_launch(const RotaryArgs& a, cudaStream_t stream) {
  RotaryParams p;
  p.q = static_cast<const uint8_t*>(a.q);
  p.key = static_cast<const uint8_t*>(a.key);
  p.value = static_cast<const uint8_t*>(a.value);
  p.q_out = static_cast<uint8_t*>(a.q_out);
  p.key_out = static_cast<uint8_t*>(a.key_out);
  p.k_cache = static_cast<uint8_t*>(a.k_cache);
  p.v_cache = static_cast<uint8_t*>(a.v_cache);
  p.q_stride = 2 * a.q_stride;
  p.key_stride = 2 * a.key_stride;
  p.value_stride = 2 * a.value_stride;
  p.q_out_stride = 2 * a.q_out_stride;
  p.key_out_stride = 2 * a.key_out_stride;
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.query_start = a.query_start;
  p.freqs = reinterpret_cast<const unsigned long long*>(a.freqs);
  p.num_seqs = a.num_seqs;
  p.num_tokens = a.num_tokens;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.log2_block = a.block_size == 8 ? 3 : (a.block_size == 16 ? 4 : 5);
  p.num_blocks = a.num_blocks;
  p.turned = a.rotary_dim / 16;
  p.amplitude = a.amplitude;
  p.err = a.err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.num_tokens);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaErrorInvalidValue;
#define PA_ROTARY_CASE(TT, DD)                                                                                \
  e = a.interleaved ? (a.k_cache ? cudaLaunchKernelEx(&cfg, rotary_kernel<TT, DD, true, true>, p)             \
                                 : cudaLaunchKernelEx(&cfg, rotary_kernel<TT, DD, true, false>, p))           \
                    : (a.k_cache ? cudaLaunchKernelEx(&cfg, rotary_kernel<TT, DD, false, true>, p)            \
                                 : cudaLaunchKernelEx(&cfg, rotary_kernel<TT, DD, false, false>, p))
  if (a.head_dim == 128) {
    if (a.bf16) PA_ROTARY_CASE(__nv_bfloat16, 128); else PA_ROTARY_CASE(__half, 128);
  } else if (a.head_dim == 64) {
    if (a.bf16) PA_ROTARY_CASE(__nv_bfloat16, 64); else PA_ROTARY_CASE(__half, 64);
  }
#undef PA_ROTARY_CASE
  return e == cudaSuccess ? 0 : -3;
}

}  // namespace pa
