// The cache write of FP8 K/V blocks that carry a scale for each (block, kv head)
// (pa_append_fp8_block).
//
// Format: E4M3 codes [num_blocks][Hkv][B][d] and float32 scales [num_blocks][Hkv]; a cached
// value is decode(code) * scale.  A scale is the smallest power of two 2^e with
// amax <= 448 * 2^e over the block's rows of that head.  For floating-point codes a scale
// only places the range, so a power of two costs no precision against amax / 448, and it
// buys two things: x / 2^e is exact, so a value is rounded once; and when a later token
// raises a block's scale, the codes of the earlier rows move by an exact factor, so they
// are rounded again only where they become subnormal.
//
// A call appends each sequence's new tokens (positions c - q .. c - 1) through the block
// table.  Per touched block and head: amax over the new rows (finite values), their scale
// 2^e, and s = max(2^e, the block's scale) when earlier rows live in the block (the first
// position is not at row 0), else 2^e; earlier rows are requantised when s grew.
//
// What bounds it is HBM: 4 d bytes in and 2 d out per token and kv head.  One warp owns one
// (block, head, K or V): at d = 128 and B = 16 its rows are 4 KB, eight 16-byte loads a
// lane, held in registers between the amax and the quantisation, so every byte moves once
// and nothing is shared between warps.  The tasks of a ragged batch are counted by a scan
// over the sequences that every CTA makes for itself, and cut into equal shares, so one
// long chunk among many single tokens keeps no SM waiting.  Measured on GB300, 13 ragged
// prompts of 300..2048 tokens (94 MB, floor 13.9 us at the copy peak), call after call on the same
// buffers, which the L2 holds: 23.3 us at first; 21.4 with the next task's table lookup under this
// one's loads; 16.3 with the magnitudes compared as integers, a second look only where one is not
// finite, and registers held to four CTAs an SM (three before).  Over rotating buffers 19.0 us, 73 %
// of the copy peak: a warp loads its rows, reduces and stores before it loads the next, so DRAM
// waits (41 % busy, 60 % of the issue slots used).  One token each of 64 sequences: 3.4 us.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_seq_scan.cuh"

namespace pa {
namespace {

struct AppendParams {
  const uint4* key;
  const uint4* value;
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* k_scales;
  float* v_scales;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  int num_seqs, num_tokens, num_blocks, num_kv_heads, max_blocks_per_seq;
  unsigned* err;
};

// A sequence's part of a call: its rows of key / value and the blocks they touch.
struct Span {
  int first_row;     // row of key / value of its first new token
  int pos, end;      // positions pos .. end - 1 are written
  int blocks;        // blocks touched (0: nothing to write)
  bool ok;
};

template <int B>
__device__ __forceinline__ Span span_of(const AppendParams& p, int s) {
  const long long a = __ldg(p.query_start + s), b = __ldg(p.query_start + s + 1);
  const long long c = __ldg(p.context_lens + s), q = b - a;
  Span sp;
  sp.ok = a >= 0 && q >= 0 && b <= p.num_tokens && c >= q &&
          c <= static_cast<long long>(p.max_blocks_per_seq) * B;
  sp.first_row = static_cast<int>(a);
  sp.pos = static_cast<int>(c - q);
  sp.end = static_cast<int>(c);
  sp.blocks = sp.ok && q > 0 ? (sp.end - 1) / B - sp.pos / B + 1 : 0;
  return sp;
}

// Larger of the magnitudes of eight 16-bit values and the running maximum `m` (bits without
// the sign, two lanes; they order as integers, infinities and NaN above everything).
// FINITE: values that are not finite are left out.
template <typename T, bool FINITE>
__device__ __forceinline__ uint32_t amax2(uint32_t m, const uint4& v) {
  constexpr uint32_t inf2 = std::is_same<T, __nv_bfloat16>::value ? 0x7f807f80u : 0x7c007c00u;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7fff7fffu;
    m = __vmaxu2(m, FINITE ? a & __vcmpltu2(a, inf2) : a);
  }
  return m;
}

// The scale of rows whose largest magnitude is amax: the smallest 2^e with amax <= 448 * 2^e,
// 448 = 1.75 * 2^8, e held in [-100, 120] (below, values under 2^-109 round to zero; a
// 16-bit float's largest value needs 2^120).  `inv` = 2^-e.
__device__ __forceinline__ float block_scale(float amax, float& inv) {
  const uint32_t b = __float_as_uint(amax);
  int e = static_cast<int>(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased
  e = min(120 + 127, max(-100 + 127, e));
  inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

// Eight 16-bit values times inv -> eight codes.
template <typename T>
__device__ __forceinline__ uint2 codes8(const uint4& v, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack2<T>(w[i]);
    o[i] = e4m3x2_of(x.y * inv, x.x * inv);
  }
  return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

// Four codes times `ratio`, rounded to codes again.
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float ratio) {
  const float2 a = e4m3x2_floats(static_cast<uint16_t>(c)), b = e4m3x2_floats(static_cast<uint16_t>(c >> 16));
  return static_cast<uint32_t>(e4m3x2_of(a.y * ratio, a.x * ratio)) |
         (static_cast<uint32_t>(e4m3x2_of(b.y * ratio, b.x * ratio)) << 16);
}

template <typename T, int D, int B>
__global__ void __launch_bounds__(kScanThreads, B == 32 && D == 128 ? 2 : 4) append_fp8_block_kernel(const AppendParams p) {
  constexpr int LPR = D / 8;          // lanes (16-byte vectors) per row
  constexpr int RPP = 32 / LPR;       // rows per pass of a warp
  constexpr int PASSES = B / RPP;
  __shared__ SeqScan scan;
  // the kernel before this one (say the projection that made key and value, or a decode that
  // still reads the cache) has finished past this point
  pdl_wait_primary();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.num_seqs + kScanThreads - 1) / kScanThreads;
  const int sa = min(p.num_seqs, tid * per), sb = min(p.num_seqs, sa + per);
  unsigned long long mine = 0;
  bool bad = false;
  for (int s = sa; s < sb; ++s) {
    const Span sp = span_of<B>(p, s);
    mine += sp.blocks;
    bad = bad || !sp.ok;
  }
  if (bad && blockIdx.x == 0) atomicOr(p.err, kErrBadContext);
  seq_scan(scan, mine);
  __syncthreads();
  const int parts = 2 * p.num_kv_heads;  // (K or V, head)
  const unsigned long long tasks = scan.pre[kScanThreads] * parts;
  const unsigned long long t1 = tasks * (blockIdx.x + 1) / gridDim.x;
  // this lane's 16-byte vector of rows r0, r0 + RPP, ..
  const int r0 = lane / LPR, ch = lane % LPR;
  const size_t row_step = static_cast<size_t>(p.num_kv_heads) * LPR;
  // Task t: (block, K or V, head).  The block of the last task is kept: a warp's tasks come
  // two by two (8 kv heads) or so from one block.
  unsigned long long have = ~0ull;  // the block (touched block number) that the next four tell of
  int blk = -1, a = 0, z = 0;       // its id; rows a .. z - 1 are new
  long long rows = 0;               // key / value vector of its row 0 (negative: before the array)
  auto block_of = [&](unsigned long long item) {
    if (item == have) return;
    have = item;
    const int u = seq_owner(scan, item);
    unsigned long long at = scan.pre[u];
    int s = u * per;
    Span sp = span_of<B>(p, s);
    while (item >= at + sp.blocks) {  // (ends inside the thread's share)
      at += sp.blocks;
      sp = span_of<B>(p, ++s);
    }
    const int j = sp.pos / B + static_cast<int>(item - at);
    blk = __ldg(p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq + j);
    a = max(sp.pos - j * B, 0);
    z = min(sp.end - j * B, B);
    // row r of the block is key row first_row + j * B + r - pos
    rows = (static_cast<long long>(sp.first_row) + j * B - sp.pos) * static_cast<long long>(row_step);
  };
  unsigned long long t = tasks * blockIdx.x / gridDim.x + warp;
  if (t < t1) block_of(t / parts);
  for (; t < t1; t += kScanWarps) {
    const int part = static_cast<int>(t % parts);
    const bool is_v = part >= p.num_kv_heads;
    const int h = is_v ? part - p.num_kv_heads : part;
    const int b0 = blk, a0 = a, z0 = z;
    const bool ok = b0 >= 0 && b0 < p.num_blocks;
    const size_t group = static_cast<size_t>(ok ? b0 : 0) * p.num_kv_heads + h;
    float* scale_at = (is_v ? p.v_scales : p.k_scales) + group;
    const float old = ok && a0 > 0 ? *scale_at : 0.f;
    const uint4* from = is_v ? p.value : p.key;
    const long long first = rows + h * LPR + ch;
    uint4 x[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = i * RPP + r0;
      x[i] = ok && r >= a0 && r < z0 ? from[first + r * static_cast<long long>(row_step)] : make_uint4(0u, 0u, 0u, 0u);
    }
    // the next task's block is looked up while these loads fly
    if (t + kScanWarps < t1) block_of((t + kScanWarps) / parts);
    if (!ok) {
      if (lane == 0) atomicOr(p.err, kErrBadBlock);
      continue;
    }
    // the largest finite magnitude, as 16-bit bits: a second look where something is not finite
    constexpr uint32_t kInf = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) m2 = amax2<T, false>(m2, x[i]);
    uint32_t top = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
    if (top >= kInf) {
      m2 = 0;
#pragma unroll
      for (int i = 0; i < PASSES; ++i) m2 = amax2<T, true>(m2, x[i]);
      top = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
    }
    const float amax = unpack2<T>(top).x;
    float inv;
    const float call = block_scale(amax, inv);
    float scale = call;
    uint2* dst = reinterpret_cast<uint2*>((is_v ? p.v_cache : p.k_cache) + group * (B * D)) + ch;
    if (a0 > 0) {
      if (old >= call) {
        scale = old;
        inv = __fdiv_rn(1.f, old);  // (exact: scales are powers of two)
      } else {
        const float ratio = __fdiv_rn(old, call);
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
          const int r = i * RPP + r0;
          if (r < a0) {
            uint2 c = dst[r * LPR];
            c.x = rescale4(c.x, ratio);
            c.y = rescale4(c.y, ratio);
            dst[r * LPR] = c;
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = i * RPP + r0;
      if (r >= a0 && r < z0) dst[r * LPR] = codes8<T>(x[i], inv);
    }
    if (lane == 0 && (a0 == 0 || scale != old)) *scale_at = scale;
  }
}

template <typename T, int D, int B>
cudaError_t launch(const AppendParams& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kScanThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append_fp8_block_kernel<T, D, B>, p);
}

}  // namespace

int append_fp8_block_launch(const void* key, const void* value, void* k_cache, void* v_cache,
                            float* k_scales, float* v_scales, const int32_t* block_tables,
                            int max_blocks_per_seq, const int32_t* context_lens,
                            const int32_t* query_start, int num_seqs, int num_tokens,
                            int num_blocks, int num_kv_heads, int head_dim, int block_size,
                            bool bf16, int sm_count, unsigned* err, cudaStream_t stream) {
  AppendParams p;
  p.key = static_cast<const uint4*>(key);
  p.value = static_cast<const uint4*>(value);
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.query_start = query_start;
  p.num_seqs = num_seqs;
  p.num_tokens = num_tokens;
  p.num_blocks = num_blocks;
  p.num_kv_heads = num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.err = err;
  // at most this many blocks are touched: a token each, and two partial blocks a sequence
  long long blocks = num_tokens / block_size + 2ll * num_seqs;
  if (blocks > num_tokens) blocks = num_tokens;
  long long grid = (blocks * 2 * num_kv_heads + kScanWarps - 1) / kScanWarps;
  const int resident = block_size == 32 && head_dim == 128 ? 2 : 4;  // CTAs per SM (registers)
  if (grid > static_cast<long long>(resident) * sm_count) grid = resident * sm_count;
  cudaError_t e = cudaErrorInvalidValue;
#define PA_APPEND_CASE(DD, BB)                                                  \
  if (head_dim == DD && block_size == BB)                                       \
    e = bf16 ? launch<__nv_bfloat16, DD, BB>(p, static_cast<int>(grid), stream) \
             : launch<__half, DD, BB>(p, static_cast<int>(grid), stream);
  PA_APPEND_CASE(128, 8)
  PA_APPEND_CASE(128, 16)
  PA_APPEND_CASE(128, 32)
  PA_APPEND_CASE(64, 8)
  PA_APPEND_CASE(64, 16)
  PA_APPEND_CASE(64, 32)
#undef PA_APPEND_CASE
  return e == cudaSuccess ? 0 : -3;
}

}  // namespace pa
