// Verification of drafted tokens against the target model's probabilities, from given random
// numbers (pa_verify_drafts).
//
// A sequence's q rows of the step hold its last token and q - 1 drafts x_1 .. x_{q-1}.  With p_i
// the target's probabilities after row i, d_i the distribution that draft x_{i+1} was drawn from
// and u_i uniform in [0, 1): drafts are accepted in order while u_i d_i(x_{i+1}) < p_i(x_{i+1}).
// At the first one refused, at row a, the token that takes its place is drawn from max(p_a - d_a, 0);
// after the last one accepted, a = q - 1, from p_a.  Then the tokens that come out have the target
// model's own distribution.  Drawn by inversion: the smallest t with C(t) > u_{q-1} C(V - 1), C the
// running sum of the weights.
//
// The running sum decides by comparison, and a rounded one decides differently from one order of
// addition to another.  So weights are whole numbers, p and d in units of 2^-56 (an fp32 value
// of 2^-33 and more exactly), their sums exact in 128 bits, and the comparison is
// floor(u C) as an integer product: the answer depends on no order, cut or cluster size.  The test
// of a draft multiplies two 24-bit numbers in fp64, exactly.
//
// What bounds it: the bytes of one row of p and, after a refusal, one of d per sequence; 4 V each
// in fp32.  A row is as long as an SM takes 20 us to read, so a cluster of CTAs shares a
// sequence: each adds up its stretch in chunks of 128 values and keeps the chunks' sums, the
// totals go round the cluster through distributed shared memory, and the CTA that holds the answer
// reads the one chunk again (from the L2).  Every CTA runs the short chain of tests itself.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 128;  // values a warp adds up at once, four to a lane
constexpr int kUnroll = 4;   // chunks of a warp whose loads are under way together
constexpr int kMaxVocab = 1 << 20;
constexpr int kMaxChunks = kMaxVocab / kChunk / kCluster;

using u64 = unsigned long long;
using u128 = unsigned __int128;

struct VerifyParams {
  const int32_t* tokens;
  const void* target;
  const void* draft;  // may be null: each draft was certain
  long long target_stride, draft_stride;  // values from row to row
  const float* uniforms;
  const int32_t* query_start;
  const int32_t* context_lens;
  int32_t* out_tokens;
  int32_t* emitted;
  int32_t* context_next;
  int num_seqs, num_tokens, vocab;
  unsigned* err;
};

__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ float value(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ float value(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// A probability in units of 2^-56; what is no number or negative counts as 0, above 1 as 1.
__device__ __forceinline__ u64 units(float x) { return __float2ull_rn(fminf(fmaxf(x, 0.f), 1.f) * 0x1p56f); }

// Four values of a row from `at` on (zeros past the row's end).  VEC: rows are aligned.
template <typename T, bool VEC>
__device__ __forceinline__ void load4(const T* row, int at, int vocab, float (&x)[4]) {
  if (VEC && at + 4 <= vocab) {
    if constexpr (std::is_same<T, float>::value) {
      const float4 v = *reinterpret_cast<const float4*>(row + at);
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(row + at);
      const float2 a = unpack2<T>(v.x), b = unpack2<T>(v.y);
      x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = at + i < vocab ? value(row + at + i) : 0.f;
  }
}

// The weight of value x of p with y of the draft (0 where there is none to take off).
__device__ __forceinline__ u64 weight(float x, float y) {
  const u64 a = units(x), b = units(y);
  return a > b ? a - b : 0;
}

__device__ __forceinline__ u64 shfl_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ u64 cluster_read(const u64* mine, int rank) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(mine)), "r"(rank));
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
  return v;
}

struct VerifySmem {
  u64 sum[kMaxChunks];   // of this CTA's chunks
  u64 total[2][2];       // its total (low, high), per pass
  int refused;           // the first draft refused
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ VerifySmem sm;
  // (the launch after this one may read context_next while this one drains: it is not let start early)
  pdl_wait_primary();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = blockIdx.x / kCluster, rank = blockIdx.x % kCluster;
  const int qs = p.query_start[s], qe = p.query_start[s + 1], ctx = p.context_lens[s];
  const bool span = qs >= 0 && qe >= qs && qe <= p.num_tokens;
  const int q = span ? qe - qs : 0;
  const bool ok = span && (q == 0 || ctx >= q);
  if (q == 0 || !ok) {  // (uniform over the cluster)
    // every CTA has read the lengths before they may be written over
    cluster_sync();
    if (rank == 0 && tid == 0) {
      if (!ok) atomicOr(p.err, kErrBadContext);
      p.emitted[s] = 0;
      p.context_next[s] = ctx;
    }
    return;
  }
  if (tid == 0) sm.refused = q - 1;
  __syncthreads();
  // ---- the drafts' tests ----
  const T* target = static_cast<const T*>(p.target) + qs * p.target_stride;
  const T* draft = p.draft ? static_cast<const T*>(p.draft) + qs * p.draft_stride : nullptr;
  for (int i = tid; i < q - 1; i += kThreads) {
    const int x = p.tokens[qs + i + 1];
    bool good = false;
    if (x >= 0 && x < p.vocab) {
      const float pt = value(target + i * p.target_stride + x);
      const float dt = draft ? value(draft + i * p.draft_stride + x) : 1.f;
      good = static_cast<double>(p.uniforms[qs + i]) * static_cast<double>(dt) < static_cast<double>(pt);
    }
    if (!good) {
      atomicMin(&sm.refused, i);
      break;
    }
  }
  __syncthreads();
  const int a = sm.refused;
  const bool refused = a < q - 1;
  const T* row = target + a * p.target_stride;
  const T* drow = refused && draft ? draft + a * p.draft_stride : nullptr;
  const int said = refused && !draft ? p.tokens[qs + a + 1] : -1;  // taken out whole
  const int chunks = (p.vocab + kChunk - 1) / kChunk, per = (chunks + kCluster - 1) / kCluster;
  const int c0 = min(chunks, rank * per), c1 = min(chunks, c0 + per);
  u64 lo = 0, hi = 0;
  int token = -1;
  // The second pass, over p alone, is for weights that are all zero (p <= d throughout).
  for (int pass = 0; pass < 2; ++pass) {
    const bool plain = pass == 1;
    auto weights = [&](int at, const float (&x)[4], const float (&y)[4], u64 (&w)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = !plain && at + i == said ? 0 : weight(x[i], y[i]);
    };
    for (int c = c0 + warp; c < c1; c += kWarps * kUnroll) {
      float x[kUnroll][4], y[kUnroll][4];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int ck = c + k * kWarps;
        const int at = ck < c1 ? ck * kChunk + lane * 4 : p.vocab;
        load4<T, VEC>(row, at, p.vocab, x[k]);
        if (drow && !plain) {
          load4<T, VEC>(drow, at, p.vocab, y[k]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) y[k][i] = 0.f;
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int ck = c + k * kWarps;
        u64 w[4];
        weights(ck * kChunk + lane * 4, x[k], y[k], w);
        const u64 sum = shfl_sum(w[0] + w[1] + w[2] + w[3]);
        if (lane == 0 && ck < c1) sm.sum[ck - c0] = sum;
      }
    }
    __syncthreads();
    if (warp == 0) {  // this CTA's total
      u128 t = 0;
      for (int c = lane; c < c1 - c0; c += 32) t += sm.sum[c];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const u64 l = __shfl_xor_sync(0xffffffffu, static_cast<u64>(t), o);
        const u64 h = __shfl_xor_sync(0xffffffffu, static_cast<u64>(t >> 64), o);
        t += (static_cast<u128>(h) << 64) | l;
      }
      if (lane == 0) {
        sm.total[pass][0] = static_cast<u64>(t);
        sm.total[pass][1] = static_cast<u64>(t >> 64);
      }
    }
    cluster_sync();
    u128 total = 0, before = 0, mine = 0;
#pragma unroll
    for (int r = 0; r < kCluster; ++r) {
      const u128 t = (static_cast<u128>(cluster_read(&sm.total[pass][1], r)) << 64) | cluster_read(&sm.total[pass][0], r);
      if (r < rank) before += t;
      if (r == rank) mine = t;
      total += t;
    }
    if (total == 0) continue;  // (uniform over the cluster)
    // the largest C(t) that is not above u total: floor(u total), u in units of 2^-64
    const float uf = p.uniforms[qe - 1];
    const u64 u = uf >= 1.f ? ~0ull : (uf > 0.f ? __double2ull_rd(static_cast<double>(uf) * 0x1p64) : 0ull);
    u128 at = (static_cast<u128>(u) * static_cast<u64>(total) >> 64) + static_cast<u128>(u) * static_cast<u64>(total >> 64);
    if (at >= before && at < before + mine) {
      // this CTA has it: the chunk, by one warp, then the place in it
      if (warp == 0) {
        u128 left = at - before;
        int c = 0;
        for (;; c += 32) {
          u64 v = c + lane < c1 - c0 ? sm.sum[c + lane] : 0;
          u128 incl = v;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const u64 l = __shfl_up_sync(0xffffffffu, static_cast<u64>(incl), o);
            const u64 h = __shfl_up_sync(0xffffffffu, static_cast<u64>(incl >> 64), o);
            if (lane >= o) incl += (static_cast<u128>(h) << 64) | l;
          }
          const uint32_t past = __ballot_sync(0xffffffffu, incl > left);
          if (past) {
            const int k = __ffs(past) - 1;
            const u128 pre = incl - v;
            const u64 l = __shfl_sync(0xffffffffu, static_cast<u64>(left - pre), k);
            c += k;
            left = l;  // (below one chunk's sum)
            break;
          }
          const u64 l = __shfl_sync(0xffffffffu, static_cast<u64>(incl), 31);
          const u64 h = __shfl_sync(0xffffffffu, static_cast<u64>(incl >> 64), 31);
          left -= (static_cast<u128>(h) << 64) | l;
        }
        const int e = (c0 + c) * kChunk + lane * 4;
        float x[4], y[4] = {0.f, 0.f, 0.f, 0.f};
        u64 w[4];
        load4<T, VEC>(row, e, p.vocab, x);
        if (drow && !plain) load4<T, VEC>(drow, e, p.vocab, y);
        weights(e, x, y, w);
        u64 incl = w[0] + w[1] + w[2] + w[3];
        const u64 all = incl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        const u64 rest = static_cast<u64>(left);
        if (incl > rest && incl - all <= rest) {
          u64 run = incl - all;
          token = e;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            run += w[i];
            if (run <= rest) token = e + i + 1;
          }
          p.out_tokens[qs + a] = token;
        }
      }
    }
    lo = static_cast<u64>(total);
    hi = static_cast<u64>(total >> 64);
    break;
  }
  // no CTA leaves while another may read its totals, and every one has read the lengths
  __syncthreads();
  cluster_sync();
  if (rank == 0) {
    const bool some = (lo | hi) != 0;
    for (int i = tid; i < q; i += kThreads) {
      if (i < a) p.out_tokens[qs + i] = p.tokens[qs + i + 1];
      else if (i > a || !some) p.out_tokens[qs + i] = -1;
    }
    if (tid == 0) {
      const int n = a + (some ? 1 : 0);
      p.emitted[s] = n;
      p.context_next[s] = ctx - q + n;
      if (!some) atomicOr(p.err, kErrBadProbs);
    }
  }
}

}  // namespace

int verify_max_vocab() { return kMaxVocab; }

int verify_drafts_launch(const VerifyArgs& a, cudaStream_t stream) {
  VerifyParams p;
  p.tokens = a.tokens;
  p.target = a.target;
  p.draft = a.draft;
  p.target_stride = a.target_stride;
  p.draft_stride = a.draft_stride;
  p.uniforms = a.uniforms;
  p.query_start = a.query_start;
  p.context_lens = a.context_lens;
  p.out_tokens = a.out_tokens;
  p.emitted = a.emitted;
  p.context_next = a.context_next;
  p.num_seqs = a.num_seqs;
  p.num_tokens = a.num_tokens;
  p.vocab = a.vocab;
  p.err = a.err;
  // four values at once where every row starts on such a boundary
  const int step = 4 * a.value_bytes;
  auto aligned = [&](const void* base, long long stride) {
    return reinterpret_cast<uintptr_t>(base) % step == 0 && stride % 4 == 0;
  };
  const bool vec = aligned(a.target, a.target_stride) && (!a.draft || aligned(a.draft, a.draft_stride));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.num_seqs * kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaErrorInvalidValue;
#define PA_VERIFY_CASE(TT) \
  e = vec ? cudaLaunchKernelEx(&cfg, verify_kernel<TT, true>, p) : cudaLaunchKernelEx(&cfg, verify_kernel<TT, false>, p)
  if (a.value_bytes == 4) PA_VERIFY_CASE(float);
  else if (a.bf16) PA_VERIFY_CASE(__nv_bfloat16);
  else PA_VERIFY_CASE(__half);
#undef PA_VERIFY_CASE
  return e == cudaSuccess ? 0 : -3;
}

}  // namespace pa
