// Attention of a few or many query rows per sequence over paged 16-bit K/V with the keys split
// over the SMs, for sm_103a: drafted tokens over their own long context (causal,
// pa_decode_drafts) and any tokens over an encoder's states (no mask, pa_cross).
//
// Row i of sequence s (q_len rows, context c) attends to t <= c - q_len + i, or to all t < c:
//   out = sum_t softmax_t(scale <q, K_t>) V_t
// Over a cut of the keys into pieces j, with m_j about the largest scaled score of a piece (in log2
// units), l_j = sum 2^(z_t - m_j) and O_j = sum 2^(z_t - m_j) V_t:
//   m = max_j m_j,   out = sum_j 2^(m_j - m) O_j / sum_j 2^(m_j - m) l_j
// which is exact, so a cut costs one fp32 rounding and no accuracy worth the name.
//
// What bounds it: with few rows the bytes of K and V (4 d bytes per key and kv head, each read
// once for all rows of its kv head), with many the two products (4 d operations per row and key).
// The prefill kernels give each (query tile, sequence, kv head) one SM, which walks all keys:
// four tokens over 8192 keys with 8 kv heads keep eight SMs busy.  Here the unit of work is 64
// keys of an item (a sequence, kv head and one or two 128-row query tiles): the batch's units are
// cut into equal shares, one per SM, wherever the cut falls, so a launch of few rows is balanced whatever
// its lengths are, and only items that a cut goes through are joined, by a second kernel.  (A causal item
// counts all keys of its context, although it stops at its last row's: of whole prompts the shares of
// early rows are short, and pa_prefill is faster.)
//
// Design: one CTA per SM (two, of one query tile at head_dim 64); every CTA finds its own share from
// the lengths (no host round trip, no counter to reset, and the cuts depend on lengths alone: the same bits
// whatever the blocks' places).  Its roles go from item to item at their own pace:
// * A query tile's rows are (token, query head of the kv head) pairs, 128 / G tokens x G heads.
//   tcgen05 multiplies all 128 rows whatever their number: at 8 kv heads of 128 in bf16 that is
//   65 K operations per key in the time in which an SM's share of HBM brings the key's 512
//   bytes, 40 % of the tensor rate, so few rows still stream at the memory's rate; the softmax,
//   which would not fit, runs in the warps that have rows only.  Weights enter P V rounded to the
//   input type, half a step each, since a product's operands have one type and V is not widened; their sum
//   is of the unrounded ones.
// * Two loader warps bring 64-key tiles of K and V into a ring, whole blocks by TMA (128-byte
//   swizzle).  What the last block holds behind the context is masked (K) or cleared in shared memory
//   (V).  Table entries are looked up 32 blocks at once, a batch ahead.  K's warp also walks the
//   share and announces its items.  A warp of its own brings q (of two query tiles, V's).
// * An MMA warp per query tile: S = Q K^T into tensor memory (two buffers), O += P V with P read
//   from tensor memory over the S it came from.  S of the next keys goes in before P V.
// * A softmax warpgroup per query tile, one thread per row, keeps m and l; O is rescaled only when
//   a row's maximum grows by more than 2^8.  f16 P is held up to 2^15, so that it rounds
//   weights below 2^-31 of the row's largest away, not below 2^-24.
// * Causal: V of keys that some row does not attend to may hold NaN or infinity, which a weight of
//   zero would spread; such values become zeros in shared memory before P V, and the rows that
//   do attend to those keys get them added as they go out.
// Every mbarrier wait is bounded (about 1 s) and checks a shared abort flag; after one that gave
// up the CTA still waits, as long again at most, for its copies and MMAs in flight.
//
// On GB300, device time: 64 contexts of 128..2048 with up to seven drafts, 32 query / 8 kv heads of
// 128, bf16, 55 us (285 MB, 5.2 TB/s); eight of 8..32 K with 5..16 rows 96 us (5.9 TB/s); 64 single rows
// over 100..1500 states, 16 heads of 64, fp16, 49 us; 32 prompts of 3..448 rows over the same 49 us; 6 texts
// of 900..2048 rows over 2000..8192 states, 32 / 8 heads, 460 us (1530 TFLOP/s) in bursts, 530 call after
// call (1330), when the power cap holds the SMs near 1.6 GHz.  With few rows a
// 64-key tile is a chain of fixed latencies (scores read 215 cycles, maximum 250, weights 125, stored and
// passed on 130, two waits of 100) against 690 (d = 64) or 1380 cycles of an SM's share of HBM: at d = 64
// that chain bounds the launch, twice over where items are a dozen tiles long and each costs its start
// and end.  Two CTAs an SM hide some of it (74 -> 51 us); of 128 they leave each a ring too short (98 -> 109).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_split_plan.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace split {

using namespace tc;

constexpr int kRows = 128;      // rows of a query tile (MMA M, tensor-memory lanes)
constexpr int kKeys = 64;       // keys of a K/V tile (MMA N of S, K of P V)
constexpr int kItems = 4;       // items in flight between the roles
constexpr int kMaxGrid = 1024;  // CTAs the workspace has descriptors for
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescale = 8.f;  // log2 growth of a row's maximum that forces a rescale of O
// Rows whose maximum is this far from zero (log2 units) have it taken off their scores before these are scaled
// (far_tiles).  Else a weight is one multiply-add of the score, relative to the scaled maximum rounded to fp32: half a
// step of it is 2^-12 at 2^12 (all of a row's weights share it), but past 2^24 a whole power of two and more, with which
// the largest weight leaves f16's or even fp32's range (scores of 4e8 in f16 came out as infinity or 0 / 0).
constexpr float kFar = 4096.f;
// P = 2^(z - m + lift) <= 2^15 in f16, whose smallest value is 2^-24: lift 7; bf16 needs none.
template <typename T>
__host__ __device__ constexpr float lift_of() { return std::is_same<T, __half>::value ? 7.f : 0.f; }

// What a cut item's first CTA leaves for the join: written by every CTA of every launch.
struct Join {
  int followers;  // CTAs after this one that hold a piece of the item; 0: nothing to join
  int s, g, qs, qlen, ctx, tok0, end;
};
// Flags of a piece.
constexpr int kFlagOdd = 1;  // V of keys that not all rows attend to was not finite and went in as 0
constexpr int kFlagBad = 2;  // (shifted by the query tile) a block id of the tile's keys is out of range

struct Params {
  CUtensorMap kmap;  // the caches as [num_blocks][Hkv][B][d] 16-bit, box (64, B, 1, 1)
  CUtensorMap vmap;
  CUtensorMap qmap;  // q as [tokens][Hq][d], box (64, G, 128 / G): one query tile's half
  int q_tma;         // qmap is valid (G divides 128)
  const uint8_t* q;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;  // [n + 1]
  uint8_t* out;
  Join* joins;    // [grid]
  float4* sums;   // [grid][2][query tiles * kRows] (m, l, flags, base) of a cut item's rows
  float4* parts;  // [grid][2][d / 4][query tiles * kRows] their O, row fastest
  int num_seqs, num_tokens, num_q_heads, num_kv_heads, group, tpt;  // tpt = tokens per query tile
  int max_blocks_per_seq, block_size, log2_block, num_blocks;
  uint32_t group_magic;  // ceil(2^16 / G): r / G = r * group_magic >> 16 for r < 128
  int cut;               // items may be cut (the join kernel follows)
  float scale_log2;
  unsigned* err;
};

// A sequence as the plan sees it.
struct Seq {
  int qs, qlen, ctx;
  int blocks;  // query blocks (items of one kv head); 0: nothing to do
  int tiles;   // key tiles of an item; 0: its rows are zeros
  bool ok;     // a possible span and context
};

template <bool CAUSAL>
__device__ __forceinline__ Seq seq_of(const Params& p, int s, int per_item) {
  Seq q;
  q.qs = p.query_start[s];
  const int qe = p.query_start[s + 1];
  q.ctx = p.context_lens[s];
  q.ok = q.qs >= 0 && qe >= q.qs && qe <= p.num_tokens;
  q.qlen = q.ok ? qe - q.qs : 0;
  q.blocks = (q.qlen + per_item - 1) / per_item;
  q.tiles = 0;
  if (q.qlen > 0) {
    const long long cap = static_cast<long long>(p.max_blocks_per_seq) << p.log2_block;
    q.ok = q.ctx >= (CAUSAL ? 1 : 0) && q.ctx <= cap && !(CAUSAL && q.qlen > q.ctx);
    if (q.ok) q.tiles = static_cast<int>((static_cast<long long>(q.ctx) + kKeys - 1) / kKeys);
  }
  return q;
}

// An item's piece as K's loader announces it.
struct Item {
  int run;  // 0: no more items
  int s, g, qs, qlen, ctx;
  int tok0, end;  // the item's tokens of the sequence
  int t0, t1;     // the piece's key tiles
  int slot;       // of the piece in the workspace; -1: the whole item, which goes to out
  int ok;         // (false: zeros)
  int flags;
};

// The end of the piece's key tiles for query tile t: up to the position of its last token.
template <bool CAUSAL>
__device__ __forceinline__ int tiles_end(const Item& it, int t, int tpt) {
  const int ntok = min(tpt, it.end - (it.tok0 + t * tpt));
  if (ntok <= 0) return it.t0;
  if (!CAUSAL) return it.t1;
  return max(it.t0, min(it.t1, (it.ctx - it.qlen + it.tok0 + t * tpt + ntok - 1) / kKeys + 1));
}

// The first key tile that not all rows of an item attend to.
__device__ __forceinline__ int first_masked(int ctx, int qlen, int tok0) {
  return (ctx - qlen + tok0 + 1) / kKeys;
}

template <int D, int NT>
struct Shape {
  static constexpr int kThreads = NT == 2 ? 384 : 256;
  static constexpr int kCtas = NT == 2 || D == 128 ? 1 : 2;  // per SM
  static constexpr int kStages = NT == 2 ? 4 : (D == 128 ? 5 : 4);
};
// Two CTAs of 256 threads have 128 registers a thread; the softmax warpgroup takes kSoftmaxRegs, the
// other keeps kOtherRegs (152 + 104 = 2 x 128).  136 to 148 bytes a thread spill all the same (-Xptxas -v), and
// 6 % of the launch's instructions are loads and stores of them.  (With one CTA an SM nothing spills with one
// query tile, 8 to 32 bytes with two.)
constexpr int kSoftmaxRegs = 152;
constexpr int kOtherRegs = 104;

template <int D, int NT>
struct Smem {
  static constexpr int kStages = Shape<D, NT>::kStages;
  uint8_t q[NT][kRows * D * 2];        // K-major, 128-byte swizzle; 1024-byte aligned
  uint8_t k[kStages][kKeys * D * 2];   // [64-column half][64 keys][128 B]
  uint8_t v[kStages][kKeys * D * 2];
  uint8_t stage[4 * NT][32 * 64];      // per softmax warp: 32 columns of its rows on their way out
  Item item[kItems];
  unsigned long long warp_sum[Shape<D, NT>::kThreads / 32];
  int from[3], to[3];                  // the share: (sequence, item of it, key tile), and its end
  long long first_cut;                 // of the item that the share's end cuts: units before the cut
  unsigned long long item_full[kItems], item_free[kItems];
  unsigned long long q_full[NT], q_free[NT];
  unsigned long long k_full[kStages], v_full[kStages];
  unsigned long long s_full[NT][2], p_full[NT][2];
  unsigned long long k_freed[kStages], v_freed[kStages];  // S, P V of them done, by every query tile
  // P V number i of the query tile done, at i % 2: the last two may both be under way when the
  // softmax waits, and a wait tells only neighbouring phases of a barrier apart
  unsigned long long pv_done[NT][2];
  unsigned long long fin[NT];          // an MMA warp's last commit
  uint32_t tmem;
  int abort;  // a wait gave up: every role stops
  // copies asked for so far (of an aborted CTA the last ones may be in flight)
  uint32_t sent[2], q_sent[NT];
};

// True where a 16-bit half of w is not finite.
template <typename T>
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
  constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
  constexpr uint32_t kOne = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
  return ((w & kExp) + kOne) & 0x80008000u;  // (an exponent of all ones carries into the sign's place)
}

// A finished value as T holds it.  Rounded weights over the sum of unrounded ones may lift an average
// of f16's largest values past them: such become the largest, infinities stay.
template <typename T>
__device__ __forceinline__ float fit(float x) {
  if (std::is_same<T, __half>::value) return fabsf(x) < 66000.f ? fminf(fmaxf(x, -65504.f), 65504.f) : x;
  return x;
}

// Adds what the values of V that went in as zeros give a row at position pos: to columns c0 .. c0 +
// n - 1 of its row of out, those that are not finite among the keys it attends to.
template <int D, typename T>
__device__ __forceinline__ void add_odd(const Params& p, int s, int g, int first_key, int pos, int c0, int n, T* out) {
  const int32_t* trow = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
#pragma unroll 1
  for (int key = first_key; key <= pos; ++key) {
    const size_t block = static_cast<size_t>(trow[key >> p.log2_block]) * p.num_kv_heads + g;
    const T* row = reinterpret_cast<const T*>(p.v_cache) + ((block << p.log2_block) + (key & (p.block_size - 1))) * D;
#pragma unroll 1
    for (int i = c0; i < c0 + n; ++i) {
      const float x = static_cast<float>(row[i]);
      if (!(fabsf(x) < INFINITY)) out[i] = from_float<T>(static_cast<float>(out[i]) + x);
    }
  }
}

// V of a key tile (in stage st, of item j) for P V, by kAll threads: keys from `rest` on, behind the context, become
// zeros, and so do, where not every row attends to all of the tile, values that are not finite.
template <int D, typename T, int NT, bool CAUSAL, int kAll>
__device__ __forceinline__ void tidy_tile(Smem<D, NT>& sm, int rest, bool masked, int j, uint32_t st, int me) {
  constexpr uint32_t kHalf = kKeys * 128, kStageBytes = kKeys * D * 2;
  const uint32_t v = smem_addr(sm.v[st]);
#pragma unroll 1
  for (int key = max(rest, 0) + (me >> 3); key < kKeys; key += kAll / 8)
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
      st_shared16(v + (me & 7) * 16 + h * kHalf + key * 128, make_uint4(0, 0, 0, 0));
  if (CAUSAL && masked) {
    const uint32_t at = v + me * 16;
    uint32_t odd = 0;
#pragma unroll 4
    for (int c = 0; c < static_cast<int>(kStageBytes / 16 / kAll); ++c) {
      if ((me + c * kAll) % (kHalf / 16) / 8 >= rest) continue;  // (behind the context: zeros)
      const uint4 w = ld_shared16(at + c * kAll * 16);
      odd |= odd_halves<T>(w.x) | odd_halves<T>(w.y) | odd_halves<T>(w.z) | odd_halves<T>(w.w);
    }
    if (odd) {
      // (the flag first: who finds the zeros has to find it)
      atomicOr(&sm.item[j % kItems].flags, kFlagOdd);
      __threadfence_block();
      auto clean = [](uint32_t x) -> uint32_t { return x & ~((odd_halves<T>(x) >> 15) * 0xffffu); };
#pragma unroll 1
      for (int c = 0; c < static_cast<int>(kStageBytes / 16 / kAll); ++c) {
        const uint4 w = ld_shared16(at + c * kAll * 16);
        st_shared16(at + c * kAll * 16, make_uint4(clean(w.x), clean(w.y), clean(w.z), clean(w.w)));
      }
    }
  }
  fence_async_smem();
  __syncwarp();
}

// What the softmax keeps of a row: its weights are relative to base * scale + m in log2 units.
struct RowState {
  float m, l, base;
  int ok;  // no wait gave up
};

// A warp's softmax over an item's key tiles k .. ntt - 1 where a row's maximum is far from zero.  A maximum that grows
// becomes the row's base, a score, which is taken off the others before they are scaled.  S of tile k has been waited for,
// its V is tidy, and O is relative to f.m; `last` is the last key that this row attends to.  A function that is not
// inlined: with this in the loop of near rows, in any of six forms, that loop lost 2 to 10 % to registers.
template <int D, typename T, int NT, bool CAUSAL>
__device__ __noinline__ RowState far_tiles(Smem<D, NT>* smp, unsigned* err, float scale_log2, RowState f, int k, int ntt,
                                           uint32_t sn, uint32_t num, int t0, int ctx, int qlen, int tok0, int j,
                                           uint32_t tl, int t, int last) {
  Smem<D, NT>& sm = *smp;
  constexpr int kStages = Shape<D, NT>::kStages;
  constexpr uint32_t kColS = kKeys, kColO = 2 * kKeys;
  const int r = threadIdx.x & (kRows - 1), lane = threadIdx.x & 31;
  auto wwait = [&](unsigned long long& bar, uint32_t parity) -> bool {
    const bool done = mbar_wait_bounded(smem_addr(&bar), parity, &sm.abort);
    if (!done && atomicExch(&sm.abort, 1) == 0) atomicOr(err, kErrTimeout);
    return __all_sync(0xffffffffu, done) != 0;
  };
  f.ok = 0;
  for (bool first = true; k < ntt; first = false, ++k, ++sn) {
    const int b = sn & 1, kt = t0 + k;
    if (!first) {
      if (!wwait(sm.s_full[t][b], (sn >> 1) & 1)) return f;
      tc_fence_after();
      const bool masked = CAUSAL && kt >= first_masked(ctx, qlen, tok0);
      if (NT == 1 && (ctx - kt * kKeys < kKeys || masked)) {
        const uint32_t x = num + k;
        if (!wwait(sm.v_full[x % kStages], (x / kStages) & 1)) return f;
        tidy_tile<D, T, NT, CAUSAL, kRows>(sm, ctx - kt * kKeys, masked, j, x % kStages, r);
      }
    }
    const int lim = last < 0 ? -1 : last - kt * kKeys;
    float top = -INFINITY;
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      float x[32];
      tmem_get32(tl + b * kColS + 32 * h, x);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (32 * h + i <= lim) top = fmaxf(top, x[i]);
    }
    const float mx = (top - f.base) * scale_log2;
    bool need = f.m == -INFINITY ? top > -INFINITY : mx > f.m + kRescale;
    if (first && top > -INFINITY && f.m == mx) {  // (taken up, and O rescaled, before the call)
      f.base = top;
      f.m = 0.f;
      need = false;
    }
    if (__any_sync(0xffffffffu, need)) {
      float alpha = 1.f;
      if (need) {
        alpha = f.m == -INFINITY ? 0.f : ex2(f.m - mx);
        f.l *= alpha;
        f.base = top;
        f.m = 0.f;
      }
      if (k > 0) {
        if (!wwait(sm.pv_done[t][(sn - 1) & 1], ((sn - 1) >> 1) & 1)) return f;
        tc_fence_after();
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          float o[32];
          tmem_get32(tl + kColO + c0, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= alpha;
          tmem_st32(tl + kColO + c0, o);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      }
    }
    const float off = (f.m == -INFINITY ? 0.f : -f.m) + lift_of<T>();
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      float x[32];
      uint32_t pk[16];
      tmem_get32(tl + b * kColS + 32 * h, x);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        x[i] = 32 * h + i <= lim ? ex2(fmaf(x[i] - f.base, scale_log2, off)) : 0.f;
        f.l += x[i];
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) pk[i] = pack2<T>(x[2 * i], x[2 * i + 1]);
      tmem_st16(tl + b * kColS + 16 * h, pk);
    }
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&sm.p_full[t][b]));
  }
  f.ok = 1;
  return f;
}

template <int D, typename T, int NT, bool CAUSAL>
__global__ void __launch_bounds__(Shape<D, NT>::kThreads, Shape<D, NT>::kCtas) split_kernel(const __grid_constant__ Params p) {
  constexpr int kThreads = Shape<D, NT>::kThreads;
  constexpr int kStages = Shape<D, NT>::kStages;
  constexpr int kLoadWarp = 4 * NT;  // K, and the share's items; V and q by the next
  constexpr int kMmaWarp = kLoadWarp + 2;
  constexpr int kQueryWarp = NT == 1 ? 7 : kLoadWarp + 1;  // loads q
  constexpr int CH = D / 8;              // 16-byte chunks of a 16-bit row
  constexpr int KS1 = D / 16;            // MMA k-steps of S = Q K^T
  constexpr int KS2 = kKeys / 16;        // MMA k-steps of P V
  constexpr uint32_t kTileCols = 256;    // TMEM columns per query tile:
  constexpr uint32_t kColS = kKeys;      //   S number i in [64 (i % 2), + 64), its P over the first
  constexpr uint32_t kColO = 2 * kKeys;  //   32 of those columns, O in [128, 128 + D)
  constexpr uint32_t kTmemCols = NT * kTileCols;
  constexpr uint32_t kHalf = kKeys * 128;  // bytes of a 64-column half of a K/V tile
  constexpr uint32_t kStageBytes = kKeys * D * 2;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_addr(smem_raw);
  using Sm = Smem<D, NT>;
  Sm& sm = *reinterpret_cast<Sm*>(smem_raw + (((raw_addr + 1023) & ~1023u) - raw_addr));

  pdl_wait_primary();
  pdl_launch_dependents();

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (known to be uniform over the warp)
  const int tpt = p.tpt, G = p.group, per_item = NT * tpt;
  T* outp = reinterpret_cast<T*>(p.out);

  // ---- set-up: barriers, tensor memory, and this CTA's share of the batch's units ----
  if (warp == kMmaWarp && lane == 0) {
    for (int i = 0; i < kItems; ++i) {
      mbar_init(smem_addr(&sm.item_full[i]), 1);
      mbar_init(smem_addr(&sm.item_free[i]), kThreads / 32 - 1);  // every warp but K's loader
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&sm.k_full[i]), 1);
      mbar_init(smem_addr(&sm.v_full[i]), 1);
      mbar_init(smem_addr(&sm.k_freed[i]), NT);
      mbar_init(smem_addr(&sm.v_freed[i]), NT);
    }
    for (int t = 0; t < NT; ++t) {
      mbar_init(smem_addr(&sm.q_full[t]), 33);  // TMA expect-tx + 32 copy lanes
      mbar_init(smem_addr(&sm.q_free[t]), 1);
      mbar_init(smem_addr(&sm.fin[t]), 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_addr(&sm.s_full[t][b]), 1);
        mbar_init(smem_addr(&sm.p_full[t][b]), 4);  // one lane of each softmax warp
        mbar_init(smem_addr(&sm.pv_done[t][b]), 1);
      }
    }
    fence_mbar_init();
    sm.abort = 0;
    sm.sent[0] = sm.sent[1] = 0;
    for (int t = 0; t < NT; ++t) sm.q_sent[t] = 0;
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&sm.tmem)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // Units: a key tile each, and kItemCost per item.  Thread u adds up its sequences' units; the
  // share's two ends are placed by the threads whose sequences they fall into.
  {
    const int per = (p.num_seqs + kThreads - 1) / kThreads;
    const int sa = min(p.num_seqs, tid * per), sb = min(p.num_seqs, sa + per);
    long long mine = 0;
    bool wrong = false;
    for (int s = sa; s < sb; ++s) {
      const Seq q = seq_of<CAUSAL>(p, s, per_item);
      mine += static_cast<long long>(q.blocks) * p.num_kv_heads * item_units(q.tiles);
      wrong = wrong || !q.ok;
    }
    if (wrong && blockIdx.x == 0) atomicOr(p.err, kErrBadContext);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sm.warp_sum[warp] = static_cast<unsigned long long>(incl);
    if (tid == 0) {
      sm.from[0] = sm.to[0] = p.num_seqs;
      sm.from[1] = sm.from[2] = sm.to[1] = sm.to[2] = 0;
      sm.first_cut = 0;
    }
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const long long x = static_cast<long long>(sm.warp_sum[w]);
      if (w < warp) before += x;
      total += x;
    }
    const long long at0 = before + incl - mine;
    const long long share = share_units(total, gridDim.x, p.cut);
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
      const long long x = (blockIdx.x + e) * share;
      if (x < at0 || x >= at0 + mine || x >= total) continue;
      long long at = at0;
      for (int s = sa; s < sb; ++s) {
        const Seq q = seq_of<CAUSAL>(p, s, per_item);
        const long long all = item_units(q.tiles) * q.blocks * p.num_kv_heads;
        if (x < at + all) {
          const Place end = place_of(x - at, q.tiles, p.cut);
          int* to = e ? sm.to : sm.from;
          to[0] = s;
          to[1] = static_cast<int>(end.item);
          to[2] = end.tile;
          if (e) sm.first_cut = end.off;
          break;
        }
        at += all;
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0) {
      // the item that the share's end cuts, if this CTA has its start
      Join j = {};
      if (sm.to[2] > 0) {
        const Seq q = seq_of<CAUSAL>(p, sm.to[0], per_item);
        const bool head = sm.from[0] < sm.to[0] || sm.from[1] < sm.to[1] || sm.from[2] == 0;
        if (head) {
          j.followers = followers_of(q.tiles, sm.first_cut, share);
          j.s = sm.to[0];
          j.g = sm.to[1] / q.blocks;
          j.qs = q.qs;
          j.qlen = q.qlen;
          j.ctx = q.ctx;
          j.tok0 = (sm.to[1] % q.blocks) * per_item;
          j.end = min(q.qlen, j.tok0 + per_item);
        }
      }
      if (p.cut) p.joins[blockIdx.x] = j;
    }
  }
  const uint32_t tmem = sm.tmem;
  // a bounded wait; on failure every role stops (the flag is checked inside the waits)
  auto wait = [&](unsigned long long& bar, uint32_t parity) -> bool {
    if (mbar_wait_bounded(smem_addr(&bar), parity, &sm.abort)) return true;
    if (atomicExch(&sm.abort, 1) == 0) atomicOr(p.err, kErrTimeout);
    return false;
  };
  auto wwait = [&](unsigned long long& bar, uint32_t parity) -> bool {  // warp-uniform result
    return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
  };
  // Item number j, once it is announced (false: a wait gave up).  A role hands it back with
  // item_done when it has no more use for the slot.
  auto item_get = [&](int j, Item& it) -> bool {
    if (!wwait(sm.item_full[j % kItems], (j / kItems) & 1)) return false;
    it = sm.item[j % kItems];
    return true;
  };
  auto item_done = [&](int j) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&sm.item_free[j % kItems]));
  };

  if (Shape<D, NT>::kCtas == 2) {
    if (warp < 4) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  }
  // An item's q, load number `loads`: each query tile once the last item's S of it are done.  A whole one
  // (tpt tokens x G heads = 128 rows, each token's G rows contiguous in q) by TMA, one copy per
  // 64-column half; a tile that runs past its sequence by 16-byte copies of the rows it has (the others'
  // S and O are garbage of their own lanes, which nothing reads).
  auto load_q = [&](const Item& it, uint32_t loads) -> bool {
    for (int t = 0; t < NT; ++t) {
      if (loads > 0 && !wwait(sm.q_free[t], (loads - 1) & 1)) return false;
      const int first = it.tok0 + t * tpt;
      const bool tma = p.q_tma && first + tpt <= it.end;
      if (lane == 0) {
        sm.q_sent[t] = loads + 1;
        mbar_arrive_expect_tx(smem_addr(&sm.q_full[t]), tma ? kRows * D * 2 : 0);
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          if (tma)
            tma_load_3d(smem_addr(sm.q[t]) + h * kRows * 128, &p.qmap, h * 64, it.g * G, it.qs + first,
                        smem_addr(&sm.q_full[t]));
      }
      __syncwarp();
      if (!tma) {
        const int live = min(tpt, it.end - first) * G * CH;
#pragma unroll 4
        for (int u = lane; u < live; u += 32) {
          const int r = u / CH, c = u % CH;
          const int tl = static_cast<int>((r * p.group_magic) >> 16);  // r / G
          const uint8_t* src =
              p.q + ((static_cast<size_t>(it.qs + first + tl) * p.num_q_heads + it.g * G + r - tl * G) * D + c * 8) * 2;
          cp_async16(smem_addr(sm.q[t]) + swz(kRows, r, c), src, 16u);
        }
      }
      cp_async_arrive(smem_addr(&sm.q_full[t]));
    }
    return true;
  };
  // V of a key tile before P V: rows behind the context become zeros, and so do values that are not finite
  // from the first tile on that not every row attends to all of (a weight of zero would spread them).
  // By every warp whose P V follows, so that one finds the zeros of another, or writes the same.  (In
  // the softmax, which has more threads; of two query tiles in the MMA warps, since there the softmax's
  // registers would spill: 460 -> 510 us on 6 x 900..2048 rows over 2000..8192 keys.)
  constexpr bool kTidySoftmax = NT == 1;
  auto untidy = [&](const Item& it, int kt) -> bool {
    return it.ctx - kt * kKeys < kKeys || (CAUSAL && kt >= first_masked(it.ctx, it.qlen, it.tok0));
  };
  auto tidy = [&](const Item& it, int j, int kt, uint32_t st, int me, auto all) {
    tidy_tile<D, T, NT, CAUSAL, decltype(all)::value>(
        sm, it.ctx - kt * kKeys, kt >= first_masked(it.ctx, it.qlen, it.tok0), j, st, me);
  };
  // The item's key tiles end here for its query tiles together.
  auto item_end = [&](const Item& it, int* e0, int* e1) -> int {
    *e0 = tiles_end<CAUSAL>(it, 0, tpt);
    *e1 = NT == 2 ? tiles_end<CAUSAL>(it, 1, tpt) : *e0;
    return max(*e0, *e1);
  };

  if (warp == kLoadWarp || warp == kLoadWarp + 1) {
    // ===== loaders: K and the share's items; V =====
    const bool is_v = warp == kLoadWarp + 1;
    const uint32_t el = elect_one();
    const CUtensorMap* tmap = is_v ? &p.vmap : &p.kmap;
    const int B = p.block_size, nbk = kKeys >> p.log2_block;
    uint32_t num = 0, loads = 0;  // key tiles and q loads so far
    Seq sq = {};
    int s = sm.from[0], i = sm.from[1], tile = sm.from[2];
    const int es = sm.to[0], ei = sm.to[1], et = sm.to[2];
    if (!is_v && s < p.num_seqs) sq = seq_of<CAUSAL>(p, s, per_item);
    bool ok = true;
    for (int j = 0; ok; ++j) {
      Item it = {};
      if (is_v) {
        if (!(ok = item_get(j, it))) break;
      } else {
        if (s < p.num_seqs && i >= sq.blocks * p.num_kv_heads) {
          // the next sequence with rows (32 at once: most of a padded batch may have none)
          i = tile = 0;
          for (++s; s < p.num_seqs; s += 32) {
            Seq x = {};
            if (s + lane < p.num_seqs) x = seq_of<CAUSAL>(p, s + lane, per_item);
            const uint32_t some = __ballot_sync(0xffffffffu, x.blocks > 0);
            if (some) {
              s += __ffs(some) - 1;
              sq = seq_of<CAUSAL>(p, s, per_item);
              break;
            }
          }
          s = min(s, p.num_seqs);
        }
        it.run = s < p.num_seqs && (s < es || (s == es && (i < ei || (i == ei && tile < et))));
        if (it.run) {
          it.s = s;
          it.qs = sq.qs;
          it.qlen = sq.qlen;
          it.ctx = sq.ctx;
          it.ok = sq.tiles > 0;
          it.g = i / sq.blocks;
          it.tok0 = (i - it.g * sq.blocks) * per_item;
          it.end = min(sq.qlen, it.tok0 + per_item);
          it.t0 = tile;
          it.t1 = s == es && i == ei ? et : sq.tiles;
          it.slot = tile > 0 ? 2 * static_cast<int>(blockIdx.x)
                             : (it.t1 < sq.tiles ? 2 * static_cast<int>(blockIdx.x) + 1 : -1);
          ++i;
          tile = 0;
        }
        if (j >= kItems && !(ok = wwait(sm.item_free[j % kItems], (j / kItems - 1) & 1))) break;
        if (lane == 0) {
          sm.item[j % kItems] = it;
          mbar_arrive(smem_addr(&sm.item_full[j % kItems]));
        }
        __syncwarp();
      }
      if (!it.run) break;
      int e0, e1;
      const int n = item_end(it, &e0, &e1);
      if (is_v) {
        item_done(j);
        if (NT == 2 && n > it.t0 && !(ok = load_q(it, loads++))) break;
      }
      const int32_t* trow = p.block_tables + static_cast<size_t>(it.s) * p.max_blocks_per_seq;
      // Table entries, 32 blocks (4 to 16 key tiles) at once, a lane each, loaded as long before they are
      // used: one lookup a tile, rotated through registers, held each tile up for the latency of the last.
      const int per_batch = 32 >> (6 - p.log2_block);  // key tiles
      auto lookup = [&](int first) -> int {
        const long long lb = static_cast<long long>(first) * nbk + lane;
        return first + lane / nbk < n && (lb << p.log2_block) < it.ctx ? trow[lb] : -1;
      };
      int entry = 0, coming = n > it.t0 ? lookup(it.t0) : -1;
      uint32_t used = 0, there = 0;  // of the batch's blocks: hold keys; and have a block id
      for (int kt = it.t0; kt < n; ++kt, ++num) {
        const int x = (kt - it.t0) & (per_batch - 1);
        if (x == 0) {
          entry = coming;
          coming = lookup(kt + per_batch);
          used = __ballot_sync(0xffffffffu, kt + lane / nbk < n &&
                                                (static_cast<long long>(kt) * nbk + lane) << p.log2_block < it.ctx);
          there = __ballot_sync(0xffffffffu, entry >= 0 && entry < p.num_blocks) & used;
        }
        const int st = num % kStages;
        if (num >= kStages && !(ok = wwait(is_v ? sm.v_freed[st] : sm.k_freed[st], (num / kStages - 1) & 1))) break;
        const uint32_t to = smem_addr(is_v ? sm.v[st] : sm.k[st]);
        const uint32_t full = smem_addr(is_v ? &sm.v_full[st] : &sm.k_full[st]);
        // the blocks that hold keys of the context, whole: what lies behind the context is masked (K), or
        // cleared before it is used (V)
        const uint32_t mask = there >> (x * nbk) & ((1u << nbk) - 1);
        if ((used & ~there) >> (x * nbk) & ((1u << nbk) - 1) && lane == 0) {
          // (for the query tiles that need these keys: before the keys are announced to them)
          atomicOr(&sm.item[j % kItems].flags, (kt < e0 ? kFlagBad : 0) | (NT == 2 && kt < e1 ? kFlagBad << 1 : 0));
          atomicOr(p.err, kErrBadBlock);
        }
        if (lane == 0) {
          sm.sent[is_v] = num + 1;
          mbar_arrive_expect_tx(full, static_cast<uint32_t>(__popc(mask)) * B * D * 2);
        }
        __syncwarp();
        // four blocks straight through, predicated (a loop over the blocks took 150 cycles for each)
#pragma unroll 1
        for (int b0 = 0; b0 < nbk; b0 += 4) {
          int e[4];
#pragma unroll
          for (int b = 0; b < 4; ++b) e[b] = __shfl_sync(0xffffffffu, entry, x * nbk + b0 + b);
          const uint32_t four = mask >> b0;
#pragma unroll
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int h = 0; h < D / 64; ++h)  // 64-column halves
              tma_load_4d_el(to + h * kHalf + (b0 + b) * B * 128, tmap, h * 64, 0, it.g, e[b], full, el & (four >> b));
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (NT == 1 && warp == kQueryWarp) {
    Item it;
    uint32_t loads = 0;
    for (int j = 0; item_get(j, it) && it.run; ++j) {
      item_done(j);
      int e0, e1;
      if (item_end(it, &e0, &e1) > it.t0 && !load_q(it, loads++)) break;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= kMmaWarp && warp < kMmaWarp + NT) {
    // ============ MMA issue: a warp per query tile ============
    // The tensor pipe runs one thread's MMAs in order, so S of a key tile may overwrite the P of
    // the tile two before, whose P V was issued earlier.  A warp whose query tile needs no more
    // keys still frees each stage, after it has landed.
    const int t = warp - kMmaWarp;
    const uint32_t el = elect_one();
    constexpr uint32_t id_s = idesc_f16<T>(kRows, kKeys, false);
    constexpr uint32_t id_o = idesc_f16<T>(kRows, D, true);
    const uint64_t qd = desc_sw128(smem_addr(sm.q[t]), 16, 1024);
    const uint64_t dk0 = desc_sw128(smem_addr(sm.k[0]), 16, 1024);
    const uint64_t dv0 = desc_sw128(smem_addr(sm.v[0]), kKeys * 128, 1024);
    const uint32_t cols = tmem + t * kTileCols;
    auto issue_s = [&](uint32_t sn, uint32_t st) {  // S number sn of this query tile, K in stage st
      const uint32_t d = cols + (sn & 1) * kColS;
      const uint64_t kd = dk0 + ((st * kStageBytes) >> 4);
#pragma unroll
      for (int ks = 0; ks < KS1; ++ks)  // 16 columns = 32 bytes of 64-column block ks / 4
        mma_el(d, qd + (((ks >> 2) * kRows * 128 + (ks & 3) * 32) >> 4),
               kd + (((ks >> 2) * kKeys * 128 + (ks & 3) * 32) >> 4), id_s, ks > 0, el);
      commit_el(smem_addr(&sm.s_full[t][sn & 1]), el);
    };
    auto issue_pv = [&](uint32_t sn, uint32_t st, bool first) {
      const uint32_t pa = cols + (sn & 1) * kColS, o = cols + kColO;
      const uint64_t vd = dv0 + ((st * kStageBytes) >> 4);
#pragma unroll
      for (int ks = 0; ks < KS2; ++ks)  // 16 keys = 8 columns of P
        mma_ts_el(o, pa + ks * 8, vd + ((ks * 16 * 128) >> 4), id_o, !first || ks > 0, el);
    };
    uint32_t sn = 0, num = 0, loads = 0;  // S of this query tile, key tiles, q loads so far
    Item it;
    bool ok = true;
    for (int j = 0; ok && (ok = item_get(j, it)); ++j) {
      if (!__shfl_sync(0xffffffffu, it.run, 0)) break;
      item_done(j);
      // (broadcast, so that the loops are known to be uniform)
      const int e0 = tiles_end<CAUSAL>(it, 0, tpt), e1 = NT == 2 ? tiles_end<CAUSAL>(it, 1, tpt) : e0;
      const int n = __shfl_sync(0xffffffffu, max(e0, e1) - it.t0, 0);
      const int ntt = __shfl_sync(0xffffffffu, (t == 0 ? e0 : e1) - it.t0, 0);
      if (n <= 0) continue;
      if (!(ok = wwait(sm.q_full[t], loads & 1))) break;
      ++loads;
      fence_async_smem();  // q rows that lanes copied -> tensor cores
      // K of key tile number x: S number sx of it, if this query tile needs it, and the stage back
      auto keys = [&](uint32_t x, bool needed, uint32_t sx) -> bool {
        const uint32_t st = x % kStages;
        if (!wwait(sm.k_full[st], (x / kStages) & 1)) return false;
        if (needed) issue_s(sx, st);
        commit_el(smem_addr(&sm.k_freed[st]), el);
        return true;
      };
      if (!(ok = keys(num, ntt > 0, sn))) break;
      if (ntt <= 1) commit_el(smem_addr(&sm.q_free[t]), el);
      for (int kt = 0; kt < n; ++kt, ++num) {
        if (kt + 1 < n) {
          if (!(ok = keys(num + 1, kt + 1 < ntt, sn + 1))) break;
          if (kt + 2 == ntt) commit_el(smem_addr(&sm.q_free[t]), el);  // the item's last S
        }
        const uint32_t st = num % kStages;
        if (!(ok = wwait(sm.v_full[st], (num / kStages) & 1))) break;
        if (kt < ntt) {
          if (!(ok = wwait(sm.p_full[t][sn & 1], (sn >> 1) & 1))) break;
          if (!kTidySoftmax && untidy(it, it.t0 + kt))
            tidy(it, j, it.t0 + kt, st, lane, std::integral_constant<int, 32>());
          tc_fence_after();
          issue_pv(sn, st, kt == 0);
          commit_el(smem_addr(&sm.pv_done[t][sn & 1]), el);
          ++sn;
        }
        commit_el(smem_addr(&sm.v_freed[st]), el);
      }
    }
    commit_el(smem_addr(&sm.fin[t]), el);  // every MMA this warp issued
    wwait(sm.fin[t], 0);
  } else if (warp < 4 * NT) {
    // ================= softmax: warpgroup t, one thread per row =================
    const int t = warp >> 2, r = tid & (kRows - 1);
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + t * kTileCols;
    const int tile_tok = static_cast<int>((r * p.group_magic) >> 16);  // r / G
    uint32_t sn = 0, num = 0;  // S of this query tile and key tiles so far
    Item it;
    bool ok = true;
    for (int j = 0; ok && (ok = item_get(j, it)) && it.run; ++j) {
      const int e0 = tiles_end<CAUSAL>(it, 0, tpt), e1 = NT == 2 ? tiles_end<CAUSAL>(it, 1, tpt) : e0;
      const int n = max(e0, e1) - it.t0, ntt = (t == 0 ? e0 : e1) - it.t0;
      const int toks = max(0, min(tpt, it.end - (it.tok0 + t * tpt)));  // tokens of this query tile
      const bool row_ok = tile_tok < toks;
      const bool warp_ok = (r & ~31) < toks * G;  // (uniform: this warp has rows)
      const int pos_lo = it.ctx - it.qlen + it.tok0 + t * tpt;  // the tile's first position
      const int pos = row_ok ? pos_lo + tile_tok : -1;
      float m_run = -INFINITY, l_run = 0.f;
      int k = 0;
      for (; k < ntt; ++k, ++sn) {
        const int b = sn & 1, kt = it.t0 + k;
        if (!(ok = wwait(sm.s_full[t][b], (sn >> 1) & 1))) break;
        tc_fence_after();
        if (kTidySoftmax && untidy(it, kt)) {
          const uint32_t x = num + k;
          if (!(ok = wwait(sm.v_full[x % kStages], (x / kStages) & 1))) break;
          tidy(it, j, kt, x % kStages, r, std::integral_constant<int, kRows>());
        }
        if (warp_ok) {
          float sv[kKeys];
          tmem_get64(tl + b * kColS, sv);
          // mask on the raw scores: past the position, or past the context.  The scores stay
          // unscaled (the scale is positive, so the maximum commutes with it) and P =
          // 2^(s * scale - m + lift) is one multiply-add per element.
          const int lim = (CAUSAL ? pos : it.ctx - 1) - kt * kKeys;
          if (CAUSAL ? kt * kKeys + kKeys - 1 > pos_lo : lim < kKeys - 1) {
#pragma unroll
            for (int i = 0; i < kKeys; ++i)
              if (i > lim) sv[i] = -INFINITY;
          }
          float pm[4];  // four chains of three-input maxima
#pragma unroll
          for (int i = 0; i < 4; ++i) pm[i] = fmaxf(sv[2 * i], sv[2 * i + 1]);
#pragma unroll
          for (int i = 8; i < kKeys; i += 8)
#pragma unroll
            for (int c = 0; c < 4; ++c) pm[c] = fmax3(pm[c], sv[i + 2 * c], sv[i + 2 * c + 1]);
          const float top = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])), mx = top * p.scale_log2;
          // (an item's first maximum grows from -inf)
          const bool need = row_ok && mx > m_run + kRescale;
          if (__any_sync(0xffffffffu, need)) {
            float alpha = 1.f;
            if (need) {
              alpha = ex2(m_run - mx);
              l_run *= alpha;
              m_run = mx;
            }
            if (k > 0) {
              // rescale O, once P V of the tile before is done (the one before that was issued
              // before this S)
              if (!(ok = wwait(sm.pv_done[t][(sn - 1) & 1], ((sn - 1) >> 1) & 1))) break;
              tc_fence_after();
#pragma unroll
              for (int c0 = 0; c0 < D; c0 += 32) {
                float o[32];
                tmem_get32(tl + kColO + c0, o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= alpha;
                tmem_st32(tl + kColO + c0, o);
              }
              asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            }
            // far from zero: far_tiles does the rest of the item
            if (__any_sync(0xffffffffu, row_ok && fabsf(m_run) >= kFar && top > -INFINITY)) break;
          }
          // P over this thread's own row of S, already in registers, rounded to the input type; its
          // unrounded sum in l (a row with every score at -inf so far: any finite offset gives 0)
          const float off = (m_run == -INFINITY ? 0.f : -m_run) + lift_of<T>();
          const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), of2 = make_float2(off, off);
          float2 ps[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                          make_float2(0.f, 0.f)};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 x = __ffma2_rn(make_float2(sv[32 * h + i], sv[32 * h + i + 1]), sc2, of2);
              const float2 e = make_float2(ex2(x.x), ex2(x.y));
              ps[(i >> 1) & 3] = __fadd2_rn(ps[(i >> 1) & 3], e);
              pk[i >> 1] = pack2<T>(e.x, e.y);
            }
            tmem_st16(tl + b * kColS + 16 * h, pk);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          const float2 sum = __fadd2_rn(__fadd2_rn(ps[0], ps[1]), __fadd2_rn(ps[2], ps[3]));
          l_run += sum.x + sum.y;
        }
        tc_fence_before();  // the P stores before the MMA warp reads them
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.p_full[t][b]));
      }
      float base = 0.f;
      if (ok && k < ntt) {
        const RowState f = far_tiles<D, T, NT, CAUSAL>(&sm, p.err, p.scale_log2, RowState{m_run, l_run, 0.f, 1}, k, ntt, sn,
                                                       num, it.t0, it.ctx, it.qlen, it.tok0, j, tl, t,
                                                       row_ok ? (CAUSAL ? pos : it.ctx - 1) : -1);
        m_run = f.m;
        l_run = f.l;
        base = f.base;
        ok = f.ok;
        sn += ntt - k;
      }
      if (!ok) break;
      if (ntt > 0 && !(ok = wwait(sm.pv_done[t][(sn - 1) & 1], ((sn - 1) >> 1) & 1))) break;
      tc_fence_after();
      num += max(0, n);
      // (this query tile's keys are done, so what concerns it is final)
      const int flags = *reinterpret_cast<volatile int*>(&sm.item[j % kItems].flags);
      const bool bad = flags & (kFlagBad << t);
      if (it.slot >= 0) {
        // ---- a piece: m, l and O for the join, row fastest: a warp's store is 512 bytes ----
        const size_t row0 = static_cast<size_t>(it.slot) * (NT * kRows) + t * kRows + r;
        if (warp_ok) {
          p.sums[row0] = make_float4(m_run, l_run, __int_as_float((bad ? kFlagBad : 0) | (flags & kFlagOdd)), base);
          if (ntt > 0) {
            float4* to = p.parts + static_cast<size_t>(it.slot) * (D / 4) * (NT * kRows) + t * kRows + r;
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 32) {
              float o[32];
              tmem_get32(tl + kColO + c0, o);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                to[(c0 / 4 + i) * (NT * kRows)] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
          }
        }
        item_done(j);
      } else {
        item_done(j);
        if (warp_ok) {
          // ---- out = O / l, through shared memory, 32 columns at a time, so that each store
          // instruction of a warp writes eight rows' 64 bytes.  Row r's 16-byte chunk c sits at
          // chunk c ^ (r / 2 % 4) of its 64-byte staging row: neither the writes nor the reads
          // collide in a bank. ----
          const bool good = it.ok && !bad;
          const bool odd = CAUSAL && good && (flags & kFlagOdd);
          const float inv = 1.f / l_run;
          const uint32_t stage = smem_addr(sm.stage[warp]);
          const int ch = lane & 3;
          T* to = outp + (static_cast<size_t>(it.qs + it.tok0 + t * tpt) * p.num_q_heads + it.g * G) * D + ch * 8;
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 32) {
            float o[32];
            if (good) {  // (uniform over the warp)
              tmem_get32(tl + kColO + c0, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = fit<T>(o[i] * inv);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = 0.f;
            }
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
              uint4 w;
              w.x = pack2<T>(o[8 * cc], o[8 * cc + 1]);
              w.y = pack2<T>(o[8 * cc + 2], o[8 * cc + 3]);
              w.z = pack2<T>(o[8 * cc + 4], o[8 * cc + 5]);
              w.w = pack2<T>(o[8 * cc + 6], o[8 * cc + 7]);
              st_shared16(stage + lane * 64 + ((cc ^ ((lane >> 1) & 3)) << 4), w);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int rr = 8 * i + (lane >> 2), row = (r - lane) + rr;  // token tk of the tile, head row % G
              const int tk = static_cast<int>((row * p.group_magic) >> 16);
              const uint4 w = ld_shared16(stage + rr * 64 + ((ch ^ ((rr >> 1) & 3)) << 4));
              if (tk < toks)
                *reinterpret_cast<uint4*>(to + static_cast<size_t>(tk * (p.num_q_heads - G) + row) * D + c0) = w;
            }
            __syncwarp();  // the reads before the next columns' stores
          }
          if (odd && row_ok) {
            // the values of V that went in as zeros (rare: a later draft's row is not finite)
            T* row = outp + ((static_cast<size_t>(it.qs + it.tok0 + t * tpt + tile_tok) * p.num_q_heads) + it.g * G +
                             r - tile_tok * G) * D;
            add_odd<D, T>(p, it.s, it.g, first_masked(it.ctx, it.qlen, it.tok0) * kKeys, pos, 0, D, row);
          }
          __syncwarp();
        }
      }
      // the O loads before this warp's next P, which lets the next item's P V overwrite O
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (sm.abort) {
    // what is in flight ends before the CTA leaves its memory (every role has stopped)
    if (tid == 0) {
      bool ended = true;
      auto land = [&](unsigned long long& bar, uint32_t sent) {  // the last of `sent` phases
        if (sent > 0) ended = mbar_wait_limit(smem_addr(&bar), (sent - 1) & 1) && ended;
      };
      for (uint32_t st = 0; st < kStages; ++st) {
        land(sm.k_full[st], (sm.sent[0] + kStages - 1 - st) / kStages);
        land(sm.v_full[st], (sm.sent[1] + kStages - 1 - st) / kStages);
      }
      for (int t = 0; t < NT; ++t) land(sm.q_full[t], sm.q_sent[t]), land(sm.fin[t], 1);
      if (!ended) atomicOr(p.err, kErrTimeout);
    }
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

// The join of cut items: grid (CTAs of the launch before, query tiles, 16-column groups), a thread
// per row.  Pieces are added in order of their keys.
template <int D, typename T, int NT, bool CAUSAL>
__global__ void __launch_bounds__(kRows) join_kernel(const __grid_constant__ Params p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const Join j = p.joins[blockIdx.x];
  if (j.followers <= 0) return;
  const int t = blockIdx.y, c4 = blockIdx.z * 4, r = threadIdx.x;
  const int tpt = p.tpt, G = p.group, tok = static_cast<int>((r * p.group_magic) >> 16);
  const int toks = min(tpt, j.end - (j.tok0 + t * tpt));
  if (tok >= toks) return;
  // piece f: slot 1 of the first CTA, slot 0 of the others; four loads under way together
  const int pieces = j.followers + 1, at = t * kRows + r;
  auto slot = [&](int f) -> size_t { return 2 * (blockIdx.x + f) + (f == 0 ? 1 : 0); };
  const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
  auto sum_of = [&](int f) { return f < pieces ? p.sums[slot(f) * (NT * kRows) + at] : none; };
  // the largest reference, as (m, base); log2 of a piece's weight over its
  float m = -INFINITY, base = 0.f;
  auto above = [&](const float4& x) { return (x.w - base) * p.scale_log2 + (x.x - m); };
  int flags = 0;
  for (int f0 = 0; f0 < pieces; f0 += 4) {
    float4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = sum_of(f0 + k);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      flags |= __float_as_int(x[k].z);
      if (x[k].y != 0.f && (m == -INFINITY || above(x[k]) > 0.f)) {
        m = x[k].x;
        base = x[k].w;
      }
    }
  }
  float l = 0.f;
  float4 o[4] = {};
  for (int f0 = 0; f0 < pieces; f0 += 2) {
    float4 x[2], v[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      x[k] = sum_of(f0 + k);
      const float4* from = p.parts + slot(f0 + k) * (D / 4) * (NT * kRows) + at;
#pragma unroll
      for (int c = 0; c < 4; ++c) v[k][c] = f0 + k < pieces ? from[(c4 + c) * (NT * kRows)] : none;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (x[k].y == 0.f) continue;  // no key of the piece counts for this row: no O was written, or zeros
      const float w = ex2(above(x[k]));
      l += x[k].y * w;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        o[c].x += v[k][c].x * w;
        o[c].y += v[k][c].y * w;
        o[c].z += v[k][c].z * w;
        o[c].w += v[k][c].w * w;
      }
    }
  }
  const float inv = 1.f / l;
  float x[16];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    x[4 * c] = fit<T>(o[c].x * inv);
    x[4 * c + 1] = fit<T>(o[c].y * inv);
    x[4 * c + 2] = fit<T>(o[c].z * inv);
    x[4 * c + 3] = fit<T>(o[c].w * inv);
  }
  if (flags & kFlagBad) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
  }
  uint4 w[2];
  uint32_t* ww = reinterpret_cast<uint32_t*>(w);
#pragma unroll
  for (int i = 0; i < 8; ++i) ww[i] = pack2<T>(x[2 * i], x[2 * i + 1]);
  T* row_out = reinterpret_cast<T*>(p.out) +
               (static_cast<size_t>(j.qs + j.tok0 + t * tpt + tok) * p.num_q_heads + j.g * G + r - tok * G) * D;
  uint4* to = reinterpret_cast<uint4*>(row_out + 4 * c4);
  to[0] = w[0];
  to[1] = w[1];
  if (CAUSAL && (flags & kFlagOdd) && !(flags & kFlagBad))
    add_odd<D, T>(p, j.s, j.g, first_masked(j.ctx, j.qlen, j.tok0) * kKeys, j.ctx - j.qlen + j.tok0 + t * tpt + tok,
                  4 * c4, 16, row_out);
}

template <int D, typename T, int NT, bool CAUSAL>
int launch(const Params& p, int sm_count, cudaStream_t stream) {
  const int grid = sm_count * Shape<D, NT>::kCtas;
  const size_t smem = sizeof(Smem<D, NT>) + 1024;
  auto* kern = split_kernel<D, T, NT, CAUSAL>;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), smem)) return -3;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(Shape<D, NT>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return -3;
  if (!p.cut) return 0;
  cfg.gridDim = dim3(grid, NT, D / 16);
  cfg.blockDim = dim3(kRows);
  cfg.dynamicSmemBytes = 0;
  if (cudaLaunchKernelEx(&cfg, join_kernel<D, T, NT, CAUSAL>, p) != cudaSuccess) return -3;
  return 0;
}

template <int D, typename T>
int launch2(const Params& p, bool two, bool causal, int sm_count, cudaStream_t stream) {
  if (causal)
    return two ? launch<D, T, 2, true>(p, sm_count, stream) : launch<D, T, 1, true>(p, sm_count, stream);
  return two ? launch<D, T, 2, false>(p, sm_count, stream) : launch<D, T, 1, false>(p, sm_count, stream);
}

size_t joins_bytes() { return sizeof(Join) * kMaxGrid; }
// (two query tiles a CTA, or two CTAs an SM)
size_t sums_bytes(int sm_count) { return sizeof(float4) * static_cast<size_t>(sm_count) * 2 * 2 * kRows; }

}  // namespace split

size_t split_workspace_bytes(int sm_count, int head_dim) {
  return split::joins_bytes() + split::sums_bytes(sm_count) +
         sizeof(float) * static_cast<size_t>(sm_count) * 2 * 2 * split::kRows * head_dim;
}

int split_attention_launch(const PrefillArgs& a, int num_tokens, bool causal, void* workspace, int sm_count,
                           cudaStream_t stream) {
  if (2 * sm_count > split::kMaxGrid) return -1;
  split::Params p;
  if (!kv_cache_map(&p.kmap, a.k_cache, 2, a.num_blocks, a.num_kv_heads, a.block_size, a.head_dim) ||
      !kv_cache_map(&p.vmap, a.v_cache, 2, a.num_blocks, a.num_kv_heads, a.block_size, a.head_dim))
    return -3;
  p.q = static_cast<const uint8_t*>(a.q);
  p.k_cache = static_cast<const uint8_t*>(a.k_cache);
  p.v_cache = static_cast<const uint8_t*>(a.v_cache);
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.query_start = a.query_start;
  p.out = static_cast<uint8_t*>(a.out);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  p.joins = reinterpret_cast<split::Join*>(w);
  p.sums = reinterpret_cast<float4*>(w + split::joins_bytes());
  p.parts = reinterpret_cast<float4*>(w + split::joins_bytes() + split::sums_bytes(sm_count));
  p.num_seqs = a.num_seqs;
  p.num_tokens = num_tokens;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.tpt = split::kRows / p.group;
  p.group_magic = (65536u + p.group - 1) / p.group;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.block_size = a.block_size;
  p.log2_block = a.block_size == 8 ? 3 : (a.block_size == 16 ? 4 : 5);
  p.num_blocks = a.num_blocks;
  p.scale_log2 = a.scale * split::kLog2e;
  p.q_tma = q_tile_map(&p.qmap, a.q, a.num_q_heads, a.head_dim, p.group, num_tokens) ? 1 : 0;
  p.err = a.err;
  // no context that the tables can hold is long enough for two pieces: no join
  p.cut = static_cast<long long>(a.max_blocks_per_seq) * a.block_size > (2 * split::kLeastPiece - 1) * split::kKeys;
  // Two query tiles per item, which share each key tile's loads, where sequences have the rows: 6 x 900..2048
  // rows of four heads each 460 us.  With 119 rows a sequence one tile takes 48.8 us, two 54.
  const bool two = static_cast<long long>(num_tokens) * p.group > static_cast<long long>(split::kRows) * a.num_seqs;
  if (a.head_dim == 128)
    return a.bf16 ? split::launch2<128, __nv_bfloat16>(p, two, causal, sm_count, stream)
                  : split::launch2<128, __half>(p, two, causal, sm_count, stream);
  if (a.head_dim == 64)
    return a.bf16 ? split::launch2<64, __nv_bfloat16>(p, two, causal, sm_count, stream)
                  : split::launch2<64, __half>(p, two, causal, sm_count, stream);
  return -1;
}

}  // namespace pa
