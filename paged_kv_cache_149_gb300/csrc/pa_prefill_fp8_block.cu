// Paged prefill attention over FP8 (E4M3) K/V blocks with a scale for each (block, kv head),
// for sm_103a: causal multi-query attention of each sequence's newest tokens over its paged
// context, on the 5th-generation tensor cores (tcgen05).
//
// With K_t = sK_t code(K_t), V_t likewise (s: the scale of token t's block and head), the token
// at position p attends to positions t <= p:
//   out = sum_t softmax_t(scale <q, K_t>) V_t
// (daiw.org "Paged Attention", section 回顾与衔接).
//
// Everything runs on the tensor cores in f16, whatever q's type: an E4M3 code is exact there, the
// widening is one instruction for two values, and P keeps 11 bits.  The scales stay out of the
// operands, so no scale, of a key that a row attends to or of one that it does not, costs another
// key's code a bit.  K's multiply the scores in the softmax, a factor per group of keys.  V's go
// into the weights, 2^(z_t + log2 sV_t - r), r a reference of each row's own: the largest
// z + log2 sV among the keys that it attends to (moved when outgrown, with O), so that f16 rounds
// weights where they count in O; the sum of weights takes the factor out again, group by group.
// Each bf16 row of q is multiplied by the power of two that brings its largest value to
// [2^14, 2^15).
//
// Design: persistent CTAs of 640 threads, one per SM; a work item is a (pair of 128-row query
// tiles, sequence, kv head).  The grid has a CTA per item; a running CTA claims items of CTAs
// that have not started (cluster launch control), so the SMs balance themselves, and its roles
// go from item to item at their own pace: the next item's codes, K, V and q arrive while this
// one's last tiles are multiplied and written out.  (One CTA per item spent about 13600 cycles
// of its 34000, 8 prompts of 2048 tokens, on starting up and writing out alone.)  A call with few
// items makes them one query tile each (see the launch).
// * A query tile's rows are (token, query head of the kv head) pairs, 128 / G tokens x G
//   heads; both tiles of the CTA share the key tiles (64 keys each).
// * Two producer warps (K, V) look blocks up four tiles at once, four ahead, and copy whole blocks
//   of codes by TMA into two buffers each; K's also hands the softmax both scales of each group.
// * Eight widening warps (four for K, four for V) turn codes into f16 in the swizzled layout
//   that the tcgen05 descriptors read, into rings of kStages K and V tiles.  Rows past the
//   context become zeros (what lies there is not used), and so do NaN codes of V from the first
//   key tile on that some token of the item does not attend to all of: a weight of zero times
//   NaN would reach that token.  The rows that attend to such a key get the NaN as they go out.
// * An MMA warp per query tile: S = Q K^T into tensor memory (two buffers of 64 columns,
//   alternate key tiles), P V from the P that the tile's softmax leaves over the first half of
//   the S buffer, into 128 columns of O.  S of the next keys goes in before P V of the current
//   ones, so each softmax finds its next scores ready.
// * Two softmax warpgroups, one per query tile, one thread per row: the row's 64 scores in
//   registers, mask, references m (of the scores) and r (of the scores with V's scale) and sum l in
//   exp2 units, P.  O is rescaled only when a row outgrows r by more than 15.9 (log2) or m by 40,
//   so P < 2^16 fits f16, whose smallest values only gain from it; the final O / l uses the same.
//   (A limit of 15: 280 us, 15.9: 277 us for 8 prompts of 2048 tokens whose blocks' scales spread
//   over 2^4; 8: 15 us more than 15, before V's scales went into the weights.)
// Every mbarrier wait is bounded (about 1 s) and checks a shared abort flag; after one that gave up
// the CTA still waits, as long again at most, for its copies and MMAs in flight.
//
// What bounds it: the softmax's step of 64 keys, 1255 instructions on each of an SM's schedulers
// (mostly exponentials, maxima, sums and the widening) and their latency, about 1710 cycles against
// 1024 of tensor work when stamped (before V's scales went into the weights); then 5300 to 9000
// cycles from an item's last P to the next item's first.
// On GB300: 8 prompts of 2048 tokens, 32 query / 8 kv heads of 128, bf16, 275 us (1000
// TFLOP/s); 16 chunks of 100..512 over 1024..3500, fp16, 185 us (1010 TFLOP/s).  The 16-bit
// prefill takes 292 and 202 us there.  (With codes widened relative to the largest scale near
// them, which let a block that a row does not attend to take its bits: 265 and 187 us.)
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace prefill8 {

using namespace tc;

constexpr int kTiles = 2;    // query tiles per CTA (softmax warpgroups)
constexpr int kRows = 128;   // rows of a query tile (MMA M, tensor-memory lanes)
constexpr int kKeys = 64;    // keys of a K/V tile (MMA N of S, K of P V)
constexpr int kStages = 3;   // K ring, V ring
constexpr int kGroups = kKeys / 8;  // groups of eight tokens, each inside one block
constexpr int kMmaWarp = 8;         // MMA issue for query tile 0; tile 1 has the next
constexpr int kItems = 4;           // work items in flight between the roles
constexpr int kCodeWarp = 10;       // claims items, looks blocks up, copies K codes; the next V's
constexpr int kWidenWarp = 12;      // the first of kWidenWarps for K, as many for V follow
constexpr int kWidenWarps = 4;
constexpr int kThreads = 32 * (kWidenWarp + 2 * kWidenWarps);
// 640 threads launch with 96 registers each; the softmax warpgroups hold a row of 64 scores
// and take kSoftmaxRegs, the other three keep kOtherRegs (2 x 144 + 3 x 64 = 5 x 96).
constexpr int kSoftmaxRegs = 144;
constexpr int kOtherRegs = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescale = 15.9f;    // log2 growth past a row's r that forces a rescale of O: P < 2^16
constexpr float kLag = 40.f;         // past its m: fp32 sums of weights up to 2^40
// Weights of groups with far smaller V scales than the row's largest are held up to 2^(z - m - kDeep),
// at most 2^-40: zero in f16 P as they would be, and they still count in l.
constexpr float kDeep = 80.f;
constexpr float kLowest = -3e38f;    // the references of a row without a score
constexpr float kLeast = 1e-37f;     // of a factor of the scores, which stays positive
constexpr int kFactorSlots = 6;      // key tiles whose scale factors are kept: as many as can be under way

struct Params {
  CUtensorMap kmap;  // codes as [num_blocks][Hkv][B][d] bytes, box (d, B, 1, 1)
  CUtensorMap vmap;
  CUtensorMap qmap;  // q as [tokens][Hq][d], box (64, G, 128 / G): one query tile's half
  int q_tma;         // qmap is valid (G divides 128)
  const uint8_t* q;
  const uint8_t* v_cache;
  const float* k_scales;
  const float* v_scales;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;  // [n + 1]
  uint8_t* out;
  int num_seqs, num_tokens, num_q_heads, num_kv_heads, group, tpt;  // tpt = tokens per query tile
  int max_blocks_per_seq, block_size, log2_block, num_blocks;
  uint32_t group_magic;  // ceil(2^16 / G): r / G = r * group_magic >> 16 for r < 128
  int tiles;       // query tiles of an item: kTiles, or 1 where that fills the SMs better
  int max_blocks;  // query blocks (of tiles x tpt tokens) taken of a sequence at most
  float scale_log2;
  unsigned* err;
};

// A work item as the claiming warp announces it.
struct Item {
  int run;  // 0: no more items, 1: attend, 2: an impossible sequence, zeros
  int g;    // kv head
  int qs, qlen, ctx;  // the sequence's first row of q, rows, context
  int tok0, end;      // the item's tokens of the sequence
  int s;
  int bad;  // a block id of its keys is out of range
  int nan;  // V codes of keys that not all of its tokens attend to were NaN and went in as zeros
};

// Keys that query tile t of an item needs, in tiles: up to the position of its last token.
__device__ __forceinline__ int key_tiles(const Item& it, int t, int tpt) {
  const int ntok = min(tpt, it.end - (it.tok0 + t * tpt));
  return it.run == 1 && ntok > 0 ? (it.ctx - it.qlen + it.tok0 + t * tpt + ntok - 1) / kKeys + 1 : 0;
}

// The first key tile that not all tokens of an item attend to.
__device__ __forceinline__ int first_masked(const Item& it) {
  return (it.ctx - it.qlen + it.tok0 + 1) / kKeys;
}

// 0xff in the bytes of `w` that are NaN codes.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xffu;
}

// NaN into the columns of one output row (D 16-bit values) in which V is NaN at a key from the
// item's first masked tile up to the row's own position.
template <int D>
__device__ __forceinline__ void nan_columns(const Params& p, const Item& it, int pos, uint16_t* out) {
  const int32_t* trow = p.block_tables + static_cast<size_t>(it.s) * p.max_blocks_per_seq;
#pragma unroll 1
  for (int key = first_masked(it) * kKeys; key <= pos; ++key) {
    const size_t group = static_cast<size_t>(trow[key >> p.log2_block]) * p.num_kv_heads + it.g;
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(
        p.v_cache + ((group << p.log2_block) + (key & (p.block_size - 1))) * D);
#pragma unroll 1
    for (int i = 0; i < D; ++i)
      if (nan_bytes(codes[i / 4]) >> (8 * (i % 4)) & 1u) out[i] = 0x7fff;
  }
}

// A place in a ring of kStages and the parity of its current use.
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == kStages) {
      st = 0;
      ph ^= 1u;
    }
  }
};

template <int D>
struct Smem {
  uint8_t q[kTiles][kRows * D * 2];     // K-major, 128-byte swizzle; 1024-byte aligned
  uint8_t k[kStages][kKeys * D * 2];    // f16, [64-column half][64 keys][128 B]
  uint8_t v[kStages][kKeys * D * 2];
  uint8_t raw[2][2][kKeys * D];         // [K, V][kt % 2]: codes as TMA lays them (128-byte swizzle at d = 128)
  // of key tile number T (over all items) at T % kFactorSlots, per group of keys: K's scale times the
  // softmax scale, and log2 of V's scale
  float2 factor[kFactorSlots][kGroups];
  uint8_t stage[8][32 * 128];          // per softmax warp: 64 columns of its rows on their way out
  uint4 claim;                         // the answer to a claim
  Item item[kItems];
  unsigned long long item_full[kItems], item_free[kItems], claim_full;
  float q_factor[kTiles][kRows];       // bf16 rows of q: what turns their f16 products back
  // a query tile's rows landed / are f16 / their last S is done
  unsigned long long q_full[kTiles], q_ready[kTiles], q_free[kTiles];
  unsigned long long raw_full[2][2], raw_free[2][2];
  unsigned long long k_full[kStages], v_full[kStages];
  unsigned long long s_full[kTiles][2], p_full[kTiles][2];
  unsigned long long o_done[kTiles][kStages];  // P V of the key tile in that stage done (frees it)
  // P V number i of the query tile done, at i % 2: the last two may both be under way when the
  // softmax waits, and a wait tells only neighbouring phases of a barrier apart
  unsigned long long pv_done[kTiles][2];
  unsigned long long fin[kTiles];              // an MMA warp's last commit
  uint32_t tmem;
  int abort;  // a wait gave up: every role stops
  // copies asked for so far (of an aborted CTA the last ones may be in flight): tiles of raw codes,
  // q tiles, claims
  uint32_t raw_sent[2], q_sent[kTiles], claim_sent;
};

// Ask for the work of a CTA of this grid that has not started; the answer (16 bytes) lands at
// `to`, counted on `bar`.
__device__ __forceinline__ void claim_ask(uint32_t to, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(to),
      "r"(bar)
      : "memory");
}
// The claimed CTA's x index, or -1 when none was left.
__device__ __forceinline__ int claim_answer(uint32_t from) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\tld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tselp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, _, _, _}, h;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(from)
      : "memory");
  return ok ? static_cast<int>(x) : -1;
}

// Eight codes (two words) -> eight f16 values.
__device__ __forceinline__ uint4 widen8(uint32_t lo, uint32_t hi) {
  auto two = [&](uint32_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
    return h;
  };
  return make_uint4(two(lo), two(lo >> 16), two(hi), two(hi >> 16));
}

__device__ __forceinline__ float2 ld_shared8(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}
// 8 or 4 columns (packed f16 pairs) written to this thread's TMEM lane.
__device__ __forceinline__ void tmem_put(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_put(uint32_t taddr, const uint32_t (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}

// A 32-bit load kept at its place in the program.  (Not by the non-coherent path: the kernel that
// wrote the scales may have run beside this one's start.)
__device__ __forceinline__ uint32_t ld_early(const void* src) {
  uint32_t v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(src));
  return v;
}

// A bf16 row of q in shared memory (row r of a 128-row tile) becomes f16 values times a power of
// two (q_lift); returns its inverse.
template <int D>
__device__ __forceinline__ float q_row_to_f16(uint32_t tile, int r) {
  constexpr int CH = D / 8;
  uint32_t m2 = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint4 w = ld_shared16(tile + swz(kRows, r, c));
    m2 = __vmaxu2(m2, w.x & 0x7fff7fffu);
    m2 = __vmaxu2(m2, w.y & 0x7fff7fffu);
    m2 = __vmaxu2(m2, w.z & 0x7fff7fffu);
    m2 = __vmaxu2(m2, w.w & 0x7fff7fffu);
  }
  const int fe = q_lift(max(m2 & 0xffffu, m2 >> 16));
  const float f = __uint_as_float(static_cast<uint32_t>(fe) << 23);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint32_t at = tile + swz(kRows, r, c);
    const uint4 w = ld_shared16(at);
    st_shared16(at, make_uint4(q_lifted(w.x, f), q_lifted(w.y, f), q_lifted(w.z, f), q_lifted(w.w, f)));
  }
  return __uint_as_float(static_cast<uint32_t>(254 - fe) << 23);
}

// NG: groups of keys with a scale in a key tile: of 16 keys, or of 8 where blocks are as short.
template <int D, typename T, int NG>
__global__ void __launch_bounds__(kThreads, 1) prefill_fp8_block_kernel(const __grid_constant__ Params p) {
  constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
  constexpr int CH = D / 8;        // 16-byte chunks of a 16-bit row
  constexpr int KS1 = D / 16;      // MMA k-steps of S = Q K^T
  constexpr int KS2 = kKeys / 16;  // MMA k-steps of P V
  constexpr int GK = kKeys / NG;   // keys of a scale group
  constexpr uint32_t kTileCols = 256;  // TMEM columns per query tile:
  constexpr uint32_t kColS = kKeys;    //   S of key tile kt in [64 (kt % 2), + 64), its P over the
  constexpr uint32_t kColO = 128;      //   first 32 of those columns, O in [128, 128 + D)
  constexpr uint32_t kTmemCols = kTiles * kTileCols;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_addr(smem_raw);
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw + (((raw_addr + 1023) & ~1023u) - raw_addr));

  pdl_wait_primary();
  pdl_launch_dependents();

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (known to be uniform over the warp)
  const int tpt = p.tpt, G = p.group;
  T* outp = reinterpret_cast<T*>(p.out);

  // ---- set-up: barriers, tensor memory ----
  if (warp == kMmaWarp && lane == 0) {
    for (int i = 0; i < kItems; ++i) {
      mbar_init(smem_addr(&sm.item_full[i]), 1);
      // every warp but the claiming one
      mbar_init(smem_addr(&sm.item_free[i]), kThreads / 32 - 1);
    }
    mbar_init(smem_addr(&sm.claim_full), 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_addr(&sm.raw_full[i >> 1][i & 1]), 1);
      mbar_init(smem_addr(&sm.raw_free[i >> 1][i & 1]), kWidenWarps);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&sm.k_full[i]), kWidenWarps);
      mbar_init(smem_addr(&sm.v_full[i]), kWidenWarps);
      for (int t = 0; t < kTiles; ++t) mbar_init(smem_addr(&sm.o_done[t][i]), 1);
    }
    for (int t = 0; t < kTiles; ++t) {
      mbar_init(smem_addr(&sm.q_full[t]), 33);  // TMA expect-tx + 32 copy lanes
      mbar_init(smem_addr(&sm.q_ready[t]), kWidenWarps);
      mbar_init(smem_addr(&sm.q_free[t]), 1);
      mbar_init(smem_addr(&sm.fin[t]), 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_addr(&sm.pv_done[t][b]), 1);
        mbar_init(smem_addr(&sm.s_full[t][b]), 2);  // the MMA warp, its MMAs
        mbar_init(smem_addr(&sm.p_full[t][b]), kRows / 32);
      }
    }
    fence_mbar_init();
    sm.abort = 0;
    sm.raw_sent[0] = sm.raw_sent[1] = sm.q_sent[0] = sm.q_sent[1] = sm.claim_sent = 0;
  }
  if (warp == kMmaWarp + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&sm.tmem)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  // a bounded wait; on failure every role stops (the flag is checked inside the waits)
  auto wait = [&](unsigned long long& bar, int parity) -> bool {
    if (mbar_wait_bounded(smem_addr(&bar), static_cast<uint32_t>(parity), &sm.abort)) return true;
    if (atomicExch(&sm.abort, 1) == 0) atomicOr(p.err, kErrTimeout);
    return false;
  };

  auto wwait = [&](unsigned long long& bar, uint32_t parity) -> bool {  // warp-uniform result
    return __all_sync(0xffffffffu, wait(bar, static_cast<int>(parity))) != 0;
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

  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp >= kWidenWarp) {
      // ===== widening: K (or V) tiles of the rings =====
      // Warp cw takes rows 16 cw .. 16 cw + 15 of each tile, two groups of eight tokens.  At
      // d = 128 a lane takes 16-byte chunk (lane % 4) + 4 hc of one row of the group: eight lanes
      // cover four chunks of rows r and r ^ 5, which makes both the swizzled code loads and the swizzled f16
      // stores (chunks 2 c and 2 c + 1 of the same row) free of bank conflicts.  At d = 64 a
      // warp covers the group's eight rows of four chunks at once.
      constexpr int NH = D / 64;  // instructions per group
      const int is_v = warp >= kWidenWarp + kWidenWarps;
      const int cw = (warp - kWidenWarp) % kWidenWarps;
      const int rr = D == 128 ? ((lane >> 3) ^ (lane & 4 ? 5 : 0)) : lane >> 2;
      const uint32_t get = D == 128 ? rr * 128 + (((lane & 3) ^ rr) << 4) : rr * 64 + ((lane & 3) << 4);
      const uint32_t put0 = rr * 128 + (((2 * (lane & 3)) ^ rr) << 4);
      const uint32_t put1 = rr * 128 + (((2 * (lane & 3) + 1) ^ rr) << 4);
      const uint32_t ring = smem_addr(is_v ? sm.v[0] : sm.k[0]) + cw * 16 * 128;
      const uint32_t raw = smem_addr(sm.raw[is_v][0]) + cw * 16 * D + get;
      unsigned long long* full = is_v ? sm.v_full : sm.k_full;
      Ring r3;
      uint32_t num = 0, loads = 0;  // key tiles and q loads so far
      Item it;
      bool ok = true;
      for (int j = 0; ok && (ok = item_get(j, it)) && it.run; ++j) {
        item_done(j);
        const int n = max(key_tiles(it, 0, tpt), key_tiles(it, 1, tpt));
        // bf16 rows of q become f16 rows here, a row per lane: V's warps take query tile 0 before
        // their first tile, K's take query tile 1 after theirs.  (The softmax warps, busy writing
        // the last item out, took 7000 cycles from its last P V to the next item's first S.)
        auto q_rows = [&](int t) -> bool {
          if (!wwait(sm.q_full[t], loads & 1)) return false;
          ++loads;
          if (key_tiles(it, t, tpt) > 0)
            sm.q_factor[t][32 * cw + lane] = q_row_to_f16<D>(smem_addr(sm.q[t]), 32 * cw + lane);
          fence_async_smem();  // the rows before the tensor cores' reads
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sm.q_ready[t]));
          return true;
        };
        if (BF && is_v && n > 0 && !(ok = q_rows(0))) break;
        for (int kt = 0; kt < n; ++kt, ++num, r3.next()) {
          const int b = num & 1;
          if (!(ok = wwait(sm.raw_full[is_v][b], (num >> 1) & 1))) break;
          uint4 c[2][NH];
#pragma unroll
          for (int gi = 0; gi < 2; ++gi)
#pragma unroll
            for (int hc = 0; hc < NH; ++hc)
              c[gi][hc] = ld_shared16((raw ^ (hc * 64)) + b * (kKeys * D) + gi * 8 * D);
          // (the row of group gi: kt * 64 + 16 cw + 8 gi + rr)
          const int left = it.ctx - (kt * kKeys + 16 * cw + rr);
          if (left <= 8) {
#pragma unroll
            for (int gi = 0; gi < 2; ++gi)
              if (left <= 8 * gi) {
#pragma unroll
                for (int hc = 0; hc < NH; ++hc) c[gi][hc] = make_uint4(0, 0, 0, 0);
              }
          }
          if (is_v && kt >= first_masked(it)) {
            // a weight of zero times NaN is NaN: such codes become zeros here, and the rows that
            // do attend to them get their NaN in the end
            uint32_t any = 0;
            auto drop = [&](uint32_t& w) {
              const uint32_t m = nan_bytes(w);
              any |= m;
              w &= ~m;
            };
#pragma unroll
            for (int gi = 0; gi < 2; ++gi)
#pragma unroll
              for (int hc = 0; hc < NH; ++hc)
                drop(c[gi][hc].x), drop(c[gi][hc].y), drop(c[gi][hc].z), drop(c[gi][hc].w);
            if (any) sm.item[j % kItems].nan = 1;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sm.raw_free[is_v][b]));
          if (num >= kStages &&
              !(ok = wwait(sm.o_done[0][r3.st], r3.ph ^ 1u) && wwait(sm.o_done[1][r3.st], r3.ph ^ 1u)))
            break;
          const uint32_t tile = ring + r3.st * (kKeys * D * 2);
#pragma unroll
          for (int gi = 0; gi < 2; ++gi) {
#pragma unroll
            for (int hc = 0; hc < NH; ++hc) {
              const uint32_t at = tile + 8 * gi * 128 + hc * (kKeys * 128);
              st_shared16(at + put0, widen8(c[gi][hc].x, c[gi][hc].y));
              st_shared16(at + put1, widen8(c[gi][hc].z, c[gi][hc].w));
            }
          }
          fence_async_smem();  // these stores before the tensor cores' reads
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&full[r3.st]));
          if (BF && !is_v && kt == 0 && !(ok = q_rows(1))) break;
        }
      }
    } else if (warp >= kCodeWarp) {
      // ===== items, blocks, scales and codes of K (or V), ahead of the widening warps =====
      const int is_v = warp != kCodeWarp;
      const int per_item = p.tiles * tpt;
      // K's warp claims the items.  Item x of the grid: kv head x % Hkv of query block x / Hkv,
      // the blocks of all sequences counted from the last one's last block down, so that a
      // sequence's long items come first; items past the last block (the grid is sized without
      // knowing the lengths) end the CTA.  Lane u keeps the blocks of sequences [u * per,
      // (u + 1) * per): `mine` of them, `before` of lower lanes.
      const int per = (p.num_seqs + 31) / 32;
      auto blocks_of = [&](int s) -> int {
        if (s >= p.num_seqs) return 0;
        const int a = __ldg(p.query_start + s), b = __ldg(p.query_start + s + 1);
        if (a < 0 || b < a || b > p.num_tokens) {  // rows that are not q's: nothing is touched
          atomicOr(p.err, kErrBadContext);
          return 0;
        }
        return min(p.max_blocks, (b - a + per_item - 1) / per_item);
      };
      auto scan32 = [&](int x) -> int {  // inclusive sum over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        return x;
      };
      int mine = 0, before = 0, total = 0;
      if (!is_v) {
        for (int i = 0; i < per; ++i) mine += blocks_of(lane * per + i);
        const int incl = scan32(mine);
        before = incl - mine;
        total = __shfl_sync(0xffffffffu, incl, 31);
      }
      auto item_of = [&](int x) -> Item {  // (uniform over the warp)
        Item it;
        it.run = it.bad = it.nan = 0;
        const int f = total - 1 - x / p.num_kv_heads;  // query block, counted from the first
        it.g = x % p.num_kv_heads;
        if (x < 0 || f < 0) return it;
        const int owner = 31 - __clz(__ballot_sync(0xffffffffu, before <= f && mine > 0));
        int left = f - __shfl_sync(0xffffffffu, before, owner);
        for (int s0 = owner * per; s0 < (owner + 1) * per; s0 += 32) {
          const int nb = s0 + lane < (owner + 1) * per ? blocks_of(s0 + lane) : 0;
          const int incl = scan32(nb);
          const int sum = __shfl_sync(0xffffffffu, incl, 31);
          if (left < sum) {
            const int o = __ffs(__ballot_sync(0xffffffffu, left < incl)) - 1;
            it.s = s0 + o;
            left -= __shfl_sync(0xffffffffu, incl - nb, o);
            it.run = 1;
            break;
          }
          left -= sum;
        }
        if (!it.run) return it;  // (never: the block is one of the owner's)
        it.qs = __ldg(p.query_start + it.s);
        it.qlen = __ldg(p.query_start + it.s + 1) - it.qs;
        it.ctx = __ldg(p.context_lens + it.s);
        it.tok0 = left * per_item;
        it.end = min(it.qlen, it.tok0 + per_item);
        if (it.ctx < 1 || it.ctx > p.max_blocks_per_seq * p.block_size || it.qlen > it.ctx) {
          it.run = 2;
          if (lane == 0) atomicOr(p.err, kErrBadContext);
        }
        return it;
      };
      // Four key tiles are looked up at once: lane 8 q + g looks after token group g of tile q of
      // the four.  (One tile at a time took this warp about 1650 cycles each, as long as the
      // softmax's step.)
      const int grp = lane & 7, quad = lane >> 3;
      const bool first_group = ((8 * grp) & (p.block_size - 1)) == 0;  // of its block
      uint32_t num = 0, claims = 0, loads = 0;  // key tiles, claims and q loads so far
      Item it;
      if (!is_v) it = item_of(blockIdx.x);
      bool ok = true;
      for (int j = 0; ok; ++j) {
        if (is_v) {
          if (!(ok = item_get(j, it))) break;
        } else {
          if (j >= kItems && !(ok = wwait(sm.item_free[j % kItems], (j / kItems - 1) & 1))) break;
          if (lane == 0) {
            sm.item[j % kItems] = it;
            mbar_arrive(smem_addr(&sm.item_full[j % kItems]));
          }
          __syncwarp();
        }
        if (!it.run) break;
        const int n = max(key_tiles(it, 0, tpt), key_tiles(it, 1, tpt));
        if (is_v) {
          item_done(j);
          if (it.run == 1) {
            // ===== q: each query tile once the last item's S of it are done =====
            // A whole query tile (tpt tokens x G heads = 128 rows, each token's G rows
            // contiguous in q) by TMA, one copy per 64-column half; a tile that runs past its
            // sequence by 16-byte copies, rows past the last token zeros.
            for (int t = 0; t < kTiles; ++t) {
              if (loads > 0 && !(ok = wwait(sm.q_free[t], (loads - 1) & 1))) break;
              const int first = it.tok0 + t * tpt;
              const bool tma = p.q_tma && first + tpt <= it.end;
              if (lane == 0) {
                sm.q_sent[t] = loads + 1;
                mbar_arrive_expect_tx(smem_addr(&sm.q_full[t]), tma ? kRows * D * 2 : 0);
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
                  if (tma)
                    tma_load_3d(smem_addr(sm.q[t]) + h * kRows * 128, &p.qmap, h * 64, it.g * G,
                                it.qs + first, smem_addr(&sm.q_full[t]));
              }
              __syncwarp();
              if (first < it.end && !tma) {
                // (rows past tpt * G, where G does not divide 128, are zeros too)
                for (int u = lane; u < kRows * CH; u += 32) {
                  const int r = u / CH, c = u % CH;
                  const int tl = static_cast<int>((r * p.group_magic) >> 16);  // r / G
                  const bool live = tl < tpt && first + tl < it.end;
                  const uint8_t* src =
                      p.q + ((static_cast<size_t>(it.qs + (live ? first + tl : 0)) * p.num_q_heads +
                              it.g * G + (live ? r - tl * G : 0)) * D + c * 8) * 2;
                  cp_async16(smem_addr(sm.q[t]) + swz(kRows, r, c), src, live ? 16u : 0u);
                }
              }
              cp_async_arrive(smem_addr(&sm.q_full[t]));
            }
            if (!ok) break;
            ++loads;
          }
        }
        const int32_t* trow = p.block_tables + static_cast<size_t>(it.s) * p.max_blocks_per_seq;
        // does tile kt's group hold keys that are used
        auto used = [&](int kt) -> bool { return kt < n && kt * kKeys + 8 * grp < it.ctx; };
        // its table entry; checked four tiles later, when it is used, so that nothing waits for the
        // load (the loads here are volatile to stay where they are written)
        auto entry = [&](int kt) -> int {
          return used(kt) ? static_cast<int>(ld_early(trow + ((kt * kKeys + 8 * grp) >> p.log2_block))) : -1;
        };
        auto block_of = [&](int kt, int e) -> int {
          if (e >= 0 && e < p.num_blocks) return e;
          if (used(kt) && !is_v) {
            sm.item[j % kItems].bad = 1;  // (read by the softmax when the item's tiles are done)
            atomicOr(p.err, kErrBadBlock);
          }
          return -1;
        };
        auto scale_of = [&](const float* scales, int e) -> float {
          return e >= 0 ? __uint_as_float(ld_early(scales + static_cast<size_t>(e) * p.num_kv_heads + it.g)) : 0.f;
        };
        const int raw0 = entry(quad);
        int raw_e = entry(4 + quad);
        int e = block_of(quad, raw0);
        float sk = 0.f, sv = 1.f;  // (K's warp: it tells the softmax both)
        auto scales_of = [&](int b) {
          if (is_v) return;
          sk = scale_of(p.k_scales, b);
          sv = scale_of(p.v_scales, b);
        };
        scales_of(e);
        for (int base = 0; ok && base < n; base += 4) {
          const int e1 = block_of(base + 4 + quad, raw_e);
          // (bf16: kept positive with the row's factor)
          const float kf = BF ? sk * p.scale_log2 : fmaxf(sk * p.scale_log2, kLeast), vl = __log2f(sv);
          scales_of(e1);
          raw_e = entry(base + 8 + quad);
          for (int q = 0; q < 4 && base + q < n; ++q, ++num) {
            // the next item is claimed three tiles before this one's end: late, so that no SM
            // sits on work that another could start, yet early enough for the answer
            if (!is_v && base + q == max(0, n - 3) && lane == 0) {
              sm.claim_sent = claims + 1;
              mbar_arrive_expect_tx(smem_addr(&sm.claim_full), 16);
              claim_ask(smem_addr(&sm.claim), smem_addr(&sm.claim_full));
            }
            const bool mine_now = quad == q && first_group && e >= 0;  // (e < 0 past the groups)
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine_now)) * p.block_size * D;
            const int b = num & 1;
            if (num >= 2 && !(ok = wwait(sm.raw_free[is_v][b], ((num >> 1) - 1) & 1))) break;
            // free: the tile two back is read; K's tile three back is widened, so the P V of six back
            // is done, and the softmax of kFactorSlots back with its factors
            if (quad == q && !is_v && grp % (8 / NG) == 0)
              sm.factor[num % kFactorSlots][grp / (8 / NG)] = make_float2(kf, vl);
            __syncwarp();  // the stores above before the arrival
            if (lane == 0) {
              sm.raw_sent[is_v] = num + 1;
              mbar_arrive_expect_tx(smem_addr(&sm.raw_full[is_v][b]), bytes);
            }
            __syncwarp();
            if (mine_now)
              tma_load_4d(smem_addr(sm.raw[is_v][b]) + 8 * grp * D, is_v ? &p.vmap : &p.kmap, 0, 0, it.g, e,
                          smem_addr(&sm.raw_full[is_v][b]));
          }
          e = e1;
        }
        if (!ok) break;
        if (!is_v) {
          if (n == 0 && lane == 0) {
            sm.claim_sent = claims + 1;
            mbar_arrive_expect_tx(smem_addr(&sm.claim_full), 16);
            claim_ask(smem_addr(&sm.claim), smem_addr(&sm.claim_full));
          }
          if (!(ok = wwait(sm.claim_full, claims & 1))) break;
          ++claims;
          const int x = claim_answer(smem_addr(&sm.claim));
          fence_async_smem();  // the read above before the next answer
          __syncwarp();
          it = item_of(x);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
      // ============ MMA issue: a warp per query tile ============
      // The tensor pipe runs one thread's MMAs in order, so S of a key tile may overwrite the P
      // of the tile two before, whose P V was issued earlier.  A warp whose query tile needs no
      // more keys still frees each stage, after it has landed.
      const int t = warp - kMmaWarp;
      const uint32_t el = elect_one();
      constexpr uint32_t id_s = idesc_f16<__half>(kRows, kKeys, false);
      constexpr uint32_t id_o = idesc_f16<__half>(kRows, D, true);
      constexpr uint32_t kStageBytes = kKeys * D * 2;
      const uint64_t qd = desc_sw128(smem_addr(sm.q[t]), 16, 1024);
      const uint64_t dk0 = desc_sw128(smem_addr(sm.k[0]), 16, 1024);
      const uint64_t dv0 = desc_sw128(smem_addr(sm.v[0]), kKeys * 128, 1024);
      const uint32_t cols = tmem + t * kTileCols;
      auto issue_s = [&](uint32_t sn, int st) {  // S number sn of this query tile, K in stage st
        const uint32_t d = cols + (sn & 1) * kColS;
        const uint64_t kd = dk0 + ((st * kStageBytes) >> 4);
#pragma unroll
        for (int ks = 0; ks < KS1; ++ks)  // 16 columns = 32 bytes of 64-column block ks / 4
          mma_el(d, qd + (((ks >> 2) * kRows * 128 + (ks & 3) * 32) >> 4),
                 kd + (((ks >> 2) * kKeys * 128 + (ks & 3) * 32) >> 4), id_s, ks > 0, el);
        commit_el(smem_addr(&sm.s_full[t][sn & 1]), el);
        if (el) mbar_arrive(smem_addr(&sm.s_full[t][sn & 1]));  // (passes k_full on to the softmax)
      };
      auto issue_pv = [&](uint32_t sn, int st, bool first) {
        const uint32_t pa = cols + (sn & 1) * kColS, o = cols + kColO;
        const uint64_t vd = dv0 + ((st * kStageBytes) >> 4);
#pragma unroll
        for (int ks = 0; ks < KS2; ++ks)  // 16 keys = 8 columns of P
          mma_ts_el(o, pa + ks * 8, vd + ((ks * 16 * 128) >> 4), id_o, !first || ks > 0, el);
      };
      Ring rk, rv;
      uint32_t sn = 0, loads = 0;  // S issued for this query tile, q loads so far
      Item it;
      bool ok = true;
      for (int j = 0; ok && (ok = item_get(j, it)); ++j) {
        if (!__shfl_sync(0xffffffffu, it.run, 0)) break;
        item_done(j);
        // (broadcast, so that the loops are known to be uniform)
        const int n0 = key_tiles(it, 0, tpt), n1 = key_tiles(it, 1, tpt);
        const int n = __shfl_sync(0xffffffffu, max(n0, n1), 0);
        const int ntt = __shfl_sync(0xffffffffu, t == 0 ? n0 : n1, 0);
        if (n == 0) continue;
        if (!(ok = wwait(BF ? sm.q_ready[t] : sm.q_full[t], loads & 1))) break;
        ++loads;
        fence_async_smem();  // q rows that lanes copied or converted -> tensor cores
        if (ntt > 0) {
          if (!(ok = wwait(sm.k_full[rk.st], rk.ph))) break;
          issue_s(sn, rk.st);
        }
        rk.next();
        // q is free once S of the last key tile is done, and the softmax has its rows' factors
        // (by the first P, which S of the third tile waits for)
        if (ntt == 0) commit_el(smem_addr(&sm.q_free[t]), el);
        for (int kt = 0; kt < n; ++kt, rk.next(), rv.next()) {
          if (kt + 1 < ntt) {
            if (!(ok = wwait(sm.k_full[rk.st], rk.ph))) break;
            issue_s(sn + 1, rk.st);
            if (kt > 0 && kt + 2 == ntt) commit_el(smem_addr(&sm.q_free[t]), el);
          }
          if (!(ok = wwait(sm.v_full[rv.st], rv.ph))) break;
          if (kt < ntt) {
            if (!(ok = wwait(sm.p_full[t][sn & 1], (sn >> 1) & 1))) break;
            tc_fence_after();
            issue_pv(sn, rv.st, kt == 0);
            commit_el(smem_addr(&sm.pv_done[t][sn & 1]), el);
            if (kt == 0 && ntt <= 2) commit_el(smem_addr(&sm.q_free[t]), el);
            ++sn;
          } else if (!(ok = wwait(sm.k_full[rv.st], rv.ph))) {
            break;
          }
          commit_el(smem_addr(&sm.o_done[t][rv.st]), el);
        }
        // rk ran one tile ahead of rv, past the item's end
        rk = rv;
      }
      commit_el(smem_addr(&sm.fin[t]), el);  // every MMA this warp issued
      wwait(sm.fin[t], 0);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ================= softmax: warpgroup t, one thread per row =================
    const int t = warp >> 2, r = tid & (kRows - 1);
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + t * kTileCols;
    const int tile_tok = static_cast<int>((r * p.group_magic) >> 16);  // r / G
    uint32_t sn = 0, num = 0;  // S of this query tile and key tiles so far
    Item it;
    bool ok = true;
    for (int j = 0; ok && (ok = item_get(j, it)) && it.run; ++j) {
      const int n0 = key_tiles(it, 0, tpt), n1 = key_tiles(it, 1, tpt);
      const int n = max(n0, n1), ntt = t == 0 ? n0 : n1;
      const int tok = it.tok0 + t * tpt + tile_tok;
      const int pos = tile_tok < tpt && tok < it.end ? it.ctx - it.qlen + tok : -1;
      const int pos_lo = it.ctx - it.qlen + it.tok0 + t * tpt;  // the tile's first position
      // (log2) references of the scores and of the scores with V's scales, and the sum of weights
      float m_ref = 0.f, r_ref = 0.f, l_run = 0.f;
      float q_fac = 1.f;  // turns this row's scores back
      for (int kt = 0; kt < ntt; ++kt, ++sn) {
        const int b = sn & 1;
        // (the factors were written before k_full of this tile, q_factor before q_ready, which
        // the MMA warp acquired before it arrived here)
        if (!(ok = wwait(sm.s_full[t][b], (sn >> 1) & 1))) break;
        tc_fence_after();
        if (BF && kt == 0) q_fac = sm.q_factor[t][r];
        const uint32_t factor = smem_addr(sm.factor[(num + kt) % kFactorSlots]);
        // group g's factor of the raw scores, positive (so that the maximum commutes with it and a
        // masked -inf stays -inf even where it would underflow), and log2 of its V scale; read
        // where they are used, twice, since the 64 scores leave few registers
        auto factors = [&](int g) -> float2 {
          float2 f = ld_shared8(factor + 8 * g);
          if (BF) f.x = fmaxf(f.x * q_fac, kLeast);
          return f;
        };
        float sv[kKeys];
        tmem_get64(tl + b * kColS, sv);
        if (kt * kKeys + kKeys - 1 > pos_lo) {  // causal mask: key kt * 64 + i > pos
          const int lim = pos - kt * kKeys;
#pragma unroll
          for (int i = 0; i < kKeys; ++i)
            if (i > lim) sv[i] = -INFINITY;
        }
        float mx = -INFINITY, my = -INFINITY;
#pragma unroll
        for (int g = 0; g < NG; g += 2) {
          float m[2], y[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 f = factors(g + k);
            const float* x = sv + (g + k) * GK;
            m[k] = fmaxf(x[0], x[1]);
#pragma unroll
            for (int i = 2; i < GK; i += 2) m[k] = fmax3(m[k], x[i], x[i + 1]);
            m[k] *= f.x;
            y[k] = m[k] + f.y;
          }
          mx = fmax3(mx, m[0], m[1]);
          my = fmax3(my, y[0], y[1]);
        }
        // (not rounded up: where one key stands out its weight is 1 then, which f16 does not round)
        if (kt == 0) {
          m_ref = mx > -INFINITY ? mx : kLowest;
          r_ref = my > -INFINITY ? my : kLowest;
        } else {
          const bool need = mx > m_ref + kLag || my > r_ref + kRescale;
          if (__any_sync(0xffffffffu, need)) {
            // rescale O, once P V of the tile before is done (the one before that was issued
            // before this S)
            if (!(ok = wwait(sm.pv_done[t][(sn - 1) & 1], ((sn - 1) >> 1) & 1))) break;
            tc_fence_after();
            float alpha = 1.f;
            if (need) {
              const float m_new = fmaxf(m_ref, mx), r_new = fmaxf(r_ref, my);
              l_run *= ex2(m_ref - m_new);
              alpha = ex2(r_ref - r_new);
              m_ref = m_new;
              r_ref = r_new;
            }
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
        }
        // P = 2^(s c + log2 sV - r), rounded to f16, packed two a column over the first half of this
        // thread's own row of S (already in registers); its unrounded sum, without the V scale, in l.
        // (the factors are read again and P leaves group by group: held in registers beside the 64
        // scores they spilled, 297 us for 8 prompts of 2048 tokens, 272 so)
        float2 l2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float2 f = factors(g);
          const float a = fmaxf(f.y - r_ref, -kDeep - m_ref);
          const float2 c2 = make_float2(f.x, f.x), a2 = make_float2(a, a);
          float2 ps[2];
          uint32_t pk[GK / 2];
#pragma unroll
          for (int i = 0; i < GK; i += 2) {
            const float2 x = __ffma2_rn(make_float2(sv[g * GK + i], sv[g * GK + i + 1]), c2, a2);
            const float2 e = make_float2(ex2(x.x), ex2(x.y));
            ps[(i >> 1) & 1] = i < 4 ? e : __fadd2_rn(ps[(i >> 1) & 1], e);
            pk[i >> 1] = pack2<__half>(e.x, e.y);
          }
          const float2 sum = __fadd2_rn(ps[0], ps[1]);
          const float w = ex2(-a - m_ref);
          l2 = __ffma2_rn(sum, make_float2(w, w), l2);
          tmem_put(tl + b * kColS + g * (GK / 2), pk);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();  // the P stores before the MMA warp reads them
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.p_full[t][b]));
        l_run += l2.x + l2.y;
      }
      if (!ok) break;
      if (ntt > 0 && !(ok = wwait(sm.pv_done[t][(sn - 1) & 1], ((sn - 1) >> 1) & 1))) break;
      tc_fence_after();
      num += n;
      // ---- out = O 2^(r - m) / l (the item's tiles are done, so its bad-block flag is final) ----
      const bool good = it.run == 1 && ntt > 0 && *reinterpret_cast<volatile int*>(&sm.item[j % kItems].bad) == 0;
      const bool nan = good && *reinterpret_cast<volatile int*>(&sm.item[j % kItems].nan) != 0;
      item_done(j);
      // (in two steps, each a float where r - m is near the exponents' ends)
      const float lift = r_ref > m_ref ? 16.f : -16.f;
      const float inv = ex2(r_ref - m_ref - lift) / l_run * ex2(lift);
      // The rows go out through shared memory, 64 columns at a time, so that each store
      // instruction of a warp writes whole 128-byte lines.  Row r's 16-byte chunk c sits at
      // chunk c ^ (r % 8) of its 128-byte staging row: neither the writes nor the reads
      // collide in a bank.  (clamped: a cached f16 value may have been rounded up past 65504)
      const uint32_t stage = smem_addr(sm.stage[warp]);
      const int ch = lane & 7;
      const int toks = min(tpt, it.end - (it.tok0 + t * tpt));  // tokens of this query tile
      T* to = outp + (static_cast<size_t>(it.qs + it.tok0 + t * tpt) * p.num_q_heads + it.g * G) * D + ch * 8;
      int at[8];  // of the eight rows that this lane stores a chunk of; -1: not a row
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = (r - lane) + 4 * i + (lane >> 3);  // token tk of the tile, head row % G
        const int tk = static_cast<int>((row * p.group_magic) >> 16);
        at[i] = tk < toks ? (tk * (p.num_q_heads - G) + row) * D : -1;
      }
      const float2 inv2 = make_float2(inv, inv);
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 64) {
#pragma unroll
        for (int c1 = 0; c1 < 64; c1 += 32) {
          float o[32];
          if (good) tmem_get32(tl + kColO + c0 + c1, o);  // (uniform over the warp)
          auto two = [&](int i) -> uint32_t {
            const float2 x = __fmul2_rn(make_float2(o[i], o[i + 1]), inv2);
            return good ? pack2_sat<T>(x.x, x.y) : 0u;
          };
#pragma unroll
          for (int cc = 0; cc < 4; ++cc)
            st_shared16(stage + lane * 128 + (((c1 / 8 + cc) ^ (lane & 7)) << 4),
                        make_uint4(two(8 * cc), two(8 * cc + 2), two(8 * cc + 4), two(8 * cc + 6)));
        }
        __syncwarp();
        uint4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = 4 * i + (lane >> 3);
          x[i] = ld_shared16(stage + rr * 128 + ((ch ^ (rr & 7)) << 4));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (at[i] >= 0) *reinterpret_cast<uint4*>(to + at[i] + c0) = x[i];
        __syncwarp();  // the reads before the next columns' stores
      }
      if (nan && pos >= 0)
        nan_columns<D>(p, it, pos,
                       reinterpret_cast<uint16_t*>(outp) +
                           ((static_cast<size_t>(it.qs + tok) * p.num_q_heads) + it.g * G + r - tile_tok * G) * D);
      __syncwarp();
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
      for (int i = 0; i < 2; ++i)
        for (uint32_t b = 0; b < 2; ++b) land(sm.raw_full[i][b], (sm.raw_sent[i] + 1 - b) / 2);
      for (int t = 0; t < kTiles; ++t) land(sm.q_full[t], sm.q_sent[t]), land(sm.fin[t], 1);
      land(sm.claim_full, sm.claim_sent);
      if (!ended) atomicOr(p.err, kErrTimeout);
    }
    __syncthreads();
  }
  if (warp == kMmaWarp + 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

template <int D, typename T, int NG>
int launch(const Params& prm, int max_query_len, int sm_count, cudaStream_t stream) {
  const size_t smem = sizeof(Smem<D>) + 1024;
  auto* kern = prefill_fp8_block_kernel<D, T, NG>;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), smem)) return -3;
  cudaLaunchConfig_t cfg = {};
  // query blocks, whatever the lengths are: a part of one per sequence beyond the whole ones
  Params q = prm;
  auto items = [&](int tiles) -> long long {
    const int per_item = tiles * prm.tpt;
    q.tiles = tiles;
    q.max_blocks = (max_query_len + per_item - 1) / per_item;
    return std::min(static_cast<long long>(prm.num_tokens / per_item) + prm.num_seqs,
                    static_cast<long long>(prm.num_seqs) * q.max_blocks) * prm.num_kv_heads;
  };
  long long count = items(kTiles);
  // Few items: one query tile each while every item still has an SM of its own.  One prompt
  // of 128 / 512 tokens, 8 kv heads, 4 query heads each: 8.3 / 14.1 us, 9.6 / 15.1 us with
  // two; a chunk of 512 over 2000 cached 39.2 us, 45.1 with two.  Past that, items queue: 8
  // chunks of 100 over 1000 cached (128 items of two) 42.1 us, 27.1 with two.
  if (2 * count <= sm_count) count = items(1);
  if (count > 0x7fffffffLL) return -1;
  cfg.gridDim = dim3(static_cast<unsigned>(count));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, q) != cudaSuccess) return -3;
  return 0;
}

}  // namespace prefill8

int prefill_fp8_block_launch(const PrefillArgs& a, int num_tokens, const float* k_scales,
                             const float* v_scales, int sm_count, cudaStream_t stream) {
  prefill8::Params p;
  p.q = static_cast<const uint8_t*>(a.q);
  p.v_cache = static_cast<const uint8_t*>(a.v_cache);
  if (!kv_cache_map(&p.kmap, a.k_cache, 1, a.num_blocks, a.num_kv_heads, a.block_size, a.head_dim) ||
      !kv_cache_map(&p.vmap, a.v_cache, 1, a.num_blocks, a.num_kv_heads, a.block_size, a.head_dim))
    return -3;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.query_start = a.query_start;
  p.out = static_cast<uint8_t*>(a.out);
  p.num_seqs = a.num_seqs;
  p.num_tokens = num_tokens;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.tpt = prefill8::kRows / p.group;
  p.group_magic = (65536u + p.group - 1) / p.group;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.block_size = a.block_size;
  p.log2_block = a.block_size == 8 ? 3 : (a.block_size == 16 ? 4 : 5);
  p.num_blocks = a.num_blocks;
  p.scale_log2 = a.scale * prefill8::kLog2e;
  p.q_tma = q_tile_map(&p.qmap, a.q, a.num_q_heads, a.head_dim, p.group, num_tokens) ? 1 : 0;
  p.err = a.err;
#define PA_PREFILL_CASE(DD, NN)                                                            \
  if (a.head_dim == DD && (a.block_size == 8) == (NN == 8))                                \
    return a.bf16 ? prefill8::launch<DD, __nv_bfloat16, NN>(p, a.max_query_len, sm_count, stream) \
                  : prefill8::launch<DD, __half, NN>(p, a.max_query_len, sm_count, stream);
  PA_PREFILL_CASE(128, 4)
  PA_PREFILL_CASE(128, 8)
  PA_PREFILL_CASE(64, 4)
  PA_PREFILL_CASE(64, 8)
#undef PA_PREFILL_CASE
  return -1;
}

}  // namespace pa
