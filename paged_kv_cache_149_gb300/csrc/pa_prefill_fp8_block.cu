// Paged prefill attention over FP8 (E4M3) K/V blocks with a scale for each (block, kv head),
// for sm_103a: causal multi-query attention of each sequence's newest tokens over its paged
// context, on the 5th-generation tensor cores (tcgen05).
//
// With K_t = sK_t code(K_t), V_t likewise (s: the scale of token t's block and head), the token
// at position p attends to positions t <= p:
//   out = sum_t softmax_t(scale <q, K_t>) V_t
// (daiw.org "Paged Attention", section 回顾与衔接; chenyuan1125 "vllm-pagedattention", section
// 它和 FlashAttention…).
//
// Everything runs on the tensor cores in f16, whatever q's type: a code times a power of two
// is exact there, the widening from E4M3 is one instruction for two values, and P keeps 11
// bits.  Range is kept by references: a key tile's codes are widened to code * s / kref, kref
// the tile's largest K scale, and its scores multiplied by kref where the softmax scales them
// anyway; V's to code * s / vref, vref the largest V scale of the CTA's first tile (it moves,
// with one rescale of O, only when a later scale is over 2^7 times it); each bf16 row of q
// is multiplied by the power of two that brings its largest value to [2^14, 2^15).  For scales
// that are powers of two no step rounds but those of values 2^-15 and more below their
// reference (an absolute 2^-25 of it); other scales round each widened value once.
//
// Design: one CTA per (pair of 128-row query tiles, sequence, kv head), 640 threads:
// * A query tile's rows are (token, query head of the kv head) pairs, 128 / G tokens x G
//   heads; both tiles of the CTA share the key tiles (64 keys each).
// * Two producer warps (K, V) look blocks and scales up a tile ahead and copy whole blocks of
//   codes by TMA into two buffers each.
// * Eight widening warps (four for K, four for V) turn codes into f16 in the swizzled layout
//   that the tcgen05 descriptors read, into a ring of four K and four V tiles.  Rows past the
//   context become zeros (what lies there is not used).
// * An MMA warp per query tile: S = Q K^T into tensor memory (two buffers of 64 columns,
//   alternate key tiles), P V from the P that the tile's softmax leaves over the first half of
//   the S buffer, into 128 columns of O.  S of the next keys goes in before P V of the current
//   ones, so each softmax finds its next scores ready.
// * Two softmax warpgroups, one per query tile, one thread per row: the row's 64 scores in
//   registers, mask, running maximum m and sum l in exp2 units, P.  O is rescaled only when a
//   row's maximum grows by more than 8 (log2), so P <= 2^8; the final O / l uses the same m.
// Every mbarrier wait is bounded (about 1 s) and checks a shared abort flag.
#include <cuda.h>
#include <cuda_runtime.h>

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
constexpr int kStages = 4;   // K ring, V ring
constexpr int kGroups = kKeys / 8;  // groups of eight tokens, each inside one block
constexpr int kMmaWarp = 8;         // MMA issue for query tile 0 (and loads Q); tile 1 has the next
constexpr int kCodeWarp = 10;       // looks blocks up, copies K codes; the next warp V's
constexpr int kWidenWarp = 12;      // the first of kWidenWarps for K, as many for V follow
constexpr int kWidenWarps = 4;
constexpr int kThreads = 32 * (kWidenWarp + 2 * kWidenWarps);
// 640 threads launch with 96 registers each; the softmax warpgroups hold a row of 64 scores
// and take kSoftmaxRegs, the other three keep kOtherRegs (2 x 144 + 3 x 64 = 5 x 96).
constexpr int kSoftmaxRegs = 144;
constexpr int kOtherRegs = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescale = 8.f;     // log2 growth of a row's maximum that forces a rescale of O
constexpr float kScaleRoom = 128.f; // growth of the largest V scale that moves vref

struct Params {
  CUtensorMap kmap;  // codes as [num_blocks][Hkv][B][d] bytes, box (d, B, 1, 1)
  CUtensorMap vmap;
  CUtensorMap qmap;  // q as [tokens][Hq][d], box (64, G, 128 / G): one query tile's half
  int q_tma;         // qmap is valid (G divides 128)
  const uint8_t* q;
  const float* k_scales;
  const float* v_scales;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;  // [n + 1]
  uint8_t* out;
  int num_seqs, num_tokens, num_q_heads, num_kv_heads, group, tpt;  // tpt = tokens per query tile
  int max_blocks_per_seq, block_size, log2_block, num_blocks;
  uint32_t group_magic;  // ceil(2^16 / G): r / G = r * group_magic >> 16 for r < 128
  int ncb;  // query blocks (of kTiles x tpt tokens) of the longest sequence
  float scale_log2;
  unsigned* err;
};

template <int D>
struct Smem {
  uint8_t q[kTiles][kRows * D * 2];     // K-major, 128-byte swizzle; 1024-byte aligned
  uint8_t k[kStages][kKeys * D * 2];    // f16, [64-column half][64 keys][128 B]
  uint8_t v[kStages][kKeys * D * 2];
  // [K, V][kt % 2]: codes as TMA lays them (128-byte swizzle at d = 128), and the groups'
  // scales over their reference
  uint8_t raw[2][2][kKeys * D];
  float ratio[2][2][kGroups];
  float kref[16], vref[16];            // of key tile kt at kt % 16
  unsigned long long q_full, q_ready;  // Q has landed; bf16 rows are f16 rows
  unsigned long long raw_full[2][2], raw_free[2][2];
  unsigned long long k_full[kStages], v_full[kStages];
  unsigned long long s_full[kTiles][2], p_full[kTiles][2];
  unsigned long long o_done[kTiles][kStages];  // P V of tile kt done (frees stage kt % kStages)
  unsigned long long fin;  // the MMA warps' last commits
  uint32_t tmem;
  int bad;    // a block id of this CTA's keys is out of range
  int abort;  // a wait gave up: every role stops
};

#define PA_R4(a) "=r"(r[a]), "=r"(r[a + 1]), "=r"(r[a + 2]), "=r"(r[a + 3])
#define PA_R16(a) PA_R4(a), PA_R4(a + 4), PA_R4(a + 8), PA_R4(a + 12)
// 64 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[64]) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : PA_R16(0), PA_R16(16), PA_R16(32), PA_R16(48)
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}
#undef PA_R16
#undef PA_R4

// tcgen05.mma and commit issued by the lane whose `el` is set.  The whole warp runs the code
// around them, so that descriptors and addresses stay in uniform registers, which the
// instruction takes; under a branch of one lane each operand is moved there first, and a
// thread issued one MMA in about 110 cycles, which bound the kernel.
__device__ __forceinline__ void mma_el(uint32_t tmem_d, uint64_t da, uint64_t db, uint32_t idesc,
                                       bool accumulate, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(da), "l"(db), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(el)
      : "memory");
}
// A from tensor memory (lane = row, column c = elements 2c and 2c + 1).
__device__ __forceinline__ void mma_ts_el(uint32_t tmem_d, uint32_t tmem_a, uint64_t db,
                                          uint32_t idesc, bool accumulate, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(db), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(el)
      : "memory");
}
__device__ __forceinline__ void commit_el(uint32_t bar, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(el)
      : "memory");
}
// One lane of a converged warp (its predicate as 0 or 1).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t el;
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(el));
  return el;
}

// Eight codes (two words) times a ratio -> eight f16 values.
__device__ __forceinline__ uint4 widen8(uint32_t lo, uint32_t hi, __half2 ratio) {
  auto two = [&](uint32_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
    const __half2 w = __hmul2(*reinterpret_cast<__half2*>(&h), ratio);
    return *reinterpret_cast<const uint32_t*>(&w);
  };
  return make_uint4(two(lo), two(lo >> 16), two(hi), two(hi >> 16));
}

__device__ __forceinline__ void st_shared16(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// A 32-bit load of data that no kernel of the call writes, kept at its place in the program.
__device__ __forceinline__ uint32_t ld_early(const void* src) {
  uint32_t v;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(src));
  return v;
}

// A bf16 row of q in shared memory (row r of a 128-row tile) becomes f16 values times 2^a, a
// chosen so that the largest magnitude lies in [2^14, 2^15); returns 2^-a.  A row that holds
// something not finite keeps a = 0.
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
  const int e = static_cast<int>(max(m2 & 0xffffu, m2 >> 16) >> 7);  // exponent field, bias 127
  const int fe = e == 255 ? 127 : min(253, 127 + 14 - (e - 127));
  const float f = __uint_as_float(static_cast<uint32_t>(fe) << 23);
  const float2 f2 = make_float2(f, f);
  auto two = [&](uint32_t w) {
    const float2 x = __fmul2_rn(unpack2<__nv_bfloat16>(w), f2);
    return pack2<__half>(x.x, x.y);
  };
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint32_t at = tile + swz(kRows, r, c);
    const uint4 w = ld_shared16(at);
    st_shared16(at, make_uint4(two(w.x), two(w.y), two(w.z), two(w.w)));
  }
  return __uint_as_float(static_cast<uint32_t>(254 - fe) << 23);
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 1) prefill_fp8_block_kernel(const __grid_constant__ Params p) {
  constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
  constexpr int CH = D / 8;        // 16-byte chunks of a 16-bit row
  constexpr int KS1 = D / 16;      // MMA k-steps of S = Q K^T
  constexpr int KS2 = kKeys / 16;  // MMA k-steps of P V
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
  // Launch order: the later half of every sequence's query blocks (the most keys) first, then
  // the earlier half, latest block first within each, so that the long CTAs do not come last;
  // the blocks of one (sequence, kv head) stay together and share their K/V in L2.
  const int s = blockIdx.y, g = blockIdx.z % p.num_kv_heads, half = blockIdx.z / p.num_kv_heads;
  const int nearly = p.ncb - static_cast<int>(gridDim.x);  // blocks in the earlier half
  if (half == 1 && static_cast<int>(blockIdx.x) >= nearly) return;  // (uniform over the CTA)
  const int cb = (half == 0 ? p.ncb : nearly) - 1 - static_cast<int>(blockIdx.x);
  const int qs = __ldg(p.query_start + s), qe = __ldg(p.query_start + s + 1);
  if (qs < 0 || qe < qs || qe > p.num_tokens) {  // rows that are not q's: nothing is touched
    if (tid == 0) atomicOr(p.err, kErrBadContext);
    return;
  }
  const int qlen = qe - qs;
  const int tpt = p.tpt, G = p.group;
  const int tok0 = cb * kTiles * tpt;
  if (tok0 >= qlen) return;  // (uniform over the CTA)
  const int ctx = __ldg(p.context_lens + s);
  T* outp = reinterpret_cast<T*>(p.out);
  if (ctx < 1 || ctx > p.max_blocks_per_seq * p.block_size || qlen > ctx) {
    const int ntok = min(kTiles * tpt, qlen - tok0);
    for (int i = tid; i < ntok * G * CH; i += kThreads) {
      const int r = i / CH, c = i % CH;
      reinterpret_cast<uint4*>(outp + ((static_cast<size_t>(qs + tok0 + r / G) * p.num_q_heads +
                                        g * G + r % G) * D))[c] = make_uint4(0, 0, 0, 0);
    }
    if (tid == 0) atomicOr(p.err, kErrBadContext);
    return;
  }
  // key tiles each query tile needs: up to the position of its last token
  int nt[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    const int ntok = min(tpt, qlen - (tok0 + t * tpt));
    nt[t] = ntok > 0 ? (ctx - qlen + tok0 + t * tpt + ntok - 1) / kKeys + 1 : 0;
  }
  const int n = max(nt[0], nt[1]);

  // ---- set-up: barriers, the first query rows on their way, tensor memory ----
  if (warp == kMmaWarp && lane == 0) {
    mbar_init(smem_addr(&sm.q_full), 33);  // TMA expect-tx + 32 copy lanes
    mbar_init(smem_addr(&sm.q_ready), kTiles * kRows);
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
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_addr(&sm.s_full[t][b]), 2);  // the MMA warp, its MMAs
        mbar_init(smem_addr(&sm.p_full[t][b]), kRows / 32);
      }
    }
    mbar_init(smem_addr(&sm.fin), kTiles);
    fence_mbar_init();
    sm.bad = 0;
    sm.abort = 0;
    // A whole query tile (tpt tokens x G heads = 128 rows, each token's G rows contiguous in
    // q) comes by TMA, one copy per 64-column half.
    uint32_t tma_bytes = 0;
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
      if (p.q_tma && tok0 + (t + 1) * tpt <= qlen) tma_bytes += kRows * D * 2;
    mbar_arrive_expect_tx(smem_addr(&sm.q_full), tma_bytes);
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      if (!(p.q_tma && tok0 + (t + 1) * tpt <= qlen)) continue;
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
        tma_load_3d(smem_addr(sm.q[t]) + h * kRows * 128, &p.qmap, h * 64, g * G, qs + tok0 + t * tpt,
                    smem_addr(&sm.q_full));
    }
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

  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp >= kWidenWarp) {
      // ===== widening: K (or V) tiles of the rings =====
      // Warp cw takes rows 16 cw .. 16 cw + 15 of each tile, two groups of eight tokens (eight
      // tokens never straddle a block, so a group has one scale).  At d = 128 a lane takes
      // 16-byte chunk (lane % 4) + 4 hc of one row of the group: eight lanes cover four chunks
      // of rows r and r ^ 5, which makes both the swizzled code loads and the swizzled f16
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
      for (int kt = 0; kt < n; ++kt) {
        const int st = kt % kStages, b = kt & 1;
        if (!wait(sm.raw_full[is_v][b], (kt >> 1) & 1)) break;
        const float2 r = *reinterpret_cast<const float2*>(&sm.ratio[is_v][b][2 * cw]);
        uint4 c[2][NH];
#pragma unroll
        for (int gi = 0; gi < 2; ++gi)
#pragma unroll
          for (int hc = 0; hc < NH; ++hc)
            c[gi][hc] = ld_shared16((raw ^ (hc * 64)) + b * (kKeys * D) + gi * 8 * D);
        // (the row of group gi: kt * 64 + 16 cw + 8 gi + rr)
        const int left = ctx - (kt * kKeys + 16 * cw + rr);
        if (left <= 8) {
#pragma unroll
          for (int gi = 0; gi < 2; ++gi)
            if (left <= 8 * gi) {
#pragma unroll
              for (int hc = 0; hc < NH; ++hc) c[gi][hc] = make_uint4(0, 0, 0, 0);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.raw_free[is_v][b]));
        if (kt >= kStages && !(wait(sm.o_done[0][st], (kt / kStages - 1) & 1) &&
                               wait(sm.o_done[1][st], (kt / kStages - 1) & 1)))
          break;
        const uint32_t tile = ring + st * (kKeys * D * 2);
#pragma unroll
        for (int gi = 0; gi < 2; ++gi) {
          const __half2 ratio = __float2half2_rn(gi ? r.y : r.x);
#pragma unroll
          for (int hc = 0; hc < NH; ++hc) {
            const uint32_t at = tile + 8 * gi * 128 + hc * (kKeys * 128);
            st_shared16(at + put0, widen8(c[gi][hc].x, c[gi][hc].y, ratio));
            st_shared16(at + put1, widen8(c[gi][hc].z, c[gi][hc].w, ratio));
          }
        }
        fence_async_smem();  // these stores before the tensor cores' reads
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&full[st]));
      }
    } else if (warp >= kCodeWarp) {
      // ===== blocks, scales and codes of K (or V): a tile ahead of the widening warps =====
      // Lane g < 8 looks after token group g of a tile.
      const int is_v = warp != kCodeWarp;
      const int32_t* trow = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
      // does tile kt's group hold keys that are used
      auto used = [&](int kt) -> bool { return lane < kGroups && kt < n && kt * kKeys + 8 * lane < ctx; };
      // its table entry; checked a tile later, when it is used, so that nothing waits for the
      // load (the loads here are volatile to stay where they are written)
      auto entry = [&](int kt) -> int {
        return used(kt) ? static_cast<int>(ld_early(trow + ((kt * kKeys + 8 * lane) >> p.log2_block))) : -1;
      };
      auto block_of = [&](int kt, int e) -> int {
        if (e >= 0 && e < p.num_blocks) return e;
        if (used(kt)) sm.bad = 1;
        return -1;
      };
      auto scale_of = [&](const float* scales, int e) -> float {
        return e >= 0 ? __uint_as_float(ld_early(scales + static_cast<size_t>(e) * p.num_kv_heads + g)) : 0.f;
      };
      const int raw0 = entry(0);
      int raw_e = entry(1);
      int e = block_of(0, raw0);
      // (K's warp follows the V scales too: it tells the softmax both references)
      float sk = is_v ? 0.f : scale_of(p.k_scales, e), sv = scale_of(p.v_scales, e);
      float vref = 0.f;
      const bool first_group = ((8 * lane) & (p.block_size - 1)) == 0;  // of its block
      for (int kt = 0; kt < n; ++kt) {
        const int e1 = block_of(kt + 1, raw_e);
        const float sk1 = is_v ? 0.f : scale_of(p.k_scales, e1), sv1 = scale_of(p.v_scales, e1);
        raw_e = entry(kt + 2);
        // (scales are positive, so their bits order as integers)
        const float kref = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(sk)));
        const float vtop = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(sv)));
        if (kt == 0 || vtop > vref * kScaleRoom) vref = vtop;
        const float ref = is_v ? vref : kref;
        const float ratio = ref > 0.f ? (is_v ? sv : sk) * __frcp_rn(ref) : 0.f;
        const int b = kt & 1;
        if (kt >= 2 && !wait(sm.raw_free[is_v][b], (kt / 2 - 1) & 1)) break;
        // free: tile kt - 2 is read, with its ratios; K's tile kt - 3 is widened, so the P V of
        // kt - 7 is done, and the softmax of kt - 16 is long done with its references
        if (lane < kGroups) sm.ratio[is_v][b][lane] = ratio;
        if (lane == 0 && !is_v) {
          sm.kref[kt & 15] = kref;
          sm.vref[kt & 15] = vref;
        }
        const bool mine = first_group && e >= 0;  // (e < 0 past the groups)
        const uint32_t blocks = __ballot_sync(0xffffffffu, mine);
        __syncwarp();  // the stores above before the arrival
        if (lane == 0)
          mbar_arrive_expect_tx(smem_addr(&sm.raw_full[is_v][b]),
                                static_cast<uint32_t>(__popc(blocks) * p.block_size * D));
        __syncwarp();
        if (mine)
          tma_load_4d(smem_addr(sm.raw[is_v][b]) + 8 * lane * D, is_v ? &p.vmap : &p.kmap, 0, 0, g, e,
                      smem_addr(&sm.raw_full[is_v][b]));
        e = e1;
        sk = sk1;
        sv = sv1;
      }
    } else {
      if (warp == kMmaWarp) {
        // ===== query tiles that run past their sequence (the whole ones are on their way) =====
        // by 16-byte copies; rows past the last token are zeros
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          const int first = tok0 + t * tpt;
          if (first >= qlen || (p.q_tma && first + tpt <= qlen)) continue;
          // (rows past tpt * G, where G does not divide 128, are zeros too)
          for (int u = lane; u < kRows * CH; u += 32) {
            const int r = u / CH, c = u % CH;
            const int tok = first + r / G;
            const bool live = r < tpt * G && tok < qlen;
            const uint8_t* src = p.q + ((static_cast<size_t>(qs + (live ? tok : 0)) * p.num_q_heads +
                                         g * G + (live ? r % G : 0)) * D + c * 8) * 2;
            cp_async16(smem_addr(sm.q[t]) + swz(kRows, r, c), src, live ? 16u : 0u);
          }
        }
        cp_async_arrive(smem_addr(&sm.q_full));
      }
      // ============ MMA issue: a warp per query tile ============
      // The tensor pipe runs one thread's MMAs in order, so S of key tile kt + 1 may overwrite
      // the P of kt - 1, whose P V was issued before it.  A warp whose query tile needs no more
      // keys still frees each stage, after it has landed.
      const int t = warp - kMmaWarp;
      const int ntt = t == 0 ? nt[0] : nt[1];
      const uint32_t el = elect_one();
      auto wwait = [&](unsigned long long& bar, int parity) -> bool {  // warp-uniform result
        return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
      };
      constexpr uint32_t id_s = idesc_f16<__half>(kRows, kKeys, false);
      constexpr uint32_t id_o = idesc_f16<__half>(kRows, D, true);
      constexpr uint32_t kStageBytes = kKeys * D * 2;
      const uint64_t qd = desc_sw128(smem_addr(sm.q[t]), 16, 1024);
      const uint64_t dk0 = desc_sw128(smem_addr(sm.k[0]), 16, 1024);
      const uint64_t dv0 = desc_sw128(smem_addr(sm.v[0]), kKeys * 128, 1024);
      const uint32_t cols = tmem + t * kTileCols;
      auto issue_s = [&](int kt) {
        const uint32_t d = cols + (kt & 1) * kColS;
        const uint64_t kd = dk0 + (((kt % kStages) * kStageBytes) >> 4);
#pragma unroll
        for (int ks = 0; ks < KS1; ++ks)  // 16 columns = 32 bytes of 64-column block ks / 4
          mma_el(d, qd + (((ks >> 2) * kRows * 128 + (ks & 3) * 32) >> 4),
                 kd + (((ks >> 2) * kKeys * 128 + (ks & 3) * 32) >> 4), id_s, ks > 0, el);
        commit_el(smem_addr(&sm.s_full[t][kt & 1]), el);
        if (el) mbar_arrive(smem_addr(&sm.s_full[t][kt & 1]));  // (passes k_full on to the softmax)
      };
      auto issue_pv = [&](int kt) {
        const uint32_t pa = cols + (kt & 1) * kColS, o = cols + kColO;
        const uint64_t vd = dv0 + (((kt % kStages) * kStageBytes) >> 4);
#pragma unroll
        for (int ks = 0; ks < KS2; ++ks)  // 16 keys = 8 columns of P
          mma_ts_el(o, pa + ks * 8, vd + ((ks * 16 * 128) >> 4), id_o, kt > 0 || ks > 0, el);
      };
      bool ok = wwait(BF ? sm.q_ready : sm.q_full, 0);
      fence_async_smem();  // q rows that lanes copied or converted -> tensor cores
      ok = ok && wwait(sm.k_full[0], 0);
      if (ok && ntt > 0) issue_s(0);
      for (int kt = 0; ok && kt < n; ++kt) {
        const int st = kt % kStages;
        if (kt + 1 < ntt) {
          if (!(ok = wwait(sm.k_full[(kt + 1) % kStages], ((kt + 1) / kStages) & 1))) break;
          issue_s(kt + 1);
        }
        if (!(ok = wwait(sm.v_full[st], (kt / kStages) & 1))) break;
        if (kt < ntt) {
          if (!(ok = wwait(sm.p_full[t][kt & 1], (kt >> 1) & 1))) break;
          tc_fence_after();
          issue_pv(kt);
        } else if (!(ok = wwait(sm.k_full[st], (kt / kStages) & 1))) {
          break;
        }
        commit_el(smem_addr(&sm.o_done[t][st]), el);
      }
      commit_el(smem_addr(&sm.fin), el);  // every MMA this warp issued
      wwait(sm.fin, 0);
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ================= softmax: warpgroup t, one thread per row =================
    const int t = warp >> 2, r = tid & (kRows - 1);
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + t * kTileCols;
    const int tok = tok0 + t * tpt + r / G;
    const bool row_ok = r / G < tpt && tok < qlen;
    const int pos = row_ok ? ctx - qlen + tok : -1;
    const int pos_lo = ctx - qlen + tok0 + t * tpt;  // the tile's first position
    float m_used = -INFINITY, l_run = 0.f, vref = 0.f;
    bool ok = true;
    auto wwait = [&](unsigned long long& bar, int parity) -> bool {  // warp-uniform result
      return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    };
    float row_scale = p.scale_log2;  // of this row's scores, before the key tile's kref
    if constexpr (BF) {
      ok = wwait(sm.q_full, 0);
      if (ok && nt[t] > 0) row_scale *= q_row_to_f16<D>(smem_addr(sm.q[t]), r);
      fence_async_smem();  // the row before the tensor cores' reads
      mbar_arrive(smem_addr(&sm.q_ready));
    }
    for (int kt = 0; ok && kt < nt[t]; ++kt) {
      const int b = kt & 1;
      // (kref and vref were written before k_full of this tile, which the MMA warp acquired
      // before it arrived here)
      if (!(ok = wwait(sm.s_full[t][b], (kt >> 1) & 1))) break;
      tc_fence_after();
      // the tile's factor of the raw scores, positive (so that the maximum commutes with it and
      // a masked -inf stays -inf even where it would underflow)
      const float c = fmaxf(sm.kref[kt & 15] * row_scale, 1e-37f);
      const float vnew = sm.vref[kt & 15];
      float sv[kKeys];
      tmem_ld64(tl + b * kColS, sv);
      if (kt * kKeys + kKeys - 1 > pos_lo) {  // causal mask: key kt * 64 + i > pos
        const int lim = pos - kt * kKeys;
#pragma unroll
        for (int i = 0; i < kKeys; ++i)
          if (i > lim) sv[i] = -INFINITY;
      }
      float pm[4];  // four chains of three-input maxima
#pragma unroll
      for (int j = 0; j < 4; ++j) pm[j] = fmaxf(sv[2 * j], sv[2 * j + 1]);
#pragma unroll
      for (int i = 8; i < kKeys; i += 8)
#pragma unroll
        for (int j = 0; j < 4; ++j) pm[j] = fmax3(pm[j], sv[i + 2 * j], sv[i + 2 * j + 1]);
      const float mx = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
      const float m_new = fmaxf(m_used, mx * c);
      const bool need = kt > 0 && m_new > m_used + kRescale;
      const bool moved = kt > 0 && vnew != vref;  // (uniform over the CTA)
      if (moved || __any_sync(0xffffffffu, need)) {
        // rescale O, once P V of tile kt - 1 is done (that of kt - 2 was issued before this S)
        if (!(ok = wwait(sm.o_done[t][(kt - 1) % kStages], ((kt - 1) / kStages) & 1))) break;
        tc_fence_after();
        float alpha = need ? ex2(m_used - m_new) : 1.f;
        if (need) {
          l_run *= alpha;
          m_used = m_new;
        }
        if (moved) alpha *= vref / vnew;
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 32) {
          float o[32];
          tmem_ld32(tl + kColO + c0, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= alpha;
          tmem_st32(tl + kColO + c0, o);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      }
      if (kt == 0) m_used = m_new;
      vref = vnew;
      // P = 2^(s c - m), rounded to f16, packed two a column over the first half of this
      // thread's own row of S (already in registers); a row with nothing unmasked yet has
      // every score at -inf, so any finite offset gives it P = 0
      const float neg_m = m_used == -INFINITY ? 0.f : -m_used;
      const float2 c2 = make_float2(c, c), nm2 = make_float2(neg_m, neg_m);
      float2 ps[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                      make_float2(0.f, 0.f)};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 x = __ffma2_rn(make_float2(sv[32 * h + i], sv[32 * h + i + 1]), c2, nm2);
          const float2 e = make_float2(ex2(x.x), ex2(x.y));
          ps[(i >> 1) & 3] = __fadd2_rn(ps[(i >> 1) & 3], e);
          pk[i >> 1] = pack2<__half>(e.x, e.y);
        }
        tmem_st16(tl + b * kColS + 16 * h, pk);
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before();  // the P stores before the MMA warp reads them
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sm.p_full[t][b]));
      const float2 s01 = __fadd2_rn(ps[0], ps[1]), s23 = __fadd2_rn(ps[2], ps[3]);
      const float2 sall = __fadd2_rn(s01, s23);
      l_run += sall.x + sall.y;
    }
    if (ok && nt[t] > 0) ok = wwait(sm.o_done[t][(nt[t] - 1) % kStages], ((nt[t] - 1) / kStages) & 1);
    // ---- out = O vref / l, after every role is done (the bad-block flag is final) ----
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const bool good = ok && sm.abort == 0 && sm.bad == 0;
    const float inv = vref / l_run;
    // (clamped: a cached f16 value may have been rounded up past 65504)
    // The rows go out through shared memory (the K ring, idle now), so that each store
    // instruction of a warp writes whole rows.  Row r's 16-byte chunk c sits at chunk
    // c ^ (r % CH) of its 2 D-byte staging row, so that neither the writes nor the reads
    // collide in a bank much.
    static_assert(kStages * kKeys >= 8 * 32, "the K ring holds a staging row per thread");
    const uint32_t stage = smem_addr(sm.k[0]) + static_cast<uint32_t>(warp) * 32 * D * 2;
    const int rw = r & 31;
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += 32) {
      float o[32];
      if (nt[t] > 0 && sm.abort == 0) tmem_ld32(tl + kColO + c0, o);  // (warp-uniform)
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (good && nt[t] > 0) {
          w.x = pack2_sat<T>(o[8 * cc + 0] * inv, o[8 * cc + 1] * inv);
          w.y = pack2_sat<T>(o[8 * cc + 2] * inv, o[8 * cc + 3] * inv);
          w.z = pack2_sat<T>(o[8 * cc + 4] * inv, o[8 * cc + 5] * inv);
          w.w = pack2_sat<T>(o[8 * cc + 6] * inv, o[8 * cc + 7] * inv);
        }
        const int ch = c0 / 8 + cc;  // 16-byte chunk of the row
        st_shared16(stage + rw * D * 2 + ((ch ^ (rw & (CH - 1))) << 4), w);
      }
    }
    __syncwarp();
    // piece i of the warp: row i / CH, chunk i % CH
    const int ch = lane % CH;
    const size_t row0 = static_cast<size_t>(qs + tok0 + t * tpt) * p.num_q_heads + g * G;
#pragma unroll 8
    for (int rr = lane / CH; rr < 32; rr += 32 / CH) {
      const int rrow = (r - rw) + rr;  // the row in the tile: token tk of it, head rrow % G
      const int tk = static_cast<int>((rrow * p.group_magic) >> 16);
      if (tk < tpt && tok0 + t * tpt + tk < qlen)
        reinterpret_cast<uint4*>(outp + (row0 + static_cast<size_t>(tk) * (p.num_q_heads - G) + rrow) * D)[ch] =
            ld_shared16(stage + rr * D * 2 + ((ch ^ (rr & (CH - 1))) << 4));
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && sm.bad) atomicOr(p.err, kErrBadBlock);
    return;
  }
  // the other roles: the two CTA-wide barriers of the softmax epilogue
  tc_fence_before();
  __syncthreads();
  __syncthreads();
  if (warp == kMmaWarp + 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

template <int D, typename T>
int launch(const Params& prm, int max_query_len, cudaStream_t stream) {
  const size_t smem = sizeof(Smem<D>) + 1024;
  auto* kern = prefill_fp8_block_kernel<D, T>;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), smem)) return -3;
  cudaLaunchConfig_t cfg = {};
  const int per_cta = kTiles * prm.tpt;
  const int ncb = (max_query_len + per_cta - 1) / per_cta;
  Params q = prm;
  q.ncb = ncb;
  // x: a block within its half (the later half has ceil(ncb / 2)), y: sequence,
  // z: half x kv head
  cfg.gridDim = dim3((ncb + 1) / 2, prm.num_seqs, 2 * prm.num_kv_heads);
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
                             const float* v_scales, cudaStream_t stream) {
  prefill8::Params p;
  p.q = static_cast<const uint8_t*>(a.q);
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
  if (a.head_dim == 128)
    return a.bf16 ? prefill8::launch<128, __nv_bfloat16>(p, a.max_query_len, stream)
                  : prefill8::launch<128, __half>(p, a.max_query_len, stream);
  if (a.head_dim == 64)
    return a.bf16 ? prefill8::launch<64, __nv_bfloat16>(p, a.max_query_len, stream)
                  : prefill8::launch<64, __half>(p, a.max_query_len, stream);
  return -1;
}

}  // namespace pa
