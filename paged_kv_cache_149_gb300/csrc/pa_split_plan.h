// The cuts of the split attention (pa_split_attention.cu), written for host and device so that they can be
// driven on the CPU as well.
//
// A batch's items (a sequence, a kv head and its query tiles) stand in a row, each as long as its key tiles
// and kItemCost more; the units are cut into equal shares, one per CTA, wherever the cuts fall.
#pragma once

#if defined(__CUDACC__)
#define PA_PLAN_FN __host__ __device__ __forceinline__
#else
#define PA_PLAN_FN inline
#endif

namespace pa {
namespace split {

// An item's start and end, in key tiles, for the shares; and the least key tiles of a piece: a cut that
// would leave fewer moves to the item's end.  (64 contexts of 128..2048 / 64 rows over 100..1500: 3 and 2
// 54.9 / 48.6 us, 2 and 4 56.8 / 50.4, 1 and 2 59.5 / 53.9, 4 and 2 55.1 / 49.3.)
constexpr int kItemCost = 3;
constexpr int kLeastPiece = 2;

// Units of an item of so many key tiles.
PA_PLAN_FN long long item_units(int tiles) { return static_cast<long long>(tiles) + kItemCost; }

// Units of a share of `total` among `grid` CTAs; `cut`: items may be cut.
PA_PLAN_FN long long share_units(long long total, long long grid, bool cut) {
  const long long even = (total + grid - 1) / grid, least = cut ? kLeastPiece : 1;
  return even > least ? even : least;
}

// Where a share ends: before key tile `tile` of item `item` (of its sequence).
struct Place {
  long long item;
  int tile;
  int off;  // units of the item before the end as it fell
};

// The place of unit x of a sequence whose items have `tiles` key tiles each.
PA_PLAN_FN Place place_of(long long x, int tiles, bool cut) {
  Place at;
  at.item = x / item_units(tiles);
  at.off = static_cast<int>(x - at.item * item_units(tiles));
  at.tile = at.off > kItemCost ? at.off - kItemCost : 0;
  if (at.tile < kLeastPiece && (cut || at.off <= 0)) {
    at.tile = 0;
  } else if (!cut || tiles - at.tile < kLeastPiece) {  // the item's end, which is the next one's start
    at.tile = 0;
    ++at.item;
  }
  return at;
}

// Pieces of an item after the first, which ends `off` units in: the later cuts lie share units apart.
PA_PLAN_FN int followers_of(int tiles, long long off, long long share) {
  return 1 + static_cast<int>((tiles - kLeastPiece + kItemCost - off) / share);
}

}  // namespace split
}  // namespace pa
