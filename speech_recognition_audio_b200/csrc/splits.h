// How many blocks of a cluster share one tile's states (host only, no CUDA).
#pragma once

namespace asr {

// Blocks a (segment, tile, head) is split into: a power of two, as long as the
// grid does not yet fill `fill` blocks and each block keeps at least `least`
// keys; up to `most` (8 is the portable cluster size, 16 goes through cap_splits).
inline int pick_splits(long long blocks, int keys, int least, long long fill, int most = 8) {
  int s = 1;
  while (s < most && blocks * s < fill && keys >= 2 * s * least) s *= 2;
  return s;
}

// The same for the tiles of 128 states: a tile of states takes about 1.5 us a
// pass, and each block of a cluster costs about 0.12 us to get going, so the S
// with the least
// cost tiles / S + blocks S, cost = 12.5 a pass.  Measured (attention, us) at 1,
// 8 and 16, or the most that leaves a block a tile: 4 blocks x 235 tiles 281,
// 48, 33; 12 x 235 282, 51, 47; 12 x 63 80, 23, 25; 12 x 12 19, 14; 48 x 12 20,
// 22; 96 x 12 20, 33.
inline int tile_splits(double blocks, int tiles, double cost, int num_sms) {
  double least = cost * tiles;
  int best = 1;
  for (int S = 2; S <= 16 && S <= tiles && blocks * S <= 2 * num_sms; S *= 2)
    if (cost * tiles / S + blocks * S < least) best = S, least = cost * tiles / S + blocks * S;
  return best;
}

// The splits as a cluster that the device holds: 16 blocks where `wide()` says
// so (a device or context with few SMs may not), else the portable 8.
template <typename Wide>
int cap_splits(int splits, Wide wide) {
  return splits > 8 && !wide() ? 8 : splits;
}

}  // namespace asr
