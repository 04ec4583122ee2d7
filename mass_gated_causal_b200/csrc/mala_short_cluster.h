// mala_short_cluster.h -- how many CTAs a short cache's decode gives to each
// (sequence, KV head). Host arithmetic only, without CUDA's headers.
#pragma once

namespace mala {

constexpr int kShortTiles = 8;     // key tiles a CTA of a short decode takes at most
constexpr int kShortCluster = 16;  // and CTAs of its cluster (more than 8 is not portable)

// CTAs per (sequence, KV head) if the whole decode is one launch of clusters, else 0.
//
//   units   (sequence, KV head) pairs
//   tiles   key tiles of the longest cache there is room for
//   ctas    CTAs of the kernel that the GPU holds at once
//   room    room(cluster, tiles of a CTA): how many such clusters the GPU holds at
//           once. A cluster lies within one part of the GPU, so that is fewer than
//           ctas / cluster (of sixteen CTAs, two to an SM, 14 and not 18), and none
//           where a part is too small for one.
//
// As many CTAs as leave each two tiles and are on the GPU at once. Where even a CTA's
// eight tiles do not reach the end, or the clusters would come in two waves, equal runs
// of all tiles are faster: 8 sequences of 2K keys, 8 KV heads, 12.8 us against 16.5 for
// the two kernels, but 16 of 4K keys in two waves 53 against 46.5; 2 sequences of 2K keys,
// 8 KV heads, 8.7 us with clusters of eight and 14.1 with sixteen in two waves (in a graph).
template <class Room>
int short_cluster(long long units, long long tiles, long long ctas, Room&& room) {
  int c = 1;
  while (c < kShortCluster && 2 * c < tiles && units * 2 * c <= ctas) c *= 2;
  for (; c >= 1; c /= 2) {
    const long long each = (tiles + c - 1) / c;
    if (each > kShortTiles) return 0;
    if (units <= room(c, static_cast<int>(each))) return c;
  }
  return 0;
}

}  // namespace mala
