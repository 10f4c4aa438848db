// How many clusters of each size the block-scaled products can count on (host
// code; no CUDA types, so that it is tested without a device).
#pragma once

namespace moe {
namespace f8b {

constexpr int MAX_SPLIT = 8;  // CTAs that may share a tile: the portable cluster size

// clusters[s], s = 2 .. MAX_SPLIT: co-resident clusters of s CTAs as query(s, &n)
// reports them (true = known). A size that cannot be asked, or has none, is 0: the
// launcher passes it over, and with all of them 0 no tile is shared. The other
// kernels of the library do not depend on any of it.
template <typename Query>
void co_resident_clusters(Query query, int* clusters) {
  for (int s = 2; s <= MAX_SPLIT; ++s) {
    int n = 0;
    clusters[s] = query(s, &n) && n > 0 ? n : 0;
  }
}

}  // namespace f8b
}  // namespace moe
