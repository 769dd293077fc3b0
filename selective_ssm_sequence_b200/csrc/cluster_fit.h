// cluster_fit.h -- how many blocks of a cluster a launch may have (host only).
#pragma once

namespace hm {

// Clusters of up to 8 blocks run on every device; of more only where the device
// (or the share of it that a process has) holds them together.  fits(cluster)
// says so; what does not fit is halved, down to 8.
template <typename Fits>
int placeable_cluster(int cluster, Fits fits) {
    while (cluster > 8 && !fits(cluster)) cluster /= 2;
    return cluster;
}

}  // namespace hm
