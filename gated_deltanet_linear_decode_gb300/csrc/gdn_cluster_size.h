// gdn_cluster_size.h -- the size of a thread-block cluster.  Host code.
#pragma once

namespace gdn {

constexpr int kPortableCluster = 8;   // CTAs that every device of this kind takes

// The size to launch where `ctas` are wanted: at most that, and more than the portable one only where a cluster of them has room.
// clusters(n): how many clusters of n CTAs run at a time; 0 or less where none does or nobody can say.
template <class F>
int cluster_that_fits(int ctas, F clusters) {
    return ctas > kPortableCluster && clusters(ctas) < 1 ? kPortableCluster : ctas;
}

}  // namespace gdn
