// gdn_chunk_strays.h -- how the two CTAs of a pair of gdn_attn_chunk (gdn_chunk_tc.cu) agree on whether a part has strays: infinite
// or NaN values among its late keys, which the softmax warps take out of shared memory, each CTA of its own channels.  Both CTAs' rows
// get what either has found.  Host and device code.
//
// A finder marks the part in both CTAs, its own and by a remote store, before it arrives for the tile's product.  At a part's end a
// thread that has waited for the part's last product -- behind which both CTAs' finders are -- takes the mark over into `now`, before a
// barrier of the CTA's softmax warps.  Behind that barrier all of them go by `now`, which no other CTA writes (whoever joins the parts
// of a unit sets it where any of them had some): the marks are the other CTA's too, and it may be at the next part already, so
// warps that looked at them would not all see the same.
//
// It is never further than that: the next part's last product is behind this CTA's weights for it, and so behind the barrier that ends
// this part.  So there are two marks, by the parity of the parts with tiles (between parts without one the CTAs are not held
// together), and one is taken back when it has been taken over, ahead of the part but one that uses it next.
#pragma once

#ifdef __CUDACC__
#define GDN_HD __host__ __device__ __forceinline__
#else
#define GDN_HD inline
#endif

namespace gdn {
namespace chunk {

struct Strays {
    volatile int found[2];
    volatile int part;       // which of them is this part's: the number of parts with tiles before it, mod 2
    volatile int now;        // this part has some

    GDN_HD void clear() {
        found[0] = 0;
        found[1] = 0;
        part = 0;
        now = 0;
    }
    GDN_HD volatile int* mark() { return found + part; }   // and the same place in the other CTA
    GDN_HD void take_over(bool tiles) {
        now = 0;
        if (!tiles) return;
        now = found[part];
        found[part] = 0;
        part = part ^ 1;
    }
};

}  // namespace chunk
}  // namespace gdn
