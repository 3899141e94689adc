// latent_loads.h -- which loads the producer of latent_prefill.cu has asked for, and
// what it waits for before its CTA may leave after a wait that ran out: every phase
// whose loads may still be in flight, and none whose loads were never asked for (such
// a phase does not complete, and each would hold the CTA for the whole limit again).
#pragma once

#ifdef __CUDACC__
#define PKV_HD_LOADS __host__ __device__ __forceinline__
#else
#define PKV_HD_LOADS inline
#endif

namespace pkv_loads {

// A key tile's loads in three parts, each with a barrier for even and one for odd
// tiles; an item's two query tiles, with a barrier each.
enum { KEY0 = 0, KEYS, VALUES, PARTS };

struct Asked {
    int tiles[PARTS] = {0, 0, 0};      // key tiles whose part has been asked for
    int queries[2] = {0, 0};           // items whose query tile has been

    // part(p, tile) and query(g, item) wait for one phase.  (The phase before it on the
    // same barrier has completed: its loads were in use before the next were asked for.)
    template <class Part, class Query>
    PKV_HD_LOADS void drain(const Part &part, const Query &query) const
    {
        for (int p = 0; p < PARTS; ++p)
            for (int t = tiles[p] < 2 ? 0 : tiles[p] - 2; t < tiles[p]; ++t) part(p, t);
        for (int g = 0; g < 2; ++g)
            if (queries[g] > 0) query(g, queries[g] - 1);
    }
};

}  // namespace pkv_loads
