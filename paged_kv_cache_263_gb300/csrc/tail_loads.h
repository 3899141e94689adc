// tail_loads.h -- what the producer of shared_tail.cu waits for before it leaves: every
// phase whose loads may still be in flight.  Consumers that gave up on a wait are gone, and
// a load may not land in shared memory that is another CTA's by then.  No phase is waited
// for that never completes (it would hold the CTA for the whole limit), nor one that a
// later phase on its barrier has followed (its parity would be taken for the other's).
#pragma once

#ifdef __CUDACC__
#define PKV_HD_TAIL __device__ __forceinline__
#else
#define PKV_HD_TAIL inline
#endif

namespace pkv_tail {

// Of a ring of `ring` stages, all `blocks` blocks were asked for in turn; of the items'
// queries, `items`, in `slots` slots.  ended: the mark that no more items come followed in
// the next slot, after the queries that were there before it had been read.
template <class Block, class Item>
PKV_HD_TAIL void drain(int blocks, int ring, int items, int slots, bool ended, const Block &block, const Item &item)
{
    for (int u = blocks < ring ? 0 : blocks - ring; u < blocks; ++u) block(u);
    const int last = ended ? slots - 1 : slots;
    for (int k = items < last ? 0 : items - last; k < items; ++k) item(k);
}

}  // namespace pkv_tail
