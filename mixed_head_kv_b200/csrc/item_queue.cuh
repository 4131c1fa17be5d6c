// item_queue.cuh — the queue through which a persistent CTA's loading thread hands
// its work items to the other warps, and the per-item marks that go with it.
// Host and device code: a host build is checked over all interleavings.
//
// Item `ord` is in slot ord % kQueueSlots. Every consumer takes every item, in order,
// and frees the slot as it takes the item, not when it is done with it. So item ord is
// published once all consumers have taken item ord - kQueueSlots, and whoever holds
// item ord knows of the others only that they are done with everything before
// ord - kQueueSlots.
//
// A mark says something of one item (some consumers set it, others read it while they
// hold the item). It is the item's number, written into place ord % kItemMarks and
// compared with the reader's: nobody has to clear it. The next item of the same place,
// ord + kItemMarks, is taken only when every reader has taken ord + kItemMarks -
// kQueueSlots, an item behind ord, and so is done with ord.
#pragma once

namespace duo {

constexpr int kQueueSlots = 4;
constexpr int kItemMarks = 8;
static_assert(kItemMarks > kQueueSlots, "a mark outlives its readers");

constexpr int kNoItem = -1;  // what the places hold at first

#if defined(__CUDACC__)
__host__ __device__
#endif
constexpr int mark_place(int ord) { return ord % kItemMarks; }

}  // namespace duo
