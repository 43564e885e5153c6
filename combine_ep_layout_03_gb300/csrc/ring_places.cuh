// ring_places.cuh -- which slot of a ring is filled and which is read next.  Plain C++ as well as device
// code: what it does after a wait that gave up cannot be provoked on a GPU, so it is tested on the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define EP_PLACES __host__ __device__ __forceinline__
#else
#define EP_PLACES inline
#endif

// A ring of DEPTH slots, filled by asynchronous copies and read in the same order, every one of them.  issue(slot)
// starts the copy into a slot; wait(slot, parity) is a bounded wait for it, false when it gave up.  Where one gives
// up, take() waits once more for it and for the others in flight there and then; no copy is started, and none
// waited for, after that.  So nothing is in flight once all have been taken, unless a copy outlasts two waits.
template <int DEPTH>
struct RingPlaces {
    int put_slot = 0, take_slot = 0;
    uint32_t parity = 0;
    bool ok = true;   // no wait gave up

    template <class Issue>
    EP_PLACES void put(Issue issue) {
        if (ok) issue(put_slot);
        put_slot = put_slot + 1 == DEPTH ? 0 : put_slot + 1;
    }

    // The slot to read: the oldest one.
    template <class Wait>
    EP_PLACES int take(Wait wait) {
        const int slot = take_slot;
        const bool arrived = !ok || wait(slot, parity);
        if (!arrived) {
            int late = slot;
            uint32_t of = parity;
            do {
                wait(late, of);
                if (++late == DEPTH) { late = 0; of ^= 1; }
            } while (late != put_slot);
            ok = false;
        }
        if (++take_slot == DEPTH) { take_slot = 0; parity ^= 1; }
        return slot;
    }
};
