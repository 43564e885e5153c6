// ring_places.cuh -- which slot of a ring is filled and which is read next.  Plain C++ as well as device
// code: what it does after a wait that gave up cannot be provoked on a GPU, so it is tested on the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define EP_PLACES __host__ __device__ __forceinline__
#else
#define EP_PLACES inline
#endif

// A ring of DEPTH slots, filled by asynchronous copies and read in the same order.  issue(slot) starts the copy
// into a slot; wait(slot, parity) is a bounded wait for it, false when it gave up.  After one that gave up no
// copy is started, none is taken for read, and drain() waits once more for just those that are in flight.
template <int DEPTH>
struct RingPlaces {
    int put_slot = 0, take_slot = 0, flying = 0;
    uint32_t parity = 0;
    bool ok = true;

    template <class Issue>
    EP_PLACES void put(Issue issue) {
        if (!ok) return;
        issue(put_slot);
        ++flying;
        put_slot = put_slot + 1 == DEPTH ? 0 : put_slot + 1;
    }

    // The slot to read: the oldest one.
    template <class Wait>
    EP_PLACES int take(Wait wait) {
        const int slot = take_slot;
        ok = ok && wait(slot, parity);
        if (ok) next();
        return slot;
    }

    // Nothing is in flight afterwards, unless a copy was not over after two waits.  False: a wait gave up.
    template <class Wait>
    EP_PLACES bool drain(Wait wait) {
        while (flying > 0) {
            ok = wait(take_slot, parity) && ok;
            next();
        }
        return ok;
    }

    EP_PLACES void next() {
        --flying;
        if (++take_slot == DEPTH) { take_slot = 0; parity ^= 1; }
    }
};
