// How the CTAs of a K-split cluster exchange their partial tiles and leave, for
// one CTA; what the steps do is the link's (device: mx_gemm.cuh).
//
// A CTA that has left may not be addressed any more: no arrival, no copy into its
// shared memory, none that still reads it.  So
//   - whatever a CTA does to others it does before it arrives at the cluster's
//     barrier, and nobody leaves before everybody has arrived.  A CTA whose main
//     loop gave up takes part like the others;
//   - no wait stops because another one gave up: a CTA that did would be missing
//     to the others, or gone.  All have a limit of their own, so all end, and with
//     them the cluster's barrier, which has none;
//   - without a failure every share has arrived before its receiver
//     arrives at the barrier, and every announcement before that, so nothing is in
//     flight when the cluster leaves.  A receiver that gave up says so to everybody
//     before it arrives, and all then wait for what may still be in flight.
#pragma once
#include "work_sched.h"

namespace qg {

// Up to the barrier.  `first`: the thread that acts for the CTA; all others call it
// too.  Returns whether all shares have arrived.
//   expect()           counts the bytes that will be received
//   announce(z)        CTA z may send: this CTA is through with its ring
//   await_announced()  every CTA has announced itself here; bounded
//   send(z)            CTA z's share of this CTA's partial tile
//   await_shares()     every CTA's share has arrived here; bounded
//   warn(z)            CTA z learns, before the barrier, that copies may be late
//   arrive()           at the cluster's barrier
template <typename Link>
QG_HD bool mx_exchange(Link& l, int splits, bool first) {
    if (first) {
        l.expect();
        for (int z = 0; z < splits; ++z) l.announce(z);
        if (l.await_announced())
            for (int z = 0; z < splits; ++z) l.send(z);
    }
    const bool got = l.await_shares();
    if (first && !got)
        for (int z = 0; z < splits; ++z) l.warn(z);
    l.arrive();
    return got;
}

// The last thing before the CTA leaves.
//   wait()    until every CTA of the cluster has arrived
//   warned()  whether one of them has warned this one
//   settle()  long enough for what is in flight to land
template <typename Link>
QG_HD void mx_exchange_leave(Link& l) {
    l.wait();
    if (l.warned()) l.settle();
}

}  // namespace qg
