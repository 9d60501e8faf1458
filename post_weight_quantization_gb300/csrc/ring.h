// Rings in shared memory whose uses several sets of warps take in turn.
#pragma once

namespace gptq {

// Use n of a ring lies in place n % places. A barrier's wait tests one bit, the parity of the barrier's uses: that tells a use only
// from the one before on the same barrier, so a waiter must know the one before to be complete. Copies land, and MMAs
// signal, in no order that may be relied on, so it knows that of a use that it has waited for itself, and of no other. A set that
// takes every `step`-th use therefore needs barriers that it alone waits on in turn: use n on barrier n % barriers, with
// as many barriers as the places or more, so that a place's earlier use is over, and a multiple of the step (which has to be the
// same all the way).
constexpr int barriers_for(int places, int step) { return (places + step - 1) / step * step; }

}  // namespace gptq
