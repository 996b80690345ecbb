// prefix_barriers.h -- the mbarriers of the shared-prefix attention kernel:
// which barrier, and which parity of it, stands for an event of tile j.
// Plain C++, so that a host program can walk through the kernel's roles.
//
// A wait by parity is safe only while its barrier cannot run a whole phase
// ahead of the waiter: the phase after the awaited one must need something
// that the waiter does later.  That holds for each event and its waiters:
//   keys(j)      the MMA thread; keys(j + 2) needs scores(j), which it issues
//   factors(j)   the softmax warps; factors(j + 4) needs scores(j + 2), whose
//                product is issued behind weights(j), which they give.  Keys
//                would not do for them: keys(j + 2) needs only scores(j), the
//                MMA thread's, and may pass a softmax warp that is late.
//   values(j)    the MMA thread; values(j + 2) needs output(j), which it issues
//   scores(j)    softmax and keys' warps; scores(j + 2) needs weights(j) and
//                keys(j + 2)
//   weights(j)   the MMA thread; weights(j + 2) needs scores(j + 2)
//   output(j)    softmax and values' warps, MMA thread; output(j + 2) needs
//                weights(j + 2) and values(j + 2)
#pragma once

#include <cstdint>

namespace dg {
namespace prefix {

constexpr int kFactorSlots = 4;   // tiles whose per-token factors are held at once

enum Barrier : int {
    kQueries = 0,
    kKeys = 1,        // two: a stage of codes is in place
    kValues = 3,      // two
    kScores = 5,      // two: the first product is done
    kWeights = 7,     // two: weights are in place
    kOutput = 9,      // two: the second product is done
    kDrain = 11,
    kFactors = 12,    // one per slot
    kBarriers = kFactors + kFactorSlots
};

struct Phase {
    int barrier;
    uint32_t parity;
};

constexpr Phase of_stream(int first, int j) {   // even and odd tiles: two streams
    return Phase{first + (j & 1), static_cast<uint32_t>(j >> 1) & 1u};
}
constexpr Phase keys(int j) { return of_stream(kKeys, j); }
constexpr Phase values(int j) { return of_stream(kValues, j); }
constexpr Phase scores(int j) { return of_stream(kScores, j); }
constexpr Phase weights(int j) { return of_stream(kWeights, j); }
constexpr Phase output(int j) { return of_stream(kOutput, j); }
constexpr int factor_slot(int j) { return j % kFactorSlots; }
constexpr Phase factors(int j) {
    return Phase{kFactors + factor_slot(j), static_cast<uint32_t>(j / kFactorSlots) & 1u};
}

}  // namespace prefix
}  // namespace dg
