// How a product's CTA waits for the operand copies that are still on their way
// when it winds down, as plain C++: ebin_gemm_tc.cuh follows it.
//
// Step j's copies land on slot j % stages; the slot's barrier takes one arrival
// with the bytes of both CTAs of a pair, made by the leader as it issues its
// copies, and the bytes of each copy.  A CTA issues j once the products of step j -
// stages are done, so of the steps issued at most the last `stages` are open.  The
// two CTAs of a pair may have stopped at different steps:
//   both issued j        its phase ends by itself
//   the peer alone       the leader's arrival is missing: it expects the peer's bytes
//   the leader alone     the peer's bytes never come: the leader counts them off
#pragma once

#ifdef __CUDACC__
#define EBIN_DRAIN_FN __host__ __device__ __forceinline__
#else
#define EBIN_DRAIN_FN inline
#endif

namespace ebin {

enum TcDrain : int { TC_DRAIN_WAIT = 0, TC_DRAIN_EXPECT = 1, TC_DRAIN_COUNT_OFF = 2 };

// Steps issued by either CTA (a single CTA is its own peer), and the first that may be open.
EBIN_DRAIN_FN int tc_drain_end(int own, int peer) { return own > peer ? own : peer; }
EBIN_DRAIN_FN int tc_drain_first(int own, int peer, int stages) {
    const int end = tc_drain_end(own, peer);
    return end > stages ? end - stages : 0;
}
// What the leader does before it waits for step j's phase, of parity (j / stages) & 1.
EBIN_DRAIN_FN TcDrain tc_drain_step(int j, int own, int peer) {
    return j >= own ? TC_DRAIN_EXPECT : j >= peer ? TC_DRAIN_COUNT_OFF : TC_DRAIN_WAIT;
}

}  // namespace ebin
