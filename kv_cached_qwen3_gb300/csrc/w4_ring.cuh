// How the steps of a product with 4-bit weights pass through a ring of slots: plain arithmetic, which a test also runs on
// the host against a model of the barriers.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define W4_BOTH __host__ __device__ __forceinline__
#else
#define W4_BOTH inline
#endif

namespace talker_k {

constexpr int kW4Slots = 4;   // steps on their way or at hand

// Step i lies in slot i % kW4Slots. Its copies complete a phase of the slot's `full`; each warp that multiplies arrives once
// a step at the slot's `empty`, whose phase lets the copies of step i + kW4Slots begin.
W4_BOTH int w4_slot(int step) { return step % kW4Slots; }
W4_BOTH uint32_t w4_full_parity(int step) { return (step / kW4Slots) & 1; }
W4_BOTH uint32_t w4_empty_parity(int step) { return (step / kW4Slots - 1) & 1; }   // that step i >= kW4Slots waits for

// A warp's own part. `empty` counts arrivals, not warps: one that gave up a wait and went on arriving would stand in for
// one that still reads, and the slot would be written under it. So it arrives no more, the ring stops, every warp gives up in
// turn, and what none of them has read is not replaced.
struct W4Ring {
    bool lost = false;
    W4_BOTH bool waits() const { return !lost; }
    W4_BOTH void waited(bool arrived) { lost = !arrived; }
    W4_BOTH bool reads() const { return !lost; }
    W4_BOTH bool releases() const { return !lost; }
};

}  // namespace talker_k
