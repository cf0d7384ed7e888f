// The state of a warp's ring of tile slots, in one word: plain arithmetic, which a test also runs on the host
// against a model of the barriers.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KV4_BOTH __host__ __device__ __forceinline__
#else
#define KV4_BOTH inline
#endif

namespace talker_k {

// A slot takes one copy at a time, and each copy completes one phase of the slot's barrier. A wait that runs
// out changes neither the slot's parity nor that its copy is in flight: the copy can still land there.
// From then on the ring is lost: what is in flight is waited for once more, and no slot is used again.
struct Kv4Ring {
    uint32_t bits = 0;   // slot i: its barrier's parity in bit i, a copy in flight in bit 8 + i; bit 16: lost

    KV4_BOTH uint32_t parity(int slot) const { return bits >> slot & 1u; }
    KV4_BOTH bool in_flight(int slot) const { return bits >> (8 + slot) & 1u; }
    KV4_BOTH bool lost() const { return bits >> 16 & 1u; }
    KV4_BOTH void issued(int slot) { bits |= 0x100u << slot; }
    KV4_BOTH void landed(int slot) { bits ^= 0x101u << slot; }
    KV4_BOTH void lose() { bits |= 1u << 16; }
};

}  // namespace talker_k
