// The places of a ring of shared memory tiles that K's and V's copies take in turn: use 2 i is the i-th tile of K, use
// 2 i + 1 the i-th of V.
//
// A stage's "full" barrier is waited for by one warp for K's uses and by others for V's.  A wait by parity cannot tell the
// phase before the last from the present one, so a waiter has to know that the phase before its own is complete, and it
// knows that of the phases that it has waited for.  With an even number of stages a stage holds K alone or V alone.  With
// an odd number it holds them by turns, and one barrier a stage would let the warp that waits for K pass while the V before
// it is still on its way: K and V then have barriers of their own, two a stage.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MHC_RING_FN __host__ __device__ __forceinline__
#else
#define MHC_RING_FN inline
#endif

namespace mhc {

template <int ST>
struct TileRing {
    static constexpr uint32_t kFull = ST % 2 == 0 ? ST : 2 * ST;   // "full" barriers; one "empty" barrier a stage
    static MHC_RING_FN uint32_t stage(uint32_t use) { return use % ST; }
    static MHC_RING_FN uint32_t full(uint32_t use) { return use % kFull; }
    static MHC_RING_FN uint32_t full_parity(uint32_t use) { return (use / kFull) & 1; }
    static MHC_RING_FN uint32_t empty_parity(uint32_t use) { return (use / ST) & 1; }   // of the release after this use
};

}  // namespace mhc
