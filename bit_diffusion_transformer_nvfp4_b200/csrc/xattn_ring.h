// xattn_ring.h -- where the cross attention keeps its key and value tiles:
// plain arithmetic, for the kernel and for host programs that check it.
//
// A ring of `slots` tiles serves `rings` sequences of fills, a part of the
// slots each; a sequence is K0 V0 K1 V1 ...  A slot's barrier is waited for
// with the parity of the fill, which tells a fill only from the one before
// it: whoever waits for a fill must know that the slot's fill before it has
// landed.  Copies need not land in the order in which they were issued, so
// that holds only where the waiter has itself waited for that earlier fill:
// the streams of the split form, which take every second key tile, have a ring
// each (in one ring for both, a stream would have waited behind fills of the
// other), those of the persistent form wait for every tile and share one.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define W4A4_HD __host__ __device__ __forceinline__
#else
#define W4A4_HD inline
#endif

namespace w4a4 {

struct XRing {
  uint32_t first, slots;  // this sequence's slots

  W4A4_HD uint32_t slot(uint32_t fill) const { return first + fill % slots; }
  W4A4_HD uint32_t parity(uint32_t fill) const { return fill / slots & 1u; }
};

// The ring of sequence t of `rings`.
W4A4_HD XRing xattn_ring(uint32_t slots, uint32_t rings, uint32_t t) { return XRing{t * (slots / rings), slots / rings}; }

// The fills of a sequence's key tile k.
W4A4_HD uint32_t xattn_fill_k(uint32_t k) { return 2 * k; }
W4A4_HD uint32_t xattn_fill_v(uint32_t k) { return 2 * k + 1; }

}  // namespace w4a4
