// The check of adapter descriptors that every kernel reading them shares.
#pragma once
#include "common.hpp"

namespace lora {

// Whether an adapter's factors A [rank][d_in] and B [d_out][rank] lie inside packs of so
// many elements.  The offsets come from device memory and may hold anything: they are
// compared with what the pack leaves, since a sum with an offset near 2^63 would wrap to
// a negative number and pass as small.
__host__ __device__ __forceinline__ bool desc_ok(const lora_adapter_desc& d, int max_rank,
                                                 int64_t d_in, int64_t d_out, int64_t a_elems,
                                                 int64_t b_elems) {
  const int64_t r = d.rank;
  return r >= 8 && r <= 64 && (r % 8) == 0 && r <= max_rank && d.a_off >= 0 && d.b_off >= 0 &&
         (d.a_off % 8) == 0 && (d.b_off % 8) == 0 && d.a_off <= a_elems - r * d_in &&
         d.b_off <= b_elems - r * d_out;
}

}  // namespace lora
