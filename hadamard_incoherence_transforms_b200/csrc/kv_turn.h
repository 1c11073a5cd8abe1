// Rotary angles as fractions of a turn, in units of 2^-64 (host and device).
#pragma once
#include <stdint.h>

namespace hit {

#ifdef __CUDACC__
__host__ __device__ __forceinline__
#else
inline
#endif
// The upper 32 bits of position times frequency modulo one turn, as a signed
// number: the angle in [-1/2, 1/2) turns.  The product wraps, on unsigned numbers.
int32_t kv_fraction(int32_t pos, uint64_t turn) {
  return int32_t(uint32_t((uint64_t(int64_t(pos)) * turn) >> 32));
}

}  // namespace hit
