// Random bits of the stochastic roundings, hashed from an element's index and
// two keys.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ob {

// A 32-bit word hashed from the quad's index and the first key, and more words
// from the word before and the second key.  The multipliers are digits of
// sqrt(5), sqrt(3) and the golden ratio; every input bit flips every output bit
// with probability 1/2 within the noise of 65536 quads, and no two bits of the
// four words correlate above it.
__device__ __forceinline__ uint32_t first_word(uint32_t quad, uint32_t key) {
  uint32_t h = quad ^ key;
  h = (h ^ (h >> 16)) * 0x3C6EF373u;
  h = (h ^ (h >> 15)) * 0xBB67AE85u;
  return h ^ (h >> 16);
}
__device__ __forceinline__ uint32_t next_word(uint32_t word, uint32_t key, uint32_t i) {
  const uint32_t h = (word ^ key) * 0x9E3779B9u + i;
  return h ^ (h >> 15);
}
// Quads past 2^32 take another key.
__device__ __forceinline__ uint32_t high_key(uint64_t quad, uint32_t key) {
  return key ^ ((uint32_t)(quad >> 32) * 0x9E3779B9u);
}
__device__ __forceinline__ uint32_t random16(uint32_t a, uint32_t b, int k) {
  const uint32_t w = k < 2 ? a : b;
  return k & 1 ? w >> 16 : w & 0xffffu;
}

// Two keys from a seed and a count, mixed in 64 bits; the multipliers are
// digits of the square roots of 2, 3 and 5.
struct Keys {
  uint32_t k0, k1;
};
__device__ __forceinline__ uint64_t mix64(uint64_t z, uint64_t mul) {
  z ^= z >> 31;
  return z * mul;
}
__device__ __forceinline__ Keys keys_of(uint64_t seed, uint64_t count) {
  uint64_t z = seed * 0x6A09E667F3BCC909ull + count * 0xBB67AE8584CAA73Bull;
  z = mix64(z, 0x3C6EF372FE94F82Bull);
  z = mix64(z, 0x6A09E667F3BCC909ull);
  z ^= z >> 32;
  return {(uint32_t)z, (uint32_t)(z >> 32)};
}

}  // namespace ob
