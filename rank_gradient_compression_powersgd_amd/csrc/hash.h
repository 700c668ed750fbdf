// Random bits of stochastic rounding: a hash of the caller's seed, the step, a tensor and an element's
// index, so that the same call gives the same bits wherever an element is computed. Two rounds of
// xor-shift and multiplication by odd constants (the fractions of the square roots of 7, made odd,
// and of 3): flipping any input bit flips every output bit with probability 0.5 +- 0.005.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace psgd {

__host__ __device__ __forceinline__ uint32_t hash_mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0xA54FF53Bu;
  x = (x ^ (x >> 15)) * 0xBB67AE85u;
  return x ^ (x >> 16);
}
__host__ __device__ __forceinline__ uint32_t hash_key(uint64_t seed, uint32_t step, uint32_t tensor) {
  uint32_t k = hash_mix((uint32_t)seed ^ 0x9E3779B9u);
  k = hash_mix(k ^ (uint32_t)(seed >> 32));
  return hash_mix(hash_mix(step ^ k) ^ tensor);
}
// the part of an element's bits that the high half of its index decides
__host__ __device__ __forceinline__ uint32_t hash_high(uint32_t key, uint64_t index) {
  return hash_mix((uint32_t)(index >> 32) ^ key);
}
__host__ __device__ __forceinline__ uint32_t hash_bits(uint32_t high, uint32_t index) { return hash_mix(index ^ high); }
// 32 more bits out of an element's 32
__host__ __device__ __forceinline__ uint32_t hash_more(uint32_t r) {
  const uint32_t t = (r ^ (r >> 15)) * 0x9E3779B1u;
  return t ^ (t >> 16);
}

}  // namespace psgd
