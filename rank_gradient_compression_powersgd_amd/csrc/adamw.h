// Arguments of the many-tensor AdamW kernels (k_adamw.hip), filled by lowbit.hip.
#pragma once

#include "psgd_internal.h"

namespace psgd {

constexpr int kAdamwChunk = 4096;       // elements per workgroup; divides 2^32 (one hash_high a chunk)
constexpr int kAdamwGroup = 64;         // elements under one exponent
constexpr int kAdamwNormGrid = 2048;    // most workgroups of the norm, and its partial sums

// One chunk of one tensor, pointers at its first element: all that a workgroup needs in one load.
struct AdamwChunk {
  void* param; const void* grad;
  void* m1; void* m2;
  uint8_t* e1; uint8_t* e2;
  int64_t first;                        // index of the chunk's first element in its tensor
  int32_t n, tensor;
};
static_assert(sizeof(AdamwChunk) == 64, "one scalar load of 16 words");

struct AdamwArgs {
  float lr, beta1, beta2, eps, weight_decay;
  double log_beta1, log_beta2;
  const int32_t* skip;
  const int32_t* step;                  // t after this step's increment
  const float* norm;                    // norm, clipping factor; NULL: no clipping
  uint64_t seed;
};

struct AdamwNorm {
  double* partial;                      // sums of the workgroups
  float max_norm;
  const int32_t* skip_in;               // or NULL
  int32_t* skip; int32_t* step; float* norm;
};

hipError_t launch_adamw_norm(const AdamwChunk* chunks, int64_t n, int gt, const AdamwNorm& a, hipStream_t s);
hipError_t launch_adamw(const AdamwChunk* chunks, int64_t n, int pt, int gt, bool low, bool stochastic, const AdamwArgs& a, hipStream_t s);
hipError_t launch_adamw_moments(const uint8_t* m1, const uint8_t* e1, const uint8_t* m2, const uint8_t* e2, int64_t n, void* out1,
                                void* out2, int ot, hipStream_t s);

}  // namespace psgd
