// AdamW over a list of tensors: one pass over the gradients for their norm and the skip decision, one
// over everything for the update. Formulas as for the pass-through tensors (k_adam.hip), with parameters
// and gradients of any type and the moments in fp32 or in 8 bits.
//
// 8-bit moments. Groups of 64 elements share an exponent byte E, that of their largest magnitude (one
// more where it rounds up past 2). A code is a small float whose largest exponent field stands for E:
// first moment sign + 4 + 3 bits, second moment 5 + 3 bits without a sign, both with subnormals; so an
// element keeps 3 fraction bits down to 2^-14 (2^-30) of its group's largest and vanishes below 2^-18
// (never, for a second moment: it would make the quotient blow up). With the exponent field moved to
// the fp32's lowest binades, code and value are one shift and one ldexp apart, subnormals included.
//
// Rounding. A moving average of 8-bit numbers rounded to nearest stands still: (1 - b2) of the
// difference is far below half a step of 2^-4. Rounded up with the probability of the fraction cut
// off, its expectation moves as in fp32. The same holds for 16-bit parameters and small lr. Random bits
// are a hash of seed, step, tensor and element (hash.h).
//
// Bound: memory. A chunk's loads are all sent for before its first use, so a workgroup (4096 elements, 256
// threads) keeps 57 KB under way. 188.9 million elements (fp32 parameters, bf16 gradients, 8-bit moments, 14.06
// bytes each): 493 us in the median of 30 passes, 473 at best (5.4 and 5.6 TB/s); their norm 105 and 74 us, their
// moments' values 199 and 194 (5.7 TB/s). 23.6 million (bf16, fp32 gradients, 12.06 bytes): 57 to 65, 15 and 23 us.
// 0.76 million: 7, 3.6 and 3.3 us, and 2.1 for the norm's last sum, which is about what a launch takes here.
//
// The moments' arithmetic is rounded operation by operation (no fused multiply-add), so that codes do
// not depend on how the compiler contracts an expression.
#include "adamw.h"
#include "hash.h"

#pragma clang fp contract(off)

namespace psgd {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;                                  // consecutive elements of a lane
constexpr int kTurns = kAdamwChunk / (kThreads * kPer);  // of a workgroup over its chunk

// 4 elements at any element's alignment: the hardware takes vector accesses at element boundaries
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef _Float16 f16x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef __bf16 bf16x4_u __attribute__((ext_vector_type(4), aligned(2)));

typedef _Float16 f16x8_u __attribute__((ext_vector_type(8), aligned(2)));
typedef __bf16 bf16x8_u __attribute__((ext_vector_type(8), aligned(2)));

// wide: what 16 bytes hold
template <int T> struct Elem;
template <> struct Elem<G_F32> { typedef float one; typedef f32x4_u four; typedef f32x4_u wide; static constexpr int WIDE = 4; };
template <> struct Elem<G_F16> { typedef _Float16 one; typedef f16x4_u four; typedef f16x8_u wide; static constexpr int WIDE = 8; };
template <> struct Elem<G_BF16> { typedef __bf16 one; typedef bf16x4_u four; typedef bf16x8_u wide; static constexpr int WIDE = 8; };

template <int T> __device__ __forceinline__ f32x4 load_four(const void* p, int i) {
  const auto v = *gcast<typename Elem<T>::four>(gbl(static_cast<const typename Elem<T>::one*>(p)) + i);
  return __builtin_convertvector(v, f32x4);
}
// the first `left` of 4, zeros behind them
template <int T> __device__ __forceinline__ f32x4 load_some(const void* p, int i, int left) {
  f32x4 v{0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < left) v[j] = (float)gbl(static_cast<const typename Elem<T>::one*>(p))[i + j];
  return v;
}

__device__ __forceinline__ uint32_t bits_of(float v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ float float_of(uint32_t v) { return __builtin_bit_cast(float, v); }

template <int CTRL> __device__ __forceinline__ uint32_t row_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
  return o > v ? o : v;
}
// largest of 16 lanes (a group of 64 elements), in all of them
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = row_max<0xB1>(v);       // neighbours
  v = row_max<0x4E>(v);       // pairs of them
  v = row_max<0x141>(v);      // mirrored in 8
  return row_max<0x140>(v);   // mirrored in 16
}

template <bool SECOND> constexpr int kTop = SECOND ? 31 : 15;

// lost: what a group of byte 255 reads as. A step takes the largest value for its second moments, and 0 for the
// first ones (theirs would move a parameter by up to 1e19 lr against it): 64 parameters stand still till the second
// moments have decayed, instead of being NaN from the next step on.
constexpr float kLargest8 = 1.875f * 0x1p127f;
template <bool SECOND> __device__ __forceinline__ float decode8(uint32_t c, int e, float lost) {
  const float v = __builtin_amdgcn_ldexpf(float_of((SECOND ? c : c & 127) << 20), e - kTop<SECOND>);
  const float s = SECOND ? v : float_of(bits_of(v) | (c & 128) << 24);
  return e == 255 ? lost : s;
}
// r: 16 random bits (read where SR)
template <bool SECOND, bool SR> __device__ __forceinline__ uint32_t encode8(float v, int e, uint32_t r) {
  const uint32_t b = bits_of(__builtin_amdgcn_ldexpf(float_of(bits_of(v) & 0x7fffffffu), kTop<SECOND> - e));
  const uint32_t c = (b + (SR ? (r << 4 | 8u) : 0x7ffffu + (b >> 20 & 1))) >> 20;
  if (SECOND) return v > 0.0f && c == 0 ? 1u : c;
  return v < 0.0f ? c | 128u : c;
}
__device__ __forceinline__ int exponent8(const f32x4& v) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t b = bits_of(v[j]) & 0x7fffffffu;
    m = b > m ? b : m;
  }
  const uint32_t e = (max16(m) + 0xfffffu) >> 23;
  return (int)(e < 1 ? 1 : e > 255 ? 255 : e);
}

// r: 32 random bits (read where SR)
template <int T, bool SR> __device__ __forceinline__ typename Elem<T>::one to_param(float v, uint32_t r) {
  if constexpr (T == G_F32) return v;
  else if constexpr (!SR) return (typename Elem<T>::one)v;
  else if constexpr (T == G_BF16) {
    const uint32_t up = (bits_of(v) + (r >> 16)) >> 16;
    return __builtin_bit_cast(__bf16, (uint16_t)(nonfinite(v) ? bits_of(v) >> 16 | (v != v ? 64u : 0u) : up));
  } else {
    // 2^-112 moves fp16's exponents, subnormals included, to where fp32 has them
    const uint32_t b = bits_of(__builtin_amdgcn_ldexpf(float_of(bits_of(v) & 0x7fffffffu), -112)) + (r >> 19);
    const uint32_t c = b >> 13;
    const uint16_t h = (uint16_t)((c < 0x7c00u ? c : 0x7c00u) | (bits_of(v) >> 31 << 15));
    return nonfinite(v) ? (_Float16)v : __builtin_bit_cast(_Float16, h);
  }
}

// sqrt without the slow path's corrections: 1 unit in the last place, small arguments moved up first,
// because the instruction takes no subnormals
__device__ __forceinline__ float fast_sqrt(float v) {
  const bool tiny = v < 0x1p-96f;
  return __builtin_amdgcn_sqrtf(tiny ? v * 0x1p64f : v) * (tiny ? 0x1p-32f : 1.0f);
}

// Sum of a workgroup's values, in thread 0.
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int w = kWave / 2; w > 0; w >>= 1) v += __shfl_xor(v, w);
  if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// The skip decision, and on a step that is not skipped t, norm and clipping factor. A sum of squares in
// fp64 of fp32 values is finite exactly when they all are.
__device__ __forceinline__ void finish_norm(const AdamwNorm& a, double total) {
  const bool bad = !(total < __builtin_inf()) || (a.skip_in && *a.skip_in != 0);
  *a.skip = bad ? 1 : 0;
  if (bad) return;
  *a.step = *a.step + 1;
  const double norm = sqrt(total);
  a.norm[0] = (float)norm;
  a.norm[1] = (float)(a.max_norm > 0.0f && norm > (double)a.max_norm ? (double)a.max_norm / norm : 1.0);
}

// Sums of squares, one per workgroup. Adding them up takes a launch of its own (2 to 4 us): left to the
// workgroup that is done last, the fences that make the sums visible across XCDs cost each workgroup
// more (23.6 million elements: 15 -> 77 us).
template <int GT>
__global__ __launch_bounds__(kThreads)
void k_adamw_sqnorm(const AdamwChunk* __restrict__ chunks, int64_t n, double* __restrict__ partial) {
  typedef typename Elem<GT>::one one;
  typedef typename Elem<GT>::wide wide;
  constexpr int WIDE = Elem<GT>::WIDE, TURNS = kAdamwChunk / (kThreads * WIDE);
  __shared__ double red[kThreads / kWave];
  double acc = 0.0;
  int64_t b = blockIdx.x;
  const void* at = chunks[b].grad;                         // the grid is no larger than the list
  int len = chunks[b].n;
  while (b < n) {
    const GLOBAL one* g = gbl(static_cast<const one*>(at));
    const int left = len;
    wide v[TURNS];
    if (left == kAdamwChunk) {
#pragma unroll
      for (int u = 0; u < TURNS; ++u) v[u] = *gcast<wide>(g + (u * kThreads + threadIdx.x) * WIDE);
    } else {
#pragma unroll
      for (int u = 0; u < TURNS; ++u) {
        const int i = (u * kThreads + threadIdx.x) * WIDE;
        v[u] = wide(0);
#pragma unroll
        for (int j = 0; j < WIDE; ++j)
          if (i + j < left) v[u][j] = g[i + j];
      }
    }
    b += gridDim.x;
    if (b < n) {                                           // the next chunk's place, while this one arrives
      at = chunks[b].grad;
      len = chunks[b].n;
    }
#pragma unroll
    for (int u = 0; u < TURNS; ++u)
#pragma unroll
      for (int j = 0; j < WIDE; ++j) acc += (double)(float)v[u][j] * (double)(float)v[u][j];
  }
  const double sum = block_sum(acc, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__global__ __launch_bounds__(kThreads)
void k_adamw_finalize(const double* __restrict__ partial, int n, AdamwNorm a) {
  __shared__ double red[kThreads / kWave];
  double acc = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) acc += partial[i];
  const double total = block_sum(acc, red);
  if (threadIdx.x == 0) finish_norm(a, total);
}

// WHOLE: a chunk of kAdamwChunk elements, no bounds to look at (with them the loads wait for one another).
template <int PT, int GT, bool LOW, bool SR, bool WHOLE>
__device__ __forceinline__ void adamw_chunk(const AdamwChunk& c, const AdamwArgs& a) {
  constexpr bool whole = WHOLE;
  const float clip = a.norm ? a.norm[1] : 1.0f;
  const int step = *a.step;
  const int len = c.n, room = (len + kAdamwGroup - 1) / kAdamwGroup * kAdamwGroup;

  f32x4 p[kTurns], g[kTurns], m1[kTurns], m2[kTurns];
  uint32_t c1[kTurns], c2[kTurns], x1[kTurns], x2[kTurns];
#pragma unroll
  for (int u = 0; u < kTurns; ++u) {
    const int i = (u * kThreads + threadIdx.x) * kPer;
    if (whole || i + kPer <= len) {
      p[u] = load_four<PT>(c.param, i);
      g[u] = load_four<GT>(c.grad, i);
    } else {
      p[u] = load_some<PT>(c.param, i, len - i);
      g[u] = load_some<GT>(c.grad, i, len - i);
    }
    if (whole || i < room) {
      if constexpr (LOW) {
        c1[u] = *gcast<uint32_t>(gbl(static_cast<const uint8_t*>(c.m1)) + i);
        c2[u] = *gcast<uint32_t>(gbl(static_cast<const uint8_t*>(c.m2)) + i);
        x1[u] = gbl(c.e1)[i / kAdamwGroup];
        x2[u] = gbl(c.e2)[i / kAdamwGroup];
      } else {
        m1[u] = *gcast<f32x4>(gbl(static_cast<const float*>(c.m1)) + i);
        m2[u] = *gcast<f32x4>(gbl(static_cast<const float*>(c.m2)) + i);
      }
    }
  }
  const float rbc1 = (float)(1.0 / (1.0 - exp(step * a.log_beta1)));
  const float rbc2 = (float)(1.0 / (1.0 - exp(step * a.log_beta2)));
  const float omb1 = 1.0f - a.beta1, omb2 = 1.0f - a.beta2;
  const uint32_t high = SR ? hash_high(hash_key(a.seed, (uint32_t)step, (uint32_t)c.tensor), (uint64_t)c.first) : 0;

#pragma unroll
  for (int u = 0; u < kTurns; ++u) {
    const int i = (u * kThreads + threadIdx.x) * kPer;
    if (!whole && i >= room) continue;
    if (LOW && x2[u] == 255) x1[u] = 255;
    uint32_t r[kPer];
    typename Elem<PT>::one out[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      r[j] = SR ? hash_bits(high, (uint32_t)c.first + i + j) : 0;
      float a1, a2;
      if constexpr (LOW) {
        a1 = decode8<false>(c1[u] >> (8 * j) & 255, (int)x1[u], 0.0f);
        a2 = decode8<true>(c2[u] >> (8 * j) & 255, (int)x2[u], kLargest8);
      } else {
        a1 = m1[u][j];
        a2 = m2[u][j];
      }
      const float gc = g[u][j] * clip;
      a1 = a1 * a.beta1 + gc * omb1;
      a2 = a2 * a.beta2 + (gc * gc) * omb2;
      if (!whole && i + j >= len) a1 = a2 = 0.0f;
      // The reciprocal takes no subnormals: below them (eps is, and a2 0) a denominator counts as 2^-126, so that a
      // moment of 0 moves nothing. rbc1 comes last, since it could take a1 past fp32, where a2 is an infinity.
      const float den = fast_sqrt(a2 * rbc2) + a.eps;
      const float upd = a1 * __builtin_amdgcn_rcpf(den < 0x1p-126f ? 0x1p-126f : den) * rbc1;
      const float th = p[u][j];
      out[j] = to_param<PT, SR>(th - a.lr * (upd + a.weight_decay * th), SR && PT != G_F32 ? hash_more(r[j]) : 0);
      m1[u][j] = a1;
      m2[u][j] = a2;
    }
    typename Elem<PT>::one* po = static_cast<typename Elem<PT>::one*>(c.param);
    if (whole || i + kPer <= len) {
      *gcast<typename Elem<PT>::four>(gbl(po) + i) = typename Elem<PT>::four{out[0], out[1], out[2], out[3]};
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (i + j < len) gbl(po)[i + j] = out[j];
    }
    if constexpr (LOW) {
      const int n1 = exponent8(m1[u]), n2 = exponent8(m2[u]);
      uint32_t w1 = 0, w2 = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        w1 |= encode8<false, SR>(m1[u][j], n1, r[j] >> 16) << (8 * j);
        w2 |= encode8<true, SR>(m2[u][j], n2, r[j] & 0xffffu) << (8 * j);
      }
      *gcast<uint32_t>(gbl(static_cast<uint8_t*>(c.m1)) + i) = n1 == 255 ? 0 : w1;
      *gcast<uint32_t>(gbl(static_cast<uint8_t*>(c.m2)) + i) = n2 == 255 ? 0 : w2;
      if ((threadIdx.x & 15) == 0) {
        gbl(c.e1)[i / kAdamwGroup] = (uint8_t)n1;
        gbl(c.e2)[i / kAdamwGroup] = (uint8_t)n2;
      }
    } else {
      *gcast<f32x4>(gbl(static_cast<float*>(c.m1)) + i) = m1[u];
      *gcast<f32x4>(gbl(static_cast<float*>(c.m2)) + i) = m2[u];
    }
  }
}

template <int PT, int GT, bool LOW, bool SR>
__global__ __launch_bounds__(kThreads)
void k_adamw(const AdamwChunk* __restrict__ chunks, AdamwArgs a) {
  const AdamwChunk c = chunks[blockIdx.x];
  if (*a.skip != 0) return;
  if (c.n == kAdamwChunk) adamw_chunk<PT, GT, LOW, SR, true>(c, a);
  else adamw_chunk<PT, GT, LOW, SR, false>(c, a);
}

// Values of 8-bit moments, 16 bytes of them a lane and turn; blockIdx.y picks the moment. bf16 holds every
// value but those below its subnormals. Four turns, whose loads are all sent for first, where that leaves four
// workgroups a CU (188.9 million elements: 200 us, 5.7 TB/s; one turn of 8 bytes 256), one elsewhere
// (0.76 million: 3.0 us, with four 4.3).
template <int OT, int TURNS>
__global__ __launch_bounds__(kThreads)
void k_adamw_moments(const uint8_t* m1, const uint8_t* e1, const uint8_t* m2, const uint8_t* e2, int64_t n, void* out1, void* out2) {
  typedef typename Elem<OT>::one one;
  constexpr int WIDE = Elem<OT>::WIDE;
  const bool second = blockIdx.y != 0;
  const GLOBAL uint8_t* m = gbl(second ? m2 : m1);
  const GLOBAL uint8_t* ex = gbl(second ? e2 : e1);
  GLOBAL one* out = gbl(static_cast<one*>(second ? out2 : out1));
  const int64_t i0 = ((int64_t)blockIdx.x * TURNS * kThreads + threadIdx.x) * WIDE;
  const float nan = __builtin_nanf("");
  uint32_t w[TURNS][WIDE / 4];
  int e[TURNS];
#pragma unroll
  for (int u = 0; u < TURNS; ++u) {
    const int64_t i = i0 + u * kThreads * WIDE;            // codes reach to the end of its group
    e[u] = 0;
#pragma unroll
    for (int q = 0; q < WIDE / 4; ++q) w[u][q] = i < n ? gcast<uint32_t>(m + i)[q] : 0;
    if (i < n) e[u] = ex[i / kAdamwGroup];
  }
#pragma unroll
  for (int u = 0; u < TURNS; ++u) {
    const int64_t i = i0 + u * kThreads * WIDE;
    typename Elem<OT>::wide v;
#pragma unroll
    for (int j = 0; j < WIDE; ++j) {
      const uint32_t c = w[u][j / 4] >> (8 * (j % 4)) & 255;
      v[j] = (one)(second ? decode8<true>(c, e[u], nan) : decode8<false>(c, e[u], nan));
    }
    if (i + WIDE <= n) {
      *gcast<typename Elem<OT>::wide>(out + i) = v;
    } else {
      for (int j = 0; i + j < n; ++j) out[i + j] = v[j];
    }
  }
}

template <int PT, int GT>
void go(const AdamwChunk* chunks, int64_t n, bool low, bool sr, const AdamwArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)n), block(kThreads);
  if (low && sr) k_adamw<PT, GT, true, true><<<grid, block, 0, s>>>(chunks, a);
  else if (low) k_adamw<PT, GT, true, false><<<grid, block, 0, s>>>(chunks, a);
  else if (sr && PT != G_F32) k_adamw<PT, GT, false, PT != G_F32><<<grid, block, 0, s>>>(chunks, a);
  else k_adamw<PT, GT, false, false><<<grid, block, 0, s>>>(chunks, a);
}

}  // namespace

hipError_t launch_adamw_norm(const AdamwChunk* chunks, int64_t n, int gt, const AdamwNorm& a, hipStream_t s) {
  const int grid = (int)(n < kAdamwNormGrid ? n : kAdamwNormGrid);
  if (grid > 0) {
    if (gt == G_F32) k_adamw_sqnorm<G_F32><<<dim3(grid), dim3(kThreads), 0, s>>>(chunks, n, a.partial);
    else if (gt == G_F16) k_adamw_sqnorm<G_F16><<<dim3(grid), dim3(kThreads), 0, s>>>(chunks, n, a.partial);
    else k_adamw_sqnorm<G_BF16><<<dim3(grid), dim3(kThreads), 0, s>>>(chunks, n, a.partial);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  k_adamw_finalize<<<dim3(1), dim3(kThreads), 0, s>>>(a.partial, grid, a);
  return hipGetLastError();
}

hipError_t launch_adamw(const AdamwChunk* chunks, int64_t n, int pt, int gt, bool low, bool stochastic, const AdamwArgs& a, hipStream_t s) {
  if (n <= 0) return hipSuccess;
  if (pt == G_F32) {
    if (gt == G_F32) go<G_F32, G_F32>(chunks, n, low, stochastic, a, s);
    else if (gt == G_F16) go<G_F32, G_F16>(chunks, n, low, stochastic, a, s);
    else go<G_F32, G_BF16>(chunks, n, low, stochastic, a, s);
  } else if (pt == G_F16) {
    if (gt == G_F32) go<G_F16, G_F32>(chunks, n, low, stochastic, a, s);
    else if (gt == G_F16) go<G_F16, G_F16>(chunks, n, low, stochastic, a, s);
    else go<G_F16, G_BF16>(chunks, n, low, stochastic, a, s);
  } else {
    if (gt == G_F32) go<G_BF16, G_F32>(chunks, n, low, stochastic, a, s);
    else if (gt == G_F16) go<G_BF16, G_F16>(chunks, n, low, stochastic, a, s);
    else go<G_BF16, G_BF16>(chunks, n, low, stochastic, a, s);
  }
  return hipGetLastError();
}

hipError_t launch_adamw_moments(const uint8_t* m1, const uint8_t* e1, const uint8_t* m2, const uint8_t* e2, int64_t n, void* out1,
                                void* out2, int ot, hipStream_t s) {
  if (n <= 0) return hipSuccess;
  const int64_t per = kThreads * (ot == G_F32 ? Elem<G_F32>::WIDE : Elem<G_BF16>::WIDE), blocks = (n + per - 1) / per;
  const bool four = 2 * blocks / 4 >= 1024;
  const dim3 grid((unsigned)(four ? (blocks + 3) / 4 : blocks), 2), block(kThreads);
  if (ot == G_F32) {
    if (four) k_adamw_moments<G_F32, 4><<<grid, block, 0, s>>>(m1, e1, m2, e2, n, out1, out2);
    else k_adamw_moments<G_F32, 1><<<grid, block, 0, s>>>(m1, e1, m2, e2, n, out1, out2);
  } else {
    if (four) k_adamw_moments<G_BF16, 4><<<grid, block, 0, s>>>(m1, e1, m2, e2, n, out1, out2);
    else k_adamw_moments<G_BF16, 1><<<grid, block, 0, s>>>(m1, e1, m2, e2, n, out1, out2);
  }
  return hipGetLastError();
}

}  // namespace psgd
