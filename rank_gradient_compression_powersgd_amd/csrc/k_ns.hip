// The two streaming kernels at the start of a Newton-Schulz call: the Frobenius norm of every
// update (with Muon's momentum), and X0 = U / max(||U||_F, eps) split into fp16 halves.
//
//   momentum:  mom <- mu mom + c g,  U = c g + mu mom (Nesterov) or mom;   without it U = in
//   norm:      fp64 sums of u^2 over parts of whole rows, added in part order by every workgroup
//              of the second kernel (the same order each time: bit-reproducible)
//   X0:        hi + lo of 2^14 u / ||U||, written s x l (transposed through LDS when m > n)
//
// Both are bound by HBM: fp32 Muon reads 8 and writes 4 bytes per element, then reads 8 and
// writes 4. A second pass over U is what the norm costs: no scale is known before the whole
// matrix has been read. Four resblock shards (9.4e7 elements): 208 us and 246 us, 5.4 and 4.6 TB/s.
#include "ns.h"

namespace psgd {
namespace {

constexpr int kThreads = 256;
constexpr int BATCH = 4;                  // vectors a thread loads together
constexpr int XT = 64;                    // X0 tile: XT x XT elements

template <int IT> __device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (IT == G_F32) return gbl(static_cast<const float*>(p))[i];
  else if constexpr (IT == G_F16) return (float)__builtin_bit_cast(_Float16, gbl(static_cast<const uint16_t*>(p))[i]);
  else return __builtin_bit_cast(float, (uint32_t)gbl(static_cast<const uint16_t*>(p))[i] << 16);
}
// four consecutive elements; the address is a multiple of their size (vec4_ok)
template <int IT> __device__ __forceinline__ f32x4 load4(const void* p, int64_t i) {
  if constexpr (IT == G_F32) return *gcast<f32x4>(gbl(static_cast<const float*>(p)) + i);
  else return GradIO<IT>::load4(gcast<char>(gbl(static_cast<const uint16_t*>(p)) + i));
}
// Muon's matrices always qualify: a compression plan's n is a multiple of 8, the pitch of its
// gradients one of 4, and gradients and momentum are 16-byte aligned.
template <int IT> __device__ __forceinline__ bool vec4_ok(const NsMat& d) {
  constexpr uintptr_t mask = IT == G_F32 ? 15 : 7;
  return ((d.n | (int)(d.ld_in & 3)) & 3) == 0 && (reinterpret_cast<uintptr_t>(d.in) & mask) == 0;
}

template <int IT>
__global__ __launch_bounds__(kThreads)
void k_ns_norm(const NsMat* __restrict__ mats, const Work* __restrict__ work, NsArgs a)
{
  if (*a.skip != 0) return;
  const Work wi = work[blockIdx.x];
  const NsMat& d = mats[wi.mat];
  const int n = d.n, r0 = wi.a, rows = min(d.part_rows, d.m - r0);
  const float clip = a.norm ? a.norm[1] : 1.0f;
  double acc = 0.0;
  // a part holds fewer than 2^32 elements (a matrix that fits the memory has at most 1024 parts)
  if (vec4_ok<IT>(d)) {
    const uint32_t n4 = (uint32_t)n >> 2, total = (uint32_t)rows * n4;
    for (uint32_t e0 = threadIdx.x; e0 < total; e0 += BATCH * kThreads) {
      f32x4 u[BATCH], mo[BATCH];
      int64_t at[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {        // past the end the last element again, not counted
        const uint32_t e = min(e0 + k * kThreads, total - 1), r = e / n4, col = (e - r * n4) << 2;
        u[k] = load4<IT>(d.in, (int64_t)(r0 + (int)r) * d.ld_in + col);
        at[k] = (int64_t)(r0 + (int)r) * n + col;
        if (a.muon) mo[k] = *gcast<f32x4>(gbl(d.mom) + at[k]);
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        if (e0 + k * kThreads >= total) break;
        f32x4 x = u[k];
        if (a.muon) {
          const f32x4 g = clip * x, m1 = a.mu * mo[k] + g;
          *gcast<f32x4>(gbl(d.mom) + at[k]) = m1;
          x = a.nesterov ? g + a.mu * m1 : m1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc += (double)x[i] * (double)x[i];
      }
    }
  } else {
    const uint32_t total = (uint32_t)rows * (uint32_t)n;
    for (uint32_t e0 = threadIdx.x; e0 < total; e0 += 2 * BATCH * kThreads) {
      float u[2 * BATCH];
#pragma unroll
      for (int k = 0; k < 2 * BATCH; ++k) {
        const uint32_t e = min(e0 + k * kThreads, total - 1), r = e / (uint32_t)n, col = e - r * (uint32_t)n;
        u[k] = load1<IT>(d.in, (int64_t)(r0 + (int)r) * d.ld_in + col);
      }
      __builtin_amdgcn_sched_barrier(0);       // or the loads sink to their uses (6.6 us become 10.3)
#pragma unroll
      for (int k = 0; k < 2 * BATCH; ++k) {
        if (e0 + k * kThreads >= total) break;
        acc += (double)u[k] * (double)u[k];
      }
    }
  }
  __shared__ double red[kThreads];
  red[threadIdx.x] = acc;
  __syncthreads();
  for (int w = kThreads / 2; w > 0; w >>= 1) {
    if ((int)threadIdx.x < w) red[threadIdx.x] += red[threadIdx.x + w];
    __syncthreads();
  }
  if (threadIdx.x == 0) gbl(d.partial)[wi.b] = red[0];
}

// hi + lo of x, both fp16: |x - hi - lo| <= 2^-22 |x| while lo is normal
__device__ __forceinline__ void split16(float x, uint16_t& hi, uint16_t& lo) {
  const _Float16 h = (_Float16)x;
  hi = f16_bits(h);
  lo = f16_bits((_Float16)(x - (float)h));
}

// One XT x XT tile of X (rows i0.., columns j0.. of the s x l matrix). Elements past s x l are
// written as zeros, so that what a call leaves in the padding never reaches the next.
template <int IT>
__global__ __launch_bounds__(kThreads)
void k_ns_x0(const NsMat* __restrict__ mats, const Work* __restrict__ work, NsArgs a)
{
  if (*a.skip != 0) return;
  const Work wi = work[blockIdx.x];
  const NsMat& d = mats[wi.mat];
  __shared__ double red[kThreads];
  __shared__ float tile[XT][XT + 1];
  const float clip = a.norm ? a.norm[1] : 1.0f;
  const int i0 = wi.a, j0 = wi.b;
  // rows and columns of the update under this tile, loaded before the norm is added up
  const int r0 = d.flip ? j0 : i0, c0 = d.flip ? i0 : j0;
  const bool v4 = vec4_ok<IT>(d);
  constexpr int PER = XT * XT / 4 / kThreads;
  f32x4 u[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int e = threadIdx.x + k * kThreads, row = r0 + (e >> 4), col = c0 + ((e & 15) << 2);
    u[k] = f32x4{0, 0, 0, 0};
    if (row < d.m && col < d.n) {
      if (v4) {
        u[k] = load4<IT>(d.in, (int64_t)row * d.ld_in + col);
        if (a.muon) {
          const f32x4 mo = *gcast<f32x4>(gbl(d.mom) + (int64_t)row * d.n + col);
          u[k] = a.nesterov ? clip * u[k] + a.mu * mo : mo;
        }
      } else {
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (col + t < d.n) u[k][t] = load1<IT>(d.in, (int64_t)row * d.ld_in + col + t);
      }
    }
  }
  double acc = 0.0;
  for (int i = threadIdx.x; i < d.parts; i += kThreads) acc += gbl(d.partial)[i];
  red[threadIdx.x] = acc;
  __syncthreads();
  for (int w = kThreads / 2; w > 0; w >>= 1) {
    if ((int)threadIdx.x < w) red[threadIdx.x] += red[threadIdx.x + w];
    __syncthreads();
  }
  const double norm = sqrt(red[0]);
  // a norm that is NaN stays NaN (max would drop it)
  const double inv = (double)kNsScaleX / (norm < a.eps ? a.eps : norm);
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int e = threadIdx.x + k * kThreads, r = e >> 4, c = (e & 15) << 2;
#pragma unroll
    for (int t = 0; t < 4; ++t) tile[r][c + t] = (float)((double)u[k][t] * inv);
  }
  __syncthreads();
  GLOBAL uint16_t* xh = gbl(d.xh[0]);
  GLOBAL uint16_t* xl = gbl(d.xl[0]);
  for (int e = threadIdx.x; e < XT * XT / 4; e += kThreads) {
    const int i = e >> 4, j = (e & 15) << 2;
    uint16_t h[4], l[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      // past s x l the update was read as 0 (times a NaN norm it would not stay 0)
      const bool in = i0 + i < d.s && j0 + j + t < d.l;
      split16(in ? (d.flip ? tile[j + t][i] : tile[i][j + t]) : 0.0f, h[t], l[t]);
    }
    const int64_t off = ((int64_t)((j0 + j) >> 5) * d.sp + i0 + i) * 32 + (j & 31);      // ns.h: panels of 32 columns
    *gcast<u32x2>(xh + off) = u32x2{(uint32_t)h[0] | ((uint32_t)h[1] << 16), (uint32_t)h[2] | ((uint32_t)h[3] << 16)};
    *gcast<u32x2>(xl + off) = u32x2{(uint32_t)l[0] | ((uint32_t)l[1] << 16), (uint32_t)l[2] | ((uint32_t)l[3] << 16)};
  }
}

}  // namespace

int ns_x0_tile() { return XT; }

hipError_t launch_ns_norm(int it, const NsMat* mats, const Work* work, int n_work, const NsArgs& a, hipStream_t s) {
  const dim3 grid(n_work), block(kThreads);
  switch (it) {
    case G_F16: k_ns_norm<G_F16><<<grid, block, 0, s>>>(mats, work, a); break;
    case G_BF16: k_ns_norm<G_BF16><<<grid, block, 0, s>>>(mats, work, a); break;
    case G_F32: k_ns_norm<G_F32><<<grid, block, 0, s>>>(mats, work, a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_ns_x0(int it, const NsMat* mats, const Work* work, int n_work, const NsArgs& a, hipStream_t s) {
  const dim3 grid(n_work), block(kThreads);
  switch (it) {
    case G_F16: k_ns_x0<G_F16><<<grid, block, 0, s>>>(mats, work, a); break;
    case G_BF16: k_ns_x0<G_BF16><<<grid, block, 0, s>>>(mats, work, a); break;
    case G_F32: k_ns_x0<G_F32><<<grid, block, 0, s>>>(mats, work, a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace psgd
