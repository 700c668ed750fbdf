// The products of one Newton-Schulz step over a group of matrices, as MFMA GEMMs on the fp16
// halves of the workspace (ns.h):
//   NS_GRAM    A = X X^T             tiles on and below the diagonal, each stored twice
//   NS_POLY    B = b A + c A A       likewise (A is symmetric: A A = A A^T)
//   NS_UPDATE  X <- a X + B X        into the other X buffer; the last step writes the caller's
//                                    output or updates the caller's parameter instead
//
// Rounding. The fast products multiply the hi halves (fp16, 2^-12 of each factor) with fp32
// accumulation; a X is formed from hi + lo in fp32 and X is stored as hi + lo again. Carrying X
// in 22 bits is what keeps the fast form usable: the rounding of a factor of B X or X X^T only
// reaches directions the update already has, while a rounded X itself would put noise into the
// directions it lacks, which every step then multiplies by a = 3.4 (an update of rank 112 came
// out 3% off, against 0.06%). The accurate products use both halves of every factor
// (hi hi + hi lo + lo hi): the result agrees with fp32 products.
#include "ns.h"

namespace psgd {
namespace {

constexpr int GM_THREADS = 256;

typedef short i16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i16x4 lds_read_tr16(const uint16_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)(p));
}

// K-outer rows (LDS row = one k): the pair of 16-byte units a transposing read touches in each of
// the rows k = 8 g + t (g = 0, 1; t = 0..3) must land on 8 distinct 32-byte groups of the banks.
template <int T> __device__ __forceinline__ int swz_outer(int k, int q) {
  if constexpr (T == 64) return q ^ (2 * (((k >> 1) & 1) | (((k >> 3) & 1) << 1)));   // 128-byte rows
  else return q ^ (2 * ((k & 3) | (((k >> 3) & 1) << 2)));                            // 256-byte rows
}
// K-contiguous rows are 128 bytes: 8 consecutive rows put one logical unit on 8 distinct groups.
__device__ __forceinline__ int swz_inner(int row, int q) { return q ^ (row & 7); }

__device__ __forceinline__ float h2f(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
__device__ __forceinline__ f32x4 h2f4(u32x2 v) { return __builtin_convertvector(__builtin_bit_cast(f16x4, v), f32x4); }
__device__ __forceinline__ u32x2 f2h4(f32x4 v) { return __builtin_bit_cast(u32x2, __builtin_convertvector(v, f16x4)); }

// hi + lo of four values stored at h and (LO) l
template <bool LO> __device__ __forceinline__ void store_split(f32x4 v, GLOBAL uint16_t* h, GLOBAL uint16_t* l) {
  const u32x2 hi = f2h4(v);
  *gcast<u32x2>(h) = hi;
  if constexpr (LO) *gcast<u32x2>(l) = f2h4(v - h2f4(hi));
}
template <bool LO> __device__ __forceinline__ void store_split1(float v, GLOBAL uint16_t* h, GLOBAL uint16_t* l) {
  const uint16_t hi = f16_bits((_Float16)v);
  *h = hi;
  if constexpr (LO) *l = f16_bits((_Float16)(v - h2f(hi)));
}

template <int OT> __device__ __forceinline__ float out_load(const void* p, int64_t i) {
  if constexpr (OT == G_F32) return gbl(static_cast<const float*>(p))[i];
  else if constexpr (OT == G_F16) return h2f(gbl(static_cast<const uint16_t*>(p))[i]);
  else return __builtin_bit_cast(float, (uint32_t)gbl(static_cast<const uint16_t*>(p))[i] << 16);
}
template <int OT> __device__ __forceinline__ void out_store(void* p, int64_t i, float v) {
  if constexpr (OT == G_F32) gbl(static_cast<float*>(p))[i] = v;
  else if constexpr (OT == G_F16) gbl(static_cast<uint16_t*>(p))[i] = f16_bits((_Float16)v);
  else gbl(static_cast<uint16_t*>(p))[i] = bf16_bits((__bf16)v);
}

// ST: stage. T: C tile side (four waves of T/2 x T/2). ACC: accurate products. OT: 0, or the
// output type of the last update. MFMA layout: operand P gives the rows i of a C tile, Q the
// columns j; a lane holds C[4 g .. 4 g + 3][c], four consecutive i. For the update i runs along
// l and j along s, so those four are consecutive in memory.
template <int ST, int T, bool ACC, int OT>
__global__ __launch_bounds__(GM_THREADS, 2)
void k_ns_gemm(const NsMat* __restrict__ mats, const Work* __restrict__ work, int step, NsArgs na)
{
  if (na.skip && *na.skip != 0) return;
  const Work wi = work[xcd_remap(blockIdx.x, gridDim.x)];
  if (wi.mat < 0) return;
  const NsMat& d = mats[wi.mat];
  constexpr bool OUTER = ST == NS_UPDATE;      // P is read K-outer
  constexpr int KS = ACC ? 32 : 64;            // k per stage: 128 bytes per row either way
  constexpr int UN = T / 32;                   // 16-byte units per thread and operand
  constexpr int WT = T / 32;                   // 16-row tiles per wave and side
  const int cur = step & 1;
  const int i0 = wi.a, j0 = wi.b;
  const int lane = threadIdx.x & (kWave - 1), wv = threadIdx.x / kWave;
  const int wm = wv & 1, wn = wv >> 1;
  const int c = lane & 15, g = lane >> 4;

  const GLOBAL uint16_t *ph, *pl, *qh, *ql;
  int64_t ldp, ldq;
  int K;
  if constexpr (ST == NS_GRAM) {
    ph = qh = gbl(d.xh[cur]); pl = ql = gbl(d.xl[cur]); ldp = ldq = d.lp; K = d.l;
  } else if constexpr (ST == NS_POLY) {
    ph = qh = gbl(d.ah); pl = ql = gbl(d.al); ldp = ldq = d.sp; K = d.s;
  } else {
    ph = gbl(d.xh[cur]); pl = gbl(d.xl[cur]); ldp = d.lp;
    qh = gbl(d.bh); ql = gbl(d.bl); ldq = d.sp; K = d.s;
  }
  const int nsteps = (K + KS - 1) / KS;        // the padding up to a whole tile holds zeros

  __shared__ __attribute__((aligned(16))) uint16_t ldsP[2][T * 64], ldsQ[2][T * 64];
  const GLOBAL uint16_t* psrc[UN];
  const GLOBAL uint16_t* qsrc[UN];
#pragma unroll
  for (int j = 0; j < UN; ++j) {
    const int e = threadIdx.x + GM_THREADS * j;
    const int row = e >> 3, q = swz_inner(row, e & 7);
    const GLOBAL uint16_t* qb = ACC && q >= 4 ? ql : qh;
    qsrc[j] = qb + (int64_t)(j0 + row) * ldq + 8 * (ACC ? (q & 3) : q);
    if constexpr (OUTER) {
      const int k = e / (T / 8), u = swz_outer<T>(k, e % (T / 8));
      const GLOBAL uint16_t* pb = ACC && k >= 32 ? pl : ph;
      psrc[j] = pb + (int64_t)(ACC ? (k & 31) : k) * ldp + i0 + 8 * u;
    } else {
      const GLOBAL uint16_t* pb = ACC && q >= 4 ? pl : ph;
      psrc[j] = pb + (int64_t)(i0 + row) * ldp + 8 * (ACC ? (q & 3) : q);
    }
  }
  u32x4 rp[UN], rq[UN];
  auto load_stage = [&](int ks) {
    const int64_t kp = OUTER ? (int64_t)ks * KS * ldp : (int64_t)ks * KS, kq = (int64_t)ks * KS;
#pragma unroll
    for (int j = 0; j < UN; ++j) {
      rp[j] = *gcast<u32x4>(psrc[j] + kp);
      rq[j] = *gcast<u32x4>(qsrc[j] + kq);
    }
  };
  auto store_stage = [&](int buf) {
#pragma unroll
    for (int j = 0; j < UN; ++j) {
      const int e = threadIdx.x + GM_THREADS * j;
      *reinterpret_cast<u32x4*>(&ldsP[buf][8 * e]) = rp[j];
      *reinterpret_cast<u32x4*>(&ldsQ[buf][8 * e]) = rq[j];
    }
  };

  f32x4 acc[WT][WT];
#pragma unroll
  for (int a = 0; a < WT; ++a)
#pragma unroll
    for (int b = 0; b < WT; ++b) acc[a][b] = f32x4{0, 0, 0, 0};

  // fragment h (k half of a fast stage; 0 hi, 1 lo of an accurate one)
  auto frag_inner = [&](const uint16_t* l, int row, int h) {
    return *reinterpret_cast<const f16x8*>(&l[row * 64 + 8 * swz_inner(row, 4 * h + g)]);
  };
  auto frag_outer = [&](const uint16_t* l, int col, int h) {
    const int k = 32 * h + 8 * g + (c >> 2), q = col / 8 + ((c & 3) >> 1);
    const uint16_t* p = &l[k * T + 8 * swz_outer<T>(k, q) + 4 * (c & 1)];
    const i16x4 x = lds_read_tr16(p), y = lds_read_tr16(p + 4 * T);
    return __builtin_bit_cast(f16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto compute = [&](int buf) {
    f16x8 q[2][WT];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = 0; b < WT; ++b) q[h][b] = frag_inner(ldsQ[buf], wn * (T / 2) + 16 * b + c, h);
#pragma unroll
    for (int a = 0; a < WT; ++a) {
      f16x8 p[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = wm * (T / 2) + 16 * a;
        if constexpr (OUTER) p[h] = frag_outer(ldsP[buf], r, h);
        else p[h] = frag_inner(ldsP[buf], r + c, h);
      }
#pragma unroll
      for (int b = 0; b < WT; ++b) {
        acc[a][b] = mfma_f16(p[0], q[0][b], acc[a][b]);
        if constexpr (ACC) {
          acc[a][b] = mfma_f16(p[0], q[1][b], acc[a][b]);
          acc[a][b] = mfma_f16(p[1], q[0][b], acc[a][b]);
        } else {
          acc[a][b] = mfma_f16(p[1], q[1][b], acc[a][b]);
        }
      }
    }
  };

  load_stage(0);
  store_stage(0);
  __syncthreads();
  for (int ks = 0; ks < nsteps; ++ks) {
    if (ks + 1 < nsteps) load_stage(ks + 1);
    compute(ks & 1);
    if (ks + 1 < nsteps) store_stage((ks + 1) & 1);
    __syncthreads();
  }

  constexpr float kProd = ST == NS_GRAM ? kNsScaleA / (kNsScaleX * kNsScaleX)
                        : ST == NS_POLY ? kNsScaleB / (kNsScaleA * kNsScaleA)
                                        : 1.0f / kNsScaleB;
#pragma unroll
  for (int a = 0; a < WT; ++a)
#pragma unroll
    for (int b = 0; b < WT; ++b) {
      const int i = i0 + wm * (T / 2) + 16 * a + 4 * g, j = j0 + wn * (T / 2) + 16 * b + c;
      f32x4 v = kProd * acc[a][b];
      if constexpr (ST != NS_UPDATE) {
        // C[i..i+3][j]; rows and columns past s are zero
        const int64_t ji = (int64_t)j * d.sp + i;
        if constexpr (ST == NS_POLY) {
          f32x4 av = h2f4(*gcast<u32x2>(gbl(d.ah) + ji));
          if constexpr (ACC) av += h2f4(*gcast<u32x2>(gbl(d.al) + ji));
          v = na.c * v + (na.b * kNsScaleB / kNsScaleA) * av;
        }
        GLOBAL uint16_t* oh = gbl(ST == NS_GRAM ? d.ah : d.bh);
        GLOBAL uint16_t* ol = gbl(ST == NS_GRAM ? d.al : d.bl);
#pragma unroll
        for (int t = 0; t < 4; ++t) if (i + t >= d.s || j >= d.s) v[t] = 0.0f;
        store_split<ACC>(v, oh + ji, ol + ji);
        if (i0 != j0) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int64_t ij = (int64_t)(i + t) * d.sp + j;
            store_split1<ACC>(v[t], oh + ij, ol + ij);
          }
        }
      } else {
        // X[j][i..i+3]
        const int64_t ji = (int64_t)j * d.lp + i;
        v += na.a * (h2f4(*gcast<u32x2>(gbl(d.xh[cur]) + ji)) + h2f4(*gcast<u32x2>(gbl(d.xl[cur]) + ji)));
        if constexpr (OT == 0) {
#pragma unroll
          for (int t = 0; t < 4; ++t) if (i + t >= d.l || j >= d.s) v[t] = 0.0f;
          store_split<true>(v, gbl(d.xh[cur ^ 1]) + ji, gbl(d.xl[cur ^ 1]) + ji);
        } else {
          v *= 1.0f / kNsScaleX;
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            if (i + t >= d.l || j >= d.s) continue;
            const int64_t o = d.flip ? (int64_t)(i + t) * d.ld_out + j : (int64_t)j * d.ld_out + i + t;
            float x = v[t];
            if (na.muon) {
              const float th = out_load<OT>(d.out, o);
              x = th - na.lr * (d.factor * x + na.weight_decay * th);
            }
            out_store<OT>(d.out, o, x);
          }
        }
      }
    }
}

template <int ST, int T, bool ACC, int OT>
void go(const NsMat* mats, const Work* work, int n_work, int step, const NsArgs& a, hipStream_t s) {
  k_ns_gemm<ST, T, ACC, OT><<<dim3(n_work), dim3(GM_THREADS), 0, s>>>(mats, work, step, a);
}
template <int T, bool ACC>
hipError_t pick(NsStage st, int ot, bool last, const NsMat* mats, const Work* work, int n_work, int step,
                const NsArgs& a, hipStream_t s) {
  if (st == NS_GRAM) go<NS_GRAM, T, ACC, 0>(mats, work, n_work, step, a, s);
  else if (st == NS_POLY) go<NS_POLY, T, ACC, 0>(mats, work, n_work, step, a, s);
  else if (!last) go<NS_UPDATE, T, ACC, 0>(mats, work, n_work, step, a, s);
  else if (ot == G_F32) go<NS_UPDATE, T, ACC, G_F32>(mats, work, n_work, step, a, s);
  else if (ot == G_F16) go<NS_UPDATE, T, ACC, G_F16>(mats, work, n_work, step, a, s);
  else if (ot == G_BF16) go<NS_UPDATE, T, ACC, G_BF16>(mats, work, n_work, step, a, s);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ns_gemm(NsStage st, int tile, bool accurate, int ot, bool last, const NsMat* mats,
                          const Work* work, int n_work, int step, const NsArgs& a, hipStream_t s) {
  if (tile == 128)
    return accurate ? pick<128, true>(st, ot, last, mats, work, n_work, step, a, s)
                    : pick<128, false>(st, ot, last, mats, work, n_work, step, a, s);
  return accurate ? pick<64, true>(st, ot, last, mats, work, n_work, step, a, s)
                  : pick<64, false>(st, ot, last, mats, work, n_work, step, a, s);
}

}  // namespace psgd
