// Matrices to microscaled 4-bit elements (mx.h) and back.
//
// An element is sign + 2 exponent + 1 fraction bits: 0, 0.5, 1, 1.5, 2, 3, 4, 6; a block of 32 shares a
// power of two 2^(s - 127). To nearest even: the largest magnitude's exponent, one more from 1.75 on,
// less 2, so that magnitudes up to 7 meet the 6 and every element is off by at most half a step. By
// random bits: one more from just past 1.5, so that none exceeds 6 and the expectation is the value itself.
// A block with an infinity or NaN gets s = 255: NaN, all of it.
//
// Both directions in one pass. A lane holds 2 columns x 32 rows: a column's block is the lane's own, a
// row's block spans 16 lanes, whose maximum is four DPP steps. No LDS; the input is read once.
#include "hash.h"
#include "mx.h"

namespace psgd {
namespace {

constexpr int kThreads = 256;

typedef float f32x2_u __attribute__((ext_vector_type(2), aligned(4)));
typedef _Float16 f16x2_u __attribute__((ext_vector_type(2), aligned(2)));
typedef __bf16 bf16x2_u __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x8_u __attribute__((ext_vector_type(8), aligned(4)));
typedef _Float16 f16x8_u __attribute__((ext_vector_type(8), aligned(2)));
typedef __bf16 bf16x8_u __attribute__((ext_vector_type(8), aligned(2)));

template <int T> struct Elem;
template <> struct Elem<G_F32> { typedef float one; typedef f32x2_u two; typedef f32x8_u eight; };
template <> struct Elem<G_F16> { typedef _Float16 one; typedef f16x2_u two; typedef f16x8_u eight; };
template <> struct Elem<G_BF16> { typedef __bf16 one; typedef bf16x2_u two; typedef bf16x8_u eight; };

__device__ __forceinline__ uint32_t mag(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
template <int CTRL> __device__ __forceinline__ uint32_t row_max(uint32_t v) {
  return umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ uint32_t max4(uint32_t v) { return row_max<0x4E>(row_max<0xB1>(v)); }       // of 4 lanes
__device__ __forceinline__ uint32_t max16(uint32_t v) { return row_max<0x140>(row_max<0x141>(max4(v))); }

// Exponent byte of a block from the bits of its largest magnitude.
template <bool SR> __device__ __forceinline__ uint32_t block_exponent(uint32_t high) {
  const int e = (int)((high + (SR ? 0x3fffffu : 0x200000u)) >> 23) - 2;
  return high >= 0x7f800000u ? 255u : (uint32_t)(e < 1 ? 1 : e);
}
// The factor 2^(s - 127) for the conversions; of a NaN block 2^127, its codes are dropped.
__device__ __forceinline__ float block_factor(uint32_t s) { return __builtin_bit_cast(float, (s < 254 ? s : 254) << 23); }

// Two elements to byte SEL of `old`, a in the low nibble.
template <int SEL> __device__ __forceinline__ uint32_t pack2(uint32_t old, float a, float b, float f) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, f, SEL);
}
// The same by random bits, in byte 0 (the others hold anything: the compiler drops this conversion's
// old value). Its bits come in at the top of a 32-bit number for the low nibble, one bit lower for the
// high one, and one instruction shares them: two elements of their own bits take two.
__device__ __forceinline__ uint32_t pack2_random(float a, float b, float f, uint32_t ra, uint32_t rb) {
  const uint32_t lo = __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, f32x2{a, 0.0f}, ra, f, 0);
  const uint32_t hi = __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, f32x2{0.0f, b}, rb >> 1, f, 0);
  return (lo & 0x0fu) | (hi & ~0x0fu);
}
// the bytes 0 of four
__device__ __forceinline__ uint32_t join4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0c0c0400u), __builtin_amdgcn_perm(b, a, 0x0c0c0400u), 0x05040100u);
}
__device__ __forceinline__ uint32_t turn16(uint32_t r) { return r << 16 | r >> 16; }

__device__ __forceinline__ int64_t scale_at(const MxView& v, int64_t panel, int64_t row, int g) {
  return (panel * v.groups + row / kMxGroup) * kMxGroupBytes + 4 * (16 * g + (row & 15)) + ((row >> 4) & 3);
}

// ---- rows only: 16 lanes a row and panel, 8 elements a lane; a workgroup takes 64 rows of a panel -----
template <int IT, bool SR>
__global__ __launch_bounds__(kThreads)
void k_mx_rows(MxQuantize a) {
  typedef typename Elem<IT>::one one;
  const int64_t panel = blockIdx.x % a.row.panels, r0 = (int64_t)(blockIdx.x / a.row.panels) * kMxGroup;
  const int q = threadIdx.x & 15, sub = threadIdx.x >> 4;
  const int64_t c0 = panel * kMxPanel + 8 * q;
  const uint32_t key = SR ? hash_key(a.seed, a.step ? (uint32_t)*a.step : 0, 0) : 0;
  const int64_t half = (a.n + 1) / 2;
  constexpr int TURNS = kMxGroup / 16;
  f32x8 v[TURNS];
#pragma unroll
  for (int u = 0; u < TURNS; ++u) {
    const int64_t r = r0 + 16 * u + sub;
    v[u] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
    if (r < a.m) {
      const GLOBAL one* x = gbl(static_cast<const one*>(a.x)) + r * a.ld + c0;
      if (c0 + 8 <= a.n) {
        v[u] = __builtin_convertvector(*gcast<typename Elem<IT>::eight>(x), f32x8);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c0 + j < a.n) v[u][j] = (float)x[j];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < TURNS; ++u) {
    const int64_t r = r0 + 16 * u + sub;
    uint32_t high = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) high = umax(high, mag(v[u][j]));
    const uint32_t s = block_exponent<SR>(max4(high));
    const float f = block_factor(s);
    uint32_t w;
    if constexpr (SR) {
      const int64_t i0 = r * half + c0 / 2;
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = hash_bits(hash_high(key, (uint64_t)(i0 + j)), (uint32_t)(i0 + j));
        b[j] = pack2_random(v[u][2 * j], v[u][2 * j + 1], f, x, turn16(x));
      }
      w = join4(b[0], b[1], b[2], b[3]);
    } else {
      w = pack2<0>(0, v[u][0], v[u][1], f);
      w = pack2<1>(w, v[u][2], v[u][3], f);
      w = pack2<2>(w, v[u][4], v[u][5], f);
      w = pack2<3>(w, v[u][6], v[u][7], f);
    }
    if (r < a.m) {
      *gcast<uint32_t>(gbl(a.row.codes) + (panel * a.row.rows + r) * kMxRowBytes + 4 * q) = s == 255 ? 0 : w;
      if ((q & 3) == 0) gbl(a.row.scales)[scale_at(a.row, panel, r, q >> 2)] = (uint8_t)s;
    }
  }
}

// ---- columns, and rows with them: a wave takes 32 rows x 128 columns, a workgroup 128 x 128 -------------
template <int IT, bool ROWS, bool SR>
__global__ __launch_bounds__(kThreads)
void k_mx_cols(MxQuantize a) {
  typedef typename Elem<IT>::one one;
  typedef typename Elem<IT>::two two;
  const int lane = threadIdx.x & (kWave - 1), wv = threadIdx.x / kWave;
  const int64_t pn = (a.n + kMxPanel - 1) / kMxPanel, panel_m = blockIdx.x / pn, panel_n = blockIdx.x - panel_m * pn;
  const int64_t r0 = panel_m * kMxPanel + 32 * wv, c0 = panel_n * kMxPanel + 2 * lane;
  const uint32_t key = SR ? hash_key(a.seed, a.step ? (uint32_t)*a.step : 0, 0) : 0;
  const int64_t half = (a.n + 1) / 2;
  const int64_t rows = a.m - r0;                         // of the block that exist, maybe none
  two v[32];
  const bool both = c0 + 1 < a.n, any = c0 < a.n;
#pragma unroll
  for (int r = 0; r < 32; ++r) {
    v[r] = two{(one)0.0f, (one)0.0f};
    if (r < rows) {
      const GLOBAL one* x = gbl(static_cast<const one*>(a.x)) + (r0 + r) * a.ld + c0;
      if (both) v[r] = *gcast<two>(x);
      else if (any) v[r][0] = x[0];
    }
  }
  uint32_t h0 = 0, h1 = 0;
#pragma unroll
  for (int r = 0; r < 32; ++r) {
    h0 = umax(h0, mag((float)v[r][0]));
    h1 = umax(h1, mag((float)v[r][1]));
  }
  const uint32_t s0 = block_exponent<SR>(h0), s1 = block_exponent<SR>(h1);
  const float f0 = block_factor(s0), f1 = block_factor(s1);
  u32x4 k0, k1;                                          // the columns' codes
  const uint32_t perm_odd = lane & 1 ? 0x07030501u : 0x02060004u, perm_two = lane & 2 ? 0x07060302u : 0x01000504u;
#pragma unroll
  for (int d = 0; d < 4; ++d) {                          // 8 rows: a word of a column, two of row bytes
    uint32_t b0[4], b1[4];                               // bytes of the columns, by random bits
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t rs[4], rb[4], w[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int r = 8 * d + 4 * e + t;
        const float x0 = (float)v[r][0], x1 = (float)v[r][1];
        if constexpr (SR) {
          const int64_t i = (r0 + r) * half + c0 / 2;
          w[t] = hash_bits(hash_high(key, (uint64_t)i), (uint32_t)i);
          if (t & 1) {
            b0[2 * e + t / 2] = pack2_random((float)v[r - 1][0], x0, f0, w[t - 1], w[t]);
            b1[2 * e + t / 2] = pack2_random((float)v[r - 1][1], x1, f1, turn16(w[t - 1]), turn16(w[t]));
          }
        }
        if constexpr (ROWS) {
          const uint32_t s = block_exponent<SR>(max16(umax(mag(x0), mag(x1))));
          const float f = block_factor(s);
          rs[t] = s;
          if constexpr (SR) rb[t] = pack2_random(x0, x1, f, w[t], turn16(w[t]));
          else rb[t] = pack2<0>(0, x0, x1, f);
          rb[t] = s == 255 ? 0 : rb[t];
        }
      }
      if constexpr (ROWS) {
        // 4 rows x 4 lanes of bytes, transposed: lane j of 4 gets row j's
        const uint32_t rw = join4(rb[0], rb[1], rb[2], rb[3]);
        uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)rw, 0xB1, 0xf, 0xf, true);
        uint32_t y = __builtin_amdgcn_perm(rw, o, perm_odd);
        o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)y, 0x4E, 0xf, 0xf, true);
        y = __builtin_amdgcn_perm(y, o, perm_two);
        const int base = 8 * d + 4 * e, r = base + (lane & 3);
        if (r < rows) *gcast<uint32_t>(gbl(a.row.codes) + (panel_n * a.row.rows + r0 + r) * kMxRowBytes + 4 * (lane >> 2)) = y;
        // lane 16 g + t: the exponent of row t, block g
        const uint32_t s = (lane & 3) == 0 ? rs[0] : (lane & 3) == 1 ? rs[1] : (lane & 3) == 2 ? rs[2] : rs[3];
        if ((lane & 15) < 4 && r < rows) gbl(a.row.scales)[scale_at(a.row, panel_n, r0 + r, lane >> 4)] = (uint8_t)s;
      }
    }
    if constexpr (SR) {
      k0[d] = join4(b0[0], b0[1], b0[2], b0[3]);
      k1[d] = join4(b1[0], b1[1], b1[2], b1[3]);
    } else {
      uint32_t w0 = 0, w1 = 0;
      const int r = 8 * d;
      w0 = pack2<0>(w0, (float)v[r][0], (float)v[r + 1][0], f0);
      w0 = pack2<1>(w0, (float)v[r + 2][0], (float)v[r + 3][0], f0);
      w0 = pack2<2>(w0, (float)v[r + 4][0], (float)v[r + 5][0], f0);
      w0 = pack2<3>(w0, (float)v[r + 6][0], (float)v[r + 7][0], f0);
      w1 = pack2<0>(w1, (float)v[r][1], (float)v[r + 1][1], f1);
      w1 = pack2<1>(w1, (float)v[r + 2][1], (float)v[r + 3][1], f1);
      w1 = pack2<2>(w1, (float)v[r + 4][1], (float)v[r + 5][1], f1);
      w1 = pack2<3>(w1, (float)v[r + 6][1], (float)v[r + 7][1], f1);
      k0[d] = w0;
      k1[d] = w1;
    }
  }
  GLOBAL uint8_t* o = gbl(a.col.codes) + (panel_m * a.col.rows + c0) * kMxRowBytes + 16 * wv;
  if (any) {
    *gcast<u32x4>(o) = s0 == 255 ? u32x4{0, 0, 0, 0} : k0;
    gbl(a.col.scales)[scale_at(a.col, panel_m, c0, wv)] = (uint8_t)s0;
  }
  if (both) {
    *gcast<u32x4>(o + kMxRowBytes) = s1 == 255 ? u32x4{0, 0, 0, 0} : k1;
    gbl(a.col.scales)[scale_at(a.col, panel_m, c0 + 1, wv)] = (uint8_t)s1;
  }
}

// ---- back to values: 16 lanes a row and panel, 8 elements a lane ----------------------------------------
template <int OT>
__global__ __launch_bounds__(kThreads)
void k_mx_dequantize(MxView a, void* out, int64_t ld) {
  typedef typename Elem<OT>::one one;
  const int64_t panel = blockIdx.x % a.panels, r0 = (int64_t)(blockIdx.x / a.panels) * kMxGroup;
  const int q = threadIdx.x & 15, sub = threadIdx.x >> 4;
  const int64_t c0 = panel * kMxPanel + 8 * q;
  constexpr int TURNS = kMxGroup / 16;
  uint32_t w[TURNS], s[TURNS];
#pragma unroll
  for (int u = 0; u < TURNS; ++u) {
    const int64_t r = r0 + 16 * u + sub;
    w[u] = s[u] = 0;
    if (r < a.rows) {
      w[u] = *gcast<uint32_t>(gbl(a.codes) + (panel * a.rows + r) * kMxRowBytes + 4 * q);
      s[u] = gbl(a.scales)[scale_at(a, panel, r, q >> 2)];
    }
  }
#pragma unroll
  for (int u = 0; u < TURNS; ++u) {
    const int64_t r = r0 + 16 * u + sub;
    const float f = s[u] == 255 ? __builtin_nanf("") : s[u] == 0 ? 0x1p-127f : __builtin_bit_cast(float, s[u] << 23);
    const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 1);
    const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 3);
    const f32x8 v = f32x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]} * f;
    if (r >= a.rows) continue;
    GLOBAL one* o = gbl(static_cast<one*>(out)) + r * ld + c0;
    if (c0 + 8 <= a.k) {
      *gcast<typename Elem<OT>::eight>(o) = __builtin_convertvector(v, typename Elem<OT>::eight);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c0 + j < a.k) o[j] = (one)v[j];
    }
  }
}

template <int IT, bool SR>
void go(const MxQuantize& a, hipStream_t s) {
  const unsigned pn = (unsigned)((a.n + kMxPanel - 1) / kMxPanel);
  if (!a.col.codes) {
    k_mx_rows<IT, SR><<<dim3(pn * (unsigned)a.row.groups), dim3(kThreads), 0, s>>>(a);
  } else {
    const dim3 grid(pn * (unsigned)((a.m + kMxPanel - 1) / kMxPanel));
    if (a.row.codes) k_mx_cols<IT, true, SR><<<grid, dim3(kThreads), 0, s>>>(a);
    else k_mx_cols<IT, false, SR><<<grid, dim3(kThreads), 0, s>>>(a);
  }
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantize& a, int it, bool stochastic, hipStream_t s) {
  if (it == G_F32) stochastic ? go<G_F32, true>(a, s) : go<G_F32, false>(a, s);
  else if (it == G_F16) stochastic ? go<G_F16, true>(a, s) : go<G_F16, false>(a, s);
  else stochastic ? go<G_BF16, true>(a, s) : go<G_BF16, false>(a, s);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const MxView& a, void* out, int64_t ld, int ot, hipStream_t s) {
  const dim3 grid((unsigned)(a.panels * a.groups)), block(kThreads);
  if (ot == G_F32) k_mx_dequantize<G_F32><<<grid, block, 0, s>>>(a, out, ld);
  else if (ot == G_F16) k_mx_dequantize<G_F16><<<grid, block, 0, s>>>(a, out, ld);
  else k_mx_dequantize<G_BF16><<<grid, block, 0, s>>>(a, out, ld);
  return hipGetLastError();
}

}  // namespace psgd
