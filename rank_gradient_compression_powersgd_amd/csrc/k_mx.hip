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
//
// Bound: to nearest, memory (20480 x 3968 bf16, both directions, 249 MB: 40 us, 6.3 TB/s, with 81 MB of it still in
// the last cache, 49 us, 5.1 TB/s, with none; rows alone 29 us; 20480 x 1984 fp16 35 to 39 us, 3.2 to 3.6 TB/s). By
// random bits the vector instructions come close to it: a conversion of 14 cycles per element and direction and
// a hash per two elements, 25 of 55 us (4.5 TB/s); 61 to 77 us where nothing is in a cache. Loads of the next block
// ahead of this one's work cost waves and gained nothing (55 -> 62 us).
#include <type_traits>
#include <utility>

#include "hash.h"
#include "mx.h"

namespace psgd {
namespace {

constexpr int kThreads = 256;

typedef float f32x2_u __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t u32_u __attribute__((aligned(2)));
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x8_u __attribute__((ext_vector_type(8), aligned(4)));
typedef _Float16 f16x8_u __attribute__((ext_vector_type(8), aligned(2)));
typedef __bf16 bf16x8_u __attribute__((ext_vector_type(8), aligned(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

template <int T> struct Elem;
template <> struct Elem<G_F32> { typedef float one; typedef f32x8_u eight; };
template <> struct Elem<G_F16> { typedef _Float16 one; typedef f16x8_u eight; };
template <> struct Elem<G_BF16> { typedef __bf16 one; typedef bf16x8_u eight; };

template <typename F, int... I> __device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F> __device__ __forceinline__ void each(F&& f) { each_of(f, std::make_integer_sequence<int, N>{}); }

__device__ __forceinline__ uint32_t mag(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
template <int CTRL> __device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kRor4 = 0x124, kRor8 = 0x128, kBcast = 0x150;   // of 4 lanes, of 16
__device__ __forceinline__ uint32_t max4(uint32_t v) {                                     // of 4 lanes
  v = umax(v, dpp<kXor1>(v));
  return umax(v, dpp<kXor2>(v));
}
// m[r]: a lane's value of row r, 16 rows; the largest of row `lane % 16` over the 16 lanes. Each of two
// exchanges halves the rows that a lane carries.
__device__ __forceinline__ uint32_t max_of_rows(const uint32_t (&m)[16], int lane) {
  uint32_t a[8], b[4];
#pragma unroll
  for (int k = 0; k < 8; ++k) a[k] = umax(lane & 1 ? m[2 * k + 1] : m[2 * k], dpp<kXor1>(lane & 1 ? m[2 * k] : m[2 * k + 1]));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    b[k] = umax(lane & 2 ? a[2 * k + 1] : a[2 * k], dpp<kXor2>(lane & 2 ? a[2 * k] : a[2 * k + 1]));
    b[k] = umax(b[k], dpp<kRor4>(b[k]));
    b[k] = umax(b[k], dpp<kRor8>(b[k]));
  }
  const uint32_t lo = lane & 4 ? b[1] : b[0], hi = lane & 4 ? b[3] : b[2];
  return lane & 8 ? hi : lo;
}

// Exponent byte of a block from the bits of its largest magnitude.
template <bool SR> __device__ __forceinline__ uint32_t block_exponent(uint32_t high) {
  const int e = (int)((high + (SR ? 0x3fffffu : 0x200000u)) >> 23) - 2;
  return high >= 0x7f800000u ? 255u : (uint32_t)(e < 1 ? 1 : e);
}
// The factor 2^(s - 127) for the conversions; of a NaN block 2^127, its codes are dropped.
__device__ __forceinline__ float block_factor(uint32_t s) { return __builtin_bit_cast(float, (s < 254 ? s : 254) << 23); }

// Two elements by random bits, in byte 0, a in the low nibble (the other bytes hold anything: the
// compiler drops this conversion's old value; from fp32, the 16-bit types' conversions keep fewer bits of
// what they cut off). Its bits come in at the top of a 32-bit number for the low nibble, one bit lower for the
// high one, and one instruction shares them: two elements of their own bits take two, each for a nibble.
__device__ __forceinline__ uint32_t pack2_random(float a, float b, float f, uint32_t ra, uint32_t rb) {
  const uint32_t lo = __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, f32x2{a, b}, ra, f, 0);
  const uint32_t hi = __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, f32x2{a, b}, rb >> 1, f, 0);
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

// Bits of pair i0 + d of a run that is shorter than 2^32: its index passes a multiple of 2^32 at most once.
struct PairBits {
  uint32_t lo, here, next;
  __device__ __forceinline__ PairBits(uint32_t key, int64_t i0)
      : lo((uint32_t)i0), here(hash_high(key, (uint64_t)i0)), next(hash_high(key, (uint64_t)i0 + (uint64_t(1) << 32))) {}
  __device__ __forceinline__ uint32_t at(uint32_t d) const { return hash_bits(lo + d < lo ? next : here, lo + d); }
};

// Two neighbours of a row as they were loaded.
template <int IT> struct Pair {
  uint32_t w;                                              // the second in the high half
  __device__ __forceinline__ void load(const GLOBAL void* x, bool both, bool any) {
    w = 0;
    if (both) w = *gcast<u32_u>(static_cast<const GLOBAL uint16_t*>(x));
    else if (any) w = *static_cast<const GLOBAL uint16_t*>(x);
  }
  __device__ __forceinline__ void load_each(const GLOBAL void* x, const GLOBAL void* y, bool first, bool second) {
    const uint32_t a = *static_cast<const GLOBAL uint16_t*>(x), b = *static_cast<const GLOBAL uint16_t*>(y);
    w = (first ? a : 0) | (second ? b << 16 : 0);
  }
  __device__ __forceinline__ static void load4(Pair (&p)[4], const GLOBAL void* x) {
    const u32x4_u v = *gcast<u32x4_u>(static_cast<const GLOBAL uint16_t*>(x));
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j].w = v[j];
  }
  // magnitudes, whose order as integers is that of the values; `bits` makes fp32's of them
  typedef u16x2 mags;
  __device__ __forceinline__ mags mag() const { return __builtin_bit_cast(u16x2, w & 0x7fff7fffu); }
  __device__ __forceinline__ static uint32_t larger(mags m) { return umax(m[0], m[1]); }
  __device__ __forceinline__ static uint32_t bits(uint32_t m) {
    if constexpr (IT == G_BF16) return m << 16;
    else return __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(_Float16, (uint16_t)m));
  }
  __device__ __forceinline__ uint32_t nearest(float f) const {                              // byte 0
    if constexpr (IT == G_BF16) return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0u, __builtin_bit_cast(bf16x2, w), f, 0);
    else return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(0u, __builtin_bit_cast(f16x2, w), f, 0);
  }
  __device__ __forceinline__ float x() const {
    if constexpr (IT == G_BF16) return __builtin_bit_cast(float, w << 16);
    else return (float)__builtin_bit_cast(f16x2, w)[0];
  }
  __device__ __forceinline__ float y() const {
    if constexpr (IT == G_BF16) return __builtin_bit_cast(float, w & 0xffff0000u);
    else return (float)__builtin_bit_cast(f16x2, w)[1];
  }
  // the same column's of two rows
  __device__ __forceinline__ static Pair first(Pair a, Pair b) { return Pair{__builtin_amdgcn_perm(b.w, a.w, 0x05040100u)}; }
  __device__ __forceinline__ static Pair second(Pair a, Pair b) { return Pair{__builtin_amdgcn_perm(b.w, a.w, 0x07060302u)}; }
};
template <> struct Pair<G_F32> {
  float v, w;
  __device__ __forceinline__ float x() const { return v; }
  __device__ __forceinline__ float y() const { return w; }
  __device__ __forceinline__ void load(const GLOBAL void* p, bool both, bool any) {
    v = w = 0.0f;
    if (both) {
      const f32x2_u u = *gcast<f32x2_u>(static_cast<const GLOBAL float*>(p));
      v = u[0];
      w = u[1];
    } else if (any) {
      v = *static_cast<const GLOBAL float*>(p);
    }
  }
  __device__ __forceinline__ void load_each(const GLOBAL void* x, const GLOBAL void* y, bool first, bool second) {
    v = *static_cast<const GLOBAL float*>(x);
    w = *static_cast<const GLOBAL float*>(y);
    if (!first) v = 0.0f;
    if (!second) w = 0.0f;
  }
  __device__ __forceinline__ static void load4(Pair (&p)[4], const GLOBAL void* x) {
    const f32x8_u v = *gcast<f32x8_u>(static_cast<const GLOBAL float*>(x));
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = Pair{v[2 * j], v[2 * j + 1]};
  }
  typedef u32x2 mags;
  __device__ __forceinline__ mags mag() const { return u32x2{psgd::mag(v), psgd::mag(w)}; }
  __device__ __forceinline__ static uint32_t larger(mags m) { return umax(m[0], m[1]); }
  __device__ __forceinline__ static uint32_t bits(uint32_t m) { return m; }
  __device__ __forceinline__ uint32_t nearest(float f) const { return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v, w, f, 0); }
  __device__ __forceinline__ static Pair first(Pair a, Pair b) { return Pair{a.v, b.v}; }
  __device__ __forceinline__ static Pair second(Pair a, Pair b) { return Pair{a.w, b.w}; }
};
// ---- rows only: 16 lanes a row and panel, 8 elements a lane; a workgroup takes 64 rows of a panel -----
// 16-byte loads, where the kernel below takes 4 bytes a lane to have columns in it (20480 x 1984 bf16: 16 us,
// columns alone 20).
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
  Pair<IT> v[TURNS][4];
#pragma unroll
  for (int u = 0; u < TURNS; ++u) {
    const int64_t r = r0 + 16 * u + sub;
    const GLOBAL one* x = gbl(static_cast<const one*>(a.x)) + r * a.ld + c0;
    if (r < a.m && c0 + 8 <= a.n) {
      Pair<IT>::load4(v[u], x);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[u][j].load(x + 2 * j, r < a.m && c0 + 2 * j + 1 < a.n, r < a.m && c0 + 2 * j < a.n);
    }
  }
#pragma unroll
  for (int u = 0; u < TURNS; ++u) {
    const int64_t r = r0 + 16 * u + sub;
    typename Pair<IT>::mags high = v[u][0].mag();
#pragma unroll
    for (int j = 1; j < 4; ++j) high = __builtin_elementwise_max(high, v[u][j].mag());
    const uint32_t s = block_exponent<SR>(Pair<IT>::bits(max4(Pair<IT>::larger(high))));
    const float f = block_factor(s);
    uint32_t b[4];
    const PairBits bits(key, r * half + c0 / 2);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (SR) {
        const uint32_t w = bits.at(j);
        b[j] = pack2_random(v[u][j].x(), v[u][j].y(), f, w, turn16(w));
      } else {
        b[j] = v[u][j].nearest(f);
      }
    }
    if (r < a.m) {
      const uint32_t w = join4(b[0], b[1], b[2], b[3]);
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
  const int lane = threadIdx.x & (kWave - 1), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t pn = (a.n + kMxPanel - 1) / kMxPanel, panel_m = blockIdx.x / pn, panel_n = blockIdx.x - panel_m * pn;
  const int64_t r0 = panel_m * kMxPanel + 32 * wv, c0 = panel_n * kMxPanel + 2 * lane;
  const int rows = (int)(a.m - r0 < 32 ? a.m - r0 : 32);     // of the block that exist, maybe none
  const bool both = c0 + 1 < a.n, any = c0 < a.n;
  Pair<IT> v[32];
  const GLOBAL one* x = gbl(static_cast<const one*>(a.x)) + r0 * a.ld + c0;
  if (rows == 32 && (panel_n + 1) * kMxPanel <= a.n) {       // all of the wave's: loads without a branch between them
#pragma unroll
    for (int r = 0; r < 32; ++r) v[r].load(x + r * a.ld, true, true);
  } else {                                                   // the matrix's nearest elements in the place of those past it
    const GLOBAL one* e = gbl(static_cast<const one*>(a.x));
    const int64_t e0 = any ? c0 : a.n - 1, e1 = both ? c0 + 1 : a.n - 1;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      const int64_t row = (r < rows ? r0 + r : a.m - 1) * a.ld;
      v[r].load_each(e + row + e0, e + row + e1, any && r < rows, both && r < rows);
    }
  }

  typename Pair<IT>::mags high{0, 0};
#pragma unroll
  for (int r = 0; r < 32; ++r) high = __builtin_elementwise_max(high, v[r].mag());
  const uint32_t s0 = block_exponent<SR>(Pair<IT>::bits(high[0])), s1 = block_exponent<SR>(Pair<IT>::bits(high[1]));
  const float f0 = block_factor(s0), f1 = block_factor(s1);
  uint32_t k0[4], k1[4];                                     // the columns' codes
  const uint32_t half = (uint32_t)((a.n + 1) / 2);
  const PairBits bits(SR ? hash_key(a.seed, a.step ? (uint32_t)*a.step : 0, 0) : 0, r0 * (int64_t)half + c0 / 2);
  const uint32_t perm_odd = lane & 1 ? 0x07030501u : 0x02060004u, perm_two = lane & 2 ? 0x07060302u : 0x01000504u;
  GLOBAL uint8_t* ro = gbl(a.row.codes) + (panel_n * a.row.rows + r0 + (lane & 3)) * kMxRowBytes + 4 * (lane >> 2);
  each<2>([&](auto hh) {                                     // 16 rows
    constexpr int h = decltype(hh)::value;
    uint32_t s = 0, f = 0;                                   // exponent and factor of row lane % 16, block lane / 16
    bool bad = false;
    if constexpr (ROWS) {
      uint32_t m[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) m[r] = Pair<IT>::larger(v[16 * h + r].mag());
      s = block_exponent<SR>(Pair<IT>::bits(max_of_rows(m, lane)));
      f = __builtin_bit_cast(uint32_t, block_factor(s));
      const int r = 16 * h + (lane & 15);
      if (r < rows) gbl(a.row.scales)[scale_at(a.row, panel_n, r0 + r, lane >> 4)] = (uint8_t)s;
      bad = __builtin_amdgcn_ballot_w64(s == 255) != 0;
    }
    each<4>([&](auto dd) {                                   // 4 rows
      constexpr int D = decltype(dd)::value;
      __builtin_amdgcn_sched_barrier(0);                     // the bits of more rows at once take registers of other waves
      const int r = 16 * h + 4 * D;
      uint32_t w[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) w[t] = SR ? bits.at((r + t) * half) : 0;
      uint32_t b0[2], b1[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const Pair<IT>&p = v[r + 2 * t], &q = v[r + 2 * t + 1];
        if constexpr (SR) {
          b0[t] = pack2_random(p.x(), q.x(), f0, w[2 * t], w[2 * t + 1]);
          b1[t] = pack2_random(p.y(), q.y(), f1, turn16(w[2 * t]), turn16(w[2 * t + 1]));
        } else {
          b0[t] = Pair<IT>::first(p, q).nearest(f0);
          b1[t] = Pair<IT>::second(p, q).nearest(f1);
        }
      }
      const uint32_t p0 = __builtin_amdgcn_perm(b0[1], b0[0], 0x0c0c0400u), p1 = __builtin_amdgcn_perm(b1[1], b1[0], 0x0c0c0400u);
      k0[2 * h + D / 2] = D & 1 ? k0[2 * h + D / 2] | p0 << 16 : p0;
      k1[2 * h + D / 2] = D & 1 ? k1[2 * h + D / 2] | p1 << 16 : p1;
      asm volatile("" : "+v"(k0[2 * h + D / 2]), "+v"(k1[2 * h + D / 2]));   // here, not with their store: the bits would stay till then
      if constexpr (ROWS) {
        uint32_t rb[4];
        each<4>([&](auto tt) {
          constexpr int T = decltype(tt)::value;
          const float fr = __builtin_bit_cast(float, dpp<kBcast + 4 * D + T>(f));
          if constexpr (SR) rb[T] = pack2_random(v[r + T].x(), v[r + T].y(), fr, w[T], turn16(w[T]));
          else rb[T] = v[r + T].nearest(fr);
        });
        // 4 rows x 4 lanes of bytes, transposed: lane j of 4 gets row j's
        const uint32_t rw = join4(rb[0], rb[1], rb[2], rb[3]);
        uint32_t y = __builtin_amdgcn_perm(rw, dpp<kXor1>(rw), perm_odd);
        y = __builtin_amdgcn_perm(y, dpp<kXor2>(y), perm_two);
        if (bad && __builtin_amdgcn_ds_bpermute(4 * ((lane & 48) + 4 * D + (lane & 3)), (int)s) == 255) y = 0;
        if (r + (lane & 3) < rows) *gcast<uint32_t>(ro + r * kMxRowBytes) = y;
      }
    });
  });
  GLOBAL uint8_t* o = gbl(a.col.codes) + (panel_m * a.col.rows + c0) * kMxRowBytes + 16 * wv;
  if (any) {
    *gcast<u32x4>(o) = s0 == 255 ? u32x4{0, 0, 0, 0} : u32x4{k0[0], k0[1], k0[2], k0[3]};
    gbl(a.col.scales)[scale_at(a.col, panel_m, c0, wv)] = (uint8_t)s0;
  }
  if (both) {
    *gcast<u32x4>(o + kMxRowBytes) = s1 == 255 ? u32x4{0, 0, 0, 0} : u32x4{k1[0], k1[1], k1[2], k1[3]};
    gbl(a.col.scales)[scale_at(a.col, panel_m, c0 + 1, wv)] = (uint8_t)s1;
  }
}

// ---- back to values: 16 lanes a row and panel, 8 elements a lane ----------------------------------------
// Bound: memory (20480 x 3968 to bf16, 206 MB: 31 to 42 us, 6.6 to 4.9 TB/s).
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
