// C = s A B^T of microscaled 4-bit matrices (mx.h) on the scaled MFMA: 16 x 16 x 128 a step, each lane
// with 32 codes of one row (16 bytes) and that block's exponent byte; sums in fp32.
//
// P is B (the columns i of C), Q is A (its rows j): a lane then holds C[j][i .. i + 3], consecutive in a
// row of C.
#include <type_traits>
#include <utility>

#include "lds_load.h"
#include "mx.h"

namespace psgd {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int RING = 4;                        // stages (panels) in LDS

template <typename F, int... I> __device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F> __device__ __forceinline__ void each(F&& f) { each_of(f, std::make_integer_sequence<int, N>{}); }

// byte SP of sp and SQ of sq are the exponents
template <int SP, int SQ> __device__ __forceinline__ f32x4 mfma_mx(u32x4 p, u32x4 q, f32x4 c, uint32_t sp, uint32_t sq) {
  const i32x4 a = __builtin_bit_cast(i32x4, p), b = __builtin_bit_cast(i32x4, q);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1),
                                                          __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1), c, 4, 4, SP, (int)sp, SQ, (int)sq);
}

typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef _Float16 f16x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef __bf16 bf16x4_u __attribute__((ext_vector_type(4), aligned(2)));
template <int T> struct Elem;
template <> struct Elem<G_F32> { typedef float one; typedef f32x4_u four; };
template <> struct Elem<G_F16> { typedef _Float16 one; typedef f16x4_u four; };
template <> struct Elem<G_BF16> { typedef __bf16 one; typedef bf16x4_u four; };

// v = C[j][i .. i + 3] of the product, scaled and written or added
template <int OT> __device__ __forceinline__ void finish(const MxProduct& a, int64_t j, int64_t i, f32x4 v, float scale) {
  typedef typename Elem<OT>::one one;
  typedef typename Elem<OT>::four four;
  if (j >= a.m || i >= a.n) return;
  GLOBAL one* c = gbl(static_cast<one*>(a.c)) + j * a.ldc + i;
  v *= scale;
  if (i + 4 <= a.n) {
    if constexpr (OT == G_F32)
      if (a.accumulate) v += *gcast<four>(c);
    *gcast<four>(c) = __builtin_convertvector(v, four);
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (i + t >= a.n) continue;
      float w = v[t];
      if constexpr (OT == G_F32)
        if (a.accumulate) w += c[t];
      c[t] = (one)w;
    }
  }
}

// ---- few rows of A: a workgroup takes 16 columns of C; its waves share the panels ------------------------
// Operands straight from memory to registers: 16 rows of a panel are one contiguous KB.
constexpr int kFewWaves = 8;
template <int MT, int OT>
__global__ __launch_bounds__(kFewWaves * kWave)
void k_mx_few(MxProduct a) {
  const int lane = threadIdx.x & (kWave - 1), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int64_t i0 = (int64_t)blockIdx.x * 16;
  const int64_t pr = i0 + c < a.n ? i0 + c : a.n - 1;
  const int shift = 8 * (int)((i0 >> 4) & 3);
  f32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = f32x4{0, 0, 0, 0};
  auto turn = [&](auto count, int p0) {
    constexpr int U = decltype(count)::value;
    u32x4 p[U], q[U][MT];
    uint32_t sp[U], sq[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t panel = p0 + u * kFewWaves;
      p[u] = *gcast<u32x4>(gbl(a.p.codes) + (panel * a.n + pr) * kMxRowBytes + 16 * g);
      sp[u] = *gcast<uint32_t>(gbl(a.p.scales) + (panel * a.p.groups + i0 / kMxGroup) * kMxGroupBytes + 4 * lane);
      sq[u] = *gcast<uint32_t>(gbl(a.q.scales) + panel * a.q.groups * kMxGroupBytes + 4 * lane);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int64_t qr = 16 * t + c < a.m ? 16 * t + c : a.m - 1;
        q[u][t] = *gcast<u32x4>(gbl(a.q.codes) + (panel * a.m + qr) * kMxRowBytes + 16 * g);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      each<MT>([&](auto t) {
        constexpr int X = decltype(t)::value;
        acc[X] = mfma_mx<0, X>(p[u], q[u][X], acc[X], sp[u] >> shift, sq[u]);
      });
  };
  const int panels = (int)a.p.panels;
  int panel = wv;
  for (; panel + 3 * kFewWaves < panels; panel += 4 * kFewWaves) turn(std::integral_constant<int, 4>{}, panel);
  for (; panel < panels; panel += kFewWaves) turn(std::integral_constant<int, 1>{}, panel);

  __shared__ f32x4 part[kFewWaves][MT][kWave];
#pragma unroll
  for (int t = 0; t < MT; ++t) part[wv][t][lane] = acc[t];
  __syncthreads();
  if (wv >= MT) return;
  f32x4 sum = part[0][wv][lane];
#pragma unroll
  for (int w = 1; w < kFewWaves; ++w) sum += part[w][wv][lane];
  finish<OT>(a, 16 * wv + c, i0 + 4 * g, sum, a.scale ? *a.scale : 1.0f);
}

// ---- tiles ------------------------------------------------------------------------------------------------
template <int T> struct Tile {
  static constexpr int WAVES = T == 256 ? 8 : 4;
  static constexpr int WI = WAVES / 2;                       // waves along i; 2 along j
  static constexpr int SI = T / WI, SJ = T / 2;              // a wave's sides
  static constexpr int NI = SI / 16, NJ = SJ / 16;           // in MFMA tiles
  static constexpr int CODES = T * kMxRowBytes;              // bytes of an operand's stage
  static constexpr int SCALES = T / kMxGroup * kMxGroupBytes;
  static constexpr int STAGE = 2 * (CODES + SCALES);
  static constexpr int LOADS = 2 * CODES / 1024 / WAVES;     // 1 KB loads of codes per wave and stage
  static constexpr int WORDS = 2 * SCALES / 256;             // 256-byte loads of exponents per stage
  static constexpr int SLOADS = (WORDS + WAVES - 1) / WAVES; // per wave (some of them twice where a wave has none of its own)
};

__device__ __forceinline__ int swz(int row, int q) { return q ^ ((row >> 1) & 3); }

__device__ __forceinline__ void load_lds4(const GLOBAL uint8_t* base, uint32_t off, uint32_t l) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(l), "v"(off), "s"(base) : "m0", "memory");
}

template <int T, int OT, bool SPLIT>
__global__ __launch_bounds__(Tile<T>::WAVES * kWave, 2)
void k_mx_gemm(MxProduct a) {
  using TL = Tile<T>;
  constexpr int NI = TL::NI, NJ = TL::NJ;
  const int lane = threadIdx.x & (kWave - 1), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int ti = (int)((a.n + T - 1) / T), tj = (int)((a.m + T - 1) / T);
  // neighbours in the list share operands: strips of 4 tiles of rows
  const int item = xcd_remap(blockIdx.x, gridDim.x);
  const int tiles = ti * tj;
  const int split = item / tiles;
  if (split >= a.splits) return;
  const int tile = item - split * tiles;
  const int strip = tile / (4 * ti), in = tile - strip * 4 * ti;
  const int high = tj - 4 * strip < 4 ? tj - 4 * strip : 4;
  const int64_t i0 = (int64_t)(in / high) * T, j0 = (int64_t)(4 * strip + in % high) * T;
  const int first = split * a.per;
  const int nst = (int)(a.p.panels - first < a.per ? a.p.panels - first : a.per);
  const int wi0 = (wv >> 1) * TL::SI, wj0 = (wv & 1) * TL::SJ;

  __shared__ __attribute__((aligned(16))) uint8_t lds[RING][TL::STAGE];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(LDS uint8_t*)&lds[0][0];
  // this wave's loads of a stage: load x of all 2 CODES / 1024, P's first
  uint32_t off[TL::LOADS], soff[TL::SLOADS];
#pragma unroll
  for (int x = 0; x < TL::LOADS; ++x) {
    const int id = wv * TL::LOADS + x;
    const bool q = id >= TL::CODES / 1024;
    const int r = (q ? id - TL::CODES / 1024 : id) * 16 + (lane >> 2);
    const int64_t left = (q ? a.m - j0 : a.n - i0) - 1;       // rows past the matrix read its last one
    off[x] = (uint32_t)((q ? j0 : i0) + (r < left ? r : left)) * kMxRowBytes + 16 * swz(r, lane & 3);
  }
#pragma unroll
  for (int x = 0; x < TL::SLOADS; ++x) {
    const int id = (wv * TL::SLOADS + x) % TL::WORDS;
    const bool q = id >= TL::WORDS / 2;
    const int64_t grp = (q ? j0 : i0) / kMxGroup + (q ? id - TL::WORDS / 2 : id), last = (q ? a.q.groups : a.p.groups) - 1;
    soff[x] = (uint32_t)(grp < last ? grp : last) * kMxGroupBytes + 4 * lane;
  }
  const int64_t pstep = a.n * kMxRowBytes, qstep = a.m * kMxRowBytes, psstep = a.p.groups * kMxGroupBytes, qsstep = a.q.groups * kMxGroupBytes;
  auto load_stage = [&](int j) {
    const int64_t panel = first + j;
    const uint32_t l = lds0 + (uint32_t)(j % RING) * TL::STAGE;
    const GLOBAL uint8_t* pc = gbl(a.p.codes) + panel * pstep;
    const GLOBAL uint8_t* qc = gbl(a.q.codes) + panel * qstep;
    const GLOBAL uint8_t* ps = gbl(a.p.scales) + panel * psstep;
    const GLOBAL uint8_t* qs = gbl(a.q.scales) + panel * qsstep;
#pragma unroll
    for (int x = 0; x < TL::LOADS; ++x) {
      const int id = wv * TL::LOADS + x;
      load_lds16(gcast<uint16_t>(id >= TL::CODES / 1024 ? qc : pc), off[x], l + id * 1024);
    }
#pragma unroll
    for (int x = 0; x < TL::SLOADS; ++x) {
      const int id = (wv * TL::SLOADS + x) % TL::WORDS;
      load_lds4(id >= TL::WORDS / 2 ? qs : ps, soff[x], l + 2 * TL::CODES + id * 256);
    }
  };
  constexpr int PER = TL::LOADS + TL::SLOADS;
  // stage j + 1 has landed when at most the `behind` later ones are under way
  auto wait_stages = [&](int behind) {
    if (behind >= 2) wait_loads<2 * PER>();
    else if (behind == 1) wait_loads<PER>();
    else wait_loads<0>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };

  constexpr int KI = (NI + 3) / 4, KJ = (NJ + 3) / 4;        // exponent words of a side
  struct Frag { u32x4 p[NI], q[NJ]; uint32_t sp[KI], sq[KJ]; };
  auto read = [&](Frag& f, int j) {
    const uint8_t* s = lds[j % RING];
#pragma unroll
    for (int x = 0; x < NI; ++x) {
      const int r = wi0 + 16 * x + c;
      f.p[x] = *reinterpret_cast<const u32x4*>(s + r * kMxRowBytes + 16 * swz(r, g));
    }
#pragma unroll
    for (int x = 0; x < NJ; ++x) {
      const int r = wj0 + 16 * x + c;
      f.q[x] = *reinterpret_cast<const u32x4*>(s + TL::CODES + r * kMxRowBytes + 16 * swz(r, g));
    }
    const uint8_t* e = s + 2 * TL::CODES + 4 * lane;
#pragma unroll
    for (int x = 0; x < KI; ++x) f.sp[x] = *reinterpret_cast<const uint32_t*>(e + (wi0 / kMxGroup + x) * kMxGroupBytes);
#pragma unroll
    for (int x = 0; x < KJ; ++x) f.sq[x] = *reinterpret_cast<const uint32_t*>(e + TL::SCALES + (wj0 / kMxGroup + x) * kMxGroupBytes);
    if constexpr (TL::SI < kMxGroup) f.sp[0] >>= wi0 % kMxGroup / 2;    // 16 rows a byte
    if constexpr (TL::SJ < kMxGroup) f.sq[0] >>= wj0 % kMxGroup / 2;
  };
  f32x4 acc[NI][NJ];
#pragma unroll
  for (int x = 0; x < NI; ++x)
#pragma unroll
    for (int y = 0; y < NJ; ++y) acc[x][y] = f32x4{0, 0, 0, 0};
  auto mul = [&](const Frag& f) {
    each<NI>([&](auto x) {
      each<NJ>([&](auto y) {
        constexpr int X = decltype(x)::value, Y = decltype(y)::value;
        acc[X][Y] = mfma_mx<X & 3, Y & 3>(f.p[X], f.q[Y], acc[X][Y], f.sp[X / 4], f.sq[Y / 4]);
      });
    });
  };

  for (int j = 0; j < RING && j < nst; ++j) load_stage(j);
  if (nst >= 4) wait_loads<3 * PER>();
  else wait_loads<0>();
  __builtin_amdgcn_s_barrier();
  Frag f0, f1;
  read(f0, 0);
  auto step = [&](Frag& now, Frag& next, int j) {
    wait_stages(nst - 2 - j);
    if (j + RING < nst) load_stage(j + RING);
    if (j + 1 < nst) read(next, j + 1);
    mul(now);
  };
  for (int j = 0; j < nst; j += 2) {
    step(f0, f1, j);
    if (j + 1 < nst) step(f1, f0, j + 1);
  }

  if constexpr (SPLIT) {
    GLOBAL float* o = gbl(a.partial) + (int64_t)split * a.m * a.n;
#pragma unroll
    for (int x = 0; x < NI; ++x)
#pragma unroll
      for (int y = 0; y < NJ; ++y) {
        const int64_t i = i0 + wi0 + 16 * x + 4 * g, j = j0 + wj0 + 16 * y + c;
        if (j >= a.m) continue;
        if (i + 4 <= a.n) *gcast<f32x4_u>(o + j * a.n + i) = acc[x][y];
        else
#pragma unroll
          for (int t = 0; t < 4; ++t)
            if (i + t < a.n) o[j * a.n + i + t] = acc[x][y][t];
      }
  } else {
    const float scale = a.scale ? *a.scale : 1.0f;
#pragma unroll
    for (int x = 0; x < NI; ++x)
#pragma unroll
      for (int y = 0; y < NJ; ++y) finish<OT>(a, j0 + wj0 + 16 * y + c, i0 + wi0 + 16 * x + 4 * g, acc[x][y], scale);
  }
}

// The parts of a split product, added in order.
template <int OT>
__global__ __launch_bounds__(256)
void k_mx_join(MxProduct a) {
  const int64_t blocks = (a.n + 1023) / 1024, j = blockIdx.x / blocks;
  const int64_t i = 4 * ((blockIdx.x - j * blocks) * 256 + threadIdx.x);
  if (i >= a.n) return;
  const GLOBAL float* p = gbl(a.partial) + j * a.n + i;
  const int64_t step = a.m * a.n;
  f32x4 sum{0, 0, 0, 0};
  if (i + 4 <= a.n) {
    for (int s = 0; s < a.splits; ++s) sum += *gcast<f32x4_u>(p + s * step);
  } else {
    for (int s = 0; s < a.splits; ++s)
      for (int t = 0; t < 4; ++t)
        if (i + t < a.n) sum[t] += p[s * step + t];
  }
  finish<OT>(a, j, i, sum, a.scale ? *a.scale : 1.0f);
}

template <int T, int OT>
hipError_t go_tiles(const MxProduct& a, hipStream_t s) {
  const int64_t tiles = ((a.n + T - 1) / T) * ((a.m + T - 1) / T) * a.splits;
  const dim3 grid((unsigned)((tiles + 7) / 8 * 8)), block(Tile<T>::WAVES * kWave);
  if (a.splits == 1) {
    k_mx_gemm<T, OT, false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
  }
  k_mx_gemm<T, G_F32, true><<<grid, block, 0, s>>>(a);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  k_mx_join<OT><<<dim3((unsigned)((a.n + 1023) / 1024 * a.m)), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}
template <int OT>
hipError_t go(const MxProduct& a, int tile, hipStream_t s) {
  if (tile == 256) return go_tiles<256, OT>(a, s);
  if (tile == 128) return go_tiles<128, OT>(a, s);
  if (tile == 64) return go_tiles<64, OT>(a, s);
  const dim3 grid((unsigned)((a.n + 15) / 16)), block(kFewWaves * kWave);
  if (a.m <= 16) k_mx_few<1, OT><<<grid, block, 0, s>>>(a);
  else if (a.m <= 32) k_mx_few<2, OT><<<grid, block, 0, s>>>(a);
  else k_mx_few<4, OT><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

MxPlan mx_plan(int64_t m, int64_t n, int64_t panels) {
  if (m <= 64) return {0, 1};
  auto tiles = [&](int64_t t) { return ((m + t - 1) / t) * ((n + t - 1) / t); };
  int tile = 64;
  if (tiles(256) >= 192) tile = 256;
  else if (tiles(128) >= 192 || panels >= 64) tile = 128;
  int splits = 1;
  while (splits < 8 && tiles(tile) * splits < 192 && panels / (2 * splits) >= 8) splits *= 2;
  return {tile, splits};
}

hipError_t launch_mx_product(const MxProduct& a, int tile, int ot, hipStream_t s) {
  if (ot == G_F32) return go<G_F32>(a, tile, s);
  if (ot == G_F16) return go<G_F16>(a, tile, s);
  return go<G_BF16>(a, tile, s);
}

}  // namespace psgd
