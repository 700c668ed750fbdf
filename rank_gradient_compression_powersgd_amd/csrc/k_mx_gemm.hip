// C = s A B^T of microscaled 4-bit matrices (mx.h) on the scaled MFMA: 16 x 16 x 128 a step, each lane
// with 32 codes of one row (16 bytes) and that block's exponent byte; sums in fp32.
//
// P is B (the columns i of C), Q is A (its rows j): a lane then holds C[j][i .. i + 3], consecutive in a
// row of C.
//
// Bound: the MFMAs at the clock that full load leaves, and beside them the operands' way into LDS. 64 MFMAs a wave
// and stage take 0.59 us with every CU at work (16 cycles each at 1.74 GHz; 0.49 on 40 CUs), 0.65 with the
// reads from LDS, 0.81 with the loads into it: 5.3 PFLOP/s. A 256-wide tile of 16-bit results takes 4 us more
// to store. 20480 x 15872, k = 3968, bf16: 601 to 622 us, 4.1 to 4.3 PFLOP/s (bf16 library products reach
// 1.37); over the whole kernel the matrix pipe is busy in 50% of the cycles, and no LDS access waits for a bank.
#include <algorithm>
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

// The same with sum I of a tile of N x N in the accumulation registers 4 I .. 4 I + 3; NEW: what the sum
// held is not read. As asm, since the compiler keeps sums of this many registers in ordinary ones, with
// a move for every use (as operands "+a" of these statements 256 of them spill), and on registers by name.
// Every statement that writes or reads sums, and settle() between the two, marks all of the tile's as written,
// so the compiler keeps nothing across any of them there and never moves a sum. What it might keep there
// between two of them the build looks for in the object (build.py: only MFMAs write accumulation
// registers in this file). Consecutive uses of one sum are a whole row of MFMAs apart; settle() stands
// between the last of them and the first read of a sum.
#define MX_A10(p) "a" #p "0", "a" #p "1", "a" #p "2", "a" #p "3", "a" #p "4", "a" #p "5", "a" #p "6", "a" #p "7", "a" #p "8", "a" #p "9"
#define MX_A16 "a0", "a1", "a2", "a3", "a4", "a5", "a6", "a7", "a8", "a9", "a10", "a11", "a12", "a13", "a14", "a15"
#define MX_A64 MX_A16, "a16", "a17", "a18", "a19", MX_A10(2), MX_A10(3), MX_A10(4), MX_A10(5), "a60", "a61", "a62", "a63"
#define MX_A256                                                                                                              \
  MX_A64, "a64", "a65", "a66", "a67", "a68", "a69", MX_A10(7), MX_A10(8), MX_A10(9), MX_A10(10), MX_A10(11), MX_A10(12),     \
      MX_A10(13), MX_A10(14), MX_A10(15), MX_A10(16), MX_A10(17), MX_A10(18), MX_A10(19), MX_A10(20), MX_A10(21), MX_A10(22), \
      MX_A10(23), MX_A10(24), "a250", "a251", "a252", "a253", "a254", "a255"
#define MX_LINE(LO, HI, Q, C, S0, S1, SP, SQ, B0, B1)                                                             \
  "v_mfma_scale_f32_16x16x128_f8f6f4 a[%" LO ":%" HI "], %0, %" Q ", " C ", %" SP ", %" SQ " op_sel:[%" S0        \
  "," B0 ",0] op_sel_hi:[%" S1 "," B1 ",0] cbsz:4 blgp:4\n\t"
#define MX_I(y) "n"(4 * (I + y)), "n"(4 * (I + y) + 3)
#define MX_KEEP(LO, HI) "a[%" LO ":%" HI "]"
#define MX_ZERO(LO, HI) "0"
#define MX_ROW4(C, CLOBBER)                                                                                        \
  asm volatile(MX_LINE("7", "8", "1", C("7", "8"), "15", "16", "5", "6", "0", "0")                                 \
               MX_LINE("9", "10", "2", C("9", "10"), "15", "16", "5", "6", "1", "0")                               \
               MX_LINE("11", "12", "3", C("11", "12"), "15", "16", "5", "6", "0", "1")                             \
               MX_LINE("13", "14", "4", C("13", "14"), "15", "16", "5", "6", "1", "1")                             \
               ::"v"(p), "v"(q[Y]), "v"(q[Y + 1]), "v"(q[Y + 2]), "v"(q[Y + 3]), "v"(sp), "v"(sq[Y / 4]), MX_I(Y), \
               MX_I(Y + 1), MX_I(Y + 2), MX_I(Y + 3), "n"(SP & 1), "n"(SP >> 1) : CLOBBER)
#define MX_ROW2(C)                                                                                                 \
  asm volatile(MX_LINE("5", "6", "1", C("5", "6"), "9", "10", "3", "4", "0", "0")                                  \
               MX_LINE("7", "8", "2", C("7", "8"), "9", "10", "3", "4", "1", "0")                                  \
               ::"v"(p), "v"(q[0]), "v"(q[1]), "v"(sp), "v"(sq[0]), MX_I(0), MX_I(1), "n"(SP & 1), "n"(SP >> 1) : MX_A16)
// Up to four MFMAs of a row of the tile: sums I + Y, ...; byte SP of sp is p's exponent, byte y % 4 of
// sq[y / 4] that of q[y].
template <int N, int I, int Y, int SP, bool NEW> __device__ __forceinline__ void mfma_row(u32x4 p, const u32x4 (&q)[N], uint32_t sp, const uint32_t* sq) {
  if constexpr (N == 8 && NEW) MX_ROW4(MX_ZERO, MX_A256);
  else if constexpr (N == 8) MX_ROW4(MX_KEEP, MX_A256);
  else if constexpr (N == 4 && NEW) MX_ROW4(MX_ZERO, MX_A64);
  else if constexpr (N == 4) MX_ROW4(MX_KEEP, MX_A64);
  else if constexpr (NEW) MX_ROW2(MX_ZERO);
  else MX_ROW2(MX_KEEP);
}
template <int N> __device__ __forceinline__ void settle() {
  if constexpr (N == 8) asm volatile("s_nop 15\n\ts_nop 15" ::: "memory", MX_A256);
  else if constexpr (N == 4) asm volatile("s_nop 15\n\ts_nop 15" ::: "memory", MX_A64);
  else asm volatile("s_nop 15\n\ts_nop 15" ::: "memory", MX_A16);
}
#define MX_READ(CLOBBER)                                                                                               \
  asm volatile("v_accvgpr_read_b32 %0, a[%4]\n\tv_accvgpr_read_b32 %1, a[%5]\n\tv_accvgpr_read_b32 %2, a[%6]\n\t"     \
               "v_accvgpr_read_b32 %3, a[%7]" : "=v"(v0), "=v"(v1), "=v"(v2), "=v"(v3)                                 \
               : "n"(4 * I), "n"(4 * I + 1), "n"(4 * I + 2), "n"(4 * I + 3) : CLOBBER)
template <int N, int I> __device__ __forceinline__ f32x4 sum_of() {
  float v0, v1, v2, v3;
  if constexpr (N == 8) MX_READ(MX_A256);
  else if constexpr (N == 4) MX_READ(MX_A64);
  else MX_READ(MX_A16);
  return f32x4{v0, v1, v2, v3};
}

typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef _Float16 f16x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef __bf16 bf16x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef _Float16 f16x8_u __attribute__((ext_vector_type(8), aligned(2)));
typedef __bf16 bf16x8_u __attribute__((ext_vector_type(8), aligned(2)));
template <int T> struct Elem;
template <> struct Elem<G_F32> { typedef float one; typedef f32x4_u four; };
template <> struct Elem<G_F16> { typedef _Float16 one; typedef f16x4_u four; typedef f16x8_u eight; };
template <> struct Elem<G_BF16> { typedef __bf16 one; typedef bf16x4_u four; typedef bf16x8_u eight; };

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
// Operands straight from memory to registers: 16 rows of a panel are one contiguous KB. Eight waves, each
// with four panels sent for at once, since all there is to do is to read B once: 16 x 11904, k = 3968,
// 25.5 MB in 5.5 us (4.6 TB/s). Every workgroup reads all of A, which bounds it from 48 rows on.
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
// 256 x 256: a wave's 128 x 128 use each fragment for 8 MFMAs, so they read a quarter less from LDS than eight
// waves' 64 x 128 (20480 x 15872, k = 3968, in first versions: 883 and 690 us); their sums fill the
// accumulation registers, so one workgroup fits a CU.
// 128 x 128 (two a CU) and 64 x 64 (four) for what leaves CUs without work: a stage of theirs takes 0.25 and
// 0.11 to 0.13 us, so for the same area 1.25 and 2.2 times as long. 128 x 256 gained nothing on either (3968 x
// 1488, k = 20480: 75 and 77 us).
template <int T> struct Tile {
  static constexpr int WAVES = 4;                            // 2 along i, 2 along j
  static constexpr int S = T / 2, N = S / 16;                // a wave's side, in rows and in MFMA tiles
  static constexpr int CODES = T * kMxRowBytes;              // bytes of an operand's stage
  static constexpr int SCALES = T / kMxGroup * kMxGroupBytes;
  static constexpr int STAGE = 2 * (CODES + SCALES);
  static constexpr int LOADS = 2 * CODES / 1024 / WAVES;     // 1 KB loads of codes per wave and stage
  static constexpr int WORDS = 2 * SCALES / 256;             // 256-byte loads of exponents per stage
  static constexpr int SLOADS = (WORDS + WAVES - 1) / WAVES; // per wave (some of them twice where a wave has none of its own)
};

__device__ __forceinline__ void load_lds4(const GLOBAL uint8_t* base, uint32_t off, uint32_t l) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(l), "v"(off), "s"(base) : "m0", "memory");
}

// Which row of P's 64 is row c of MFMA tile x. A lane's results are rows 4 g .. 4 g + 3 of each tile; with
// PAIRS tiles 2 x and 2 x + 1 give it 8 columns of C in a row, 16 bytes of a 16-bit output, and the four g
// of a row 64.
template <bool PAIRS> __device__ __forceinline__ int p_row(int x, int c) {
  return PAIRS ? 32 * (x >> 1) + 8 * (c >> 2) + 4 * (x & 1) + (c & 3) : 16 * x + c;
}
// Place of a row's 16-byte unit q: 8 lanes of one LDS pass, rows of 64 bytes, on 8 distinct places.
template <bool PAIRS> __device__ __forceinline__ int p_place(int row, int q) {
  return q ^ (PAIRS ? (row >> 1 & 1) | (row >> 2 & 2) : row >> 1 & 3);
}
__device__ __forceinline__ int q_place(int row, int q) { return q ^ (row >> 1 & 3); }

// Workgroups stay: each takes items (a tile, or a part of one's panels) off its XCD's range until there
// are none. Stages of one panel go straight from L2 to a ring of four LDS buffers (the global addresses
// carry the places), three stages ahead of their use and on into the next item's. While a stage is
// multiplied out of registers, the fragments of the next one are read from LDS into the other set and
// the one after three more is sent for, a few between the rows of MFMAs. One barrier a stage: it says
// that the next stage has landed for every wave and that every wave has read this one out of the
// buffer that is then loaded into. An item's results leave while the next one's stages arrive.
template <int T, int OT, bool SPLIT>
__global__ __launch_bounds__(Tile<T>::WAVES * kWave, T == 256 ? 1 : 2)
void k_mx_gemm(MxProduct a, int items) {
  using TL = Tile<T>;
  constexpr int N = TL::N;
  constexpr bool PAIRS = OT != G_F32;
  const int lane = threadIdx.x & (kWave - 1), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int ti = (int)((a.n + T - 1) / T), tj = (int)((a.m + T - 1) / T), tiles = ti * tj;
  const int per_xcd = (items + kXcds - 1) / kXcds, slots = gridDim.x / kXcds;     // the grid is a multiple of 8
  const int range = (int)(blockIdx.x & (kXcds - 1)) * per_xcd, end = min(per_xcd, items - range);
  const int wi0 = (wv >> 1) * TL::S, wj0 = (wv & 1) * TL::S;

  struct Item { int64_t i0, j0; int split, first, stages; };
  // neighbours in the list share operands: strips of 4 tiles of rows
  auto locate = [&](int slot) {
    const int item = range + slot, split = item / tiles, tile = item - split * tiles;
    const int strip = tile / (4 * ti), in = tile - strip * 4 * ti, high = min(tj - 4 * strip, 4);
    const int first = split * a.per;
    return Item{(int64_t)(in / high) * T, (int64_t)(4 * strip + in % high) * T, split, first, min((int)a.p.panels - first, a.per)};
  };
  int slot = (int)(blockIdx.x / kXcds);
  if (slot >= end) return;

  __shared__ __attribute__((aligned(16))) uint8_t lds[RING][TL::STAGE];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(LDS uint8_t*)&lds[0][0];
  // ---- sending for stages: half of the waves load P, the others Q; rows past a matrix read its last -----
  const bool wq = wv >= TL::WAVES / 2;
  const MxView& mv = wq ? a.q : a.p;
  const int64_t step = mv.rows * kMxRowBytes, sstep = mv.groups * kMxGroupBytes;
  const GLOBAL uint8_t* codes;
  const GLOBAL uint8_t* scales;
  uint32_t off[TL::LOADS], soff[TL::SLOADS];
  const uint32_t lcodes = lds0 + (wq ? TL::CODES : 0) + (wv & 1) * TL::LOADS * 1024;
  const uint32_t lscales = lds0 + 2 * TL::CODES + (wq ? TL::SCALES : 0);
  int send_slot = slot, send_left, ahead = 0;
  uint32_t send_to = 0;                                      // its buffer
  auto aim = [&] {                                           // at the first stage of the item in send_slot
    const Item it = locate(send_slot);
    const int64_t t0 = wq ? it.j0 : it.i0;
    codes = gbl(mv.codes) + it.first * step;
    scales = gbl(mv.scales) + it.first * sstep;
    send_left = it.stages;
    const int left = (int)min(mv.rows - t0 - 1, (int64_t)T);
#pragma unroll
    for (int x = 0; x < TL::LOADS; ++x) {
      const int r = ((wv & 1) * TL::LOADS + x) * 16 + (lane >> 2);
      off[x] = (uint32_t)((int)t0 + min(r, left)) * kMxRowBytes + 16 * (wq ? q_place(r, lane & 3) : p_place<PAIRS>(r, lane & 3));
    }
#pragma unroll
    for (int x = 0; x < TL::SLOADS; ++x) {
      const int grp = (int)(t0 / kMxGroup) + ((wv & 1) * TL::SLOADS + x) % (TL::WORDS / 2);
      soff[x] = (uint32_t)min(grp, (int)mv.groups - 1) * kMxGroupBytes + 4 * lane;
    }
  };
  constexpr int PER = TL::LOADS + TL::SLOADS;
  // loads x = 0 .. PER - 1 of the next stage, and then sent()
  auto send = [&](int x) {
    if (x < TL::LOADS) {
      load_lds16(gcast<uint16_t>(codes), off[x], send_to + lcodes + x * 1024);
    } else {
      const int id = ((wv & 1) * TL::SLOADS + x - TL::LOADS) % (TL::WORDS / 2);
      load_lds4(scales, soff[x - TL::LOADS], send_to + lscales + id * 256);
    }
  };
  auto sent = [&] {
    send_to = send_to == (RING - 1) * TL::STAGE ? 0 : send_to + TL::STAGE;
    codes += step;
    scales += sstep;
  };
  auto sent_one = [&] {                                      // and on to the next item
    sent();
    ++ahead;
    if (--send_left > 0) return;
    send_slot += slots;
    if (send_slot < end) aim();
  };
  auto more = [&] { return send_slot < end; };

  // ---- fragments ---------------------------------------------------------------------------------------
  // words of exponents of 64 rows: with PAIRS a lane's rows have two places in them and a byte of its own
  constexpr int KP = (N + 3) / 4 * (PAIRS ? 2 : 1), KQ = (N + 3) / 4;
  struct Frag { u32x4 p[N], q[N]; uint32_t sp[KP], sq[KQ]; };
  const int pshift = (PAIRS ? 8 * (c >> 3) : 0) + wi0 % kMxGroup / 2;   // 16 rows a byte
  const int prow = wi0 + p_row<PAIRS>(0, c), qrow = wj0 + c;
  const uint32_t plane = lds0 + prow * kMxRowBytes + 16 * p_place<PAIRS>(prow, g);
  const uint32_t qlane = lds0 + TL::CODES + qrow * kMxRowBytes + 16 * q_place(qrow, g);
  const uint32_t splane = lds0 + 2 * TL::CODES + wi0 / kMxGroup * kMxGroupBytes + 4 * (PAIRS ? 16 * g + 8 * (c >> 2 & 1) + (c & 3) : lane);
  const uint32_t sqlane = lds0 + 2 * TL::CODES + TL::SCALES + wj0 / kMxGroup * kMxGroupBytes + 4 * lane;
  uint32_t read_from = 0;                                    // buffer of the stage to be read next
  auto ld4 = [](uint32_t at) { return *(const LDS u32x4*)(uintptr_t)at; };
  auto ld1 = [](uint32_t at) { return *(const LDS uint32_t*)(uintptr_t)at; };
  // a lane's first addresses, as asm: the compiler would give every read one of its own
  auto at = [&](uint32_t lane_part) {
    uint32_t v;
    asm("v_add_u32 %0, %1, %2" : "=v"(v) : "s"(read_from), "v"(lane_part));
    return v;
  };
  // reads of a stage: 0 the exponents, then p and q in turn
  constexpr int READS = 2 * N + 1;
  struct Places { uint32_t p, q, sp, sq; };
  auto read = [&](Frag& f, const Places& b, int i) {
    if (i == 0) {
#pragma unroll
      for (int x = 0; x < KP; ++x) f.sp[x] = ld1(b.sp + (PAIRS ? x / 2 : x) * kMxGroupBytes + (PAIRS ? 16 * (x & 1) : 0));
#pragma unroll
      for (int x = 0; x < KQ; ++x) f.sq[x] = ld1(b.sq + x * kMxGroupBytes);
    } else if (i & 1) {
      const int x = i / 2;
      f.p[x] = ld4(b.p + (64 * (x / 4) + p_row<PAIRS>(x & 3, 0)) * kMxRowBytes);
    } else {
      f.q[i / 2 - 1] = ld4(b.q + 16 * (i / 2 - 1) * kMxRowBytes);
    }
  };
  auto read_done = [&] { read_from = read_from == (RING - 1) * TL::STAGE ? 0 : read_from + TL::STAGE; };

  // ---- a stage -------------------------------------------------------------------------------------------
  // Stores of a whole tile's results, all younger than the stages that are then under way. Three stages
  // later every stage waited for is younger than they are.
  constexpr int STORES = N * N / 2;
  constexpr bool LATE = PAIRS && 2 * PER + STORES <= 63;
  int late = 0;
  // Before a stage (`now`) is multiplied: its fragments are there, the next stage has landed, and every
  // wave is this far. ahead: stages sent for and not multiplied, this one among them.
  // STEADY: four stages ahead, nothing late.
  auto turn = [&](Frag& now, auto steady) {
    if (decltype(steady)::value || (ahead >= 4 && late == 0)) {
      wait_loads<2 * PER>();
    } else if (ahead >= 4) {
      wait_loads<LATE ? 2 * PER + STORES : 0>();
      --late;
    } else if (ahead == 3) {
      wait_loads<PER>();
    } else {
      wait_loads<0>();
    }
    if (PAIRS || TL::S < kMxGroup) {
#pragma unroll
      for (int x = 0; x < KP; ++x) now.sp[x] >>= pshift;
    }
    if (TL::S < kMxGroup) {
#pragma unroll
      for (int x = 0; x < KQ; ++x) now.sq[x] >>= wj0 % kMxGroup / 2;
    }
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 3\n\ts_barrier" ::: "memory");      // the shifts are written before an MFMA reads them
    __builtin_amdgcn_sched_barrier(0);
  };
  // Reads over the first three quarters of the MFMAs, loads over the second half, one or two ahead of four
  // MFMAs: more at once wait for the LDS, and the matrix pipe with them. Behind the last stage the reads
  // fetch what nobody uses.
  auto mul = [&](Frag& now, Frag& next, auto fresh, auto steady) {
    constexpr int STEPS = N == 8 ? 16 : N, RSTEPS = N == 8 ? 12 : N == 4 ? 3 : 1, LFIRST = STEPS / 2, LSTEPS = STEPS - LFIRST;
    const bool sends = decltype(steady)::value || more();
    const Places b{at(plane), at(qlane), at(splane), at(sqlane)};
    each<STEPS>([&](auto hh) {
      constexpr int H = decltype(hh)::value, X = N == 8 ? H / 2 : H, Y = N == 8 ? 4 * (H & 1) : 0;
#pragma unroll
      for (int i = H * READS / RSTEPS; i < (H + 1) * READS / RSTEPS && i < READS; ++i) read(next, b, i);
      if constexpr (H >= LFIRST) {
        if (sends) {
#pragma unroll
          for (int x = (H - LFIRST) * PER / LSTEPS; x < (H - LFIRST + 1) * PER / LSTEPS; ++x) send(x);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      constexpr int BP = PAIRS ? 2 * (X >> 1 & 1) : X & 3, WP = PAIRS ? 2 * (X / 4) + (X & 1) : X / 4;
      mfma_row<N, X * N, Y, BP, decltype(fresh)::value>(now.p[X], now.q, now.sp[WP], now.sq);
      __builtin_amdgcn_sched_barrier(0);
    });
    read_done();
    if (decltype(steady)::value) {
      sent();
    } else {
      if (sends) sent_one();
      --ahead;
    }
  };

  // ---- results -------------------------------------------------------------------------------------------
  const float scale = !SPLIT && a.scale ? *a.scale : 1.0f;
  auto results = [&](const Item& it) {
    settle<N>();
    const int64_t i0 = it.i0 + wi0, j0 = it.j0 + wj0;
    if constexpr (SPLIT) {
      GLOBAL float* o = gbl(a.partial) + ((int64_t)it.split * a.m + j0 + c) * a.n + i0 + 4 * g;
      const int rows = (int)min(a.m - j0 - c, (int64_t)T), cols = (int)min(a.n - i0 - 4 * g, (int64_t)T);   // from this lane's first on
      each<N>([&](auto yy) {
        constexpr int Y = decltype(yy)::value;
        each<N>([&](auto xx) {
          constexpr int X = decltype(xx)::value;
          const f32x4 v = sum_of<N, X * N + Y>();
          if (16 * Y < rows && 16 * X < cols) {
            if (16 * X + 4 <= cols) *gcast<f32x4_u>(o + 16 * X) = v;
            else
#pragma unroll
              for (int t = 0; t < 3; ++t)
                if (16 * X + t < cols) o[16 * X + t] = v[t];
          }
        });
        o += 16 * a.n;
      });
    } else if constexpr (PAIRS) {
      typedef typename Elem<OT>::one one;
      typedef typename Elem<OT>::eight eight;
      GLOBAL one* o = gbl(static_cast<one*>(a.c)) + (j0 + c) * a.ldc + i0 + 8 * g;
      const int rows = (int)min(a.m - j0 - c, (int64_t)T), cols = (int)min(a.n - i0 - 8 * g, (int64_t)T);
      const bool eights = (a.n & 7) == 0;
      if (it.i0 + T <= a.n && it.j0 + T <= a.m && eights) late = 3;
      each<N>([&](auto yy) {
        constexpr int Y = decltype(yy)::value;
        each<N / 2>([&](auto xx) {
          constexpr int X = 2 * decltype(xx)::value;
          const f32x4 v = sum_of<N, X * N + Y>() * scale, w = sum_of<N, (X + 1) * N + Y>() * scale;
          const eight u = __builtin_convertvector(f32x8{v[0], v[1], v[2], v[3], w[0], w[1], w[2], w[3]}, eight);
          if (16 * Y < rows && 16 * X < cols) {
            if (eights || 16 * X + 8 <= cols) {
              *gcast<eight>(o + 16 * X) = u;
            } else {
#pragma unroll
              for (int t = 0; t < 8; ++t)
                if (16 * X + t < cols) o[16 * X + t] = u[t];
            }
          }
        });
        o += 16 * a.ldc;
      });
    } else if (it.i0 + T <= a.n && it.j0 + T <= a.m) {
      GLOBAL float* o = gbl(static_cast<float*>(a.c)) + (j0 + c) * a.ldc + i0 + 4 * g;
      f32x4 old[2][N];                                       // of this row of tiles and the next: their way takes longer than the rest
      auto get = [&](int y) {
#pragma unroll
        for (int x = 0; x < N; ++x) old[y & 1][x] = *gcast<f32x4_u>(o + 16 * y * a.ldc + 16 * x);
      };
#pragma unroll
      for (int x = 0; x < 2 * N; ++x) old[x / N][x % N] = f32x4{0, 0, 0, 0};
      if (a.accumulate) get(0);
      each<N>([&](auto yy) {
        constexpr int Y = decltype(yy)::value;
        if (Y + 1 < N && a.accumulate) get(Y + 1);
        __builtin_amdgcn_sched_barrier(0);
        each<N>([&](auto xx) {
          constexpr int X = decltype(xx)::value;
          *gcast<f32x4_u>(o + 16 * Y * a.ldc + 16 * X) = sum_of<N, X * N + Y>() * scale + old[Y & 1][X];
        });
      });
    } else {
      each<N>([&](auto yy) {
        constexpr int Y = decltype(yy)::value;
        each<N>([&](auto xx) {
          constexpr int X = decltype(xx)::value;
          finish<OT>(a, j0 + 16 * Y + c, i0 + 16 * X + 4 * g, sum_of<N, X * N + Y>(), scale);
        });
      });
    }
  };

  aim();
  for (int j = 0; j < RING; ++j)
    if (more()) {
#pragma unroll
      for (int x = 0; x < PER; ++x) send(x);
      sent_one();
    }
  if (ahead == 4) wait_loads<3 * PER>();
  else wait_loads<0>();
  __builtin_amdgcn_s_barrier();
  Frag f0, f1;
  {
    const Places b{at(plane), at(qlane), at(splane), at(sqlane)};
#pragma unroll
    for (int i = 0; i < READS; ++i) read(f0, b, i);
  }
  read_done();
  Item it = locate(slot);
  bool fresh = true;
  // one stage; false behind the last
  auto stage = [&](Frag& now, Frag& next) {
    using No = std::false_type;
    turn(now, No{});
    if (fresh) mul(now, next, std::true_type{}, No{});
    else mul(now, next, No{}, No{});
    fresh = --it.stages == 0;
    if (!fresh) return true;
    results(it);
    slot += slots;
    if (slot >= end) return false;
    it = locate(slot);
    return true;
  };
  // Most stages pass through a loop without choices: with one wave a SIMD nothing else runs while a wave
  // branches.
  do {
    if (!fresh && ahead == 4 && late == 0 && more()) {
      using Yes = std::true_type;
      const int twos = (min(send_left, it.stages) - 1) / 2;
      send_left -= 2 * twos;
      it.stages -= 2 * twos;
      for (int x = 0; x < twos; ++x) {
        turn(f0, Yes{});
        mul(f0, f1, std::false_type{}, Yes{});
        turn(f1, Yes{});
        mul(f1, f0, std::false_type{}, Yes{});
      }
    }
  } while (stage(f0, f1) && stage(f1, f0));
}

// The parts of a split product, added in order; of none, zeros.
template <int OT>
__global__ __launch_bounds__(256)
void k_mx_join(MxProduct a) {
  const int64_t blocks = (a.n + 1023) / 1024, step = a.m * a.n;
  const int parts = a.p.panels > 0 ? a.splits : 0;
  const float scale = a.scale ? *a.scale : 1.0f;
  for (int64_t block = blockIdx.x; block < blocks * a.m; block += gridDim.x) {
    const int64_t j = block / blocks, i = 4 * ((block - j * blocks) * 256 + threadIdx.x);
    if (i >= a.n) continue;
    const GLOBAL float* p = gbl(a.partial) + j * a.n + i;
    f32x4 sum{0, 0, 0, 0};
    if (i + 4 <= a.n) {
      for (int s = 0; s < parts; ++s) sum += *gcast<f32x4_u>(p + s * step);
    } else {
      for (int s = 0; s < parts; ++s)
        for (int t = 0; t < 4; ++t)
          if (i + t < a.n) sum[t] += p[s * step + t];
    }
    finish<OT>(a, j, i, sum, scale);
  }
}

template <int T, int OT>
hipError_t go_tiles(const MxProduct& a, hipStream_t s) {
  const int64_t items = ((a.n + T - 1) / T) * ((a.m + T - 1) / T) * a.splits;
  constexpr int64_t fit = 256 * (T == 256 ? 1 : T == 128 ? 2 : 4);            // what 256 CUs hold
  const dim3 grid((unsigned)std::min<int64_t>((items + kXcds - 1) / kXcds * kXcds, fit)), block(Tile<T>::WAVES * kWave);
  if (a.splits == 1) k_mx_gemm<T, OT, false><<<grid, block, 0, s>>>(a, (int)items);
  else k_mx_gemm<T, G_F32, true><<<grid, block, 0, s>>>(a, (int)items);
  return hipGetLastError();
}
template <int OT>
hipError_t go_join(const MxProduct& a, hipStream_t s) {
  const int64_t blocks = (a.n + 1023) / 1024 * a.m;
  k_mx_join<OT><<<dim3((unsigned)std::min<int64_t>(blocks, 1 << 20)), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}
template <int OT>
hipError_t go(const MxProduct& a, int tile, hipStream_t s) {
  if (a.p.panels == 0) return go_join<OT>(a, s);                              // no parts: zeros
  if (tile != 0) {
    const hipError_t e = tile == 256 ? go_tiles<256, OT>(a, s) : tile == 128 ? go_tiles<128, OT>(a, s) : go_tiles<64, OT>(a, s);
    return e != hipSuccess || a.splits == 1 ? e : go_join<OT>(a, s);
  }
  const dim3 grid((unsigned)((a.n + 15) / 16)), block(kFewWaves * kWave);
  if (a.m <= 16) k_mx_few<1, OT><<<grid, block, 0, s>>>(a);
  else if (a.m <= 32) k_mx_few<2, OT><<<grid, block, 0, s>>>(a);
  else k_mx_few<4, OT><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

// Kernel, tiles and parts by a sum of what they cost, in microseconds: a launch that ends with one tile's
// results, stages of the CU with most tiles, and the parts' way through memory; for few rows a launch, and
// what its workgroups read at the rate of the L2s, or one workgroup's way through all panels where that takes
// longer. Measured, tiles of 256 / 128 / 64:
//   1280 x 1984, k = 3968    28.3 / 13.8 / 14.1     512 x 4096, k = 4096      27.9 / 13.4 / 11.5
//   2048 x 2048, k = 2048    19.6 / 10.6 / 12.4     4096 x 4096, k = 4096     40.6 / 49.0 / 69.0
//   20480 x 1984, k = 3968   88.5 / 95.3 / 144      20480 x 15872, k = 3968    601 /  726 / 1170
// in two parts 1280 x 1984, k = 3968: 33.3 / 23.8 / 22.6; 3968 x 1488, k = 20480: 104 / 77.6 / 103 whole,
// 79.6 / 84.1 / 118 in two parts; few rows / tiles of 64, 64 x 1984, k = 3968: 4.9 / 8.3; 64 x 11904: 11.8 / 9.0;
// 16 x 11904: 5.5 / 8.6; 1 x 32768, k = 4096: 18.0 / 14.0; few rows / tiles of 64 in eight parts, 64 x 64, k = 8192:
// 7.6 / 9.8; 20480: 14.3 / 11.3; 81920: 48 / 19; 327680: 295 / 49; 16 x 64, k = 40960: 12.3 / 13.8; 81920: 22 / 18.
MxPlan mx_plan(int64_t m, int64_t n, int64_t panels) {
  static constexpr struct { int tile; double start, stage; } kinds[] = {{64, 4.9, 0.11}, {128, 4.8, 0.27}, {256, 8.3, 0.80}};
  MxPlan best{0, 1};
  double least = -1;
  if (m <= 64) {
    const int64_t high = (m + 15) / 16, held = high > 2 ? 4 : high;      // MFMA tiles that exist, and that are multiplied
    least = 2.6 + std::max((double)((n + 15) / 16) * (double)((high + 1) * panels) * 16 * kMxRowBytes / 13e6,
                           (double)panels * (0.017 + 0.014 * (double)held));
  }
  for (const auto& k : kinds) {
    const int64_t tiles = ((m + k.tile - 1) / k.tile) * ((n + k.tile - 1) / k.tile);
    for (int splits = 1; splits <= 8 && (splits == 1 || panels / splits >= 8); splits *= 2) {
      double cost = k.start + (double)((tiles * splits + 255) / 256) * (double)((panels + splits - 1) / splits) * k.stage;
      if (splits > 1) cost += 4.0 + 8.0 * (double)m * (double)n * splits / 2.9e6;
      if (least < 0 || cost < least) {
        least = cost;
        best = {k.tile, splits};
      }
    }
  }
  return best;
}

hipError_t launch_mx_product(const MxProduct& a, int tile, int ot, hipStream_t s) {
  if (ot == G_F32) return go<G_F32>(a, tile, s);
  if (ot == G_F16) return go<G_F16>(a, tile, s);
  return go<G_BF16>(a, tile, s);
}

}  // namespace psgd
