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
// out 3% off, against 0.15%). The accurate products use both halves of every factor
// (hi hi + hi lo + lo hi): the result's error, 1e-6 to 5e-6 of its norm, is that of fp32 products.
//
// Measured. Four resblock shards (s 496..1984, l 3968), fast: A 181 us, B 106, update 350; the
// unsharded resblock (s 3968, l up to 15872): A 596, B 243, update 1256, 1.2 PFLOP/s.
// One resblock shard, accurate: A 135, B 75, update 255. Large groups run at the chip's power limit,
// 82% of what a large library product reaches; small ones (496 x 3968: 5 to 8 us a launch) wait for
// their first loads.
#include <type_traits>

#include "lds_load.h"
#include "ns.h"

namespace psgd {
namespace {

constexpr int KB = 32;                         // k per stage
constexpr int RING = 4;                        // stages in LDS

typedef short i16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i16x4 lds_read_tr16(const uint16_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)(p));
}

// A stage of P read K-outer is 32 x 32 blocks, 64 bytes per k. A transposing read touches 32 bytes
// in each of the rows k = 8 g + t (+ 4): the rows of lanes 0..31 (g = 0, 1; t = 0..3) and those of
// lanes 32..63 each have to land on 8 distinct 32-byte groups of the 256 bytes of banks, so the two
// 32-byte halves of a row change places with every 8 k.
__device__ __forceinline__ int swz_outer(int k, int q) { return q ^ (((k >> 3) & 1) << 1); }
// K-contiguous rows are 64 bytes (4 units): 8 consecutive rows put one logical unit on the 8
// distinct 16-byte groups of one LDS pass.
__device__ __forceinline__ int swz_inner(int row, int q) { return q ^ ((row >> 1) & 3); }

__device__ __forceinline__ float h2f(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
__device__ __forceinline__ f32x4 h2f4(u32x2 v) { return __builtin_convertvector(__builtin_bit_cast(f16x4, v), f32x4); }
__device__ __forceinline__ u32x2 f2h4(f32x4 v) { return __builtin_bit_cast(u32x2, __builtin_convertvector(v, f16x4)); }

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

template <int OT> __device__ __forceinline__ f32x4 out_load4(const void* p, int64_t i) {
  if constexpr (OT == G_F32) return *gcast<f32x4>(gbl(static_cast<const float*>(p)) + i);
  else return GradIO<OT>::load4(gcast<char>(gbl(static_cast<const uint16_t*>(p)) + i));
}
template <int OT> __device__ __forceinline__ void out_store4(void* p, int64_t i, f32x4 v) {
  if constexpr (OT == G_F32) *gcast<f32x4>(gbl(static_cast<float*>(p)) + i) = v;
  else if constexpr (OT == G_F16) *gcast<u32x2>(gbl(static_cast<uint16_t*>(p)) + i) = f2h4(v);
  else *gcast<u32x2>(gbl(static_cast<uint16_t*>(p)) + i) = __builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4));
}

template <int T> struct Tile {
  static constexpr int WAVES = T == 256 ? 8 : 4;
  static constexpr int THREADS = WAVES * kWave;
  static constexpr int WN = T == 256 ? 4 : 2;              // waves along j; 2 along i
  static constexpr int TA = T / 32, TB = T / (16 * WN);    // 16-wide MFMA tiles per wave along i, j
  static constexpr int BYTES = T * KB * 2;                 // one operand's stage
  static constexpr int LOADS = 2 * BYTES / (WAVES * 1024); // 1 KB loads per wave and stage
};

// ST: stage. T: C tile side. ACC: accurate products. OT: 0, or the output type of the last update.
// MFMA layout: operand P gives the rows i of a C tile, Q the columns j; a lane holds C[4 g .. 4 g
// + 3][c], four consecutive i. For the update i runs along l and j along s, so those four are
// consecutive in memory.
//
// Main loop. Stages of 32 k go straight from L2 to a ring of four LDS buffers (16 bytes per lane,
// the global addresses carry the swizzle), three stages ahead of their use. While stage j is
// multiplied out of registers, the fragments of stage j + 1 are read from LDS into the other set,
// so the MFMAs after a barrier depend on nothing younger than it. One barrier per stage: it
// says that stage j + 1 has landed for every wave and that every wave has read stage j out of the
// buffer that stage j + 4 is then loaded into. Accurate products take the hi and the lo plane of
// 32 k as two stages: hi hi in the first, lo hi + hi lo in the second.
//
// Split items. A tile whose K is cut into wi.b & 63 parts leaves part wi.a & 63 as raw fp32
// accumulators in slot wi.c of `partial`; the launch with REDUCE adds a tile's slots wi.c, wi.c + 1,
// ... in order and runs the epilogue, each wave of the tile as a workgroup of its own.
template <int ST, int T, bool ACC, int OT, bool REDUCE>
__global__ __launch_bounds__(REDUCE ? kWave : Tile<T>::THREADS, 2)
void k_ns_gemm(const NsItem* __restrict__ items, float* __restrict__ partial, int step, NsArgs na)
{
  using TL = Tile<T>;
  constexpr int PER = REDUCE ? TL::WAVES : 1;  // workgroups per item: the sums' waves are on their own
  const int item = xcd_remap(blockIdx.x, gridDim.x);
  const Work wi = items[item / PER].w;
  const NsMat& d = items[item / PER].d;
  constexpr bool OUTER = ST == NS_UPDATE;      // P is read K-outer
  const int cur = step & 1;
  const int i0 = wi.a & ~63, j0 = wi.b & ~63, split = wi.a & 63, splits = wi.b & 63;
  const int lane = threadIdx.x & (kWave - 1), wv = REDUCE ? item % PER : __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wv & 1, wn = wv >> 1;
  const int wi0 = wm * (T / 2), wj0 = wn * (T / TL::WN);
  const int c = lane & 15, g = lane >> 4;

  const GLOBAL uint16_t *ph, *pl, *qh, *ql;
  if constexpr (ST == NS_GRAM) {
    ph = qh = gbl(d.xh[cur]); pl = ql = gbl(d.xl[cur]);
  } else if constexpr (ST == NS_POLY) {
    ph = qh = gbl(d.ah); pl = ql = gbl(d.al);
  } else {
    ph = gbl(d.xh[cur]); pl = gbl(d.xl[cur]);
    qh = gbl(d.bh); ql = gbl(d.bl);
  }
  const int K = ST == NS_GRAM ? d.l : d.s;
  const int64_t panel = (int64_t)d.sp * KB;    // elements from one panel of 32 columns to the next
  const int skip = *na.skip;
  // all of these loads are under way together before the first is looked at
  asm volatile("" ::"s"(ph), "s"(pl), "s"(qh), "s"(ql), "s"(K), "s"(panel), "s"(skip), "s"(wi.mat));
  if (skip != 0 || wi.mat < 0) return;
  // whole pairs of 32 k (the padding up to a tile holds zeros); accurate: two stages per 32 k
  int nst = ns_stages(K, ACC);
  int k0 = 0;                                  // first k of this part
  if (splits > 1) {
    const int per = ns_part(nst, splits, ACC), first = split * per;
    nst = min(per, nst - first);
    k0 = first * (ACC ? KB / 2 : KB);
  }

  __shared__ __attribute__((aligned(16))) uint16_t lds[RING][TL::BYTES / PER];   // P, then Q
  const uint32_t lds0 = (uint32_t)(uintptr_t)(LDS uint16_t*)&lds[0][0];
  // this wave's loads of a stage: load x < PL is 1 KB of P, the others of Q
  constexpr int PL = TL::LOADS / 2;
  uint32_t poff[PL], qoff[PL];
  const int64_t pfirst = OUTER ? i0 / KB * panel + k0 * KB : k0 / KB * panel + i0 * KB, qfirst = k0 / KB * panel + j0 * KB;
  const int64_t pstage = OUTER ? KB * KB : panel;             // elements from stage to stage
  const GLOBAL uint16_t* const pbase_h = ph + pfirst;
  const GLOBAL uint16_t* const qbase_h = qh + qfirst;
  const GLOBAL uint16_t* const pbase_l = pl + pfirst;
  const GLOBAL uint16_t* const qbase_l = ql + qfirst;
#pragma unroll
  for (int x = 0; x < PL; ++x) {
    const int e = (wv * PL + x) * kWave + lane;              // 16-byte slot of the operand's stage
    const int r = e >> 2;                                    // its row: 64 bytes, contiguous with the next
    qoff[x] = (uint32_t)(r * KB + 8 * swz_inner(r, e & 3)) * 2u;
    if constexpr (OUTER) poff[x] = (uint32_t)((r / KB) * panel + (r % KB) * KB + 8 * swz_outer(r % KB, e & 3)) * 2u;
    else poff[x] = qoff[x];
  }
  // load x of stage j: P and Q in turn
  auto load_part = [&](int j, int x) {
    const int ks = ACC ? j >> 1 : j;
    const uint32_t l = lds0 + (uint32_t)(j % RING) * (2 * TL::BYTES) + wv * (PL * 1024) + (x >> 1) * 1024;
    if (x & 1) load_lds16((ACC && (j & 1) ? qbase_l : qbase_h) + ks * panel, qoff[x >> 1], l + TL::BYTES);
    else load_lds16((ACC && (j & 1) ? pbase_l : pbase_h) + ks * pstage, poff[x >> 1], l);
  };

  f32x4 acc[TL::TA][TL::TB];
#pragma unroll
  for (int a = 0; a < TL::TA; ++a)
#pragma unroll
    for (int b = 0; b < TL::TB; ++b) acc[a][b] = f32x4{0, 0, 0, 0};

  // hi lo + lo hi: on their own in 64-wide tiles, where the accumulators are few and K short, so that
  // they are not cut to the size of hi hi
  constexpr bool CROSS = ACC && T == 64;
  f32x4 own[CROSS ? TL::TA : 1][CROSS ? TL::TB : 1];
  f32x4 (&cross)[TL::TA][TL::TB] = [&]() -> f32x4 (&)[TL::TA][TL::TB] {
    if constexpr (CROSS) return own; else return acc;
  }();
  if constexpr (CROSS) {
#pragma unroll
    for (int a = 0; a < TL::TA; ++a)
#pragma unroll
      for (int b = 0; b < TL::TB; ++b) own[a][b] = f32x4{0, 0, 0, 0};
  }

  struct Frag { f16x8 p[TL::TA], q[TL::TB]; };
  auto read_p = [&](Frag& f, int j, int a) {
    const uint16_t* lp = lds[j % RING];
    if constexpr (OUTER) {
      const int k = 8 * g + (c >> 2), col = wi0 + 16 * a, u = 2 * ((col / 16) & 1) + ((c & 3) >> 1);
      const uint16_t* s = &lp[col / KB * (KB * KB) + k * KB + 8 * swz_outer(k, u) + 4 * (c & 1)];
      const i16x4 x = lds_read_tr16(s), y = lds_read_tr16(s + 4 * KB);
      f.p[a] = __builtin_bit_cast(f16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const int r = wi0 + 16 * a + c;
      f.p[a] = *reinterpret_cast<const f16x8*>(&lp[r * KB + 8 * swz_inner(r, g)]);
    }
  };
  auto read_q = [&](Frag& f, int j, int b) {
    const uint16_t* lq = lds[j % RING] + TL::BYTES / 2;
    const int r = wj0 + 16 * b + c;
    f.q[b] = *reinterpret_cast<const f16x8*>(&lq[r * KB + 8 * swz_inner(r, g)]);
  };
  // One pass over the wave's MFMA tiles, row by row; `before(a)` is issued ahead of row a's MFMAs
  // and `after(a)` behind them, so that LDS reads and stage loads trickle in between MFMAs that do
  // not depend on them.
  auto mul_to = [&](f32x4 (&to)[TL::TA][TL::TB], const Frag& fp, const Frag& fq, auto before, auto after) {
#pragma unroll
    for (int a = 0; a < TL::TA; ++a) {
      before(a);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int b = 0; b < TL::TB; ++b) to[a][b] = mfma_f16(fp.p[a], fq.q[b], to[a][b]);
      __builtin_amdgcn_sched_barrier(0);
      after(a);
    }
  };
  auto mul = [&](const Frag& fp, const Frag& fq, auto before, auto after) { mul_to(acc, fp, fq, before, after); };
  auto none = [](int) {};
  // stage j's fragments over the first half of the rows, so that the last of them is answered before
  // the wait; the stage loads over the second half
  constexpr int HALF = TL::TA / 2;
  auto read_some = [&](Frag& f, int j, int a) {
    if (a >= HALF) return;
#pragma unroll
    for (int b = a * TL::TB / HALF; b < (a + 1) * TL::TB / HALF; ++b) read_q(f, j, b);
    read_p(f, j, 2 * a);
    read_p(f, j, 2 * a + 1);
  };
  auto send_some = [&](int j, int a) {
    if (a < HALF) return;
#pragma unroll
    for (int x = (a - HALF) * TL::LOADS / HALF; x < (a - HALF + 1) * TL::LOADS / HALF; ++x) load_part(j, x);
  };
  // Before stage j is multiplied: stage j + 1 has landed (BEHIND later stages may still be under
  // way) and nobody reads stage j's buffer any more.
  auto turn = [&](auto behind) {
    wait_loads<decltype(behind)::value * TL::LOADS>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  Frag f0, f1;
  // stages j (even) and j + 1; send: stages j + 4 and j + 5 are sent for; more: stage j + 2 follows
  // and its first fragments are read
  auto pair = [&](int j, auto behind0, auto behind1, auto send, auto more) {
    constexpr bool SEND = decltype(send)::value, MORE = decltype(more)::value;
    turn(behind0);
    mul(f0, f0, [&](int a) {
      read_some(f1, j + 1, a);
      if (SEND) send_some(j + RING, a);
    }, none);
    if constexpr (MORE) turn(behind1);
    if constexpr (ACC) {
      mul_to(cross, f1, f0, [&](int a) { if (SEND) send_some(j + 1 + RING, a); }, none);
      // f0.q is free from here on, and each f0.p[a] behind its last row
      mul_to(cross, f0, f1, [&](int a) { if (MORE && a < TL::TB) read_q(f0, j + 2, a); }, [&](int a) { if (MORE) read_p(f0, j + 2, a); });
    } else {
      mul(f1, f1, [&](int a) {
        if (MORE) read_some(f0, j + 2, a);
        if (SEND) send_some(j + 1 + RING, a);
      }, none);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  using N0 = std::integral_constant<int, 0>;
  using N1 = std::integral_constant<int, 1>;
  using N2 = std::integral_constant<int, 2>;
  using Yes = std::true_type;
  using No = std::false_type;
  auto load_stage = [&](int j) {
#pragma unroll
    for (int x = 0; x < TL::LOADS; ++x) load_part(j, x);
  };

  if constexpr (REDUCE) {
    const GLOBAL f32x4* s = gcast<f32x4>(gbl(partial)) + (int64_t)wi.c * (T * T / 4) + wv * (TL::TA * TL::TB * kWave) + lane;
    auto add_slots = [&](auto count) {                        // loads of several slots at once, added in order
      constexpr int N = decltype(count)::value;
      f32x4 v[N][TL::TA][TL::TB];
#pragma unroll
      for (int x = 0; x < N; ++x)
#pragma unroll
        for (int a = 0; a < TL::TA; ++a)
#pragma unroll
          for (int b = 0; b < TL::TB; ++b) v[x][a][b] = s[x * (T * T / 4) + (a * TL::TB + b) * kWave];
#pragma unroll
      for (int x = 0; x < N; ++x)
#pragma unroll
        for (int a = 0; a < TL::TA; ++a)
#pragma unroll
          for (int b = 0; b < TL::TB; ++b) acc[a][b] += v[x][a][b];
      s += N * (T * T / 4);
    };
    int x = 0;
    constexpr int GO = T == 64 ? 4 : T == 128 ? 2 : 1;
    for (; x + GO <= splits; x += GO) add_slots(std::integral_constant<int, GO>{});
    if constexpr (GO > 1)
      for (; x < splits; ++x) add_slots(N1{});
  } else if constexpr (T == 256) {
    static_assert(!ACC, "128-wide tiles at most: both halves' fragments beside 128 accumulators do not fit");
    // Two waves per SIMD take turns: while waves 0..3 multiply, waves 4..7 read their fragments and
    // send for loads, and the other way round, a barrier between the phases. Each phase's MFMAs
    // find their operands in registers, so the matrix pipe of every SIMD passes from one wave to the
    // other without a gap to fill. Stage j is read in one phase by each half; after both, its
    // buffer is free: stage j + 3 is sent for while stage j is read.
    const bool second = wv >= TL::WAVES / 2;
    auto read_all = [&](Frag& f, int j) {
#pragma unroll
      for (int b = 0; b < TL::TB; ++b) read_q(f, j, b);
#pragma unroll
      for (int a = 0; a < TL::TA; ++a) read_p(f, j, a);
    };
    auto none1 = [](int) {};
    auto phase_read = [&](Frag& f, int j, auto behind, auto send) {
      read_all(f, j);
      if constexpr (decltype(send)::value) load_stage(j + RING - 1);
      wait_loads<decltype(behind)::value * TL::LOADS>();
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
    };
    auto phase_end = [&] {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
    };
    auto two = [&](int j, auto behind0, auto behind1, auto send0, auto send1) {   // stages j (even), j + 1
      phase_read(f0, j, behind0, send0);
      mul(f0, f0, none1, none1);
      phase_end();
      phase_read(f0, j + 1, behind1, send1);
      mul(f0, f0, none1, none1);
      phase_end();
    };
    load_stage(0);
    load_stage(1);
    if (nst > 2) {
      load_stage(2);
      wait_loads<2 * TL::LOADS>();
    } else {
      wait_loads<TL::LOADS>();
    }
    __builtin_amdgcn_s_barrier();
    if (second) __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    int j = 0;
    for (; j + 4 < nst; j += 2) two(j, N2{}, N2{}, Yes{}, Yes{});
    if (nst > 2) {                             // four stages left, the last of them to be sent for
      two(j, N2{}, N1{}, Yes{}, No{});
      j += 2;
    }
    two(j, N0{}, N0{}, No{}, No{});
    if (!second) __builtin_amdgcn_s_barrier();
  } else {
    load_stage(0);
    load_stage(1);
    if (nst > 2) {                               // nst is even
      load_stage(2);
      load_stage(3);
      wait_loads<3 * TL::LOADS>();
    } else {
      wait_loads<TL::LOADS>();
    }
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int b = 0; b < TL::TB; ++b) read_q(f0, 0, b);
#pragma unroll
    for (int a = 0; a < TL::TA; ++a) read_p(f0, 0, a);
    int j = 0;
    if constexpr (ACC) {
      // Every MFMA rounds its accumulator (to nearest even), three times per 32 k here. Every 128 k
      // the chain's sum moves to another one, so that the large sum is rounded once per 128 k: five
      // steps on 1500 x 4096 come out 1.2e-6 off instead of 2.9e-6, positive elements, whose sums
      // round alike, 0.07e-6 instead of 0.4e-6 in one A X.
      f32x4 sum[TL::TA][TL::TB];
#pragma unroll
      for (int a = 0; a < TL::TA; ++a)
#pragma unroll
        for (int b = 0; b < TL::TB; ++b) sum[a][b] = f32x4{0, 0, 0, 0};
      for (int n = 1; j + RING < nst; j += 2, ++n) {
        pair(j, N2{}, N2{}, Yes{}, Yes{});
        if ((n & 3) == 0) {
#pragma unroll
          for (int a = 0; a < TL::TA; ++a)
#pragma unroll
            for (int b = 0; b < TL::TB; ++b) {
              sum[a][b] += acc[a][b];
              acc[a][b] = f32x4{0, 0, 0, 0};
            }
        }
      }
      if (nst > 2) {
        pair(j, N2{}, N1{}, No{}, Yes{});
        j += 2;
      }
      pair(j, N0{}, N0{}, No{}, No{});
#pragma unroll
      for (int a = 0; a < TL::TA; ++a)
#pragma unroll
        for (int b = 0; b < TL::TB; ++b) {
          acc[a][b] += sum[a][b];
          if constexpr (CROSS) acc[a][b] += own[a][b];
        }
    } else {
      for (; j + RING < nst; j += 2) pair(j, N2{}, N2{}, Yes{}, Yes{});
      if (nst > 2) {
        pair(j, N2{}, N1{}, No{}, Yes{});
        j += 2;
      }
      pair(j, N0{}, N0{}, No{}, No{});
    }
  }

  if constexpr (!REDUCE && ST != NS_UPDATE) {
    if (splits > 1) {
      GLOBAL f32x4* s = gcast<f32x4>(gbl(partial)) + (int64_t)wi.c * (T * T / 4) + wv * (TL::TA * TL::TB * kWave) + lane;
#pragma unroll
      for (int a = 0; a < TL::TA; ++a)
#pragma unroll
        for (int b = 0; b < TL::TB; ++b) s[(a * TL::TB + b) * kWave] = acc[a][b];
      return;
    }
  }

  // ---- epilogue --------------------------------------------------------------------------
  // Through this wave's own part of the ring, so that memory sees whole rows, 16 bytes a lane: a
  // lane's accumulators are 8 bytes in each of 16 rows. 16-byte units are XOR-ed by their row, which keeps both sides conflict-free.
  constexpr int WI = T / 2, WJ = T / TL::WN;                 // the wave's tile of C
  __syncthreads();                                           // the ring is read out
  const int part = REDUCE ? 0 : wv * (WI * WJ);
  uint16_t* const reg = &lds[0][0] + part;
  const uint32_t reg0 = lds0 + 2 * part;
  const int ib = i0 + wi0, jb = j0 + wj0;

  // In the workspace's layout: panels of 32 columns, 64 bytes per row, so a wave's tile is a
  // contiguous block per panel.
  auto swz_out = [](int r, int u) { return u ^ ((r >> 2) & 3); };
  // rows j, columns i: a lane's four values are half a unit
  auto at_ji = [&](int a, int b) {
    const int r = 16 * b + c, u = 2 * (a & 1) + (g >> 1);
    return reg + (a >> 1) * (WJ * KB) + r * KB + 8 * swz_out(r, u) + 4 * (g & 1);
  };
  auto fetch = [&](const GLOBAL uint16_t* src) {
    const GLOBAL uint16_t* s = src + ib / KB * panel + jb * KB;
#pragma unroll
    for (int x = 0; x < WI * WJ / 512; ++x) {
      const int e = x * kWave + lane, r = (e >> 2) % WJ;
      load_lds16(s + x * 512 / (WJ * KB) * panel, (uint32_t)(r * KB + 8 * swz_out(r, e & 3)) * 2u, reg0 + x * 1024);
    }
    wait_loads<0>();
  };
  auto add = [&](float f) {                                  // acc += f * fetched, few at a time: no registers to spare
#pragma unroll
    for (int a = 0; a < TL::TA; ++a)
#pragma unroll
      for (int b = 0; b < TL::TB; ++b) {
        __builtin_amdgcn_sched_barrier(0);
        acc[a][b] += f * h2f4(*reinterpret_cast<const u32x2*>(at_ji(a, b)));
      }
    wait_loads<0>();
  };
  // what stands in `reg`, panels of R rows, to rows row.. of the panels from `col` on
  auto send_out = [&](GLOBAL uint16_t* dst, int row, int col, auto rows) {
    constexpr int R = decltype(rows)::value;
    GLOBAL uint16_t* o = dst + col / KB * panel + row * KB;
#pragma unroll
    for (int x = 0; x < WI * WJ / 512; ++x) {
      const int e = x * kWave + lane, r = (e >> 2) % R;
      *gcast<u32x4>(o + x * 512 / (R * KB) * panel + r * KB + 8 * (e & 3)) =
          *reinterpret_cast<const u32x4*>(reg + x * 512 / (R * KB) * (R * KB) + r * KB + 8 * swz_out(r, e & 3));
    }
  };
  // the fp16 of acc (LO: of what rounding to it leaves) to rows j of dst
  auto flush_ji = [&](GLOBAL uint16_t* dst, bool lo) {
#pragma unroll
    for (int a = 0; a < TL::TA; ++a)
#pragma unroll
      for (int b = 0; b < TL::TB; ++b) {
        const u32x2 h = f2h4(acc[a][b]);
        *reinterpret_cast<u32x2*>(at_ji(a, b)) = lo ? f2h4(acc[a][b] - h2f4(h)) : h;
      }
    send_out(dst, jb, ib, std::integral_constant<int, WJ>{});
  };
  // the same to rows i of dst
  auto flush_ij = [&](GLOBAL uint16_t* dst, bool lo) {
#pragma unroll
    for (int a = 0; a < TL::TA; ++a)
#pragma unroll
      for (int b = 0; b < TL::TB; ++b) {
        const u32x2 h = f2h4(acc[a][b]), v = lo ? f2h4(acc[a][b] - h2f4(h)) : h;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int r = 16 * a + 4 * g + t, u = 2 * (b & 1) + (c >> 3);
          reg[(b >> 1) * (WI * KB) + r * KB + 8 * swz_out(r, u) + (c & 7)] = (uint16_t)(v[t >> 1] >> (16 * (t & 1)));
        }
      }
    send_out(dst, ib, jb, std::integral_constant<int, WI>{});
  };
  // Nothing masks the padding. Sums run over whole pairs of 32 k: up to there rows and columns past s
  // and l are products of X0's zeros. What lies further out, up to the wider of two products' tiles,
  // may never have been written and only reaches elements as far out. A NaN in X is in all of X by
  // way of the norm, so the padding may be NaN beside it; the next call writes all of it anew.

  constexpr float kProd = ST == NS_GRAM ? kNsScaleA / (kNsScaleX * kNsScaleX)
                        : ST == NS_POLY ? kNsScaleB / (kNsScaleA * kNsScaleA)
                                        : 1.0f / kNsScaleB;
  const float prod = ST == NS_POLY ? na.c * kProd : kProd;
#pragma unroll
  for (int a = 0; a < TL::TA; ++a)
#pragma unroll
    for (int b = 0; b < TL::TB; ++b) acc[a][b] *= prod;

  if constexpr (ST != NS_UPDATE) {
    if constexpr (ST == NS_POLY) {
      fetch(gbl(d.ah));
      add(na.b * (kNsScaleB / kNsScaleA));
      if constexpr (ACC) {
        fetch(gbl(d.al));
        add(na.b * (kNsScaleB / kNsScaleA));
      } else if (i0 == j0) {
        // the fast form multiplies by a I + B: the hi half of a X comes out of the product
#pragma unroll
        for (int a = 0; a < TL::TA; ++a)
#pragma unroll
          for (int b = 0; b < TL::TB; ++b)
#pragma unroll
            for (int t = 0; t < 4; ++t)
              if (ib + 16 * a + 4 * g + t == jb + 16 * b + c) acc[a][b][t] += na.a * kNsScaleB;
      }
    }
    GLOBAL uint16_t* oh = gbl(ST == NS_GRAM ? d.ah : d.bh);
    GLOBAL uint16_t* ol = gbl(ST == NS_GRAM ? d.al : d.bl);
    flush_ji(oh, false);
    if constexpr (ACC) flush_ji(ol, true);
    if (i0 != j0) {
      flush_ij(oh, false);
      if constexpr (ACC) flush_ij(ol, true);
    }
  } else {
    if constexpr (ACC) {
      fetch(gbl(d.xh[cur]));
      add(na.a);
    }
    // The fast form needs no lo in the last step: nothing multiplies that rounding again.
    if constexpr (ACC || OT == 0) {
      fetch(gbl(d.xl[cur]));
      add(na.a);
    }
    if constexpr (OT == 0) {
      flush_ji(gbl(d.xh[cur ^ 1]), false);
      if (ACC || step + 2 < na.steps) flush_ji(gbl(d.xl[cur ^ 1]), true);
    } else {
      // half of the wave's i at a time, as fp32 rows of the output (rows i when X is transposed)
      constexpr int HI = WI / 2;
      float* const regf = reinterpret_cast<float*>(reg);
      const bool vec = ((d.ld_out | d.n) & 3) == 0 && (reinterpret_cast<uintptr_t>(d.out) & (OT == G_F32 ? 15 : 7)) == 0;
      const int cols = d.flip ? WJ : HI;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int a = 0; a < TL::TA / 2; ++a)
#pragma unroll
          for (int b = 0; b < TL::TB; ++b) {
            const f32x4 v = acc[h * (TL::TA / 2) + a][b] * (1.0f / kNsScaleX);
            if (d.flip) {
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                const int r = 16 * a + 4 * g + t;
                regf[r * WJ + 4 * ((4 * b + (c >> 2)) ^ (r & (WJ / 4 - 1))) + (c & 3)] = v[t];
              }
            } else {
              const int r = 16 * b + c;
              *reinterpret_cast<f32x4*>(&regf[r * HI + 4 * ((4 * a + g) ^ (r & (HI / 4 - 1)))]) = v;
            }
          }
        const int row0 = d.flip ? ib + h * HI : jb, col0 = d.flip ? jb : ib + h * HI;
        const int units = cols / 4;
        // A batch of loads before the first is waited for (one at a time: four resblocks' last update
        // 448 us, so 391). Their addresses are clamped into the parameter, nothing is stored past it.
        constexpr int BATCH = 8;
        static_assert(HI * WJ / 256 % BATCH == 0 || HI * WJ / 256 < BATCH);
        constexpr int PASS = HI * WJ / 256 < BATCH ? HI * WJ / 256 : BATCH;
        for (int x0 = 0; x0 < HI * WJ / 256; x0 += PASS) {
          f32x4 th[PASS];
          if (vec && na.muon) {
#pragma unroll
            for (int y = 0; y < PASS; ++y) {
              const int e = (x0 + y) * kWave + lane;
              const int row = min(row0 + e / units, d.m - 1), col = min(col0 + 4 * (e % units), d.n - 4);
              th[y] = out_load4<OT>(d.out, (int64_t)row * d.ld_out + col);
            }
          }
#pragma unroll
          for (int y = 0; y < PASS; ++y) {
            const int e = (x0 + y) * kWave + lane, r = e / units, u = e % units;
            const int row = row0 + r, col = col0 + 4 * u;
            if (row >= d.m || col >= d.n) continue;
            f32x4 v = *reinterpret_cast<const f32x4*>(&regf[r * cols + 4 * (u ^ (r & (units - 1)))]);
            const int64_t o = (int64_t)row * d.ld_out + col;
            if (vec) {
              if (na.muon) v = th[y] - na.lr * (d.factor[na.adjust] * v + na.weight_decay * th[y]);
              out_store4<OT>(d.out, o, v);
            } else {
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                if (col + t >= d.n) continue;
                float w = v[t];
                if (na.muon) {
                  const float one = out_load<OT>(d.out, o + t);
                  w = one - na.lr * (d.factor[na.adjust] * w + na.weight_decay * one);
                }
                out_store<OT>(d.out, o + t, w);
              }
            }
          }
        }
      }
    }
  }
}

template <int ST, int T, bool ACC, int OT, bool REDUCE = false>
void go(const NsList& l, int step, const NsArgs& a, hipStream_t s) {
  k_ns_gemm<ST, T, ACC, OT, REDUCE><<<dim3(REDUCE ? l.n_reduce * Tile<T>::WAVES : l.n_work), dim3(REDUCE ? kWave : Tile<T>::THREADS), 0, s>>>(
      REDUCE ? l.reduce : l.work, l.partial, step, a);
}
template <int ST, int T, bool ACC>
void go_split(const NsList& l, int step, const NsArgs& a, hipStream_t s) {
  go<ST, T, ACC, 0>(l, step, a, s);
  if (l.n_reduce > 0) go<ST, T, ACC, 0, true>(l, step, a, s);
}
template <int T, bool ACC>
hipError_t pick(NsStage st, int ot, bool last, const NsList& l, int step, const NsArgs& a, hipStream_t s) {
  if (st == NS_GRAM) go_split<NS_GRAM, T, ACC>(l, step, a, s);
  else if (st == NS_POLY) go_split<NS_POLY, T, ACC>(l, step, a, s);
  else if (!last) go<NS_UPDATE, T, ACC, 0>(l, step, a, s);
  else if (ot == G_F32) go<NS_UPDATE, T, ACC, G_F32>(l, step, a, s);
  else if (ot == G_F16) go<NS_UPDATE, T, ACC, G_F16>(l, step, a, s);
  else if (ot == G_BF16) go<NS_UPDATE, T, ACC, G_BF16>(l, step, a, s);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ns_gemm(NsStage st, bool accurate, int ot, bool last, const NsList& l, int step,
                          const NsArgs& a, hipStream_t s) {
  if (l.tile == 256)
    return accurate ? hipErrorInvalidValue : pick<256, false>(st, ot, last, l, step, a, s);
  if (l.tile == 128)
    return accurate ? pick<128, true>(st, ot, last, l, step, a, s) : pick<128, false>(st, ot, last, l, step, a, s);
  return accurate ? pick<64, true>(st, ot, last, l, step, a, s) : pick<64, false>(st, ot, last, l, step, a, s);
}

}  // namespace psgd
