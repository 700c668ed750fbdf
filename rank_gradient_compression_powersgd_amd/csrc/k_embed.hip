// Embedding rows with scaling, and the embedding's gradient by sorted tokens.
//
//   lookup:    out[t] = round(scale * W[id_t]); a token outside [0, vocab) gives a row of zeros
//   gradient:  dW[v] = scale * sum over t with id_t = v of dx[t]   (+ dW[v] when accumulating)
//
// The embeddings are the uncompressed 32-bit tensors of the step (Korean summary of the paper,
// section "Mixed-Precision Training"): the gradient formed here is a pass-through gradient.
//
// Both are bound by HBM. The gradient adds the rows of a token in fp32 with no atomics on data: the
// tokens are sorted stably first, then fixed chunks of the sorted order are summed, each in the
// order of the batch, and the chunks' sums of a token added. The same inputs give the same bits on
// every run (where chunks cut a token's rows depends on the tokens sorted before it), and a token
// that fills half the batch is spread over the chip like any other.
#include <algorithm>

#include "embed.h"

namespace psgd {
namespace {

// ---- element access ------------------------------------------------------------------------
template <int T, int V> struct Vec {
  typedef float f __attribute__((ext_vector_type(V)));
  // V consecutive elements at p[i], widened; V > 1: 16-byte aligned. 16-bit types take 8 or 1.
  static __device__ __forceinline__ f load(const void* p, int64_t i) {
    if constexpr (T == G_F32) {
      const GLOBAL float* q = gbl(static_cast<const float*>(p)) + i;
      if constexpr (V == 1) return f{*q};
      else if constexpr (V == 4) return *gcast<f32x4>(q);
      else { const f32x4 a = gcast<f32x4>(q)[0], b = gcast<f32x4>(q)[1]; return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }
    } else {
      const GLOBAL uint16_t* q = gbl(static_cast<const uint16_t*>(p)) + i;
      if constexpr (V == 1) {
        if constexpr (T == G_F16) return f{(float)__builtin_bit_cast(_Float16, *q)};
        else return f{__builtin_bit_cast(float, (uint32_t)*q << 16)};
      } else {
        static_assert(V == 8);
        return GradIO<T>::load8(gcast<char>(q));
      }
    }
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, f v) {
    if constexpr (T == G_F32) {
      GLOBAL float* q = gbl(static_cast<float*>(p)) + i;
      if constexpr (V == 1) *q = v[0];
      else if constexpr (V == 4) *gcast<f32x4>(q) = v;
      else { gcast<f32x4>(q)[0] = __builtin_shufflevector(v, v, 0, 1, 2, 3); gcast<f32x4>(q)[1] = __builtin_shufflevector(v, v, 4, 5, 6, 7); }
    } else {
      GLOBAL uint16_t* q = gbl(static_cast<uint16_t*>(p)) + i;
      if constexpr (V == 1) {
        if constexpr (T == G_F16) *q = f16_bits((_Float16)v[0]); else *q = bf16_bits((__bf16)v[0]);
      } else {
        typedef _Float16 h __attribute__((ext_vector_type(V)));
        typedef __bf16 b __attribute__((ext_vector_type(V)));
        typedef uint32_t w __attribute__((ext_vector_type(V / 2)));
        if constexpr (T == G_F16) *gcast<w>(q) = __builtin_bit_cast(w, __builtin_convertvector(v, h));
        else *gcast<w>(q) = __builtin_bit_cast(w, __builtin_convertvector(v, b));
      }
    }
  }
};
template <int ID> __device__ __forceinline__ int64_t load_id(const void* ids, int64_t i) {
  if constexpr (ID == 4) return gbl(static_cast<const int32_t*>(ids))[i];
  else return gbl(static_cast<const int64_t*>(ids))[i];
}

// ---- lookup --------------------------------------------------------------------------------
constexpr int LK_THREADS = 256, LK_ROWS = 4;

// blockIdx.x: LK_ROWS tokens, whose rows are loaded together; blockIdx.y: 256 V columns.
template <int T, int O, int V, int ID>
__global__ __launch_bounds__(LK_THREADS)
void k_embed_lookup(EmbedLookup a)
{
  const int64_t col = ((int64_t)blockIdx.y * LK_THREADS + threadIdx.x) * V;
  if (col >= a.dim) return;
  const int64_t t0 = (int64_t)blockIdx.x * LK_ROWS;
  typename Vec<T, V>::f v[LK_ROWS];
  bool ok[LK_ROWS];
#pragma unroll
  for (int r = 0; r < LK_ROWS; ++r) {
    const int64_t id = t0 + r < a.n ? load_id<ID>(a.ids, t0 + r) : -1;
    ok[r] = id >= 0 && id < a.vocab;
    v[r] = 0.0f;
    if (ok[r]) v[r] = Vec<T, V>::load(a.table, id * a.ld_table + col);
  }
#pragma unroll
  for (int r = 0; r < LK_ROWS; ++r) {
    if (t0 + r >= a.n) break;
    // a row of zeros stays +0 under a negative scale
    Vec<O, V>::store(a.out, (t0 + r) * a.ld_out + col, ok[r] ? a.scale * v[r] : v[r]);
  }
}

// ---- the tokens sorted ---------------------------------------------------------------------
// A stable sort by id in ranges of `range` ids: first the ranges in order, each with its tokens in
// batch order (`list`), then each range by id (`sorted`, with the first place of every id in `seg`).
// A token's place is its key's first place, plus the tokens of that key in earlier waves, plus
// those before it in its own wave: stable, and free of atomics' order.
constexpr int SO_THREADS = 1024, SO_WAVES = SO_THREADS / kWave, SO_UNROLL = 8;

__device__ __forceinline__ int prefix(uint64_t mask, int lane) { return __popcll(mask & ((1ull << lane) - 1)); }

// lanes that hold the same key, among those of `has`
template <int BITS> __device__ __forceinline__ uint64_t same_key(uint32_t key, bool has) {
  uint64_t same = __builtin_amdgcn_ballot_w64(has);
#pragma unroll
  for (int bit = 0; bit < BITS; ++bit) {
    const bool set = (key >> bit) & 1;
    const uint64_t one = __builtin_amdgcn_ballot_w64(set);
    same &= set ? one : ~one;
  }
  return same;
}
constexpr int bits_of(int n) { return n <= 1 ? 0 : 1 + bits_of((n + 1) / 2); }

// place of this lane's key: lanes with the same key take consecutive places from at[key], which the
// last of them moves on
template <int BITS> __device__ __forceinline__ int32_t take_place(int32_t* at, uint32_t key, bool has, int lane) {
  const uint64_t same = same_key<BITS>(key, has);
  int32_t p = 0;
  if (has) p = at[key] + prefix(same, lane);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (has && (same >> lane) == 1) at[key] = p + 1;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return p;
}

// Exclusive sum over the workgroup's threads; `sums` holds a word per wave.
__device__ __forceinline__ int32_t block_exclusive(int32_t v, int32_t* sums) {
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  int32_t inc = v;
  for (int o = 1; o < kWave; o <<= 1) { const int32_t u = __shfl_up(inc, o); if (lane >= o) inc += u; }
  if (lane == kWave - 1) sums[w] = inc;
  __syncthreads();
  for (int i = 0; i < w; ++i) inc += sums[i];
  __syncthreads();
  return inc - v;
}

// hist[w][k] (tokens of key k in wave w's share) becomes the first place of key k in wave w, the
// keys in order from `base`; returns the first place of key threadIdx.x.
template <int N> __device__ __forceinline__ int32_t places(int32_t (*hist)[N], int n, int32_t base, int32_t* sums) {
  int32_t cnt = 0;
  if ((int)threadIdx.x < n)
    for (int i = 0; i < SO_WAVES; ++i) cnt += hist[i][threadIdx.x];
  const int32_t first = base + block_exclusive(cnt, sums);
  if ((int)threadIdx.x < n) {
    int32_t at = first;
    for (int i = 0; i < SO_WAVES; ++i) { const int32_t h = hist[i][threadIdx.x]; hist[i][threadIdx.x] = at; at += h; }
  }
  __syncthreads();
  return first;
}

// The tokens of range `lo`.., which stand in `list` in batch order (n of them from `base`), sorted by
// id. The waves take contiguous shares.
struct SortMem {
  int32_t hist[SO_WAVES][kEmbedRange];
  int32_t sums[SO_WAVES];
};
__device__ __forceinline__ void sort_range(const EmbedGrad& a, SortMem& m, int64_t lo, int nr, int32_t base, int32_t n) {
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  const int32_t share = (n + SO_THREADS - 1) / SO_THREADS * kWave;
  const int32_t b0 = min(w * share, n), b1 = min(b0 + share, n);
  const GLOBAL uint64_t* list = gbl((const uint64_t*)a.list) + base;
  for (int i = threadIdx.x; i < SO_WAVES * kEmbedRange; i += SO_THREADS) (&m.hist[0][0])[i] = 0;
  __syncthreads();
  for (int32_t b = b0 + lane; b < b1; b += kWave) atomicAdd(&m.hist[w][(uint32_t)(list[b] >> 32)], 1);
  __syncthreads();
  const int32_t first = places(m.hist, nr, base, m.sums);
  if ((int)threadIdx.x < nr) gbl(a.seg)[lo + threadIdx.x] = first;
  if (lo + nr == a.vocab && threadIdx.x == 0) gbl(a.seg)[a.vocab] = base + n;
  for (int32_t b = b0; b < b1; b += kWave) {
    const bool has = b + lane < b1;
    const uint64_t e = has ? list[b + lane] : ~0ull;
    const int32_t at = take_place<bits_of(kEmbedRange)>(m.hist[w], (uint32_t)(e >> 32), has, lane);
    if (has) gbl(a.sorted)[at] = ((uint64_t)(lo + (e >> 32)) << 32) | (uint32_t)e;
  }
}

// Short batches, one launch: the workgroup of a range reads all tokens (a few bytes each, from L2),
// counts those below its range, which is where its part of the order begins, and keeps its own.
// No workgroup waits for another. The time grows with n for every workgroup: 14 us at 20480 tokens
// and 34 at 65537, where the three launches below take 17 and 20.
template <int ID>
__global__ __launch_bounds__(SO_THREADS)
void k_embed_sort(EmbedGrad a)
{
  __shared__ SortMem m;
  __shared__ int32_t below_w[SO_WAVES], in_w[SO_WAVES];
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  const int64_t lo = (int64_t)blockIdx.x * a.range, hi = min(lo + a.range, a.vocab);
  const int64_t share = (a.n + SO_THREADS - 1) / SO_THREADS * kWave;
  const int64_t b0 = min(w * share, a.n), b1 = min(b0 + share, a.n);
  int32_t below = 0, in = 0;
  for (int64_t b = b0; b < b1; b += SO_UNROLL * kWave) {
    int64_t id[SO_UNROLL];
#pragma unroll
    for (int u = 0; u < SO_UNROLL; ++u) {
      const int64_t t = b + u * kWave + lane;
      id[u] = t < b1 ? load_id<ID>(a.ids, t) : -1;
    }
#pragma unroll
    for (int u = 0; u < SO_UNROLL; ++u) {
      below += __popcll(__builtin_amdgcn_ballot_w64(id[u] >= 0 && id[u] < lo));
      in += __popcll(__builtin_amdgcn_ballot_w64(id[u] >= lo && id[u] < hi));
    }
  }
  if (lane == 0) { below_w[w] = below; in_w[w] = in; }
  __syncthreads();
  int32_t base = 0, mine = 0, total = 0;
  for (int i = 0; i < SO_WAVES; ++i) { base += below_w[i]; mine += i < w ? in_w[i] : 0; total += in_w[i]; }
  GLOBAL uint64_t* list = gbl(a.list) + base + mine;
  int32_t put = 0;
  if (in > 0)
    for (int64_t b = b0; b < b1; b += SO_UNROLL * kWave) {
      int64_t id[SO_UNROLL];
#pragma unroll
      for (int u = 0; u < SO_UNROLL; ++u) {
        const int64_t t = b + u * kWave + lane;
        id[u] = t < b1 ? load_id<ID>(a.ids, t) : -1;
      }
#pragma unroll
      for (int u = 0; u < SO_UNROLL; ++u) {
        const bool mineid = id[u] >= lo && id[u] < hi;
        const uint64_t bal = __builtin_amdgcn_ballot_w64(mineid);
        if (mineid) list[put + prefix(bal, lane)] = ((uint64_t)(id[u] - lo) << 32) | (uint32_t)(b + u * kWave + lane);
        put += __popcll(bal);
      }
    }
  __syncthreads();
  sort_range(a, m, lo, (int)(hi - lo), base, total);
}

// Long batches, three launches. Tokens are dealt to workgroups in contiguous shares of `tokens`.
// 1: tokens of every range in each share.
template <int ID>
__global__ __launch_bounds__(SO_THREADS)
void k_embed_count(EmbedGrad a)
{
  __shared__ int32_t hist[kEmbedRanges];
  const int nb = (int)((a.vocab + a.range - 1) / a.range);
  for (int i = threadIdx.x; i < nb; i += SO_THREADS) hist[i] = 0;
  __syncthreads();
  const int64_t b0 = (int64_t)blockIdx.x * a.tokens, b1 = min(b0 + a.tokens, a.n);
  for (int64_t t = b0 + threadIdx.x; t < b1; t += SO_THREADS) {
    const int64_t id = load_id<ID>(a.ids, t);
    if (id >= 0 && id < a.vocab) atomicAdd(&hist[(uint32_t)id / (uint32_t)a.range], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nb; i += SO_THREADS) gbl(a.count)[(int64_t)blockIdx.x * nb + i] = hist[i];
}

// 2: every share's tokens to their range's part of `list`. A range begins behind all tokens of the
// ranges before it, a share's part of it behind those of the shares before.
template <int ID>
__global__ __launch_bounds__(SO_THREADS)
void k_embed_deal(EmbedGrad a)
{
  __shared__ int32_t hist[SO_WAVES][kEmbedRanges];
  __shared__ int32_t sums[SO_WAVES];
  const int nb = (int)((a.vocab + a.range - 1) / a.range);
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave, r = threadIdx.x;
  for (int i = threadIdx.x; i < SO_WAVES * kEmbedRanges; i += SO_THREADS) (&hist[0][0])[i] = 0;
  int32_t total = 0, before = 0;
  for (int g0 = 0; r < nb && g0 < (int)gridDim.x; g0 += 16) {
    int32_t c[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) c[u] = g0 + u < (int)gridDim.x ? gbl((const int32_t*)a.count)[(int64_t)(g0 + u) * nb + r] : 0;
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      total += c[u];
      before += g0 + u < (int)blockIdx.x ? c[u] : 0;
    }
  }
  const int32_t start = block_exclusive(total, sums);
  if (blockIdx.x == 0 && r < nb) gbl(a.start)[r] = start;
  if (blockIdx.x == 0 && r == nb - 1) gbl(a.start)[nb] = start + total;
  const int64_t share = (a.tokens + SO_THREADS - 1) / SO_THREADS * kWave;
  const int64_t g0 = (int64_t)blockIdx.x * a.tokens, g1 = min(g0 + a.tokens, a.n);
  const int64_t b0 = min(g0 + w * share, g1), b1 = min(b0 + share, g1);
  for (int64_t t = b0 + lane; t < b1; t += kWave) {
    const int64_t id = load_id<ID>(a.ids, t);
    if (id >= 0 && id < a.vocab) atomicAdd(&hist[w][(uint32_t)id / (uint32_t)a.range], 1);
  }
  __syncthreads();
  if (r < nb) {
    int32_t at = start + before;
    for (int i = 0; i < SO_WAVES; ++i) { const int32_t h = hist[i][r]; hist[i][r] = at; at += h; }
  }
  __syncthreads();
  for (int64_t b = b0; b < b1; b += kWave) {
    const int64_t t = b + lane, id = t < b1 ? load_id<ID>(a.ids, t) : -1;
    const bool has = id >= 0 && id < a.vocab;
    const uint32_t bucket = has ? (uint32_t)id / (uint32_t)a.range : 0;
    const int32_t at = take_place<bits_of(kEmbedRanges)>(hist[w], bucket, has, lane);
    if (has) gbl(a.list)[at] = ((uint64_t)((uint32_t)id - bucket * (uint32_t)a.range) << 32) | (uint32_t)t;
  }
}

// 3: every range by id.
__global__ __launch_bounds__(SO_THREADS)
void k_embed_order(EmbedGrad a)
{
  __shared__ SortMem m;
  const int64_t lo = (int64_t)blockIdx.x * a.range;
  const int32_t base = gbl((const int32_t*)a.start)[blockIdx.x], end = gbl((const int32_t*)a.start)[blockIdx.x + 1];
  sort_range(a, m, lo, (int)min(a.range, a.vocab - lo), base, end - base);
}

// ---- the sums ------------------------------------------------------------------------------
constexpr int SU_THREADS = 256, SU_UNROLL = 8, JO_UNROLL = 16, JO_WAYS = 4;

// blockIdx.x < chunks: one chunk of the sorted order; blockIdx.y: blockDim.x V columns. A token
// whose tokens all lie in the chunk is finished here; a token that goes on into the next chunk or
// comes from the one before leaves a partial row: slot 2 j + 1 where it begins in chunk j, 2 j
// where it does not. Where a run begins and ends is read off the neighbours in the sorted order, so
// nothing but the rows themselves is waited for. The remaining workgroups write the zero rows of
// absent tokens.
template <int T, int V, bool ADD>
__global__ __launch_bounds__(SU_THREADS)
void k_embed_sum(EmbedGrad a)
{
  typedef typename Vec<T, V>::f vf;
  __shared__ uint64_t ent[kEmbedChunk + 2];      // the chunk's entries, and one before and behind
  const int64_t col = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V;
  const int64_t vocab = a.vocab;
  if ((int64_t)blockIdx.x >= a.chunks) {
    const int64_t v0 = ((int64_t)blockIdx.x - a.chunks) * kEmbedZeroRows;
    const int lane = threadIdx.x & (kWave - 1);
    const int32_t s = gbl((const int32_t*)a.seg)[min(v0 + min(lane, kEmbedZeroRows), vocab)];
    const int32_t next = __shfl_down(s, 1);      // by every lane, also those that ask for no row
    uint64_t gone = __builtin_amdgcn_ballot_w64(lane < kEmbedZeroRows && v0 + lane < vocab && s == next);
    if (col >= a.dim) return;
    for (; gone; gone &= gone - 1) Vec<G_F32, V>::store(a.dtable, (v0 + __builtin_ctzll(gone)) * a.ld_dtable + col, vf(0.0f));
    return;
  }
  const int32_t total = gbl((const int32_t*)a.seg)[vocab];
  const int64_t p0 = (int64_t)blockIdx.x * a.chunk;
  if (p0 >= total) return;
  const int cnt = (int)min((int64_t)a.chunk, total - p0);
  for (int i = threadIdx.x; i < cnt + 2; i += blockDim.x) {
    const int64_t p = p0 - 1 + i;
    ent[i] = p >= 0 && p < total ? gbl((const uint64_t*)a.sorted)[p] : ~0ull;
  }
  __syncthreads();
  if (col >= a.dim) return;
  auto id_of = [&](int i) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)(ent[i + 1] >> 32)); };   // -1: before
  auto pos_of = [&](int i) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)ent[i + 1]); };
  vf acc = 0.0f;
  bool begins = id_of(-1) != id_of(0);
  for (int i0 = 0; i0 < cnt; i0 += SU_UNROLL) {
    vf x[SU_UNROLL], old[ADD ? SU_UNROLL : 1];
#pragma unroll
    for (int u = 0; u < SU_UNROLL; ++u) {
      // past the chunk its last row again: without a branch the loads of a batch are under way
      // together
      const int i = min(i0 + u, cnt - 1);
      x[u] = Vec<T, V>::load(a.dx, (int64_t)pos_of(i) * a.ld_dx + col);
      // the row to add to, where a token may end (one that leaves a partial row after all only
      // reads it for nothing)
      if (ADD && id_of(i) != id_of(i + 1)) old[ADD ? u : 0] = Vec<G_F32, V>::load(a.dtable, (int64_t)id_of(i) * a.ld_dtable + col);
    }
    __builtin_amdgcn_sched_barrier(0);           // or the loads sink to their uses
#pragma unroll
    for (int u = 0; u < SU_UNROLL; ++u) {
      const int i = i0 + u;
      if (i >= cnt) break;
      acc += x[u];
      const uint32_t v = id_of(i);
      const bool ends = id_of(i + 1) != v;
      if (!ends && i + 1 < cnt) continue;
      if (begins && ends) {
        vf r = a.scale * acc;
        if constexpr (ADD) r = old[u] + r;
        Vec<G_F32, V>::store(a.dtable, (int64_t)v * a.ld_dtable + col, r);
      } else {
        Vec<G_F32, V>::store(a.partial, (2 * (int64_t)blockIdx.x + (begins ? 1 : 0)) * a.ld_partial + col, acc);
      }
      acc = 0.0f;
      begins = true;
    }
  }
}

// A token that begins in chunk blockIdx.x and goes on: its partial rows, added in order by the rows of
// threads (threadIdx.y), each a share of them, whose sums are then added in order: a token that is
// a tenth of the batch has hundreds. Four rows of threads where one workgroup holds all columns (65536 x
// 64: 56 us in all, one row 63), one where they are spread over several anyway and most of the
// extra waves would only start and end (65536 x 3968: 386 us, four rows 412).
template <int V>
__global__ __launch_bounds__(SU_THREADS * JO_WAYS)
void k_embed_join(EmbedGrad a)
{
  typedef typename Vec<G_F32, V>::f vf;
  __shared__ vf sums[JO_WAYS - 1][SU_THREADS];
  const int32_t total = gbl(a.seg)[a.vocab];
  const int64_t j = blockIdx.x, p0 = j * a.chunk, p1 = p0 + a.chunk;
  if (p1 >= total) return;
  const uint32_t v = (uint32_t)(gbl(a.sorted)[p1 - 1] >> 32);
  const int32_t s0 = gbl(a.seg)[v], s1 = gbl(a.seg)[(int64_t)v + 1];
  if (s0 < p0 || s1 <= p1) return;
  const int64_t col = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V;
  const bool in = col < a.dim;
  const int64_t je = (s1 - 1) / a.chunk;
  const int ways = blockDim.y;
  const int64_t share = max((int64_t)JO_UNROLL, (je - j + ways - 1) / ways);
  const int64_t first = j + 1 + threadIdx.y * share, last = min(first + share - 1, je);
  vf acc = 0.0f;
  if (in && threadIdx.y == 0) acc = Vec<G_F32, V>::load(a.partial, (2 * j + 1) * a.ld_partial + col);
  if (in)
    for (int64_t k0 = first; k0 <= last; k0 += JO_UNROLL) {    // a batch of loads at a time, the last one too
      vf x[JO_UNROLL];
#pragma unroll
      for (int u = 0; u < JO_UNROLL; ++u) {
        x[u] = 0.0f;
        if (k0 + u <= last) x[u] = Vec<G_F32, V>::load(a.partial, 2 * (k0 + u) * a.ld_partial + col);
      }
#pragma unroll
      for (int u = 0; u < JO_UNROLL; ++u) acc += x[u];
    }
  if (threadIdx.y > 0) sums[threadIdx.y - 1][threadIdx.x] = acc;
  __syncthreads();
  if (!in || threadIdx.y > 0) return;
  for (int w = 1; w < ways && j + 1 + w * share <= je; ++w) acc += sums[w - 1][threadIdx.x];
  const int64_t o = (int64_t)v * a.ld_dtable + col;
  vf r = a.scale * acc;
  if (a.accumulate) r = Vec<G_F32, V>::load(a.dtable, o) + r;
  Vec<G_F32, V>::store(a.dtable, o, r);
}

bool aligned(const void* p, int64_t ld, int size, int vec) {
  const int bytes = size * vec < 16 ? size * vec : 16;
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld % vec == 0;
}

template <int T, int O, int V>
void lookup_ids(const EmbedLookup& a, int id_bytes, hipStream_t s) {
  const dim3 grid((unsigned)((a.n + LK_ROWS - 1) / LK_ROWS), (unsigned)((a.dim + LK_THREADS * V - 1) / (LK_THREADS * V)));
  if (id_bytes == 4) k_embed_lookup<T, O, V, 4><<<grid, dim3(LK_THREADS), 0, s>>>(a);
  else k_embed_lookup<T, O, V, 8><<<grid, dim3(LK_THREADS), 0, s>>>(a);
}
template <int T, int O> void lookup_vec(const EmbedLookup& a, int id_bytes, hipStream_t s) {
  const int ts = T == G_F32 ? 4 : 2, os = O == G_F32 ? 4 : 2;
  if (a.dim % 8 == 0 && aligned(a.table, a.ld_table, ts, 8) && aligned(a.out, a.ld_out, os, 8)) lookup_ids<T, O, 8>(a, id_bytes, s);
  else lookup_ids<T, O, 1>(a, id_bytes, s);
}
template <int T> hipError_t lookup_out(const EmbedLookup& a, int ot, int id_bytes, hipStream_t s) {
  switch (ot) {
    case G_F32: lookup_vec<T, G_F32>(a, id_bytes, s); break;
    case G_F16: lookup_vec<T, G_F16>(a, id_bytes, s); break;
    case G_BF16: lookup_vec<T, G_BF16>(a, id_bytes, s); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

// Columns of V values over workgroups of whole waves, evenly.
struct Cols { unsigned blocks, threads; };
Cols cols_of(int64_t dim, int v) {
  const int64_t vecs = (dim + v - 1) / v, blocks = (vecs + SU_THREADS - 1) / SU_THREADS;
  return {(unsigned)blocks, (unsigned)(((vecs + blocks - 1) / blocks + kWave - 1) / kWave * kWave)};
}
template <int T, int V> hipError_t grad_sum(const EmbedGrad& a, hipStream_t s) {
  const Cols c = cols_of(a.dim, V);
  const int64_t zero = a.accumulate ? 0 : (a.vocab + kEmbedZeroRows - 1) / kEmbedZeroRows;
  const dim3 grid((unsigned)(a.chunks + zero), c.blocks), block(c.threads);
  if (a.accumulate && a.chunks > 0) k_embed_sum<T, V, true><<<grid, block, 0, s>>>(a);
  else if (!a.accumulate) k_embed_sum<T, V, false><<<grid, block, 0, s>>>(a);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess || a.chunks < 2) return e;
  constexpr int VJ = V == 1 ? 1 : 4;
  const Cols j = cols_of(a.dim, VJ);
  k_embed_join<VJ><<<dim3((unsigned)(a.chunks - 1), j.blocks), dim3(j.threads, j.blocks == 1 ? JO_WAYS : 1), 0, s>>>(a);
  return hipGetLastError();
}
template <int T> hipError_t grad_vec(const EmbedGrad& a, hipStream_t s) {
  constexpr int V = T == G_F32 ? 4 : 8, size = T == G_F32 ? 4 : 2;
  if (a.dim % V == 0 && aligned(a.dx, a.ld_dx, size, V) && aligned(a.dtable, a.ld_dtable, 4, V)) return grad_sum<T, V>(a, s);
  return grad_sum<T, 1>(a, s);
}

}  // namespace

hipError_t launch_embed_lookup(const EmbedLookup& a, int tt, int ot, int id_bytes, hipStream_t s) {
  if (a.n <= 0) return hipSuccess;
  switch (tt) {
    case G_F32: return lookup_out<G_F32>(a, ot, id_bytes, s);
    case G_F16: return lookup_out<G_F16>(a, ot, id_bytes, s);
    case G_BF16: return lookup_out<G_BF16>(a, ot, id_bytes, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_embed_grad(const EmbedGrad& a, int dt, int id_bytes, hipStream_t s) {
  const dim3 ranges((unsigned)((a.vocab + a.range - 1) / a.range)), block(SO_THREADS);
  if (a.tokens == 0) {
    if (id_bytes == 4) k_embed_sort<4><<<ranges, block, 0, s>>>(a);
    else k_embed_sort<8><<<ranges, block, 0, s>>>(a);
  } else {
    const dim3 shares((unsigned)((a.n + a.tokens - 1) / a.tokens));
    if (id_bytes == 4) {
      k_embed_count<4><<<shares, block, 0, s>>>(a);
      k_embed_deal<4><<<shares, block, 0, s>>>(a);
    } else {
      k_embed_count<8><<<shares, block, 0, s>>>(a);
      k_embed_deal<8><<<shares, block, 0, s>>>(a);
    }
    k_embed_order<<<ranges, block, 0, s>>>(a);
  }
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  switch (dt) {
    case G_F32: return grad_vec<G_F32>(a, s);
    case G_F16: return grad_vec<G_F16>(a, s);
    case G_BF16: return grad_vec<G_BF16>(a, s);
  }
  return hipErrorInvalidValue;
}

// Sorted tokens per summing workgroup: 32, or one batch of loads where all rows together are few (333
// x 1000: 13 us instead of 19, 4096 x 1000: 19 instead of 22; 8192 x 1000: 31 instead of 27) and a
// frequent token does not leave too many partial rows (65536 x 24: 84 us instead of 64).
constexpr int64_t kFewTokens = 8192, kFewElements = 1 << 22;
int embed_chunk(int64_t n, int64_t dim) { return n <= kFewTokens && n * dim <= kFewElements ? SU_UNROLL : kEmbedChunk; }
// Most chunks of a batch of up to n tokens, and most shares of the three-launch sort: a workspace for n
// tokens has to serve fewer.
int64_t embed_max_chunks(int64_t n, int64_t dim) {
  const int64_t few = std::min({n, kFewTokens, kFewElements / dim});
  return std::max((n + kEmbedChunk - 1) / kEmbedChunk, (few + SU_UNROLL - 1) / SU_UNROLL);
}
int64_t embed_max_shares(int64_t n, int64_t vocab) {
  return embed_tokens(n, vocab) == 0 ? 0 : std::min<int64_t>(128, (n + 2047) / 2048);
}
// Ids per sorting workgroup: enough workgroups for the chip, at most the counters' room.
int64_t embed_range(int64_t vocab) {
  const int64_t r = (vocab + 255) / 256;
  return r < 16 ? 16 : r > kEmbedRange ? kEmbedRange : r;
}
// Tokens per workgroup of the three-launch sort (at most 128 workgroups, since each adds up the
// counts of all), or 0: one launch. That one takes any vocabulary, and reads every id once per range:
// 2^20 ids, 2048 ranges, take 0.2 ms with 65537 tokens, 2.3 with 2^20, 76 with 2^25.
int64_t embed_tokens(int64_t n, int64_t vocab) {
  const int64_t ranges = (vocab + embed_range(vocab) - 1) / embed_range(vocab);
  if (n <= kEmbedShort || ranges > kEmbedRanges) return 0;
  const int64_t t = (n + 127) / 128;
  return t < 2048 ? 2048 : t;
}

}  // namespace psgd
