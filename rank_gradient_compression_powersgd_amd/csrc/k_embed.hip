// Embedding rows with scaling, and the embedding's gradient by sorted tokens.
//
//   lookup:    out[t] = round(scale * W[id_t]); a token outside [0, vocab) gives a row of zeros
//   gradient:  dW[v] = scale * sum over t with id_t = v of dx[t]   (+ dW[v] when accumulating)
//
// The embeddings are the uncompressed 32-bit tensors of the step (Korean summary of the paper,
// section "Mixed-Precision Training"): the gradient formed here is a pass-through gradient.
//
// Both are bound by HBM. The gradient adds the rows of a token in the order of the batch, in
// fp32, with no atomics on data: the tokens are sorted stably first, then fixed chunks of the
// sorted order are summed, so the result is the same bits on every run and a token that fills
// half the batch is spread over the chip like any other.
#include "embed.h"

namespace psgd {
namespace {

// ---- element access ------------------------------------------------------------------------
template <int T, int V> struct Vec {
  typedef float f __attribute__((ext_vector_type(V)));
  // V consecutive elements at p[i], widened; V > 1: 16-byte (8-byte for 4 half-width) aligned
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
      } else if constexpr (V == 4) return GradIO<T>::load4(gcast<char>(q));
      else return GradIO<T>::load8(gcast<char>(q));
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
constexpr int SO_THREADS = 1024, SO_WAVES = SO_THREADS / kWave, SO_UNROLL = 8;

// One workgroup per range of `range` ids. Every workgroup reads all tokens (a few bytes each,
// from L2): it counts those below its range, which is where its part of the sorted order
// begins, so no workgroup waits for another and one launch sorts. Each wave keeps one contiguous
// share of the batch; a token's place is its id's first place, plus the tokens of that id in
// earlier waves, plus those before it in its own wave: stable, and free of atomics' order.
template <int ID>
__global__ __launch_bounds__(SO_THREADS)
void k_embed_sort(EmbedGrad a)
{
  __shared__ int32_t hist[SO_WAVES][kEmbedRange];       // tokens of an id per wave, then places
  __shared__ int32_t below_w[SO_WAVES], in_w[SO_WAVES], scan_w[SO_WAVES];
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  const int64_t lo = (int64_t)blockIdx.x * a.range, hi = min(lo + a.range, a.vocab);
  const int nr = (int)(hi - lo);
  const int64_t share = (a.n + SO_WAVES * kWave - 1) / (SO_WAVES * kWave) * kWave;
  const int64_t b0 = min(w * share, a.n), b1 = min(b0 + share, a.n);
  for (int i = threadIdx.x; i < SO_WAVES * kEmbedRange; i += SO_THREADS) (&hist[0][0])[i] = 0;

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

  // the range's tokens, in batch order, each wave's share contiguous
  uint64_t* __restrict__ list = a.list + base + mine;
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
        if (mineid) {
          const int32_t key = (int32_t)(id[u] - lo);
          list[put + __popcll(bal & ((1ull << lane) - 1))] = ((uint64_t)key << 32) | (uint32_t)(b + u * kWave + lane);
          atomicAdd(&hist[w][key], 1);
        }
        put += __popcll(bal);
      }
    }
  __syncthreads();

  // first place of every id (exclusive sums over ids, then over waves within an id)
  int32_t cnt = 0;
  if ((int)threadIdx.x < nr)
    for (int i = 0; i < SO_WAVES; ++i) cnt += hist[i][threadIdx.x];
  int32_t inc = cnt;
  for (int o = 1; o < kWave; o <<= 1) { const int32_t v = __shfl_up(inc, o); if (lane >= o) inc += v; }
  if (lane == kWave - 1) scan_w[w] = inc;
  __syncthreads();
  int32_t first = base + inc - cnt;
  for (int i = 0; i < w; ++i) first += scan_w[i];
  if ((int)threadIdx.x < nr) {
    gbl(a.seg)[lo + threadIdx.x] = first;
    for (int i = 0; i < SO_WAVES; ++i) { const int32_t h = hist[i][threadIdx.x]; hist[i][threadIdx.x] = first; first += h; }
  }
  if (hi == a.vocab && threadIdx.x == 0) gbl(a.seg)[a.vocab] = base + total;
  __syncthreads();

  // stable placement: 64 tokens of the wave's list at a time. Lanes with the same id take
  // consecutive places; the last of them moves the id's place on.
  for (int32_t i0 = 0; i0 < in; i0 += kWave) {
    const bool has = i0 + lane < in;
    const uint64_t e = has ? list[i0 + lane] : ~0ull;
    const uint32_t key = (uint32_t)(e >> 32);
    uint64_t same = __builtin_amdgcn_ballot_w64(has);
    for (int bit = 0; bit < 32 - __builtin_clz(kEmbedRange - 1); ++bit) {
      const uint64_t one = __builtin_amdgcn_ballot_w64((key >> bit) & 1);
      same &= ((key >> bit) & 1) ? one : ~one;
    }
    int32_t at = 0;
    if (has) at = hist[w][key] + __popcll(same & ((1ull << lane) - 1));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (has) {
      if ((same >> lane) == 1) hist[w][key] = at + 1;
      gbl(a.sorted)[at] = ((uint64_t)(lo + key) << 32) | (uint32_t)e;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// ---- the sums ------------------------------------------------------------------------------
constexpr int SU_THREADS = 256, SU_UNROLL = 8;

// blockIdx.x < chunks: one chunk of the sorted order, 256 V columns. A token whose tokens all
// lie in the chunk is finished here; a token that goes on into the next chunk or comes from the
// one before leaves a partial row: slot 2 j + 1 where it begins in chunk j, 2 j where it does
// not. The remaining workgroups write the zero rows of absent tokens.
template <int T, int V>
__global__ __launch_bounds__(SU_THREADS)
void k_embed_sum(EmbedGrad a)
{
  typedef typename Vec<T, V>::f vf;
  const int64_t col = ((int64_t)blockIdx.y * SU_THREADS + threadIdx.x) * V;
  const int64_t vocab = a.vocab;
  if ((int64_t)blockIdx.x >= a.chunks) {
    const int64_t v0 = ((int64_t)blockIdx.x - a.chunks) * kEmbedZeroRows;
    if (col >= a.dim) return;
    for (int64_t v = v0; v < min(v0 + kEmbedZeroRows, vocab); ++v)
      if (gbl(a.seg)[v] == gbl(a.seg)[v + 1]) Vec<G_F32, V>::store(a.dtable, v * a.ld_dtable + col, vf(0.0f));
    return;
  }
  const int32_t total = gbl(a.seg)[vocab];
  const int64_t p0 = (int64_t)blockIdx.x * a.chunk;
  if (p0 >= total || col >= a.dim) return;
  const int cnt = (int)min((int64_t)a.chunk, total - p0);
  const GLOBAL uint64_t* sorted = gbl(a.sorted) + p0;
  vf acc = 0.0f;
  int run = 0;                                   // first position of the running token
  for (int i0 = 0; i0 < cnt; i0 += SU_UNROLL) {
    uint64_t e[SU_UNROLL + 1];
    vf x[SU_UNROLL];
#pragma unroll
    for (int u = 0; u < SU_UNROLL; ++u) {
      e[u] = i0 + u < cnt ? sorted[i0 + u] : ~0ull;
      x[u] = 0.0f;
      if (i0 + u < cnt) x[u] = Vec<T, V>::load(a.dx, (int64_t)(uint32_t)e[u] * a.ld_dx + col);
    }
    e[SU_UNROLL] = i0 + SU_UNROLL < cnt ? sorted[i0 + SU_UNROLL] : ~0ull;
#pragma unroll
    for (int u = 0; u < SU_UNROLL; ++u) {
      if (i0 + u >= cnt) break;
      acc += x[u];
      const uint32_t v = (uint32_t)(e[u] >> 32);
      if (i0 + u + 1 < cnt && (uint32_t)(e[u + 1] >> 32) == v) continue;
      // the token's run in this chunk ends here
      const int32_t s0 = gbl(a.seg)[v], s1 = gbl(a.seg)[(int64_t)v + 1];
      const bool begins = s0 == p0 + run, ends = s1 == p0 + i0 + u + 1;
      if (begins && ends) {
        const int64_t o = (int64_t)v * a.ld_dtable + col;
        vf r = a.scale * acc;
        if (a.accumulate) r = Vec<G_F32, V>::load(a.dtable, o) + r;
        Vec<G_F32, V>::store(a.dtable, o, r);
      } else {
        Vec<G_F32, V>::store(a.partial, (2 * (int64_t)blockIdx.x + (begins ? 1 : 0)) * a.ld_partial + col, acc);
      }
      acc = 0.0f;
      run = i0 + u + 1;
    }
  }
}

// A token that begins in chunk blockIdx.x and goes on: its partial rows, added in order.
template <int V>
__global__ __launch_bounds__(SU_THREADS)
void k_embed_join(EmbedGrad a)
{
  typedef typename Vec<G_F32, V>::f vf;
  const int32_t total = gbl(a.seg)[a.vocab];
  const int64_t j = blockIdx.x, p0 = j * a.chunk, p1 = p0 + a.chunk;
  if (p1 >= total) return;
  const uint32_t v = (uint32_t)(gbl(a.sorted)[p1 - 1] >> 32);
  const int32_t s0 = gbl(a.seg)[v], s1 = gbl(a.seg)[(int64_t)v + 1];
  if (s0 < p0 || s1 <= p1) return;
  const int64_t col = ((int64_t)blockIdx.y * SU_THREADS + threadIdx.x) * V;
  if (col >= a.dim) return;
  vf acc = Vec<G_F32, V>::load(a.partial, (2 * j + 1) * a.ld_partial + col);
  const int64_t je = (s1 - 1) / a.chunk;
#pragma unroll 8
  for (int64_t k = j + 1; k <= je; ++k) acc += Vec<G_F32, V>::load(a.partial, 2 * k * a.ld_partial + col);
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

template <int T, int V> hipError_t grad_sum(const EmbedGrad& a, hipStream_t s) {
  const unsigned cols = (unsigned)((a.dim + SU_THREADS * V - 1) / (SU_THREADS * V));
  const int64_t zero = a.accumulate ? 0 : (a.vocab + kEmbedZeroRows - 1) / kEmbedZeroRows;
  if (a.chunks + zero > 0) k_embed_sum<T, V><<<dim3((unsigned)(a.chunks + zero), cols), dim3(SU_THREADS), 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.chunks < 2) return e;
  k_embed_join<V><<<dim3((unsigned)(a.chunks - 1), cols), dim3(SU_THREADS), 0, s>>>(a);
  return hipGetLastError();
}
template <int T> hipError_t grad_vec(const EmbedGrad& a, hipStream_t s) {
  if (a.dim % 4 == 0 && aligned(a.dx, a.ld_dx, T == G_F32 ? 4 : 2, 4) && aligned(a.dtable, a.ld_dtable, 4, 4)) return grad_sum<T, 4>(a, s);
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
  const dim3 grid((unsigned)((a.vocab + a.range - 1) / a.range)), block(SO_THREADS);
  if (id_bytes == 4) k_embed_sort<4><<<grid, block, 0, s>>>(a);
  else k_embed_sort<8><<<grid, block, 0, s>>>(a);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  switch (dt) {
    case G_F32: return grad_vec<G_F32>(a, s);
    case G_F16: return grad_vec<G_F16>(a, s);
    case G_BF16: return grad_vec<G_BF16>(a, s);
  }
  return hipErrorInvalidValue;
}

// Ids per sorting workgroup: enough workgroups for the chip, at most the counters' room.
int64_t embed_range(int64_t vocab) {
  const int64_t r = (vocab + 255) / 256;
  return r < 16 ? 16 : r > kEmbedRange ? kEmbedRange : r;
}
int embed_chunk(int64_t, int64_t) { return 32; }

}  // namespace psgd
