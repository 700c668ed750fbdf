// Arguments of the embedding kernels (k_embed.hip), filled by the runtime.
#pragma once

#include "psgd_internal.h"

namespace psgd {

constexpr int kEmbedRange = 512;        // most ids one sorting workgroup takes
constexpr int kEmbedRanges = 512;       // most ranges the three-launch sort deals tokens to
constexpr int64_t kEmbedShort = 24576;  // longest batch sorted by one launch
constexpr int kEmbedChunk = 32;         // sorted tokens per summing workgroup, at most
constexpr int kEmbedZeroRows = 16;      // table rows per workgroup that clears absent tokens

struct EmbedLookup {
  const void* table; int64_t ld_table, vocab, dim;
  const void* ids;   int64_t n;
  void* out;         int64_t ld_out;
  float scale;
};

struct EmbedGrad {
  const void* dx;    int64_t ld_dx;
  const void* ids;   int64_t n, vocab, dim;
  float* dtable;     int64_t ld_dtable;
  float scale;
  int32_t accumulate;
  int64_t range;                        // ids per sorting workgroup
  int64_t chunks;                       // ceil(n / chunk)
  int32_t chunk;                        // sorted tokens per summing workgroup
  int64_t tokens;                       // tokens per workgroup of the three-launch sort, 0: one launch
  // workspace
  uint64_t* list;                       // n: (id - range start, position), in batch order per range
  uint64_t* sorted;                     // n: (id, position) sorted by id, then position
  int32_t* seg;                         // vocab + 1: first place of every id in `sorted`
  int32_t* count; int32_t* start;       // three-launch sort: tokens per share and range, first places
  float* partial; int64_t ld_partial;   // 2 chunks rows of partial sums
};

int embed_chunk(int64_t n, int64_t dim);
int64_t embed_max_chunks(int64_t n, int64_t dim);
int64_t embed_max_shares(int64_t n, int64_t vocab);
int64_t embed_range(int64_t vocab);
int64_t embed_tokens(int64_t n, int64_t vocab);
hipError_t launch_embed_lookup(const EmbedLookup& a, int tt, int ot, int id_bytes, hipStream_t s);
hipError_t launch_embed_grad(const EmbedGrad& a, int dt, int id_bytes, hipStream_t s);

}  // namespace psgd
