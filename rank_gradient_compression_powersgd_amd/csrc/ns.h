// Newton-Schulz orthogonalisation of a group of matrices: descriptors shared by its kernels
// (k_ns.hip, k_ns_gemm.hip) and its host side (ns_group.hip).
#pragma once

#include <vector>

#include "psgd_internal.h"

namespace psgd {

// The iteration works on the smaller side: X is s x l with s = min(m, n), l = max(m, n), the
// update transposed when m > n. Everything between the first and the last kernel lives in the
// workspace as fp16 values times a fixed power of two, zero-padded to whole tiles:
//   X  (sp x lp)  as hi + lo, X * 2^14 = hi + lo to 2^-22 of itself, or to lo's floor of 2^-25 for
//                 |X| below 2^-17: singular values stay below 4
//   A  (sp x sp)  X X^T, times 2^14 (entries bounded by the squared singular values)
//   B  (sp x sp)  b A + c A A, times 2^10
// All of them are stored as panels of 32 columns, one after another, 64 bytes per row within a panel:
// what a product stage of 32 k loads of a tile's rows (and, read the other way round, of its columns)
// is then contiguous (a stage of a 256-wide tile that has the chip to itself: 0.43 us, 0.75 row by
// row).
// A and B are symmetric: only the tiles on and below the diagonal are computed, and each is
// stored twice.
constexpr float kNsScaleX = 16384.0f, kNsScaleA = 16384.0f, kNsScaleB = 1024.0f;

struct NsMat {
  const void* in;    int64_t ld_in;      // update (Newton-Schulz) or gradient (Muon), m x n
  float* mom;                            // Muon: m x n fp32 momentum (leading dimension n)
  void* out;         int64_t ld_out;     // orthogonal factor (Newton-Schulz) or parameter (Muon)
  int32_t m, n;
  int32_t s, l, sp, lp;
  int32_t flip;                          // 1: X holds the transposed update (m > n)
  int32_t parts, part_rows;              // partial sums of squares: rows per part
  float factor[2];                       // Muon: scale of the orthogonal update, by NsArgs::adjust
  uint16_t* xh[2];   uint16_t* xl[2];    // X, ping-pong between steps
  uint16_t* ah;      uint16_t* al;       // A (lo: accurate products only)
  uint16_t* bh;      uint16_t* bl;       // B likewise
  double* partial;                       // parts fp64 sums of u^2
};

// Scalars of one call.
struct NsArgs {
  float a, b, c;
  double eps;
  int steps;
  // Muon (mu unused otherwise)
  int muon, nesterov, adjust;
  float lr, mu, weight_decay;
  const int32_t* skip;                   // the step's skip word (NULL, up to NsGroup::run: never skipped)
  const float* norm;                     // norm[1] = clipping factor; NULL: 1
};

// An item of a product list: its tile, and a copy of its matrix, so that a workgroup waits for one
// load and not for two in a row before it can ask for its operands.
struct NsItem {
  Work w;
  NsMat d;
};

// The products of one step: A = X X^T, B = b A + c A A, X <- a X + B X.
enum NsStage : int { NS_GRAM = 0, NS_POLY = 1, NS_UPDATE = 2 };

hipError_t launch_ns_norm(int it, const NsMat* mats, const Work* work, int n_work, const NsArgs& a, hipStream_t s);
hipError_t launch_ns_x0(int it, const NsMat* mats, const Work* work, int n_work, const NsArgs& a, hipStream_t s);
// One product stage's tiles: (matrix, first row, first column, partial slot), padded for
// xcd_remap. Tiles are multiples of 64 wide, so the low 6 bits of the row and the column carry the
// part of a tile whose K is split and the number of parts (0: not split).
struct NsList {
  int tile = 0;
  const NsItem* work = nullptr;   int n_work = 0;
  const NsItem* reduce = nullptr; int n_reduce = 0;    // the split tiles, with their first slot
  float* partial = nullptr;                          // tile * tile floats per slot
};
// Stages of 32 k a product over K takes (accurate: the hi and the lo plane each), always even, and
// the stages of one of `splits` parts (whole k and an even number).
__host__ __device__ inline int ns_stages(int K, bool accurate) { return 2 * ((K + 63) / 64) * (accurate ? 2 : 1); }
__host__ __device__ inline int ns_part(int stages, int splits, bool accurate) {
  const int unit = accurate ? 4 : 2;
  return ((stages + splits - 1) / splits + unit - 1) / unit * unit;
}
// One product stage of step `step` (0-based); `last` writes the caller's output.
hipError_t launch_ns_gemm(NsStage st, bool accurate, int ot, bool last, const NsList& l, int step,
                          const NsArgs& a, hipStream_t s);

// A group of matrices orthogonalised together: validated by the caller, laid out and allocated
// here. One instance serves one call at a time.
class NsGroup {
 public:
  struct Item { const void* in; int64_t ld_in; float* mom; void* out; int64_t ld_out; int64_t m, n; };
  ~NsGroup();
  // types are GradType; adds no host work to later calls. Sides are at most 2^22 (the caller has
  // checked). Returns hipErrorOutOfMemory when the workspace does not fit.
  hipError_t create(const std::vector<Item>& items, int in_type, int out_type, bool accurate);
  // adjust selects NsMat::factor for Muon calls: 0 sqrt(max(1, m/n)), 1 0.2 sqrt(max(m, n))
  hipError_t run(const NsArgs& a, int adjust, hipStream_t s);
  size_t workspace_bytes() const { return bytes_; }

 private:
  struct List { int off = 0, cnt = 0; };
  void* buf_ = nullptr;                  // workspace, descriptors, work lists
  size_t bytes_ = 0;
  NsMat* d_mats_ = nullptr;
  int32_t* d_zero_ = nullptr;            // a skip word for calls that have none
  Work* d_work_ = nullptr;
  List norm_, x0_;
  NsList gram_, poly_, update_;
  int it_ = 0, ot_ = 0;
  bool accurate_ = false;
};

}  // namespace psgd
