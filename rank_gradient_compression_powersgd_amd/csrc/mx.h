// Microscaled 4-bit matrices: layout, and the arguments of their kernels (k_mx.hip, k_mx_gemm.hip).
//
// A matrix of `rows` x k, k the dimension its products sum over. Columns are padded with zeros to panels
// of 128. Codes: panel after panel, 64 bytes a row (element 2 i in the low nibble of byte i), so 16 rows
// of a panel are one contiguous KB: an MFMA operand. Exponent bytes, one per row and 32 columns: panel
// after panel, per 64 rows 256 bytes, byte 4 (16 g + r % 16) + r / 16 % 4 for block g of the panel: lane
// (r % 16, g) of an MFMA finds those of four 16-row tiles in one word. Rows of the exponents are
// padded to 64.
#pragma once

#include "psgd_internal.h"

namespace psgd {

constexpr int kMxBlock = 32;            // elements under one exponent
constexpr int kMxPanel = 128;           // columns of a panel
constexpr int kMxRowBytes = 64;         // bytes of a row's codes in a panel
constexpr int kMxGroup = 64;            // rows of an exponent group
constexpr int kMxGroupBytes = 256;      // its bytes in a panel

struct MxView {
  uint8_t* codes; uint8_t* scales;
  int64_t rows, k, panels, groups;
};
inline MxView mx_view(void* data, int64_t rows, int64_t k) {
  const int64_t panels = (k + kMxPanel - 1) / kMxPanel, groups = (rows + kMxGroup - 1) / kMxGroup;
  uint8_t* p = static_cast<uint8_t*>(data);
  return MxView{p, p + panels * rows * kMxRowBytes, rows, k, panels, groups};
}
inline int64_t mx_bytes(int64_t rows, int64_t k) {
  const MxView v = mx_view(nullptr, rows, k);
  return v.panels * (rows * kMxRowBytes + v.groups * kMxGroupBytes);
}

struct MxQuantize {
  const void* x; int64_t ld, m, n;
  MxView row, col;                      // of x and of its transpose; codes NULL: not wanted
  uint64_t seed;
  const int32_t* step;                  // NULL: 0
};

struct MxProduct {
  MxView p, q;                          // C's columns and rows: B (n rows) and A (m rows)
  int64_t m, n;
  void* c; int64_t ldc;
  const float* scale;                   // NULL: 1
  int32_t accumulate;
  int32_t splits, per;                  // parts of the panels, panels of a part
  float* partial;                       // splits > 1: their fp32 results, m x n each
};

struct MxPlan { int tile; int splits; };  // tile 0: few rows
MxPlan mx_plan(int64_t m, int64_t n, int64_t panels);

hipError_t launch_mx_quantize(const MxQuantize& a, int it, bool stochastic, hipStream_t s);
hipError_t launch_mx_dequantize(const MxView& a, void* out, int64_t ld, int ot, hipStream_t s);
hipError_t launch_mx_product(const MxProduct& a, int tile, int ot, hipStream_t s);

}  // namespace psgd
