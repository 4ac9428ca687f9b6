// Launchers of the grouped products (grouped.hip); arguments are validated by the C ABI.
#pragma once

#include "common.h"

namespace exmoe {

struct GroupedArgs {
  const uint16_t* a;         // x of the forward product, dy of both gradients
  const uint16_t* b;         // W of the forward product and of the gradient of x; x of the gradient of W
  size_t lda, ldb, b_stride; // elements per row of a and b, elements per expert of W
  int len_a, len_b;          // readable elements of a row (past its length: zeros)
  const int32_t* offsets;    // [E + 1]
  const int32_t* row_index;  // sorted row -> row_index / row_div = row of x; or null (same row)
  int row_div, x_rows;
  int rows, N, K, E;
  void* out;
  size_t ldo, o_stride;      // elements per output row, per expert (gradient of W)
  int fp16, out_f32;
  int vec;                   // 16-byte stores: the base and every row and expert of out are 16-byte aligned
  const int32_t* flat_to_sorted;   // gradient of x summed per token, or null
  int k;
  float* ws;                 // rows of the summed gradient, or the partial sums of W's
  uint16_t *pack_a, *pack_b; // room for operands with padded rows (see grouped_workspace)
};

// Workspace of a call: bytes of its parts (0: not needed); op as in enum exmoe_grouped_op.
struct GroupedWorkspace {
  size_t sums;               // fp32: rows of the summed gradient, or partial sums
  size_t pack_a, pack_b;     // operands whose rows are no multiple of 16 bytes, with padded rows
  size_t total() const { return sums + pack_a + pack_b; }
};
GroupedWorkspace grouped_workspace(int op, int rows, int N, int K, int E, int k);
hipError_t launch_grouped_mm(const GroupedArgs& a, hipStream_t s);
hipError_t launch_grouped_dgrad(const GroupedArgs& a, hipStream_t s);
hipError_t launch_grouped_wgrad(const GroupedArgs& a, hipStream_t s);

}  // namespace exmoe
