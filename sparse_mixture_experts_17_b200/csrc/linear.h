// linear.h -- host-side interface between linear.cu (entry points, elementwise
// passes) and linear_tc.cu (the tensor-core products).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

// The three products, as out[c, m] = sum_k A[m, k] B[c, k] with m contiguous in
// the output:
//   LIN_FWD  m = d_out, c = rows,  k = d_in          A = W_e, B = x
//   LIN_DX   m = d_in,  c = rows,  k = d_out         A = W_e^T, B = dz
//   LIN_DW   m = d_in,  c = d_out, k = the group's rows  A = x^T, B = dz^T
enum LinMode { LIN_FWD = 0, LIN_DX = 1, LIN_DW = 2 };

struct LinArgs {
    const uint16_t *x, *W, *dz;
    const float *bias;            // LIN_FWD, [E, d_out] or NULL
    const uint16_t *residual;     // LIN_FWD, or NULL
    uint16_t *out, *z;            // z: LIN_FWD, or NULL
    float *part;                  // LIN_DW split along the rows: fp32 sums [splits, E, d_out, d_in]
    const int32_t *offsets;       // NULL: one group of all rows
    int rows, d_in, d_out, E, act;
    int splits;                   // LIN_DW
    // The product needs nothing of the kernel launched just before it, and what it does
    // need had completed before that one was let start its successor: it starts at once,
    // beside that kernel, and lets its own successor start at once too; it waits for its
    // predecessor only before it ends, on every way out (so that whatever waits for this
    // product has waited for both). See moe_linear_backward.
    bool late;
    bool starve;                  // MOE_FLAG_TEST_TIMEOUT
    uint32_t *status;
};

// Parts that LIN_DW cuts the rows of each group into (1: none).
int lin_dw_splits(const moe_linear_t &s);

int launch_linear(LinMode mode, const LinArgs &p, cudaStream_t st);

} // namespace moe
