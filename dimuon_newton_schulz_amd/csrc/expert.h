// Experts: what the kernels (expert_kernels.hip, linear_kernels.hip) and the
// host side (expert_api.hip) share.
#pragma once

#include "common.h"

namespace muon {

// ---------------------------------------------------------------------------
// Tokens sorted by expert and back
// ---------------------------------------------------------------------------
struct Routes {
  int32_t* offsets;   // experts + 1
  int32_t* order;     // slots
  int32_t* place;     // slots
  int32_t tokens, top, experts, slots;
};

constexpr int kSortThreads = 1024;
constexpr int kSortAlone = 8192;        // slots that one workgroup sorts, alone if they are all
constexpr int kSortSummed = 256;        // workgroups up to which each adds up the others' counts itself
constexpr int kMaxExperts = 1024;

// Slots of a workgroup, number of workgroups and rows of counts of a sort.
inline void sort_shape(int64_t slots, int64_t& per, int64_t& blocks) {
  per = slots;
  if (slots > kSortAlone) {
    per = (slots + kSortSummed - 1) / kSortSummed;
    per = (per + kSortThreads - 1) / kSortThreads * kSortThreads;
    per = per < kSortAlone ? per : kSortAlone;
  }
  blocks = slots > kSortAlone ? (slots + per - 1) / per : 1;
}

// Rows between tokens and experts.  Strides in elements.
struct MoveArgs {
  const void* tok;        // token rows (x, dy, or the residual; may be NULL as a residual)
  void* tok_out;          // token rows written (combine)
  const void* rows;       // sorted rows read
  void* rows_out;         // sorted rows written
  const void* weights;    // slots, or NULL
  void* dweights;         // slots
  int64_t tok_ld, tok_out_ld, rows_ld, rows_out_ld;
  const int32_t* place;
  int32_t tokens, top, width, slots, w_dt;
};

hipError_t launch_expert_sort(const void* ids, int id_bytes, const Routes& r, int32_t* counts, hipStream_t s);
hipError_t launch_expert_gather(const MoveArgs& a, int dt, bool vec, hipStream_t s);
hipError_t launch_expert_combine(const MoveArgs& a, int dt, bool vec, hipStream_t s);
hipError_t launch_expert_combine_grad(const MoveArgs& a, int dt, bool vec, hipStream_t s);

// ---------------------------------------------------------------------------
// Products over groups of rows
// ---------------------------------------------------------------------------
enum LinearMode : int32_t {
  LIN_FORWARD = 0,    // y = act(x W^T + b) + residual    rows x out, k = in
  LIN_INPUT = 1,      // dx = (dz W) act'(x_pre)          rows x in,  k = out
  LIN_WEIGHT = 2      // dW (+)= dz^T x                   out x in,   k = rows of the group
};

struct LinArgs {
  const void* p;            // rows' operand: x (forward), dz (gradients)
  const void* q;            // W (forward, input), x (weight gradient)
  void* c;                  // y, dx or dW
  void* pre;                // forward: z, or NULL
  const void* bias;         // forward: groups x n, or NULL
  const void* aux;          // forward: residual; input gradient: x_pre; or NULL
  const int32_t* offsets;   // groups + 1, or NULL: one group of all rows
  float* part;              // weight gradient in several parts: their sums, parts x groups x m x n
  int64_t ldp, ldq, ldc, ldpre, ldaux;   // row strides, elements
  int64_t gq, gc;           // group strides of W (q) and dW (c), elements
  int32_t rows, m, n, k;    // m: weight gradient only (out); k: not the weight gradient
  int32_t groups, act, c_dt, accumulate, parts;
};

// `align`: 16 where every row lies on 16-byte borders and holds whole runs of
// eight, 4 where rows lie on 4-byte borders, else 2.
hipError_t launch_linear(const LinArgs& a, int mode, int dt, int align, hipStream_t s);
// Whether the product's tiles fit one launch.
bool linear_fits(const LinArgs& a, int mode, int dt, int align);
// Sum of the parts of a weight gradient.
hipError_t launch_linear_join(const LinArgs& a, hipStream_t s);
// Parts that the rows of a weight gradient (a bias gradient) are split in.
int linear_weight_parts(int64_t rows, int64_t out, int64_t in, int64_t groups);
// dz = dy act'(pre) on the groups' rows.
hipError_t launch_linear_slope(const void* dy, int64_t ld_dy, const void* pre, int64_t ld_pre, void* dz, int64_t ld_dz,
                               const int32_t* offsets, int groups, int64_t rows, int64_t out, int act, int dt, int align,
                               hipStream_t s);
// The same for bf16, with the unrounded terms' column sums per tile of rows,
// linear_slope_tiles x out; and db (a.c) (+)= the groups' sums of them.  a:
// n = out, rows, groups, offsets, act; c, c_dt, accumulate.  dz may be NULL.
int64_t linear_slope_tiles(int64_t rows, int64_t out, int64_t groups);
hipError_t launch_linear_slope_sums(const LinArgs& a, const void* dy, int64_t ld_dy, const void* pre, int64_t ld_pre,
                                    void* dz, int64_t ld_dz, float* sums, hipStream_t s);
hipError_t launch_linear_sums(const LinArgs& a, const float* sums, hipStream_t s);
int linear_bias_parts(int64_t rows, int64_t groups);
bool linear_bias_fits(int64_t out, int64_t groups);
// db (+)= column sums of every group's rows, in `parts` parts.
hipError_t launch_linear_bias(const void* dz, int64_t ld, const int32_t* offsets, int groups, int64_t rows, int64_t out,
                              void* db, int dt, int grad_dt, int accumulate, float* part, int parts, hipStream_t s);

}  // namespace muon
