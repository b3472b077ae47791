// Expert products on rows grouped by expert: what their kernels share.
#pragma once

#include "moe_device.h"

namespace moe {

// A rows operand as the kernels take it (moe_rows_t): grouped row i is matrix
// row i, or ids[i]/div; `rows` bounds it.
struct RowsArg {
  uint8_t* p;
  int64_t stride;  // elements
  int rows, div;
  const int32_t* ids;
};

// Matrix row of grouped row i with id f (read only where there are ids), or -1
// when its id is outside the matrix.
__device__ __forceinline__ int row_of(const RowsArg& r, int i, int f) {
  if (!r.ids) return i < r.rows ? i : -1;
  const int m = f < 0 ? -1 : (r.div == 1 ? f : (int)((unsigned)f / (unsigned)r.div));
  return m < r.rows ? m : -1;
}
__device__ __forceinline__ int row_of(const RowsArg& r, int i) { return row_of(r, i, r.ids ? r.ids[i] : 0); }

struct GroupedArgs {
  int R, E, N, K;
  const int32_t* offsets;
  RowsArg in, out;
  const uint8_t* w;
  const uint8_t* w_scale;
};

struct GroupedWgradArgs {
  int R, E, N, K;
  const int32_t* offsets;
  RowsArg dy, in;
  uint8_t* dw;
};

// Row range of expert e, its ends clamped so that no offset leads outside
// [0, R].
__device__ __forceinline__ void group_range(const int32_t* offsets, int e, int R, int* lo, int* hi) {
  const int a = offsets[e], b = offsets[e + 1];
  *lo = min(max(a, 0), R);
  *hi = min(max(b, *lo), R);
}

// Host launchers; false when the launch could not be set up.
bool launch_grouped_tile(bool dgrad, bool f32, hipStream_t st, const GroupedArgs& a);
bool launch_grouped_wgrad(bool f32, bool accumulate, hipStream_t st, const GroupedWgradArgs& a);
bool launch_grouped_stream(int format, bool f32, hipStream_t st, const GroupedArgs& a);

}  // namespace moe
