// Host side of the grouped expert products and the checkpointed activation
// (include/moe.h): argument validation and launches.  The activation's
// kernels are compiled here.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe.h"
#include "grouped.h"
#include "swiglu.h"

using namespace moe;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

moe_status_t launch_status() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE; }

constexpr int64_t kMaxStride = (int64_t)1 << 20;         // elements of a row stride: tile offsets stay below 2^31 bytes
constexpr int64_t kMaxExpertBytes = (int64_t)1 << 31;    // one expert's matrix, addressed by 32-bit offsets
constexpr int64_t kMaxGatherBytes = ((int64_t)1 << 32) - ((int64_t)1 << 22);  // a gathered matrix, by unsigned 32-bit
                                                                              // offsets (the tiled kernels' kOob)
constexpr int kMaxRows = 1 << 26;                        // keeps the tiled products' row tiles times column tiles,
                                                         // which workgroups number in 32 bits, below 2^31
constexpr int64_t kMaxGroups = (int64_t)1 << 30;  // rows * scale groups: the activation's grid has at most 2^32 threads

bool known_out(moe_out_t t) { return t == MOE_OUT_BF16 || t == MOE_OUT_FP32; }

// A rows operand of `width` elements of `esz` bytes for R grouped rows.
moe_status_t check_rows(const moe_rows_t& r, int R, int width, int esz, bool input) {
  if (!r.data || !aligned(r.data, 16) || !aligned(r.ids, 4) || r.rows < 0 || r.div < 1) return MOE_ERR_INVALID_ARG;
  if (!r.ids && (r.rows < R || r.div != 1)) return MOE_ERR_INVALID_ARG;
  if (!input && r.div != 1) return MOE_ERR_INVALID_ARG;
  if (r.stride < width || r.stride * esz % 16) return MOE_ERR_INVALID_ARG;
  if (r.stride >= kMaxStride) return MOE_ERR_UNSUPPORTED;
  if (input && r.ids && (int64_t)r.rows * r.stride * esz > kMaxGatherBytes) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status_t check_sizes(int R, int E, int N, int K) {
  if (R < 0 || E < 1 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  if (R >= kMaxRows || E > kMaxExperts || N % 8 || K % 8 || (int64_t)N * K * 2 >= kMaxExpertBytes)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool activation_sizes(int R, int I) {
  return I % 8 == 0 && I < kMaxStride / 2 && R < kMaxRows &&
         (int64_t)R * ((I + kCkptGroup - 1) / kCkptGroup) < kMaxGroups;
}

RowsArg rows_arg(const moe_rows_t& r) { return RowsArg{(uint8_t*)r.data, r.stride, r.rows, r.div, r.ids}; }

moe_status_t grouped(const moe_grouped_args_t* a, bool dgrad, hipStream_t st) {
  if (!a) return MOE_ERR_INVALID_ARG;
  moe_status_t rc = check_sizes(a->R, a->E, a->N, a->K);
  if (rc != MOE_OK) return rc;
  if (!known_out(a->out_type)) return MOE_ERR_INVALID_ARG;
  int group = 8;
  switch (a->weight) {
    case MOE_WEIGHT_BF16: break;
    case MOE_WEIGHT_MXFP4: group = 32; break;
    case MOE_WEIGHT_INT4: group = 128; break;
    default: return MOE_ERR_INVALID_ARG;
  }
  const bool q4 = a->weight != MOE_WEIGHT_BF16;
  if ((q4 && dgrad) || a->K % group) return MOE_ERR_UNSUPPORTED;
  if (a->R == 0) return MOE_OK;
  if (!a->offsets || !aligned(a->offsets, 4) || !a->w || !aligned(a->w, 16)) return MOE_ERR_INVALID_ARG;
  if (q4 != (a->w_scale != nullptr) || !aligned(a->w_scale, a->weight == MOE_WEIGHT_INT4 ? 2 : 1))
    return MOE_ERR_INVALID_ARG;
  const bool f32 = a->out_type == MOE_OUT_FP32;
  if ((rc = check_rows(a->in, a->R, dgrad ? a->N : a->K, 2, true)) != MOE_OK) return rc;
  if ((rc = check_rows(a->out, a->R, dgrad ? a->K : a->N, f32 ? 4 : 2, false)) != MOE_OK) return rc;
  const GroupedArgs g{a->R, a->E, a->N, a->K, a->offsets, rows_arg(a->in), rows_arg(a->out), (const uint8_t*)a->w,
                      (const uint8_t*)a->w_scale};
  const bool ok = q4 ? launch_grouped_stream(a->weight, f32, st, g) : launch_grouped_tile(dgrad, f32, st, g);
  const moe_status_t launched = launch_status();
  return ok ? launched : MOE_ERR_DEVICE;
}

}  // namespace

extern "C" {

moe_status_t moe_grouped_gemm(const moe_grouped_args_t* args, void* stream) {
  return grouped(args, false, (hipStream_t)stream);
}

moe_status_t moe_grouped_gemm_dgrad(const moe_grouped_args_t* args, void* stream) {
  return grouped(args, true, (hipStream_t)stream);
}

moe_status_t moe_grouped_gemm_wgrad(const moe_grouped_wgrad_args_t* a, void* stream) {
  if (!a) return MOE_ERR_INVALID_ARG;
  moe_status_t rc = check_sizes(a->R, a->E, a->N, a->K);
  if (rc != MOE_OK) return rc;
  if (!known_out(a->out_type) || (a->accumulate != 0 && a->accumulate != 1)) return MOE_ERR_INVALID_ARG;
  const bool f32 = a->out_type == MOE_OUT_FP32;
  if (a->accumulate && !f32) return MOE_ERR_INVALID_ARG;
  if (!a->offsets || !aligned(a->offsets, 4) || !a->dw || !aligned(a->dw, 16)) return MOE_ERR_INVALID_ARG;
  if ((rc = check_rows(a->dy, a->R, a->N, 2, true)) != MOE_OK) return rc;
  if ((rc = check_rows(a->in, a->R, a->K, 2, true)) != MOE_OK) return rc;
  const GroupedWgradArgs g{a->R, a->E, a->N, a->K, a->offsets, rows_arg(a->dy), rows_arg(a->in), (uint8_t*)a->dw};
  const bool ok = launch_grouped_wgrad(f32, a->accumulate != 0, (hipStream_t)stream, g);
  const moe_status_t launched = launch_status();
  return ok ? launched : MOE_ERR_DEVICE;
}

moe_status_t moe_swiglu_checkpoint(const void* gu, int64_t gu_stride, const float* row_weight, int32_t R, int32_t I,
                                   const int32_t* num_rows, void* h, uint8_t* codes, uint8_t* scales, void* stream) {
  if (R < 0 || I < 1) return MOE_ERR_INVALID_ARG;
  if (!activation_sizes(R, I)) return MOE_ERR_UNSUPPORTED;
  if (R == 0) return MOE_OK;
  if (!gu || !aligned(gu, 16) || gu_stride < 2 * (int64_t)I || gu_stride % 8) return MOE_ERR_INVALID_ARG;
  if (gu_stride >= kMaxStride) return MOE_ERR_UNSUPPORTED;
  if ((!h && !codes) || (codes != nullptr) != (scales != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned(h, 16) || !aligned(codes, 16) || !aligned(row_weight, 4) || !aligned(num_rows, 4))
    return MOE_ERR_INVALID_ARG;
  launch_swiglu_checkpoint((const uint8_t*)gu, gu_stride, row_weight, R, I, num_rows, (uint8_t*)h, codes, scales,
                           (hipStream_t)stream);
  return launch_status();
}

moe_status_t moe_swiglu_checkpoint_grad(const uint8_t* codes, const uint8_t* scales, const void* dh,
                                        const float* row_weight, int32_t R, int32_t I, const int32_t* num_rows,
                                        void* dgu, void* h, float* dweight, void* stream) {
  if (R < 0 || I < 1) return MOE_ERR_INVALID_ARG;
  if (!activation_sizes(R, I)) return MOE_ERR_UNSUPPORTED;
  if (R == 0) return MOE_OK;
  if (!codes || !scales || !dh || !dgu) return MOE_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(dh, 16) || !aligned(dgu, 16) || !aligned(h, 16) || !aligned(row_weight, 4) ||
      !aligned(dweight, 4) || !aligned(num_rows, 4))
    return MOE_ERR_INVALID_ARG;
  launch_swiglu_grad(codes, scales, (const uint8_t*)dh, row_weight, R, I, num_rows, (uint8_t*)dgu, (uint8_t*)h,
                     dweight, (hipStream_t)stream);
  return launch_status();
}

}  // extern "C"
