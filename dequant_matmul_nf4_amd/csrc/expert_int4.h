// Launches of the expert products and of int4 weights, and what their kernels share.
#pragma once

#include "nf4_internal.h"

namespace nf4i {

// ---- uniform 4-bit weights with group scales (nf4_int4_weight)
struct Int4Weight {
  const uint8_t* packed;
  int64_t rows, cols;
  int group;             // 32, 64 or 128; cols is a multiple of it
  const void* scales;    // [rows][cols / group]
  int scale_type;        // nf4_dtype: 0 float32, 1 bfloat16, 2 float16
  const uint8_t* zeros;  // [rows][cols / group], or null: 8 everywhere
};
hipError_t launch_int4_quantize(const void* x, int x_type, int64_t n, int group, uint8_t* packed, void* scales,
                                int scale_type, uint8_t* zeros, hipStream_t s);
hipError_t launch_int4_dequantize(const Int4Weight& w, void* out, int out_type, hipStream_t s);
hipError_t launch_int4_gemv(const Int4Weight& w, const uint16_t* x, int x_f16, int64_t m, void* y, int y_type,
                            hipStream_t s);

// ---- mixture-of-experts products: `experts` weights stacked along the rows
constexpr int kMaxExperts = 1024;
struct ExpertRows {        // which rows of the product belong to which expert
  const int32_t* offsets;  // [experts + 1]
  int experts;
  int64_t m;               // rows of the product's buffers: offsets are clamped to them
  // Where two kernels share a product: a first one takes tiles of kCoverRows
  // rows in full rounds of `cover_slots` workgroups, cover_units of them per
  // tile, and the other the rest.  0: not shared.
  int cover_slots, cover_units;
};
constexpr int kCoverRows = 256;
struct ExpertX {           // where the product's row p finds its activations
  const uint16_t* x;       // [rows][cols]
  int64_t rows;
  const int32_t* index;    // row index[p] / slots of x, or null: row p
  int slots;
};
size_t expert_plan_workspace(int64_t n, int experts);
hipError_t launch_expert_plan(const int32_t* ids, int64_t n, int experts, int32_t* order, int32_t* position,
                              int32_t* offsets, void* ws, hipStream_t s);
hipError_t launch_expert_gemm(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const ExpertRows& er,
                              const ExpertX& ex, uint16_t* y, hipStream_t s);
// Its form for few rows per expert.
hipError_t launch_expert_skinny(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const ExpertRows& er,
                                const ExpertX& ex, uint16_t* y, hipStream_t s);
hipError_t launch_expert_gemm_dx(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const ExpertRows& er,
                                 const uint16_t* dy, uint16_t* dx, hipStream_t s);
// Its form for few tiles: the reduction split over the waves of a workgroup.
hipError_t launch_expert_skinny_dx(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const ExpertRows& er,
                                   const uint16_t* dy, uint16_t* dx, hipStream_t s);
hipError_t launch_expert_combine(const uint16_t* y, int64_t m, const int32_t* position, int64_t tokens, int slots,
                                 int64_t cols, const float* weights, uint16_t* out, hipStream_t s);
hipError_t launch_expert_combine_backward(const uint16_t* dout, const uint16_t* y, int64_t m, const int32_t* position,
                                          int64_t tokens, int slots, int64_t cols, const float* weights, uint16_t* dy,
                                          float* dweights, hipStream_t s);

// Workgroups numbered over a grid of two dimensions: the threads of one are
// counted in 32 bits.  Kernels leave where the number is past their last.
inline dim3 block_grid(int64_t blocks) {
  const int64_t gy = (blocks + (1 << 20) - 1) >> 20;
  return dim3(static_cast<unsigned>((blocks + gy - 1) / gy), static_cast<unsigned>(gy));
}
__device__ __forceinline__ int64_t block_number() {
  return static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
}

}  // namespace nf4i
