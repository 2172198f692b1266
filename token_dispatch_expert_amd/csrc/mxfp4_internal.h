// Launchers of the MXFP4 kernels, for the C ABI host code.
#pragma once

#include "moe_internal.h"

namespace moe {

// E matrices of `rows` rows, or (f2s [rows, k], E = 1) each row into its k sorted rows; codes [.., d / 2], scales
// [E][ceil(d/256)][rows * k][8]; d a multiple of 32.
long long mx_row_grid(long long rows, int d);  // workgroups, at most
hipError_t launch_mx_quantize(const void* x, bool bf16, int E, int rows, int k, int d, const int32_t* f2s,
                              void* codes, void* scales, hipStream_t stream);
hipError_t launch_mx_dequantize(const void* codes, const void* scales, int E, int rows, int d, void* out,
                                bool bf16, hipStream_t stream);

// Products by expert: g.a = x [rows, K] in bf16, or MXFP4 codes with a_scales; g.b = W [E, N, K] codes with b_scales.
// With g.b2 (the same, b2_scales) the gate and up products with SwiGLU: out h [rows, N] in bf16, or MXFP4 codes
// with out_scales; else out y in fp32 or bf16.
struct MxGemmArgs {
  GroupedGemmArgs g;
  bool x4;  // rows in MXFP4
  const uint8_t *a_scales, *b_scales, *b2_scales;
  uint8_t* out_scales;
};
bool mx_gemm_fits(const MxGemmArgs& a);
bool mx_ffn_fits(int rows, int E, int d, int d_ff);  // the products of a grouped FFN
hipError_t launch_mx_gemm(const MxGemmArgs& a, hipStream_t stream);
// Their input gradient: g.a = dy [rows, N] in bf16, g.b = W's codes with b_scales, g.a2, g.b2 and b2_scales a second pair
// or null; g.out = dx [rows, K].
bool mx_dgrad_fits(const MxGemmArgs& a);
hipError_t launch_mx_dgrad(const MxGemmArgs& a, hipStream_t stream);

}  // namespace moe
