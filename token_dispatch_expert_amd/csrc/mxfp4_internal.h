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

}  // namespace moe
