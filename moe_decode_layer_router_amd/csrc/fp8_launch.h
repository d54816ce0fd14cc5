// fp8_launch.h -- enqueue functions of the FP8 steps (arguments already checked).
#pragma once

#include "host.h"

namespace moeblk {

// rows [M][K] (in_type) -> e4m3 [M][Kb * 128] and scales [Kb][M]
void launch_fp8_quant(const void* x, int in_type, uint8_t* xq, float* xs, int M, int K,
                      hipStream_t stream);
// n canonical matrices [N][K] with scales [Nb][Kb] -> packed (fp8_dev.h);
// which = MOE_W13: rows interleaved gate / up (common.h packed_row)
void launch_fp8_pack(const void* q, const void* scales, void* packed, int n, int N, int K,
                     int which, hipStream_t stream);

}  // namespace moeblk
