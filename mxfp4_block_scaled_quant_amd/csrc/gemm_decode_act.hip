// The small-M kernels with an activation, a gate and a residual in their
// epilogue: the source of gemm_decode.hip built again.
#define MXFP4_DECODE_ACT 1
#include "gemm_decode.hip"
