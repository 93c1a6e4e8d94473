// The large-M kernel with an activation, a gate and a residual in its epilogue at 256-wide
// output tiles: the source of gemm_prefill.hip built again.
#define MXFP4_PREFILL_FORM 1
#define MXFP4_PREFILL_BN 256
#include "gemm_prefill.hip"
