// The large-M kernel over the experts' row tiles at 256-wide
// output tiles: the source of gemm_prefill.hip built again.
#define MXFP4_PREFILL_FORM 2
#define MXFP4_PREFILL_BN 256
#include "gemm_prefill.hip"
