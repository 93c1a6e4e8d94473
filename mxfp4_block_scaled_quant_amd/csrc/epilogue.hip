// The epilogue of mxfp4_linear_act: out = act(y) (times the gate's other
// half) + residual, from fp32 y, rounded once (gfx950).
#include "mxfp4_device.h"
#include "mxfp4_launch.h"

namespace mxfp4 {

__global__ __launch_bounds__(256) void epilogue_kernel(EpilogueArgs p) {
  const int cols = p.gated ? p.N / 2 : p.N;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)p.M * cols) return;
  const int64_t m = i / cols;
  const int n = (int)(i % cols);
  const float* y = p.y + m * p.N;
  float v = activate(y[n], p.act);
  if (p.gated) v *= y[cols + n];
  if (p.residual) v += bf16_to_f32(p.residual[m * p.ldr + n]);
  if (p.out_f32)
    static_cast<float*>(p.out)[m * p.ldo + n] = v;
  else
    static_cast<uint16_t*>(p.out)[m * p.ldo + n] = f32_to_bf16_rne(v);
}

hipError_t launch_epilogue(const EpilogueArgs& p, hipStream_t stream) {
  const int64_t n = (int64_t)p.M * (p.gated ? p.N / 2 : p.N);
  epilogue_kernel<<<dim3((unsigned)((n + 255) / 256)), 256, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace mxfp4
