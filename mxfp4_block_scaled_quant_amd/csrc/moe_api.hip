// C ABI of the feed-forward operators (declared in include/mxfp4.h): argument
// validation on the host, before any HIP call, and dispatch.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/mxfp4.h"
#include "moe_launch.h"
#include "mxfp4_launch.h"

namespace mxfp4 {

namespace {

constexpr int64_t kMaxInt = 0x7FFFFFFF;
constexpr int64_t kMaxDim = 1 << 20;        // hidden and inner sizes
constexpr int64_t kMaxPairs = 1 << 24;      // tokens * top_k
constexpr int64_t kMaxStride = 1ll << 40;   // elements: products with sizes stay in 64 bits

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int launched(hipError_t e) { return e == hipSuccess ? MXFP4_OK : MXFP4_ERR_LAUNCH; }
// A row stride over rows of n elements; one row's is never used.
inline bool row_ok(int64_t stride, int64_t n, int64_t rows) {
  return rows <= 1 || (stride >= n && stride <= kMaxStride);
}
inline int64_t used(int64_t stride, int64_t rows) { return rows > 1 ? stride : 0; }

// Bytes of one expert's weight of N rows of K in the GEMM layout.
inline int64_t one_weight(int64_t N, int64_t K) { return cdiv(N, 16) * cdiv(K, 128) * 1024; }

int moe_shape(int64_t tokens, int64_t top_k, int64_t experts, int64_t hidden, int64_t inner, int gated) {
  if (tokens < 0 || top_k < 1 || top_k > kMaxTopK || experts < 1 || experts > kMaxExperts) return MXFP4_ERR_SHAPE;
  if (hidden < 32 || hidden % 32 || hidden > kMaxDim || inner < 32 || inner % 32 || inner > kMaxDim)
    return MXFP4_ERR_SHAPE;
  if (tokens > kMaxPairs / top_k) return MXFP4_ERR_SHAPE;
  if (one_weight(inner * (gated ? 2 : 1), hidden) > kMaxInt || one_weight(hidden, inner) > kMaxInt)
    return MXFP4_ERR_SHAPE;
  // x in MXFP4 through 32-bit buffer offsets
  if (tokens * cdiv(hidden, 128) * 64 > kMaxInt) return MXFP4_ERR_SHAPE;
  // workgroups of a launch: 16-row strips times 32-column blocks or K-steps
  const int64_t strips = (tokens * top_k + 15 * experts) / 16;
  const int64_t widest = (hidden > inner ? hidden : inner) / 32 + 16;
  if (strips * widest > kMaxInt) return MXFP4_ERR_SHAPE;
  return MXFP4_OK;
}

}  // namespace

}  // namespace mxfp4

using namespace mxfp4;

extern "C" {

int moe_route(const void* logits, int64_t ld, int logits_dtype, const void* bias, int64_t tokens, int64_t experts,
              int64_t top_k, int scoring, int64_t groups, int64_t top_groups, int64_t group_top, int renormalize,
              float scale, void* weights, int64_t ldw, void* ids, int64_t ldi, void* stream) {
  if (logits_dtype != MXFP4_OUT_BF16 && logits_dtype != MXFP4_OUT_F32) return MXFP4_ERR_ARG;
  if (scoring != MOE_SCORE_SOFTMAX && scoring != MOE_SCORE_SIGMOID) return MXFP4_ERR_ARG;
  if (group_top != 1 && group_top != 2) return MXFP4_ERR_ARG;
  if (tokens < 0 || tokens > kMaxInt || experts < 1 || experts > kMaxExperts) return MXFP4_ERR_SHAPE;
  if (top_k < 1 || top_k > kMaxTopK || top_k > experts) return MXFP4_ERR_SHAPE;
  if (groups < 1 || groups > kMaxTopK || experts % groups || top_groups < 1 || top_groups > groups)
    return MXFP4_ERR_SHAPE;
  if (groups > 1 && top_k > top_groups * (experts / groups)) return MXFP4_ERR_SHAPE;
  if (!row_ok(ld, experts, tokens) || !row_ok(ldw, top_k, tokens) || !row_ok(ldi, top_k, tokens))
    return MXFP4_ERR_SHAPE;
  if (tokens == 0) return MXFP4_OK;
  if (!logits || !weights || !ids) return MXFP4_ERR_NULL;
  if (!aligned(logits, logits_dtype == MXFP4_OUT_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(weights, 4) ||
      !aligned(ids, 4))
    return MXFP4_ERR_ALIGN;
  const int st = device_cus(nullptr);
  if (st) return st;
  RouteArgs p{};
  p.logits = logits;
  p.ld = used(ld, tokens);
  p.bias = (const float*)bias;
  p.weights = (float*)weights;
  p.ldw = used(ldw, tokens);
  p.ids = (int32_t*)ids;
  p.ldi = used(ldi, tokens);
  p.tokens = tokens;
  p.experts = (int)experts;
  p.top_k = (int)top_k;
  p.groups = top_groups < groups ? (int)groups : 1;
  p.kept = (int)top_groups;
  p.group_top = (int)group_top;
  p.renormalize = renormalize != 0;
  p.scale = scale;
  return launched(launch_moe_route(p, logits_dtype == MXFP4_OUT_F32, scoring == MOE_SCORE_SIGMOID,
                                   (hipStream_t)stream));
}

size_t mxfp4_moe_workspace_bytes(int64_t tokens, int64_t top_k, int64_t experts, int64_t hidden, int64_t inner) {
  if (moe_shape(tokens, top_k, experts, hidden, inner, 0) || tokens == 0) return 0;
  return moe_workspace_bytes(tokens, top_k, experts, hidden, inner);
}

int mxfp4_moe(const void* x, int64_t ldx, const void* ids, int64_t ldi, const void* weights, int64_t ldw,
              const void* up_pre, const void* up_scales, const void* up_bias, const void* down_pre,
              const void* down_scales, const void* down_bias, const void* residual, int64_t ldr, void* out,
              int64_t ldo, int64_t tokens, int64_t top_k, int64_t experts, int64_t hidden, int64_t inner,
              int activation, int gated, void* workspace, size_t workspace_bytes, void* stream) {
  if (activation < MXFP4_ACT_NONE || activation > MXFP4_ACT_RELU) return MXFP4_ERR_ARG;
  int st = moe_shape(tokens, top_k, experts, hidden, inner, gated);
  if (st) return st;
  if (!row_ok(ldx, hidden, tokens) || !row_ok(ldi, top_k, tokens) || !row_ok(ldw, top_k, tokens) ||
      !row_ok(ldo, hidden, tokens) || (residual && !row_ok(ldr, hidden, tokens)))
    return MXFP4_ERR_SHAPE;
  if (workspace_bytes < mxfp4_moe_workspace_bytes(tokens, top_k, experts, hidden, inner)) return MXFP4_ERR_WORKSPACE;
  if (tokens == 0) return MXFP4_OK;
  if (!x || !ids || !weights || !up_pre || !up_scales || !down_pre || !down_scales || !out || !workspace)
    return MXFP4_ERR_NULL;
  if (!aligned(x, 16) || (tokens > 1 && ldx % 8) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(up_pre, 16) || !aligned(up_scales, 4) || !aligned(down_pre, 16) || !aligned(down_scales, 4) ||
      !aligned(up_bias, 2) || !aligned(down_bias, 2) || !aligned(out, 8) || (tokens > 1 && ldo % 4) ||
      !aligned(residual, 8) || (residual && tokens > 1 && ldr % 4) || !aligned(workspace, 256))
    return MXFP4_ERR_ALIGN;
  int cus = 0;
  st = device_cus(&cus);
  if (st) return st;
  MoeArgs p{};
  p.x = (const uint16_t*)x;
  p.ldx = used(ldx, tokens);
  p.ids = (const int32_t*)ids;
  p.ldi = used(ldi, tokens);
  p.weights = (const float*)weights;
  p.ldw = used(ldw, tokens);
  p.up = (const uint8_t*)up_pre;
  p.up_scales = (const uint8_t*)up_scales;
  p.up_bias = (const uint16_t*)up_bias;
  p.down = (const uint8_t*)down_pre;
  p.down_scales = (const uint8_t*)down_scales;
  p.down_bias = (const uint16_t*)down_bias;
  p.residual = (const uint16_t*)residual;
  p.ldr = used(ldr, tokens);
  p.out = (uint16_t*)out;
  p.ldo = used(ldo, tokens);
  p.tokens = tokens;
  p.top_k = (int)top_k;
  p.experts = (int)experts;
  p.hidden = (int)hidden;
  p.inner = (int)inner;
  p.gated = gated != 0;
  p.act = activation;
  p.cus = cus;
  p.work = (uint8_t*)workspace;
  return launched(launch_moe(p, (hipStream_t)stream));
}

size_t mxfp4_linear_act_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return mxfp4_linear_workspace_bytes(M, N, K);
}

int mxfp4_linear_act(const void* x, int64_t ldx, const void* w_pre, const void* ws_pre, const void* bias,
                     int activation, int gated, const void* residual, int64_t ldr, void* out, int64_t ldo,
                     int out_dtype, int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                     void* stream) {
  if (activation < MXFP4_ACT_NONE || activation > MXFP4_ACT_RELU) return MXFP4_ERR_ARG;
  if (gated && N % 32) return MXFP4_ERR_SHAPE;
  const int64_t cols = gated ? N / 2 : N;
  if (!row_ok(ldo, cols, M) || (residual && !row_ok(ldr, cols, M))) return MXFP4_ERR_SHAPE;
  // 256 rows (one tile of the large-M kernel) stay addressable by 32-bit offsets
  if (M > 1 && (ldo > kMaxInt / 256 / (out_dtype == MXFP4_OUT_F32 ? 4 : 2) || (residual && ldr > kMaxInt / 256 / 2)))
    return MXFP4_ERR_SHAPE;
  int st = linear_check(x, M > 1 ? ldx : K, w_pre, ws_pre, bias, out, N, out_dtype, M, N, K);
  if (st) return st;
  if (workspace_bytes < mxfp4_linear_act_workspace_bytes(M, N, K)) return MXFP4_ERR_WORKSPACE;
  if (M == 0) return MXFP4_OK;
  const size_t need = mxfp4_linear_act_workspace_bytes(M, N, K);
  if (need && !workspace) return MXFP4_ERR_NULL;
  if ((need && !aligned(workspace, 256)) || !aligned(residual, 2)) return MXFP4_ERR_ALIGN;
  int cus = 0;
  st = device_cus(&cus);
  if (st) return st;
  GemmArgs e{};
  // (a call without anything to add is mxfp4_linear's)
  e.epilogue = activation != MXFP4_ACT_NONE || gated || residual;
  e.act = activation;
  e.gated = gated != 0;
  e.res = (const uint16_t*)residual;
  e.ldr = used(ldr, M);
  e.res_vec = aligned(residual, 8) && e.ldr % 4 == 0 && cols % 4 == 0;
  return linear_run_act(e, x, M > 1 ? ldx : K, w_pre, ws_pre, bias, out, M > 1 ? ldo : cols, out_dtype, M, N, K,
                        workspace, workspace_bytes, cus, (hipStream_t)stream);
}

}  // extern "C"
