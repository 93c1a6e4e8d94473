// C ABI of the latent-attention operators (declared in include/mxfp4.h):
// argument validation on the host, before any HIP call, and dispatch.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/mxfp4.h"
#include "../../include/mxfp4_testing.h"
#include "mla_launch.h"
#include "mxfp4_launch.h"

namespace mxfp4 {

// The test hook's forced row block: per thread, like the GEMM path's.
static thread_local int t_rows = 0;
static thread_local int t_prefill_rows = 0;
int get_mla_rows_override() { return t_rows; }

namespace {

constexpr int64_t kMaxRows = 1 << 22;      // query rows of a decode call
constexpr int64_t kMaxTokens = 1 << 30;    // rows of a page table: 32-bit key numbers
constexpr int64_t kMaxInt = 0x7FFFFFFF;
constexpr int64_t kMaxStride = 1ll << 40;  // elements: products with sizes stay in 64 bits

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }
// The stride of a dimension of n elements: one element's is never used, and a
// view may have any number there.
inline int64_t used(int64_t stride, int64_t n) { return n > 1 ? stride : 0; }
inline int launched(hipError_t e) { return e == hipSuccess ? MXFP4_OK : MXFP4_ERR_LAUNCH; }

// Whether rows of `width` elements at the given strides keep apart: walking
// the dimensions from the smallest stride, each steps over all before it.
bool rows_apart(int64_t width, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2) {
  int64_t n[3] = {n0, n1, n2}, s[3] = {s0, s1, s2};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (s[j] < s[i]) {
        const int64_t a = s[i], b = n[i];
        s[i] = s[j], n[i] = n[j], s[j] = a, n[j] = b;
      }
  int64_t extent = width;
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (s[i] < extent) return false;
    extent += (n[i] - 1) * s[i];
  }
  return true;
}

int cache_check(const void* cache, int64_t pages, int64_t page_size, int64_t cache_page, int64_t cache_row) {
  if (pages < 0 || pages > kMaxInt || page_size < 1 || page_size > kMaxTokens) return MXFP4_ERR_SHAPE;
  if (!stride_ok(cache_page) || !stride_ok(cache_row)) return MXFP4_ERR_SHAPE;
  if ((page_size > 1 && cache_row < kRowDim) ||
      (pages > 1 && cache_page < (page_size - 1) * cache_row + kRowDim))
    return MXFP4_ERR_SHAPE;
  if (pages > 0 && !cache) return MXFP4_ERR_NULL;
  if (!aligned(cache, 16) || cache_page % 8 || cache_row % 8) return MXFP4_ERR_ALIGN;
  return MXFP4_OK;
}

PagedRows paged(const void* cache, int64_t pages, int64_t page_size, int64_t cache_page, int64_t cache_row) {
  PagedRows r{};
  r.base = (const char*)cache;
  r.page_bytes = cache_page * 2;
  r.row_bytes = cache_row * 2;
  r.pages = (int)pages;
  r.page_size = (int)page_size;
  // magic = floor(2^(32 + shift) / d) + 1 exceeds 2^(32 + shift) / d by at
  // most 1, so the quotient is exact while t * d <= 2^(32 + shift): with
  // 2^(shift + 2) > d that holds for every t < 2^30.
  if (page_size == 1) {
    r.whole = ~0u;
  } else {
    while ((2ll << (r.shift + 1)) <= page_size) ++r.shift;
    r.magic = (uint32_t)((1ull << (32 + r.shift)) / (uint64_t)page_size + 1);
  }
  return r;
}

bool decode_shape(int64_t B, int64_t S, int64_t H, int64_t max_tokens, int64_t prefix_len) {
  if (B < 0 || S < 1 || H < 1 || max_tokens < 0 || prefix_len < 0) return false;
  if (B > kMaxRows || S > kMaxRows || H > kMaxRows || S * H > kMaxRows || B * S * H > kMaxRows) return false;
  if (max_tokens > kMaxTokens || prefix_len > kMaxTokens) return false;
  // work units are counted in 32 bits (at most one per 64 keys and 16 rows)
  return B * cdiv(S * H, 16) * cdiv(max_tokens, 64) <= kMaxInt &&
         cdiv(B * S * H, 16) * cdiv(prefix_len, 64) <= kMaxInt;
}

int decode_call(const void* q, int64_t q_batch, int64_t q_token, int64_t q_head, const void* cache, int64_t pages,
                int64_t page_size, int64_t cache_page, int64_t cache_row, const void* prefix_table,
                int64_t prefix_pages, int64_t prefix_len, const void* block_table, int64_t ldt, int64_t max_pages,
                const void* lengths, int64_t B, int64_t S, int64_t H, float scale, void* out, int64_t out_batch,
                int64_t out_token, int64_t out_head, void* lse, void* workspace, size_t workspace_bytes,
                void* stream) {
  if (!(scale > 0.0f) || isinf(scale)) return MXFP4_ERR_ARG;
  q_batch = used(q_batch, B), out_batch = used(out_batch, B), ldt = used(ldt, B);
  q_token = used(q_token, S), out_token = used(out_token, S);
  q_head = used(q_head, H), out_head = used(out_head, H);
  cache_page = used(cache_page, pages), cache_row = used(cache_row, page_size);
  if (page_size < 1 || max_pages < 0 || max_pages > kMaxTokens || page_size > kMaxTokens) return MXFP4_ERR_SHAPE;
  if (max_pages * page_size > kMaxTokens || !decode_shape(B, S, H, max_pages * page_size, prefix_len))
    return MXFP4_ERR_SHAPE;
  if ((ldt < max_pages && ldt != 0) || ldt > kMaxStride) return MXFP4_ERR_SHAPE;
  if (prefix_pages < 0 || prefix_pages > kMaxTokens || prefix_pages * page_size < prefix_len) return MXFP4_ERR_SHAPE;
  if (!stride_ok(q_batch) || !stride_ok(q_token) || !stride_ok(q_head) || !stride_ok(out_batch) ||
      !stride_ok(out_token) || !stride_ok(out_head))
    return MXFP4_ERR_SHAPE;
  if (!rows_apart(kLatent, B, out_batch, S, out_token, H, out_head)) return MXFP4_ERR_SHAPE;
  int st = cache_check(cache, pages, page_size, cache_page, cache_row);
  if (st) return st;
  if (B == 0) return MXFP4_OK;
  if (!q || !out || !lengths || (max_pages > 0 && !block_table) || (prefix_len > 0 && !prefix_table))
    return MXFP4_ERR_NULL;
  if (!aligned(q, 16) || q_batch % 8 || q_token % 8 || q_head % 8 || !aligned(out, 16) || out_batch % 8 ||
      out_token % 8 || out_head % 8 || !aligned(block_table, 4) || !aligned(lengths, 4) ||
      !aligned(prefix_table, 4) || !aligned(lse, 4))
    return MXFP4_ERR_ALIGN;
  if (workspace_bytes < mla_decode_workspace_bytes(B, S, H, max_pages * page_size, prefix_len))
    return MXFP4_ERR_WORKSPACE;
  if (!workspace) return MXFP4_ERR_NULL;
  if (!aligned(workspace, 16)) return MXFP4_ERR_ALIGN;
  int cus = 0;
  st = device_cus(&cus);
  if (st) return st;
  DecodeArgs p{};
  p.q = (const uint16_t*)q;
  p.sqb = q_batch;
  p.sqs = q_token;
  p.sqh = q_head;
  p.cache = paged(cache, pages, page_size, cache_page, cache_row);
  p.table = (const int32_t*)block_table;
  p.ldt = ldt;
  p.max_pages = (int)max_pages;
  p.lens = (const int32_t*)lengths;
  p.prefix_table = (const int32_t*)prefix_table;
  p.prefix_len = (int)prefix_len;
  p.B = (int)B;
  p.S = (int)S;
  p.H = (int)H;
  p.c = scale * 1.4426950408889634f;
  p.out = (uint16_t*)out;
  p.sob = out_batch;
  p.sos = out_token;
  p.soh = out_head;
  p.lse = (float*)lse;
  p.work = (float*)workspace;
  return launched(launch_mla_decode(p, decode_plan(B, S, H, max_pages * page_size, prefix_len, cus),
                                    (hipStream_t)stream));
}

}  // namespace
}  // namespace mxfp4

using namespace mxfp4;

extern "C" {

int mla_cache_append(const void* kv, int64_t ldkv, const void* norm_weight, float eps, const void* cos_sin,
                     int64_t max_position, const void* positions, const void* slots, int interleaved,
                     const void* q_pe, int64_t q_token, int64_t q_head, void* q_out, int64_t qo_token,
                     int64_t qo_head, void* cache, int64_t pages, int64_t page_size, int64_t cache_page,
                     int64_t cache_row, int64_t T, int64_t H, void* stream) {
  if (interleaved != 0 && interleaved != 1) return MXFP4_ERR_ARG;
  if (!(eps >= 0.0f) || isinf(eps)) return MXFP4_ERR_ARG;
  ldkv = used(ldkv, T), q_token = used(q_token, T), qo_token = used(qo_token, T);
  q_head = used(q_head, H), qo_head = used(qo_head, H);
  cache_page = used(cache_page, pages), cache_row = used(cache_row, page_size);
  if (T < 0 || T > kMaxInt || H < 0 || H > (1 << 20) || max_position < 0 || max_position > kMaxStride)
    return MXFP4_ERR_SHAPE;
  if ((T > 1 && ldkv < kRowDim) || !stride_ok(ldkv)) return MXFP4_ERR_SHAPE;
  const bool with_q = q_pe && q_out && H > 0;
  if (!with_q && (q_pe || q_out) && H > 0) return MXFP4_ERR_NULL;
  if (with_q) {
    if (!stride_ok(q_token) || !stride_ok(q_head) || !stride_ok(qo_token) || !stride_ok(qo_head))
      return MXFP4_ERR_SHAPE;
    if (!rows_apart(kRope, T, qo_token, H, qo_head, 1, 0)) return MXFP4_ERR_SHAPE;
  }
  int st = cache_check(cache, pages, page_size, cache_page, cache_row);
  if (st) return st;
  if (T == 0) return MXFP4_OK;
  if (!kv || !norm_weight || !positions || !slots || (max_position > 0 && !cos_sin)) return MXFP4_ERR_NULL;
  if (!aligned(kv, 16) || ldkv % 8 || !aligned(norm_weight, 16) || !aligned(cos_sin, 16) || !aligned(positions, 8) ||
      !aligned(slots, 8))
    return MXFP4_ERR_ALIGN;
  if (with_q && (!aligned(q_pe, 16) || q_token % 8 || q_head % 8 || !aligned(q_out, 16) || qo_token % 8 ||
                 qo_head % 8))
    return MXFP4_ERR_ALIGN;
  if ((st = device_cus(nullptr))) return st;
  AppendArgs p{};
  p.kv = (const uint16_t*)kv;
  p.ldkv = ldkv;
  p.weight = (const uint16_t*)norm_weight;
  p.eps = eps;
  p.cos_sin = (const float*)cos_sin;
  p.positions_max = max_position;
  p.positions = (const int64_t*)positions;
  p.slots = (const int64_t*)slots;
  p.q = with_q ? (const uint16_t*)q_pe : nullptr;
  p.sqt = q_token;
  p.sqh = q_head;
  p.q_out = (uint16_t*)q_out;
  p.sot = qo_token;
  p.soh = qo_head;
  p.H = (int)H;
  p.cache = paged(cache, pages, page_size, cache_page, cache_row);
  p.T = T;
  p.interleaved = interleaved;
  return launched(launch_mla_append(p, (hipStream_t)stream));
}

size_t mla_decode_workspace_bytes(int64_t B, int64_t S, int64_t H, int64_t max_tokens, int64_t prefix_len) {
  if (!decode_shape(B, S, H, max_tokens, prefix_len) || B == 0) return 0;
  return decode_plan(B, S, H, max_tokens, prefix_len, kMlaMaxCus).floats * sizeof(float);
}

int mla_decode(const void* q, int64_t q_batch, int64_t q_token, int64_t q_head, const void* cache, int64_t pages,
               int64_t page_size, int64_t cache_page, int64_t cache_row, const void* block_table, int64_t ldt,
               int64_t max_pages, const void* lengths, int64_t B, int64_t S, int64_t H, float scale, void* out,
               int64_t out_batch, int64_t out_token, int64_t out_head, void* lse, void* workspace,
               size_t workspace_bytes, void* stream) {
  return decode_call(q, q_batch, q_token, q_head, cache, pages, page_size, cache_page, cache_row, nullptr, 0, 0,
                     block_table, ldt, max_pages, lengths, B, S, H, scale, out, out_batch, out_token, out_head, lse,
                     workspace, workspace_bytes, stream);
}

int mla_decode_shared_prefix(const void* q, int64_t q_batch, int64_t q_token, int64_t q_head, const void* cache,
                             int64_t pages, int64_t page_size, int64_t cache_page, int64_t cache_row,
                             const void* prefix_table, int64_t prefix_pages, int64_t prefix_len,
                             const void* block_table, int64_t ldt, int64_t max_pages, const void* lengths, int64_t B,
                             int64_t S, int64_t H, float scale, void* out, int64_t out_batch, int64_t out_token,
                             int64_t out_head, void* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return decode_call(q, q_batch, q_token, q_head, cache, pages, page_size, cache_page, cache_row, prefix_table,
                     prefix_pages, prefix_len, block_table, ldt, max_pages, lengths, B, S, H, scale, out, out_batch,
                     out_token, out_head, lse, workspace, workspace_bytes, stream);
}

int mla_prefill(const void* q, int64_t q_token, int64_t q_head, const void* k_nope, int64_t k_token, int64_t k_head,
                const void* k_pe, int64_t pe_token, const void* v, int64_t v_token, int64_t v_head, const void* cu_q,
                const void* cu_k, int64_t B, int64_t H, int64_t Tq, int64_t Tk, int64_t dn, int64_t dv, int causal,
                float scale, void* out, int64_t out_token, int64_t out_head, void* lse, void* stream) {
  if (!(scale > 0.0f) || isinf(scale) || (causal != 0 && causal != 1)) return MXFP4_ERR_ARG;
  if (!((dn == 128 && dv == 128) || (dn == 192 && dv == 256))) return MXFP4_ERR_SHAPE;
  if (B < 0 || B > (1 << 24) || H < 1 || H > (1 << 16) || Tq < 0 || Tk < 0 || Tq > kMaxTokens || Tk > kMaxTokens ||
      (Tq / 64 + (Tq < B ? Tq : B)) * H > kMaxInt)
    return MXFP4_ERR_SHAPE;
  // 256 threads a block of 128 query rows and head: a launch does no more than 2^32 work items
  if ((Tq / 128 + (Tq < B ? Tq : B)) * H >= (1 << 24)) return MXFP4_ERR_SHAPE;
  q_token = used(q_token, Tq), out_token = used(out_token, Tq);
  k_token = used(k_token, Tk), pe_token = used(pe_token, Tk), v_token = used(v_token, Tk);
  q_head = used(q_head, H), k_head = used(k_head, H), v_head = used(v_head, H), out_head = used(out_head, H);
  const int64_t in[] = {q_token, q_head, k_token, k_head, pe_token, v_token, v_head, out_token, out_head};
  for (int64_t s : in)
    if (!stride_ok(s)) return MXFP4_ERR_SHAPE;
  if (k_token >= (1 << 25) || pe_token >= (1 << 25) || v_token >= (1 << 25)) return MXFP4_ERR_SHAPE;
  if (!rows_apart(dv, Tq, out_token, H, out_head, 1, 0)) return MXFP4_ERR_SHAPE;
  if (Tq == 0 || B == 0) return MXFP4_OK;
  if (!q || !cu_q || !cu_k || !out || (Tk > 0 && (!k_nope || !k_pe || !v))) return MXFP4_ERR_NULL;
  for (int64_t s : in)
    if (s % 8) return MXFP4_ERR_ALIGN;
  if (!aligned(q, 16) || !aligned(k_nope, 16) || !aligned(k_pe, 16) || !aligned(v, 16) || !aligned(out, 16) ||
      !aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(lse, 4))
    return MXFP4_ERR_ALIGN;
  int cus = 0;
  const int st = device_cus(&cus);
  if (st) return st;
  MlaPrefillArgs p{};
  p.q = (const uint16_t*)q;
  p.sqt = q_token;
  p.sqh = q_head;
  p.k = (const uint16_t*)k_nope;
  p.skt = k_token;
  p.skh = k_head;
  p.k_pe = (const uint16_t*)k_pe;
  p.spt = pe_token;
  p.v = (const uint16_t*)v;
  p.svt = v_token;
  p.svh = v_head;
  p.cu_q = (const int32_t*)cu_q;
  p.cu_k = (const int32_t*)cu_k;
  p.B = (int)B;
  p.H = (int)H;
  p.Tq = Tq;
  p.Tk = Tk;
  p.causal = causal;
  p.c = scale * 1.4426950408889634f;
  p.out = (uint16_t*)out;
  p.sot = out_token;
  p.soh = out_head;
  p.lse = (float*)lse;
  return launched(launch_mla_prefill(p, (int)dn, (int)dv, t_prefill_rows, cus, (hipStream_t)stream));
}

// Test hooks (include/mxfp4_testing.h): force the forms on this thread.
int mla_testing_set_rows(int rows) {
  if (rows != 0 && rows != 16 && rows != 32 && rows != 128) return MXFP4_ERR_ARG;
  t_rows = rows;
  return MXFP4_OK;
}

int mla_testing_set_prefill_rows(int rows) {
  if (rows != 0 && rows != 32 && rows != 128) return MXFP4_ERR_ARG;
  t_prefill_rows = rows;
  return MXFP4_OK;
}

}  // extern "C"
