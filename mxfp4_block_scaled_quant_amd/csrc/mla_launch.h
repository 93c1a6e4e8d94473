// Internal launchers of the latent-attention operators (csrc/mla_*.hip).
// Arguments are already validated by the caller (csrc/mla_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mxfp4 {

constexpr int kLatent = 512, kRope = 64, kRowDim = kLatent + kRope;
constexpr int kMlaMaxCus = 256;   // workgroups of an attention launch at most

// Paged rows: page p's row i at base + p * page_bytes + i * row_bytes.
struct PagedRows {
  const char* base;
  int64_t page_bytes, row_bytes;
  int pages, page_size;
  // t / page_size for t < 2^30 as (mulhi(t, magic) >> shift) + (t & whole)
  // (magic 0 and whole ~0 for pages of one row).
  uint32_t magic, shift, whole;
};

struct AppendArgs {
  const uint16_t* kv;             // [T, 576]
  int64_t ldkv;
  const uint16_t* weight;         // [512]
  float eps;
  const float* cos_sin;           // [positions_max, 64]: cos of 32 angles, sin of 32 angles
  int64_t positions_max;
  const int64_t* positions;
  const int64_t* slots;
  const uint16_t* q;              // [T, H, 64] or nullptr
  int64_t sqt, sqh;
  uint16_t* q_out;
  int64_t sot, soh;
  int H;
  PagedRows cache;
  int64_t T;
  int interleaved;
};
hipError_t launch_mla_append(const AppendArgs& p, hipStream_t stream);

// One absorbed attention call: B requests of S tokens, H heads.
struct DecodeArgs {
  const uint16_t* q;              // [B, S, H, 576]
  int64_t sqb, sqs, sqh;
  PagedRows cache;
  const int32_t* table;           // [B, max_pages]
  int64_t ldt;
  int max_pages;
  const int32_t* lens;            // [B]
  const int32_t* prefix_table;    // nullptr: no shared prefix
  int prefix_len;
  int B, S, H;
  float c;                        // scale * log2(e)
  uint16_t* out;                  // [B, S, H, 512]
  int64_t sob, sos, soh;
  float* lse;                     // [B, S, H] or nullptr
  float* work;
};
// The split of a call: query rows per workgroup of its requests and of its
// prefix, workgroups, and where the parts lie in the workspace (float offsets).
struct DecodePlan {
  int rows, prows;                // 16, 32 (four waves share the keys), 128 (four waves share the rows)
  int grid, pgrid, cus;
  size_t part, pml, ppart, ppml, ipart, ipml, floats;
};
int get_mla_rows_override();  // 0: none (set by the test hook)
DecodePlan decode_plan(int64_t B, int64_t S, int64_t H, int64_t max_tokens, int64_t prefix_len, int cus);
hipError_t launch_mla_decode(const DecodeArgs& p, const DecodePlan& plan, hipStream_t stream);

struct MlaPrefillArgs {
  const uint16_t* q;              // [Tq, H, dn + 64]
  int64_t sqt, sqh;
  const uint16_t* k;              // [Tk, H, dn]
  int64_t skt, skh;
  const uint16_t* k_pe;           // [Tk, 64]
  int64_t spt;
  const uint16_t* v;              // [Tk, H, dv]
  int64_t svt, svh;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int B, H;
  int64_t Tq, Tk;
  int causal;
  float c;
  uint16_t* out;                  // [Tq, H, dv]
  int64_t sot, soh;
  float* lse;                     // [Tq, H] or nullptr
};
// rows: per workgroup, 32 or 128; 0 = by the rows.
hipError_t launch_mla_prefill(const MlaPrefillArgs& p, int dn, int dv, int rows, int cus, hipStream_t stream);

}  // namespace mxfp4
