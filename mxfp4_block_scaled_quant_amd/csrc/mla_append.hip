// The cache write of latent attention on gfx950: one wave per token norms
// the latent (fp32 sum of squares over 512 values), rotates the key part and
// every head's query part by the token's position, and writes the row into
// its page slot.  One pass, each byte once; bound by HBM for many tokens and
// by one load's latency for few: 16001 tokens of 16 heads (107 MB) 24.6 us,
// 4.35 TB/s, where a 1 GiB copy reaches 5.2 and 107 MB is too few bytes for
// its start and end to vanish; non-temporal stores and loads of the next
// token ahead measured the same.  64 tokens: 4 us, and the call's host side
// takes longer.
//
// Lane l holds latent elements 8l..8l+7 (one 16-byte load: the row is 1 KiB
// a wave).  A 64-element rotated part is four units of two 16-byte pieces
// and 8 angles: unit u takes elements 16u..16u+15 (pairs 2i, 2i+1) or
// 8u..8u+7 and 32+8u..+7 (pairs i, 32+i), so 16 heads are one pass of a wave.
#include "mla_device.h"
#include "mla_launch.h"

namespace mxfp4 {
namespace {

constexpr int kWaves = 4;

__device__ __forceinline__ void unpack8(const int4& v, float (&x)[8]) {
  const uint32_t w[4] = {(uint32_t)v.x, (uint32_t)v.y, (uint32_t)v.z, (uint32_t)v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ int4 pack8(const float (&x)[8]) {
  return make_int4((int)pack_bf16x2(x[0], x[1]), (int)pack_bf16x2(x[2], x[3]), (int)pack_bf16x2(x[4], x[5]),
                   (int)pack_bf16x2(x[6], x[7]));
}

// Unit u of a 64-element part: a and b are its two pieces, cs its token's
// angles (cos of 32, sin of 32).
template <bool INTER>
__device__ __forceinline__ void rotate_unit(int4& a, int4& b, const float* cs, int u) {
  float x[8], y[8], c[8], s[8];
  unpack8(a, x);
  unpack8(b, y);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const v4f cc = *(const v4f*)(cs + 8 * u + 4 * i), ss = *(const v4f*)(cs + 32 + 8 * u + 4 * i);
#pragma unroll
    for (int j = 0; j < 4; ++j) c[4 * i + j] = cc[j], s[4 * i + j] = ss[j];
  }
  float p[8], r[8];
  if (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[2 * i] = x[2 * i] * c[i] - x[2 * i + 1] * s[i];
      p[2 * i + 1] = x[2 * i + 1] * c[i] + x[2 * i] * s[i];
      r[2 * i] = y[2 * i] * c[4 + i] - y[2 * i + 1] * s[4 + i];
      r[2 * i + 1] = y[2 * i + 1] * c[4 + i] + y[2 * i] * s[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = x[i] * c[i] - y[i] * s[i];
      r[i] = y[i] * c[i] + x[i] * s[i];
    }
  }
  a = pack8(p);
  b = pack8(r);
}

template <bool INTER>
__global__ __launch_bounds__(64 * kWaves) void mla_append_kernel(AppendArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= p.T) return;
  const int64_t pos = p.positions[t], slot = p.slots[t];
  // A position outside the table has no angles: nothing is written for it.
  if ((uint64_t)pos >= (uint64_t)p.positions_max) return;
  const float* cs = p.cos_sin + pos * kRope;
  const bool keep = slot >= 0 && slot / p.cache.page_size < p.cache.pages;  // padding, or past the cache: no row
  const uint16_t* src = p.kv + t * p.ldkv;
  char* row = const_cast<char*>(p.cache.base);
  if (keep) {
    const int64_t page = slot / p.cache.page_size;
    row += page * p.cache.page_bytes + (slot - page * p.cache.page_size) * p.cache.row_bytes;
    const int4 v = *(const int4*)(src + lane * 8), wv = *(const int4*)(p.weight + lane * 8);
    float x[8], w[8];
    unpack8(v, x);
    unpack8(wv, w);
    float ss = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
    const float r = rsqrtf(wave_sum(ss) * (1.0f / kLatent) + p.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
    *(int4*)(row + lane * 16) = pack8(x);
  }
  // Units of the key part (first) and of the heads' query parts.
  const int units = 4 * ((p.q ? p.H : 0) + 1);
  for (int i = lane; i < units; i += 64) {
    const int h = (i >> 2) - 1, u = i & 3;
    if (h < 0 && !keep) continue;
    const uint16_t* s = h < 0 ? src + kLatent : p.q + t * p.sqt + h * p.sqh;
    uint16_t* d = h < 0 ? (uint16_t*)row + kLatent : p.q_out + t * p.sot + h * p.soh;
    const int e0 = INTER ? 16 * u : 8 * u, e1 = INTER ? 16 * u + 8 : 32 + 8 * u;
    int4 a = *(const int4*)(s + e0), b = *(const int4*)(s + e1);
    rotate_unit<INTER>(a, b, cs, u);
    *(int4*)(d + e0) = a;
    *(int4*)(d + e1) = b;
  }
}

}  // namespace

hipError_t launch_mla_append(const AppendArgs& p, hipStream_t stream) {
  // (2^25 tokens a launch, a wave each: one does no more than 2^32 work items)
  constexpr int64_t kTokens = 1 << 25;
  for (int64_t t = 0; t < p.T; t += kTokens) {
    AppendArgs a = p;
    a.T = p.T - t < kTokens ? p.T - t : kTokens;
    a.kv += t * p.ldkv;
    a.positions += t;
    a.slots += t;
    if (p.q) a.q += t * p.sqt, a.q_out += t * p.sot;
    const dim3 grid((unsigned)((a.T + kWaves - 1) / kWaves));
    if (a.interleaved) mla_append_kernel<true><<<grid, 64 * kWaves, 0, stream>>>(a);
    else mla_append_kernel<false><<<grid, 64 * kWaves, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace mxfp4
