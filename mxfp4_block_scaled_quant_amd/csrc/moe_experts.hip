// The chosen experts' MXFP4 products and their weighted sum (gfx950).
//
// For every pair (token t, choice j) with e = ids[t, j] in [0, E):
//   h = bf16(act(gate) * up),  (gate, up) = dq(Q(x_t)) dq(U_e)^T + bias
//   y = dq(Q(h)) dq(D_e)^T + bias
//   out_t = residual_t + sum_j weights[t, j] y   (fp32, in the order of j)
//
// Five launches:
//  * plan: counts the pairs of each expert and gives every pair a row; an
//    expert's rows are consecutive and begin with a 16-row strip, so that
//    the products find them as whole operands of the matrix instruction;
//  * gather: the rows of x quantised per 1x32 into the GEMM layout there;
//  * up: the product, the activation and the quantisation of its rows, which
//    stay in the same order;
//  * down: the product, one fp32 row a pair;
//  * combine: a token's rows, weighted and added.
#include "moe_launch.h"
#include "mxfp4_device.h"
#include "mxfp4_launch.h"

namespace mxfp4 {

namespace {

constexpr int kAuxNT = 2;  // cache policy bits of a buffer load: non-temporal

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ------------------------------------------------------------ the workspace

// Where things are in the workspace (byte offsets).  rows: 16 per strip, at
// most as many strips as pairs, and 15 rows of padding per expert met.
struct MoeLayout {
  int64_t strips, max_blocks;
  size_t head, blocks, pos, src, a, as, h, hs, part, total;
};

MoeLayout moe_layout(int64_t tokens, int64_t top_k, int64_t experts, int64_t hidden, int64_t inner) {
  MoeLayout l{};
  const int64_t pairs = tokens * top_k;
  const int64_t met = pairs < experts ? pairs : experts;
  l.strips = (pairs + 15 * met) / 16;
  l.max_blocks = l.strips;
  const int64_t kt1 = cdiv(hidden, 128), kt2 = cdiv(inner, 128);
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t o = at;
    at += (size_t)cdiv(bytes, 256) * 256;
    return o;
  };
  l.head = take(sizeof(MoeHead));
  l.blocks = take(l.max_blocks * (int64_t)sizeof(MoeBlock));
  l.pos = take(pairs * 4);
  l.src = take(l.strips * 16 * 4);
  l.a = take(l.strips * kt1 * 1024);
  l.as = take(l.strips * cdiv(kt1, 4) * 256);
  l.h = take(l.strips * kt2 * 1024);
  l.hs = take(l.strips * cdiv(kt2, 4) * 256);
  l.part = take(l.strips * 16 * hidden * 4);
  l.total = at;
  return l;
}

// ------------------------------------------------------------------ the plan

// Inclusive scan over the workgroup's 1024 threads (16 waves).
__device__ __forceinline__ int scan1024(int v, int* tmp) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();
  if (lane == 63) tmp[wv] = v;
  __syncthreads();
  int add = 0;
  for (int w = 0; w < wv; ++w) add += tmp[w];
  return v + add;
}

// One workgroup: an expert's pairs are counted and ranked by atomics in LDS.
// Their order gives a pair its row among its expert's, and no row's result
// depends on which row it is, so the outputs do not depend on that order.
__global__ __launch_bounds__(1024) void moe_plan_kernel(const int32_t* ids, int64_t ldi, int pairs, int top_k,
                                                        int experts, int block_strips, MoeHead* head,
                                                        MoeBlock* blocks, int32_t* pos, int32_t* src) {
  __shared__ int count[kMaxExperts], first[kMaxExperts], tmp[16];
  const int tid = threadIdx.x;
  count[tid] = 0;
  __syncthreads();
  for (int i = tid; i < pairs; i += 1024) {
    const int e = ids[(int64_t)(i / top_k) * ldi + i % top_k];
    pos[i] = (uint32_t)e < (uint32_t)experts ? atomicAdd(&count[e], 1) : -1;
  }
  __syncthreads();
  const int rows = tid < experts ? count[tid] : 0;
  const int strips = (rows + 15) / 16;
  const int nb = (strips + block_strips - 1) / block_strips;
  const int end = scan1024(strips, tmp);
  const int bend = scan1024(nb, tmp);
  first[tid] = (end - strips) * 16;
  for (int b = 0; b < nb; ++b) {
    const int left = rows - b * block_strips * 16;
    blocks[bend - nb + b] = {tid, end - strips + b * block_strips, left < block_strips * 16 ? left : block_strips * 16, 0};
  }
  for (int r = rows; r < strips * 16; ++r) src[(end - strips) * 16 + r] = -1;
  if (tid == 1023) *head = {bend, end};
  __syncthreads();
  for (int i = tid; i < pairs; i += 1024) {
    const int rank = pos[i];
    if (rank < 0) continue;
    const int row = first[ids[(int64_t)(i / top_k) * ldi + i % top_k]] + rank;
    pos[i] = row;
    src[row] = i;
  }
}

// ---------------------------------------------------------------- the gather

// Rows of x quantised into the GEMM layout at their places: as
// quant_1x32_gemm_kernel, a 256-thread workgroup per 1 KiB unit (16 rows x
// one K-step), whose rows come from the pairs' tokens.  A strip's padding
// rows become zeros with scale 1.
// The first workgroup of a strip also writes the padding of its rows in
// the second product's input (K2 values in Kt2 K-steps): zeros with scale 1
// past K2.
__global__ __launch_bounds__(256) void moe_gather_kernel(const uint16_t* x, int64_t ldx, const MoeHead* head,
                                                         const int32_t* src, int top_k, int K, int Kt, int G,
                                                         uint8_t* q, uint8_t* scales, int K2, int Kt2, int G2,
                                                         uint8_t* h, uint8_t* hs) {
  const int L = threadIdx.x;
  const int r = L >> 4, kb = (L >> 2) & 3, sub = L & 3;
  const int s = (int)(blockIdx.x / (unsigned)(4 * G)), tq = (int)(blockIdx.x % (unsigned)(4 * G));
  if (s >= head->strips) return;
  const int pair = src[s * 16 + r];
  const int c = tq * 4 + kb;
  const bool valid = pair >= 0 && c < (K >> 5);
  uint32_t w0 = 0, w1 = 0, w2 = 0, w3 = 0;
  if (valid) {
    const int4 v = *reinterpret_cast<const int4*>(x + (int64_t)(pair / top_k) * ldx + (int64_t)c * 32 + sub * 8);
    w0 = (uint32_t)v.x, w1 = (uint32_t)v.y, w2 = (uint32_t)v.z, w3 = (uint32_t)v.w;
  }
  const uint32_t amax = quad_amax_bits(w0, w1, w2, w3);
  const uint32_t b = valid ? e8m0_of_amax_bits(amax) : kE8M0One;
  if (tq < Kt) {
    const uint32_t packed = valid ? e2m1_pack8(w0, w1, w2, w3, e8m0_value(b)) : 0u;
    *reinterpret_cast<uint32_t*>(q + ((int64_t)s * Kt + tq) * 1024 + (kb * 16 + r) * 16 + sub * 4) = packed;
  }
  if (sub == 0) scales[((int64_t)s * G + (tq >> 2)) * 256 + (kb * 16 + r) * 4 + (tq & 3)] = (uint8_t)b;
  if (tq == 0)
    for (int c2 = (K2 >> 5) + (L & 15); c2 < G2 * 16; c2 += 16) {
      const int t2 = c2 >> 2, k2 = c2 & 3;
      if (t2 < Kt2) *reinterpret_cast<int4*>(h + ((int64_t)s * Kt2 + t2) * 1024 + (k2 * 16 + r) * 16) = (int4){0, 0, 0, 0};
      hs[((int64_t)s * G2 + (t2 >> 2)) * 256 + (k2 * 16 + r) * 4 + (t2 & 3)] = (uint8_t)kE8M0One;
    }
}

// -------------------------------------------------------------- the products

// One side's operands: quantised rows (GEMM layouts) and the experts'
// weights.
struct ProductArgs {
  const MoeHead* head;
  const MoeBlock* blocks;
  const uint8_t *a, *as, *w, *ws;
  const uint16_t* bias;  // [experts, Ns * 16] or nullptr
  int Kt, G, Ns;         // of the weights
  int cols;              // workgroups of 32 output columns
  int act;
  int inner;             // up: columns of h
  uint8_t *h, *hs;       // up: h in the GEMM layouts (Kt2, G2 of its own)
  float* part;           // down: [rows, hidden]
  int hidden;
};

// A workgroup takes 32 output columns of one block of MT row tiles: NS weight
// strips (up, gated: two of the gate and the two beside them of the other
// half; else two), its KW waves the groups of 4 K-steps in turn.  All of a
// group's loads go out before its first product.  The waves' partial sums
// meet in LDS and are added in wave order.
constexpr int stream_waves(int mt) { return mt == 1 ? 12 : mt == 2 ? 8 : 4; }

template <int MT, int NS, bool UP>
__global__ __launch_bounds__(64 * stream_waves(MT)) void moe_stream_kernel(ProductArgs p) {
  extern __shared__ float red[];
  const int bi = (int)(blockIdx.x / (unsigned)p.cols), c = (int)(blockIdx.x % (unsigned)p.cols);
  if (bi >= p.head->blocks) return;
  const MoeBlock blk = p.blocks[bi];
  const int expert = __builtin_amdgcn_readfirstlane(blk.expert);
  const int strip = __builtin_amdgcn_readfirstlane(blk.strip);
  const int rows = __builtin_amdgcn_readfirstlane(blk.rows);
  const int lane = threadIdx.x & 63;
  const int wv = threadIdx.x >> 6;
  const int KW = blockDim.x >> 6;

  const int nst = (rows + 15) >> 4;
  const auto ra = make_rsrc(p.a + (int64_t)strip * p.Kt * 1024, (uint32_t)(nst * p.Kt) * 1024u);
  const auto ras = make_rsrc(p.as + (int64_t)strip * p.G * 256, (uint32_t)(nst * p.G) * 256u);
  const auto rw = make_rsrc(p.w + (int64_t)expert * p.Ns * p.Kt * 1024, (uint32_t)p.Ns * p.Kt * 1024u);
  const auto rws = make_rsrc(p.ws + (int64_t)expert * p.Ns * p.G * 256, (uint32_t)p.Ns * p.G * 256u);

  v4f acc[MT][NS];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NS; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};

  for (int g = wv; g < p.G; g += KW) {
    int4 bf[4][NS], af[4][MT];
    uint32_t sa[MT], sb[NS];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = g * 4 + u;
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const int s = (NS == 4 && j >= 2 ? p.Ns / 2 : 0) + 2 * c + (j & 1);
        bf[u][j] = __builtin_bit_cast(
            int4, __builtin_amdgcn_raw_buffer_load_b128(
                      rw, t < p.Kt ? (uint32_t)((s * p.Kt + t) * 1024 + lane * 16) : kOOB, 0, kAuxNT));
      }
    }
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const int s = (NS == 4 && j >= 2 ? p.Ns / 2 : 0) + 2 * c + (j & 1);
      sb[j] = buf_load4(rws, (uint32_t)((s * p.G + g) * 256 + lane * 4));
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) sa[i] = buf_load4(ras, (uint32_t)((i * p.G + g) * 256 + lane * 4));
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = g * 4 + u;
#pragma unroll
      for (int i = 0; i < MT; ++i)
        af[u][i] = buf_load16(ra, (t < p.Kt && i * 16 + (lane & 15) < rows)
                                      ? (uint32_t)((i * p.Kt + t) * 1024 + lane * 16) : kOOB);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          switch (u) {
            case 0: acc[i][j] = mfma_fp4<0, 0>(af[u][i], bf[u][j], sa[i], sb[j], acc[i][j]); break;
            case 1: acc[i][j] = mfma_fp4<1, 1>(af[u][i], bf[u][j], sa[i], sb[j], acc[i][j]); break;
            case 2: acc[i][j] = mfma_fp4<2, 2>(af[u][i], bf[u][j], sa[i], sb[j], acc[i][j]); break;
            default: acc[i][j] = mfma_fp4<3, 3>(af[u][i], bf[u][j], sa[i], sb[j], acc[i][j]); break;
          }
        }
  }

#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) red[(((i * NS + j) * 4 + r) * KW + wv) * 64 + lane] = acc[i][j][r];
  __syncthreads();
  auto sum = [&](int tile, int reg, int l) {
    const float* s = red + (tile * 4 + reg) * KW * 64 + l;
    float v = s[0];
    for (int w = 1; w < KW; ++w) v += s[w * 64];
    return v;
  };
  const uint16_t* bias = p.bias ? p.bias + (int64_t)expert * p.Ns * 16 : nullptr;
  if constexpr (UP) {
    uint16_t* stg = reinterpret_cast<uint16_t*>(red + MT * NS * 4 * KW * 64);  // [MT * 16][32] bf16
    for (int idx = threadIdx.x; idx < MT * 512; idx += blockDim.x) {
      const int l = idx & 63, reg = (idx >> 6) & 3, jj = (idx >> 8) & 1, i = idx >> 9;
      const int m = i * 16 + 4 * (l >> 4) + reg, n = jj * 16 + (l & 15);
      float g = sum(i * NS + jj, reg, l);
      if (bias) g += bf16_to_f32(bias[c * 32 + n]);
      float v = activate(g, p.act);
      if constexpr (NS == 4) {
        float up = sum(i * NS + 2 + jj, reg, l);
        if (bias) up += bf16_to_f32(bias[p.inner + c * 32 + n]);
        v *= up;
      }
      stg[m * 32 + n] = f32_to_bf16_rne(v);
    }
    __syncthreads();
    const int Kt2 = (p.inner + 127) >> 7, G2 = (Kt2 + 3) >> 2;
    for (int idx = threadIdx.x; idx < MT * 64; idx += blockDim.x) {
      const int m = idx >> 2, piece = idx & 3;
      const int4 v = *reinterpret_cast<const int4*>(stg + m * 32 + piece * 8);
      const uint32_t b =
          e8m0_of_amax_bits(quad_amax_bits((uint32_t)v.x, (uint32_t)v.y, (uint32_t)v.z, (uint32_t)v.w));
      const uint32_t code = e2m1_pack8((uint32_t)v.x, (uint32_t)v.y, (uint32_t)v.z, (uint32_t)v.w, e8m0_value(b));
      if (m < rows) {
        const int64_t s = strip + (m >> 4);
        const int r = m & 15, t = c >> 2, kb = c & 3;
        *reinterpret_cast<uint32_t*>(p.h + (s * Kt2 + t) * 1024 + (kb * 16 + r) * 16 + piece * 4) = code;
        if (piece == 0) p.hs[(s * G2 + (t >> 2)) * 256 + (kb * 16 + r) * 4 + (t & 3)] = (uint8_t)b;
      }
    }
  } else {
    for (int idx = threadIdx.x; idx < MT * 512; idx += blockDim.x) {
      const int l = idx & 63, reg = (idx >> 6) & 3, jj = (idx >> 8) & 1, i = idx >> 9;
      const int m = i * 16 + 4 * (l >> 4) + reg, n = c * 32 + jj * 16 + (l & 15);
      if (m >= rows) continue;
      float v = sum(i * NS + jj, reg, l);
      if (bias) v += bf16_to_f32(bias[n]);
      p.part[((int64_t)strip * 16 + m) * p.hidden + n] = v;
    }
  }
}

template <int MT, int NS, bool UP>
hipError_t launch_stream(const ProductArgs& p, int64_t max_blocks, hipStream_t stream) {
  const int kw = p.G < stream_waves(MT) ? p.G : stream_waves(MT);
  const size_t lds = (size_t)MT * NS * 4 * kw * 64 * 4 + (UP ? MT * 16 * 32 * 2 : 0);
  moe_stream_kernel<MT, NS, UP><<<dim3((unsigned)(max_blocks * p.cols)), 64 * kw, lds, stream>>>(p);
  return hipGetLastError();
}

template <int MT>
hipError_t launch_up(const ProductArgs& p, bool gated, int64_t max_blocks, hipStream_t stream) {
  return gated ? launch_stream<MT, 4, true>(p, max_blocks, stream) : launch_stream<MT, 2, true>(p, max_blocks, stream);
}

// Mean rows of an expert up to which its weights are streamed once per block
// of up to 64 rows; with more the products run on tiles of 256 rows.
constexpr int64_t kStreamRows = 48;

// The large-M kernel over the plan's row tiles.
hipError_t launch_tiles(const GemmArgs& p, int64_t max_blocks, hipStream_t stream) {
  const int out_strips = p.gated ? p.Ns / 2 : p.Ns;
  const int wide = p.gated ? 8 : 16;
  const int64_t tiles = max_blocks * cdiv(out_strips, wide);
  return launch_prefill_experts_256(p, (int)(tiles < p.cus ? tiles : p.cus), stream);
}

// --------------------------------------------------------------- the combine

// A token's rows, weighted and added in the order of its choices: four
// columns a thread.
__global__ __launch_bounds__(256) void moe_combine_kernel(MoeArgs p, const int32_t* pos, const float* part) {
  const int64_t quads = p.hidden / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.tokens * quads) return;
  const int64_t t = i / quads;
  const int n = (int)(i % quads) * 4;
  v4f v = {0.f, 0.f, 0.f, 0.f};
  if (p.residual) {
    const uint2 r = *reinterpret_cast<const uint2*>(p.residual + t * p.ldr + n);
    v = (v4f){__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
              __uint_as_float(r.y & 0xFFFF0000u)};
  }
  for (int j = 0; j < p.top_k; ++j) {
    const int row = pos[t * p.top_k + j];
    if (row < 0) continue;
    const float w = p.weights[t * p.ldw + j];
    const v4f y = *reinterpret_cast<const v4f*>(part + (int64_t)row * p.hidden + n);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] += w * y[q];
  }
  uint2 o;
  o.x = pack_bf16x2(v[0], v[1]);
  o.y = pack_bf16x2(v[2], v[3]);
  *reinterpret_cast<uint2*>(p.out + t * p.ldo + n) = o;
}

}  // namespace

size_t moe_workspace_bytes(int64_t tokens, int64_t top_k, int64_t experts, int64_t hidden, int64_t inner) {
  return moe_layout(tokens, top_k, experts, hidden, inner).total;
}

hipError_t launch_moe(const MoeArgs& p, hipStream_t stream) {
  const MoeLayout l = moe_layout(p.tokens, p.top_k, p.experts, p.hidden, p.inner);
  const int pairs = (int)(p.tokens * p.top_k);
  MoeHead* head = reinterpret_cast<MoeHead*>(p.work + l.head);
  MoeBlock* blocks = reinterpret_cast<MoeBlock*>(p.work + l.blocks);
  int32_t* pos = reinterpret_cast<int32_t*>(p.work + l.pos);
  int32_t* src = reinterpret_cast<int32_t*>(p.work + l.src);
  const int64_t mean = pairs / p.experts;
  const bool tiles = mean > kStreamRows;
  const int mt = mean <= 10 ? 1 : mean <= 24 ? 2 : 4;
  const int block_strips = tiles ? 16 : mt;
  moe_plan_kernel<<<1, 1024, 0, stream>>>(p.ids, p.ldi, pairs, p.top_k, p.experts, block_strips, head, blocks, pos, src);
  const int kt1 = (int)cdiv(p.hidden, 128), g1 = (int)cdiv(kt1, 4);
  const int kt2 = (int)cdiv(p.inner, 128), g2 = (int)cdiv(kt2, 4);
  moe_gather_kernel<<<dim3((unsigned)(l.strips * 4 * g1)), 256, 0, stream>>>(
      p.x, p.ldx, head, src, p.top_k, p.hidden, kt1, g1, p.work + l.a, p.work + l.as, p.inner, kt2, g2, p.work + l.h,
      p.work + l.hs);
  // at most one block per strip, one part block per expert met
  const int64_t met = pairs < p.experts ? pairs : p.experts;
  int64_t max_blocks = l.strips / block_strips + met;
  if (max_blocks > l.strips) max_blocks = l.strips;
  float* part = reinterpret_cast<float*>(p.work + l.part);
  hipError_t e;
  if (tiles) {
    GemmArgs u{};
    u.cus = p.cus, u.head = head, u.blocks = blocks;
    u.a = p.work + l.a, u.as = p.work + l.as, u.w = p.up, u.ws = p.up_scales, u.bias = p.up_bias;
    u.N = p.inner * (p.gated ? 2 : 1), u.K = p.hidden, u.Kt = kt1, u.G = g1, u.Ns = u.N / 16;
    u.w_expert = (int64_t)u.Ns * kt1 * 1024, u.ws_expert = (int64_t)u.Ns * g1 * 256;
    u.epilogue = 1, u.act = p.act, u.gated = p.gated;
    u.rows_out = p.work + l.h, u.rows_scales = p.work + l.hs, u.rows_kt = kt2, u.rows_g = g2;
    e = launch_tiles(u, max_blocks, stream);
    if (e != hipSuccess) return e;
    GemmArgs d{};
    d.cus = p.cus, d.head = head, d.blocks = blocks;
    d.a = p.work + l.h, d.as = p.work + l.hs, d.w = p.down, d.ws = p.down_scales, d.bias = p.down_bias;
    d.N = p.hidden, d.K = p.inner, d.Kt = kt2, d.G = g2, d.Ns = p.hidden / 16;
    d.w_expert = (int64_t)d.Ns * kt2 * 1024, d.ws_expert = (int64_t)d.Ns * g2 * 256;
    d.out = part, d.ldo = p.hidden, d.out_f32 = 1;
    e = launch_tiles(d, max_blocks, stream);
    if (e != hipSuccess) return e;
  } else {
    ProductArgs u{};
    u.head = head, u.blocks = blocks;
    u.a = p.work + l.a, u.as = p.work + l.as, u.w = p.up, u.ws = p.up_scales, u.bias = p.up_bias;
    u.Kt = kt1, u.G = g1, u.Ns = p.inner * (p.gated ? 2 : 1) / 16, u.cols = p.inner / 32;
    u.act = p.act, u.inner = p.inner, u.h = p.work + l.h, u.hs = p.work + l.hs;
    e = mt == 1 ? launch_up<1>(u, p.gated, max_blocks, stream)
        : mt == 2 ? launch_up<2>(u, p.gated, max_blocks, stream)
                  : launch_up<4>(u, p.gated, max_blocks, stream);
    if (e != hipSuccess) return e;
    ProductArgs d{};
    d.head = head, d.blocks = blocks;
    d.a = p.work + l.h, d.as = p.work + l.hs, d.w = p.down, d.ws = p.down_scales, d.bias = p.down_bias;
    d.Kt = kt2, d.G = g2, d.Ns = p.hidden / 16, d.cols = p.hidden / 32;
    d.part = part, d.hidden = p.hidden;
    e = mt == 1 ? launch_stream<1, 2, false>(d, max_blocks, stream)
        : mt == 2 ? launch_stream<2, 2, false>(d, max_blocks, stream)
                  : launch_stream<4, 2, false>(d, max_blocks, stream);
    if (e != hipSuccess) return e;
  }
  const int64_t n = p.tokens * (p.hidden / 4);
  moe_combine_kernel<<<dim3((unsigned)cdiv(n, 256)), 256, 0, stream>>>(p, pos, part);
  return hipGetLastError();
}

}  // namespace mxfp4
