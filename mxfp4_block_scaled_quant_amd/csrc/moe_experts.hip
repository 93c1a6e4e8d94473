// The chosen experts' MXFP4 products and their weighted sum (gfx950).
//
// For every pair (token t, choice j) with e = ids[t, j] in [0, E):
//   h = bf16(act(gate) * up),  (gate, up) = dq(Q(x_t)) dq(U_e)^T + bias
//   y = dq(Q(h)) dq(D_e)^T + bias
//   out_t = residual_t + sum_j weights[t, j] y   (fp32, in the order of j)
//
// Launches:
//  * prepare: the plan (the pairs of each expert are counted and every pair
//    given a row; an expert's rows are consecutive and begin with a 16-row
//    strip) and the quantisation of x, side by side; over 1024 pairs a second
//    launch places the chunks that the first one counted;
//  * up: the product of the rows gathered by their tokens, the activation and
//    the quantisation of its rows, stored in the order of the plan;
//  * down: the product, one fp32 row a pair, and combine: a token's rows,
//    weighted and added; or, for up to 1024 pairs of short blocks, both in
//    one launch.
// Up to 64 pairs of 4 tokens take two launches: every wave makes the plan for
// itself and quantises the rows it multiplies.
#include "moe_launch.h"
#include "mxfp4_device.h"
#include "mxfp4_launch.h"

namespace mxfp4 {

namespace {

constexpr int kAuxNT = 2;  // cache policy bits of a buffer load: non-temporal

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kChunk = 1024;  // pairs that one workgroup counts

// ------------------------------------------------------------ the workspace

// Mean rows of an expert up to which its weights are streamed into registers,
// once per block of one or two 16-row tiles; with more the products run on
// tiles of 256 rows.  Measured (us, streamed / tiles; experts, choices, hidden,
// inner): 64, 8, 5120, 1024 with mean 12.5 124 / 140, 20 148 / 148, 25
// 158 / 150; 128, 8, 2048, 768 with mean 16 85 / 115, 24 96 / 118, 32
// 110 / 122; 32, 4, 5120, 1504 with mean 20 111 / 128, 25 119 / 129.  (The
// first, with the most weights, decides; the mean counts pairs whose expert is
// elsewhere too, since the host sees no ids.)
constexpr int64_t kStreamRows = 24;
inline bool moe_tiles(int64_t pairs, int64_t experts) { return pairs / experts > kStreamRows; }

// Where things are in the workspace (byte offsets).  rows: 16 per strip, at
// most as many strips as pairs, and 15 rows of padding per expert met.
struct MoeLayout {
  int64_t strips, max_blocks;
  size_t head, blocks, counts, pos, src, tok, a, as, h, hs, part, total;
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
  l.counts = take(cdiv(pairs, kChunk) * experts * 4);
  l.pos = take(pairs * 4);
  l.src = take(l.strips * 16 * 4);
  l.tok = take(l.strips * 16 * 4);
  l.a = take(tokens * kt1 * 64);
  l.as = take(tokens * cdiv(kt1, 4) * 16);
  l.h = take(l.strips * kt2 * 1024);
  l.hs = take(l.strips * cdiv(kt2, 4) * 256);
  l.part = take(l.strips * 16 * hidden * 4);
  l.total = at;
  return l;
}

// ------------------------------------------------------------------ the plan

// Where things of a plan are written.
struct PlanArgs {
  const int32_t* ids;
  int64_t ldi;
  int pairs, top_k, experts, block_strips, chunks;
  MoeHead* head;
  MoeBlock* blocks;
  int32_t* counts;  // [chunks][experts]
  int32_t* pos;     // a pair's row, -1 without one
  int32_t* src;     // a row's pair, -1 in a strip's padding
  int32_t* tok;     // a row's token, -1
};

// From the rows of four experts a thread (e0 = 4 threadIdx.x) the first row
// of each; `writes`: the list of blocks, the padding and the head too.
__device__ __forceinline__ void place_experts(const PlanArgs& p, const int (&rows)[4], int* first, int (*tmp)[4],
                                              bool writes) {
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, e0 = tid * 4;
  int strips = 0, nb = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int st = (rows[i] + 15) >> 4;
    strips += st;
    nb += (st + p.block_strips - 1) / p.block_strips;
  }
  int se = strips, be = nb;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int a = __shfl_up(se, d), b = __shfl_up(be, d);
    if (lane >= d) se += a, be += b;
  }
  if (lane == 63) tmp[0][wv] = se, tmp[1][wv] = be;
  __syncthreads();
  int all = 0, ball = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < wv) se += tmp[0][w], be += tmp[1][w];
    all += tmp[0][w], ball += tmp[1][w];
  }
  int s0 = se - strips, b0 = be - nb;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (e0 + i >= p.experts) break;
    first[e0 + i] = s0 * 16;
    const int st = (rows[i] + 15) >> 4;
    if (writes) {
      for (int b = 0; b < st; b += p.block_strips) {
        const int left = rows[i] - b * 16;
        p.blocks[b0++] = {e0 + i, s0 + b, left < p.block_strips * 16 ? left : p.block_strips * 16, 0};
      }
      for (int r = rows[i]; r < st * 16; ++r) p.src[s0 * 16 + r] = p.tok[s0 * 16 + r] = -1;
    }
    s0 += st;
  }
  if (writes && tid == 0) *p.head = {ball, all};
}

// Chunk w of the pairs: each ranked among its expert's of the chunk by an
// atomic in LDS.  (Their order gives a pair its row among its expert's, and
// no row's result depends on which row it is, so the outputs do not depend on
// it.)  With one chunk that is the whole plan; else the counts and ranks go to
// memory for moe_scatter_kernel.
__device__ void plan_chunk(const PlanArgs& p, int w) {
  __shared__ int count[kMaxExperts], first[kMaxExperts], tmp[2][4];
  const int tid = threadIdx.x;
#pragma unroll
  for (int i = 0; i < kMaxExperts; i += 256) count[i + tid] = 0;
  __syncthreads();
  int e[4], rank[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = w * kChunk + u * 256 + tid;
    e[u] = i < p.pairs ? p.ids[(int64_t)(i / p.top_k) * p.ldi + i % p.top_k] : -1;
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) rank[u] = (uint32_t)e[u] < (uint32_t)p.experts ? atomicAdd(&count[e[u]], 1) : -1;
  __syncthreads();
  if (p.chunks > 1) {
    for (int i = tid; i < p.experts; i += 256) p.counts[w * p.experts + i] = count[i];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = w * kChunk + u * 256 + tid;
      if (i < p.pairs) p.pos[i] = rank[u];
    }
    return;
  }
  int rows[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) rows[i] = count[tid * 4 + i];
  place_experts(p, rows, first, tmp, true);
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = u * 256 + tid;
    if (i >= p.pairs) break;
    const int row = rank[u] < 0 ? -1 : first[e[u]] + rank[u];
    p.pos[i] = row;
    if (row >= 0) p.src[row] = i, p.tok[row] = i / p.top_k;
  }
}

// The rest of a plan of several chunks: workgroup w adds up the chunks'
// counts (those before its own apart), places the experts, and gives its
// chunk's pairs their rows.  All workgroups find the same places; the first
// writes the list.
__global__ __launch_bounds__(256) void moe_scatter_kernel(PlanArgs p) {
  __shared__ int all[kMaxExperts], before[kMaxExperts], first[kMaxExperts], tmp[2][4];
  const int tid = threadIdx.x, w = blockIdx.x;
#pragma unroll
  for (int i = 0; i < kMaxExperts; i += 256) all[i + tid] = before[i + tid] = 0;
  __syncthreads();
  for (int i = tid; i < p.chunks * p.experts; i += 256) {
    const int n = p.counts[i], c = i / p.experts, e = i - c * p.experts;
    if (n) {
      atomicAdd(&all[e], n);
      if (c < w) atomicAdd(&before[e], n);
    }
  }
  __syncthreads();
  int rows[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) rows[i] = all[tid * 4 + i];
  place_experts(p, rows, first, tmp, w == 0);
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = w * kChunk + u * 256 + tid;
    if (i >= p.pairs) break;
    const int rank = p.pos[i];
    if (rank < 0) continue;
    const int t = i / p.top_k;
    const int e = p.ids[(int64_t)t * p.ldi + i % p.top_k];
    const int row = first[e] + before[e] + rank;
    p.pos[i] = row;
    p.src[row] = i;
    p.tok[row] = t;
  }
}

// The lanes of the wave whose expert (0 .. 1023) is this lane's, among those
// with `there`: ten votes, one a bit.
__device__ __forceinline__ uint64_t same_expert(int e, bool there) {
  uint64_t m = __ballot(there);
#pragma unroll
  for (int b = 0; b < 10; ++b) {
    const bool one = (e >> b) & 1;
    const uint64_t v = __ballot(one);
    m &= one ? v : ~v;
  }
  return m;
}
__device__ __forceinline__ uint64_t lanes_below(int lane) { return (1ull << lane) - 1; }

// ---- Up to 64 pairs (kFewPairs): lane i of a wave holds pair i, and every wave
// makes the plan for itself.  A pair's place among its expert's is its rank
// in pair order; a block is up to 16 of them, from a rank that 16 divides.
constexpr int kFewPairs = 64, kFewTokens = 4;
constexpr int kSomePairs = kChunk;  // pairs of the one-launch sum (moe_down_sum_kernel)
struct FewPlan {
  int e, rank;
  uint64_t same;     // the lanes of this lane's expert
  uint64_t leaders;  // the lanes that begin a block, in block order
};
__device__ __forceinline__ FewPlan few_plan(const int32_t* ids, int64_t ldi, int pairs, int top_k, int experts,
                                            int lane) {
  FewPlan f;
  const int i = lane < pairs ? lane : 0;
  f.e = ids[(int64_t)(i / top_k) * ldi + i % top_k];
  const bool there = lane < pairs && (uint32_t)f.e < (uint32_t)experts;
  f.same = same_expert(f.e, there);
  f.rank = there ? __popcll(f.same & lanes_below(lane)) : -1;
  f.leaders = __ballot(there && (f.rank & 15) == 0);
  return f;
}
// Block b: its expert, rows, and the lanes (pairs) that are its rows; the
// lane that begins it.  (Uniform.)
struct FewBlock {
  int expert, rows, rank0;
  uint64_t lanes;
};
__device__ __forceinline__ FewBlock few_block(const FewPlan& f, int b) {
  uint64_t m = f.leaders;
  for (int i = 0; i < b; ++i) m &= m - 1;
  const int l = __builtin_ctzll(m);
  FewBlock k;
  k.expert = __builtin_amdgcn_readlane(f.e, l);
  k.rank0 = __builtin_amdgcn_readlane(f.rank, l);
  k.lanes = __ballot(f.e == k.expert && f.rank >= k.rank0 && f.rank < k.rank0 + 16);
  k.rows = __popcll(k.lanes);
  return k;
}

// --------------------------------------------------------- the rows' padding

// The padding of row r of strip s of the second product's input past its K2
// values, to whole K-steps and scale groups: zeros with scale 1.  Thread `at`
// of `step` takes every step-th block.
__device__ __forceinline__ void pad_rows(int s, int r, int at, int step, int K2, int Kt2, int G2, uint8_t* h,
                                         uint8_t* hs) {
  for (int c2 = (K2 >> 5) + at; c2 < G2 * 16; c2 += step) {
    const int t2 = c2 >> 2, k2 = c2 & 3;
    if (t2 < Kt2) *reinterpret_cast<int4*>(h + ((int64_t)s * Kt2 + t2) * 1024 + (k2 * 16 + r) * 16) = (int4){0, 0, 0, 0};
    hs[((int64_t)s * G2 + (t2 >> 2)) * 256 + (k2 * 16 + r) * 4 + (t2 & 3)] = (uint8_t)kE8M0One;
  }
}

// ------------------------------------------------------ plan and quantisation

// The rows of x per 1x32, by token: codes [tokens][Kt * 64], scales
// [tokens][G * 16], of a group of 4 K-steps byte kb * 4 + j for block kb of
// step j, so that a row's blocks of a step are 64 consecutive bytes and a
// lane's scales of a group one word.  Past K: zeros with scale 1.  The products
// gather the rows from here by their tokens.
struct QuantArgs {
  const uint16_t* x;
  int64_t ldx;
  int64_t tokens;
  int K, Kt, G;
  uint8_t *q, *scales;
};
// A wave takes U segments of 512 values (one scale group), 8 a lane, all loads
// first.
template <int U>
__device__ __forceinline__ void quant_segments(const QuantArgs& a, int64_t first) {
  const int lane = threadIdx.x & 63;
  const int64_t total = a.tokens * a.G;
  uint32_t w[U][4];
  bool valid[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t s = first + j;
    const int64_t row = s / a.G;
    const int k0 = (int)(s % a.G) * 512 + lane * 8;
    valid[j] = s < total && k0 < a.K;
    w[j][0] = w[j][1] = w[j][2] = w[j][3] = 0;
    if (valid[j]) {
      const int4 v = *reinterpret_cast<const int4*>(a.x + row * a.ldx + k0);
      w[j][0] = (uint32_t)v.x, w[j][1] = (uint32_t)v.y, w[j][2] = (uint32_t)v.z, w[j][3] = (uint32_t)v.w;
    }
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t s = first + j;
    if (s >= total) break;  // uniform across the wave
    const int64_t row = s / a.G;
    const int g = (int)(s % a.G), c = lane >> 2;
    const uint32_t b = valid[j] ? e8m0_of_amax_bits(quad_amax_bits(w[j][0], w[j][1], w[j][2], w[j][3])) : kE8M0One;
    const uint32_t code = valid[j] ? e2m1_pack8(w[j][0], w[j][1], w[j][2], w[j][3], e8m0_value(b)) : 0u;
    if (g * 4 + (c >> 2) < a.Kt)
      *reinterpret_cast<uint32_t*>(a.q + row * a.Kt * 64 + g * 256 + lane * 4) = code;
    if ((lane & 3) == 0) a.scales[row * a.G * 16 + g * 16 + (c & 3) * 4 + (c >> 2)] = (uint8_t)b;
  }
}

// The first `chunks` workgroups make the plan (or its chunks), the others
// quantise: neither needs the other.
template <int U>
__global__ __launch_bounds__(256) void moe_prepare_kernel(PlanArgs p, QuantArgs a) {
  if ((int)blockIdx.x < p.chunks)
    plan_chunk(p, blockIdx.x);
  else
    quant_segments<U>(a, (((int64_t)blockIdx.x - p.chunks) * 4 + (threadIdx.x >> 6)) * U);
}

hipError_t launch_prepare(const PlanArgs& p, const QuantArgs& a, hipStream_t stream) {
  const int64_t segs = a.tokens * a.G;
  // four segments a wave where there are many (as in the quantisation kernels)
  if (segs >= 8192)
    moe_prepare_kernel<4><<<dim3((unsigned)(p.chunks + cdiv(segs, 16))), 256, 0, stream>>>(p, a);
  else
    moe_prepare_kernel<1><<<dim3((unsigned)(p.chunks + cdiv(segs, 4))), 256, 0, stream>>>(p, a);
  if (p.chunks > 1) moe_scatter_kernel<<<dim3((unsigned)p.chunks), 256, 0, stream>>>(p);
  return hipGetLastError();
}

// -------------------------------------------------------------- the products

// One side's operands: quantised rows (GEMM layouts) and the experts'
// weights.
struct ProductArgs {
  const MoeHead* head;
  const MoeBlock* blocks;
  const int32_t* tok;    // up: the rows' tokens
  uint32_t a_bytes, as_bytes;  // up: of the quantised tokens
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

// The waves' partial tiles in LDS, [tile][register][wave][lane], and their sum
// in wave order.
template <int MT, int NS>
__device__ __forceinline__ void store_parts(float* red, const v4f (&acc)[MT][NS]) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, KW = blockDim.x >> 6;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) red[(((i * NS + j) * 4 + r) * KW + wv) * 64 + lane] = acc[i][j][r];
}
__device__ __forceinline__ float sum_parts(const float* red, int tile, int reg, int l) {
  const int KW = blockDim.x >> 6;
  const float* s = red + (tile * 4 + reg) * KW * 64 + l;
  float v = s[0];
  for (int w = 1; w < KW; ++w) v += s[w * 64];
  return v;
}

// The end of the first product's workgroup: its 32 columns' sums activated,
// rounded to bf16, encoded per row (one 1x32 block) and stored in the GEMM
// layout of the second.  The last column's workgroup also pads the rows.
template <int MT, int NS>
__device__ __forceinline__ void finish_rows(const ProductArgs& p, float* red, const uint16_t* bias, int strip, int rows,
                                            int c) {
  const int KW = blockDim.x >> 6;
  uint16_t* stg = reinterpret_cast<uint16_t*>(red + MT * NS * 4 * KW * 64);  // [MT * 16][32] bf16
  for (int idx = threadIdx.x; idx < MT * 512; idx += blockDim.x) {
    const int l = idx & 63, reg = (idx >> 6) & 3, jj = (idx >> 8) & 1, i = idx >> 9;
    const int m = i * 16 + 4 * (l >> 4) + reg, n = jj * 16 + (l & 15);
    float g = sum_parts(red, i * NS + jj, reg, l);
    if (bias) g += bf16_to_f32(bias[c * 32 + n]);
    float v = activate(g, p.act);
    if constexpr (NS == 4) {
      float up = sum_parts(red, i * NS + 2 + jj, reg, l);
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
      if (c == p.cols - 1) pad_rows((int)s, r, piece, 4, p.inner, Kt2, G2, p.h, p.hs);
    }
  }
}

// A workgroup takes 32 output columns of one block of MT row tiles: NS weight
// strips (up, gated: two of the gate and the two beside them of the other
// half; else two), its KW waves the groups of 4 K-steps in turn.  All of a
// group's loads go out before its first product.  The waves' partial sums
// meet in LDS and are added in wave order.
constexpr int stream_waves(int mt) { return mt == 1 ? 12 : 8; }

template <int MT, int NS, bool UP>
__global__ __launch_bounds__(64 * stream_waves(MT)) void moe_stream_kernel(ProductArgs p) {
  extern __shared__ float red[];
  const int bi = blockIdx.y, c = blockIdx.x;
  if (bi >= p.head->blocks) return;
  const MoeBlock blk = p.blocks[bi];
  const int expert = __builtin_amdgcn_readfirstlane(blk.expert);
  const int strip = __builtin_amdgcn_readfirstlane(blk.strip);
  const int rows = __builtin_amdgcn_readfirstlane(blk.rows);
  const int lane = threadIdx.x & 63;
  const int wv = threadIdx.x >> 6;
  const int KW = blockDim.x >> 6;

  // up: rows gathered from the quantised tokens; down: the block's strips
  const int nst = (rows + 15) >> 4;
  const auto ra = UP ? make_rsrc(p.a, p.a_bytes)
                     : make_rsrc(p.a + (int64_t)strip * p.Kt * 1024, (uint32_t)(nst * p.Kt) * 1024u);
  const auto ras = UP ? make_rsrc(p.as, p.as_bytes)
                      : make_rsrc(p.as + (int64_t)strip * p.G * 256, (uint32_t)(nst * p.G) * 256u);
  uint32_t arow[MT], srow[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = i * 16 + (lane & 15);
    arow[i] = srow[i] = kOOB;
    if (m < rows) {
      if constexpr (UP) {
        const uint32_t t = (uint32_t)p.tok[strip * 16 + m];
        arow[i] = t * (uint32_t)p.Kt * 64u + (uint32_t)(lane >> 4) * 16u;
        srow[i] = t * (uint32_t)p.G * 16u + (uint32_t)(lane >> 4) * 4u;
      } else {
        arow[i] = (uint32_t)(i * p.Kt) * 1024u + (uint32_t)lane * 16u;
        srow[i] = (uint32_t)(i * p.G) * 256u + (uint32_t)lane * 4u;
      }
    }
  }
  constexpr uint32_t kStep = UP ? 64u : 1024u, kGroup = UP ? 16u : 256u;
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
    for (int i = 0; i < MT; ++i) sa[i] = buf_load4(ras, srow[i] + (uint32_t)g * kGroup);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = g * 4 + u;
#pragma unroll
      for (int i = 0; i < MT; ++i)
        af[u][i] = buf_load16(ra, t < p.Kt ? arow[i] + (uint32_t)t * kStep : kOOB);
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

  store_parts<MT, NS>(red, acc);
  __syncthreads();
  const uint16_t* bias = p.bias ? p.bias + (int64_t)expert * p.Ns * 16 : nullptr;
  if constexpr (UP) {
    finish_rows<MT, NS>(p, red, bias, strip, rows, c);
  } else {
    for (int idx = threadIdx.x; idx < MT * 512; idx += blockDim.x) {
      const int l = idx & 63, reg = (idx >> 6) & 3, jj = (idx >> 8) & 1, i = idx >> 9;
      const int m = i * 16 + 4 * (l >> 4) + reg, n = c * 32 + jj * 16 + (l & 15);
      if (m >= rows) continue;
      float v = sum_parts(red, i * NS + jj, reg, l);
      if (bias) v += bf16_to_f32(bias[n]);
      p.part[((int64_t)strip * 16 + m) * p.hidden + n] = v;
    }
  }
}

template <int MT, int NS, bool UP>
hipError_t launch_stream(const ProductArgs& p, int64_t max_blocks, hipStream_t stream) {
  const int kw = p.G < stream_waves(MT) ? p.G : stream_waves(MT);
  const size_t lds = (size_t)MT * NS * 4 * kw * 64 * 4 + (UP ? MT * 16 * 32 * 2 : 0);
  // (columns and blocks in two dimensions of the grid: a launch does no more
  // than 2^32 work items of one; blocks are fewer than 2^12, kStreamRows rows of
  // kMaxExperts experts at most)
  moe_stream_kernel<MT, NS, UP><<<dim3((unsigned)p.cols, (unsigned)max_blocks), 64 * kw, lds, stream>>>(p);
  return hipGetLastError();
}

template <int MT>
hipError_t launch_up(const ProductArgs& p, bool gated, int64_t max_blocks, hipStream_t stream) {
  return gated ? launch_stream<MT, 4, true>(p, max_blocks, stream) : launch_stream<MT, 2, true>(p, max_blocks, stream);
}

// What the kernels of few pairs read besides ProductArgs.
struct FewArgs {
  const int32_t* ids;
  int64_t ldi;
  int pairs, top_k, experts;
  const uint16_t* x;
  int64_t ldx;
  int K;
};

// The first product of up to 64 pairs: plan, quantisation and product in one
// launch.  The K split is the streaming form's; a wave encodes its groups'
// blocks of the rows, four rows at a time, one block a lane (lane l: row l / 16,
// block l % 16 of the group), and moves them to their operand lanes by
// permutes while the weights are in flight.
template <int NS>
__global__ __launch_bounds__(768) void moe_up_few_kernel(ProductArgs p, FewArgs a) {
  extern __shared__ float red[];
  const int bi = (int)(blockIdx.x / (unsigned)p.cols), c = (int)(blockIdx.x % (unsigned)p.cols);
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, KW = blockDim.x >> 6;
  const FewPlan f = few_plan(a.ids, a.ldi, a.pairs, a.top_k, a.experts, lane);
  if (bi >= __popcll(f.leaders)) return;
  const FewBlock blk = few_block(f, bi);
  const auto rw = make_rsrc(p.w + (int64_t)blk.expert * p.Ns * p.Kt * 1024, (uint32_t)p.Ns * p.Kt * 1024u);
  const auto rws = make_rsrc(p.ws + (int64_t)blk.expert * p.Ns * p.G * 256, (uint32_t)p.Ns * p.G * 256u);
  const int nblk = a.K >> 5;
  // the token of this lane's row in each pass of four rows: row n is the
  // n-th of the block's lanes
  const int er = lane >> 4, ec = lane & 15;
  int token[4];
  {
    uint64_t m = blk.lanes;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      token[q] = -1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int pair = m ? __builtin_ctzll(m) : -1;
        if (m) m &= m - 1;
        if (er == i && pair >= 0) token[q] = pair / a.top_k;
      }
    }
  }
  const int mr = lane & 15;
  const uint32_t src0 = (uint32_t)((mr & 3) * 16 + (lane >> 4)) * 4u;

  v4f acc[1][NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) acc[0][j] = (v4f){0.f, 0.f, 0.f, 0.f};
  for (int g = wv; g < p.G; g += KW) {
    const bool block_in = g * 16 + ec < nblk;
    int4 xv[4];
    const auto load_x = [&](int tok) {
      const bool ok = tok >= 0 && block_in;
      const int4* xp = reinterpret_cast<const int4*>(a.x + (int64_t)(ok ? tok : 0) * a.ldx + (ok ? (g * 16 + ec) * 32 : 0));
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int4 v = xp[q];
        xv[q] = {ok ? v.x : 0, ok ? v.y : 0, ok ? v.z : 0, ok ? v.w : 0};
      }
    };
    load_x(token[0]);
    int4 bf[4][NS];
    uint32_t sb[NS];
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
    __builtin_amdgcn_sched_barrier(0);
    int4 af[4];
    uint32_t sa[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) af[u] = (int4){0, 0, 0, 0}, sa[u] = kE8M0One;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q * 4 >= blk.rows) continue;  // (uniform)
      if (q) load_x(token[q]);
      uint32_t b;
      const int4 code = quant_block32(xv, b);
      const bool here = (mr >> 2) == q && mr < blk.rows;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int src = (int)(src0 + (uint32_t)u * 16u);
        const int4 v = {__builtin_amdgcn_ds_bpermute(src, code.x), __builtin_amdgcn_ds_bpermute(src, code.y),
                        __builtin_amdgcn_ds_bpermute(src, code.z), __builtin_amdgcn_ds_bpermute(src, code.w)};
        const uint32_t sc = (uint32_t)__builtin_amdgcn_ds_bpermute(src, (int)b);
        af[u] = {here ? v.x : af[u].x, here ? v.y : af[u].y, here ? v.z : af[u].z, here ? v.w : af[u].w};
        sa[u] = here ? sc : sa[u];
      }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        switch (u) {
          case 0: acc[0][j] = mfma_fp4<0, 0>(af[u], bf[u][j], sa[u], sb[j], acc[0][j]); break;
          case 1: acc[0][j] = mfma_fp4<0, 1>(af[u], bf[u][j], sa[u], sb[j], acc[0][j]); break;
          case 2: acc[0][j] = mfma_fp4<0, 2>(af[u], bf[u][j], sa[u], sb[j], acc[0][j]); break;
          default: acc[0][j] = mfma_fp4<0, 3>(af[u], bf[u][j], sa[u], sb[j], acc[0][j]); break;
        }
      }
  }
  store_parts<1, NS>(red, acc);
  __syncthreads();
  // block b of the plan is strip b of the rows
  finish_rows<1, NS>(p, red, p.bias ? p.bias + (int64_t)blk.expert * p.Ns * 16 : nullptr, bi, blk.rows, c);
}

// The second product and the sum over a token's choices in one launch, for up
// to kSomePairs pairs in blocks of one row tile: a workgroup takes 16 output
// columns of every block, its waves one (block, share of K) each in turn.
// The products, bias added, meet in LDS, [share][pair][16 columns]; then a
// thread adds an output's choices in their order.  FEW: the plan is made in
// the wave, block b's rows in strip b.
struct SumArgs {
  MoeArgs m;
  const MoeHead* head;
  const MoeBlock* blocks;
  const int32_t* src;
  const uint8_t *h, *hs;
  int Kt, G, Ns;    // of the weights
  int shares, gps;  // shares of K, groups of one
};
constexpr int kSumWaves = 8;
template <bool FEW>
__global__ __launch_bounds__(64 * kSumWaves) void moe_down_sum_kernel(SumArgs p) {
  extern __shared__ float y[];
  __shared__ float weight[kSomePairs];
  __shared__ uint8_t counts[kSomePairs];
  const MoeArgs& m = p.m;
  const int pairs = (int)m.tokens * m.top_k;
  for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
    const int t = i / m.top_k, j = i % m.top_k;
    counts[i] = (uint32_t)m.ids[t * m.ldi + j] < (uint32_t)m.experts;
    weight[i] = m.weights[t * m.ldw + j];
  }
  const int c = blockIdx.x;  // 16-column strip
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), NW = blockDim.x >> 6;
  FewPlan f;
  int nb;
  if constexpr (FEW) {
    f = few_plan(m.ids, m.ldi, pairs, m.top_k, m.experts, lane);
    nb = __popcll(f.leaders);
  } else {
    nb = p.head->blocks;
  }
  for (int task = wv; task < nb * p.shares; task += NW) {
    const int b = task / p.shares, share = task % p.shares;
    int expert, strip, rows, pair = -1;
    if constexpr (FEW) {
      const FewBlock k = few_block(f, b);
      expert = k.expert, strip = b, rows = k.rows;
      uint64_t left = k.lanes;
      for (int r = 0; r < rows; ++r) {
        if ((lane & 15) == r) pair = __builtin_ctzll(left);
        left &= left - 1;
      }
    } else {
      const MoeBlock k = p.blocks[b];
      expert = __builtin_amdgcn_readfirstlane(k.expert);
      strip = __builtin_amdgcn_readfirstlane(k.strip);
      rows = __builtin_amdgcn_readfirstlane(k.rows);
      if ((lane & 15) < rows) pair = p.src[strip * 16 + (lane & 15)];
    }
    const auto ra = make_rsrc(p.h + (int64_t)strip * p.Kt * 1024, (uint32_t)p.Kt * 1024u);
    const auto ras = make_rsrc(p.hs + (int64_t)strip * p.G * 256, (uint32_t)p.G * 256u);
    const auto rw = make_rsrc(m.down + ((int64_t)expert * p.Ns + c) * p.Kt * 1024, (uint32_t)p.Kt * 1024u);
    const auto rws = make_rsrc(m.down_scales + ((int64_t)expert * p.Ns + c) * p.G * 256, (uint32_t)p.G * 256u);
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    const int g1 = min((share + 1) * p.gps, p.G);
    for (int g = share * p.gps; g < g1; g += 2) {
      int4 w[8], a[8];
      uint32_t sw[2], sa[2];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int t = g * 4 + u;
        const bool in = t < p.Kt && g + u / 4 < g1;
        w[u] = __builtin_bit_cast(int4, __builtin_amdgcn_raw_buffer_load_b128(
                                            rw, in ? (uint32_t)(t * 1024 + lane * 16) : kOOB, 0, kAuxNT));
      }
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint32_t off = g + v < g1 ? (uint32_t)((g + v) * 256 + lane * 4) : kOOB;
        sw[v] = buf_load4(rws, off);
        sa[v] = buf_load4(ras, off);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int t = g * 4 + u;
        const bool in = t < p.Kt && g + u / 4 < g1 && (lane & 15) < rows;
        a[u] = buf_load16(ra, in ? (uint32_t)(t * 1024 + lane * 16) : kOOB);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint32_t s0 = sw[u / 4], s1 = sa[u / 4];
        switch (u & 3) {
          case 0: acc = mfma_fp4<0, 0>(w[u], a[u], s0, s1, acc); break;
          case 1: acc = mfma_fp4<1, 1>(w[u], a[u], s0, s1, acc); break;
          case 2: acc = mfma_fp4<2, 2>(w[u], a[u], s0, s1, acc); break;
          default: acc = mfma_fp4<3, 3>(w[u], a[u], s0, s1, acc); break;
        }
      }
    }
    // lane: columns 4 (l / 16) .. + 3 of row l % 16
    const int n = 4 * (lane >> 4);
    if (m.down_bias && share == 0) {
      const uint16_t* bias = m.down_bias + (int64_t)expert * m.hidden + c * 16 + n;
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] += bf16_to_f32(bias[r]);
    }
    if (pair >= 0) *reinterpret_cast<v4f*>(y + ((int64_t)share * pairs + pair) * 16 + n) = acc;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < (int)m.tokens * 16; i += blockDim.x) {
    const int t = i >> 4, n = i & 15;
    float v = m.residual ? bf16_to_f32(m.residual[t * m.ldr + c * 16 + n]) : 0.f;
    for (int j = 0; j < m.top_k; ++j) {
      const int pair = t * m.top_k + j;
      if (!counts[pair]) continue;
      float s = y[pair * 16 + n];
      for (int k = 1; k < p.shares; ++k) s += y[(k * pairs + pair) * 16 + n];
      v += weight[pair] * s;
    }
    m.out[t * m.ldo + c * 16 + n] = f32_to_bf16_rne(v);
  }
}

hipError_t launch_down_sum(const MoeArgs& p, const MoeLayout& l, bool few, int64_t max_blocks, hipStream_t stream) {
  SumArgs s{};
  s.m = p;
  s.head = reinterpret_cast<const MoeHead*>(p.work + l.head);
  s.blocks = reinterpret_cast<const MoeBlock*>(p.work + l.blocks);
  s.src = reinterpret_cast<const int32_t*>(p.work + l.src);
  s.h = p.work + l.h, s.hs = p.work + l.hs;
  s.Kt = (int)cdiv(p.inner, 128), s.G = (int)cdiv(s.Kt, 4), s.Ns = p.hidden / 16;
  const int pairs = (int)p.tokens * p.top_k;
  // shares of K so that few blocks still fill the workgroup's waves
  int shares = (int)(kSumWaves / max_blocks);
  if (shares > s.G) shares = s.G;
  if (shares > kSomePairs / pairs) shares = kSomePairs / pairs;
  if (shares < 1) shares = 1;
  s.gps = (s.G + shares - 1) / shares;
  s.shares = (s.G + s.gps - 1) / s.gps;
  const int64_t tasks = max_blocks * s.shares;
  const int waves = tasks < kSumWaves ? (int)tasks : kSumWaves;
  const size_t lds = (size_t)s.shares * pairs * 64;
  if (few)
    moe_down_sum_kernel<true><<<dim3((unsigned)s.Ns), 64 * waves, lds, stream>>>(s);
  else
    moe_down_sum_kernel<false><<<dim3((unsigned)s.Ns), 64 * waves, lds, stream>>>(s);
  return hipGetLastError();
}

// The large-M kernel over the plan's row tiles.
hipError_t launch_tiles(const GemmArgs& p, int64_t max_blocks, hipStream_t stream) {
  const int out_strips = p.gated ? p.Ns / 2 : p.Ns;
  const int wide = p.gated ? 8 : 16;
  const int64_t tiles = max_blocks * cdiv(out_strips, wide);
  return launch_prefill_experts(p, (int)(tiles < p.cus ? tiles : p.cus), stream);
}

// --------------------------------------------------------------- the combine

// A token's rows, weighted and added in the order of its choices: four columns
// a thread, the rows of up to eight choices under way together.
__global__ __launch_bounds__(256) void moe_combine_kernel(MoeArgs p, const int32_t* pos, const float* part) {
  const int64_t quads = p.hidden / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.tokens * quads) return;
  const int64_t t = i / quads;
  const int n = (int)(i % quads) * 4;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.residual) {
    const uint2 r = *reinterpret_cast<const uint2*>(p.residual + t * p.ldr + n);
    v[0] = __uint_as_float(r.x << 16), v[1] = __uint_as_float(r.x & 0xFFFF0000u);
    v[2] = __uint_as_float(r.y << 16), v[3] = __uint_as_float(r.y & 0xFFFF0000u);
  }
  for (int j0 = 0; j0 < p.top_k; j0 += 8) {
    int row[8];
    float w[8];
    v4f y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool in = j0 + j < p.top_k;
      row[j] = in ? pos[t * p.top_k + j0 + j] : -1;
      w[j] = in ? p.weights[t * p.ldw + j0 + j] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (row[j] >= 0) y[j] = *reinterpret_cast<const v4f*>(part + (int64_t)row[j] * p.hidden + n);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (row[j] < 0) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = fmaf(w[j], y[j][q], v[q]);
    }
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
  PlanArgs plan{};
  plan.ids = p.ids, plan.ldi = p.ldi, plan.pairs = pairs, plan.top_k = p.top_k, plan.experts = p.experts;
  plan.chunks = (int)cdiv(pairs, kChunk);
  plan.head = reinterpret_cast<MoeHead*>(p.work + l.head);
  plan.blocks = reinterpret_cast<MoeBlock*>(p.work + l.blocks);
  plan.counts = reinterpret_cast<int32_t*>(p.work + l.counts);
  plan.pos = reinterpret_cast<int32_t*>(p.work + l.pos);
  plan.src = reinterpret_cast<int32_t*>(p.work + l.src);
  plan.tok = reinterpret_cast<int32_t*>(p.work + l.tok);
  const int64_t mean = pairs / p.experts;
  const bool tiles = moe_tiles(pairs, p.experts);
  const int mt = mean <= 10 ? 1 : 2;
  const int block_strips = tiles ? 16 : mt;
  const int kt1 = (int)cdiv(p.hidden, 128), g1 = (int)cdiv(kt1, 4);
  const int kt2 = (int)cdiv(p.inner, 128), g2 = (int)cdiv(kt2, 4);
  // at most one block per strip, one part block per expert met
  const int64_t met = pairs < p.experts ? pairs : p.experts;
  int64_t max_blocks = l.strips / block_strips + met;
  if (max_blocks > l.strips) max_blocks = l.strips;
  ProductArgs u{};
  u.head = plan.head, u.blocks = plan.blocks, u.tok = plan.tok;
  u.a_bytes = (uint32_t)(p.tokens * kt1 * 64), u.as_bytes = (uint32_t)(p.tokens * g1 * 16);
  u.a = p.work + l.a, u.as = p.work + l.as, u.w = p.up, u.ws = p.up_scales, u.bias = p.up_bias;
  u.Kt = kt1, u.G = g1, u.Ns = p.inner * (p.gated ? 2 : 1) / 16, u.cols = p.inner / 32;
  u.act = p.act, u.inner = p.inner, u.h = p.work + l.h, u.hs = p.work + l.hs;
  hipError_t e;
  if (pairs <= kFewPairs && p.tokens <= kFewTokens) {
    FewArgs f{};
    f.ids = p.ids, f.ldi = p.ldi, f.pairs = pairs, f.top_k = p.top_k, f.experts = p.experts;
    f.x = p.x, f.ldx = p.ldx, f.K = p.hidden;
    const int kw = g1 < 12 ? g1 : 12;
    const int64_t nb = l.strips;
    const dim3 grid((unsigned)(nb * u.cols));
    if (p.gated)
      moe_up_few_kernel<4><<<grid, 64 * kw, (size_t)4 * 4 * kw * 256 + 1024, stream>>>(u, f);
    else
      moe_up_few_kernel<2><<<grid, 64 * kw, (size_t)2 * 4 * kw * 256 + 1024, stream>>>(u, f);
    e = hipGetLastError();
    return e != hipSuccess ? e : launch_down_sum(p, l, true, nb, stream);
  }
  plan.block_strips = block_strips;
  QuantArgs qa{};
  qa.x = p.x, qa.ldx = p.ldx, qa.tokens = p.tokens, qa.K = p.hidden, qa.Kt = kt1, qa.G = g1;
  qa.q = p.work + l.a, qa.scales = p.work + l.as;
  e = launch_prepare(plan, qa, stream);
  if (e != hipSuccess) return e;
  if (pairs <= kSomePairs && mt == 1 && !tiles) {
    e = launch_up<1>(u, p.gated, max_blocks, stream);
    return e != hipSuccess ? e : launch_down_sum(p, l, false, max_blocks, stream);
  }
  float* part = reinterpret_cast<float*>(p.work + l.part);
  if (tiles) {
    GemmArgs v{};
    v.cus = p.cus, v.head = plan.head, v.blocks = plan.blocks, v.row_tokens = plan.tok;
    v.a_bytes = u.a_bytes, v.as_bytes = u.as_bytes;
    v.a = u.a, v.as = u.as, v.w = p.up, v.ws = p.up_scales, v.bias = p.up_bias;
    v.N = p.inner * (p.gated ? 2 : 1), v.K = p.hidden, v.Kt = kt1, v.G = g1, v.Ns = u.Ns;
    v.w_expert = (int64_t)u.Ns * kt1 * 1024, v.ws_expert = (int64_t)u.Ns * g1 * 256;
    v.epilogue = 1, v.act = p.act, v.gated = p.gated;
    v.rows_out = u.h, v.rows_scales = u.hs, v.rows_kt = kt2, v.rows_g = g2;
    e = launch_tiles(v, max_blocks, stream);
    if (e != hipSuccess) return e;
    GemmArgs d{};
    d.cus = p.cus, d.head = plan.head, d.blocks = plan.blocks;
    d.a = p.work + l.h, d.as = p.work + l.hs, d.w = p.down, d.ws = p.down_scales, d.bias = p.down_bias;
    d.N = p.hidden, d.K = p.inner, d.Kt = kt2, d.G = g2, d.Ns = p.hidden / 16;
    d.w_expert = (int64_t)d.Ns * kt2 * 1024, d.ws_expert = (int64_t)d.Ns * g2 * 256;
    d.out = part;
    e = launch_tiles(d, max_blocks, stream);
    if (e != hipSuccess) return e;
  } else {
    e = mt == 1 ? launch_up<1>(u, p.gated, max_blocks, stream) : launch_up<2>(u, p.gated, max_blocks, stream);
    if (e != hipSuccess) return e;
    ProductArgs d{};
    d.head = plan.head, d.blocks = plan.blocks;
    d.a = p.work + l.h, d.as = p.work + l.hs, d.w = p.down, d.ws = p.down_scales, d.bias = p.down_bias;
    d.Kt = kt2, d.G = g2, d.Ns = p.hidden / 16, d.cols = p.hidden / 32;
    d.part = part, d.hidden = p.hidden;
    e = mt == 1 ? launch_stream<1, 2, false>(d, max_blocks, stream) : launch_stream<2, 2, false>(d, max_blocks, stream);
    if (e != hipSuccess) return e;
  }
  moe_combine_kernel<<<dim3((unsigned)cdiv(p.tokens * (p.hidden / 4), 256)), 256, 0, stream>>>(p, plan.pos, part);
  return hipGetLastError();
}

}  // namespace mxfp4
