// Absorbed latent attention over a paged cache, for gfx950.
//
// A cached row is a key for every head (576 values) and, in its first 512
// values, also the value, so a request's S tokens x H heads are S*H query
// rows over ONE sequence of rows:
//   z = scale q . row,  out = softmax(z) rows[:, :512],  lse = ln sum exp z.
// Each row has to be read once for 2 * S*H * (576 + 512) operations: 30 per
// byte at 16 query rows (bound by HBM), 242 at 128 (near the ridge of the
// matrix units), and a prefix that all requests share is bound by the matrix
// units.  A sequence's row blocks read it each for themselves, from L2 where
// they meet in one: 12 requests of 4 row blocks fetch 2.8 times their rows'
// bytes from HBM, one row block each 1.0 times.  Measured on MI355X: 128 requests of 16 heads over up to
// 16000 rows (1.06 GB) 188 us, 5.6 TB/s; 6 of 40000 to 65000 76 us, 4.6 TB/s;
// one of 777 rows 14 us, the time of two launches and one pass of each; 12
// requests of 4 tokens x 128 heads over 1500 to 8191 rows 100 us and 96
// requests of 16 heads sharing 24571 rows 121 us, 0.7 PFLOP/s: at 32 query
// rows a wave one wave is all that a SIMD's registers hold, a 32-key tile
// takes it over 2 us (its products are half of that), and the 64 MB of parts
// and their join are some 25 us of each.
//
// Work is cut along the keys.  The list of all requests' key units (128 keys
// for 16 and 32 query rows, 64 above, and an item's setup) is dealt to the
// workgroups in equal contiguous shares, computed by each workgroup from the
// lengths on the device, so ragged batches stay balanced and a captured graph
// follows new lengths.  A workgroup that holds a whole (request, row block) writes its
// output; otherwise the fp32 accumulators, maxima and sums go to the
// workspace, and a second kernel joins a row's parts in key order (results
// do not depend on timing).
//
// Two forms, by the query rows of a workgroup:
//  * 16 or 32 (attend_split): the four waves of a workgroup take
//    32-key tiles in turn, each with its own LDS tile, accumulators and
//    running softmax, and meet once at the end of the share: no barrier in
//    the loop, and four independent waves keep loads in flight.
//  * 128 (attend_shared): the four waves share each tile (a ring of four in
//    LDS) and take 32 query rows each.
#include "mla_device.h"
#include "mla_launch.h"

namespace mxfp4 {
namespace {

constexpr int kTile = 32;                                  // keys per LDS tile
// A tile in LDS: nine blocks of 64 values (128 bytes) of all 32 rows, so that
// a load covers 8 rows' whole cache lines and a lane that loads keeps one row
// address for all nine.
constexpr uint32_t kBlock = kTile * 128;
constexpr int kBlocks = kRowDim / 64;
constexpr uint32_t kTileBytes = kTile * kRowDim * 2;       // 36 KiB
constexpr uint32_t kTabLds = 4 * kTileBytes;               // page numbers of the shared form's window
constexpr int kTabEntries = 3000;
constexpr uint32_t kMiscLds = kTabLds + kTabEntries * 4;   // scan and softmax exchange
constexpr uint32_t kLdsBytes = kMiscLds + 4096;
static_assert(kLdsBytes <= 160 * 1024, "LDS per workgroup");

// What masked keys load: a key past the end or in a page the cache does not
// have scores -inf and must add 0 * value with a finite value.
// (16-byte loads read it: so its elements are 16 bytes.)
__device__ const int4 zero_row[kRowDim / 8] = {};
static_assert(sizeof(zero_row) == kRowDim * 2 && alignof(decltype(zero_row)) == 16, "a row, in 16-byte pieces");

// One list of work: `B` sequences of rows, `rows` query rows each.
struct ListArgs {
  DecodeArgs d;
  const int32_t* table;
  int64_t ldt;
  const int32_t* lens;   // nullptr: one sequence of `fixed` rows, seen whole by the rows of every request
  int fixed, capacity;   // lengths are clamped to the capacity of a table row
  int B, rows, nt;       // nt row blocks per sequence
  int grid;
  float *part, *pml;     // parts of items that several workgroups share: [2 grid][RB][512], [..][4] (maximum, sums)
  float *ipart, *ipml;   // parts of whole items, by query row (nullptr: write the output)
};

__device__ __forceinline__ int list_len(const ListArgs& a, int b) {
  if (!a.lens) return a.fixed;
  const int n = a.lens[b];
  return n < 0 ? 0 : n > a.capacity ? a.capacity : n;
}

template <int UNIT>
__device__ __forceinline__ int units_of(int n) { return (int)(((uint32_t)n + UNIT - 1) / UNIT); }

// Sum over the workgroup's 256 threads of v before this thread's, and the
// total, through LDS.
__device__ __forceinline__ int scan256(int v, int& total) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  lds_i32_t s = (lds_i32_t)(uintptr_t)kMiscLds;
  if (lane == 63) s[wv] = x;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int w = s[i];
    if (i < wv) before += w;
    total += w;
  }
  __syncthreads();
  return before + x - v;
}

// Workgroups go to the 8 XCDs in turn, each with an L2 of its own: an XCD
// takes consecutive shares of `n`, so that the row blocks of a sequence,
// which read the same rows, meet in one L2.
__device__ __forceinline__ int xcd_order(int w, int n) {
  const int x = w & 7;
  return x * (n >> 3) + min(x, n & 7) + (w >> 3);
}

// One sequence whose row blocks are no more than the workgroups: its keys are
// cut into the same `chunks` pieces of `size` units for every row block, piece
// by piece (all row blocks of a piece run side by side).
struct Single {
  int chunks, size;
};
__device__ __forceinline__ bool is_single(const ListArgs& a) { return a.B == 1 && a.nt <= a.grid; }
__device__ __forceinline__ Single single_split(const ListArgs& a, int units) {
  const int size = (units + a.grid / a.nt - 1) / (a.grid / a.nt);
  return {size ? (units + size - 1) / size : 0, size};
}

template <int RB>
__host__ __device__ constexpr int unit_tiles() { return RB <= 32 ? 4 : 2; }

// What an item costs a workgroup before and after its keys, in units: the
// shares count it, so that a workgroup that ends one item and starts another
// has fewer keys (us with 0, 2, 4, 6 units for 128 rows: 12 requests of 4
// tokens x 128 heads 110, 104.5, 102, 102.5; with 0, 1, 2 for 16 rows: 128
// requests 192.5, 188.5, 188; one or two units a workgroup are cut less
// evenly for it: 8 equal requests of 128 heads and 1000 keys 21.7 -> 24.7,
// 100 of 16 heads and 100 to 700 keys 31.7 -> 27.9).
template <int RB>
__host__ __device__ constexpr int setup_units() { return RB <= 32 ? 1 : 4; }
// Units of an item of n keys in the list that the shares cut (0: no keys).
template <int RB>
__device__ __forceinline__ int item_units(int n) {
  const int units = units_of<unit_tiles<RB>() * kTile>(n);
  return units ? units + setup_units<RB>() : 0;
}

// Share w of `total` units over at most `most` workgroups, each with at least
// one unit: [lo, hi), empty for workgroups without.
__device__ __forceinline__ void share_of(int& w, int total, int most, int& lo, int& hi) {
  const int grid = min(most, total);
  lo = hi = 0;
  if (w < grid) {
    w = xcd_order(w, grid);
    lo = (int)((int64_t)w * total / grid);
    hi = (int)((int64_t)(w + 1) * total / grid);
  }
}

// This workgroup's share w of the list, units [lo, hi), the sequence that
// holds unit lo, and the units before that sequence.
template <int RB>
__device__ __forceinline__ void find_share(const ListArgs& a, int& w, int& b, int& base, int& lo, int& hi) {
  if (a.B <= 64) {  // each wave by itself, one sequence a lane
    const int lane = threadIdx.x & 63;
    const int u = lane < a.B ? a.nt * item_units<RB>(list_len(a, lane)) : 0;
    int upto = u;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(upto, d);
      if (lane >= d) upto += y;
    }
    share_of(w, __builtin_amdgcn_readlane(upto, 63), a.grid, lo, hi);
    const uint64_t holds = __builtin_amdgcn_ballot_w64(upto - u <= lo && lo < upto);
    b = holds ? __builtin_ctzll(holds) : 0;
    base = __builtin_amdgcn_readlane(upto - u, b);
    return;
  }
  const int chunk = (a.B + 255) / 256, b0 = threadIdx.x * chunk, b1 = min(a.B, b0 + chunk);
  int sum = 0;
  for (int i = b0; i < b1; ++i) sum += a.nt * item_units<RB>(list_len(a, i));
  int total;
  int at = scan256(sum, total);
  share_of(w, total, a.grid, lo, hi);
  lds_i32_t s = (lds_i32_t)(uintptr_t)kMiscLds;
  if (at <= lo && lo < at + sum) {
    int i = b0;
    for (;; ++i) {
      const int u = a.nt * item_units<RB>(list_len(a, i));
      if (lo < at + u) break;
      at += u;
    }
    s[0] = i;
    s[1] = at;
  }
  __syncthreads();
  b = __builtin_amdgcn_readfirstlane(s[0]);
  base = __builtin_amdgcn_readfirstlane(s[1]);
  __syncthreads();
}

// The address of key t's row, given its page number (-1: none).
__device__ __forceinline__ uint32_t page_of(const PagedRows& k, uint32_t t) {
  return (__umulhi(t, k.magic) >> k.shift) + (t & k.whole);
}
__device__ __forceinline__ const char* row_at(const PagedRows& k, uint32_t t, int page, bool& ok) {
  ok = (uint32_t)page < (uint32_t)k.pages;
  const uint32_t i = t - page_of(k, t) * (uint32_t)k.page_size;
  return ok ? k.base + page * k.page_bytes + i * k.row_bytes : (const char*)zero_row;
}

// Lane l loads, of each group of 8 rows, row l / 8's chunk l % 8 of every
// block (permuted): its bytes past the row's address.
__device__ __forceinline__ uint32_t load_chunk(uint32_t lane) {
  return ((lane & 7) ^ swizzle128(lane >> 3)) * 16;
}
// Groups g and g ^ 1 differ in bit 3 of the row, which the swizzle maps to bit 0.
__device__ __forceinline__ uint32_t load_chunk(uint32_t lane, uint32_t group) {
  return load_chunk(lane) ^ ((group & 1) << 4);
}
template <bool STREAM, int... J>
__device__ __forceinline__ void load_blocks(uint32_t at, const char* p, std::integer_sequence<int, J...>) {
  (dma16_at<J * 128, STREAM>(at + J * kBlock, p), ...);
}
template <bool STREAM>
__device__ __forceinline__ void load_group(uint32_t at, const char* p) {
  load_blocks<STREAM>(at, p, std::make_integer_sequence<int, kBlocks>{});
}

// Accumulators and query operands of RW query rows.
template <int RW>
struct Rows;
template <>
struct Rows<16> {
  static constexpr int kSteps = kRowDim / 32, kCols = kLatent / 16;
  v8bf q[kSteps];
  v4f o[kCols];
};
template <>
struct Rows<32> {
  static constexpr int kSteps = kRowDim / 16, kCols = kLatent / 32;
  v8bf q[kSteps];
  v16f o[kCols];
};

template <int RW>
__device__ __forceinline__ void clear(Rows<RW>& s) {
#pragma unroll
  for (int i = 0; i < Rows<RW>::kCols; ++i)
#pragma unroll
    for (int j = 0; j < RW * RW / 64; ++j) s.o[i][j] = 0;
}

// Where a lane reads a tile's operands: rows start at multiples of their
// length, so a step's chunk is one XOR away and its row group an immediate
// offset.
template <int RW>
struct LaneAddr {
  uint32_t k, v;
  __device__ __forceinline__ explicit LaneAddr(uint32_t lane) {
    const uint32_t row = lane % RW, part = lane / RW;  // the lane's key row and its 8-value piece of a step
    const uint32_t i16 = lane & 15, vrow = 4 * (lane >> (RW == 16 ? 4 : 5)) + (i16 >> 2);
    const uint32_t vchunk = (RW == 16 ? 0 : 2 * ((lane >> 4) & 1)) + ((i16 & 3) >> 1);
    k = row * 128 + ((part ^ swizzle128(row)) << 4);
    v = vrow * 128 + (i16 & 1) * 8 + ((vchunk ^ swizzle128(vrow)) << 4);
  }
};
// The same within one tile, opaque, so that the steps' addresses are computed
// where they are used and not kept in registers.
template <int RW>
struct TileAddr {
  uint32_t k, v;
  __device__ __forceinline__ TileAddr(const LaneAddr<RW>& l, uint32_t tile) : k(l.k + tile), v(l.v + tile) {
    asm volatile("" : "+v"(k), "+v"(v));
  }
  // Step i of the scores: for 16 rows, keys 0-15 and 16-31 in turn.
  __device__ __forceinline__ v8bf key(int i) const {
    if constexpr (RW == 16) {
      const int s = i >> 1;
      return lds_read16((k ^ ((s & 1) << 6)) + (s >> 1) * kBlock + (i & 1) * 16 * 128);
    } else {
      return lds_read16((k ^ ((i & 3) << 5)) + (i >> 2) * kBlock);
    }
  }
  // Step i of the values: for 16 rows column tile i over all keys, for 32
  // rows column tile i / 2 over keys 0-15 or 16-31.
  __device__ __forceinline__ v8bf value(int i) const {
    if constexpr (RW == 16) {
      const uint32_t a = (v ^ ((i & 3) << 5)) + (i >> 2) * kBlock;
      return join_keys(lds_read_tr(a), lds_read_tr(a + 16 * 128));
    } else {
      const int ct = i >> 1;
      const uint32_t c0 = (ct & 1) << 6, c1 = (ct >> 1) * kBlock + (i & 1) * 16 * 128;
      return join_keys(lds_read_tr((v ^ c0) + c1), lds_read_tr((v ^ (c0 | 16)) + c1 + 8 * 128));
    }
  }
};

// Hides masked keys' scores: `seen` (per lane): keys below it are visible to
// the lane's row; `bad`: bit t set if key t is masked for every row.
template <int RW, int NX>
__device__ __forceinline__ void mask_scores(float (&x)[NX], uint32_t lane, int seen, uint32_t bad) {
  asm volatile("" : "+v"(lane));  // (keeps the keys' numbers out of registers elsewhere)
#pragma unroll
  for (int i = 0; i < NX; ++i) {
    const int t = key_of<RW>(i, lane);
    if (t >= seen || ((bad >> t) & 1)) x[i] = kNegInf;
  }
}

// Product i of the 36 of a 32-row score tile.
__device__ __forceinline__ void score_product(v16f& s, int i, v8bf f, v8bf q) {
  if (i == 0) mfma_vgpr<true, false>(s, f, q);
  else if (i == 35) mfma_vgpr<false, true>(s, f, q);
  else mfma_vgpr<false, false>(s, f, q);
}

// Products between LDS reads and their use: the short ones need more of them.
template <int RW>
constexpr int kValueGroup = RW == 16 ? 8 : 4;
template <int RW>
__device__ __forceinline__ void tile_values(const TileAddr<RW>& at, v8bf (&first)[kValueGroup<RW>], Rows<RW>& st,
                                            const v8bf (&p)[RW / 16]) {
  pipeline<32, kValueGroup<RW>>(first, [&](int i) { return at.value(i); }, [&](int i, v8bf f) {
    if constexpr (RW == 16) st.o[i] = mfma_rows(f, p[0], st.o[i]);
    else st.o[i >> 1] = mfma_rows(f, p[i & 1], st.o[i >> 1]);
  });
}

// One 32-key tile in LDS: scores, softmax step, values; `full`: nothing is masked.
template <int RW>
__device__ __forceinline__ void attend_tile(uint32_t tile, const LaneAddr<RW>& la, Rows<RW>& st, float& m, RowSums& l,
                                            float c, uint32_t lane, bool full, int seen, uint32_t bad) {
  constexpr int NX = RW / 2;
  float x[NX];
  const TileAddr<RW> at(la, tile);
  auto key = [&](int i) { return at.key(i); };
  auto value = [&](int i) { return at.value(i); };
  if constexpr (RW == 16) {
    v8bf ahead[6];
    read_group(ahead, key);
    v4f s[2] = {};
    pipeline<36, 6>(ahead, key, [&](int i, v8bf f) { s[i & 1] = mfma_rows(f, st.q[i >> 1], s[i & 1]); });
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = s[i >> 2][i & 3];
  } else {
    v8bf ahead[3];  // (groups of three: the registers end there)
    read_group(ahead, key);
    v16f s;
    pipeline<36, 3>(ahead, key, [&](int i, v8bf f) { score_product(s, i, f, st.q[i]); });
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = s[i];
  }
  v8bf first[kValueGroup<RW>];
  read_group(first, value);
  if (!full) mask_scores<RW, NX>(x, lane, seen, bad);
  float alpha;
  v8bf p[NX / 8];
  if (softmax_step<RW, NX>(x, c, m, l, alpha, p)) rescale(st.o, alpha);
  tile_values<RW>(at, first, st, p);
}

// Query row r of sequence b: its request, token and head.
struct RowId {
  int b, s, h;
};
__device__ __forceinline__ RowId row_id(const ListArgs& a, int b, int r) {
  if (!a.lens) {
    const int sh = a.d.S * a.d.H;
    b = r / sh;
    r -= b * sh;
  }
  const int s = r / a.d.H;
  return {b, s, r - s * a.d.H};
}

template <int RW>
__device__ __forceinline__ void load_query(const ListArgs& a, const RowId& id, uint32_t lane, Rows<RW>& st) {
  const uint16_t* q = a.d.q + id.b * a.d.sqb + id.s * a.d.sqs + id.h * a.d.sqh + 8 * (lane / RW);
#pragma unroll
  for (int k = 0; k < Rows<RW>::kSteps; ++k)
    st.q[k] = __builtin_bit_cast(v8bf, *(const int4*)(q + k * (512 / RW)));
}

__device__ __forceinline__ int64_t flat_row(const DecodeArgs& d, const RowId& id) {
  return ((int64_t)id.b * d.S + id.s) * d.H + id.h;
}

// Where a segment's rows go: the output, the part of a whole item, or part slot `slot`.
struct Dest {
  bool whole;
  int slot;
};

template <int RB>
__device__ __forceinline__ void store_ml(const ListArgs& a, const Dest& to, const RowId& id, int r_in_block, float m,
                                         const RowSums& l) {
  if (to.whole && !a.ipart) {
    if (a.d.lse) a.d.lse[flat_row(a.d, id)] = l.log_sum_exp(m);
    return;
  }
  float* p = to.whole ? a.ipml + 4 * flat_row(a.d, id) : a.pml + 4 * ((int64_t)to.slot * RB + r_in_block);
  *(v4f*)p = v4f{m, l.exact, l.used, 0};
}

// A share's piece of one item: tiles [t0, t1) of sequence b for row block rt.
template <int RW>
__device__ __forceinline__ void attend_split(const ListArgs& a, int b, int n, int rt, int t0, int t1, Dest to) {
  const uint32_t lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = wv * kTileBytes;
  const int r0 = rt * RW;
  const RowId id = row_id(a, b, min(r0 + (int)(lane % RW), a.rows - 1));
  const int causal = a.lens ? n - a.d.S + 1 : n;      // keys the first token of a request sees
  const int seen = a.lens ? causal + id.s : n;
  const int seen_all = a.lens ? causal + r0 / a.d.H : n;

  float m = kNegInf;
  RowSums l;
  const LaneAddr<RW> la(lane);
  const int32_t* table = a.table + b * a.ldt;
  // Rows 8g + lane / 8 of a tile: page numbers one tile ahead.
  int page[4];
  auto lookup = [&](int t) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int key = t * kTile + 8 * g + (int)(lane >> 3);
      page[g] = t < t1 && key < n ? table[page_of(a.d.cache, key)] : -1;
    }
  };
  lookup(t0 + wv);
  Rows<RW> st;  // (behind the page numbers, which the first rows wait for)
  load_query<RW>(a, id, lane, st);
  clear(st);
  for (int t = t0 + wv; t < t1; t += 4) {
    uint64_t hidden[4];
    wait_lds();
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      bool ok;
      const char* ptr = row_at(a.d.cache, t * kTile + 8 * g + (lane >> 3), page[g], ok) + load_chunk(lane, g);
      hidden[g] = __builtin_amdgcn_ballot_w64(!ok && t * kTile + 8 * g + (int)(lane >> 3) < n);
      // One row block: nothing else reads these rows, and loads that leave
      // no trace in the caches run faster (128 requests of up to 16000 rows:
      // 218 -> 196 us, 5.4 TB/s).
      if (a.nt == 1) load_group<true>(tile + g * 1024, ptr);
      else load_group<false>(tile + g * 1024, ptr);
    }
    lookup(t + 4);
    uint32_t bad = 0;  // keys in pages that the cache does not have (those past the end are not `seen`)
    if ((hidden[0] | hidden[1] | hidden[2] | hidden[3]) != 0) {
#pragma unroll
      for (int i = 0; i < 32; ++i) bad |= (uint32_t)((hidden[i >> 3] >> (8 * (i & 7))) & 1) << i;
    }
    wait_loads<0>();
    attend_tile<RW>(tile, la, st, m, l, a.d.c, lane, bad == 0 && (t + 1) * kTile <= seen_all, seen - t * kTile, bad);
  }

  // The four waves' accumulators meet: rescaled to the rows' common maximum,
  // through the wave's own tile, summed in wave order.
  acc_settle();
  l.exact = rows_sum<RW>(l.exact);
  l.used = rows_sum<RW>(l.used);
  lds_v4f_t ml = (lds_v4f_t)(uintptr_t)kMiscLds;
  if (lane < RW) ml[wv * RW + lane] = v4f{m, l.exact, l.used, 0};
  lds_barrier();
  float mm = kNegInf;
  RowSums ll;
#pragma unroll
  for (int w = 0; w < 4; ++w) mm = fmaxf(mm, ml[w * RW + lane % RW][0]);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const v4f o = ml[w * RW + lane % RW];
    const float fw = o[0] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(o[0] - mm);
    ll.exact += o[1] * fw;
    ll.used += o[2] * fw;
  }
  const float f = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - mm);
  const bool direct = to.whole && !a.ipart;
  // Per row, for the stores: the factor of an output, and where the row goes.
  lds_f32_t inv = (lds_f32_t)(uintptr_t)(kMiscLds + 2048);
  lds_i64_t off = (lds_i64_t)(uintptr_t)(kMiscLds + 2048 + 32 * 4);
  if (threadIdx.x < RW) {
    inv[lane] = direct ? ll.inverse() : 1.0f;
    off[lane] = direct     ? id.b * a.d.sob + id.s * a.d.sos + id.h * a.d.soh
                : to.whole ? flat_row(a.d, id) * kLatent
                           : ((int64_t)to.slot * RW + lane) * kLatent;
    if (r0 + (int)lane < a.rows) store_ml<RW>(a, to, id, lane, mm, ll);
  }
  float* part = to.whole ? a.ipart : a.part;
  const int rows = min(RW, a.rows - r0);
  constexpr int C = RW == 16 ? 512 : 256, LD = C * 4 + 16;  // columns per pass, padded row bytes
  constexpr int kPer = Rows<RW>::kCols * C / 512;
#pragma unroll
  for (int pass = 0; pass < 512 / C; ++pass) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
#pragma unroll
      for (int j = 0; j < RW * RW / 256; ++j) {
        const uint32_t col = i * RW + (RW == 16 ? 4 * (lane >> 4) : 8 * j + 4 * (lane >> 5));
        v4f v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc_read(st.o[pass * kPer + i][4 * j + e]) * f;
        *(lds_v4f_t)(uintptr_t)(tile + (lane % RW) * LD + col * 4) = v;
      }
    }
    lds_barrier();
#pragma unroll 4
    for (int it = 0; it < RW * C / 1024; ++it) {
      const int e = it * 256 + threadIdx.x, r = e / (C / 4), col = e % (C / 4) * 4;
      v4f v = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < 4; ++w) v += *(lds_v4f_t)(uintptr_t)(w * kTileBytes + r * LD + col * 4);
      if (r < rows) {
        const int64_t at = off[r] + pass * C + col;
        if (direct) {
          v *= inv[r];
          *(uint2*)(a.d.out + at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        } else {
          *(v4f*)(part + at) = v;
        }
      }
    }
    lds_barrier();
  }
}

template <int RW>
__device__ __forceinline__ void attend_shared(const ListArgs& a, int b, int n, int rt, int t0, int t1, Dest to) {
  constexpr int RB = 4 * RW;
  const uint32_t lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r0 = rt * RB + wv * RW;
  const RowId id = row_id(a, b, min(r0 + (int)(lane % RW), a.rows - 1));
  const int causal = a.lens ? n - a.d.S + 1 : n;
  const int seen = a.lens ? causal + id.s : n;
  const int seen_all = a.lens ? causal + min(r0, a.rows - 1) / a.d.H : n;

  Rows<RW> st;
  load_query<RW>(a, id, lane, st);
  clear(st);
  float m = kNegInf;
  RowSums l;
  const int32_t* table = a.table + b * a.ldt;
  const int last_page = (int)page_of(a.d.cache, n - 1);
  lds_i32_t tab = (lds_i32_t)(uintptr_t)kTabLds;
  int p0 = 0, p1 = 0;  // the window of page numbers in LDS
  auto window = [&](int t) {
    p0 = (int)page_of(a.d.cache, t * kTile);
    p1 = min(last_page + 1, p0 + kTabEntries);
    for (int i = threadIdx.x; i < p1 - p0; i += 256) tab[i] = table[p0 + i];
  };
  auto covered = [&](int t) { return (int)page_of(a.d.cache, min(n, (t + 1) * kTile) - 1) < p1; };
  // A tile's loads in three steps: page numbers (of the row this lane loads,
  // and of key lane % 32), the row's address and the hidden keys, then the
  // nine loads of this wave's 8 rows.  (Tiles past the end have no rows:
  // their loads fetch zeros.)
  const char* ptr = nullptr;
  const uint32_t chunk = load_chunk(lane, wv);
  const int end = min(n, t1 * kTile);
  auto page_at = [&](int key) {
    const int page = tab[min((int)page_of(a.d.cache, key), p1 - 1) - p0];
    return key < end ? page : -1;
  };
  auto lookup = [&](int t, int& mine, int& all) {
    mine = page_at(t * kTile + 8 * wv + (int)(lane >> 3));
    all = page_at(t * kTile + (int)(lane & 31));
  };
  auto locate = [&](int t, int mine, int all) {
    bool ok;
    ptr = row_at(a.d.cache, t * kTile + 8 * wv + (lane >> 3), mine, ok) + chunk;
    return (uint32_t)__builtin_amdgcn_ballot_w64((uint32_t)all >= (uint32_t)a.d.cache.pages);
  };
  auto load = [&](uint32_t stage) {
    load_group<false>(stage + wv * 1024, ptr);
  };
  auto stage_of = [&](int t) { return ((t - t0) & 3) * kTileBytes; };
  auto refill = [&](int t) {  // a new window if tile t's pages lie past this one
    if (t < t1 && !covered(t)) {
      __syncthreads();
      window(t);
      __syncthreads();
    }
  };
  const LaneAddr<RW> la(lane);
  window(t0);
  __syncthreads();
  // bad[i]: the masked keys of tile t + i
  uint32_t bad[5] = {};
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    refill(t0 + i);
    int mine, all;
    lookup(t0 + i, mine, all);
    bad[i] = locate(t0 + i, mine, all);
    load(stage_of(t0 + i));
  }
  // One wave a SIMD: nothing else fills the matrix unit while this wave
  // does anything but issue products.  So tile t's softmax runs between the
  // value products of tile t - 1, and the loads of tile t + 2 and the
  // addresses of tile t + 3 between the score products of tile t.
  auto full = [&](int t) { return bad[0] == 0 && (t + 1) * kTile <= seen_all; };
  v8bf p[2];            // the probabilities of the tile before,
  bool grew = false;    // whether its maxima rose, and by what the
  float alpha = 1;      // accumulators are to be scaled then
  wait_loads<18>();
  wave_barrier();
  {
    const TileAddr<RW> at(la, stage_of(t0));
    auto key = [&](int i) { return at.key(i); };
    v8bf first[4];
    read_group(first, key);
    v16f s;
    pipeline<36, 4>(first, key, [&](int i, v8bf f) { score_product(s, i, f, st.q[i]); });
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = s[i];
    if (!full(t0)) mask_scores<RW, 16>(x, lane, seen - t0 * kTile, bad[0]);
    softmax_step<RW, 16>(x, a.d.c, m, l, alpha, p);  // (nothing to rescale yet)
  }
  refill(t0 + 3);
  int mine, all;
  lookup(t0 + 3, mine, all);
  bad[3] = locate(t0 + 3, mine, all);
#pragma unroll
  for (int i = 0; i < 4; ++i) bad[i] = bad[i + 1];
  for (int t = t0 + 1; t < t1; ++t) {
    wait_loads<9>();  // tile t is there, t + 1 may be in flight
    wait_lds();
    wave_barrier();   // tile t is whole, and tile t - 2 no longer read
    refill(t + 3);
    const uint32_t fill = stage_of(t + 2);
    v16f s;
    {
      const TileAddr<RW> at(la, stage_of(t));
      auto key = [&](int i) { return at.key(i); };
      v8bf first[4];
      read_group(first, key);
      pipeline<36, 4>(first, key, [&](auto ic, v8bf f) {
        constexpr int i = ic;
        score_product(s, i, f, st.q[i]);
        if constexpr (i < 9) dma16_at<i * 128, false>(fill + wv * 1024 + i * kBlock, ptr);
        else if constexpr (i == 15) lookup(t + 3, mine, all);
        else if constexpr (i == 27) bad[3] = locate(t + 3, mine, all);
      });
    }
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = s[i];
    if (!full(t)) mask_scores<RW, 16>(x, lane, seen - t * kTile, bad[0]);
    float mx = x[0], mu = 0;
    if (grew) rescale(st.o, alpha);
    const TileAddr<RW> at(la, stage_of(t - 1));
    auto value = [&](int i) { return at.value(i); };
    v8bf first[4];
    read_group(first, value);
    pipeline<32, 4>(first, value, [&](int i, v8bf f) {
      st.o[i >> 1] = mfma_rows(f, p[i & 1], st.o[i >> 1]);
      if (i == 0) {
#pragma unroll
        for (int j = 1; j < 16; ++j) mx = fmaxf(mx, x[j]);
      } else if (i == 1) {
        mx = rows_max<RW>(mx) * a.d.c;
        const float mn = mx > m + kLag ? mx : m;
        alpha = mn == m || m == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
        grew = __builtin_amdgcn_ballot_w64(alpha != 1.0f) != 0;
        m = mn;
        mu = m == kNegInf ? 0.0f : m;
        l.scale(alpha);
      } else if (i >= 4 && i < 20) {
        const int e = i - 4;
        x[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], a.d.c, -mu));
        l.exact += x[e];
        asm volatile("" : "+v"(x[e]));  // here, not where the values are used
      }
    });
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i >> 3][i & 7] = (__bf16)x[i];
    l.used = add_rounded(p[1], add_rounded(p[0], l.used));
#pragma unroll
    for (int i = 0; i < 3; ++i) bad[i] = bad[i + 1];
  }
  if (grew) rescale(st.o, alpha);
  {
    const TileAddr<RW> at(la, stage_of(t1 - 1));
    auto value = [&](int i) { return at.value(i); };
    v8bf first[4];
    read_group(first, value);
    tile_values<RW>(at, first, st, p);
  }
  wait_loads<0>();
  __syncthreads();

  acc_settle();
  l.exact = rows_sum<RW>(l.exact);
  l.used = rows_sum<RW>(l.used);
  const int r_in_block = wv * RW + lane % RW;
  auto column = [&](int i, int j) {  // of a lane's values 4j..4j+3 of column tile i
    return i * RW + (RW == 16 ? 4 * (int)(lane >> 4) : 8 * j + 4 * (int)(lane >> 5));
  };
  if (!to.whole) {
    // A part goes out through the wave's share of LDS, so that whole lines
    // are stored (in registers a lane holds 4 columns of its row); rows past
    // the last are stored too, into their place in the part.
    constexpr int C = 256, LD = C * 4 + 16;  // columns per pass, padded row bytes
    constexpr int kPer = Rows<RW>::kCols * C / 512;
    const uint32_t mine = wv * kTileBytes;
    float* part = a.part + ((int64_t)to.slot * RB + wv * RW) * kLatent + 4 * lane;
#pragma unroll
    for (int pass = 0; pass < 512 / C; ++pass) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
#pragma unroll
        for (int j = 0; j < RW * RW / 256; ++j) {
          v4f v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc_read(st.o[pass * kPer + i][4 * j + e]);
          *(lds_v4f_t)(uintptr_t)(mine + (lane % RW) * LD + column(i, j) * 4) = v;
        }
      }
      wait_lds();
#pragma unroll 8
      for (int r = 0; r < RW; ++r)
        *(v4f*)(part + r * kLatent + pass * C) = *(lds_v4f_t)(uintptr_t)(mine + r * LD + lane * 16);
      wait_lds();
    }
  } else if (r0 + (int)(lane % RW) < a.rows) {
    const bool direct = !a.ipart;
    const float inv = l.inverse();
    float* part = direct ? nullptr : a.ipart + flat_row(a.d, id) * kLatent;
    uint16_t* out = a.d.out + id.b * a.d.sob + id.s * a.d.sos + id.h * a.d.soh;
#pragma unroll
    for (int i = 0; i < Rows<RW>::kCols; ++i) {
#pragma unroll
      for (int j = 0; j < RW * RW / 256; ++j) {
        v4f v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc_read(st.o[i][4 * j + e]);
        if (direct) {
          const uint2 w = {pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv)};
          *(uint2*)(out + column(i, j)) = w;
        } else {
          *(v4f*)(part + column(i, j)) = v;
        }
      }
    }
  }
  if (lane < RW && r0 + (int)lane < a.rows) store_ml<RB>(a, to, id, r_in_block, m, l);
  lds_barrier();
}

// Workgroup w's share of one list.
template <int RB>
__device__ __forceinline__ void attend_list(const ListArgs& a, int w) {
  constexpr int kUnitTiles = unit_tiles<RB>(), kUnit = kUnitTiles * kTile;
  constexpr int kSetup = setup_units<RB>();
  int b = 0, base = 0, lo, hi;
  const bool single = is_single(a);
  if (!single) find_share<RB>(a, w, b, base, lo, hi);
  else lo = 0, hi = 1;
  for (int cur = lo; cur < hi;) {
    const int n = __builtin_amdgcn_readfirstlane(list_len(a, b));
    const int units = units_of<kUnit>(n);
    int rt, u0, u1;
    Dest to;
    if (single) {
      const Single cut = single_split(a, units);
      if (w >= cut.chunks * a.nt) break;
      w = xcd_order(w, cut.chunks * a.nt);
      const int k = w / a.nt;
      rt = w - k * a.nt;
      u0 = k * cut.size;
      u1 = min(units, u0 + cut.size);
      to = {cut.chunks == 1, w};
      cur = hi;
    } else {
      const int item = item_units<RB>(n);
      if (cur - base >= item * a.nt) {  // past this sequence (or it is empty)
        base += item * a.nt;
        ++b;
        continue;
      }
      rt = (cur - base) / item;
      const int at = (cur - base) - rt * item, end = min(item, at + hi - cur);
      cur += end - at;
      u0 = max(0, at - kSetup);
      u1 = max(0, end - kSetup);
      if (u0 == u1) continue;  // (nothing but the item's setup)
      to = {u0 == 0 && u1 == units, 2 * w + (u0 == 0)};
    }
    const int tiles = (int)(((uint32_t)n + kTile - 1) / kTile);
    if constexpr (RB <= 32)
      attend_split<RB>(a, b, n, rt, u0 * kUnitTiles, min(tiles, u1 * kUnitTiles), to);
    else
      attend_shared<RB / 4>(a, b, n, rt, u0 * kUnitTiles, min(tiles, u1 * kUnitTiles), to);
  }
}

// One list (PRB = 0), or a prefix's list and then the requests' own: a
// workgroup that has stored its prefix part starts on its requests at once,
// and where there is little work, the requests start from the other end and
// meet workgroups that have no prefix part.
template <int RB, int PRB>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void mla_attend_kernel(ListArgs a,
                                                                                                   ListArgs p) {
  __shared__ int4 lds_raw[kLdsBytes / 16];
  uint32_t anchor = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int4*)lds_raw;
  asm volatile("" : "+s"(anchor)::"memory");  // LDS is addressed by number: its array starts at 0
  if constexpr (PRB != 0) {
    attend_list<PRB>(p, blockIdx.x);
    attend_list<RB>(a, gridDim.x - 1 - blockIdx.x);
  } else {
    attend_list<RB>(a, blockIdx.x);
  }
}

// The workgroups that hold pieces of query row r of sequence b in a list:
// count 0 if the sequence is empty, 1 if one workgroup held the whole item.
// Part i lies in slot first + i * step - (i > 0) * skip.
struct Parts {
  int count, first, step, skip;
};
template <int RB>
__device__ __forceinline__ Parts find_parts(const ListArgs& a, int b, int r) {
  constexpr int kUnit = unit_tiles<RB>() * kTile;
  if (is_single(a)) return {single_split(a, units_of<kUnit>(list_len(a, 0))).chunks, r / RB, a.nt, 0};
  int before = 0, total = 0;  // units of the sequences before b, and of all (each wave by itself)
  for (int i = threadIdx.x & 63; i < a.B; i += 64) {
    const int u = a.nt * item_units<RB>(list_len(a, i));
    if (i < b) before += u;
    total += u;
  }
  before = wave_sum(before);
  total = wave_sum(total);
  const int item = item_units<RB>(list_len(a, b));
  if (item == 0) return {0, 0, 0, 0};
  const int u0 = before + r / RB * item;
  const int grid = min(a.grid, total);
  const int w0 = (int)((((int64_t)u0 + setup_units<RB>() + 1) * grid - 1) / total);
  const int w1 = (int)((((int64_t)u0 + item) * grid - 1) / total);
  // the first workgroup's second slot (the item begins there), then the others' first
  return {w1 - w0 + 1, 2 * w0 + 1, 2, 1};
}

// Where a query row's parts of one list lie: part i is row
// first + i * step - (i > 0) * skip; whole items lie by query row.
struct RowParts {
  const float *part, *pml;
  int count;
  int64_t first;
  int step, skip;
};
template <int RB>
__device__ __forceinline__ RowParts row_parts(const ListArgs& a, int b, int r, int64_t flat) {
  const Parts q = find_parts<RB>(a, b, r);
  const bool whole = q.count == 1;
  return {whole ? a.ipart : a.part, whole ? a.ipml : a.pml, q.count, whole ? flat : (int64_t)q.first * RB + r % RB,
          q.step * RB, q.skip * RB};
}

// Joins the parts of query row r of sequence b, columns c0 .. c0 + 512 / CS: a
// wave's lanes fetch 64 parts' maxima and sums at once, then it runs over the
// parts' values, 8 / CS a lane, one part after another (the loop is not
// unrolled: its lane read keeps the compiler from it).  ALONE: one wave takes
// all parts; otherwise wave w of a workgroup takes parts w, w + 4, .., and the
// four waves' sums meet in LDS in wave order.  Rows that one workgroup of a
// call without a prefix wrote itself are left alone; rows without any key
// become 0 and -inf.
template <int RB, int PRB, int CS, bool ALONE>
__device__ __forceinline__ void join_row(const ListArgs& a, const ListArgs& p, int b, int r, int c0, float (*so)[512 / CS],
                                         float (*sml)[3]) {
  constexpr int W = 8 / CS;                      // columns per lane
  typedef float vec __attribute__((ext_vector_type(CS == 1 ? 4 : W)));
  constexpr int V = CS == 1 ? 4 : W, NV = W / V;  // read as NV vectors, 64 lanes apart
  constexpr int kStride = ALONE ? 1 : 4;         // waves that share the parts
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const RowId id = row_id(a, b, r);
  const int64_t flat = flat_row(a.d, id);
  const RowParts own = row_parts<RB>(a, b, r, flat);
  if (!PRB && own.count == 1) return;
  RowParts pre = {};
  if constexpr (PRB != 0) pre = row_parts<PRB>(p, 0, (int)flat, flat);
  auto part_at = [&](int i, const float*& po, const float*& pm) {  // the prefix's parts, then the request's own
    const bool in_prefix = PRB != 0 && i < pre.count;
    const RowParts& q = in_prefix ? pre : own;
    i -= in_prefix ? 0 : pre.count;
    const int64_t k = q.first + (int64_t)i * q.step - (i > 0 ? q.skip : 0);
    po = q.part + k * kLatent + c0;
    pm = q.pml + 4 * k;
  };
  const int count = pre.count + own.count;
  float m = kNegInf;
  RowSums l;
  vec o[NV] = {};
  for (int i0 = ALONE ? 0 : wv; i0 < count; i0 += 64 * kStride) {  // 64 parts of this wave
    const int mine = i0 + kStride * lane, n = min(64, (count - i0 + kStride - 1) / kStride);
    const float *po, *pm;
    v4f pl = {kNegInf, 0, 0, 0};
    if (lane < n) {
      part_at(mine, po, pm);
      pl = *(const v4f*)pm;
    }
    const float mn = fmaxf(wave_max(pl[0]), m);
    const float keep = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - mn);
    const float f = pl[1] == 0 ? 0.0f : __builtin_amdgcn_exp2f(pl[0] - mn);  // a part without keys counts nothing
    l.scale(keep);
    l.exact += wave_sum(pl[1] * f);
    l.used += wave_sum(pl[2] * f);
    m = mn;
#pragma unroll
    for (int v = 0; v < NV; ++v) o[v] *= keep;
    for (int i = 0; i < n; ++i) {
      const float fi = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), i));
      part_at(i0 + kStride * i, po, pm);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const vec x = *(const vec*)(po + v * 64 * V + V * lane);
#pragma unroll
        for (int e = 0; e < V; ++e) o[v][e] += fi == 0 ? 0.0f : x[e] * fi;
      }
    }
  }
  uint16_t* out = a.d.out + id.b * a.d.sob + id.s * a.d.sos + id.h * a.d.soh + c0;
  if constexpr (ALONE) {
    const float inv = l.inverse();
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const uint2 w = {pack_bf16x2(o[v][0] * inv, o[v][1] * inv), pack_bf16x2(o[v][2] * inv, o[v][3] * inv)};
      *(uint2*)(out + v * 64 * V + V * lane) = w;
    }
    if (a.d.lse && lane == 0) a.d.lse[flat] = l.log_sum_exp(m);
    return;
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) *(vec*)&so[wv][v * 64 * V + V * lane] = o[v];
  if (lane == 0) {
    sml[wv][0] = m;
    sml[wv][1] = l.exact;
    sml[wv][2] = l.used;
  }
  __syncthreads();
  if (threadIdx.x >= 128 / CS) return;
  m = fmaxf(fmaxf(sml[0][0], sml[1][0]), fmaxf(sml[2][0], sml[3][0]));
  l = RowSums();
  v4f t = {0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float f = sml[w][1] == 0 ? 0.0f : __builtin_amdgcn_exp2f(sml[w][0] - m);
    l.exact += sml[w][1] * f;
    l.used += sml[w][2] * f;
    t += *(const v4f*)&so[w][4 * threadIdx.x] * f;
  }
  const float inv = l.inverse();
  const uint2 w = {pack_bf16x2(t[0] * inv, t[1] * inv), pack_bf16x2(t[2] * inv, t[3] * inv)};
  *(uint2*)(out + 4 * threadIdx.x) = w;
  if (a.d.lse && threadIdx.x == 0 && c0 == 0) a.d.lse[flat] = l.log_sum_exp(m);
}

// One workgroup of four waves per query row, or CS workgroups per row with
// 512 / CS columns each.
template <int RB, int PRB, int CS>
__global__ __launch_bounds__(256) void mla_join_kernel(ListArgs a, ListArgs p) {
  __shared__ alignas(16) float so[4][512 / CS];  // (read 16 bytes at a time)
  __shared__ float sml[4][3];
  const int b = blockIdx.x / a.rows, r = blockIdx.x - b * a.rows;
  join_row<RB, PRB, CS, false>(a, p, b, r, blockIdx.y * (512 / CS), so, sml);
}

// One wave per query row, where the rows are many.
template <int RB, int PRB>
__global__ __launch_bounds__(256) void mla_join_waves_kernel(ListArgs a, ListArgs p) {
  const int at = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (at >= a.B * a.rows) return;
  const int b = at / a.rows, r = at - b * a.rows;
  join_row<RB, PRB, 1, true>(a, p, b, r, 0, nullptr, nullptr);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int unit_keys(int rb) { return rb <= 32 ? unit_tiles<16>() * kTile : unit_tiles<128>() * kTile; }
int setup_keys(int rb) { return rb <= 32 ? setup_units<16>() * unit_keys(rb) : setup_units<128>() * unit_keys(rb); }

// Query rows per workgroup for B sequences of `rows` query rows and up to n
// keys.  Blocks of 16 read a sequence's rows once per 16 query rows, but from
// L2, with little to set up and small parts, so they win until the matrix
// units' work counts: up to ten units of 128 keys a compute unit.  Past that,
// 32 rows where there are no more, else 128 (the waves share the loads).
// Measured on MI355X (us, blocks of 16 / 32 / 128): 8 sequences of 64 rows
// and 8000 keys (7.9 units a compute unit) 41.4 / 42.3 / 44.7, one of 128
// rows and 32000 (7.8) 42.7 / 42.8 / 55.2; 8 of 128 and 8000 (15.8) 63.6 /
// 51.2 / 51.0, 32 of 32 and 8000 (15.8) 88.5 / 76.9 / 91.9, 8 of 64 and
// 32000 (31) 144 / 99 / 94, 4 of 512 and 32000 (125) 370 / 214 / 156.  n is
// what the page table can hold, the lengths being known on the device alone
// (and the workspace is sized before them), so short requests in a wide table
// take the form of long ones: 32 requests of 64 rows and 1000 keys 29.6 us in
// a table of 1024 rows, 37.8 in one of 131072.
int rows_per_block(int64_t B, int64_t rows, int64_t n) {
  if (const int forced = get_mla_rows_override()) return forced;
  if (rows <= 16 || B * cdiv(rows, 16) * cdiv(n, 128) <= 10ll * kMlaMaxCus) return 16;
  return rows <= 32 ? 32 : 128;
}

template <int PRB>
void launch_attend(int rb, const ListArgs& a, const ListArgs& p, int cus, hipStream_t s) {
  if constexpr (PRB == 0) {
    switch (rb) {
      case 16: mla_attend_kernel<16, 0><<<a.grid, 256, 0, s>>>(a, p); break;
      case 32: mla_attend_kernel<32, 0><<<a.grid, 256, 0, s>>>(a, p); break;
      default: mla_attend_kernel<128, 0><<<a.grid, 256, 0, s>>>(a, p); break;
    }
  } else {
    const int grid = a.grid + p.grid < cus ? a.grid + p.grid : cus;
    switch (rb) {
      case 16: mla_attend_kernel<16, PRB><<<grid, 256, 0, s>>>(a, p); break;
      case 32: mla_attend_kernel<32, PRB><<<grid, 256, 0, s>>>(a, p); break;
      default: mla_attend_kernel<128, PRB><<<grid, 256, 0, s>>>(a, p); break;
    }
  }
}
template <int PRB, int CS>
void launch_join_columns(int rb, const ListArgs& a, const ListArgs& p, hipStream_t s) {
  const dim3 grid(a.B * a.rows, CS);
  switch (rb) {
    case 16: mla_join_kernel<16, PRB, CS><<<grid, 256, 0, s>>>(a, p); break;
    case 32: mla_join_kernel<32, PRB, CS><<<grid, 256, 0, s>>>(a, p); break;
    default: mla_join_kernel<128, PRB, CS><<<grid, 256, 0, s>>>(a, p); break;
  }
}
template <int PRB>
void launch_join_waves(int rb, const ListArgs& a, const ListArgs& p, hipStream_t s) {
  const int grid = (a.B * a.rows + 3) / 4;
  switch (rb) {
    case 16: mla_join_waves_kernel<16, PRB><<<grid, 256, 0, s>>>(a, p); break;
    case 32: mla_join_waves_kernel<32, PRB><<<grid, 256, 0, s>>>(a, p); break;
    default: mla_join_waves_kernel<128, PRB><<<grid, 256, 0, s>>>(a, p); break;
  }
}
// A row's parts by one workgroup, or by four where the rows are too few to
// keep the compute units' loads in flight (16 rows of 250 parts: 17.3 -> 9.7
// us), or by one wave where workgroups of a row each would not all fit the
// chip (16 heads, a workgroup against a wave a row: 64 requests 5.4, 7.0 us;
// 160 9.0, 6.4; 512 24, 12).
template <int PRB>
void launch_join(int rb, const ListArgs& a, const ListArgs& p, int cus, hipStream_t s) {
  if (a.B * a.rows < 2 * cus) launch_join_columns<PRB, 4>(rb, a, p, s);
  else if (a.B * a.rows < 8 * cus) launch_join_columns<PRB, 1>(rb, a, p, s);
  else launch_join_waves<PRB>(rb, a, p, s);
}

}  // namespace

DecodePlan decode_plan(int64_t B, int64_t S, int64_t H, int64_t max_tokens, int64_t prefix_len, int cus) {
  DecodePlan d{};
  if (cus > kMlaMaxCus) cus = kMlaMaxCus;
  d.cus = cus;
  const int64_t rows = S * H;
  d.rows = rows_per_block(B, rows, max_tokens);
  // (one sequence's shares are cut without the setup: Single)
  int64_t units = B * cdiv(rows, d.rows) * cdiv(max_tokens + (B > 1 ? setup_keys(d.rows) : 0), unit_keys(d.rows));
  d.grid = (int)(units < cus ? (units < 1 ? 1 : units) : cus);
  size_t at = 0;
  auto take = [&](int64_t n) {
    const size_t r = at;
    at += (size_t)((n + 63) / 64 * 64);
    return r;
  };
  d.part = take(2ll * d.grid * d.rows * kLatent);
  d.pml = take(2ll * d.grid * d.rows * 4);
  if (prefix_len > 0) {
    d.prows = rows_per_block(1, B * rows, prefix_len);
    units = cdiv(B * rows, d.prows) * cdiv(prefix_len, unit_keys(d.prows));
    d.pgrid = (int)(units < cus ? units : cus);
    d.ppart = take(2ll * d.pgrid * d.prows * kLatent);
    d.ppml = take(2ll * d.pgrid * d.prows * 4);
    d.ipart = take(2 * B * rows * kLatent);
    d.ipml = take(2 * B * rows * 4);
  }
  d.floats = at;
  return d;
}

hipError_t launch_mla_decode(const DecodeArgs& d, const DecodePlan& plan, hipStream_t stream) {
  const int rows = d.S * d.H;
  ListArgs a{};
  a.d = d;
  a.table = d.table;
  a.ldt = d.ldt;
  a.lens = d.lens;
  a.capacity = (int)((int64_t)d.max_pages * d.cache.page_size);
  a.B = d.B;
  a.rows = rows;
  a.nt = (rows + plan.rows - 1) / plan.rows;
  a.grid = plan.grid;
  a.part = d.work + plan.part;
  a.pml = d.work + plan.pml;
  if (d.prefix_len > 0) {
    const int64_t all = (int64_t)d.B * rows;
    a.ipart = d.work + plan.ipart;
    a.ipml = d.work + plan.ipml;
    ListArgs p = a;
    p.table = d.prefix_table;
    p.ldt = 0;
    p.lens = nullptr;
    p.fixed = d.prefix_len;
    p.B = 1;
    p.rows = (int)all;
    p.nt = (int)cdiv(all, plan.prows);
    p.grid = plan.pgrid;
    p.part = d.work + plan.ppart;
    p.pml = d.work + plan.ppml;
    p.ipart = a.ipart + all * kLatent;
    p.ipml = a.ipml + 4 * all;
    // (Prefix blocks of 32 rows, a batch of 17 to 32 rows over a long prefix,
    // take two launches: no code of their own for every pair of forms.)
    hipError_t e;
    switch (plan.prows) {
      case 16: launch_attend<16>(plan.rows, a, p, plan.cus, stream); break;
      case 128: launch_attend<128>(plan.rows, a, p, plan.cus, stream); break;
      default:
        launch_attend<0>(plan.prows, p, p, plan.cus, stream);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        launch_attend<0>(plan.rows, a, a, plan.cus, stream);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    switch (plan.prows) {
      case 16: launch_join<16>(plan.rows, a, p, plan.cus, stream); break;
      case 32: launch_join<32>(plan.rows, a, p, plan.cus, stream); break;
      default: launch_join<128>(plan.rows, a, p, plan.cus, stream); break;
    }
    return hipGetLastError();
  }
  launch_attend<0>(plan.rows, a, a, plan.cus, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  launch_join<0>(plan.rows, a, a, plan.cus, stream);
  return hipGetLastError();
}

}  // namespace mxfp4
