// Causal attention over keys and values expanded per head (latent
// attention's prompt form), for gfx950: sequences of unequal lengths packed
// along the tokens, keys made of a per-head part and a rotated part that all
// heads share (never copied per head).
//
// One pass over the keys with a running maximum and sum (fp32).  A workgroup
// takes 128 query rows of one head of one sequence, 32 rows a wave, and walks
// the keys in 32-key tiles that its waves share in a ring of LDS stages; loads
// run ahead of the barrier that hands a tile over.  A stage is 32 KiB at
// values of 256 (two stages) and 20 KiB at 128 (four), so that a compute unit
// holds two workgroups, and one's start and barriers pass under the other's
// products.  Eight waves with four stages at 256 measured 1 to 3% slower, and
// softmax steps spread between the products, or a wave priority for them, the
// same.
//
// 2 (dn + 64 + dv) operations per (query, key) pair.  16384 causal tokens of
// 16 heads at 192 + 64 and 256: 1.93-2.12 ms, 1.04-1.14 PFLOP/s; 2 x 1900-2048
// tokens after 14003 others at 128 + 64 and 128: 0.63-0.68 ms, 0.90-0.96; 9
// prompts of 17 to 4001 tokens at 192 + 64 and 256: 0.39-0.41 ms, 0.83-0.87; a
// library product of random 8192 x 8192 matrices 1.44.  What bounds them
// differs.  The long prompt keeps the matrix units busy 64% of the time, and
// the card's power holds the clock at 1.5 to 1.8 GHz under it (the same launch
// on zeros reaches 1.35 PFLOP/s).  The chunks keep them busy 47% at 2.1 GHz:
// there 6.6 vector instructions go with each product (softmax and addresses of
// a tile, for 20 products a wave instead of 32), against 4.6 at 256 values.
// The ragged prompts keep them busy 48% at 2.05 GHz, with 5.2 instructions a
// product and the masked tiles and last blocks of nine sequences.
//
// Few query rows leave most compute units idle that way, each workgroup
// walking all of its keys alone: there the four waves of a workgroup take 32
// rows together and a quarter of the keys each (mla_prefill_few_kernel).
#include "mla_device.h"
#include "mla_launch.h"

namespace mxfp4 {
namespace {

constexpr int kTile = 32, kWaves = 4;

// LDS of one stage: the keys' first 128 values (256-byte rows), the next 64
// (DN = 192; 128-byte rows), the rotated 64, then the values (DV * 2-byte rows).
template <int DN, int DV>
struct Stage {
  static constexpr uint32_t kB = kTile * 256;                       // second part of the keys
  static constexpr uint32_t kPe = kB + (DN > 128 ? kTile * 128 : 0);
  static constexpr uint32_t kV = kPe + kTile * 128;
  static constexpr uint32_t kBytes = kV + kTile * DV * 2;
  static constexpr int kLoads = kBytes / 1024;                      // wave loads of a tile
};

template <int DN, int DV, int NS>
struct Cfg {
  using St = Stage<DN, DV>;
  static constexpr int kPer = St::kLoads / kWaves;
  static_assert(NS == 2 || NS == 4, "the kernel's waits");
  static_assert(St::kLoads % kWaves == 0, "equal loads per wave");
  static constexpr uint32_t kLds = NS * St::kBytes;
  static_assert(kLds <= 80 * 1024, "two workgroups a compute unit");
};

// The rows of sequence b.  Offsets are clamped to the packed tensors: bad ones
// cannot leave them, as long as every use of the offsets goes through here (a
// block counted from the offsets themselves can lie at rows below 0, where the
// products of wild ones wrap).
struct Span {
  int64_t q0, k0;
  int nq, nk;
  __device__ __forceinline__ Span(const MlaPrefillArgs& a, int b) {
    q0 = max((int64_t)0, min(a.Tq, (int64_t)a.cu_q[b]));
    k0 = max((int64_t)0, min(a.Tk, (int64_t)a.cu_k[b]));
    nq = (int)(max(q0, min(a.Tq, (int64_t)a.cu_q[b + 1])) - q0);
    nk = (int)(max(k0, min(a.Tk, (int64_t)a.cu_k[b + 1])) - k0);
  }
};

// Query block `blk` of R rows, counted by the keys it sees from the most down
// (whatever sequence it is of: where all blocks run at once, long and short
// ones then share the compute units; the chunks above 0.67 -> 0.63 ms), 64
// sequences at a time: its sequence and its number there; false past the end.
// A block's level is its keys' end in units of R: per sequence the blocks of a
// level and above are counted without a list, so the level that holds `blk` is
// found by bisection, one sequence a lane.
template <int R>
__device__ __forceinline__ bool find_block(const MlaPrefillArgs& a, int blk, int& b, int& i) {
  const int lane = threadIdx.x & 63;
  for (int s = 0; s < a.B; s += 64) {
    const int k = s + lane;
    int n = 0, first = 0;  // blocks, and the level of the first (causal) or of all
    if (k < a.B) {
      const Span rows(a, k);
      n = (rows.nq + R - 1) / R;
      first = (a.causal ? rows.nk - rows.nq : rows.nk) >> __builtin_ctz(R);
    }
    const int total = wave_sum(n);
    if (blk >= total) {
      blk -= total;
      continue;
    }
    if (a.B == 1) {
      b = 0;
      i = total - 1 - blk;
      return true;
    }
    auto from = [&](int level) {  // the lane's blocks at `level` or above
      return a.causal ? max(0, min(n, n + first - level)) : level <= first ? n : 0;
    };
    int lo = wave_reduce(n ? first : 0x7FFFFFFF, [](int x, int y) { return min(x, y); });
    int hi = wave_reduce(n ? first + (a.causal ? n : 1) : -0x7FFFFFFF, [](int x, int y) { return max(x, y); });
    while (hi - lo > 1) {  // blocks from lo: more than blk; from hi: no more
      const int mid = lo + (hi - lo) / 2;
      if (wave_sum(from(mid)) > blk) lo = mid;
      else hi = mid;
    }
    const int above = from(hi), here = from(lo) - above, rank = blk - wave_sum(above);
    int x = here;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(x, d);
      if (lane >= d) x += y;
    }
    const int f = __builtin_ctzll(__builtin_amdgcn_ballot_w64(x > rank));
    b = s + f;
    i = __builtin_amdgcn_readlane(n - 1 - above, f) - (rank - __builtin_amdgcn_readlane(x - here, f));
    return true;
  }
  return false;
}

// A row's outputs: columns 32 i + 8 j + 4 (lane / 32) + (0..3) are 4 j.. of
// the lane's accumulator of column tile i.
__device__ __forceinline__ void store_columns(uint16_t* out, uint32_t lane, int i, int j, v4f o, float inv) {
  const uint2 w = {pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv)};
  *(uint2*)(out + 32 * i + 8 * j + 4 * (lane >> 5)) = w;
}

// A wave's work on one tile of keys in LDS, for its 32 query rows: scores,
// softmax step, values.  G: LDS operands read ahead.
template <int DN, int DV, int G>
struct Tile {
  using St = Stage<DN, DV>;
  static constexpr int kSteps = (DN + kRope) / 16, kCols = DV / 32;
  // Lane addresses within a stage.  Rows start at multiples of their length,
  // so a step's chunk is one XOR away and its row group an immediate offset.
  uint32_t lane, ka, kb, va;
  __device__ __forceinline__ explicit Tile(uint32_t lane) : lane(lane) {
    const uint32_t kr = lane & 31, hh = lane >> 5, i16 = lane & 15, vr = 4 * hh + (i16 >> 2);
    ka = kr * 256 + ((hh ^ bitrev4(kr & 15)) << 4);
    kb = St::kB + kr * 128 + ((hh ^ ((kr >> 1) & 7)) << 4);
    va = St::kV + vr * (DV * 2) + (i16 & 1) * 8 +
         (((2 * ((lane >> 4) & 1) + ((i16 & 3) >> 1)) ^ bitrev4(vr)) << 4);
  }
  // `at`: the tile in LDS; `key`: its first key; `seen`: keys the lane's row
  // sees; `masked`: some row of the wave does not see all of the tile;
  // `scored()` runs between the last read of the keys and the first of the values.
  template <typename Scored>
  __device__ __forceinline__ void attend(uint32_t at, int key, const v8bf (&q)[kSteps], v16f (&o)[kCols], float& m,
                                         RowSums& l, float c, int seen, bool masked, Scored scored) const {
    // (opaque, so that the steps' addresses are computed here and not kept)
    uint32_t ta = ka + at, tb = kb + at, tv = va + at;
    asm volatile("" : "+v"(ta), "+v"(tb), "+v"(tv));
    auto key_frag = [&](int k) {
      if (k < 8) return lds_read16(ta ^ ((2 * k) << 4));
      const int i = k < DN / 16 ? k - 8 : k - DN / 16;
      return lds_read16((tb ^ ((2 * i) << 4)) + (k < DN / 16 ? 0 : St::kPe - St::kB));
    };
    v8bf first[G];
    read_group(first, key_frag);
    v16f s = {};
    pipeline<kSteps, G>(first, key_frag, [&](int k, v8bf f) { s = mfma_rows(f, q[k], s); });
    scored();
    // Step i of the values: column tile i / 2 over keys 0-15 or 16-31.
    auto value_frag = [&](int i) {
      const int ct = i >> 1;
      const uint32_t c0 = ((4 * ct) & 15) << 4, c1 = (ct >> 2) * 256 + (i & 1) * 16 * DV * 2;
      return join_keys(lds_read_tr((tv ^ c0) + c1), lds_read_tr((tv ^ (c0 | 16)) + c1 + 8 * DV * 2));
    };
    read_group(first, value_frag);
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = s[i];
    if (masked) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (key + key_of<32>(i, lane) >= seen) x[i] = kNegInf;
    }
    float alpha;
    v8bf p[2];
    if (softmax_step<32, 16>(x, c, m, l, alpha, p)) {
#pragma unroll
      for (int i = 0; i < kCols; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] *= alpha;
    }
    pipeline<2 * kCols, G>(first, value_frag, [&](int i, v8bf f) { o[i >> 1] = mfma_rows(f, p[i & 1], o[i >> 1]); });
  }
};

template <int DN, int DV, int NS>
__global__ __launch_bounds__(64 * kWaves, 2) void mla_prefill_kernel(MlaPrefillArgs a) {
  using St = Stage<DN, DV>;
  using C = Cfg<DN, DV, NS>;
  constexpr int R = 32 * kWaves, kSteps = (DN + kRope) / 16, kCols = DV / 32;
  __shared__ int4 lds_raw[C::kLds / 16];
  uint32_t anchor = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int4*)lds_raw;
  asm volatile("" : "+s"(anchor)::"memory");  // LDS is addressed by number: its array starts at 0

  const uint32_t lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = blockIdx.x % a.H;
  int b, blk;
  if (!find_block<R>(a, blockIdx.x / a.H, b, blk)) return;
  b = __builtin_amdgcn_readfirstlane(b);
  blk = __builtin_amdgcn_readfirstlane(blk);
  const auto [q0, k0, nq, nk] = Span(a, b);
  const int r0 = blk * R;                      // first query row of the block
  if (r0 >= nq) return;
  const int wr0 = r0 + wv * 32;                // of the wave
  const int row = wr0 + (int)(lane & 31);
  const int past = a.causal ? nk - nq + 1 : nk;  // keys the first query sees
  auto sees = [&](int r) { return a.causal ? min(nk, past + r) : nk; };
  const int seen = sees(row), seen_first = sees(wr0), seen_wave = sees(min(wr0 + 31, nq - 1));
  const int nt = (max(0, sees(min(r0 + R, nq) - 1)) + kTile - 1) / kTile;
  const int wave_tiles = wr0 < nq ? (max(0, seen_wave) + kTile - 1) / kTile : 0;

  v8bf q[kSteps];
  {
    const uint16_t* p = a.q + (q0 + min(row, nq - 1)) * a.sqt + h * a.sqh + 8 * (lane >> 5);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) q[k] = __builtin_bit_cast(v8bf, *(const int4*)(p + k * 16));
  }
  v16f o[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[i][j] = 0;
  float m = kNegInf;
  RowSums l;

  // This wave's loads of a tile, 1 KiB each: a running base (the tile's
  // first row), its step per tile, and the lane's offset, which names a row
  // and the row's permuted chunk.  All of it is fixed before the loop.
  const char* base[C::kPer];
  int64_t step[C::kPer];
  uint32_t off[C::kPer], pitch[C::kPer];
  int first_row[C::kPer], shift[C::kPer];
#pragma unroll
  for (int i = 0; i < C::kPer; ++i) {
    const uint32_t at = (wv * C::kPer + i) * 1024;
    const bool second = DN > 128 && at >= St::kB && at < St::kPe;
    if (at < St::kPe) base[i] = (const char*)(a.k + k0 * a.skt + h * a.skh + (second ? 128 : 0));
    else if (at < St::kV) base[i] = (const char*)(a.k_pe + k0 * a.spt);
    else base[i] = (const char*)(a.v + k0 * a.svt + h * a.svh);
    pitch[i] = (uint32_t)(at < St::kPe ? a.skt : at < St::kV ? a.spt : a.svt) * 2;
    step[i] = (int64_t)kTile * pitch[i];
    shift[i] = at < St::kB ? 4 : at < St::kV ? 3 : DV == 256 ? 5 : 4;      // log2 of a row's chunks
    first_row[i] = (int)((at - (at < St::kB ? 0 : second ? St::kB : at < St::kV ? St::kPe : St::kV)) >> (shift[i] + 4));
    const uint32_t r = first_row[i] + (lane >> shift[i]), ch = lane & ((1u << shift[i]) - 1);
    off[i] = r * pitch[i] + ((ch ^ (shift[i] == 3 ? (r >> 1) & 7 : bitrev4(r & 15))) << 4);
  }
  auto issue = [&](int t, uint32_t lds) {
    const int left = nk - t * kTile;  // rows of the tile that exist
#pragma unroll
    for (int i = 0; i < C::kPer; ++i) {
      uint32_t o = off[i];
      if (left < kTile) {             // past them the last row is loaded again
        const int over = first_row[i] + (int)(lane >> shift[i]) - (left - 1);
        o -= (over > 0 ? over : 0) * pitch[i];
      }
      dma16(lds + (wv * C::kPer + i) * 1024, base[i], o);
      base[i] += step[i];
    }
  };

#pragma unroll
  for (int t = 0; t < NS - 1; ++t)
    if (t < nt) issue(t, t * St::kBytes);
  const Tile<DN, DV, DV == 256 ? 2 : 4> at_tile(lane);  // (groups: what the registers leave)
  uint32_t tile = 0, fill = (NS - 1) * St::kBytes;  // this tile's stage, and the next to load
  for (int t = 0; t < nt; ++t) {
    if (NS == 4 && t + 2 < nt) wait_loads<2 * C::kPer>();  // tile t is there, the next may be under way
    else if (NS == 4 && t + 1 < nt) wait_loads<C::kPer>();
    else wait_loads<0>();
    wait_lds();
    wave_barrier();
    if (t + NS - 1 < nt) issue(t + NS - 1, fill);
    const uint32_t at = tile;
    fill = tile;
    tile = tile + St::kBytes == NS * St::kBytes ? 0 : tile + St::kBytes;
    if (t >= wave_tiles) continue;

    at_tile.attend(at, t * kTile, q, o, m, l, a.c, seen, (t + 1) * kTile > seen_first, [] {});
  }

  l.exact = rows_sum<32>(l.exact);
  l.used = rows_sum<32>(l.used);
  if (row >= nq) return;
  const float inv = l.inverse();  // (a row that sees no key: 0 and -inf)
  uint16_t* out = a.out + (q0 + row) * a.sot + h * a.soh;
#pragma unroll
  for (int i = 0; i < kCols; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      store_columns(out, lane, i, j, v4f{o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]}, inv);
  if (a.lse && lane < 32)
    a.lse[(q0 + row) * a.H + h] = l.log_sum_exp(m);
}

// The same for few query rows: a workgroup takes 32 of them, its four waves
// walk every fourth tile of their keys, each through a ring of LDS stages of
// its own (no barriers), and join their sums at the end, in the waves' order.
template <int DN, int DV, int NS>
__global__ __launch_bounds__(256, 1) void mla_prefill_few_kernel(MlaPrefillArgs a) {
  using St = Stage<DN, DV>;
  constexpr int kSteps = (DN + kRope) / 16, kCols = DV / 32, kMine = kCols / 4;
  constexpr uint32_t kSums = 4 * 32 * DV * 4;  // after the waves' outputs: maxima, sums
  constexpr uint32_t kLds = 4 * NS * St::kBytes > kSums + 4 * 64 * 16 ? 4 * NS * St::kBytes : kSums + 4 * 64 * 16;
  static_assert(kLds <= 160 * 1024, "LDS per workgroup");
  __shared__ int4 lds_raw[kLds / 16];
  uint32_t anchor = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int4*)lds_raw;
  asm volatile("" : "+s"(anchor)::"memory");  // LDS is addressed by number: its array starts at 0

  const uint32_t lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = blockIdx.x % a.H;
  int b, blk;
  if (!find_block<32>(a, blockIdx.x / a.H, b, blk)) return;
  b = __builtin_amdgcn_readfirstlane(b);
  blk = __builtin_amdgcn_readfirstlane(blk);
  const auto [q0, k0, nq, nk] = Span(a, b);
  const int r0 = blk * 32;
  if (r0 >= nq) return;
  const int row = r0 + (int)(lane & 31);
  const int past = a.causal ? nk - nq + 1 : nk;
  auto sees = [&](int r) { return a.causal ? min(nk, past + r) : nk; };
  const int seen = sees(row), seen_first = sees(r0);
  const int nt = (max(0, sees(min(r0 + 32, nq) - 1)) + kTile - 1) / kTile;

  // A tile's loads, 1 KiB each: a part's base (the tile's first row) and the
  // lane's offset, which names a row and the row's permuted chunk.
  const char* base[3] = {(const char*)(a.k + k0 * a.skt + h * a.skh), (const char*)(a.k_pe + k0 * a.spt),
                         (const char*)(a.v + k0 * a.svt + h * a.svh)};
  const uint32_t pitch[3] = {(uint32_t)a.skt * 2, (uint32_t)a.spt * 2, (uint32_t)a.svt * 2};
  constexpr int kKeyLoads = St::kV / 1024, kValueLoads = St::kLoads - kKeyLoads;
  auto issue = [&](int t, uint32_t lds, auto values) {
    const int left = nk - t * kTile;  // rows of the tile that exist: past them the last one is loaded again
    const char* tile[3];
#pragma unroll
    for (int p = 0; p < 3; ++p) tile[p] = base[p] + (int64_t)t * kTile * pitch[p];
#pragma unroll
    for (int i = values ? kKeyLoads : 0; i < (values ? St::kLoads : kKeyLoads); ++i) {
      const uint32_t at = i * 1024;
      const bool second = DN > 128 && at >= St::kB && at < St::kPe;
      const int part = at < St::kPe ? 0 : at < St::kV ? 1 : 2;
      const int shift = at < St::kB ? 4 : at < St::kV ? 3 : DV == 256 ? 5 : 4;  // log2 of a row's chunks
      const uint32_t start = at < St::kB ? 0 : second ? St::kB : at < St::kV ? St::kPe : St::kV;
      const uint32_t r = ((at - start) >> (shift + 4)) + (lane >> shift), ch = lane & ((1u << shift) - 1);
      const uint32_t o = (uint32_t)min((int)r, left - 1) * pitch[part] + (second ? 256 : 0) +
                         ((ch ^ (shift == 3 ? (r >> 1) & 7 : bitrev4(r & 15))) << 4);
      dma16(lds + at, tile[part], o);
    }
  };
  const uint32_t ring = wv * NS * St::kBytes;
#pragma unroll
  for (int i = 0; i < NS; ++i)
    if (wv + 4 * i < nt) {
      issue(wv + 4 * i, ring + i * St::kBytes, std::false_type{});
      issue(wv + 4 * i, ring + i * St::kBytes, std::true_type{});
    }

  v8bf q[kSteps];
  {
    const uint16_t* p = a.q + (q0 + min(row, nq - 1)) * a.sqt + h * a.sqh + 8 * (lane >> 5);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) q[k] = __builtin_bit_cast(v8bf, *(const int4*)(p + k * 16));
  }
  v16f o[kCols] = {};
  float m = kNegInf;
  RowSums l;
  const Tile<DN, DV, 4> at_tile(lane);
  uint32_t at = ring;
  for (int t = wv; t < nt; t += 4) {
    // A tile's keys and values are waited for apart, and each part of the
    // stage is filled again once it is read.
    const bool next = NS == 2 && t + 4 < nt, refill = t + 4 * NS < nt;
    if (next) wait_loads<kValueLoads + St::kLoads>();
    else wait_loads<kValueLoads>();
    at_tile.attend(at, t * kTile, q, o, m, l, a.c, seen, (t + 1) * kTile > seen_first, [&] {
      wait_lds();
      if (refill) {
        issue(t + 4 * NS, at, std::false_type{});
        wait_loads<(NS - 1) * St::kLoads + kKeyLoads>();
      } else if (next) {
        wait_loads<St::kLoads>();
      } else {
        wait_loads<0>();
      }
    });
    wait_lds();
    if (refill) issue(t + 4 * NS, at, std::true_type{});
    at = at + St::kBytes == ring + NS * St::kBytes ? ring : at + St::kBytes;
  }

  lds_barrier();  // the stages become the waves' outputs
  float4* const sums = (float4*)((char*)lds_raw + kSums);
  float4* const parts = (float4*)lds_raw;
  sums[wv * 64 + lane] = {m, rows_sum<32>(l.exact), rows_sum<32>(l.used), 0};
#pragma unroll
  for (int i = 0; i < kCols; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      parts[((wv * kCols + i) * 4 + j) * 64 + lane] = {o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]};
  lds_barrier();
  float4 w[4];
  float top = kNegInf, f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = sums[i * 64 + lane];
    top = fmaxf(top, w[i].x);
  }
  RowSums all;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = w[i].x == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(w[i].x - top);
    all.exact += f[i] * w[i].y;
    all.used += f[i] * w[i].z;
  }
  if (row >= nq) return;
  const float inv = all.inverse();  // (a row that sees no key: 0 and -inf)
  uint16_t* out = a.out + (q0 + row) * a.sot + h * a.soh;
#pragma unroll
  for (int i = 0; i < kMine; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v4f sum = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 x = parts[((k * kCols + wv * kMine + i) * 4 + j) * 64 + lane];
        sum += v4f{x.x, x.y, x.z, x.w} * f[k];
      }
      store_columns(out, lane, wv * kMine + i, j, sum, inv);
    }
  if (a.lse && wv == 0 && lane < 32) a.lse[(q0 + row) * a.H + h] = all.log_sum_exp(top);
}

}  // namespace

hipError_t launch_mla_prefill(const MlaPrefillArgs& p, int dn, int dv, int rows, int cus, hipStream_t stream) {
  // at most one part-filled block per sequence
  auto blocks = [&](int rows) { return (p.Tq / rows + (p.Tq < p.B ? p.Tq : p.B)) * p.H; };
  auto grid = [&](int rows) { return dim3((unsigned)blocks(rows)); };
  // The waves share 32 rows' keys where one workgroup per compute unit, or
  // two with keys enough to share, take all rows (16 heads, us, shared keys
  // against shared rows: 333 tokens 9.3, 14.5; 1000 22, 34; 32 after 4000
  // others 42, 114; but 8 x 333 40, 22 and one of 20 5.7, 5.3).
  const int64_t mean_rows = p.B ? (p.Tq + p.B - 1) / p.B : 0, mean_keys = p.B ? p.Tk / p.B : 0;
  const int64_t few_blocks = p.B * ((mean_rows + 31) / 32) * p.H;
  const bool few = rows ? rows == 32 : few_blocks <= cus * (mean_keys >= 256 ? 2 : mean_keys > kTile ? 1 : 0);
  if (few && dn == 192) mla_prefill_few_kernel<192, 256, 1><<<grid(32), 256, 0, stream>>>(p);
  else if (few) mla_prefill_few_kernel<128, 128, 2><<<grid(32), 256, 0, stream>>>(p);
  else if (dn == 192) mla_prefill_kernel<192, 256, 2><<<grid(128), 256, 0, stream>>>(p);
  else mla_prefill_kernel<128, 128, 4><<<grid(128), 256, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace mxfp4
