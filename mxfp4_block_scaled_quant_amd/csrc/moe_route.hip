// Routing to experts: scores, choice by group and score, renormalised
// weights (gfx950).
//
// Per token, over its E logits x (one that is NaN or -inf, or whose bias is,
// is not available; +inf counts as the largest finite value):
//   s = softmax(x) over the available, or 1 / (1 + exp(-x));  c = s + bias
//   group g = experts [g E/G, (g+1) E/G): its score is its largest available
//   c, or the sum of its two largest; the best `kept` groups stay
//   the best top_k by (c, x), equal ones by index; w = s (/ their sum) * scale
//
// L lanes hold one token's experts, V consecutive ones each, in registers:
// one read of the logits, and every step of the choice is a few lane
// permutations (DPP within 16 lanes) of a register value.  Each of the top_k
// rounds finds the largest value left, then the lowest index that holds it,
// and takes it out.
//
// The choice is that of 64-bit scores.  Without a bias (or with the same one
// everywhere) the order of a token's scores is the logits' own, and they are
// compared instead.  With one, fp32 scores decide wherever the values they
// compare differ by more than twice their error (the margins below); where
// one comparison of a wave's tokens does not, the wave chooses again in 64
// bits.
#include <float.h>

#include <type_traits>

#include "moe_launch.h"
#include "mxfp4_device.h"

namespace mxfp4 {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// Bounds of the difference of two fp32 scores c from that of the exact ones:
// base + |c| * kMarginRel (c = s + bias is rounded once: 2^-24 |c| each).
// A sigmoid's exponent is off by |x| 2^-23 relative, its power by an ulp,
// the quotient by two: s (1 - s) (|x| + 2) 2^-23 + 3 * 2^-24 < 2^-21.5 each.
// A softmax term is off by (|x - max| 2 + 2) 2^-23 relative, its sum by the
// terms' error and one rounding per addition (at most 16 + 6): < 2.1e-6 of
// s <= 1 each.
// A group's score a + c of two terms is off by as much in all where each counts
// with its own magnitude: base covers the two s, kMarginRel (|a| + |c|) both
// terms' rounding, the sum's and that of the bounds below, 2^-24 each.  (|a + c|
// in place of |a| + |c| would not do: the roundings stay where terms of large
// biases of both signs cancel.)
constexpr float kMarginSigmoid = 1.0e-6f;
constexpr float kMarginSoftmax = 5.0e-6f;
constexpr float kMarginRel = 2.5e-7f;

template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(int, v)));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  int w[2];
  __builtin_memcpy(w, &v, 8);
  w[0] = dpp<CTRL>(w[0]);
  w[1] = dpp<CTRL>(w[1]);
  __builtin_memcpy(&v, w, 8);
  return v;
}

// The lane that step S of a reduction over 2^S neighbours pairs this one
// with: lane ^ 1, lane ^ 2, then the mirror image in 8 and in 16 lanes (as
// good as ^ 4 and ^ 8 once the lanes of a half agree), lane ^ 16, lane ^ 32.
template <int S, typename T>
__device__ __forceinline__ T partner(T v) {
  if constexpr (S == 0) return dpp<0xB1>(v);
  if constexpr (S == 1) return dpp<0x4E>(v);
  if constexpr (S == 2) return dpp<0x141>(v);
  if constexpr (S == 3) return dpp<0x140>(v);
  if constexpr (S == 4) return __shfl_xor(v, 16);
  if constexpr (S == 5) return __shfl_xor(v, 32);
}

constexpr int log2of(int n) { return n <= 1 ? 0 : 1 + log2of(n / 2); }

// Reductions over the L lanes of a token; every lane has the result.
template <int L, int S = 0, typename T>
__device__ __forceinline__ T all_max(T v) {
  if constexpr (S == log2of(L)) return v;
  else {
    const T o = partner<S>(v);
    return all_max<L, S + 1>(o > v ? o : v);
  }
}
template <int L, int S = 0, typename T>
__device__ __forceinline__ T all_min(T v) {
  if constexpr (S == log2of(L)) return v;
  else {
    const T o = partner<S>(v);
    return all_min<L, S + 1>(o < v ? o : v);
  }
}
template <int L, int S = 0, typename T>
__device__ __forceinline__ T all_sum(T v) {
  if constexpr (S == log2of(L)) return v;
  else return all_sum<L, S + 1>(v + partner<S>(v));
}

// The two largest of two pairs (a >= b).
template <typename F>
__device__ __forceinline__ void merge2(F& a, F& b, F oa, F ob) {
  const F lo = a < oa ? a : oa;
  const F hb = b > ob ? b : ob;
  a = a > oa ? a : oa;
  b = lo > hb ? lo : hb;
}
// ... over the 2^n lanes that share a group (n uniform).
template <int L, int S = 0, typename F>
__device__ __forceinline__ void merge_lanes(F& a, F& b, int n) {
  if constexpr (S < log2of(L)) {
    if (S < n) {
      const F oa = partner<S>(a), ob = partner<S>(b);
      merge2(a, b, oa, ob);
      merge_lanes<L, S + 1>(a, b, n);
    }
  }
}

__device__ __forceinline__ float exp_of(float v) { return __builtin_amdgcn_exp2f(v * kLog2e); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }
__device__ __forceinline__ float quotient(float a, float b) { return a * __builtin_amdgcn_rcpf(b); }
__device__ __forceinline__ double quotient(double a, double b) { return a / b; }

template <typename F>
struct Lowest;
template <>
struct Lowest<float> {
  static constexpr float v = -__builtin_huge_valf();
};
template <>
struct Lowest<double> {
  static constexpr double v = -__builtin_huge_val();
};

// A group's score in fp32 (-inf for a group without an available expert), and
// what the exact one lies between.  a, c: its largest two (c = -inf: one term).
// Sums past fp32 count as its largest number of that sign in `mine`, and leave
// the bound on their far side infinite.
struct GroupScore {
  float mine, low, high;
};
__device__ __forceinline__ GroupScore group_score(float a, float c, int group_top, float base) {
  constexpr float kLow = -__builtin_huge_valf();
  const bool two = group_top == 2 && c > kLow;
  const float sum = two ? a + c : a;
  const float off = base + kMarginRel * fabsf(a) + (two ? kMarginRel * fabsf(c) : 0.f);
  GroupScore g;
  const bool open = a > kLow;
  g.mine = open ? fmaxf(sum, -FLT_MAX) : kLow;
  g.low = open ? fminf(sum, FLT_MAX) - off : kLow;
  g.high = open ? fmaxf(sum, -FLT_MAX) + off : kLow;
  return g;
}

// What the choice needs of the call, the same in every lane.
struct Choice {
  int experts, top_k, groups, kept, group_top;
  int size;          // experts of a group
  int lanes2;        // log2 of the lanes that hold one group, -1: groups do not fill whole lanes
  bool by_logit;     // the logits' order is the scores'
};

// The choice for one token in precision F.  x: the lane's logits (-inf where
// not available), b: their biases.  Returns the expert of round `lane`
// (lane < top_k; -1: none left); `unsure` is set where a comparison was
// closer than fp32 can tell (F = float only).
template <int L, int V, bool SIGMOID, typename F>
__device__ __forceinline__ int choose(const Choice& p, const float (&x)[V], const float (&b)[V], int lane,
                                      bool& unsure) {
  constexpr F kLow = Lowest<F>::v;
  constexpr bool kFast = sizeof(F) == 4;
  constexpr float kBase = SIGMOID ? kMarginSigmoid : kMarginSoftmax;
  F key[V];
  const bool grouped = p.groups > 1;  // groups are compared by their scores
  if (!p.by_logit || grouped) {
    if constexpr (SIGMOID) {
#pragma unroll
      for (int r = 0; r < V; ++r) key[r] = quotient((F)1, (F)1 + exp_of(-(F)x[r]));
    } else {
      float m = x[0];
#pragma unroll
      for (int r = 1; r < V; ++r) m = fmaxf(m, x[r]);
      m = all_max<L>(m);
      F z = 0;
#pragma unroll
      for (int r = 0; r < V; ++r) {
        key[r] = x[r] > -__builtin_huge_valf() ? exp_of((F)x[r] - (F)m) : (F)0;
        z += key[r];
      }
      z = all_sum<L>(z);
      const F inv = quotient((F)1, z);
#pragma unroll
      for (int r = 0; r < V; ++r) key[r] *= inv;
    }
#pragma unroll
    for (int r = 0; r < V; ++r) key[r] = x[r] > -__builtin_huge_valf() ? key[r] + (F)b[r] : kLow;
  } else {
#pragma unroll
    for (int r = 0; r < V; ++r) key[r] = (F)x[r];
  }

  if (p.groups > 1) {
    // every lane g < groups gets group g's score
    F mine = kLow;
    float low = -__builtin_huge_valf(), high = low;
    const auto score_of = [&](F a, F c) {
      if constexpr (kFast) {
        const GroupScore g = group_score(a, c, p.group_top, kBase);
        mine = g.mine, low = g.low, high = g.high;
      } else {
        mine = (p.group_top == 2 && c > kLow) ? a + c : a;
      }
    };
    if (p.lanes2 >= 0) {
      F a = kLow, c = kLow;
#pragma unroll
      for (int r = 0; r < V; ++r) merge2(a, c, key[r], kLow);
      merge_lanes<L>(a, c, p.lanes2);
      score_of(a, c);
      const int from = (lane << p.lanes2) & (L - 1);
      mine = __shfl(mine, from, L);
      if constexpr (kFast) low = __shfl(low, from, L), high = __shfl(high, from, L);
    } else {
      F a1 = kLow, c1 = kLow;
      for (int g = 0; g < p.groups; ++g) {
        F a = kLow, c = kLow;
#pragma unroll
        for (int r = 0; r < V; ++r) {
          const int e = lane * V + r;
          merge2(a, c, (e >= g * p.size && e < (g + 1) * p.size) ? key[r] : kLow, kLow);
        }
        merge_lanes<L>(a, c, log2of(L));
        if (lane == g) a1 = a, c1 = c;
      }
      score_of(a1, c1);
    }
    if (lane >= p.groups) mine = kLow;
    int ahead = 0;
    for (int g = 0; g < p.groups; ++g) {
      const F other = __shfl(mine, g, L);
      ahead += (other > mine || (other == mine && g < lane)) ? 1 : 0;
    }
    const bool stays = lane < p.groups && ahead < p.kept && mine > kLow;
    if constexpr (kFast) {
      const float lo = all_min<L>(stays ? low : __builtin_huge_valf());
      const float hi = all_max<L>(!stays && mine > kLow ? high : kLow);
      if (hi > kLow && !(lo > hi)) unsure = true;
    }
    const uint64_t votes = __ballot(stays);
    const uint64_t here = votes >> ((threadIdx.x & 63) & ~(L - 1));
    int g = lane * V / p.size, at = lane * V - g * p.size;
#pragma unroll
    for (int r = 0; r < V; ++r) {
      const bool in = g < p.groups && (here >> (g & 63) & 1);
      key[r] = in ? (p.by_logit ? (F)x[r] : key[r]) : kLow;
      if (++at == p.size) at = 0, ++g;
    }
  }

  int id = -1;
  F before = kLow;
  const bool check = kFast && !p.by_logit;
  for (int j = 0; j < p.top_k + (check ? 1 : 0); ++j) {
    F best = key[0];
#pragma unroll
    for (int r = 1; r < V; ++r) best = key[r] > best ? key[r] : best;
    best = all_max<L>(best);
    if constexpr (kFast) {
      if (check && j > 0 && best > kLow && !(before - best > kBase + kMarginRel * fabsf(best))) unsure = true;
      before = best;
    }
    int at = 1 << 20;
    if constexpr (kFast) {
#pragma unroll
      for (int r = V - 1; r >= 0; --r) at = key[r] == best ? lane * V + r : at;
    } else {
      float bx = -__builtin_huge_valf();
#pragma unroll
      for (int r = 0; r < V; ++r) bx = key[r] == best ? fmaxf(bx, x[r]) : bx;
      bx = all_max<L>(bx);
#pragma unroll
      for (int r = V - 1; r >= 0; --r) at = (key[r] == best && x[r] == bx) ? lane * V + r : at;
    }
    at = all_min<L>(at);
    if (lane == j) id = best > kLow ? at : -1;
#pragma unroll
    for (int r = 0; r < V; ++r) key[r] = lane * V + r == at ? kLow : key[r];
  }
  return id;
}

// fp32 values as integers of the same order (0 and -0 equal), and back.
constexpr int kNone = (int)0x807FFFFFu;  // -inf
__device__ __forceinline__ int order_of(float v) {
  const int i = __builtin_bit_cast(int, v + 0.f);
  return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float value_of(int i) {
  return __builtin_bit_cast(float, i ^ ((i >> 31) & 0x7FFFFFFF));
}

// The largest integer of a wave, in a scalar register: shifts within rows of
// 16 lanes, then row 0 into row 1 and 2 into 3, then the lower half into the
// upper, one instruction each.
template <int CTRL, int ROWS>
__device__ __forceinline__ int max_step(int v) {
  return max(v, __builtin_amdgcn_update_dpp((int)0x80000000u, v, CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ int wave_max(int v) {
  v = max_step<0x111, 0xF>(v);
  v = max_step<0x112, 0xF>(v);
  v = max_step<0x114, 0xF>(v);
  v = max_step<0x118, 0xF>(v);
  v = max_step<0x142, 0xA>(v);
  v = max_step<0x143, 0xC>(v);
  return __builtin_amdgcn_readlane(v, 63);
}

// choose() in fp32 for a token that has a wave of its own (and whose groups,
// if any, fill whole lanes): a round's largest value is in a scalar register,
// so that one comparison and vote per register finds the lanes that hold it,
// and the rest of the round is scalar.  Lane j gets round j's
// expert.
template <int V, bool SIGMOID>
__device__ __forceinline__ int choose_wave(const Choice& p, const float (&x)[V], const float (&b)[V], int lane,
                                           bool& unsure) {
  constexpr float kLow = -__builtin_huge_valf();
  constexpr float kBase = SIGMOID ? kMarginSigmoid : kMarginSoftmax;
  float key[V];
  const bool grouped = p.groups > 1;
  if (!p.by_logit || grouped) {
    if constexpr (SIGMOID) {
#pragma unroll
      for (int r = 0; r < V; ++r) key[r] = quotient(1.f, 1.f + exp_of(-x[r]));
    } else {
      float m = x[0];
#pragma unroll
      for (int r = 1; r < V; ++r) m = fmaxf(m, x[r]);
      m = value_of(wave_max(order_of(m)));
      float z = 0.f;
#pragma unroll
      for (int r = 0; r < V; ++r) {
        key[r] = x[r] > kLow ? exp_of(x[r] - m) : 0.f;
        z += key[r];
      }
      const float inv = quotient(1.f, all_sum<64>(z));
#pragma unroll
      for (int r = 0; r < V; ++r) key[r] *= inv;
    }
#pragma unroll
    for (int r = 0; r < V; ++r) key[r] = x[r] > kLow ? key[r] + b[r] : kLow;
  } else {
#pragma unroll
    for (int r = 0; r < V; ++r) key[r] = x[r];
  }
  if (grouped) {
    float a = kLow, c = kLow;
#pragma unroll
    for (int r = 0; r < V; ++r) {
      c = fmaxf(c, fminf(a, key[r]));
      a = fmaxf(a, key[r]);
    }
    merge_lanes<64>(a, c, p.lanes2);
    const GroupScore mine = group_score(a, c, p.group_top, kBase);
    // groups ahead of this lane's: for certain, and at most (its own among
    // them); between the two fp32 cannot tell
    int certain = 0, most = 0;
    for (int g = 0; g < p.groups; ++g) {
      const auto of = [&](float v) {
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), g << p.lanes2));
      };
      certain += of(mine.low) > mine.high ? 1 : 0;
      most += !(of(mine.high) < mine.low) ? 1 : 0;
    }
    const bool in = (lane >> p.lanes2) < p.groups && mine.mine > kLow;
    const bool stays = in && most - 1 < p.kept;
    unsure = unsure || (in && !stays && certain < p.kept);
#pragma unroll
    for (int r = 0; r < V; ++r) key[r] = stays ? (p.by_logit ? x[r] : key[r]) : kLow;
  }
  int left[V], got = kNone;
#pragma unroll
  for (int r = 0; r < V; ++r) left[r] = order_of(key[r]);
  int id = -1;
  const int rounds = p.by_logit ? p.top_k : min(p.top_k + 1, 64);  // the one after the last shows how sure it is
  for (int j = 0; j < rounds; ++j) {
    int best = left[0];
#pragma unroll
    for (int r = 1; r < V; ++r) best = max(best, left[r]);
    best = wave_max(best);
    if (best <= kNone) break;
    uint64_t held[V], any = 0;
#pragma unroll
    for (int r = 0; r < V; ++r) any |= held[r] = __ballot(left[r] == best);
    const int at = __builtin_ctzll(any);
    int reg = 0;
#pragma unroll
    for (int r = V - 1; r >= 0; --r) reg = (held[r] >> at & 1) ? r : reg;
    id = lane == j ? at * V + reg : id;
    got = lane == j ? best : got;
#pragma unroll
    for (int r = 0; r < V; ++r) left[r] = (lane == at && reg == r) ? kNone : left[r];
  }
  const float value = value_of(got);
  if (!p.by_logit) {
    // round j and the next one closer than fp32 can tell
    const float next = __shfl_down(value, 1);
    if (lane < p.top_k && lane < 63 && next > kLow && !(value - next > kBase + kMarginRel * fabsf(next))) unsure = true;
    if (p.top_k == 64) unsure = true;  // (lane 64, the first that is not chosen, does not exist)
  }
  return id;
}

// One token's logits and biases in registers, V consecutive ones a lane; -inf
// for an expert that is not available.  Returns whether all biases are the
// same.
template <int L, int V, bool F32>
__device__ __forceinline__ bool load_row(const RouteArgs& p, int64_t row, int lane, float (&x)[V], float (&b)[V]) {
  constexpr float kLow = -__builtin_huge_valf();
  float lo = -kLow, hi = kLow;
#pragma unroll
  for (int r = 0; r < V; ++r) {
    const int e = lane * V + r;
    const int at = e < p.experts ? e : p.experts - 1;
    x[r] = F32 ? static_cast<const float*>(p.logits)[row + at]
               : bf16_to_f32(static_cast<const uint16_t*>(p.logits)[row + at]);
    b[r] = p.bias ? p.bias[at] : 0.f;
  }
#pragma unroll
  for (int r = 0; r < V; ++r) {
    const int e = lane * V + r;
    lo = fminf(lo, b[r]);
    hi = fmaxf(hi, b[r]);
    // false for a NaN
    const bool open = e < p.experts && x[r] > kLow && b[r] > kLow;
    x[r] = open ? fminf(x[r], FLT_MAX) : kLow;
  }
  // (every lane reads the last expert's bias at least, so lo <= hi; a NaN
  // leaves both as they are, and is the same as -inf to the choice)
  return !p.bias || !__any(lo != hi || lo != __shfl(lo, 0));
}

// The weights of the chosen experts, one a lane: s, or s over their sum.
template <int L, int V, bool SIGMOID, bool F32>
__device__ __forceinline__ void store_choice(const RouteArgs& p, int64_t token, int64_t row, bool live, int lane,
                                             int id, const float (&x)[V]) {
  constexpr float kLow = -__builtin_huge_valf();
  const bool mine = lane < p.top_k && id >= 0;
  float xi = kLow;
  if (mine)
    xi = fminf(F32 ? static_cast<const float*>(p.logits)[row + id]
                   : bf16_to_f32(static_cast<const uint16_t*>(p.logits)[row + id]),
               FLT_MAX);
  float w = 0.f;
  if (p.renormalize) {
    // s / sum s with a common factor taken out, so that small scores do not
    // vanish: exp(x) / (1 + exp(x)) below 0 (times exp(-top) where every
    // chosen logit is below 0)
    const float top = all_max<L>(xi);
    if (SIGMOID) {
      const float shift = fminf(top, 0.f);
      w = xi > 0.f ? 1.f / (1.f + expf(-xi)) : expf(xi - shift) / (1.f + expf(xi));
    } else {
      w = expf(xi - top);
    }
    if (!mine) w = 0.f;
    const float total = all_sum<L>(w);
    w = mine ? w / total * p.scale : 0.f;
  } else if (SIGMOID) {
    w = mine ? p.scale / (1.f + expf(-xi)) : 0.f;
  } else {
    float m = x[0];
#pragma unroll
    for (int r = 1; r < V; ++r) m = fmaxf(m, x[r]);
    m = all_max<L>(m);
    float z = 0.f;
#pragma unroll
    for (int r = 0; r < V; ++r) z += x[r] > kLow ? expf(x[r] - m) : 0.f;
    z = all_sum<L>(z);
    w = mine ? expf(xi - m) / z * p.scale : 0.f;
  }
  if (live && lane < p.top_k) {
    p.weights[token * p.ldw + lane] = w;
    p.ids[token * p.ldi + lane] = id;
  }
}

__device__ __forceinline__ Choice choice_of(const RouteArgs& p, int lanes2, bool by_logit) {
  Choice c;
  c.experts = p.experts, c.top_k = p.top_k, c.groups = p.groups, c.kept = p.kept, c.group_top = p.group_top;
  c.size = p.experts / p.groups;
  c.lanes2 = lanes2;
  c.by_logit = by_logit;
  return c;
}

// Batcher's odd-even merge sort of V values in registers, descending: merges of
// P values, in each the exchanges over a distance of D = P, P / 2, ..., 1.
template <int V, int P = 1, int D = P>
__device__ __forceinline__ void sort_down(int (&k)[V]) {
#pragma unroll
  for (int i = D % P; i + D < V; ++i)
    if ((i - D % P) / D % 2 == 0 && i / (2 * P) == (i + D) / (2 * P)) {
      const int a = k[i], b = k[i + D];
      k[i] = max(a, b);
      k[i + D] = min(a, b);
    }
  if constexpr (D > 1)
    sort_down<V, P, D / 2>(k);
  else if constexpr (2 * P < V)
    sort_down<V, 2 * P>(k);
}

// Many tokens: 16 lanes a token, V experts each, expert 64 (r / 4) + 4 lane +
// r % 4 in register r (so that the lanes read whole lines).  Each lane sorts its
// keys once; a round then is the largest of the 16 heads (four DPP steps), and
// the lane that holds it moves its list up by one.  A key is the score's order
// with its last four bits replaced by the register; bf16 logits that decide
// by themselves keep all their bits above the expert's number.  Where two keys
// next to each other are too close for what they leave out, or two lanes
// have the same key, the wave chooses that token's experts again in 64 bits.
// 16001 tokens of 256 fp32 logits in 8 groups take 22 us, 17.4 MB at 0.8 TB/s
// (kManyTokens has the wave per token's): about half of it is vector
// instructions (1490 a wave, 4 cycles each, four waves a SIMD), the rest waits:
// the waves, all resident in one round, meet at two barriers, and the fourth
// of a wave whose token is chosen again holds up the others.
constexpr int kGone = (int)0x80000000u;
template <int V, bool SIGMOID, bool F32>
__global__ __launch_bounds__(256) void moe_route_many_kernel(RouteArgs p, int lanes2, int wave_lanes2) {
  constexpr float kLow = -__builtin_huge_valf();
  constexpr float kBase = SIGMOID ? kMarginSigmoid : kMarginSoftmax;
  __shared__ float glow[16][17], ghigh[16][17];
  __shared__ int won[16][17];
  const int lane = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const int64_t token = (int64_t)blockIdx.x * 16 + slot;
  const bool live = token < p.tokens;
  const int64_t row = (live ? token : p.tokens - 1) * p.ld;
  float x[V], b[V];
  float lo = -kLow, hi = kLow;
#pragma unroll
  for (int c = 0; c < V / 4; ++c) {
    const int e = c * 64 + lane * 4;
    const int at = e < p.experts ? e : p.experts - 4;  // (experts % 4 == 0)
    if constexpr (F32) {
      const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.logits) + row + at);
      x[c * 4] = v.x, x[c * 4 + 1] = v.y, x[c * 4 + 2] = v.z, x[c * 4 + 3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.logits) + row + at);
      x[c * 4] = __uint_as_float(v.x << 16), x[c * 4 + 1] = __uint_as_float(v.x & 0xFFFF0000u);
      x[c * 4 + 2] = __uint_as_float(v.y << 16), x[c * 4 + 3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
  }
#pragma unroll
  for (int r = 0; r < V; ++r) b[r] = 0.f;
  if (p.bias) {
#pragma unroll
    for (int r = 0; r < V; ++r) {
      const int e = r / 4 * 64 + lane * 4;
      b[r] = p.bias[(e < p.experts ? e : p.experts - 4) + r % 4];
    }
  }
#pragma unroll
  for (int r = 0; r < V; ++r) {
    lo = fminf(lo, b[r]);
    hi = fmaxf(hi, b[r]);
    const bool open = (r / 4) * 64 + lane * 4 < p.experts && x[r] > kLow && b[r] > kLow;
    x[r] = open ? fminf(x[r], FLT_MAX) : kLow;
  }
  const bool by_logit = !p.bias || !__any(lo != hi || lo != __shfl(lo, 0));
  const bool grouped = p.groups > 1;
  const bool exact = !F32 && by_logit;  // the key holds the whole logit
  float score[V];
  if (!by_logit || grouped) {
    if constexpr (SIGMOID) {
#pragma unroll
      for (int r = 0; r < V; ++r) score[r] = quotient(1.f, 1.f + exp_of(-x[r]));
    } else {
      float m = x[0];
#pragma unroll
      for (int r = 1; r < V; ++r) m = fmaxf(m, x[r]);
      m = all_max<16>(m);
      float z = 0.f;
#pragma unroll
      for (int r = 0; r < V; ++r) {
        score[r] = x[r] > kLow ? exp_of(x[r] - m) : 0.f;
        z += score[r];
      }
      const float inv = quotient(1.f, all_sum<16>(z));
#pragma unroll
      for (int r = 0; r < V; ++r) score[r] *= inv;
    }
#pragma unroll
    for (int r = 0; r < V; ++r) score[r] = x[r] > kLow ? score[r] + b[r] : kLow;
  }
  bool unsure = false;
  bool in[V / 4];
#pragma unroll
  for (int c = 0; c < V / 4; ++c) in[c] = true;
  if (grouped) {
    // 2^lanes2 lanes hold a group's experts of register quad c
    GroupScore mine[V / 4];
    const int per = 16 >> lanes2;  // groups of a quad
#pragma unroll
    for (int c = 0; c < V / 4; ++c) {
      float a = kLow, d = kLow;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        d = fmaxf(d, fminf(a, score[c * 4 + q]));
        a = fmaxf(a, score[c * 4 + q]);
      }
      merge_lanes<16>(a, d, lanes2);
      mine[c] = group_score(a, d, p.group_top, kBase);
      const int g = c * per + (lane >> lanes2);
      if ((lane & ((1 << lanes2) - 1)) == 0 && g < p.groups) glow[slot][g] = mine[c].low, ghigh[slot][g] = mine[c].high;
    }
    __syncthreads();
    int certain[V / 4] = {}, most[V / 4] = {};
    for (int g = 0; g < p.groups; ++g) {
      const float low = glow[slot][g], high = ghigh[slot][g];
#pragma unroll
      for (int c = 0; c < V / 4; ++c) {
        certain[c] += low > mine[c].high ? 1 : 0;
        most[c] += !(high < mine[c].low) ? 1 : 0;
      }
    }
#pragma unroll
    for (int c = 0; c < V / 4; ++c) {
      const bool there = c * per + (lane >> lanes2) < p.groups && mine[c].mine > kLow;
      in[c] = there && most[c] - 1 < p.kept;
      unsure = unsure || (there && !in[c] && certain[c] < p.kept);
    }
  }
  int key[V];
#pragma unroll
  for (int r = 0; r < V; ++r) {
    float v = x[r];
    if (!by_logit) v = score[r];
    int k;
    if (exact)  // (FLT_MAX stands for +inf, above every finite bf16 number)
      k = (order_of(v == FLT_MAX ? -kLow : v) & (int)0xFFFF0000u) | (0xFFFF - ((r / 4) * 64 + lane * 4 + r % 4));
    else
      k = (order_of(v) & ~15) | (15 - r);
    key[r] = v > kLow && in[r / 4] ? k : kGone;
  }
  sort_down<V>(key);
  int got = kGone;
  uint64_t twice = 0;
  for (int j = 0; j <= p.top_k; ++j) {
    const int best = all_max<16>(key[0]);
    const bool hit = key[0] == best && best != kGone;
    const uint64_t votes = __ballot(hit), any = __ballot(best != kGone);
    // more than one vote of a token: every field of 16 that has votes, less one
    twice |= votes & (votes - (0x0001000100010001ull & ((any >> 15) & 0x0001000100010001ull)));
    if (hit) won[slot][j] = exact ? 0xFFFF - (key[0] & 0xFFFF) : 15 - (key[0] & 15) + lane * 16;
    got = lane == j ? best : got;
#pragma unroll
    for (int r = 0; r + 1 < V; ++r) {
      const int kept = key[r], next = key[r + 1];  // (of two elements ?: takes an address, and the list leaves its registers)
      key[r] = hit ? next : kept;
    }
    key[V - 1] = hit ? kGone : key[V - 1];
  }
  __syncthreads();
  int id = -1;
  if (lane < p.top_k && got != kGone) {
    const int w = won[slot][lane];
    id = exact ? w : (w & 15) / 4 * 64 + (w >> 4) * 4 + (w & 3);
  }
  if (!exact) {
    const int next = __builtin_amdgcn_update_dpp(kGone, got, 0x101, 0xF, 0xF, false);  // lane + 1's
    if (lane < p.top_k && next != kGone) {
      if (by_logit) {
        unsure = unsure || (got >> 4) == (next >> 4);
      } else {
        const float v = value_of(got), n = value_of(next);
        unsure = unsure || !(v - n > kBase + (kMarginRel + 3.9e-6f) * fmaxf(fabsf(v), fabsf(n)));  // + 2^-18: the last bits
      }
    }
  }
  const uint64_t again = __ballot(unsure) | twice;
  for (int s = 0; s < 4; ++s) {
    if (!(again >> (16 * s) & 0xFFFF)) continue;
    const int64_t t0 = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 6) * 4 + s;
    const int64_t r0 = (t0 < p.tokens ? t0 : p.tokens - 1) * p.ld;
    const int wl = threadIdx.x & 63;
    float xs[V / 4], bs[V / 4];
    const bool same = load_row<64, V / 4, F32>(p, r0, wl, xs, bs);
    bool never = false;
    const int other = choose<64, V / 4, SIGMOID, double>(choice_of(p, wave_lanes2, same), xs, bs, wl, never);
    const int moved = __shfl(other, lane);
    if ((wl >> 4) == s) id = moved;
  }
  store_choice<16, V, SIGMOID, F32>(p, token, row, live, lane, id, x);
}

// A wave per token.
template <int V, bool SIGMOID, bool F32>
__global__ __launch_bounds__(256) void moe_route_wave_kernel(RouteArgs p, int lanes2) {
  const int lane = threadIdx.x & 63;
  const int64_t token = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (token >= p.tokens) return;
  const int64_t row = token * p.ld;
  float x[V], b[V];
  const bool same = load_row<64, V, F32>(p, row, lane, x, b);
  const Choice c = choice_of(p, lanes2, same);
  bool unsure = false;
  int id = choose_wave<V, SIGMOID>(c, x, b, lane, unsure);
  if (__any(unsure)) {
    bool never = false;
    id = choose<64, V, SIGMOID, double>(c, x, b, lane, never);
  }
  store_choice<64, V, SIGMOID, F32>(p, token, row, true, lane, id, x);
}

template <int L, int V, bool SIGMOID, bool F32>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteArgs p, int lanes2) {
  const int lane = threadIdx.x & (L - 1);
  const int64_t token = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  const bool live = token < p.tokens;
  const int64_t row = (live ? token : p.tokens - 1) * p.ld;

  float x[V], b[V];
  const bool same = load_row<L, V, F32>(p, row, lane, x, b);
  const Choice c = choice_of(p, lanes2, same);
  bool unsure = false;
  int id = choose<L, V, SIGMOID, float>(c, x, b, lane, unsure);
  if (__any(unsure)) {
    bool never = false;
    id = choose<L, V, SIGMOID, double>(c, x, b, lane, never);
  }
  store_choice<L, V, SIGMOID, F32>(p, token, row, live, lane, id, x);
}

// log2 of the lanes that a group of `size` experts fills, -1 if it does not
// fill whole lanes, a power of two of them.
int group_lanes(int size, int V, int L) {
  for (int n = 0; (1 << n) <= L; ++n)
    if (size == V << n) return n;
  return -1;
}

// Whether a call's rows suit moe_route_many_kernel: whole aligned quads, groups
// that fill lanes of one quad of registers, and a lane for the first expert that
// is not chosen.
bool many_fits(const RouteArgs& p, bool f32) {
  const uintptr_t a = f32 ? 15 : 7;
  if (p.experts % 4 || p.top_k > 15 || p.groups > 16) return false;
  if (((uintptr_t)p.logits & a) || (p.tokens > 1 && p.ld % 4)) return false;
  return p.groups == 1 || group_lanes(p.experts / p.groups, 4, 16) >= 0;
}

#define MOE_ROUTE(KERNEL, GRID, ...)                                              \
  if (sigmoid && f32)                                                               \
    KERNEL<__VA_ARGS__, true, true><<<GRID, 256, 0, stream>>>(p, lanes2);           \
  else if (sigmoid)                                                                 \
    KERNEL<__VA_ARGS__, true, false><<<GRID, 256, 0, stream>>>(p, lanes2);          \
  else if (f32)                                                                     \
    KERNEL<__VA_ARGS__, false, true><<<GRID, 256, 0, stream>>>(p, lanes2);          \
  else                                                                              \
    KERNEL<__VA_ARGS__, false, false><<<GRID, 256, 0, stream>>>(p, lanes2)

template <int L, int V>
hipError_t launch_parts(const RouteArgs& p, bool f32, bool sigmoid, hipStream_t stream) {
  const int lanes2 = group_lanes(p.experts / p.groups, V, L);
  const dim3 grid((unsigned)((p.tokens + 256 / L - 1) / (256 / L)));
  MOE_ROUTE(moe_route_kernel, grid, L, V);
  return hipGetLastError();
}

template <int V>
hipError_t launch_wave(const RouteArgs& p, bool f32, bool sigmoid, hipStream_t stream) {
  const int lanes2 = group_lanes(p.experts / p.groups, V, 64);
  if (p.groups > 1 && lanes2 < 0) return launch_parts<64, V>(p, f32, sigmoid, stream);
  const dim3 grid((unsigned)((p.tokens + 3) / 4));
  MOE_ROUTE(moe_route_wave_kernel, grid, V);
  return hipGetLastError();
}

// From here on moe_route_many_kernel, us against a wave a token (bf16 logits of
// 256 experts; fp32, sigmoid, 8 groups; fp32 logits of 128 experts):
//   4096 tokens:  6.2 |  6.0   15.9 | 13.6    6.8 |  4.8
//   8192          7.0 |  8.6   17.1 | 16.4    7.0 |  6.7
//   16001         9.5 | 14.1   21.9 | 24.6    8.2 | 10.6
//   40000        21.0 | 31.1   35.7 | 47.8   15.3 | 22.9
// Few tokens leave no second wave to hide one token's 64-bit choice behind.  Up
// to 64 experts, where moe_route_kernel has 16 lanes a token as well, it is the
// faster without groups (16001 tokens: 5.4 | 4.8, with them 9.5 | 11.1).
constexpr int64_t kManyTokens = 8192;

template <int V>
hipError_t launch_many(const RouteArgs& p, bool f32, bool sigmoid, hipStream_t stream) {
  const int size = p.experts / p.groups;
  const int lanes2 = p.groups > 1 ? group_lanes(size, 4, 16) : 0, wave2 = group_lanes(size, V / 4, 64);
  const dim3 grid((unsigned)((p.tokens + 15) / 16));
  if (sigmoid && f32)
    moe_route_many_kernel<V, true, true><<<grid, 256, 0, stream>>>(p, lanes2, wave2);
  else if (sigmoid)
    moe_route_many_kernel<V, true, false><<<grid, 256, 0, stream>>>(p, lanes2, wave2);
  else if (f32)
    moe_route_many_kernel<V, false, true><<<grid, 256, 0, stream>>>(p, lanes2, wave2);
  else
    moe_route_many_kernel<V, false, false><<<grid, 256, 0, stream>>>(p, lanes2, wave2);
  return hipGetLastError();
}

// The tokens of one launch: 64 lanes each stay below the 2^32 work items of a grid.
constexpr int64_t kLaunchTokens = 1 << 25;

hipError_t launch_tokens(const RouteArgs& p, bool f32, bool sigmoid, hipStream_t stream) {
  // Lane j keeps round j's expert and lane g group g's score, so a token has
  // at least as many lanes as either.
  const int need = p.top_k > p.groups ? p.top_k : p.groups;
  if (p.tokens >= kManyTokens && p.experts > 64 && p.experts <= 256 && many_fits(p, f32)) {
    if (p.experts <= 128) return launch_many<8>(p, f32, sigmoid, stream);
    return launch_many<16>(p, f32, sigmoid, stream);
  }
  if (need <= 16 && p.experts <= 64) return launch_parts<16, 4>(p, f32, sigmoid, stream);
  if (p.experts <= 64) return launch_wave<1>(p, f32, sigmoid, stream);
  if (p.experts <= 128) return launch_wave<2>(p, f32, sigmoid, stream);
  if (p.experts <= 256) return launch_wave<4>(p, f32, sigmoid, stream);
  if (p.experts <= 512) return launch_wave<8>(p, f32, sigmoid, stream);
  return launch_wave<16>(p, f32, sigmoid, stream);
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& p, bool f32, bool sigmoid, hipStream_t stream) {
  for (int64_t t = 0; t < p.tokens; t += kLaunchTokens) {
    RouteArgs q = p;
    q.tokens = p.tokens - t < kLaunchTokens ? p.tokens - t : kLaunchTokens;
    q.logits = static_cast<const uint8_t*>(p.logits) + t * p.ld * (f32 ? 4 : 2);
    q.weights = p.weights + t * p.ldw;
    q.ids = p.ids + t * p.ldi;
    const hipError_t e = launch_tokens(q, f32, sigmoid, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace mxfp4
