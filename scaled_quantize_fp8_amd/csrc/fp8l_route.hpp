// Routing of tokens to a mixture's experts, and the exchange of their rows.
//
// Choice.  With p[e] = softmax(z)[e] or sigmoid(z[e]) and c = p + b (b: a bias
// that balances the experts; without it c = p):
//   groups     E / G consecutive experts each; a group's score is the sum of
//              its one or two largest c; the best `kept` groups stay
//   experts    the k largest c in them, best first
// Ties go to the lowest index, and the order is that of scores held in 64
// bits (without a bias that of the logits, which is the scores' order).  An
// expert with c or z = -inf is never chosen: a slot that finds none has index
// -1 and weight 0.  A row that holds a NaN (softmax: or +inf) chooses 0 .. k-1
// with NaN weights.
//
// Weights.  w[i] = s p[idx[i]], or s p[idx[i]] / sum_j p[idx[j]].  The quotient
// is taken of scores scaled by the largest chosen one, so it stands where all
// chosen scores underflow:
//   softmax   q[i] = exp(z[i] - m) / sum,   m the largest chosen logit
//   sigmoid   n[i] = exp(min(z[i], 0) - m) / (1 + exp(-|z[i]|)), q = n / sum n,
//             m the largest chosen min(z, 0)
//
// Gradient.  With d[i] = s dw[i] and q as above (plain weights: q = p):
//   softmax, quotient   dz[i] = q[i] (d[i] - sum_j q[j] d[j])
//   sigmoid, quotient   the same times 1 - p[i]
//   sigmoid, plain      dz[i] = p[i] (1 - p[i]) d[i]
//   softmax, plain      dz[e] = (p d at the chosen) - p[e] sum_j p[j] d[j]
// All other logits get 0; the bias has no gradient.
#pragma once

#include "fp8l_values.hpp"

namespace fp8l {

constexpr int kRThreads = 256;
constexpr int kRouteMaxE = 1024, kRouteMaxK = 64;
enum { kSoftmax = 0, kSigmoid = 1 };

struct RouteArgs {
  const void* z;      // [T][E]
  const float* bias;  // [E] or null
  int32_t* idx;       // [T][k]
  float* w;           // [T][k]
  int32_t T, E, k, score, groups, kept, group_top, renorm;
  float scale;
  int32_t vec;    // a lane's experts by wide loads
  int32_t lanes;  // lanes of a group where 16 hold a row, 0: groups end inside a lane
};

// ---------------------------------------------------------------- lanes

// Lane groups of L (16 or 64) consecutive lanes hold one row.  All-reduce
// steps inside 16 lanes are DPP: xor 1, xor 2, then the mirrors of 8 and of 16
// lanes (quads, then eights are uniform by then, so these act as xor 4 and
// xor 8).  Every step adds the same two numbers in both its lanes, so all
// lanes end with the same bits: equal scores stay equal.
template <int STEP>
FP8L_DEV uint32_t lane_step(uint32_t v) {
  if constexpr (STEP == 1) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false);
  else if constexpr (STEP == 2) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false);
  else if constexpr (STEP == 4) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false);
  else if constexpr (STEP == 8) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false);
  else return (uint32_t)__shfl_xor((int)v, STEP);
}
template <int STEP>
FP8L_DEV float lane_step(float v) { return __uint_as_float(lane_step<STEP>(__float_as_uint(v))); }
template <int STEP>
FP8L_DEV int lane_step(int v) { return (int)lane_step<STEP>((uint32_t)v); }
template <int STEP>
FP8L_DEV double lane_step(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint64_t lo = lane_step<STEP>((uint32_t)u), hi = lane_step<STEP>((uint32_t)(u >> 32));
  return __longlong_as_double((long long)(lo | (hi << 32)));
}
// f(step tag) for steps 1, 2, .. L / 2
template <int L, int STEP = 1, class F>
FP8L_DEV void lane_steps(F&& f) {
  if constexpr (STEP < L) {
    f(std::integral_constant<int, STEP>{});
    lane_steps<L, 2 * STEP>(f);
  }
}
template <int L>
FP8L_DEV float lanes_max(float v) {
  lane_steps<L>([&](auto s) { v = fmaxf(v, lane_step<decltype(s)::value>(v)); });
  return v;
}
template <int L, class S>
FP8L_DEV S lanes_sum(S v) {
  lane_steps<L>([&](auto s) { v += lane_step<decltype(s)::value>(v); });
  return v;
}
template <int L>
FP8L_DEV bool lanes_any(bool b) {
  const uint64_t m = __ballot(b);
  if constexpr (L == 64) return m != 0;
  return (m >> (threadIdx.x & 63 & ~(L - 1)) & ((1ull << (L & 63)) - 1)) != 0;
}

// LDS written by lanes of this wave, before lanes of it read (a wave's LDS
// accesses run in order; this keeps the compiler from moving them).
FP8L_DEV void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Largest of the row's values c[V] (lane l holds indices l V ..), the lowest
// index on a tie; its index in `at` (unspecified where all are -inf).
template <int L, int V, class S>
FP8L_DEV S row_best(const S (&c)[V], int sl, int& at) {
  S best = c[0];
  at = sl * V;
#pragma unroll
  for (int v = 1; v < V; ++v)
    if (c[v] > best) best = c[v], at = sl * V + v;
  lane_steps<L>([&](auto s) {
    const S o = lane_step<decltype(s)::value>(best);
    const int oa = lane_step<decltype(s)::value>(at);
    if (o > best || (o == best && oa < at)) best = o, at = oa;
  });
  return best;
}

template <int V, class S>
FP8L_DEV void strike(S (&c)[V], int sl, int at) {
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (at == sl * V + v) c[v] = -(S)INFINITY;
}

// LDS of one row: its scores, then the marks of the kept groups.
template <int L, int V, class S>
constexpr int group_lds() { return L * V * ((int)sizeof(S) + 1); }

// c of the experts in groups that are not kept becomes -inf.  g: the values
// that the groups are scored by.  Any groups: a lane reads a group's values
// from LDS.  The smallest score of a kept group and the largest of the others.
template <int L, int V, class S>
FP8L_DEV void keep_groups(const RouteArgs& a, S (&c)[V], const S (&g)[V], int sl, uint8_t* row,
                          S& least, S& best) {
  S* const sc = reinterpret_cast<S*>(row);
  uint8_t* const mark = row + L * V * sizeof(S);
  const int n = a.E / a.groups;
#pragma unroll
  for (int v = 0; v < V; ++v) sc[sl * V + v] = g[v];
  wave_fence();
  S gs[V], left[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {  // neighbouring lanes take neighbouring groups
    if (v * L >= a.groups) break;
    const int q = v * L + sl;
    if (q >= a.groups) continue;
    S hi = -(S)INFINITY, lo = -(S)INFINITY;
#pragma unroll 4
    for (int i = q * n; i < q * n + n; ++i) {
      const S x = sc[i];
      lo = max(lo, min(hi, x));
      hi = max(hi, x);
    }
    gs[v] = a.group_top == 2 && lo > -(S)INFINITY ? hi + lo : hi;
  }
  wave_fence();
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (v * L + sl < a.groups) sc[v * L + sl] = gs[v];
  wave_fence();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int q = sl * V + v;
    left[v] = gs[v] = q < a.groups ? sc[q] : -(S)INFINITY;
    mark[q] = 0;
  }
  wave_fence();
  for (int i = 0; i < a.kept; ++i) {
    int at;
    if (row_best<L>(left, sl, at) > -(S)INFINITY && at / V == sl) mark[at] = 1;
    strike(left, sl, at);
  }
  wave_fence();
  least = (S)INFINITY, best = -(S)INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int q = sl * V + v, e = q;
    if (q < a.groups) {
      if (mark[q]) least = min(least, gs[v]);
      else best = max(best, gs[v]);
    }
    if (e < a.E && !mark[e / n]) c[v] = -(S)INFINITY;
  }
  wave_fence();
}

// Score of this lane's group of `lanes` (2^j) lanes, whose experts they hold.
template <int L, int V, class S>
FP8L_DEV S lane_group(const RouteArgs& a, const S (&g)[V], int lanes) {
  S hi = -(S)INFINITY, lo = -(S)INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    lo = max(lo, min(hi, g[v]));
    hi = max(hi, g[v]);
  }
  lane_steps<L>([&](auto s) {
    constexpr int STEP = decltype(s)::value;
    if (STEP < lanes) {
      const S oh = lane_step<STEP>(hi), ol = lane_step<STEP>(lo);
      lo = max(min(hi, oh), max(lo, ol));
      hi = max(hi, oh);
    }
  });
  return a.group_top == 2 && lo > -(S)INFINITY ? hi + lo : hi;
}

// The same where 64 lanes hold a row and `lanes` (2^j) of them a group.
template <int V>
FP8L_DEV void keep_groups_wide(const RouteArgs& a, double (&c)[V], const double (&g)[V], int lane,
                               int lanes) {
  const double mark = lane_group<64>(a, g, lanes);
  const uint64_t u = (uint64_t)__double_as_longlong(mark);
  const int grp = lane / lanes;
  int ahead = 0;  // better groups
  for (int q = 0; q < a.groups; ++q) {
    const uint64_t lo = (uint32_t)__builtin_amdgcn_readlane((int)u, q * lanes);
    const uint64_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), q * lanes);
    const double o = __longlong_as_double((long long)(lo | hi << 32));
    ahead += o > mark || (o == mark && q < grp) ? 1 : 0;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) c[v] = ahead < a.kept ? c[v] : -(double)INFINITY;
}

template <int N>
FP8L_DEV uint32_t turn_lane(uint32_t v) {  // row_ror:N
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + N, 0xF, 0xF, false);
}
template <int N>
FP8L_DEV int turn_lane(int v) { return (int)turn_lane<N>((uint32_t)v); }
template <int N>
FP8L_DEV float turn_lane(float v) { return __uint_as_float(turn_lane<N>(__float_as_uint(v))); }
template <int N>
FP8L_DEV double turn_lane(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint64_t lo = turn_lane<N>((uint32_t)u), hi = turn_lane<N>((uint32_t)(u >> 32));
  return __longlong_as_double((long long)(lo | (hi << 32)));
}
// f(N tag) for N = 1 .. 15
template <int N = 1, class F>
FP8L_DEV void other_lanes(F&& f) {
  if constexpr (N < 16) {
    f(std::integral_constant<int, N>{});
    other_lanes<N + 1>(f);
  }
}

// c of the experts in groups that are not kept becomes -inf, for rows of 16
// lanes and groups of 2^j lanes (RouteArgs::lanes): every lane ranks its group
// among those of the other lanes.  g: what groups are scored by.  Whether the
// group stays, and its score, for the caller's proof.
template <int V>
FP8L_DEV bool keep_groups_lanes(const RouteArgs& a, float (&c)[V], const float (&g)[V], int sl,
                                float& mark) {
  mark = lane_group<16>(a, g, a.lanes);
  const int grp = sl / a.lanes;
  int ahead = 0;  // lanes of better groups
  other_lanes([&](auto n) {
    constexpr int N = decltype(n)::value;
    const float o = turn_lane<N>(mark);
    const int og = turn_lane<N>(grp);
    ahead += o > mark || (o == mark && og < grp) ? 1 : 0;
  });
  const bool in = ahead < a.kept * a.lanes;
#pragma unroll
  for (int v = 0; v < V; ++v) c[v] = in ? c[v] : -INFINITY;
  return in;
}

// The scores p of a row in S; m: its largest logit.  (Both kinds share the
// exponential's and the division's code, whose fetch is much of what a rare row
// costs.)
template <int L, int V, class S>
FP8L_DEV void row_scores(const RouteArgs& a, const float (&z)[V], float m, S (&p)[V]) {
  const bool sig = a.score == kSigmoid;
  S sum = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    p[v] = exp(sig ? -(S)z[v] : (S)z[v] - (S)m);
    sum += p[v];
  }
  sum = lanes_sum<L>(sum);
#pragma unroll
  for (int v = 0; v < V; ++v) p[v] = (sig ? (S)1 : p[v]) / (sig ? (S)1 + p[v] : sum);
}

// The chosen experts of a row, of scores in S: slot i's in lane i (-1: none).
template <int L, int V, class S>
FP8L_DEV int choose(const RouteArgs& a, const float (&z)[V], const float (&b)[V], float m, int sl,
                    uint8_t* row) {
  S c[V], g[V];
  const S none = -(S)INFINITY;
  const bool by_score = a.bias || (a.groups > 1 && a.group_top == 2);
  if (by_score) row_scores<L>(a, z, m, g);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const bool off = z[v] == -INFINITY;
    if (by_score) g[v] = off ? none : g[v] + (S)b[v];
    else g[v] = (S)z[v];
    c[v] = a.bias ? g[v] : (S)z[v];
  }
  if (a.groups > 1 && a.kept < a.groups) {
    S least, best;
    if (a.lanes) keep_groups_wide(a, c, g, sl, V > 1 ? 4 * a.lanes : a.E / a.groups);
    else keep_groups<L>(a, c, g, sl, row, least, best);
  }
  int mine = -1;
  for (int i = 0; i < a.k; ++i) {
    int at;
    const S best = row_best<L>(c, sl, at);
    if (sl == i && best > none) mine = at;
    strike(c, sl, at);
  }
  return mine;
}

// Weights of a row's slots: slot i's in lane i.  zi: the chosen one's logit.
template <int L, int V>
FP8L_DEV float slot_weight(const RouteArgs& a, const float (&z)[V], float m, bool live, float zi) {
  float q;
  if (a.score == kSoftmax) {
    const float top = a.renorm ? lanes_max<L>(live ? zi : -INFINITY) : m;
    q = live ? expf(zi - top) : 0.0f;
    float sum;
    if (a.renorm) {
      sum = lanes_sum<L>(q);
    } else {
      sum = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) sum += expf(z[v] - m);
      sum = lanes_sum<L>(sum);
    }
    q = live ? q / sum : 0.0f;
  } else {
    const float lo = fminf(zi, 0.0f);
    const float top = a.renorm ? lanes_max<L>(live ? lo : -INFINITY) : 0.0f;
    q = live ? expf(lo - top) / (1.0f + expf(-fabsf(zi))) : 0.0f;
    if (a.renorm) {
      const float sum = lanes_sum<L>(q);
      q = live ? q / sum : 0.0f;
    }
  }
  return q;
}

// ---------------------------------------------------------------- choice in 32 bits

// The choice of scores held in 64 bits, from scores in 32 bits and a proof
// (16384 rows of 256 experts entirely in 64 bits: 105 us).
//
//   keys     every expert gets an upper bound of its c as an integer below
//            2^31 whose lowest bits give way to the expert's index, lower ones
//            larger: a fixed-point number over the range of the row's c (24 bits
//            less one, so as fine as the scores), or the float's ordered bits
//            where logits of 16 bits are compared as they are, without loss.
//            All keys differ, so a round of the top-k is a maximum over the
//            lanes, and the largest key below the last one is
//            last + max(key - last) in unsigned numbers, without striking
//            anything out.
//   proof    the chosen experts' c, one per lane, in 32 bits with its bound:
//            all others have c <= what the (k + 1)-th key stands for, so the
//            set is right if every chosen c is larger, and the order if they
//            are further apart than their errors.  If not, the same in 64 bits,
//            where the order is also mended.
//   errors   a score in 32 bits is off by less than (|x| + n) 2^-23 of itself,
//            x its exponential's argument (rounded to 2^-24, and by the factor
//            log2 e); n = 4 for exp (1), 1 + exp (1/2) and reciprocal (1) of a
//            sigmoid, 24 with a softmax's sum: 20 additions, and its terms' |x|,
//            whose mean is at most log E.
//   groups   scored in 32 bits, in lanes or, where groups end inside a lane, from
//            LDS; right if the least kept and the best dropped group are further
//            apart than the scores' errors.
//   else     the wave does the row again in 64 bits, with all of its lanes.  So
//            it is wherever the k-th and the (k + 1)-th c are equal, but for
//            16-bit logits without a bias: no proof settles a tie there.  Few
//            rows of fp32 logits, but 9% of bf16 ones of 256 experts under a bias
//            of zeros, k 8 (16384 rows 29 us, under a bias of 24 bits 15.5;
//            4096 27 and 6.1; 131072 118 and 67).
//
// One row per 16 lanes, V experts per lane.

// Key bits of the index.
template <int V>
constexpr int key_low() { return V == 1 ? 4 : V == 4 ? 6 : V == 8 ? 7 : 8; }

// Order-preserving integer of a float that is no NaN.  The sum makes -0 a +0,
// which it ties with.
FP8L_DEV uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
// Value of the next lane of 16 (the last one's: its own).
FP8L_DEV uint32_t next_lane(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x101, 0xF, 0xF, false);  // row_shl:1
}
FP8L_DEV double next_lane(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint64_t lo = next_lane((uint32_t)u), hi = next_lane((uint32_t)(u >> 32));
  return __longlong_as_double((long long)(lo | (hi << 32)));
}

// The groups in 32 bits; false where that cannot tell which ones stay.  err:
// the largest error of a group's score (< 0: none).
template <int V>
FP8L_DEV bool keep_groups32(const RouteArgs& a, float (&c)[V], const float (&g)[V], int sl,
                            uint8_t* row, float err) {
  float least, best;
  if (a.lanes) {
    float mark;
    const bool in = keep_groups_lanes<V>(a, c, g, sl, mark);
    least = in ? mark : INFINITY;
    best = in ? -INFINITY : mark;
  } else {
    keep_groups<16>(a, c, g, sl, row, least, best);
  }
  if (err < 0.0f) return true;
  least = -lanes_max<16>(-least);
  best = lanes_max<16>(best);
  return best == -INFINITY || least - best > 2.0f * err + 0x1p-21f * (fabsf(least) + fabsf(best));
}

// A score in 32 bits; x: what its error grows with.  m, r: the row's largest
// logit and the reciprocal of the softmax's sum.
FP8L_DEV float score32(const RouteArgs& a, float z, float m, float r, float& x) {
  if (a.score == kSigmoid) {
    x = fabsf(z);
    return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
  }
  x = m - z;
  return __expf(z - m) * r;
}
// c's error: the score's, the addition's, and what underflows.
FP8L_DEV float c_error(const RouteArgs& a, float p, float x, float c) {
  const float n = a.score == kSigmoid ? 4.0f : 24.0f;
  return p * ((fminf(x, 128.0f) + n) * 0x1p-23f) + 0x1p-23f * fabsf(c) + 0x1p-120f;
}

// The chosen expert of slot i in lane i (-1: none) and its logit; sure: false
// where the row has to be done in 64 bits.  m: the row's largest logit.
template <int IN, int V>
FP8L_DEV int choose32(const RouteArgs& a, const float (&z)[V], const float (&b)[V], int64_t t,
                      float m, int sl, uint8_t* row, bool& sure, float& zi) {
  constexpr int LOW = key_low<V>();
  constexpr uint32_t MASK = (1u << LOW) - 1;
  const bool grouped = a.groups > 1 && a.kept < a.groups;
  const bool by_score = a.bias || (grouped && a.group_top == 2);
  float c[V], g[V], sum = 1.0f, rs = 1.0f, err = 0.0f;
  if (by_score) {
    if (a.score == kSoftmax) {
      sum = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) sum += g[v] = __expf(z[v] - m);
      sum = lanes_sum<16>(sum);
      rs = __builtin_amdgcn_rcpf(sum);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool off = z[v] == -INFINITY;
      float x, p = score32(a, z[v], m, rs, x);
      g[v] = off ? -INFINITY : p + b[v];
      const float d = g[v] == -INFINITY ? 0.0f : c_error(a, p, x, g[v]);
      err = fmaxf(err, d);
      c[v] = a.bias ? g[v] + 2.0f * d : z[v];  // twice: the addition of the bound
      if (g[v] == -INFINITY) c[v] = -INFINITY;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = g[v] = z[v];
  }
  sure = !grouped || keep_groups32<V>(a, c, g, sl, row, by_score ? 2.0f * lanes_max<16>(err) : -1.0f);
  // keys
  const bool exact = IN != kInF32 && !a.bias;
  uint32_t key[V], last = 0;
  float low = 0.0f, scale = 1.0f;
  if (exact) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      key[v] = ((ordered(c[v]) >> (LOW + 1)) << LOW) | (MASK - (uint32_t)(sl * V + v));
  } else {
    float hi = -INFINITY, lo = INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      hi = fmaxf(hi, c[v]);
      lo = fminf(lo, c[v] == -INFINITY ? INFINITY : c[v]);
    }
    hi = lanes_max<16>(hi);
    // masks of very small logits do not count: what lies below is one key apart
    low = fmaxf(-lanes_max<16>(-lo), hi - 64.0f);
    scale = 8388600.0f / fmaxf(hi - low, 0x1p-60f);
#pragma unroll
    for (int v = 0; v < V; ++v)
      key[v] = ((1u + (uint32_t)fmaxf((c[v] - low) * scale, 0.0f)) << LOW) |
               (MASK - (uint32_t)(sl * V + v));
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (c[v] == -INFINITY) key[v] = 0;
    last = max(last, key[v]);
  }
  lane_steps<16>([&](auto s) { last = max(last, lane_step<decltype(s)::value>(last)); });
  uint32_t slot = 0;  // this lane's slot's key
  for (int i = 0; i < a.k; ++i) {
    if (sl == i) slot = last;
    uint32_t r = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) r = max(r, key[v] - last);
    lane_steps<16>([&](auto s) { r = max(r, lane_step<decltype(s)::value>(r)); });
    last = (int32_t)r < 0 ? r + last : 0u;  // no key below the last one: none is left
  }
  const bool live = slot != 0;
  int e = live ? (int)(MASK - (slot & MASK)) : -1;
  zi = live ? load1<IN>(a.z, t * a.E + e) : 0.0f;
  if (exact) return e;

  // (last: the (k + 1)-th key, of a c at most `units` units above low: 1.5 for
  // the roundings of its three steps)
  const float units = (float)(last >> LOW) + 2.0f;
  const float bi = live && a.bias ? a.bias[e] : 0.0f;
  {
    float x, p = 0.0f, ci = live ? zi : -INFINITY, d = 0.0f;
    if (a.bias && live) {
      p = score32(a, zi, m, rs, x);
      ci = p + bi;
      d = c_error(a, p, x, ci);
    }
    const float above = units / scale;
    const float bound =
        last == 0 ? -INFINITY : low + above + 0x1p-22f * (fabsf(low) + above);
    const float cn = __uint_as_float(next_lane(__float_as_uint(ci)));
    const float dn = __uint_as_float(next_lane(__float_as_uint(d)));
    const int en = (int)next_lane((uint32_t)e);
    const bool both = sl + 1 < a.k && live && en >= 0;
    const bool ok = !live || (ci - 2.0f * d > bound && (!both || ci - cn > 2.0f * (d + dn) ||
                                                        (!a.bias && ci == cn && e < en)));
    if (!__any(!ok)) return e;
  }
  double ci = -INFINITY, p = 0.0;
  if (live) {
    if (a.bias) {
      const bool sig = a.score == kSigmoid;
      const double x = exp(sig ? -(double)zi : (double)zi - (double)m);
      p = (sig ? 1.0 : x) / (sig ? 1.0 + x : (double)sum);
      ci = p + (double)bi;
    } else {
      ci = zi;
    }
  }
  const bool loose = a.bias && a.score == kSoftmax;  // p carries the 32-bit sum's error
  const double slack = loose ? 0x1p-16 : 0.0;
  const double bound = last == 0 ? -INFINITY : ((double)low + (double)units / (double)scale);
  bool ok = !live || ci - slack * p > bound + 0x1p-30 * fabs(bound);
  const double cn = next_lane(ci), pn = next_lane(p);
  const int en = (int)next_lane((uint32_t)e);
  const bool both = sl + 1 < a.k && live && en >= 0;
  const bool wrong = both && (ci < cn || (ci == cn && e > en));
  if (loose) ok = ok && !wrong && !(both && p != pn && fabs(ci - cn) <= slack * fabs(p - pn));
  sure = sure && !lanes_any<16>(!ok);
  if (!loose && __any(wrong)) {
    // slots without an expert keep their places behind the others
    const int id = live ? e : 1024 + sl;
    int rank = 0;
    other_lanes([&](auto n) {
      constexpr int N = decltype(n)::value;
      const double o = turn_lane<N>(ci);
      const int oid = turn_lane<N>(id);
      rank += o > ci || (o == ci && oid < id) ? 1 : 0;
    });
    const int to = ((threadIdx.x & 48) + rank) * 4;
    e = __builtin_amdgcn_ds_permute(to, e);
    zi = __int_as_float(__builtin_amdgcn_ds_permute(to, __float_as_int(zi)));
  }
  return e;
}

// V consecutive logits (or biases) from element i on.
template <int IN, int V>
FP8L_DEV void load_v(const void* p, int64_t i, float (&v)[V]) {
  if constexpr (V >= 8) {
#pragma unroll
    for (int j = 0; j < V; j += 8) load8<IN>(p, i + j, v + j);
  } else if constexpr (V == 4 && IN == kInF32) {
    const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = load1<IN>(p, i + j);
  }
}

// A lane's logits and biases of row t (-inf, 0 past the last expert).
template <int IN, int V>
FP8L_DEV void load_row(const RouteArgs& a, int64_t t, int sl, bool vec, float (&z)[V],
                       float (&b)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) z[v] = -INFINITY, b[v] = 0.0f;
  if (vec) {
    if (sl * V < a.E) {
      load_v<IN>(a.z, t * a.E + sl * V, z);
      if (a.bias) load_v<kInF32>(a.bias, sl * V, b);
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = sl * V + v;
      if (e < a.E) {
        z[v] = load1<IN>(a.z, t * a.E + e);
        if (a.bias) b[v] = a.bias[e];
      }
    }
  }
}

// Experts per lane where 64 lanes take a row of 16 V, and its LDS.
template <int V>
constexpr int wide_v() { return V < 4 ? 1 : V / 4; }
template <int L, int V>
constexpr int route_wave_lds() {
  constexpr int rows = L == 64 ? 0 : 4 * group_lds<16, V, float>();
  constexpr int wide = group_lds<64, L == 64 ? V : wide_v<V>(), double>();
  return rows > wide ? rows : wide;
}

// One row of L lanes, V experts per lane (E <= L V, k <= L): the slot of lane
// sl: its expert, and its weight in w.  lds: route_wave_lds of this wave.
template <int IN, int L, int V>
FP8L_DEV int route_row(const RouteArgs& a, int64_t t, int sl, uint8_t* lds, float& w) {
  float z[V], b[V];
  load_row<IN>(a, t, sl, a.vec, z, b);
  bool bad = false;
  float m = -INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    bad = bad || z[v] != z[v] || b[v] != b[v] || (a.score == kSoftmax && z[v] == INFINITY);
    m = fmaxf(m, z[v]);
  }
  m = lanes_max<L>(m);
  bad = lanes_any<L>(bad);
  int mine = -1;
  float zi = 0.0f;
  if constexpr (L == 64) {
    mine = choose<L, V, double>(a, z, b, m, sl, lds);
    zi = sl < a.k && mine >= 0 ? load1<IN>(a.z, t * a.E + mine) : 0.0f;
  } else {
    bool sure;
    const int lane = threadIdx.x & 63;
    mine = choose32<IN, V>(a, z, b, t, m, sl, lds + (lane >> 4) * group_lds<16, V, float>(), sure,
                           zi);
    for (uint64_t todo = __ballot(!sure && !bad && sl == 0); todo; todo &= todo - 1) {
      const int from = __builtin_ctzll(todo);
      const int64_t row = __builtin_amdgcn_readlane((int)t, from);  // T < 2^31
      constexpr int W = wide_v<V>();
      float zw[W], bw[W];
      load_row<IN>(a, row, lane, false, zw, bw);
      const int all = choose<64, W, double>(a, zw, bw, __shfl(m, from), lane, lds);
      const int again = __shfl(all, sl);
      if (lane >> 4 == from >> 4) {
        mine = again;
        zi = sl < a.k && mine >= 0 ? load1<IN>(a.z, t * a.E + mine) : 0.0f;
      }
    }
  }
  const bool live = sl < a.k && !bad && mine >= 0;
  w = a.scale * slot_weight<L>(a, z, m, live, zi);
  if (bad) w = __uint_as_float(0x7fc00000u);
  return bad ? sl : mine;
}

template <int IN, int L, int V>
__global__ __launch_bounds__(kRThreads) void route_kernel(RouteArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kRThreads / 64 * route_wave_lds<L, V>()];
  const int sl = threadIdx.x % L;
  const int64_t t = (int64_t)blockIdx.x * (kRThreads / L) + threadIdx.x / L;
  float w;
  const int e = route_row<IN, L, V>(a, t < a.T ? t : a.T - 1, sl,
                                    lds + threadIdx.x / 64 * route_wave_lds<L, V>(), w);
  if (t < a.T && sl < a.k) {
    a.idx[t * a.k + sl] = e;
    a.w[t * a.k + sl] = w;
  }
}

// ---------------------------------------------------------------- gradient

struct RouteBwdArgs {
  RouteArgs r;        // z, idx, k, E, T, score, renorm, scale; w unused
  const float* dw;    // [T][k]
  void* dz;           // [T][E], z's type
};

template <int IN, int L, int V>
__global__ __launch_bounds__(kRThreads) void route_bwd_kernel(RouteBwdArgs a) {
  const RouteArgs& r = a.r;
  const int sl = threadIdx.x % L;
  const int64_t t0 = (int64_t)blockIdx.x * (kRThreads / L) + threadIdx.x / L;
  const bool there = t0 < r.T;
  const int64_t t = there ? t0 : r.T - 1;
  float z[V];
  float m = -INFINITY;
  const bool dense = r.score == kSoftmax && !r.renorm;  // every logit gets a part
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = sl * V + v;
    z[v] = dense && e < r.E ? load1<IN>(r.z, t * r.E + e) : -INFINITY;
    m = fmaxf(m, z[v]);
  }
  if (dense) m = lanes_max<L>(m);
  int e = -1;
  float d = 0.0f;
  if (sl < r.k) {
    e = r.idx[t * r.k + sl];
    if (e < 0 || e >= r.E) e = -1;
    else d = r.scale * a.dw[t * r.k + sl];
  }
  const bool live = e >= 0;
  const float zi = live ? load1<IN>(r.z, t * r.E + e) : 0.0f;
  const float q = slot_weight<L>(r, z, m, live, zi);
  float part = live ? q * d : 0.0f;
  const float dot = r.renorm || dense ? lanes_sum<L>(part) : 0.0f;
  if (r.renorm) part = live ? q * (d - dot) : 0.0f;
  // 1 - p = sigmoid(-z)
  if (r.score == kSigmoid) part = live ? part / (1.0f + expf(zi)) : 0.0f;
  float g[V];
  if (dense) {
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) sum += g[v] = expf(z[v] - m);
    sum = lanes_sum<L>(sum);
#pragma unroll
    for (int v = 0; v < V; ++v) g[v] = m == -INFINITY && dot == 0.0f ? 0.0f : -dot * (g[v] / sum);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) g[v] = 0.0f;
  }
  for (int i = 0; i < r.k; ++i) {
    const int src = (threadIdx.x & 63 & ~(L - 1)) + i;
    const int ei = __shfl(e, src);
    const float pi = __shfl(part, src);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (ei == sl * V + v) g[v] += pi;
  }
  if (!there) return;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (sl * V + v < r.E) store1<IN>(a.dz, t * r.E + sl * V + v, g[v]);
}

// ---------------------------------------------------------------- places

// Rows sorted by expert, in the order of the slots (a stable counting sort):
// slot j = t k + i with expert e goes to offsets[e] + the number of earlier
// slots of e.  Slots of no expert get -1.  The slots are cut into chunks, one
// per block.  With few of them every block counts all slots itself; with many,
// a first launch counts each chunk's, and a block adds up what lies before its
// own.  Nothing is counted by atomics across blocks: places do not depend on
// timing.
struct PlanArgs {
  const int32_t* idx;
  int32_t* offsets;  // [E + 1]
  int32_t* pos;      // [n]
  int32_t* counts;   // [chunks][E], null: each block counts all slots
  int32_t n, E, chunk, chunks;
};

FP8L_DEV int slot_expert(const PlanArgs& a, int j) {
  const int e = a.idx[j];
  return e >= 0 && e < a.E ? e : a.E;
}

__global__ __launch_bounds__(kRThreads) void plan_count_kernel(PlanArgs a) {
  __shared__ int32_t h[kRouteMaxE + 1];
  for (int e = threadIdx.x; e <= a.E; e += kRThreads) h[e] = 0;
  __syncthreads();
  const int j1 = min((int)(blockIdx.x + 1) * a.chunk, a.n);
  constexpr int U = 8;  // loads in flight
  for (int j = blockIdx.x * a.chunk + threadIdx.x; j < j1; j += U * kRThreads) {
    int e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) e[u] = slot_expert(a, min(j + u * kRThreads, a.n - 1));
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (j + u * kRThreads < j1) atomicAdd(&h[e[u]], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kRThreads) a.counts[(int64_t)blockIdx.x * a.E + e] = h[e];
}

// Lanes of the wave with the same key (< 2^bits).
FP8L_DEV uint64_t same_key(int key, int bits) {
  uint64_t peers = ~0ull;
  for (int i = 0; i < bits; ++i) {
    const uint64_t m = __ballot((key >> i) & 1);
    peers &= (key >> i) & 1 ? m : ~m;
  }
  return peers;
}

// Places the slots of one chunk, NT threads; expert(j): slot j's expert, a.E
// for none.  lds: NW (E + 1) integers, then 3 NT more.
template <int NT>
__host__ __device__ constexpr int place_lds(int E) {
  return (4 * ((NT / 64 + 2) * (E + 1) + 3 * NT) + 15) & ~15;
}

template <int NT, class F>
FP8L_DEV void place_chunk(const PlanArgs& a, int block, int32_t* lds, F&& expert) {
  constexpr int NW = NT / 64, COLS = NT < 256 ? NT : 256, SPLIT = NT / COLS;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, W = a.E + 1;
  int32_t* const next = lds;  // [wave][expert]: the wave's slots, then its next place
  int32_t* const before_part = lds + NW * W;  // [SPLIT][COLS]
  int32_t* const total_part = before_part + NT;
  int32_t* const wave_total = total_part + NT;
  int32_t* const all = wave_total + NT;  // without counts: [before this chunk, from it on][expert]
  const bool count_all = a.chunks > 1 && !a.counts;
  for (int i = tid; i < NW * W; i += NT) next[i] = 0;
  if (count_all)
    for (int i = tid; i < 2 * W; i += NT) all[i] = 0;
  __syncthreads();
  // wave w's slots: the w-th part of the chunk, steps of 64, U of them in flight
  constexpr int U = 4;
  const int per = a.chunk / NW;
  const int j0 = block * a.chunk + wave * per, j1 = min(j0 + per, a.n);
  int32_t* const mine = next + wave * W;
  int slot[U];
  auto load_slots = [&](int j) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = j + 64 * u + lane;
      slot[u] = i < j1 ? expert(i) : a.E;
    }
  };
  const int last = per > 0 ? (per - 1) / (64 * U) * (64 * U) : 0;
  load_slots(j0 + last);
  if (count_all) {
    constexpr int Q = 8;  // loads of four slots in flight
    typedef int32_t four __attribute__((ext_vector_type(4), aligned(4)));
    const int before = block * a.chunk, quads = a.n / 4;  // (a chunk is a multiple of 4)
    auto count = [&](int j, int e) {
      atomicAdd(&all[(j < before ? 0 : W) + (e >= 0 && e < a.E ? e : a.E)], 1);
    };
    for (int q0 = tid; q0 < quads; q0 += Q * NT) {
      four v[Q];
#pragma unroll
      for (int u = 0; u < Q; ++u)
        v[u] = reinterpret_cast<const four*>(a.idx)[min(q0 + u * NT, quads - 1)];
#pragma unroll
      for (int u = 0; u < Q; ++u) {
        const int q = q0 + u * NT;
        if (q < quads)
          for (int i = 0; i < 4; ++i) count(4 * q, v[u][i]);
      }
    }
    if (tid < a.n % 4) count(4 * quads + tid, a.idx[4 * quads + tid]);
  }
  // from the last steps to the first, which stay for the places below
  for (int j = j0 + last;; j -= 64 * U) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (j + 64 * u + lane < j1) atomicAdd(&mine[slot[u]], 1);
    if (j <= j0) break;
    load_slots(j - 64 * U);
  }
  __syncthreads();
  // first places of 256 experts at a time; SPLIT threads add up an expert's chunks
  int carry = 0;
  for (int e0 = 0; e0 < a.E; e0 += COLS) {
    const int col = tid % COLS, part = tid / COLS, e = e0 + col;
    int before = 0, total = 0;
    if (e < a.E) {
      if (a.chunks == 1) {
        for (int w = part; w < NW; w += SPLIT) total += next[w * W + e];
      } else if (count_all) {
        if (part == 0) before = all[e], total = all[e] + all[W + e];
      } else {
        constexpr int U = 16;  // loads in flight
        for (int c0 = part; c0 < a.chunks; c0 += U * SPLIT) {
          int n[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int c = c0 + u * SPLIT;
            n[u] = a.counts[min(c, a.chunks - 1) * a.E + e];
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int c = c0 + u * SPLIT;
            if (c < a.chunks) total += n[u];
            if (c < block) before += n[u];
          }
        }
      }
    }
    before_part[tid] = before;
    total_part[tid] = total;
    __syncthreads();
    before = total = 0;
    if (tid < COLS)
      for (int s = 0; s < SPLIT; ++s) {
        before += before_part[s * COLS + tid];
        total += total_part[s * COLS + tid];
      }
    int incl = total;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 63) wave_total[wave] = incl;
    __syncthreads();
    int first = carry + incl - total;
    for (int w = 0; w < COLS / 64; ++w) {
      if (w < wave) first += wave_total[w];
      carry += wave_total[w];
    }
    if (tid < COLS && e < a.E) {
      if (block == 0) {
        a.offsets[e] = first;
        if (e == a.E - 1) a.offsets[a.E] = first + total;
      }
      int at = first + before;
      for (int w = 0; w < NW; ++w) {
        const int n = next[w * W + e];
        next[w * W + e] = at;
        at += n;
      }
    }
    __syncthreads();
  }
  const int bits = 32 - __builtin_clz(a.E);
  for (int jb = j0; jb < j1; jb += 64 * U) {
    if (jb > j0) load_slots(jb);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (jb + 64 * u >= j1) break;
      const int j = jb + 64 * u + lane, e = slot[u];
      const uint64_t peers = same_key(e, bits);
      const int rank = __popcll(peers & ((1ull << lane) - 1));
      const int at = mine[e] + rank;
      wave_fence();
      if (rank == 0) mine[e] += __popcll(peers);
      wave_fence();
      if (j < j1) a.pos[j] = e < a.E ? at : -1;
    }
  }
}

constexpr int kPlaceThreads = 512;
__global__ __launch_bounds__(kPlaceThreads) void plan_place_kernel(PlanArgs a) {
  extern __shared__ __attribute__((aligned(16))) int32_t place_mem[];
  place_chunk<kPlaceThreads>(a, blockIdx.x, place_mem, [&](int j) { return slot_expert(a, j); });
}

// Few tokens: choice and places by one block, in one launch.
template <int IN, int V>
__global__ __launch_bounds__(kPlaceThreads) void route_place_kernel(RouteArgs a, PlanArgs p) {
  extern __shared__ __attribute__((aligned(16))) int32_t place_mem[];
  int32_t* const slots = place_mem;  // [T][k]
  int32_t* const place = slots + kPlaceThreads;
  uint8_t* const rows = reinterpret_cast<uint8_t*>(place) + place_lds<kPlaceThreads>(p.E);
  const int sl = threadIdx.x % 16, t = threadIdx.x / 16;
  float w;
  const int e = route_row<IN, 16, V>(a, min(t, a.T - 1), sl,
                                     rows + threadIdx.x / 64 * route_wave_lds<16, V>(), w);
  if (t < a.T && sl < a.k) {
    a.idx[t * a.k + sl] = e;
    a.w[t * a.k + sl] = w;
    slots[t * a.k + sl] = e < 0 ? p.E : e;
  }
  __syncthreads();
  place_chunk<kPlaceThreads>(p, 0, place, [&](int j) { return slots[j]; });
}
constexpr int kRoutePlaceRows = kPlaceThreads / 16;
template <int V>
constexpr int route_place_lds(int E) {
  return 4 * kPlaceThreads + place_lds<kPlaceThreads>(E) +
         kPlaceThreads / 64 * route_wave_lds<16, V>();
}

// ---------------------------------------------------------------- rows

// A row's pieces go to `width` neighbouring threads (a power of two up to the
// block's), the block's 256 / width tokens side by side, further pieces over
// blockIdx.y.  A piece is 16 bytes (8 values), at any address; the last one of a
// row ends with it and may overlap the one before, which then holds the same
// (4096 x 8 rows of 4097 bf16 values, us so / value by value: there 64 / 138,
// back 61 / 177, gradients 123 / 360).  Rows shorter than a piece go by single
// bytes or values.
struct RowGrid {
  int32_t width_log, pieces;
};

template <int U>
struct Bytes {
  typedef uint32_t T __attribute__((ext_vector_type(4), aligned(1)));
};
template <> struct Bytes<1> { typedef uint8_t T; };

struct GatherArgs {
  const uint8_t* x;    // [T] rows
  uint8_t* out;        // [R] rows
  const int32_t* pos;  // [T][k]
  int32_t T, k, R;
  int64_t row;         // bytes
  RowGrid grid;
};

template <int U>
__global__ __launch_bounds__(kRThreads) void gather_kernel(GatherArgs a) {
  typedef typename Bytes<U>::T P;
  const int piece = blockIdx.y * (1 << a.grid.width_log) + (threadIdx.x & ((1 << a.grid.width_log) - 1));
  if (piece >= a.grid.pieces) return;
  const int per = kRThreads >> a.grid.width_log;
  const int64_t at = min<int64_t>((int64_t)piece * U, a.row - U);
  for (int64_t t = (int64_t)blockIdx.x * per + (threadIdx.x >> a.grid.width_log); t < a.T;
       t += (int64_t)gridDim.x * per) {
    const P v = *reinterpret_cast<const P*>(a.x + t * a.row + at);
    for (int i = 0; i < a.k; ++i) {
      const int p = a.pos[t * a.k + i];
      if (p >= 0 && p < a.R) *reinterpret_cast<P*>(a.out + p * a.row + at) = v;
    }
  }
}

struct CombineArgs {
  const void* y;       // [R][D]
  const int32_t* pos;  // [T][k]
  const float* w;      // [T][k], null: ones
  void* out;           // [T][D]
  int32_t T, k, R;
  int64_t D;
  RowGrid grid;
};

// A piece of N values of a row, 8 or 1.
template <int IN, int N>
FP8L_DEV void store_n(void* p, int64_t i, const float (&v)[N]) {
  if constexpr (N == 8) store8<IN>(p, i, v);
  else store1<IN>(p, i, v[0]);
}

constexpr int kSlotBatch = 8;  // slots whose rows are loaded together

// Places and weights of slots i0 .. i0 + 7 of a token (-1, 0 past the last).
// UNI: the token is the wave's, so its slots come by scalar loads (nothing
// writes them meanwhile) and every row's address is a scalar.
template <bool UNI>
FP8L_DEV void load_slots(const int32_t* pos, const float* w, int64_t t, int k, int i0, int R,
                         int (&p)[kSlotBatch], float (&wt)[kSlotBatch]) {
  typedef const __attribute__((address_space(4))) int32_t* SInt;
  typedef const __attribute__((address_space(4))) float* SFloat;
#pragma unroll
  for (int s = 0; s < kSlotBatch; ++s) {
    const int64_t at = t * k + min(i0 + s, k - 1);
    if constexpr (UNI) {
      p[s] = ((SInt)(uintptr_t)pos)[at];
      wt[s] = w ? ((SFloat)(uintptr_t)w)[at] : 1.0f;
    } else {
      p[s] = pos[at];
      wt[s] = w ? w[at] : 1.0f;
    }
    if (i0 + s >= k || p[s] >= R) p[s] = -1;
  }
}

// out[t] = sum_i w[t, i] y[pos[t, i]], in slot order in 32 bits, rounded once.
// Bound by reading y: a thread has its piece of eight rows in flight (4096
// tokens, 8 slots of 4096 bf16 values, 302 MB: 52 us; one row after the
// other 91).
template <int IN, int N, bool UNI>
__global__ __launch_bounds__(kRThreads) void combine_kernel(CombineArgs a) {
  const int piece = blockIdx.y * (1 << a.grid.width_log) + (threadIdx.x & ((1 << a.grid.width_log) - 1));
  const int per = kRThreads >> a.grid.width_log;
  const int64_t at = min<int64_t>((int64_t)piece * N, a.D - N);
  for (int64_t t0 = (int64_t)blockIdx.x * per + (threadIdx.x >> a.grid.width_log); t0 < a.T;
       t0 += (int64_t)gridDim.x * per) {
    const int t = UNI ? __builtin_amdgcn_readfirstlane((int)t0) : (int)t0;
    float acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.0f;
    for (int i0 = 0; i0 < a.k; i0 += kSlotBatch) {
      int p[kSlotBatch];
      float w[kSlotBatch];
      load_slots<UNI>(a.pos, a.w, t, a.k, i0, a.R, p, w);
      Raw<IN, N> v[kSlotBatch];
#pragma unroll
      for (int s = 0; s < kSlotBatch; ++s) {
        v[s].zero();
        if (p[s] >= 0 && piece < a.grid.pieces) v[s].template load<true>(a.y, p[s] * a.D + at);
      }
#pragma unroll
      for (int s = 0; s < kSlotBatch; ++s)
#pragma unroll
        for (int j = 0; j < N; ++j)
          acc[j] = __builtin_fmaf(p[s] >= 0 ? w[s] : 0.0f, v[s].get(j), acc[j]);
    }
    if (piece < a.grid.pieces) store_n<IN>(a.out, t * a.D + at, acc);
  }
}

struct CombineBwdArgs {
  const void* dout;    // [T][D]
  const void* y;       // [R][D]
  const int32_t* pos;
  const float* w;
  void* dy;            // [R][D] or null
  float* dw;           // [T][k] or null
  int32_t T, k, R;
  int64_t D;
};

// dy[pos[t, i]] = w[t, i] dout[t] and dw[t, i] = dout[t] . y[pos[t, i]]: one
// wave per token, eight slots at a time.
template <int IN, int N>
__global__ __launch_bounds__(kRThreads) void combine_bwd_kernel(CombineBwdArgs a) {
  constexpr int S = kSlotBatch;
  const int lane = threadIdx.x & 63;
  const int64_t pieces = (a.D + N - 1) / N;
  for (int64_t t0 = (int64_t)blockIdx.x * (kRThreads / 64) + (threadIdx.x >> 6); t0 < a.T;
       t0 += (int64_t)gridDim.x * (kRThreads / 64)) {
    const int t = __builtin_amdgcn_readfirstlane((int)t0);
    for (int i0 = 0; i0 < a.k; i0 += S) {
      int p[S];
      float w[S], dot[S];
      load_slots<true>(a.pos, a.w, t, a.k, i0, a.R, p, w);
#pragma unroll
      for (int s = 0; s < S; ++s) dot[s] = 0.0f;
      for (int64_t c = lane; c < pieces; c += 64) {
        const int64_t at = min<int64_t>(c * N, a.D - N);
        const int seen = (int)(c * N - at);  // values of the piece before
        Raw<IN, N> raw;
        raw.load(a.dout, t * a.D + at);
        float g[N];
#pragma unroll
        for (int j = 0; j < N; ++j) g[j] = raw.get(j);
        if (a.dw) {
          Raw<IN, N> v[S];
#pragma unroll
          for (int s = 0; s < S; ++s) {
            if (p[s] >= 0) v[s].template load<true>(a.y, p[s] * a.D + at);
            else v[s].zero();
          }
#pragma unroll
          for (int s = 0; s < S; ++s)
#pragma unroll
            for (int j = 0; j < N; ++j)
              if (p[s] >= 0 && j >= seen) dot[s] = __builtin_fmaf(g[j], v[s].get(j), dot[s]);
        }
        if (a.dy) {
#pragma unroll
          for (int s = 0; s < S; ++s) {
            if (p[s] < 0) continue;
            float v[N];
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = w[s] * g[j];
            store_n<IN>(a.dy, p[s] * a.D + at, v);
          }
        }
      }
      if (a.dw) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const float d = lanes_sum<64>(dot[s]);
          if (lane == 0 && i0 + s < a.k) a.dw[(int64_t)t * a.k + i0 + s] = d;
        }
      }
    }
  }
}

}  // namespace fp8l
