// Routing to experts from given logits, its gradient, and the grouping of the
// chosen (token, slot) rows by expert.
//
//   s    = softmax(l) or sigmoid(l)                     scores, all E experts
//   key  = s + b                                        b selects only (balance)
//   score of a group = the sum of its group_top (1 or 2) largest keys; the
//   topk_groups best groups stay; the k largest keys in them are chosen, ties to
//   the lower index; w_j = scale * s_j [/ sum_i s_i over the chosen].
// (nxmr.cn "V4" article, §2.2; DeepSeek V4 infra notes, §6.3; the linux.do post on
// MoE variants, "QuantileBalancing".)
//
// Without a bias the scores grow with the logits, so the logits themselves are the
// keys and every comparison of two experts is exact.  With one, keys are formed in
// fp32; where two neighbours in the order lie within the error bound below, the slots'
// keys (and those of the experts just left out) are formed again in fp64, one a lane.
// A row whose groups' fp32 sums are that close goes to a second pass in fp64, which
// places groups without a bias by the logits (group_position).
#include <cfloat>

#include "common.cuh"
#include "moe_internal.h"
#include "ops_internal.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// fp32 as an unsigned integer of the same order; 0 is below every number (it
// stands for "cannot be chosen").  -0 and +0 are one value.
__device__ __forceinline__ uint32_t order_of(float v) {
  const int b = __float_as_int(v + 0.0f);
  return static_cast<uint32_t>(b ^ ((b >> 31) | 0x80000000));
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ uint32_t key_of(float v) {
  // NaN and -inf can never be chosen.
  return v > -INFINITY ? order_of(v) : 0u;
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

__device__ __forceinline__ float sigmoid_f32(float l) { return 1.0f / (1.0f + expf(-l)); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// The same to about 1e-7: its own rounding and the exponent's, |l| s (1 - s) 2^-23 at
// most (for keys, whose near neighbours are settled in fp64).
__device__ __forceinline__ float sigmoid_fast(float l) { return __fdividef(1.0f, 1.0f + __expf(-l)); }

// Descending, by Batcher's odd-even merge network.
template <int N>
__device__ __forceinline__ void sort_desc(uint32_t (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int q = p; q >= 1; q >>= 1)
#pragma unroll
      for (int j = q % p; j <= N - 1 - q; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i <= N - j - q - 1 && (i + j) / (p * 2) == (i + j + q) / (p * 2)) {
            const uint32_t hi = max(v[i + j], v[i + j + q]), lo = min(v[i + j], v[i + j + q]);
            v[i + j] = hi;
            v[i + j + q] = lo;
          }
}

// Sum of N values in pairs: log2 N roundings of each, not N - 1.
template <int N, typename F>
__device__ __forceinline__ float sum_in_pairs(F value) {
  float part[6];   // part[b]: the sum of 2^b values
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = value(i);
    int b = 0;
#pragma unroll
    for (; b < 6 && (i >> b & 1); ++b) s += part[b];
    part[b] = s;
  }
  int top = 0;
#pragma unroll
  for (int b = 0; b < 6; ++b)
    if (N >> b == 1) top = b;
  return part[top];
}

// How far the difference of two fp32 keys of about this size can be from the exact
// one, u = 2^-24.  sigmoid: below 3e-7 each for s <= 1 (sigmoid_fast).  softmax, of
// d = max - l: e^-d errs by |d| u (the argument) and 4 u (2 ulp), the reciprocal and
// the product by 2 u, so p by (0.37 + 6 p) u; the sum by (ln E + 4) u and its at most
// 5 + 5 additions (sum_in_pairs, warp_sum), an error that the two keys share: it counts
// by p - p'.  As p + p' <= 1: 0.74 + 6 + 21 = 28 u.  The sum with the bias: u |key|
// each.  (A bound that shrinks with the largest p spares softmax rows fp64 work but
// costs the others a register: 13.65 -> 14.05 us for sigmoid rows of 256.)
__device__ __forceinline__ float close_bound(float key, int softmax) {
  return fmaf(1.3e-7f, fabsf(key), softmax ? 1.7e-6f : 6.5e-7f);
}

// Where a group without a bias stands whose best logits are a >= b (-inf: it has only
// one), as hi + lo that grows with the sum S of their scores and tells sums apart
// where fp64 scores would all be 1 or 0:
//   softmax  log S + const = a + log(1 + e^(b - a))
//   sigmoid  S - 1 = sigmoid(a) - sigmoid(-b) = (1 - e^-(a + b)) sigmoid(a) sigmoid(b)
//            between 1/2 and 3/2, log S below, -log(2 - S) above; 2 - S is the sum of
//            (-b, -a), so that only sums below 1 have to be formed.
__device__ __noinline__ double2 group_position(double a, double b, int softmax) {
  const double ninf = -static_cast<double>(INFINITY);
  auto sigmoid = [](double v) { return 1.0 / (1.0 + exp(-v)); };
  double x = a, small;
  bool low = true;
  if (softmax) {
    if (!(fabs(x) < -ninf)) return make_double2(x, 0.0);
    small = log1p(exp(b - a));
  } else {
    const double s = b > ninf ? a + b : ninf;   // S < 1 exactly where a + b < 0
    low = s < 0.0;
    const double y = low ? b : -a;
    if (!low) x = -b;
    const double t = -expm1(-fabs(s)) * sigmoid(-x) * sigmoid(-y);   // 1 - S of (x, y)
    if (t <= 0.5) return make_double2(low ? -t : t, 0.0);
    if (!(fabs(x) < -ninf)) return make_double2(low ? x : -x, 0.0);
    const double ex = exp(x);                   // S < 1/2, so x < 0
    small = log1p(exp(y - x) * (1.0 + ex) / (1.0 + exp(y))) - log1p(ex);
  }
  const double hi = x + small, z = hi - x, lo = (x - (hi - z)) + (small - z);   // hi + lo = x + small
  return low ? make_double2(hi, lo) : make_double2(-hi, -lo);
}

// The whole row again in fp64, for rows whose fp32 keys are too close to order.
// Without a bias the logits stay the keys.
// Returns the expert of slot `lane` (-1: none).
template <int CPL, typename In>
__device__ __noinline__ int select_exact(const RouteOpArgs& a, const In* row, int lane, int first, int count) {
  const double ninf = -static_cast<double>(INFINITY);
  double key[CPL];
  auto load = [&]() {
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const double l = i < count ? static_cast<double>(to_float(row[first + i])) : ninf;
      key[i] = l > ninf ? l : ninf;
    }
  };
  load();
  if (a.bias != nullptr) {
    if (a.softmax) {
      double m = ninf, sum = 0.0;
#pragma unroll
      for (int i = 0; i < CPL; ++i) m = fmax(m, key[i]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kFull, m, o));
#pragma unroll
      for (int i = 0; i < CPL; ++i)
        if (key[i] > ninf) { key[i] = exp(key[i] - m); sum += key[i]; }
        else key[i] = ninf;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
#pragma unroll
      for (int i = 0; i < CPL; ++i)
        if (key[i] > ninf) key[i] /= sum;
    } else {
#pragma unroll
      for (int i = 0; i < CPL; ++i)
        if (key[i] > ninf) key[i] = 1.0 / (1.0 + exp(-key[i]));
    }
#pragma unroll
    for (int i = 0; i < CPL; ++i)
      if (key[i] > ninf) {
        key[i] += static_cast<double>(a.bias[first + i]);
        if (!(key[i] > ninf)) key[i] = ninf;
      }
  }
  if (a.topk_groups < a.n_groups) {
    double m1 = ninf, m2 = ninf;
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      if (key[i] > m1) { m2 = m1; m1 = key[i]; }
      else if (key[i] > m2) m2 = key[i];
    }
    for (int o = 1; o < a.lpg; o <<= 1) {
      const double o1 = __shfl_xor_sync(kFull, m1, o), o2 = __shfl_xor_sync(kFull, m2, o);
      const double hi = fmax(m1, o1), lo = fmin(m1, o1);
      m2 = fmax(lo, fmax(m2, o2));
      m1 = hi;
    }
    // A group with one expert left scores by that one.  Positions that come out equal
    // are ordered by the logits: b first, whose part in the sum is the smaller one.
    double2 at = make_double2((a.group_top == 2 && m2 > ninf) ? m1 + m2 : m1, 0.0);
    if (a.bias != nullptr) {
      m1 = m2 = 0.0;
    } else if (a.group_top == 2) {
      if (m1 > ninf) at = group_position(m1, m2, a.softmax);
      load();   // again: no register holds them over the call
    }
    const int g = lane / a.lpg;
    int rank = 0;
    for (int q = 0; q < a.n_groups; ++q) {
      const int from = q * a.lpg;
      const double hq = __shfl_sync(kFull, at.x, from), lq = __shfl_sync(kFull, at.y, from);
      const double bq = __shfl_sync(kFull, m2, from), aq = __shfl_sync(kFull, m1, from);
      bool above = q < g;
      if (aq != m1) above = aq > m1;
      if (bq != m2) above = bq > m2;
      if (lq != at.y) above = lq > at.y;
      if (hq != at.x) above = hq > at.x;
      rank += above ? 1 : 0;
    }
    if (rank >= a.topk_groups)
#pragma unroll
      for (int i = 0; i < CPL; ++i) key[i] = ninf;
  }
  int chosen = -1;
  for (int j = 0; j < a.k; ++j) {
    double bk = ninf;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < CPL; ++i)
      if (key[i] > bk) { bk = key[i]; be = first + i; }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ok = __shfl_xor_sync(kFull, bk, o);
      const int oe = __shfl_xor_sync(kFull, be, o);
      if (ok > bk || (ok == bk && oe < be)) { bk = ok; be = oe; }
    }
    if (!(bk > ninf)) break;
    if (lane == j) chosen = be;
#pragma unroll
    for (int i = 0; i < CPL; ++i)
      if (first + i == be) key[i] = ninf;
  }
  return chosen;
}

// One warp per token.  Lane l owns cpl consecutive experts of group l / lpg, so
// lanes hold experts in index order: the lowest lane with the greatest key, and
// its first position with it, is the lowest index.  Every lane sorts its keys; each
// of the k rounds takes the maximum of the lanes' heads with one redux and the
// winner moves up its list; lane j notes the key and the winner of slot j and looks
// its expert up among the winner's keys when all are known.
// Bound by instructions issued: T = 8192, E = 256, k = 8 in 8 groups reads 8.4 MB fp32
// (1.3 us of memory) and takes 13.8 us, one token 4.1.  A lane's whole sort network
// is cheaper than searching its keys in every round; a row that has to be decided
// in fp64 costs the launch up to 8 us.
// The resident CTAs keep the fp64 pass, which few rows take, from costing the others
// registers (8 experts a lane: 70 without it, and 14.6 instead of 13.6 us for 8192 x
// 256).  Two a lane would have to spill for more than four CTAs: 8192 x 64 takes 6.45
// us with four, 6.84 with six.
template <int CPL, typename In>
__global__ void __launch_bounds__(256, CPL == 4 ? 5 : CPL <= 8 ? 4 : CPL <= 16 ? 2 : 1) k_route(const RouteOpArgs a) {
  griddep_wait();
  griddep_launch();
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (t >= a.T) return;
  const In* row = static_cast<const In*>(a.logits) + static_cast<long long>(t) * a.ld;
  const int g = lane / a.lpg, sub = lane - g * a.lpg;
  const int first = g * a.gs + sub * a.cpl;
  const int count = g < a.n_groups ? max(0, min(a.cpl, a.gs - sub * a.cpl)) : 0;
  const bool groups = a.topk_groups < a.n_groups;

  float l[CPL];
  constexpr int kPer16 = 16 / sizeof(In);
  bool loaded = false;
  if constexpr (CPL >= kPer16) if (a.vec) {
    loaded = true;
    // count is cpl or 0 here, and cpl a multiple of kPer16.
#pragma unroll
    for (int i = 0; i < CPL; i += kPer16) {
      union { uint4 u; In e[kPer16]; } v;
      v.u = make_uint4(0, 0, 0, 0);
      if (i < count) v.u = *reinterpret_cast<const uint4*>(row + first + i);
#pragma unroll
      for (int z = 0; z < kPer16; ++z) l[i + z] = i + z < count ? to_float(v.e[z]) : -INFINITY;
    }
  }
  if (!loaded) {
#pragma unroll
    for (int i = 0; i < CPL; ++i) l[i] = i < count ? to_float(row[first + i]) : -INFINITY;
  }

  // Softmax over the whole row where a value of it is needed.
  float rmax = 0.f, rsum = 1.f;
  if (a.softmax && (!a.renorm || a.bias != nullptr || (groups && a.group_top == 2))) {
    rmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < CPL; ++i) rmax = fmaxf(rmax, l[i]);   // fmaxf drops a NaN
    rmax = warp_max(rmax);
    rsum = warp_sum(sum_in_pairs<CPL>([&](int i) { return l[i] > -INFINITY ? expf(l[i] - rmax) : 0.f; }));
  }
  auto score = [&](float v) { return a.softmax ? expf(v - rmax) / rsum : sigmoid_f32(v); };

  uint32_t key[CPL], top[CPL];   // in index order; descending
  const float rscale = 1.f / rsum;
  if (a.bias != nullptr) {
    float bias[CPL];
    bool whole = false;
    if constexpr (CPL >= 4) if (a.vec_bias) {
      whole = true;
#pragma unroll
      for (int i = 0; i < CPL; i += 4) {
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < count) f = *reinterpret_cast<const float4*>(a.bias + first + i);
        bias[i] = f.x; bias[i + 1] = f.y; bias[i + 2] = f.z; bias[i + 3] = f.w;
      }
    }
    if (!whole) {
#pragma unroll
      for (int i = 0; i < CPL; ++i) bias[i] = i < count ? a.bias[first + i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const float s = a.softmax ? expf(l[i] - rmax) * rscale : sigmoid_fast(l[i]);
      key[i] = l[i] > -INFINITY ? key_of(s + bias[i]) : 0u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < CPL; ++i) key[i] = key_of(l[i]);
  }

#pragma unroll
  for (int i = 0; i < CPL; ++i) top[i] = key[i];
  sort_desc(top);

  bool close_groups = false;   // an order that fp32 cannot decide
  if (groups) {
    uint32_t m1 = top[0], m2 = CPL > 1 ? top[1] : 0u;
    for (int o = 1; o < a.lpg; o <<= 1) {
      const uint32_t o1 = __shfl_xor_sync(kFull, m1, o), o2 = __shfl_xor_sync(kFull, m2, o);
      m2 = max(max(m2, o2), min(m1, o1));
      m1 = max(m1, o1);
    }
    uint32_t gscore = m1;
    // What the keys' and their sum's own roundings can be, 2 2^-24 of the keys' sizes:
    // the sum may be far smaller than they are.  Infinite with them.
    float slack = 0.f;
    if (m1 != 0 && (a.bias != nullptr || a.group_top == 2)) {
      // Keys are logits without a bias; the sum is of their scores.
      const float v1 = a.bias != nullptr ? value_of(m1) : score(value_of(m1));
      float v2 = 0.f;
      if (a.group_top == 2 && m2 != 0) v2 = a.bias != nullptr ? value_of(m2) : score(value_of(m2));
      gscore = order_of(v1 + v2);
      slack = 1.3e-7f * (fabsf(v1) + fabsf(v2));
    }
    int rank = 0;
    for (int q = 0; q < a.n_groups; ++q) {
      const uint32_t sq = __shfl_sync(kFull, gscore, q * a.lpg);
      rank += (sq > gscore || (sq == gscore && q < g)) ? 1 : 0;
    }
    const bool stays = rank < a.topk_groups;
    if (a.bias != nullptr || a.group_top == 2) {
      // The lowest that a kept group may be, the highest that another may.
      const float v = value_of(gscore);
      const uint32_t low = slack < INFINITY ? order_of(v - slack) : order_of(-INFINITY);
      const uint32_t high = slack < INFINITY ? order_of(v + slack) : order_of(INFINITY);
      const bool has = g < a.n_groups && gscore != 0;
      const uint32_t worst = __reduce_min_sync(kFull, has && stays ? low : 0xffffffffu);
      const uint32_t best = __reduce_max_sync(kFull, has && !stays ? high : 0u);
      if (best != 0 && worst != 0xffffffffu)
        close_groups = !(value_of(worst) - value_of(best) > (a.softmax ? 1.8e-6f : 1.3e-6f));   // four scores' errors
    }
    if (!stays) {
#pragma unroll
      for (int i = 0; i < CPL; ++i) top[i] = 0;
    }
  }

  // Rounds beyond the k-th only with fp32 keys: the experts left out that come within
  // the bound of the last one in.
  bool close = false, many = false;
  uint32_t prev = 0, mine = 0;   // mine: the key of this lane's slot (0: none)
  int from = 0;                  // and the lane that had it
  float last = 0.f;              // key of slot k - 1
  for (int j = 0;; ++j) {
    if (a.bias == nullptr && j == a.k) break;
    const uint32_t m = __reduce_max_sync(kFull, top[0]);
    if (m == 0) break;
    if (a.bias != nullptr) {
      const float v = value_of(m);
      if (j > 0) close |= value_of(prev) - v <= close_bound(v, a.softmax);
      if (j >= a.k) {
        if (j == a.k) last = value_of(prev);
        if (!close || last - v > close_bound(v, a.softmax)) break;
        if (j == 32) { many = true; break; }
      }
      prev = m;
    }
    const int win = __ffs(__ballot_sync(kFull, top[0] == m)) - 1;
    if (lane == j) { mine = m; from = win; }
    const bool up = lane == win;
#pragma unroll
    for (int i = 0; i < CPL; ++i) top[i] = up ? (i + 1 < CPL ? top[i + 1] : 0u) : top[i];
  }
  // Slot `lane`: the expert of lane `from` with key `mine`; of several equal ones the
  // one after those that earlier slots took.
  int chosen = -1;
  {
    // Equal keys of one lane fill neighbouring slots: how many before this one.
    const uint32_t mine_below = __shfl_up_sync(kFull, mine, 1);   // every lane takes part in both
    const int from_below = __shfl_up_sync(kFull, from, 1);
    const bool same = lane > 0 && mine_below == mine && from_below == from;
    const unsigned starts = ~__ballot_sync(kFull, same) & (0xffffffffu >> (31 - lane));
    int skip = lane - (31 - __clz(starts));
    const int f0 = __shfl_sync(kFull, first, from);
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const uint32_t v = __shfl_sync(kFull, key[i], from);
      if (mine != 0 && v == mine && chosen < 0 && skip-- == 0) chosen = f0 + i;
    }
  }
  int slot = lane;
  if (close_groups || many) {   // uniform over the warp, as close
    chosen = select_exact<CPL, In>(a, row, lane, first, count);
  } else if (close) {
    double m = 0.0, sum = 1.0, k64 = -static_cast<double>(INFINITY);
    if (a.softmax) {
      m = rmax;
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < CPL; ++i)
        if (l[i] > -INFINITY) sum += exp(static_cast<double>(l[i]) - m);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    }
    if (chosen >= 0) {
      const double v = static_cast<double>(to_float(row[chosen]));
      k64 = (a.softmax ? exp(v - m) / sum : 1.0 / (1.0 + exp(-v))) + static_cast<double>(a.bias[chosen]);
    }
    const int n = __popc(__ballot_sync(kFull, chosen >= 0));   // slots 0 .. n - 1 are filled
    int rank = 0;
    for (int j = 0; j < n; ++j) {
      const double kj = __shfl_sync(kFull, k64, j);
      const int ej = __shfl_sync(kFull, chosen, j);
      rank += (kj > k64 || (kj == k64 && ej < chosen)) ? 1 : 0;
    }
    if (chosen >= 0) slot = rank;
  }
  if (slot >= a.k) chosen = -1;

  // Weights; every lane has one slot.
  const bool have = chosen >= 0;
  const float lj = have ? to_float(row[chosen]) : -INFINITY;
  float w = 0.f;
  if (a.renorm) {
    float s = 0.f;
    if (a.softmax) {
      const float m = warp_max(lj);
      s = have ? expf(lj - m) : 0.f;
    } else {
      s = have ? sigmoid_f32(lj) : 0.f;
      // Far below zero a sigmoid is the exponential: shift it, so that nothing
      // underflows (and the sum is never zero).
      const float m = warp_max(lj);
      if (m < -60.f) s = have ? expf(lj - m) : 0.f;
    }
    const float total = warp_sum(s);
    w = have ? s / total * a.scale : 0.f;
  } else if (have) {
    w = score(lj) * a.scale;
  }
  if (slot < a.k) {
    a.idx[static_cast<long long>(t) * a.k + slot] = chosen;
    a.w[static_cast<long long>(t) * a.k + slot] = w;
  }
}

// Gradient of the weights with respect to the logits, one warp per token.  With
// u_j = dw_j (slots of one expert added in slot order):
//   softmax, renormalised   dl_j = w_j (dw_j - sum_i dw_i w_i / scale), chosen only
//   softmax                 dl_e = scale p_e (u_e - sum_j dw_j p_j), every expert
//   sigmoid                 dl_j = ds_j s_j (1 - s_j), ds_j = scale dw_j, or
//                           scale (dw_j - sum_i dw_i s_i / S) / S with S = sum s_i
// The row is written once (zeros, or the softmax's common term); the chosen
// experts' lanes then write theirs.
// Bound by memory: every logit of the row is written, and read for a plain
// softmax (T = 16384, E = 128 fp32: 17.8 MB, 6.2 us with the rows in L2, 12.7 without).
// The row is in the caches by the time the chosen lanes' part is known.
template <int PER, int VEC, typename In>
__global__ void __launch_bounds__(256) k_route_backward(const RouteBackArgs a) {
  griddep_wait();
  griddep_launch();
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (t >= a.T) return;
  const In* row = static_cast<const In*>(a.logits) + static_cast<long long>(t) * a.ld;
  In* out = static_cast<In*>(a.dlogits) + static_cast<long long>(t) * a.ld_out;
  struct alignas(sizeof(In) * VEC) Vec { In e[VEC]; };
  const bool whole = a.softmax && !a.renorm;

  int e = -1;
  float dw = 0.f;
  if (lane < a.k) {
    e = a.idx[static_cast<long long>(t) * a.k + lane];
    dw = a.dw[static_cast<long long>(t) * a.k + lane];
    if (e < 0 || e >= a.E) { e = -1; dw = 0.f; }
  }
  const float lj = e >= 0 ? to_float(row[e]) : -INFINITY;
  // -inf and NaN logits are never chosen; an index given for one gets no gradient, and
  // its dw, whatever it is, is in no sum.
  const bool have = lj > -INFINITY;
  if (!have) dw = 0.f;

  auto store = [](float v) {
    if constexpr (sizeof(In) == 2) return static_cast<In>(pack_bf16x2(v, 0.f) & 0xFFFFu);
    else return v;
  };

  float l[PER];
  float rmax = -INFINITY, rsum = 1.f;
  if (whole) {
#pragma unroll
    for (int i = 0; i < PER; i += VEC) {
      const int c = (i * 32 + lane * VEC);
      Vec v;
#pragma unroll
      for (int z = 0; z < VEC; ++z) l[i + z] = -INFINITY;
      if (c < a.E) {
        v = *reinterpret_cast<const Vec*>(row + c);
#pragma unroll
        for (int z = 0; z < VEC; ++z) l[i + z] = to_float(v.e[z]);
      }
#pragma unroll
      for (int z = 0; z < VEC; ++z) rmax = fmaxf(rmax, l[i + z]);
    }
    rmax = warp_max(rmax);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      l[i] = l[i] > -INFINITY ? expf(l[i] - rmax) : 0.f;
      s += l[i];
    }
    rsum = warp_sum(s);
  }

  float dl = 0.f, common = 0.f;   // common: -sum_j dw_j p_j
  float p = 0.f;
  if (whole) {
    p = have ? expf(lj - rmax) / rsum : 0.f;
    common = -warp_sum(dw * p);
    dl = p * dw;
  } else if (a.softmax) {
    const float m = warp_max(lj);
    const float s = have ? expf(lj - m) : 0.f;
    const float total = warp_sum(s);
    const float q = have ? s / total : 0.f;
    const float mean = warp_sum(dw * q);
    dl = q * (dw - mean);
  } else {
    float s = have ? sigmoid_f32(lj) : 0.f;
    // 1 - s without cancellation: sigmoid(-l).
    const float c = have ? sigmoid_f32(-lj) : 0.f;
    if (a.renorm) {
      const float m = warp_max(lj);
      if (m < -60.f) s = have ? expf(lj - m) : 0.f;   // as the forward pass does
      const float total = warp_sum(s);
      const float q = have ? s / total : 0.f;
      const float mean = warp_sum(dw * q);
      dl = q * c * (dw - mean);
    } else {
      dl = s * c * dw;
    }
  }
  // Slots that name the same expert add up, in slot order.
  float mine = 0.f;
  for (int j = 0; j < a.k; ++j) {
    const int ej = __shfl_sync(kFull, e, j);
    const float dj = __shfl_sync(kFull, dl, j);
    if (ej == e) mine += dj;
  }
  if (whole && have) mine += p * common;
  mine *= a.scale;
  const float base = whole ? common * a.scale / rsum : 0.f;
#pragma unroll
  for (int i = 0; i < PER; i += VEC) {
    const int c = (i * 32 + lane * VEC);
    if (c >= a.E) break;
    Vec v;
#pragma unroll
    for (int z = 0; z < VEC; ++z) v.e[z] = store(whole && l[i + z] > 0.f ? l[i + z] * base : 0.f);
    *reinterpret_cast<Vec*>(out + c) = v;
  }
  __syncwarp();
  if (have) out[e] = store(mine);
}

// ---------------------------------------------------------------- grouping
// One cluster of 8 CTAs; CTA c takes the c-th eighth of the flattened (token,
// slot) list and each of its warps a run of it.  A warp counts its run per expert
// in its own row of shared memory; the prefix over warps, over CTAs (through
// distributed shared memory) and over experts gives every warp its first row of
// every expert; a second walk hands the rows out 32 entries at a time (the lanes
// with one expert come from a vote on each of its bits: match.any costs the SM
// about 40 cycles a time).  Integers only, the order is the
// list's: stable by token, then slot.  No workspace and one launch, whatever T.
// Bound by latency: the list is small (T = 8192, k = 8, E = 256: 262 KB in 12.1 us;
// one token 6.5 us, most of it the two cluster barriers and the prefix over warps).
constexpr int kGroupCtas = 8;
constexpr int kGroupThreads = 1024;
constexpr int kAtOnce = 8;

// Lanes whose `e` (its `bits` low bits, at most 11) equals this lane's.
__device__ __forceinline__ unsigned lanes_with(int e, int bits) {
  unsigned same = kFull;
#pragma unroll
  for (int b = 0; b < 11; ++b) {
    if (b >= bits) break;   // uniform
    const bool one = (e >> b) & 1;
    const unsigned v = __ballot_sync(kFull, one);
    same &= one ? v : ~v;
  }
  return same;
}

__global__ void __launch_bounds__(kGroupThreads)
    k_group_rows(const int32_t* idx, int n, int k, int E, int32_t* offsets,
                 int32_t* token_of_row, int32_t* row_of_slot) {
  extern __shared__ int32_t gsm[];
  constexpr int kWarps = kGroupThreads / 32;
  int32_t* hist = gsm;                  // [kWarps][E]
  int32_t* mine = gsm + kWarps * E;     // [E] this CTA's counts (read by the others)
  __shared__ int32_t warp_tot[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = static_cast<int>(cluster_ctarank());
  // Runs are whole multiples of 32 entries; n < 2^31.
  const uint32_t per_warp = ((static_cast<uint32_t>(n) + kGroupCtas * kWarps - 1) / (kGroupCtas * kWarps) + 31) / 32 * 32;
  const uint32_t lo = static_cast<uint32_t>(min(static_cast<unsigned long long>(n),
                                                (static_cast<unsigned long long>(cta) * kWarps + warp) * per_warp));
  const uint32_t hi = static_cast<uint32_t>(min(static_cast<unsigned long long>(n),
                                                static_cast<unsigned long long>(lo) + per_warp));
  for (int i = tid; i < kWarps * E; i += kGroupThreads) hist[i] = 0;
  griddep_wait();
  griddep_launch();
  __syncthreads();

  int32_t* h = hist + warp * E;
  const int bits = 32 - __clz(E);   // E itself stands for no expert
  // kAtOnce loads are in flight before their entries are counted.
  int e[kAtOnce];
  auto read = [&](uint32_t b) {
#pragma unroll
    for (int z = 0; z < kAtOnce; ++z) {
      const uint32_t i = b + 32 * z + lane;
      e[z] = i < hi ? idx[i] : -1;
      if (e[z] >= E) e[z] = -1;
    }
  };
  for (uint32_t b = lo; b < hi; b += 32 * kAtOnce) {
    read(b);
#pragma unroll
    for (int z = 0; z < kAtOnce; ++z) {
      if (e[z] >= 0) atomicAdd(&h[e[z]], 1);   // a count: any order
    }
  }
  __syncthreads();
  for (int e = tid; e < E; e += kGroupThreads) {
    int run = 0;
#pragma unroll 8
    for (int w = 0; w < kWarps; ++w) {
      const int c = hist[w * E + e];
      hist[w * E + e] = run;
      run += c;
    }
    mine[e] = run;
  }
  cluster_sync();
  // kGroupThreads >= E: thread e has expert e.
  int before = 0, total = 0;
  if (tid < E) {
#pragma unroll
    for (int c = 0; c < kGroupCtas; ++c) {
      int v;
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(mine + tid, c)));
      if (c < cta) before += v;
      total += v;
    }
  }
  int incl = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_tot[warp] = incl;
  __syncthreads();
  int base = 0, all = 0;
#pragma unroll 8
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) base += warp_tot[w];
    all += warp_tot[w];
  }
  const int start = base + incl - total;
  if (tid < E) {
    if (cta == 0) {
      offsets[tid] = start;
      if (tid == E - 1) offsets[E] = all;
    }
    const int add = start + before;
#pragma unroll 8
    for (int w = 0; w < kWarps; ++w) hist[w * E + tid] += add;
  }
  __syncthreads();
  for (uint32_t b = lo; b < hi; b += 32 * kAtOnce) {
    if (hi - lo > 32 * kAtOnce) read(b);   // else still there from the count
#pragma unroll
    for (int z = 0; z < kAtOnce; ++z) {
      const uint32_t i = b + 32 * z + lane;
      const bool ok = e[z] >= 0;
      const unsigned same = lanes_with(ok ? e[z] : E, bits);
      int pos = -1;
      if (ok) pos = h[e[z]] + __popc(same & ((1u << lane) - 1u));
      __syncwarp();
      if (ok && lane == __ffs(same) - 1) h[e[z]] += __popc(same);
      __syncwarp();
      if (i < hi) {
        row_of_slot[i] = pos;
        if (ok) token_of_row[pos] = static_cast<int32_t>(i / static_cast<uint32_t>(k));
      }
    }
  }
  // Rows behind the last group come from no token.
  for (long long r = all + static_cast<long long>(cta) * kGroupThreads + tid; r < n; r += kGroupCtas * kGroupThreads)
    token_of_row[r] = -1;
  cluster_sync();   // no CTA leaves while another may still read its counts
}

template <typename In>
cudaError_t route_by_width(const RouteOpArgs& a, cudaStream_t s) {
  const dim3 grid((a.T + 7) / 8), block(256);
  if (a.cpl <= 2) return launch_k(k_route<2, In>, grid, block, 0, s, false, a);
  if (a.cpl <= 4) return launch_k(k_route<4, In>, grid, block, 0, s, false, a);
  if (a.cpl <= 8) return launch_k(k_route<8, In>, grid, block, 0, s, false, a);
  if (a.cpl <= 16) return launch_k(k_route<16, In>, grid, block, 0, s, false, a);
  return launch_k(k_route<32, In>, grid, block, 0, s, false, a);
}

template <int VEC, typename In>
cudaError_t route_back_by_width(const RouteBackArgs& a, cudaStream_t s) {
  const dim3 grid((a.T + 7) / 8), block(256);
  if (a.E <= 128) return launch_k(k_route_backward<4, VEC, In>, grid, block, 0, s, false, a);
  if (a.E <= 256) return launch_k(k_route_backward<8, VEC, In>, grid, block, 0, s, false, a);
  if (a.E <= 512) return launch_k(k_route_backward<16, VEC, In>, grid, block, 0, s, false, a);
  return launch_k(k_route_backward<32, VEC, In>, grid, block, 0, s, false, a);
}

}  // namespace

cudaError_t launch_route(const RouteOpArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? route_by_width<uint16_t>(a, s) : route_by_width<float>(a, s);
}

cudaError_t launch_route_backward(const RouteBackArgs& a, bool bf16, cudaStream_t s) {
  if (a.vec) return bf16 ? route_back_by_width<4, uint16_t>(a, s) : route_back_by_width<4, float>(a, s);
  return bf16 ? route_back_by_width<1, uint16_t>(a, s) : route_back_by_width<1, float>(a, s);
}

cudaError_t launch_group_rows(const int32_t* idx, int T, int k, int E, int32_t* offsets, int32_t* token_of_row,
                              int32_t* row_of_slot, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(kGroupThreads / 32 + 1) * E * sizeof(int32_t);
  const cudaError_t rc = cudaFuncSetAttribute(k_group_rows, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              (kGroupThreads / 32 + 1) * kRouteMaxE * 4);
  if (rc != cudaSuccess) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kGroupCtas);
  cfg.blockDim = dim3(kGroupThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kGroupCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_group_rows, idx, T * k, k, E, offsets, token_of_row, row_of_slot);
}

}  // namespace moe
