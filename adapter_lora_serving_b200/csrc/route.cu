// Routing of tokens to experts, the grouping of (token, choice) pairs by
// expert, and the weighted combine of the experts' rows: what stands between
// the router fold (lora_apply_router), the expert fold (lora_expert_apply) and
// the layer's output.
//
// Sources: spark_model/lora/expert_apply.rs, module text (the router delta
// lands before top-k; the fold works on rows sorted by expert_offsets, before
// moe_unpermute_reduce_indexed).
#include <mutex>

#include "elem.cuh"
#include "experts.h"

namespace lora {

namespace {

// ---------------------------------------------------------------------------
// Ordered keys: unsigned integers that compare as the numbers they come from
// (+0 and -0 alike).  What cannot be chosen has the key of -inf, or 0.
// ---------------------------------------------------------------------------

LORA_DEV uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
LORA_DEV float value_of(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
LORA_DEV uint64_t order_of(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
LORA_DEV double value_of(uint64_t u) {
  return __longlong_as_double((long long)((u >> 63) ? (u & 0x7fffffffffffffffull) : ~u));
}
LORA_DEV bool is_open(uint32_t u) { return u > 0x007fffffu; }
LORA_DEV bool is_open(uint64_t u) { return u > 0x000fffffffffffffull; }

LORA_DEV uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }
LORA_DEV uint64_t warp_max(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
  const uint32_t lo =
      __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((uint64_t)hi << 32) | lo;
}

template <typename V>
struct KeyOf;
template <>
struct KeyOf<float> { typedef uint32_t U; };
template <>
struct KeyOf<double> { typedef uint64_t U; };

// The warp's row of logits: lane l holds experts [l * VPL, (l + 1) * VPL), those
// past E as -inf.
template <int VPL, typename LT>
LORA_DEV void load_row(const LT* row, int lane, int E, float (&x)[VPL]) {
  const int e0 = lane * VPL;
  constexpr int kBytes = VPL * (int)sizeof(LT);
  if (E % VPL == 0 && kBytes >= 4) {
    // the lane's share is whole or empty, and aligned to its size (or 16 bytes)
    constexpr int kVec = kBytes >= 16 ? 16 : kBytes;
    constexpr int kN = kBytes / kVec == 0 ? 1 : kBytes / kVec;
    uint32_t w[kBytes < 4 ? 1 : kBytes / 4];
    if (e0 < E) {
      const LT* p = row + e0;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        if (kVec == 16) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
          w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        } else if (kVec == 8) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
          w[0] = v.x; w[1] = v.y;
        } else {
          w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
        }
      }
      const LT* q = reinterpret_cast<const LT*>(w);
#pragma unroll
      for (int i = 0; i < VPL; ++i) x[i] = to_f32(q[i]);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) x[i] = -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] = e0 + i < E ? to_f32(row[e0 + i]) : -INFINITY;
  }
}

// Masked logits: NaN and +inf become -inf (and set *bad).  Returns whether every
// lane's share is finite, or wholly past E.
template <int VPL>
LORA_DEV bool mask_row(float (&x)[VPL], bool past_end, bool* bad) {
  bool fine = true;
#pragma unroll
  for (int i = 0; i < VPL; ++i) fine = fine && fabsf(x[i]) < INFINITY;
  if (__all_sync(0xffffffffu, fine || past_end)) return true;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (!(x[i] < INFINITY)) {
      x[i] = -INFINITY;
      *bad = true;
    }
  return false;
}

// The lane's biases: 0 without any, -inf past E and where one is NaN or +inf
// (*bad).
template <int VPL>
LORA_DEV void load_bias(const RouteParams& p, int lane, float (&bias)[VPL], bool* bad) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    bias[i] = e >= p.E ? -INFINITY : p.bias != nullptr ? __ldg(p.bias + e) : 0.0f;
    if (!(bias[i] < INFINITY)) {
      bias[i] = -INFINITY;
      *bad = true;
    }
  }
}

// Whether all experts have one bias, a finite one (VPL of them in each lane, e0 the
// lane's first; the caller votes), and no sum of two scores counts: then the order of
// the keys is that of the logits, also where scores are equal in 64 bits.  Asked only
// where keys are close.
template <int VPL>
LORA_DEV bool one_bias(const RouteParams& p, const float (&bias)[VPL], int e0) {
  if (p.bias == nullptr || (p.num_groups > 1 && p.group_score == LORA_GROUP_TOP_PAIR)) return false;
  const float first = __ldg(p.bias);
  bool same = fabsf(first) < INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) same = same && (e0 + i >= p.E || bias[i] == first);
  return same;
}

// e^z and 1 / a: in 64 bits, or for fp32 keys whose error is accounted for (Within)
// the fast ones: 2 + 1.173 |z| ulps and 2 ulps.
LORA_DEV double power(double z) { return exp(z); }
LORA_DEV float power(float z) { return __expf(z); }
LORA_DEV double inverse(double a) { return 1.0 / a; }
LORA_DEV float inverse(float a) { return __fdividef(1.0f, a); }

// Scores of the lane's experts in V.  Returns the largest score of the row.
template <int VPL, typename V>
LORA_DEV V scores(const RouteParams& p, const float (&x)[VPL], V (&s)[VPL]) {
  if (p.score == LORA_SCORE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = inverse((V)1 + power(-(V)x[i]));
    return (V)1;
  }
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) m = fmaxf(m, x[i]);
  {
    const uint32_t u = warp_max(order_of(m));
    m = is_open(u) ? value_of(u) : 0.0f;
  }
  V sum = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    s[i] = power((V)x[i] - (V)m);
    sum += s[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const V inv = inverse(sum);
#pragma unroll
  for (int i = 0; i < VPL; ++i) s[i] = s[i] * inv;
  return inv;   // the largest: exp(0) / sum
}

// What a chosen expert's weight is a share of: softmax relative to the logit `top`, or
// the sigmoid, to be renormalised relative to that of a negative `top`, the largest
// chosen (so that nothing underflows to 0 / 0).
LORA_DEV float weight_of(const RouteParams& p, float x, float top) {
  if (p.score == LORA_SCORE_SOFTMAX) return expf(x - top);
  if (x >= 0.0f || !p.renormalize) return 1.0f / (1.0f + expf(-x));
  return expf(x - fminf(top, 0.0f)) / (1.0f + expf(x));
}

// Selection keys s + bias of the lane's experts; a masked logit has key 0, a masked
// bias the key of -inf.
template <int VPL, typename V>
LORA_DEV void make_keys(const float (&x)[VPL], const V (&s)[VPL], const float (&bias)[VPL],
                        bool finite, typename KeyOf<V>::U (&u)[VPL]) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) u[i] = order_of(s[i] + (V)bias[i]);
  if (!finite) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (!(x[i] > -INFINITY)) u[i] = 0;
  }
}

LORA_DEV uint32_t magnitude_of(uint32_t u) {
  return is_open(u) ? __float_as_uint(fabsf(value_of(u))) : 0u;
}
LORA_DEV uint32_t magnitude_of(uint64_t) { return 0; }   // (exact keys only)

// How close two keys may come before fp32 cannot tell them apart.
struct Exact {
  static constexpr bool kExact = true;
  template <typename V>
  LORA_DEV V operator()(V) const { return (V)-1; }
  LORA_DEV float of_sum(uint32_t) const { return -1.0f; }
};
// Twice the error of an fp32 key, in units of u = 2^-23.
//   sigmoid: e^-x moves the score by s (1 - s) (2 + 1.173 |x|) u < u (|x| s (1 - s)
//     < .23); the sum and the quotient by 3 s u: 4 u in all, 8 for two.
//   softmax: a term e^z is off by (2 + 1.173 |z|) u, and by half a |z| u for the
//     rounding of z: e^z (2 + 1.68 |z|) u <= 2 u, and half a u for the product with
//     the inverse.  The sum is off by the mean of (2 + 1.68 |z|) u over its terms, half
//     a u for each of VPL + 4 additions and 2 u for the quotient.  That mean is largest
//     with one expert at 0 and the others at one -w (w = 5.4 of 1024 experts): 5.1,
//     5.9, 6.8, 7.7, 8.6 and 9.5 for 32, 64 ... 1024 experts.  It is a factor that all
//     scores share, so it acts on the difference of two, at most smax: counted once.
//     Two keys: (mean + VPL / 2 + 4 + 5) u smax, at most 35 for VPL = 32 and 15 for 1
//     (a thread's EM - 1 additions: 28 for 32); here VPL + 22.
//   the bias sum: half a u of the key; the place within the lane that fills its
//     three lowest bits (Sorted): 7 u of it.  Two keys: 15 u, here 16.
// A pair's sum has the errors of both its keys, whose magnitudes its own can be
// far below, and half a u for the sum: 31 u of the row's largest key, here 34.
struct Within {
  static constexpr bool kExact = false;
  float of_score;
  LORA_DEV float operator()(float v) const { return of_score + 0x1p-19f * fabsf(v); }
  LORA_DEV float of_sum(uint32_t magnitude) const {
    return 2.0f * of_score + 0x1.1p-18f * __uint_as_float(warp_max(magnitude));
  }
};
template <int VPL>
LORA_DEV Within key_error(const RouteParams& p, float smax) {
  Within w;
  w.of_score = p.score == LORA_SCORE_SIGMOID ? 8.0f * 0x1p-23f : (float)(VPL + 22) * 0x1p-23f * smax;
  return w;
}

// Ranks the groups' scores, lane g holding group g's (`count` of them): which
// groups are kept, as a mask, and whether the border is within the error.
template <typename U, typename Tol>
LORA_DEV uint32_t best_groups(const RouteParams& p, int lane, U score, uint32_t magnitude, Tol tol,
                              bool* close) {
  const bool real = lane < p.num_groups;
  int rank = 0;
  for (int g = 0; g < p.num_groups; ++g) {
    const U other = __shfl_sync(0xffffffffu, score, g);
    rank += (other > score || (other == score && g < lane)) ? 1 : 0;
  }
  const bool kept = real && rank < p.top_groups;
  const uint32_t keep = __ballot_sync(0xffffffffu, kept && is_open(score));
  if (!Tol::kExact) {
    const U worst_kept = ~warp_max(kept && is_open(score) ? (U)~score : (U)0);
    const U best_out = warp_max(real && !kept ? score : (U)0);
    const float border = tol.of_sum(magnitude);
    // (keys of 2^127 and more, whose sums fp32 cannot hold, show in the border)
    *close |= border >= 0x1p109f ||
              (is_open(best_out) && value_of(worst_kept) - value_of(best_out) <= border);
  }
  return keep;
}

// A pair's score from the two largest keys of a group (one alone counts alone).
template <typename U>
LORA_DEV U group_score_of(const RouteParams& p, U top, U second) {
  return p.group_score == LORA_GROUP_TOP_PAIR && is_open(second)
             ? order_of(value_of(top) + value_of(second))
             : top;
}

// Keeps the experts of the best top_groups groups (ties to the lowest group),
// clearing the others' keys.  Group g holds the E / num_groups experts from
// g * E / num_groups on.  Any group size.
template <int VPL, typename U, typename Tol>
LORA_DEV void keep_groups(const RouteParams& p, int lane, U (&u)[VPL], Tol tol, bool* close) {
  const int n = p.E / p.num_groups;
  U score = 0;   // this lane's group's
  uint32_t magnitude = 0;
  for (int g = 0; g < p.num_groups; ++g) {
    U a = 0, b = 0;   // the lane's two largest keys in group g
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      const U v = (e >= g * n && e < (g + 1) * n) ? u[i] : 0;
      b = max(b, min(a, v));
      a = max(a, v);
    }
    const U top = warp_max(a);
    U second = 0;
    if (p.group_score == LORA_GROUP_TOP_PAIR) {
      // the best lane's runner-up, or another lane's best
      const uint32_t holders = __ballot_sync(0xffffffffu, a == top);
      second = warp_max(lane == __ffs((int)holders) - 1 ? b : a);
    }
    const U of_group = group_score_of(p, top, second);
    if (lane == g) score = of_group;
    if (!Tol::kExact) magnitude = max(magnitude, max(magnitude_of(a), magnitude_of(b)));
  }
  const uint32_t keep = best_groups(p, lane, score, magnitude, tol, close);
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    if (e < p.E && !((keep >> (e / n)) & 1u)) u[i] = 0;
  }
}

// The top_k largest keys in descending order, ties to the lowest expert: lane
// j returns the j-th choice (-1 when nothing is left).  *close is set when two
// neighbours in that order, or the last choice and the best one left, are
// within the keys' error.
template <int VPL, typename U, typename Tol>
LORA_DEV int take_best(const RouteParams& p, int lane, U (&u)[VPL], Tol tol, bool* close) {
  U best = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) best = max(best, u[i]);
  int id = -1;
  U prev = 0;
  const int rounds = p.top_k + (Tol::kExact ? 0 : 1);
  for (int j = 0; j < rounds; ++j) {
    const U m = warp_max(best);
    if (!is_open(m)) break;
    if (!Tol::kExact) {
      if (prev != 0 && value_of(prev) - value_of(m) <= tol(value_of(prev))) *close = true;
      prev = m;
      if (j == p.top_k) break;
    }
    const int src = __ffs((int)__ballot_sync(0xffffffffu, best == m)) - 1;
    int at = 0;
    if (lane == src) {
#pragma unroll
      for (int i = VPL - 1; i >= 0; --i)
        if (u[i] == m) at = i;
      best = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (i == at) u[i] = 0;
        best = max(best, u[i]);
      }
    }
    at = __shfl_sync(0xffffffffu, at, src);
    if (lane == j) id = src * VPL + at;
  }
  return id;
}

// Batcher's odd-even merge sort of the VPL keys of a lane, descending.
template <int VPL, typename Swap>
LORA_DEV void sort_network(Swap order) {
#pragma unroll
  for (int p = 1; p < VPL; p <<= 1)
#pragma unroll
    for (int k = p; k >= 1; k >>= 1)
#pragma unroll
      for (int j = k % p; j + k < VPL; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < VPL && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order(i + j, i + j + k);
}

// A lane's keys (VPL <= 8; with 16 the rounds over unsorted keys are faster, 29 us
// against 39 for 8192 tokens of 384 experts) in descending order: one sorting
// network, after which a round of the selection looks at the lanes' first keys
// alone (the list of the lane that gave one moves up).  Equal keys stay in order of
// their places.  Where the place in the lane is held:
//   kLow    in the key's three lowest bits (7 - i), which moves an approximate key by
//           7 ulps at most (accounted for in Within);
//   kExpert in the ten lowest bits (1023 - e) of a 16-bit logit's key, whose own
//           lowest 13 are constant: exact, and no two are equal;
//   kBeside beside the key: exact keys that need all their bits.
enum Place { kLow, kExpert, kBeside };

template <int VPL, typename V, Place kPlace>
struct Sorted {
  typedef typename KeyOf<V>::U U;
  static constexpr bool kAt = kPlace == kBeside;
  U u[VPL];
  int at[kAt ? VPL : 1];

  LORA_DEV void sort(int lane) {
    if (kAt) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) at[kAt ? i : 0] = i;
      sort_network<VPL>([&](int i, int j) {
        const int ai = at[kAt ? i : 0], aj = at[kAt ? j : 0];
        const bool swap = u[j] > u[i] || (u[j] == u[i] && aj < ai);
        const U hi = swap ? u[j] : u[i];
        u[j] = swap ? u[i] : u[j];
        u[i] = hi;
        at[kAt ? i : 0] = swap ? aj : ai;
        at[kAt ? j : 0] = swap ? ai : aj;
      });
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        u[i] = kPlace == kLow ? (u[i] & ~(U)7) | (U)(7 - i)
                              : (u[i] & ~(U)1023) | (U)(1023 - (lane * VPL + i));
      sort_network<VPL>([&](int i, int j) {
        const U hi = max(u[i], u[j]);
        u[j] = min(u[i], u[j]);
        u[i] = hi;
      });
    }
  }

  // keep_groups for groups of `span` whole lanes, a power of two of them.
  template <typename Tol>
  LORA_DEV void keep(const RouteParams& p, int lane, int span, Tol tol, bool* close) {
    U a = u[0], b = VPL > 1 ? u[VPL > 1 ? 1 : 0] : (U)0;
    for (int o = 1; o < span; o <<= 1) {
      const U c = __shfl_xor_sync(0xffffffffu, a, o), d = __shfl_xor_sync(0xffffffffu, b, o);
      b = max(min(a, c), max(b, d));
      a = max(a, c);
    }
    // every lane of a group has its score: to the lane of the group's number
    const U score = __shfl_sync(0xffffffffu, group_score_of(p, a, b), (lane * span) & 31);
    const uint32_t magnitude = Tol::kExact ? 0u : max(magnitude_of(a), magnitude_of(b));
    const uint32_t kept = best_groups(p, lane, score, magnitude, tol, close);
    if (!((kept >> (lane / span)) & 1u)) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) u[i] = 0;
    }
  }

  // One round: the largest key left and the lane that gives it up (its place, with
  // kAt, in *place).
  LORA_DEV U round(int lane, int* from, int* place) {
    const U m = warp_max(u[0]);
    bool mine = u[0] == m;
    if (kPlace != kExpert) {
      *from = __ffs((int)__ballot_sync(0xffffffffu, mine)) - 1;
      mine = lane == *from;
      if (kAt) *place = __shfl_sync(0xffffffffu, at[0], *from);
    }
    if (mine) {
#pragma unroll
      for (int i = 0; i + 1 < VPL; ++i) {
        u[i] = u[i + 1];
        if (kAt) at[kAt ? i : 0] = at[kAt ? i + 1 : 0];
      }
      u[VPL - 1] = 0;
    }
    return m;
  }
  LORA_DEV int expert(U key, int from, int place) const {
    if (!is_open(key)) return -1;
    if (kAt) return from * VPL + place;
    if (kPlace == kLow) return from * VPL + 7 - (int)((uint32_t)key & 7u);
    return 1023 - (int)((uint32_t)key & 1023u);
  }

  // take_best: lane j notes the j-th key and the lane it came from.  Where
  // neighbours in that order come too close, the next ones are taken too until one
  // is clear of the last, and `exact` (of a lane's expert) ranks them all; *close
  // if 32 lanes do not hold them.
  template <typename Tol, typename ExactKey>
  LORA_DEV int take(const RouteParams& p, int lane, Tol tol, bool* close, ExactKey exact) {
    U key = 0;
    int from = 0, place = 0;
    int rounds = p.top_k + (Tol::kExact || p.top_k == 32 ? 0 : 1);
    for (int j = 0; j < rounds; ++j) {
      int f = 0, a = 0;
      const U m = round(lane, &f, &a);
      if (lane == j) {
        key = m;
        from = f;
        place = a;
      }
    }
    int id = expert(key, from, place);
    if (!Tol::kExact) {
      const U before = __shfl_up_sync(0xffffffffu, key, 1);
      const bool near = lane > 0 && lane < rounds && id >= 0 &&
                        value_of(before) - value_of(key) <= tol(value_of(before));
      if (__any_sync(0xffffffffu, near)) {
        U last = __shfl_sync(0xffffffffu, key, rounds - 1);
        while (true) {
          const U next = warp_max(u[0]);
          if (!is_open(next) || value_of(last) - value_of(next) > tol(value_of(last))) break;
          if (rounds == 32) {
            *close = true;
            break;
          }
          int f = 0, a = 0;
          last = round(lane, &f, &a);
          if (lane == rounds) id = expert(last, f, a);
          ++rounds;
        }
        if (!*close) {
          const auto mine = exact(id);
          int rank = 0;
          for (int j = 0; j < rounds; ++j) {
            const auto other = __shfl_sync(0xffffffffu, mine, j);
            const int e = __shfl_sync(0xffffffffu, id, j);
            rank += e >= 0 && (other > mine || (other == mine && e < id)) ? 1 : 0;
          }
          if (id < 0 || lane >= rounds) rank = 32;
          int sorted = -1;
          for (int j = 0; j < p.top_k; ++j) {
            const uint32_t who = __ballot_sync(0xffffffffu, rank == j);
            const int e = __shfl_sync(0xffffffffu, id, who != 0 ? __ffs((int)who) - 1 : 0);
            if (lane == j && who != 0) sorted = e;
          }
          id = sorted;
        }
      } else if (p.top_k == 32) {
        // no lane for the best one left
        const U next = warp_max(u[0]), last = __shfl_sync(0xffffffffu, key, 31);
        if (is_open(next) && value_of(last) - value_of(next) <= tol(value_of(last))) *close = true;
      }
    }
    return lane < p.top_k ? id : -1;
  }
};

// The exact key of expert e of a row, for a few experts whose fp32 keys are close:
// every lane its own e (or -1), the whole warp together.
template <int VPL, typename LT>
__device__ __noinline__ double exact_key(const RouteParams& p, const LT* row, int lane, int e);

// Lanes per expert group where groups are whole lanes, a power of two of them;
// else 0.
template <int VPL>
LORA_DEV int group_span(const RouteParams& p) {
  if (p.num_groups == 1) return 1;
  const int n = p.E / p.num_groups;
  const int span = n / VPL;
  return n % VPL == 0 && (span & (span - 1)) == 0 ? span : 0;
}

// The selection by keys s + bias, in V.
template <int VPL, typename V, Place kPlace, typename Tol, typename ExactKey>
LORA_DEV int select_by_score(const RouteParams& p, int lane, int span, const float (&x)[VPL],
                             const V (&s)[VPL], const float (&bias)[VPL], bool finite, Tol tol,
                             bool* close, ExactKey exact) {
  if (VPL <= 8 && span > 0) {
    Sorted<VPL, V, kPlace> k;
    make_keys<VPL, V>(x, s, bias, finite, k.u);
    k.sort(lane);
    if (p.num_groups > 1) k.keep(p, lane, span, tol, close);
    if (*close) return -1;
    return k.take(p, lane, tol, close, exact);
  }
  typename KeyOf<V>::U u[VPL];
  make_keys<VPL, V>(x, s, bias, finite, u);
  if (p.num_groups > 1) keep_groups(p, lane, u, tol, close);
  return take_best(p, lane, u, tol, close);
}

struct NoKey {
  LORA_DEV double operator()(int) const { return 0.0; }
};

template <int VPL, typename LT>
__device__ __noinline__ double exact_key(const RouteParams& p, const LT* row, int lane, int e) {
  const double x = e >= 0 ? (double)to_f32(row[e]) : 0.0;
  const double b = e >= 0 && p.bias != nullptr ? (double)__ldg(p.bias + e) : 0.0;
  if (p.score == LORA_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-x)) + b;
  float v[VPL];
  bool bad = false;
  load_row<VPL, LT>(row, lane, p.E, v);
  mask_row<VPL>(v, lane * VPL >= p.E, &bad);
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) m = fmaxf(m, v[i]);
  m = value_of(warp_max(order_of(m)));   // finite: there are keys to compare
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) sum += exp((double)v[i] - (double)m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return exp(x - (double)m) / sum + b;
}

// The same selection in 64 bits, for the tokens whose fp32 keys come too close to
// tell apart.
template <int VPL, typename LT>
__device__ __noinline__ int select_in_double(const RouteParams& p, const LT* row, int lane) {
  float x[VPL], bias[VPL];
  double s[VPL];
  bool bad = false, close = false;
  load_row<VPL, LT>(row, lane, p.E, x);
  const bool finite = mask_row<VPL>(x, lane * VPL >= p.E, &bad);
  load_bias<VPL>(p, lane, bias, &bad);
  if (__all_sync(0xffffffffu, one_bias<VPL>(p, bias, lane * VPL))) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      s[i] = (double)x[i];
      bias[i] = 0.0f;
    }
  } else {
    scores<VPL, double>(p, x, s);
  }
  return select_by_score<VPL, double, kBeside>(p, lane, group_span<VPL>(p), x, s, bias, finite,
                                               Exact(), &close, NoKey());
}

// One warp per token.  Without a bias (and without pair scores of groups) the order
// of the scores is the order of the logits, so the logits themselves are the keys and
// the choice is exact.  Else the keys are fp32 scores plus bias; where two that decide
// the outcome lie within their error bound they are compared in 64 bits (the filter),
// or by their logits where all have one bias, so that the chosen experts are those of
// keys in 64 bits.  Bound by its instructions (about 950 a token with groups and a bias,
// 48 of them loads and stores of spilled registers: the 64-bit calls within the loop
// keep a token's state across them; issued in 69 % of the cycles; 16384 tokens of 256
// experts: 23.2 us, of which the rounds 6, the groups 5 and the close calls 1.3;
// without groups and bias, 2048 of 128: 2.7 us).
template <int VPL, typename LT>
__global__ void __launch_bounds__(256, VPL <= 8 ? 4 : VPL <= 16 ? 3 : 2) route_kernel(const __grid_constant__ RouteParams p) {
  const int lane = threadIdx.x & 31;
  const int warps = (int)(blockDim.x >> 5);
  const bool by_score =
      p.bias != nullptr || (p.num_groups > 1 && p.group_score == LORA_GROUP_TOP_PAIR);
  const int span = group_span<VPL>(p);
  bool bad = false;
  float bias[VPL];
  if (by_score) load_bias<VPL>(p, lane, bias, &bad);
  for (long long t = (long long)blockIdx.x * warps + (threadIdx.x >> 5); t < p.T;
       t += (long long)gridDim.x * warps) {
    const LT* row = reinterpret_cast<const LT*>(p.logits) + (size_t)t * p.E;
    float x[VPL];
    bool close = false;
    load_row<VPL, LT>(row, lane, p.E, x);
    const bool finite = mask_row<VPL>(x, lane * VPL >= p.E, &bad);
    int id;
    if (by_score) {
      float s[VPL];
      const float smax = scores<VPL, float>(p, x, s);
      id = select_by_score<VPL, float, kLow>(p, lane, span, x, s, bias, finite,
                                             key_error<VPL>(p, smax), &close, [&](int e) {
                                               if (__all_sync(0xffffffffu, one_bias<VPL>(p, bias, lane * VPL)))
                                                 return e >= 0 ? (double)to_f32(row[e]) : 0.0;
                                               return exact_key<VPL, LT>(p, row, lane, e);
                                             });
      if (close) id = select_in_double<VPL, LT>(p, row, lane);
    } else if (VPL <= 8 && span > 0) {
      Sorted<VPL, float, sizeof(LT) == 2 ? kExpert : kBeside> k;
#pragma unroll
      for (int i = 0; i < VPL; ++i) k.u[i] = order_of(x[i]);
      k.sort(lane);
      if (p.num_groups > 1) k.keep(p, lane, span, Exact(), &close);
      id = k.take(p, lane, Exact(), &close, NoKey());
    } else {
      uint32_t u[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) u[i] = order_of(x[i]);
      if (p.num_groups > 1) keep_groups(p, lane, u, Exact(), &close);
      id = take_best(p, lane, u, Exact(), &close);
    }
    // weights: lane j has the j-th choice
    const bool live = id >= 0;
    const float xs = live ? to_f32(row[id]) : -INFINITY;
    float w;
    if (p.renormalize) {
      const uint32_t mu = warp_max(order_of(xs));
      const float top = is_open(mu) ? value_of(mu) : 0.0f;
      w = live ? weight_of(p, xs, top) : 0.0f;
      float sum = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      w = live ? w / sum : 0.0f;
    } else if (p.score == LORA_SCORE_SOFTMAX) {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i) m = fmaxf(m, x[i]);
      const uint32_t mu = warp_max(order_of(m));
      m = is_open(mu) ? value_of(mu) : 0.0f;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum += expf(x[i] - m);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      w = live ? weight_of(p, xs, m) / sum : 0.0f;
    } else {
      w = live ? weight_of(p, xs, 0.0f) : 0.0f;
    }
    if (lane < p.top_k) {
      const size_t o = (size_t)t * p.top_k + lane;
      p.ids[o] = id;
      p.weights[o] = w * p.scale;
    }
  }
  if (p.flags != nullptr && __any_sync(0xffffffffu, bad) && lane == 0)
    raise_flag(p.flags, LORA_FLAG_NONFINITE);
}

// Few experts (E <= EM <= 32), no groups, many tokens: a thread per token, its row in
// registers.  The same keys and the same filter; the choices as five bits each.
// 500000 tokens of 8 experts 12.8 us against 152.6 with a warp each, 262144 of 16 with
// a bias 26.5 against 117.6.  A thread's time grows with its row and its choices and a
// few tokens leave SMs idle, so it is used from 16384 tokens on and from
// 16 EM E (top_k + 1) (us with a thread and with a warp each, sigmoid and a bias, the
// slowest kind; softmax without one turns at half as many tokens):
//   8 experts, 8 of them:  16384 tokens 10.3 and 10.4, 32768 10.7 and 18.4
//   16, 4:    16384 9.4 and 8.7, 32768 10.4 and 15.5
//   16, 12:   16384 18.7 and 12.0, 32768 19.5 and 21.8, 65536 23.7 and 40.0
//   32, 1:    16384 10.3 and 7.8, 32768 12.7 and 13.4
//   32, 4:    32768 18.5 and 15.5, 65536 29.2 and 28.5, 262144 83 and 114
//   32, 8:    65536 41 and 33, 262144 122 and 130
//   32, 12:   262144 165 and 149, 524288 311 and 293: a warp
constexpr int kThreadTokens = 16384;
constexpr int kThreadTopK = 12;       // 60 bits

template <int EM>
bool thread_per_token(const RouteParams& p) {   // EM: E rounded up to 8, 16 or 32
  return p.E <= EM && p.num_groups == 1 && p.top_k <= (EM == 32 ? 8 : kThreadTopK) &&
         p.T >= kThreadTokens && p.T >= 16 * EM * p.E * (p.top_k + 1);
}

template <int EM, typename V, typename Tol>
LORA_DEV uint64_t choose_in_thread(int top_k, V (&key)[EM], Tol tol, int* count, bool* close) {
  uint64_t picks = 0;
  V prev = 0;
  int n = 0;
  for (int j = 0; j <= top_k; ++j) {
    V best = -(V)INFINITY;
    int at = -1;
#pragma unroll
    for (int i = 0; i < EM; ++i)
      if (key[i] > best) {   // ties: the lowest
        best = key[i];
        at = i;
      }
    if (at < 0) break;
    if (!Tol::kExact && j > 0 && prev - best <= tol(prev)) *close = true;
    if (j == top_k) break;
    prev = best;
    picks |= (uint64_t)at << (5 * j);
    n = j + 1;
#pragma unroll
    for (int i = 0; i < EM; ++i)
      if (i == at) key[i] = -(V)INFINITY;
  }
  *count = n;
  return picks;
}

template <int EM, typename V>
LORA_DEV V scores_in_thread(const RouteParams& p, const float (&x)[EM], V (&s)[EM]) {
  if (p.score == LORA_SCORE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < EM; ++i) s[i] = inverse((V)1 + power(-(V)x[i]));
    return (V)1;
  }
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < EM; ++i) m = fmaxf(m, x[i]);
  if (!(m > -INFINITY)) m = 0.0f;
  V sum = 0;
#pragma unroll
  for (int i = 0; i < EM; ++i) {
    s[i] = power((V)x[i] - (V)m);
    sum += s[i];
  }
  const V inv = inverse(sum);
#pragma unroll
  for (int i = 0; i < EM; ++i) s[i] *= inv;
  return inv;
}

template <int EM, typename LT>
LORA_DEV void load_in_thread(const LT* row, int E, float (&x)[EM], bool* bad) {
#pragma unroll
  for (int i = 0; i < EM; ++i) {
    x[i] = i < E ? to_f32(row[i]) : -INFINITY;
    if (!(x[i] < INFINITY)) {
      x[i] = -INFINITY;
      *bad = true;
    }
  }
}

// Keys s + bias; -inf where logit or bias is masked.
template <int EM, typename V>
LORA_DEV void keys_in_thread(const RouteParams& p, const float (&x)[EM], V (&s)[EM], bool* bad) {
#pragma unroll
  for (int i = 0; i < EM; ++i) {
    float b = i < p.E ? __ldg(p.bias + i) : -INFINITY;
    if (!(b < INFINITY)) {
      b = -INFINITY;
      *bad = true;
    }
    s[i] = x[i] > -INFINITY ? s[i] + (V)b : -(V)INFINITY;
  }
}

template <int EM, typename LT>
__device__ __noinline__ uint64_t choose_in_thread_double(const RouteParams& p, const LT* row, int* count) {
  float x[EM];
  double s[EM];
  bool bad = false, close = false;
  load_in_thread<EM, LT>(row, p.E, x, &bad);
  float bias[EM];
#pragma unroll
  for (int i = 0; i < EM; ++i) bias[i] = i < p.E ? __ldg(p.bias + i) : 0.0f;
  if (one_bias<EM>(p, bias, 0)) {
#pragma unroll
    for (int i = 0; i < EM; ++i) s[i] = (double)x[i];
  } else {
    scores_in_thread<EM, double>(p, x, s);
    keys_in_thread<EM, double>(p, x, s, &bad);
  }
  return choose_in_thread<EM, double>(p.top_k, s, Exact(), count, &close);
}

template <int EM, typename LT>
__global__ void __launch_bounds__(128) route_thread_kernel(const __grid_constant__ RouteParams p) {
  const long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  bool bad = false;
  if (t < p.T) {
    const LT* row = reinterpret_cast<const LT*>(p.logits) + (size_t)t * p.E;
    float x[EM], key[EM];
    load_in_thread<EM, LT>(row, p.E, x, &bad);
    int count = 0;
    bool close = false;
    uint64_t picks;
    if (p.bias != nullptr) {
      const float smax = scores_in_thread<EM, float>(p, x, key);
      const Within tol = key_error<EM>(p, smax);
      keys_in_thread<EM, float>(p, x, key, &bad);
      picks = choose_in_thread<EM, float>(p.top_k, key, tol, &count, &close);
      if (close) picks = choose_in_thread_double<EM, LT>(p, row, &count);
    } else {
#pragma unroll
      for (int i = 0; i < EM; ++i) key[i] = x[i];
      picks = choose_in_thread<EM, float>(p.top_k, key, Exact(), &count, &close);
    }
    float top = -INFINITY, sum = 0.0f;
    if (p.renormalize) {
      for (int j = 0; j < count; ++j) top = fmaxf(top, to_f32(row[(picks >> (5 * j)) & 31]));
    } else if (p.score == LORA_SCORE_SOFTMAX) {
#pragma unroll
      for (int i = 0; i < EM; ++i) top = fmaxf(top, x[i]);
#pragma unroll
      for (int i = 0; i < EM; ++i) sum += expf(x[i] - top);
    }
    if (p.renormalize)
      for (int j = 0; j < count; ++j) sum += weight_of(p, to_f32(row[(picks >> (5 * j)) & 31]), top);
    else if (p.score == LORA_SCORE_SIGMOID)
      sum = 1.0f;
    const size_t o = (size_t)t * p.top_k;
    for (int j = 0; j < p.top_k; ++j) {
      const int id = j < count ? (int)((picks >> (5 * j)) & 31) : -1;
      p.ids[o + j] = id;
      p.weights[o + j] = id >= 0 ? weight_of(p, to_f32(row[id]), top) / sum * p.scale : 0.0f;
    }
  }
  if (p.flags != nullptr && __any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0)
    raise_flag(p.flags, LORA_FLAG_NONFINITE);
}

template <typename LT>
cudaError_t route_typed(const RouteParams& p, cudaStream_t stream) {
  const bool by_thread = p.E <= 8    ? thread_per_token<8>(p)
                         : p.E <= 16 ? thread_per_token<16>(p)
                                     : thread_per_token<32>(p);
  if (by_thread) {
    const unsigned blocks = (unsigned)((p.T + 127LL) / 128);
    if (p.E <= 8) route_thread_kernel<8, LT><<<blocks, 128, 0, stream>>>(p);
    else if (p.E <= 16) route_thread_kernel<16, LT><<<blocks, 128, 0, stream>>>(p);
    else route_thread_kernel<32, LT><<<blocks, 128, 0, stream>>>(p);
    return cudaGetLastError();
  }
  const int warps = 8;
  const int threads = p.T < warps ? 32 * p.T : 32 * warps;
  // several tokens a warp where there are many: the biases are loaded once (16384
  // tokens: 23.2 us with as many blocks as run at once, 25.5 with one more per SM)
  const long long blocks = ((long long)p.T + warps - 1) / warps;
  const unsigned grid = (unsigned)(blocks < 148 * 4 ? blocks : 148 * 4);
  const int per_lane = (p.E + 31) / 32;
  if (per_lane <= 1) route_kernel<1, LT><<<grid, threads, 0, stream>>>(p);
  else if (per_lane <= 2) route_kernel<2, LT><<<grid, threads, 0, stream>>>(p);
  else if (per_lane <= 4) route_kernel<4, LT><<<grid, threads, 0, stream>>>(p);
  else if (per_lane <= 8) route_kernel<8, LT><<<grid, threads, 0, stream>>>(p);
  else if (per_lane <= 16) route_kernel<16, LT><<<grid, threads, 0, stream>>>(p);
  else route_kernel<32, LT><<<grid, threads, 0, stream>>>(p);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Grouping: a stable counting sort of the pairs by expert (bound by latency: 37 x 8
// pairs 4.1 us, 131072 pairs 11.5 us).
// Few pairs: one CTA of NT threads.  Warp w takes the w-th share of the pairs, so
// (warp, position) order is pair order.
//   1. every warp counts its pairs per expert (in its own table: no atomics);
//   2. per expert, a prefix over the warps, then over the experts;
//   3. every warp walks its pairs again and hands out rows.
// ---------------------------------------------------------------------------

LORA_DEV int pair_expert(const GroupParams& p, int i, int end, bool* bad) {
  int e = -1;
  if (i < end) {
    e = __ldg(p.ids + i);
    if (e < -1 || e >= p.E) {
      e = -1;
      *bad = true;
    }
  }
  return e;
}

// Counts a warp's pairs [begin, end) in its table.
LORA_DEV void count_share(const GroupParams& p, int begin, int end, int* mine, bool* bad) {
  const int lane = threadIdx.x & 31;
  for (int e = lane; e < p.E; e += 32) mine[e] = 0;
  __syncwarp();
  for (int i0 = begin; i0 < end; i0 += 128) {
    int e[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) e[q] = pair_expert(p, i0 + 32 * q + lane, end, bad);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (i0 + 32 * q >= end) break;
      const uint32_t same = __match_any_sync(0xffffffffu, e[q]);
      if (e[q] >= 0 && lane == __ffs((int)same) - 1) mine[e[q]] += __popc(same);
      __syncwarp();
    }
  }
}

// Hands out the rows of a warp's pairs, from its table of first rows.
LORA_DEV void place_share(const GroupParams& p, int begin, int end, int* mine) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  for (int i0 = begin; i0 < end; i0 += 128) {
    int e[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) e[q] = pair_expert(p, i0 + 32 * q + lane, end, &bad);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = i0 + 32 * q + lane;
      if (i0 + 32 * q >= end) break;
      const uint32_t same = __match_any_sync(0xffffffffu, e[q]);
      int row = -1;
      if (e[q] >= 0) row = mine[e[q]] + __popc(same & ((1u << lane) - 1u));
      __syncwarp();
      if (e[q] >= 0 && lane == __ffs((int)same) - 1) mine[e[q]] += __popc(same);
      __syncwarp();
      if (i < end) {
        p.pair_row[i] = row;
        if (row >= 0) {
          const int t = i / p.top_k;
          p.row_token[row] = t;
          if (p.row_slot != nullptr) p.row_slot[row] = __ldg(p.token_slot + t);
        }
      }
    }
  }
}

template <int NT>
__global__ void __launch_bounds__(NT) group_small_kernel(const GroupParams p) {
  constexpr int kWarps = NT / 32;
  extern __shared__ int gr_smem[];   // [kWarps][E]
  __shared__ int scratch[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (p.n + NT - 1) / NT * 32;   // whole warps' steps
  const int begin = min(warp * per, p.n), end = min(begin + per, p.n);
  int* mine = gr_smem + warp * p.E;
  bool bad = false;
  count_share(p, begin, end, mine, &bad);
  if (p.flags != nullptr && __any_sync(0xffffffffu, bad) && lane == 0)
    raise_flag(p.flags, LORA_FLAG_BAD_EXPERT);
  __syncthreads();
  int carry = 0;
  for (int e0 = 0; e0 < p.E; e0 += NT) {
    const int e = e0 + (int)threadIdx.x;
    int total = 0;
    if (e < p.E) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const int c = gr_smem[w * p.E + e];
        gr_smem[w * p.E + e] = total;
        total += c;
      }
    }
    int rows = 0;
    const int first = carry + block_inclusive_scan<NT>(total, scratch, &rows) - total;
    carry += rows;
    if (e < p.E) {
      p.expert_offsets[e] = first;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) gr_smem[w * p.E + e] += first;
    }
  }
  if (threadIdx.x == 0) p.expert_offsets[p.E] = carry;
  __syncthreads();
  place_share(p, begin, end, mine);
}

// Many pairs: three launches over all SMs, without a workspace.  pair_row is
// written in full by the last one, so until then run b of the pairs holds its own
// table (pairs per expert, then the rows before it) at its place in pair_row;
// runs are at least E long.
//   1. count: a CTA counts its run per expert;
//   2. scan: one CTA turns the tables into rows before each run and the totals
//      into expert_offsets;
//   3. place: a CTA takes its table, ranks its run and writes the rows.

constexpr int kSmallPairs = 2048;   // one CTA up to here (7.4 us; three launches 7.5 at 4096)
constexpr int kRunThreads = 512;
constexpr int kRunWarps = kRunThreads / 32;

struct Runs {
  int count, length;   // the last run takes the rest
};

LORA_DEV void run_bounds(const GroupParams& p, const Runs& r, int b, int* begin, int* end) {
  *begin = b * r.length;
  *end = b + 1 == r.count ? p.n : (b + 1) * r.length;
}

LORA_DEV void share_of(int begin, int end, int* lo, int* hi) {
  const int warp = threadIdx.x >> 5;
  const int per = ((end - begin + kRunWarps - 1) / kRunWarps + 31) / 32 * 32;
  *lo = min(begin + warp * per, end);
  *hi = min(*lo + per, end);
}

__global__ void __launch_bounds__(kRunThreads) group_count_kernel(const GroupParams p, const Runs r) {
  extern __shared__ int gr_smem[];   // [E]
  grid_dep_launch_dependents();
  const int lane = threadIdx.x & 31;
  int begin, end;
  run_bounds(p, r, (int)blockIdx.x, &begin, &end);
  for (int e = threadIdx.x; e < p.E; e += kRunThreads) gr_smem[e] = 0;
  __syncthreads();
  bool bad = false;
  for (int i = begin + (int)threadIdx.x; i < end; i += kRunThreads) {
    const int e = pair_expert(p, i, end, &bad);
    if (e >= 0) atomicAdd(gr_smem + e, 1);
  }
  if (p.flags != nullptr && __any_sync(0xffffffffu, bad) && lane == 0)
    raise_flag(p.flags, LORA_FLAG_BAD_EXPERT);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kRunThreads) p.pair_row[begin + e] = gr_smem[e];
}

constexpr int kScanThreads = 1024;

__global__ void __launch_bounds__(kScanThreads) group_scan_kernel(const GroupParams p, const Runs r) {
  __shared__ int scratch[kScanThreads / 32];
  __shared__ int part[kScanThreads];
  grid_dep_launch_dependents();
  grid_dep_wait();
  // `parts` threads per expert, each over a share of the runs
  const int parts = kScanThreads / p.E > 0 ? kScanThreads / p.E : 1;   // E <= kScanThreads
  const int per = (r.count + parts - 1) / parts;
  const int e = threadIdx.x % p.E, q = threadIdx.x / p.E;
  const int b0 = min(q * per, r.count), b1 = q < parts ? min(b0 + per, r.count) : b0;
  int sum = 0;
  for (int b = b0; b < b1; b += 8) {
    int t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = b + k < b1 ? p.pair_row[(b + k) * r.length + e] : 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += t[k];
  }
  part[threadIdx.x] = q < parts ? sum : 0;
  __syncthreads();
  // totals per expert, their prefix, and the rows before this thread's share
  int total = 0, before = 0;
  if (threadIdx.x < p.E)
    for (int k = 0; k < parts; ++k) total += part[k * p.E + threadIdx.x];
  int rows = 0;
  const int incl = block_inclusive_scan<kScanThreads>(total, scratch, &rows);
  if (q < parts)
    for (int k = 0; k < q; ++k) before += part[k * p.E + e];
  __syncthreads();
  if (threadIdx.x < p.E) {
    part[threadIdx.x] = incl - total;   // first row of each expert
    p.expert_offsets[threadIdx.x] = incl - total;
  }
  if (threadIdx.x == 0) p.expert_offsets[p.E] = rows;
  __syncthreads();
  int run = part[e] + before;
  for (int b = b0; b < b1; b += 8) {
    int t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = b + k < b1 ? p.pair_row[(b + k) * r.length + e] : 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (b + k < b1) p.pair_row[(b + k) * r.length + e] = run;
      run += t[k];
    }
  }
}

__global__ void __launch_bounds__(kRunThreads) group_place_kernel(const GroupParams p, const Runs r) {
  extern __shared__ int gr_smem[];   // [kRunWarps][E]
  const int warp = threadIdx.x >> 5;
  int begin, end, lo, hi;
  run_bounds(p, r, (int)blockIdx.x, &begin, &end);
  share_of(begin, end, &lo, &hi);
  int* mine = gr_smem + warp * p.E;
  bool bad = false;
  count_share(p, lo, hi, mine, &bad);
  grid_dep_wait();   // the tables are there (the pairs are inputs of the whole call)
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kRunThreads) {
    int run = p.pair_row[begin + e];
    for (int w = 0; w < kRunWarps; ++w) {
      const int c = gr_smem[w * p.E + e];
      gr_smem[w * p.E + e] = run;
      run += c;
    }
  }
  __syncthreads();
  place_share(p, lo, hi, mine);
}

template <typename K>
cudaError_t launch_after(K kernel, int grid, int threads, size_t smem, bool overlap,
                         cudaStream_t stream, const GroupParams& p, const Runs& r) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p, r);
}

// ---------------------------------------------------------------------------
// Combine: out[t] = residual[t] + sum_j w[t, j] y[pair_row[t, j]], fp32, in
// order of j, rounded once.  A thread owns eight columns of one token and has the
// loads of eight rows in flight (predicated: with branches around them the
// compiler kept few in flight, 70 us).  Memory bound: top_k rows read and one
// written per token.  8192 tokens of 8 x 2048 bf16 and a residual: 55.9 us, 51.4
// being the bytes at the copy rate (65.9 with one index over all columns, a 64-bit
// division a thread; 57.6 with 256 threads a block).
// ---------------------------------------------------------------------------

template <typename T>
__global__ void __launch_bounds__(128)
combine_kernel(const __grid_constant__ CombineParams p) {
  const int t = (int)(blockIdx.x * blockDim.y + threadIdx.y);
  if (t >= p.T) return;
  const T* y = reinterpret_cast<const T*>(p.y);
  bool bad = false;
  const int c = (int)(blockIdx.y * blockDim.x + threadIdx.x) * 8;
  if (c >= p.F) return;
  float acc[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) acc[q] = 0.0f;
  if (p.residual != nullptr) {
    Raw8<T> r;
    r.load(reinterpret_cast<const T*>(p.residual) + (size_t)t * p.F + c);
    r.get(acc);
  }
  for (int j0 = 0; j0 < p.top_k; j0 += 8) {
    const size_t at = (size_t)t * p.top_k + j0;
    int row[8];
    float w[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      row[q] = j0 + q < p.top_k ? __ldg(p.pair_row + at + q) : -1;
      w[q] = j0 + q < p.top_k ? __ldg(p.weights + at + q) : 0.0f;
    }
    Raw8<T> v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const bool valid = row[q] >= 0 && row[q] < p.rows_cap;
      bad |= !valid && row[q] != -1;
      if (!valid) w[q] = 0.0f;
      v[q].load_if(y + (size_t)(valid ? row[q] : 0) * p.F + c, valid);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float f[8];
      v[q].get(f);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = fmaf(w[q], f[k], acc[k]);
    }
  }
  Raw8<T> o;
  o.set(acc);
  o.store(reinterpret_cast<T*>(p.out) + (size_t)t * p.F + c);
  if (bad && c == 0) raise_flag(p.flags, LORA_FLAG_BAD_ROW);
}

template <typename T>
cudaError_t combine_typed(const CombineParams& p, cudaStream_t stream) {
  const int cols = p.F >> 3;
  const int x = cols < 128 ? cols : 128, rows = 128 / x;
  combine_kernel<T><<<dim3((unsigned)((p.T + rows - 1) / rows), (cols + x - 1) / x), dim3(x, rows), 0, stream>>>(p);
  return cudaGetLastError();
}

template <int NT>
cudaError_t group_small(const GroupParams& p, cudaStream_t stream) {
  group_small_kernel<NT><<<1, NT, (size_t)(NT / 32) * p.E * 4, stream>>>(p);
  return cudaGetLastError();
}

std::mutex g_mu;
bool g_group_attr[64];

}  // namespace

cudaError_t route_launch(const RouteParams& p, int type, cudaStream_t stream) {
  if (type == LORA_TYPE_BF16) return route_typed<__nv_bfloat16>(p, stream);
  if (type == LORA_TYPE_F16) return route_typed<__half>(p, stream);
  return route_typed<float>(p, stream);
}

cudaError_t group_launch(const GroupParams& p, cudaStream_t stream) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_group_attr[dev]) {
      const int smem = kRunWarps * kRouteMaxExperts * 4;   // 64 KB
      err = cudaFuncSetAttribute(group_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (err == cudaSuccess)
        err = cudaFuncSetAttribute(group_small_kernel<512>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (err != cudaSuccess) return err;
      g_group_attr[dev] = true;
    }
  }
  if (p.n <= 512) return group_small<128>(p, stream);
  if (p.n <= kSmallPairs) return group_small<512>(p, stream);
  Runs r;
  // runs of 1024 or (half the tables to scan) 2048: 11.5 us against 13.2 at 131072 pairs
  r.length = p.n > 65536 ? 2048 : 1024;   // at least E
  while (p.n / r.length > 592) r.length *= 2;
  r.count = p.n / r.length;
  err = launch_after(group_count_kernel, r.count, kRunThreads, (size_t)p.E * 4, false, stream, p, r);
  if (err != cudaSuccess) return err;
  err = launch_after(group_scan_kernel, 1, kScanThreads, 0, true, stream, p, r);
  if (err != cudaSuccess) return err;
  return launch_after(group_place_kernel, r.count, kRunThreads, (size_t)kRunWarps * p.E * 4, true,
                      stream, p, r);
}

cudaError_t combine_launch(const CombineParams& p, int type, cudaStream_t stream) {
  if (type == LORA_TYPE_BF16) return combine_typed<__nv_bfloat16>(p, stream);
  if (type == LORA_TYPE_F16) return combine_typed<__half>(p, stream);
  return combine_typed<float>(p, stream);
}

}  // namespace lora
