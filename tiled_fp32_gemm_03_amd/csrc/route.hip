// Routing of tokens to experts (gemm_route.h): LANES lanes to a token, lane l of them
// holding experts l, l + LANES, ...  Scores, keys and sums are in 64 bits, so that the
// order of experts next to a tie does not depend on how an exponential was rounded.
//
// What bounds it is the instructions, half of them the 64-bit exponentials: 16,384
// tokens, 256 experts, sigmoid scores, a bias, 4 of 8 groups, top 8 take 23 to 26 us by box (their 17
// MB of logits 3.3).
#include "launch_util.hpp"
#include "mx_thin.hpp"
#include "route_internal.hpp"

namespace gemm_f32_impl {
namespace {

// Waves of a workgroup (a few, where groups' keys take LDS).
template <int LANES>
constexpr int kRouteWaves = LANES == 64 ? 4 : 2;
constexpr int kRor1 = 0x121, kRor2 = 0x122, kRor4 = 0x124, kRor8 = 0x128;

// ---- reductions over a token's lanes, by lane rotations inside rows of 16 --------

template <int CTRL>
__device__ inline uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ inline double dpp(double v) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, u32x2{dpp<CTRL>(b[0]), dpp<CTRL>(b[1])});
}
__device__ inline uint32_t lane_of(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
__device__ inline double lane_of(double v, int lane) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, u32x2{lane_of(b[0], lane), lane_of(b[1], lane)});
}
template <int LANES, class V, class Op>
__device__ inline V over_token(V v, Op op) {
  v = op(v, dpp<kRor8>(v));
  v = op(v, dpp<kRor4>(v));
  v = op(v, dpp<kRor2>(v));
  v = op(v, dpp<kRor1>(v));
  if constexpr (LANES == 16) return v;
  else return op(op(lane_of(v, 0), lane_of(v, 16)), op(lane_of(v, 32), lane_of(v, 48)));
}
// One instruction; a NaN operand gives the other one.
__device__ inline double max_of(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
template <int LANES>
__device__ inline double token_max(double v) {
  return over_token<LANES>(v, [](double a, double b) { return max_of(a, b); });
}
template <int LANES>
__device__ inline uint32_t token_min(uint32_t v) {
  return over_token<LANES>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int LANES>
__device__ inline double token_sum(double v) {
  return over_token<LANES>(v, [](double a, double b) { return a + b; });
}

constexpr double kLow = -__builtin_inf();

// exp(z - top), where equals of an infinite top are 1.
__device__ inline double exp_below(double z, double top) { return z == top ? 1.0 : exp(z - top); }
__device__ inline double sigmoid(double z) { return 1.0 / (1.0 + exp(-z)); }

// What the choice goes by: numbers as they are, -infinity and NaN as kLowest; less than
// that an expert that is taken (marked in the high word alone), and kLow one that is none.
constexpr double kLowest = -0x1p1023;
constexpr uint32_t kTaken = 0xffefffffu;
__device__ inline double key_of(double v) { return v > kLow ? v : kLowest; }

// A token's logits: experts `sub` + LANES i, kLow past E.
template <int FMT, int P, int LANES>
__device__ inline void load_logits(const RouteProblem &p, long long t, int sub, double (&z)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = sub + LANES * i;
    z[i] = e < p.E ? (double)load1<FMT>(p.Z, t * p.ldz + e) : kLow;
  }
}

// ---- the forward pass ----------------------------------------------------------

// Whether each of the token's groups is one of the top_groups: bit L g, L = LANES / (groups,
// or the power of 2 above it).  `key`: the token's keys, one place free after each group.
template <int LANES>
__device__ inline unsigned long long kept_groups(const RouteProblem &p, const double *key, int lane,
                                                 int L, int S) {
  const int sub = lane & (LANES - 1), g = sub / L;
  double first = kLow, second = kLow;
  if (g < p.groups)
    for (int i = sub & (L - 1); i < S; i += L) {
      const double v = key[g * (S + 1) + i];  // no NaN
      second = max_of(second, v < first ? v : first);
      first = max_of(first, v);
    }
  for (int d = 1; d < L; d <<= 1) {
    const double f = __shfl_xor(first, d), s = __shfl_xor(second, d);
    second = max_of(f < first ? f : first, max_of(second, s));
    first = max_of(first, f);
  }
  // (kLowest: masked experts, which are in no sum)
  const double mine = p.group_score == kGroupTop2 && second > kLowest ? first + second : first;
  int above = 0;
  for (int o = 0; o < p.groups; ++o) {
    const double other = __shfl(mine, (lane & ~(LANES - 1)) + o * L);
    above += other > mine || (other == mine && o < g);
  }
  const unsigned long long kept = __ballot(g < p.groups && above < p.top_groups);
  return LANES == 64 ? kept : kept >> (lane & 48) & 0xffffu;
}

// P: experts to a lane.  Choosing is `top` times the largest key, and of those who have
// it the lowest index.
template <int FMT, int P, int LANES>
__global__ void __launch_bounds__(64 * kRouteWaves<LANES>) route_kernel(RouteProblem p) {
  constexpr int kTokens = kRouteWaves<LANES> * 64 / LANES;
  extern __shared__ double keys[];  // [tokens][E + groups], where groups are chosen
  __shared__ int chosen[kTokens][kRouteMaxTop];
  const int lane = threadIdx.x & 63, sub = lane & (LANES - 1), slot = threadIdx.x / LANES;
  const long long mine = (long long)kTokens * blockIdx.x + slot;
  const bool in = mine < p.T;
  if (__ballot(in) == 0) return;
  const long long t = in ? mine : p.T - 1;  // lanes without a token go along
  const bool softmax = p.score == kSoftmax;
  const bool choose_groups = p.top_groups < p.groups;
  double z[P];
  load_logits<FMT, P, LANES>(p, t, sub, z);
  double key[P];
  double zmax = kLow, total = 0.0;  // of the softmax over all experts; a NaN only enters `total`
  if (softmax) {
#pragma unroll
    for (int i = 0; i < P; ++i) zmax = max_of(zmax, z[i]);
    zmax = token_max<LANES>(zmax);
  }
  // Keys are scores where a bias or a sum enters, else logits.
  const bool by_score = p.bias != nullptr || (choose_groups && p.group_score == kGroupTop2);
  if (softmax && (by_score || !p.renormalize)) {
    double numbers = 0.0;
    uint32_t number = 1;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      key[i] = 0.0;
      if (LANES * i >= p.E) continue;  // uniform
      const bool nan = z[i] != z[i];
      if (nan) number = 0;
      key[i] = nan || sub + LANES * i >= p.E ? 0.0 : exp_below(z[i], zmax);
      numbers += key[i];
    }
    total = token_sum<LANES>(numbers);
    number = token_min<LANES>(number);
#pragma unroll
    for (int i = 0; i < P; ++i) key[i] = key[i] / total;
    if (number == 0) total = __builtin_nan("");
  } else if (!softmax && by_score) {
#pragma unroll
    for (int i = 0; i < P; ++i) key[i] = LANES * i < p.E ? sigmoid(z[i]) : 0.0;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = sub + LANES * i;
    const bool is = e < p.E;
    double v = by_score ? key[i] : z[i];
    if (p.bias && is) v += (double)p.bias[e];
    v = is ? key_of(z[i] > kLow ? v : kLow) : kLow;
    key[i] = v;
  }
  if (choose_groups) {
    const int S = p.E / p.groups;
    const float per = 1.f / (float)S;
    int L = LANES;
    for (int g = 1; g < p.groups; g <<= 1) L >>= 1;
    double *own = keys + slot * (p.E + p.groups);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = sub + LANES * i, g = (int)(((float)e + 0.5f) * per);
      if (e < p.E) own[e + g] = key[i];
    }
    __builtin_amdgcn_wave_barrier();  // (a wave's LDS operations are in order)
    const unsigned long long kept = kept_groups<LANES>(p, own, lane, L, S);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = sub + LANES * i, g = (int)(((float)e + 0.5f) * per);
      const bool stays = e < p.E && (kept >> ((e < p.E ? g : 0) * L) & 1);
      // (without a bias scores are for the groups' sums alone: they may be rounded to 0 or 1)
      const double mine = p.bias ? key[i] : key_of(z[i]);
      key[i] = stays ? mine : kLow;
    }
  }
  for (int s = 0; s < p.top; ++s) {
    double best = key[0];
#pragma unroll
    for (int i = 1; i < P; ++i) best = max_of(best, key[i]);
    best = token_max<LANES>(best);
    uint32_t at = 0xffffu;
#pragma unroll
    for (int i = P - 1; i >= 0; --i) at = key[i] == best ? (uint32_t)i : at;
    const uint32_t e = token_min<LANES>(at * LANES + sub);
    const bool own = (e & (LANES - 1)) == (uint32_t)sub;
    if (own) chosen[slot][s] = (int)e;
    const uint32_t taken = own ? e / LANES : 0xffffu;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      u32x2 b = __builtin_bit_cast(u32x2, key[i]);
      b[1] = taken == (uint32_t)i ? kTaken : b[1];
      key[i] = __builtin_bit_cast(double, b);
    }
  }
  __builtin_amdgcn_wave_barrier();
  // Gates: lane s has choice s.
  const bool has = sub < p.top;
  const int id = has ? chosen[slot][sub] : 0;
  double value = has ? (double)load1<FMT>(p.Z, t * p.ldz + id) : kLow;
  double w;
  if (softmax) {
    const double from = p.renormalize ? token_max<LANES>(value) : zmax;
    w = has && !(value == kLow) ? exp_below(value, from) : 0.0;
  } else {
    w = has ? sigmoid(value) : 0.0;
  }
  if (p.renormalize) {
    total = token_sum<LANES>(w);
    if (total == 0.0) total = 1.0;
  } else if (!softmax) {
    total = 1.0;
  }
  if (has && in) {
    p.ids[t * p.top + sub] = id;
    p.gates[t * p.top + sub] = (float)(p.scale * (w / total));
  }
}

// ---- the backward pass -----------------------------------------------------------
// With s the scores, c the scale and d the gates' gradients, summed over the choices of
// an expert:
//   softmax:               dz[e] = c s[e] (d[e] - sum_j d[j] s[j]), for every expert
//   softmax, renormalised: dz[e] = c r[e] (d[e] - sum_j d[j] r[j]), r = s / sum of the chosen s
//   sigmoid:               dz[e] = c s[e] (1 - s[e]) d[e]
//   sigmoid, renormalised: dz[e] = c r[e] (1 - s[e]) (d[e] - sum_j d[j] r[j])
// A share near 1 leaves little of its difference: with a logit 30 above the others it was
// off by 3e-4, from 37 on 0.  So 1 - s is 1 / (1 + exp(z)), and tokens with a share above
// kNear form, over the other choices j (softmax: over other experts, `rest` the share of
// those not chosen),
//   d[e] - sum_j d[j] r[j] = sum_j r[j] (d[e] - d[j]) + rest d[e]
// (for all tokens, 4,097 on 6 of 63 experts, 7.8 us instead of 5.8).
constexpr double kNear = 1.0 - 0x1p-8;
template <int FMT, int P>
__global__ void __launch_bounds__(64 * kRouteWaves<64>) route_backward_kernel(RouteProblem p) {
  const int lane = threadIdx.x & 63;
  const long long t = (long long)kRouteWaves<64> * blockIdx.x + wave_id();
  if (t >= p.T) return;
  const bool softmax = p.score == kSoftmax, all = softmax && !p.renormalize;
  const bool mine = lane < p.top;
  int id = mine ? p.given[t * p.top + lane] : -1;
  if (id < 0 || id >= p.E) id = -1;
  const double d = id >= 0 ? p.scale * (double)p.dgates[t * p.top + lane] : 0.0;
  const double chosen = id >= 0 ? (double)load1<FMT>(p.Z, t * p.ldz + id) : kLow;
  double z[P], zmax = kLow, total = 0.0;
  if (all) {
    load_logits<FMT, P, 64>(p, t, lane, z);
#pragma unroll
    for (int i = 0; i < P; ++i) zmax = max_of(zmax, z[i]);
    zmax = token_max<64>(zmax);
    double part = 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      z[i] = z[i] == kLow ? 0.0 : exp_below(z[i], zmax);  // the share, over the total
      part += z[i];
    }
    total = token_sum<64>(part);
  } else if (softmax) {
    zmax = token_max<64>(chosen);
  }
  double score = 0.0;
  if (id >= 0) score = softmax ? (chosen == kLow ? 0.0 : exp_below(chosen, zmax)) : sigmoid(chosen);
  if (!all) total = p.renormalize ? token_sum<64>(score) : 1.0;
  if (total == 0.0) total = 1.0;
  const double r = id >= 0 ? score / total : 0.0;
  const double slope = softmax ? 1.0 : sigmoid(-chosen);
  const bool near = __ballot((all || p.renormalize) && r > kNear) != 0;  // uniform
  double add, mean = 0.0;
  unsigned own = 0;  // bit i: `add` is all of the gradient of expert lane + 64 i
  int of = id;       // -1 where an earlier choice is of the same expert and has its sum
  if (!near) {
    if (all || p.renormalize) mean = token_sum<64>(d * r);
    add = all ? d : r * slope * (d - mean);
  } else {
    double sum = d, rest = 0.0;
    if (all) {
      sum = 0.0;
      for (int s = 0; s < p.top; ++s) {
        const int e = (int)lane_of((uint32_t)id, s);
        const double v = lane_of(d, s);
        if (e == id) sum += v;
        if (e == id && s < lane) of = -1;
#pragma unroll
        for (int i = 0; i < P; ++i)
          if (e == lane + 64 * i) own |= 1u << i;
      }
#pragma unroll
      for (int i = 0; i < P; ++i) rest += own >> i & 1 ? 0.0 : z[i];
      rest = token_sum<64>(rest) / total;
      mean = token_sum<64>(of >= 0 ? sum * r : 0.0);
    }
    add = rest > 0.0 ? rest * sum : 0.0;
    const double share = of >= 0 ? r : 0.0;
    for (int s = 0; s < p.top; ++s)
      if ((int)lane_of((uint32_t)of, s) >= 0 && s != lane)
        add += lane_of(share, s) * (sum - lane_of(sum, s));
    add *= share * slope;
  }
  double out[P];
#pragma unroll
  for (int i = 0; i < P; ++i) out[i] = 0.0;
  for (int s = 0; s < p.top; ++s) {
    const int e = (int)lane_of((uint32_t)of, s);
    const double v = lane_of(add, s);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (e == lane + 64 * i) out[i] += v;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 64 * i;
    if (e >= p.E) continue;
    if (all && !(own >> i & 1)) out[i] = z[i] / total * (out[i] - mean);
    store1<FMT>(p.dZ, t * p.lddz + e, (float)out[i]);
  }
}

template <int LANES, class Launch>
hipError_t by_experts(int E, Launch launch) {
  if (E <= LANES) return launch(std::integral_constant<int, 1>{});
  if (E <= 2 * LANES) return launch(std::integral_constant<int, 2>{});
  if (E <= 4 * LANES) return launch(std::integral_constant<int, 4>{});
  if (E <= 8 * LANES) return launch(std::integral_constant<int, 8>{});
  if constexpr (LANES == 16) return launch(std::integral_constant<int, 16>{});
  return hipErrorInvalidValue;  // (E is at most 256 with 16 lanes, 512 with 64)
}
template <class Launch>
hipError_t by_format(int format, Launch launch) {
  if (format == kBf16) return launch(std::integral_constant<int, kBf16>{});
  if (format == kF16) return launch(std::integral_constant<int, kF16>{});
  return launch(std::integral_constant<int, kF32>{});
}

template <int LANES>
hipError_t launch_lanes(const RouteProblem &p, hipStream_t s) {
  return by_format(p.format, [&](auto fmt) {
    constexpr int FMT = decltype(fmt)::value;
    return by_experts<LANES>(p.E, [&](auto per) {
      constexpr int kTokens = kRouteWaves<LANES> * 64 / LANES;
      RouteProblem q = p;
      void *args[] = {&q};
      const size_t lds = p.top_groups < p.groups ? sizeof(double) * kTokens * (p.E + p.groups) : 0;
      return hipLaunchKernel(
          reinterpret_cast<const void *>(route_kernel<FMT, decltype(per)::value, LANES>),
          dim3((unsigned)ceil_div(p.T, kTokens)), dim3(64 * kRouteWaves<LANES>), args, lds, s);
    });
  });
}

}  // namespace

hipError_t launch_route(const RouteProblem &p, hipStream_t s) {
  // A quarter of the waves, each with four times the chain, where tokens are many to an
  // expert.  16 and 64 lanes, us: 16,384 tokens on 64 experts 4.9 and 12.8, on 256 (as
  // above) 22.9 and 29.5, on 500 74 and 55; 4,097 on 63 4.3 and 6.3, 4,096 on 256 16.3
  // and 10.6; one on 256 13.5 and 6.6.
  if (p.groups <= 16 && p.E <= 256 && p.T >= 1024 && p.T >= 40 * p.E)
    return launch_lanes<16>(p, s);
  return launch_lanes<64>(p, s);
}

hipError_t launch_route_backward(const RouteProblem &p, hipStream_t s) {
  return by_format(p.format, [&](auto fmt) {
    constexpr int FMT = decltype(fmt)::value;
    return by_experts<64>(p.E, [&](auto per) {
      return launch_kernel(route_backward_kernel<FMT, decltype(per)::value>,
                           dim3((unsigned)ceil_div(p.T, kRouteWaves<64>)),
                           dim3(64 * kRouteWaves<64>), s, p);
    });
  });
}

}  // namespace gemm_f32_impl
