// Routing of tokens to experts (gemm_route.h): a wave to a token, lane l holding
// experts l, l + 64, ...  Scores, keys and sums are in 64 bits, so that the order of
// experts next to a tie does not depend on how an exponential was rounded.
#include "launch_util.hpp"
#include "mx_thin.hpp"
#include "route_internal.hpp"

namespace gemm_f32_impl {
namespace {

constexpr int kRouteWaves = 4, kRouteThreads = 64 * kRouteWaves;
constexpr int kRor1 = 0x121, kRor2 = 0x122, kRor4 = 0x124, kRor8 = 0x128;

// ---- reductions over a wave, by lane rotations inside rows of 16 lanes -----

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
template <class V, class Op>
__device__ inline V over_wave(V v, Op op) {
  v = op(v, dpp<kRor8>(v));
  v = op(v, dpp<kRor4>(v));
  v = op(v, dpp<kRor2>(v));
  v = op(v, dpp<kRor1>(v));
  return op(op(lane_of(v, 0), lane_of(v, 16)), op(lane_of(v, 32), lane_of(v, 48)));
}
__device__ inline uint32_t wave_max(uint32_t v) {
  return over_wave(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
// Of numbers and NaN: the largest number.
__device__ inline double wave_max(double v) {
  return over_wave(v, [](double a, double b) { return __builtin_fmax(a, b); });
}
__device__ inline double wave_sum(double v) {
  return over_wave(v, [](double a, double b) { return a + b; });
}

constexpr double kLow = -__builtin_inf();

// exp(z - top), where equals of an infinite top are 1.
__device__ inline double exp_below(double z, double top) { return z == top ? 1.0 : exp(z - top); }
__device__ inline double sigmoid(double z) { return 1.0 / (1.0 + exp(-z)); }

// Numbers as integers of the same order; kLowest: -infinity and NaN.  0 is less than all.
constexpr uint64_t kLowest = 1;
__device__ inline uint64_t ordered(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v == 0.0 ? 0.0 : v);  // -0 equals 0
  return v > kLow ? b ^ ((uint64_t)((int64_t)b >> 63) | 1ULL << 63) : kLowest;
}

// A token's logits: experts lane + 64 i, kLow past E.
template <int FMT, int P>
__device__ inline void load_logits(const RouteProblem &p, long long t, int lane, double (&z)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 64 * i;
    z[i] = e < p.E ? (double)load1<FMT>(p.Z, t * p.ldz + e) : kLow;
  }
}

// ---- the forward pass ----------------------------------------------------------

// Bit L g of the result: whether group g is one of the top_groups, L = 64 / (groups,
// or the power of 2 above it).  `key`: this wave's E keys.
__device__ inline unsigned long long kept_groups(const RouteProblem &p, const double *key, int lane,
                                                 int L) {
  const int S = p.E / p.groups, g = lane / L;
  double first = kLow, second = kLow;
  if (g < p.groups)
    for (int i = lane & (L - 1); i < S; i += L) {
      const double v = key[g * S + i];  // no NaN
      second = __builtin_fmax(second, __builtin_fmin(first, v));
      first = __builtin_fmax(first, v);
    }
  for (int d = 1; d < L; d <<= 1) {
    const double f = __shfl_xor(first, d), s = __shfl_xor(second, d);
    second = __builtin_fmax(__builtin_fmin(first, f), __builtin_fmax(second, s));
    first = __builtin_fmax(first, f);
  }
  const bool two = p.group_score == kGroupTop2 && second > kLow;
  const uint64_t mine = ordered(two ? first + second : first);
  int above = 0;
  for (int o = 0; o < p.groups; ++o) {
    const uint64_t other = (uint64_t)lane_of((uint32_t)(mine >> 32), o * L) << 32 |
                           lane_of((uint32_t)mine, o * L);
    above += other > mine || (other == mine && o < g);
  }
  return __ballot(g < p.groups && above < p.top_groups);
}

// P: experts to a lane.  Choosing is `top` times the largest key, by its high word and
// then its low one: 32-bit maxima over the wave.
template <int FMT, int P>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(RouteProblem p) {
  extern __shared__ double keys[];  // [waves][E], where groups are chosen
  const int lane = threadIdx.x & 63, wave = wave_id();
  const long long t = (long long)kRouteWaves * blockIdx.x + wave;
  if (t >= p.T) return;
  const bool softmax = p.score == kSoftmax;
  const bool choose_groups = p.top_groups < p.groups;
  double z[P];  // logits; of sigmoid scores the scores, once the keys are formed
  load_logits<FMT>(p, t, lane, z);
  uint64_t key[P] = {};  // 0: cannot be chosen
  double zmax = kLow, total = 0.0;  // of the softmax over all experts; a NaN only enters `total`
  if (softmax) {
#pragma unroll
    for (int i = 0; i < P; ++i) zmax = __builtin_fmax(zmax, z[i]);
    zmax = wave_max(zmax);
  }
  // The choice: by the scores where a bias or a sum enters, else by the logits.
  const bool by_score = p.bias != nullptr || (choose_groups && p.group_score == kGroupTop2);
  if (softmax && (by_score || !p.renormalize)) {
    double numbers = 0.0;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (64 * i >= p.E) continue;  // uniform
      if (z[i] != z[i]) nan = true;
      else if (lane + 64 * i < p.E) numbers += exp_below(z[i], zmax);
    }
    total = wave_sum(numbers);
    if (by_score) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (64 * i >= p.E) continue;
        const int e = lane + 64 * i;
        const double b = p.bias && e < p.E ? (double)p.bias[e] : 0.0;
        const double v = z[i] > kLow ? exp_below(z[i], zmax) / total + b : kLow;
        key[i] = ordered(v);
        if (choose_groups && e < p.E) keys[wave * p.E + e] = v == v ? v : kLow;
      }
    }
    if (__any(nan)) total = __builtin_nan("");
  }
  if (!softmax || !by_score) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (64 * i >= p.E) continue;
      const int e = lane + 64 * i;
      const double b = p.bias && e < p.E ? (double)p.bias[e] : 0.0;
      const double logit = z[i];
      if (!softmax) z[i] = sigmoid(logit);
      const double v = logit > kLow ? (by_score ? z[i] + b : logit) : kLow;
      key[i] = ordered(v);
      if (choose_groups && e < p.E) keys[wave * p.E + e] = v == v ? v : kLow;
    }
  }
  unsigned long long kept = ~0ULL;
  int L = 64, S = p.E;
  if (choose_groups) {
    S = p.E / p.groups;
    for (int g = 1; g < p.groups; g <<= 1) L >>= 1;
    __builtin_amdgcn_wave_barrier();  // (a wave's LDS operations are in order)
    kept = kept_groups(p, keys + wave * p.E, lane, L);
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 64 * i, group = e < p.E ? e / S : 0;
    // (as a mask: the compiler has lost a conditional assignment here)
    key[i] &= e < p.E ? 0 - (uint64_t)(kept >> (group * L) & 1) : 0;
  }
  int id = 0;            // lane s: choice s,
  double value = 0.0;    // its logit or sigmoid score
  for (int s = 0; s < p.top; ++s) {
    uint32_t high = 0, low = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const uint32_t h = (uint32_t)(key[i] >> 32);
      high = h > high ? h : high;
    }
    high = wave_max(high);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if ((uint32_t)(key[i] >> 32) == high) low = (uint32_t)key[i] > low ? (uint32_t)key[i] : low;
    low = wave_max(low);
    const uint64_t best = (uint64_t)high << 32 | low;
    bool found = false;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (found || 64 * i >= p.E) continue;  // uniform
      const unsigned long long m = __ballot(key[i] == best);
      if (m == 0) continue;
      found = true;
      const int at = __builtin_ctzll(m);
      if (lane == at) key[i] = 0;
      const double v = lane_of(z[i], at);
      if (lane == s) id = 64 * i + at, value = v;
    }
  }
  // Gates.
  const bool mine = lane < p.top;
  double w = mine ? value : 0.0;
  if (softmax) {
    double from = zmax;
    if (p.renormalize) from = wave_max(mine ? value : kLow);
    w = mine && !(value == kLow) ? exp_below(value, from) : 0.0;
  }
  if (p.renormalize) {
    total = wave_sum(w);
    if (total == 0.0) total = 1.0;
  } else if (!softmax) {
    total = 1.0;
  }
  if (mine) {
    p.ids[t * p.top + lane] = id;
    p.gates[t * p.top + lane] = (float)(p.scale * (w / total));
  }
}

// ---- the backward pass -----------------------------------------------------------
// With s the scores, c the scale and d the gates' gradients, summed over the choices of
// an expert:
//   softmax:               dz[e] = c s[e] (d[e] - sum_j d[j] s[j]), for every expert
//   softmax, renormalised: dz[e] = c r[e] (d[e] - sum_j d[j] r[j]), r = s / sum of the chosen s
//   sigmoid:               dz[e] = c s[e] (1 - s[e]) d[e]
//   sigmoid, renormalised: dz[e] = c r[e] (1 - s[e]) (d[e] - sum_j d[j] r[j])
template <int FMT, int P>
__global__ void __launch_bounds__(kRouteThreads) route_backward_kernel(RouteProblem p) {
  const int lane = threadIdx.x & 63;
  const long long t = (long long)kRouteWaves * blockIdx.x + wave_id();
  if (t >= p.T) return;
  const bool softmax = p.score == kSoftmax, all = softmax && !p.renormalize;
  const bool mine = lane < p.top;
  int id = mine ? p.given[t * p.top + lane] : -1;
  if (id >= p.E) id = -1;
  const double d = id >= 0 ? p.scale * (double)p.dgates[t * p.top + lane] : 0.0;
  const double chosen = id >= 0 ? (double)load1<FMT>(p.Z, t * p.ldz + id) : kLow;
  double z[P], zmax = kLow, total = 0.0;
  if (all) {
    load_logits<FMT>(p, t, lane, z);
#pragma unroll
    for (int i = 0; i < P; ++i) zmax = __builtin_fmax(zmax, z[i]);
    zmax = wave_max(zmax);
    double part = 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (z[i] != z[i] || z[i] > kLow) part += exp_below(z[i], zmax);
    total = wave_sum(part);
    if (total == 0.0) total = 1.0;
  } else if (softmax) {
    zmax = wave_max(chosen);
  }
  // r, the choice's share, and what it is multiplied with
  double score = 0.0, r = 0.0;
  if (id >= 0) score = softmax ? (chosen == kLow ? 0.0 : exp_below(chosen, zmax)) : sigmoid(chosen);
  if (!all) total = p.renormalize ? wave_sum(score) : 1.0;
  if (total == 0.0) total = 1.0;
  r = score / total;
  const double mean = all || p.renormalize ? wave_sum(d * r) : 0.0;
  const double slope = softmax ? 1.0 : 1.0 - score;
  const double add = all ? d : r * slope * (d - mean);
  double out[P];
#pragma unroll
  for (int i = 0; i < P; ++i) out[i] = 0.0;
  for (int s = 0; s < p.top; ++s) {
    const int e = (int)lane_of((uint32_t)id, s);
    const double v = lane_of(add, s);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (e == lane + 64 * i) out[i] += v;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 64 * i;
    if (e >= p.E) continue;
    if (all) {
      const double share = z[i] == kLow ? 0.0 : exp_below(z[i], zmax) / total;
      out[i] = share * (out[i] - mean);
    }
    store1<FMT>(p.dZ, t * p.lddz + e, (float)out[i]);
  }
}

template <int FMT, class Launch>
hipError_t by_experts(int E, Launch launch) {
  if (E <= 64) return launch(std::integral_constant<int, 1>{});
  if (E <= 128) return launch(std::integral_constant<int, 2>{});
  if (E <= 256) return launch(std::integral_constant<int, 4>{});
  return launch(std::integral_constant<int, 8>{});
}
template <class Launch>
hipError_t by_format(int format, Launch launch) {
  if (format == kBf16) return launch(std::integral_constant<int, kBf16>{});
  if (format == kF16) return launch(std::integral_constant<int, kF16>{});
  return launch(std::integral_constant<int, kF32>{});
}

}  // namespace

hipError_t launch_route(const RouteProblem &p, hipStream_t s) {
  return by_format(p.format, [&](auto fmt) {
    constexpr int FMT = decltype(fmt)::value;
    return by_experts<FMT>(p.E, [&](auto per) {
      RouteProblem q = p;
      void *args[] = {&q};
      const size_t lds = p.top_groups < p.groups ? sizeof(double) * kRouteWaves * p.E : 0;
      return hipLaunchKernel(reinterpret_cast<const void *>(route_kernel<FMT, decltype(per)::value>),
                             dim3((unsigned)ceil_div(p.T, kRouteWaves)), dim3(kRouteThreads), args,
                             lds, s);
    });
  });
}

hipError_t launch_route_backward(const RouteProblem &p, hipStream_t s) {
  return by_format(p.format, [&](auto fmt) {
    constexpr int FMT = decltype(fmt)::value;
    return by_experts<FMT>(p.E, [&](auto per) {
      return launch_kernel(route_backward_kernel<FMT, decltype(per)::value>,
                           dim3((unsigned)ceil_div(p.T, kRouteWaves)), dim3(kRouteThreads), s, p);
    });
  });
}

}  // namespace gemm_f32_impl
