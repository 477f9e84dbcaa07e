// The mixture-of-experts layer for a few tokens (gemm_moe.h): the router's
// logits, the choice of experts, and the two products over the chosen
// experts' weights.  The products read each chosen expert's weights once,
// straight into the matrix instructions' operands (mx_thin.hpp); the tokens
// of one expert share them, 16 rows at a time.  Three launches for up to 8
// tokens (the choice is made again by each workgroup of the first product),
// four for more.
#include "mx_internal.hpp"
#include "mx_thin.hpp"

namespace gemm_f32_impl {
namespace {

template <class T>
__device__ inline T *ws_at(const MoeProblem &p, long long off) {
  return reinterpret_cast<T *>(p.ws + off);
}

// ---- reductions over a wave, by lane rotations inside rows of 16 lanes -----

template <int CTRL>
__device__ inline double dpp_f64(double v) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(
      double, u32x2{(uint32_t)__builtin_amdgcn_update_dpp(0, (int)b[0], CTRL, 0xf, 0xf, false),
                    (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b[1], CTRL, 0xf, 0xf, false)});
}
__device__ inline double lane_f64(double v, int lane) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double,
                            u32x2{(uint32_t)__builtin_amdgcn_readlane((int)b[0], lane),
                                  (uint32_t)__builtin_amdgcn_readlane((int)b[1], lane)});
}
constexpr int kRor1 = 0x121, kRor2 = 0x122, kRor4 = 0x124, kRor8 = 0x128;
__device__ inline double wave_max(double v) {
  v = __builtin_fmax(v, dpp_f64<kRor8>(v));
  v = __builtin_fmax(v, dpp_f64<kRor4>(v));
  v = __builtin_fmax(v, dpp_f64<kRor2>(v));
  v = __builtin_fmax(v, dpp_f64<kRor1>(v));
  return __builtin_fmax(__builtin_fmax(lane_f64(v, 0), lane_f64(v, 16)),
                        __builtin_fmax(lane_f64(v, 32), lane_f64(v, 48)));
}
__device__ inline double wave_sum(double v) {
  v += dpp_f64<kRor8>(v);
  v += dpp_f64<kRor4>(v);
  v += dpp_f64<kRor2>(v);
  v += dpp_f64<kRor1>(v);
  return (lane_f64(v, 0) + lane_f64(v, 16)) + (lane_f64(v, 32) + lane_f64(v, 48));
}

// ---- router logits -------------------------------------------------------
// A wave takes one expert and TB tokens; a lane 8 consecutive h of each 512.
// Products and sums in 64 bits, so that the order of experts next to a tie
// does not depend on the order of the sum.

template <int FMT, int TB>
__global__ void __launch_bounds__(256) moe_logits_kernel(MoeProblem p) {
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int e = 4 * blockIdx.x + wave;
  if (e >= p.E) return;
  const int t0 = TB * blockIdx.y;
  double acc[TB] = {};
  const uint16_t *row = p.R + e * p.ldr, *x[TB];
#pragma unroll
  for (int i = 0; i < TB; ++i) x[i] = p.X + (t0 + i < p.T ? t0 + i : p.T - 1) * p.ldx;
  auto add = [&](const u32x4 &rw, const u32x4 (&xw)[TB]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double r = to_f32<FMT>((uint16_t)(rw[j >> 1] >> (16 * (j & 1))));
#pragma unroll
      for (int i = 0; i < TB; ++i)
        acc[i] = fma(r, (double)to_f32<FMT>((uint16_t)(xw[i][j >> 1] >> (16 * (j & 1)))), acc[i]);
    }
  };
  const int whole = p.H & ~511;
#pragma unroll 4
  for (int h = 8 * lane; h < whole; h += 512) {
    u32x4 xw[TB];
    const u32x4 rw = *reinterpret_cast<const u32x4h *>(row + h);
#pragma unroll
    for (int i = 0; i < TB; ++i) xw[i] = *reinterpret_cast<const u32x4h *>(x[i] + h);
    add(rw, xw);
  }
  if (whole + 8 * lane < p.H) {
    const int h = whole + 8 * lane;
    u32x4 xw[TB];
    const u32x4 rw = load_guarded(reinterpret_cast<const unsigned char *>(row), h, p.H - h);
#pragma unroll
    for (int i = 0; i < TB; ++i)
      xw[i] = load_guarded(reinterpret_cast<const unsigned char *>(x[i]), h, p.H - h);
    add(rw, xw);
  }
#pragma unroll
  for (int i = 0; i < TB; ++i) {
    const double v = wave_sum(acc[i]);
    if (lane == 0 && t0 + i < p.T) ws_at<double>(p, p.at.logits)[(t0 + i) * p.E + e] = v;
  }
}

// ---- the choice of experts --------------------------------------------------
// A wave takes a token: `top` times the largest logit not yet taken (ties to
// the lower index; a NaN counts as -infinity), then the gates.  Then the
// pairs (token, choice) are listed by expert: ranks inside 64 pairs by
// ballots, added to the counts of the 64-pair chunks before.

constexpr int kPerLane = kMoeMaxExperts / 64;
constexpr int kFusedTokens = 8;

template <int MAX_PAIRS>
struct Route {
  float gate[MAX_PAIRS];               // by pair
  unsigned short chosen[MAX_PAIRS];    // by pair
  unsigned short list[MAX_PAIRS];      // pairs by expert
  unsigned short count[(MAX_PAIRS + 63) / 64][kMoeMaxExperts];
  unsigned short start[kMoeMaxExperts + 1];
  unsigned short ufirst[kMoeMaxExperts];
  unsigned short active[kMoeMaxExperts];
  int nactive;
};

template <int MAX_PAIRS>
__device__ inline void choose_experts(const MoeProblem &p, Route<MAX_PAIRS> &r, int t) {
  const int lane = threadIdx.x & 63;
  const double *logits = ws_at<double>(p, p.at.logits) + t * p.E;
  const double low = -__builtin_inf();
  double z[kPerLane], key[kPerLane];
  unsigned taken = 0;  // bit i: expert lane + 64 i is taken, or past E
  bool nan = false;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + 64 * i;
    const bool in = e < p.E;
    z[i] = in ? logits[e] : low;
    taken |= in ? 0u : 1u << i;
    nan |= z[i] != z[i];
    key[i] = z[i] != z[i] ? low : z[i];
  }
  int id = 0;          // lane s: choice s,
  double value = 0.0;  // its logit
  for (int s = 0; s < p.top; ++s) {
    double best = low;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (64 * i < p.E && !(taken >> i & 1)) best = __builtin_fmax(best, key[i]);
    best = wave_max(best);
    bool found = false;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      if (found || 64 * i >= p.E) continue;  // uniform
      const unsigned long long m = __ballot(!(taken >> i & 1) && key[i] == best);
      if (m == 0) continue;
      found = true;
      const int at = __builtin_ctzll(m);
      if (lane == at) taken |= 1u << i;
      if (lane == s) id = 64 * i + at, value = best;
    }
  }
  // Gates: a NaN among the logits makes every one NaN.
  const double zmax = lane_f64(value, 0);
  double w = lane < p.top ? exp(value - zmax) : 0.0, part = w;
  if (!p.renormalize) {
    part = 0.0;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (64 * i < p.E) part += lane + 64 * i < p.E ? exp(z[i] - zmax) : 0.0;
  }
  const double total = __any(nan) ? __builtin_nan("") : wave_sum(part);
  if (lane < p.top) {
    r.chosen[t * p.top + lane] = (unsigned short)id;
    r.gate[t * p.top + lane] = (float)(w / total);
  }
}

// Lanes of the wave whose pair has the same expert as this lane's.
__device__ inline unsigned long long same_expert(int e) {
  unsigned long long same = ~0ULL;
#pragma unroll
  for (int b = 0; b < 10; ++b) {
    const unsigned long long m = __ballot((e >> b) & 1);
    same &= (e >> b) & 1 ? m : ~m;
  }
  return same;
}

template <int THREADS, int MAX_PAIRS>
__device__ inline void route_all(const MoeProblem &p, Route<MAX_PAIRS> &r) {
  constexpr int kWaves = THREADS / 64;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int pairs = p.T * p.top, chunks = (pairs + 63) / 64;
  const unsigned long long before = (1ULL << lane) - 1;
  for (int c = 0; c < chunks; ++c)
    for (int e = threadIdx.x; e < p.E; e += THREADS) r.count[c][e] = 0;
  for (int t = wave; t < p.T; t += kWaves) choose_experts(p, r, t);
  __syncthreads();
  for (int c = wave; c < chunks; c += kWaves) {
    const int i = 64 * c + lane, e = i < pairs ? r.chosen[i] : kMoeMaxExperts;
    const unsigned long long same = same_expert(e);
    if (i < pairs && (same & before) == 0) r.count[c][e] = (unsigned short)__popcll(same);
  }
  __syncthreads();
  if (wave == 0) {  // where each expert's pairs begin, and the chosen experts
    int base = 0, ubase = 0, nact = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      const int e = e0 + lane;
      int n = 0;
      if (e < p.E)
        for (int c = 0; c < chunks; ++c) n += r.count[c][e];
      const int u = (n + 3) & ~3;  // rows of u
      int upto = n, uupto = u;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(upto, d), uv = __shfl_up(uupto, d);
        if (lane >= d) upto += v, uupto += uv;
      }
      if (e < p.E) {
        r.start[e] = (unsigned short)(base + upto - n);
        r.ufirst[e] = (unsigned short)(ubase + uupto - u);
      }
      const unsigned long long on = __ballot(n > 0);
      if (n > 0) r.active[nact + __popcll(on & before)] = (unsigned short)e;
      base += __shfl(upto, 63);
      ubase += __shfl(uupto, 63);
      nact += __popcll(on);
    }
    if (lane == 0) {
      r.nactive = nact;
      r.start[p.E] = (unsigned short)pairs;
    }
  }
  __syncthreads();
  for (int c = wave; c < chunks; c += kWaves) {
    const int i = 64 * c + lane, e = i < pairs ? r.chosen[i] : kMoeMaxExperts;
    const unsigned long long same = same_expert(e);
    if (i < pairs) {
      int at = r.start[e] + __popcll(same & before);
      for (int q = 0; q < c; ++q) at += r.count[q][e];
      r.list[at] = (unsigned short)i;
    }
  }
  __syncthreads();
}

// The route in the workspace, for the kernels that follow, and the caller's
// ids and gates.
template <int THREADS, int MAX_PAIRS>
__device__ inline void write_route(const MoeProblem &p, const Route<MAX_PAIRS> &r) {
  const int pairs = p.T * p.top;
  int *list = ws_at<int>(p, p.at.list), *start = ws_at<int>(p, p.at.start);
  int *active = ws_at<int>(p, p.at.active), *ufirst = ws_at<int>(p, p.at.ufirst);
  float *gates = ws_at<float>(p, p.at.gates);
  for (int i = threadIdx.x; i < pairs; i += THREADS) {
    list[i] = r.list[i];
    gates[i] = r.gate[i];
    if (p.ids) p.ids[i] = r.chosen[i];
    if (p.gates) p.gates[i] = r.gate[i];
  }
  for (int e = threadIdx.x; e <= p.E; e += THREADS) start[e] = r.start[e];
  for (int e = threadIdx.x; e < p.E; e += THREADS) ufirst[e] = r.ufirst[e];
  for (int a = threadIdx.x; a < r.nactive; a += THREADS) active[1 + a] = r.active[a];
  if (threadIdx.x == 0) active[0] = r.nactive;
}

constexpr int kRouteThreads = 1024;
__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(MoeProblem p) {
  __shared__ Route<kMoeMaxTokens * kMoeMaxTop> r;
  route_all<kRouteThreads>(p, r);
  write_route<kRouteThreads>(p, r);
}

// ---- first product: u = silu(gate) * other ------------------------------------
// A unit is one chosen expert and 16 of its inner columns, both factors.  `ks`
// waves share a unit, taking the pieces of H in turn: one wave per unit where
// there are units enough to fill the chip, more where there are few.

constexpr int kUpWaves = 4;
typedef f32x4 UpPart[1][2][64];  // [block of rows][factor][lane]

template <int W, int AF, int MB, bool ODD>
__device__ __forceinline__ void moe_up_rows(const MoeProblem &p, const Rows (&w)[2],
                                            const Row (&x)[MB], int ufirst, int n, int i0, int ks,
                                            bool any, UpPart *part) {
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int l16 = lane & 15, g = lane >> 4, kw = wave & (ks - 1);
  bool valid[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) valid[i] = 16 * i + l16 < n;
  Thin<W, AF, MB, 2, ODD> t;
  t.clear();
  if (any) t.run(x, valid, w, kw, ks, p.H, lane);
  if (ks > 1) {
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      part[wave][i][0][lane] = t.acc[i][0];
      part[wave][i][1][lane] = t.acc[i][1];
    }
    __syncthreads();
    if (kw == 0)
      for (int q = 1; q < ks; ++q)
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          t.acc[i][0] += part[wave + q][i][0][lane];
          t.acc[i][1] += part[wave + q][i][1][lane];
        }
    __syncthreads();
  }
  if (kw != 0 || !any) return;
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int m = 16 * i + l16;
    if (m >= n) continue;
    uint16_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = t.acc[i][0][j], b = t.acc[i][1][j];
      const float u = a / (1.f + expf(-a)) * b;
      const float v = i0 + 4 * g + j < p.I ? u : 0.f;  // rows are padded with zeros
      hi[j] = from_f32<kBf16>(v);
      const float h = to_f32<kBf16>(hi[j]);
      lo[j] = mag_bits(h) < 0x7f800000u ? from_f32<kBf16>(v - h) : (uint16_t)0;
    }
    const long long at = split_at<W>(ufirst + m, i0 + 4 * g, p.at.pitch);
    *reinterpret_cast<u32x2 *>(p.ws + p.at.hi + at) =
        u32x2{hi[0] | (uint32_t)hi[1] << 16, hi[2] | (uint32_t)hi[3] << 16};
    *reinterpret_cast<u32x2 *>(p.ws + p.at.lo + at) =
        u32x2{lo[0] | (uint32_t)lo[1] << 16, lo[2] | (uint32_t)lo[3] << 16};
  }
}

// FUSED: at most kFusedTokens tokens, each workgroup makes the choice itself.
template <int W, int AF, bool FUSED, bool ODD>
__global__ void __launch_bounds__(64 * kUpWaves, 3) moe_up_kernel(MoeProblem p, int ks) {
  __shared__ UpPart part[kUpWaves];
  __shared__ Route<FUSED ? kFusedTokens * kMoeMaxTop : 1> route;
  const int wave = wave_id(), l16 = threadIdx.x & 15;
  int e, first, n, ufirst;
  if constexpr (FUSED) {
    route_all<64 * kUpWaves>(p, route);
    if (blockIdx.x == 0 && blockIdx.y == 0) write_route<64 * kUpWaves>(p, route);
    if ((int)blockIdx.y >= route.nactive) return;
    e = __builtin_amdgcn_readfirstlane(route.active[blockIdx.y]);
    first = __builtin_amdgcn_readfirstlane(route.start[e]);
    n = __builtin_amdgcn_readfirstlane(route.start[e + 1]) - first;
    ufirst = __builtin_amdgcn_readfirstlane(route.ufirst[e]);
  } else {
    const int *active = ws_at<int>(p, p.at.active), *start = ws_at<int>(p, p.at.start);
    if ((int)blockIdx.y >= active[0]) return;
    e = active[1 + blockIdx.y];
    first = start[e];
    n = start[e + 1] - first;
    ufirst = ws_at<int>(p, p.at.ufirst)[e];
  }
  const int lane = threadIdx.x & 63;
  const int units = kUpWaves / ks;
  const int i0 = 16 * (int)(blockIdx.x * units + wave / ks);
  const bool any = i0 < p.at.pitch;  // the last workgroup may have units too many
  auto inner = [&](int r) { return 2LL * p.I * e + (i0 + r < p.I ? i0 + r : p.I - 1); };
  Rows w[2];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const long long r = inner(load_row(lane, t));
    w[0].p[t] = p.W1 + r * p.ld1;
    w[1].p[t] = p.W1 + (r + p.I) * p.ld1;
  }
  if constexpr (W == kMx) {
    w[0].q = p.S1 + inner(l16) * p.lds1;
    w[1].q = p.S1 + (inner(l16) + p.I) * p.lds1;
  }
  for (int m = 0; m < n; m += 16) {
    const int at = first + (m + l16 < n ? m + l16 : n - 1);
    const int pair = FUSED ? (int)route.list[at] : ws_at<int>(p, p.at.list)[at];
    const Row x[1] = {{reinterpret_cast<const unsigned char *>(p.X + pair / p.top * p.ldx), nullptr}};
    moe_up_rows<W, AF, 1, ODD>(p, w, x, ufirst + m, n - m, i0, ks, any, part);
  }
}

// ---- second product and the weighted sum -----------------------------------------
// A workgroup owns 16 columns of Y for all tokens.  The pieces of all chosen
// experts' inner columns, one expert after the other, are dealt to its waves
// in equal runs; a wave loads the next piece's weights while it uses one, and
// adds each piece's rows, times their gates, to a sum of its own in LDS.  The
// waves' sums are added in wave order at the end.

// LDS of the second product: sums [wave][token][16], then the route.
struct DownLds {
  int gates, start, ufirst, active, tokens, bytes;
};
constexpr DownLds down_lds(int waves, int T, int E, int top) {
  const int pairs = T * top;
  const int gates = waves * T * 64, start = gates + 4 * pairs, ufirst = start + 2 * (E + 1),
            active = ufirst + 2 * E, tokens = active + 2 * E;
  return {gates, start, ufirst, active, tokens, tokens + 2 * pairs};
}

template <int W, int WAVES, bool ODD>
__global__ void __launch_bounds__(64 * WAVES, WAVES == 16 ? 4 : 2) moe_down_kernel(MoeProblem p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  constexpr int kThreads = 64 * WAVES;
  const DownLds at = down_lds(WAVES, p.T, p.E, p.top);
  float *gate = reinterpret_cast<float *>(lds + at.gates);  // by place in the list
  unsigned short *start = reinterpret_cast<unsigned short *>(lds + at.start);
  unsigned short *ufirst = reinterpret_cast<unsigned short *>(lds + at.ufirst);
  unsigned short *active = reinterpret_cast<unsigned short *>(lds + at.active);
  unsigned short *token = reinterpret_cast<unsigned short *>(lds + at.tokens);  // by place
  const int wave = wave_id(), lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int nact = ws_at<int>(p, p.at.active)[0], pairs = p.T * p.top;
  for (int i = threadIdx.x; i < 4 * p.T * WAVES; i += kThreads)
    reinterpret_cast<f32x4 *>(lds)[i] = f32x4{0, 0, 0, 0};
  for (int i = threadIdx.x; i < pairs; i += kThreads) {
    const int pair = ws_at<int>(p, p.at.list)[i];
    gate[i] = ws_at<float>(p, p.at.gates)[pair];
    token[i] = (unsigned short)(pair / p.top);
  }
  for (int i = threadIdx.x; i <= p.E; i += kThreads)
    start[i] = (unsigned short)ws_at<int>(p, p.at.start)[i];
  for (int i = threadIdx.x; i < p.E; i += kThreads)
    ufirst[i] = (unsigned short)ws_at<int>(p, p.at.ufirst)[i];
  for (int i = threadIdx.x; i < nact; i += kThreads)
    active[i] = (unsigned short)ws_at<int>(p, p.at.active)[1 + i];
  __syncthreads();

  float *sum = reinterpret_cast<float *>(lds) + wave * 16 * p.T;
  const int n0 = 16 * blockIdx.x, nb = (int)mx_blocks(p.I);
  const int pieces = (int)ceil_div(p.I, kPieceK<W>), whole = p.I / kPieceK<W>;
  const long long all = (long long)nact * pieces;
  const int from = (int)(all * wave / WAVES), to = (int)(all * (wave + 1) / WAVES);
  typedef Thin<W, kSplit, 1, 1, ODD> Product;
#pragma unroll 1
  for (int v = from; v < to; ++v) {
    const int e = __builtin_amdgcn_readfirstlane(active[v / pieces]), piece = v % pieces;
    const int first = __builtin_amdgcn_readfirstlane(start[e]);
    const int last = __builtin_amdgcn_readfirstlane(start[e + 1]);
    auto row = [&](int r) { return (long long)p.H * e + (n0 + r < p.H ? n0 + r : p.H - 1); };
    Rows w[1];
#pragma unroll
    for (int t = 0; t < 4; ++t) w[0].p[t] = p.W2 + row(load_row(lane, t)) * p.ld2;
    if constexpr (W == kMx) w[0].q = p.S2 + row(l16) * p.lds2;
    typename Product::Weights x;
    if (piece < whole) {
      Product::template load_weights<false>(x, w, piece, lane, p.I, nb);
      Product::template turn_weights<false>(x, w, piece, lane, nb);
    } else {
      Product::template load_weights<true>(x, w, piece, lane, p.I, nb);
      Product::template turn_weights<true>(x, w, piece, lane, nb);
    }
    const int u0 = __builtin_amdgcn_readfirstlane(ufirst[e]);
    for (int m0 = first; m0 < last; m0 += 16) {
      const int m = m0 + l16;
      const bool valid[1] = {m < last};
      const long long at_u = split_at<W>(u0 + m - first, 0, p.at.pitch) + 64 * g;
      const Row u[1] = {{p.ws + p.at.hi + at_u, p.ws + p.at.lo + at_u}};
      Product t;
      t.clear();
      t.template use<false>(x, u, valid, piece, lane, p.I, nb);
      if (valid[0]) {
        f32x4 *y = reinterpret_cast<f32x4 *>(sum + 16 * token[m] + 4 * g);
        *y += gate[m] * t.acc[0][0];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 4 * p.T; i += kThreads) {
    const f32x4 *s = reinterpret_cast<const f32x4 *>(lds) + i;
    f32x4 v = s[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += s[w * 4 * p.T];
    const int t = i / 4, n = n0 + 4 * (i % 4);
    store4_fmt(p.y_format, p.Y, t * p.ldy + n, p.H - n < 4 ? p.H - n : 4, v);
  }
}

template <int FMT>
hipError_t launch_logits(const MoeProblem &p, hipStream_t s) {
  const unsigned gx = (unsigned)ceil_div(p.E, 4);
  if (p.T == 1) return launch_kernel(moe_logits_kernel<FMT, 1>, dim3(gx), dim3(256), s, p);
  return launch_kernel(moe_logits_kernel<FMT, 4>, dim3(gx, (unsigned)ceil_div(p.T, 4)), dim3(256),
                       s, p);
}

template <int W, int AF, bool ODD>
hipError_t launch_up(const MoeProblem &p, hipStream_t s) {
  const int pairs = p.T * p.top;
  const long long experts = p.E < pairs ? p.E : pairs, cols = p.at.pitch / 16;
  // Waves per unit: neighbours read neighbouring pieces of the same rows.
  int ks = 1;
  while (ks < kUpWaves && 2 * ks * kPieceK<W> <= p.H) ks *= 2;
  const dim3 grid((unsigned)ceil_div(cols * ks, kUpWaves), (unsigned)experts);
  return launch_kernel(p.T <= kFusedTokens ? moe_up_kernel<W, AF, true, ODD>
                                           : moe_up_kernel<W, AF, false, ODD>,
                       grid, dim3(64 * kUpWaves), s, p, ks);
}

template <int W, int WAVES, bool ODD>
hipError_t launch_down_waves(const MoeProblem &p, hipStream_t s) {
  MoeProblem q = p;
  void *args[] = {&q};
  return hipLaunchKernel(reinterpret_cast<const void *>(moe_down_kernel<W, WAVES, ODD>),
                         dim3((unsigned)ceil_div(p.H, 16)), dim3(64 * WAVES), args,
                         (size_t)down_lds(WAVES, p.T, p.E, p.top).bytes, s);
}
template <int W, bool ODD>
hipError_t launch_down(const MoeProblem &p, hipStream_t s) {
  return p.T <= 64 ? launch_down_waves<W, 16, ODD>(p, s) : launch_down_waves<W, 8, ODD>(p, s);
}

// Whether a product's 16-bit rows are to be read by whole words (Eight<true>):
// some start in the middle of one, and both matrices start on one.
bool odd_rows(const void *a, long long a_pitch, const void *b, long long b_pitch) {
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 3) == 0 &&
         ((a_pitch | b_pitch) & 3) != 0;
}

template <int W, int AF>
hipError_t launch_products(const MoeProblem &p, hipStream_t s) {
  constexpr bool kHalf = W != kMx;
  const hipError_t e = odd_rows(p.X, 2 * p.ldx, kHalf ? p.W1 : nullptr, kHalf ? p.ld1 : 0)
                           ? launch_up<W, AF, true>(p, s)
                           : launch_up<W, AF, false>(p, s);
  if (e != hipSuccess) return e;
  if (kHalf && odd_rows(p.W2, p.ld2, nullptr, 0)) return launch_down<W, kHalf>(p, s);
  return launch_down<W, false>(p, s);
}

}  // namespace

hipError_t launch_moe(const MoeProblem &p, hipStream_t s) {
  const bool bf16 = p.format == kBf16;
  hipError_t e = bf16 ? launch_logits<kBf16>(p, s) : launch_logits<kF16>(p, s);
  if (e != hipSuccess) return e;
  if (p.T > kFusedTokens) {
    e = launch_kernel(moe_route_kernel, dim3(1), dim3(kRouteThreads), s, p);
    if (e != hipSuccess) return e;
  }
  if (p.mx) return bf16 ? launch_products<kMx, kBf16>(p, s) : launch_products<kMx, kF16>(p, s);
  return bf16 ? launch_products<kBf16, kBf16>(p, s) : launch_products<kF16, kF16>(p, s);
}

}  // namespace gemm_f32_impl
