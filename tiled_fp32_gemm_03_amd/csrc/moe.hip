// The mixture-of-experts layer for a few tokens (gemm_moe.h): the router's
// logits, the choice of experts, and the two products over the chosen
// experts' weights.  The products read each chosen expert's weights once,
// straight into the matrix instructions' operands (mx_thin.hpp); the tokens
// of one expert share them, 16 rows at a time.  Four launches for one token
// (logits, first product, second product, sum), one or two more for the choice
// of experts of several.
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
    const u32x4 rw = load_guarded(reinterpret_cast<const unsigned char *>(row), h, p.H);
#pragma unroll
    for (int i = 0; i < TB; ++i)
      xw[i] = load_guarded(reinterpret_cast<const unsigned char *>(x[i]), h, p.H);
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

template <int MAX_PAIRS>
struct Route {
  float gate[MAX_PAIRS];               // by pair
  unsigned short chosen[MAX_PAIRS];    // by pair
  unsigned short list[MAX_PAIRS];      // pairs by expert
  unsigned short count[(MAX_PAIRS + 63) / 64][kMoeMaxExperts];
  unsigned short start[kMoeMaxExperts + 1];
  unsigned short active[kMoeMaxExperts];
  int nactive;
};

// Token t, as number `slot` of `r`.
template <bool GATES, int MAX_PAIRS>
__device__ inline void choose_experts(const MoeProblem &p, Route<MAX_PAIRS> &r, int slot, int t) {
  const int lane = threadIdx.x & 63;
  const double *logits = ws_at<double>(p, p.at.logits) + t * p.E;
  const double low = -__builtin_inf();
  double z[kPerLane], key[kPerLane];
  unsigned taken = 0;  // bit i: expert lane + 64 i is taken, or past E
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + 64 * i;
    const bool in = e < p.E;
    z[i] = in ? logits[e] : low;
    taken |= in ? 0u : 1u << i;
    key[i] = z[i] != z[i] ? low : z[i];
  }
  int id = 0;          // lane s: choice s,
  double value = 0.0;  // its logit (a NaN stays one)
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
      const double logit = lane_f64(z[i], at);
      if (lane == s) id = 64 * i + at, value = logit;
    }
  }
  if (lane < p.top) r.chosen[slot * p.top + lane] = (unsigned short)id;
  if (!GATES) return;
  // Gates: a NaN among the logits that the sum takes makes every one NaN.
  const double zmax = lane_f64(value, 0);
  double w = lane < p.top ? exp(value - zmax) : 0.0, part = w;
  if (!p.renormalize) {
    part = 0.0;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (64 * i < p.E) part += lane + 64 * i < p.E ? exp(z[i] - zmax) : 0.0;
  }
  const double total = wave_sum(part);
  if (lane < p.top) r.gate[slot * p.top + lane] = (float)(w / total);
}

// The lists of chosen pairs, from r.chosen.
template <int THREADS, int MAX_PAIRS>
__device__ inline void list_pairs(const MoeProblem &p, Route<MAX_PAIRS> &r) {
  constexpr int kWaves = THREADS / 64;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int pairs = p.T * p.top, chunks = (pairs + 63) / 64;
  const unsigned long long before = (1ULL << lane) - 1;
  for (int c = 0; c < chunks; ++c)
    for (int e = threadIdx.x; e < p.E; e += THREADS) r.count[c][e] = 0;
  __syncthreads();
  for (int c = wave; c < chunks; c += kWaves) {
    const int i = 64 * c + lane, e = i < pairs ? r.chosen[i] : kMoeMaxExperts;
    const unsigned long long same = same_expert(e);
    if (e < p.E && (same & before) == 0) r.count[c][e] = (unsigned short)__popcll(same);
  }
  __syncthreads();
  if (wave == 0) {  // where each expert's pairs begin, and the chosen experts
    int base = 0, nact = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      const int e = e0 + lane;
      int n = 0;
      if (e < p.E)
        for (int c = 0; c < chunks; ++c) n += r.count[c][e];
      int upto = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
      }
      if (e < p.E) r.start[e] = (unsigned short)(base + upto - n);
      const unsigned long long on = __ballot(n > 0);
      if (n > 0) r.active[nact + __popcll(on & before)] = (unsigned short)e;
      base += __shfl(upto, 63);
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
    if (e < p.E) {  // pair i has an expert
      int at = r.start[e] + __popcll(same & before);
      for (int q = 0; q < c; ++q) at += r.count[q][e];
      r.list[at] = (unsigned short)i;
    }
  }
  __syncthreads();
}

// Chosen experts and gates, to the workspace and the caller.
template <int THREADS, int MAX_PAIRS>
__device__ inline void write_choice(const MoeProblem &p, const Route<MAX_PAIRS> &r, int from,
                                    int to) {
  int *ids = ws_at<int>(p, p.at.ids);
  float *gates = ws_at<float>(p, p.at.gates);
  for (int i = from + threadIdx.x; i < to; i += THREADS) {
    ids[i] = r.chosen[i - from];
    gates[i] = r.gate[i - from];
    if (p.ids) p.ids[i] = r.chosen[i - from];
    if (p.gates) p.gates[i] = r.gate[i - from];
  }
}
// The lists, to the workspace.
template <int THREADS, int MAX_PAIRS>
__device__ inline void write_lists(const MoeProblem &p, const Route<MAX_PAIRS> &r) {
  int *list = ws_at<int>(p, p.at.list), *start = ws_at<int>(p, p.at.start);
  int *active = ws_at<int>(p, p.at.active);
  for (int i = threadIdx.x; i < p.T * p.top; i += THREADS) list[i] = r.list[i];
  for (int e = threadIdx.x; e <= p.E; e += THREADS) start[e] = r.start[e];
  for (int a = threadIdx.x; a < r.nactive; a += THREADS) active[1 + a] = r.active[a];
  if (threadIdx.x == 0) active[0] = r.nactive;
}

// Up to kRouteTokens tokens: choice and lists by one workgroup, a wave to a
// token (6.2 us, in two launches 9.5).  More: the choice, four tokens to a workgroup, then the lists.  (One
// token: the first product's workgroups choose for themselves.)
constexpr int kRouteTokens = 16;
__global__ void __launch_bounds__(64 * kRouteTokens) moe_route_kernel(MoeProblem p) {
  __shared__ Route<kRouteTokens * kMoeMaxTop> r;
  if (wave_id() < p.T) choose_experts<true>(p, r, wave_id(), wave_id());
  __syncthreads();
  write_choice<64 * kRouteTokens>(p, r, 0, p.T * p.top);
  list_pairs<64 * kRouteTokens>(p, r);
  write_lists<64 * kRouteTokens>(p, r);
}
constexpr int kChooseTokens = 4;
__global__ void __launch_bounds__(64 * kChooseTokens) moe_choose_kernel(MoeProblem p) {
  __shared__ Route<kChooseTokens * kMoeMaxTop> r;
  const int t0 = kChooseTokens * blockIdx.x;
  const int last = t0 + kChooseTokens < p.T ? t0 + kChooseTokens : p.T;
  if (t0 + wave_id() < last) choose_experts<true>(p, r, wave_id(), t0 + wave_id());
  __syncthreads();
  write_choice<64 * kChooseTokens>(p, r, t0 * p.top, last * p.top);
}
constexpr int kListThreads = 1024;
// The lists of a choice made before (several tokens): as above, without the pairs
// that have no expert, which come last.
__global__ void __launch_bounds__(kListThreads) moe_given_kernel(MoeProblem p) {
  __shared__ Route<kMoeMaxTokens * kMoeMaxTop> r;
  __shared__ int valid;
  const int pairs = p.T * p.top;
  if (threadIdx.x == 0) valid = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += kListThreads) {
    const int e = p.given_ids[i];
    const bool in = e >= 0 && e < p.E;
    r.chosen[i] = (unsigned short)(in ? e : kMoeMaxExperts);
    if (in) atomicAdd(&valid, 1);
  }
  __syncthreads();
  list_pairs<kListThreads>(p, r);
  if (threadIdx.x == 0) r.start[p.E] = (unsigned short)valid;
  __syncthreads();
  write_lists<kListThreads>(p, r);
}
__global__ void __launch_bounds__(kListThreads) moe_list_kernel(MoeProblem p) {
  __shared__ Route<kMoeMaxTokens * kMoeMaxTop> r;
  for (int i = threadIdx.x; i < p.T * p.top; i += kListThreads)
    r.chosen[i] = (unsigned short)ws_at<int>(p, p.at.ids)[i];
  list_pairs<kListThreads>(p, r);
  write_lists<kListThreads>(p, r);
}

// ---- the two products ---------------------------------------------------------
// A workgroup takes one chosen expert and some groups of 16 columns; `ks` of
// its waves share a group, taking the pieces of K in turn: one where there
// are groups enough to fill the chip, more where there are few.  A wave goes
// through `each` groups, its weights loaded ahead across them.
//
// Memory bounds the first: the chosen experts' weights once, at 4.2 to 4.5 TB/s
// (268 MB of fp16 weights with odd rows 64 us, the same loads alone 59; 285 MB of
// MX weights 64 us, alone 58).  Second ones run at 2.7 to 3.2 TB/s (134 MB of fp16
// weights 50 us, alone 37: 16 rows of 64 bytes at a time; 142 MB of MX weights 44
// us, alone 32): their activations are three terms, of six bytes a value in LDS,
// which leaves a compute unit eight waves.

constexpr int kWaves = 4, kThreads = 64 * kWaves;  // of the first product's workgroups
constexpr int kMostWaves = 8;                      // of the second one's: 4 or 8

// Two workgroups of four waves to a compute unit: one streams while another
// stages its activations.  The LDS that leaves each for its tile, and the most that
// a tile which needs more may take; then the second product's workgroups have
// eight waves, where there are groups for them.
constexpr int kTileLds = 74 * 1024;
constexpr int kMostLds = 140 * 1024, kCuLds = 160 * 1024;

// The number of pair i's expert in a choice made before, or -1.
__device__ inline int given_expert(const MoeProblem &p, int i) {
  const int e = p.given_ids[i];
  return e >= 0 && e < p.E ? e : -1;
}

// What the launch chose: waves, waves per group, groups per wave, the tile's LDS, and the
// most rows that it has room for.
struct MoeShape {
  int waves, ks, each, lds, rows;
  __host__ __device__ int threads() const { return 64 * waves; }
};

// An expert's part in a launch.
struct Expert {
  int e, first, n;  // its number, its first place in the list, its pairs
};
__device__ inline bool expert_of(const MoeProblem &p, int a, Expert &x) {
  if (p.T == 1 && p.given_ids) {
    x = {given_expert(p, a), a, 1};
    return x.e >= 0;
  }
  const int *active = ws_at<int>(p, p.at.active), *start = ws_at<int>(p, p.at.start);
  if (a >= active[0]) return false;
  x.e = active[1 + a];
  x.first = p.T == 1 ? a : start[x.e];  // one token: in the order of the choice
  x.n = p.T == 1 ? 1 : start[x.e + 1] - x.first;
  return true;
}

// Columns 16 c .. 16 c + 15 of the product of up to 16 rows, NB factors each,
// for each group c of this wave: `weights(c)` gives the lane's rows,
// `done(c, acc)` takes the sums of the group's first wave.  The weights of two
// pieces are on their way while a third is used.  STAGED: the first tile is in
// LDS, or on its way there, already.
template <int W, int A, int NB, int ROWS, bool STAGED, class RowOf, class WeightsOf, class Done>
__device__ __forceinline__ void expert_columns(unsigned char *lds, RowOf row, int n, int K,
                                               int groups, const MoeShape &sh,
                                               WeightsOf weights, Done done) {
  typedef Thin<W, A, NB, ROWS> Product;
  constexpr int kK = Product::kK;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int ks = sh.ks;
  const Tile tile = tile_of<A>(tile_rows(n), K, ks * kK, kTileLds);
  const bool whole = tile.kc >= K;
  f32x4 *part = reinterpret_cast<f32x4 *>(lds + sh.lds);  // [waves][NB][64], if ks > 1
  const int side = sh.waves / ks;  // groups side by side
  const int c0 = (int)blockIdx.x * side * sh.each + wave / ks, first = wave & (ks - 1);
  // A wave's turns: for each of its groups, pieces first, first + ks, ... (an even
  // number of rounds, and of rounds in a tile, unless it holds all).
  const int pieces = (int)ceil_div(K, kK), need = (int)ceil_div(pieces, ks);
  const int rounds = whole ? need : (need + 1) & ~1;
  const int per = tile.kc / (kK * ks);  // rounds in a tile
  struct Turn {
    int group, round;
  };
  auto step = [&](Turn &t) __attribute__((always_inline)) {
    if (++t.round == rounds) t = {t.group + 1, 0};
  };
  auto piece = [&](const Turn &t) __attribute__((always_inline)) { return first + t.round * ks; };
  typename Product::Weights x[2];
  Row w[NB];
  int at = -1;  // whose group's rows w are
  auto load = [&](typename Product::Weights &x, const Turn &t) __attribute__((always_inline)) {
    if (t.group != at) {
      at = t.group;
      const int c = c0 + at * side;
      weights(at < sh.each && c < groups ? c : groups - 1, w);
    }
    Product::load(x, w, piece(t) < pieces ? piece(t) : pieces - 1, lane, K);
  };
  Turn ahead{0, 0}, now{0, 0};
  // The first tile before the weights, which it would wait for otherwise.
  if constexpr (!STAGED) stage_acts<A, W, ROWS>(lds, tile, row, n, 0, K, threadIdx.x, sh.threads());
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    load(x[u], ahead);
    step(ahead);
    __builtin_amdgcn_sched_barrier(0);  // in order of use, or the first wait is for both
  }
  __syncthreads();
  Product t;
  t.clear();
#pragma unroll 1
  while (now.group < sh.each) {
    if (!whole && now.round % per == 0 && now.round + now.group > 0) {
      __syncthreads();
      stage_acts<A, W, ROWS>(lds, tile, row, n, now.round * ks * kK, K, threadIdx.x,
                             sh.threads());
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {  // a turn past the end multiplies nothing
      if (now.group < sh.each) {
        const int c = c0 + now.group * side;
        if (c < groups && piece(now) < pieces)
          t.use(x[u], [&](Row (&w)[NB]) { weights(c, w); }, lds, tile, now.round % per * ks + first,
                piece(now), lane, K);
        if (now.round == rounds - 1) {
          if (ks > 1) {  // the waves' sums, added in wave order
            __syncthreads();
#pragma unroll
            for (int b = 0; b < NB; ++b) part[(wave * NB + b) * 64 + lane] = t.acc[b];
            __syncthreads();
            if (first == 0)
              for (int q = 1; q < ks; ++q)
#pragma unroll
                for (int b = 0; b < NB; ++b) t.acc[b] += part[((wave + q) * NB + b) * 64 + lane];
          }
          if (c < groups && first == 0 && (lane & 15) < n) done(c, t.acc);
          t.clear();
        }
      }
      step(now);
      load(x[u], ahead);
      step(ahead);
    }
  }
}

// First product: u = silu(gate) * other.  ONE: a single token; each workgroup
// makes the choice itself, one of them writes it, and the pairs are listed in
// the order of the choice.
template <int W, int AF, bool ONE, int ROWS>
__global__ void __launch_bounds__(kThreads, 2) moe_up_kernel(MoeProblem p, MoeShape sh) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ Route<kMoeMaxTop> route;
  __shared__ long long starts[16];  // of the tokens' rows
  Expert x;
  if constexpr (ONE) {
    const bool writes = blockIdx.x == 0 && blockIdx.y == 0 && !p.given_ids;
    if (p.given_ids && given_expert(p, blockIdx.y) < 0) return;
    if (wave_id() == 0 && !p.given_ids) choose_experts<false>(p, route, 0, 0);
    if (writes && wave_id() == 1) choose_experts<true>(p, route, 0, 0);  // the same, and the gates
    if (wave_id() >= 2)  // meanwhile the token's first tile
      stage_acts<AF, W, ROWS>(
          lds, tile_of<AF>(tile_rows(1), p.H, sh.ks * kPieceK<W>, kTileLds),
          [&](int) { return reinterpret_cast<const unsigned char *>(p.X); }, 1, 0, p.H,
          threadIdx.x - 128, kThreads - 128);
    __syncthreads();
    if (writes) {
      write_choice<kThreads>(p, route, 0, p.top);
      if ((int)threadIdx.x < p.top) {
        ws_at<int>(p, p.at.list)[threadIdx.x] = threadIdx.x;
        ws_at<int>(p, p.at.active)[1 + threadIdx.x] = route.chosen[threadIdx.x];
      }
      if (threadIdx.x == 0) ws_at<int>(p, p.at.active)[0] = p.top;
    }
    x = {p.given_ids ? given_expert(p, blockIdx.y)
                     : __builtin_amdgcn_readfirstlane(route.chosen[blockIdx.y]),
         (int)blockIdx.y, 1};
  } else if (!expert_of(p, blockIdx.y, x)) {
    return;
  }
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  auto weights = [&](int c, Row (&w)[2]) __attribute__((always_inline)) {
    const long long i = 16LL * c + (lane >> 2) < p.I ? 16LL * c + (lane >> 2) : p.I - 1;
    const long long r = 2LL * p.I * x.e + i;
    w[0] = {p.W1 + r * p.ld1, p.S1 + r * p.lds1};
    w[1] = {p.W1 + (r + p.I) * p.ld1, p.S1 + (r + p.I) * p.lds1};
  };
  for (int m0 = 0; m0 < x.n; m0 += sh.rows) {
    const int n = x.n - m0 < sh.rows ? x.n - m0 : sh.rows;
    if ((int)threadIdx.x < n) {
      const int at = x.first + m0 + threadIdx.x;
      const int pair = ONE ? at : ws_at<int>(p, p.at.list)[at];
      starts[threadIdx.x] = pair / p.top * p.ldx;
    }
    __syncthreads();
    auto row = [&](int r) __attribute__((always_inline)) {
      return reinterpret_cast<const unsigned char *>(p.X + starts[r]);
    };
    auto done = [&](int c, const f32x4 (&acc)[2]) __attribute__((always_inline)) {
      f32x4 u;
      const long long i = 16LL * c + 4 * g;
#pragma unroll
      for (int j = 0; j < 4; ++j)  // zeros from I to the pitch
        u[j] = i + j < p.I ? acc[0][j] / (1.f + expf(-acc[0][j])) * acc[1][j] : 0.f;
      if (i < p.at.upitch)
        *reinterpret_cast<f32x4 *>(ws_at<float>(p, p.at.u) + (x.first + m0 + l16) * p.at.upitch + i) = u;
    };
    const int groups = (int)ceil_div(p.I, 16);
    expert_columns<W, AF, 2, ROWS, ONE>(lds, row, n, p.H, groups, sh, weights, done);
    __syncthreads();
  }
}

// Second product: each pair's result, before its gate.
template <int W, int ROWS>
__global__ void __launch_bounds__(64 * kMostWaves, 2) moe_down_kernel(MoeProblem p, MoeShape sh) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  Expert x;
  if (!expert_of(p, blockIdx.y, x)) return;
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  auto weights = [&](int c, Row (&w)[1]) __attribute__((always_inline)) {
    const long long h = 16LL * c + (lane >> 2) < p.H ? 16LL * c + (lane >> 2) : p.H - 1;
    const long long r = (long long)p.H * x.e + h;
    w[0] = {p.W2 + r * p.ld2, p.S2 + r * p.lds2};
  };
  for (int m0 = 0; m0 < x.n; m0 += sh.rows) {
    const int n = x.n - m0 < sh.rows ? x.n - m0 : sh.rows;
    auto row = [&](int r) __attribute__((always_inline)) {
      return p.ws + p.at.u + 4 * (x.first + m0 + r) * p.at.upitch;
    };
    const int at = x.first + m0 + (l16 < n ? l16 : 0);
    const int pair = p.T == 1 ? at : ws_at<int>(p, p.at.list)[at];
    auto done = [&](int c, const f32x4 (&acc)[1]) __attribute__((always_inline)) {
      const long long h = 16LL * c + 4 * g, left = p.H - h;
      store4<kF32>(ws_at<float>(p, p.at.part), pair * p.at.ypitch + h, (int)(left < 4 ? left : 4),
                   acc[0]);
    };
    const int groups = (int)ceil_div(p.H, 16);
    expert_columns<W, kF32, 1, ROWS, false>(lds, row, n, p.I, groups, sh, weights, done);
    __syncthreads();
  }
}

// Y: each token's results times their gates, in the order of the choice.
__global__ void __launch_bounds__(256) moe_sum_kernel(MoeProblem p) {
  const int t = blockIdx.y;
  const long long h = 4LL * (blockIdx.x * 256 + threadIdx.x), left = p.H - h;
  if (left <= 0) return;
  const float *gates = (p.given_ids ? p.given_gates : ws_at<float>(p, p.at.gates)) + t * p.top;
  const float *part = ws_at<float>(p, p.at.part) + (long long)t * p.top * p.at.ypitch + h;
  f32x4 y{0, 0, 0, 0};
#pragma unroll 4
  for (int s = 0; s < p.top; ++s) {
    if (p.given_ids && given_expert(p, t * p.top + s) < 0) continue;
    y += gates[s] * *reinterpret_cast<const f32x4 *>(part + s * p.at.ypitch);
  }
  store4_fmt(p.y_format, p.Y, t * p.ldy + h, (int)(left < 4 ? left : 4), y);
}

template <int FMT>
hipError_t launch_logits(const MoeProblem &p, hipStream_t s) {
  const unsigned gx = (unsigned)ceil_div(p.E, 4);
  // A wave to each logit while four waves a SIMD hold them all (16 tokens, 8
  // experts, 4096 wide: 3.7 us against 5.4 with four tokens to a wave).
  if (p.T * p.E <= 4096)
    return launch_kernel(moe_logits_kernel<FMT, 1>, dim3(gx, (unsigned)p.T), dim3(256), s, p);
  return launch_kernel(moe_logits_kernel<FMT, 4>, dim3(gx, (unsigned)ceil_div(p.T, 4)), dim3(256),
                       s, p);
}

// The LDS of a product of up to `rows` rows to an expert.
template <int W, int A>
int tile_bytes(int rows, int K, int ks) {
  int most = 0;
  for (int keep = 4; keep <= tile_rows(rows); keep *= 2) {
    const int bytes = act_bytes<A>(tile_of<A>(keep, K, ks * kPieceK<W>, kTileLds));
    most = most < bytes ? bytes : most;
  }
  return most;
}
// The shape of a product over `experts` experts, `columns` columns and K, of
// at most `rows` rows each.  (Where a choice made before names an expert more than once in
// a row, it may have more than that: they are taken in turns of as many as the LDS is for.)
template <int W, int A>
MoeShape shape_of(long long experts, int columns, int K, int rows) {
  const long long groups = experts * ceil_div(columns, 16);
  MoeShape sh;
  // Waves per group: until they are four to a compute unit; and two where groups
  // are fewer than eight to one and 16-bit rows have 16 pieces or more.  One and
  // two, us (experts' pairs, H / I, weights): 2, 2049 / 2049, bf16 88 and 82; 2,
  // 2048 / 2048, bf16 62 and 64; 16, 2048 / 2048, bf16 95 and 88; 16, 3501 / 3501, fp16
  // 256 and 230; 16, 2101 / 8001, fp16 389 and 322; but MX, 16, 8000 / 2100 193 and
  // 211.  Two and four, where two make more than four to a compute unit: 20, 4001 / 2501,
  // bf16 160 and 168; 2, 4000 / 2500, bf16 70 and 67; 20, 8000 / 2100, fp16 202 and 219.
  const long long pieces = ceil_div(K, kPieceK<W>);
  sh.waves = kWaves;
  sh.rows = tile_rows(rows);
  sh.ks = 1;
  while (sh.ks < kWaves && 2 * sh.ks <= pieces && groups * sh.ks < 4 * 256) sh.ks *= 2;
  if (W != kMx && sh.ks == 1 && groups < 8 * 256 && pieces >= 16) sh.ks = 2;
  while (sh.ks > 1 && tile_bytes<W, A>(rows, K, sh.ks) > kMostLds) sh.ks /= 2;
  // Groups per wave: while workgroups are left for two on each compute unit
  // (three, us: 33 tokens, 8 of 64 experts, 2048 / 1024, MX 83 against 76; 8
  // tokens, 1024 / 2816 76 against 82).
  sh.each = 1;
  while (groups * sh.ks / (2 * sh.each) >= 2 * 256 * kWaves) sh.each *= 2;
  // Eight waves to a workgroup of the second product where those of four do not
  // all fit the chip and those of eight do (four and eight, us: 64 tokens on 64
  // experts, 4096 / 1024, MX 149 and 128; 16 tokens on fp16 W2 rows of 4095 136
  // and 127; on bf16 ones of 4096, which fit, 184 and 192).
  sh.lds = tile_bytes<W, A>(rows, K, sh.ks);
  auto rounds = [&](int waves) {
    const long long all = experts * ceil_div(ceil_div(columns, 16), waves / sh.ks * sh.each);
    return ceil_div(all, 256 * (kCuLds / (sh.lds + (sh.ks > 1 ? waves * 1024 : 0))));
  };
  if (A == kF32 && rounds(kMostWaves) < rounds(kWaves)) sh.waves = kMostWaves;
  return sh;
}
template <int W, int A, int NB, class Kernel>
hipError_t launch_experts(Kernel kern, const MoeProblem &p, int columns, int K, hipStream_t s) {
  // Workgroups to an expert that is asked or, one token, to each of its choices (a choice
  // made before may name an expert more than once).
  const int experts = p.T == 1 || p.T * p.top < p.E ? p.T * p.top : p.E;
  MoeShape sh = shape_of<W, A>(experts, columns, K, p.T);
  MoeProblem q = p;
  void *args[] = {&q, &sh};
  const dim3 grid((unsigned)ceil_div(ceil_div(columns, 16), sh.waves / sh.ks * sh.each),
                  (unsigned)experts);
  return hipLaunchKernel(reinterpret_cast<const void *>(kern), grid,
                         dim3(sh.threads()), args,
                         (size_t)(sh.lds + (sh.ks > 1 ? sh.waves * NB * 1024 : 0)), s);
}

template <int W, int AF, int ROWS>
hipError_t launch_up(const MoeProblem &p, hipStream_t s) {
  return launch_experts<W, AF, 2>(p.T == 1 ? moe_up_kernel<W, AF, true, ROWS>
                                        : moe_up_kernel<W, AF, false, ROWS>,
                               p, p.I, p.H, s);
}
template <int W, int ROWS>
hipError_t launch_down(const MoeProblem &p, hipStream_t s) {
  return launch_experts<W, kF32, 1>(moe_down_kernel<W, ROWS>, p, p.H, p.I, s);
}

// Whether a product's 16-bit rows are to be read by whole words (Eight<kOdd>):
// some start in the middle of one, and both matrices start on one.
bool odd_rows(const void *a, long long a_pitch, const void *b, long long b_pitch) {
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 3) == 0 &&
         ((a_pitch | b_pitch) & 3) != 0;
}

template <int W, int AF>
hipError_t launch_products(const MoeProblem &p, hipStream_t s) {
  constexpr bool kHalf = W != kMx;
  hipError_t e;
  if (p.H < 8)
    e = launch_up<W, AF, kShort>(p, s);
  else if (odd_rows(p.X, 2 * p.ldx, kHalf ? p.W1 : nullptr, kHalf ? p.ld1 : 0))
    e = launch_up<W, AF, kOdd>(p, s);
  else
    e = launch_up<W, AF, kWords>(p, s);
  if (e != hipSuccess) return e;
  if constexpr (kHalf) {
    if (p.I < 8) return launch_down<W, kShort>(p, s);
    if (odd_rows(p.W2, p.ld2, nullptr, 0)) return launch_down<W, kOdd>(p, s);
  }
  return launch_down<W, kWords>(p, s);
}

}  // namespace

hipError_t launch_moe(const MoeProblem &p, hipStream_t s) {
  const bool bf16 = p.format == kBf16;
  hipError_t e = hipSuccess;
  if (!p.given_ids) e = bf16 ? launch_logits<kBf16>(p, s) : launch_logits<kF16>(p, s);
  if (e != hipSuccess) return e;
  if (p.given_ids) {
    if (p.T > 1) e = launch_kernel(moe_given_kernel, dim3(1), dim3(kListThreads), s, p);
    if (e != hipSuccess) return e;
  } else if (p.T > 1 && p.T <= kRouteTokens) {
    e = launch_kernel(moe_route_kernel, dim3(1), dim3(64 * kRouteTokens), s, p);
    if (e != hipSuccess) return e;
  } else if (p.T > 1) {
    e = launch_kernel(moe_choose_kernel, dim3((unsigned)ceil_div(p.T, kChooseTokens)),
                      dim3(64 * kChooseTokens), s, p);
    if (e == hipSuccess) e = launch_kernel(moe_list_kernel, dim3(1), dim3(kListThreads), s, p);
    if (e != hipSuccess) return e;
  }
  e = p.mx ? (bf16 ? launch_products<kMx, kBf16>(p, s) : launch_products<kMx, kF16>(p, s))
           : (bf16 ? launch_products<kBf16, kBf16>(p, s) : launch_products<kF16, kF16>(p, s));
  if (e != hipSuccess) return e;
  return launch_kernel(moe_sum_kernel, dim3((unsigned)ceil_div(p.H, 1024), (unsigned)p.T), dim3(256),
                       s, p);
}

}  // namespace gemm_f32_impl
