// The mixture-of-experts layer for a few tokens (gemm_moe.h), in four
// launches: the router's logits, the choice of experts, and the two products
// over the chosen experts' weights.  The products read each chosen expert's
// weights once, straight into the matrix instructions' operands
// (mx_thin.hpp); the tokens of one expert share them, 16 rows at a time.
#include "mx_internal.hpp"
#include "mx_thin.hpp"

namespace gemm_f32_impl {
namespace {

template <class T>
__device__ inline T *ws_at(const MoeProblem &p, long long off) {
  return reinterpret_cast<T *>(p.ws + off);
}

// ---- router logits -------------------------------------------------------
// A wave takes one expert and 4 tokens; a lane 8 consecutive h at a time.
// Products and sums in 64 bits, so that the order of experts next to a tie
// does not depend on the order of the sum.
constexpr int kLogitTokens = 4;

template <int FMT>
__global__ void __launch_bounds__(256) moe_logits_kernel(MoeProblem p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = 4 * blockIdx.x + wave;
  if (e >= p.E) return;
  const int t0 = kLogitTokens * blockIdx.y;
  double acc[kLogitTokens] = {};
  for (long long h = 8 * lane; h < p.H; h += 512) {
    float r[8];
    load8<FMT>(p.R, e * p.ldr + h, (int)(p.H - h < 8 ? p.H - h : 8), r);
#pragma unroll
    for (int i = 0; i < kLogitTokens; ++i) {
      const int t = t0 + i < p.T ? t0 + i : p.T - 1;
      float x[8];
      load8<FMT>(p.X, t * p.ldx + h, (int)(p.H - h < 8 ? p.H - h : 8), x);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i] = fma((double)r[j], (double)x[j], acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kLogitTokens; ++i) {
    double v = acc[i];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    if (lane == 0 && t0 + i < p.T) ws_at<double>(p, p.at.logits)[(long long)(t0 + i) * p.E + e] = v;
  }
}

// ---- the choice of experts --------------------------------------------------
// One workgroup.  A wave takes a token: `top` times the largest of the logits
// not yet taken (ties to the lower index), then the gates.  Then the pairs
// (token, choice) are listed by expert: ranks inside 64 pairs by ballots,
// added to the counts of the 64-pair chunks before.
constexpr int kRouteThreads = 1024;
constexpr int kMaxPairs = kMoeMaxTokens * kMoeMaxTop;
constexpr int kPerLane = kMoeMaxExperts / 64;

// Doubles as integers of the same order; NaN as -infinity, so that every
// expert can be chosen and INT64_MIN is below all.
__device__ inline long long order_key(double v) {
  if (v != v) v = -__builtin_inf();
  const long long b = __builtin_bit_cast(long long, v);
  return b >= 0 ? b : b ^ 0x7fffffffffffffffLL;
}

__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(MoeProblem p) {
  __shared__ unsigned short chosen[kMaxPairs];
  __shared__ unsigned short count[kMaxPairs / 64][kMoeMaxExperts];
  __shared__ int first[kMoeMaxExperts + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int kWaves = kRouteThreads / 64;
  const int pairs = p.T * p.top, chunks = (pairs + 63) / 64;
  const double *logits = ws_at<double>(p, p.at.logits);
  int *ids = ws_at<int>(p, p.at.ids);
  float *gates = ws_at<float>(p, p.at.gates);

  for (int i = threadIdx.x; i < chunks * kMoeMaxExperts; i += kRouteThreads)
    (&count[0][0])[i] = 0;

  for (int t = wave; t < p.T; t += kWaves) {
    double z[kPerLane];
    long long key[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int e = lane + 64 * i;
      z[i] = e < p.E ? logits[(long long)t * p.E + e] : 0.0;
      key[i] = e < p.E ? order_key(z[i]) : (long long)0x8000000000000000ULL;
    }
    double zmax = 0.0, total = 0.0, mine = 0.0;
    for (int s = 0; s < p.top; ++s) {
      long long best = key[0];
      int at = lane;
#pragma unroll
      for (int i = 1; i < kPerLane; ++i)
        if (key[i] > best) best = key[i], at = lane + 64 * i;
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) {
        const long long ob = __shfl_xor(best, d);
        const int oa = __shfl_xor(at, d);
        if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
      }
      double v = 0.0;  // the chosen logit, from the lane that holds it
#pragma unroll
      for (int i = 0; i < kPerLane; ++i)
        if (at == lane + 64 * i) {
          v = z[i];
          key[i] = (long long)0x8000000000000000ULL;
        }
      v = __shfl(v, at & 63);
      if (s == 0) {
        // The largest logit; a NaN among the logits makes every gate NaN.
        zmax = v;
        double part = 0.0;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
          if (lane + 64 * i < p.E) {
            nan |= z[i] != z[i];
            if (!p.renormalize) part += exp(z[i] - zmax);
          }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) part += __shfl_xor(part, d);
        total = __any(nan) ? __builtin_nan("") : part;
      }
      const double w = exp(v - zmax);
      if (p.renormalize) total += w;
      if (lane == s) mine = w;
      if (lane == 0) {
        chosen[t * p.top + s] = (unsigned short)at;
        ids[t * p.top + s] = at;
        if (p.ids) p.ids[t * p.top + s] = at;
      }
    }
    if (lane < p.top) {
      const float gate = (float)(mine / total);
      gates[t * p.top + lane] = gate;
      if (p.gates) p.gates[t * p.top + lane] = gate;
    }
  }
  __syncthreads();

  // Counts per chunk of 64 pairs, and each pair's rank in its chunk.
  for (int c = wave; c < chunks; c += kWaves) {
    const int i = 64 * c + lane;
    const int e = i < pairs ? chosen[i] : kMoeMaxExperts;
    unsigned long long same = __ballot(1);
#pragma unroll
    for (int b = 0; b < 10; ++b) {
      const unsigned long long m = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? m : ~m;
    }
    if (i < pairs && (same & ((1ULL << lane) - 1)) == 0)
      count[c][e] = (unsigned short)__popcll(same);
  }
  __syncthreads();
  if (wave == 0) {  // where each expert's pairs begin, and the chosen experts
    int base = 0, nact = 0;
    int *active = ws_at<int>(p, p.at.active), *start = ws_at<int>(p, p.at.start);
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      const int e = e0 + lane;
      int n = 0;
      if (e < p.E)
        for (int c = 0; c < chunks; ++c) n += count[c][e];
      int upto = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
      }
      if (e < p.E) first[e] = start[e] = base + upto - n;
      const unsigned long long on = __ballot(n > 0);
      if (n > 0) active[1 + nact + __popcll(on & ((1ULL << lane) - 1))] = e;
      base += __shfl(upto, 63);
      nact += __popcll(on);
    }
    if (lane == 0) {
      active[0] = nact;
      start[p.E] = pairs;
    }
  }
  __syncthreads();
  int *list = ws_at<int>(p, p.at.list);
  for (int c = wave; c < chunks; c += kWaves) {
    const int i = 64 * c + lane;
    const int e = i < pairs ? chosen[i] : kMoeMaxExperts;
    unsigned long long same = __ballot(1);
#pragma unroll
    for (int b = 0; b < 10; ++b) {
      const unsigned long long m = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? m : ~m;
    }
    if (i < pairs) {
      int at = first[e] + __popcll(same & ((1ULL << lane) - 1));
      for (int q = 0; q < c; ++q) at += count[q][e];
      list[at] = i;
    }
  }
}

// ---- first product: u = silu(gate) * other ------------------------------------
// A workgroup takes one chosen expert and 16 of its inner columns, both
// factors; its waves take 128-deep steps of H in turn.

constexpr int kUpWaves = 8;

template <int W, int AF, int MB>
__device__ inline void moe_up_rows(const MoeProblem &p, const Row (&w)[2], int first, int n,
                                   int i0, f32x4 (*part)[2][2][64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  const int *list = ws_at<int>(p, p.at.list) + first;
  Row x[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int m = 16 * i + l16 < n ? 16 * i + l16 : n - 1;
    x[i] = {reinterpret_cast<const unsigned char *>(p.X + list[m] / p.top * p.ldx), nullptr};
  }
  Thin<W, AF, MB, 2> t;
  t.clear();
  t.run(x, w, wave, kUpWaves, (int)ceil_div(p.H, kPieceK<W>), p.H, g);
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    part[wave][i][0][lane] = t.acc[i][0];
    part[wave][i][1][lane] = t.acc[i][1];
  }
  __syncthreads();
  if (wave < MB) {
    f32x4 a = part[0][wave][0][lane], b = part[0][wave][1][lane];
#pragma unroll
    for (int q = 1; q < kUpWaves; ++q) {
      a += part[q][wave][0][lane];
      b += part[q][wave][1][lane];
    }
    const int m = 16 * wave + l16;
    if (m < n) {
      uint16_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float u = a[j] / (1.f + expf(-a[j])) * b[j];
        const float v = i0 + 4 * g + j < p.I ? u : 0.f;  // rows are padded with zeros
        hi[j] = from_f32<kBf16>(v);
        const float h = to_f32<kBf16>(hi[j]);
        lo[j] = mag_bits(h) < 0x7f800000u ? from_f32<kBf16>(v - h) : (uint16_t)0;
      }
      const long long at = (first + m) * p.at.pitch + i0 + 4 * g;
      *reinterpret_cast<u32x2 *>(ws_at<uint16_t>(p, p.at.hi) + at) =
          u32x2{hi[0] | (uint32_t)hi[1] << 16, hi[2] | (uint32_t)hi[3] << 16};
      *reinterpret_cast<u32x2 *>(ws_at<uint16_t>(p, p.at.lo) + at) =
          u32x2{lo[0] | (uint32_t)lo[1] << 16, lo[2] | (uint32_t)lo[3] << 16};
    }
  }
  __syncthreads();
}

template <int W, int AF>
__global__ void __launch_bounds__(64 * kUpWaves) moe_up_kernel(MoeProblem p) {
  __shared__ f32x4 part[kUpWaves][2][2][64];
  const int *active = ws_at<int>(p, p.at.active), *start = ws_at<int>(p, p.at.start);
  if ((int)blockIdx.y >= active[0]) return;
  const int e = active[1 + blockIdx.y];
  const int first = start[e], n = start[e + 1] - first;
  const int i0 = 16 * blockIdx.x, l16 = threadIdx.x & 15;
  const int i = i0 + l16 < p.I ? i0 + l16 : p.I - 1;
  const long long r0 = 2LL * p.I * e + i, r1 = r0 + p.I;
  Row w[2] = {{p.W1 + r0 * p.ld1, nullptr}, {p.W1 + r1 * p.ld1, nullptr}};
  if constexpr (W == kMx) w[0].q = p.S1 + r0 * p.lds1, w[1].q = p.S1 + r1 * p.lds1;
  if (n <= 16) {
    moe_up_rows<W, AF, 1>(p, w, first, n, i0, part);
  } else {
    for (int m = 0; m < n; m += 32) moe_up_rows<W, AF, 2>(p, w, first + m, n - m, i0, part);
  }
}

// ---- second product and the weighted sum -----------------------------------------
// A workgroup owns 16 columns of Y for all tokens.  Its waves take pieces of
// an expert's inner columns in turn, over all chosen experts, and add each
// run of pieces, times the gates, to a sum of their own in LDS; the waves'
// sums are added in wave order at the end.
constexpr int kDownWaves = 8;
template <int W>
constexpr int kRunPieces = W == kMx ? 1 : 4;  // 512 k

template <int W, int MB>
__device__ inline void moe_down_run(const MoeProblem &p, const Row &row, int first, int n, int p0,
                                    int p1, float *sum) {
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  Row u[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int m = 16 * i + l16 < n ? 16 * i + l16 : n - 1;
    u[i] = {p.ws + p.at.hi + 2 * (first + m) * p.at.pitch,
            p.ws + p.at.lo + 2 * (first + m) * p.at.pitch};
  }
  Thin<W, kSplit, MB, 1> t;
  t.clear();
  const Row w[1] = {row};
  t.run(u, w, p0, 1, p1, p.I, g);
  const int *list = ws_at<int>(p, p.at.list) + first;
  const float *gates = ws_at<float>(p, p.at.gates);
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int m = 16 * i + l16;
    if (m < n) {
      const int pair = list[m];
      f32x4 *to = reinterpret_cast<f32x4 *>(sum + 16 * (pair / p.top) + 4 * g);
      *to += gates[pair] * t.acc[i][0];
    }
  }
}

template <int W>
__global__ void __launch_bounds__(64 * kDownWaves) moe_down_kernel(MoeProblem p) {
  extern __shared__ __attribute__((aligned(16))) float sums[];  // [wave][token][16]
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  float *sum = sums + wave * 16 * p.T;
  for (int i = lane; i < 4 * p.T; i += 64) reinterpret_cast<f32x4 *>(sum)[i] = f32x4{0, 0, 0, 0};
  __syncthreads();
  const int *active = ws_at<int>(p, p.at.active), *start = ws_at<int>(p, p.at.start);
  const int n0 = 16 * blockIdx.x, l16 = lane & 15;
  const int col = n0 + l16 < p.H ? n0 + l16 : p.H - 1;
  const int pieces = (int)ceil_div(p.I, kPieceK<W>), runs = (int)ceil_div(pieces, kRunPieces<W>);
  const int units = active[0] * runs;
  for (int v = wave; v < units; v += kDownWaves) {
    const int e = active[1 + v / runs], run = v % runs;
    const int first = start[e], n = start[e + 1] - first;
    const long long r = (long long)p.H * e + col;
    const Row row{p.W2 + r * p.ld2, W == kMx ? p.S2 + r * p.lds2 : nullptr};
    const int p0 = run * kRunPieces<W>;
    const int p1 = p0 + kRunPieces<W> < pieces ? p0 + kRunPieces<W> : pieces;
    if (n <= 16) {
      moe_down_run<W, 1>(p, row, first, n, p0, p1, sum);
    } else {
      for (int m = 0; m < n; m += 32)
        moe_down_run<W, 2>(p, row, first + m, n - m, p0, p1, sum);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 4 * p.T; i += 64 * kDownWaves) {
    f32x4 v = reinterpret_cast<const f32x4 *>(sums)[i];
#pragma unroll
    for (int w = 1; w < kDownWaves; ++w) v += reinterpret_cast<const f32x4 *>(sums + w * 16 * p.T)[i];
    const int t = i / 4, n = n0 + 4 * (i % 4);
    store4_fmt(p.y_format, p.Y, t * p.ldy + n, p.H - n < 4 ? p.H - n : 4, v);
  }
}

}  // namespace

hipError_t launch_moe(const MoeProblem &p, hipStream_t s) {
  const int pairs = p.T * p.top;
  const dim3 lgrid((unsigned)ceil_div(p.E, 4), (unsigned)ceil_div(p.T, kLogitTokens));
  hipError_t e = launch_kernel(
      p.format == kBf16 ? moe_logits_kernel<kBf16> : moe_logits_kernel<kF16>, lgrid, dim3(256), s, p);
  if (e != hipSuccess) return e;
  e = launch_kernel(moe_route_kernel, dim3(1), dim3(kRouteThreads), s, p);
  if (e != hipSuccess) return e;
  const dim3 ugrid((unsigned)(p.at.pitch / 16), (unsigned)(p.E < pairs ? p.E : pairs));
  auto up = p.mx ? (p.format == kBf16 ? moe_up_kernel<kMx, kBf16> : moe_up_kernel<kMx, kF16>)
                 : (p.format == kBf16 ? moe_up_kernel<kBf16, kBf16> : moe_up_kernel<kF16, kF16>);
  e = launch_kernel(up, ugrid, dim3(64 * kUpWaves), s, p);
  if (e != hipSuccess) return e;
  auto down = p.mx                ? moe_down_kernel<kMx>
              : p.format == kBf16 ? moe_down_kernel<kBf16>
                                  : moe_down_kernel<kF16>;
  MoeProblem q = p;
  void *args[] = {&q};
  return hipLaunchKernel(reinterpret_cast<const void *>(down), dim3((unsigned)ceil_div(p.H, 16)),
                         dim3(64 * kDownWaves), args, (size_t)kDownWaves * 64 * p.T, s);
}

}  // namespace gemm_f32_impl
