// The experts' products for a choice made before (gemm_experts.h): the order of
// the pairs by expert, the sums over a token's pairs, and the calls of a pass.
//
// A few tokens without a backward pass run on the mixture-of-experts layer's thin
// products (moe.hip), which read each weight once for up to 16 pairs; others on
// tiles (row_tiles.hpp).
#include "experts_tiles.hpp"
#include "mx_internal.hpp"

namespace gemm_f32_impl {
namespace {

// ---- the order of the pairs ----------------------------------------------------
// A stable sort by expert: counts, their sums, then each pair's place.  Up to
// kOneLaunch pairs in one launch, whose workgroups each count all pairs, and take
// kListPairs of them; more in three launches, the sums by one workgroup.  One launch and
// three, us, by experts (64, 512, 8, 1): 4,096 pairs 5.7, 6.2, 5.6, 7.5 and 11.1, 13.0,
// 10.5, 11.6; 65,536 16.0, 17.1, 17.5, 52.5 and 16.4, 19.5, 18.6, 35.9; 131,072 26.7,
// 28.4, 30.3, 99.9 and 22.8, 27.2, 26.2, 60.6.  Three at 2^20 pairs 115, 145, 144, 418; at
// 2^22 433, 867, 548, 1,655; at 2^26 11,500, 14,800, 10,700, 26,900: linear, and beside
// 262,144 tokens' products of 7,500 (8 experts, 4096 / 1024) 45.  Pairs whose expert is
// not in 0 .. E - 1 get no place.

constexpr int kMostGroups = 1 << 20;
constexpr int kOneLaunch = 1 << 16, kOneThreads = kListPairs, kListThreads = 256;

__device__ inline int expert_of(const ExpertsProblem &p, long long pair, long long pairs) {
  if (pair >= pairs) return kMoeMaxExperts;  // none
  const int e = p.ids[pair], last = p.E - (p.rest ? 1 : 0);
  return e >= 0 && e < last ? e : p.rest ? p.E - 1 : kMoeMaxExperts;
}

// Counts of pairs from .. from + pairs' by expert, onto zeros in `count`.
template <int THREADS>
__device__ inline void count_pairs(const ExpertsProblem &p, int *count, long long from, long long to,
                                   long long pairs) {
  for (int e = threadIdx.x; e < p.E; e += THREADS) count[e] = 0;
  __syncthreads();
  for (long long i = from + threadIdx.x; i < to; i += THREADS) {
    const int e = expert_of(p, i, pairs);
    if (e < p.E) atomicAdd(&count[e], 1);
  }
  __syncthreads();
}

// Where each expert's places begin, and the row tiles, from the experts' counts
// `n` of the first kMoeMaxExperts threads.  On return begin[e] is expert e's first place.
// `writes`: into the workspace too.
__device__ inline void lay_out(const ExpertsProblem &p, int n, int (*scan)[3], int *begin,
                               bool writes = true) {
  const int e = threadIdx.x, lane = e & 63, wave = wave_id();
  const bool in = e < kMoeMaxExperts;
  const int tiles = p.rest && e == p.E - 1 ? 0 : (n + p.tile - 1) / p.tile;
  int upto[3] = {n, tiles, n > 0};  // sums up to this expert: in the wave, then in all
  if (in) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const int v = __shfl_up(upto[q], d);
        if (lane >= d) upto[q] += v;
      }
#pragma unroll
    for (int q = 0; q < 3; ++q)
      if (lane == 63) scan[wave][q] = upto[q];
  }
  __syncthreads();
  if (in)
    for (int w = 0; w < wave; ++w)
#pragma unroll
      for (int q = 0; q < 3; ++q) upto[q] += scan[w][q];
  if (in && e < p.E) begin[e] = upto[0] - n;
  if (writes && in && e < p.E) {
    const int last = upto[0], first = last - n;
    int *start = ws_at<int>(p, p.at.start), *table = ws_at<int>(p, p.at.tiles);
    start[e] = first;
    const int t0 = upto[1] - tiles;
    for (int t = 0; t < tiles; ++t) {
      int *at = table + 4 + 4LL * (t0 + t);
      at[0] = e;
      at[1] = first + t * p.tile;
      at[2] = n - t * p.tile < p.tile ? n - t * p.tile : p.tile;
    }
    if (p.rest && n > 0) {
      const int run = upto[2] - 1;
      int *at = ws_at<int>(p, p.at.runs) + 4 + 4 * run, *tile_run = ws_at<int>(p, p.at.tile_run);
      at[0] = e, at[1] = first, at[2] = n;
      for (int t = (first + p.run_tile - 1) / p.run_tile; t * p.run_tile < last; ++t) tile_run[t] = run;
    }
    if (e == p.E - 1) {
      start[p.E] = last;
      table[0] = t0 + tiles;
      if (p.rest) *ws_at<int>(p, p.at.runs) = upto[2];
    }
  }
  __syncthreads();
}

// The places of pairs from .. to, `begin` those of their experts' first ones.
template <int THREADS>
__device__ inline void place_pairs(const ExpertsProblem &p, int *begin,
                                   unsigned short (*count)[kMoeMaxExperts], long long from,
                                   long long to, long long pairs) {
  constexpr int kWaves = THREADS / 64;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const unsigned long long before = (1ULL << lane) - 1;
  int *list = ws_at<int>(p, p.at.list), *token = ws_at<int>(p, p.at.token);
  int *where = ws_at<int>(p, p.at.where);
  for (long long i0 = from; i0 < to; i0 += THREADS) {
    for (int w = 0; w < kWaves; ++w)
      for (int e = threadIdx.x; e < p.E; e += THREADS) count[w][e] = 0;
    __syncthreads();
    const long long i = i0 + threadIdx.x;
    const int e = expert_of(p, i < to ? i : pairs, pairs);
    const unsigned long long same = same_expert(e);
    if (e < p.E && (same & before) == 0) count[wave][e] = (unsigned short)__popcll(same);
    __syncthreads();
    if (e < p.E) {
      int at = begin[e] + __popcll(same & before);
      for (int w = 0; w < wave; ++w) at += count[w][e];
      list[at] = (int)i;
      token[at] = (int)(i / p.top);
      where[i] = at;
    } else if (i < to) {
      where[i] = -1;
    }
    __syncthreads();
    for (int x = threadIdx.x; x < p.E; x += THREADS) {
      int n = 0;
      for (int w = 0; w < kWaves; ++w) n += count[w][x];
      begin[x] += n;
    }
    // the next round's counts are zeroed by the threads that have just read them
  }
}

// Counts are kept in kCopies, by lane, so that a wave's pairs of one expert do not
// wait for one another.
constexpr int kCopies = 8;
__global__ void __launch_bounds__(kOneThreads) experts_list_kernel(ExpertsProblem p) {
  __shared__ int scan[kMoeMaxExperts / 64][3];
  __shared__ int begin[kMoeMaxExperts];
  __shared__ int counts[2][kCopies][kMoeMaxExperts];  // of the pairs before this workgroup's; of the others
  __shared__ unsigned short count[kOneThreads / 64][kMoeMaxExperts];
  const int pairs = p.T * p.top, from = kListPairs * (int)blockIdx.x;
  const int copy = threadIdx.x & (kCopies - 1);
  for (int i = threadIdx.x; i < 2 * kCopies * kMoeMaxExperts; i += kOneThreads)
    counts[0][0][i] = 0;
  __syncthreads();
#pragma unroll 4
  for (int i = threadIdx.x; i < pairs; i += kOneThreads) {
    const int e = expert_of(p, i, pairs);
    if (e < p.E) atomicAdd(&counts[i >= from][copy][e], 1);
  }
  __syncthreads();
  int before = 0, n = 0;
  if ((int)threadIdx.x < p.E)
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      before += counts[0][c][threadIdx.x];
      n += counts[1][c][threadIdx.x];
    }
  n += before;
  lay_out(p, n, scan, begin, blockIdx.x == 0);
  if ((int)threadIdx.x < p.E) begin[threadIdx.x] += before;
  __syncthreads();
  place_pairs<kOneThreads>(p, begin, count, from, from + kListPairs < pairs ? from + kListPairs : pairs,
                           pairs);
}

__global__ void __launch_bounds__(kListThreads) experts_count_kernel(ExpertsProblem p) {
  __shared__ int count[kMoeMaxExperts];
  const long long pairs = (long long)p.T * p.top, from = (long long)kListPairs * blockIdx.x;
  const long long to = from + kListPairs < pairs ? from + kListPairs : pairs;
  count_pairs<kListThreads>(p, count, from, to, pairs);
  int *counts = ws_at<int>(p, p.at.counts) + (long long)blockIdx.x * p.E;
  for (int e = threadIdx.x; e < p.E; e += kListThreads) counts[e] = count[e];
}

// One workgroup: each group's counts become the places of its first pairs.
__global__ void __launch_bounds__(kMoeMaxExperts) experts_scan_kernel(ExpertsProblem p) {
  __shared__ int scan[kMoeMaxExperts / 64][3];
  __shared__ int begin[kMoeMaxExperts];
  int *counts = ws_at<int>(p, p.at.counts) + threadIdx.x;
  int n = 0;
  const bool in = (int)threadIdx.x < p.E;
  if (in)
#pragma unroll 8
    for (long long g = 0; g < p.at.list_groups; ++g) n += counts[g * p.E];
  lay_out(p, n, scan, begin);
  if (!in) return;
  n = begin[threadIdx.x];
#pragma unroll 8
  for (long long g = 0; g < p.at.list_groups; ++g) {
    const int c = counts[g * p.E];
    counts[g * p.E] = n;
    n += c;
  }
}

__global__ void __launch_bounds__(kListThreads) experts_place_kernel(ExpertsProblem p) {
  __shared__ int begin[kMoeMaxExperts];
  __shared__ unsigned short count[kListThreads / 64][kMoeMaxExperts];
  const long long pairs = (long long)p.T * p.top, from = (long long)kListPairs * blockIdx.x;
  const long long to = from + kListPairs < pairs ? from + kListPairs : pairs;
  const int *counts = ws_at<int>(p, p.at.counts) + (long long)blockIdx.x * p.E;
  for (int e = threadIdx.x; e < p.E; e += kListThreads) begin[e] = counts[e];
  __syncthreads();
  place_pairs<kListThreads>(p, begin, count, from, to, pairs);
}

}  // namespace

hipError_t launch_list(const ExpertsProblem &p, hipStream_t s) {
  const dim3 groups((unsigned)(p.at.list_groups > 0 ? p.at.list_groups : 1));
  if ((long long)p.T * p.top <= kOneLaunch)
    return launch_kernel(experts_list_kernel, groups, dim3(kOneThreads), s, p);
  hipError_t e = launch_kernel(experts_count_kernel, groups, dim3(kListThreads), s, p);
  if (e != hipSuccess) return e;
  e = launch_kernel(experts_scan_kernel, dim3(1), dim3(kMoeMaxExperts), s, p);
  if (e != hipSuccess) return e;
  return launch_kernel(experts_place_kernel, groups, dim3(kListThreads), s, p);
}

namespace {

// ---- sums over a token's pairs --------------------------------------------------

// out[t] = the sum of token t's rows of `part`, in the order of its choices.  A row
// of threads takes a token, each 8 values.
template <int FMT>
__global__ void __launch_bounds__(256) experts_sum_kernel(ExpertsProblem p, uint16_t *out,
                                                          long long ldo) {
  const int per = blockDim.x;
  for (long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y; t < p.T;
       t += (long long)gridDim.x * blockDim.y) {
    const int *ids = p.ids + t * p.top;
    const float *part = ws_at<float>(p, p.at.part) + t * p.top * p.at.hpitch;
    for (int h = 8 * threadIdx.x; h < p.H; h += 8 * per) {
      float v[8] = {};
#pragma unroll 4
      for (int s = 0; s < p.top; ++s) {
        if (ids[s] < 0 || ids[s] >= p.E) continue;
        const f32x4 *w = reinterpret_cast<const f32x4 *>(part + s * p.at.hpitch + h);
        const f32x4 a = w[0], b = w[1];
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] += a[c], v[4 + c] += b[c];
      }
      store8<FMT>(out, t * ldo + h, p.H - h, v);
    }
  }
}
hipError_t launch_sum(const ExpertsProblem &p, uint16_t *out, long long ldo, hipStream_t s) {
  unsigned per = 1;
  while (per < 256 && 8 * per < (unsigned)p.H) per *= 2;
  const dim3 block(per, 256 / per);
  const long long groups = ceil_div(p.T, block.y);
  const dim3 grid((unsigned)(groups < kMostGroups ? groups : kMostGroups));
  return p.format == kBf16 ? launch_kernel(experts_sum_kernel<kBf16>, grid, block, s, p, out, ldo)
                           : launch_kernel(experts_sum_kernel<kF16>, grid, block, s, p, out, ldo);
}

// The gates' gradients: their parts added in order of the columns; 0 for a pair without an expert.
__global__ void __launch_bounds__(256) experts_dgates_kernel(ExpertsProblem p) {
  const long long pairs = (long long)p.T * p.top, i = 256LL * blockIdx.x + threadIdx.x;
  if (i >= pairs) return;
  const int place = ws_at<int>(p, p.at.where)[i];
  float sum = 0.f;
  if (place >= 0) {
    const float *dg = ws_at<float>(p, p.at.dg) + place;
#pragma unroll 8
    for (long long q = 0; q < p.at.slices; ++q) sum += dg[q * pairs];
  }
  p.dgates[i] = sum;
}

}  // namespace

// The products of a pass take the list's row tiles, so all of them are of one size.
hipError_t launch_experts_forward(const ExpertsProblem &call, hipStream_t s) {
  ExpertsProblem p = call;
  p.tile = up_direct(p) && down_direct(p) ? experts_tile(p.T, p.E, p.top, p.H, p.I, p.saved != nullptr)
                                          : Small::BM;
  p.at = experts_space(p.T, p.E, p.top, p.H, p.I, p.tile, false);
  hipError_t e = launch_list(p, s);
  if (e == hipSuccess) e = launch_experts_up(p, s);
  if (e == hipSuccess) e = launch_experts_down(p, s);
  return e == hipSuccess ? launch_sum(p, p.Y, p.ldy, s) : e;
}

hipError_t launch_experts_backward(const ExpertsProblem &call, hipStream_t s) {
  ExpertsProblem p = call;
  p.tile = du_direct(p) && dx_direct(p) ? experts_tile(p.T, p.E, p.top, p.H, p.I, true) : Small::BM;
  p.at = experts_space(p.T, p.E, p.top, p.H, p.I, p.tile, true);
  hipError_t e = launch_list(p, s);
  if (e == hipSuccess && (p.dgates || p.dX || p.dW1 || p.dW2)) e = launch_experts_du(p, s);
  if (e == hipSuccess && p.dgates && p.T > 0)
    e = launch_kernel(experts_dgates_kernel, dim3((unsigned)ceil_div((long long)p.T * p.top, 256)),
                      dim3(256), s, p);
  if (e == hipSuccess && p.dX && p.T > 0) {
    e = launch_experts_dx(p, s);
    if (e == hipSuccess) e = launch_sum(p, p.dX, p.lddx, s);
  }
  return e == hipSuccess ? launch_experts_dw(p, s) : e;
}

}  // namespace gemm_f32_impl
