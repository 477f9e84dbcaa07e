// Host-only planning of routing, the experts' products and adapters (see
// experts_plan.hpp).
#include "experts_plan.hpp"

namespace gemm_f32_impl {

int route_check_sizes(int T, int E, int top) {
  if (T < 0 || E < 0 || top < 0) return kInvalidDim;
  if (T > kRouteMaxTokens || E > kRouteMaxExperts || top < 1 || top > kRouteMaxTop || top > E)
    return kBadArg;
  return kOk;
}

int experts_check_sizes(int T, int E, int top, int H, int I) {
  if (T < 0 || E < 0 || top < 0 || H < 1 || I < 1) return kInvalidDim;
  if (T > kExpertsMaxTokens || E < 1 || E > kMoeMaxExperts || top < 1 || top > kMoeMaxTop ||
      H > kExpertsMaxWidth || I > kExpertsMaxWidth)
    return kBadArg;
  return kOk;
}

bool experts_thin(int T, int E, int top) {
  const long long pairs = (long long)T * top;
  return T <= kMoeMaxTokens && pairs <= 16LL * E;
}

int experts_tile(int T, int E, int top, int H, int I) {
  const long long pairs = (long long)T * top;
  const long long asked = E < pairs ? E : pairs;
  const long long rows = asked ? ceil_div(pairs, asked) : 0;
  // 256 x 256 tiles where they can fill most of the chip
  const long long large = asked * ceil_div(rows, 256) * ceil_div(H < 2 * I ? H : 2 * I, 256);
  return rows > 64 && large >= 192 ? 256 : 128;
}

ExpertsSpace experts_space(int T, int E, int top, int H, int I, int tile, bool backward) {
  ExpertsSpace w;
  long long at = 0;
  const long long pairs = (long long)T * top;
  auto take = [&at](long long bytes) {
    const long long from = at;
    at += ceil_div(bytes, 256) * 256;
    return from;
  };
  w.ipitch = ceil_div(I, 64) * 64;
  w.hpitch = ceil_div(H, 8) * 8;
  w.most_tiles = pairs / tile + (E < pairs ? E : pairs);
  w.list_groups = ceil_div(pairs, kListPairs);
  w.slices = backward ? 2 * ceil_div(I, tile) : 0;
  w.start = take(4LL * (E + 1));
  w.tiles = take(16 + 16 * w.most_tiles);
  w.list = take(4 * pairs);
  w.token = take(4 * pairs);
  w.where = take(4 * pairs);
  w.counts = take(4 * w.list_groups * E);
  w.u = take(2 * pairs * w.ipitch);
  w.part = take(2 * pairs * w.hpitch);
  w.dh = backward ? take(4 * pairs * w.ipitch) : at;
  w.dg = backward ? take(4 * pairs * w.slices) : at;
  w.runs = w.tile_run = at;
  w.bytes = at;
  return w;
}

int adapters_check_sizes(int T, int N, int K, int R, int count) {
  if (T < 0 || count < 0 || N < 1 || K < 1 || R < 1) return kInvalidDim;
  if (T > kAdaptersMaxRows || N > kAdaptersMaxWidth || K > kAdaptersMaxWidth ||
      R > kAdaptersMaxRank || count > kAdaptersMaxCount)
    return kBadArg;
  return kOk;
}

AdaptersSpace adapters_space(int T, int N, int K, int R, int count) {
  AdaptersSpace w{};
  long long at = 0;
  auto take = [&at](long long bytes) {
    const long long from = at;
    at += ceil_div(bytes, 256) * 256;
    return from;
  };
  w.rpitch = ceil_div(R, 64) * 64;
  w.v = take(2 * T * w.rpitch);
  w.splits = 1;
  w.chunk = K;
  if (T > kAdaptersThin) {
    w.tile = ceil_div(T, 256) * ceil_div(N, 256) >= 192 ? 256 : 128;
    // The products with A: row tiles of kAdaptersRows, K in parts until there are
    // two workgroups to a compute unit, of 256 values at least.
    const long long tiles = (ceil_div(T, kAdaptersRows) + count / 2) * ceil_div(R, kAdaptersRows);
    while (tiles * w.splits < 512 && ceil_div(K, 2 * w.splits) >= 256) w.splits *= 2;
    w.chunk = (int)(ceil_div(ceil_div(K, w.splits), 64) * 64);
    w.splits = (int)ceil_div(K, w.chunk);
    w.part = take(4LL * w.splits * T * w.rpitch);
    const int E = count + 1;
    ExpertsSpace &o = w.order;
    o.most_tiles = T / kAdaptersRows + (E < T ? E : T);
    o.list_groups = ceil_div(T, kListPairs);
    o.start = take(4LL * (E + 1));
    o.tiles = take(16 + 16 * o.most_tiles);
    o.list = take(4LL * T);
    o.token = take(4LL * T);
    o.where = take(4LL * T);
    o.counts = take(4 * o.list_groups * E);
    o.runs = take(16 + 16LL * (E < T ? E : T));
    o.tile_run = take(4 * ceil_div(T, w.tile));
  }
  w.bytes = at;
  return w;
}

}  // namespace gemm_f32_impl
