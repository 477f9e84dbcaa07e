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
  w.bytes = at;
  return w;
}

}  // namespace gemm_f32_impl
