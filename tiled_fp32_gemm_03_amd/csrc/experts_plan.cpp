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

// Thin products where an expert has few pairs: they read its weights once for 16 of
// them.  Thin and tiles, us, by pairs to an expert (experts, widths): 4 (8, 4096 / 2048)
// 114 and 124, 8 136 and 125, 16 166 and 130; 4 (64, 2048 / 1024) 163 and 171, 8 286
// and 174; 8 (8, 512 / 512) 21 and 25.
bool experts_thin(int T, int E, int top) {
  const long long pairs = (long long)T * top;
  return T <= kMoeMaxTokens && pairs <= 6LL * E;
}

namespace {

// Microseconds of n tiles of `steps`: rounds of what the chip holds at once (partial
// ones cost half of what is missing), each step and a tile's start and end.
double tiles_us(int tile, double n, double steps) {
  const bool large = tile == 256;
  const double r = n / (large ? 256 : 512);
  const double rounds = r <= 1 ? 1 : (r + (double)(long long)(r + 0.999)) / 2;
  return rounds * (steps * (large ? 2.0 : 1.35) + (large ? 12 : 6));
}

}  // namespace

// The tile of less modelled time.  128 and 256, us (tokens, experts, choices, widths;
// forward and training step): 512, 8, 2, 4096 / 2048 153 and 192, 529 and 613; 1,024,
// the same, 243 and 192, 763 and 678; 4,096, 64, 4, 2048 / 1024 368 and 384, 1,440 and
// 1,385; 8,192, the same, 620 and 575, 2,250 and 1,992; 8,192, 4, 1, 512 / 2048 108 and
// 125, 453 and 578; 8,192, 8, 2, 4096 / 4096 2,005 and 1,628.
int experts_tile(int T, int E, int top, int H, int I, bool trains) {
  const double pairs = (double)T * top, asked = E < pairs ? E : pairs, rows = asked ? pairs / asked : 0;
  auto cost = [&](int tile) {
    const double m = asked * (rows / tile + 0.5);  // experts' last tiles are half full
    const double h = (double)ceil_div(H, tile), i = (double)ceil_div(I, tile), i2 = (double)ceil_div(2LL * I, tile);
    double t = tiles_us(tile, m * i2, H / 64.0) + tiles_us(tile, m * h, I / 64.0);
    if (trains)
      t += tiles_us(tile, m * i, H / 64.0) + tiles_us(tile, m * h, I / 32.0) +
           tiles_us(tile, E * i2 * h, rows / 64) + tiles_us(tile, E * h * i, rows / 64);
    return t;
  };
  return cost(256) < cost(128) ? 256 : 128;
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
  w.part = take(4 * pairs * w.hpitch);
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

// Thin products while 64 rows at a time cost less than the tiles' five launches.  Tiles
// and thin, us (rows, N x K): 65, 4096 x 4096 51 and 35; 128 56 and 44; 256 52 and 80;
// 512, 1024 x 1024 35 and 31; 1,024 37 and 58; 256, 8192 x 2048 58 and 83; 200, 2048 x
// 8192 65 and 60; 192, 16384 x 4096 85 and 113.
bool adapters_thin(int T, int N, int K) {
  return T <= kAdaptersThin ||
         (T <= kAdaptersMostThin && ceil_div(T, kAdaptersThin) * N * K <= 1LL << 25);
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
  w.v = take(4LL * T * w.rpitch);
  w.splits = w.wide_splits = 1;
  w.chunk = w.wide_chunk = K;
  if (!adapters_thin(T, N, K)) {
    // Tiles of 256 where those of 128 are more than the chip holds at once (else they take
    // K in parts) and the modelled time is less, with a tenth off for the larger ones.  128
    // and 256, us (rows, N x K): 2,048, 4096 x 1024 41 and 60; 1,280, 6656 x 4096 123 and
    // 115; 512, 18432 x 8192 289 and 209; 20,000, 300 x 4096 114 and 145; 20,000, 390 x
    // 4096 166 and 147; 8,192, 1536 x 4096 161 and 127; 4,096, 4096 x 4096 161 and 136;
    // 100,000, 100 x 4096 481 and 533; 100,000, 160 x 2048 328 and 312.  Of 47 sizes the
    // rule loses 10% in two: 33,000, 500 x 2048 141 and 156; 30,000, 640 x 1024 106 and 115.
    const long long wide = ceil_div(T, 128) * ceil_div(N, 128), large = ceil_div(T, 256) * ceil_div(N, 256);
    const double steps = K / 64.0;
    w.tile = wide > 512 && 0.9 * tiles_us(256, large, steps) < tiles_us(128, wide, steps) ? 256 : 128;
    // The products with A: row tiles of kAdaptersRows, K in parts until there are
    // two workgroups to a compute unit, of 256 values at least.
    const long long tiles = (ceil_div(T, kAdaptersRows) + count / 2) * ceil_div(R, kAdaptersRows);
    while (tiles * w.splits < 512 && ceil_div(K, 2 * w.splits) >= 256) w.splits *= 2;
    w.chunk = (int)(ceil_div(ceil_div(K, w.splits), 64) * 64);
    w.splits = (int)ceil_div(K, w.chunk);
    w.part = take(4LL * w.splits * T * w.rpitch);
    // The projection: K in parts while there are two tiles to a compute unit at most, of
    // 512 values at least (a compute unit is fed 35 to 45 KB a microsecond, so few tiles
    // take long however they are scheduled).
    while (2 * wide * w.wide_splits <= 512 && ceil_div(K, 2 * w.wide_splits) >= 512) w.wide_splits *= 2;
    w.wide_chunk = (int)(ceil_div(ceil_div(K, w.wide_splits), 64) * 64);
    w.wide_splits = (int)ceil_div(K, w.wide_chunk);
    w.npitch = ceil_div(N, 8) * 8;
    w.wide_part = take(w.wide_splits > 1 ? 4 * w.wide_splits * T * w.npitch : 0);
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
    o.tile_run = take(4 * ceil_div(T, 128));  // (of either tile)
  }
  w.bytes = at;
  return w;
}

}  // namespace gemm_f32_impl
