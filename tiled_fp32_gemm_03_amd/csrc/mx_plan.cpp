// Host-only planning of the MX operators (see mx_plan.hpp).
#include "mx_plan.hpp"

#include <cstdint>

namespace gemm_f32_impl {

namespace {

bool misaligned(const void *p, int align) {
  return (reinterpret_cast<std::uintptr_t>(p) & static_cast<std::uintptr_t>(align - 1)) != 0;
}

}  // namespace

int check_mx_ld(int K, int ld, int lds) {
  const long long c = mx_code_bytes(K), s = mx_scale_bytes(K);
  if (ld < (c > 16 ? c : 16) || lds < (s > 16 ? s : 16)) return kInvalidLd;
  return (ld % 16 || lds % 16) ? kMisaligned : kOk;
}

int check_mx_pointers(const void *codes, const void *scales) {
  if (codes == nullptr || scales == nullptr) return kNullPtr;
  return misaligned(codes, 16) || misaligned(scales, 16) ? kMisaligned : kOk;
}

int check_plain_pointer(const void *p, int format) {
  if (p == nullptr) return kNullPtr;
  return misaligned(p, format_bytes(format)) ? kMisaligned : kOk;
}

namespace {

// Index = launch-table entry of gemm_mx.
const MxEntry kMxEntries[] = {
    {64, 64, 128, 256},    // operands straight from memory, any size
    {256, 256, 256, 256},  // direct-load tiles, 128 x 128 per wave
    {128, 128, 256, 256},  // direct-load tiles, 64 x 64 per wave
    {32, 16, 256, 256},    // few rows: K shared by the waves, B read once
};

}  // namespace

int mx_num_entries() { return (int)(sizeof(kMxEntries) / sizeof(kMxEntries[0])); }
const MxEntry &mx_entry(int index) { return kMxEntries[index]; }
// 256 x 256 tiles where they fill most of the chip; otherwise the entry with
// the least modelled time in ns, from rounds of workgroups on 256 compute
// units and a straight line in K through measured times, us (entries 0, 2 and
// 3): 64 x 2048 x 16384 113, -, 12.0; 100 x 8192 x 4096 31, -, 35; 128 x 8192 x
// 4096 31, 17, 37; 256 x 512 x 16384 113, 51, 12; 256 x 2048 x 4096 31, 13.4,
// 18.6; 256 x 8192 x 512 8.7, 6.3, 19; 512 x 8192 x 16384 448, 60, -; 33 x 8192 x
// 512 4.9, -, 6.0.
int mx_choose(int M, int N, int K) {
  if (M >= 256 && N >= 256 && ceil_div(M, 256) * ceil_div(N, 256) >= 192) return 1;
  if (M <= 32) return 3;
  const double k = K / 1024.0;
  auto rounds = [&](int bm, int bn) { return ceil_div(ceil_div(M, bm) * ceil_div(N, bn), 256); };
  const double direct = 2000 + (300 + 6850 * k) * (double)rounds(64, 64);
  const double few = 2400 + (900 + 530 * k) * (double)rounds(32, 16);
  int best = few < direct ? 3 : 0;
  if (M >= 128 && N >= 128) {
    const double filled = (double)(ceil_div(M, 128) * ceil_div(N, 128)) * 0.95 / 256;
    double tiles = 1500 + (1000 + 2950 * k) * (filled > 1 ? filled : 1);
    if (tiles < 5300) tiles = 5300;  // its start and end alone
    if (tiles < (best == 3 ? few : direct)) best = 2;
  }
  return best;
}

int moe_check_sizes(int T, int E, int top, int H, int I) {
  if (T < 0 || E < 0 || top < 0 || H < 1 || I < 1) return kInvalidDim;
  if (T > kMoeMaxTokens || E > kMoeMaxExperts || top < 1 || top > kMoeMaxTop || top > E ||
      H > kMoeMaxWidth || I > kMoeMaxWidth)
    return kBadArg;
  return kOk;
}

MoeSpace moe_space(int T, int E, int top, int H, int I) {
  MoeSpace w;
  long long at = 0;
  const long long pairs = (long long)T * top;
  auto take = [&at](long long bytes) {
    const long long from = at;
    at += ceil_div(bytes, 16) * 16;
    return from;
  };
  w.upitch = ceil_div(I, 8) * 8;
  w.ypitch = ceil_div(H, 4) * 4;
  w.logits = take(8LL * T * E);
  w.ids = take(4 * pairs);
  w.gates = take(4 * pairs);
  w.start = take(4LL * (E + 1));
  w.list = take(4 * pairs);
  w.active = take(4LL * (E + 1));
  w.u = take(4 * pairs * w.upitch);
  w.part = take(4 * pairs * w.ypitch);
  w.bytes = at;
  return w;
}

}  // namespace gemm_f32_impl
