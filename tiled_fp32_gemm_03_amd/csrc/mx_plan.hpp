// Host-only planning of the MX (4-bit microscaled) operators and the
// mixture-of-experts layer: sizes, argument checks and the choice of a
// kernel.  Plain C++17 with no HIP types, like host_plan.hpp; nothing here
// touches a GPU.
#pragma once

#include "host_plan.hpp"

namespace gemm_f32_impl {

// Formats of unquantised matrices (gemm_mixed.h, gemm_mx.h).
constexpr int kBf16 = 0, kF16 = 1, kF32 = 2;
constexpr int kAlongRows = 0, kAlongColumns = 1;

// Values per block, and the bytes of a row's blocks (16 of codes each) and
// scales (one each, rows padded to whole 16 bytes).
constexpr int kMxBlock = 32;
constexpr long long mx_blocks(int K) { return ceil_div(K, kMxBlock); }
constexpr long long mx_code_bytes(int K) { return 16 * mx_blocks(K); }
constexpr long long mx_scale_bytes(int K) { return 16 * ceil_div(mx_blocks(K), 16); }

constexpr bool is_format(int f) { return f == kBf16 || f == kF16 || f == kF32; }
constexpr int format_bytes(int f) { return f == kF32 ? 4 : 2; }

// One MX matrix's row pitches: too short (kInvalidLd) or not multiples of 16
// (kMisaligned).
int check_mx_ld(int K, int ld, int lds);
// Its pointers, for a matrix with elements: null, or not 16-byte aligned.
int check_mx_pointers(const void *codes, const void *scales);
// A row-major matrix with elements: null, or not aligned to its element.
int check_plain_pointer(const void *p, int format);

// ---- gemm_mx's launch table ------------------------------------------------

struct MxEntry {
  int BM, BN, BK, threads;
};
int mx_num_entries();
const MxEntry &mx_entry(int index);
int mx_choose(int M, int N, int K);

// ---- the mixture-of-experts layer ------------------------------------------

constexpr int kMoeMaxTokens = 256, kMoeMaxExperts = 512, kMoeMaxTop = 16,
              kMoeMaxWidth = 1 << 24;
int moe_check_sizes(int T, int E, int top, int H, int I);

// The workspace of one call, as byte offsets (each a multiple of 16).  A pair
// is a token's choice, number token * top + choice; `list` has the pairs by
// expert, then by number.
struct MoeSpace {
  long long logits;  // double [T][E]
  long long ids;     // int [T top]
  long long gates;   // float [T top]
  long long start;   // int [E + 1]: expert e's pairs are list[start[e]] .. list[start[e + 1] - 1]
  long long list;    // int [T top]
  long long active;  // int [1 + E]: how many experts were chosen, and which, rising
  long long u;       // float [T top][upitch], by place in the list: the inner values
  long long part;    // float [T top][ypitch], by pair: the experts' results
  long long bytes;
  long long upitch, ypitch;
};
MoeSpace moe_space(int T, int E, int top, int H, int I);

}  // namespace gemm_f32_impl
