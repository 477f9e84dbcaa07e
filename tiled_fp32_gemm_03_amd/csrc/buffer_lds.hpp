// Direct loads from a bounded buffer into LDS (gfx950), shared by the kernels
// whose lanes may have nothing to load.
#pragma once

#include <hip/hip_runtime.h>

namespace gemm_f32_impl {
namespace {

typedef __amdgpu_buffer_rsrc_t rsrc_t;
constexpr int kOutside = (int)0x80000000u;  // an offset past every record count

// 16 bytes per lane from rsrc[voff + soff] to LDS at lds_addr + 16 lane.
// M0 holds the LDS destination: see ks_load_to_lds16 (w16_tiles.hpp).
__device__ inline void buffer_load_to_lds16(int voff, rsrc_t rsrc, int soff, unsigned lds_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %3 offen lds"
               :
               : "v"(voff), "s"(rsrc), "s"(lds_addr), "s"(soff)
               : "memory", "m0");
}

}  // namespace
}  // namespace gemm_f32_impl
