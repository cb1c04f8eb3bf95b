// Device helpers shared by the tiled GEMM kernels (gemm.hip, int8.hip):
// buffer descriptors, LDS swizzle, the counted barrier and the tile order.
#pragma once

#include "device_common.h"

namespace qlora {

constexpr uint32_t kOOB = 0x80000000u;         // buffer offset that reads as 0

// LDS tile of 128-byte rows in 8 chunks of 16 bytes: chunk' = chunk ^ swz_g(row)
__device__ __forceinline__ int swz_g(int row) {
  return ((row >> 1) & 7) ^ ((row & 1) << 1);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

// s_waitcnt vmcnt(n) lgkmcnt(0), then a workgroup barrier that is also a
// compiler memory barrier.  Outstanding LDS-DMA loads beyond the n newest
// are complete afterwards.
template <int N>
__device__ __forceinline__ void barrier_keep_vmem() {
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (7 << 4) | (0 << 8));
  asm volatile("s_barrier" ::: "memory");
}

// tile index -> (token tile, column tile): XCD-major, then groups of 4 token tiles
__device__ __forceinline__ void tile_coords(int pid, int mt, int nt, int& tm, int& tn) {
  const int total = mt * nt;
  const int xcd = pid & 7;
  const int base = total >> 3;
  const int rem = total & 7;
  const int q = xcd * base + (xcd < rem ? xcd : rem) + (pid >> 3);
  constexpr int GM = 4;
  const int group = q / (GM * nt);
  const int first = group * GM;
  const int gm = (mt - first) < GM ? (mt - first) : GM;
  const int local = q - group * GM * nt;
  tm = first + local % gm;
  tn = local / gm;
}

}  // namespace qlora
