// Global memory to LDS by DMA: the pieces that gemm.hip, grouped.hip and ns_backward.hip share.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

namespace mns {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

constexpr int kChunks = 8;                  // 16-byte chunks of a 128-byte LDS row (one k-tile)
constexpr int kBufferFlags = 0x00020000;    // buffer resource word 3: raw loads, gfx9 family

// Loads are checked dword by dword against `bytes` (>= 0), the scalar offset counted: one that starts at or
// past the end, or that the end falls inside of, reads as zero.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  const int n = bytes > 0x7FFFFFFFLL ? 0x7FFFFFFF : (int)bytes;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, n, kBufferFlags);
}

// 16 bytes per lane, global -> LDS: lane l's land at dst + 16 l (dst wave-uniform, carried in M0).
// Kept out of lambdas: the host pass of a kernel must not see the LDS address-space cast.
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, u32x4* dst, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 16, voff, soff, 0, 0);
}

__device__ __forceinline__ int swz(int row, int chunk) {
  return row * kChunks + (chunk ^ ((row ^ ((row >> 3) & 3)) & 7));
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(lds_void*)p;
}

// s_waitcnt immediate (gfx9 encoding: vmcnt[3:0] | expcnt[6:4] | lgkmcnt[11:8] | vmcnt[15:14]).
constexpr int kWaitVm0Lgkm0 = 0x0070;       // vmcnt(0) lgkmcnt(0)

// This wave's DMA and LDS accesses are done, then the workgroup meets. No memory fence: the DMA
// traffic is ordered by the explicit counters.
__device__ __forceinline__ void block_sync() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(kWaitVm0Lgkm0);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace mns
