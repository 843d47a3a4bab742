// Device helpers of the tiled products: raw buffer resources, the global -> LDS DMA and its
// waits (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace awq {

typedef int int32x4 __attribute__((ext_vector_type(4)));
typedef int int32x16 __attribute__((ext_vector_type(16)));

// Raw buffer resource (gfx9 layout): 48-bit base, stride 0, byte range, 32-bit data format.
// Accesses at offsets >= num_bytes read zero.
__device__ __forceinline__ int32x4 buffer_rsrc(const void* base, unsigned num_bytes) {
  const unsigned long long b = (unsigned long long)base;
  int32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(unsigned)(b & 0xffffffffu));
  r[1] = __builtin_amdgcn_readfirstlane((int)(unsigned)((b >> 32) & 0xffffu));
  r[2] = __builtin_amdgcn_readfirstlane((int)num_bytes);
  r[3] = 0x00020000;
  return r;
}

__device__ __forceinline__ unsigned lds_address(const void* p) {
  return __builtin_amdgcn_readfirstlane(
      (int)(unsigned)(size_t)(const __attribute__((address_space(3))) void*)p);
}

// One wave-level 16-byte-per-lane DMA: lane l's 16 bytes at buffer offset voff + soff land at
// LDS byte lds + 16 l.  Inline assembly keeps the compiler's automatic waits from draining
// the DMA queue before unrelated LDS reads; every wait for these transfers is explicit.  Its data
// goes to LDS: no VGPR of the asm is overwritten after the statement.
__device__ __forceinline__ void lds_dma16(const int32x4& rsrc, unsigned lds, unsigned voff,
                                          unsigned soff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
      : "memory", "m0");
}

// s_waitcnt immediate: vmcnt(VM), lgkmcnt(0).
template <int VM>
struct WaitVmLgkm0 {
  static_assert(VM >= 0 && VM < 64, "vmcnt range");
  static constexpr int value = (VM & 0xF) | ((VM >> 4) << 14) | (7 << 4);
};

}  // namespace awq
