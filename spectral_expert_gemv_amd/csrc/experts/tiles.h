// What the tiled products (16-bit and 8-bit operands) share: copies into LDS
// that are waited for by count, and the order of the output tiles.
#pragma once
#include "experts.h"

namespace bitsmoe {
namespace experts {

// Copies 16 bytes per lane from `src` to LDS at lds + 16 lane.  (The
// compiler would wait for all such copies before any LDS read, so the copy is
// an opaque statement without register outputs; the loop below waits for its
// copies by count.  The LDS address is an operand in m0, so the compiler knows
// what it holds; the copy may not be the instruction after the one that sets it.)
__device__ __forceinline__ void copy16(const void* src, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(src), "{m0}"(lds) : "memory");
}
// all but the last kLeft copies of the wave have landed
template <int kLeft>
__device__ __forceinline__ void wait_copies() {
  static_assert(kLeft < 16, "vmcnt field");
  __builtin_amdgcn_s_waitcnt(0x0F70 | kLeft);
}
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

constexpr int kUnits = 256;  // compute units of an MI355X, one work-group each (its LDS)

// Tile `id` of mt x nt in the order that keeps the 32 work-groups of an XCD on
// shared operand rows (in its L2): 4 row tiles by 8 column tiles, then the
// next columns.
__device__ __forceinline__ void tile_place(uint32_t id, int mt, int nt, int& m, int& n) {
  const uint32_t g = id / (4u * nt), r = id - g * (4u * nt);
  const uint32_t gm = min(4, mt - (int)g * 4);
  m = g * 4 + r % gm;
  n = r / gm;
}

}  // namespace experts
}  // namespace bitsmoe
