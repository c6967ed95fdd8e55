// Vector access to tensors of any alignment, and reductions over small groups
// of lanes: shared by the AdamW and MX4 kernels.
#pragma once

#include "common.h"

namespace shp {

// Global-memory access (see ldg, stg) for a vector at an address aligned to ALIGN bytes only (global
// memory takes vector accesses at any element's address).
template <class V, int ALIGN>
__device__ __forceinline__ V ldg_any(const void* p) {
  typedef V U __attribute__((aligned(ALIGN)));
  return *(const __attribute__((address_space(1))) U*)p;
}
template <class V, int ALIGN>
__device__ __forceinline__ void stg_any(void* p, const V& v) {
  typedef V U __attribute__((aligned(ALIGN)));
  *(__attribute__((address_space(1))) U*)p = v;
}

// The same for data that is read or written once: not kept in the caches.
template <class V, int ALIGN>
__device__ __forceinline__ V ldg_once(const void* p) {
  typedef V U __attribute__((aligned(ALIGN)));
  return __builtin_nontemporal_load((const __attribute__((address_space(1))) U*)p);
}
template <class V, int ALIGN>
__device__ __forceinline__ void stg_once(void* p, const V& v) {
  typedef V U __attribute__((aligned(ALIGN)));
  __builtin_nontemporal_store(v, (__attribute__((address_space(1))) U*)p);
}

// Largest of v over groups of 4, 8 or 16 consecutive lanes, in every lane.
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  static_assert(LANES == 4 || LANES == 8 || LANES == 16, "lanes of a group");
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));  // quad_perm 1 0 3 2
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true));  // quad_perm 2 3 0 1
  if constexpr (LANES >= 8)
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true));  // row_half_mirror
  if constexpr (LANES == 16)
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true));  // row_mirror
  return v;
}

}  // namespace shp
