// Loads and stores of the attention's and the trees' kernels (gfx950).
#pragma once

#include "sv_device.h"

namespace sv {

namespace {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));    // 16 bytes at any element's address

// A load or store of memory that the compiler cannot tell to be global (an address that was itself
// loaded): as a flat access it would wait for every LDS access under way too.
#define SV_GLOBAL __attribute__((address_space(1)))
template <typename T> __device__ inline T load_global(const void *p)
{
    return *(const SV_GLOBAL T *)p;
}
template <typename T> __device__ inline T load_once(const void *p)       // streams past the caches
{
    return __builtin_nontemporal_load((const SV_GLOBAL T *)p);
}
template <typename T> __device__ inline void store_global(void *p, T v) { *(SV_GLOBAL T *)p = v; }

}  // namespace

}  // namespace sv
