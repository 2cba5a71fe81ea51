// What the kernel files share: the launch that times a kernel, element access, and reductions and
// scans over a wave64.  Included by sv_kernels.hip, sv_filter.hip and sv_cache.hip.
#pragma once

#include <math.h>
#include <hip/hip_ext.h>

#include "sv_internal.h"

namespace sv {

// Launches one kernel on the call's stream.  When its kind is being timed, the kind's start
// and stop events are handed to the dispatch itself (hipExtLaunchKernel stamps them with the
// kernel's own begin and end), so timing puts no marker packets, and no extra gaps, between
// dependent kernels.  Untimed launches are ordinary launches (capturable in a HIP graph).
inline bool timed(const Launch &ln, int kind) { return ln.ev && ((ln.mask >> kind) & 1u); }

#define SV_LAUNCH(ln, kind, kernel, grid, block, lds, ...)                                        \
    do {                                                                                          \
        if (timed((ln), (kind)))                                                                  \
            hipExtLaunchKernelGGL(kernel, (grid), (block), (std::uint32_t)(lds), (ln).stream,     \
                                  (ln).ev[2 * (kind)], (ln).ev[2 * (kind) + 1], 0u, __VA_ARGS__); \
        else                                                                                      \
            hipLaunchKernelGGL(kernel, (grid), (block), (lds), (ln).stream, __VA_ARGS__);         \
    } while (0)

// ------------------------------------------------------------------ element access

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// 16-byte load that streams past the caches (logits are read once per pass)
__device__ inline uint4 load_stream(const char *p)
{
    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
}

__device__ inline uint4 load_plain(const char *p) { return *reinterpret_cast<const uint4 *>(p); }

template <int DT> struct Elt;

template <> struct Elt<0> {  // float32
    static constexpr int EPV = 4;
    static constexpr int BYTES = 4;
    __device__ static inline void unpack(const uint4 v, float (&x)[4])
    {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
    __device__ static inline float one(const char *base, size_t i)
    {
        return reinterpret_cast<const float *>(base)[i];
    }
};

template <> struct Elt<1> {  // bfloat16 = the upper half of a float32: widening is exact
    static constexpr int EPV = 8;
    static constexpr int BYTES = 2;
    __device__ static inline void unpack(const uint4 v, float (&x)[8])
    {
        x[0] = __uint_as_float(v.x << 16);
        x[1] = __uint_as_float(v.x & 0xffff0000u);
        x[2] = __uint_as_float(v.y << 16);
        x[3] = __uint_as_float(v.y & 0xffff0000u);
        x[4] = __uint_as_float(v.z << 16);
        x[5] = __uint_as_float(v.z & 0xffff0000u);
        x[6] = __uint_as_float(v.w << 16);
        x[7] = __uint_as_float(v.w & 0xffff0000u);
    }
    __device__ static inline float one(const char *base, size_t i)
    {
        return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(base)[i] << 16);
    }
};

__device__ inline bool aligned16(const char *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// EPV ids e0..e0+EPV-1 of a row; ids >= V read as `fill`.  One 16-byte load when the
// row is 16-byte aligned and the vector is whole, element loads otherwise.
template <int DT>
__device__ inline void load_elems(const char *row, bool aligned, int e0, int V, float fill,
                                  float (&x)[Elt<DT>::EPV])
{
    constexpr int E = Elt<DT>::EPV;
    if (aligned && e0 + E <= V) {
        Elt<DT>::unpack(load_plain(row + (size_t)e0 * Elt<DT>::BYTES), x);
    } else {
#pragma unroll
        for (int k = 0; k < E; ++k)
            x[k] = (e0 + k < V) ? Elt<DT>::one(row, (size_t)(e0 + k)) : fill;
    }
}

// 2^(d * log2(e)/T) for d <= 0 with the scale split in two floats (see Scale).
__device__ inline float exp2s(float d, float hi, float lo)
{
    float a = d * hi;
    a = __builtin_fmaf(d, lo, a);
    return __builtin_amdgcn_exp2f(a);
}

template <int E> __device__ inline float tree_sum(const float (&t)[E]);
template <> __device__ inline float tree_sum<4>(const float (&t)[4]) { return (t[0] + t[1]) + (t[2] + t[3]); }
template <> __device__ inline float tree_sum<8>(const float (&t)[8])
{
    return ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
}

// ------------------------------------------------------------------ wave64 / block reductions
// Butterfly reductions whose lane exchanges run on the VALU, with no LDS round trip: steps 0
// and 1 are the DPP quad permutations lane^1 and lane^2; steps 2 and 3 mirror lanes within 8
// and within 16 (once the quads are reduced, the mirrored lane holds what lane^4, lane^8
// would); step 4 swaps 16-lane rows (lane^16, v_permlane16_swap) and step 5 the wave's halves
// (lane^32, v_permlane32_swap).  Each step combines the same two operands in both lanes of a
// pair, so every lane ends with the same bits and the results are deterministic.  The whole
// wave (or, for the half-wave forms, the whole 32-lane half) must be active.

template <int S>
__device__ __forceinline__ int lane_xch(int v)
{
    const int lane = threadIdx.x & 63;
    if constexpr (S == 0)
        return __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, false);   // quad_perm 1,0,3,2
    else if constexpr (S == 1)
        return __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, false);   // quad_perm 2,3,0,1
    else if constexpr (S == 2)
        return __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, false);  // row_half_mirror
    else if constexpr (S == 3)
        return __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, false);  // row_mirror
    else if constexpr (S == 4) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return (lane & 16) ? (int)r[0] : (int)r[1];
    } else {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return (lane & 32) ? (int)r[0] : (int)r[1];
    }
}

template <int S> __device__ __forceinline__ float xch(float v)
{
    return __int_as_float(lane_xch<S>(__float_as_int(v)));
}

template <int S> __device__ __forceinline__ double xch(double v)
{
    return __hiloint2double(lane_xch<S>(__double2hiint(v)), lane_xch<S>(__double2loint(v)));
}

template <int NS, typename T> __device__ __forceinline__ T xmax(T v)
{
    v = fmaxf(v, xch<0>(v));
    v = fmaxf(v, xch<1>(v));
    v = fmaxf(v, xch<2>(v));
    v = fmaxf(v, xch<3>(v));
    v = fmaxf(v, xch<4>(v));
    if constexpr (NS == 6)
        v = fmaxf(v, xch<5>(v));
    return v;
}

template <int NS, typename T> __device__ __forceinline__ T xsum(T v)
{
    v += xch<0>(v);
    v += xch<1>(v);
    v += xch<2>(v);
    v += xch<3>(v);
    v += xch<4>(v);
    if constexpr (NS == 6)
        v += xch<5>(v);
    return v;
}

__device__ inline float wave_max(float v) { return xmax<6>(v); }
__device__ inline double wave_sum(double v) { return xsum<6>(v); }

// The same reductions with the exchanges through the LDS crossbar (ds_bpermute): a longer
// latency per call, but they leave the VALU alone, which matters where the VALU is as busy
// as the memory pipe: the row statistics kernels and the draw's row pass.
template <typename T> __device__ inline T wave_max_lds(T v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor(v, o));
    return v;
}

template <typename T> __device__ inline T wave_sum_lds(T v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v += __shfl_xor(v, o);
    return v;
}

// max and sum over each 32-lane half of the wave (the halves reduce independently)
__device__ inline float half_max(float v) { return xmax<5>(v); }
__device__ inline double half_sum(double v) { return xsum<5>(v); }

// Inclusive prefix sum of a double over the wave's lanes, with DPP moves (fixed order): row
// shifts by 1, 2, 4, 8 give each 16-lane row its own scan, then lane 15's total is added into
// rows 1 and 3 (row_bcast:15) and lane 31's into rows 2 and 3 (row_bcast:31).  Lanes with no
// source read 0.  The whole wave must be active.
template <int CTRL, int ROWS> __device__ __forceinline__ double dpp_move(double v)
{
    const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, ROWS, 0xF, false);
    const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, ROWS, 0xF, false);
    return __hiloint2double(hi, lo);
}

__device__ inline double wave_incl_scan(double v)
{
    v += dpp_move<0x111, 0xF>(v);  // row_shr:1
    v += dpp_move<0x112, 0xF>(v);  // row_shr:2
    v += dpp_move<0x114, 0xF>(v);  // row_shr:4
    v += dpp_move<0x118, 0xF>(v);  // row_shr:8
    v += dpp_move<0x142, 0xA>(v);  // row_bcast:15, rows 1 and 3
    v += dpp_move<0x143, 0xC>(v);  // row_bcast:31, rows 2 and 3
    return v;
}

// The exclusive prefix from the inclusive one: each lane takes its left neighbour's value
// (DPP wave_shr:1), lane 0 takes 0.
__device__ inline double wave_excl_from_incl(double inc) { return dpp_move<0x138, 0xF>(inc); }

// A lane's value read by the whole wave; the lane index must be the same in every lane.
__device__ __forceinline__ int lane_value(int v, int l) { return __builtin_amdgcn_readlane(v, l); }
__device__ __forceinline__ double lane_value(double v, int l)
{
    return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), l),
                            __builtin_amdgcn_readlane(__double2loint(v), l));
}

// lexicographic "better": larger value, then lower id
__device__ inline void take_better(float &v, int &i, float v2, int i2)
{
    if (v2 > v || (v2 == v && i2 < i)) {
        v = v2;
        i = i2;
    }
}

template <int S> __device__ __forceinline__ void argmax_step(float &v, int &i)
{
    const float v2 = xch<S>(v);
    const int i2 = lane_xch<S>(i);
    take_better(v, i, v2, i2);
}

__device__ inline void wave_argmax(float &v, int &i)
{
    argmax_step<0>(v, i);
    argmax_step<1>(v, i);
    argmax_step<2>(v, i);
    argmax_step<3>(v, i);
    argmax_step<4>(v, i);
    argmax_step<5>(v, i);
}

}  // namespace sv
