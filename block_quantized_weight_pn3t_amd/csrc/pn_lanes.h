// pn_lanes.h -- values of other lanes of a wave.
#pragma once

#include <type_traits>

#include "pn_common.h"

namespace pn {

typedef unsigned long long u64;

// v of the lane whose number differs in the bits of MASK: moves within rows of 16 lanes, swaps between them. (By
// ds_bpermute an exchange takes some 100 clocks, so about 40.)
template <int MASK>
__device__ __forceinline__ uint32_t moved_by(uint32_t v)
{
    constexpr auto dpp = [](uint32_t w, auto ctrl) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, ctrl.value, 0xF, 0xF, true);
    };
    if constexpr (MASK & 1)
        v = dpp(v, std::integral_constant<int, MASK & 2 ? 0x1B : 0xB1>());  // quad_perm
    else if constexpr (MASK & 2)
        v = dpp(v, std::integral_constant<int, 0x4E>());
    if constexpr (MASK & 4) {  // row_half_mirror is 7: the other two bits back
        v = dpp(v, std::integral_constant<int, 0x141>());
        v = dpp(v, std::integral_constant<int, 0x1B>());
    }
    if constexpr (MASK & 8)
        v = dpp(v, std::integral_constant<int, 0x128>());  // row_ror 8
    if constexpr (MASK & 16) {
        const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);  // the even row's, the odd one's
        v = threadIdx.x & 16 ? p[0] : p[1];
    }
    if constexpr (MASK & 32) {
        const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = threadIdx.x & 32 ? p[0] : p[1];
    }
    return v;
}
template <int MASK>
__device__ __forceinline__ u64 moved_by(u64 v)
{
    return (u64)moved_by<MASK>((uint32_t)(v >> 32)) << 32 | moved_by<MASK>((uint32_t)v);
}

// The sum and the largest over the wave's lanes, in every lane.
template <int MASK = 1>
__device__ __forceinline__ double over_lanes_sum(double v)
{
    v += __builtin_bit_cast(double, moved_by<MASK>(__builtin_bit_cast(u64, v)));
    if constexpr (MASK < 32)
        return over_lanes_sum<2 * MASK>(v);
    else
        return v;
}
template <int MASK = 1, typename V>
__device__ __forceinline__ V over_lanes_max(V v)
{
    typedef typename std::conditional<sizeof(V) == 8, u64, uint32_t>::type Bits;
    const V o = __builtin_bit_cast(V, moved_by<MASK>(__builtin_bit_cast(Bits, v)));
    v = v > o ? v : o;
    if constexpr (MASK < 32)
        return over_lanes_max<2 * MASK>(v);
    else
        return v;
}

}  // namespace pn
