// kdn_lanes.h -- sums over adjacent lanes of a wave.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

namespace kdn {

// The sum of v over groups of N adjacent lanes, in each of them.
template <int N>
__device__ __forceinline__ float lane_sum(float v)
{
    auto dpp = [](float x, auto ctrl) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value,
                                                          0xF, 0xF, true));
    };
    if constexpr (N >= 2)
        v += dpp(v, std::integral_constant<int, 0xB1>{});  // quad [1,0,3,2]
    if constexpr (N >= 4)
        v += dpp(v, std::integral_constant<int, 0x4E>{});  // quad [2,3,0,1]
    if constexpr (N >= 8)
        v += dpp(v, std::integral_constant<int, 0x141>{});  // mirror within 8
    if constexpr (N >= 16)
        v += dpp(v, std::integral_constant<int, 0x140>{});  // mirror within 16
    if constexpr (N >= 32)
        v += __shfl_xor(v, 16);
    if constexpr (N >= 64)
        v += __shfl_xor(v, 32);
    return v;
}

}  // namespace kdn
