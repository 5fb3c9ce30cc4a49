// ls_wave64.hpp -- moves and sums of 64-bit values across a wave (gfx950): the steps of
// wave_inclusive_scan, each moving both halves.
#pragma once
#include "ls_device.hpp"

namespace ls {

template <int CTRL, int ROW_MASK, class T>
__device__ __forceinline__ T dpp_move64(T v)
{
    static_assert(sizeof(T) == 8, "64-bit values");
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = dpp_move<CTRL, ROW_MASK>(0u, uint32_t(b));
    const uint32_t hi = dpp_move<CTRL, ROW_MASK>(0u, uint32_t(b >> 32));
    return __builtin_bit_cast(T, (uint64_t(hi) << 32) | lo);
}

template <class T>
__device__ __forceinline__ T wave_inclusive_sum64(T v)
{
    v += dpp_move64<DPP_ROW_SHR1, 0xf>(v);
    v += dpp_move64<DPP_ROW_SHR2, 0xf>(v);
    v += dpp_move64<DPP_ROW_SHR4, 0xf>(v);
    v += dpp_move64<DPP_ROW_SHR8, 0xf>(v);
    v += dpp_move64<DPP_ROW_BCAST15, 0xa>(v);
    v += dpp_move64<DPP_ROW_BCAST31, 0xc>(v);
    return v;
}

template <class T>
__device__ __forceinline__ T read_lane64(T v, int lane)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = read_lane(uint32_t(b), lane), hi = read_lane(uint32_t(b >> 32), lane);
    return __builtin_bit_cast(T, (uint64_t(hi) << 32) | lo);
}

}  // namespace ls
