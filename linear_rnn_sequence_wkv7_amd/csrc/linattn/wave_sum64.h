// Running sums over the lanes of a wave in 64 bits.
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace wkv7 {
namespace linattn {

// The value of another lane of the row of 16 (0 where there is none), of one lane.
template <int CTRL>
__device__ __forceinline__ double dpp64(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const int lo = __builtin_amdgcn_update_dpp(0, int(u), CTRL, 0xF, 0xF, true);
    const int hi = __builtin_amdgcn_update_dpp(0, int(u >> 32), CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(double, uint64_t(uint32_t(hi)) << 32 | uint32_t(lo));
}
__device__ __forceinline__ double lane64(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane(int(u), lane), hi = __builtin_amdgcn_readlane(int(u >> 32), lane);
    return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}
// The sum over lanes 0 .. lane: within a row of 16, then the rows before it.
__device__ __forceinline__ double running_sum(double v, int lane) {
    v += dpp64<0x111>(v);   // row_shr by 1, 2, 4, 8
    v += dpp64<0x112>(v);
    v += dpp64<0x114>(v);
    v += dpp64<0x118>(v);
    const double r0 = lane64(v, 15), r1 = lane64(v, 31), r2 = lane64(v, 47);
    return v + (lane >= 48 ? r0 + r1 + r2 : lane >= 32 ? r0 + r1 : lane >= 16 ? r0 : 0.0);
}

}  // namespace linattn
}  // namespace wkv7
