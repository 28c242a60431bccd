// Device helpers of the per-channel operators (ssm_*.hip, shortconv.hip,
// groupnorm.hip): short vectors of consecutive channels, the order of
// workgroups over the XCDs, exact-enough softplus and SiLU, and the
// column sum that joins partial gradients.
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

#include "wkv7_device.h"

namespace wkv7 {

// E consecutive elements, loaded and stored in pieces of at most 16 bytes.
template <typename T, int E>
struct alignas(sizeof(T) * E < 16 ? sizeof(T) * E : 16) Pack {
    T e[E];
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(bf16_t x) { return bf16_to_f32(x); }
__device__ __forceinline__ void narrow(float x, float& o) { o = x; }
__device__ __forceinline__ void narrow(float x, bf16_t& o) { o = f32_to_bf16(x); }

// p[0 .. E): as one piece where `whole` (all there and aligned), else the first n, zeros after.
template <int E, typename T>
__device__ __forceinline__ Pack<T, E> ld_pack(const T* p, bool whole, int n) {
    if (whole) return *reinterpret_cast<const Pack<T, E>*>(p);
    Pack<T, E> r;
    #pragma unroll
    for (int i = 0; i < E; ++i) r.e[i] = i < n ? p[i] : T(0);
    return r;
}
template <int E, typename T>
__device__ __forceinline__ void st_pack(T* p, const float* v, bool whole, int n) {
    Pack<T, E> r;
    #pragma unroll
    for (int i = 0; i < E; ++i) narrow(v[i], r.e[i]);
    if (whole) {
        *reinterpret_cast<Pack<T, E>*>(p) = r;
        return;
    }
    #pragma unroll
    for (int i = 0; i < E; ++i)
        if (i < n) p[i] = r.e[i];
}
// The same into an array whose type is only known at run time.
template <int E>
__device__ __forceinline__ void st_pack_as(void* p, int64_t i, bool bf16, const float* v, bool whole, int n) {
    if (bf16) st_pack<E>(static_cast<bf16_t*>(p) + i, v, whole, n);
    else st_pack<E>(static_cast<float*>(p) + i, v, whole, n);
}
template <int E>
__device__ __forceinline__ void ld_pack_as(const void* p, int64_t i, bool bf16, float* v, bool whole, int n) {
    if (bf16) {
        const Pack<bf16_t, E> r = ld_pack<E>(static_cast<const bf16_t*>(p) + i, whole, n);
        #pragma unroll
        for (int k = 0; k < E; ++k) v[k] = widen(r.e[k]);
    } else {
        const Pack<float, E> r = ld_pack<E>(static_cast<const float*>(p) + i, whole, n);
        #pragma unroll
        for (int k = 0; k < E; ++k) v[k] = r.e[k];
    }
}

// Workgroups go to the 8 XCDs in turn.  Give each XCD a run of consecutive
// items instead, so that neighbours (which share cache lines) share an L2.
__device__ __forceinline__ int64_t xcd_order(int64_t i, int64_t n) {
    const int64_t q = n >> 3, r = n & 7, x = i & 7;
    return x * q + (x < r ? x : r) + (i >> 3);
}

// Order LDS traffic between the lanes of one wave.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ float sigmoidf_(float x) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// log(1 + e) for 0 <= e <= 1 to fp32 relative accuracy: 2 atanh(s), s = e / (2 + e) <= 1/3,
// by its odd series to s^15 (the next term is below 2^-26 of the first).
__device__ __forceinline__ float log1p_unit(float e) {
    const float s = e * __builtin_amdgcn_rcpf(2.f + e), q = s * s;
    float p = 2.f / 15.f;
    p = fmaf(p, q, 2.f / 13.f);
    p = fmaf(p, q, 2.f / 11.f);
    p = fmaf(p, q, 2.f / 9.f);
    p = fmaf(p, q, 2.f / 7.f);
    p = fmaf(p, q, 2.f / 5.f);
    p = fmaf(p, q, 2.f / 3.f);
    return fmaf(p * q, s, 2.f * s);
}
// softplus(v) = max(v, 0) + log(1 + exp(-|v|)); NaN stays NaN.
__device__ __forceinline__ float softplusf_(float v) {
    const float l = log1p_unit(__builtin_amdgcn_exp2f(-kLog2e * fabsf(v)));
    return (v > 0.f ? v : 0.f) + l;
}

// Tokens of sequence b that are there: lengths[b] held to [0, T].
__device__ __forceinline__ int seq_length(const int32_t* lengths, int64_t b, int T) {
    if (!lengths) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : (n > T ? T : n);
}

// Whether row b comes first of the rows that name its state (a later row of the
// same index has no request).  Every thread of the workgroup calls it with the
// same b; `threads` is the workgroup's size.
__device__ __forceinline__ bool first_of_slot(const int32_t* index, int b, int slot, int threads) {
    int seen = 0;
    for (int j = threadIdx.x; j < b; j += threads) seen |= index[j] == slot;
    return !__syncthreads_or(seen);
}

}  // namespace wkv7
