// Device helpers of the per-channel operators (ssm_*.hip, shortconv.hip,
// groupnorm.hip): short vectors of consecutive channels, the order of
// workgroups over the XCDs, loads through descriptors, softplus and SiLU, row
// broadcasts and halving sums, and the lookup of a step's states.
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>
#include <type_traits>
#include <utility>

#include "wkv7_device.h"

namespace wkv7 {

// E consecutive elements, loaded and stored in pieces of at most 16 bytes.
constexpr int pack_align(int bytes) { return (bytes & -bytes) < 16 ? (bytes & -bytes) : 16; }
template <typename T, int E>
struct alignas(pack_align(int(sizeof(T)) * E)) Pack {
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

// Buffer descriptors: loads past `bytes` give 0 and stores past it are dropped.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t buf_rsrc(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, int(bytes > 0 ? bytes : 0), 0x00020000);
}

// An offset past any descriptor's end (they have less than 2^31 bytes), also with the offsets within a
// load added: those must not come round to the start.
constexpr uint32_t kNowhere = 0x80000000u;

// E consecutive elements as they were loaded, for loads that are in flight while other work
// goes on: nothing is computed from the registers until get().  WHOLE: they start on 4 bytes and
// come in loads of up to 16 bytes; else one by one, those past the first n as 0.
template <typename T, int E, bool WHOLE>
struct Raw {
    static constexpr bool kWhole = WHOLE && sizeof(T) * E >= 4;
    static constexpr int W = kWhole ? int(sizeof(T)) * E / 4 : E;
    uint32_t w[W];

    __device__ __forceinline__ void load(rsrc_t r, uint32_t off, int n) {
        if constexpr (!kWhole) {
            #pragma unroll
            for (int i = 0; i < E; ++i) {
                const uint32_t o = i < n ? off + uint32_t(sizeof(T)) * i : kNowhere;
                if constexpr (sizeof(T) == 4) w[i] = __builtin_amdgcn_raw_buffer_load_b32(r, o, 0, 0);
                else w[i] = uint32_t(__builtin_amdgcn_raw_buffer_load_b16(r, o, 0, 0));
            }
        } else if constexpr (W >= 4) {
            #pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                const auto x = __builtin_amdgcn_raw_buffer_load_b128(r, off + 16 * i, 0, 0);
                w[4 * i] = x[0]; w[4 * i + 1] = x[1]; w[4 * i + 2] = x[2]; w[4 * i + 3] = x[3];
            }
        } else if constexpr (W == 2) {
            const auto x = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0);
            w[0] = x[0]; w[1] = x[1];
        } else {
            w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else if constexpr (!kWhole) return __uint_as_float(w[i] << 16);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};

// Store E floats in type T; dropped past the descriptor's end.  WHOLE as above, n: how many are there.
template <typename T, int E, bool WHOLE>
__device__ __forceinline__ void buf_store(rsrc_t r, uint32_t off, const float* v, int n) {
    Pack<T, E> o;
    #pragma unroll
    for (int i = 0; i < E; ++i) narrow(v[i], o.e[i]);
    if (WHOLE && n >= E && sizeof(T) * E >= 4) {
        if constexpr (sizeof(T) * E == 4) {
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, o), r, off, 0, 0);
        } else if constexpr (sizeof(T) * E == 8) {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, o), r, off, 0, 0);
        } else if constexpr (sizeof(T) * E >= 16) {
            typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
            struct Q { u32x4 q[sizeof(T) * E / 16]; };
            const Q q = __builtin_bit_cast(Q, o);
            #pragma unroll
            for (int i = 0; i < int(sizeof(T)) * E / 16; ++i) __builtin_amdgcn_raw_buffer_store_b128(q.q[i], r, off + 16 * i, 0, 0);
        }
        return;
    }
    #pragma unroll
    for (int i = 0; i < E; ++i)
        if (i < n) {
            if constexpr (sizeof(T) == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, o.e[i]), r, off + 4 * i, 0, 0);
            else __builtin_amdgcn_raw_buffer_store_b16(o.e[i], r, off + 2 * i, 0, 0);
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

// log(1 + e) for 0 <= e <= 1 to fp32 relative accuracy: 2 atanh(s) = 2 s + 2 s^3 p(s^2) with
// s = e / (2 + e) <= 1/3 and p the cubic nearest to its series there (5e-9 of the result;
// fitted by least squares reweighted towards the largest error).
__device__ __forceinline__ float log1p_unit(float e) {
    const float s = e * __builtin_amdgcn_rcpf(2.f + e), q = s * s, s2 = s + s;
    float p = 0.28024465f;
    p = fmaf(p, q, 0.27999139f);
    p = fmaf(p, q, 0.40021700f);
    p = fmaf(p, q, 0.66666412f);
    return fmaf(p * q, s, s2);
}
// softplus(v) = max(v, 0) + log(1 + exp(-|v|)); NaN stays NaN.
__device__ __forceinline__ float softplusf_(float v) {
    const float l = log1p_unit(__builtin_amdgcn_exp2f(-kLog2e * fabsf(v)));
    return fmaxf(v, 0.f) + l;
}

// f(0), f(1) .. f(N - 1) with the index known at compile time.
template <int N, typename F, int... I>
__device__ __forceinline__ void static_for_(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
    static_for_<N>(f, std::make_integer_sequence<int, N>{});
}

// The value that lane T of the row of 16 lanes has, in all of them (an operand modifier of the
// instruction that uses it).
template <int T>
__device__ __forceinline__ float row_lane(float x) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x150 + T, 0xF, 0xF, true));   // row_newbcast
}

// y[j] = sum_i c[i] of lane T + j of the row times h[j][i], for j = 0 .. 3.  Written out because
// the compiler folds a row broadcast into products but not into fused multiply-adds.  The four
// sums take turns, so that none waits for itself; the wait before the first instruction is the one
// between the write of a register and its read across lanes.
template <int T, int N>
__device__ __forceinline__ void row_dot4(const float* c, const float (&h)[4][N], f32x4& y) {
    constexpr int A = T, B = T + 1, C = T + 2, D = T + 3;
    float y0, y1, y2, y3;
#define WKV7_BC(t) " row_newbcast:%c[" t "] row_mask:0xf bank_mask:0xf\n"
    asm("s_nop 1\n"
        "v_mul_f32_dpp %0, %4, %5" WKV7_BC("a") "v_mul_f32_dpp %1, %4, %6" WKV7_BC("b")
        "v_mul_f32_dpp %2, %4, %7" WKV7_BC("c") "v_mul_f32_dpp %3, %4, %8" WKV7_BC("d")
        : "=&v"(y0), "=&v"(y1), "=&v"(y2), "=&v"(y3)
        : "v"(c[0]), "v"(h[0][0]), "v"(h[1][0]), "v"(h[2][0]), "v"(h[3][0]), [a] "n"(A), [b] "n"(B), [c] "n"(C), [d] "n"(D));
    #pragma unroll
    for (int i = 1; i < N; ++i)
        asm("s_nop 1\n"
            "v_fmac_f32_dpp %0, %4, %5" WKV7_BC("a") "v_fmac_f32_dpp %1, %4, %6" WKV7_BC("b")
            "v_fmac_f32_dpp %2, %4, %7" WKV7_BC("c") "v_fmac_f32_dpp %3, %4, %8" WKV7_BC("d")
            : "+v"(y0), "+v"(y1), "+v"(y2), "+v"(y3)
            : "v"(c[i]), "v"(h[0][i]), "v"(h[1][i]), "v"(h[2][i]), "v"(h[3][i]), [a] "n"(A), [b] "n"(B), [c] "n"(C), [d] "n"(D));
#undef WKV7_BC
    y = f32x4{y0, y1, y2, y3};
}

// a where the bits of m are set, b where they are not: a choice made once, without a branch.
__device__ __forceinline__ float bit_select(uint32_t m, float a, float b) {
    return __uint_as_float((__float_as_uint(a) & m) | (__float_as_uint(b) & ~m));
}

// lo where bit M of the lane is 0, hi where it is 1, each summed over the pair of lanes that
// differ in it.
template <int M>
__device__ __forceinline__ float halve(float lo, float hi, int lane) {
    if constexpr (M == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(lo), __float_as_uint(hi), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    } else if constexpr (M == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(lo), __float_as_uint(hi), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    } else {
        static_assert(M <= 2);
        constexpr int ctrl = M == 2 ? kDppQuadXor2 : kDppQuadXor1;
        const bool b = lane & M;
        return (b ? hi : lo) + dpp<ctrl>(b ? lo : hi);
    }
}

// Tokens of sequence b that are there: lengths[b] held to [0, T].
__device__ __forceinline__ int seq_length(const int32_t* lengths, int64_t b, int T) {
    if (!lengths) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : (n > T ? T : n);
}

// Of the rows b0 .. b0 + R, with states slot[], keep those as mine[] that come first of the rows
// that name their state (a later row of the same index has no request).  Every thread of the
// workgroup calls it with the same arguments; `threads` is the workgroup's size.
template <int R>
__device__ __forceinline__ void first_of_slots(const int32_t* index, int b0, const int* slot, bool* mine, int threads) {
    int seen = 0;
    for (int j = threadIdx.x; j < b0; j += threads) {
        const int s = index[j];
        #pragma unroll
        for (int r = 0; r < R; ++r) seen |= (s == slot[r]) << r;
    }
    #pragma unroll
    for (int r = 0; r < R; ++r)
        #pragma unroll
        for (int q = 0; q < r; ++q) seen |= (slot[q] == slot[r]) << r;
    // one barrier for all the rows: each wave's bits, then everybody's
    __shared__ int s_seen;
    if (threadIdx.x == 0) s_seen = 0;
    __syncthreads();
    #pragma unroll
    for (int r = 0; r < R; ++r)
        if (__any(seen >> r & 1) && (threadIdx.x & 63) == 0) atomicOr(&s_seen, 1 << r);
    __syncthreads();
    const int all = s_seen;
    #pragma unroll
    for (int r = 0; r < R; ++r) mine[r] = mine[r] && !(all >> r & 1);
}

}  // namespace wkv7
