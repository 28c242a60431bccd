// Linear attention where an array is fp32: v_mfma_f32_16x16x4_f32, every operand fp32 in LDS.
// bf16 arrays beside it are widened on the way there.
#include "linattn_core.h"

namespace wkv7 {
namespace linattn {
namespace {

struct F32Ops {
    using elem = float;
    using Frag = f32x4;
    static constexpr int E = 4, K = 16, L = 32;
    static constexpr int NPY = 1, NPU = 1;

    // Four products of depth 4: element e of the lanes' groups is the e-th one's contraction.
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
        #pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
    template <int D>
    static __device__ __forceinline__ int at(int row, int piece) {
        if constexpr (D >= 64) return row * D * 4 + (piece ^ (row & 15)) * 16;
        else return row * 128 + (piece ^ (row >> 1 & 7)) * 16;
    }
    template <int D>
    static __device__ __forceinline__ Frag row(const char* tile, int r, int m, int g) {
        return *reinterpret_cast<const Frag*>(tile + at<D>(r, 4 * m + g));
    }
    template <int D>
    static __device__ __forceinline__ Frag row_of_state(const char* tile, int r, int m, int g) { return row<D>(tile, r, m, g); }
    // Rows 16 m + 4 g .. of column c.
    template <int D>
    static __device__ __forceinline__ Frag col(const char* tile, int m, int, int c, int lane) {
        Frag f;
        #pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = *reinterpret_cast<const float*>(tile + at<D>(16 * m + 4 * (lane >> 4) + e, c / 4) + c % 4 * 4);
        return f;
    }
    static __device__ __forceinline__ float get(Frag f, int e) { return f[e]; }
    template <int N>
    static __device__ __forceinline__ void split(const float* v, Frag* f) { f[0] = Frag{v[0], v[1], v[2], v[3]}; }
    template <int N>
    static __device__ __forceinline__ void store_p(char* P, int t, int i0, const float* v) {
        *reinterpret_cast<Frag*>(P + at<L>(t, i0 / 4)) = Frag{v[0], v[1], v[2], v[3]};
    }

    template <bool WHOLE>
    struct Piece {
        uint32_t w0, w1, w2, w3;
        __device__ __forceinline__ void load(rsrc_t d, uint32_t off, int n, bool bf16) {
            if (bf16) {
                Raw<bf16_t, 4, WHOLE> r;
                r.load(d, off, n);
                w0 = r.w[0]; w1 = r.w[1];
                w2 = WHOLE ? 0 : r.w[r.W - 2]; w3 = WHOLE ? 0 : r.w[r.W - 1];
            } else {
                Raw<float, 4, WHOLE> r;
                r.load(d, off, n);
                w0 = r.w[0]; w1 = r.w[1]; w2 = r.w[2]; w3 = r.w[3];
            }
        }
        __device__ __forceinline__ void store(char* p, bool bf16) const {
            typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
            u32x4 v = {w0, w1, w2, w3};
            if (bf16) v = WHOLE ? u32x4{w0 << 16, w0 & 0xffff0000u, w1 << 16, w1 & 0xffff0000u} : v << 16;
            *reinterpret_cast<u32x4*>(p) = v;
        }
        __device__ __forceinline__ void get(float* v, bool bf16) const {
            v[0] = __uint_as_float(bf16 ? w0 << 16 : w0);
            v[1] = __uint_as_float(bf16 ? (WHOLE ? w0 & 0xffff0000u : w1 << 16) : w1);
            v[2] = __uint_as_float(bf16 ? (WHOLE ? w1 : w2) << 16 : w2);
            v[3] = __uint_as_float(bf16 ? (WHOLE ? w1 & 0xffff0000u : w3 << 16) : w3);
        }
    };
    template <bool WHOLE>
    using Four = Piece<WHOLE>;   // four neighbouring columns of a row
};

}  // namespace

hipError_t parts_f32(const Chunks& w, const Sweep& s, hipStream_t st) { return launch_parts<F32Ops>(w, s, st); }
hipError_t forward_f32(const Chunks& w, const Sweep& s, hipStream_t st) { return launch_outs<F32Ops, F32Ops::NPY, false, false>(w, s, s, 1, st); }
hipError_t backward_f32(const Chunks& w, const Sweep& q, const Sweep& k, const Sweep& v, hipStream_t st) { return launch_backward<F32Ops>(w, q, k, v, st); }

}  // namespace linattn
}  // namespace wkv7
