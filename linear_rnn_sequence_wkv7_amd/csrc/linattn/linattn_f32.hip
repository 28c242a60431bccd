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
    static constexpr int NP = 1;

    // Four products of depth 4: element e of the lanes' groups is the e-th one's contraction.
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
        #pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
    // A row's pieces of 16 bytes trade places, as in linattn_bf16.hip.
    template <int D>
    static __device__ __forceinline__ uint32_t at(uint32_t row, uint32_t piece) {
        return row * (4 * D) + (piece ^ (D >= 64 ? row & 15 : row >> 1 & 7)) * 16;
    }
    static __device__ __forceinline__ constexpr int row_of(int a, int c) { return 16 * a + 4 * c; }

    template <int D>
    struct Lanes {
        uint32_t row, col;
        __device__ __forceinline__ Lanes(uint32_t ln) : row(at<D>(ln & 15, ln >> 4)), col(at<D>(ln >> 4 << 2, (ln & 15) >> 2) + (ln & 3) * 4) {}
    };
    // Elements 16 m + 4 g .. of row 16 t + the lane's.
    template <int D>
    static __device__ __forceinline__ Frag row(const char* tile, const Lanes<D>& at, int t, int m) {
        return *reinterpret_cast<const Frag*>(tile + (at.row ^ m * 64) + t * 64 * D);
    }
    // Rows 16 m + 4 g .. of column 16 t + the lane's (D >= 64: a row's last two bits go into its pieces' numbers as they are).
    template <int D>
    static __device__ __forceinline__ Frag col(const char* tile, const Lanes<D>& at, int t, int m) {
        Frag f;
        #pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = *reinterpret_cast<const float*>(tile + (at.col ^ (t * 64 | e * 16)) + (m * 64 + e * 4) * D);
        return f;
    }
    template <int D>
    static __device__ __forceinline__ Frag col_of_state(const char* tile, const Lanes<D>& at, int a, int m) { return col<D>(tile, at, a, m); }
    static __device__ __forceinline__ float get(Frag f, int e) { return f[e]; }
    template <int N>
    static __device__ __forceinline__ void split(const float* v, Frag* f) { f[0] = Frag{v[0], v[1], v[2], v[3]}; }
    // P of row 16 t + the lane's, columns 16 i + 4 g ..
    template <int N>
    static __device__ __forceinline__ void store_p(char* P, const Lanes<L>& at, int t, int i, const float* v) {
        *reinterpret_cast<Frag*>(P + (at.row ^ i * 64) + t * 64 * L) = Frag{v[0], v[1], v[2], v[3]};
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
hipError_t forward_f32(const Chunks& w, const Sweep& s, hipStream_t st) { return launch_outs<F32Ops, false, false>(w, s, st); }
hipError_t backward_f32(const Chunks& w, const Sweep& q, const Sweep& k, const Sweep& v, hipStream_t st) { return launch_backward<F32Ops>(w, q, k, v, st); }

}  // namespace linattn
}  // namespace wkv7
