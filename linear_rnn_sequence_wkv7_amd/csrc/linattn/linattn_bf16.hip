// Linear attention on bf16 operands: v_mfma_f32_16x16x32_bf16.
//
// q, k, v (and dy) are bf16 already and go into the products as they are.  What is not, the
// state, P and c times its decay, is split into three bf16 operands whose sum it is: the
// products and sums are then as good as fp32's, and only what is stored is rounded.  (Two
// operands, 2^-17 off, move a bf16 y by a step in one of a thousand places, and an fp32 y by
// more than all else; replays of y of 4 x 4096 tokens, 40 heads of 64, take 125 us with them,
// 131 with three; of 1 x 2048, 32 heads of 128, 51 and 54; of 8 x 1024, 32 heads of 64, 47 and 52.)
#include "linattn_core.h"

namespace wkv7 {
namespace linattn {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

struct Bf16Ops {
    using elem = bf16_t;
    using Frag = bf16x8;
    static constexpr int E = 8, K = 32, L = 64;
    static constexpr int NP = 3;   // operands that a value which is no bf16 is split into

    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

    // The pieces of 16 bytes of a row in an LDS tile of D columns trade places, each with the one whose
    // number differs by swap(), so that reads of one piece of 16 rows (row(); they go by lanes 0-3, 12-15,
    // 20-27 and so on) and of two pieces of rows r .. r + 3 and r + 8 .. r + 11 (col()) use every bank once.
    // (Columns of a state, four pieces' halves of those rows, meet in pairs: 4 of 12 clocks.)
    template <int D>
    static __device__ __forceinline__ uint32_t swap(uint32_t row) {
        if constexpr (D == 128) {
            const uint32_t q = row >> 2;
            return (row & 3) << 2 | (((q & 1) << 1 | (q >> 1 & 1)) ^ (q & 2));
        } else {
            const uint32_t u = row >> 1;
            return (u << 1 & 7) ^ (u >> 2 & 1) * 5;
        }
    }
    template <int D>
    static __device__ __forceinline__ uint32_t at(uint32_t row, uint32_t piece) { return row * (2 * D) + (piece ^ swap<D>(row)) * 16; }

    // The first of the four rows of a state that tile a's rows 4 c .. 4 c + 3 are.  In two tiles a group of
    // lanes has 8 neighbours, which is how row() reads what they are multiplied with.
    static __device__ __forceinline__ constexpr int row_of(int a, int c) { return 32 * (a / 2) + 8 * c + 4 * (a % 2); }

    // Where a lane reads a tile.  swap() goes by the row's last four bits and the pieces' numbers are
    // xors, so that another piece is an xor and other rows by 16 an offset away.
    template <int D>
    struct Lanes {
        uint32_t row, half, col[2], state[2];
        __device__ __forceinline__ Lanes(uint32_t ln) {
            const uint32_t l = ln & 15, g = ln >> 4, r = 8 * g + (l >> 2);
            row = at<D>(l, g);
            half = at<D>(l, g >> 1) + (g & 1) * 8;
            col[0] = at<D>(r, (l & 3) >> 1) + (l & 1) * 8;
            col[1] = at<D>(r + 4, (l & 3) >> 1) + (l & 1) * 8;
            state[0] = at<D>(r, l & 3);
            state[1] = at<D>(r + 4, l & 3);
        }
    };
    // Elements 32 m + 8 g .. of row 16 t + the lane's.
    template <int D>
    static __device__ __forceinline__ Frag row(const char* tile, const Lanes<D>& at, int t, int m) {
        return *reinterpret_cast<const Frag*>(tile + (at.row ^ m * 64) + t * 32 * D);
    }
    // Rows 32 m + 8 g .. of a column.  A transposing read takes 4 neighbouring columns of 4 rows from 4 lanes
    // each and gives every lane of the 16 its own column.
    static __device__ __forceinline__ Frag transposed(const char* lo4, const char* hi4) {
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(lo4));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(hi4));
        return __builtin_bit_cast(Frag, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    // Column 16 t + the lane's.
    template <int D>
    static __device__ __forceinline__ Frag col(const char* tile, const Lanes<D>& at, int t, int m) {
        return transposed(tile + (at.col[0] ^ t * 32) + m * 64 * D, tile + (at.col[1] ^ t * 32) + m * 64 * D);
    }
    // The column that row_of(a) gives the lane.
    template <int D>
    static __device__ __forceinline__ Frag col_of_state(const char* tile, const Lanes<D>& at, int a, int m) {
        const int more = m * 64 * D + a % 2 * 8;
        return transposed(tile + (at.state[0] ^ a / 2 * 64) + more, tile + (at.state[1] ^ a / 2 * 64) + more);
    }
    static __device__ __forceinline__ float get(Frag f, int e) {
        const u32x4 w = __builtin_bit_cast(u32x4, f);
        return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    }

    // Two values as N words of two bf16: all but the last cut off, the last rounded.
    template <int N>
    static __device__ __forceinline__ void split2(float x, float y, uint32_t (&w)[N]) {
        #pragma unroll
        for (int p = 0; p < N - 1; ++p) {
            w[p] = __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302);
            x -= __uint_as_float(__float_as_uint(x) & 0xffff0000u);
            y -= __uint_as_float(__float_as_uint(y) & 0xffff0000u);
        }
        w[N - 1] = __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(x), static_cast<__bf16>(y)});
    }
    template <int N>
    static __device__ __forceinline__ void split(const float* v, Frag* f) {
        u32x4 q[N];
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[N];
            split2<N>(v[2 * i], v[2 * i + 1], w);
            #pragma unroll
            for (int p = 0; p < N; ++p) q[p][i] = w[p];
        }
        #pragma unroll
        for (int p = 0; p < N; ++p) f[p] = __builtin_bit_cast(Frag, q[p]);
    }
    // P of row 16 t + the lane's, columns 16 i + 4 g ..
    template <int N>
    static __device__ __forceinline__ void store_p(char* P, const Lanes<L>& at, int t, int i, const float* v) {
        uint32_t lo[N], hi[N];
        split2<N>(v[0], v[1], lo);
        split2<N>(v[2], v[3], hi);
        #pragma unroll
        for (int p = 0; p < N; ++p) *reinterpret_cast<uint2*>(P + p * L * L * 2 + (at.half ^ i * 32) + t * 32 * L) = uint2{lo[p], hi[p]};
    }

    // Four neighbouring columns of a row.
    template <bool WHOLE>
    struct Four {
        Raw<bf16_t, 4, WHOLE> r;
        __device__ __forceinline__ void load(rsrc_t d, uint32_t off, int n, bool) { r.load(d, off, n); }
        __device__ __forceinline__ void get(float* v, bool) const {
            #pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = r.get(i);
        }
    };
    template <bool WHOLE>
    struct Piece {
        Raw<bf16_t, 8, WHOLE> r;
        __device__ __forceinline__ void load(rsrc_t d, uint32_t off, int n, bool) { r.load(d, off, n); }
        __device__ __forceinline__ void store(char* p, bool) const {
            if constexpr (WHOLE) {
                *reinterpret_cast<u32x4*>(p) = u32x4{r.w[0], r.w[1], r.w[2], r.w[3]};
            } else {
                u32x4 w;
                #pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = r.w[2 * i] | r.w[2 * i + 1] << 16;
                *reinterpret_cast<u32x4*>(p) = w;
            }
        }
    };
};

}  // namespace

hipError_t parts_bf16(const Chunks& w, const Sweep& s, hipStream_t st) { return launch_parts<Bf16Ops>(w, s, st); }
hipError_t forward_bf16(const Chunks& w, const Sweep& s, hipStream_t st) { return launch_outs<Bf16Ops, false, false>(w, s, st); }
hipError_t backward_bf16(const Chunks& w, const Sweep& q, const Sweep& k, const Sweep& v, hipStream_t st) { return launch_backward<Bf16Ops>(w, q, k, v, st); }

}  // namespace linattn
}  // namespace wkv7
