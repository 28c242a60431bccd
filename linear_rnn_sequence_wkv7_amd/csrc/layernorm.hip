// Layer norm on gfx950, with the residual stream's sum in front of it:
//
//   h = x + residual,  xh = (h - mean) rstd,  y = xh weight + bias             per row
//   dxh = dy weight,  dresidual = rstd (dxh - mean(dxh) - xh mean(dxh xh)) + dh
//   dweight = sum dy xh,  dbias = sum dy                                        over the rows
//
// Memory bounds it: every array is read or written once.  A row stays in the registers that
// loaded it: R waves take one, each lane K times 8 neighbouring channels.  The variance is that
// of the differences from the mean; h is rounded to the stream's type first, so that the
// statistics, y and the backward all mean the h that is stored.
//
// Pieces of 8 channels start where the array's element number is a multiple of 8, in every row,
// so that they are aligned for any C; a row's first and last piece may belong to it in part.  A
// row's offset in its pieces repeats with 8 / gcd(C, 8) rows; workgroups take rows that many (or a
// multiple) apart, so that a lane has the same channels in all its rows: it keeps their weights
// and sums their gradients in registers.  Each workgroup leaves a row of gradient sums, which a
// second kernel adds in a fixed order.
//
// 8 x 4096 x 4096 in bf16, forward: 208 us, 5.2 TB/s.  Forward, backward and the sums' kernel: 8 x 1024 x 2048 in
// bf16 23, 32 and 4 us; 4 x 2048 x 4096 with the stream in fp32 71, 113 and 5.
#include "layernorm.h"
#include "seq_device.h"

namespace wkv7 {
namespace {

// 8 elements as they were loaded.
template <typename T>
struct Oct {
    uint32_t w[sizeof(T) * 2];

    // p[lo .. hi) of the piece at p, which is 16-byte aligned; the others 0.  WHOLE: all or none.
    template <bool WHOLE>
    __device__ __forceinline__ void load(const T* p, int lo, int hi) {
        if (WHOLE && hi == 0) {
            #pragma unroll
            for (int i = 0; i < int(sizeof(T)) * 2; ++i) w[i] = 0;
        } else if (WHOLE || (lo == 0 && hi == 8)) {
            const uint4* q = reinterpret_cast<const uint4*>(p);
            #pragma unroll
            for (int i = 0; i < int(sizeof(T)) / 2; ++i) {
                const uint4 v = q[i];
                w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
            }
        } else {
            T e[8];
            #pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = i >= lo && i < hi ? p[i] : T(0);
            #pragma unroll
            for (int i = 0; i < int(sizeof(T)) * 2; ++i) {
                if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(e[i]);
                else w[i] = uint32_t(e[2 * i]) | uint32_t(e[2 * i + 1]) << 16;
            }
        }
    }
    // From here on the values are formed from the loaded words again, and not kept beside them.
    __device__ __forceinline__ void fresh() {
        #pragma unroll
        for (int i = 0; i < int(sizeof(T)) * 2; ++i) settle(w[i]);
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};
template <bool WHOLE, typename T>
__device__ __forceinline__ void st_oct(T* p, const float* v, int lo, int hi) {
    if (WHOLE || (lo == 0 && hi == 8)) {
        st_pack<8>(p, v, true, 8);
        return;
    }
    #pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i >= lo && i < hi) narrow(v[i], p[i]);
}
template <bool WHOLE>
__device__ __forceinline__ void st_oct_as(void* p, int64_t e, bool bf16, const float* v, int lo, int hi) {
    if (bf16) st_oct<WHOLE>(static_cast<bf16_t*>(p) + e, v, lo, hi);
    else st_oct<WHOLE>(static_cast<float*>(p) + e, v, lo, hi);
}

// The rows of a launch and how they are shared out: `slots` rows at a time, a multiple of `period`.
struct Share {
    int64_t rows, slots;
};

// Where a lane's K pieces lie in a row that starts `phase` elements into its first piece.
// WHOLE: rows of whole pieces.
template <int R, int K, bool WHOLE>
struct Pieces {
    int c[K], lo[K], hi[K];   // first channel (negative at the row's start), and which of the 8 are there
    __device__ __forceinline__ Pieces(int C, int phase, int lane_of_row) {
        #pragma unroll
        for (int k = 0; k < K; ++k) {
            c[k] = (k * 64 * R + lane_of_row) * 8 - phase;
            lo[k] = c[k] < 0 ? -c[k] : 0;
            hi[k] = C - c[k] < 0 ? 0 : C - c[k] > 8 ? 8 : C - c[k];
            if (lo[k] >= hi[k]) lo[k] = hi[k] = 0;
            if (WHOLE) {
                lo[k] = 0;
                hi[k] = c[k] < C ? 8 : 0;
            }
        }
    }
};

__device__ __forceinline__ float wave_sum(float x) {
    x = sum16(x);
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}
// Sums over the R waves of a row; `turn` alternates between the two places.
template <int R, int N>
__device__ __forceinline__ void row_sum(float (&x)[N], float (*lds)[16][N], int turn) {
    #pragma unroll
    for (int i = 0; i < N; ++i) x[i] = wave_sum(x[i]);
    if constexpr (R > 1) {
        const int wave = threadIdx.x / 64;
        if ((threadIdx.x & 63) == 0)
            #pragma unroll
            for (int i = 0; i < N; ++i) lds[turn][wave][i] = x[i];
        __syncthreads();
        #pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = 0.f;
            #pragma unroll
            for (int r = 0; r < R; ++r) x[i] += lds[turn][r][i];
        }
    }
}

constexpr int group_threads(int R) { return R < 4 ? 256 : 64 * R; }

template <bool WHOLE, int K>
__device__ __forceinline__ void load_params(const float* p, float other, const int* c, const int* lo, const int* hi, float (&v)[K][8]) {
    #pragma unroll
    for (int k = 0; k < K; ++k)
        if (WHOLE && p && hi[k]) {
            const Pack<float, 8> w = ld_pack<8>(p + c[k], true, 8);
            #pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] = w.e[i];
        } else
        #pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = p && i >= lo[k] && i < hi[k] ? p[c[k] + i] : other;
}

template <typename Tx, typename Th, int R, int K, bool WHOLE>
__global__ __launch_bounds__(group_threads(R)) void ln_forward_kernel(LayerNormParams p, Share s) {
    constexpr int AT_ONCE = group_threads(R) / (64 * R);   // rows of a workgroup
    __shared__ float lds[2][16][1];
    const int in_row = threadIdx.x % (64 * R);
    int64_t row = int64_t(blockIdx.x) * AT_ONCE + threadIdx.x / (64 * R);
    const int C = p.C, phase = WHOLE ? 0 : int(row * C % 8);
    const Pieces<R, K, WHOLE> at(C, phase, in_row);
    float wt[K][8], bs[K][8];
    load_params<WHOLE, K>(p.weight, 1.f, at.c, at.lo, at.hi, wt);
    load_params<WHOLE, K>(p.bias, 0.f, at.c, at.lo, at.hi, bs);
    const float inv = C ? 1.f / C : 0.f;
    for (; row < s.rows; row += s.slots) {
        const int64_t e0 = row * C - phase;
        const bool there = !p.lengths || row % p.T < seq_length(p.lengths, row / p.T, p.T);
        Oct<Tx> xr[K];
        Oct<Th> rr[K];
        float v[K][8];
        if (there) {
            #pragma unroll
            for (int k = 0; k < K; ++k) {
                xr[k].template load<WHOLE>(static_cast<const Tx*>(p.x) + e0 + at.c[k] + phase, at.lo[k], at.hi[k]);
                if (p.res) rr[k].template load<WHOLE>(static_cast<const Th*>(p.res) + e0 + at.c[k] + phase, at.lo[k], at.hi[k]);
            }
        }
        float sum[1] = {0.f};
        #pragma unroll
        for (int k = 0; k < K; ++k)
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[k][i] = there ? xr[k].get(i) : 0.f;
                if (there && p.res) {
                    Th o;
                    narrow(v[k][i] + rr[k].get(i), o);
                    v[k][i] = widen(o);
                }
                sum[0] += v[k][i];
            }
        row_sum<R, 1>(sum, lds, 0);
        const float mean = sum[0] * inv;
        float sq[1] = {0.f};
        #pragma unroll
        for (int k = 0; k < K; ++k)
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = v[k][i] - mean;
                if (WHOLE ? at.hi[k] : i >= at.lo[k] && i < at.hi[k]) sq[0] = fmaf(d, d, sq[0]);
            }
        row_sum<R, 1>(sq, lds, 1);
        const float rstd = 1.f / __builtin_sqrtf(fmaf(sq[0], inv, p.eps));
        #pragma unroll
        for (int k = 0; k < K; ++k) {
            if (at.hi[k] == 0) continue;
            if (p.res) st_oct<WHOLE>(static_cast<Th*>(p.h) + e0 + at.c[k] + phase, v[k], at.lo[k], at.hi[k]);
            float y[8];
            #pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = there ? fmaf((v[k][i] - mean) * rstd, wt[k][i], bs[k][i]) : 0.f;
            st_oct_as<WHOLE>(p.y, e0 + at.c[k] + phase, p.y_bf16, y, at.lo[k], at.hi[k]);
        }
        if (p.mean && in_row == 0) {
            p.mean[row] = mean;
            p.rstd[row] = rstd;
        }
    }
}

// part: [workgroups][2][C], the sums of dy xh and of dy over the workgroup's rows.
// The widest rows' weights are read for every row and dh only where it is added: with them in
// registers too, a row would not fit.
template <typename Th, typename Ty, int R, int K, bool WHOLE>
__global__ __launch_bounds__(group_threads(R)) void ln_backward_kernel(LayerNormParams p, Share s, float* part) {
    constexpr int AT_ONCE = group_threads(R) / (64 * R);
    constexpr bool LATE = K == 4;
    __shared__ float lds[2][16][2];
    __shared__ float join[AT_ONCE > 1 ? 2 * (R * K * 512) : 1];
    const int in_row = threadIdx.x % (64 * R), at_row = threadIdx.x / (64 * R);
    int64_t row = int64_t(blockIdx.x) * AT_ONCE + at_row;
    const int C = p.C, phase = WHOLE ? 0 : int(row * C % 8);
    const Pieces<R, K, WHOLE> at(C, phase, in_row);
    float wt[LATE ? 1 : K][8], dw[K][8] = {}, db[K][8] = {};
    if constexpr (!LATE) load_params<WHOLE, K>(p.weight, 1.f, at.c, at.lo, at.hi, wt);
    const float inv = C ? 1.f / C : 0.f;
    int turn = 0;
    for (; row < s.rows; row += s.slots, turn ^= 1) {
        const int64_t e0 = row * C - phase;
        const bool there = !p.lengths || row % p.T < seq_length(p.lengths, row / p.T, p.T);
        Oct<Th> hr[K], gr[K];
        Oct<Ty> dr[K];
        #pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t e = e0 + at.c[k] + phase;
            hr[k].template load<WHOLE>(static_cast<const Th*>(p.h) + e, there ? at.lo[k] : 0, there ? at.hi[k] : 0);
            dr[k].template load<WHOLE>(static_cast<const Ty*>(p.dy) + e, there ? at.lo[k] : 0, there ? at.hi[k] : 0);
            if (!LATE) gr[k].template load<WHOLE>(static_cast<const Th*>(p.dh) + e, there && p.dh ? at.lo[k] : 0, there && p.dh ? at.hi[k] : 0);
        }
        const float mean = there ? p.mean[row] : 0.f, rstd = there ? p.rstd[row] : 0.f;
        float m[2] = {0.f, 0.f};
        #pragma unroll
        for (int k = 0; k < K; ++k) {
            float (&w)[8] = wt[LATE ? 0 : k];
            if constexpr (LATE) load_params<WHOLE, 1>(p.weight, 1.f, at.c + k, at.lo + k, at.hi + k, wt);
            #pragma unroll
            for (int i = 0; i < 8; ++i) {   // dy is 0 where there is no element, and xh of no matter
                const float dy = dr[k].get(i), xh = (hr[k].get(i) - mean) * rstd, dxh = dy * w[i];
                m[0] += dxh;
                m[1] = fmaf(dxh, xh, m[1]);
                dw[k][i] = fmaf(dy, xh, dw[k][i]);
                db[k][i] += dy;
            }
            if constexpr (LATE) __builtin_amdgcn_sched_barrier(0);   // one piece's weights at a time
        }
        row_sum<R, 2>(m, lds, turn);
        m[0] *= inv;
        m[1] *= inv;
        #pragma unroll
        for (int k = 0; k < K; ++k) {
            if (at.hi[k] == 0) continue;
            uint32_t c = at.c[k] + phase;
            settle(c);   // addresses are formed again, too
            const int64_t e = e0 + c;
            float (&w)[8] = wt[LATE ? 0 : k];
            if constexpr (LATE) {
                load_params<WHOLE, 1>(p.weight, 1.f, at.c + k, at.lo + k, at.hi + k, wt);
                gr[k].template load<WHOLE>(static_cast<const Th*>(p.dh) + e, there && p.dh ? at.lo[k] : 0, there && p.dh ? at.hi[k] : 0);
            }
            hr[k].fresh();
            dr[k].fresh();
            float o[8];
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xh = (hr[k].get(i) - mean) * rstd;
                o[i] = there ? rstd * (dr[k].get(i) * w[i] - m[0] - xh * m[1]) + gr[k].get(i) : 0.f;
            }
            st_oct<WHOLE>(static_cast<Th*>(p.dres) + e, o, at.lo[k], at.hi[k]);
            if (p.dx) st_oct_as<WHOLE>(p.dx, e, p.x_bf16, o, at.lo[k], at.hi[k]);
            if constexpr (LATE) __builtin_amdgcn_sched_barrier(0);   // one piece's dh and weights at a time
        }
    }
    float* out = part + int64_t(blockIdx.x) * 2 * C;
    if constexpr (AT_ONCE > 1) {   // the rows at once have their channels in other places where C is no multiple of 8
        for (int i = threadIdx.x; i < 2 * R * K * 512; i += group_threads(R)) join[i] = 0.f;
        for (int r = 0; r < AT_ONCE; ++r) {
            __syncthreads();
            if (at_row == r)
                #pragma unroll
                for (int k = 0; k < K; ++k)
                    #pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i >= at.lo[k] && i < at.hi[k]) {
                            join[at.c[k] + i] += dw[k][i];
                            join[R * K * 512 + at.c[k] + i] += db[k][i];
                        }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < C; i += group_threads(R)) {
            out[i] = join[i];
            out[C + i] = join[R * K * 512 + i];
        }
    } else {
        #pragma unroll
        for (int k = 0; k < K; ++k)
            #pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i >= at.lo[k] && i < at.hi[k]) {
                    out[at.c[k] + i] = dw[k][i];
                    out[C + at.c[k] + i] = db[k][i];
                }
    }
}

// Rows past the registers of a workgroup, and those past 8185 channels that are no multiple of 8: read again for each
// pass, element by element, out of the caches.  8192 rows in bf16 with a residual, of 9001 channels: forward 334 us,
// backward 451 (of 9008, in registers: 127 and 181).
constexpr int kLong = 1024;
__device__ __forceinline__ float block_sum(float x, float* lds) {
    x = wave_sum(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x / 64] = x;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < kLong / 64; ++i) s += lds[i];
    return s;
}
template <typename Tx, typename Th>
__global__ __launch_bounds__(kLong) void ln_forward_long_kernel(LayerNormParams p, Share s) {
    __shared__ float lds[kLong / 64];
    const int C = p.C;
    const float inv = C ? 1.f / C : 0.f;
    for (int64_t row = blockIdx.x; row < s.rows; row += gridDim.x) {
        const int64_t e = row * C;
        const bool there = !p.lengths || row % p.T < seq_length(p.lengths, row / p.T, p.T);
        float sum = 0.f, sq = 0.f;
        auto value = [&](int c) { return p.res ? widen(static_cast<const Th*>(p.h)[e + c]) : widen(static_cast<const Tx*>(p.x)[e + c]); };
        for (int c = threadIdx.x; c < C; c += kLong) {   // a thread reads only what it wrote itself
            float v = there ? widen(static_cast<const Tx*>(p.x)[e + c]) : 0.f;
            if (p.res) {
                Th o;
                narrow(there ? v + widen(static_cast<const Th*>(p.res)[e + c]) : 0.f, o);
                static_cast<Th*>(p.h)[e + c] = o;
                v = widen(o);
            }
            sum += v;
        }
        const float mean = block_sum(sum, lds) * inv;
        for (int c = threadIdx.x; there && c < C; c += kLong) {
            const float d = value(c) - mean;
            sq = fmaf(d, d, sq);
        }
        const float rstd = 1.f / __builtin_sqrtf(fmaf(block_sum(sq, lds), inv, p.eps));
        for (int c = threadIdx.x; c < C; c += kLong) {
            const float y = there ? fmaf((value(c) - mean) * rstd, p.weight ? p.weight[c] : 1.f, p.bias ? p.bias[c] : 0.f) : 0.f;
            if (p.y_bf16) static_cast<bf16_t*>(p.y)[e + c] = f32_to_bf16(y);
            else static_cast<float*>(p.y)[e + c] = y;
        }
        if (p.mean && threadIdx.x == 0) {
            p.mean[row] = mean;
            p.rstd[row] = rstd;
        }
    }
}
template <typename Th, typename Ty>
__global__ __launch_bounds__(kLong) void ln_backward_long_kernel(LayerNormParams p, Share s, float* part) {
    __shared__ float lds[kLong / 64];
    const int C = p.C;
    const float inv = C ? 1.f / C : 0.f;
    float* out = part + int64_t(blockIdx.x) * 2 * C;
    for (int c = threadIdx.x; c < 2 * C; c += kLong) out[c] = 0.f;
    __syncthreads();
    for (int64_t row = blockIdx.x; row < s.rows; row += gridDim.x) {
        const int64_t e = row * C;
        const bool there = !p.lengths || row % p.T < seq_length(p.lengths, row / p.T, p.T);
        const float mean = there ? p.mean[row] : 0.f, rstd = there ? p.rstd[row] : 0.f;
        float m1 = 0.f, m2 = 0.f;
        for (int c = threadIdx.x; there && c < C; c += kLong) {
            const float dy = widen(static_cast<const Ty*>(p.dy)[e + c]), xh = (widen(static_cast<const Th*>(p.h)[e + c]) - mean) * rstd;
            const float dxh = dy * (p.weight ? p.weight[c] : 1.f);
            m1 += dxh;
            m2 = fmaf(dxh, xh, m2);
            out[c] = fmaf(dy, xh, out[c]);
            out[C + c] += dy;
        }
        m1 = block_sum(m1, lds) * inv;
        m2 = block_sum(m2, lds) * inv;
        for (int c = threadIdx.x; c < C; c += kLong) {
            float o = 0.f;
            if (there) {
                const float dy = widen(static_cast<const Ty*>(p.dy)[e + c]), xh = (widen(static_cast<const Th*>(p.h)[e + c]) - mean) * rstd;
                o = rstd * (dy * (p.weight ? p.weight[c] : 1.f) - m1 - xh * m2) + (p.dh ? widen(static_cast<const Th*>(p.dh)[e + c]) : 0.f);
            }
            narrow(o, static_cast<Th*>(p.dres)[e + c]);
            if (p.dx && p.x_bf16) static_cast<bf16_t*>(p.dx)[e + c] = f32_to_bf16(o);
            else if (p.dx) static_cast<float*>(p.dx)[e + c] = o;
        }
    }
}

// dweight and dbias: 32 neighbouring sums a workgroup, 32 threads to each, then over those.
__global__ __launch_bounds__(1024) void ln_sum_kernel(const float* part, int64_t groups, int C, float* dweight, float* dbias) {
    __shared__ float lds[32][33];
    const int x = threadIdx.x % 32, y = threadIdx.x / 32;
    const int64_t at = int64_t(blockIdx.x) * 32 + x;
    float s = 0.f;
    if (at < 2 * int64_t(C))
        #pragma unroll 8
        for (int64_t g = y; g < groups; g += 32) s += part[g * 2 * C + at];
    lds[y][x] = s;
    __syncthreads();
    if (y == 0 && at < 2 * int64_t(C)) {
        s = 0.f;
        #pragma unroll
        for (int i = 0; i < 32; ++i) s += lds[i][x];
        float* out = at < C ? dweight : dbias;
        if (out) out[at < C ? at : at - C] = s;
    }
}
__global__ __launch_bounds__(256) void ln_zero_kernel(float* a, float* b, int n) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < n && a) a[i] = 0.f;
    if (i < n && b) b[i] = 0.f;
}

// ---------------------------------------------------------------- forms

struct Form {
    int R, K;         // R 0: a long row
    int64_t slots;    // rows at a time
    int64_t groups;
};
Form form_of(const LayerNormParams& p, bool bwd) {
    const int64_t rows = int64_t(p.B) * p.T;
    const int period = p.C % 8 == 0 ? 1 : p.C % 4 == 0 ? 2 : p.C % 2 == 0 ? 4 : 8;
    const int64_t need = int64_t(p.C) + (period > 1 ? 7 : 0);   // with what stands before a row in its first piece
    Form f{0, 0, 0, 0};
    for (const auto& c : {Form{1, 1}, Form{1, 2}, Form{4, 1}, Form{4, 2}, Form{8, 2}, bwd ? Form{8, 4} : Form{16, 2}})
        if (!f.R && need <= int64_t(c.R) * c.K * 512 && (c.R * c.K < 32 || period == 1)) f = c;
    if (!f.R) {
        f.groups = f.slots = rows < 1024 ? rows : 1024;
        return f;
    }
    const int at_once = group_threads(f.R) / (64 * f.R), waves = group_threads(f.R) / 64;
    // Waves on the chip: 16 to a compute unit, in the backward 8, since each group leaves a row of sums.
    int64_t groups = (rows + at_once - 1) / at_once;
    const int64_t most = 256 * (bwd ? 8 : 16) / waves;
    if (groups > most) groups = most;   // most is a multiple of 8, so of the period
    f.groups = groups;
    f.slots = groups * at_once;
    return f;
}

template <typename Tx, typename Th>
hipError_t forward(const LayerNormParams& p, hipStream_t st) {
    const Form f = form_of(p, false);
    const Share s{int64_t(p.B) * p.T, f.slots};
    const dim3 grid{unsigned(f.groups)};
#define WKV7_LN(r, k, w) case r * 32 + k * 2 + w: ln_forward_kernel<Tx, Th, r, k, w><<<grid, group_threads(r), 0, st>>>(p, s); break
    switch (f.R * 32 + f.K * 2 + (p.C % 8 == 0)) {
        WKV7_LN(1, 1, true); WKV7_LN(1, 2, true); WKV7_LN(4, 1, true); WKV7_LN(4, 2, true); WKV7_LN(8, 2, true); WKV7_LN(16, 2, true);
        WKV7_LN(1, 1, false); WKV7_LN(1, 2, false); WKV7_LN(4, 1, false); WKV7_LN(4, 2, false); WKV7_LN(8, 2, false);
        default: ln_forward_long_kernel<Tx, Th><<<grid, kLong, 0, st>>>(p, s);
    }
#undef WKV7_LN
    return hipGetLastError();
}
template <typename Th, typename Ty>
hipError_t backward(const LayerNormParams& p, hipStream_t st) {
    const Form f = form_of(p, true);
    const Share s{int64_t(p.B) * p.T, f.slots};
    const dim3 grid{unsigned(f.groups)};
    float* part = static_cast<float*>(p.ws);
#define WKV7_LN(r, k, w) case r * 32 + k * 2 + w: ln_backward_kernel<Th, Ty, r, k, w><<<grid, group_threads(r), 0, st>>>(p, s, part); break
    switch (f.R * 32 + f.K * 2 + (p.C % 8 == 0)) {
        WKV7_LN(1, 1, true); WKV7_LN(1, 2, true); WKV7_LN(4, 1, true); WKV7_LN(4, 2, true); WKV7_LN(8, 2, true); WKV7_LN(8, 4, true);
        WKV7_LN(1, 1, false); WKV7_LN(1, 2, false); WKV7_LN(4, 1, false); WKV7_LN(4, 2, false); WKV7_LN(8, 2, false);
        default: ln_backward_long_kernel<Th, Ty><<<grid, kLong, 0, st>>>(p, s, part);
    }
#undef WKV7_LN
    if (p.dweight || p.dbias) ln_sum_kernel<<<unsigned((2 * int64_t(p.C) + 31) / 32), 1024, 0, st>>>(part, f.groups, p.C, p.dweight, p.dbias);
    return hipGetLastError();
}

}  // namespace

int64_t layernorm_backward_workspace(const LayerNormParams& p) {
    if (int64_t(p.B) * p.T * p.C == 0) return 0;
    return form_of(p, true).groups * 2 * p.C * 4;
}
int64_t layernorm_threads(const LayerNormParams& p, bool bwd) { return bwd ? int64_t(p.C) * 64 + 1024 : 0; }

hipError_t launch_layernorm_forward(const LayerNormParams& p, hipStream_t st) {
    if (p.x_bf16) return p.h_bf16 ? forward<bf16_t, bf16_t>(p, st) : forward<bf16_t, float>(p, st);
    return p.h_bf16 ? forward<float, bf16_t>(p, st) : forward<float, float>(p, st);
}
hipError_t launch_layernorm_backward(const LayerNormParams& p, hipStream_t st) {
    if (int64_t(p.B) * p.T == 0) {
        if (p.dweight || p.dbias) ln_zero_kernel<<<(p.C + 255) / 256, 256, 0, st>>>(p.dweight, p.dbias, p.C);
        return hipGetLastError();
    }
    if (p.h_bf16) return p.y_bf16 ? backward<bf16_t, bf16_t>(p, st) : backward<bf16_t, float>(p, st);
    return p.y_bf16 ? backward<float, bf16_t>(p, st) : backward<float, float>(p, st);
}

}  // namespace wkv7
