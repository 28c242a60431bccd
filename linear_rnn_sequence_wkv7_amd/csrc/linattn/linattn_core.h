// Linear attention with a decay for each head: the sweep over chunks of tokens that the forward
// and all three gradients are made of.  Included by one source per matrix-core opcode, which
// brings the operand type O (Bf16Ops, F32Ops).
//
// With rows a_t, b_t (DA wide) and c_t (DC wide), X_t the running sum of g and S (DA x DC) the
// state before a chunk of L tokens:
//
//     out_t = sp sum_{i <= t} exp(X_t - X_i) (a_t . b_i) c_i + si exp(X_t) S^T a_t
//     S'    = exp(X_L) S + su sum_i exp(X_L - X_i) b_i c_i^T
//
//              a   b   c   out  state
//   forward    q   k   v   y    S
//   dq         dy  v   k   dq   S^T
//   dk, back   v   dy  q   dk   E^T       E: the gradient of the state behind a token
//   dv, back   k   q   dy  dv   E
//
// Backwards the tokens of a chunk are read in the other order and X_t leaves the token's own g
// out; all the rest is the same.  X is summed in 64 bits, in units of log2, and kept as two
// floats, so that exp(X_t - X_i) is good to fp32 however far the sum has come.
//
// A wave for each 16 columns of c: together they compute the L x L matrix P = exp(X_t - X_i)
// (a_t . b_i), and each holds its columns of S in registers, as the matrix cores left them:
// rows (DA) by group of 16 lanes and register, columns by lane.  In that layout the state
// is at once the operand of S^T a_t (the order of a contraction is free as long as both
// operands agree), so it never goes through LDS.  out is computed transposed, so that a lane
// has neighbouring columns of one token and stores them as one piece.
#pragma once

#include "../seq_device.h"
#include "linattn_internal.h"
#include "wave_sum64.h"

namespace wkv7 {
namespace linattn {

// Which rows of a state the index 4 c .. 4 c + 3 of a 16-wide tile stands for.  In pairs of
// tiles the lanes of one group have 8 neighbours: 4 in each tile.
__device__ __forceinline__ constexpr int pair_col(int tile, int c) { return 32 * (tile / 2) + 8 * c + 4 * (tile % 2); }
__device__ __forceinline__ constexpr int flat_col(int tile, int c) { return 16 * tile + 4 * c; }

// x, which the compiler takes for a new value: what is formed from it is formed here, and not
// kept in registers over the loop (LDS addresses alone would take 60 of them).
__device__ __forceinline__ int fresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

template <typename O, int DA, int DC, int NPP>
struct Layout {
    static constexpr int L = O::L, es = int(sizeof(typename O::elem));
    static constexpr int A = 0, B = A + L * DA * es, C = B + L * DA * es, P = C + L * DC * es;
    static constexpr int TAB = P + NPP * L * L * es;      // float [4][64]: X, its low part, exp(X) si, exp(X_L - X) su;
    static constexpr int DOT = TAB + (4 * 64 + 16) * 4;   // exp(X_L); [8] sums of the waves.  float [waves][64]
    static constexpr int END = DOT + DC / 16 * 64 * 4;
};

// The rows of one operand in a chunk: 16-byte pieces (8 bf16, 4 fp32), a few to a thread, held
// as they were loaded until stage() brings them to LDS.
template <typename O, int D, int THREADS, bool WHOLE>
struct Rows {
    static constexpr int PER = D / O::E, N = O::L * PER / THREADS;
    static_assert(O::L * PER % THREADS == 0);
    typename O::template Piece<WHOLE> r[N];

    __device__ __forceinline__ void load(const Operand& x, int64_t row0, int n, bool back, int head) {
        const int tid = fresh(int(threadIdx.x));
        const uint32_t es = x.bf16 ? 2 : 4, stride = uint32_t(x.heads) * x.D * es;
        const char* p = static_cast<const char*>(x.p) + (row0 * x.heads + head) * x.D * es;
        const rsrc_t d = buf_rsrc(p, n > 0 ? int64_t(n - 1) * stride + x.D * es : 0);
        #pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = i * THREADS + tid, row = at / PER, col = at % PER * O::E;
            const uint32_t off = uint32_t(back ? n - 1 - row : row) * stride + uint32_t(col) * es;
            r[i].load(d, row < n && col < x.D ? off : kNowhere, x.D - col, x.bf16);
        }
    }
    __device__ __forceinline__ void stage(char* tile, bool bf16) const {
        const int tid = fresh(int(threadIdx.x));
        #pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = i * THREADS + tid;
            r[i].store(tile + O::template at<D>(at / PER, at % PER), bf16);
        }
    }
};

// The decays of a chunk's tokens, by the first wave: lane = row of the chunk.
__device__ __forceinline__ float load_g(const Chunks& w, const float* g, int64_t row0, int n, bool back, int h, int lane) {
    if (lane >= n) return 0.f;
    return w.g_per_token ? g[(row0 + (back ? n - 1 - lane : lane)) * w.H + h] : g[h];
}
// Returns exp(X_L).
__device__ __forceinline__ void make_tables(float* tab, float g, int n, bool back, float si, float su, int lane) {
    double u = double(g) * 1.4426950408889634074;
    u = u < kNoDecayLog2 ? kNoDecayLog2 : u;   // NaN stays NaN
    const double in = running_sum(u, lane), all = lane64(in, 63), X = back ? in - u : in;
    const float hi = float(X), out = exp2f(float(all - X));
    tab[lane] = hi;
    tab[64 + lane] = float(X - hi);
    tab[128 + lane] = exp2f(hi) * si;
    tab[192 + lane] = out * su;
    if (lane == 0) tab[256] = exp2f(float(all));
}

// S (or the part of it that a run of tokens adds) for the wave's columns.
template <typename O, int DA>
struct State {
    static constexpr int NA = DA / 16;
    f32x4 s[NA];

    // f(element, its byte offset in fp32 [DA][DC] (the state as it is stored) or its transpose) of every element.
    template <typename F>
    __device__ __forceinline__ void each(F&& f, int da, int dc, bool transposed, int wave, int lane) {
        const int j = 16 * wave + (lane & 15);
        #pragma unroll
        for (int a = 0; a < NA; ++a)
            #pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = O::row_of(a, lane >> 4) + r;
                float x = s[a][r];
                f(x, i < da && j < dc ? uint32_t(transposed ? j * da + i : i * dc + j) * 4 : kNowhere);
                s[a][r] = x;
            }
    }
    __device__ __forceinline__ void load(const float* p, int da, int dc, bool transposed, int wave, int lane) {
        const rsrc_t d = buf_rsrc(p, p ? da * dc * 4 : 0);
        each([&](float& x, uint32_t off) { x = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(d, off, 0, 0)); }, da, dc, transposed, wave, lane);
    }
    __device__ __forceinline__ void store(float* p, int da, int dc, bool transposed, int wave, int lane) {
        const rsrc_t d = buf_rsrc(p, da * dc * 4);
        each([&](float& x, uint32_t off) { __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), d, off, 0, 0); }, da, dc, transposed, wave, lane);
    }
    __device__ __forceinline__ float dot(const float* p, int da, int dc, bool transposed, int wave, int lane) {
        const rsrc_t d = buf_rsrc(p, da * dc * 4);
        float sum = 0.f;
        each([&](float& x, uint32_t off) { sum = fmaf(x, __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(d, off, 0, 0)), sum); }, da, dc, transposed, wave, lane);
        return sum;
    }
};

// The workgroup's place in the launch: segments of a head, heads, sequences, and what is computed
// for them (`kinds`) fastest, in runs of neighbours for each XCD.
struct Place {
    int kind, seg, h, b;
    __device__ __forceinline__ Place(const Chunks& w, int kinds) {
        int64_t i = xcd_order(blockIdx.x, gridDim.x);
        kind = int(i % kinds); i /= kinds;
        seg = int(i % w.segs); i /= w.segs;
        h = int(i % w.H);
        b = int(i / w.H);
    }
};

// One sweep over the tokens of a segment of sequence b, head h.
//   OUT: computes out; else only what the segment adds to a state.
//   NPS, NPP: how many operands of the matrix cores a value of S (for out) and of P is split into.
template <typename O, int DA, int DC, int NPS, int NPP, bool OUT, bool WHOLE>
__device__ void sweep(const Chunks& w, const Sweep& s, int b, int h, int seg, char* smem) {
    using Lay = Layout<O, DA, DC, NPP>;
    using St = State<O, DA>;
    constexpr int L = O::L, K = O::K, NL = L / 16, NA = St::NA, kThreads = 4 * DC;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    float* tab = reinterpret_cast<float*>(smem + Lay::TAB);
    float* dots = reinterpret_cast<float*>(smem + Lay::DOT);
    const bool back = s.back;
    const int len = seq_length(w.lengths, b, w.T);
    const int t0 = seg * w.seg_tokens, t1 = min(t0 + w.seg_tokens, w.T), end = min(t1, max(len, t0));
    const int nch = (end - t0 + L - 1) / L;
    const int64_t bh = int64_t(b) * w.H + h;
    const int ha = h / (w.H / s.a.heads), hb = h / (w.H / s.b.heads), hc = h / (w.H / s.c.heads), hx = s.dot ? h / (w.H / s.x.heads) : 0;

    St S;
    {
        const float* from = w.segs > 1 ? (OUT ? s.ws + (bh * w.segs + seg) * int64_t(s.a.D) * s.c.D : nullptr)
                                       : (s.s_in ? s.s_in + bh * int64_t(s.a.D) * s.c.D : nullptr);
        S.load(from, s.a.D, s.c.D, s.transposed, wave, lane);
    }
    float kept = 1.f;   // what is left of a state behind the segment

    Rows<O, DA, kThreads, WHOLE> ra, rb;
    Rows<O, DC, kThreads, WHOLE> rc;
    float rg = 0.f;
    auto fetch = [&](int c) {
        const int c0 = t0 + (back ? nch - 1 - c : c) * L, n = min(L, end - c0);
        const int64_t row0 = int64_t(b) * w.T + c0;
        if constexpr (OUT) ra.load(s.a, row0, n, back, ha);
        rb.load(s.b, row0, n, back, hb);
        rc.load(s.c, row0, n, back, hc);
        if (wave == 0) rg = load_g(w, w.g, row0, n, back, h, lane);
    };
    if (nch > 0) fetch(0);
    if constexpr (OUT && O::K > 16) {   // the blocks of P that a wider contraction reads past the diagonal
        for (int i = tid; i < NPP * L * L * Lay::es / 16; i += kThreads) *reinterpret_cast<uint4*>(smem + Lay::P + 16 * i) = uint4{0, 0, 0, 0};
    }

    for (int ch = 0; ch < nch; ++ch) {
        const int c0 = t0 + (back ? nch - 1 - ch : ch) * L, n = min(L, end - c0);
        if constexpr (OUT) ra.stage(smem + Lay::A, s.a.bf16);
        rb.stage(smem + Lay::B, s.b.bf16);
        rc.stage(smem + Lay::C, s.c.bf16);
        if (wave == 0) make_tables(tab, rg, n, back, s.si, s.su, lane);
        __syncthreads();
        if (ch + 1 < nch) fetch(ch + 1);

        f32x4 out[NL];
        if constexpr (OUT) {
            // P: lane has row t, four neighbouring i
            const int ln = fresh(lane), l16 = ln & 15, g4 = ln >> 4;
            for (int p = wave; p < NL * (NL + 1) / 2; p += DC / 16) {
                int ti = 0, ii = p;
                while (ii > ti) ii -= ++ti;
                f32x4 acc = {0.f, 0.f, 0.f, 0.f};
                #pragma unroll
                for (int m = 0; m < DA / K; ++m)
                    acc = O::mma(O::template row<DA>(smem + Lay::B, 16 * ii + l16, m, g4), O::template row<DA>(smem + Lay::A, 16 * ti + l16, m, g4), acc);
                const int t = 16 * ti + l16, i0 = 16 * ii + 4 * g4;
                const float xh = tab[t], xl = tab[64 + t];
                const f32x4 ih = *reinterpret_cast<const f32x4*>(tab + i0), il = *reinterpret_cast<const f32x4*>(tab + 64 + i0);
                float v[4];
                #pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float e = __builtin_amdgcn_exp2f((xh - ih[r]) + (xl - il[r]));
                    v[r] = i0 + r <= t ? s.sp * acc[r] * e : 0.f;
                }
                O::template store_p<NPP>(smem + Lay::P, t, i0, v);
            }
            // what the state before the chunk gives
            #pragma unroll
            for (int ti = 0; ti < NL; ++ti) out[ti] = f32x4{0.f, 0.f, 0.f, 0.f};
            #pragma unroll
            for (int m = 0; m < DA / K; ++m) {
                typename O::Frag sf[NPS];
                float v[O::E];
                #pragma unroll
                for (int e = 0; e < O::E; ++e) v[e] = S.s[m * (K / 16) + e / 4][e % 4];
                O::template split<NPS>(v, sf);
                #pragma unroll
                for (int ti = 0; ti < NL; ++ti) {
                    const typename O::Frag af = O::template row<DA>(smem + Lay::A, 16 * ti + l16, m, g4);
                    #pragma unroll
                    for (int p = 0; p < NPS; ++p) out[ti] = O::mma(sf[p], af, out[ti]);
                }
            }
            #pragma unroll
            for (int ti = 0; ti < NL; ++ti) out[ti] *= tab[128 + 16 * ti + l16];
            __syncthreads();
        }
        const int ln = fresh(lane), l16 = ln & 15, g4 = ln >> 4;
        const float all = tab[256];
        kept *= all;
        #pragma unroll
        for (int a = 0; a < NA; ++a) S.s[a] *= all;
        #pragma unroll
        for (int m = 0; m < L / K; ++m) {
            const typename O::Frag cf = O::template col<DC>(smem + Lay::C, m, flat_col(wave, l16 & 3), 16 * wave + l16, ln);
            if constexpr (OUT) {
                #pragma unroll
                for (int ti = m * K / 16; ti < NL; ++ti)
                    #pragma unroll
                    for (int p = 0; p < NPP; ++p)
                        out[ti] = O::mma(cf, O::template row<L>(smem + Lay::P + p * L * L * Lay::es, 16 * ti + l16, m, g4), out[ti]);
            }
            // c times its decay to the chunk's end
            typename O::Frag cs[O::NPU];
            float v[O::E];
            #pragma unroll
            for (int e = 0; e < O::E; ++e) v[e] = O::get(cf, e) * tab[192 + K * m + O::E * g4 + e];
            O::template split<O::NPU>(v, cs);
            #pragma unroll
            for (int a = 0; a < NA; ++a) {
                const typename O::Frag bf = O::template col<DA>(smem + Lay::B, m, O::row_of(a, l16 & 3), O::row_of(a, l16 >> 2) + (l16 & 3), ln);
                #pragma unroll
                for (int p = 0; p < O::NPU; ++p) S.s[a] = O::mma(bf, cs[p], S.s[a]);
            }
        }
        if constexpr (OUT) {
            const int j = 16 * wave + 4 * g4, D = s.c.D;
            const int64_t row0 = int64_t(b) * w.T + c0;
            const uint32_t stride = uint32_t(s.out_heads) * D, xstride = uint32_t(s.x.heads) * D;
            const int es = s.out_bf16 ? 2 : 4, xs = s.x.bf16 ? 2 : 4;
            const rsrc_t od = buf_rsrc(static_cast<char*>(s.out) + (row0 * s.out_heads + h) * D * es, (int64_t(n - 1) * stride + D) * es);
            const rsrc_t xd = buf_rsrc(static_cast<const char*>(s.x.p) + (row0 * s.x.heads + hx) * D * xs, s.dot ? (int64_t(n - 1) * xstride + D) * xs : 0);
            #pragma unroll
            for (int ti = 0; ti < NL; ++ti) {
                const int t = 16 * ti + l16, row = back ? n - 1 - t : t;
                const bool there = t < n && j < D;
                float v[4];
                #pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = out[ti][e];
                const uint32_t off = there ? (row * stride + j) * es : kNowhere;
                if (s.out_bf16) buf_store<bf16_t, 4, WHOLE>(od, off, v, D - j);
                else buf_store<float, 4, WHOLE>(od, off, v, D - j);
                if (s.dot) {
                    const uint32_t xo = there ? (row * xstride + j) * xs : kNowhere;
                    float dot = 0.f;
                    if (s.x.bf16) {
                        Raw<bf16_t, 4, WHOLE> x;
                        x.load(xd, xo, D - j);
                        #pragma unroll
                        for (int e = 0; e < 4; ++e) dot = fmaf(v[e], x.get(e), dot);
                    } else {
                        Raw<float, 4, WHOLE> x;
                        x.load(xd, xo, D - j);
                        #pragma unroll
                        for (int e = 0; e < 4; ++e) dot = fmaf(v[e], x.get(e), dot);
                    }
                    dot += __shfl_xor(dot, 16);
                    dot += __shfl_xor(dot, 32);
                    if (g4 == 0) dots[wave * 64 + t] = dot;
                }
            }
        }
        __syncthreads();
        if constexpr (OUT) {
            if (s.dot && tid < n) {
                float d = 0.f;
                #pragma unroll
                for (int i = 0; i < DC / 16; ++i) d += dots[64 * i + tid];
                s.dot[bh * w.T + c0 + (back ? n - 1 - tid : tid)] = d;
            }
        }
    }
    if constexpr (OUT) {
        // padding
        const int D = s.c.D;
        if (end < t1) {
            for (int64_t i = tid; i < int64_t(t1 - end) * D; i += kThreads) {
                const int64_t o = ((int64_t(b) * w.T + end + i / D) * s.out_heads + h) * D + i % D;
                if (s.out_bf16) static_cast<bf16_t*>(s.out)[o] = 0;
                else static_cast<float*>(s.out)[o] = 0.f;
            }
            if (s.dot)
                for (int i = end + tid; i < t1; i += kThreads) s.dot[bh * w.T + i] = 0.f;
        }
        if (w.segs == 1 && s.s_out) S.store(s.s_out + bh * int64_t(s.a.D) * s.c.D, s.a.D, s.c.D, s.transposed, wave, lane);
        if (s.end_dot && seg == (back ? 0 : w.segs - 1)) {   // <the last state, its gradient>
            float d = S.dot(s.end_grad + bh * int64_t(s.a.D) * s.c.D, s.a.D, s.c.D, s.transposed, wave, lane);
            #pragma unroll
            for (int m = 1; m < 64; m *= 2) d += __shfl_xor(d, m);
            if (lane == 0) tab[257 + wave] = d;
            __syncthreads();
            if (tid == 0) {
                d = 0.f;
                for (int i = 0; i < DC / 16; ++i) d += tab[257 + i];
                s.end_dot[bh] = d;
            }
        }
    } else {
        S.store(s.ws + (bh * w.segs + seg) * int64_t(s.a.D) * s.c.D, s.a.D, s.c.D, s.transposed, wave, lane);
        if (tid == 0) s.kept[bh * w.segs + seg] = kept;
    }
}

// The states that segments add, of one or both directions.
template <typename O, int DK, int DV, bool WHOLE>
__global__ __launch_bounds__(4 * DV, 2) void parts_kernel(Chunks w, Sweep f, Sweep r, int kinds) {
    __shared__ alignas(16) char smem[Layout<O, DK, DV, 0>::END];
    const Place at(w, kinds);
    sweep<O, DK, DV, 1, 0, false, WHOLE>(w, at.kind ? r : f, at.b, at.h, at.seg, smem);
}
// One to three outputs of the same widths side by side.
template <typename O, int DA, int DC, int NP, bool WHOLE>
__global__ __launch_bounds__(4 * DC, 2) void outs_kernel(Chunks w, Sweep x, Sweep y, Sweep z, int kinds) {
    __shared__ alignas(16) char smem[Layout<O, DA, DC, NP>::END];
    const Place at(w, kinds);
    sweep<O, DA, DC, NP, NP, true, WHOLE>(w, at.kind == 0 ? x : at.kind == 1 ? y : z, at.b, at.h, at.seg, smem);
}

// Heads are computed at 64 or 128, with zeros behind a smaller one's values.
template <typename F>
inline hipError_t with_widths(int da, int dc, F&& f) {
    using N64 = std::integral_constant<int, 64>;
    using N128 = std::integral_constant<int, 128>;
    if (da <= 64) return dc <= 64 ? f(N64{}, N64{}) : f(N64{}, N128{});
    return dc <= 64 ? f(N128{}, N64{}) : f(N128{}, N128{});
}
inline bool same_width(int d, int e) { return (d <= 64) == (e <= 64); }

template <typename O>
inline hipError_t launch_parts(const Chunks& w, const Sweep& f, const Sweep& r, int kinds, hipStream_t st) {
    return with_widths(f.a.D, f.c.D, [&](auto dk, auto dv) {
        const dim3 grid(uint32_t(int64_t(w.B) * w.H * w.segs * kinds));
        if (f.a.D % O::E == 0 && f.c.D % O::E == 0) parts_kernel<O, dk, dv, true><<<grid, 4 * dv, 0, st>>>(w, f, r, kinds);
        else parts_kernel<O, dk, dv, false><<<grid, 4 * dv, 0, st>>>(w, f, r, kinds);
        return hipGetLastError();
    });
}
template <typename O, int NP>
inline hipError_t launch_outs(const Chunks& w, const Sweep& x, const Sweep& y, const Sweep& z, int kinds, hipStream_t st) {
    return with_widths(x.a.D, x.c.D, [&](auto da, auto dc) {
        const dim3 grid(uint32_t(int64_t(w.B) * w.H * w.segs * kinds));
        if (x.a.D % O::E == 0 && x.c.D % O::E == 0) outs_kernel<O, da, dc, NP, true><<<grid, 4 * dc, 0, st>>>(w, x, y, z, kinds);
        else outs_kernel<O, da, dc, NP, false><<<grid, 4 * dc, 0, st>>>(w, x, y, z, kinds);
        return hipGetLastError();
    });
}
template <typename O>
inline hipError_t launch_backward(const Chunks& w, const Sweep& q, const Sweep& k, const Sweep& v, hipStream_t st) {
    if (same_width(v.a.D, v.c.D)) return launch_outs<O, O::NPU>(w, q, k, v, 3, st);
    const hipError_t e = launch_outs<O, O::NPU>(w, q, k, k, 2, st);
    return e != hipSuccess ? e : launch_outs<O, O::NPU>(w, v, v, v, 1, st);
}

}  // namespace linattn
}  // namespace wkv7
