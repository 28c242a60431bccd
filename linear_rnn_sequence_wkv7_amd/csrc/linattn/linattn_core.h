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
// Backwards t <= i in both sums, and X_t is the sum over the later tokens of the chunk, without the
// token's own g; all the rest is the same.  X is summed in 64 bits, in units of log2, and kept as two
// floats, so that exp(X_t - X_i) is good to fp32 however far the sum has come.
//
// A wave for each 16 columns of c: together they compute the L x L matrix P = exp(X_t - X_i)
// (a_t . b_i), and each holds its columns of S in registers, as the matrix cores left them:
// rows (DA) by group of 16 lanes and register, columns by lane.  In that layout the state
// is at once the operand of S^T a_t (the order of a contraction is free as long as both
// operands agree), so it never goes through LDS.  out is computed transposed, so that a lane
// has neighbouring columns of one token and stores them as one piece.
//
// Bound by no unit alone: vector work (splits into bf16, decays, addresses) and the matrix cores, which a
// wave does in turn, and the waits at two barriers a chunk.  Replays of one call, whose inputs the caches hold in
// part: y of 8 x 1024 tokens, 32 heads of 64, bf16, 52 us (2.7 TB/s), its three gradients 105 (vector units 45 %,
// matrix cores 22 %, LDS 31 % busy); of 2 x 16384 tokens, 32 heads of 128, q and k shared by four, y with the segments'
// pass 434 us (62, 37 and 35 %) and the gradients 1085 (56, 32 and 30 %).  One workgroup by itself on a compute unit
// takes 3 us for a chunk at heads of 64 and 5 at 128.
#pragma once

#include "../seq_device.h"
#include "linattn_internal.h"
#include "wave_sum64.h"

namespace wkv7 {
namespace linattn {

// x, which the compiler takes for a new value: what is formed from it is formed here, and not
// kept in registers over the loop (LDS addresses alone would take 60 of them).
template <bool DO = true>
__device__ __forceinline__ uint32_t fresh(uint32_t x) {
    if constexpr (DO) asm volatile("" : "+v"(x));
    return x;
}

// float [2 chunks][4][64] X, its low part, exp(X) si, exp(X_L - X) su; [2] exp(X_L)
constexpr int kTab = 4 * 64 + 16;
// Nothing is moved across: operands of the next products are not loaded before these are done, which
// keeps registers free for more waves.
__device__ __forceinline__ void hold() { __builtin_amdgcn_sched_barrier(0); }

// N fragments of READS LDS reads each, that MMAS products use: reads are issued AHEAD fragments before their products.
template <int AHEAD, int READS, int MMAS, int N>
__device__ __forceinline__ void pace() {
    #pragma unroll
    for (int i = 0; i < N + AHEAD; ++i) {
        if (i < N) __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
        if (i >= AHEAD) __builtin_amdgcn_sched_group_barrier(0x008, MMAS, 0);
    }
    hold();
}

template <typename O, int DA, int DC, int NPP>
struct Layout {
    static constexpr int L = O::L, es = int(sizeof(typename O::elem));
    static constexpr int A = 0, B = A + (NPP ? L * DA * es : 0), C = B + L * DA * es;
    static constexpr int NEXT = NPP ? 0 : L * (DA + DC) * es;   // where no out is computed the next chunk's rows have a place of their own
    static constexpr int P = C + L * DC * es + NEXT;
    static constexpr int TAB = P + NPP * L * L * es;
    static constexpr int DOT = TAB + 2 * kTab * 4;        // float [waves][64], behind them a double of each
    static constexpr int END = DOT + (DC / 16 * 64 + 16) * 4;
};

// A row of a chunk times its stride (16384 heads of 128 fp32 at the most: 2^23): full rate, unlike 32 bits.
__device__ __forceinline__ uint32_t mul24(uint32_t row, uint32_t stride) { return __umul24(row, stride); }

// One operand's rows of a head, chunk after chunk.
struct Stream {
    const char* p;      // the chunk's first row
    uint32_t stride, width;
    __device__ __forceinline__ Stream(const Operand& x, int64_t row0, int head) {
        const uint32_t es = x.bf16 ? 2 : 4;
        stride = uint32_t(x.heads) * x.D * es;
        width = x.D * es;
        p = static_cast<const char*>(x.p) + row0 * stride + uint32_t(head) * width;
    }
    // n rows (none: also less than 0); what is read behind them is 0
    __device__ __forceinline__ rsrc_t rows(int n) const { return buf_rsrc(p, n > 0 ? (n - 1) * stride + width : 0); }
    __device__ __forceinline__ void move(int rows) { p += int64_t(rows) * stride; }
};

// Four neighbouring columns, dropped past the descriptor's end; n: how many there are.
template <typename T, bool WHOLE>
__device__ __forceinline__ void store4(rsrc_t d, uint32_t off, f32x4 x, int n) {
    const float v[4] = {x[0], x[1], x[2], x[3]};
    if constexpr (WHOLE) buf_store<T, 4, true>(d, off, v, 4);   // all or, at an offset that is nowhere, none
    else buf_store<T, 4, false>(d, off, v, n);
}

// The rows of one operand in a chunk: 16-byte pieces (8 bf16, 4 fp32), a few to a thread, held
// as they were loaded until stage() brings them to LDS.
template <typename O, int D, int THREADS, bool WHOLE, bool KEEP>
struct Rows {
    static constexpr int PER = D / O::E, N = O::L * PER / THREADS, APART = THREADS / PER;   // rows between a thread's pieces
    static_assert(O::L * PER % THREADS == 0 && THREADS % PER == 0);
    typename O::template Piece<WHOLE> r[N];

    uint32_t off;   // of the first piece; kept over the chunks where registers allow

    __device__ __forceinline__ Rows(const Stream& x, int D_, bool bf16) : off(KEEP ? place(x, D_, bf16) : 0) {}
    // A column past the last is nowhere.
    static __device__ __forceinline__ uint32_t place(const Stream& x, int D_, bool bf16) {
        const uint32_t tid = fresh<!KEEP>(threadIdx.x), col = tid % PER * O::E;
        return int(col) < D_ ? mul24(tid / PER, x.stride) + col * (bf16 ? 2 : 4) : kNowhere;
    }
    __device__ __forceinline__ void load(const Stream& x, int n, int D_, bool bf16) {
        const int col = WHOLE ? 0 : int(fresh<!KEEP>(threadIdx.x) % PER * O::E);
        const uint32_t o = KEEP ? off : place(x, D_, bf16);
        const rsrc_t d = x.rows(n);
        #pragma unroll
        for (int i = 0; i < N; ++i) r[i].load(d, o + uint32_t(i * APART) * x.stride, D_ - col, bf16);
    }
    __device__ __forceinline__ void stage(char* tile, bool bf16) const {
        const uint32_t tid = fresh<!KEEP>(threadIdx.x);
        #pragma unroll
        for (int i = 0; i < N; ++i) r[i].store(tile + O::template at<D>(tid / PER + i * APART, tid % PER), bf16);
    }
};

// The decays of a chunk's tokens, lane = token: g from memory, 0 behind the last.
__device__ __forceinline__ float load_g(const Chunks& w, float constant, int64_t row0, int n, int h, int lane) {
    if (!w.g_per_token) return lane < n ? constant : 0.f;
    const rsrc_t d = buf_rsrc(w.g + row0 * w.H, int64_t(n) * w.H * 4);
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(d, lane < n ? uint32_t(lane * w.H + h) * 4 : kNowhere, 0, 0));
}
template <bool BACK>
__device__ __forceinline__ void make_tables(float* tab, float g, float si, float su, int lane) {
    double u = double(g) * 1.4426950408889634074;
    u = u < kNoDecayLog2 ? kNoDecayLog2 : u;   // NaN stays NaN
    const double in = running_sum(u, lane), all = lane64(in, 63), X = BACK ? all - in : in, out = BACK ? in : all - in;
    const float hi = float(X);
    tab[lane] = hi;
    tab[64 + lane] = float(X - hi);
    tab[128 + lane] = __builtin_amdgcn_exp2f(hi) * si;
    tab[192 + lane] = __builtin_amdgcn_exp2f(float(out)) * su;
    if (lane == 0) tab[256] = __builtin_amdgcn_exp2f(float(all));
}

// S (or the part of it that a run of tokens adds) for the wave's columns.
template <typename O, int DA>
struct State {
    static constexpr int NA = DA / 16;
    f32x4 s[NA];

    // f(element, its byte offset in fp32 [DA][DC] (the state as it is stored) or its transpose) of every element.
    template <typename F>
    __device__ __forceinline__ void each(F&& f, int da, int dc, bool transposed, int wave, int lane) {
        lane = fresh(lane);
        const int j = 16 * wave + (lane & 15), si = transposed ? 1 : dc, sj = transposed ? da : 1;
        #pragma unroll
        for (int a = 0; a < NA; ++a) {
            const int i = O::row_of(a, lane >> 4);
            const uint32_t off = uint32_t(i * si + j * sj) * 4;
            #pragma unroll
            for (int r = 0; r < 4; ++r) {
                float x = s[a][r];
                f(x, (i + r < da) & (j < dc) ? off + uint32_t(r * si) * 4 : kNowhere);
                s[a][r] = x;
            }
            hold();
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
    // As it is held, in whole pieces.
    __device__ __forceinline__ void leave(float* p, int wave, int lane) {
        #pragma unroll
        for (int a = 0; a < NA; ++a) *reinterpret_cast<f32x4*>(p + ((wave * NA + a) * 64 + lane) * 4) = s[a];
    }
    __device__ __forceinline__ double dot(const float* p, int da, int dc, bool transposed, int wave, int lane) {
        const rsrc_t d = buf_rsrc(p, da * dc * 4);
        double sum = 0.0;
        each([&](float& x, uint32_t off) { sum += double(x) * __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(d, off, 0, 0)); }, da, dc, transposed, wave, lane);
        return sum;
    }
};

// The workgroup's place in the launch, in runs of neighbours for each XCD: the heads that share an operand
// fastest, then what is computed for them (`kinds`), segments, heads, sequences, so that rows that several
// read come from the XCD's L2.  The gradients of 2 x 16384 tokens, 32 heads of 128 sharing q and k in
// fours read 1.75 GB in this order; with heads slowest 3.0, and 3 % slower.
struct Place {
    int kind, seg, h, b;
    __device__ __forceinline__ Place(const Chunks& w, int segs, int kinds) {
        uint32_t i = uint32_t(xcd_order(blockIdx.x, gridDim.x));   // less than 2^32 threads
        const int in = int(i % w.group); i /= w.group;
        kind = int(i % kinds); i /= kinds;
        seg = int(i % segs); i /= segs;
        const int groups = w.H / w.group;
        h = int(i % groups) * w.group + in;
        b = int(i / groups);
    }
};

// One sweep over the tokens of a segment of sequence b, head h.
//   NP: how many operands of the matrix cores a value of S (for out) and of P is split into; 0: no out is
//       computed, only what the segment adds to a state.
//   DOTS: with s.dot, the rows' sums of out x.
template <typename O, int DA, int DC, int NP, bool BACK, bool DOTS, bool WHOLE>
__device__ void sweep(const Chunks& w, const Sweep& s, int b, int h, int seg, char* smem) {
    constexpr bool OUT = NP > 0;
    using Lay = Layout<O, DA, DC, NP>;
    using St = State<O, DA>;
    constexpr int L = O::L, K = O::K, NL = L / 16, NA = St::NA, kThreads = 4 * DC, kWaves = DC / 16;
    constexpr bool kTight = !(O::E == 8 && DA == 64 && DC == 64 && WHOLE);   // registers are short: less is kept and overlapped
    constexpr bool kShort = OUT && O::E == 8 && DA == 128 && DC == 128 && WHOLE;   // shorter: the next c is loaded late, too
    constexpr bool kKeep = WHOLE && O::E == 8 && !(DA == 128 && DC == 128);
    constexpr bool kPace = O::E == 8;
    constexpr bool kLateX = kShort || (DA == 128 && DC == 128);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    float* tabs = reinterpret_cast<float*>(smem + Lay::TAB);
    float* dots = reinterpret_cast<float*>(smem + Lay::DOT);
    const int len = seq_length(w.lengths, b, w.T);
    const int t0 = seg * w.seg_tokens, t1 = min(t0 + w.seg_tokens, w.T), end = min(t1, max(len, t0));
    const int nch = (end - t0 + L - 1) / L;
    const int64_t bh = int64_t(b) * w.H + h, row_t0 = int64_t(b) * w.T + t0;
    const int da = s.a.D, dc = s.c.D, elems = da * dc;
    const float si = s.si, su = s.su, sp = s.sp;

    float kept = 1.f;   // what is left of a state behind the segment

    auto bf16 = [](const Operand& x) { return O::E == 8 || x.bf16; };   // known where every operand is
    auto stream = [&](const Operand& x, int64_t row0, bool there = true) {
        return Stream({x.p, x.heads, x.D, bf16(x)}, row0, there ? h / (w.H / x.heads) : 0);
    };
    // chunk c0 .. c0 + n of the segment's tokens, the last of them first where it runs backwards
    constexpr int STEP = BACK ? -L : L;
    int c0 = BACK ? (nch - 1) * L : 0;
    Stream xa = stream(s.a, row_t0 + c0), xb = stream(s.b, row_t0 + c0), xc = stream(s.c, row_t0 + c0);
    Stream xx = stream(s.x, row_t0 + c0, DOTS && s.dot), xo({s.out, s.out_heads, dc, s.out_bf16}, row_t0 + c0, h);
    const bool a16 = bf16(s.a), b16 = bf16(s.b), c16 = bf16(s.c), x16 = bf16(s.x), o16 = s.out_bf16;
    const bool dot = DOTS && s.dot;

    Rows<O, DA, kThreads, WHOLE, kKeep> ra(xa, da, a16), rb(xb, da, b16);
    Rows<O, DC, kThreads, WHOLE, kKeep> rc(xc, dc, c16);
    const int tokens = end - t0;
    typename O::template Four<WHOLE> xr[NL];
    auto fetch_ab = [&](int n) {   // the next chunk's rows
        if constexpr (OUT) ra.load(xa, n, da, a16);
        rb.load(xb, n, da, b16);
        if constexpr (OUT) xa.move(STEP);
        xb.move(STEP);
    };
    auto fetch_c = [&](int n) {
        rc.load(xc, n, dc, c16);
        xc.move(STEP);
    };
    auto fetch_x = [&](int n) {   // (nothing where no sums are asked for)
        if constexpr (DOTS) {
            const uint32_t ln = fresh<kTight>(lane), l16 = ln & 15, j = 16 * wave + 4 * (ln >> 4);
            const rsrc_t d = xx.rows(dot ? n : 0);
            const uint32_t off = int(j) < dc ? mul24(l16, xx.stride) + j * (x16 ? 2 : 4) : kNowhere;
            #pragma unroll
            for (int ti = 0; ti < NL; ++ti) xr[ti].load(d, off + uint32_t(16 * ti) * xx.stride, dc - int(j), x16);
            xx.move(STEP);
        }
    };
    auto stage = [&](int ch) {
        char* tile = smem + (ch & 1) * Lay::NEXT;
        if constexpr (OUT) ra.stage(tile + Lay::A, a16);
        rb.stage(tile + Lay::B, b16);
        rc.stage(tile + Lay::C, c16);
    };
    // how many tokens the chunk `ahead` of the one at c0 has, or 0
    auto count = [&](int ch, int c0, int ahead) { return ch + ahead < nch ? min(L, tokens - c0 - ahead * STEP) : 0; };
    // Before the barrier that opens a chunk its rows are in LDS and the next one's under way.  The tables
    // are made by one wave a chunk ahead, from decays that were asked for a chunk before that: a wait for
    // them would be one for all the rows that were asked for since.
    constexpr int kTabWave = kWaves - 1;
    float g1 = 0.f, g2 = 0.f;
    const float gc = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(nch > 0 && !w.g_per_token ? w.g[h] : 0.f)));
    auto fetch_g = [&](int c, int n) { return load_g(w, gc, row_t0 + c, n, h, int(fresh(lane))); };
    float g0 = 0.f;
    if (nch > 0) {
        fetch_ab(count(0, c0, 0));
        fetch_c(count(0, c0, 0));
        if (wave == kTabWave) g0 = fetch_g(c0, count(0, c0, 0));
    }
    St S;
    {
        const float* first = s.s_in ? s.s_in + bh * elems : nullptr;
        const float* parts = OUT && w.segs > 1 ? s.ws + bh * w.segs * int64_t(elems) : nullptr;
        if (parts && w.chained) first = parts + int64_t(seg) * elems;
        S.load(OUT ? first : nullptr, da, dc, s.transposed, wave, lane);
        if (parts && !w.chained) {   // what the segments before this one add, one after another
            for (int i = 0; i < (BACK ? w.segs - 1 - seg : seg); ++i) {
                const int at = BACK ? w.segs - 1 - i : i;
                St U;
                U.load(parts + int64_t(at) * elems, da, dc, s.transposed, wave, lane);
                const float k = s.kept[bh * w.segs + at];
                #pragma unroll
                for (int a = 0; a < NA; ++a)
                    #pragma unroll
                    for (int r = 0; r < 4; ++r) S.s[a][r] = fmaf(S.s[a][r], k, U.s[a][r]);
            }
        }
    }
    if (nch > 0) {
        if (wave == kTabWave) {
            g1 = fetch_g(c0 + STEP, count(0, c0, 1));
            g2 = fetch_g(c0 + 2 * STEP, count(0, c0, 2));
            make_tables<BACK>(tabs, g0, si, su, lane);
            settle(g1);
        }
        if constexpr (OUT && K > 16) {   // the blocks of P that a wider contraction reads past the diagonal
            for (int i = tid; i < NP * L * L * Lay::es / 16; i += kThreads) *reinterpret_cast<uint4*>(smem + Lay::P + 16 * i) = uint4{0, 0, 0, 0};
        }
        stage(0);
        if constexpr (!kLateX) fetch_x(count(0, c0, 0));
        fetch_ab(count(0, c0, 1));
        if constexpr (!kShort) fetch_c(count(0, c0, 1));
    }
    auto put_dots = [&](int c, int n) {   // of the chunk at c, behind a barrier
        if (!dot || tid >= n) return;
        float d = 0.f;
        #pragma unroll
        for (int i = 0; i < kWaves; ++i) d += dots[64 * i + tid];
        s.dot[bh * w.T + t0 + c + tid] = d;
    };

    for (int ch = 0; ch < nch; ++ch) {
        const int n = count(ch, c0, 0);
        const float* tab = tabs + (ch & 1) * kTab;
        const char* tile = smem + (ch & 1) * Lay::NEXT;
        if constexpr (DOTS) {
            const int t = t0 + c0 + (BACK ? L : 0);
            if (s.marks && t % kMark == 0 && t > 0 && t < len) S.leave(s.marks + (bh * (w.runs - 1) + t / kMark - 1) * (DA * DC), wave, lane);
        }
        __syncthreads();
        if (OUT && ch > 0) put_dots(c0 - STEP, count(ch - 1, c0 - STEP, 0));
        if (wave == kTabWave) make_tables<BACK>(tabs + (ch + 1 & 1) * kTab, g1, si, su, lane);

        f32x4 out[NL];
        typename O::Frag cf[L / K];
        const uint32_t ln = fresh<kTight>(lane), l16 = ln & 15, g4 = ln >> 4;
        const typename O::template Lanes<DA> at_a(ln);
        const typename O::template Lanes<DC> at_c(ln);
        const typename O::template Lanes<L> at_p(ln);
        if constexpr (OUT) {
            // P: lane has row t, four neighbouring i
            constexpr int kTiles = NL * (NL + 1) / 2;
            #pragma unroll
            for (int q = 0; q < (kTiles + kWaves - 1) / kWaves; ++q) {
                const int p = wave + q * kWaves;
                if (p >= kTiles) break;
                const int far = p < 1 ? 0 : p < 3 ? 1 : p < 6 ? 2 : 3, near = p - far * (far + 1) / 2;
                const int ti = BACK ? near : far, ii = BACK ? far : near;
                f32x4 acc = {0.f, 0.f, 0.f, 0.f};
                #pragma unroll
                for (int m = 0; m < DA / K; ++m)
                    acc = O::mma(O::template row<DA>(smem + Lay::B, at_a, ii, m), O::template row<DA>(smem + Lay::A, at_a, ti, m), acc);
                const int t = 16 * ti + l16, i0 = 16 * ii + 4 * g4;
                const float xh = tab[t], xl = tab[64 + t];
                const f32x4 ih = *reinterpret_cast<const f32x4*>(tab + i0), il = *reinterpret_cast<const f32x4*>(tab + 64 + i0);
                float v[4];
                #pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float e = __builtin_amdgcn_exp2f((xh - ih[r]) + (xl - il[r]));
                    v[r] = (BACK ? i0 + r >= t : i0 + r <= t) ? sp * acc[r] * e : 0.f;
                }
                O::template store_p<NP>(smem + Lay::P, at_p, ti, ii, v);
                if constexpr (kTight) hold();
            }
            // what the state before the chunk gives
            #pragma unroll
            for (int ti = 0; ti < NL; ++ti) out[ti] = f32x4{0.f, 0.f, 0.f, 0.f};
            #pragma unroll
            for (int m = 0; m < DA / K; ++m) {
                typename O::Frag sf[NP];
                float v[O::E];
                #pragma unroll
                for (int e = 0; e < O::E; ++e) v[e] = S.s[m * (K / 16) + e / 4][e % 4];
                O::template split<NP>(v, sf);
                #pragma unroll
                for (int ti = 0; ti < NL; ++ti) {
                    const typename O::Frag af = O::template row<DA>(smem + Lay::A, at_a, ti, m);
                    #pragma unroll
                    for (int p = 0; p < NP; ++p) out[ti] = O::mma(sf[p], af, out[ti]);
                }
            }
            #pragma unroll
            for (int ti = 0; ti < NL; ++ti) out[ti] *= tab[128 + 16 * ti + l16];
            if constexpr (kTight) hold();
        }
        // the state behind the chunk: c times its decay to the chunk's end
        const float all = tab[256];
        if constexpr (!OUT) kept *= all;
        #pragma unroll
        for (int a = 0; a < NA; ++a) S.s[a] *= all;
        #pragma unroll
        for (int m = 0; m < L / K; ++m) {
            cf[m] = O::template col<DC>(tile + Lay::C, at_c, wave, m);
            const typename O::template Lanes<DA> at_b(fresh<O::E == 4>(ln));   // (32 addresses of single floats are not worth keeping)
            typename O::Frag cs[O::NP];
            float v[O::E];
            #pragma unroll
            for (int e = 0; e < O::E; ++e) v[e] = O::get(cf[m], e) * tab[192 + K * m + O::E * g4 + e];
            O::template split<O::NP>(v, cs);
            if constexpr (kPace) hold();
            #pragma unroll
            for (int a = 0; a < NA; ++a) {
                const typename O::Frag bf = O::template col_of_state<DA>(tile + Lay::B, at_b, a, m);
                #pragma unroll
                for (int p = 0; p < O::NP; ++p) S.s[a] = O::mma(bf, cs[p], S.s[a]);
            }
            if constexpr (kPace) pace<OUT ? 1 : 2, 2, O::NP, NA>();
        }
        if constexpr (kShort) {
            hold();
            fetch_c(count(ch, c0, 1));
        }
        if constexpr (kLateX) fetch_x(n);
        if constexpr (OUT) {
            if constexpr (kTight) {   // again, and in front of the barrier, behind which other waves write the next chunk there
                hold();
                #pragma unroll
                for (int m = 0; m < L / K; ++m) cf[m] = O::template col<DC>(tile + Lay::C, at_c, wave, m);
            }
            __syncthreads();
            #pragma unroll
            for (int m = 0; m < L / K; ++m) {
                #pragma unroll
                for (int ti = BACK ? 0 : m * K / 16; ti < (BACK ? (m + 1) * K / 16 : NL); ++ti)
                    #pragma unroll
                    for (int p = 0; p < NP; ++p)
                        out[ti] = O::mma(cf[m], O::template row<L>(smem + Lay::P + p * L * L * Lay::es, at_p, ti, m), out[ti]);
            }
        }
        stage(ch + 1);
        if constexpr (DOTS) {   // over a wave's columns by halves: the group of 16 lanes then has tile 0, 2, 1 or 3 (0, 0, 1, 1 of two)
            float v[NL], x[4];
            #pragma unroll
            for (int ti = 0; ti < NL; ++ti) {
                xr[ti].get(x, x16);
                v[ti] = 0.f;
                #pragma unroll
                for (int e = 0; e < 4; ++e) v[ti] = fmaf(out[ti][e], x[e], v[ti]);
            }
            if constexpr (NL == 4) {
                const float sum = halve<16>(halve<32>(v[0], v[1], ln), halve<32>(v[2], v[3], ln), ln);
                dots[wave * 64 + 16 * (g4 >> 1 | (g4 & 1) << 1) + l16] = sum;
            } else {
                static_assert(NL == 2);
                const float both = halve<32>(v[0], v[1], ln);
                dots[wave * 64 + 16 * (g4 >> 1) + l16] = halve<16>(both, both, ln);
            }
        }
        // the rows asked for a chunk ago are all there; the next ones are asked for before anything is stored,
        // since waiting for them waits for what was issued earlier
        g1 = g2;
        settle(g1);
        if (wave == kTabWave) g2 = fetch_g(c0 + 3 * STEP, count(ch, c0, 3));
        if constexpr (!kLateX) fetch_x(count(ch, c0, 1));
        fetch_ab(count(ch, c0, 2));
        if constexpr (!kShort) fetch_c(count(ch, c0, 2));
        if constexpr (OUT) {
            const int j = 16 * wave + 4 * g4;
            const rsrc_t d = xo.rows(n);
            const uint32_t off = j < dc ? mul24(l16, xo.stride) + uint32_t(j) * (o16 ? 2 : 4) : kNowhere;
            xo.move(STEP);
            if (o16) {
                #pragma unroll
                for (int ti = 0; ti < NL; ++ti) store4<bf16_t, WHOLE>(d, off + uint32_t(16 * ti) * xo.stride, out[ti], dc - j);
            } else {
                #pragma unroll
                for (int ti = 0; ti < NL; ++ti) store4<float, WHOLE>(d, off + uint32_t(16 * ti) * xo.stride, out[ti], dc - j);
            }
        }
        c0 += STEP;
    }
    if (OUT && dot && nch > 0) {
        __syncthreads();
        put_dots(c0 - STEP, count(nch - 1, c0 - STEP, 0));
    }
    if constexpr (OUT) {
        if (end < t1) {   // padding
            for (int64_t i = tid; i < int64_t(t1 - end) * dc; i += kThreads) {
                const int64_t o = ((int64_t(b) * w.T + end + i / dc) * s.out_heads + h) * dc + i % dc;
                if (o16) static_cast<bf16_t*>(s.out)[o] = 0;
                else static_cast<float*>(s.out)[o] = 0.f;
            }
            if (dot)
                for (int i = end + tid; i < t1; i += kThreads) s.dot[bh * w.T + i] = 0.f;
        }
        if (s.s_out && seg == (BACK ? 0 : w.segs - 1)) S.store(s.s_out + bh * elems, da, dc, s.transposed, wave, lane);
        if (DOTS && s.end_dot && seg == (BACK ? 0 : w.segs - 1)) {
            const double d = running_sum(S.dot(s.end_with + bh * elems, da, dc, s.transposed, wave, lane), lane);
            double* sums = reinterpret_cast<double*>(dots + kWaves * 64);
            if (lane == 63) sums[wave] = d;
            __syncthreads();
            if (tid == 0) {
                double all = 0.0;
                for (int i = 0; i < kWaves; ++i) all += sums[i];
                s.end_dot[bh] = all;
            }
        }
    } else {
        S.store(s.ws + (bh * w.segs + seg) * elems, da, dc, s.transposed, wave, lane);
        if (tid == 0) s.kept[bh * w.segs + seg] = kept;
    }
}

// What the segments add to a state; but the last, behind which none follows.
template <typename O, int DA, int DC, bool BACK, bool WHOLE>
__global__ __launch_bounds__(4 * DC, DA == 128 && DC == 64 ? 3 : WHOLE || O::E == 4 || DA == 64 ? 4 : 2) void parts_kernel(Chunks w, Sweep s) {
    __shared__ alignas(16) char smem[Layout<O, DA, DC, 0>::END];
    const Place at(w, w.segs - 1, 1);
    sweep<O, DA, DC, 0, BACK, false, WHOLE>(w, s, at.b, at.h, at.seg + BACK, smem);
}
// Waves to a SIMD: as many workgroups as their LDS allows, and no more than their registers do (rows
// that are not in whole pieces come in single elements, of which each takes a register).
template <typename O, int DA, int DC, int NP, bool WHOLE>
constexpr int waves_per_simd() {
    constexpr int lds = 160 * 1024 / Layout<O, DA, DC, NP>::END * (DC / 64), regs = DA == 128 ? (DC == 128 && WHOLE ? 4 : 2) : (WHOLE || O::E == 4) ? 4 : DC == 128 ? 2 : 3;
    return lds < regs ? lds : regs;
}
// One output.
template <typename O, int DA, int DC, int NP, bool BACK, bool DOTS, bool WHOLE>
__global__ __launch_bounds__(4 * DC, (waves_per_simd<O, DA, DC, NP, WHOLE>())) void outs_kernel(Chunks w, Sweep s) {
    __shared__ alignas(16) char smem[Layout<O, DA, DC, NP>::END];
    const Place at(w, w.segs, 1);
    sweep<O, DA, DC, NP, BACK, DOTS, WHOLE>(w, s, at.b, at.h, at.seg, smem);
}

struct Three {
    Sweep s[3];
};
// dq, dk and dv side by side, where keys and values are of one width.
template <typename O, int D, bool WHOLE>
__global__ __launch_bounds__(4 * D, (waves_per_simd<O, D, D, O::NP, WHOLE>())) void grads_kernel(Chunks w, Three s) {
    __shared__ alignas(16) char smem[Layout<O, D, D, O::NP>::END];
    const Place at(w, w.segs, 3);
    if (at.kind == 0) sweep<O, D, D, O::NP, false, true, WHOLE>(w, s.s[0], at.b, at.h, at.seg, smem);
    else sweep<O, D, D, O::NP, true, true, WHOLE>(w, s.s[at.kind], at.b, at.h, at.seg, smem);
}

// Heads are computed at 64 or 128, with zeros behind a smaller one's values; WHOLE: rows in whole 16-byte pieces.
template <typename O, typename F>
inline hipError_t with_widths(int da, int dc, F&& f) {
    using N64 = std::integral_constant<int, 64>;
    using N128 = std::integral_constant<int, 128>;
    auto whole = [&](auto a, auto c) { return da % O::E == 0 && dc % O::E == 0 ? f(a, c, std::true_type{}) : f(a, c, std::false_type{}); };
    if (da <= 64) return dc <= 64 ? whole(N64{}, N64{}) : whole(N64{}, N128{});
    return dc <= 64 ? whole(N128{}, N64{}) : whole(N128{}, N128{});
}
inline bool same_width(int d, int e) { return (d <= 64) == (e <= 64); }

template <typename O>
inline hipError_t launch_parts(const Chunks& w, const Sweep& s, hipStream_t st) {
    return with_widths<O>(s.a.D, s.c.D, [&](auto da, auto dc, auto whole) {
        const dim3 grid(uint32_t(int64_t(w.B) * w.H * (w.segs - 1)));
        if (s.back) parts_kernel<O, da, dc, true, whole><<<grid, 4 * dc, 0, st>>>(w, s);
        else parts_kernel<O, da, dc, false, whole><<<grid, 4 * dc, 0, st>>>(w, s);
        return hipGetLastError();
    });
}
template <typename O, bool BACK, bool DOTS>
inline hipError_t launch_outs(const Chunks& w, const Sweep& s, hipStream_t st) {
    return with_widths<O>(s.a.D, s.c.D, [&](auto da, auto dc, auto whole) {
        if constexpr (DOTS && da == dc) {
            return hipErrorInvalidValue;   // grads_kernel's
        } else {
            outs_kernel<O, da, dc, O::NP, BACK, DOTS, whole><<<dim3(uint32_t(int64_t(w.B) * w.H * w.segs)), 4 * dc, 0, st>>>(w, s);
            return hipGetLastError();
        }
    });
}
template <typename O>
inline hipError_t launch_backward(const Chunks& w, const Sweep& q, const Sweep& k, const Sweep& v, hipStream_t st) {
    if (same_width(v.a.D, v.c.D))
        return with_widths<O>(v.a.D, v.c.D, [&](auto d, auto, auto whole) {
            grads_kernel<O, d, whole><<<dim3(uint32_t(int64_t(w.B) * w.H * w.segs * 3)), 4 * d, 0, st>>>(w, Three{{q, k, v}});
            return hipGetLastError();
        });
    hipError_t e = launch_outs<O, false, true>(w, q, st);
    if (e == hipSuccess) e = launch_outs<O, true, true>(w, k, st);
    return e != hipSuccess ? e : launch_outs<O, true, true>(w, v, st);
}

}  // namespace linattn
}  // namespace wkv7
