// Gradients of the selective state space scan on gfx950.  With do_t = dy_t
// silu(z_t) and e_t = dL/dh_t, per channel and state n:
//
//   e_t = do_t C_t + exp(d_{t+1} A) e_{t+1}          (from the last token back; dstate_out enters there)
//   dB_t = sum_c e_t d_t x_t,   dC_t = sum_c do_t h_t,
//   q_t = e_t exp(d_t A) h_{t-1},   dA = sum_t q_t d_t,
//   du_t = sum_n e_t B_t,   dd_t = sum_n q_t A + du_t x_t,
//   dx_t = du_t d_t + do_t D,   ddt_t = dd_t softplus'(dt_t + dt_bias),
//   dz_t = dy_t y'_t silu'(z_t)   with y' the output before the gate
//
// A wave has 16 channels, 16 tokens and 8 states: lane (q, c) of its 4 rows of 16
// lanes has states 2 q, 2 q + 1 of channel c, and holds B and C of token c for them,
// which an operand modifier hands to the whole row when their token comes.  WS waves
// share the states of a token run and its elements (step sizes, products, gates, which
// each computes a part of, through LDS); the WT runs of a workgroup follow one another.
// The workgroup goes from its last 16 WT tokens to its first.  A round computes the
// decays of its tokens (kept in registers), each run's state from zero and its
// gradient from zero, and exchanges both with the run's decay through LDS, so that
// every run has its incoming state, from the checkpoint of the round, and its incoming
// gradient, from the later round's; it runs the states forward once more, into
// registers, and then the gradients backward.  Two states a lane keep it within 128
// registers, which is what lets four waves share a SIMD: with four states a lane and
// two waves the same work issued a fifth more slowly.
//
// Bound: the vector units, busy 83% of the time.  33 instructions per state and token:
// 9 run the gradients back and 6 or 7 are the sums over rows and channels; the others are
// the decays, the states from zero and once more, the gradients from zero, the exchange and
// the elements.  4 x 2048 tokens x 2048 channels of 16 states, bf16: 306 to 320 us,
// 154 MB read and 236 MB written, 134 of which are the blocks' dB and dC.
//
// Sums over the rows and over a row's channels are transposing butterflies: a step
// halves the values that a lane holds while it doubles the lanes summed.  dB and dC of
// a wave's channels go to the workspace, one row for each block of channels, and a
// second kernel adds the rows; no atomics, so the order is fixed.  dA, dD and ddt_bias
// are kept in registers over the whole sequence and added over the batch by a third.
#include "seq_device.h"
#include "seq_internal.h"

namespace wkv7 {
namespace {

constexpr int TW = 16, CH = 16, TP = 20, NPL = 2;
constexpr int PT = 8;   // tokens whose states are in registers at once
constexpr float kLn2 = 0.6931471805599453f;

struct BwdWs {
    float* bc;    // [ncb][B][T][G][2][N]: dB and dC of each block of channels
    float* par;   // [B][C N + 2 C]: dA, dD, ddt_bias of each sequence
    const float* ck;
};

// One token backward, for the two states of a lane.  In: e, the gradient of the state as later
// tokens left it.  e += C do; y = C . h and us = B . e are the lane's parts of the readout and of
// the input's gradient.  B and C of lane T of the row, by operand modifiers (the compiler folds
// them into products only).
template <int T>
__device__ __forceinline__ void token_back(float (&e)[2], const float* C, const float* B, float o, const float* h, float& y, float& us) {
#define WKV7_BC " row_newbcast:%c[t] row_mask:0xf bank_mask:0xf\n"
    asm("s_nop 1\n"
        "v_fmac_f32_dpp %0, %4, %8" WKV7_BC "v_fmac_f32_dpp %1, %5, %8" WKV7_BC
        "v_mul_f32_dpp %2, %4, %9" WKV7_BC "v_mul_f32_dpp %3, %6, %0" WKV7_BC
        "v_fmac_f32_dpp %2, %5, %10" WKV7_BC "v_fmac_f32_dpp %3, %7, %1" WKV7_BC
        : "+&v"(e[0]), "+&v"(e[1]), "=&v"(y), "=&v"(us)
        : "v"(C[0]), "v"(C[1]), "v"(B[0]), "v"(B[1]), "v"(o), "v"(h[0]), "v"(h[1]), [t] "n"(T));
#undef WKV7_BC
}

// lo in the lanes whose bit 3 (2) is 0, hi in the others, each summed over the lane and its mirror
// in 16 (8): the second sum is written to the upper banks of four lanes only.
template <int M>
__device__ __forceinline__ void halve_banks(float& a0, float b0, float& a1, float b1) {
    float r0, r1;
    if constexpr (M == 8)
        asm("s_nop 1\nv_add_f32_dpp %0, %2, %2 row_mirror row_mask:0xf bank_mask:0xf\nv_add_f32_dpp %1, %4, %4 row_mirror row_mask:0xf bank_mask:0xf\n"
            "v_add_f32_dpp %0, %3, %3 row_mirror row_mask:0xf bank_mask:0xc\nv_add_f32_dpp %1, %5, %5 row_mirror row_mask:0xf bank_mask:0xc"
            : "=&v"(r0), "=&v"(r1) : "v"(a0), "v"(b0), "v"(a1), "v"(b1));
    else
        asm("s_nop 1\nv_add_f32_dpp %0, %2, %2 row_half_mirror row_mask:0xf bank_mask:0xf\nv_add_f32_dpp %1, %4, %4 row_half_mirror row_mask:0xf bank_mask:0xf\n"
            "v_add_f32_dpp %0, %3, %3 row_half_mirror row_mask:0xf bank_mask:0xa\nv_add_f32_dpp %1, %5, %5 row_half_mirror row_mask:0xf bank_mask:0xa"
            : "=&v"(r0), "=&v"(r1) : "v"(a0), "v"(b0), "v"(a1), "v"(b1));
    a0 = r0;
    a1 = r1;
}

// x, by a way that the compiler does not see through: what is computed from it is computed where it
// is used, and not kept in registers over the loop.
__device__ __forceinline__ int opaque(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// Waves to a SIMD that the registers are held to: 4 where they fit, or have to because the
// workgroup has 16 waves.
constexpr int waves_of(int WS, int WT, bool vec) { return WS * WT >= 16 || (vec && WT > 1 && WS * WT >= 8) ? 4 : 2; }

// WS waves with 8 states each; WT runs of 16 tokens.  VEC: rows of channels and of states start on
// 4 bytes, for each group too, and no lane has only one of its two states.
template <typename Tin, typename Ty, int WS, int WT, bool VEC>
__global__ __launch_bounds__(64 * WS * WT, waves_of(WS, WT, VEC)) void ssm_backward_kernel(SsmParams g, BwdWs ws) {
    constexpr int ROUND = TW * WT, NP = 8 * WS, E = WS <= 2 ? 4 / WS : 1, ES = int(sizeof(Tin)), YS = int(sizeof(Ty));
    __shared__ float s_d[WT][CH][TP], s_u[WT][CH][TP], s_o[WT][CH][TP], s_k[2][WT][CH][TP];   // d, d x, do; softplus', dz's factor
    __shared__ float s_r[WT][WS][3][CH][TP];
    __shared__ float s_x[3][WT][WS][NPL][64];      // decay, state and gradient of each run
    __shared__ float s_bc[WT][TW][2][NP];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int s = wv % WS, w = wv / WS;            // part of the states, run
    const unsigned item = unsigned(xcd_order(blockIdx.x, gridDim.x));
    const int Cg = g.C / g.G;
    const unsigned ncb = (Cg + CH - 1) / CH;
    const int cb = int(item % ncb), grp = int(item / ncb % g.G);
    const int64_t b = item / ncb / g.G;
    const int c0 = grp * Cg + cb * CH, nc = min(CH, Cg - cb * CH);
    const int len = __builtin_amdgcn_readfirstlane(seq_length(g.lengths, b, g.T));

    const int ch = lane & 15, q = lane >> 4, n0 = s * 8 + q * NPL;
    const int64_t srow = (b * g.C + c0 + ch) * g.N + n0;
    float A2[NPL], gc[NPL], dA[NPL] = {};
    bool n_in[NPL];
    #pragma unroll
    for (int i = 0; i < NPL; ++i) {
        n_in[i] = ch < nc && n0 + i < g.N;
        A2[i] = n_in[i] ? g.A[int64_t(c0 + ch) * g.N + n0 + i] * kLog2e : 0.f;
        gc[i] = n_in[i] && g.ds1 ? g.ds1[srow + i] : 0.f;   // gradient of the state after the round
    }
    // A thread's elements: token te, channels e0 .. e0 + E of its run (WS = 8: the first half's threads).
    const int idx = (s * 64 + lane) * E, te = idx >> 4 & 15, e0 = idx & 15, ne = idx < 256 ? nc - e0 : 0;
    const bool el_in = ne > 0;
    float dD[E] = {}, dbias[E] = {};
    __shared__ float s_par[2][CH];   // dt_bias and D of the channels
    if (threadIdx.x < 2 * CH) {
        const float* p = threadIdx.x < CH ? g.dt_bias : g.D;
        s_par[threadIdx.x >> 4][ch] = p && ch < nc ? p[c0 + ch] : 0.f;
    }
    __syncthreads();
    const uint32_t soft = g.softplus ? ~0u : 0u;
    const float no_z = g.z ? 0.f : 1.f;

    // Rows of a round through descriptors that end with the sequence: a padded token's values are 0.
    const int64_t erow = int64_t(g.C) * ES, vrow = int64_t(g.G) * g.N * ES, yrow = int64_t(g.C) * YS;
    const uint32_t eoff = el_in ? uint32_t((w * TW + te) * g.C + c0 + e0) : 0u;
    const uint32_t voff = n0 < g.N ? uint32_t((w * TW + ch) * g.G * g.N + grp * g.N + n0) * ES : kNowhere;
    struct Inputs {
        Raw<Tin, E, VEC> x, dt, z;
        Raw<Ty, E, VEC> dy;
        Raw<Tin, NPL, VEC> b, c;
        Raw<float, NPL, VEC> h;
    } nx;
    auto load = [&](int t0) {
        const int n = max(0, min(len - t0, ROUND));
        const int64_t row = b * g.T + t0;
        auto rows = [&](const void* p, int64_t width) { return buf_rsrc(static_cast<const char*>(p) + row * width, p ? n * width : 0); };
        nx.dt.load(rows(g.dt, erow), eoff * ES, ne);
        nx.x.load(rows(g.x, erow), eoff * ES, ne);
        nx.z.load(rows(g.z, erow), eoff * ES, ne);
        nx.dy.load(rows(g.dy, yrow), eoff * YS, ne);
        nx.b.load(rows(g.Bm, vrow), voff, g.N - n0);
        nx.c.load(rows(g.Cm, vrow), voff, g.N - n0);
        const rsrc_t ck = buf_rsrc(ws.ck + ((b * g.nck + t0 / SSM_CHECKPOINT_TOKENS) * g.C + c0) * g.N, int64_t(nc) * g.N * 4);
        nx.h.load(ck, n0 < g.N ? uint32_t(ch * g.N + n0) * 4 : kNowhere, g.N - n0);
    };
    auto store = [&](void* p, int t0, int end, const float* v, uint32_t eoff, int ne) {   // of the tokens before `end`
        const int n = min(end - t0, ROUND);
        buf_store<Tin, E, VEC>(buf_rsrc(static_cast<char*>(p) + (b * g.T + t0) * erow, n * erow), eoff * ES, v, ne);
    };

    const int rounds = (len + ROUND - 1) / ROUND;
    for (int t0 = len; t0 < g.T; t0 += ROUND) {   // padding: 0, also where a state or its gradient is no number
        const float zero[E] = {};
        store(g.dx, t0, g.T, zero, eoff, ne);
        store(g.ddt, t0, g.T, zero, eoff, ne);
        if (g.z) store(g.dz, t0, g.T, zero, eoff, ne);
    }
    if (rounds > 0) load((rounds - 1) * ROUND);
    for (int rd = rounds - 1; rd >= 0; --rd) {
        const int t0 = rd * ROUND, tw = t0 + w * TW;
        float Bv[NPL], Cv[NPL], hin[NPL];
        const auto x_c = nx.x;
        {   // elements; a padded token, and a channel that is not there, have x = d = do = 0
            const uint32_t keep = tw + te < len && el_in ? ~0u : 0u;
            #pragma unroll
            for (int i = 0; i < E; ++i) {
                const uint32_t k = i < ne ? keep : 0u;
                // softplus and its derivative from one exponential: e = exp(-|v|), 1 / (1 + e) or e / (1 + e)
                const float v = nx.dt.get(i) + s_par[0][e0 + i], ex = __builtin_amdgcn_exp2f(-kLog2e * fabsf(v));
                const float r = __builtin_amdgcn_rcpf(1.f + ex), sp = fmaxf(v, 0.f) + log1p_unit(ex), sg = v > 0.f ? r : ex * r;
                const float z = nx.z.get(i), sz = sigmoidf_(z), dy = nx.dy.get(i);
                auto kept = [&](float f) { return __uint_as_float(__float_as_uint(f) & k); };
                const float d = kept(bit_select(soft, sp, v));
                if (idx < 256) {
                    s_k[0][w][e0 + i][te] = kept(bit_select(soft, sg, 1.f));
                    s_k[1][w][e0 + i][te] = kept(dy * sz * fmaf(z, 1.f - sz, 1.f));
                    s_d[w][e0 + i][te] = d;
                    s_u[w][e0 + i][te] = kept(d * nx.x.get(i));
                    s_o[w][e0 + i][te] = kept(dy * fmaf(z, sz, no_z));
                }
            }
            #pragma unroll
            for (int i = 0; i < NPL; ++i) {
                Bv[i] = nx.b.get(i);
                Cv[i] = nx.c.get(i);
                hin[i] = nx.h.get(i);
            }
        }
        __syncthreads();

        // Decays; the state and the gradient that the run gives from zero, and its decay.
        float a[TW][NPL], Hm[NPL], dm = 0.f;   // after the first PT tokens: the state from zero, the sum of d
        {
            float hl[NPL] = {}, el[NPL] = {}, ds = 0.f;
            static_for<TW / 4>([&](auto t4) {
                if constexpr (t4 * 4 == PT) {
                    dm = ds;
                    #pragma unroll
                    for (int i = 0; i < NPL; ++i) Hm[i] = hl[i];
                }
                const f32x4 d4 = *reinterpret_cast<const f32x4*>(&s_d[w][ch][t4 * 4]);
                const f32x4 u4 = *reinterpret_cast<const f32x4*>(&s_u[w][ch][t4 * 4]);
                static_for<4>([&](auto j_) {
                    constexpr int j = j_, tt = t4 * 4 + j;
                    ds += d4[j];
                    #pragma unroll
                    for (int i = 0; i < NPL; ++i) {
                        a[tt][i] = __builtin_amdgcn_exp2f(d4[j] * A2[i]);
                        hl[i] = fmaf(a[tt][i], hl[i], u4[j] * row_lane<tt>(Bv[i]));
                    }
                });
            });
            if constexpr (WT > 1) {
                static_for<TW / 4>([&](auto r4) {
                    constexpr int t4 = TW / 4 - 1 - r4;
                    const f32x4 o4 = *reinterpret_cast<const f32x4*>(&s_o[w][ch][t4 * 4]);
                    static_for<4>([&](auto j_) {
                        constexpr int j = 3 - j_, tt = t4 * 4 + j;
                        #pragma unroll
                        for (int i = 0; i < NPL; ++i) el[i] = a[tt][i] * (o4[j] * row_lane<tt>(Cv[i]) + el[i]);
                    });
                });
                #pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    s_x[0][w][s][i][lane] = __builtin_amdgcn_exp2f(ds * A2[i]);
                    s_x[1][w][s][i][lane] = hl[i];
                    s_x[2][w][s][i][lane] = el[i];
                }
            }
        }
        float gi[NPL];   // gradient of the state after the run
        if constexpr (WT > 1) {
            __syncthreads();
            #pragma unroll
            for (int v = 0; v < WT - 1; ++v) {
                if (v >= w) break;
                #pragma unroll
                for (int i = 0; i < NPL; ++i) hin[i] = fmaf(s_x[0][v][s][i][lane], hin[i], s_x[1][v][s][i][lane]);
            }
            #pragma unroll
            for (int v = WT - 1; v >= 0; --v) {
                if (v == w) {
                    #pragma unroll
                    for (int i = 0; i < NPL; ++i) gi[i] = gc[i];
                }
                #pragma unroll
                for (int i = 0; i < NPL; ++i) gc[i] = fmaf(s_x[0][v][s][i][lane], gc[i], s_x[2][v][s][i][lane]);
            }
        } else {
            #pragma unroll
            for (int i = 0; i < NPL; ++i) gi[i] = gc[i];
        }
        // The run's states and gradients, the later PT tokens first.
        float dAr[NPL] = {};
        static_for<TW / PT>([&](auto rp) {
        constexpr int tp = TW - PT - rp * PT;
        float h[PT][NPL], hb[NPL];   // hb: the state before the part
        #pragma unroll
        for (int i = 0; i < NPL; ++i) hb[i] = tp ? fmaf(__builtin_amdgcn_exp2f(dm * A2[i]), hin[i], Hm[i]) : hin[i];
        static_for<PT / 4>([&](auto p4) {
            const f32x4 u4 = *reinterpret_cast<const f32x4*>(&s_u[w][ch][tp + p4 * 4]);
            static_for<4>([&](auto j_) {
                constexpr int j = j_, tt = p4 * 4 + j;
                #pragma unroll
                for (int i = 0; i < NPL; ++i)
                    h[tt][i] = fmaf(a[tp + tt][i], tt ? h[tt ? tt - 1 : 0][i] : hb[i], u4[j] * row_lane<tp + tt>(Bv[i]));
            });
        });
        // four tokens at a time
        static_for<PT / 4>([&](auto r4) {
            constexpr int t4 = (tp + PT) / 4 - 1 - r4;
            __builtin_amdgcn_sched_barrier(0);
            const f32x4 d4 = *reinterpret_cast<const f32x4*>(&s_d[w][ch][t4 * 4]);
            const f32x4 u4 = *reinterpret_cast<const f32x4*>(&s_u[w][ch][t4 * 4]);
            const f32x4 o4 = *reinterpret_cast<const f32x4*>(&s_o[w][ch][t4 * 4]);
            float y[4], us[4], ds[4], bc[16];
            static_for<4>([&](auto j_) {
                constexpr int j = 3 - j_, tt = t4 * 4 + j;
                token_back<tt>(gi, Cv, Bv, o4[j], h[tt - tp], y[j], us[j]);
                ds[j] = 0.f;
                #pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    bc[j * 4 + i] = gi[i] * u4[j];
                    bc[j * 4 + 2 + i] = h[tt - tp][i] * o4[j];
                    gi[i] *= a[tt][i];
                    const float qt = gi[i] * (tt > tp ? h[tt > tp ? tt - tp - 1 : 0][i] : hb[i]);
                    ds[j] = fmaf(qt, A2[i], ds[j]);
                    dAr[i] = fmaf(qt, d4[j], dAr[i]);
                }
                // over the rows, and the channels: as soon as the pair of tokens is there
                if constexpr (j < 2) {
                    asm("s_nop 1" : "+v"(y[j]), "+v"(us[j]));   // from their write, which the compiler does not see, to the swap
                    y[j] = halve<32>(y[j], y[j + 2], lane);
                    us[j] = halve<32>(us[j], us[j + 2], lane);
                    ds[j] = halve<32>(ds[j], ds[j + 2], lane);
                    halve_banks<8>(bc[j * 4], bc[j * 4 + 8], bc[j * 4 + 1], bc[j * 4 + 9]);
                    halve_banks<8>(bc[j * 4 + 2], bc[j * 4 + 10], bc[j * 4 + 3], bc[j * 4 + 11]);
                }
            });
            // dB and dC: values (token, which, state); a lane keeps the one that its bits 3 .. 0 name
            #pragma unroll
            for (int v = 0; v < 4; v += 2) halve_banks<4>(bc[v], bc[v + 4], bc[v + 1], bc[v + 5]);
            #pragma unroll
            for (int v = 0; v < 2; ++v) bc[v] = halve<2>(bc[v], bc[v + 2], lane);
            s_bc[w][t4 * 4 + (ch >> 2)][ch >> 1 & 1][n0 + (ch & 1)] = halve<1>(bc[0], bc[1], lane);
            // row q keeps token q
            s_r[w][s][0][ch][t4 * 4 + q] = halve<16>(y[0], y[1], lane);
            s_r[w][s][1][ch][t4 * 4 + q] = halve<16>(us[0], us[1], lane);
            s_r[w][s][2][ch][t4 * 4 + q] = halve<16>(ds[0], ds[1], lane);
            // (without this the compiler puts off the sum and keeps all its terms)
            #pragma unroll
            for (int i = 0; i < NPL; ++i) settle(dAr[i]);
        });
        });
        if (rd > 0) load(t0 - ROUND);   // here, where the registers of the decays and states are free
        #pragma unroll
        for (int i = 0; i < NPL; ++i) {
            dA[i] += dAr[i];
            if constexpr (WT == 1) gc[i] = gi[i];
        }
        __syncthreads();
        const int thr = opaque(s * 64 + lane);
        if (thr * E < 256) {
            const int te = thr * E >> 4, e0 = thr * E & 15, ne = nc - e0;
            const uint32_t eoff = uint32_t((w * TW + te) * g.C + c0 + e0);
            float dx[E], ddt[E], dz[E];
            #pragma unroll
            for (int i = 0; i < E; ++i) {
                const float x = x_c.get(i), d = s_d[w][e0 + i][te], o = s_o[w][e0 + i][te], Dv = s_par[1][e0 + i];
                float y = Dv * x, du = 0.f, dd = 0.f;
                #pragma unroll
                for (int v = 0; v < WS; ++v) {
                    y += s_r[w][v][0][e0 + i][te];
                    du += s_r[w][v][1][e0 + i][te];
                    dd += s_r[w][v][2][e0 + i][te];
                }
                dd = fmaf(du, x, dd * kLn2);
                dx[i] = fmaf(du, d, o * Dv);
                ddt[i] = dd * s_k[0][w][e0 + i][te];
                dz[i] = s_k[1][w][e0 + i][te] * y;
                dD[i] = fmaf(o, x, dD[i]);
                dbias[i] += ddt[i];
            }
            store(g.dx, t0, len, dx, eoff, ne);
            store(g.ddt, t0, len, ddt, eoff, ne);
            if (g.z) store(g.dz, t0, len, dz, eoff, ne);
        }
        // dB and dC of the run, 4 tokens at once.
        {
            const int r = thr & (2 * NP - 1), kind = r / NP, n = r % NP, width = g.G * 2 * g.N;
            const rsrc_t bc = buf_rsrc(ws.bc + (((int64_t(cb) * g.B + b) * g.T + tw) * g.G + grp) * 2 * g.N,
                                       int64_t(max(0, min(len - tw, TW))) * width * 4);
            if (n < g.N) {
                #pragma unroll
                for (int k = 0; k < TW; k += 4) {
                    const int tt = k + thr / (2 * NP);
                    if (tw + tt < len)
                        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(s_bc[w][tt][kind][n]), bc, uint32_t(tt * width + kind * g.N + n) * 4, 0, 0);
                }
            }
        }
        __syncthreads();   // the LDS rows are free again
    }
    // Places once more, from scratch.
    const int lane_ = opaque(lane), ch_ = lane_ & 15, n0_ = s * 8 + (lane_ >> 4) * NPL;
    auto there = [&](int i) { return ch_ < nc && n0_ + i < g.N; };
    if (g.ds0 && w == 0) {
        #pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (there(i)) g.ds0[(b * g.C + c0 + ch_) * g.N + n0_ + i] = gc[i];
    }
    // The parameters' gradients of this sequence, summed over the runs, and over the tokens of a channel.
    __syncthreads();
    #pragma unroll
    for (int i = 0; i < NPL; ++i) s_x[0][w][s][i][lane_] = dA[i];
    const int idx_ = (s * 64 + lane_) * E;
    if (idx_ < 256) {
        #pragma unroll
        for (int i = 0; i < E; ++i) {
            s_d[w][(idx_ & 15) + i][idx_ >> 4] = dD[i];
            s_u[w][(idx_ & 15) + i][idx_ >> 4] = dbias[i];
        }
    }
    __syncthreads();
    float* out = ws.par + b * (int64_t(g.C) * g.N + 2 * g.C);
    if (w == 0) {
        #pragma unroll
        for (int i = 0; i < NPL; ++i) {
            float sum = 0.f;
            #pragma unroll
            for (int v = 0; v < WT; ++v) sum += s_x[0][v][s][i][lane_];
            if (there(i)) out[int64_t(c0 + ch_) * g.N + n0_ + i] = sum;
        }
    }
    if (wv == 0 && lane_ < 2 * CH && ch_ < nc) {
        const bool second = lane_ >= CH;
        float sum = 0.f;
        for (int v = 0; v < WT; ++v)
            #pragma unroll
            for (int t = 0; t < TW; ++t) sum += second ? s_u[v][ch_][t] : s_d[v][ch_][t];
        out[int64_t(g.C) * g.N + (second ? g.C : 0) + c0 + ch_] = sum;
    }
}

// dBm and dCm: the sums over the blocks of channels.  A workgroup has 64 runs of V values and 4
// threads to each, which take every fourth block.
template <int V>
__global__ __launch_bounds__(256) void ssm_sum_bc_kernel(SsmParams g, const float* bc, int ncb) {
    const int64_t M = int64_t(g.B) * g.T * g.G * 2 * g.N;
    const int64_t m = (int64_t(blockIdx.x) * 64 + (threadIdx.x & 63)) * V;
    const int y = threadIdx.x >> 6;
    const bool in = m < M;
    const int64_t bt = m / (2 * g.N), row = bt / g.G, b = in ? row / g.T : 0;
    float s[V] = {};
    if (in && row - b * g.T < seq_length(g.lengths, b, g.T)) {
        #pragma unroll 4
        for (int i = y; i < ncb; i += 4) {
            const Pack<float, V> p = ld_pack<V>(bc + i * M + m, true, V);
            #pragma unroll
            for (int v = 0; v < V; ++v) s[v] += p.e[v];
        }
    }
    __shared__ float sm[3][64][V];
    if (y > 0) {
        #pragma unroll
        for (int v = 0; v < V; ++v) sm[y - 1][threadIdx.x & 63][v] = s[v];
    }
    __syncthreads();
    if (y > 0 || !in) return;
    #pragma unroll
    for (int v = 0; v < V; ++v)
        for (int o = 0; o < 3; ++o) s[v] += sm[o][threadIdx.x][v];
    const int n = int(m % g.N);
    st_pack_as<V>(m / g.N % 2 ? g.dCm : g.dBm, bt * g.N + n, g.in_bf16, s, true, V);
}

// dA, dD and ddt_bias: the sums over the batch.
__global__ __launch_bounds__(256) void ssm_sum_batch_kernel(SsmParams g, const float* par) {
    const int64_t CN = int64_t(g.C) * g.N, M = CN + 2 * g.C;
    const int64_t m = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (m >= M) return;
    float s = 0.f;
    for (int b = 0; b < g.B; ++b) s += par[b * M + m];
    if (m < CN) g.dA[m] = s;
    else if (m < CN + g.C) {
        if (g.dD) g.dD[m - CN] = s;
    } else if (g.dbias) g.dbias[m - CN - g.C] = s;
}

// Without tokens: the state's gradient goes back as it came (or 0).
__global__ __launch_bounds__(256) void ssm_no_tokens_kernel(const float* from, float* to, int64_t n) {
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) to[i] = from ? from[i] : 0.f;
}

int blocks_of(const SsmParams& p) { return (p.C / p.G + CH - 1) / CH; }
int64_t up(int64_t x) { return (x + 255) & ~int64_t(255); }
int64_t bc_bytes(const SsmParams& p) { return up(int64_t(blocks_of(p)) * p.B * p.T * p.G * 2 * p.N * 4); }
int64_t par_bytes(const SsmParams& p) { return up(int64_t(p.B) * (int64_t(p.C) * p.N + 2 * p.C) * 4); }

// Waves over the states, 8 to each.
int states_waves(const SsmParams& p) { return p.N <= 8 ? 1 : p.N <= 16 ? 2 : p.N <= 32 ? 4 : 8; }
// Token runs of a workgroup, as many as the chip has room for: 16 waves while it has a compute unit to
// itself, then fewer, which saves the waits of many.  A round starts at a checkpoint, so more than 16
// tokens take two runs or more.  1024 tokens, N = 16, us with 2, 4, 8 runs: 256 workgroups 145, 109, 99;
// 512: 196, 173, 185; 1536: 454, 458, 528; 4096: 1105, 1183, 1403.  N = 8 with 4, 8: 256: 85, 70; 1024: 203,
// 248.  512 tokens, N = 32, with 2, 4: 256: 103, 92; 512: 155, 168; 4096: 1123, 1357.
int runs_of(const SsmParams& p) {
    static_assert(SSM_CHECKPOINT_TOKENS == 2 * TW);
    const int ws = states_waves(p);
    const int64_t blocks = int64_t(p.B) * p.G * blocks_of(p);
    if (p.T <= TW) return 1;
    if (ws == 8) return 2;
    if (ws == 4) return blocks <= 256 ? 4 : 2;
    if (blocks <= 256 && p.T > 16 * TW && ssm_backward_words(p)) return 8;
    return ws == 1 || blocks <= 1024 ? 4 : 2;
}

template <typename Tin, typename Ty, int WS, bool VEC>
hipError_t launch_ws(const SsmParams& p, const BwdWs& ws, hipStream_t stream) {
    const dim3 grid{unsigned(int64_t(p.B) * p.G * blocks_of(p))};
    const int runs = runs_of(p);
    if (runs == 1) hipLaunchKernelGGL((ssm_backward_kernel<Tin, Ty, WS, 1, VEC>), grid, dim3(64 * WS), 0, stream, p, ws);
    if constexpr (WS >= 2)
        if (runs == 2) hipLaunchKernelGGL((ssm_backward_kernel<Tin, Ty, WS, 2, VEC>), grid, dim3(128 * WS), 0, stream, p, ws);
    if constexpr (WS <= 4)
        if (runs == 4) hipLaunchKernelGGL((ssm_backward_kernel<Tin, Ty, WS, 4, VEC>), grid, dim3(256 * WS), 0, stream, p, ws);
    if constexpr (WS <= 2 && VEC)
        if (runs == 8) hipLaunchKernelGGL((ssm_backward_kernel<Tin, Ty, WS, 8, VEC>), grid, dim3(512 * WS), 0, stream, p, ws);
    return hipGetLastError();
}
template <typename Tin, typename Ty, bool VEC>
hipError_t launch_vec(const SsmParams& p, const BwdWs& ws, hipStream_t stream) {
    switch (states_waves(p)) {
        case 1: return launch_ws<Tin, Ty, 1, VEC>(p, ws, stream);
        case 2: return launch_ws<Tin, Ty, 2, VEC>(p, ws, stream);
        case 4: return launch_ws<Tin, Ty, 4, VEC>(p, ws, stream);
        default: return launch_ws<Tin, Ty, 8, VEC>(p, ws, stream);
    }
}
template <typename Tin, typename Ty>
hipError_t launch_types(const SsmParams& p, const BwdWs& ws, hipStream_t stream) {
    return ssm_backward_words(p) ? launch_vec<Tin, Ty, true>(p, ws, stream) : launch_vec<Tin, Ty, false>(p, ws, stream);
}

}  // namespace

int64_t ssm_backward_workspace(const SsmParams& p, bool own_checkpoints) {
    if (int64_t(p.B) * p.T * p.C == 0) return 0;
    return bc_bytes(p) + par_bytes(p) + (own_checkpoints ? up(int64_t(p.B) * p.nck * p.C * p.N * 4) : 0);
}

int64_t ssm_backward_threads(const SsmParams& p) {
    if (p.C == 0) return 0;
    const int64_t own = int64_t(p.B) * p.G * blocks_of(p) * states_waves(p) * runs_of(p) * 64, sums = int64_t(p.B) * p.T * p.G * 2 * p.N * (p.N % 4 ? 4 : 1);
    const int64_t first = ssm_forward_threads(p), most = own > sums ? own : sums;
    return (most > first ? most : first) + 1024;
}

hipError_t launch_ssm_backward(const SsmParams& p, hipStream_t stream) {
    const int64_t Mp = int64_t(p.C) * p.N + 2 * p.C;
    const dim3 batch{unsigned((Mp + 255) / 256)};
    if (p.T == 0) {   // nothing to add up, and no workspace
        const int64_t n = p.ds0 ? int64_t(p.B) * p.C * p.N : 0, nb = (n + 255) / 256;
        if (n > 0) hipLaunchKernelGGL(ssm_no_tokens_kernel, dim3(unsigned(nb < 4096 ? nb : 4096)), dim3(256), 0, stream, p.ds1, p.ds0, n);
        SsmParams none = p;
        none.B = 0;
        if (Mp > 0) hipLaunchKernelGGL(ssm_sum_batch_kernel, batch, dim3(256), 0, stream, none, static_cast<const float*>(nullptr));
        return hipGetLastError();
    }
    char* at = static_cast<char*>(p.ws);
    BwdWs ws{reinterpret_cast<float*>(at), reinterpret_cast<float*>(at + bc_bytes(p)), p.ck};
    if (!p.ck && int64_t(p.B) * p.T * p.C > 0) {   // the states first
        SsmParams f = p;
        f.ck = reinterpret_cast<float*>(at + bc_bytes(p) + par_bytes(p));
        f.y = nullptr;
        f.s1 = nullptr;
        const hipError_t e = launch_ssm_forward(f, stream);
        if (e != hipSuccess) return e;
        ws.ck = f.ck;
    }
    if (int64_t(p.B) * p.C > 0) {
        const hipError_t e = p.in_bf16 ? p.y_bf16 ? launch_types<bf16_t, bf16_t>(p, ws, stream) : launch_types<bf16_t, float>(p, ws, stream)
                                       : p.y_bf16 ? launch_types<float, bf16_t>(p, ws, stream) : launch_types<float, float>(p, ws, stream);
        if (e != hipSuccess) return e;
    }
    // The sums; without channels or sequences, the zeros.
    const int ncb = blocks_of(p);
    const int64_t M = int64_t(p.B) * p.T * p.G * 2 * p.N;
    if (M > 0) {
        if (p.N % 4 == 0) hipLaunchKernelGGL((ssm_sum_bc_kernel<4>), dim3(unsigned((M / 4 + 63) / 64)), dim3(256), 0, stream, p, ws.bc, ncb);
        else hipLaunchKernelGGL((ssm_sum_bc_kernel<1>), dim3(unsigned((M + 63) / 64)), dim3(256), 0, stream, p, ws.bc, ncb);
    }
    if (Mp > 0) hipLaunchKernelGGL(ssm_sum_batch_kernel, batch, dim3(256), 0, stream, p, ws.par);
    return hipGetLastError();
}

}  // namespace wkv7
