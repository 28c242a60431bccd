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
// The lanes are the forward's (ssm_scan.hip): LPC to a channel with NPL states
// each, the WT waves of a workgroup on consecutive runs of 16 tokens of the same
// channels.  The workgroup goes from its last 16 WT tokens to its first.  A round
// computes the decays of its tokens (kept in registers), each wave's state from
// zero and its gradient from zero, exchanges both and the wave's decay through
// LDS (one barrier, double buffered), so that every wave has its incoming state,
// starting from the checkpoint of the round, and its incoming gradient, starting
// from the later round's; runs the states forward once more, into registers, and
// then the gradients backward.
//
// Sums over a channel's lanes and over the channels of a wave are transposing
// butterflies: a step halves the values that a lane holds while it doubles the
// lanes summed.  dB and dC of a wave's channels go to the workspace, one row for
// each block of channels, and a second kernel adds the rows; no atomics, so the
// order is fixed.  dA, dD and ddt_bias are kept in registers over the whole
// sequence and added over the batch by a third kernel.
#include "seq_device.h"
#include "seq_internal.h"

namespace wkv7 {
namespace {

constexpr int TW = 16, TP = 20;
constexpr int PT = 4, PARTS = TW / PT;   // tokens whose states and decays are in registers at once
constexpr float kLn2 = 0.6931471805599453f;

// The value of lane ^ M.
template <int M>
__device__ __forceinline__ float from_xor(float x) {
    if constexpr (M == 1) return dpp<kDppQuadXor1>(x);
    if constexpr (M == 2) return dpp<kDppQuadXor2>(x);
    if constexpr (M == 8) return dpp<0x128>(x);   // row_ror:8
    // 4: down for the odd banks of four lanes, up for the even ones
    const int v = __float_as_int(x);
    const int t = __builtin_amdgcn_update_dpp(v, v, 0x114, 0xF, 0xA, false);   // row_shr:4
    return __int_as_float(__builtin_amdgcn_update_dpp(t, v, 0x104, 0xF, 0x5, false));   // row_shl:4
}
// lo where the lane's bit M is 0, hi where it is 1, each summed over the pair of lanes.
template <int M>
__device__ __forceinline__ float halve(float lo, float hi, int lane) {
    if constexpr (M == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(lo), __float_as_uint(hi), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    } else if constexpr (M == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(lo), __float_as_uint(hi), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    } else {
        const bool b = lane & M;
        return (b ? hi : lo) + from_xor<M>(b ? lo : hi);
    }
}
// Sum over a channel's lanes of 4 tokens, into LDS (row of the channel, from the first token).
template <int LPC>
__device__ __forceinline__ void sum_lanes_to(float* row, float* y, int lane) {
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (LPC >= 16) y[k] += dpp<kDppRowMirror>(y[k]);
        if constexpr (LPC >= 8) y[k] += dpp<kDppRowHalfMirror>(y[k]);
    }
    const float s = halve<1>(halve<2>(y[0], y[2], lane), halve<2>(y[1], y[3], lane), lane);
    if (lane % LPC < 4) row[lane & 3] = s;
}
// Values read from LDS are not to be kept in registers across this point: read them again.
__device__ __forceinline__ void forget_lds() { wave_sync(); }

struct BwdWs {
    float* bc;    // [ncb][B][T][G][2][N]: dB and dC of each block of channels
    float* par;   // [B][C N + 2 C]: dA, dD, ddt_bias of each sequence
    const float* ck;
};

template <typename Tin, int LPC, int NPL, int WT>
__global__ __launch_bounds__(64 * WT, 2) void ssm_backward_kernel(SsmParams g, BwdWs ws) {
    constexpr int CH = 64 / LPC, E = CH / 4, NP = LPC * NPL, BN = NP / 4, ROUND = TW * WT;
    constexpr int NV = 4 * 2 * NPL;   // values of dB and dC of 4 tokens in a lane
    __shared__ float s_d[WT][CH][TP], s_u[WT][CH][TP], s_o[WT][CH][TP];
    __shared__ float s_b[WT][TW][NP], s_c[WT][TW][NP];
    __shared__ float s_keep[WT][5][E][64];   // a lane's own x, d, softplus', do and dz factor, while it computes
    __shared__ float s_p[2][WT][64 * NPL], s_h[2][WT][64 * NPL], s_g[2][WT][64 * NPL];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t item = xcd_order(blockIdx.x, gridDim.x);
    const int Cg = g.C / g.G, ncb = (Cg + CH - 1) / CH;
    const int cb = int(item % ncb), grp = int(item / ncb % g.G);
    const int64_t b = item / ncb / g.G;
    const int c0 = grp * Cg + cb * CH, nc = min(CH, Cg - cb * CH);
    const int len = seq_length(g.lengths, b, g.T);

    const int ch = lane / LPC, q = lane % LPC;
    const bool ch_in = ch < nc;
    const int64_t srow = (b * g.C + c0 + ch) * g.N + q * NPL;
    float A2[NPL], gc[NPL], dA[NPL] = {};
    bool n_in[NPL];
    #pragma unroll
    for (int i = 0; i < NPL; ++i) {
        n_in[i] = ch_in && q * NPL + i < g.N;
        A2[i] = n_in[i] ? g.A[int64_t(c0 + ch) * g.N + q * NPL + i] * kLog2e : 0.f;
        gc[i] = n_in[i] && g.ds1 ? g.ds1[srow + i] : 0.f;   // gradient of the state after the round
    }
    const int te = lane >> 2, e0 = (lane & 3) * E, ne = nc - e0;
    const bool whole = g.vec_c && ne >= E;
    const int bn0 = (lane & 3) * BN, nb = g.N - bn0;
    float bias[E], Dv[E], dD[E] = {}, dbias[E] = {};
    #pragma unroll
    for (int i = 0; i < E; ++i) {
        bias[i] = g.dt_bias && i < ne ? g.dt_bias[c0 + e0 + i] : 0.f;
        Dv[i] = g.D && i < ne ? g.D[c0 + e0 + i] : 0.f;
    }
    const Tin *xp = static_cast<const Tin*>(g.x), *dtp = static_cast<const Tin*>(g.dt), *zp = static_cast<const Tin*>(g.z);
    const Tin *bp = static_cast<const Tin*>(g.Bm), *cp = static_cast<const Tin*>(g.Cm);
    auto store = [&](void* p, int64_t e, const float* v) { st_pack<E>(static_cast<Tin*>(p) + e, v, whole, ne); };

    const int rounds = (len + ROUND - 1) / ROUND;
    {   // padding after the last round
        const float zero[E] = {};
        for (int t = rounds * ROUND + w * TW + te; t < g.T; t += ROUND) {
            const int64_t e = (b * g.T + t) * g.C + c0 + e0;
            store(g.dx, e, zero);
            store(g.ddt, e, zero);
            if (g.z) store(g.dz, e, zero);
        }
    }
    int par = 0;
    for (int rd = rounds - 1; rd >= 0; --rd) {
        const int tw = rd * ROUND + w * TW, t = tw + te;
        const bool in = t < len;
        const int64_t row = b * g.T + min(t, g.T - 1), e = row * g.C + c0 + e0;
        float hin[NPL];
        {   // elements, and the round's checkpoint
            const Pack<Tin, E> xr = ld_pack<E>(xp + e, whole, ne), dr = ld_pack<E>(dtp + e, whole, ne);
            Pack<Tin, E> zr;
            if (g.z) zr = ld_pack<E>(zp + e, whole, ne);
            const int64_t r = (row * g.G + grp) * g.N + bn0;
            const Pack<Tin, BN> br = ld_pack<BN>(bp + r, g.vec_n, nb), cr = ld_pack<BN>(cp + r, g.vec_n, nb);
            float dyv[E];
            ld_pack_as<E>(g.dy, e, g.y_bf16, dyv, whole, ne);
            const float* ck = ws.ck + ((b * g.nck + rd * (ROUND < SSM_CHECKPOINT_TOKENS ? 1 : ROUND / SSM_CHECKPOINT_TOKENS)) * g.C + c0 + ch) * g.N + q * NPL;
            #pragma unroll
            for (int i = 0; i < NPL; ++i) hin[i] = n_in[i] ? ck[i] : 0.f;
            #pragma unroll
            for (int i = 0; i < E; ++i) {
                const float v = widen(dr.e[i]) + bias[i], x = in ? widen(xr.e[i]) : 0.f, dy = in ? dyv[i] : 0.f;
                const float d = in ? (g.softplus ? softplusf_(v) : v) : 0.f;
                float o = dy, dzf = 0.f;
                if (g.z) {
                    const float z = in ? widen(zr.e[i]) : 0.f, s = sigmoidf_(z);
                    o = dy * (z * s);
                    dzf = dy * s * fmaf(z, 1.f - s, 1.f);
                }
                s_d[w][e0 + i][te] = d;
                s_u[w][e0 + i][te] = d * x;
                s_o[w][e0 + i][te] = o;
                s_keep[w][0][i][lane] = x;
                s_keep[w][1][i][lane] = d;
                s_keep[w][2][i][lane] = in ? (g.softplus ? sigmoidf_(v) : 1.f) : 0.f;
                s_keep[w][3][i][lane] = o;
                s_keep[w][4][i][lane] = dzf;
            }
            #pragma unroll
            for (int i = 0; i < BN; ++i) {
                s_b[w][te][bn0 + i] = in ? widen(br.e[i]) : 0.f;
                s_c[w][te][bn0 + i] = in ? widen(cr.e[i]) : 0.f;
            }
        }
        wave_sync();
        auto Bv = [&](int tt) { return *reinterpret_cast<const Pack<float, NPL>*>(&s_b[w][tt][q * NPL]); };
        auto Cv = [&](int tt) { return *reinterpret_cast<const Pack<float, NPL>*>(&s_c[w][tt][q * NPL]); };

        // The state and the gradient that the wave's tokens give from zero, and their decay;
        // the state from zero and the decay up to each part of PT tokens.
        float Pm[PARTS - 1][NPL], Hm[PARTS - 1][NPL];
        {
            float hl[NPL] = {}, gl[NPL] = {}, pr[NPL];
            #pragma unroll
            for (int i = 0; i < NPL; ++i) pr[i] = 1.f;
            #pragma unroll
            for (int tt = 0; tt < (WT > 1 ? TW : TW - PT); ++tt) {
                if (tt % 4 == 0) forget_lds();
                if (tt % PT == 0 && tt > 0) {
                    #pragma unroll
                    for (int i = 0; i < NPL; ++i) {
                        Pm[tt / PT - 1][i] = pr[i];
                        Hm[tt / PT - 1][i] = hl[i];
                    }
                }
                const float dd = s_d[w][ch][tt], u = s_u[w][ch][tt], od = s_o[w][ch][tt];
                const Pack<float, NPL> B = Bv(tt), C = Cv(tt);
                #pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    const float at = __builtin_amdgcn_exp2f(dd * A2[i]);
                    hl[i] = fmaf(at, hl[i], u * B.e[i]);
                    pr[i] *= at;
                    if constexpr (WT > 1) gl[i] = fmaf(pr[i], C.e[i] * od, gl[i]);
                }
            }
            if constexpr (WT == 1) {
                #pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    Pm[PARTS - 2][i] = pr[i];
                    Hm[PARTS - 2][i] = hl[i];
                }
            }
            if constexpr (WT > 1) {
                Pack<float, NPL> P, H, Gl;
                #pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    P.e[i] = pr[i];
                    H.e[i] = hl[i];
                    Gl.e[i] = gl[i];
                }
                *reinterpret_cast<Pack<float, NPL>*>(&s_p[par][w][lane * NPL]) = P;
                *reinterpret_cast<Pack<float, NPL>*>(&s_h[par][w][lane * NPL]) = H;
                *reinterpret_cast<Pack<float, NPL>*>(&s_g[par][w][lane * NPL]) = Gl;
            }
        }
        float gi[NPL];   // gradient of the state after the wave's tokens
        if constexpr (WT > 1) {
            __syncthreads();
            #pragma unroll
            for (int v = 0; v < WT - 1; ++v) {
                if (v >= w) break;
                const Pack<float, NPL> P = *reinterpret_cast<const Pack<float, NPL>*>(&s_p[par][v][lane * NPL]);
                const Pack<float, NPL> H = *reinterpret_cast<const Pack<float, NPL>*>(&s_h[par][v][lane * NPL]);
                #pragma unroll
                for (int i = 0; i < NPL; ++i) hin[i] = fmaf(P.e[i], hin[i], H.e[i]);
            }
            #pragma unroll
            for (int v = WT - 1; v >= 0; --v) {
                if (v == w) {
                    #pragma unroll
                    for (int i = 0; i < NPL; ++i) gi[i] = gc[i];
                }
                const Pack<float, NPL> P = *reinterpret_cast<const Pack<float, NPL>*>(&s_p[par][v][lane * NPL]);
                const Pack<float, NPL> Gl = *reinterpret_cast<const Pack<float, NPL>*>(&s_g[par][v][lane * NPL]);
                #pragma unroll
                for (int i = 0; i < NPL; ++i) gc[i] = fmaf(P.e[i], gc[i], Gl.e[i]);
            }
            par ^= 1;
        } else {
            #pragma unroll
            for (int i = 0; i < NPL; ++i) gi[i] = gc[i];
        }
        // Part by part from the last: the part's states, then its gradients.
        float dAr[NPL] = {};
        #pragma unroll
        for (int t8 = TW - PT; t8 >= 0; t8 -= PT) {
        float a[PT][NPL], h[PT][NPL], hb[NPL];   // hb: the state before the part
        #pragma unroll
        for (int i = 0; i < NPL; ++i)
            hb[i] = t8 ? fmaf(Pm[t8 ? t8 / PT - 1 : 0][i], hin[i], Hm[t8 ? t8 / PT - 1 : 0][i]) : hin[i];
        #pragma unroll
        for (int tt = 0; tt < PT; ++tt) {
            if (tt % 4 == 0) forget_lds();
            const float dd = s_d[w][ch][t8 + tt], u = s_u[w][ch][t8 + tt];
            const Pack<float, NPL> B = Bv(t8 + tt);
            #pragma unroll
            for (int i = 0; i < NPL; ++i) {
                a[tt][i] = __builtin_amdgcn_exp2f(dd * A2[i]);
                h[tt][i] = fmaf(a[tt][i], tt ? h[tt ? tt - 1 : 0][i] : hb[i], u * B.e[i]);
            }
        }
        // Backward, in groups of 4 tokens.
        #pragma unroll
        for (int tg = t8 + PT - 4; tg >= t8; tg -= 4) {
            forget_lds();
            float ys[4], us[4], ds[4], bc[NV];
            #pragma unroll
            for (int k = 3; k >= 0; --k) {
                const int tt = tg + k;
                const float dd = s_d[w][ch][tt], u = s_u[w][ch][tt], od = s_o[w][ch][tt];
                const Pack<float, NPL> B = Bv(tt), C = Cv(tt);
                ys[k] = us[k] = ds[k] = 0.f;
                #pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    const float et = fmaf(C.e[i], od, gi[i]);
                    gi[i] = a[tt - t8][i] * et;
                    const float qt = gi[i] * (tt > t8 ? h[tt > t8 ? tt - t8 - 1 : 0][i] : hb[i]);
                    ys[k] = fmaf(C.e[i], h[tt - t8][i], ys[k]);
                    us[k] = fmaf(et, B.e[i], us[k]);
                    ds[k] = fmaf(qt, A2[i], ds[k]);
                    dAr[i] = fmaf(qt, dd, dAr[i]);
                    bc[k * 2 * NPL + i] = et * u;
                    bc[k * 2 * NPL + NPL + i] = h[tt - t8][i] * od;
                }
            }
            // over the channels: the values are (token, dB or dC, state), the highest index bit first
            #pragma unroll
            for (int v = 0; v < NV / 2; ++v) bc[v] = halve<32>(bc[v], bc[v + NV / 2], lane);
            #pragma unroll
            for (int v = 0; v < NV / 4; ++v) bc[v] = halve<16>(bc[v], bc[v + NV / 4], lane);
            if constexpr (LPC <= 8) {
                #pragma unroll
                for (int v = 0; v < NV / 8; ++v) bc[v] = halve<8>(bc[v], bc[v + NV / 8], lane);
            }
            if constexpr (LPC <= 4) {
                #pragma unroll
                for (int v = 0; v < NV / 16; ++v) bc[v] = halve<4>(bc[v], bc[v + NV / 16], lane);
            }
            constexpr int LEFT = NV / CH;   // values that stay with a lane
            const int tt = tw + tg + (lane >> 4), v0 = (lane & 15) / LPC * LEFT;
            if (tt < len) {
                float* p = ws.bc + (((int64_t(cb) * g.B + b) * g.T + tt) * g.G + grp) * 2 * g.N;
                #pragma unroll
                for (int v = 0; v < LEFT; ++v) {
                    const int n = q * NPL + (v0 + v) % NPL;
                    if (n < g.N) p[(v0 + v) / NPL * g.N + n] = bc[v];
                }
            }
            // over the channel's lanes; these tokens' d, u and o have been read
            sum_lanes_to<LPC>(&s_d[w][ch][tg], ys, lane);
            sum_lanes_to<LPC>(&s_u[w][ch][tg], us, lane);
            sum_lanes_to<LPC>(&s_o[w][ch][tg], ds, lane);
        }
        }
        #pragma unroll
        for (int i = 0; i < NPL; ++i) {
            dA[i] += dAr[i];
            if constexpr (WT == 1) gc[i] = gi[i];
        }
        wave_sync();
        float dx[E], ddt[E], dz[E];
        #pragma unroll
        for (int i = 0; i < E; ++i) {
            const float x = s_keep[w][0][i][lane], d = s_keep[w][1][i][lane], o = s_keep[w][3][i][lane];
            const float y = fmaf(Dv[i], x, s_d[w][e0 + i][te]), du = s_u[w][e0 + i][te];
            const float dd = fmaf(du, x, s_o[w][e0 + i][te] * kLn2);
            dx[i] = fmaf(du, d, o * Dv[i]);
            ddt[i] = in ? dd * s_keep[w][2][i][lane] : 0.f;
            dz[i] = s_keep[w][4][i][lane] * y;
            dD[i] = fmaf(o, x, dD[i]);
            dbias[i] += ddt[i];
        }
        if (t < g.T) {
            store(g.dx, e, dx);
            store(g.ddt, e, ddt);
            if (g.z) store(g.dz, e, dz);
        }
        wave_sync();   // the LDS rows are free again
    }
    #pragma unroll
    for (int i = 0; i < NPL; ++i)
        if (g.ds0 && n_in[i] && w == 0) g.ds0[srow + i] = gc[i];

    // The parameters' gradients of this sequence: over the lanes of the same channels, then over the waves.
    #pragma unroll
    for (int i = 0; i < E; ++i) {
        #pragma unroll
        for (int m = 4; m < 64; m *= 2) {
            dD[i] += __shfl_xor(dD[i], m);
            dbias[i] += __shfl_xor(dbias[i], m);
        }
    }
    __syncthreads();
    #pragma unroll
    for (int i = 0; i < NPL; ++i) s_p[0][w][lane * NPL + i] = dA[i];
    if (te == 0) {
        #pragma unroll
        for (int i = 0; i < E; ++i) {
            s_d[w][e0 + i][0] = dD[i];
            s_d[w][e0 + i][1] = dbias[i];
        }
    }
    __syncthreads();
    if (w != 0) return;
    float* out = ws.par + b * (int64_t(g.C) * g.N + 2 * g.C);
    #pragma unroll
    for (int i = 0; i < NPL; ++i) {
        float s = 0.f;
        #pragma unroll
        for (int v = 0; v < WT; ++v) s += s_p[0][v][lane * NPL + i];
        if (n_in[i]) out[int64_t(c0 + ch) * g.N + q * NPL + i] = s;
    }
    if (lane < 2 * CH && lane / 2 < nc) {
        float s = 0.f;
        #pragma unroll
        for (int v = 0; v < WT; ++v) s += s_d[v][lane / 2][lane & 1];
        out[int64_t(g.C) * g.N + (lane & 1) * g.C + c0 + lane / 2] = s;
    }
}

// dBm and dCm: the sums over the blocks of channels.
__global__ __launch_bounds__(256) void ssm_sum_bc_kernel(SsmParams g, const float* bc, int ncb) {
    const int64_t M = int64_t(g.B) * g.T * g.G * 2 * g.N;
    const int64_t m = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (m >= M) return;
    const int n = int(m % g.N), kind = int(m / g.N % 2);
    const int64_t bt = m / (2 * g.N), row = bt / g.G, b = row / g.T;
    float s = 0.f;
    if (row - b * g.T < seq_length(g.lengths, b, g.T))
        for (int i = 0; i < ncb; ++i) s += bc[i * M + m];
    st_pack_as<1>(kind ? g.dCm : g.dBm, bt * g.N + n, g.in_bf16, &s, true, 1);
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

int lanes_of(int N) { return N <= 16 ? 4 : N <= 32 ? 8 : 16; }
int blocks_of(const SsmParams& p) {
    const int CH = 64 / lanes_of(p.N);
    return (p.C / p.G + CH - 1) / CH;
}
int64_t up(int64_t x) { return (x + 255) & ~int64_t(255); }
int64_t bc_bytes(const SsmParams& p) { return up(int64_t(blocks_of(p)) * p.B * p.T * p.G * 2 * p.N * 4); }
int64_t par_bytes(const SsmParams& p) { return up(int64_t(p.B) * (int64_t(p.C) * p.N + 2 * p.C) * 4); }

template <typename Tin, int LPC, int NPL>
hipError_t launch_lpc(SsmParams p, const BwdWs& ws, hipStream_t stream) {
    constexpr int E = 16 / LPC;
    p.vec_c = p.C % E == 0 && (p.C / p.G) % E == 0;
    p.vec_n = p.N == LPC * NPL;
    const int ncb = blocks_of(p);
    const dim3 grid{unsigned(int64_t(p.B) * p.G * ncb)};
    if (grid.x == 0) {   // no channels or no sequences: only zeros to write
    } else if (p.T <= TW) hipLaunchKernelGGL((ssm_backward_kernel<Tin, LPC, NPL, 1>), grid, dim3(64), 0, stream, p, ws);
    else hipLaunchKernelGGL((ssm_backward_kernel<Tin, LPC, NPL, 4>), grid, dim3(256), 0, stream, p, ws);
    const int64_t M = int64_t(p.B) * p.T * p.G * 2 * p.N, Mp = int64_t(p.C) * p.N + 2 * p.C;
    if (M > 0)
        hipLaunchKernelGGL(ssm_sum_bc_kernel, dim3(unsigned((M + 255) / 256)), dim3(256), 0, stream, p, ws.bc, ncb);
    if (Mp > 0) hipLaunchKernelGGL(ssm_sum_batch_kernel, dim3(unsigned((Mp + 255) / 256)), dim3(256), 0, stream, p, ws.par);
    return hipGetLastError();
}
template <typename Tin>
hipError_t launch_in(const SsmParams& p, const BwdWs& ws, hipStream_t stream) {
    if (p.N <= 8) return launch_lpc<Tin, 4, 2>(p, ws, stream);
    switch (lanes_of(p.N)) {
        case 4: return launch_lpc<Tin, 4, 4>(p, ws, stream);
        case 8: return launch_lpc<Tin, 8, 4>(p, ws, stream);
        default: return launch_lpc<Tin, 16, 4>(p, ws, stream);
    }
}

}  // namespace

int64_t ssm_backward_workspace(const SsmParams& p, bool own_checkpoints) {
    if (int64_t(p.B) * p.C == 0) return 0;
    return bc_bytes(p) + par_bytes(p) + (own_checkpoints ? up(int64_t(p.B) * p.nck * p.C * p.N * 4) : 0);
}

hipError_t launch_ssm_backward(const SsmParams& p, hipStream_t stream) {
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
    return p.in_bf16 ? launch_in<bf16_t>(p, ws, stream) : launch_in<float>(p, ws, stream);
}

}  // namespace wkv7
