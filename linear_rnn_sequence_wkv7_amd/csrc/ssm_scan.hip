// Selective state space scan on gfx950: prompts (ssm_forward) and single tokens
// (ssm_step).
//
//   d_t = softplus(dt_t + dt_bias),  h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,
//   y_t = (C_t . h_t + D x_t) silu(z_t)
//
// per batch and channel with N states.  The decay exp(d_t A[c][n]) has a factor
// for every channel and state, so the readout is no matrix product: the work is
// elementwise, a product, an exponential, the update and the readout per state.
//
// Lanes: LPC neighbouring lanes share a channel, each with NPL of its states in
// registers (LPC NPL >= N, unused states have A = B = C = 0), so a wave has
// 64 / LPC channels.  The WT waves of a workgroup have the same channels and
// consecutive runs of 16 tokens, which is how few channels still fill the chip:
// each wave first runs its tokens from a zero state, which gives its state H and,
// from the sum of its d_t, the factor P that an incoming state is multiplied by;
// the pairs (P, H) go through LDS, every wave composes those before it to its
// incoming state and all of them to the next round's, and runs its tokens again
// with the decays kept in registers.  One barrier a round; the pairs are double
// buffered.
//
// x, dt and z are loaded for the next round while this one computes, 4 lanes to a
// token's channels; step sizes and products d x are formed there, once per
// element, and change to the lanes' layout through LDS private to the wave, as
// do B and C and, on the way back, y (summed over the LPC lanes by a transposing
// butterfly that leaves each lane one token).  Everything is fp32 between the
// loads and the stores of y.
#include "seq_device.h"
#include "seq_internal.h"

namespace wkv7 {
namespace {

constexpr int TW = 16;   // tokens of one wave in a round
constexpr int TP = 20;   // LDS row of 16 tokens, padded

// Sum y[t] over the LPC lanes of a channel for LPC tokens; lane q keeps token q.
template <int LPC>
__device__ __forceinline__ float sum_transposed(float* y, int lane) {
    if constexpr (LPC >= 16) {
        const bool hi = lane & 8;
        #pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = (hi ? y[i + 8] : y[i]) + dpp<kDppRowMirror>(hi ? y[i] : y[i + 8]);
    }
    if constexpr (LPC >= 8) {
        const bool hi = lane & 4;
        #pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = (hi ? y[i + 4] : y[i]) + dpp<kDppRowHalfMirror>(hi ? y[i] : y[i + 4]);
    }
    if constexpr (LPC >= 4) {
        const bool hi = lane & 2;
        #pragma unroll
        for (int i = 0; i < 2; ++i) y[i] = (hi ? y[i + 2] : y[i]) + dpp<kDppQuadXor2>(hi ? y[i] : y[i + 2]);
    }
    const bool hi = lane & 1;
    return (hi ? y[1] : y[0]) + dpp<kDppQuadXor1>(hi ? y[0] : y[1]);
}

template <typename Tin, int LPC, int NPL, int WT>
__global__ __launch_bounds__(64 * WT) void ssm_scan_kernel(SsmParams g) {
    constexpr int CH = 64 / LPC, E = CH / 4, NP = LPC * NPL, BN = NP / 4;
    __shared__ float s_d[WT][CH][TP], s_u[WT][CH][TP];
    __shared__ float s_b[WT][TW][NP], s_c[WT][TW][NP];
    __shared__ float s_p[WT > 1 ? 2 : 1][WT][64 * NPL], s_h[WT > 1 ? 2 : 1][WT][64 * NPL];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    // The workgroup's sequence, group and channels.
    const int64_t item = xcd_order(blockIdx.x, gridDim.x);
    const int Cg = g.C / g.G, ncb = (Cg + CH - 1) / CH;
    const int cb = int(item % ncb), grp = int(item / ncb % g.G);
    const int64_t b = item / ncb / g.G;
    const int c0 = grp * Cg + cb * CH, nc = min(CH, Cg - cb * CH);   // first channel, channels there
    const int len = seq_length(g.lengths, b, g.T);

    // A lane's share of the states ...
    const int ch = lane / LPC, q = lane % LPC;
    const bool ch_in = ch < nc;
    float A2[NPL], h[NPL];
    const int64_t srow = (b * g.C + c0 + ch) * g.N + q * NPL;
    #pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const bool in = ch_in && q * NPL + i < g.N;
        A2[i] = in ? g.A[int64_t(c0 + ch) * g.N + q * NPL + i] * kLog2e : 0.f;
        h[i] = in && g.s0 ? g.s0[srow + i] : 0.f;
    }
    // ... and of the elements: token lane / 4, channels e0 .. e0 + E.
    const int te = lane >> 2, e0 = (lane & 3) * E, ne = nc - e0;
    const bool whole = g.vec_c && ne >= E, bwhole = g.vec_n;
    const int bn0 = (lane & 3) * BN, nb = g.N - bn0;
    float bias[E], Dv[E];
    #pragma unroll
    for (int i = 0; i < E; ++i) {
        bias[i] = g.dt_bias && i < ne ? g.dt_bias[c0 + e0 + i] : 0.f;
        Dv[i] = g.D && i < ne ? g.D[c0 + e0 + i] : 0.f;
    }
    const Tin *xp = static_cast<const Tin*>(g.x), *dtp = static_cast<const Tin*>(g.dt), *zp = static_cast<const Tin*>(g.z);
    const Tin *bp = static_cast<const Tin*>(g.Bm), *cp = static_cast<const Tin*>(g.Cm);

    Pack<Tin, E> x_n, dt_n, z_n;
    Pack<Tin, BN> b_n, c_n;
    auto load = [&](int t0) {
        const int64_t t = b * g.T + min(t0 + w * TW + te, g.T - 1);
        const int64_t e = t * g.C + c0 + e0;
        x_n = ld_pack<E>(xp + e, whole, ne);
        dt_n = ld_pack<E>(dtp + e, whole, ne);
        if (g.z) z_n = ld_pack<E>(zp + e, whole, ne);
        const int64_t r = (t * g.G + grp) * g.N + bn0;
        b_n = ld_pack<BN>(bp + r, bwhole, nb);
        c_n = ld_pack<BN>(cp + r, bwhole, nb);
    };
    if (len > 0) load(0);
    int par = 0;
    for (int t0 = 0; t0 < len; t0 += TW * WT) {
        const Pack<Tin, E> x_c = x_n, z_c = z_n;
        const int t = t0 + w * TW + te;
        const bool in = t < len;
        {   // elements into the wave's LDS; a padded token has d = 0 and B = 0: it leaves the state as it is
            #pragma unroll
            for (int i = 0; i < E; ++i) {
                float d = widen(dt_n.e[i]) + bias[i];
                if (g.softplus) d = softplusf_(d);
                d = in ? d : 0.f;
                s_d[w][e0 + i][te] = d;
                s_u[w][e0 + i][te] = in ? d * widen(x_c.e[i]) : 0.f;
            }
            #pragma unroll
            for (int i = 0; i < BN; ++i) {
                s_b[w][te][bn0 + i] = in ? widen(b_n.e[i]) : 0.f;
                s_c[w][te][bn0 + i] = widen(c_n.e[i]);
            }
        }
        if (t0 + TW * WT < len) load(t0 + TW * WT);
        wave_sync();

        float a[WT > 1 ? TW : 1][NPL];
        if constexpr (WT > 1) {
            float hl[NPL] = {}, ds = 0.f;
            #pragma unroll
            for (int t4 = 0; t4 < TW; t4 += 4) {
                const f32x4 d4 = *reinterpret_cast<const f32x4*>(&s_d[w][ch][t4]);
                const f32x4 u4 = *reinterpret_cast<const f32x4*>(&s_u[w][ch][t4]);
                #pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const Pack<float, NPL> Bv = *reinterpret_cast<const Pack<float, NPL>*>(&s_b[w][t4 + j][q * NPL]);
                    ds += d4[j];
                    #pragma unroll
                    for (int i = 0; i < NPL; ++i) {
                        a[t4 + j][i] = __builtin_amdgcn_exp2f(d4[j] * A2[i]);
                        hl[i] = fmaf(a[t4 + j][i], hl[i], u4[j] * Bv.e[i]);
                    }
                }
            }
            Pack<float, NPL> P, H;
            #pragma unroll
            for (int i = 0; i < NPL; ++i) {
                P.e[i] = __builtin_amdgcn_exp2f(ds * A2[i]);
                H.e[i] = hl[i];
            }
            *reinterpret_cast<Pack<float, NPL>*>(&s_p[par][w][lane * NPL]) = P;
            *reinterpret_cast<Pack<float, NPL>*>(&s_h[par][w][lane * NPL]) = H;
            __syncthreads();
            float hin[NPL];
            #pragma unroll
            for (int v = 0; v < WT; ++v) {
                if (v == w) {
                    #pragma unroll
                    for (int i = 0; i < NPL; ++i) hin[i] = h[i];
                }
                const Pack<float, NPL> Pv = *reinterpret_cast<const Pack<float, NPL>*>(&s_p[par][v][lane * NPL]);
                const Pack<float, NPL> Hv = *reinterpret_cast<const Pack<float, NPL>*>(&s_h[par][v][lane * NPL]);
                #pragma unroll
                for (int i = 0; i < NPL; ++i) h[i] = fmaf(Pv.e[i], h[i], Hv.e[i]);
            }
            par ^= 1;
            // h: the state after the round; hc: this wave's own
            float hc[NPL];
            #pragma unroll
            for (int i = 0; i < NPL; ++i) hc[i] = hin[i];
            const int tw = t0 + w * TW;
            if (g.ck && tw % SSM_CHECKPOINT_TOKENS == 0 && tw < g.T) {
                #pragma unroll
                for (int i = 0; i < NPL; ++i)
                    if (ch_in && q * NPL + i < g.N)
                        g.ck[((b * g.nck + tw / SSM_CHECKPOINT_TOKENS) * g.C + c0 + ch) * g.N + q * NPL + i] = hc[i];
            }
            #pragma unroll
            for (int tg = 0; tg < TW; tg += LPC) {
                float y[LPC];
                #pragma unroll
                for (int j = 0; j < LPC; ++j) {
                    const float u = s_u[w][ch][tg + j];
                    const Pack<float, NPL> Bv = *reinterpret_cast<const Pack<float, NPL>*>(&s_b[w][tg + j][q * NPL]);
                    const Pack<float, NPL> Cv = *reinterpret_cast<const Pack<float, NPL>*>(&s_c[w][tg + j][q * NPL]);
                    y[j] = 0.f;
                    #pragma unroll
                    for (int i = 0; i < NPL; ++i) {
                        hc[i] = fmaf(a[tg + j][i], hc[i], u * Bv.e[i]);
                        y[j] = fmaf(Cv.e[i], hc[i], y[j]);
                    }
                }
                s_d[w][ch][tg + q] = sum_transposed<LPC>(y, lane);
            }
        } else {
            if (g.ck && t0 % SSM_CHECKPOINT_TOKENS == 0) {
                #pragma unroll
                for (int i = 0; i < NPL; ++i)
                    if (ch_in && q * NPL + i < g.N)
                        g.ck[((b * g.nck + t0 / SSM_CHECKPOINT_TOKENS) * g.C + c0 + ch) * g.N + q * NPL + i] = h[i];
            }
            #pragma unroll
            for (int tg = 0; tg < TW; tg += LPC) {
                float y[LPC];
                #pragma unroll
                for (int j = 0; j < LPC; ++j) {
                    const float d = s_d[w][ch][tg + j], u = s_u[w][ch][tg + j];
                    const Pack<float, NPL> Bv = *reinterpret_cast<const Pack<float, NPL>*>(&s_b[w][tg + j][q * NPL]);
                    const Pack<float, NPL> Cv = *reinterpret_cast<const Pack<float, NPL>*>(&s_c[w][tg + j][q * NPL]);
                    y[j] = 0.f;
                    #pragma unroll
                    for (int i = 0; i < NPL; ++i) {
                        h[i] = fmaf(__builtin_amdgcn_exp2f(d * A2[i]), h[i], u * Bv.e[i]);
                        y[j] = fmaf(Cv.e[i], h[i], y[j]);
                    }
                }
                const float ys = sum_transposed<LPC>(y, lane);
                wave_sync();   // every lane has read these tokens' d
                s_d[w][ch][tg + q] = ys;
            }
        }
        wave_sync();
        float out[E];
        #pragma unroll
        for (int i = 0; i < E; ++i) {
            float y = fmaf(Dv[i], widen(x_c.e[i]), s_d[w][e0 + i][te]);
            if (g.z) {
                const float z = widen(z_c.e[i]);
                y *= z * sigmoidf_(z);
            }
            out[i] = in ? y : 0.f;
        }
        if (t < g.T && g.y) st_pack_as<E>(g.y, (b * g.T + t) * g.C + c0 + e0, g.y_bf16, out, whole, ne);
        wave_sync();   // the LDS rows are free again
    }
    // Padding after the last round: y = 0, and the state as it is at the checkpoints there.
    const int done = (len + TW * WT - 1) / (TW * WT) * (TW * WT);
    const float zero[E] = {};
    for (int t = done + w * TW + te; t < g.T && g.y; t += TW * WT)
        st_pack_as<E>(g.y, (b * g.T + t) * g.C + c0 + e0, g.y_bf16, zero, whole, ne);
    #pragma unroll
    for (int i = 0; i < NPL; ++i) {
        if (!ch_in || q * NPL + i >= g.N || w != 0) continue;
        if (g.ck)
            for (int k = (done + SSM_CHECKPOINT_TOKENS - 1) / SSM_CHECKPOINT_TOKENS; k < g.nck; ++k)
                g.ck[((b * g.nck + k) * g.C + c0 + ch) * g.N + q * NPL + i] = h[i];
        if (g.s1) g.s1[srow + i] = h[i];
    }
}

template <typename Tin, int LPC, int NPL>
hipError_t launch_scan_wt(const SsmParams& p, hipStream_t stream) {
    constexpr int CH = 64 / LPC;
    const int Cg = p.C / p.G;
    const int64_t blocks = int64_t(p.B) * p.G * ((Cg + CH - 1) / CH);
    const dim3 grid{unsigned(blocks)};
    // Waves over the tokens while the chip has room for them.
    const int wt = blocks >= 2048 || p.T <= TW ? 1 : blocks >= 512 || p.T <= 4 * TW ? 4 : 8;
    if (wt == 1) hipLaunchKernelGGL((ssm_scan_kernel<Tin, LPC, NPL, 1>), grid, dim3(64), 0, stream, p);
    else if (wt == 4) hipLaunchKernelGGL((ssm_scan_kernel<Tin, LPC, NPL, 4>), grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((ssm_scan_kernel<Tin, LPC, NPL, 8>), grid, dim3(512), 0, stream, p);
    return hipGetLastError();
}

template <typename Tin>
hipError_t launch_scan_in(SsmParams p, hipStream_t stream) {
    const int lpc = p.N <= 8 ? 2 : p.N <= 16 ? 4 : p.N <= 32 ? 8 : 16;
    const int E = 16 / lpc;
    p.vec_c = p.C % E == 0 && (p.C / p.G) % E == 0;
    p.vec_n = p.N == lpc * 4;
    switch (lpc) {
        case 2: return launch_scan_wt<Tin, 2, 4>(p, stream);
        case 4: return launch_scan_wt<Tin, 4, 4>(p, stream);
        case 8: return launch_scan_wt<Tin, 8, 4>(p, stream);
        default: return launch_scan_wt<Tin, 16, 4>(p, stream);
    }
}

// One token per row.  LN lanes to a channel, 4 states each: a wave's loads and
// stores of the states are 1 KiB runs.  A workgroup has 64 / LN channels of each
// of its 4 waves, and RB rows one after another (A stays in registers).
constexpr int SB = 256;

template <typename Tin, int LN>
__global__ __launch_bounds__(SB) void ssm_step_kernel(SsmParams g) {
    constexpr int CHB = SB / LN;
    const int ch = threadIdx.x / LN, q = threadIdx.x % LN;
    const int ncb = (g.C + CHB - 1) / CHB;
    const int64_t item = blockIdx.x;
    const int c = int(item % ncb) * CHB + ch;
    const int b = int(item / ncb);
    const bool in = c < g.C;
    const int n0 = q * 4, nn = in ? g.N - n0 : 0;
    const bool whole = g.vec_n && nn >= 4;
    const int slot = g.index ? g.index[b] : b;
    bool mine = slot >= 0 && slot < g.S;
    float hv[4] = {};
    const int64_t sr = (int64_t(slot) * g.C + c) * g.N + n0;
    if (mine && nn > 0) ld_pack_as<4>(g.s0, sr, false, hv, whole, nn);
    if (g.index && mine) mine = first_of_slot(g.index, b, slot, SB);
    const int64_t e = int64_t(b) * g.C + (in ? c : 0);
    const int grp = (in ? c : 0) / (g.C / g.G);
    const int64_t r = (int64_t(b) * g.G + grp) * g.N + n0;
    float Av[4], Bv[4], Cv[4];
    ld_pack_as<4>(g.A, int64_t(in ? c : 0) * g.N + n0, false, Av, whole, nn);
    ld_pack_as<4>(g.Bm, r, sizeof(Tin) == 2, Bv, whole, nn);
    ld_pack_as<4>(g.Cm, r, sizeof(Tin) == 2, Cv, whole, nn);
    const float x = widen(static_cast<const Tin*>(g.x)[e]);
    float d = widen(static_cast<const Tin*>(g.dt)[e]) + (g.dt_bias && in ? g.dt_bias[c] : 0.f);
    if (g.softplus) d = softplusf_(d);
    float y = 0.f;
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        hv[i] = fmaf(__builtin_amdgcn_exp2f(d * (Av[i] * kLog2e)), hv[i], d * x * Bv[i]);
        y = fmaf(Cv[i], hv[i], y);
    }
    if (mine && nn > 0) st_pack<4>(g.s1 + sr, hv, whole, nn);
    if constexpr (LN >= 2) y += dpp<kDppQuadXor1>(y);
    if constexpr (LN >= 4) y += dpp<kDppQuadXor2>(y);
    if constexpr (LN >= 8) y += dpp<kDppRowHalfMirror>(y);
    if constexpr (LN >= 16) y += dpp<kDppRowMirror>(y);
    if (!in || q != 0) return;
    if (g.D) y = fmaf(g.D[c], x, y);
    if (g.z) {
        const float z = widen(static_cast<const Tin*>(g.z)[e]);
        y *= z * sigmoidf_(z);
    }
    y = mine ? y : 0.f;
    st_pack_as<1>(g.y, e, g.y_bf16, &y, true, 1);
}

template <typename Tin>
hipError_t launch_step_in(SsmParams p, hipStream_t stream) {
    const int ln = p.N <= 4 ? 1 : p.N <= 8 ? 2 : p.N <= 16 ? 4 : p.N <= 32 ? 8 : 16;
    p.vec_n = p.N % 4 == 0;
    const int chb = SB / ln;
    const dim3 grid{unsigned(int64_t(p.B) * ((p.C + chb - 1) / chb))}, block{SB};
    switch (ln) {
        case 1: hipLaunchKernelGGL((ssm_step_kernel<Tin, 1>), grid, block, 0, stream, p); break;
        case 2: hipLaunchKernelGGL((ssm_step_kernel<Tin, 2>), grid, block, 0, stream, p); break;
        case 4: hipLaunchKernelGGL((ssm_step_kernel<Tin, 4>), grid, block, 0, stream, p); break;
        case 8: hipLaunchKernelGGL((ssm_step_kernel<Tin, 8>), grid, block, 0, stream, p); break;
        default: hipLaunchKernelGGL((ssm_step_kernel<Tin, 16>), grid, block, 0, stream, p); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ssm_forward(const SsmParams& p, hipStream_t stream) {
    return p.in_bf16 ? launch_scan_in<bf16_t>(p, stream) : launch_scan_in<float>(p, stream);
}

hipError_t launch_ssm_step(const SsmParams& p, hipStream_t stream) {
    return p.in_bf16 ? launch_step_in<bf16_t>(p, stream) : launch_step_in<float>(p, stream);
}

}  // namespace wkv7
