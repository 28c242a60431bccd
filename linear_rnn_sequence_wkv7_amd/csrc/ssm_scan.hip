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
// Lanes: a wave has 16 channels; lane (q, c) of its 4 rows of 16 lanes has NPL
// states of channel c in registers, q NPL and on (4 NPL >= N, unused states have
// A = B = C = 0).  B and C of 16 tokens lie across a row, token t in lane t, and an
// operand modifier hands lane t's to the whole row when token t comes: no LDS
// traffic and no extra instruction, which is why a row has 16 channels and not
// some states of fewer.  The readout is left in four parts, one a row, that are
// added where y is written.
//
// Tokens: the WT waves of a workgroup have the same channels and consecutive runs
// of 16 tokens, which is how few channels still fill the chip: each wave first runs
// its tokens from a zero state, which gives its state H and, from the sum of its
// d_t, the factor P that an incoming state is multiplied by; the pairs (P, H) go
// through LDS, every wave composes those before it to its incoming state and all of
// them to the next round's, and runs its tokens again with the decays kept in
// registers.  One barrier a round; the pairs are double buffered.  That is one more
// update per state and token than WT = 1 does, which is taken as soon as its waves
// fill the chip.
//
// x, dt, z, B and C are loaded a round ahead as raw words (a conversion would wait
// for them), 4 lanes to a token's channels, through descriptors that end with the
// sequence, so that padding reads as zeros without a branch; step sizes and products
// d x are formed there, once per element, and change to the lanes' layout through LDS
// private to the wave, as y does on the way back.  Everything is fp32 between the
// loads and the stores of y.
//
// Bound: the vector units.  A state and token needs a multiplication and an
// exponential for its decay, a product, an update and a readout (two updates where
// WT > 1); an exponential takes the time of two of the others and a half.  Measured at
// N = 16, G = 1, bf16: 8 x 4096 tokens x 4096 channels 625 us (vector units 81% busy, 8.3
// instructions a state and token; 1.7 TB/s), 1 x 2048 x 4096 54 us (67% busy: a round's
// barrier and LDS traffic stand open with two waves to a SIMD).  Tried and left: 2 states a
// lane and twice the waves (786 and 72 us: the elements and barriers count twice), the
// next round's elements formed between this one's updates (no faster).
#include "seq_device.h"
#include "seq_internal.h"

namespace wkv7 {
namespace {

constexpr int TW = 16;   // tokens of one wave in a round
constexpr int CH = 16;   // channels of a wave
constexpr int E = 4;     // channels of a lane where it loads and stores elements
constexpr int TP = 20;   // LDS row of 16 tokens, padded

// VEC: every row of channels (of the inputs and of y) and of states starts on 4 bytes, for each group
// too, and no lane has only some of its NPL states.
template <typename Tin, int NPL, int WT, bool VEC>
__global__ __launch_bounds__(64 * WT) void ssm_scan_kernel(SsmParams g) {
    constexpr int ROUND = TW * WT, ES = int(sizeof(Tin));
    // Step sizes, products and the rows' parts of y; where a wave's decays stay in its registers y takes
    // the place of the others.
    constexpr int Y0 = WT > 1 ? 0 : 2;
    __shared__ float s_e[WT][Y0 + 4][CH][TP];
    __shared__ Pack<float, NPL> s_p[WT > 1 ? 2 : 1][WT][64], s_h[WT > 1 ? 2 : 1][WT][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    // The workgroup's sequence, group and channels.
    const unsigned item = unsigned(xcd_order(blockIdx.x, gridDim.x));
    const int Cg = g.C / g.G;
    const unsigned ncb = (Cg + CH - 1) / CH;
    const int cb = int(item % ncb), grp = int(item / ncb % g.G);
    const int64_t b = item / ncb / g.G;
    const int c0 = grp * Cg + cb * CH, nc = min(CH, Cg - cb * CH);   // first channel, channels there
    const int len = __builtin_amdgcn_readfirstlane(seq_length(g.lengths, b, g.T));

    // A lane's share of the states: channel ch, states n0 .. n0 + NPL ...
    const int ch = lane & 15, q = lane >> 4, n0 = q * NPL;
    const bool ch_in = ch < nc;
    float A2[NPL], h[NPL];
    const int64_t srow = (b * g.C + c0 + ch) * g.N + n0;
    #pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const bool in = ch_in && n0 + i < g.N;
        A2[i] = in ? g.A[int64_t(c0 + ch) * g.N + n0 + i] * kLog2e : 0.f;
        h[i] = in && g.s0 ? g.s0[srow + i] : 0.f;
    }
    // ... of the elements: token te, channels e0 .. e0 + E; and of B and C: token ch, states n0 .. n0 + NPL.
    // What a lane makes of channels that are not there no other lane sees.
    const int te = lane >> 2, e0 = (lane & 3) * E, ne = nc - e0;
    float bias[E], Dv[E];
    #pragma unroll
    for (int i = 0; i < E; ++i) {
        bias[i] = g.dt_bias && i < ne ? g.dt_bias[c0 + e0 + i] : 0.f;
        Dv[i] = g.D && i < ne ? g.D[c0 + e0 + i] : 0.f;
    }

    // Rows of a round through descriptors that end with the sequence, at offsets that stay the same:
    // a padded token's x, z, B and C are 0.
    const uint32_t eoff = uint32_t((w * TW + te) * g.C + c0 + e0);
    const uint32_t voff = n0 < g.N ? uint32_t((w * TW + ch) * g.G * g.N + grp * g.N + n0) * ES : kNowhere;
    const int64_t erow = int64_t(g.C) * ES, vrow = int64_t(g.G) * g.N * ES, yrow = int64_t(g.C) * (g.y_bf16 ? 2 : 4);
    const char *xp = static_cast<const char*>(g.x) + b * g.T * erow, *dtp = static_cast<const char*>(g.dt) + b * g.T * erow;
    const char *zp = g.z ? static_cast<const char*>(g.z) + b * g.T * erow : xp;
    const char *bp = static_cast<const char*>(g.Bm) + b * g.T * vrow, *cp = static_cast<const char*>(g.Cm) + b * g.T * vrow;
    char* yp = static_cast<char*>(g.y) + b * g.T * yrow;
    const int zkeep = g.z ? -1 : 0, ykeep = g.y ? -1 : 0;
    struct Inputs {
        Raw<Tin, E, VEC> x, dt, z;
        Raw<Tin, NPL, VEC> b, c;
    } nx;
    int left = len;   // tokens from the next load on
    auto load = [&]() {
        const int n = max(0, min(left, ROUND)), eb = n * int(erow), vb = n * int(vrow);
        nx.dt.load(buf_rsrc(dtp, eb), eoff * ES, ne);
        nx.x.load(buf_rsrc(xp, eb), eoff * ES, ne);
        nx.b.load(buf_rsrc(bp, vb), voff, g.N - n0);
        nx.c.load(buf_rsrc(cp, vb), voff, g.N - n0);
        nx.z.load(buf_rsrc(zp, eb & zkeep), eoff * ES, ne);
        dtp += ROUND * erow;
        xp += ROUND * erow;
        zp += ROUND * erow;
        bp += ROUND * vrow;
        cp += ROUND * vrow;
        left -= ROUND;
    };
    auto store_y = [&](int t0, int end, const float* v) {   // of the tokens before `end`
        const rsrc_t r = buf_rsrc(yp + t0 * yrow, (t0 < 0 ? 0 : max(0, min(end - t0, ROUND)) * int(yrow)) & ykeep);
        if (g.y_bf16) buf_store<bf16_t, E, VEC>(r, eoff * 2, v, ne);
        else buf_store<float, E, true>(r, eoff * 4, v, ne);
    };
    auto checkpoint = [&](int t, const float* v) {
        #pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (ch_in && n0 + i < g.N) g.ck[((b * g.nck + t / SSM_CHECKPOINT_TOKENS) * g.C + c0 + ch) * g.N + n0 + i] = v[i];
    };
    // Step sizes and products d x of a round into LDS; a padded token has d = 0: it leaves the state as it is.
    const uint32_t soft = g.softplus ? ~0u : 0u;
    const float no_z = g.z ? 0.f : 1.f;   // the gate's factor without z
    auto stage = [&](int t0) {
        const bool in = t0 + w * TW + te < len;
        const uint32_t keep = in ? ~0u : 0u;
        #pragma unroll
        for (int i = 0; i < E; ++i) {
            const float v = nx.dt.get(i) + bias[i];
            const float d = __uint_as_float(__float_as_uint(bit_select(soft, softplusf_(v), v)) & keep);
            s_e[w][0][e0 + i][te] = d;
            s_e[w][1][e0 + i][te] = d * nx.x.get(i);
        }
    };
    // y of a round, from the rows' parts in LDS.
    auto x_p = nx.x, z_p = nx.z;
    auto output = [&](int t0) {
        float out[E];
        #pragma unroll
        for (int i = 0; i < E; ++i) {
            const float y = fmaf(Dv[i], x_p.get(i), (s_e[w][Y0][e0 + i][te] + s_e[w][Y0 + 1][e0 + i][te]) + (s_e[w][Y0 + 2][e0 + i][te] + s_e[w][Y0 + 3][e0 + i][te]));
            const float z = z_p.get(i);
            out[i] = y * fmaf(z, sigmoidf_(z), no_z);
        }
        store_y(t0, len, out);
    };
    load();
    int par = 0;
    for (int t0 = 0; t0 < len; t0 += ROUND) {
        const auto x_c = nx.x, z_c = nx.z;
        const int tw = t0 + w * TW;
        stage(t0);
        float Bv[NPL], Cv[NPL];
        #pragma unroll
        for (int i = 0; i < NPL; ++i) {
            Bv[i] = nx.b.get(i);
            Cv[i] = nx.c.get(i);
        }
        load();
        // With a wave to itself the round before is finished here, while LDS turns this one's elements
        // round (8 x 4096 x 4096 bf16: 700 -> 664 us; with more waves it is no faster).
        if constexpr (WT == 1) output(t0 - ROUND);
        wave_sync();

        // The wave's tokens from a state: decay(token, state, d) and input(token, state, u).
        auto run = [&](float* hs, auto&& decay, auto&& input) {
            static_for<TW / 4>([&](auto t4) {
                f32x4 d4, u4, y;
                float hh[4][NPL];
                if constexpr (WT == 1) {
                    d4 = *reinterpret_cast<const f32x4*>(&s_e[w][0][ch][t4 * 4]);
                    u4 = *reinterpret_cast<const f32x4*>(&s_e[w][1][ch][t4 * 4]);
                }
                static_for<4>([&](auto j_) {
                    constexpr int j = j_, tt = t4 * 4 + j;
                    #pragma unroll
                    for (int i = 0; i < NPL; ++i) {
                        hh[j][i] = fmaf(decay(tt, i, d4[j]), hs[i], input(j_, t4, i, u4[j]));
                        hs[i] = hh[j][i];
                    }
                });
                row_dot4<t4 * 4, NPL>(Cv, hh, y);
                *reinterpret_cast<f32x4*>(&s_e[w][Y0 + q][ch][t4 * 4]) = y;
            });
        };
        if constexpr (WT > 1) {
            float a[TW][NPL], in_[TW][NPL], hl[NPL] = {}, ds = 0.f;
            static_for<TW / 4>([&](auto t4) {
                const f32x4 d4 = *reinterpret_cast<const f32x4*>(&s_e[w][0][ch][t4 * 4]);
                const f32x4 u4 = *reinterpret_cast<const f32x4*>(&s_e[w][1][ch][t4 * 4]);
                static_for<4>([&](auto j_) {
                    constexpr int j = j_, tt = t4 * 4 + j;
                    ds += d4[j];
                    #pragma unroll
                    for (int i = 0; i < NPL; ++i) {
                        a[tt][i] = __builtin_amdgcn_exp2f(d4[j] * A2[i]);
                        in_[tt][i] = u4[j] * row_lane<tt>(Bv[i]);
                        hl[i] = fmaf(a[tt][i], hl[i], in_[tt][i]);
                    }
                });
            });
            Pack<float, NPL> P, H;
            #pragma unroll
            for (int i = 0; i < NPL; ++i) {
                P.e[i] = __builtin_amdgcn_exp2f(ds * A2[i]);
                H.e[i] = hl[i];
            }
            s_p[par][w][lane] = P;
            s_h[par][w][lane] = H;
            __syncthreads();
            float hc[NPL];   // the state before this wave's tokens; h goes on to the state after the round
            #pragma unroll
            for (int v = 0; v < WT; ++v) {
                if (v == w) {
                    #pragma unroll
                    for (int i = 0; i < NPL; ++i) hc[i] = h[i];
                }
                const Pack<float, NPL> P = s_p[par][v][lane], H = s_h[par][v][lane];
                #pragma unroll
                for (int i = 0; i < NPL; ++i) h[i] = fmaf(P.e[i], h[i], H.e[i]);
            }
            if (g.ck && tw % SSM_CHECKPOINT_TOKENS == 0 && tw < g.T) checkpoint(tw, hc);
            run(hc, [&](int tt, int i, float) { return a[tt][i]; }, [&](auto j, auto t4, int i, float) { return in_[t4 * 4 + j][i]; });
        } else {
            if (g.ck && t0 % SSM_CHECKPOINT_TOKENS == 0) checkpoint(t0, h);
            run(h, [&](int, int i, float dd) { return __builtin_amdgcn_exp2f(dd * A2[i]); },
                [&](auto j, auto t4, int i, float uu) { return uu * row_lane<t4 * 4 + j>(Bv[i]); });
        }
        par ^= 1;
        x_p = x_c;
        z_p = z_c;
        wave_sync();
        if constexpr (WT > 1) {
            output(t0);
            wave_sync();
        }
    }
    if (WT == 1 && len > 0) output((len + ROUND - 1) / ROUND * ROUND - ROUND);
    // Padding: y = 0, also where the state is no number, and after the last round the state as it is at the
    // checkpoints there.
    const int done = (len + ROUND - 1) / ROUND * ROUND;
    const float zero[E] = {};
    for (int t0 = len; t0 < g.T; t0 += ROUND) store_y(t0, g.T, zero);
    if (w != 0) return;
    if (g.ck)
        for (int k = (done + SSM_CHECKPOINT_TOKENS - 1) / SSM_CHECKPOINT_TOKENS; k < g.nck; ++k)
            checkpoint(k * SSM_CHECKPOINT_TOKENS, h);
    if (g.s1) {
        #pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (ch_in && n0 + i < g.N) g.s1[srow + i] = h[i];
    }
}

int64_t scan_blocks(const SsmParams& p) { return int64_t(p.B) * p.G * ((p.C / p.G + CH - 1) / CH); }
// Waves over the tokens while the chip has room for them: 8 while each workgroup has a compute unit
// to itself, 1 from two waves for every SIMD on.  1024 tokens, N = 16, bf16, us with 1, 4, 8 waves: 256
// workgroups 112, 41, 32; 320: 120, 56, 58; 1024: 118, 102, 110; 2048: 161, 192, 217.  More than 16 states
// are 8 or 16 of a lane, and the decays and inputs of 16 tokens that several waves keep for their second run
// would be 256 registers or more: always one wave, however few channels (1 x 2048 x 4096 with N = 16, 32, 64:
// 60, 301, 500 us; 8 x 4096 x 4096 with 16, 32: 624, 988).
int scan_waves(const SsmParams& p) {
    const int64_t blocks = scan_blocks(p);
    return p.N > 16 || blocks >= 2048 || p.T <= TW ? 1 : blocks > 256 || p.T <= 4 * TW ? 4 : 8;
}

template <typename Tin, int NPL, bool VEC>
hipError_t launch_scan_wt(const SsmParams& p, hipStream_t stream) {
    const dim3 grid{unsigned(scan_blocks(p))};
    const int wt = scan_waves(p);
    if (wt == 1) hipLaunchKernelGGL((ssm_scan_kernel<Tin, NPL, 1, VEC>), grid, dim3(64), 0, stream, p);
    else if constexpr (NPL <= 4) {
        if (wt == 4) hipLaunchKernelGGL((ssm_scan_kernel<Tin, NPL, 4, VEC>), grid, dim3(256), 0, stream, p);
        else hipLaunchKernelGGL((ssm_scan_kernel<Tin, NPL, 8, VEC>), grid, dim3(512), 0, stream, p);
    }
    return hipGetLastError();
}
template <typename Tin, int NPL>
hipError_t launch_scan_n(const SsmParams& p, hipStream_t stream) {
    return ssm_forward_words(p, NPL) ? launch_scan_wt<Tin, NPL, true>(p, stream) : launch_scan_wt<Tin, NPL, false>(p, stream);
}

template <typename Tin>
hipError_t launch_scan_in(const SsmParams& p, hipStream_t stream) {
    if (p.N <= 4) return launch_scan_n<Tin, 1>(p, stream);
    if (p.N <= 8) return launch_scan_n<Tin, 2>(p, stream);
    if (p.N <= 16) return launch_scan_n<Tin, 4>(p, stream);
    if (p.N <= 32) return launch_scan_n<Tin, 8>(p, stream);
    return launch_scan_n<Tin, 16>(p, stream);
}

// One token per row.  LN lanes to a channel, 4 states each: a wave's loads and
// stores of the states are 1 KiB runs.  A workgroup has 256 / LN channels of R
// rows, whose states are in flight together; A is loaded once for them.
// Bound: memory, each state read and written once; 256 rows x 4096 channels of 16 states
// in bf16 33 us, 4.3 TB/s, one row x 2048 4 us.
constexpr int SB = 256;

template <typename Tin, int LN, int R>
__global__ __launch_bounds__(SB) void ssm_step_kernel(SsmParams g) {
    constexpr int CHB = SB / LN;
    const int q = threadIdx.x % LN;
    const int ncb = (g.C + CHB - 1) / CHB;
    const int c = int(blockIdx.x % ncb) * CHB + threadIdx.x / LN, b0 = int(blockIdx.x / ncb) * R;
    const bool in = c < g.C;
    const int cc = in ? c : 0, grp = cc / (g.C / g.G);
    const int n0 = q * 4, nn = in ? g.N - n0 : 0;
    const bool whole = g.vec_n && nn >= 4;
    int slot[R];
    bool mine[R];
    float hv[R][4] = {}, Bv[R][4], Cv[R][4], x[R], d[R], z[R], Av[4];
    #pragma unroll
    for (int r = 0; r < R; ++r) {
        const int b = min(b0 + r, g.B - 1);
        slot[r] = g.index ? g.index[b] : b;
        mine[r] = b0 + r < g.B && slot[r] >= 0 && slot[r] < g.S;
        if (mine[r] && nn > 0) ld_pack_as<4>(g.s0, (int64_t(slot[r]) * g.C + c) * g.N + n0, false, hv[r], whole, nn);
        const int64_t e = int64_t(b) * g.C + cc, v = (int64_t(b) * g.G + grp) * g.N + n0;
        ld_pack_as<4>(g.Bm, v, sizeof(Tin) == 2, Bv[r], whole, nn);
        ld_pack_as<4>(g.Cm, v, sizeof(Tin) == 2, Cv[r], whole, nn);
        x[r] = widen(static_cast<const Tin*>(g.x)[e]);
        d[r] = widen(static_cast<const Tin*>(g.dt)[e]);
        z[r] = g.z ? widen(static_cast<const Tin*>(g.z)[e]) : 0.f;
    }
    ld_pack_as<4>(g.A, int64_t(cc) * g.N + n0, false, Av, whole, nn);
    const float bias = g.dt_bias ? g.dt_bias[cc] : 0.f, Dv = g.D ? g.D[cc] : 0.f;
    if (g.index) first_of_slots<R>(g.index, b0, slot, mine, SB);
    #pragma unroll
    for (int r = 0; r < R; ++r) {
        const float v = d[r] + bias, dd = g.softplus ? softplusf_(v) : v;
        float y = 0.f;
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            hv[r][i] = fmaf(__builtin_amdgcn_exp2f(dd * (Av[i] * kLog2e)), hv[r][i], dd * x[r] * Bv[r][i]);
            y = fmaf(Cv[r][i], hv[r][i], y);
        }
        if (mine[r] && nn > 0) st_pack<4>(g.s1 + (int64_t(slot[r]) * g.C + c) * g.N + n0, hv[r], whole, nn);
        if constexpr (LN >= 2) y += dpp<kDppQuadXor1>(y);
        if constexpr (LN >= 4) y += dpp<kDppQuadXor2>(y);
        if constexpr (LN >= 8) y += dpp<kDppRowHalfMirror>(y);
        if constexpr (LN >= 16) y += dpp<kDppRowMirror>(y);
        y = fmaf(Dv, x[r], y);
        if (g.z) y *= z[r] * sigmoidf_(z[r]);
        y = mine[r] ? y : 0.f;
        if (in && q == 0 && b0 + r < g.B) st_pack_as<1>(g.y, int64_t(b0 + r) * g.C + c, g.y_bf16, &y, true, 1);
    }
}

// Lanes to a channel, rows to a workgroup (four where that leaves four workgroups to a compute unit),
// workgroups.
struct StepPlan {
    int lanes, rows;
    int64_t blocks;
};
StepPlan step_plan(const SsmParams& p) {
    const int lanes = p.N <= 4 ? 1 : p.N <= 8 ? 2 : p.N <= 16 ? 4 : p.N <= 32 ? 8 : 16;
    const int64_t ncb = (int64_t(p.C) * lanes + SB - 1) / SB;
    const int rows = ncb * p.B >= 4096 ? 4 : 1;
    return {lanes, rows, ncb * ((int64_t(p.B) + rows - 1) / rows)};
}

template <typename Tin, int LN>
hipError_t launch_step_ln(const SsmParams& p, const StepPlan& s, hipStream_t stream) {
    const dim3 grid{unsigned(s.blocks)};
    if (s.rows == 4) hipLaunchKernelGGL((ssm_step_kernel<Tin, LN, 4>), grid, dim3(SB), 0, stream, p);
    else hipLaunchKernelGGL((ssm_step_kernel<Tin, LN, 1>), grid, dim3(SB), 0, stream, p);
    return hipGetLastError();
}

template <typename Tin>
hipError_t launch_step_in(SsmParams p, hipStream_t stream) {
    p.vec_n = p.N % 4 == 0;
    const StepPlan s = step_plan(p);
    switch (s.lanes) {
        case 1: return launch_step_ln<Tin, 1>(p, s, stream);
        case 2: return launch_step_ln<Tin, 2>(p, s, stream);
        case 4: return launch_step_ln<Tin, 4>(p, s, stream);
        case 8: return launch_step_ln<Tin, 8>(p, s, stream);
        default: return launch_step_ln<Tin, 16>(p, s, stream);
    }
}

}  // namespace

int64_t ssm_forward_threads(const SsmParams& p) { return p.C ? scan_blocks(p) * scan_waves(p) * 64 : 0; }
int64_t ssm_step_threads(const SsmParams& p) { return step_plan(p).blocks * SB; }

hipError_t launch_ssm_forward(const SsmParams& p, hipStream_t stream) {
    return p.in_bf16 ? launch_scan_in<bf16_t>(p, stream) : launch_scan_in<float>(p, stream);
}

hipError_t launch_ssm_step(const SsmParams& p, hipStream_t stream) {
    return p.in_bf16 ? launch_step_in<bf16_t>(p, stream) : launch_step_in<float>(p, stream);
}

}  // namespace wkv7
