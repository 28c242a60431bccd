// Group norm on gfx950, channels last, with an activation and an output gate:
//
//   xh = (x - mean) rstd,  y = act(xh weight + bias) gate
//
// with the statistics of T positions and C / G channels.  Memory bounds it: x
// (and the gate) are read and y is written once wherever a group's values fit the
// registers that loaded them; a pass over the same values for the variance costs
// registers only.  The forms, the first that fits:
//
// T = 1 (a recurrence's heads), groups of 8 LG channels (LG = 1, 2 .. 64): a thread
// has 8 channels of a row, LG neighbouring lanes a group.  The variance is that of the
// differences from the mean.  A workgroup takes several rows, so that weights are
// loaded once and, in the backward, a thread sums its channels' parameter gradients
// over its rows.  32768 x 4096 bf16 in 64 groups with a gate, 805 MB (as counted): forward 162 us
// (5.0 TB/s, a copy's rate); 8192 x 2048 forward and backward 61 us, the kernels at 5.1 TB/s.
//
// T = 1, other groups of up to 1024 or, even, 2048 channels: the same with one wave
// to a group, one load of 4 bytes a lane and run: far from a copy.  32768 rows of about 4000 channels, bf16
// with a gate: groups of 80 604 us (1.3 TB/s), of 96 516, of 160 421, of 192 382 (2.1 TB/s).  Whole rows of
// 4096 go through the three passes below: 370 us (2.2 TB/s).
//
// T > 1, a group's values within the registers of a workgroup of 1024: one pass, the
// sums over the workgroup; 3 x 1531 x 960 fp32 in 30 groups 13.0 us (bf16 12.8),
// which the 90 workgroups bound (35 MB at most, vector units 9% busy).
//
// Otherwise three passes: partial (mean, sum of squared differences) of up to 64
// positions of a channel slot (8 channels of one group, or 1), formed block by
// block in registers around the block's own mean and joined by the parallel
// variance formula; their join per group; and the elementwise pass.  The backward
// has the same shape with the sums of dpre and dpre xh per channel in place of
// the statistics: they are the parameters' gradients and, weighted, the two means
// that dx needs:
//
//   dpre = dy gate act'(pre),  dxh = dpre weight,
//   dx = rstd (dxh - mean(dxh) - xh mean(dxh xh)),  dgate = dy act(pre)
//
// All sums are fp32 and in a fixed order.
#include "seq_device.h"
#include "seq_internal.h"

namespace wkv7 {
namespace {

constexpr int NTG = 256;
constexpr int V8 = 8;

// Sum over aligned groups of n lanes (a power of two up to 64); every lane gets it.
template <int LG>
__device__ __forceinline__ float sum_lanes(float x) {
    if constexpr (LG >= 2) x += dpp<kDppQuadXor1>(x);
    if constexpr (LG >= 4) x += dpp<kDppQuadXor2>(x);
    if constexpr (LG >= 8) x += dpp<kDppRowHalfMirror>(x);
    if constexpr (LG >= 16) x += dpp<kDppRowMirror>(x);
    if constexpr (LG >= 32) x += __shfl_xor(x, 16);
    if constexpr (LG >= 64) x += __shfl_xor(x, 32);
    return x;
}

// weight and bias of V channels (c a multiple of V).
template <int V>
__device__ __forceinline__ void channel_params(const NormParams& g, int c, float* wt, float* bs) {
    Pack<float, V> w, b;
    #pragma unroll
    for (int j = 0; j < V; ++j) {
        w.e[j] = 1.f;
        b.e[j] = 0.f;
    }
    if (g.weight) w = ld_pack<V>(g.weight + c, true, V);
    if (g.bias) b = ld_pack<V>(g.bias + c, true, V);
    #pragma unroll
    for (int j = 0; j < V; ++j) {
        wt[j] = w.e[j];
        bs[j] = b.e[j];
    }
}

struct Rows {
    int slots;   // 8-channel slots of a row
    int cols;    // slots of a workgroup: threads are (row, slot), slots fastest
    int ncol;    // workgroups side by side
    int64_t nrow;  // rows of workgroups: workgroup y takes rows y, y + nrow .. (times its own rows at once)
};

// Forward and backward of rows by themselves, groups of 8 LG channels.
template <typename Tin, typename Ty, int LG, bool BWD>
__global__ __launch_bounds__(NTG) void norm_rows_kernel(NormParams g, Rows r, float* part) {
    const int at_once = NTG / r.cols;
    const int ry = threadIdx.x / r.cols, sx = threadIdx.x % r.cols;
    const int64_t wg_row = blockIdx.x / r.ncol;
    const int slot = int(blockIdx.x % r.ncol) * r.cols + sx;
    const bool in = ry < at_once && slot < r.slots;
    const int c = in ? slot * V8 : 0;
    float wt[V8], bs[V8], dw[V8] = {}, db[V8] = {};
    channel_params<V8>(g, c, wt, bs);
    const Tin *xp = static_cast<const Tin*>(g.x), *gp = static_cast<const Tin*>(g.gate);
    constexpr float inv = 1.f / (8 * LG);
    for (int64_t row = wg_row * at_once + ry; in && row < g.B; row += r.nrow * at_once) {
        const int64_t e = row * g.C + c;
        const int grp = slot / LG;
        const bool there = seq_length(g.lengths, row, 1) > 0;
        const Pack<Tin, V8> xr = ld_pack<V8>(xp + e, true, V8);
        Pack<Tin, V8> gr;
        Pack<Ty, V8> dyr;
        if (g.gate) gr = ld_pack<V8>(gp + e, true, V8);
        if constexpr (BWD) dyr = ld_pack<V8>(static_cast<const Ty*>(g.dy) + e, true, V8);
        float x[V8], pre[V8], xh[V8], out[V8];
        #pragma unroll
        for (int j = 0; j < V8; ++j) x[j] = widen(xr.e[j]);
        float mean, rstd;
        if constexpr (!BWD) {
            float s = 0.f, q = 0.f;
            #pragma unroll
            for (int j = 0; j < V8; ++j) s += x[j];
            mean = sum_lanes<LG>(s) * inv;
            #pragma unroll
            for (int j = 0; j < V8; ++j) q = fmaf(x[j] - mean, x[j] - mean, q);
            rstd = 1.f / __builtin_sqrtf(fmaf(sum_lanes<LG>(q), inv, g.eps));
            if (!there) {
                mean = 0.f;
                rstd = 1.f / __builtin_sqrtf(g.eps);
            }
            if (g.mean && slot % LG == 0) {
                g.mean[row * g.G + grp] = mean;
                g.rstd[row * g.G + grp] = rstd;
            }
        } else {
            mean = g.mean[row * g.G + grp];
            rstd = g.rstd[row * g.G + grp];
        }
        #pragma unroll
        for (int j = 0; j < V8; ++j) {
            xh[j] = (x[j] - mean) * rstd;
            pre[j] = fmaf(xh[j], wt[j], bs[j]);
        }
        if constexpr (!BWD) {
            #pragma unroll
            for (int j = 0; j < V8; ++j) {
                float y = g.silu ? pre[j] * sigmoidf_(pre[j]) : pre[j];
                if (g.gate) y *= widen(gr.e[j]);
                out[j] = there ? y : 0.f;
            }
            st_pack_as<V8>(g.y, e, g.y_bf16, out, true, V8);
        } else {
            float dxh[V8], s1 = 0.f, s2 = 0.f;
            #pragma unroll
            for (int j = 0; j < V8; ++j) {
                float act = pre[j], da = 1.f;
                if (g.silu) {
                    const float sg = sigmoidf_(pre[j]);
                    act = pre[j] * sg;
                    da = sg * fmaf(pre[j], 1.f - sg, 1.f);
                }
                float d = widen(dyr.e[j]);
                out[j] = there ? d * act : 0.f;
                if (g.gate) d *= widen(gr.e[j]);
                const float dpre = there ? d * da : 0.f;
                xh[j] = there ? xh[j] : 0.f;
                db[j] += dpre;
                dw[j] = fmaf(dpre, xh[j], dw[j]);
                dxh[j] = dpre * wt[j];
                s1 += dxh[j];
                s2 = fmaf(dxh[j], xh[j], s2);
            }
            if (g.gate) st_pack<V8>(static_cast<Tin*>(g.dgate) + e, out, true, V8);
            s1 = sum_lanes<LG>(s1) * inv;
            s2 = sum_lanes<LG>(s2) * inv;
            #pragma unroll
            for (int j = 0; j < V8; ++j) out[j] = there ? (dxh[j] - s1 - xh[j] * s2) * rstd : 0.f;
            st_pack<V8>(static_cast<Tin*>(g.dx) + e, out, true, V8);
        }
    }
    if constexpr (BWD) {   // the workgroup's sums over its rows: [nrow][2][C]
        __shared__ float s_w[NTG][V8], s_b[NTG][V8];
        #pragma unroll
        for (int j = 0; j < V8; ++j) {
            s_w[threadIdx.x][j] = dw[j];
            s_b[threadIdx.x][j] = db[j];
        }
        __syncthreads();
        if (!in || ry != 0) return;
        for (int o = 1; o < at_once; ++o) {
            #pragma unroll
            for (int j = 0; j < V8; ++j) {
                dw[j] += s_w[o * r.cols + sx][j];
                db[j] += s_b[o * r.cols + sx][j];
            }
        }
        st_pack<V8>(part + (wg_row * 2) * g.C + c, dw, true, V8);
        st_pack<V8>(part + (wg_row * 2 + 1) * g.C + c, db, true, V8);
    }
}

// Rows by themselves, any group of up to 64 K V channels: one wave a row and group, V neighbouring
// channels in each of K runs of 64 lanes.  Wave (chunk, group) takes the rows chunk, chunk + nrow ..
template <typename Tin, typename Ty, int K, int V, bool BWD>
__global__ __launch_bounds__(NTG) void norm_wave_kernel(NormParams g, int64_t nrow, float* part) {
    const int64_t wave = int64_t(blockIdx.x) * (NTG / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, grp = int(wave % g.G), Cg = g.C / g.G;
    const int64_t chunk = wave / g.G;
    if (chunk >= nrow) return;
    const int c0 = grp * Cg + lane * V;
    bool in[K];
    float wt[K][V], bs[K][V], dw[K][V] = {}, db[K][V] = {};
    #pragma unroll
    for (int k = 0; k < K; ++k) {
        in[k] = (k * 64 + lane) * V < Cg;
        #pragma unroll
        for (int v = 0; v < V; ++v) {
            wt[k][v] = in[k] && g.weight ? g.weight[c0 + k * 64 * V + v] : 1.f;
            bs[k][v] = in[k] && g.bias ? g.bias[c0 + k * 64 * V + v] : 0.f;
        }
    }
    const float inv = 1.f / float(Cg);
    for (int64_t row = chunk; row < g.B; row += nrow) {
        const int64_t e = row * g.C + c0, st = row * g.G + grp;
        const bool there = seq_length(g.lengths, row, 1) > 0;
        float x[K][V], gt[K][V];
        #pragma unroll
        for (int k = 0; k < K; ++k) {
            const Pack<Tin, V> r = ld_pack<V>(static_cast<const Tin*>(g.x) + e + k * 64 * V, false, in[k] ? V : 0);
            Pack<Tin, V> q;
            if (g.gate) q = ld_pack<V>(static_cast<const Tin*>(g.gate) + e + k * 64 * V, false, in[k] ? V : 0);
            #pragma unroll
            for (int v = 0; v < V; ++v) {
                x[k][v] = widen(r.e[v]);
                gt[k][v] = g.gate ? widen(q.e[v]) : 1.f;
            }
        }
        float mean, rstd;
        if constexpr (!BWD) {
            float s = 0.f, q = 0.f;
            #pragma unroll
            for (int k = 0; k < K; ++k)
                #pragma unroll
                for (int v = 0; v < V; ++v) s += x[k][v];
            mean = sum_lanes<64>(s) * inv;
            #pragma unroll
            for (int k = 0; k < K; ++k)
                #pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float d = in[k] ? x[k][v] - mean : 0.f;
                    q = fmaf(d, d, q);
                }
            rstd = 1.f / __builtin_sqrtf(fmaf(sum_lanes<64>(q), inv, g.eps));
            if (!there) {
                mean = 0.f;
                rstd = 1.f / __builtin_sqrtf(g.eps);
            }
            if (g.mean && lane == 0) {
                g.mean[st] = mean;
                g.rstd[st] = rstd;
            }
        } else {
            mean = g.mean[st];
            rstd = g.rstd[st];
        }
        float out[K][V], dxh[K][V], s1 = 0.f, s2 = 0.f;
        #pragma unroll
        for (int k = 0; k < K; ++k) {
            float dy[V];
            if constexpr (BWD) {
                const Pack<Ty, V> r = ld_pack<V>(static_cast<const Ty*>(g.dy) + e + k * 64 * V, false, in[k] ? V : 0);
                #pragma unroll
                for (int v = 0; v < V; ++v) dy[v] = widen(r.e[v]);
            }
            #pragma unroll
            for (int v = 0; v < V; ++v) {
                const float xh = (x[k][v] - mean) * rstd, pre = fmaf(xh, wt[k][v], bs[k][v]);
                float act = pre, da = 1.f;
                if (g.silu) {
                    const float sg = sigmoidf_(pre);
                    act = pre * sg;
                    da = sg * fmaf(pre, 1.f - sg, 1.f);
                }
                if constexpr (!BWD) {
                    out[k][v] = there ? act * gt[k][v] : 0.f;
                } else {
                    const bool on = there && in[k];
                    out[k][v] = on ? dy[v] * act : 0.f;
                    const float dpre = on ? dy[v] * gt[k][v] * da : 0.f;
                    x[k][v] = on ? xh : 0.f;
                    db[k][v] += dpre;
                    dw[k][v] = fmaf(dpre, x[k][v], dw[k][v]);
                    dxh[k][v] = dpre * wt[k][v];
                    s1 += dxh[k][v];
                    s2 = fmaf(dxh[k][v], x[k][v], s2);
                }
            }
            if constexpr (!BWD) st_pack_as<V>(g.y, e + k * 64 * V, g.y_bf16, out[k], false, in[k] ? V : 0);
            else if (g.gate) st_pack<V>(static_cast<Tin*>(g.dgate) + e + k * 64 * V, out[k], false, in[k] ? V : 0);
        }
        if constexpr (BWD) {
            s1 = sum_lanes<64>(s1) * inv;
            s2 = sum_lanes<64>(s2) * inv;
            #pragma unroll
            for (int k = 0; k < K; ++k) {
                #pragma unroll
                for (int v = 0; v < V; ++v) out[k][v] = there ? (dxh[k][v] - s1 - x[k][v] * s2) * rstd : 0.f;
                st_pack<V>(static_cast<Tin*>(g.dx) + e + k * 64 * V, out[k], false, in[k] ? V : 0);
            }
        }
    }
    if constexpr (BWD) {
        #pragma unroll
        for (int k = 0; k < K; ++k) {
            st_pack<V>(part + chunk * 2 * g.C + c0 + k * 64 * V, dw[k], false, in[k] ? V : 0);
            st_pack<V>(part + (chunk * 2 + 1) * g.C + c0 + k * 64 * V, db[k], false, in[k] ? V : 0);
        }
    }
}

// dweight and dbias: column sums of [rows][2][C]; 32 columns a workgroup, 32 threads to each.
__global__ __launch_bounds__(1024) void norm_sum_kernel(NormParams g, const float* part, int64_t rows) {
    const int64_t m = int64_t(blockIdx.x) * 32 + (threadIdx.x & 31), M = 2 * int64_t(g.C);
    const int y = threadIdx.x >> 5;
    float s = 0.f;
    if (m < M) {
        #pragma unroll 4
        for (int64_t i = y; i < rows; i += 32) s += part[i * M + m];
    }
    __shared__ float sm[32][32];
    sm[y][threadIdx.x & 31] = s;
    __syncthreads();
    if (y != 0 || m >= M) return;
    s = 0.f;
    #pragma unroll
    for (int i = 0; i < 32; ++i) s += sm[i][threadIdx.x & 31];
    float* out = m < g.C ? g.dweight : g.dbias;
    if (out) out[m < g.C ? m : m - g.C] = s;
}

// ---- statistics over positions --------------------------------------------

struct Stats {
    float n, mean, m2;   // count, mean, sum of squared differences from it
};
__device__ __forceinline__ Stats join(Stats a, Stats b) {
    const float n = a.n + b.n;
    if (n == 0.f) return a;
    const float f = b.n / n, d = b.mean - a.mean;
    return {n, fmaf(d, f, a.mean), a.m2 + b.m2 + d * d * a.n * f};
}

// Thread (sequence, run of run_len positions (a multiple of 8), slot of V channels), slots fastest: [B][runs][slots][2].
template <typename Tin, int V>
__global__ __launch_bounds__(NTG) void norm_stats_kernel(NormParams g, int slots, int runs, int run_len, float* part) {
    const int64_t id = int64_t(blockIdx.x) * NTG + threadIdx.x;
    const int slot = int(id % slots), run = int(id / slots % runs);
    const int64_t b = id / slots / runs;
    if (b >= g.B) return;
    const int len = seq_length(g.lengths, b, g.T), t0 = run * run_len, t1 = min(t0 + run_len, len);
    constexpr int U = 8;
    Stats st{0.f, 0.f, 0.f};
    for (int t = t0; t < t1; t += U) {
        const int n = min(U, t1 - t);
        Pack<Tin, V> rows[U];
        #pragma unroll
        for (int i = 0; i < U; ++i)
            rows[i] = ld_pack<V>(static_cast<const Tin*>(g.x) + (b * g.T + min(t + i, t1 - 1)) * g.C + slot * V, true, V);
        float s = 0.f, q = 0.f;
        #pragma unroll
        for (int i = 0; i < U; ++i) {
            #pragma unroll
            for (int j = 0; j < V; ++j) s += i < n ? widen(rows[i].e[j]) : 0.f;
        }
        const float cnt = float(n * V), m = s / cnt;
        #pragma unroll
        for (int i = 0; i < U; ++i) {
            #pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = i < n ? widen(rows[i].e[j]) - m : 0.f;
                q = fmaf(d, d, q);
            }
        }
        st = join(st, Stats{cnt, m, q});
    }
    part[2 * id] = st.mean;
    part[2 * id + 1] = st.m2;
}

// One workgroup per (sequence, group): the join of its partials, in a fixed order.
__global__ __launch_bounds__(NTG) void norm_join_kernel(NormParams g, int slots, int runs, int run_len, int V, const float* part,
                                                        float* mean, float* rstd) {
    const int64_t b = blockIdx.x / g.G;
    const int grp = int(blockIdx.x % g.G);
    const int len = seq_length(g.lengths, b, g.T);
    const int gs = slots / g.G, used = (len + run_len - 1) / run_len;
    Stats st{0.f, 0.f, 0.f};
    for (int64_t i = threadIdx.x; i < int64_t(used) * gs; i += NTG) {
        const int run = int(i / gs), s = grp * gs + int(i % gs);
        const int64_t id = (b * runs + run) * slots + s;
        st = join(st, Stats{float(min(run_len, len - run * run_len) * V), part[2 * id], part[2 * id + 1]});
    }
    __shared__ Stats sm[NTG];
    sm[threadIdx.x] = st;
    for (int o = NTG / 2; o > 0; o /= 2) {
        __syncthreads();
        if (threadIdx.x < o) sm[threadIdx.x] = join(sm[threadIdx.x], sm[threadIdx.x + o]);
    }
    if (threadIdx.x != 0) return;
    const Stats all = sm[0];
    mean[blockIdx.x] = all.mean;
    rstd[blockIdx.x] = 1.f / __builtin_sqrtf((all.n > 0.f ? all.m2 / all.n : 0.f) + g.eps);
}

// The value before the activation and what follows from it, for one slot of one position.
template <typename Tin, int V>
struct Slot {
    float xh[V], act[V], da[V], gate[V];
    __device__ __forceinline__ void load(const NormParams& g, int64_t e, const float* wt, const float* bs, float mean, float rstd) {
        const Pack<Tin, V> x = ld_pack<V>(static_cast<const Tin*>(g.x) + e, true, V);
        Pack<Tin, V> gt;
        if (g.gate) gt = ld_pack<V>(static_cast<const Tin*>(g.gate) + e, true, V);
        #pragma unroll
        for (int j = 0; j < V; ++j) {
            gate[j] = g.gate ? widen(gt.e[j]) : 1.f;
            xh[j] = (widen(x.e[j]) - mean) * rstd;
            const float pre = fmaf(xh[j], wt[j], bs[j]);
            act[j] = pre;
            da[j] = 1.f;
            if (g.silu) {
                const float s = sigmoidf_(pre);
                act[j] = pre * s;
                da[j] = s * fmaf(pre, 1.f - s, 1.f);
            }
        }
    }
};

// Elementwise passes; BWD: dx and dgate, with the two means of each group in m12.  A thread keeps its
// channels and goes over `per` positions of a sequence, `at_once` apart.
template <typename Tin, int V, bool BWD>
__global__ __launch_bounds__(NTG) void norm_apply_kernel(NormParams g, int slots, int cols, int ncol, int per, const float* mean,
                                                         const float* rstd, const float* m12) {
    const int at_once = NTG / cols, ry = threadIdx.x / cols;
    const int slot = int(blockIdx.x % ncol) * cols + threadIdx.x % cols, c = slot * V;
    const unsigned rest = blockIdx.x / ncol, chunks = (g.T + per * at_once - 1) / (per * at_once);
    const int64_t b = rest / chunks;
    const int t0 = int(rest % chunks) * per * at_once + ry, t1 = min(g.T, t0 - ry + per * at_once);
    if (ry >= at_once || slot >= slots) return;
    const int len = seq_length(g.lengths, b, g.T);
    const int64_t bg = b * g.G + c / (g.C / g.G);
    const float mu = mean[bg], rs = rstd[bg];
    const float m1 = BWD ? m12[2 * bg] : 0.f, m2 = BWD ? m12[2 * bg + 1] : 0.f;
    float wt[V], bs[V];
    channel_params<V>(g, c, wt, bs);
    for (int t = t0; t < t1; t += at_once) {
        const int64_t e = (b * g.T + t) * g.C + c;
        const bool there = t < len;
        float out[V] = {}, dg[V] = {};
        if (there) {
            Slot<Tin, V> s;
            s.load(g, e, wt, bs, mu, rs);
            if constexpr (!BWD) {
                #pragma unroll
                for (int j = 0; j < V; ++j) out[j] = s.act[j] * s.gate[j];
            } else {
                float dy[V];
                ld_pack_as<V>(g.dy, e, g.y_bf16, dy, true, V);
                #pragma unroll
                for (int j = 0; j < V; ++j) {
                    dg[j] = dy[j] * s.act[j];
                    const float dxh = dy[j] * s.gate[j] * s.da[j] * wt[j];
                    out[j] = (dxh - m1 - s.xh[j] * m2) * rs;
                }
            }
        }
        if constexpr (!BWD) {
            st_pack_as<V>(g.y, e, g.y_bf16, out, true, V);
        } else {
            st_pack<V>(static_cast<Tin*>(g.dx) + e, out, true, V);
            if (g.gate) st_pack<V>(static_cast<Tin*>(g.dgate) + e, dg, true, V);
        }
    }
}

// Per channel, over run_len positions: sums of dpre xh and of dpre, [B][runs][2][C].
template <typename Tin, int V>
__global__ __launch_bounds__(NTG) void norm_grad_kernel(NormParams g, int slots, int runs, int run_len, float* part) {
    const int64_t id = int64_t(blockIdx.x) * NTG + threadIdx.x;
    const int slot = int(id % slots), run = int(id / slots % runs), c = slot * V;
    const int64_t b = id / slots / runs;
    if (b >= g.B) return;
    const int len = seq_length(g.lengths, b, g.T), t0 = run * run_len, t1 = min(t0 + run_len, len);
    const int64_t bg = b * g.G + c / (g.C / g.G);
    const float mean = g.mean[bg], rstd = g.rstd[bg];
    float dw[V] = {}, db[V] = {}, wt[V], bs[V];
    channel_params<V>(g, c, wt, bs);
    for (int t = t0; t < t1; ++t) {
        const int64_t e = (b * g.T + t) * g.C + c;
        Slot<Tin, V> s;
        s.load(g, e, wt, bs, mean, rstd);
        float dy[V];
        ld_pack_as<V>(g.dy, e, g.y_bf16, dy, true, V);
        #pragma unroll
        for (int j = 0; j < V; ++j) {
            const float dpre = dy[j] * s.gate[j] * s.da[j];
            db[j] += dpre;
            dw[j] = fmaf(dpre, s.xh[j], dw[j]);
        }
    }
    float* row = part + (b * runs + run) * 2 * g.C + c;
    st_pack<V>(row, dw, true, V);
    st_pack<V>(row + g.C, db, true, V);
}

// One workgroup per (sequence, group): the means of dxh and dxh xh from the channels' sums.
__global__ __launch_bounds__(NTG) void norm_means_kernel(NormParams g, int runs, int run_len, const float* part, float* m12) {
    const int64_t b = blockIdx.x / g.G;
    const int Cg = g.C / g.G, c0 = int(blockIdx.x % g.G) * Cg;
    const int len = seq_length(g.lengths, b, g.T), used = (len + run_len - 1) / run_len;
    float s1 = 0.f, s2 = 0.f;
    for (int64_t i = threadIdx.x; i < int64_t(used) * Cg; i += NTG) {
        const int run = int(i / Cg), c = c0 + int(i % Cg);
        const float* row = part + (b * runs + run) * 2 * g.C + c;
        const float w = g.weight ? g.weight[c] : 1.f;
        s2 = fmaf(w, row[0], s2);
        s1 = fmaf(w, row[g.C], s1);
    }
    __shared__ float sm[2][NTG];
    sm[0][threadIdx.x] = s1;
    sm[1][threadIdx.x] = s2;
    for (int o = NTG / 2; o > 0; o /= 2) {
        __syncthreads();
        if (threadIdx.x < o) {
            sm[0][threadIdx.x] += sm[0][threadIdx.x + o];
            sm[1][threadIdx.x] += sm[1][threadIdx.x + o];
        }
    }
    if (threadIdx.x != 0) return;
    const float n = float(len) * float(Cg);
    m12[2 * blockIdx.x] = n > 0.f ? sm[0][0] / n : 0.f;
    m12[2 * blockIdx.x + 1] = n > 0.f ? sm[1][0] / n : 0.f;
}

// A group's values over all positions in the registers of one workgroup: x is read once and the
// statistics, or in the backward the two means, need no other pass.  A thread has V neighbouring channels
// of up to R positions, `apart` positions from one to the next.
constexpr int NTS = 1024;

// Sum over the workgroup; every thread gets it.  Wave sums, then their sum in a fixed order.
__device__ __forceinline__ float sum_group(float x, float* s_wave) {
    x = sum_lanes<64>(x);
    if ((threadIdx.x & 63) == 0) s_wave[threadIdx.x >> 6] = x;
    __syncthreads();
    float s = 0.f;
    #pragma unroll
    for (int i = 0; i < NTS / 64; ++i) s += s_wave[i];
    return s;
}

template <typename Tin, typename Ty, int V, int R, bool BWD>
__global__ __launch_bounds__(NTS) void norm_slab_kernel(NormParams g, float* part) {
    __shared__ float s_wave[2][NTS / 64];
    const int64_t b = blockIdx.x / g.G;
    const int grp = int(blockIdx.x % g.G), Cg = g.C / g.G, slots = Cg / V, apart = NTS / slots;
    const int ry = threadIdx.x / slots, c = grp * Cg + int(threadIdx.x % slots) * V;
    const int len = seq_length(g.lengths, b, g.T);
    const bool in = ry < apart;
    const float count = float(len) * float(Cg), inv = count > 0.f ? 1.f / count : 0.f;
    Pack<Tin, V> xr[R];
    #pragma unroll
    for (int r = 0; r < R; ++r) {
        const int t = r * apart + ry;
        if (in && t < len) xr[r] = ld_pack<V>(static_cast<const Tin*>(g.x) + (b * g.T + t) * g.C + c, true, V);
    }
    float mean, rstd;
    if constexpr (!BWD) {
        float s = 0.f, q = 0.f;
        #pragma unroll
        for (int r = 0; r < R; ++r)
            if (in && r * apart + ry < len) {
                float sr = 0.f;
                #pragma unroll
                for (int j = 0; j < V; ++j) sr += widen(xr[r].e[j]);
                s += sr;
            }
        mean = sum_group(s, s_wave[0]) * inv;
        #pragma unroll
        for (int r = 0; r < R; ++r)
            if (in && r * apart + ry < len) {
                float qr = 0.f;
                #pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float d = widen(xr[r].e[j]) - mean;
                    qr = fmaf(d, d, qr);
                }
                q += qr;
            }
        rstd = 1.f / __builtin_sqrtf(fmaf(sum_group(q, s_wave[1]), inv, g.eps));
        if (g.mean && threadIdx.x == 0) {
            g.mean[blockIdx.x] = mean;
            g.rstd[blockIdx.x] = rstd;
        }
    } else {
        mean = g.mean[blockIdx.x];
        rstd = g.rstd[blockIdx.x];
    }
    float wt[V], bs[V];
    channel_params<V>(g, in ? c : 0, wt, bs);
    if constexpr (!BWD) {
        #pragma unroll
        for (int r = 0; r < R; ++r) {
            const int t = r * apart + ry;
            if (!in || t >= g.T) break;
            const int64_t e = (b * g.T + t) * g.C + c;
            float out[V] = {};
            if (t < len) {
                Pack<Tin, V> gt;
                if (g.gate) gt = ld_pack<V>(static_cast<const Tin*>(g.gate) + e, true, V);
                #pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float pre = fmaf((widen(xr[r].e[j]) - mean) * rstd, wt[j], bs[j]);
                    out[j] = g.silu ? pre * sigmoidf_(pre) : pre;
                    if (g.gate) out[j] *= widen(gt.e[j]);
                }
            }
            st_pack_as<V>(g.y, e, g.y_bf16, out, true, V);
        }
    } else {
        Pack<Ty, V> dyr[R];
        #pragma unroll
        for (int r = 0; r < R; ++r) {
            const int t = r * apart + ry;
            if (in && t < len) dyr[r] = ld_pack<V>(static_cast<const Ty*>(g.dy) + (b * g.T + t) * g.C + c, true, V);
        }
        float dxh[R][V], dw[V] = {}, db[V] = {}, s1 = 0.f, s2 = 0.f;
        #pragma unroll
        for (int r = 0; r < R; ++r) {
            const int t = r * apart + ry;
            if (!in || t >= g.T) break;
            const int64_t e = (b * g.T + t) * g.C + c;
            Pack<Tin, V> gt;
            float dg[V] = {}, s1r = 0.f, s2r = 0.f;
            if (t < len && g.gate) gt = ld_pack<V>(static_cast<const Tin*>(g.gate) + e, true, V);
            #pragma unroll
            for (int j = 0; j < V; ++j) {
                dxh[r][j] = 0.f;
                if (t >= len) continue;
                const float xh = (widen(xr[r].e[j]) - mean) * rstd, pre = fmaf(xh, wt[j], bs[j]);
                float act = pre, da = 1.f, d = widen(dyr[r].e[j]);
                if (g.silu) {
                    const float sg = sigmoidf_(pre);
                    act = pre * sg;
                    da = sg * fmaf(pre, 1.f - sg, 1.f);
                }
                dg[j] = d * act;
                if (g.gate) d *= widen(gt.e[j]);
                d *= da;
                db[j] += d;
                dw[j] = fmaf(d, xh, dw[j]);
                dxh[r][j] = d * wt[j];
                s1r += dxh[r][j];
                s2r = fmaf(dxh[r][j], xh, s2r);
            }
            s1 += s1r;
            s2 += s2r;
            if (g.gate) st_pack<V>(static_cast<Tin*>(g.dgate) + e, dg, true, V);
        }
        s1 = sum_group(s1, s_wave[0]) * inv;
        s2 = sum_group(s2, s_wave[1]) * inv;
        #pragma unroll
        for (int r = 0; r < R; ++r) {
            const int t = r * apart + ry;
            if (!in || t >= g.T) break;
            float out[V];
            #pragma unroll
            for (int j = 0; j < V; ++j)
                out[j] = t < len ? (dxh[r][j] - s1 - (widen(xr[r].e[j]) - mean) * rstd * s2) * rstd : 0.f;
            st_pack<V>(static_cast<Tin*>(g.dx) + (b * g.T + t) * g.C + c, out, true, V);
        }
        // The channels' sums of this sequence, [B][2][C]: over the threads of a channel, through LDS.
        __shared__ float s_par[2][NTS * V];
        #pragma unroll
        for (int j = 0; j < V; ++j) {
            s_par[0][threadIdx.x * V + j] = dw[j];
            s_par[1][threadIdx.x * V + j] = db[j];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * Cg; i += NTS) {
            const int which = i >= Cg, cc = i - which * Cg;
            float s = 0.f;
            for (int r = 0; r < apart; ++r) s += s_par[which][(r * slots) * V + cc];
            part[(b * 2 + which) * g.C + grp * Cg + cc] = s;
        }
    }
}

constexpr int64_t kMaxThreads = int64_t(1) << 32;

// Lanes of a group in the row form (0: the general form).
int row_lanes(const NormParams& p) {
    const int Cg = p.C / p.G;
    if (p.T != 1 || Cg % 8 != 0) return 0;
    const int lg = Cg / 8;
    return lg <= 64 && (lg & (lg - 1)) == 0 ? lg : 0;
}
Rows rows_of(const NormParams& p, bool bwd) {
    Rows r;
    r.slots = p.C / V8;
    r.cols = r.slots < NTG ? r.slots : NTG;
    r.ncol = (r.slots + r.cols - 1) / r.cols;
    const int64_t at_once = NTG / r.cols, rows = (p.B + at_once - 1) / at_once;
    // Workgroups to a compute unit: 8; in the backward 2, since each leaves a row of sums to be added.
    const int64_t all = bwd ? 512 : 2048, most = all / r.ncol > 0 ? all / r.ncol : 1;
    r.nrow = rows < most ? rows : most;
    return r;
}
// Runs of 64 lanes of the wave form (0: the general form), and its rows of waves.
int wave_runs(const NormParams& p) {
    const int Cg = p.C / p.G, V = Cg % 2 == 0 ? 2 : 1;
    return p.T != 1 ? 0 : Cg <= 64 * 4 * V ? 4 : Cg <= 64 * 16 * V ? 16 : 0;
}
int64_t wave_rows(const NormParams& p, bool bwd) {
    const int64_t all = bwd ? 4096 : 16384, most = all / p.G > 0 ? all / p.G : 1;
    return p.B < most ? p.B : most;
}
int channels_per_thread(const NormParams& p) {
    const int Cg = p.C / p.G;
    return Cg % 8 == 0 ? 8 : Cg % 2 == 0 ? 2 : 1;
}
// Channels (up to 16 bytes of them) and positions of a thread in the slab form (0 positions: the group
// does not fit the registers of a workgroup).  1 x 1531 x 1024 in 32 groups: 11 us, with three passes 12;
// 8 x 1531 x 1024: 19 and 30; 8 x 500 x 1024: 8 and 16, with gradients 15 and 30 (fp32).
int slab_channels(const NormParams& p, bool bwd) {
    const int Cg = p.C / p.G;
    return p.in_bf16 && !bwd && Cg % 8 == 0 ? 8 : Cg % 4 == 0 ? 4 : Cg % 2 == 0 ? 2 : 1;
}
int slab_positions(const NormParams& p, bool bwd) {
    const int Cg = p.C / p.G, V = slab_channels(p, bwd), slots = Cg / V;
    if (p.T <= 1 || slots > NTS || int64_t(p.B) * p.G * NTS >= kMaxThreads) return 0;
    const int apart = NTS / slots, r = (p.T + apart - 1) / apart;
    return r <= 4 ? 4 : r <= 8 ? 8 : r <= 16 && V < 8 && !bwd ? 16 : 0;   // (the backward has three arrays)
}
// Positions of one partial sum: 64, fewer where that leaves less than a wave for every SIMD.
int run_of(const NormParams& p) {
    int pr = 64;
    while (pr > 8 && int64_t(p.B) * ((p.T + pr - 1) / pr) * (p.C / channels_per_thread(p)) < 65536) pr /= 2;
    return pr;
}
int runs_of(const NormParams& p) { return (p.T + run_of(p) - 1) / run_of(p); }
int64_t up(int64_t x) { return (x + 255) & ~int64_t(255); }

// The elementwise pass: slots of a workgroup, workgroups side by side, positions of a thread, workgroups.
struct Apply {
    int cols, ncol, per;
    int64_t blocks;
};
Apply apply_of(const NormParams& p, int slots) {
    const int cols = slots < NTG ? slots : NTG, ncol = (slots + cols - 1) / cols, at_once = NTG / cols;
    // Positions of a thread: 8, fewer where that leaves less than 16 workgroups to a compute unit
    // (3 x 1531 x 960 fp32: 18.6 us with 8, 8 with 1).
    int per = 8;
    while (per > 1 && int64_t(p.B) * p.T * ncol / (at_once * per) < 4096) per /= 2;
    return {cols, ncol, per, (p.T + int64_t(per) * at_once - 1) / (int64_t(per) * at_once) * p.B * ncol};
}

template <typename Tin, int LG>
hipError_t launch_rows(const NormParams& p, bool bwd, hipStream_t stream) {
    const Rows r = rows_of(p, bwd);
    float* part = static_cast<float*>(p.ws);
    const dim3 grid{unsigned(r.nrow * r.ncol)};
    if (!bwd) {
        hipLaunchKernelGGL((norm_rows_kernel<Tin, Tin, LG, false>), grid, dim3(NTG), 0, stream, p, r, part);
        return hipGetLastError();
    }
    if (p.y_bf16) hipLaunchKernelGGL((norm_rows_kernel<Tin, bf16_t, LG, true>), grid, dim3(NTG), 0, stream, p, r, part);
    else hipLaunchKernelGGL((norm_rows_kernel<Tin, float, LG, true>), grid, dim3(NTG), 0, stream, p, r, part);
    hipLaunchKernelGGL(norm_sum_kernel, dim3(unsigned((2 * int64_t(p.C) + 31) / 32)), dim3(1024), 0, stream, p, part, r.nrow);
    return hipGetLastError();
}

template <typename Tin, int K, int V>
hipError_t launch_wave(const NormParams& p, bool bwd, hipStream_t stream) {
    const int64_t nrow = wave_rows(p, bwd), per = NTG / 64;
    float* part = static_cast<float*>(p.ws);
    const dim3 grid{unsigned((nrow * p.G + per - 1) / per)};
    if (!bwd) {
        hipLaunchKernelGGL((norm_wave_kernel<Tin, Tin, K, V, false>), grid, dim3(NTG), 0, stream, p, nrow, part);
        return hipGetLastError();
    }
    if (p.y_bf16) hipLaunchKernelGGL((norm_wave_kernel<Tin, bf16_t, K, V, true>), grid, dim3(NTG), 0, stream, p, nrow, part);
    else hipLaunchKernelGGL((norm_wave_kernel<Tin, float, K, V, true>), grid, dim3(NTG), 0, stream, p, nrow, part);
    hipLaunchKernelGGL(norm_sum_kernel, dim3(unsigned((2 * int64_t(p.C) + 31) / 32)), dim3(1024), 0, stream, p, part, nrow);
    return hipGetLastError();
}

template <typename Tin, int V, int R>
hipError_t launch_slab(const NormParams& p, bool bwd, hipStream_t stream) {
    float* part = static_cast<float*>(p.ws);
    const dim3 grid{unsigned(int64_t(p.B) * p.G)};
    constexpr bool kBwd = R <= 8 && V <= 4;
    if (!bwd || !kBwd) {
        hipLaunchKernelGGL((norm_slab_kernel<Tin, Tin, V, R, false>), grid, dim3(NTS), 0, stream, p, part);
        return hipGetLastError();
    }
    if constexpr (kBwd) {
        if (p.y_bf16) hipLaunchKernelGGL((norm_slab_kernel<Tin, bf16_t, V, R, true>), grid, dim3(NTS), 0, stream, p, part);
        else hipLaunchKernelGGL((norm_slab_kernel<Tin, float, V, R, true>), grid, dim3(NTS), 0, stream, p, part);
        hipLaunchKernelGGL(norm_sum_kernel, dim3(unsigned((2 * int64_t(p.C) + 31) / 32)), dim3(1024), 0, stream, p, part, int64_t(p.B));
    }
    return hipGetLastError();
}
template <typename Tin, int V>
hipError_t launch_slab_r(const NormParams& p, bool bwd, hipStream_t stream) {
    switch (slab_positions(p, bwd)) {
        case 4: return launch_slab<Tin, V, 4>(p, bwd, stream);
        case 8: return launch_slab<Tin, V, 8>(p, bwd, stream);
        default: return launch_slab<Tin, V, 16>(p, bwd, stream);
    }
}

template <typename Tin, int V>
hipError_t launch_general(const NormParams& p, bool bwd, hipStream_t stream) {
    const int slots = p.C / V, runs = runs_of(p), run_len = run_of(p);
    const int64_t threads = int64_t(p.B) * runs * slots;
    const dim3 g1{unsigned((threads + NTG - 1) / NTG)}, g2{unsigned(int64_t(p.B) * p.G)};
    const auto [cols, ncol, per, blocks] = apply_of(p, slots);
    const dim3 g3{unsigned(blocks)};
    float* ws = static_cast<float*>(p.ws);
    if (!bwd) {
        float *mean = p.mean, *rstd = p.rstd;
        if (!mean) {
            mean = ws;
            rstd = ws + int64_t(p.B) * p.G;
        }
        float* part = ws + up(2 * int64_t(p.B) * p.G);
        hipLaunchKernelGGL((norm_stats_kernel<Tin, V>), g1, dim3(NTG), 0, stream, p, slots, runs, run_len, part);
        hipLaunchKernelGGL(norm_join_kernel, g2, dim3(NTG), 0, stream, p, slots, runs, run_len, V, part, mean, rstd);
        hipLaunchKernelGGL((norm_apply_kernel<Tin, V, false>), g3, dim3(NTG), 0, stream, p, slots, cols, ncol, per, mean, rstd,
                           static_cast<const float*>(nullptr));
        return hipGetLastError();
    }
    float *m12 = ws, *part = ws + up(2 * int64_t(p.B) * p.G);
    hipLaunchKernelGGL((norm_grad_kernel<Tin, V>), g1, dim3(NTG), 0, stream, p, slots, runs, run_len, part);
    hipLaunchKernelGGL(norm_means_kernel, g2, dim3(NTG), 0, stream, p, runs, run_len, part, m12);
    hipLaunchKernelGGL(norm_sum_kernel, dim3(unsigned((2 * int64_t(p.C) + 31) / 32)), dim3(1024), 0, stream, p, part,
                       int64_t(p.B) * runs);
    hipLaunchKernelGGL((norm_apply_kernel<Tin, V, true>), g3, dim3(NTG), 0, stream, p, slots, cols, ncol, per, p.mean, p.rstd, m12);
    return hipGetLastError();
}

template <typename Tin>
hipError_t launch_in(const NormParams& p, bool bwd, hipStream_t stream) {
    switch (row_lanes(p)) {
        case 1: return launch_rows<Tin, 1>(p, bwd, stream);
        case 2: return launch_rows<Tin, 2>(p, bwd, stream);
        case 4: return launch_rows<Tin, 4>(p, bwd, stream);
        case 8: return launch_rows<Tin, 8>(p, bwd, stream);
        case 16: return launch_rows<Tin, 16>(p, bwd, stream);
        case 32: return launch_rows<Tin, 32>(p, bwd, stream);
        case 64: return launch_rows<Tin, 64>(p, bwd, stream);
        default: break;
    }
    const bool even = p.C / p.G % 2 == 0;
    switch (wave_runs(p)) {
        case 4: return even ? launch_wave<Tin, 4, 2>(p, bwd, stream) : launch_wave<Tin, 4, 1>(p, bwd, stream);
        case 16: return even ? launch_wave<Tin, 16, 2>(p, bwd, stream) : launch_wave<Tin, 16, 1>(p, bwd, stream);
        default: break;
    }
    if (slab_positions(p, bwd)) {
        switch (slab_channels(p, bwd)) {
            case 8:
                if constexpr (sizeof(Tin) == 2) return slab_positions(p, bwd) == 4 ? launch_slab<Tin, 8, 4>(p, bwd, stream) : launch_slab<Tin, 8, 8>(p, bwd, stream);
            case 4: return launch_slab_r<Tin, 4>(p, bwd, stream);
            case 2: return launch_slab_r<Tin, 2>(p, bwd, stream);
            default: return launch_slab_r<Tin, 1>(p, bwd, stream);
        }
    }
    switch (channels_per_thread(p)) {
        case 8: return launch_general<Tin, 8>(p, bwd, stream);
        case 2: return launch_general<Tin, 2>(p, bwd, stream);
        default: return launch_general<Tin, 1>(p, bwd, stream);
    }
}

}  // namespace

int64_t groupnorm_threads(const NormParams& p, bool bwd) {
    if (int64_t(p.B) * p.T * p.C == 0) return 0;
    int64_t n;
    if (row_lanes(p)) {
        const Rows r = rows_of(p, bwd);
        n = r.nrow * r.ncol * NTG;
    } else if (wave_runs(p)) {
        n = wave_rows(p, bwd) * p.G * 64 + NTG;
    } else if (slab_positions(p, bwd)) {
        n = int64_t(p.B) * p.G * NTS;
    } else {
        const int slots = p.C / channels_per_thread(p);
        const int64_t stats = int64_t(p.B) * runs_of(p) * slots + NTG, join = int64_t(p.B) * p.G * NTG, apply = apply_of(p, slots).blocks * NTG;
        n = stats > join ? stats : join;
        n = n > apply ? n : apply;
    }
    const int64_t sums = bwd ? int64_t(p.C) * 64 + 1024 : 0;
    return n > sums ? n : sums;
}
int64_t groupnorm_workspace(const NormParams& p) {
    if (int64_t(p.B) * p.T * p.C == 0 || row_lanes(p) || wave_runs(p) || slab_positions(p, false)) return 0;
    const int64_t slots = p.C / channels_per_thread(p);
    return up(4 * (up(2 * int64_t(p.B) * p.G) + 2 * int64_t(p.B) * runs_of(p) * slots));
}
int64_t groupnorm_backward_workspace(const NormParams& p) {
    if (int64_t(p.B) * p.T * p.C == 0) return 0;
    if (row_lanes(p)) return up(4 * rows_of(p, true).nrow * 2 * p.C);
    if (wave_runs(p)) return up(4 * wave_rows(p, true) * 2 * p.C);
    if (slab_positions(p, true)) return up(4 * int64_t(p.B) * 2 * p.C);
    return up(4 * (up(2 * int64_t(p.B) * p.G) + 2 * int64_t(p.B) * runs_of(p) * p.C));
}

namespace {
__global__ __launch_bounds__(256) void norm_fill_kernel(float* a, float va, float* b, float vb, int64_t n) {
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
        if (a) a[i] = va;
        if (b) b[i] = vb;
    }
}
}  // namespace

hipError_t launch_groupnorm_forward(const NormParams& p, hipStream_t stream) {
    if (int64_t(p.B) * p.T * p.C == 0) {   // only the statistics of empty sequences
        if (!p.mean || p.B == 0) return hipSuccess;
        const int64_t n = int64_t(p.B) * p.G;
        hipLaunchKernelGGL(norm_fill_kernel, dim3(unsigned(n / 256 + 1 < 4096 ? n / 256 + 1 : 4096)), dim3(256), 0, stream,
                           p.mean, 0.f, p.rstd, float(1.0 / __builtin_sqrt(double(p.eps))), n);
        return hipGetLastError();
    }
    return p.in_bf16 ? launch_in<bf16_t>(p, false, stream) : launch_in<float>(p, false, stream);
}
hipError_t launch_groupnorm_backward(const NormParams& p, hipStream_t stream) {
    if (int64_t(p.B) * p.T * p.C == 0) {
        if (p.C == 0 || (!p.dweight && !p.dbias)) return hipSuccess;
        hipLaunchKernelGGL(norm_fill_kernel, dim3(unsigned(p.C / 256 + 1)), dim3(256), 0, stream, p.dweight, 0.f, p.dbias,
                           0.f, int64_t(p.C));
        return hipGetLastError();
    }
    return p.in_bf16 ? launch_in<bf16_t>(p, true, stream) : launch_in<float>(p, true, stream);
}

}  // namespace wkv7
