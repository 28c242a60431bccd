// Group norm on gfx950, channels last, with an activation and an output gate:
//
//   xh = (x - mean) rstd,  y = act(xh weight + bias) gate
//
// with the statistics of T positions and C / G channels.  Memory bounds it: x
// (and the gate) are read and y is written once where a group's values fit the
// registers that loaded them, which is the case of a recurrence's heads (T = 1).
//
// T = 1, groups of 8 LG channels (LG = 1, 2 .. 64): a thread has 8 channels of a
// row, LG neighbouring lanes a group.  The variance is that of the differences
// from the mean, in registers.  A workgroup takes several rows, so that weights
// are loaded once and, in the backward, a thread sums its channels' parameter
// gradients over its rows.
//
// Otherwise three passes: partial (mean, sum of squared differences) of 64
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
constexpr int PR = 64;   // positions of one partial sum

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

struct Rows {
    int slots;   // 8-channel slots of a row
    int cols;    // slots of a workgroup: threads are (row, slot), slots fastest
    int ncol;    // workgroups side by side
    int64_t nrow;  // rows of workgroups: workgroup y takes rows y, y + nrow .. (times its own rows at once)
};

// Forward and backward of rows by themselves, groups of 8 LG channels.
template <typename Tin, int LG, bool BWD>
__global__ __launch_bounds__(NTG) void norm_rows_kernel(NormParams g, Rows r, float* part) {
    const int at_once = NTG / r.cols;
    const int ry = threadIdx.x / r.cols, sx = threadIdx.x % r.cols;
    const int64_t wg_row = blockIdx.x / r.ncol;
    const int slot = int(blockIdx.x % r.ncol) * r.cols + sx;
    const bool in = ry < at_once && slot < r.slots;
    const int c = in ? slot * V8 : 0;
    float wt[V8], bs[V8], dw[V8] = {}, db[V8] = {};
    #pragma unroll
    for (int j = 0; j < V8; ++j) {
        wt[j] = g.weight ? g.weight[c + j] : 1.f;
        bs[j] = g.bias ? g.bias[c + j] : 0.f;
    }
    const Tin *xp = static_cast<const Tin*>(g.x), *gp = static_cast<const Tin*>(g.gate);
    constexpr float inv = 1.f / (8 * LG);
    for (int64_t row = wg_row * at_once + ry; in && row < g.B; row += r.nrow * at_once) {
        const int64_t e = row * g.C + c;
        const int grp = slot / LG;
        const bool there = seq_length(g.lengths, row, 1) > 0;
        const Pack<Tin, V8> xr = ld_pack<V8>(xp + e, true, V8);
        Pack<Tin, V8> gr;
        if (g.gate) gr = ld_pack<V8>(gp + e, true, V8);
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
            float dy[V8], dxh[V8], s1 = 0.f, s2 = 0.f;
            ld_pack_as<V8>(g.dy, e, g.y_bf16, dy, true, V8);
            #pragma unroll
            for (int j = 0; j < V8; ++j) {
                float act = pre[j], da = 1.f;
                if (g.silu) {
                    const float sg = sigmoidf_(pre[j]);
                    act = pre[j] * sg;
                    da = sg * fmaf(pre[j], 1.f - sg, 1.f);
                }
                float d = dy[j];
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

// dweight and dbias: column sums of [rows][2][C]; 16 columns a workgroup, 16 threads to each.
__global__ __launch_bounds__(256) void norm_sum_kernel(NormParams g, const float* part, int64_t rows) {
    const int64_t m = int64_t(blockIdx.x) * 16 + (threadIdx.x & 15), M = 2 * int64_t(g.C);
    const int y = threadIdx.x >> 4;
    float s = 0.f;
    if (m < M)
        for (int64_t i = y; i < rows; i += 16) s += part[i * M + m];
    __shared__ float sm[16][16];
    sm[y][threadIdx.x & 15] = s;
    __syncthreads();
    if (y != 0 || m >= M) return;
    s = 0.f;
    #pragma unroll
    for (int i = 0; i < 16; ++i) s += sm[i][threadIdx.x & 15];
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

// Thread (sequence, run of PR positions, slot of V channels), slots fastest: [B][runs][slots][2].
template <typename Tin, int V>
__global__ __launch_bounds__(NTG) void norm_stats_kernel(NormParams g, int slots, int runs, float* part) {
    const int64_t id = int64_t(blockIdx.x) * NTG + threadIdx.x;
    const int slot = int(id % slots), run = int(id / slots % runs);
    const int64_t b = id / slots / runs;
    if (b >= g.B) return;
    const int len = seq_length(g.lengths, b, g.T), t0 = run * PR, t1 = min(t0 + PR, len);
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
__global__ __launch_bounds__(NTG) void norm_join_kernel(NormParams g, int slots, int runs, int V, const float* part,
                                                        float* mean, float* rstd) {
    const int64_t b = blockIdx.x / g.G;
    const int grp = int(blockIdx.x % g.G);
    const int len = seq_length(g.lengths, b, g.T);
    const int gs = slots / g.G, used = (len + PR - 1) / PR;
    Stats st{0.f, 0.f, 0.f};
    for (int64_t i = threadIdx.x; i < int64_t(used) * gs; i += NTG) {
        const int run = int(i / gs), s = grp * gs + int(i % gs);
        const int64_t id = (b * runs + run) * slots + s;
        st = join(st, Stats{float(min(PR, len - run * PR) * V), part[2 * id], part[2 * id + 1]});
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
    float xh[V], act[V], da[V], gate[V], wt[V];
    __device__ __forceinline__ void load(const NormParams& g, int64_t e, int c, float mean, float rstd) {
        const Pack<Tin, V> x = ld_pack<V>(static_cast<const Tin*>(g.x) + e, true, V);
        Pack<Tin, V> gt;
        if (g.gate) gt = ld_pack<V>(static_cast<const Tin*>(g.gate) + e, true, V);
        #pragma unroll
        for (int j = 0; j < V; ++j) {
            wt[j] = g.weight ? g.weight[c + j] : 1.f;
            gate[j] = g.gate ? widen(gt.e[j]) : 1.f;
            xh[j] = (widen(x.e[j]) - mean) * rstd;
            const float pre = fmaf(xh[j], wt[j], g.bias ? g.bias[c + j] : 0.f);
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

// Elementwise passes; BWD: dx and dgate, with the two means of each group in m12.
template <typename Tin, int V, bool BWD>
__global__ __launch_bounds__(NTG) void norm_apply_kernel(NormParams g, int slots, const float* mean, const float* rstd,
                                                         const float* m12) {
    const int64_t n = int64_t(g.B) * g.T * slots;
    for (int64_t id = int64_t(blockIdx.x) * NTG + threadIdx.x; id < n; id += int64_t(gridDim.x) * NTG) {
        const int slot = int(id % slots), c = slot * V;
        const int64_t row = id / slots, b = row / g.T, e = row * g.C + c;
        const int64_t bg = b * g.G + c / (g.C / g.G);
        float out[V] = {};
        const bool there = row - b * g.T < seq_length(g.lengths, b, g.T);
        if constexpr (!BWD) {
            if (there) {
                Slot<Tin, V> s;
                s.load(g, e, c, mean[bg], rstd[bg]);
                #pragma unroll
                for (int j = 0; j < V; ++j) out[j] = s.act[j] * s.gate[j];
            }
            st_pack_as<V>(g.y, e, g.y_bf16, out, true, V);
        } else {
            float dg[V] = {};
            if (there) {
                Slot<Tin, V> s;
                s.load(g, e, c, mean[bg], rstd[bg]);
                float dy[V];
                ld_pack_as<V>(g.dy, e, g.y_bf16, dy, true, V);
                const float m1 = m12[2 * bg], m2 = m12[2 * bg + 1], rs = rstd[bg];
                #pragma unroll
                for (int j = 0; j < V; ++j) {
                    dg[j] = dy[j] * s.act[j];
                    const float dxh = dy[j] * s.gate[j] * s.da[j] * s.wt[j];
                    out[j] = (dxh - m1 - s.xh[j] * m2) * rs;
                }
            }
            st_pack<V>(static_cast<Tin*>(g.dx) + e, out, true, V);
            if (g.gate) st_pack<V>(static_cast<Tin*>(g.dgate) + e, dg, true, V);
        }
    }
}

// Per channel, over PR positions: sums of dpre xh and of dpre, [B][runs][2][C].
template <typename Tin, int V>
__global__ __launch_bounds__(NTG) void norm_grad_kernel(NormParams g, int slots, int runs, float* part) {
    const int64_t id = int64_t(blockIdx.x) * NTG + threadIdx.x;
    const int slot = int(id % slots), run = int(id / slots % runs), c = slot * V;
    const int64_t b = id / slots / runs;
    if (b >= g.B) return;
    const int len = seq_length(g.lengths, b, g.T), t0 = run * PR, t1 = min(t0 + PR, len);
    const int64_t bg = b * g.G + c / (g.C / g.G);
    const float mean = g.mean[bg], rstd = g.rstd[bg];
    float dw[V] = {}, db[V] = {};
    for (int t = t0; t < t1; ++t) {
        const int64_t e = (b * g.T + t) * g.C + c;
        Slot<Tin, V> s;
        s.load(g, e, c, mean, rstd);
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
__global__ __launch_bounds__(NTG) void norm_means_kernel(NormParams g, int runs, const float* part, float* m12) {
    const int64_t b = blockIdx.x / g.G;
    const int Cg = g.C / g.G, c0 = int(blockIdx.x % g.G) * Cg;
    const int len = seq_length(g.lengths, b, g.T), used = (len + PR - 1) / PR;
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

// Lanes of a group in the row form (0: the general form).
int row_lanes(const NormParams& p) {
    const int Cg = p.C / p.G;
    if (p.T != 1 || Cg % 8 != 0) return 0;
    const int lg = Cg / 8;
    return lg <= 64 && (lg & (lg - 1)) == 0 ? lg : 0;
}
Rows rows_of(const NormParams& p) {
    Rows r;
    r.slots = p.C / V8;
    r.cols = r.slots < NTG ? r.slots : NTG;
    r.ncol = (r.slots + r.cols - 1) / r.cols;
    const int64_t at_once = NTG / r.cols, rows = (p.B + at_once - 1) / at_once;
    const int64_t most = 2048 / r.ncol > 0 ? 2048 / r.ncol : 1;   // 8 workgroups to a compute unit
    r.nrow = rows < most ? rows : most;
    return r;
}
int channels_per_thread(const NormParams& p) {
    const int Cg = p.C / p.G;
    return Cg % 8 == 0 ? 8 : Cg % 2 == 0 ? 2 : 1;
}
int runs_of(const NormParams& p) { return (p.T + PR - 1) / PR; }
int64_t up(int64_t x) { return (x + 255) & ~int64_t(255); }

template <typename Tin, int LG>
hipError_t launch_rows(const NormParams& p, bool bwd, hipStream_t stream) {
    const Rows r = rows_of(p);
    float* part = static_cast<float*>(p.ws);
    const dim3 grid{unsigned(r.nrow * r.ncol)};
    if (!bwd) {
        hipLaunchKernelGGL((norm_rows_kernel<Tin, LG, false>), grid, dim3(NTG), 0, stream, p, r, part);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((norm_rows_kernel<Tin, LG, true>), grid, dim3(NTG), 0, stream, p, r, part);
    hipLaunchKernelGGL(norm_sum_kernel, dim3(unsigned((2 * int64_t(p.C) + 15) / 16)), dim3(256), 0, stream, p, part, r.nrow);
    return hipGetLastError();
}

template <typename Tin, int V>
hipError_t launch_general(const NormParams& p, bool bwd, hipStream_t stream) {
    const int slots = p.C / V, runs = runs_of(p);
    const int64_t threads = int64_t(p.B) * runs * slots, n = int64_t(p.B) * p.T * slots;
    const dim3 g1{unsigned((threads + NTG - 1) / NTG)}, g2{unsigned(int64_t(p.B) * p.G)};
    const int64_t nb = (n + NTG - 1) / NTG;
    const dim3 g3{unsigned(nb < (1 << 20) ? nb : (1 << 20))};
    float* ws = static_cast<float*>(p.ws);
    if (!bwd) {
        float *mean = p.mean, *rstd = p.rstd;
        if (!mean) {
            mean = ws;
            rstd = ws + int64_t(p.B) * p.G;
        }
        float* part = ws + up(2 * int64_t(p.B) * p.G);
        hipLaunchKernelGGL((norm_stats_kernel<Tin, V>), g1, dim3(NTG), 0, stream, p, slots, runs, part);
        hipLaunchKernelGGL(norm_join_kernel, g2, dim3(NTG), 0, stream, p, slots, runs, V, part, mean, rstd);
        hipLaunchKernelGGL((norm_apply_kernel<Tin, V, false>), g3, dim3(NTG), 0, stream, p, slots, mean, rstd,
                           static_cast<const float*>(nullptr));
        return hipGetLastError();
    }
    float *m12 = ws, *part = ws + up(2 * int64_t(p.B) * p.G);
    hipLaunchKernelGGL((norm_grad_kernel<Tin, V>), g1, dim3(NTG), 0, stream, p, slots, runs, part);
    hipLaunchKernelGGL(norm_means_kernel, g2, dim3(NTG), 0, stream, p, runs, part, m12);
    hipLaunchKernelGGL(norm_sum_kernel, dim3(unsigned((2 * int64_t(p.C) + 15) / 16)), dim3(256), 0, stream, p, part,
                       int64_t(p.B) * runs);
    hipLaunchKernelGGL((norm_apply_kernel<Tin, V, true>), g3, dim3(NTG), 0, stream, p, slots, p.mean, p.rstd, m12);
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
    switch (channels_per_thread(p)) {
        case 8: return launch_general<Tin, 8>(p, bwd, stream);
        case 2: return launch_general<Tin, 2>(p, bwd, stream);
        default: return launch_general<Tin, 1>(p, bwd, stream);
    }
}

}  // namespace

int64_t groupnorm_workspace(const NormParams& p) {
    if (int64_t(p.B) * p.T * p.C == 0 || row_lanes(p)) return 0;
    const int64_t slots = p.C / channels_per_thread(p);
    return up(4 * (up(2 * int64_t(p.B) * p.G) + 2 * int64_t(p.B) * runs_of(p) * slots));
}
int64_t groupnorm_backward_workspace(const NormParams& p) {
    if (int64_t(p.B) * p.T * p.C == 0) return 0;
    if (row_lanes(p)) return up(4 * rows_of(p).nrow * 2 * p.C);
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
