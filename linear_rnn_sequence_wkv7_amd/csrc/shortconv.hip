// Short causal convolution on gfx950: y_t = act(bias + sum_k w_k x_{t-K+1+k}) per
// channel, for prompts, single tokens and training.
//
// Every direction reads and writes each element once and does a few operations
// on it, so memory bounds it first.  A thread has V consecutive channels (16
// bytes of bf16 inputs where C allows) and a run of tokens; the last K - 1 inputs
// stay in its registers, so a token's row is loaded once and only the K - 1 rows
// before a run are read twice.  The backward goes over a run once more from the
// same loads: it recomputes the value before the activation, and the gradient of
// input t is complete when output t + K - 1 has been passed.  Measured with K = 4,
// bf16: forward 8 x 4096 x 4096 (537 MB; counted 564, the rows before each run with them)
// 118 to 122 us, 4.4 to 4.6 TB/s where a copy of that size makes 5.2, vector units 62% busy; forward and
// backward 4 x 2048 x 2048 51 us, the backward's kernel 29 to 31 of them: counted 146 MB, 1.4
// times what it needs (a run of 16 tokens loads 22 rows of x and 19 of dy), at 4.9 TB/s, vector units 69% busy; a
// step of 256 x 4096 8.6 us, most of it the launch.
#include "seq_device.h"
#include "seq_internal.h"

namespace wkv7 {
namespace {

constexpr int NTC = 256;

// Threads are numbered (sequence, run of tokens, channel slot), slots fastest.
struct Runs {
    int slots, runs, len;   // channel slots of a row, runs of a sequence, tokens of a run
};

__device__ __forceinline__ float act_of(float pre, bool silu) { return silu ? pre * sigmoidf_(pre) : pre; }
// d act / d pre
__device__ __forceinline__ float act_grad(float pre, bool silu) {
    if (!silu) return 1.f;
    const float s = sigmoidf_(pre);
    return s * fmaf(pre, 1.f - s, 1.f);
}

// Input t of sequence b (t < 0: from the state, t >= len: none), V channels from c.
template <typename Tin, int V>
__device__ __forceinline__ void input_row(const ConvParams& g, int64_t b, int t, int c, float* v) {
    if (t < 0) {
        const int i = t + g.K - 1;
        if (!g.s0 || i < 0) {
            #pragma unroll
            for (int j = 0; j < V; ++j) v[j] = 0.f;
            return;
        }
        const Pack<Tin, V> r = ld_pack<V>(static_cast<const Tin*>(g.s0) + (b * (g.K - 1) + i) * g.C + c, true, V);
        #pragma unroll
        for (int j = 0; j < V; ++j) v[j] = widen(r.e[j]);
        return;
    }
    const Pack<Tin, V> r = ld_pack<V>(static_cast<const Tin*>(g.x) + (b * g.T + t) * g.C + c, true, V);
    #pragma unroll
    for (int j = 0; j < V; ++j) v[j] = widen(r.e[j]);
}

// A thread's V x K taps lie one after another.
template <int K, int V>
__device__ __forceinline__ void load_taps(const ConvParams& g, int c, float (&w)[K][V], float (&bias)[V]) {
    const Pack<float, V * K> t = ld_pack<V * K>(g.w + int64_t(c) * K, V >= 4, V * K);
    #pragma unroll
    for (int j = 0; j < V; ++j) {
        #pragma unroll
        for (int k = 0; k < K; ++k) w[k][j] = t.e[j * K + k];
    }
    const Pack<float, V> b = g.bias ? ld_pack<V>(g.bias + c, true, V) : Pack<float, V>{};
    #pragma unroll
    for (int j = 0; j < V; ++j) bias[j] = b.e[j];
}

template <typename Tin, int K, int V>
__global__ __launch_bounds__(NTC) void conv_forward_kernel(ConvParams g, Runs r) {
    const int64_t id = xcd_order(blockIdx.x, gridDim.x) * NTC + threadIdx.x;
    const int slot = int(id % r.slots), run = int(id / r.slots % r.runs);
    const int64_t b = id / r.slots / r.runs;
    if (b >= g.B) return;
    const int c = slot * V, t0 = run * r.len, t1 = min(t0 + r.len, g.T);
    const int len = seq_length(g.lengths, b, g.T);
    float w[K][V], bias[V], win[K][V];
    load_taps<K, V>(g, c, w, bias);
    if (t0 < len) {
        #pragma unroll
        for (int k = 0; k < K - 1; ++k) input_row<Tin, V>(g, b, t0 - K + 1 + k, c, win[k + 1]);
    }
    // Rows are loaded a group ahead.
    constexpr int U = 4;
    Pack<Tin, V> next[U];
    auto load = [&](int tb) {
        #pragma unroll
        for (int i = 0; i < U; ++i)
            next[i] = ld_pack<V>(static_cast<const Tin*>(g.x) + (b * g.T + min(tb + i, t1 - 1)) * g.C + c, true, V);
    };
    load(t0);
    for (int tb = t0; tb < t1; tb += U) {
        Pack<Tin, V> rows[U];
        #pragma unroll
        for (int i = 0; i < U; ++i) rows[i] = next[i];
        load(tb + U);
        #pragma unroll
        for (int i = 0; i < U; ++i) {
            const int t = tb + i;
            if (t >= t1) break;
            float y[V];
            #pragma unroll
            for (int j = 0; j < V; ++j) {
                #pragma unroll
                for (int k = 0; k < K - 1; ++k) win[k][j] = win[k + 1][j];
                win[K - 1][j] = widen(rows[i].e[j]);
                float pre = bias[j];
                #pragma unroll
                for (int k = 0; k < K; ++k) pre = fmaf(w[k][j], win[k][j], pre);
                y[j] = t < len ? act_of(pre, g.silu) : 0.f;
            }
            st_pack_as<V>(g.y, (b * g.T + t) * g.C + c, g.y_bf16, y, true, V);
        }
    }
    if (run == 0 && g.s1) {
        #pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            float v[V];
            input_row<Tin, V>(g, b, len - (K - 1) + k, c, v);
            st_pack<V>(static_cast<Tin*>(g.s1) + (b * (K - 1) + k) * g.C + c, v, true, V);
        }
    }
}

// R rows at once: their loads are in flight together and the taps are loaded once.
template <typename Tin, int K, int V, int R>
__global__ __launch_bounds__(NTC) void conv_step_kernel(ConvParams g) {
    const int slots = g.C / V, nsb = (slots + NTC - 1) / NTC;
    const int b0 = int(blockIdx.x / nsb) * R, s = int(blockIdx.x % nsb) * NTC + threadIdx.x;
    const bool in = s < slots;
    const int c = in ? s * V : 0;
    int slot[R];
    bool mine[R];
    Pack<Tin, V> row[R][K];
    #pragma unroll
    for (int r = 0; r < R; ++r) {
        const int b = min(b0 + r, g.B - 1);
        slot[r] = g.index ? g.index[b] : b;
        mine[r] = b0 + r < g.B && slot[r] >= 0 && slot[r] < g.S;
        const Tin* st = static_cast<const Tin*>(g.s1) + int64_t(mine[r] ? slot[r] : 0) * (K - 1) * g.C + c;
        row[r][K - 1] = ld_pack<V>(static_cast<const Tin*>(g.x) + int64_t(b) * g.C + c, true, V);
        #pragma unroll
        for (int k = 0; k < K - 1; ++k)
            if (mine[r]) row[r][k] = ld_pack<V>(st + int64_t(k) * g.C, true, V);
    }
    float w[K][V], bias[V];
    load_taps<K, V>(g, c, w, bias);
    if (g.index) first_of_slots<R>(g.index, b0, slot, mine, NTC);
    if (!in) return;
    #pragma unroll
    for (int r = 0; r < R; ++r) {
        if (b0 + r >= g.B) break;
        float y[V];
        #pragma unroll
        for (int j = 0; j < V; ++j) {
            float pre = bias[j];
            #pragma unroll
            for (int k = 0; k < K; ++k) pre = fmaf(w[k][j], widen(row[r][k].e[j]), pre);
            y[j] = mine[r] ? act_of(pre, g.silu) : 0.f;
        }
        st_pack_as<V>(g.y, int64_t(b0 + r) * g.C + c, g.y_bf16, y, true, V);
        if (!mine[r]) continue;
        Tin* st = static_cast<Tin*>(g.s1) + int64_t(slot[r]) * (K - 1) * g.C + c;
        #pragma unroll
        for (int k = 0; k < K - 1; ++k) *reinterpret_cast<Pack<Tin, V>*>(st + int64_t(k) * g.C) = row[r][k + 1];
    }
}

// A workgroup has 64 slots and 4 neighbouring runs of one sequence; its sums of the
// taps' and the bias' gradients go to one row of the workspace, [rows][K + 1][C].
template <typename Tin, typename Ty, int K, int V>
__global__ __launch_bounds__(NTC) void conv_backward_kernel(ConvParams g, Runs r, float* part) {
    const int nsb = (r.slots + 63) / 64, nrb = (r.runs + 3) / 4;
    const int64_t item = xcd_order(blockIdx.x, gridDim.x);
    const int lane = threadIdx.x & 63, rw = threadIdx.x >> 6;
    const int slot = int(item % nsb) * 64 + lane, run = int(item / nsb % nrb) * 4 + rw;
    const int64_t b = item / nsb / nrb;
    const bool in = slot < r.slots;
    const int c = in ? slot * V : 0, t0 = run * r.len, t1 = min(t0 + r.len, g.T);
    const int len = seq_length(g.lengths, b, g.T);
    float dw[K][V] = {}, db[V] = {};
    if (in && t0 < t1) {
        float w[K][V], bias[V], win[K][V], dp[K][V] = {};
        load_taps<K, V>(g, c, w, bias);
        #pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            input_row<Tin, V>(g, b, min(t0 - K + 1 + k, g.T - 1), c, win[k + 1]);
            if (t0 - K + 1 + k >= len) {   // padding: it meets gradients of 0 only, but may be no number
                #pragma unroll
                for (int j = 0; j < V; ++j) win[k + 1][j] = 0.f;
            }
        }
        // Outputs t0 .. t1 + K - 2; input t - K + 1 is done after output t.  The first run has the state's too.
        const int first = run == 0 ? 1 - K : t0;
        // Rows are loaded a group ahead.
        constexpr int U = 4;
        Pack<Tin, V> x_n[U];
        Pack<Ty, V> dy_n[U];
        auto load = [&](int tb) {
            #pragma unroll
            for (int i = 0; i < U; ++i) {
                const int64_t e = (b * g.T + min(tb + i, g.T - 1)) * g.C + c;
                x_n[i] = ld_pack<V>(static_cast<const Tin*>(g.x) + e, true, V);
                dy_n[i] = ld_pack<V>(static_cast<const Ty*>(g.dy) + e, true, V);
            }
        };
        load(t0);
        for (int tb = t0; tb < t1 + K - 1; tb += U) {
            Pack<Tin, V> xr[U];
            Pack<Ty, V> dyr[U];
            #pragma unroll
            for (int i = 0; i < U; ++i) {
                xr[i] = x_n[i];
                dyr[i] = dy_n[i];
            }
            load(tb + U);
            #pragma unroll
            for (int i = 0; i < U; ++i) {
                const int t = tb + i;
                if (t >= t1 + K - 1) break;
                const bool there = t < len;
                #pragma unroll
                for (int j = 0; j < V; ++j) {
                    #pragma unroll
                    for (int k = 0; k < K - 1; ++k) {
                        win[k][j] = win[k + 1][j];
                        dp[k][j] = dp[k + 1][j];
                    }
                    win[K - 1][j] = there ? widen(xr[i].e[j]) : 0.f;
                    float pre = bias[j];
                    #pragma unroll
                    for (int k = 0; k < K; ++k) pre = fmaf(w[k][j], win[k][j], pre);
                    const float d = there ? widen(dyr[i].e[j]) * act_grad(pre, g.silu) : 0.f;
                    dp[K - 1][j] = d;
                    if (t < t1) {
                        db[j] += d;
                        #pragma unroll
                        for (int k = 0; k < K; ++k) dw[k][j] = fmaf(d, win[k][j], dw[k][j]);
                    }
                }
                const int ti = t - (K - 1);
                if (ti < first) continue;
                float dx[V];
                #pragma unroll
                for (int j = 0; j < V; ++j) {
                    dx[j] = 0.f;
                    #pragma unroll
                    for (int k = 0; k < K; ++k) dx[j] = fmaf(w[K - 1 - k][j], dp[k][j], dx[j]);
                    if (ti >= len) dx[j] = 0.f;   // padding: also where a tap is no number
                }
                const int k1 = ti - (len - (K - 1));   // its place in state_out
                if (g.ds1 && k1 >= 0 && k1 < K - 1) {
                    float s[V];
                    ld_pack_as<V>(g.ds1, (b * (K - 1) + k1) * g.C + c, false, s, true, V);
                    #pragma unroll
                    for (int j = 0; j < V; ++j) dx[j] += s[j];
                }
                if (ti >= 0) st_pack<V>(static_cast<Tin*>(g.dx) + (b * g.T + ti) * g.C + c, dx, true, V);
                else if (g.ds0) st_pack<V>(g.ds0 + (b * (K - 1) + ti + K - 1) * g.C + c, dx, true, V);
            }
        }
    }
    // Sum over the 4 runs, in their order.
    __shared__ float s_sum[3][K + 1][64 * V];
    if (rw > 0) {
        #pragma unroll
        for (int j = 0; j < V; ++j) {
            #pragma unroll
            for (int k = 0; k < K; ++k) s_sum[rw - 1][k][j * 64 + lane] = dw[k][j];
            s_sum[rw - 1][K][j * 64 + lane] = db[j];
        }
    }
    __syncthreads();
    if (rw > 0 || !in) return;
    float* row = part + (b * nrb + item / nsb % nrb) * (K + 1) * g.C + c;
    #pragma unroll
    for (int k = 0; k <= K; ++k) {
        float v[V];
        #pragma unroll
        for (int j = 0; j < V; ++j) {
            v[j] = k < K ? dw[k < K ? k : 0][j] : db[j];
            #pragma unroll
            for (int o = 0; o < 3; ++o) v[j] += s_sum[o][k][j * 64 + lane];
        }
        st_pack<V>(row + int64_t(k) * g.C, v, true, V);
    }
}

// Column sums of the workspace rows: 32 columns a workgroup, 32 threads to each.
template <int K>
__global__ __launch_bounds__(1024) void conv_sum_kernel(ConvParams g, const float* part, int64_t rows) {
    const int64_t m = int64_t(blockIdx.x) * 32 + (threadIdx.x & 31), M = int64_t(K + 1) * g.C;
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
    const int k = int(m / g.C), c = int(m % g.C);
    if (k < K) g.dw[int64_t(c) * K + k] = s;
    else if (g.dbias) g.dbias[c] = s;
}

// Without tokens: the state goes over unchanged (its gradient too).
template <typename Tst>
__global__ __launch_bounds__(NTC) void conv_copy_kernel(const Tst* from, Tst* to, int64_t n) {
    for (int64_t i = int64_t(blockIdx.x) * NTC + threadIdx.x; i < n; i += int64_t(gridDim.x) * NTC)
        to[i] = from ? from[i] : Tst(0);
}
template <typename Tst>
hipError_t copy_state(const void* from, void* to, int64_t n, hipStream_t stream) {
    if (!to || n == 0) return hipSuccess;
    const int64_t nb = (n + NTC - 1) / NTC;
    hipLaunchKernelGGL((conv_copy_kernel<Tst>), dim3(unsigned(nb < 4096 ? nb : 4096)), dim3(NTC), 0, stream,
                       static_cast<const Tst*>(from), static_cast<Tst*>(to), n);
    return hipGetLastError();
}

// Run lengths: 32 tokens where that leaves two waves (in the backward four) for every SIMD, shorter
// for small calls.
Runs runs_of(const ConvParams& p, int V, bool bwd) {
    Runs r{p.C / V, 0, 32};
    while (r.len > 8 && int64_t(p.B) * ((p.T + r.len - 1) / r.len) * r.slots < (bwd ? 4 : 2) * 65536) r.len /= 2;
    r.runs = (p.T + r.len - 1) / r.len;
    return r;
}
// 8 channels of bf16 are a 16-byte load.  The backward's 4 K + 3 registers a channel leave room for two
// waves to a SIMD with 8 channels, for four with 4 (4 x 2048 x 2048 x 4 bf16: 48 and 36 us).
int channels_per_thread(const ConvParams& p, bool bwd) {
    return p.C % 8 == 0 && !bwd ? 8 : p.C % 4 == 0 ? 4 : p.C % 2 == 0 ? 2 : 1;
}

template <typename Tin, int K, int V>
hipError_t launch_k(const ConvParams& p, int what, hipStream_t stream) {
    const Runs r = runs_of(p, V, what == 2);
    if constexpr (V == 8) {
        if (what == 2) return hipErrorInvalidValue;   // channels_per_thread gives 4 at most
    }
    if (what == 1) {
        const int64_t nsb = (p.C / V + NTC - 1) / NTC;
        // two rows to a workgroup where that leaves one for every compute unit
        if (nsb * p.B >= 512) {
            hipLaunchKernelGGL((conv_step_kernel<Tin, K, V, 2>), dim3(unsigned(nsb * ((p.B + 1) / 2))), dim3(NTC), 0, stream, p);
        } else {
            hipLaunchKernelGGL((conv_step_kernel<Tin, K, V, 1>), dim3(unsigned(nsb * p.B)), dim3(NTC), 0, stream, p);
        }
        return hipGetLastError();
    }
    if (what == 0) {
        const int64_t threads = int64_t(p.B) * r.runs * r.slots;
        hipLaunchKernelGGL((conv_forward_kernel<Tin, K, V>), dim3(unsigned((threads + NTC - 1) / NTC)), dim3(NTC), 0, stream, p, r);
        return hipGetLastError();
    }
    if constexpr (V < 8) {
        const int64_t nsb = (r.slots + 63) / 64, nrb = (r.runs + 3) / 4;
        float* part = static_cast<float*>(p.ws);
        const dim3 grid{unsigned(nsb * nrb * p.B)};
        if (p.y_bf16) hipLaunchKernelGGL((conv_backward_kernel<Tin, bf16_t, K, V>), grid, dim3(NTC), 0, stream, p, r, part);
        else hipLaunchKernelGGL((conv_backward_kernel<Tin, float, K, V>), grid, dim3(NTC), 0, stream, p, r, part);
        hipLaunchKernelGGL((conv_sum_kernel<K>), dim3(unsigned((int64_t(K + 1) * p.C + 31) / 32)), dim3(1024), 0, stream, p, part, nrb * p.B);
    }
    return hipGetLastError();
}

template <typename Tin, int K>
hipError_t launch_v(const ConvParams& p, int what, hipStream_t stream) {
    switch (channels_per_thread(p, what == 2)) {
        case 8: return launch_k<Tin, K, 8>(p, what, stream);
        case 4: return launch_k<Tin, K, 4>(p, what, stream);
        case 2: return launch_k<Tin, K, 2>(p, what, stream);
        default: return launch_k<Tin, K, 1>(p, what, stream);
    }
}
template <typename Tin>
hipError_t launch_in(const ConvParams& p, int what, hipStream_t stream) {
    switch (p.K) {
        case 2: return launch_v<Tin, 2>(p, what, stream);
        case 3: return launch_v<Tin, 3>(p, what, stream);
        default: return launch_v<Tin, 4>(p, what, stream);
    }
}
hipError_t launch(const ConvParams& p, int what, hipStream_t stream) {
    return p.in_bf16 ? launch_in<bf16_t>(p, what, stream) : launch_in<float>(p, what, stream);
}

}  // namespace

int64_t shortconv_forward_threads(const ConvParams& p) {
    if (int64_t(p.T) * p.C == 0) return 0;
    const Runs r = runs_of(p, channels_per_thread(p, false), false);
    return int64_t(p.B) * r.runs * r.slots + NTC;
}
int64_t shortconv_step_threads(const ConvParams& p) { return (p.C / channels_per_thread(p, false) / NTC + 1) * ((int64_t(p.B) + 1) / 2 + 512) * NTC; }
int64_t shortconv_backward_threads(const ConvParams& p) {
    if (int64_t(p.T) * p.C == 0) return 0;
    const Runs r = runs_of(p, channels_per_thread(p, true), true);
    const int64_t own = int64_t(p.B) * ((r.slots + 63) / 64) * ((r.runs + 3) / 4) * NTC, sums = int64_t(p.K + 1) * p.C * 32 + 1024;
    return own > sums ? own : sums;
}
int64_t shortconv_backward_workspace(const ConvParams& p) {
    if (int64_t(p.B) * p.T * p.C == 0) return 0;
    const Runs r = runs_of(p, channels_per_thread(p, true), true);
    return (int64_t(p.B) * ((r.runs + 3) / 4) * (p.K + 1) * p.C * 4 + 255) & ~int64_t(255);
}

hipError_t launch_shortconv_forward(const ConvParams& p, hipStream_t stream) {
    if (p.T == 0) {
        const int64_t n = int64_t(p.B) * (p.K - 1) * p.C;
        return p.in_bf16 ? copy_state<bf16_t>(p.s0, p.s1, n, stream) : copy_state<float>(p.s0, p.s1, n, stream);
    }
    return launch(p, 0, stream);
}
hipError_t launch_shortconv_step(const ConvParams& p, hipStream_t stream) { return launch(p, 1, stream); }
hipError_t launch_shortconv_backward(const ConvParams& p, hipStream_t stream) {
    if (p.B == 0 || p.T == 0) {   // no tokens: no gradient of the parameters
        hipError_t e = copy_state<float>(nullptr, p.dw, int64_t(p.C) * p.K, stream);
        if (e == hipSuccess) e = copy_state<float>(nullptr, p.dbias, p.C, stream);
        if (e == hipSuccess) e = copy_state<float>(p.ds1, p.ds0, int64_t(p.B) * (p.K - 1) * p.C, stream);
        return e;
    }
    return launch(p, 2, stream);
}

}  // namespace wkv7
