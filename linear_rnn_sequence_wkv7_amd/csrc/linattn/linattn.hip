// Linear attention with a decay for each head: how a call is split up, and what runs beside the
// sweeps of linattn_core.h: the chain of the segments' states, the gradient of g, sums over heads
// that share an operand, and the step on a pool of states.
#include "../seq_device.h"
#include "linattn_internal.h"
#include "wave_sum64.h"

namespace wkv7 {
namespace linattn {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------- chain of segments

struct Chain {
    float* ws;            // [B, H, segs, Dk, Dv]: what the segments add (but the last); becomes the state before each
    const float* kept;    // [B, H, segs]
    const float* first;   // [B, H, Dk, Dv] or null
};
// A thread per element of a state.  Eight segments' parts are read before the first is needed.  8 segments of
// 64 heads' states and gradients of 128 x 128 take 25 us.
__global__ __launch_bounds__(kThreads) void chain_kernel(Chain f, Chain r, int segs, int elems) {
    const bool back = blockIdx.z;
    const Chain c = back ? r : f;
    const int e = blockIdx.x * kThreads + threadIdx.x;
    const int64_t bh = blockIdx.y;
    if (e >= elems) return;
    float s = c.first ? c.first[bh * elems + e] : 0.f;
    float* p = c.ws + bh * segs * int64_t(elems) + e;
    const float* k = c.kept + bh * segs;
    for (int i0 = 0; i0 < segs; i0 += 8) {
        float u[8];
        #pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = back ? segs - 1 - i0 - i : i0 + i;
            u[i] = i0 + i < segs - 1 ? p[int64_t(at) * elems] : 0.f;
        }
        #pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i0 + i >= segs) break;
            const int at = back ? segs - 1 - i0 - i : i0 + i;
            p[int64_t(at) * elems] = s;
            if (i0 + i < segs - 1) s = fmaf(k[at], s, u[i]);
        }
    }
}

// ---------------------------------------------------------------- gradient of g

// The gradient of g_t is the sum over u >= t of <q_u, dq_u> - <k_u, dk_u>, and <state, its
// gradient> behind the last token: what a change of every running sum from t on does.  Each of these
// differences is off by its terms' rounding, and a sum over the rest of the sequence by the root of its length
// times that.  So the sum runs to the next of the marks, kMark tokens apart, where the sweeps leave the state and
// its gradient, and their product is what all behind it comes to.  The mark in front gives the sum over the run
// between them once more (the first run's mark is the state that was given): what it is off by there is taken back
// evenly over the run's tokens.  8 x 1024 tokens, 32 heads of 64 that decay by exp(-0.05) to exp(-0.8) a token: a
// relative error of 7.6e-7, with one sum over the sequence 1.9e-6, for 1 % of the call's time (heads of 128, whose
// states are larger: 4 %).  In 64 bits.
__device__ __forceinline__ double block_sum(double v, double* sums, int threads) {
    const int lane = threadIdx.x & 63;
    const double in = running_sum(v, lane);
    __syncthreads();
    if (lane == 63) sums[threadIdx.x >> 6] = in;
    __syncthreads();
    v = 0.0;
    for (int i = 0; i < threads / 64; ++i) v += sums[i];
    return v;
}
// products [B, H, runs - 1]: <state, its gradient> at the marks, `elems` of both in one order.
__global__ __launch_bounds__(kThreads) void mark_kernel(const float* state, const float* grad, Chunks w, int elems, double* products) {
    __shared__ double sums[kThreads / 64];
    const int run = int(blockIdx.x % (w.runs - 1)) + 1;
    const int64_t bh = blockIdx.x / (w.runs - 1), at = int64_t(blockIdx.x) * elems;
    double v = 0.0;
    if (run * kMark < seq_length(w.lengths, bh / w.H, w.T))
        #pragma unroll 4
        for (int i = threadIdx.x * 4; i < elems; i += kThreads * 4) {
            const float4 x = *reinterpret_cast<const float4*>(state + at + i), y = *reinterpret_cast<const float4*>(grad + at + i);
            v += double(x.x) * y.x + double(x.y) * y.y + (double(x.z) * y.z + double(x.w) * y.w);
        }
    v = block_sum(v, sums, kThreads);
    if (threadIdx.x == 0) products[blockIdx.x] = v;
}
// A thread per token, from a run's last to its first.  start, end [B, H]: <state, its gradient> in front of the
// first token and behind the last, or null (0).
__global__ __launch_bounds__(kMark) void dg_kernel(const float* qd, const float* kd, const double* start, const double* end, const double* products, Chunks w,
                                                   float* dg, float* part) {
    __shared__ double sums[kMark / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int run = int(blockIdx.x % w.runs);
    const int64_t bh = blockIdx.x / w.runs, b = bh / w.H;
    const int h = int(bh % w.H), first = run * kMark, t = first + kMark - 1 - tid;
    const int len = seq_length(w.lengths, b, w.T), count = min(len - first, kMark);
    const double d = t < len ? double(qd[bh * w.T + t]) - double(kd[bh * w.T + t]) : 0.0;
    const double in = running_sum(d, lane);
    if (lane == 63) sums[wave] = in;
    __syncthreads();
    double before = in, all = 0.0;
    for (int i = 0; i < kMark / 64; ++i) {
        if (i < wave) before += sums[i];
        all += sums[i];
    }
    const double* marks = products + bh * (w.runs - 1);   // of run 1 and on
    const double behind = len - first > kMark ? marks[run] : end ? end[bh] : 0.0;
    const double off = all + behind - (run > 0 ? marks[run - 1] : start ? start[bh] : 0.0);
    double total = 0.0;
    if (t < w.T) {
        const float g = w.g_per_token ? w.g[(b * w.T + t) * w.H + h] : w.g[h];
        const bool none = t >= len || double(g) * 1.4426950408889634074 < kNoDecayLog2;
        total = none ? 0.0 : before + behind - off * (double(count - (t - first)) / count);
        if (w.g_per_token) dg[(b * w.T + t) * w.H + h] = float(total);
    }
    if (!w.g_per_token) {
        total = block_sum(total, sums, kMark);
        if (tid == 0) part[bh * w.runs + run] = float(total);
    }
}
// part [B, H, runs] -> dg [H]; a wave per head.
__global__ __launch_bounds__(64) void dg_heads_kernel(const float* part, float* dg, int B, int H, int runs) {
    const int h = blockIdx.x, lane = threadIdx.x;
    double s = 0.0;
    for (int64_t i = lane; i < int64_t(B) * runs; i += 64) s += part[(i / runs * H + h) * runs + i % runs];
    s = running_sum(s, lane);
    if (lane == 63) dg[h] = float(s);
}

// ---------------------------------------------------------------- sums over shared heads

// out [rows, heads, D] = the sum over each head's H / heads gradients in x [rows, H, D], in their order.  In
// fours, 2 x 16384 tokens of 8 heads of 128: 110 us, 5.5 TB/s.
template <int E>
__global__ __launch_bounds__(kThreads) void shared_sum_kernel(const float* x, void* out, int64_t items, int group, int D, bool bf16) {
    const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= items) return;
    const int64_t at = i * E, head = at / D;
    const float* p = x + head * group * D + at % D;
    float s[E] = {};
    for (int j = 0; j < group; ++j) {
        const Pack<float, E> v = ld_pack<E>(p + int64_t(j) * D, true, E);
        #pragma unroll
        for (int e = 0; e < E; ++e) s[e] += v.e[e];
    }
    st_pack_as<E>(out, at, bf16, s, true, E);
}

// ---------------------------------------------------------------- step

// Columns of a state for a workgroup: 64, or 16 where that is needed to occupy the chip.
// A thread has 4 columns (VEC: in one piece) of every RG-th row; the state is read once, kept in
// registers and written once, everything else is small beside it.  256 rows of 64 heads of 64: 110 us, 4.4 TB/s.
template <typename T, int CB, int ROWS, bool VEC>
__global__ __launch_bounds__(kThreads) void step_kernel(LinAttnParams p) {
    constexpr int CL = CB / 4, RG = kThreads / CL, N = ROWS / RG;
    __shared__ float part[kThreads / 64][CB];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int blocks = (p.Dv + CB - 1) / CB;
    const int64_t item = xcd_order(blockIdx.x, gridDim.x);
    const int cb = int(item % blocks), h = int(item / blocks % p.H), b = int(item / blocks / p.H);
    const int j = cb * CB + tid % CL * 4, r0 = tid / CL, Dk = p.Dk, Dv = p.Dv;
    const int slot = p.index ? p.index[b] : b;
    bool mine[1] = {slot >= 0 && slot < p.S};
    float* st = p.s1 + (int64_t(mine[0] ? slot : 0) * p.H + h) * Dk * Dv;
    const T* q = static_cast<const T*>(p.q) + (int64_t(b) * p.Hq + h / (p.H / p.Hq)) * Dk;
    const T* k = static_cast<const T*>(p.k) + (int64_t(b) * p.Hk + h / (p.H / p.Hk)) * Dk;
    const T* v = static_cast<const T*>(p.v) + (int64_t(b) * p.Hv + h / (p.H / p.Hv)) * Dv;
    Pack<float, 4> s[N];
    float qi[N], ki[N], vj[4], y[4] = {};
    if (mine[0] && j < Dv) {
        #pragma unroll
        for (int n = 0; n < N; ++n) {
            const int i = r0 + n * RG;
            if (i < Dk) s[n] = ld_pack<4>(st + i * Dv + j, VEC, Dv - j);
        }
    }
    #pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = r0 + n * RG;
        qi[n] = i < Dk ? widen(q[i]) : 0.f;
        ki[n] = i < Dk ? widen(k[i]) : 0.f;
    }
    #pragma unroll
    for (int e = 0; e < 4; ++e) vj[e] = j + e < Dv ? widen(v[j + e]) : 0.f;
    const float a = expf(p.g_per_token ? p.g[int64_t(b) * p.H + h] : p.g[h]);
    if (p.index) first_of_slots<1>(p.index, b, &slot, mine, kThreads);
    if (mine[0] && j < Dv) {
        #pragma unroll
        for (int n = 0; n < N; ++n) {
            const int i = r0 + n * RG;
            if (i >= Dk) continue;
            float o[4];
            #pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[e] = fmaf(a, s[n].e[e], ki[n] * vj[e]);
                y[e] = fmaf(qi[n], o[e], y[e]);
            }
            st_pack<4>(st + i * Dv + j, o, VEC, Dv - j);
        }
    }
    #pragma unroll
    for (int e = 0; e < 4; ++e)
        #pragma unroll
        for (int m = CL; m < 64; m *= 2) y[e] += __shfl_xor(y[e], m);
    if (lane < CL)
        #pragma unroll
        for (int e = 0; e < 4; ++e) part[wave][lane * 4 + e] = y[e];
    __syncthreads();
    if (tid < CB && cb * CB + tid < Dv) {
        const float sum = p.scale * (part[0][tid] + part[1][tid] + (part[2][tid] + part[3][tid]));
        const int64_t o = (int64_t(b) * p.H + h) * Dv + cb * CB + tid;
        if (p.y_bf16) static_cast<bf16_t*>(p.y)[o] = f32_to_bf16(mine[0] ? sum : 0.f);
        else static_cast<float*>(p.y)[o] = mine[0] ? sum : 0.f;
    }
}

int step_columns(const LinAttnParams& p) { return int64_t(p.B) * p.H * ((p.Dv + 63) / 64) >= 512 ? 64 : 16; }

template <typename T, int CB>
hipError_t step_rows(const LinAttnParams& p, dim3 grid, hipStream_t st) {
    if (p.Dk <= 64) {
        if (p.Dv % 4 == 0) step_kernel<T, CB, 64, true><<<grid, kThreads, 0, st>>>(p);
        else step_kernel<T, CB, 64, false><<<grid, kThreads, 0, st>>>(p);
    } else {
        if (p.Dv % 4 == 0) step_kernel<T, CB, 128, true><<<grid, kThreads, 0, st>>>(p);
        else step_kernel<T, CB, 128, false><<<grid, kThreads, 0, st>>>(p);
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------- how a call is split up

// Sequences are cut into segments, computed side by side, where their heads alone do not occupy the
// chip.  The number is the one with the least time by what was measured (in 0.1 us): a workgroup by
// itself takes `lat` for a chunk, several on a compute unit `thr` each, and about two chunks' time goes
// before the first; more than one segment costs a pass over two of the operands and the joining of the states.
// us by the number of segments, bf16:
//   forward   1 x 2048, 32 heads of 128   1: 172   4: 73    6: 60   8: 52   16: 60
//             4 x 4096, 40 heads of 64    1: 232   2: 202   3: 136  4: 153  8: 142
//             8 x 1024, 32 heads of 64    1: 52    2: 50    4: 57
//             1 x 65536, 16 heads of 64   8: 546   16: 295  32: 213
//   backward  2 x 2048, 32 heads of 64    1: 123   2: 122   4: 90   8: 96   16: 114
//             4 x 1024, 32 heads of 128   1: 157   2: 190   4: 224
// The gradients are counted as one launch.  Of keys and values on different sides of 64 they are three, one
// after another, of a third of the workgroups each, which the rule does not know.
void plan(const LinAttnParams& p, int kinds, Chunks* w) {
    const int64_t heads = int64_t(p.B) * p.H, chunks = (int64_t(p.T) + 63) / 64;
    const bool wide = p.Dk > 64 || p.Dv > 64, both = p.Dk > 64 && p.Dv > 64;
    const int groups = both ? 2 : 3, lat = both ? 45 : wide ? 36 : 28, thr = both ? 36 : wide ? 28 : 20;
    auto rounds = [&](int64_t jobs, int64_t segs, int64_t each, int groups, int lat, int thr) {   // the fullest compute unit's
        int64_t time = 0;
        for (int64_t k = (jobs * segs + 255) / 256; k > 0; k -= groups) {
            const int64_t c = k < groups ? k : groups;
            time += (each + 2) * (c * thr > lat ? c * thr : lat);
            if (k > 64 * groups) return time * (k / groups);   // many rounds alike
        }
        return time;
    };
    int64_t best = 1, least = -1;
    for (int64_t segs = 1; segs <= chunks && segs <= 64 && (segs == 1 || heads * kinds < 768); ++segs) {
        const int64_t each = (chunks + segs - 1) / segs;
        if (segs > 1 && (chunks + each - 1) / each != segs) continue;   // the same as fewer
        int64_t time = rounds(heads * kinds, segs, each, groups, lat, thr);
        if (segs > 1) time += (kinds > 1 ? 2 : 1) * (rounds(heads, segs - 1, each, 2, both ? 28 : 12, both ? 22 : 8) + heads * segs * p.Dk * p.Dv / 200000) + 60;
        if (least < 0 || time < least) {
            least = time;
            best = segs;
        }
    }
    const int64_t each = chunks > 0 ? (chunks + best - 1) / best : 1;
    const int least_heads = p.Hq < p.Hk ? (p.Hq < p.Hv ? p.Hq : p.Hv) : (p.Hk < p.Hv ? p.Hk : p.Hv), group = p.H ? p.H / least_heads : 1;
    *w = Chunks{p.B, p.T, p.H, group, int((int64_t(p.T) + kMark - 1) / kMark), int(best), int(each * 64), p.g_per_token, p.g, p.lengths, false};
    // Either each workgroup adds up the states of the segments before its own or, if there are more, a launch
    // does it for all (and where a state is moved in place, since a segment's workgroup would write it while
    // others still read it).  The gradients read two of three states transposed, a fourth of the speed.  1 x
    // 4096, 16 heads of 64: forward 8 segments 43 us without the launch, 42 with it, 16 35 and 31; backward 2
    // 189 and 194, 4 111 and 109, 8 89 and 77.  1 x 2048, 32 heads of 128, forward: 8 52 and 55, 16 70 and 60.
    w->chained = best > (kinds > 1 ? 2 : 8) || (best > 1 && p.s0 && p.s0 == p.s1);
}

// A state as the sweeps' waves hold it: at widths of 64 or 128.
int mark_elems(const LinAttnParams& p) { return (p.Dk > 64 ? 128 : 64) * (p.Dv > 64 ? 128 : 64); }

struct Carve {   // pieces of a workspace
    char* base;
    int64_t at = 0;
    float* floats(int64_t n) {
        float* r = base ? reinterpret_cast<float*>(base + at) : nullptr;   // (a size query has no base)
        at += (n * 4 + 255) / 256 * 256;
        return r;
    }
};
struct ForwardWs {
    float *states, *kept;
    int64_t bytes;
    ForwardWs(const LinAttnParams& p, const Chunks& w, void* ws) {
        Carve c{static_cast<char*>(ws)};
        const int64_t n = w.segs > 1 ? int64_t(p.B) * p.H * w.segs : 0;
        states = c.floats(n * p.Dk * p.Dv);
        kept = c.floats(n);
        bytes = c.at;
    }
};
struct BackwardWs {
    float *qd, *kd, *part, *states[2], *kept[2], *dq, *dk, *dv;
    double *start, *end, *products;
    float* marked[2];   // [B, H, runs - 1, mark_elems]: states, and their gradients
    int64_t bytes;
    BackwardWs(const LinAttnParams& p, const Chunks& w, void* ws) {
        Carve c{static_cast<char*>(ws)};
        const int64_t bh = int64_t(p.B) * p.H, n = w.segs > 1 ? bh * w.segs : 0, marks = w.runs > 1 ? bh * (w.runs - 1) : 0;
        auto doubles = [&](int64_t n) { return reinterpret_cast<double*>(c.floats(2 * n)); };
        qd = c.floats(bh * p.T);
        kd = c.floats(bh * p.T);
        part = c.floats(bh * w.runs);
        start = doubles(bh);
        end = doubles(bh);
        products = doubles(marks);
        for (float*& m : marked) m = c.floats(marks * mark_elems(p));
        for (int i = 0; i < 2; ++i) {
            states[i] = c.floats(n * p.Dk * p.Dv);
            kept[i] = c.floats(n);
        }
        dq = c.floats(p.Hq < p.H ? bh * p.T * p.Dk : 0);
        dk = c.floats(p.Hk < p.H ? bh * p.T * p.Dk : 0);
        dv = c.floats(p.Hv < p.H ? bh * p.T * p.Dv : 0);
        bytes = c.at;
    }
};

hipError_t chain(const Chunks& w, const Chain& f, const Chain& r, int kinds, int elems, hipStream_t st) {
    // heads by 32768, the most that a grid's second dimension is asked for
    const int64_t bh = int64_t(w.B) * w.H;
    for (int64_t h0 = 0; h0 < bh; h0 += 32768) {
        const uint32_t n = uint32_t(bh - h0 < 32768 ? bh - h0 : 32768);
        auto from = [&](Chain c) {
            c.ws += h0 * w.segs * elems;
            c.kept += h0 * w.segs;
            c.first = c.first ? c.first + h0 * elems : nullptr;
            return c;
        };
        chain_kernel<<<dim3((elems + kThreads - 1) / kThreads, n, kinds), kThreads, 0, st>>>(from(f), kinds > 1 ? from(r) : from(f), w.segs, elems);
    }
    return hipGetLastError();
}

int64_t shared_sum_threads(int64_t rows, int heads, int D) { return (rows * heads * D / (D % 4 ? 1 : 4) + kThreads - 1) / kThreads * kThreads; }
hipError_t shared_sum(const float* x, void* out, int64_t rows, int heads, int group, int D, bool bf16, hipStream_t st) {
    const int64_t n = rows * heads * D;
    const uint32_t grid = uint32_t(shared_sum_threads(rows, heads, D) / kThreads);
    if (D % 4 == 0) shared_sum_kernel<4><<<grid, kThreads, 0, st>>>(x, out, n / 4, group, D, bf16);
    else shared_sum_kernel<1><<<grid, kThreads, 0, st>>>(x, out, n, group, D, bf16);
    return hipGetLastError();
}

#define TRY(call)                            \
    do {                                     \
        const hipError_t e_ = (call);        \
        if (e_ != hipSuccess) return e_;     \
    } while (0)

}  // namespace
}  // namespace linattn

using namespace linattn;

int64_t linattn_forward_workspace(const LinAttnParams& p) {
    Chunks w;
    plan(p, 1, &w);
    return ForwardWs(p, w, nullptr).bytes;
}
int64_t linattn_backward_workspace(const LinAttnParams& p) {
    if (int64_t(p.B) * p.T * p.H == 0) return 0;
    Chunks w;
    plan(p, 3, &w);
    return BackwardWs(p, w, nullptr).bytes;
}
int64_t linattn_forward_threads(const LinAttnParams& p) {
    Chunks w;
    plan(p, 1, &w);
    return int64_t(p.B) * p.H * w.segs * 512;
}
int64_t linattn_step_threads(const LinAttnParams& p) {
    const int cb = step_columns(p);
    return int64_t(p.B) * p.H * ((p.Dv + cb - 1) / cb) * kThreads;
}
int64_t linattn_backward_threads(const LinAttnParams& p) {
    Chunks w;
    plan(p, 3, &w);
    // the sweeps together, the gradient of g, and the sums over heads that share an operand
    int64_t most = int64_t(p.B) * p.H * w.segs * 3 * 512;
    auto at_least = [&](int64_t n) { most = n > most ? n : most; };
    at_least(int64_t(p.B) * p.H * w.runs * kMark);
    auto sums = [&](int heads, int D) { at_least(heads < p.H ? shared_sum_threads(int64_t(p.B) * p.T, heads, D) : 0); };
    sums(p.Hq, p.Dk);
    sums(p.Hk, p.Dk);
    sums(p.Hv, p.Dv);
    return most;
}

hipError_t launch_linattn_forward(const LinAttnParams& p, hipStream_t st) {
    Chunks w;
    plan(p, 1, &w);
    const ForwardWs ws(p, w, p.ws);
    Sweep s{};
    s.a = {p.q, p.Hq, p.Dk, p.in_bf16};
    s.b = {p.k, p.Hk, p.Dk, p.in_bf16};
    s.c = {p.v, p.Hv, p.Dv, p.in_bf16};
    s.out = p.y; s.out_heads = p.H; s.out_bf16 = p.y_bf16;
    s.sp = s.si = p.scale; s.su = 1.f;
    s.ws = ws.states; s.kept = ws.kept;
    s.s_in = p.s0; s.s_out = p.s1;
    if (w.segs > 1) {
        TRY(p.in_bf16 ? parts_bf16(w, s, st) : parts_f32(w, s, st));
        if (w.chained) TRY(chain(w, {ws.states, ws.kept, p.s0}, {}, 1, p.Dk * p.Dv, st));
    }
    return p.in_bf16 ? forward_bf16(w, s, st) : forward_f32(w, s, st);
}

hipError_t launch_linattn_step(const LinAttnParams& p, hipStream_t st) {
    const int cb = step_columns(p);
    const dim3 grid(uint32_t(int64_t(p.B) * p.H * ((p.Dv + cb - 1) / cb)));
    if (cb == 64) return p.in_bf16 ? step_rows<bf16_t, 64>(p, grid, st) : step_rows<float, 64>(p, grid, st);
    return p.in_bf16 ? step_rows<bf16_t, 16>(p, grid, st) : step_rows<float, 16>(p, grid, st);
}

hipError_t launch_linattn_backward(const LinAttnParams& p, hipStream_t st) {
    Chunks w;
    plan(p, 3, &w);
    const int64_t rows = int64_t(p.B) * p.T;
    const BackwardWs ws(p, w, rows > 0 ? p.ws : nullptr);   // without tokens none is needed: what is given may be of any size
    const bool bf16 = p.in_bf16 && p.y_bf16;
    const Operand q{p.q, p.Hq, p.Dk, p.in_bf16}, k{p.k, p.Hk, p.Dk, p.in_bf16}, v{p.v, p.Hv, p.Dv, p.in_bf16}, dy{p.dy, p.H, p.Dv, p.y_bf16};
    // a gradient goes to its place, or, where heads share one, each head's to the workspace
    if (p.B == 0) {
        if (p.dg && !p.g_per_token) dg_heads_kernel<<<p.H, 64, 0, st>>>(ws.part, p.dg, 0, p.H, 1);
        return hipGetLastError();
    }
    auto make = [&](const Operand& a, const Operand& b, const Operand& c, void* out, float* each, int heads, bool back, bool transposed) {
        Sweep s{};
        s.a = a; s.b = b; s.c = c;
        const bool shared = heads < p.H;
        s.out = shared ? each : out; s.out_heads = p.H; s.out_bf16 = !shared && p.in_bf16;
        s.sp = p.scale; s.si = back ? 1.f : p.scale; s.su = back ? p.scale : 1.f;
        s.ws = ws.states[back]; s.kept = ws.kept[back];
        s.s_in = back ? p.ds1 : p.s0;
        s.back = back; s.transposed = transposed;
        return s;
    };
    Sweep sq = make(dy, v, k, p.dq, ws.dq, p.Hq, false, true);
    Sweep sk = make(v, dy, q, p.dk, ws.dk, p.Hk, true, true);
    Sweep sv = make(k, q, dy, p.dv, ws.dv, p.Hv, true, false);
    if (p.dg) {
        sq.x = q; sq.dot = ws.qd;
        sk.x = k; sk.dot = ws.kd;
        if (w.runs > 1) {
            sq.marks = ws.marked[0];
            sk.marks = ws.marked[1];
        }
        sq.end_with = p.ds1; sq.end_dot = p.ds1 ? ws.end : nullptr;
        sk.end_with = p.s0; sk.end_dot = p.s0 ? ws.start : nullptr;
    }
    if (w.segs > 1) {
        Sweep f = sv;
        f.b = k; f.c = v; f.back = false; f.su = 1.f; f.ws = ws.states[0]; f.kept = ws.kept[0];
        TRY(bf16 ? parts_bf16(w, f, st) : parts_f32(w, f, st));
        TRY(bf16 ? parts_bf16(w, sv, st) : parts_f32(w, sv, st));
        if (w.chained) TRY(chain(w, {ws.states[0], ws.kept[0], p.s0}, {ws.states[1], ws.kept[1], p.ds1}, 2, p.Dk * p.Dv, st));
    }
    sv.s_out = p.ds0;
    TRY(bf16 ? backward_bf16(w, sq, sk, sv, st) : backward_f32(w, sq, sk, sv, st));
    if (p.Hq < p.H && rows > 0) TRY(shared_sum(ws.dq, p.dq, rows, p.Hq, p.H / p.Hq, p.Dk, p.in_bf16, st));
    if (p.Hk < p.H && rows > 0) TRY(shared_sum(ws.dk, p.dk, rows, p.Hk, p.H / p.Hk, p.Dk, p.in_bf16, st));
    if (p.Hv < p.H && rows > 0) TRY(shared_sum(ws.dv, p.dv, rows, p.Hv, p.H / p.Hv, p.Dv, p.in_bf16, st));
    if (p.dg) {
        const uint32_t jobs = uint32_t(int64_t(p.B) * p.H * w.runs);
        if (w.runs > 1) mark_kernel<<<jobs - jobs / w.runs, kThreads, 0, st>>>(ws.marked[0], ws.marked[1], w, mark_elems(p), ws.products);
        if (rows > 0) dg_kernel<<<jobs, kMark, 0, st>>>(ws.qd, ws.kd, sk.end_dot, sq.end_dot, ws.products, w, p.dg, ws.part);
        if (!p.g_per_token) dg_heads_kernel<<<p.H, 64, 0, st>>>(ws.part, p.dg, rows > 0 ? p.B : 0, p.H, rows > 0 ? w.runs : 1);
    }
    return hipGetLastError();
}

}  // namespace wkv7
