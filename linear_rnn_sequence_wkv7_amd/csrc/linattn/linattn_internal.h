// Internal interface of linear attention: the entry points' validated arguments, what a sweep
// over chunks is told (linattn_core.h) and its launchers, one pair per matrix-core opcode
// (linattn_bf16.hip, linattn_f32.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace wkv7 {

struct LinAttnParams {
    int B, T, H, Hq, Hk, Hv, Dk, Dv, S;
    bool in_bf16, y_bf16, g_per_token;
    float scale;
    const int32_t *lengths, *index;   // null: all of T; null: state b
    const void *q, *k, *v;
    const float *g, *s0;
    void* y;
    float* s1;
    // backward
    const void* dy;
    const float* ds1;
    void *dq, *dk, *dv;
    float *dg, *ds0;
    void* ws;
};
int64_t linattn_forward_workspace(const LinAttnParams& p);
int64_t linattn_backward_workspace(const LinAttnParams& p);
// The threads of a call's largest launch.
int64_t linattn_forward_threads(const LinAttnParams& p);
int64_t linattn_step_threads(const LinAttnParams& p);
int64_t linattn_backward_threads(const LinAttnParams& p);
hipError_t launch_linattn_forward(const LinAttnParams& p, hipStream_t stream);
hipError_t launch_linattn_step(const LinAttnParams& p, hipStream_t stream);
hipError_t launch_linattn_backward(const LinAttnParams& p, hipStream_t stream);

namespace linattn {

constexpr double kNoDecayLog2 = -2000.0;   // a log2 of a decay below this counts as -inf: it is 0 in fp32 by far

constexpr int kMark = 512;   // tokens; a multiple of every chunk's

struct Operand {   // [B, T, heads, D]
    const void* p;
    int heads, D;
    bool bf16;
};
struct Chunks {
    int B, T, H;
    int group;                // how many consecutive heads share an operand
    int runs;                 // of kMark tokens, the last one shorter
    int segs, seg_tokens;     // sequences are computed in parts side by side, of a multiple of 64 tokens
    bool g_per_token;
    const float* g;
    const int32_t* lengths;
    bool chained;             // the states before the segments are there; else each adds up the parts before it
};
struct Sweep {
    Operand a, b, c;
    Operand x;                // with dot: [B, H, T] sums of out x over the columns, before out is rounded
    void* out;                // [B, T, out_heads, c.D]
    float* dot;
    float* ws;                // [B, H, segs, Dk, Dv]: what segments add; chained: then the state before each
    float* kept;              // [B, H, segs]: what is left of a state behind each
    const float* s_in;        // [B, H, Dk, Dv] or null
    float* s_out;             // or null
    const float* end_with;    // with end_dot [B, H]: <the state that s_out would get, end_with>
    double* end_dot;
    float* marks;             // [B, H, runs - 1, widths' product] or null: the state in front of every run but the first, as waves hold it
    float sp, si, su;
    int out_heads;
    bool out_bf16, back, transposed;   // transposed: the state is stored [c.D][a.D]
};

hipError_t parts_bf16(const Chunks& w, const Sweep& s, hipStream_t st);
hipError_t parts_f32(const Chunks& w, const Sweep& s, hipStream_t st);
hipError_t forward_bf16(const Chunks& w, const Sweep& s, hipStream_t st);
hipError_t forward_f32(const Chunks& w, const Sweep& s, hipStream_t st);
hipError_t backward_bf16(const Chunks& w, const Sweep& q, const Sweep& k, const Sweep& v, hipStream_t st);
hipError_t backward_f32(const Chunks& w, const Sweep& q, const Sweep& k, const Sweep& v, hipStream_t st);

}  // namespace linattn
}  // namespace wkv7
