// Internal interface between the C-ABI entry points of the per-channel
// operators (seq_api.cpp) and their kernel launchers (ssm_scan.hip,
// ssm_backward.hip, shortconv.hip, groupnorm.hip).  The structures hold
// validated arguments and go to the kernels as they are.
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

#include "../../include/ssm.h"
#include "../../include/shortconv.h"
#include "../../include/groupnorm.h"

namespace wkv7 {

struct SsmParams {
    int B, T, C, N, G, S;
    bool in_bf16, y_bf16, softplus;
    const int32_t *lengths, *index;   // null: all of T; null: state b
    const void *x, *dt, *z, *Bm, *Cm;
    const float *A, *D, *dt_bias, *s0;
    void* y;
    float *s1, *ck;
    int nck;                          // checkpoints of a sequence
    bool vec_n;                       // set by the step's launcher: runs of 4 states are aligned
    // backward
    const void* dy;
    const float* ds1;
    void *dx, *ddt, *dz, *dBm, *dCm;
    float *dA, *dD, *dbias, *ds0;
    void* ws;
};
// Rows of channels, of every group and in each type that a kernel moves them in, start on 4 bytes.
inline bool channels_on_words(const SsmParams& p) { return (!p.in_bf16 && !p.y_bf16) || (p.C % 2 == 0 && p.C / p.G % 2 == 0); }
// The forward and the backward, with npl states of a lane: runs of channels and of states move as whole
// words, and no lane has only some of its states.
inline bool ssm_forward_words(const SsmParams& p, int npl) {
    return p.N % npl == 0 && (!p.in_bf16 || p.N % 2 == 0) && channels_on_words(p);
}
inline bool ssm_backward_words(const SsmParams& p) { return p.N % 2 == 0 && channels_on_words(p); }
int64_t ssm_backward_workspace(const SsmParams& p, bool own_checkpoints);
// The threads of a call's largest launch: HIP takes less than 2^32.
int64_t ssm_forward_threads(const SsmParams& p);
int64_t ssm_step_threads(const SsmParams& p);
int64_t ssm_backward_threads(const SsmParams& p);
hipError_t launch_ssm_forward(const SsmParams& p, hipStream_t stream);
hipError_t launch_ssm_step(const SsmParams& p, hipStream_t stream);
hipError_t launch_ssm_backward(const SsmParams& p, hipStream_t stream);

struct ConvParams {
    int B, T, C, K, S;
    bool in_bf16, y_bf16, silu;
    const int32_t *lengths, *index;
    const void* x;
    const float *w, *bias;
    const void* s0;
    void *y, *s1;
    // backward
    const void* dy;
    const float* ds1;
    void* dx;
    float *dw, *dbias, *ds0;
    void* ws;
};
int64_t shortconv_backward_workspace(const ConvParams& p);
int64_t shortconv_forward_threads(const ConvParams& p);
int64_t shortconv_step_threads(const ConvParams& p);
int64_t shortconv_backward_threads(const ConvParams& p);
hipError_t launch_shortconv_forward(const ConvParams& p, hipStream_t stream);
hipError_t launch_shortconv_step(const ConvParams& p, hipStream_t stream);
hipError_t launch_shortconv_backward(const ConvParams& p, hipStream_t stream);

struct NormParams {
    int B, T, C, G;
    bool in_bf16, y_bf16, silu;
    float eps;
    const int32_t* lengths;
    const void *x, *gate;
    const float *weight, *bias;
    void* y;
    float *mean, *rstd;
    // backward
    const void* dy;
    void *dx, *dgate;
    float *dweight, *dbias;
    void* ws;
};
int64_t groupnorm_workspace(const NormParams& p);
int64_t groupnorm_backward_workspace(const NormParams& p);
int64_t groupnorm_threads(const NormParams& p, bool bwd);
hipError_t launch_groupnorm_forward(const NormParams& p, hipStream_t stream);
hipError_t launch_groupnorm_backward(const NormParams& p, hipStream_t stream);

}  // namespace wkv7
