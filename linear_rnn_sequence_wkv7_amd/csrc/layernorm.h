// Internal interface of the layer norm: the entry points' validated arguments and its launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace wkv7 {

struct LayerNormParams {
    int B, T, C;
    bool x_bf16, h_bf16, y_bf16;
    float eps;
    const int32_t* lengths;
    const void *x, *res;
    const float *weight, *bias;
    void *h, *y;
    float *mean, *rstd;
    // backward (h is read)
    const void *dy, *dh;
    void *dres, *dx;
    float *dweight, *dbias;
    void* ws;
};
int64_t layernorm_backward_workspace(const LayerNormParams& p);
int64_t layernorm_threads(const LayerNormParams& p, bool bwd);
hipError_t launch_layernorm_forward(const LayerNormParams& p, hipStream_t stream);
hipError_t launch_layernorm_backward(const LayerNormParams& p, hipStream_t stream);

}  // namespace wkv7
