// One element of the Adam step (Kingma & Ba, 2015), shared by the per-tensor
// and the many-tensor kernels so that both give the same bits.
#pragma once

#include <hip/hip_runtime.h>

namespace ia {

// p -= step_size * m / (sqrt(v * v_scale) + eps) after the moment updates;
// step_size = lr / (1 - b1^t), v_scale = 1 / (1 - b2^t) (host, double).
struct AdamConsts {
    float b1, b2, eps, v_scale;
};

__device__ __forceinline__ float adam_element(float p, float g, float& m, float& v, const AdamConsts& c,
                                              float step_size) {
    m = c.b1 * m + (1.0f - c.b1) * g;
    v = c.b2 * v + (1.0f - c.b2) * (g * g);
    return p - step_size * m / (sqrtf(v * c.v_scale) + c.eps);
}

}  // namespace ia
