// Dropout of a matrix: out = x / (1 - p) where kept, else 0, with a mask that
// is computed from the place of a value (philox.h) and stored nowhere.  The
// gradient is the same call on the upstream gradient.
#include <hip/hip_runtime.h>

#include "mx4_common.h"
#include "philox.h"

namespace ia {
namespace {

// A thread takes eight values of a row: two counters give their eight words.
template <typename T>
__global__ void __launch_bounds__(256) dropout_kernel(const T* x, int64_t ldx, T* out, int64_t ldo, int64_t rows,
                                                      uint32_t cols, float factor, DropArgs a) {
    const uint32_t chunks = (cols + 7) / 8;
    const int64_t total = rows * chunks;
    const Dropper drop(a);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const uint32_t r = (uint32_t)(i / chunks), c = (uint32_t)(i - (int64_t)r * chunks) * 8;
        float v[8];
        load8(x + (int64_t)r * ldx + c, (int64_t)cols - c, v);
        drop.apply(v, r, c, factor);
        store8(out + (int64_t)r * ldo + c, (int64_t)cols - c, v);
    }
}

template <typename T>
hipError_t launch(const void* x, int64_t ldx, void* out, int64_t ldo, int64_t rows, int64_t cols, float factor,
                  const DropArgs& a, hipStream_t s) {
    IA_LAUNCH("dropout_kernel", dropout_kernel<T>, dim3(grid_for(rows * ceil_div(cols, 8))), dim3(256), 0, s,
              (const T*)x, ldx, (T*)out, ldo, rows, (uint32_t)cols, factor, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx, const DropArgs& a,
                          float factor, void* out, int64_t ldo, hipStream_t s) {
    if (rows == 0 || cols == 0) return hipSuccess;
    return IA_BY_DTYPE(dtype, launch, x, ldx, out, ldo, rows, cols, factor, a, s);
}

}  // namespace ia
