// Dropout of a matrix: out = x / (1 - p) where kept, else 0, with a mask that
// is computed from the place of a value (philox.h) and stored nowhere.  The
// gradient is the same call on the upstream gradient.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "mx4_common.h"
#include "philox.h"

namespace ia {
namespace {

// A thread takes eight values of a row: two counters give their eight words.
// Rows from row0 on, fewer than 2^31 threads.  300,000 x 256 fp16 values (307 MB) take
// 54 us (5.7 TB/s, a copy 6.2); the generator's multiplications alone, at a quarter
// of the rate of other instructions, keep the SIMDs busy for about as long.
template <typename T>
__global__ void __launch_bounds__(256) dropout_kernel(const T* x, int64_t ldx, T* out, int64_t ldo, uint32_t row0,
                                                      uint32_t rows, uint32_t cols, Divisor chunks, float factor, bool stream, DropArgs a) {
    const uint32_t i = blockIdx.x * 256u + threadIdx.x, k = chunks.of(i), r = row0 + k, c = (i - k * chunks.d) * 8;
    if (k >= rows) return;
    const Dropper drop(a);
    const T* const from = x + r * ldx + c;
    T* const to = out + r * ldo + c;
    float v[8];
    if (c + 8 <= cols) {
        load8(from, 8, v);
        drop.apply(v, r, c, factor);
        store8(to, 8, v, stream);
    } else {
        load8(from, (int64_t)cols - c, v);
        drop.apply(v, r, c, factor);
        store8(to, (int64_t)cols - c, v);
    }
}

template <typename T>
hipError_t launch(const void* x, int64_t ldx, void* out, int64_t ldo, int64_t rows, int64_t cols, float factor,
                  const DropArgs& a, hipStream_t s) {
    const Divisor chunks((uint32_t)ceil_div(cols, 8));
    const int64_t most = (((int64_t)1 << 31) - 256) / chunks.d;
    for (int64_t r = 0; r < rows; r += most) {
        const int64_t here = std::min(most, rows - r);
        IA_LAUNCH("dropout_kernel", dropout_kernel<T>, dim3((unsigned)ceil_div(here * chunks.d, 256)), dim3(256), 0, s,
                  (const T*)x, ldx, (T*)out, ldo, (uint32_t)r, (uint32_t)here, (uint32_t)cols, chunks, factor,
                  rows * cols * (int64_t)sizeof(T) >= kStreamBytes, a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx, const DropArgs& a,
                          float factor, void* out, int64_t ldo, hipStream_t s) {
    if (rows == 0 || cols == 0) return hipSuccess;
    return IA_BY_DTYPE(dtype, launch, x, ldx, out, ldo, rows, cols, factor, a, s);
}

}  // namespace ia
