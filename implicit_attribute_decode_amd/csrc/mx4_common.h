// What the MXFP4 translation units share: the format's constants, the matrix
// instruction with E2M1 operands and the host's small arithmetic.
#pragma once

#include <hip/hip_runtime.h>

#include "ia_internal.h"

namespace ia {

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));
typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef uint32_t uintx4 __attribute__((ext_vector_type(4)));
typedef uint32_t loose_uintx4 __attribute__((ext_vector_type(4), aligned(2)));  // at any element
typedef unsigned short ushortx2 __attribute__((ext_vector_type(2)));

constexpr int kBlock = 32;  // values per scale
constexpr int kFp4 = 4;     // the MFMA's format code of E2M1
constexpr int kNaNByte = 255;

__device__ __forceinline__ intx8 widen(intx4 v) { return intx8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// 16 x 16 x 128; the first operand's scale in byte BYTE of its word, the
// second's in the lowest.
template <int BYTE>
__device__ __forceinline__ floatx4 mfma16(intx4 a, int as, intx4 b, int bs, floatx4 c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(a), widen(b), c, kFp4, kFp4, BYTE, as, 0, bs);
}

// 32 x 32 x 64; both scales in byte BYTE of their words.
template <int BYTE>
__device__ __forceinline__ floatx16 mfma32(intx4 a, int as, intx4 b, int bs, floatx16 c) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(a), widen(b), c, kFp4, kFp4, BYTE, as, BYTE, bs);
}

__device__ __forceinline__ float activate(float v, int act) {
    return act == IA_ACT_RELU && v < 0.0f ? 0.0f : v;  // a NaN stays
}

// Tile index of a block so that blocks of one XCD (every eighth block) take
// neighbouring tiles: runs of 8 tile rows, column by column.
__device__ __forceinline__ void tile_of(int64_t b, int64_t tm, int64_t tn, int64_t& im, int64_t& in) {
    const int64_t total = tm * tn, per = total / 8, rest = total % 8, x = b % 8;
    int64_t t = x * per + min(x, rest) + b / 8;
    const int64_t group = 8 * tn, g = t / group, h = min((int64_t)8, tm - 8 * g);
    t -= g * group;
    im = 8 * g + t % h;
    in = t / h;
}

// LDS written by the lanes of one wave is read back by other lanes of the same
// wave: order the accesses at wavefront scope.
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Every copy of this wave has landed, and every wave's after the barrier.
__device__ __forceinline__ void stage_barrier() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
}

// Row of block i of a matrix with `blocks` blocks a row, where i is at most 255
// past `base`, which is the same for all threads: one 64-bit division for the
// workgroup and a 32-bit one a thread.
__device__ __forceinline__ int64_t row_of(int64_t i, int64_t blocks, int64_t base) {
    const int64_t r = base / blocks;
    const int64_t k = i - r * blocks;
    return r + (blocks < ((int64_t)1 << 31) ? (int64_t)((uint32_t)k / (uint32_t)blocks) : k / blocks);
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t round_up(size_t n) { return (n + 255) & ~(size_t)255; }
inline int64_t mx4_blocks(int64_t cols) { return ceil_div(cols, kBlock); }

// Blocks of 256 threads for a grid-stride loop.
inline unsigned grid_for(int64_t threads) {
    const int64_t b = ceil_div(threads, 256);
    return (unsigned)(b < (int64_t)1 << 22 ? b : (int64_t)1 << 22);
}

#define IA_BY_DTYPE(dtype, fn, ...)                                   \
    ((dtype) == IA_DTYPE_F32   ? fn<float>(__VA_ARGS__)               \
     : (dtype) == IA_DTYPE_F16 ? fn<_Float16>(__VA_ARGS__)            \
                               : fn<__bf16>(__VA_ARGS__))

}  // namespace ia
