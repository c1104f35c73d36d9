// What the translation units of the group-scaled 4-bit matrices share.
//
// Format: a row of `cols` values is ceil(cols / G) groups of G = 32, 64 or 128.
// A group has a scale s and a zero z in 0..15 and stands for s (q - z), q in
// 0..15; two codes q to a byte, the earlier one in the low half.  One 32-bit
// word holds both: s as a float whose lowest byte is zero (16 significant bits:
// every fp16 or bf16 scale, and (k + 1/2) s is exact in fp32) and z in that
// byte.  A row of words is padded to a multiple of four.
#pragma once

#include <hip/hip_runtime.h>

#include "mx4_common.h"
#include "philox.h"

namespace ia {

typedef _Float16 halfx2 __attribute__((ext_vector_type(2)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));
typedef __bf16 bfloatx2 __attribute__((ext_vector_type(2)));
typedef __bf16 bfloatx8 __attribute__((ext_vector_type(8)));

__host__ __device__ inline int64_t q4_groups(int64_t cols, int group) { return (cols + group - 1) / group; }
__host__ __device__ inline int64_t q4_word_stride(int64_t groups) { return (groups + 3) & ~(int64_t)3; }

__device__ __forceinline__ float scale_of(uint32_t word) { return __builtin_bit_cast(float, word & ~255u); }
__device__ __forceinline__ float zero_of(uint32_t word) { return (float)(word & 255u); }

// Eight codes as bytes.
struct Nibbles {
    uint32_t even, odd;

    __device__ __forceinline__ explicit Nibbles(uint32_t codes) {
        even = codes & 0x0f0f0f0fu;
        odd = (codes >> 4) & 0x0f0f0f0fu;
        // a byte is converted by one instruction as long as the compiler does not know that half of it is zero
        asm("" : "+v"(even), "+v"(odd));
    }
    // code 2 j + ODD
    template <int ODD>
    __device__ __forceinline__ float value(int j) const {
        return (float)(((ODD ? odd : even) >> (8 * j)) & 255u);
    }
};

// u (q - z) of eight codes, u a power of two from 2^-24 to 2^8, given as 512 u, and
// zu = -z u twice: exact in fp16, which ends at 2^-24 and 2^16.
__device__ __forceinline__ halfx8 codes_times(uint32_t codes, float u512, halfx2 zu) {
    // e4m3's values of the bytes 0..15 are 0..15 times 2^-9: the scaled conversion reads them as whole numbers
    const uint32_t even = codes & 0x0f0f0f0fu, odd = (codes >> 4) & 0x0f0f0f0fu;
    const int lo = (int)__builtin_amdgcn_perm(odd, even, 0x05010400u), hi = (int)__builtin_amdgcn_perm(odd, even, 0x07030602u);
    halfx2 h[4] = {__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, u512, false), __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, u512, true),
                   __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, u512, false), __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, u512, true)};
    halfx8 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        h[j] += zu;
        r[2 * j] = h[j][0];
        r[2 * j + 1] = h[j][1];
    }
    return r;
}
__device__ __forceinline__ halfx2 twice(float v) { return halfx2{(_Float16)v, (_Float16)v}; }
// u (q - z) of eight codes, u a power of two and zu = -z u (exact but for u under 2^-133).
__device__ __forceinline__ bfloatx8 codes_times(uint32_t codes, float u, float zu) {
    const Nibbles n(codes);
    bfloatx8 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const floatx2 v = {__builtin_fmaf(n.value<0>(j), u, zu), __builtin_fmaf(n.value<1>(j), u, zu)};
        const bfloatx2 w = __builtin_convertvector(v, bfloatx2);
        r[2 * j] = w[0];
        r[2 * j + 1] = w[1];
    }
    return r;
}

template <typename T>
struct Raw {
    T v[8];
};

// count of them exist (0 or less: none)
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p, int64_t count) {
    Raw<T> r;
    if (count >= 8) {
        __builtin_memcpy(&r, p, sizeof(r));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = j < count ? p[j] : (T)0.0f;
    }
    return r;
}

// The operand's parts, largest first: cut off, so that they add up to the value (to
// within 2^-133, where bf16 ends).
__device__ __forceinline__ void split(const Raw<_Float16>& r, halfx8 (&p)[1]) { __builtin_memcpy(&p[0], &r, sizeof(r)); }
__device__ __forceinline__ void split(const Raw<__bf16>& r, bfloatx8 (&p)[1]) { __builtin_memcpy(&p[0], &r, sizeof(r)); }
__device__ __forceinline__ void split(const Raw<float>& r, bfloatx8 (&p)[3]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float v = r.v[j];
        const uint32_t b = __builtin_bit_cast(uint32_t, v);
        const bool finite = (b & 0x7f800000u) != 0x7f800000u;
        const uint32_t h0 = v != v ? 0x7fc00000u : b & 0xffff0000u;
        const float r1 = finite ? v - __builtin_bit_cast(float, h0) : 0.0f;
        const uint32_t h1 = __builtin_bit_cast(uint32_t, r1) & 0xffff0000u;
        const float r2 = r1 - __builtin_bit_cast(float, h1);
        p[0][j] = __builtin_bit_cast(__bf16, (uint16_t)(h0 >> 16));
        p[1][j] = __builtin_bit_cast(__bf16, (uint16_t)(h1 >> 16));
        p[2][j] = __builtin_bit_cast(__bf16, (uint16_t)(__builtin_bit_cast(uint32_t, r2) >> 16));
    }
}

struct Q4Linear {
    const uint8_t* codes;
    const uint32_t* words;
    int64_t N, K, groups;
    const float* bias;
    int act;
    void* y;
    int64_t ldy;
};

// Many rows, in tiles (q4_matmul.hip), where that is faster; the workspace holds
// rows of x that cannot be read as they are, and the sums of splits.
bool q4_takes_tiles(int32_t dtype, int group, int64_t M, int64_t K, int64_t N);
size_t q4_matmul_workspace(int32_t dtype, int64_t M, int64_t K, int64_t N);
hipError_t launch_q4_matmul(const void* x, int32_t dtype, int64_t M, int64_t ldx, int group, const Q4Linear& p, void* ws,
                            hipStream_t s);

}  // namespace ia
