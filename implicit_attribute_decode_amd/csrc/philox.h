// Philox4x32-10, the counter-based generator of Salmon, Moraes, Dror & Shaw,
// "Parallel random numbers: as easy as 1, 2, 3" (SC 2011): four words from a
// counter of four words and a key of two, with no state between calls.
//
// Dropout's use of it: value (r, c) of a matrix takes word c mod 4 of the
// counter (c / 4, r, offset low, offset high) under the key `seed`, so the mask
// of a value depends on its place alone, not on strides, alignment or the shape
// of a launch, and is computed again wherever it is needed.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ia_internal.h"

namespace ia {

struct Words4 {
    uint32_t w[4];
};

__device__ __forceinline__ Words4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int round = 0; round < 10; ++round) {
        const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return Words4{{c0, c1, c2, c3}};
}

// What a kernel needs of a dropout: `limit` = p 2^32 rounded (2^32 keeps
// nothing), the key, the call's number and, where not null, a number in device
// memory that is added to it.
struct DropArgs {
    uint64_t limit, seed, offset;
    const int64_t* step;
};

// The call's number is read once by a thread, before its loop.
struct Dropper {
    uint64_t limit;
    uint32_t k0, k1, o0, o1;

    __device__ __forceinline__ explicit Dropper(const DropArgs& a) {
        const uint64_t o = a.offset + (a.step ? (uint64_t)a.step[0] : 0u);
        limit = a.limit;
        k0 = (uint32_t)a.seed;
        k1 = (uint32_t)(a.seed >> 32);
        o0 = (uint32_t)o;
        o1 = (uint32_t)(o >> 32);
    }
    // zero where dropped, for values c .. c + 3 of row r (c a multiple of 4)
    template <typename V>
    __device__ __forceinline__ void apply(V& v, uint32_t r, uint32_t c) const {
        const Words4 x = philox(c >> 2, r, o0, o1, k0, k1);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = x.w[j] >= limit ? v[j] : 0.0f;
    }
    // v times factor where kept, else 0, for values c0 .. c0 + 7 of row r (c0 a multiple of 8)
    __device__ __forceinline__ void apply(float (&v)[8], uint32_t r, uint32_t c0, float factor) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const Words4 x = philox((c0 >> 2) + h, r, o0, o1, k0, k1);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * h + j] = x.w[j] >= limit ? v[4 * h + j] * factor : 0.0f;
        }
    }
};

// Eight consecutive values as floats; `count` of them exist, the rest are zero.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int64_t count, float (&v)[8]) {
    if (count >= 8) {
        T t[8];
        __builtin_memcpy(t, p, sizeof(t));
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (float)t[j];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < count ? (float)p[j] : 0.0f;
    }
}

// The first `count` of eight values, each rounded once.
template <typename T>
__device__ __forceinline__ void store8(T* p, int64_t count, const float (&v)[8]) {
    if (count >= 8) {
        T t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = (T)v[j];
        __builtin_memcpy(p, t, sizeof(t));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < count) p[j] = (T)v[j];
    }
}

}  // namespace ia
