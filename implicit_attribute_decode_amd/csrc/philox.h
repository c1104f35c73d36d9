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
    uint32_t most;  // words up to it drop, unless none do
    bool none;
    uint32_t k0, k1, o0, o1;

    __device__ __forceinline__ explicit Dropper(const DropArgs& a) {
        const uint64_t o = a.offset + (a.step ? (uint64_t)a.step[0] : 0u);
        none = a.limit == 0;
        most = (uint32_t)(a.limit - 1);
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
        for (int j = 0; j < 4; ++j) v[j] = x.w[j] > most || none ? v[j] : 0.0f;
    }
    // v times factor where kept, else 0, for values c0 .. c0 + 7 of row r (c0 a multiple of 8)
    __device__ __forceinline__ void apply(float (&v)[8], uint32_t r, uint32_t c0, float factor) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const Words4 x = philox((c0 >> 2) + h, r, o0, o1, k0, k1);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * h + j] = x.w[j] > most || none ? v[4 * h + j] * factor : 0.0f;
        }
    }
};

// Division of numbers below 2^31 by a fixed one, which the host prepares: with
// 2^(l - 1) < d <= 2^l and m = ceil(2^(31 + l) / d), n m / 2^(31 + l) exceeds n / d by
// less than n / 2^31 / d, so by less than what is missing to the next whole number.
struct Divisor {
    uint32_t d, m, shift;

    explicit Divisor(uint32_t divisor) : d(divisor), m(0), shift(31) {
        while (((uint64_t)1 << (shift - 31)) < d) ++shift;
        m = (uint32_t)((((uint64_t)1 << shift) + d - 1) / d);
    }
    __device__ __forceinline__ uint32_t of(uint32_t n) const { return (uint32_t)((uint64_t)n * m >> shift); }
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

// Outputs of this many bytes and more go past the memory-side cache, which they
// would only sweep: 300,000 x 256 fp16 values with dropout 56 -> 54 us.
constexpr int64_t kStreamBytes = (int64_t)64 << 20;

// The first `count` of eight values, each rounded once.
template <typename T>
__device__ __forceinline__ void store8(T* p, int64_t count, const float (&v)[8], bool stream = false) {
    if (count >= 8) {
        T t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = (T)v[j];
        if (stream) {
            typedef uint32_t quad __attribute__((ext_vector_type(4)));
            typedef uint32_t loose_quad __attribute__((ext_vector_type(4), aligned(2)));  // at any element
            quad q[sizeof(t) / 16];
            __builtin_memcpy(q, t, sizeof(t));
#pragma unroll
            for (size_t j = 0; j < sizeof(t) / 16; ++j)
                __builtin_nontemporal_store(q[j], reinterpret_cast<loose_quad*>(p) + j);
        } else {
            __builtin_memcpy(p, t, sizeof(t));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < count) p[j] = (T)v[j];
    }
}

}  // namespace ia
