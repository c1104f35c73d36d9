// 4-bit weights with group scales (q4_common.h): quantisation, read-back and the
// product of a few unquantised rows with them.
#include <hip/hip_runtime.h>

#include "q4_common.h"

namespace ia {
namespace {

// ------------------------------------------------------------ quantisation

// w / s rounded to the nearest whole number, ties to even, exactly: the product
// with the reciprocal is off by one at most, and next to a border only; r s and
// the rest of w are exact in fp32 (r has 4 bits, s 16).
__device__ __forceinline__ float nearest_code(float w, float s, float inverse) {
    float r = rintf(w * inverse);
    const float d = __builtin_fmaf(-r, s, w), h = 0.5f * s;
    const bool odd = ((int)r & 1) != 0;
    if (d > h || (d == h && odd)) r += 1.0f;
    if (d < -h || (d == -h && odd)) r -= 1.0f;
    return r;
}

// Eight values a thread, G / 8 threads a group.  lo and hi include zero; s =
// (hi - lo) / 15 in double, rounded up to 16 bits (at least 2^-100), z = the
// code nearest to -lo / s.  A group that is not finite has the scale NaN.
template <typename T, int G>
__global__ void __launch_bounds__(256) q4_quantize_kernel(const T* x, int64_t ldx, int64_t rows, int64_t cols, uint32_t* codes,
                                                          uint32_t* words) {
    constexpr int LANES = G / 8;
    const int64_t groups = q4_groups(cols, G), chunks = groups * LANES, total = rows * chunks, ldw = q4_word_stride(groups);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / chunks, k = i - r * chunks, g = k / LANES;
        float v[8];
        load8(x + r * ldx + 8 * k, cols - 8 * k, v);
        float lo = 0.0f, hi = 0.0f;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            lo = fminf(lo, v[j]);
            hi = fmaxf(hi, v[j]);
            top = max(top, __builtin_bit_cast(uint32_t, v[j]) & 0x7fffffffu);
        }
#pragma unroll
        for (int m = 1; m < LANES; m *= 2) {
            lo = fminf(lo, __shfl_xor(lo, m));
            hi = fmaxf(hi, __shfl_xor(hi, m));
            top = max(top, (uint32_t)__shfl_xor((int)top, m));
        }
        const double range = ((double)hi - (double)lo) / 15.0;
        const uint64_t low = ((uint64_t)1 << 37) - 1;
        const uint64_t bits = (__builtin_bit_cast(uint64_t, range) + low) & ~low;
        float s = fmaxf((float)__builtin_bit_cast(double, bits), 0x1p-100f);
        const float inverse = 1.0f / s;
        const float z = nearest_code(-lo, s, inverse);
        uint32_t q = 0, word = __builtin_bit_cast(uint32_t, s) | (uint32_t)z;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            q |= (uint32_t)fminf(fmaxf(nearest_code(v[j], s, inverse) + z, 0.0f), 15.0f) << (4 * j);
        if (hi == lo) q = word = 0;  // zeros
        if (top >= 0x7f800000u) {
            q = 0;
            word = 0x7fc00000u;
        }
        codes[r * chunks + k] = q;
        if (k % LANES == 0) {
            words[r * ldw + g] = word;
            if (g == groups - 1)
                for (int64_t j = groups; j < ldw; ++j) words[r * ldw + j] = 0;
        }
    }
}

// Eight values a thread.  s (q - z) is exact in fp32, then rounded once.
template <typename T, int G>
__global__ void __launch_bounds__(256) q4_dequantize_kernel(const uint32_t* codes, const uint32_t* words, int64_t rows,
                                                            int64_t cols, T* x, int64_t ldx) {
    const int64_t groups = q4_groups(cols, G), chunks = groups * (G / 8), total = rows * chunks, ldw = q4_word_stride(groups);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / chunks, k = i - r * chunks;
        const uint32_t q = codes[i], w = words[r * ldw + k / (G / 8)];
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = scale_of(w) * ((float)((q >> (4 * j)) & 15u) - zero_of(w));
        store8(x + r * ldx + 8 * k, cols - 8 * k, v);
    }
}

// ------------------------------------------------------------ product

// Eight values of a row of x as matrix operands.  fp32 goes as three bf16 parts
// of 8 bits each, cut off and not rounded, so that they add up to the value
// exactly (a value that is not finite is its first part alone).
template <typename T>
struct Operand;
template <>
struct Operand<_Float16> {
    typedef halfx8 vec;
    static constexpr int kParts = 1;
};
template <>
struct Operand<__bf16> {
    typedef bfloatx8 vec;
    static constexpr int kParts = 1;
};
template <>
struct Operand<float> {
    typedef bfloatx8 vec;
    static constexpr int kParts = 3;
};

__device__ __forceinline__ floatx4 mfma(halfx8 a, halfx8 b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ floatx4 mfma(bfloatx8 a, bfloatx8 b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Lane groups of 16: lane group a's register b and lane group b's register a change places.
__device__ __forceinline__ void transpose(uint32_t (&r)[4]) {
    const auto swap32 = [&](int a, int b) {
        const auto t = __builtin_amdgcn_permlane32_swap(r[a], r[b], false, false);
        r[a] = t[0];
        r[b] = t[1];
    };
    const auto swap16 = [&](int a, int b) {
        const auto t = __builtin_amdgcn_permlane16_swap(r[a], r[b], false, false);
        r[a] = t[0];
        r[b] = t[1];
    };
    swap32(0, 2);
    swap32(1, 3);
    swap16(0, 1);
    swap16(2, 3);
}

constexpr int kWaves = 8;

// y = act(x W^T + bias) for 16 MT rows and 16 NT outputs a block.  The waves of
// a block take every eighth step of 128 inputs each; a lane loads 16 bytes of
// codes (32 inputs of its output), four lanes' worth is transposed so that each
// matrix instruction covers 32 consecutive inputs, which lie in one group.  The
// codes less their zero are exact matrix operands; a group's sum is
// scaled in fp32.
template <typename T, int MT, int NT, int G>
__global__ void __launch_bounds__(64 * kWaves) q4_few_rows_kernel(const T* x, int64_t M, int64_t ldx, Q4Linear p) {
    typedef typename Operand<T>::vec vec;
    constexpr int PARTS = Operand<T>::kParts, PER = 128 / G;
    __shared__ float sums[kWaves][16 * MT][16 * NT];
    const int lane = threadIdx.x & 63, q = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t across = (p.N + 16 * NT - 1) / (16 * NT);
    const int64_t m0 = (int64_t)blockIdx.x / across * (16 * MT), n0 = (int64_t)blockIdx.x % across * (16 * NT);
    const int64_t ldw = q4_word_stride(p.groups), ldc = p.groups * (G / 2), steps = (p.groups + PER - 1) / PER;
    floatx4 acc[MT][NT] = {};
    for (int64_t step = wave; step < steps; step += kWaves) {
        uint32_t code[NT][4], word[NT][PER];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int64_t n = min(n0 + 16 * t + c, p.N - 1);
            const int64_t at = step * 64 + 16 * q;
            uintx4 v = {0, 0, 0, 0};
            if (at < ldc) v = *reinterpret_cast<const uintx4*>(p.codes + n * ldc + at);
#pragma unroll
            for (int j = 0; j < 4; ++j) code[t][j] = v[j];
            __builtin_memcpy(word[t], p.words + n * ldw + step * PER, sizeof(word[t]));
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (step * PER + j >= p.groups) word[t][j] = 0;
        }
        Raw<T> raw[4][MT];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t k = step * 128 + 32 * i + 8 * q;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int64_t m = m0 + 16 * t + c;
                raw[i][t] = load_raw(x + m * ldx + k, m < M ? p.K - k : 0);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) transpose(code[t]);
        floatx4 part[MT][NT];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int g = 32 * i / G;
            const bool first = 32 * i % G == 0, last = 32 * (i + 1) % G == 0;
            vec a[MT][PARTS];
#pragma unroll
            for (int t = 0; t < MT; ++t) split(raw[i][t], a[t]);
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                const vec b = codes_less(code[u][i], zero_of(word[u][g]), vec());
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    if (first) part[t][u] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int h = 0; h < PARTS; ++h) part[t][u] = mfma(a[t][h], b, part[t][u]);
                    if (last) {
                        const float s = scale_of(word[u][g]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[t][u][j] = __builtin_fmaf(s, part[t][u][j], acc[t][u][j]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) sums[wave][16 * t + 4 * q + j][16 * u + c] = acc[t][u][j];
    __syncthreads();
    for (int i = threadIdx.x; i < 256 * MT * NT; i += 64 * kWaves) {
        const int r = i / (16 * NT), o = i % (16 * NT);
        const int64_t m = m0 + r, n = n0 + o;
        if (m >= M || n >= p.N) continue;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += sums[w][r][o];
        reinterpret_cast<T*>(p.y)[m * p.ldy + n] = (T)activate(v + (p.bias ? p.bias[n] : 0.0f), p.act);
    }
}

template <typename T, int MT, int NT, int G>
hipError_t few(const T* x, int64_t M, int64_t ldx, const Q4Linear& p, hipStream_t s) {
    IA_LAUNCH("q4_few_rows_kernel", (q4_few_rows_kernel<T, MT, NT, G>),
              dim3((unsigned)(ceil_div(p.N, 16 * NT) * ceil_div(M, 16 * MT))), dim3(64 * kWaves), 0, s, x, M, ldx, p);
    return hipGetLastError();
}
template <typename T, int G>
hipError_t linear(const T* x, int64_t M, int64_t ldx, const Q4Linear& p, hipStream_t s) {
    if (M <= 16) return few<T, 1, 1, G>(x, M, ldx, p, s);
    if (M <= 32) return few<T, 2, 1, G>(x, M, ldx, p, s);
    return few<T, 4, 1, G>(x, M, ldx, p, s);
}

template <typename T>
hipError_t launch_linear(const void* x, int64_t M, int64_t ldx, int group, const Q4Linear& p, hipStream_t s) {
    const T* const t = (const T*)x;
    return group == 32 ? linear<T, 32>(t, M, ldx, p, s) : group == 64 ? linear<T, 64>(t, M, ldx, p, s)
                                                                      : linear<T, 128>(t, M, ldx, p, s);
}

template <typename T, int G>
hipError_t quantize(const void* x, int64_t ldx, const Q4View& o, hipStream_t s) {
    IA_LAUNCH("q4_quantize_kernel", (q4_quantize_kernel<T, G>), dim3(grid_for(o.rows * q4_groups(o.cols, G) * (G / 8))),
              dim3(256), 0, s, (const T*)x, ldx, o.rows, o.cols, (uint32_t*)o.codes, o.words);
    return hipGetLastError();
}
template <typename T>
hipError_t launch_quantize(const void* x, int64_t ldx, const Q4View& o, hipStream_t s) {
    return o.group == 32 ? quantize<T, 32>(x, ldx, o, s) : o.group == 64 ? quantize<T, 64>(x, ldx, o, s)
                                                                         : quantize<T, 128>(x, ldx, o, s);
}

template <typename T, int G>
hipError_t dequantize(const Q4View& q, void* x, int64_t ldx, hipStream_t s) {
    IA_LAUNCH("q4_dequantize_kernel", (q4_dequantize_kernel<T, G>), dim3(grid_for(q.rows * q4_groups(q.cols, G) * (G / 8))),
              dim3(256), 0, s, (const uint32_t*)q.codes, q.words, q.rows, q.cols, (T*)x, ldx);
    return hipGetLastError();
}
template <typename T>
hipError_t launch_dequantize(const Q4View& q, void* x, int64_t ldx, hipStream_t s) {
    return q.group == 32 ? dequantize<T, 32>(q, x, ldx, s) : q.group == 64 ? dequantize<T, 64>(q, x, ldx, s)
                                                                           : dequantize<T, 128>(q, x, ldx, s);
}

}  // namespace

hipError_t launch_q4_quantize(const void* x, int32_t dtype, int64_t ldx, const Q4View& out, hipStream_t s) {
    if (out.rows == 0 || out.cols == 0) return hipSuccess;
    return IA_BY_DTYPE(dtype, launch_quantize, x, ldx, out, s);
}

hipError_t launch_q4_dequantize(const Q4View& q, int32_t dtype, void* x, int64_t ldx, hipStream_t s) {
    if (q.rows == 0 || q.cols == 0) return hipSuccess;
    return IA_BY_DTYPE(dtype, launch_dequantize, q, x, ldx, s);
}

// Up to 64 rows in one reading of the weights, more in tiles (whose offsets have
// 32 bits).
bool is_few(int64_t M, int64_t K) { return M <= 64 || K == 0 || K >= (int64_t)1 << 22; }

size_t q4_linear_workspace(int32_t dtype, int64_t M, int64_t K, int64_t N) {
    return is_few(M, K) || N == 0 ? 0 : q4_matmul_workspace(dtype, M, K, N);
}

hipError_t launch_q4_linear(const void* x, int32_t dtype, int64_t M, int64_t ldx, const Q4View& w, const float* bias,
                            int32_t act, void* y, int64_t ldy, void* ws, hipStream_t s) {
    if (M == 0 || w.rows == 0) return hipSuccess;
    const Q4Linear p{w.codes, w.words, w.rows, w.cols, q4_groups(w.cols, w.group), bias, act, y, ldy};
    if (!is_few(M, w.cols)) return launch_q4_matmul(x, dtype, M, ldx, w.group, p, ws, s);
    return IA_BY_DTYPE(dtype, launch_linear, x, M, ldx, w.group, p, s);
}

}  // namespace ia
