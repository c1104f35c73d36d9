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

// Whether a step's inputs are loaded whole, a step ahead, or quarter by quarter, as
// registers allow.
template <typename T, int MT>
constexpr bool kWhole = MT * sizeof(T) <= 4;

template <typename T, int MT>
struct Inputs {
    Raw<T> x[kWhole<T, MT> ? 4 : 1][MT];  // a step's quarters
};

// A step of 128 inputs: a lane holds 16 bytes of codes (32 inputs of its output);
// four lanes' worth is transposed, so that each matrix instruction covers 32
// consecutive inputs, which lie in one group.  get(x, i) loads quarter i of the
// inputs, where they were not all loaded ahead.
template <typename T, int MT, int NT, int G, typename Get>
__device__ __forceinline__ void multiply(const uintx4 (&codes)[NT], const uint32_t (&words)[NT][128 / G], Inputs<T, MT>& x,
                                         const Get& get, floatx4 (&acc)[MT][NT]) {
    typedef typename Operand<T>::vec vec;
    constexpr int PARTS = Operand<T>::kParts;
    uint32_t code[NT][4];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
#pragma unroll
        for (int j = 0; j < 4; ++j) code[u][j] = codes[u][j];
        transpose(code[u]);
    }
    floatx4 part[MT][NT];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int g = 32 * i / G;
        const bool first = 32 * i % G == 0, last = 32 * (i + 1) % G == 0;
        vec a[MT][PARTS];
#pragma unroll
        for (int t = 0; t < MT; ++t) split(x.x[kWhole<T, MT> ? i : 0][t], a[t]);
        if (!kWhole<T, MT> && i < 3) get(x, i + 1);
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            const vec b = codes_less(code[u][i], zero_of(words[u][g]), vec());
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                if (first) part[t][u] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int h = 0; h < PARTS; ++h) part[t][u] = mfma(a[t][h], b, part[t][u]);
                if (last) {
                    const float f = scale_of(words[u][g]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[t][u][j] = __builtin_fmaf(f, part[t][u][j], acc[t][u][j]);
                }
            }
        }
    }
}

// y = act(x W^T + bias) for 16 MT rows and 16 NT outputs a block.  The waves take
// every WAVES-th unit of four groups: one load brings a lane its output's four
// words, and the codes are consecutive.  The codes less their zero are exact matrix
// operands; a group's sum is scaled in fp32; the waves' sums are added in order.
template <typename T, int MT, int NT, int G, int WAVES>
__global__ void __launch_bounds__(64 * WAVES) q4_few_rows_kernel(const T* x, int64_t M, int64_t ldx, Q4Linear p) {
    constexpr int PER = 128 / G, STEPS = 4 / PER;  // groups of a step, steps of a unit
    constexpr bool WHOLE = kWhole<T, MT>;
    __shared__ float sums[WAVES][16 * MT][16 * NT];
    const int lane = threadIdx.x & 63, q = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t across = (p.N + 16 * NT - 1) / (16 * NT), blocks = across * ((M + 16 * MT - 1) / (16 * MT));
    const int64_t ldw = q4_word_stride(p.groups), ldc = p.groups * (G / 2);
    const int64_t whole = p.K / (4 * G);  // units that lie within a row
    for (int64_t block = blockIdx.x; block < blocks; block += gridDim.x) {
        const int64_t m0 = block / across * (16 * MT), n0 = block % across * (16 * NT);
        // rows and outputs past the end repeat the last one, and are not stored
        const uint8_t* codes[NT];
        const uint32_t* words[NT];
        const T* rows[MT];
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            const int64_t n = min(n0 + 16 * u + c, p.N - 1);
            codes[u] = p.codes + n * ldc + 16 * q;
            words[u] = p.words + n * ldw;
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) rows[t] = x + min(m0 + 16 * t + c, M - 1) * ldx + 8 * q;
        floatx4 acc[MT][NT] = {};
        struct Unit {
            uintx4 code[STEPS][NT];
            uint32_t word[NT][4];
        };
        typedef Inputs<T, MT> inputs_t;
        const auto load_unit = [&](int64_t unit, Unit& s) {
#pragma unroll
            for (int u = 0; u < NT; ++u) {
#pragma unroll
                for (int j = 0; j < STEPS; ++j)
                    s.code[j][u] = *reinterpret_cast<const uintx4*>(codes[u] + (unit * STEPS + j) * 64);
                const uintx4 w = *reinterpret_cast<const uintx4*>(words[u] + unit * 4);
#pragma unroll
                for (int g = 0; g < 4; ++g) s.word[u][g] = w[g];
            }
        };
        const auto load_quarter = [&](int64_t step, inputs_t& s, int i) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
                __builtin_memcpy(&s.x[WHOLE ? i : 0][t], rows[t] + step * 128 + 32 * i, sizeof(s.x[0][t]));
        };
        const auto load_inputs = [&](int64_t step, inputs_t& s) {
#pragma unroll
            for (int i = 0; i < (WHOLE ? 4 : 1); ++i) load_quarter(step, s, i);
        };
        const auto words_of = [&](const Unit& s, int j, uint32_t (&w)[NT][PER]) {
#pragma unroll
            for (int u = 0; u < NT; ++u)
#pragma unroll
                for (int g = 0; g < PER; ++g) w[u][g] = s.word[u][j * PER + g];
        };
        if (wave < whole) {
            Unit now, then;
            inputs_t in;
            load_unit(wave, now);
            load_inputs((int64_t)wave * STEPS, in);
            for (int64_t unit = wave; unit < whole; unit += WAVES) {
                const bool more = unit + WAVES < whole;
                if (more) load_unit(unit + WAVES, then);
#pragma unroll
                for (int j = 0; j < STEPS; ++j) {
                    const int64_t step = unit * STEPS + j, next = j + 1 < STEPS ? step + 1 : (unit + WAVES) * STEPS;
                    inputs_t have = in;
                    if (WHOLE && (j + 1 < STEPS || more)) load_inputs(next, in);
                    uint32_t w[NT][PER];
                    words_of(now, j, w);
                    multiply<T, MT, NT, G>(now.code[j], w, have, [&](inputs_t& e, int i) { load_quarter(step, e, i); }, acc);
                    if (!WHOLE && (j + 1 < STEPS || more)) load_inputs(next, in);
                }
                now = then;
            }
        }
        if (whole * 4 * G < p.K && whole % WAVES == wave) {  // the last inputs: zero past the row's end
#pragma unroll
            for (int j = 0; j < STEPS; ++j) {
                const int64_t step = whole * STEPS + j;
                if (step * 128 >= p.K) break;
                uintx4 code[NT];
                uint32_t w[NT][PER];
#pragma unroll
                for (int u = 0; u < NT; ++u) {
                    code[u] = uintx4{0, 0, 0, 0};
                    if (step * 64 + 16 * q < ldc) code[u] = *reinterpret_cast<const uintx4*>(codes[u] + step * 64);
#pragma unroll
                    for (int g = 0; g < PER; ++g) w[u][g] = step * PER + g < p.groups ? words[u][step * PER + g] : 0u;
                }
                inputs_t in;
                const auto rest = [&](inputs_t& e, int i) {
#pragma unroll
                    for (int t = 0; t < MT; ++t)
                        e.x[WHOLE ? i : 0][t] = load_raw(rows[t] + step * 128 + 32 * i, p.K - step * 128 - 32 * i - 8 * q);
                };
#pragma unroll
                for (int i = 0; i < (WHOLE ? 4 : 1); ++i) rest(in, i);
                multiply<T, MT, NT, G>(code, w, in, rest, acc);
            }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int u = 0; u < NT; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) sums[wave][16 * t + 4 * q + j][16 * u + c] = acc[t][u][j];
        __syncthreads();
        for (int i = threadIdx.x; i < 256 * MT * NT; i += 64 * WAVES) {
            const int r = i / (16 * NT), o = i % (16 * NT);
            const int64_t m = m0 + r, n = n0 + o;
            if (m >= M || n >= p.N) continue;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) v += sums[w][r][o];
            reinterpret_cast<T*>(p.y)[m * p.ldy + n] = (T)activate(v + (p.bias ? p.bias[n] : 0.0f), p.act);
        }
        __syncthreads();  // the sums have been read
    }
}

template <typename T, int MT, int NT, int G, int WAVES>
hipError_t few(const T* x, int64_t M, int64_t ldx, const Q4Linear& p, hipStream_t s) {
    const int64_t blocks = ceil_div(p.N, 16 * NT) * ceil_div(M, 16 * MT);
    IA_LAUNCH("q4_few_rows_kernel", (q4_few_rows_kernel<T, MT, NT, G, WAVES>), dim3((unsigned)(blocks < 1 << 20 ? blocks : 1 << 20)),
              dim3(64 * WAVES), 0, s, x, M, ldx, p);
    return hipGetLastError();
}
template <typename T, int G>
hipError_t linear(const T* x, int64_t M, int64_t ldx, const Q4Linear& p, hipStream_t s) {
    // Two tiles of outputs a wave halve the reading of x, where blocks of four waves fill
    // the chip all the same (5 x 8,192 -> 16,384: 31 -> 26 us; -> 8,192: 12 either way)
    if (M <= 16) return p.N >= 16384 ? few<T, 1, 2, G, 4>(x, M, ldx, p, s) : few<T, 1, 1, G, 8>(x, M, ldx, p, s);
    if (M <= 32) return few<T, 2, 1, G, 8>(x, M, ldx, p, s);
    return few<T, 4, 1, G, 8>(x, M, ldx, p, s);
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

size_t q4_linear_workspace(int32_t dtype, int64_t M, int64_t K, int64_t N) {
    return M == 0 || N == 0 ? 0 : q4_matmul_workspace(dtype, M, K, N);
}

hipError_t launch_q4_linear(const void* x, int32_t dtype, int64_t M, int64_t ldx, const Q4View& w, const float* bias,
                            int32_t act, void* y, int64_t ldy, void* ws, hipStream_t s) {
    if (M == 0 || w.rows == 0) return hipSuccess;
    const Q4Linear p{w.codes, w.words, w.rows, w.cols, q4_groups(w.cols, w.group), bias, act, y, ldy};
    if (q4_takes_tiles(dtype, w.group, M, w.cols, w.rows)) return launch_q4_matmul(x, dtype, M, ldx, w.group, p, ws, s);
    return IA_BY_DTYPE(dtype, launch_linear, x, M, ldx, w.group, p, s);
}

}  // namespace ia
