// 4-bit weights with group scales (q4_common.h): quantisation, read-back and the
// product of a few unquantised rows with them.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "q4_common.h"

namespace ia {
namespace {

// ------------------------------------------------------------ quantisation

// The scale of a group from its least and greatest value (at most 0 and at least
// 0): (hi - lo) / 15 rounded up to 16 bits, which is the least 16-bit number s with
// 15 s >= hi - lo.  (Where 15 s is below hi - lo in double, it is so by at least the
// last place of 15 s, more than the rounding of the quotient can hide.)  The
// quotient in fp32 is off by a few 2^-24, so one of three numbers.
__device__ __forceinline__ float group_scale(float lo, float hi) {
    constexpr float k15 = 1.0f / 15.0f;
    const uint32_t c = __builtin_bit_cast(uint32_t, __builtin_fmaf(-lo, k15, hi * k15)) & ~255u;
    const double range = (double)hi - (double)lo;
    const float s0 = __builtin_bit_cast(float, c), s1 = __builtin_bit_cast(float, c + 256u);
    const float s = 15.0 * (double)s0 >= range ? s0 : 15.0 * (double)s1 >= range ? s1 : __builtin_bit_cast(float, c + 512u);
    return fmaxf(s, 0x1p-100f);
}

// w / s rounded to the nearest whole number r, ties to even: the product with the
// reciprocal is off by one at most, and next to a border only.  r s and d = w - r s
// are exact in fp32 (r has 4 bits, s 16), so d tells.
__device__ __forceinline__ float near_code(float w, float s, float inverse, float& d) {
    const float r = rintf(w * inverse);
    d = __builtin_fmaf(-r, s, w);
    return r;
}
__device__ __forceinline__ float nearest_code(float w, float s, float inverse) {
    float d, r = near_code(w, s, inverse, d);
    const float h = 0.5f * s;
    const bool odd = ((int)r & 1) != 0;
    if (d > h || (d == h && odd)) r += 1.0f;
    if (d < -h || (d == -h && odd)) r -= 1.0f;
    return r;
}

// A value of another lane: of pairs, pairs of pairs and so on exchanged (once the
// lanes of a pair agree, mirrored ones do as well).
constexpr int kPairs = 0xB1, kTwos = 0x4E, kFours = 0x141, kEights = 0x140;  // DPP: quad permutations, half row and row mirrored
template <int CTRL>
__device__ __forceinline__ float exchanged(float v) {
    const int b = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(b, b, CTRL, 0xf, 0xf, true));
}

// Rows from row0 on, fewer than 2^31 threads.
struct Q4Rows {
    uint32_t row0, rows;
    int64_t cols;
    Divisor chunks;  // of eight values a row, all its groups' (threads)
};

// Eight values a thread, G / 8 threads a group.  z = the code nearest to -lo / s.  A
// group that is not finite has the scale NaN.  8,192 x 8,192 bf16 values (170 MB) take
// 45 us (3.8 TB/s): with the limits exchanged through LDS they took 52, with a 64-bit
// division for every place and a double one for every scale 68.
template <typename T, int G>
__global__ void __launch_bounds__(256) q4_quantize_kernel(const T* x, int64_t ldx, Q4Rows p, uint32_t* codes, uint32_t* words) {
    constexpr uint32_t LANES = G / 8;
    const uint32_t i = blockIdx.x * 256u + threadIdx.x, at = p.chunks.of(i), r = p.row0 + at, k = i - at * p.chunks.d;
    if (at >= p.rows) return;  // whole groups of threads
    float v[8];
    const T* const from = x + r * ldx + 8 * (int64_t)k;
    if (8 * ((int64_t)k + 1) <= p.cols) {
        load8(from, 8, v);
    } else {
        load8(from, p.cols - 8 * (int64_t)k, v);
    }
    float lo = 0.0f, hi = 0.0f;
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        lo = fminf(lo, v[j]);
        hi = fmaxf(hi, v[j]);
        top = max(top, __builtin_bit_cast(uint32_t, v[j]) & 0x7fffffffu);
    }
    if (top >= 0x7f800000u) hi = __builtin_huge_valf();  // also for a NaN
    const auto reduce = [&](auto exchange) {
        constexpr int CTRL = decltype(exchange)::value;
        lo = fminf(lo, exchanged<CTRL>(lo));
        hi = fmaxf(hi, exchanged<CTRL>(hi));
    };
    reduce(std::integral_constant<int, kPairs>{});
    reduce(std::integral_constant<int, kTwos>{});
    if (LANES > 4) reduce(std::integral_constant<int, kFours>{});
    if (LANES > 8) reduce(std::integral_constant<int, kEights>{});
    const float s = group_scale(lo, hi), inverse = 1.0f / s, z = nearest_code(-lo, s, inverse);
    float c[8], most = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float d;
        c[j] = near_code(v[j], s, inverse, d);
        most = fmaxf(most, fabsf(d));
    }
    if (most >= 0.5f * s) {  // a border
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = nearest_code(v[j], s, inverse);
    }
    uint32_t q = 0, word = __builtin_bit_cast(uint32_t, s) | (uint32_t)z;
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = fminf(fmaxf(c[j] + z, 0.0f), 15.0f);
#pragma unroll
    for (int j = 0; j < 4; ++j) q = __builtin_amdgcn_cvt_pk_u8_f32(__builtin_fmaf(c[2 * j + 1], 16.0f, c[2 * j]), j, q);
    if (hi == lo) q = word = 0;  // zeros
    if (hi == __builtin_huge_valf()) {
        q = 0;
        word = 0x7fc00000u;
    }
    const uint32_t groups = p.chunks.d / LANES, g = k / LANES;
    const int64_t ldw = q4_word_stride(groups);
    codes[(int64_t)r * p.chunks.d + k] = q;
    if (k % LANES == 0) {
        words[r * ldw + g] = word;
        if (g == groups - 1)
            for (int64_t j = groups; j < ldw; ++j) words[r * ldw + j] = 0;
    }
}

// Eight values a thread.  s (q - z) is exact in fp32, then rounded once.  8,192 x
// 8,192 values to bf16 (170 MB) take 26 us (6.6 TB/s, the codes partly from the
// memory-side cache).
template <typename T, int G>
__global__ void __launch_bounds__(256) q4_dequantize_kernel(const uint32_t* codes, const uint32_t* words, Q4Rows p, T* x,
                                                            int64_t ldx, bool stream) {
    const uint32_t i = blockIdx.x * 256u + threadIdx.x, at = p.chunks.of(i), r = p.row0 + at, k = i - at * p.chunks.d;
    if (at >= p.rows) return;
    const int64_t ldw = q4_word_stride(p.chunks.d / (G / 8));
    const uint32_t w = words[r * ldw + k / (G / 8)];
    const Nibbles q(codes[(int64_t)r * p.chunks.d + k]);
    const float s = scale_of(w), z = zero_of(w);
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = s * (q.value<0>(j) - z);
        v[2 * j + 1] = s * (q.value<1>(j) - z);
    }
    T* const to = x + r * ldx + 8 * (int64_t)k;
    if (8 * ((int64_t)k + 1) <= p.cols)
        store8(to, 8, v, stream);
    else
        store8(to, p.cols - 8 * (int64_t)k, v);
}

// Launches over at most 2^31 threads each.
template <typename Fn>
hipError_t for_rows(const Q4View& q, const Fn& launch) {
    const Divisor chunks((uint32_t)(q4_groups(q.cols, q.group) * (q.group / 8)));
    const int64_t most = (((int64_t)1 << 31) - 256) / chunks.d;
    for (int64_t r = 0; r < q.rows; r += most) {
        const int64_t here = std::min(most, q.rows - r);
        launch(Q4Rows{(uint32_t)r, (uint32_t)here, q.cols, chunks}, dim3((unsigned)ceil_div(here * chunks.d, 256)));
    }
    return hipGetLastError();
}

// ------------------------------------------------------------ product

// Eight values of a row of x as matrix operands.  fp32 goes as three bf16 parts
// of 8 bits each, cut off and not rounded, so that they add up to the value (to
// within 2^-133, bf16's least; a value that is not finite is its first part alone).
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

// What a group's word does to its codes: operands are the codes less their zero, and
// the sum of a group is scaled.  Inputs in bf16 and fp32 reach the end of fp32's range,
// which their sums would pass where the scale brings the result back: their operands
// are 2^-11 times that, so that 128 terms of less than 2^132 stay below 2^128, and the
// scale 2^11 times as large (not one past 2^64, where the result is out of range as well).
template <typename V>
struct Group;
template <>
struct Group<halfx8> {
    halfx2 zu;
    float scale;
    __device__ __forceinline__ explicit Group(uint32_t word) : zu(twice(-zero_of(word))), scale(scale_of(word)) {}
    __device__ __forceinline__ halfx8 operand(uint32_t codes) const { return codes_times(codes, 512.0f, zu); }
};
template <>
struct Group<bfloatx8> {
    float u, zu, scale;
    __device__ __forceinline__ explicit Group(uint32_t word) {
        const bool past = fabsf(scale_of(word)) >= 0x1p64f;
        u = past ? 1.0f : 0x1p-11f;
        zu = -zero_of(word) * u;
        scale = scale_of(word) * (past ? 1.0f : 0x1p11f);
    }
    __device__ __forceinline__ bfloatx8 operand(uint32_t codes) const { return codes_times(codes, u, zu); }
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
            const Group<vec> group(words[u][g]);
            const vec b = group.operand(code[u][i]);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                if (first) part[t][u] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int h = 0; h < PARTS; ++h) part[t][u] = mfma(a[t][h], b, part[t][u]);
                if (last) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[t][u][j] = __builtin_fmaf(group.scale, part[t][u][j], acc[t][u][j]);
                }
            }
        }
    }
}

// y = act(x W^T + bias) for 16 MT rows and 16 NT outputs a block.  The waves take
// every WAVES-th unit of four groups: one load brings a lane its output's four
// words, and the codes are consecutive.  The codes less their zero are exact matrix
// operands; a group's sum is scaled in fp32; the waves' sums are added in order.
// One fp16 row through 4,096 -> 4,096 (8.9 MB): 7.3 us, most of it the launch and one
// round of loads.  Five bf16 rows through 8,192 -> 16,384 (71 MB): 26 us (2.7 TB/s).
// There the loads' own handling binds: without x's 24, without x and words 23, and
// without the conversions too 19 (measured with one tile of outputs a wave, 33 in all).
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
    // Two tiles of outputs a wave halve the reading of x, and blocks of four waves leave fewer
    // rounds of them on the chip; up to 8,192 outputs there are few blocks then (times of calls
    // with one and with two, us):
    //   outputs                         8,192        10,240       12,288       16,384
    //   1 fp16 row of 4,096          9.9  10.2    14.0  13.3    14.3  13.7    17.1  14.1
    //   5 bf16 rows of 8,192        17.2  16.8    23.4  24.0    24.3  24.1    30.1  24.8
    //   16 bf16 rows of 4,096       14.6  12.2    20.6  18.0    21.1  18.1    25.5  18.6
    //   8 fp32 rows of 4,096        22.2  16.7    32.0  25.1    32.5  24.9    42.2  25.8
    if (M <= 16) return p.N > 8192 ? few<T, 1, 2, G, 4>(x, M, ldx, p, s) : few<T, 1, 1, G, 8>(x, M, ldx, p, s);
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
    return for_rows(o, [&](const Q4Rows& p, dim3 grid) {
        IA_LAUNCH("q4_quantize_kernel", (q4_quantize_kernel<T, G>), grid, dim3(256), 0, s, (const T*)x, ldx, p,
                  (uint32_t*)o.codes, o.words);
    });
}
template <typename T>
hipError_t launch_quantize(const void* x, int64_t ldx, const Q4View& o, hipStream_t s) {
    return o.group == 32 ? quantize<T, 32>(x, ldx, o, s) : o.group == 64 ? quantize<T, 64>(x, ldx, o, s)
                                                                         : quantize<T, 128>(x, ldx, o, s);
}

template <typename T, int G>
hipError_t dequantize(const Q4View& q, void* x, int64_t ldx, hipStream_t s) {
    return for_rows(q, [&](const Q4Rows& p, dim3 grid) {
        IA_LAUNCH("q4_dequantize_kernel", (q4_dequantize_kernel<T, G>), grid, dim3(256), 0, s, (const uint32_t*)q.codes, q.words,
                  p, (T*)x, ldx, q.rows * q.cols * (int64_t)sizeof(T) >= kStreamBytes);
    });
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
