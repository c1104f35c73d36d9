// 4-bit microscaled floating point (MXFP4 of the OCP Microscaling Formats
// specification v1.0): quantisation, read-back, products and the gradients of
// a linear layer whose products run in it.
//
// Format: 32 consecutive values of a row form a block with one scale
// 2^(byte - 127) (E8M0; byte 255 is NaN) and 32 E2M1 codes (sign, then
// 0 0.5 1 1.5 2 3 4 6), two to a byte, the earlier one in the low half.  A row
// of `cols` values holds ceil(cols / 32) blocks; the values past its end are
// zero.  The scale of a block is 2^(floor(log2 max|x|) - 2), so that the
// largest value lands in [4, 8): its byte is the exponent field of the fp32
// maximum minus 2 (0 when that is negative).  Codes are rounded to nearest,
// ties to the even code, and values of 6 and more give 6.  A block that holds
// a NaN or an infinity has the NaN scale and zero codes: it reads back as NaN
// and every product it enters is NaN.
//
// The conversions are gfx950's scaled ones (v_cvt_scalef32_pk_fp4_*), which
// take the scale as a float of that exponent (bits byte << 23; 0 stands for
// 2^-127) and round as above.
//
// Products use v_mfma_scale_f32_16x16x128_f8f6f4 (wave64, lane l, q = l / 16,
// c = l % 16): a lane supplies row c of its operand at the 32 values of
// k-block q, 16 bytes, and that block's scale byte, so one lane's share of an
// operand is exactly one block of the format; D holds rows 4 q .. 4 q + 3 of
// the first operand against row c of the second, accumulated in fp32.
#include <hip/hip_runtime.h>

#include "ia_internal.h"

namespace ia {
namespace {

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef unsigned short ushortx2 __attribute__((ext_vector_type(2)));

constexpr int kBlock = 32;   // values per scale
constexpr int kFp4 = 4;      // the MFMA's format code of E2M1
constexpr int kNaNByte = 255;

template <typename T>
struct Pair;
template <>
struct Pair<float> {
    typedef float type __attribute__((ext_vector_type(2)));
};
template <>
struct Pair<_Float16> {
    typedef _Float16 type __attribute__((ext_vector_type(2)));
};
template <>
struct Pair<__bf16> {
    typedef __bf16 type __attribute__((ext_vector_type(2)));
};
template <typename T>
using pair_t = typename Pair<T>::type;

// 32 values of one block, in pairs
template <typename T>
struct Values {
    pair_t<T> p[16];
};

template <int BYTE>
__device__ __forceinline__ uint32_t cvt_pair(uint32_t old, pair_t<float> v, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, v[0], v[1], scale, BYTE);
}
template <int BYTE>
__device__ __forceinline__ uint32_t cvt_pair(uint32_t old, pair_t<_Float16> v, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, v, scale, BYTE);
}
template <int BYTE>
__device__ __forceinline__ uint32_t cvt_pair(uint32_t old, pair_t<__bf16> v, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, v, scale, BYTE);
}

// fp32 bits of the largest magnitude (integer comparison orders magnitudes,
// infinities and NaN above every finite one)
__device__ __forceinline__ uint32_t max_bits(const Values<float>& v) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        m = max(m, __builtin_bit_cast(uint32_t, (float)v.p[i][0]) & 0x7fffffffu);
        m = max(m, __builtin_bit_cast(uint32_t, (float)v.p[i][1]) & 0x7fffffffu);
    }
    return m;
}
template <typename T>
__device__ __forceinline__ uint32_t max_bits16(const Values<T>& v) {
    ushortx2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        m = __builtin_elementwise_max(
            m, __builtin_bit_cast(ushortx2, __builtin_bit_cast(uint32_t, v.p[i]) & 0x7fff7fffu));
    return max((uint32_t)m[0], (uint32_t)m[1]);
}
__device__ __forceinline__ uint32_t max_bits(const Values<_Float16>& v) {
    return __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(_Float16, (uint16_t)max_bits16(v)));
}
__device__ __forceinline__ uint32_t max_bits(const Values<__bf16>& v) { return max_bits16(v) << 16; }

// Codes and scale byte of one block.
template <typename T>
__device__ __forceinline__ intx4 quantize(const Values<T>& v, uint32_t& byte) {
    const uint32_t e = max_bits(v) >> 23;
    byte = e < 2u ? 0u : e - 2u;
    const float scale = __builtin_bit_cast(float, byte << 23);
    intx4 c;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint32_t r = cvt_pair<0>(0u, v.p[4 * w], scale);
        r = cvt_pair<1>(r, v.p[4 * w + 1], scale);
        r = cvt_pair<2>(r, v.p[4 * w + 2], scale);
        r = cvt_pair<3>(r, v.p[4 * w + 3], scale);
        c[w] = (int)r;
    }
    if (e == 255u) {
        byte = kNaNByte;
        c = intx4{0, 0, 0, 0};
    }
    return c;
}

// Values k0 .. k0 + 31 of a row of `cols` (zero past its end).
template <typename T>
__device__ __forceinline__ Values<T> load_values(const T* row, int64_t k0, int64_t cols) {
    Values<T> v;
    if (k0 + kBlock <= cols) {
        __builtin_memcpy(&v, row + k0, sizeof(v));
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            v.p[i][0] = k0 + 2 * i < cols ? row[k0 + 2 * i] : (T)0.0f;
            v.p[i][1] = k0 + 2 * i + 1 < cols ? row[k0 + 2 * i + 1] : (T)0.0f;
        }
    }
    return v;
}

// v where the matching value of y is above zero, else zero (a ReLU's gradient)
template <typename T>
__device__ __forceinline__ void mask(Values<T>& v, const Values<T>& y) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        v.p[i][0] = (float)y.p[i][0] > 0.0f ? v.p[i][0] : (T)0.0f;
        v.p[i][1] = (float)y.p[i][1] > 0.0f ? v.p[i][1] : (T)0.0f;
    }
}

// A matrix to quantise: x [rows][cols], rows ldx apart; with y (the same
// shape, rows ldy apart) the values where y <= 0 count as zero.
template <typename T>
struct Source {
    const T* x;
    const T* y;
    int64_t rows, cols, ldx, ldy;
};

// One thread per block of a row.
template <typename T>
__global__ void __launch_bounds__(256) mx4_quantize_rows_kernel(Source<T> s, int64_t blocks, uint8_t* codes,
                                                                uint8_t* scales) {
    const int64_t total = s.rows * blocks;
    for (int64_t base = (int64_t)blockIdx.x * 256; base < total; base += (int64_t)gridDim.x * 256) {
        const int64_t i = base + threadIdx.x;
        if (i >= total) return;
        const int64_t r = i / blocks, k0 = (i - r * blocks) * kBlock;
        Values<T> v = load_values(s.x + r * s.ldx, k0, s.cols);
        if (s.y) mask(v, load_values(s.y + r * s.ldy, k0, s.cols));
        uint32_t byte;
        const intx4 c = quantize(v, byte);
        *reinterpret_cast<intx4*>(codes + i * 16) = c;
        scales[i] = (uint8_t)byte;
    }
}

// Blocks along the columns of x: output row j holds column j.  One thread per
// (column, block of 32 rows), neighbouring threads on neighbouring columns.
template <typename T>
__global__ void __launch_bounds__(256) mx4_quantize_cols_kernel(Source<T> s, int64_t blocks, uint8_t* codes,
                                                                uint8_t* scales) {
    const int64_t total = s.cols * blocks;
    for (int64_t base = (int64_t)blockIdx.x * 256; base < total; base += (int64_t)gridDim.x * 256) {
        const int64_t i = base + threadIdx.x;
        if (i >= total) return;
        const int64_t b = i / s.cols, j = i - b * s.cols, r0 = b * kBlock;
        Values<T> v;
#pragma unroll
        for (int k = 0; k < kBlock; ++k) {
            const int64_t r = r0 + k;
            T e = (T)0.0f;
            if (r < s.rows) {
                e = s.x[r * s.ldx + j];
                if (s.y && !((float)s.y[r * s.ldy + j] > 0.0f)) e = (T)0.0f;
            }
            v.p[k >> 1][k & 1] = e;
        }
        uint32_t byte;
        const intx4 c = quantize(v, byte);
        *reinterpret_cast<intx4*>(codes + (j * blocks + b) * 16) = c;
        scales[j * blocks + b] = (uint8_t)byte;
    }
}

// Value 2^(byte - 127) * code, in fp32; a NaN scale gives NaN.
__device__ __forceinline__ float value_of(uint32_t code, float scale) {
    const uint32_t m = code & 7u;
    const float a = m < 4u ? 0.5f * (float)m : (m < 6u ? (float)m - 2.0f : 2.0f * (float)m - 8.0f);
    return (code & 8u ? -a : a) * scale;
}

__device__ __forceinline__ float scale_of(uint32_t byte) {
    if (byte == (uint32_t)kNaNByte) return __builtin_nanf("");
    return __builtin_bit_cast(float, byte ? byte << 23 : 0x00400000u);  // 2^-127 is subnormal
}

template <typename T>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const uint8_t* codes, const uint8_t* scales,
                                                             int64_t rows, int64_t cols, int64_t blocks, T* x,
                                                             int64_t ldx) {
    const int64_t total = rows * blocks;
    for (int64_t base = (int64_t)blockIdx.x * 256; base < total; base += (int64_t)gridDim.x * 256) {
        const int64_t i = base + threadIdx.x;
        if (i >= total) return;
        const int64_t r = i / blocks, k0 = (i - r * blocks) * kBlock;
        const intx4 c = *reinterpret_cast<const intx4*>(codes + i * 16);
        const float s = scale_of(scales[i]);
        T* out = x + r * ldx + k0;
        T v[kBlock];
#pragma unroll
        for (int k = 0; k < kBlock; ++k) v[k] = (T)value_of((uint32_t)c[k >> 3] >> (4 * (k & 7)), s);
        if (k0 + kBlock <= cols) {
            __builtin_memcpy(out, v, sizeof(v));
        } else {
#pragma unroll
            for (int k = 0; k < kBlock; ++k)
                if (k0 + k < cols) out[k] = v[k];
        }
    }
}

// ------------------------------------------------------------------ product

struct MatArgs {
    const uint8_t* a;   // M rows of `blocks` blocks
    const uint8_t* as;
    const uint8_t* b;   // N rows
    const uint8_t* bs;
    int64_t M, N, blocks;
    const float* bias;  // [N] or null
    int act;
    void* c;            // [M][ldc]
    int64_t ldc;
};

__device__ __forceinline__ intx8 widen(intx4 v) { return intx8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

__device__ __forceinline__ floatx4 mfma(intx4 a, int as, intx4 b, int bs, floatx4 c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(a), widen(b), c, kFp4, kFp4, 0, as, 0, bs);
}

// C[m][n] = act(sum_k a[m][k] b[n][k] + bias[n]).  One wave per 64 x 64 tile.
// The n rows are the MFMA's first operand: row 4 q + r of n tile j stands for
// n = 16 q + 4 j + r, so that a lane ends with 16 consecutive n of one row m.
template <typename T>
__global__ void __launch_bounds__(256) mx4_matmul_kernel(MatArgs p) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4, c = lane & 15;
    const int64_t m0 = (int64_t)blockIdx.x * 128 + (wave & 1) * 64, n0 = (int64_t)blockIdx.y * 128 + (wave >> 1) * 64;
    int64_t ra[4], rb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        ra[i] = min(m0 + 16 * i + c, p.M - 1);
        rb[i] = min(n0 + 16 * (c >> 2) + 4 * i + (c & 3), p.N - 1);
    }
    floatx4 acc[4][4] = {};
    for (int64_t k = 0; k < p.blocks; k += 4) {
        const int64_t kb = k + q;
        const bool in = kb < p.blocks;
        intx4 a[4], b[4];
        int as[4], bs[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t ia = ra[i] * p.blocks + kb, ib = rb[i] * p.blocks + kb;
            a[i] = in ? *reinterpret_cast<const intx4*>(p.a + ia * 16) : intx4{0, 0, 0, 0};
            b[i] = in ? *reinterpret_cast<const intx4*>(p.b + ib * 16) : intx4{0, 0, 0, 0};
            as[i] = in ? (int)p.as[ia] : 127;
            bs[i] = in ? (int)p.bs[ib] : 127;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = mfma(b[j], bs[j], a[i], as[i], acc[i][j]);
    }
    T* out = reinterpret_cast<T*>(p.c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + 16 * i + c;
        if (m >= p.M) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t n = n0 + 16 * q + 4 * j + r;
                if (n >= p.N) continue;
                float v = acc[i][j][r] + (p.bias ? p.bias[n] : 0.0f);
                if (p.act == IA_ACT_RELU) v = v < 0.0f ? 0.0f : v;  // a NaN stays
                out[m * p.ldc + n] = (T)v;
            }
    }
}

// ------------------------------------------------------------- bias gradient

constexpr int kSumRows = 1024;  // rows per partial sum

// part[chunk][col]: sums of kSumRows rows, one thread per column.
template <typename T>
__global__ void __launch_bounds__(256) mx4_colsum_kernel(Source<T> s, float* part) {
    const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (j >= s.cols) return;
    const int64_t r0 = (int64_t)blockIdx.y * kSumRows, r1 = min(r0 + kSumRows, s.rows);
    float sum = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
        const float v = (float)s.x[r * s.ldx + j];
        sum += s.y && !((float)s.y[r * s.ldy + j] > 0.0f) ? 0.0f : v;
    }
    part[(int64_t)blockIdx.y * s.cols + j] = sum;
}

__global__ void __launch_bounds__(256) mx4_colsum_finish_kernel(const float* part, int64_t chunks, int64_t cols,
                                                                float* out) {
    const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (j >= cols) return;
    double sum = 0.0;
    for (int64_t k = 0; k < chunks; ++k) sum += (double)part[k * cols + j];
    out[j] = (float)sum;
}

// ------------------------------------------------------------------- host

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t round_up(size_t n) { return (n + 255) & ~(size_t)255; }

unsigned grid_for(int64_t threads) {
    const int64_t b = ceil_div(threads, 256);
    return (unsigned)(b < (int64_t)1 << 22 ? b : (int64_t)1 << 22);
}

template <typename T>
hipError_t quantize_t(const Mx4Source& x, bool transpose, const Mx4View& out, hipStream_t s) {
    const Source<T> src{(const T*)x.x, (const T*)x.y, x.rows, x.cols, x.ldx, x.ldy};
    const int64_t blocks = mx4_blocks(out.cols);
    if (out.rows == 0 || blocks == 0) return hipSuccess;
    if (transpose)
        IA_LAUNCH("mx4_quantize_cols_kernel", mx4_quantize_cols_kernel<T>, dim3(grid_for(out.rows * blocks)), dim3(256),
                  0, s, src, blocks, out.codes, out.scales);
    else
        IA_LAUNCH("mx4_quantize_rows_kernel", mx4_quantize_rows_kernel<T>, dim3(grid_for(out.rows * blocks)), dim3(256),
                  0, s, src, blocks, out.codes, out.scales);
    return hipGetLastError();
}

template <typename T>
hipError_t dequantize_t(const Mx4View& q, void* x, int64_t ldx, hipStream_t s) {
    const int64_t blocks = mx4_blocks(q.cols);
    if (q.rows == 0 || blocks == 0) return hipSuccess;
    IA_LAUNCH("mx4_dequantize_kernel", mx4_dequantize_kernel<T>, dim3(grid_for(q.rows * blocks)), dim3(256), 0, s,
              (const uint8_t*)q.codes, (const uint8_t*)q.scales, q.rows, q.cols, blocks, (T*)x, ldx);
    return hipGetLastError();
}

template <typename T>
hipError_t matmul_t(const MatArgs& p, hipStream_t s) {
    const dim3 grid((unsigned)ceil_div(p.M, 128), (unsigned)ceil_div(p.N, 128));
    IA_LAUNCH("mx4_matmul_kernel", mx4_matmul_kernel<T>, grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

template <typename T>
hipError_t colsum_t(const Mx4Source& x, float* part, float* out, hipStream_t s) {
    const Source<T> src{(const T*)x.x, (const T*)x.y, x.rows, x.cols, x.ldx, x.ldy};
    const int64_t chunks = ceil_div(x.rows, kSumRows), cb = ceil_div(x.cols, 256);
    if (x.cols == 0) return hipSuccess;
    if (chunks > 0) {
        IA_LAUNCH("mx4_colsum_kernel", mx4_colsum_kernel<T>, dim3((unsigned)cb, (unsigned)chunks), dim3(256), 0, s, src,
                  part);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    IA_LAUNCH("mx4_colsum_finish_kernel", mx4_colsum_finish_kernel, dim3((unsigned)cb), dim3(256), 0, s,
              (const float*)part, chunks, x.cols, out);
    return hipGetLastError();
}

#define IA_BY_DTYPE(dtype, fn, ...)                                   \
    ((dtype) == IA_DTYPE_F32   ? fn<float>(__VA_ARGS__)               \
     : (dtype) == IA_DTYPE_F16 ? fn<_Float16>(__VA_ARGS__)            \
                               : fn<__bf16>(__VA_ARGS__))

// Scratch of one quantised matrix: codes, then scales.
size_t scratch_bytes(int64_t rows, int64_t cols) {
    const size_t n = (size_t)rows * (size_t)mx4_blocks(cols);
    return round_up(16 * n) + round_up(n);
}
Mx4View scratch_view(void* at, int64_t rows, int64_t cols) {
    uint8_t* p = (uint8_t*)at;
    return Mx4View{p, p + round_up(16 * (size_t)rows * (size_t)mx4_blocks(cols)), rows, cols};
}

}  // namespace

int64_t mx4_blocks(int64_t cols) { return ceil_div(cols, kBlock); }

hipError_t launch_mx4_quantize(const Mx4Source& x, bool transpose, const Mx4View& out, hipStream_t s) {
    return IA_BY_DTYPE(x.dtype, quantize_t, x, transpose, out, s);
}

hipError_t launch_mx4_dequantize(const Mx4View& q, int32_t dtype, void* x, int64_t ldx, hipStream_t s) {
    return IA_BY_DTYPE(dtype, dequantize_t, q, x, ldx, s);
}

size_t mx4_matmul_workspace(int64_t M, int64_t N, int64_t K) { return 0; }

hipError_t launch_mx4_matmul(const Mx4View& a, const Mx4View& b, const float* bias, int32_t act, int32_t dtype, void* c,
                             int64_t ldc, void* ws, hipStream_t s) {
    if (a.rows == 0 || b.rows == 0) return hipSuccess;
    const MatArgs p{a.codes, a.scales, b.codes, b.scales, a.rows, b.rows, mx4_blocks(a.cols), bias, act, c, ldc};
    return IA_BY_DTYPE(dtype, matmul_t, p, s);
}

size_t mx4_linear_workspace(int64_t M, int64_t K, int64_t N) { return scratch_bytes(M, K); }

hipError_t launch_mx4_linear(const Mx4Source& x, const Mx4View& w, const float* bias, int32_t act, void* y,
                             int64_t ldy, void* ws, hipStream_t s) {
    const Mx4View q = scratch_view(ws, x.rows, x.cols);
    hipError_t e = launch_mx4_quantize(x, false, q, s);
    if (e != hipSuccess) return e;
    return launch_mx4_matmul(q, w, bias, act, x.dtype, y, ldy, nullptr, s);
}

size_t mx4_linear_backward_workspace(int64_t M, int64_t N, int64_t K) {
    return scratch_bytes(M, N) + scratch_bytes(N, M) + scratch_bytes(K, M) +
           round_up((size_t)ceil_div(M, kSumRows) * (size_t)N * sizeof(float));
}

hipError_t launch_mx4_linear_backward(const Mx4Source& dy, const Mx4Source& x, const Mx4View& wt, void* dx, int64_t lddx,
                                      float* dw, float* db, void* ws, hipStream_t s) {
    const int64_t M = dy.rows, N = dy.cols, K = x.cols;
    char* at = (char*)ws;
    const Mx4View dr = scratch_view(at, M, N), dc = scratch_view(at += scratch_bytes(M, N), N, M),
                  xc = scratch_view(at += scratch_bytes(N, M), K, M);
    float* part = (float*)(at += scratch_bytes(K, M));
    hipError_t e = hipSuccess;
    if (dx) {
        e = launch_mx4_quantize(dy, false, dr, s);
        if (e == hipSuccess) e = launch_mx4_matmul(dr, wt, nullptr, kMx4NoAct, dy.dtype, dx, lddx, nullptr, s);
    }
    if (e == hipSuccess && dw) {
        e = launch_mx4_quantize(dy, true, dc, s);
        if (e == hipSuccess) e = launch_mx4_quantize(x, true, xc, s);
        if (e == hipSuccess) e = launch_mx4_matmul(dc, xc, nullptr, kMx4NoAct, IA_DTYPE_F32, dw, K, nullptr, s);
    }
    if (e == hipSuccess && db) e = IA_BY_DTYPE(dy.dtype, colsum_t, dy, part, db, s);
    return e;
}

}  // namespace ia
