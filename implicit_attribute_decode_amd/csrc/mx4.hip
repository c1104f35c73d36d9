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

#include "mx4_common.h"

namespace ia {
namespace {

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

// The ReLU mask of 16 rows (lanes c) by 128 columns (32 in each lane group q)
// turned to bits along the rows: bit c of word [column] of `words`.  A
// comparison's lane mask holds the column 32 q + k of all four q.
template <typename T>
__device__ __forceinline__ void store_mask(const Values<T>& y, uint16_t* words, int lane) {
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int k = 0; k < kBlock; ++k) {
        const uint64_t b = __ballot((float)y.p[k >> 1][k & 1] > 0.0f);
        lo = lane == k ? (uint32_t)b : lo;
        hi = lane == k ? (uint32_t)(b >> 32) : hi;
    }
    if (lane < kBlock) {
        words[lane] = (uint16_t)lo;
        words[32 + lane] = (uint16_t)(lo >> 16);
        words[64 + lane] = (uint16_t)hi;
        words[96 + lane] = (uint16_t)(hi >> 16);
    }
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

// Row of block i of a matrix with `blocks` blocks a row, where i is at most 255
// past `base`, which is the same for all threads: one 64-bit division for the
// workgroup and a 32-bit one a thread.
__device__ __forceinline__ int64_t row_of(int64_t i, int64_t blocks, int64_t base) {
    const int64_t r = base / blocks;
    const int64_t k = i - r * blocks;
    return r + (blocks < ((int64_t)1 << 31) ? (int64_t)((uint32_t)k / (uint32_t)blocks) : k / blocks);
}

// One thread per block of a row.  Bound by its bytes: 8,192 x 8,192 in bf16, 170 MB
// in 36 us (4.7 TB/s).
template <typename T>
__global__ void __launch_bounds__(256) mx4_quantize_rows_kernel(Source<T> s, int64_t blocks, uint8_t* codes,
                                                                uint8_t* scales) {
    const int64_t total = s.rows * blocks;
    for (int64_t base = (int64_t)blockIdx.x * 256; base < total; base += (int64_t)gridDim.x * 256) {
        const int64_t i = base + threadIdx.x;
        if (i >= total) return;
        const int64_t r = row_of(i, blocks, base), k0 = (i - r * blocks) * kBlock;
        Values<T> v = load_values(s.x + r * s.ldx, k0, s.cols);
        if (s.y) mask(v, load_values(s.y + r * s.ldy, k0, s.cols));
        uint32_t byte;
        const intx4 c = quantize(v, byte);
        *reinterpret_cast<intx4*>(codes + i * 16) = c;
        scales[i] = (uint8_t)byte;
    }
}

// Blocks along the columns of x (output row j holds column j) and, from the
// same reading of x, its column sums and blocks along the rows.  A tile of 256
// rows and 128 bytes of columns is read in whole lines, masked, and laid in
// LDS with a row pitch of 144 bytes: 16-byte reads along a row and reads down
// the columns both touch every bank once.  A thread takes one block of a
// column at a time; the column codes go back through LDS so that a column's
// eight blocks leave as one line.  Bound by this chain of steps in each tile
// rather than by bytes: 30,011 x 250 in fp32, 34 MB in 13 us; 4,096 x 4,096 in bf16
// with a mask and both ways, 85 MB in 24 us (3.5 TB/s).
constexpr int kTileRows = 256;
constexpr int kTilePitch = 144;

struct ColumnOut {
    uint8_t* codes;   // [cols][blocks] along x's columns, or null
    uint8_t* scales;
    int64_t blocks;
    uint8_t* rcodes;  // [rows][rblocks] along x's rows, or null
    uint8_t* rscales;
    int64_t rblocks;
    float* sums;      // [tile row][cols] sums of 256 rows, or null
};

template <typename T>
__device__ __forceinline__ void quantize_tile(const Source<T>& s, const ColumnOut& o, int64_t it, int64_t jt) {
    constexpr int C = 128 / (int)sizeof(T), E = 16 / (int)sizeof(T);  // columns of a tile, of a 16-byte piece
    __shared__ __attribute__((aligned(16))) uint8_t tile[kTileRows * kTilePitch];
    __shared__ uint8_t cscale[C][8];
    __shared__ float sum[8][C];
    const int t = threadIdx.x;
    const int64_t r0 = it * kTileRows, c0 = jt * C;
    const int piece = t & 7;
    struct Piece {
        T e[E];
    };
    Piece x[8], y[8];
    const int64_t j0 = c0 + piece * E;
    const bool whole = j0 + E <= s.cols;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 32 * i + (t >> 3);
        if (r < s.rows && whole) {
            __builtin_memcpy(&x[i], s.x + r * s.ldx + j0, 16);
            if (s.y) __builtin_memcpy(&y[i], s.y + r * s.ldy + j0, 16);
        } else {
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const bool in = r < s.rows && j0 + k < s.cols;
                x[i].e[k] = in ? s.x[r * s.ldx + j0 + k] : (T)0.0f;
                if (s.y) y[i].e[k] = in ? s.y[r * s.ldy + j0 + k] : (T)0.0f;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (s.y) {
#pragma unroll
            for (int k = 0; k < E; ++k) x[i].e[k] = (float)y[i].e[k] > 0.0f ? x[i].e[k] : (T)0.0f;
        }
        __builtin_memcpy(tile + (32 * i + (t >> 3)) * kTilePitch + 16 * piece, &x[i], 16);
    }
    __syncthreads();
    if (o.rcodes) {
#pragma unroll
        for (int i = 0; i < C / 32; ++i) {
            const int p = t + 256 * i, row = p / (C / 32), b = p % (C / 32);
            const int64_t r = r0 + row, kb = c0 / 32 + b;
            Values<T> v;
            __builtin_memcpy(&v, tile + row * kTilePitch + b * (int)sizeof(v), sizeof(v));
            uint32_t byte;
            const intx4 q = quantize(v, byte);
            if (r < s.rows && kb < o.rblocks) {
                *reinterpret_cast<intx4*>(o.rcodes + (r * o.rblocks + kb) * 16) = q;
                o.rscales[r * o.rblocks + kb] = (uint8_t)byte;
            }
        }
    }
    if (!o.codes && !o.sums) return;
    intx4 q[C / 32];
#pragma unroll
    for (int i = 0; i < C / 32; ++i) {
        const int col = t % C, b = t / C + (256 / C) * i;
        Values<T> v;
#pragma unroll
        for (int k = 0; k < kBlock; ++k)
            v.p[k >> 1][k & 1] = *reinterpret_cast<const T*>(tile + (32 * b + k) * kTilePitch + col * (int)sizeof(T));
        uint32_t byte;
        q[i] = quantize(v, byte);
        cscale[col][b] = (uint8_t)byte;
        float a = 0.0f;
#pragma unroll
        for (int k = 0; k < kBlock; ++k) a += (float)v.p[k >> 1][k & 1];
        sum[b][col] = a;
    }
    __syncthreads();  // the tile has been read
    if (o.sums && t < C && c0 + t < s.cols) {
        float a = 0.0f;
#pragma unroll
        for (int b = 0; b < 8; ++b) a += sum[b][t];
        o.sums[it * s.cols + c0 + t] = a;
    }
    if (!o.codes) return;
    const int64_t b0 = r0 / kBlock;
#pragma unroll
    for (int i = 0; i < C / 32; ++i)
        *reinterpret_cast<intx4*>(tile + ((t % C) * 8 + t / C + (256 / C) * i) * 16) = q[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < C / 32; ++i) {
        const int p = t + 256 * i, col = p >> 3, b = p & 7;
        if (c0 + col < s.cols && b0 + b < o.blocks) {
            const int64_t at = (c0 + col) * o.blocks + b0 + b;
            *reinterpret_cast<intx4*>(o.codes + at * 16) = *reinterpret_cast<const intx4*>(tile + p * 16);
            o.scales[at] = cscale[col][b];
        }
    }
}

// Tiles column by column within a run of rows, so that neighbouring blocks
// read neighbouring lines of a row.
template <typename T>
__global__ void __launch_bounds__(256) mx4_quantize_tile_kernel(Source<T> s, ColumnOut o) {
    constexpr int C = 128 / (int)sizeof(T);
    const int64_t across = (s.cols + C - 1) / C, total = across * ((s.rows + kTileRows - 1) / kTileRows);
    for (int64_t k = blockIdx.x; k < total; k += gridDim.x) {
        quantize_tile(s, o, k / across, k % across);
        __syncthreads();
    }
}

template <int BYTE>
__device__ __forceinline__ pair_t<float> value_pair(uint32_t codes, float scale, float) {
    return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, BYTE);
}
template <int BYTE>
__device__ __forceinline__ pair_t<_Float16> value_pair(uint32_t codes, float scale, _Float16) {
    const pair_t<float> v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, BYTE);
    return pair_t<_Float16>{(_Float16)v[0], (_Float16)v[1]};
}
template <int BYTE>
__device__ __forceinline__ pair_t<__bf16> value_pair(uint32_t codes, float scale, __bf16) {
    const pair_t<float> v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, BYTE);
    return pair_t<__bf16>{(__bf16)v[0], (__bf16)v[1]};
}

// One thread per 8 values: a wave reads 256 bytes of codes and writes whole
// lines.  The conversion to fp32 is exact, then one rounding to T.  Bound by its
// bytes: 16.8M values to fp16, 42 MB in 9.6 us (4.4 TB/s).
template <typename T>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const uint8_t* codes, const uint8_t* scales,
                                                             int64_t rows, int64_t cols, int64_t blocks, T* x,
                                                             int64_t ldx) {
    const int64_t total = rows * blocks * 4;
    for (int64_t base = (int64_t)blockIdx.x * 256; base < total; base += (int64_t)gridDim.x * 256) {
        const int64_t i = base + threadIdx.x;
        if (i >= total) return;
        const int64_t block = i >> 2, r = row_of(block, blocks, base >> 2), k0 = (block - r * blocks) * kBlock + 8 * (i & 3);
        const uint32_t c = reinterpret_cast<const uint32_t*>(codes)[i], byte = scales[block];
        const float s = __builtin_bit_cast(float, byte << 23);
        pair_t<T> v[4] = {value_pair<0>(c, s, T()), value_pair<1>(c, s, T()), value_pair<2>(c, s, T()),
                          value_pair<3>(c, s, T())};
        if (byte == (uint32_t)kNaNByte) {
            const T nan = (T)__builtin_nanf("");
            v[0] = v[1] = v[2] = v[3] = pair_t<T>{nan, nan};
        }
        T* out = x + r * ldx + k0;
        if (k0 + 8 <= cols) {
            __builtin_memcpy(out, v, sizeof(v));
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k0 + k < cols) out[k] = v[k >> 1][k & 1];
        }
    }
}

// ------------------------------------------------------- narrow layers, fused

// act(Q(x) w^T + bias) for layers whose weights for up to 256 outputs (64 G) fit
// LDS; wider layers are taken 256 outputs at a time (blockIdx.y).  A lane's share
// of the MFMA operand is one block of one row, so a wave quantises 16 rows of x
// in its registers on the way to the matrix cores: x is read once (once for 256
// outputs) and only y is written.  Bound by those bytes: 300,000 x 256 -> 256 in fp16,
// 307 MB in 64 us (4.8 TB/s), where quantising first and the tiled product
// take 125.  Loading the next step's values ahead of the current product was not
// faster (64 -> 66 us): other waves cover the latency.
struct NarrowArgs {
    const uint8_t* w;   // [N][blocks]
    const uint8_t* ws;
    int N, blocks, steps;  // steps of 4 blocks
    const float* bias;
    int act;
    void* y;
    int64_t ldy;
    uint16_t* bits;     // with a mask: [rows / 16][128 steps] words of store_mask, or null
    bool lines;         // y's rows are whole lines (writes_lines)
};

constexpr int kNarrowUnits = 14;  // 64 outputs x 128 inputs: 4 KiB of codes, 256 B of scales; within 64 KiB

// Output rows that are whole 128-byte lines, and long, are written past the
// memory-side cache: 300,000 x 256 -> 256 in fp16 69 -> 64 us.  Rows that share
// lines must not be: 100,000 x 64 -> 250 in fp32 would take 88 us instead of 29,
// 300,000 x 192 -> 201 in bf16 130 instead of 58.
bool writes_lines(const void* y, int64_t ldy, int64_t N, size_t es) {
    return (uintptr_t)y % 128 == 0 && (size_t)ldy * es % 128 == 0 && (size_t)N * es >= 512;
}

size_t narrow_lds(int groups, int steps) {
    return (size_t)groups * steps * (4096 + 256) + (size_t)groups * 64 * sizeof(float);
}

// Column n of register r of n tile j in a group of 64, for lane group q: a
// lane's 16 values are 16-byte runs, the four lanes of a row side by side.
template <typename T>
__device__ __forceinline__ int narrow_column(int j, int q, int r) {
    constexpr int E = 16 / (int)sizeof(T);
    const int p = 4 * j + r;
    return p / E * (4 * E) + q * E + p % E;
}

template <typename T, int G, bool MASK>
__global__ void __launch_bounds__(256) mx4_narrow_linear_kernel(Source<T> s, NarrowArgs p) {
    constexpr int NT = 4 * G, E = 16 / (int)sizeof(T);
    extern __shared__ intx4 shared[];
    intx4* wc = shared;                                                         // [step][tile][lane]
    uint8_t* wsc = reinterpret_cast<uint8_t*>(shared + (size_t)p.steps * NT * 64);  // [step][lane][tile]
    float* sbias = reinterpret_cast<float*>(wsc + (size_t)p.steps * 64 * NT);       // [group][64]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4, c = lane & 15;
    const int n0 = (int)blockIdx.y * 64 * G;
    for (int i = threadIdx.x; i < p.steps * NT * 64; i += 256) {
        const int l = i & 63, j = (i >> 6) % NT, step = (i >> 6) / NT;
        const int n = n0 + 64 * (j >> 2) + narrow_column<T>(j & 3, (l & 15) >> 2, l & 3), b = 4 * step + (l >> 4);
        const bool in = n < p.N && b < p.blocks;
        const int64_t at = (int64_t)n * p.blocks + b;
        wc[i] = in ? *reinterpret_cast<const intx4*>(p.w + at * 16) : intx4{0, 0, 0, 0};
        wsc[(step * 64 + l) * NT + j] = in ? p.ws[at] : (uint8_t)0;
    }
    for (int n = threadIdx.x; n < 64 * G; n += 256) sbias[n] = p.bias && n0 + n < p.N ? p.bias[n0 + n] : 0.0f;
    __syncthreads();
    T* out = reinterpret_cast<T*>(p.y);
    for (int64_t m0 = ((int64_t)blockIdx.x * 4 + wave) * 16; m0 < s.rows; m0 += (int64_t)gridDim.x * 64) {
        const int64_t row = min(m0 + c, s.rows - 1);
        const T* x = s.x + row * s.ldx;
        const T* y = s.y + row * s.ldy;
        floatx4 acc[NT] = {};
        for (int step = 0; step < p.steps; ++step) {
            const int64_t k0 = (int64_t)(4 * step + q) * kBlock;
            Values<T> v = load_values(x, k0, s.cols);
            if (MASK) {
                const Values<T> r = load_values(y, k0, s.cols);
                if (p.bits) store_mask(r, p.bits + ((m0 >> 4) * p.steps + step) * 128, lane);
                mask(v, r);
            }
            uint32_t xs;
            const intx4 xc = quantize(v, xs);
            int sc[G];
            __builtin_memcpy(sc, wsc + (step * 64 + lane) * NT, NT);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const intx4* w = wc + (step * NT + 4 * g) * 64 + lane;
                acc[4 * g] = mfma16<0>(w[0], sc[g], xc, (int)xs, acc[4 * g]);
                acc[4 * g + 1] = mfma16<1>(w[64], sc[g], xc, (int)xs, acc[4 * g + 1]);
                acc[4 * g + 2] = mfma16<2>(w[128], sc[g], xc, (int)xs, acc[4 * g + 2]);
                acc[4 * g + 3] = mfma16<3>(w[192], sc[g], xc, (int)xs, acc[4 * g + 3]);
            }
        }
        if (m0 + c >= s.rows) continue;
        T* to = out + (m0 + c) * p.ldy + n0;
        const int N = p.N - n0;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int h = 0; h < 16 / E; ++h) {  // runs of 16 bytes
                const int n = 64 * g + 4 * E * h + E * q;
                T o[E];
#pragma unroll
                for (int e = 0; e < E; ++e)
                    o[e] = (T)activate(acc[4 * g + (E * h + e) / 4][(E * h + e) % 4] + sbias[n + e], p.act);
                if (n + E <= N) {
                    if (p.lines) {
                        uintx4 w;
                        __builtin_memcpy(&w, o, sizeof(w));
                        __builtin_nontemporal_store(w, reinterpret_cast<loose_uintx4*>(to + n));
                    } else {
                        __builtin_memcpy(to + n, o, sizeof(o));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (n + e < N) to[n + e] = o[e];
                }
            }
    }
}

// ------------------------------------------------------------ few rows

// act(Q(x) w^T + bias) for up to 64 rows (16 MT), where the weights are what
// there is to read (1 x 4,096 -> 4,096 in fp16: 8.9 MB in 5.2 us, most of it the
// launch and one round of loads): a block of 8 waves takes 16 outputs, each wave every eighth
// step of 128 inputs.  The weights of a chunk are loaded first; while they come,
// the block quantises the chunk of x once, one block of 32 a thread, into LDS,
// where every wave takes it as its operand.  The waves' sums meet in LDS and
// are added in order.
struct FewArgs {
    const uint8_t* w;  // [N][blocks]
    const uint8_t* ws;
    int64_t N, blocks;
    const float* bias;
    int act;
    void* y;
    int64_t ldy;
};

constexpr int kFewRows = 64;
constexpr int kFewWaves = 8;
constexpr int kFewUnits = 2048;  // blocks of x in LDS

template <typename T, int MT>
__global__ void __launch_bounds__(64 * kFewWaves) mx4_few_rows_kernel(Source<T> s, FewArgs p) {
    constexpr int ROWS = 16 * MT, CHUNK = kFewUnits / ROWS, STEPS = CHUNK / 4 / kFewWaves;  // blocks, a wave's steps
    __shared__ intx4 xc[kFewUnits];  // [block][row]
    __shared__ uint8_t xs[kFewUnits];
    const int lane = threadIdx.x & 63, q = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * 16, row = min(n0 + c, p.N - 1) * p.blocks;
    floatx4 acc[MT] = {};
    for (int64_t b0 = 0; b0 < p.blocks; b0 += CHUNK) {
        intx4 wc[STEPS];
        int wb[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int64_t b = b0 + 4 * (kFewWaves * i + wave) + q;
            const int64_t at = row + min(b, p.blocks - 1);
            wc[i] = *reinterpret_cast<const intx4*>(p.w + at * 16);
            wb[i] = b < p.blocks ? (int)p.ws[at] : 0;
        }
        // whole steps: blocks past the end are zero
        const int here = (int)min((int64_t)CHUNK, (p.blocks - b0 + 3) / 4 * 4);
        __syncthreads();  // the last chunk has been read
        for (int i = threadIdx.x; i < here * (int)s.rows; i += 64 * kFewWaves) {
            const int m = i / here, b = i - m * here;
            uint32_t byte;
            xc[b * ROWS + m] = quantize(load_values(s.x + m * s.ldx, (b0 + b) * kBlock, s.cols), byte);
            xs[b * ROWS + m] = (uint8_t)byte;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int b = 4 * (kFewWaves * i + wave);
            if (b < here) {
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const int at = (b + q) * ROWS + 16 * t + c;
                    acc[t] = mfma16<0>(wc[i], wb[i], xc[at], (int)xs[at], acc[t]);
                }
            }
        }
    }
    __syncthreads();
    float* sum = reinterpret_cast<float*>(xc);  // [wave][row][16 outputs]
    static_assert(kFewWaves * kFewRows * 16 * sizeof(float) <= sizeof(xc), "the sums fit");
#pragma unroll
    for (int t = 0; t < MT; ++t) *reinterpret_cast<floatx4*>(sum + (wave * ROWS + 16 * t + c) * 16 + 4 * q) = acc[t];
    __syncthreads();
    for (int i = threadIdx.x; i < ROWS * 16; i += 64 * kFewWaves) {
        const int64_t m = i >> 4, n = n0 + (i & 15);
        if (m >= s.rows || n >= p.N) continue;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) v += sum[w * ROWS * 16 + i];
        reinterpret_cast<T*>(p.y)[m * p.ldy + n] = (T)activate(v + (p.bias ? p.bias[n] : 0.0f), p.act);
    }
}

// The mask words alone, for a backward that needs no input gradient.
template <typename T>
__global__ void __launch_bounds__(256) mx4_mask_kernel(Source<T> s, int steps, uint16_t* bits) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4, c = lane & 15;
    const int64_t total = (s.rows + 15) / 16 * steps;
    for (int64_t i = (int64_t)blockIdx.x * 4 + wave; i < total; i += (int64_t)gridDim.x * 4) {
        const int64_t m = i / steps * 16 + c;
        const int step = (int)(i % steps);
        store_mask(load_values(s.y + min(m, s.rows - 1) * s.ldy, (int64_t)(4 * step + q) * kBlock, s.cols),
                   bits + i * 128, lane);
    }
}

// dw = Qc(d)^T Qc(x) and db = column sums of d for up to 256 x 256 weights:
// both matrices are read once and quantised along their rows m in registers.
// A block of 8 waves takes a run of rows in steps of 128.  The columns are cut
// into panels of 16 lanes x 4 bytes (32 columns, 16 in fp32); in a step each
// wave takes every eighth of them, lane (q, c) the rows 32 q .. 32 q + 31 of its 4
// bytes, which hold 2 (1) whole blocks, one for each of 2 (1) MFMA tiles whose
// row c is the lane's column.  The codes meet in LDS (two buffers, one barrier
// a step); wave w multiplies the n tiles 2 w, 2 w + 1 with every k tile.  Two
// panels' loads are in flight but for the one being quantised.  The blocks' sums
// go to `part` in register order and are added in a fixed order by
// mx4_narrow_join_kernel.
// Bound by the bytes of d and x: 300,000 rows, 192 -> 256 in fp16, 279 MB in 80 us
// (3.5 TB/s), and 11 us for the join of the 50 MB of sums.
template <typename T>
struct NarrowGradArgs {
    const T* d;
    int64_t ldd;
    const uint16_t* bits;  // mask words, `words` to a group of 16 rows, or null
    int64_t words;
    const T* x;
    int64_t ldx;
    int64_t M, run;  // rows, rows a block takes
    int N, K;
    floatx4* part;  // [block][n tile][k tile][lane]
    float* sums;    // [block][N]
};

constexpr int kGradRows = 128;
constexpr int kGradTiles = 32;  // n and k tiles of 16 columns

// A lane's share of a panel: 32 rows of 4 bytes, as words.
template <typename T>
struct Panel {
    static constexpr int E = 4 / (int)sizeof(T), COLS = 16 * E;
    uint32_t w[kBlock];
    uint16_t bits[2][E];  // mask words of rows 0..15 and 16..31
};

// Rows row0 + 32 q + k of the lane's columns, zero from row `end` on.  The rows'
// addresses are uniform, the lane adds 32 bits where `ld` is below kMaxGradStride
// and takes whole addresses where it is not (FAR).  A piece that crosses the last
// column is read from before its place (cols is at least E); shift_panel puts it
// right.
constexpr int64_t kMaxGradStride = 1 << 22;

template <bool FAR, typename T>
__device__ __forceinline__ void load_panel(Panel<T>& v, const T* m, int64_t ld, int cols, int panel, int q, int c,
                                           int64_t row0, int64_t end) {
    constexpr int E = Panel<T>::E, COLS = Panel<T>::COLS;
    const int col = panel * COLS + E * c, from = min(col, cols - E);
    const char* base = reinterpret_cast<const char*>(m + row0 * ld);
    const int64_t pitch = ld * (int64_t)sizeof(T);
    if (FAR) {
        const int r = 32 * q, last = (int)min((int64_t)kGradRows, end - row0) - 1;
        int64_t off = min(r, last) * pitch + (int64_t)from * (int64_t)sizeof(T);
        asm volatile("" : "+v"(off));  // one address that goes along, not 32 at once
#pragma unroll
        for (int k = 0; k < kBlock; ++k) {
            uint32_t w;
            __builtin_memcpy(&w, base + off, 4);
            v.w[k] = r + k <= last ? w : 0u;
            off += r + k < last ? pitch : 0;
        }
    } else if (row0 + kGradRows <= end) {
        // the offset is opaque: else 32 loop-invariant addresses take 64 registers
        uint32_t off = (uint32_t)((32 * q * (int)ld + from) * (int)sizeof(T));
        asm volatile("" : "+v"(off));
#pragma unroll
        for (int k = 0; k < kBlock; ++k) __builtin_memcpy(&v.w[k], base + k * pitch + off, 4);
    } else {
        const int last = (int)(end - row0) - 1;
        int r = 32 * q;
        asm volatile("" : "+v"(r));
#pragma unroll
        for (int k = 0; k < kBlock; ++k) {
            const uint32_t off = (uint32_t)((min(r + k, last) * (int)ld + from) * (int)sizeof(T));
            uint32_t w;
            __builtin_memcpy(&w, base + off, 4);
            v.w[k] = w & (uint32_t)((r + k - last - 1) >> 31);
        }
    }
}

// The columns of a piece that load_panel read from before its place.
template <typename T>
__device__ __forceinline__ void shift_panel(Panel<T>& v, int cols, int panel, int c) {
    constexpr int E = Panel<T>::E, COLS = Panel<T>::COLS;
    if ((panel + 1) * COLS <= cols) return;
    const int col = panel * COLS + E * c, shift = (col - min(col, cols - E)) * 8 * (int)sizeof(T);
#pragma unroll
    for (int k = 0; k < kBlock; ++k) v.w[k] = shift < 32 ? v.w[k] >> (shift & 31) : 0u;
}

// The mask words of the lane's columns (`words` to a group of 16 rows; a
// multiple of 128, so the piece is whole; past the last row or column any
// words will do, the values there are zero).
template <typename T>
__device__ __forceinline__ void load_bits(Panel<T>& v, const uint16_t* bits, int64_t words, int col, int64_t r0,
                                          int64_t end) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t group = min(r0 / 16 + i, (end - 1) / 16);
        __builtin_memcpy(v.bits[i], bits + group * words + min(col, (int)words - Panel<T>::E), sizeof(v.bits[i]));
    }
}
template <typename T>
__device__ __forceinline__ uint32_t mask_bits(const Panel<T>& v, int e) {
    return (uint32_t)v.bits[0][e] | (uint32_t)v.bits[1][e] << 16;
}

// Rows 2 i, 2 i + 1 of column e.
__device__ __forceinline__ pair_t<float> panel_pair(const Panel<float>& v, int i, int) {
    return pair_t<float>{__builtin_bit_cast(float, v.w[2 * i]), __builtin_bit_cast(float, v.w[2 * i + 1])};
}
template <typename T>
__device__ __forceinline__ pair_t<T> panel_pair(const Panel<T>& v, int i, int e) {
    return __builtin_bit_cast(pair_t<T>,
                              __builtin_amdgcn_perm(v.w[2 * i + 1], v.w[2 * i], e & 1 ? 0x07060302u : 0x05040100u));
}
// The pair where its bits 2 i, 2 i + 1 of m are set, else zero.
__device__ __forceinline__ pair_t<float> keep_pair(pair_t<float> v, uint32_t m, int i) {
    return pair_t<float>{m >> (2 * i) & 1u ? v[0] : 0.0f, m >> (2 * i + 1) & 1u ? v[1] : 0.0f};
}
template <typename T>
__device__ __forceinline__ T keep_pair(T v, uint32_t m, int i) {
    const uint32_t lo = (uint32_t)((int32_t)(m << (31 - 2 * i)) >> 31), hi = (uint32_t)((int32_t)(m << (30 - 2 * i)) >> 31);
    return __builtin_bit_cast(T, __builtin_bit_cast(uint32_t, v) & ((lo & 0xffffu) | (hi & 0xffff0000u)));
}

template <typename T, bool FAR>
__global__ void __launch_bounds__(512) mx4_narrow_grad_kernel(NarrowGradArgs<T> p) {
    constexpr int E = Panel<T>::E, COLS = Panel<T>::COLS, SUBS = kGradTiles / E / 8;  // panels a wave takes
    __shared__ intx4 codes[2][kGradTiles][64];
    __shared__ __attribute__((aligned(16))) uint8_t scales[2][64][kGradTiles];
    const int lane = threadIdx.x & 63, q = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int np = (p.N + COLS - 1) / COLS, kp = (p.K + COLS - 1) / COLS, tn = np * E, tk = kp * E;
    const int64_t begin = (int64_t)blockIdx.x * p.run, end = min(begin + p.run, p.M);
    floatx4 acc[2][16] = {};
    double sum[SUBS][E] = {};  // of blocks of 32 rows: a run may be of any length
    // panels in turn: one on its way while the other is quantised (in fp32, which
    // has no registers for it, one)
    constexpr int AHEAD = sizeof(T) == 2 ? 2 : 1;
    Panel<T> v[AHEAD];
    const int64_t steps = (end - begin + kGradRows - 1) / kGradRows;
    auto load = [&](Panel<T>& to, int64_t step, int sub) {  // panels from np on are x's
        const int all = 8 * sub + wave;
        if (all >= np + kp) return;
        const bool of_d = all < np;
        const int panel = of_d ? all : all - np;
        const int64_t row0 = begin + step * kGradRows;
        if (of_d && p.bits) load_bits(to, p.bits, p.words, panel * COLS + E * c, row0 + 32 * q, end);
        load_panel<FAR>(to, of_d ? p.d : p.x, of_d ? p.ldd : p.ldx, of_d ? p.N : p.K, panel, q, c, row0, end);
    };
    if (steps > 0) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) load(v[i], 0, i);
    }
    for (int64_t step = 0; step < steps; ++step) {
        const int buf = (int)(step & 1);
#pragma unroll
        for (int sub = 0; sub < SUBS; ++sub) {
            const int panel = 8 * sub + wave;
            Panel<T>& from = v[sub % AHEAD];
            if (panel < np + kp) {
                uint32_t bytes = 0;
                shift_panel(from, panel < np ? p.N : p.K, panel < np ? panel : panel - np, c);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    Values<T> b;
#pragma unroll
                    for (int i = 0; i < 16; ++i) b.p[i] = panel_pair(from, i, e);
                    if (panel < np) {
                        if (p.bits) {
                            const uint32_t m = mask_bits(from, e);
#pragma unroll
                            for (int i = 0; i < 16; ++i) b.p[i] = keep_pair(b.p[i], m, i);
                        }
                        float part = 0.0f;
#pragma unroll
                        for (int k = 0; k < kBlock; ++k) part += (float)b.p[k >> 1][k & 1];
                        sum[sub][e] += (double)part;
                    }
                    uint32_t byte;
                    codes[buf][panel * E + e][lane] = quantize(b, byte);
                    bytes |= byte << (8 * e);
                    __builtin_amdgcn_sched_barrier(0);  // one column's temporaries at a time
                }
                __builtin_memcpy(&scales[buf][lane][panel * E], &bytes, E);
            }
            if (sub + AHEAD < SUBS)
                load(from, step, sub + AHEAD);
            else if (step + 1 < steps)
                load(from, step + 1, sub + AHEAD - SUBS);
        }
        __syncthreads();
        if (2 * wave < tn) {
            const bool two = 2 * wave + 1 < tn;
            const int second = two ? 2 * wave + 1 : 2 * wave;
            const intx4 d0 = codes[buf][2 * wave][lane], d1 = codes[buf][second][lane];
            const int s0 = scales[buf][lane][2 * wave], s1 = scales[buf][lane][second];
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (k < tk) {
                    const intx4 xc = codes[buf][tn + k][lane];
                    const int xs = scales[buf][lane][tn + k];
                    acc[0][k] = mfma16<0>(xc, xs, d0, s0, acc[0][k]);
                    acc[1][k] = mfma16<0>(xc, xs, d1, s1, acc[1][k]);
                }
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (2 * wave + h < tn) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (k < tk) p.part[(((int64_t)blockIdx.x * tn + 2 * wave + h) * tk + k) * 64 + lane] = acc[h][k];
        }
    if (!p.sums) return;
#pragma unroll
    for (int sub = 0; sub < SUBS; ++sub)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            double a = sum[sub][e];
            a += __shfl_xor(a, 16, 64);
            a += __shfl_xor(a, 32, 64);
            const int n = (8 * sub + wave) * COLS + E * c + e;
            if (q == 0 && 8 * sub + wave < np && n < p.N) p.sums[(int64_t)blockIdx.x * p.N + n] = (float)a;
        }
}

// The blocks' sums added in a fixed order, 16 waves each taking every
// sixteenth.  Blocks below tn tk join one tile of dw, the others 64 columns of
// db (in double).
template <int E>
__global__ void __launch_bounds__(1024) mx4_narrow_join_kernel(const floatx4* part, const float* sums, int blocks,
                                                               int tn, int tk, int N, int K, float* dw, float* db) {
    __shared__ floatx4 tile[16][64];
    __shared__ double column[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4, c = lane & 15;
    if ((int)blockIdx.x < tn * tk) {
        const int nt = blockIdx.x / tk, kt = blockIdx.x % tk;
        floatx4 a = {0, 0, 0, 0};
#pragma unroll 8
        for (int b = wave; b < blocks; b += 16) a += part[((int64_t)b * tn * tk + blockIdx.x) * 64 + lane];
        tile[wave][lane] = a;
        __syncthreads();
        if (wave != 0) return;
        for (int w = 1; w < 16; ++w) a += tile[w][lane];
        const int n = nt / E * (16 * E) + E * c + nt % E;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int k = kt / E * (16 * E) + E * (4 * q + r) + kt % E;
            if (n < N && k < K) dw[(int64_t)n * K + k] = a[r];
        }
    } else {
        const int n = ((int)blockIdx.x - tn * tk) * 64 + lane;
        double a = 0.0;
        if (n < N) {
#pragma unroll 8
            for (int b = wave; b < blocks; b += 16) a += (double)sums[(int64_t)b * N + n];
        }
        column[wave][lane] = a;
        __syncthreads();
        if (wave != 0 || n >= N) return;
        for (int w = 1; w < 16; ++w) a += column[w][lane];
        db[n] = (float)a;
    }
}

// ------------------------------------------------------------- column sums

// out[col] = sum over the tile rows of part[chunk][col], in double: 16 waves
// each take every sixteenth chunk of 64 columns.
__global__ void __launch_bounds__(1024) mx4_column_sums_kernel(const float* part, int64_t chunks, int64_t cols,
                                                               float* out) {
    __shared__ double sum[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t j = (int64_t)blockIdx.x * 64 + lane;
    double a = 0.0;
    if (j < cols) {
#pragma unroll 8
        for (int64_t k = wave; k < chunks; k += 16) a += (double)part[k * cols + j];
    }
    sum[wave][lane] = a;
    __syncthreads();
    if (wave == 0 && j < cols) {
        a = 0.0;
        for (int w = 0; w < 16; ++w) a += sum[w][lane];
        out[j] = (float)a;
    }
}

// ------------------------------------------------------------------- host

template <typename T>
hipError_t quantize_rows_t(const Mx4Source& x, const Mx4View& out, hipStream_t s) {
    const Source<T> src{(const T*)x.x, (const T*)x.y, x.rows, x.cols, x.ldx, x.ldy};
    const int64_t blocks = mx4_blocks(out.cols);
    if (out.rows == 0 || blocks == 0) return hipSuccess;
    IA_LAUNCH("mx4_quantize_rows_kernel", mx4_quantize_rows_kernel<T>, dim3(grid_for(out.rows * blocks)), dim3(256), 0, s,
              src, blocks, out.codes, out.scales);
    return hipGetLastError();
}

template <typename T>
hipError_t quantize_tile_t(const Mx4Source& x, const ColumnOut& o, hipStream_t s) {
    if (x.rows == 0 || x.cols == 0) return hipSuccess;
    const Source<T> src{(const T*)x.x, (const T*)x.y, x.rows, x.cols, x.ldx, x.ldy};
    const int64_t tiles = ceil_div(x.rows, kTileRows) * ceil_div(x.cols, 128 / (int64_t)sizeof(T));
    IA_LAUNCH("mx4_quantize_tile_kernel", mx4_quantize_tile_kernel<T>, dim3(grid_for(tiles * 256)), dim3(256), 0, s, src,
              o);
    return hipGetLastError();
}

template <typename T>
hipError_t dequantize_t(const Mx4View& q, void* x, int64_t ldx, hipStream_t s) {
    const int64_t blocks = mx4_blocks(q.cols);
    if (q.rows == 0 || blocks == 0) return hipSuccess;
    IA_LAUNCH("mx4_dequantize_kernel", mx4_dequantize_kernel<T>, dim3(grid_for(q.rows * blocks * 4)), dim3(256), 0, s,
              (const uint8_t*)q.codes, (const uint8_t*)q.scales, q.rows, q.cols, blocks, (T*)x, ldx);
    return hipGetLastError();
}

template <typename T, bool MASK>
hipError_t narrow_linear_masked(const Source<T>& src, const NarrowArgs& p, hipStream_t s) {
    // 64 outputs to a group, up to four groups in a block, the blocks' alike
    const int parts = (p.N + 255) / 256, groups = ((p.N + 63) / 64 + parts - 1) / parts;
    const size_t lds = narrow_lds(groups, p.steps);
    // each block reads the weights once; as many blocks as fit the CUs
    const int64_t tiles = ceil_div(src.rows, 64), most = 256 * (int64_t)(163840 / lds < 8 ? 163840 / lds : 8);
    const dim3 grid((unsigned)(tiles < most ? tiles : most), (unsigned)((p.N + 64 * groups - 1) / (64 * groups)));
    switch (groups) {
        case 1:
            IA_LAUNCH("mx4_narrow_linear_kernel", (mx4_narrow_linear_kernel<T, 1, MASK>), grid, dim3(256), lds, s, src, p);
            break;
        case 2:
            IA_LAUNCH("mx4_narrow_linear_kernel", (mx4_narrow_linear_kernel<T, 2, MASK>), grid, dim3(256), lds, s, src, p);
            break;
        case 3:
            IA_LAUNCH("mx4_narrow_linear_kernel", (mx4_narrow_linear_kernel<T, 3, MASK>), grid, dim3(256), lds, s, src, p);
            break;
        default:
            IA_LAUNCH("mx4_narrow_linear_kernel", (mx4_narrow_linear_kernel<T, 4, MASK>), grid, dim3(256), lds, s, src, p);
            break;
    }
    return hipGetLastError();
}

template <typename T>
hipError_t narrow_linear_t(const Mx4Source& x, const NarrowArgs& p, hipStream_t s) {
    const Source<T> src{(const T*)x.x, (const T*)x.y, x.rows, x.cols, x.ldx, x.ldy};
    return x.y ? narrow_linear_masked<T, true>(src, p, s) : narrow_linear_masked<T, false>(src, p, s);
}

template <typename T>
hipError_t few_rows_t(const Mx4Source& x, const FewArgs& p, hipStream_t s) {
    const Source<T> src{(const T*)x.x, nullptr, x.rows, x.cols, x.ldx, 0};
    const dim3 grid((unsigned)ceil_div(p.N, 16)), block(64 * kFewWaves);
    if (x.rows <= 16)
        IA_LAUNCH("mx4_few_rows_kernel", (mx4_few_rows_kernel<T, 1>), grid, block, 0, s, src, p);
    else if (x.rows <= 32)
        IA_LAUNCH("mx4_few_rows_kernel", (mx4_few_rows_kernel<T, 2>), grid, block, 0, s, src, p);
    else
        IA_LAUNCH("mx4_few_rows_kernel", (mx4_few_rows_kernel<T, 4>), grid, block, 0, s, src, p);
    return hipGetLastError();
}

// Blocks and rows a block takes of a narrow gradient: one block a CU, whole
// blocks of 32 rows.
constexpr int64_t kGradBlocks = 256;
struct GradPlan {
    int64_t run, blocks;
    int tn, tk;  // tiles
};
GradPlan grad_plan(int64_t M, int64_t N, int64_t K, size_t es) {
    GradPlan g;
    g.run = ceil_div(ceil_div(M, kGradBlocks), kBlock) * kBlock;
    if (g.run < kGradRows) g.run = kGradRows;
    g.blocks = ceil_div(M, g.run);
    const int64_t e = 4 / (int64_t)es, cols = 16 * e;
    g.tn = (int)(ceil_div(N, cols) * e);
    g.tk = (int)(ceil_div(K, cols) * e);
    return g;
}

// Scratch of a narrow gradient: mask words, tiles, column sums.
struct GradScratch {
    size_t bits, part, sums, total;
};
GradScratch grad_scratch(int64_t M, int64_t N, const GradPlan& g) {
    GradScratch s;
    s.bits = 0;
    s.part = round_up((size_t)ceil_div(M, 16) * (size_t)ceil_div(N, 128) * 256);
    s.sums = s.part + round_up((size_t)g.blocks * g.tn * g.tk * 64 * sizeof(floatx4));
    s.total = s.sums + round_up((size_t)g.blocks * (size_t)N * sizeof(float));
    return s;
}

template <typename T>
hipError_t narrow_grad_t(const Mx4Source& dy, const Mx4Source& x, const Mx4View& wt, void* dx, int64_t lddx, float* dw,
                         float* db, void* ws, hipStream_t s) {
    const int64_t M = dy.rows, N = dy.cols, K = x.cols, blocks = mx4_blocks(N);
    const GradPlan g = grad_plan(M, N, K, sizeof(T));
    const GradScratch at = grad_scratch(M, N, g);
    const int steps = (int)ceil_div(blocks, 4);
    const Source<T> src{(const T*)dy.x, (const T*)dy.y, M, N, dy.ldx, dy.ldy};
    uint16_t* bits = dy.y && (dw || db) ? (uint16_t*)((char*)ws + at.bits) : nullptr;
    hipError_t e = hipSuccess;
    if (dx) {
        const NarrowArgs p{wt.codes, wt.scales, (int)K, (int)blocks, steps, nullptr, IA_ACT_NONE, dx, lddx, bits,
                           writes_lines(dx, lddx, K, sizeof(T))};
        e = narrow_linear_t<T>(dy, p, s);
    } else if (bits) {
        IA_LAUNCH("mx4_mask_kernel", mx4_mask_kernel<T>, dim3(grid_for(ceil_div(M, 16) * steps * 64)), dim3(256), 0, s,
                  src, steps, bits);
        e = hipGetLastError();
    }
    if (e != hipSuccess || !(dw || db)) return e;
    floatx4* part = (floatx4*)((char*)ws + at.part);
    float* sums = db ? (float*)((char*)ws + at.sums) : nullptr;
    const NarrowGradArgs<T> p{src.x, src.ldx, bits, steps * 128, (const T*)x.x, x.ldx, M, g.run, (int)N,
                              dw ? (int)K : 0, part, sums};
    const int tk = dw ? g.tk : 0;
    if (src.ldx < kMaxGradStride && (!dw || x.ldx < kMaxGradStride))
        IA_LAUNCH("mx4_narrow_grad_kernel", (mx4_narrow_grad_kernel<T, false>), dim3((unsigned)g.blocks), dim3(512), 0, s, p);
    else
        IA_LAUNCH("mx4_narrow_grad_kernel", (mx4_narrow_grad_kernel<T, true>), dim3((unsigned)g.blocks), dim3(512), 0, s, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    constexpr int E = Panel<T>::E;
    const int columns = db ? (int)ceil_div(N, 64) : 0;
    IA_LAUNCH("mx4_narrow_join_kernel", mx4_narrow_join_kernel<E>, dim3((unsigned)(g.tn * tk + columns)), dim3(1024), 0,
              s, (const floatx4*)part, (const float*)sums, (int)g.blocks, g.tn, tk, (int)N, (int)K, dw, db);
    return hipGetLastError();
}

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

hipError_t launch_mx4_quantize(const Mx4Source& x, bool transpose, const Mx4View& out, hipStream_t s) {
    if (!transpose) return IA_BY_DTYPE(x.dtype, quantize_rows_t, x, out, s);
    const ColumnOut o{out.codes, out.scales, mx4_blocks(out.cols), nullptr, nullptr, 0, nullptr};
    return IA_BY_DTYPE(x.dtype, quantize_tile_t, x, o, s);
}

hipError_t launch_mx4_dequantize(const Mx4View& q, int32_t dtype, void* x, int64_t ldx, hipStream_t s) {
    return IA_BY_DTYPE(dtype, dequantize_t, q, x, ldx, s);
}

// Whether a layer of M rows, K inputs and N outputs goes through the narrow
// kernel: where 256 outputs' weights fit LDS, and with more outputs where a row has
// at most 256 inputs, so that taking it again for each 256 outputs costs little.
// Against quantising and the tiled product: 150,000 x 32 -> 512 in fp16 81 -> 50 us,
// 50,000 x 200 -> 2,000 in fp16 133 -> 83, 1,000 x 256 -> 10,000 in fp32 25 -> 20;
// 200,000 x 380 -> 1,000 in fp32 would be 386 -> 529.
bool is_narrow(int64_t M, int64_t K, int64_t N) {
    const int64_t steps = ceil_div(mx4_blocks(K), 4);
    if (K == 0) return false;
    if (N <= 256) return ceil_div(N, 64) * steps <= kNarrowUnits;
    return M > kFewRows && steps <= 2 && N <= 16384;
}

// Whether a layer goes through the few rows' kernel.  Each block quantises all of
// x, a chunk of kFewUnits blocks at a time, so chunks have to be few, and blocks
// not more than run at once.  fp16, us against quantising and the tiled product:
//   1 x 256 -> 256 4, 8                  64 x 1,024 -> 4,096 7, 13
//   1 x 4,096 -> 4,096 5, 15             64 x 4,096 -> 64 (fp32) 34, 18
//   7 x 16,384 -> 256 15, 15             32 x 8,192 -> 2,048 17, 17
//   1 x 32,768 -> 16 20, 13              4 x 8,192 -> 32,768 48, 40
bool is_few(int64_t M, int64_t K, int64_t N) {
    if (M > kFewRows) return false;
    const int64_t chunk = kFewUnits / (M <= 16 ? 16 : M <= 32 ? 32 : 64);
    const int64_t chunks = ceil_div(mx4_blocks(K), chunk);
    return chunks <= (M <= 16 ? 4 : 2) && chunks * ceil_div(N, 16) <= 1024;
}

size_t mx4_linear_workspace(int64_t M, int64_t K, int64_t N) {
    return is_few(M, K, N) || is_narrow(M, K, N) ? 0 : scratch_bytes(M, K) + mx4_matmul_workspace(M, N, K);
}

hipError_t launch_narrow_linear(const Mx4Source& x, const Mx4View& w, const float* bias, int32_t act, void* y, int64_t ldy,
                                hipStream_t s) {
    const int64_t blocks = mx4_blocks(x.cols);
    const NarrowArgs p{w.codes, w.scales, (int)w.rows, (int)blocks, (int)ceil_div(blocks, 4), bias, act, y, ldy,
                       nullptr, writes_lines(y, ldy, w.rows, x.dtype == IA_DTYPE_F32 ? 4 : 2)};
    return IA_BY_DTYPE(x.dtype, narrow_linear_t, x, p, s);
}

hipError_t launch_mx4_linear(const Mx4Source& x, const Mx4View& w, const float* bias, int32_t act, void* y,
                             int64_t ldy, void* ws, hipStream_t s) {
    if (x.rows == 0 || w.rows == 0) return hipSuccess;
    if (is_few(x.rows, x.cols, w.rows)) {
        const FewArgs p{w.codes, w.scales, w.rows, mx4_blocks(x.cols), bias, act, y, ldy};
        return IA_BY_DTYPE(x.dtype, few_rows_t, x, p, s);
    }
    if (is_narrow(x.rows, x.cols, w.rows)) return launch_narrow_linear(x, w, bias, act, y, ldy, s);
    const Mx4View q = scratch_view(ws, x.rows, x.cols);
    hipError_t e = launch_mx4_quantize(x, false, q, s);
    if (e != hipSuccess) return e;
    return launch_mx4_matmul(q, w, bias, act, x.dtype, y, ldy, (char*)ws + scratch_bytes(x.rows, x.cols), s);
}

// Whether a layer's gradients go through the fused kernels.  All of a backward,
// against quantising and two tiled products: 300,000 rows, 192 -> 256 in fp16 179
// and 318 us; 300,000, 64 -> 64 in fp16 47 and 102; 1,000, 64 -> 64 in fp32 17 and 38;
// 64, 256 -> 256 in fp16 25 and 34.
bool is_narrow_grad(int64_t M, int64_t N, int64_t K) { return M > 0 && N >= 4 && K >= 4 && N <= 256 && K <= 256; }

size_t mx4_linear_backward_workspace(int64_t M, int64_t N, int64_t K) {
    if (is_narrow_grad(M, N, K)) {
        const size_t a = grad_scratch(M, N, grad_plan(M, N, K, 2)).total, b = grad_scratch(M, N, grad_plan(M, N, K, 4)).total;
        return a > b ? a : b;
    }
    const size_t x = mx4_matmul_workspace(M, K, N), w = mx4_matmul_workspace(N, K, M);
    return scratch_bytes(M, N) + scratch_bytes(N, M) + scratch_bytes(K, M) +
           round_up((size_t)ceil_div(M, kTileRows) * (size_t)N * sizeof(float)) + (x > w ? x : w);
}

hipError_t launch_mx4_linear_backward(const Mx4Source& dy, const Mx4Source& x, const Mx4View& wt, void* dx, int64_t lddx,
                                      float* dw, float* db, void* ws, hipStream_t s) {
    const int64_t M = dy.rows, N = dy.cols, K = x.cols;
    if (is_narrow_grad(M, N, K))
        return IA_BY_DTYPE(dy.dtype, narrow_grad_t, dy, x, wt, dx, lddx, dw, db, ws, s);
    char* at = (char*)ws;
    const Mx4View dr = scratch_view(at, M, N), dc = scratch_view(at += scratch_bytes(M, N), N, M),
                  xc = scratch_view(at += scratch_bytes(N, M), K, M);
    float* part = (float*)(at += scratch_bytes(K, M));
    void* mat = at + round_up((size_t)ceil_div(M, kTileRows) * (size_t)N * sizeof(float));
    ColumnOut o{};
    // dx is a layer of N inputs and K outputs on d.  Where d is quantised for dw
    // anyway, its blocks along the rows come cheaper from the same tiles, but for few
    // columns of 16 bits.  A backward of 30,000 rows so, and with a second reading:
    //   817 -> 18 bf16 85, 106     600 -> 64 f32 90, 100      192 -> 300 f32 71, 79
    //   256 -> 1,000 f32 137, 155  64 -> 2,000 f32 190, 198   64 -> 2,000 bf16 157, 149
    // (us; 1,700 -> 11 in bf16 at 3,122 and at 60,000 rows 56, 66 and 239, 297).
    const bool few = N <= 64 && dy.dtype != IA_DTYPE_F32;
    const bool narrow = dx && M > 0 && is_narrow(M, N, K) && (few || !(dw || db));
    if (dx && !narrow) {
        o.rcodes = dr.codes;
        o.rscales = dr.scales;
        o.rblocks = mx4_blocks(N);
    }
    if (dw) {
        o.codes = dc.codes;
        o.scales = dc.scales;
        o.blocks = mx4_blocks(M);
    }
    if (db) o.sums = part;
    hipError_t e = hipSuccess;
    if (o.rcodes || o.codes || o.sums) e = IA_BY_DTYPE(dy.dtype, quantize_tile_t, dy, o, s);
    if (e == hipSuccess && narrow) e = launch_narrow_linear(dy, wt, nullptr, kMx4NoAct, dx, lddx, s);
    if (e == hipSuccess && dx && !narrow) e = launch_mx4_matmul(dr, wt, nullptr, kMx4NoAct, dy.dtype, dx, lddx, mat, s);
    if (e == hipSuccess && dw) {
        e = launch_mx4_quantize(x, true, xc, s);
        if (e == hipSuccess) e = launch_mx4_matmul(dc, xc, nullptr, kMx4NoAct, IA_DTYPE_F32, dw, K, mat, s);
    }
    if (e == hipSuccess && db && N > 0) {
        IA_LAUNCH("mx4_column_sums_kernel", mx4_column_sums_kernel, dim3((unsigned)ceil_div(N, 64)), dim3(1024), 0, s,
                  (const float*)part, ceil_div(M, kTileRows), N, db);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace ia
