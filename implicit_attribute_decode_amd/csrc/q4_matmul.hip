// Products of many rows with group-scaled 4-bit weights on the 16-bit matrix
// instructions (v_mfma_f32_32x32x16: wave64, lane l, h = l / 32, r = l % 32: a
// lane supplies row r of its operand at 8 values, 8 h of the 16 on; D holds rows
// (e % 4) + 8 (e / 4) + 4 h, e = 0..15, of the first operand against row r of
// the second).
//
// Weights become operands exactly: s (q - z) = m u (q - z), where u (q - z) has
// at most 4 significant bits and m goes to the sums.  A sum is kept in units of
// its weight row's current m: where a group ends it is multiplied by m / m', m'
// being the next group's, and at the end by the last m.
//   bf16: u = the power of two of s, so 1 <= |m| < 2 and nothing grows.
//   fp16: u = 1 and m = s, which fp16's range needs.  A group with |s| under
//   2^-80 counts as zero: with 2^31 inputs of at most 2^16 it adds less than
//   2^-29, under half of fp16's smallest value.
//   fp32 rows go as three bf16 parts of 8 bits each, cut off and not rounded,
//   which add up to them exactly, one part after the other.
#include <hip/hip_runtime.h>

#include "q4_common.h"

namespace ia {
namespace {

template <typename V>
struct Elem;  // the operands' element, as the instructions' vectors hold it
template <>
struct Elem<_Float16> {
    typedef halfx8 vec;
};
template <>
struct Elem<__bf16> {
    typedef bfloatx8 vec;
};

__device__ __forceinline__ floatx16 mfma(halfx8 a, halfx8 b, floatx16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ floatx16 mfma(bfloatx8 a, bfloatx8 b, floatx16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// A group's m.
template <typename V>
__device__ __forceinline__ float unit_of(uint32_t word);
template <>
__device__ __forceinline__ float unit_of<_Float16>(uint32_t word) {
    const float s = scale_of(word);
    return fabsf(s) < 0x1p-80f ? 0x1p-80f : s;
}
template <>
__device__ __forceinline__ float unit_of<__bf16>(uint32_t word) {
    const uint32_t e = word & 0x7f800000u;
    if (e == 0x7f800000u || (word & 0x7fffff00u) == 0) return 1.0f;
    return e ? __builtin_bit_cast(float, (word & 0x807fff00u) | 0x3f800000u) : scale_of(word) * 0x1p126f;
}

// u (q - z) of eight codes.
__device__ __forceinline__ halfx8 operand(uint32_t codes, uint32_t word, halfx8) {
    if (fabsf(scale_of(word)) < 0x1p-80f) codes = 0, word = 0;
    return codes_less(codes, zero_of(word), halfx8());
}
__device__ __forceinline__ bfloatx8 operand(uint32_t codes, uint32_t word, bfloatx8) {
    const uint32_t e = word & 0x7f800000u;
    // a scale that is not finite goes into the operand as it is
    const float u = e == 0x7f800000u ? scale_of(word) : __builtin_bit_cast(float, e ? e : (word & 0x7fff00u) ? 0x00800000u : 0u);
    const float zu = zero_of(word) * u;
    const uint32_t even = codes & 0x0f0f0f0fu, odd = (codes >> 4) & 0x0f0f0f0fu;
    bfloatx8 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        r[2 * j] = (__bf16)__builtin_fmaf((float)((even >> (8 * j)) & 255u), u, -zu);
        r[2 * j + 1] = (__bf16)__builtin_fmaf((float)((odd >> (8 * j)) & 255u), u, -zu);
    }
    return r;
}

struct ManyArgs {
    const void* x;       // parts planes of [M][ldx] operands
    int64_t ldx, plane;  // in elements
    int parts;
    int64_t M, pairs;    // pairs of stages: K in steps of 128
    Q4Linear w;
    int64_t tiles_m, tiles_n, per_split;  // pairs of a split
    float* sums;         // [splits][M][N], or null
};

constexpr int kStage = 64;  // inputs of a stage: a line of 128 bytes a row

// Slot of 16 bytes in which block b of eight inputs of a row stands: the lanes
// that LDS serves together read different banks.
__device__ __forceinline__ int slot_of(int row, int b) { return b ^ ((row >> 1 & 1) | (row >> 2 & 6)); }

// 32 rows (of m) by C columns of sums that a wave keeps in LDS to the output, 8
// columns a lane.
template <typename T, int C>
__device__ __forceinline__ void store_tile(const float* sums, int pitch, const ManyArgs& p, T* out, int64_t ldo, bool whole,
                                           int64_t m, int64_t n, int lane) {
    constexpr int L = C / 8;
    const int64_t n1 = n + (lane % L) * 8;
    float bias[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[e] = whole && p.w.bias ? p.w.bias[min(n1 + e, p.w.N - 1)] : 0.0f;
#pragma unroll
    for (int i = 0; i < 32 * L / 64; ++i) {
        const int r = i * (64 / L) + lane / L;
        if (m + r >= p.M) continue;
        float v[8];
        const float* from = sums + r * pitch + (lane % L) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = whole ? activate(from[e] + bias[e], p.w.act) : from[e];
        store8(out + (m + r) * ldo + n1, p.w.N - n1, v);
    }
}

// A block computes BM rows by BN outputs, a wave 32 TI by 32 TJ of them.  A
// stage is 64 inputs in one of two LDS buffers: the rows of x are copied there
// by the LDS-DMA loads, the codes pass through registers, where each thread
// turns 32 of them into operands between the current stage's products.
template <typename V, typename T, int G, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN) q4_matmul_kernel(ManyArgs p) {
    typedef typename Elem<V>::vec vec;
    constexpr int WAVES = WM * WN, TI = BM / WM / 32, TJ = BN / WN / 32, PER = 128 / G;
    constexpr int COPIES = BM / 8 / WAVES;
    static_assert(2 * BN == 64 * WAVES, "two threads for every row of codes");
    // apart, so that a read of one buffer need not wait for copies into the other
    __shared__ uintx4 x0[BM * 8], x1[BM * 8], w0[BN * 8], w1[BN * 8];
    const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t im, in;
    tile_of(blockIdx.x, p.tiles_m, p.tiles_n, im, in);
    const int64_t m0 = im * BM, n0 = in * BN;
    const int wm = wave % WM * 32 * TI, wn = wave / WM * 32 * TJ;
    const int64_t total = p.parts * p.pairs, q0 = blockIdx.y * p.per_split, q1 = min(q0 + p.per_split, total);
    const int64_t ldc = p.w.groups * (G / 2), ldw = q4_word_stride(p.w.groups);

    // this thread's copies of x: rows 8 (WAVES i + wave) + lane / 8
    const char* xrow[COPIES];
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
        const int row = 8 * (WAVES * i + wave) + (lane >> 3);
        xrow[i] = (const char*)p.x + (min(m0 + row, p.M - 1) * p.ldx + 8 * slot_of(row, lane & 7)) * 2;
    }
    const auto copy = [&](int64_t pair, int s) {
        const int64_t part = pair / p.pairs, at = (part * p.plane + (pair - part * p.pairs) * 128 + s * kStage) * 2;
#pragma unroll
        for (int i = 0; i < COPIES; ++i)
            __builtin_amdgcn_global_load_lds((const void*)(xrow[i] + at),
                                             (__attribute__((address_space(3))) void*)((s ? x1 : x0) + (WAVES * i + wave) * 64), 16, 0, 0);
    };
    // and its half row of codes
    const int crow = threadIdx.x >> 1, half = threadIdx.x & 1;
    const int64_t cn = min(n0 + crow, p.w.N - 1);
    struct Codes {
        uintx4 q[2];
        uint32_t w[2];
    };
    const auto load_codes = [&](int64_t pair) {
        Codes c;
        const int64_t k = pair % p.pairs;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int64_t at = k * 64 + 32 * s + 16 * half, g = at / (G / 2);
            c.q[s] = uintx4{0, 0, 0, 0};
            c.w[s] = 0;
            if (at < ldc) {
                c.q[s] = *reinterpret_cast<const uintx4*>(p.w.codes + cn * ldc + at);
                c.w[s] = p.w.words[cn * ldw + g];
            }
        }
        return c;
    };
    const auto convert = [&](const Codes& c, int s, int i, int buf) {
        const vec v = operand(c.q[s][i], c.w[s], vec());
        (buf ? w1 : w0)[crow * 8 + slot_of(crow, 4 * half + i)] = __builtin_bit_cast(uintx4, v);
    };
    // the words of this lane's columns
    const auto load_words = [&](int64_t pair, uint32_t (&w)[TJ][PER]) {
        const int64_t k = pair % p.pairs;
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            const int64_t n = min(n0 + wn + 32 * j + r, p.w.N - 1);
            __builtin_memcpy(w[j], p.w.words + n * ldw + k * PER, sizeof(w[j]));
#pragma unroll
            for (int g = 0; g < PER; ++g)
                if (k * PER + g >= p.w.groups) w[j][g] = 0;
        }
    };

    floatx16 acc[TI][TJ] = {};
    float unit[TJ];
    if (q0 < q1) {
        Codes cur = load_codes(q0), nxt;
        uint32_t word[TJ][PER], word_next[TJ][PER];
        load_words(q0, word);
        copy(q0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) convert(cur, 0, i, 0);
#pragma unroll
        for (int j = 0; j < TJ; ++j) unit[j] = unit_of<V>(word[j][0]);
        stage_barrier();
        for (int64_t pair = q0; pair < q1; ++pair) {
            const bool more = pair + 1 < q1;
            if (more) {
                nxt = load_codes(pair + 1);
                load_words(pair + 1, word_next);
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (s == 0)
                    copy(pair, 1);
                else if (more)
                    copy(pair + 1, 0);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if ((kStage * s + 16 * k) % G == 0) {
#pragma unroll
                        for (int j = 0; j < TJ; ++j) {
                            const float u = unit_of<V>(word[j][(kStage * s + 16 * k) / G]), f = unit[j] / u;
                            unit[j] = u;
#pragma unroll
                            for (int i = 0; i < TI; ++i)
#pragma unroll
                                for (int e = 0; e < 16; ++e) acc[i][j][e] *= f;
                        }
                    }
                    vec a[TI], b[TJ];
                    const int slot = slot_of(r, 2 * k + h);
#pragma unroll
                    for (int i = 0; i < TI; ++i) a[i] = __builtin_bit_cast(vec, (s ? x1 : x0)[(wm + 32 * i + r) * 8 + slot]);
#pragma unroll
                    for (int j = 0; j < TJ; ++j) b[j] = __builtin_bit_cast(vec, (s ? w1 : w0)[(wn + 32 * j + r) * 8 + slot]);
#pragma unroll
                    for (int i = 0; i < TI; ++i)
#pragma unroll
                        for (int j = 0; j < TJ; ++j) acc[i][j] = mfma(a[i], b[j], acc[i][j]);
                    if (s == 0)
                        convert(cur, 1, k, 1);
                    else if (more)
                        convert(nxt, 0, k, 0);
                }
                stage_barrier();
            }
            cur = nxt;
#pragma unroll
            for (int j = 0; j < TJ; ++j)
#pragma unroll
                for (int g = 0; g < PER; ++g) word[j][g] = word_next[j][g];
        }
    } else {
#pragma unroll
        for (int j = 0; j < TJ; ++j) unit[j] = 1.0f;
    }

    // The sums leave through LDS, 32 rows of a wave at a time, as whole lines.
    constexpr int PITCH = 32 * TJ;
    static_assert(WAVES / 2 * 32 * PITCH * 4 <= sizeof(x0), "half of the waves' rows fit");
    float* mine = reinterpret_cast<float*>(wave < WAVES / 2 ? x0 : x1) + wave % (WAVES / 2) * 32 * PITCH;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
        wave_lds_sync();
#pragma unroll
        for (int j = 0; j < TJ; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) mine[((e & 3) + 8 * (e >> 2) + 4 * h) * PITCH + 32 * j + r] = acc[i][j][e] * unit[j];
        wave_lds_sync();
        if (p.sums)
            store_tile<float, 32 * TJ>(mine, PITCH, p, p.sums + blockIdx.y * p.M * p.w.N, p.w.N, false, m0 + wm + 32 * i, n0 + wn, lane);
        else
            store_tile<T, 32 * TJ>(mine, PITCH, p, (T*)p.w.y, p.w.ldy, true, m0 + wm + 32 * i, n0 + wn, lane);
    }
}

// Rows of x as planes of operands [parts][M][Kp], zero past K.
template <typename T, typename V, int PARTS>
__global__ void __launch_bounds__(256) q4_pack_kernel(const T* x, int64_t ldx, int64_t M, int64_t K, int64_t Kp, V* out) {
    const int64_t chunks = Kp / 8, total = M * chunks;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / chunks, k = (i - m * chunks) * 8;
        typename Elem<V>::vec v[PARTS];
        split(load_raw(x + m * ldx + k, K - k), v);
#pragma unroll
        for (int h = 0; h < PARTS; ++h) __builtin_memcpy(out + (h * M + m) * Kp + k, &v[h], 16);
    }
}

// Sums of splits in order, then bias and activation.
template <typename T>
__global__ void __launch_bounds__(256) q4_join_kernel(const float* sums, int splits, int64_t M, Q4Linear p) {
    const int64_t total = M * p.N;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / p.N, n = i - m * p.N;
        float v = 0.0f;
        for (int s = 0; s < splits; ++s) v += sums[s * total + i];
        reinterpret_cast<T*>(p.y)[m * p.ldy + n] = (T)activate(v + (p.bias ? p.bias[n] : 0.0f), p.act);
    }
}

struct Plan {
    int tile;    // rows of a tile; outputs of a tile
    int splits;
    int64_t per_split;
};

Plan plan_of(int parts, int64_t M, int64_t K, int64_t N) {
    const int64_t pairs = ceil_div(K, 128) * parts;
    Plan p{256, 1, pairs};
    return p;
}

size_t pack_bytes(int parts, int64_t M, int64_t K) { return round_up((size_t)parts * (size_t)M * (size_t)ceil_div(K, 128) * 256); }

template <typename V, typename T, int G, int BM, int BN, int WM, int WN>
hipError_t run(const ManyArgs& a, int splits, hipStream_t s) {
    ManyArgs p = a;
    p.tiles_m = ceil_div(p.M, BM);
    p.tiles_n = ceil_div(p.w.N, BN);
    IA_LAUNCH("q4_matmul_kernel", (q4_matmul_kernel<V, T, G, BM, BN, WM, WN>), dim3((unsigned)(p.tiles_m * p.tiles_n), splits),
              dim3(64 * WM * WN), 0, s, p);
    return hipGetLastError();
}

template <typename V, typename T, int PARTS, int G>
hipError_t matmul(const T* x, int64_t M, int64_t ldx, const Q4Linear& w, void* ws, hipStream_t s) {
    const Plan plan = plan_of(PARTS, M, w.K, w.N);
    const int64_t Kp = ceil_div(w.K, 128) * 128;
    ManyArgs p{};
    p.M = M;
    p.parts = PARTS;
    p.pairs = Kp / 128;
    p.w = w;
    p.per_split = plan.per_split;
    // x as it is where its rows are whole lines of 16-bit values
    if (PARTS == 1 && w.K == Kp && (uintptr_t)x % 16 == 0 && ldx % 8 == 0) {
        p.x = x;
        p.ldx = ldx;
    } else {
        V* out = (V*)ws;
        IA_LAUNCH("q4_pack_kernel", (q4_pack_kernel<T, V, PARTS>), dim3(grid_for(M * Kp / 8)), dim3(256), 0, s, x, ldx, M, w.K, Kp, out);
        p.x = out;
        p.ldx = Kp;
        p.plane = M * Kp;
    }
    if (plan.splits > 1) p.sums = (float*)((char*)ws + pack_bytes(PARTS, M, w.K));
    hipError_t e = run<V, T, G, 256, 256, 2, 4>(p, plan.splits, s);
    if (e != hipSuccess || plan.splits == 1) return e;
    IA_LAUNCH("q4_join_kernel", q4_join_kernel<T>, dim3(grid_for(M * w.N)), dim3(256), 0, s, p.sums, plan.splits, M, w);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_matmul(const void* x, int64_t M, int64_t ldx, int group, const Q4Linear& w, void* ws, hipStream_t s) {
    typedef std::conditional_t<std::is_same<T, _Float16>::value, _Float16, __bf16> V;
    constexpr int PARTS = std::is_same<T, float>::value ? 3 : 1;
    const T* const t = (const T*)x;
    return group == 32   ? matmul<V, T, PARTS, 32>(t, M, ldx, w, ws, s)
           : group == 64 ? matmul<V, T, PARTS, 64>(t, M, ldx, w, ws, s)
                         : matmul<V, T, PARTS, 128>(t, M, ldx, w, ws, s);
}

}  // namespace

size_t q4_matmul_workspace(int32_t dtype, int64_t M, int64_t K, int64_t N) {
    const int parts = dtype == IA_DTYPE_F32 ? 3 : 1;
    const Plan p = plan_of(parts, M, K, N);
    return pack_bytes(parts, M, K) + (p.splits > 1 ? (size_t)p.splits * (size_t)M * (size_t)N * 4 : 0);
}

hipError_t launch_q4_matmul(const void* x, int32_t dtype, int64_t M, int64_t ldx, int group, const Q4Linear& p, void* ws,
                            hipStream_t s) {
    return IA_BY_DTYPE(dtype, launch_matmul, x, M, ldx, group, p, ws, s);
}

}  // namespace ia
