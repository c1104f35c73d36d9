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
//   bf16: u = the power of two of s, so 1 <= |m| < 2 and nothing grows; 2^123 at most
//   (15 u is in range) and 2^-126 at least, past which m goes on.
//   fp16: the same from 2^-24 to 2^8, where u (q - z) is a number of fp16; u ends
//   there, and m goes on below 1 and above 2.  Powers of two in s below 2^-66 count
//   as 2^-66: with the 2^20 inputs of less than 2^16 that tiles take, such groups add
//   less than 2^-25, half of fp16's least value.  (They are not left out: an infinite
//   input gives an infinity against any weight but zero.)  Those past 2^45 count as
//   2^45: fp16 inputs are at least 2^-24, so what such a group adds is 0 or at least
//   2^21, past fp16's range.  A sum, of 2^20 terms of at most 15 * 2^46 * 65504, is
//   below 2^86 then and in units of m, 2^-42 or more, below 2^128: a change of unit
//   never makes it infinite.
//   fp32 rows go as three bf16 parts of 8 bits each, cut off and not rounded,
//   which add up to them (to within 2^-133, where bf16 ends), one part after the
//   other.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

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

// The power of two in a scale, as bits, held between two powers.
__device__ __forceinline__ uint32_t power_of(uint32_t word, int least, int most) {
    return min(max(word & 0x7f800000u, (uint32_t)(127 + least) << 23), (uint32_t)(127 + most) << 23);
}
// A group's u in fp16, as bits.
__device__ __forceinline__ uint32_t half_unit(uint32_t word) { return power_of(word, -24, 8); }

constexpr int kMostPower = 123;  // of u in bf16: times 15 it is in range

// A group's m.
template <typename V>
__device__ __forceinline__ float unit_of(uint32_t word);
template <>
__device__ __forceinline__ float unit_of<_Float16>(uint32_t word) {
    return __builtin_bit_cast(float, (word & 0x807fff00u) | (power_of(word, -66, 45) - half_unit(word) + 0x3f800000u));
}
template <>
__device__ __forceinline__ float unit_of<__bf16>(uint32_t word) {
    const float s = scale_of(word);
    return s == 0.0f ? 1.0f : s * __builtin_bit_cast(float, (254u << 23) - power_of(word, -126, kMostPower));  // 1 / u
}

// What a group's word does to its codes; operands are u (q - z).
template <typename V>
struct Group;
template <>
struct Group<_Float16> {
    float u512;
    halfx2 zu;
    __device__ __forceinline__ explicit Group(uint32_t word) {
        // a scale that is not finite goes into the operand as it is, as zero does (codes times 2^-118 are zero in fp16)
        const bool other = (word & 0x7f800000u) == 0x7f800000u || (word & 0x7fffff00u) == 0;
        const uint32_t u = other ? word & 0x7fffff00u : half_unit(word);
        u512 = __builtin_bit_cast(float, u + (9u << 23));
        zu = twice(-zero_of(word) * __builtin_bit_cast(float, u));
    }
    __device__ __forceinline__ halfx8 operand(uint32_t codes) const { return codes_times(codes, u512, zu); }
};
template <>
struct Group<__bf16> {
    float u, zu;
    __device__ __forceinline__ explicit Group(uint32_t word) {
        const uint32_t e = word & 0x7f800000u, low = (word & 0x7fff00u) ? 0x00800000u : 0u;
        // a scale that is not finite goes into the operand as it is
        u = __builtin_bit_cast(float, e == 0x7f800000u ? word & ~255u : e ? power_of(word, -126, kMostPower) : low);
        zu = -zero_of(word) * u;
    }
    __device__ __forceinline__ bfloatx8 operand(uint32_t codes) const { return codes_times(codes, u, zu); }
};

// A pointer that is the same for all lanes, in scalar registers.
__device__ __forceinline__ const char* uniform(const char* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return reinterpret_cast<const char*>((uint64_t)hi << 32 | lo);
}

struct ManyArgs {
    const void* x;       // parts planes of [M][ldx] operands
    int64_t ldx, plane;  // in elements
    int parts;
    int64_t M, pairs;    // pairs of stages: K in steps of 128
    Q4Linear w;
    int64_t tile0, tiles_m, tiles_n;  // of the launch; of all
    int64_t per_split;   // pairs of a split
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
// stage is 64 inputs: the rows of x are copied into one of three LDS buffers by the
// LDS-DMA loads, the codes reach one of two through registers, where each thread
// turns 32 of them into operands between the current stage's products.  4,096 cubed
// in bf16 and groups of 128: 157 us of normally distributed rows, 144 of rows of
// different sizes (875 and 960 TFLOP/s; the library's product of bf16 matrices reaches 1,210).
// The matrix cores are busy 38 % of the time and the vector units, with conversions
// and the sums' changes of unit, 39 %: what does not overlap is the distance.  About
// 20 us are a tile's start and its stores, with one tile a CU.  Waves that raise their
// priority for the matrix instructions take 166, operands made before or in fixed turn
// with them no less.
template <typename V, typename T, int G, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN) q4_matmul_kernel(ManyArgs p) {
    typedef typename Elem<V>::vec vec;
    constexpr int WAVES = WM * WN, TI = BM / WM / 32, TJ = BN / WN / 32;
    constexpr int COPIES = BM / 8 / WAVES;
    static_assert(2 * BN == 64 * WAVES, "two threads for every row of codes");
    // apart, so that a read of one buffer need not wait for copies into the other
    __shared__ uintx4 x0[BM * 8], x1[BM * 8], x2[BM * 8], w0[BN * 8], w1[BN * 8];
    const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t im, in;
    tile_of(p.tile0 + blockIdx.x, p.tiles_m, p.tiles_n, im, in);
    const int64_t m0 = im * BM, n0 = in * BN;
    const int wm = wave % WM * 32 * TI, wn = wave / WM * 32 * TJ;
    const int64_t ldc = p.w.groups * (G / 2), ldw = q4_word_stride(p.w.groups);

    // The pairs of stages of this split, one after the other through the parts of
    // x.  Addresses are uniform, the threads' offsets to them have 32 bits.
    struct At {
        const char* x;  // the tile's first row there
        int k;          // pair of the weights
    };
    const int pairs = (int)p.pairs, groups = (int)p.w.groups;
    const int q0 = (int)(blockIdx.y * p.per_split), q1 = (int)min((int64_t)q0 + p.per_split, p.parts * p.pairs);
    At at{(const char*)p.x + (q0 / pairs * p.plane + m0 * p.ldx + q0 % pairs * 128) * 2, q0 % pairs};
    const auto advance = [&](At& t) {
        t.x += 256;
        if (++t.k == pairs) {
            t.k = 0;
            t.x += (p.plane - p.pairs * 128) * 2;
        }
    };
    // this thread's copies of x: rows 8 (WAVES i + wave) + lane / 8
    uint32_t xoff[COPIES];
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
        const int row = 8 * (WAVES * i + wave) + (lane >> 3);
        xoff[i] = (uint32_t)((min((int64_t)row, p.M - 1 - m0) * p.ldx + 8 * slot_of(row, lane & 7)) * 2);
    }
    const auto copy = [&](const char* x, uintx4* to) {
        x = uniform(x);
#pragma unroll
        for (int i = 0; i < COPIES; ++i)
            __builtin_amdgcn_global_load_lds((const void*)(x + xoff[i]),
                                             (__attribute__((address_space(3))) void*)(to + (WAVES * i + wave) * 64), 16, 0, 0);
    };
    // and its half row of codes: 16 bytes and their word each stage
    // (neighbouring threads take rows whose slots differ: their stores meet different banks)
    const int ct = threadIdx.x >> 1, half = threadIdx.x & 1;
    const int crow = (ct & ~15) | (ct & 1) << 1 | (ct & 2) << 2 | (ct >> 2 & 1) | (ct >> 1 & 4);
    const uint8_t* const codes = p.w.codes + n0 * ldc;
    const uint32_t* const words = p.w.words + n0 * ldw;
    const uint32_t cn = (uint32_t)min((int64_t)crow, p.w.N - 1 - n0), coff = cn * (uint32_t)ldc + 16 * half, cw = cn * (uint32_t)ldw;
    const int last_block = groups * (G / 32) - 1;  // of 32 inputs
    struct Codes {
        uintx4 q;
        uint32_t w;
    };
    const auto load_codes = [&](int k, int s) {
        const int here = min(4 * k + 2 * s + half, last_block);  // past the row's end: the last codes again
        Codes c;
        c.q = *reinterpret_cast<const uintx4*>(codes + (coff + 16 * (here - half)));
        c.w = words[cw + here / (G / 32)];
        return c;
    };
    // and there their scale is zero
    const auto group_of = [&](const Codes& c, int k, int s) { return Group<V>(4 * k + 2 * s + half <= last_block ? c.w : 0u); };
    int wslot[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) wslot[i] = crow * 8 + slot_of(crow, 4 * half + i);
    // the words of this lane's columns, those of a stage
    constexpr int PER = G < kStage ? kStage / G : 1;
    uint32_t dw[TJ];
#pragma unroll
    for (int j = 0; j < TJ; ++j) dw[j] = (uint32_t)min((int64_t)(wn + 32 * j + r), p.w.N - 1 - n0) * (uint32_t)ldw;
    const auto load_words = [&](int k, int s, uint32_t (&w)[TJ][PER]) {
        const int g0 = (128 * k + kStage * s) / G;
#pragma unroll
        for (int j = 0; j < TJ; ++j)
#pragma unroll
            for (int g = 0; g < PER; ++g) w[j][g] = words[dw[j] + min(g0 + g, groups - 1)];  // past the end: no matter, times zero
    };

    floatx16 acc[TI][TJ] = {};
    float unit[TJ];
#pragma unroll
    for (int j = 0; j < TJ; ++j) unit[j] = 1.0f;
    if (q0 < q1) {
        uint32_t word[TJ][PER];
        load_words(at.k, 0, word);
        Codes code = load_codes(at.k, 0);
        copy(at.x, x0);
        copy(at.x + 128, x1);
        {
            const Group<V> g = group_of(code, at.k, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) w0[wslot[i]] = __builtin_bit_cast(uintx4, g.operand(code.q[i]));
        }
        code = load_codes(at.k, 1);
#pragma unroll
        for (int j = 0; j < TJ; ++j) unit[j] = unit_of<V>(word[j][0]);
        stage_barrier();
        // Copies land in the order of their issue: the next stage has landed when
        // no more are under way than the last COPIES.
        const auto ready = [] { asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(COPIES) : "memory"); };
        // Stage s of a pair out of xa and wb; meanwhile the next one's codes become
        // operands in wc, those of the one after it are loaded and its x is
        // copied from `from` to xc.
        const auto stage = [&](auto half_pair, const At& then, const uintx4* xa, const uintx4* wb, uintx4* xc, uintx4* wc) {
            constexpr int s = decltype(half_pair)::value;
            Codes more = load_codes(then.k, s);
            uint32_t word_next[TJ][PER];
            if (s == 1 || G < 128) load_words(s ? then.k : at.k, s ^ 1, word_next);
            __builtin_amdgcn_sched_barrier(0);  // the copies come last
            copy(then.x + s * 128, xc);
            __builtin_amdgcn_sched_barrier(0);
            const Group<V> group = s ? group_of(code, then.k, 0) : group_of(code, at.k, 1);
            vec a[2][TI], b[2][TJ];  // this step's operands and the next one's
            const auto read = [&](int k) {
                const int slot = slot_of(r, 2 * k + h);
#pragma unroll
                for (int i = 0; i < TI; ++i) a[k & 1][i] = __builtin_bit_cast(vec, xa[(wm + 32 * i + r) * 8 + slot]);
#pragma unroll
                for (int j = 0; j < TJ; ++j) b[k & 1][j] = __builtin_bit_cast(vec, wb[(wn + 32 * j + r) * 8 + slot]);
            };
            read(0);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k < 3) read(k + 1);
                if ((kStage * s + 16 * k) % G == 0) {
#pragma unroll
                    for (int j = 0; j < TJ; ++j) {
                        const float u = unit_of<V>(word[j][16 * k / G]), f = unit[j] / u;
                        unit[j] = u;
#pragma unroll
                        for (int i = 0; i < TI; ++i)
#pragma unroll
                            for (int e = 0; e < 16; ++e) acc[i][j][e] *= f;
                    }
                }
#pragma unroll
                for (int i = 0; i < TI; ++i)
#pragma unroll
                    for (int j = 0; j < TJ; ++j) acc[i][j] = mfma(a[k & 1][i], b[k & 1][j], acc[i][j]);
                wc[wslot[k]] = __builtin_bit_cast(uintx4, group.operand(code.q[k]));
            }
            // what was loaded is used from here on, not waited for above
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("" : "+v"(more.q), "+v"(more.w));
            code = more;
            if (s == 1 || G < 128)
#pragma unroll
                for (int j = 0; j < TJ; ++j)
#pragma unroll
                    for (int g = 0; g < PER; ++g) {
                        asm volatile("" : "+v"(word_next[j][g]));
                        word[j][g] = word_next[j][g];
                    }
            ready();
        };
        const auto pair_of = [&](int pair, uintx4* xa, uintx4* xb, uintx4* xc) {
            // the last pair makes itself ready again, for nothing
            At then = at;
            if (pair + 1 < q1) advance(then);
            stage(std::integral_constant<int, 0>{}, then, xa, w0, xc, w1);
            stage(std::integral_constant<int, 1>{}, then, xb, w1, xa, w0);
            at = then;
        };
        for (int pair = q0;;) {
            pair_of(pair, x0, x1, x2);
            if (++pair >= q1) break;
            pair_of(pair, x2, x0, x1);
            if (++pair >= q1) break;
            pair_of(pair, x1, x2, x0);
            if (++pair >= q1) break;
        }
        stage_barrier();
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

int parts_of(int32_t dtype) { return dtype == IA_DTYPE_F32 ? 3 : 1; }

// Microseconds that a product takes, as measured on bf16 in groups of 128 over M of
// 33 to 100,000, K of 32 to 8,192 and N of 58 to 11,008 (in brackets a case):
//   few rows' kernel: 16 outputs of 64 rows a block, 256 blocks side by side take
//     16.3 for 4,096 inputs (fp32 twice that), 1.75 at least (256 x 8,192 -> 1,024: 36)
//   tiles of 128: 6.5 and 1.75 a pair of stages for up to 256 blocks, 0.8 of that
//     for each 256 more, two to a CU (2,048 x 4,096 -> 4,096: 101)
//   tiles of 256: 4 and 3.7 a pair for up to 128 blocks, 8 and 4.8 for 256 (4,096
//     cubed: 163, in tiles of 128 226)
//   joining splits: 3 and 8 bytes a sum at 4 TB/s (128 x 4,096 -> 4,096 in four
//     splits: 28, in one 59).
// It stands for the other types and groups as well, whose tiles take longer: 4,096 cubed
// in groups of 32 takes 244 where this says 200.  Packing x, for fp32 rows and for
// rows that are no whole lines, is not counted.
enum Way { kFew, kSmall, kLarge };
struct Plan {
    Way way;
    int splits;
    int64_t per_split;
};

Plan plan_of(int32_t dtype, int group, int64_t M, int64_t K, int64_t N) {
    const int parts = parts_of(dtype);
    const int64_t pairs = ceil_div(K, 128) * parts;
    const auto tiles = [&](int64_t m, int64_t n) { return (double)(ceil_div(M, m) * ceil_div(N, n)); };
    Plan best{kFew, 1, pairs};
    // a tile's offsets have 32 bits, fp16 sums 2^20 terms
    if (M <= 16 || K >= (int64_t)1 << (dtype == IA_DTYPE_F16 ? 20 : 22)) return best;
    double least = 2.5 + std::max(0.8, tiles(64, 16) / 256) * std::max(1.75, (parts > 1 ? 32.6 : 16.3) * (double)K / 4096);
    const auto offer = [&](Way way, int64_t splits, double blocks) {
        const int64_t per = ceil_div(pairs, splits);
        double t;
        if (way == kSmall)
            t = std::max(1.0, 0.8 * blocks / 256) * (6.5 + 1.75 * (double)per);
        else
            t = blocks <= 128 ? 4 + 3.7 * (double)per : std::ceil(blocks / 256) * (8 + 4.8 * (double)per);
        if (splits > 1) t += 3 + (double)splits * (double)M * (double)N * 8 / 4e6;
        if (t < least) least = t, best = Plan{way, (int)ceil_div(pairs, per), per};
    };
    for (int64_t s = 1; s <= 8 && s <= pairs; s *= 2) {
        offer(kSmall, s, tiles(128, 128) * (double)s);
        // with groups of 32 the wide tile's sums do not fit the registers
        if (group > 32) offer(kLarge, s, tiles(256, 256) * (double)s);
    }
    return best;
}

size_t pack_bytes(int parts, int64_t M, int64_t K) { return round_up((size_t)parts * (size_t)M * (size_t)ceil_div(K, 128) * 256); }

template <typename V, typename T, int G, int BM, int BN, int WM, int WN>
hipError_t run(const ManyArgs& a, int splits, hipStream_t s) {
    ManyArgs p = a;
    p.tiles_m = ceil_div(p.M, BM);
    p.tiles_n = ceil_div(p.w.N, BN);
    const int64_t tiles = p.tiles_m * p.tiles_n, most = 1 << 20;  // a grid has less than 2^32 threads
    for (p.tile0 = 0; p.tile0 < tiles; p.tile0 += most)
        IA_LAUNCH(BM == 256 ? "q4_matmul_kernel<256>" : "q4_matmul_kernel<128>", (q4_matmul_kernel<V, T, G, BM, BN, WM, WN>),
                  dim3((unsigned)std::min(most, tiles - p.tile0), splits), dim3(64 * WM * WN), 0, s, p);
    return hipGetLastError();
}

template <typename V, typename T, int PARTS, int G>
hipError_t matmul(const Plan& plan, const T* x, int64_t M, int64_t ldx, const Q4Linear& w, void* ws, hipStream_t s) {
    const int64_t Kp = ceil_div(w.K, 128) * 128;
    ManyArgs p{};
    p.M = M;
    p.parts = PARTS;
    p.pairs = Kp / 128;
    p.w = w;
    p.per_split = plan.per_split;
    // x as it is where its rows are whole lines of 16-bit values and a tile's offsets fit 32 bits
    if (PARTS == 1 && w.K == Kp && (uintptr_t)x % 16 == 0 && ldx % 8 == 0 && ldx < (int64_t)1 << 22) {
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
    hipError_t e;
    if constexpr (G > 32)
        e = plan.way == kLarge ? run<V, T, G, 256, 256, 2, 4>(p, plan.splits, s) : run<V, T, G, 128, 128, 2, 2>(p, plan.splits, s);
    else
        e = run<V, T, G, 128, 128, 2, 2>(p, plan.splits, s);
    if (e != hipSuccess || plan.splits == 1) return e;
    IA_LAUNCH("q4_join_kernel", q4_join_kernel<T>, dim3(grid_for(M * w.N)), dim3(256), 0, s, p.sums, plan.splits, M, w);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_matmul(const void* x, int64_t M, int64_t ldx, int group, const Q4Linear& w, void* ws, hipStream_t s) {
    typedef std::conditional_t<std::is_same<T, _Float16>::value, _Float16, __bf16> V;
    constexpr int PARTS = std::is_same<T, float>::value ? 3 : 1;
    const T* const t = (const T*)x;
    constexpr int32_t DTYPE = PARTS > 1 ? IA_DTYPE_F32 : std::is_same<T, _Float16>::value ? IA_DTYPE_F16 : IA_DTYPE_BF16;
    const Plan plan = plan_of(DTYPE, group, M, w.K, w.N);
    return group == 32   ? matmul<V, T, PARTS, 32>(plan, t, M, ldx, w, ws, s)
           : group == 64 ? matmul<V, T, PARTS, 64>(plan, t, M, ldx, w, ws, s)
                         : matmul<V, T, PARTS, 128>(plan, t, M, ldx, w, ws, s);
}

}  // namespace

bool q4_takes_tiles(int32_t dtype, int group, int64_t M, int64_t K, int64_t N) {
    return K > 0 && plan_of(dtype, group, M, K, N).way != kFew;
}

size_t q4_matmul_workspace(int32_t dtype, int64_t M, int64_t K, int64_t N) {
    const int parts = parts_of(dtype);
    size_t most = 0;  // of any group
    for (int group : {32, 128}) {
        const Plan p = plan_of(dtype, group, M, K, N);
        if (K > 0 && p.way != kFew)
            most = std::max(most, pack_bytes(parts, M, K) + (p.splits > 1 ? (size_t)p.splits * (size_t)M * (size_t)N * 4 : 0));
    }
    return most;
}

hipError_t launch_q4_matmul(const void* x, int32_t dtype, int64_t M, int64_t ldx, int group, const Q4Linear& p, void* ws,
                            hipStream_t s) {
    return IA_BY_DTYPE(dtype, launch_matmul, x, M, ldx, group, p, ws, s);
}

}  // namespace ia
