// Product of two MXFP4 matrices, C[m][n] = act(sum_k a[m][k] b[n][k] + bias[n]),
// on v_mfma_scale_f32_32x32x64_f8f6f4 (wave64, lane l, h = l / 32, r = l % 32:
// a lane supplies row r of its operand at the 32 values of k-block h, 16 bytes,
// and that block's scale; D holds rows (e % 4) + 8 (e / 4) + 4 h, e = 0..15, of
// the first operand against row r of the second, accumulated in fp32).
//
// A block computes a tile of R x R; a wave 64 rows m by 128 or 64 columns n of
// it.  The codes of 8 blocks (256 values, one 128-byte line of a row) of every
// row pass through LDS in two buffers, copied there by the LDS-DMA loads one
// stage ahead.  The operands of the next MFMA step (64 values) are read from
// LDS while the current step's products run, across the stages' barrier too:
// the barrier stands before the last step of a stage, when every wave has that
// step's operands in registers and the next stage's codes have landed.
//   Block b of a row stands in slot b ^ key(row) of its line, so that the 16
// lanes that LDS serves in one cycle (0-3, 12-15, 20-23, 24-27 and the like;
// rows alternate between its two halves of 128 bytes) read 16 different banks.
//   The n rows are the first operand: row i of n tile j stands for
// n = 32 j + 16 (i / 4 % 2) + i % 4 + 4 (i / 8), so that a lane ends with 16
// consecutive n of one row m and stores them together.
//   Rows past the end repeat the last one (their results are not stored).
// Blocks past the end of a row are other rows' codes with scale byte 0 on both
// sides: such a product is below 2^-240, under half of fp32's smallest value.
//   Bound by the matrix cores and the power they draw; the figures stand at
// mat_plan.
#include "mx4_common.h"

namespace ia {
namespace {

struct MatArgs {
    const uint8_t* a;   // M rows of `blocks` blocks
    const uint8_t* as;
    const uint8_t* b;   // N rows
    const uint8_t* bs;
    int64_t M, N, blocks;
    const float* bias;  // [N] or null
    int act;
    void* c;            // [M][ldc]; with splits [splits][M][N] fp32
    int64_t ldc;
    int64_t tiles_m, tiles_n, stages;  // tiles, and stages of 8 blocks a split takes
};

constexpr int kStageBlocks = 8;

// Bits 1, 3 and 4 of the lane row of either operand (n_row spreads b's bits).
__device__ __forceinline__ int key_a(int row) { return (row >> 1 & 1) | (row >> 2 & 6); }
__device__ __forceinline__ int key_b(int row) { return row >> 1 & 7; }

// The row (within a wave's n rows) that is lane row i of n tile j.
__device__ __forceinline__ int n_row(int j, int i) { return 32 * j + 16 * (i >> 2 & 1) + (i & 3) + 4 * (i >> 3); }

// The copies of one operand's tile rows into LDS: a uniform base that follows
// the stages and lane offsets, of 32 bits (OFF) where a tile's rows span less
// than 2^32 bytes.  Blocks past the end of a row are the next row's, or for
// the last row the operand's last block.
template <typename OFF, int ROWS, int WAVES, bool B>
struct Codes {
    static constexpr int N = ROWS / 8 / WAVES;  // copies of 8 rows a wave
    const uint8_t* base;  // first block of the tile's first row
    int64_t bytes;        // from there to the operand's end, less one block
    OFF off[N];

    __device__ __forceinline__ Codes(const uint8_t* codes, int64_t row0, int64_t rows, int64_t blocks, int wave,
                                     int lane) {
        base = codes + row0 * blocks * 16;
        bytes = (rows - row0) * blocks * 16 - 16;
        const int64_t last = rows - 1 - row0;
        // the keys take bits up to 4 of the row, the same for all of a wave's copies
        const int r = 8 * wave + (lane >> 3), slot = (lane & 7) ^ (B ? key_b(r) : key_a(r));
#pragma unroll
        for (int i = 0; i < N; ++i)
            off[i] = (OFF)(min((int64_t)(8 * WAVES * i + r), last) * blocks * 16 + slot * 16);
    }

    // blocks 8 t .. 8 t + 7
    __device__ __forceinline__ void copy(intx4* buf, int t, int wave) const {
        const int64_t skip = (int64_t)t * (kStageBlocks * 16), left = max(bytes - skip, (int64_t)0);
        const uint8_t* at = base + min(skip, bytes);
        const OFF most = sizeof(OFF) == 4 ? (OFF)min(left, (int64_t)0xffffffff) : (OFF)left;
#pragma unroll
        for (int i = 0; i < N; ++i)
            __builtin_amdgcn_global_load_lds((const void*)(at + min(off[i], most)),
                                             (__attribute__((address_space(3))) void*)(buf + (WAVES * i + wave) * 64),
                                             16, 0, 0);
    }
};

// Scale bytes of one row of a tile.
template <typename OFF>
struct ScaleRow {
    const uint8_t* base;  // uniform: the tile's first row
    OFF off;
    int64_t left;  // bytes from base to the operand's end
    int blocks;

    __device__ __forceinline__ ScaleRow(const uint8_t* scales, int64_t row0, int64_t rows, int64_t nblocks, int row) {
        base = scales + row0 * nblocks;
        off = (OFF)(min((int64_t)row, rows - 1 - row0) * nblocks);
        left = (rows - row0) * nblocks;
        blocks = (int)nblocks;
    }

    // Bytes k0 .. k0 + 15 of the row: one 16-byte load, from before its place
    // where it would pass the operand's end (finish() shifts it).  Needs 16
    // bytes from base on: so for every k0 >= 16 within the row.
    __device__ __forceinline__ uint4 load(int k0) const {
        uint4 w = {0, 0, 0, 0};
        if (k0 < blocks) {
            const int64_t room = left - 16 - k0;
            __builtin_memcpy(&w, base + k0 + min(room, (int64_t)0) + min(off, most(room)), 16);
        }
        return w;
    }

    // The same for the first group, byte by byte where fewer are left.
    __device__ __forceinline__ uint4 load_first(int k0) const {
        if (left >= 16) return load(k0);
        uint64_t v[2] = {0, 0};
#pragma unroll 1
        for (int i = 0; i < blocks; ++i) {
            const uint64_t byte = (uint64_t)base[off + (OFF)i] << (8 * (i & 7));
            v[0] |= i < 8 ? byte : 0;
            v[1] |= i < 8 ? 0 : byte;
        }
        return make_uint4((uint32_t)v[0], (uint32_t)(v[0] >> 32), (uint32_t)v[1], (uint32_t)(v[1] >> 32));
    }

    // The loaded bytes in their places, zero past the row's end, as four
    // words: the even blocks of the first stage, its odd ones, and the same of
    // the second stage.
    __device__ __forceinline__ uint4 finish(uint4 w, int k0) const {
        uint64_t v[2] = {(uint64_t)w.y << 32 | w.x, (uint64_t)w.w << 32 | w.z};
        if (left >= 16) {
            const int64_t room = left - 16 - k0;
            const uint32_t s = 8 * (uint32_t)(off - min(off, most(room)) - (OFF)min(room, (int64_t)0)) & 127u;
            const uint64_t up = (v[1] << 1) << (63 - (s & 63));
            v[0] = s < 64 ? v[0] >> s | up : v[1] >> (s & 63);
            v[1] = s < 64 ? v[1] >> s : 0;
        }
        const int n = max(blocks - k0, 0);  // uniform
        v[0] &= n < 8 ? ((uint64_t)1 << (8 * n)) - 1 : ~(uint64_t)0;
        v[1] &= n < 16 ? ((uint64_t)1 << (8 * max(n - 8, 0))) - 1 : ~(uint64_t)0;
        const uint32_t a = (uint32_t)v[0], b = (uint32_t)(v[0] >> 32), c = (uint32_t)v[1], d = (uint32_t)(v[1] >> 32);
        return make_uint4(__builtin_amdgcn_perm(b, a, 0x06040200u), __builtin_amdgcn_perm(b, a, 0x07050301u),
                          __builtin_amdgcn_perm(d, c, 0x06040200u), __builtin_amdgcn_perm(d, c, 0x07050301u));
    }

    static __device__ __forceinline__ OFF most(int64_t room) {
        room = max(room, (int64_t)0);
        return sizeof(OFF) == 4 ? (OFF)min(room, (int64_t)0xffffffff) : (OFF)room;
    }
};

// 32 rows by C columns of sums, which a wave keeps in LDS (16-byte units, unit u
// of row r in place u ^ r), to the output: a lane takes runs of 16 bytes, so
// that an instruction writes whole lines.
template <typename T, int C>
__device__ __forceinline__ void store_rows(const floatx4* sums, const MatArgs& p, T* out, int64_t m, int64_t n, int lane) {
    constexpr int E = 16 / (int)sizeof(T), L = C / E, UNITS = C / 4;  // values a run, lanes a row
    const int64_t n1 = n + (lane % L) * E;
    float bias[E];
#pragma unroll
    for (int e = 0; e < E; ++e) bias[e] = p.bias ? p.bias[min(n1 + e, p.N - 1)] : 0.0f;
#pragma unroll
    for (int i = 0; i < 32 * L / 64; ++i) {
        const int r = i * (64 / L) + lane / L;
        if (m + r >= p.M) continue;
        T o[E];
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            const floatx4 v = sums[r * UNITS + (((lane % L) * (E / 4) + e / 4) ^ (r % UNITS))];
#pragma unroll
            for (int k = 0; k < 4; ++k) o[e + k] = (T)activate(v[k] + bias[e + k], p.act);
        }
        T* to = out + (m + r) * p.ldc + n1;
        if (n1 + E <= p.N) {
            __builtin_memcpy(to, o, sizeof(o));
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (n1 + e < p.N) to[e] = o[e];
        }
    }
}

// Tile index of a block so that blocks of one XCD (every eighth block) take
// neighbouring tiles: runs of 8 tile rows, column by column.
__device__ __forceinline__ void tile_of(int64_t b, int64_t tm, int64_t tn, int64_t& im, int64_t& in) {
    const int64_t total = tm * tn, per = total / 8, rest = total % 8, x = b % 8;
    int64_t t = x * per + min(x, rest) + b / 8;
    const int64_t group = 8 * tn, g = t / group, h = min((int64_t)8, tm - 8 * g);
    t -= g * group;
    im = 8 * g + t % h;
    in = t / h;
}

// Operands of one step of 64 values.
template <int TI, int TJ>
struct Step {
    intx4 a[TI], b[TJ];

    __device__ __forceinline__ void read(const intx4* la, const intx4* lb, int s, int wm, int wn, int lane) {
        const int r = lane & 31, slot = (2 * s + (lane >> 5)) ^ key_a(r);  // key_b(n_row(j, r)) too
#pragma unroll
        for (int i = 0; i < TI; ++i) a[i] = la[(wm + 32 * i + r) * 8 + slot];
#pragma unroll
        for (int j = 0; j < TJ; ++j) b[j] = lb[(wn + n_row(j, r)) * 8 + slot];
    }
};

// Scales of one stage: byte s of a word is the lane's block in step s.
template <int TI, int TJ>
struct Scales {
    int a[TI], b[TJ];

    // rows: the words of the tile's rows, of a and then of b
    template <int R>
    __device__ __forceinline__ void read(const uint4* rows, int stage, int wm, int wn, int lane) {
        const int r = lane & 31, word = 2 * stage + (lane >> 5);
#pragma unroll
        for (int i = 0; i < TI; ++i) a[i] = reinterpret_cast<const int*>(rows + wm + 32 * i + r)[word];
#pragma unroll
        for (int j = 0; j < TJ; ++j) b[j] = reinterpret_cast<const int*>(rows + R + wn + n_row(j, r))[word];
    }
};

template <int S, int TI, int TJ>
__device__ __forceinline__ void multiply(const Step<TI, TJ>& o, const Scales<TI, TJ>& sc, floatx16 (&acc)[TI][TJ]) {
    __builtin_amdgcn_sched_barrier(0);  // the next step's reads stay above
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = mfma32<S>(o.b[j], sc.b[j], o.a[i], sc.a[i], acc[i][j]);
    // the sums exist here: left to the compiler, products sink behind the
    // next barrier
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) asm volatile("" : "+v"(acc[i][j]));
    __builtin_amdgcn_sched_barrier(0);
}

// LDS written by the lanes of one wave is read back by other lanes of the same
// wave: order the accesses at wavefront scope.
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Every copy of this wave has landed, and every wave's after the barrier.
__device__ __forceinline__ void stage_barrier() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
}

template <typename T, typename OFF, int R, int WAVES_M, int WAVES_N>
__global__ void __launch_bounds__(64 * WAVES_M * WAVES_N) mx4_matmul_kernel(MatArgs p) {
    constexpr int WAVES = WAVES_M * WAVES_N, TI = R / WAVES_M / 32, TJ = R / WAVES_N / 32;
    __shared__ intx4 a0[R * 8], a1[R * 8], b0[R * 8], b1[R * 8];
    __shared__ uint4 scales[2][2 * R];  // the rows of a, then of b
    static_assert(64 * WAVES == 2 * R, "a thread for every row's scales");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t im, in;
    tile_of(blockIdx.x, p.tiles_m, p.tiles_n, im, in);
    const int64_t m0 = im * R, n0 = in * R;
    const int wm = wave % WAVES_M * 32 * TI, wn = wave / WAVES_M * 32 * TJ;
    const int blocks = (int)p.blocks;
    const int t0 = (int)(blockIdx.y * p.stages), t1 = min(t0 + (int)p.stages, (blocks + kStageBlocks - 1) / kStageBlocks);
    const Codes<OFF, R, WAVES, false> ca(p.a, m0, p.M, p.blocks, wave, lane);
    const Codes<OFF, R, WAVES, true> cb(p.b, n0, p.N, p.blocks, wave, lane);
    const bool of_a = wave < WAVES / 2;
    const ScaleRow<OFF> row(of_a ? p.as : p.bs, of_a ? m0 : n0, of_a ? p.M : p.N, p.blocks, (int)threadIdx.x % R);
    floatx16 acc[TI][TJ] = {};

    // Stages go in pairs that share a group of scales; the missing second half
    // of a last pair has zero scales.
    if (t0 < t1) {
        Step<TI, TJ> x, y;
        Scales<TI, TJ> sc, sd;
        ca.copy(a0, t0, wave);
        cb.copy(b0, t0, wave);
        scales[0][threadIdx.x] = row.finish(row.load_first(t0 * kStageBlocks), t0 * kStageBlocks);
        stage_barrier();
        // scales are read before copies start: the compiler lets a read of
        // them wait for every copy in flight
        sc.template read<R>(scales[0], 0, wm, wn, lane);
        __builtin_amdgcn_sched_barrier(0);
        ca.copy(a1, t0 + 1, wave);
        cb.copy(b1, t0 + 1, wave);
        x.read(a0, b0, 0, wm, wn, lane);
        int buf = 0;
        for (int t = t0; t < t1; t += 2, buf ^= 1) {
            const uint4 next = row.load((t + 2) * kStageBlocks);
            y.read(a0, b0, 1, wm, wn, lane);
            multiply<0>(x, sc, acc);
            x.read(a0, b0, 2, wm, wn, lane);
            multiply<1>(y, sc, acc);
            y.read(a0, b0, 3, wm, wn, lane);
            multiply<2>(x, sc, acc);
            scales[buf ^ 1][threadIdx.x] = row.finish(next, (t + 2) * kStageBlocks);
            stage_barrier();
            sd.template read<R>(scales[buf], 1, wm, wn, lane);
            __builtin_amdgcn_sched_barrier(0);
            if (t + 2 < t1) {
                ca.copy(a0, t + 2, wave);
                cb.copy(b0, t + 2, wave);
            }
            x.read(a1, b1, 0, wm, wn, lane);
            multiply<3>(y, sc, acc);
            y.read(a1, b1, 1, wm, wn, lane);
            multiply<0>(x, sd, acc);
            x.read(a1, b1, 2, wm, wn, lane);
            multiply<1>(y, sd, acc);
            y.read(a1, b1, 3, wm, wn, lane);
            multiply<2>(x, sd, acc);
            stage_barrier();
            sc.template read<R>(scales[buf ^ 1], 0, wm, wn, lane);
            __builtin_amdgcn_sched_barrier(0);
            if (t + 3 < t1) {
                ca.copy(a1, t + 3, wave);
                cb.copy(b1, t + 3, wave);
            }
            x.read(a0, b0, 0, wm, wn, lane);
            multiply<3>(y, sd, acc);
        }
    }
    // The sums leave through LDS, 32 rows of a wave at a time: a lane holds 16
    // columns of one row, and stores of those alone write lines piece by piece
    // (measured with that change alone: 4,096^3 in bf16 58 -> 48 us, 150,000 x 32 -> 512
    // in fp16 127 -> 76).
    constexpr int C = 32 * TJ;
    static_assert(32 * C * 4 * WAVES <= 4 * R * 8 * 16, "the buffers hold every wave's rows");
    __syncthreads();
    constexpr int EACH = R * 8 / (32 * C / 4);  // waves a buffer holds
    floatx4* sums = reinterpret_cast<floatx4*>(wave / EACH == 0 ? a0 : wave / EACH == 1 ? a1 : wave / EACH == 2 ? b0 : b1) +
                    wave % EACH * (32 * C / 4);
    T* out = reinterpret_cast<T*>(p.c) + (int64_t)blockIdx.y * p.M * p.N;
    const int r = lane & 31;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
#pragma unroll
        for (int j = 0; j < TJ; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                sums[r * (C / 4) + ((8 * j + 4 * (lane >> 5) + k) ^ (r % (C / 4)))] =
                    floatx4{acc[i][j][4 * k], acc[i][j][4 * k + 1], acc[i][j][4 * k + 2], acc[i][j][4 * k + 3]};
        wave_lds_sync();
        store_rows<T, C>(sums, p, out, m0 + wm + 32 * i, n0 + wn, lane);
        wave_lds_sync();
    }
}

// The splits of a long sum added in a fixed order: c = act(sum of part[s] +
// bias).  A thread adds four neighbouring outputs over every WAYS-th split, and
// the WAYS waves' sums meet in LDS.
template <typename T, int WAYS>
__global__ void __launch_bounds__(256) mx4_join_kernel(MatArgs p, const float* part, int splits) {
    __shared__ floatx4 sum[WAYS][256 / WAYS];
    const int64_t total = p.M * p.N;
    const int way = threadIdx.x / (256 / WAYS), u = threadIdx.x % (256 / WAYS);
    const int64_t i = ((int64_t)blockIdx.x * (256 / WAYS) + u) * 4;
    floatx4 v = {};
    if (i + 4 <= total) {
#pragma unroll 8
        for (int s = way; s < splits; s += WAYS) {
            floatx4 w;
            __builtin_memcpy(&w, part + s * total + i, sizeof(w));
            v += w;
        }
    } else {
        for (int s = way; s < splits; s += WAYS)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < total) v[e] += part[s * total + i + e];
    }
    if (WAYS > 1) {
        sum[way][u] = v;
        __syncthreads();
        if (way != 0) return;
#pragma unroll
        for (int w = 1; w < WAYS; ++w) v += sum[w][u];
    }
    if (i >= total) return;
    int64_t m = i / p.N, n = i - m * p.N;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (i + e >= total) return;
        reinterpret_cast<T*>(p.c)[m * p.ldc + n] = (T)activate(v[e] + (p.bias ? p.bias[n] : 0.0f), p.act);
        if (++n == p.N) {
            n = 0;
            ++m;
        }
    }
}

// How a product is cut.  A CU holds one block of 256 x 256 (half the bytes to
// copy) or two of 128 x 128, one of which multiplies while the other starts or
// stores.  Measured, a round of 256 of the former takes 16 + 2.4 stages us, of
// 512 of the latter 3.5 + 1.7 stages; the larger tiles leave CUs idle in their
// last round, the smaller ones hardly.  Us with tiles of 256 and of 128 (products
// of normally distributed values alone, one after another):
//   8,192^3 bf16 317, 376           4,096^3 bf16 49, 55
//   4,096 x 4,096 -> 4,400 bf16 79, 68       3,328 x 16,384 -> 4,096 bf16 133, 161
//   20,000 x 1,438 -> 1,548 bf16 70, 59      100,000 x 512 -> 512 f16 61, 52
//   8,704 x 1,000 -> 1,920 f16 36, 27        150,000 x 300 -> 512 f16 75, 74
//   6,000^3 f16 180, 182            200,000 x 380 -> 1,000 f32 247, 259
// The two times leave out what the stores of a large output cost: in the last line
// the rule takes tiles of 128, 1 % and 5 % slower.
// Where blocks of 128 are few, the sum over k goes in up to `splits` parts of
// at least 4 stages (1,024 values), joined in order: 130 tiles of 68 stages so
// 60 us, whole 85; but 225 tiles of 10 stages would take 29 instead of 20.
struct MatPlan {
    int tile;
    bool wide;  // 64-bit offsets
    int64_t tiles_m, tiles_n, stages;
    int splits;
};
MatPlan mat_plan(int64_t M, int64_t N, int64_t blocks) {
    MatPlan p{};
    p.wide = blocks >= (int64_t)1 << 20;  // 128 rows of 2^25 values: 2^31 bytes
    const int64_t all = ceil_div(blocks, kStageBlocks);
    const int64_t large = ceil_div(M, 256) * ceil_div(N, 256), small = ceil_div(M, 128) * ceil_div(N, 128);
    const double large_us = (double)ceil_div(large, 256) * (16.0 + 2.4 * (double)all);
    const double small_us = (small > 512 ? (double)small / 512 : 1.0) * (3.5 + 1.7 * (double)all);
    p.tile = large_us < small_us && !p.wide ? 256 : 128;
    p.tiles_m = ceil_div(M, p.tile);
    p.tiles_n = ceil_div(N, p.tile);
    const int64_t tiles = p.tiles_m * p.tiles_n;
    const bool few = tiles <= 128 || (tiles < 256 && all >= 32);
    int64_t splits = p.tile == 128 && tiles > 0 && few ? 512 / tiles : 1;
    if (splits > all / 4) splits = all / 4;
    if (splits < 1) splits = 1;
    p.stages = ceil_div(ceil_div(all, splits), 2) * 2;  // whole groups of 16 scales
    if (p.stages < 2) p.stages = 2;
    p.splits = (int)ceil_div(all, p.stages);
    if (p.splits < 1) p.splits = 1;
    return p;
}

template <typename T>
hipError_t launch_tiles(const MatArgs& p, const MatPlan& plan, hipStream_t s) {
    const dim3 grid((unsigned)(plan.tiles_m * plan.tiles_n), (unsigned)plan.splits);
    if (plan.tile == 256)
        IA_LAUNCH("mx4_matmul_kernel", (mx4_matmul_kernel<T, uint32_t, 256, 4, 2>), grid, dim3(512), 0, s, p);
    else if (plan.wide)
        IA_LAUNCH("mx4_matmul_kernel", (mx4_matmul_kernel<T, int64_t, 128, 2, 2>), grid, dim3(256), 0, s, p);
    else
        IA_LAUNCH("mx4_matmul_kernel", (mx4_matmul_kernel<T, uint32_t, 128, 2, 2>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

template <typename T>
hipError_t matmul_t(MatArgs p, void* ws, hipStream_t s) {
    const MatPlan plan = mat_plan(p.M, p.N, p.blocks);
    p.tiles_m = plan.tiles_m;
    p.tiles_n = plan.tiles_n;
    p.stages = plan.stages;
    if (plan.splits == 1) return launch_tiles<T>(p, plan, s);
    MatArgs part = p;
    part.bias = nullptr;
    part.act = IA_ACT_NONE;
    part.c = ws;
    part.ldc = p.N;
    hipError_t e = launch_tiles<float>(part, plan, s);
    if (e != hipSuccess) return e;
    const int64_t quads = ceil_div(p.M * p.N, 4);
    if (plan.splits >= 8)
        IA_LAUNCH("mx4_join_kernel", (mx4_join_kernel<T, 4>), dim3((unsigned)ceil_div(quads, 64)), dim3(256), 0, s, p,
                  (const float*)ws, plan.splits);
    else
        IA_LAUNCH("mx4_join_kernel", (mx4_join_kernel<T, 1>), dim3((unsigned)ceil_div(quads, 256)), dim3(256), 0, s, p,
                  (const float*)ws, plan.splits);
    return hipGetLastError();
}

}  // namespace

size_t mx4_matmul_workspace(int64_t M, int64_t N, int64_t K) {
    const int splits = mat_plan(M, N, mx4_blocks(K)).splits;
    return splits > 1 ? round_up((size_t)splits * (size_t)M * (size_t)N * sizeof(float)) : 0;
}

hipError_t launch_mx4_matmul(const Mx4View& a, const Mx4View& b, const float* bias, int32_t act, int32_t dtype, void* c,
                             int64_t ldc, void* ws, hipStream_t s) {
    if (a.rows == 0 || b.rows == 0) return hipSuccess;
    const MatArgs p{a.codes, a.scales, b.codes, b.scales, a.rows, b.rows, mx4_blocks(a.cols), bias, act, c, ldc, 0, 0, 0};
    return IA_BY_DTYPE(dtype, matmul_t, p, ws, s);
}

}  // namespace ia
