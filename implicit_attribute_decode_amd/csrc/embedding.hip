// Rows of a table picked by index, scaled, with dropout where asked, and the
// table's gradient.
//
// The gradient of entry v is the sum of the rows of dy whose index is v.  The
// rows' numbers are sorted by index (stable, so the rows of an entry stay in
// order), then each entry's rows are added in that order in fp32: the sums are
// the same on every run, no floating-point atomics take part.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>

#include "mx4_common.h"
#include "philox.h"

namespace ia {
namespace {

// ------------------------------------------------------------ lookup

template <typename T>
struct DenseTable {
    const T* t;
    int64_t ld;
    uint32_t dim;

    struct Raw {
        T v[8];
    };
    // values c .. c + 7 of entry v: loaded at once where they all exist, and as floats
    __device__ __forceinline__ Raw load(int64_t v, uint32_t c) const {
        Raw r;
        __builtin_memcpy(&r, t + v * ld + c, sizeof(r));
        return r;
    }
    __device__ __forceinline__ Raw load_some(int64_t v, uint32_t c) const {
        Raw r;
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = t[v * ld + min(c + j, dim - 1)];
        return r;
    }
    __device__ __forceinline__ void get(const Raw& r, float (&x)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (float)r.v[j];
    }
};

// A quarter of a block of 32 codes and the block's scale; values past the row's
// end are whatever the codes there say and are not stored.
struct Mx4Table {
    const uint32_t* codes;
    const uint8_t* scales;
    int64_t blocks;

    struct Raw {
        uint32_t codes;
        uint8_t scale;
    };
    __device__ __forceinline__ Raw load(int64_t v, uint32_t c) const {
        const int64_t block = v * blocks + (c >> 5);
        return Raw{codes[4 * block + ((c >> 3) & 3)], scales[block]};
    }
    __device__ __forceinline__ Raw load_some(int64_t v, uint32_t c) const { return load(v, c); }
    __device__ __forceinline__ void get(const Raw& r, float (&x)[8]) const {
        const uint32_t byte = r.scale;
        const float s = __builtin_bit_cast(float, byte << 23);
        const floatx2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r.codes, s, 0),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r.codes, s, 1),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r.codes, s, 2),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r.codes, s, 3)};
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = byte == (uint32_t)kNaNByte ? __builtin_nanf("") : (float)p[j >> 1][j & 1];
    }
};

// Eight values of EACH rows a thread: rows k, k + step, ... of `rows` from row0 on,
// fewer than 2^31 threads.  An index outside [0, entries) gives zeros (entry 0 is
// loaded for it).  A row's load waits for its index's, so several are under way.
// 300,000 rows of 256 bf16 values, the k-th entry picked 1 / k as often as the first,
// with dropout: 61 us, 2.5 TB/s of the rows written, bound by the generator
// (dropout.hip) as much as by the rows; with one row a thread 62.
template <typename Table, typename I, typename O, bool DROP, int EACH>
__global__ void __launch_bounds__(256) embedding_kernel(Table t, const I* index, int64_t istride, uint32_t row0, uint32_t rows,
                                                        uint32_t step, int64_t entries, uint32_t dim, Divisor chunks,
                                                        float factor, O* out, int64_t ldo, bool stream, DropArgs a) {
    const uint32_t i = blockIdx.x * 256u + threadIdx.x, k = chunks.of(i), c = (i - k * chunks.d) * 8;
    if (k >= step) return;
    int64_t v[EACH];
#pragma unroll
    for (int e = 0; e < EACH; ++e) v[e] = (int64_t)index[(int64_t)(row0 + min(k + e * step, rows - 1)) * istride];
    const Dropper drop(a);
    const auto there = [&](int e) { return v[e] >= 0 && v[e] < entries; };
    const auto put = [&](const typename Table::Raw& raw, int e, int64_t count) {
        const uint32_t r = row0 + k + e * step;
        if (k + e * step >= rows) return;
        float x[8];
        t.get(raw, x);
        if (DROP) {
            drop.apply(x, r, c, factor);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= factor;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = there(e) ? x[j] : 0.0f;
        store8(out + (int64_t)r * ldo + c, count, x, stream);
    };
    if (c + 8 <= dim) {
        typename Table::Raw raw[EACH];
#pragma unroll
        for (int e = 0; e < EACH; ++e) raw[e] = t.load(there(e) ? v[e] : 0, c);
#pragma unroll
        for (int e = 0; e < EACH; ++e) put(raw[e], e, 8);
    } else {
#pragma unroll
        for (int e = 0; e < EACH; ++e) put(t.load_some(there(e) ? v[e] : 0, c), e, (int64_t)dim - c);
    }
}

// No entries: zeros.
template <typename O>
__global__ void __launch_bounds__(256) embedding_none_kernel(O* out, int64_t ldo, int64_t n, int64_t dim) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n * dim; i += (int64_t)gridDim.x * 256)
        out[i / dim * ldo + i % dim] = (O)0.0f;
}

struct LookupArgs {
    const void* index;
    int64_t istride, n, entries, dim;
    int index_bytes;
    float factor;
    void* out;
    int64_t ldo;
    const DropArgs* drop;
    hipStream_t s;
};

template <typename O, typename Table, typename I, bool DROP, int EACH>
void launch_rows(const Table& t, const LookupArgs& p, const Divisor& chunks, int64_t row0, int64_t rows) {
    const int64_t step = ceil_div(rows, EACH);
    IA_LAUNCH("embedding_kernel", (embedding_kernel<Table, I, O, DROP, EACH>), dim3((unsigned)ceil_div(step * chunks.d, 256)),
              dim3(256), 0, p.s, t, (const I*)p.index, p.istride, (uint32_t)row0, (uint32_t)rows, (uint32_t)step, p.entries,
              (uint32_t)p.dim, chunks, p.factor, (O*)p.out, p.ldo, p.n * p.dim * (int64_t)sizeof(O) >= kStreamBytes,
              p.drop ? *p.drop : DropArgs{});
}
template <typename O, typename Table, typename I, bool DROP>
hipError_t launch_lookup(const Table& t, const LookupArgs& p) {
    const Divisor chunks((uint32_t)ceil_div(p.dim, 8));
    const int64_t most = (((int64_t)1 << 31) - 256) / chunks.d;
    for (int64_t r = 0; r < p.n; r += most) {
        const int64_t here = std::min(most, p.n - r);
        // four rows a thread where that leaves waves for the whole chip
        if (here * chunks.d >= (int64_t)4 * 64 * 8192)
            launch_rows<O, Table, I, DROP, 4>(t, p, chunks, r, here);
        else
            launch_rows<O, Table, I, DROP, 1>(t, p, chunks, r, here);
    }
    return hipGetLastError();
}
template <typename O, typename Table>
hipError_t lookup(const Table& t, const LookupArgs& p) {
    if (p.entries == 0) {
        IA_LAUNCH("embedding_none_kernel", embedding_none_kernel<O>, dim3(grid_for(p.n * p.dim)), dim3(256), 0, p.s, (O*)p.out,
                  p.ldo, p.n, p.dim);
        return hipGetLastError();
    }
    if (p.index_bytes == 8)
        return p.drop ? launch_lookup<O, Table, int64_t, true>(t, p) : launch_lookup<O, Table, int64_t, false>(t, p);
    return p.drop ? launch_lookup<O, Table, int32_t, true>(t, p) : launch_lookup<O, Table, int32_t, false>(t, p);
}
template <typename T>
hipError_t lookup_dense(const void* table, int64_t ld, int32_t out_dtype, const LookupArgs& p) {
    const DenseTable<T> t{(const T*)table, ld, (uint32_t)p.dim};
    return IA_BY_DTYPE(out_dtype, lookup, t, p);
}

// ------------------------------------------------------------ gradient

// Sorted by index: (index << 32) | row; rows without an entry have index
// `entries` and come last.
__device__ __forceinline__ uint32_t key_of(uint64_t w) { return (uint32_t)(w >> 32); }

template <typename I>
__device__ __forceinline__ uint64_t word_of(const I* index, int64_t istride, int64_t i, int64_t entries) {
    const int64_t v = (int64_t)index[i * istride];
    return ((uint64_t)(v >= 0 && v < entries ? v : entries) << 32) | (uint32_t)i;
}

constexpr int kThreads = 256;

// A share of the gradient's zeros, written by the blocks from `first` on of a
// kernel that leaves most of the chip idle: part k of `parts` of it.  (With the
// 102 MB of 50,021 x 512 values the six kernels of a sort of 131,071 rows take 38 us;
// the three of a pass over 300,000 rows with next to none 14.)
struct Zeros {
    float* grad;
    int64_t values;
    int first, blocks, part, parts;
};
__device__ __forceinline__ bool zero_share(const Zeros& z) {
    const int b = (int)blockIdx.x - z.first;
    if (b < 0) return false;
    const int64_t quads = (z.values + 3) / 4, lo = quads * z.part / z.parts, hi = quads * (z.part + 1) / z.parts;
    for (int64_t i = lo + (int64_t)b * blockDim.x + threadIdx.x; i < hi; i += (int64_t)z.blocks * blockDim.x) {
        if (4 * i + 4 <= z.values) {
            const floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
            __builtin_memcpy(z.grad + 4 * i, &v, 16);
        } else {
            for (int64_t k = 4 * i; k < z.values; ++k) z.grad[k] = 0.0f;
        }
    }
    return true;
}

// Stable sort, eight bits of the index at a time, least first: every block counts
// the digits of its items, the counts are summed over the blocks before it, and
// every block puts its items in their places.  The items of a block are few, so
// that 100,000 of them occupy the chip: two passes of 131,071 take 20 us here,
// where tiles of 4,096 took 39.
constexpr int kDigits = 256;
constexpr int kItems = 4;                    // of a thread
constexpr int kSortTile = kThreads * kItems;
constexpr int kSortBlocks = 512;

struct SortArgs {
    const uint64_t* in;
    uint64_t* out;
    int64_t n, per;    // items; of a block, whole tiles
    int blocks, shift;
    uint32_t* counts;  // [kDigits][blocks]
    uint32_t* totals;  // [kDigits]
};

__device__ __forceinline__ uint32_t digit_of(uint64_t w, int shift) { return (uint32_t)(w >> shift) & (kDigits - 1); }

// Lanes of the wave that are valid and hold the same digit.
__device__ __forceinline__ uint64_t same_digit(uint32_t d, bool valid) {
    uint64_t peers = __ballot(valid);
#pragma unroll
    for (int bit = 0; bit < 8; ++bit) {
        const uint64_t b = __ballot((d >> bit) & 1u);
        peers &= ((d >> bit) & 1u) ? b : ~b;
    }
    return peers;
}

__device__ __forceinline__ void count_digit(uint32_t* hist, uint32_t d, bool valid) {
    // a wave of one digit (indices in order) adds once
    const uint32_t d0 = __builtin_amdgcn_readfirstlane(d);
    if (__ballot(valid && d == d0) == ~0ull) {
        if ((threadIdx.x & 63) == 0) atomicAdd(&hist[d0], 64u);
    } else if (valid) {
        atomicAdd(&hist[d], 1u);
    }
}

// Counts of the first pass, and the words themselves.
template <typename I>
__global__ void __launch_bounds__(kThreads) embedding_keys_kernel(const I* index, int64_t istride, int64_t entries,
                                                                  uint64_t* words, SortArgs p, uint32_t* listed, Zeros z) {
    if (zero_share(z)) return;
    __shared__ uint32_t hist[kDigits];
    hist[threadIdx.x] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) listed[0] = 0;
    __syncthreads();
    const int64_t begin = blockIdx.x * p.per, end = min(begin + p.per, p.n);
    for (int64_t base = begin; base < end; base += kThreads) {
        const int64_t i = base + threadIdx.x;
        uint64_t w = 0;
        if (i < end) words[i] = w = word_of(index, istride, i, entries);
        count_digit(hist, digit_of(w, p.shift), i < end);
    }
    __syncthreads();
    p.counts[threadIdx.x * p.blocks + blockIdx.x] = hist[threadIdx.x];
}

__global__ void __launch_bounds__(kThreads) embedding_count_kernel(SortArgs p, Zeros z) {
    if (zero_share(z)) return;
    __shared__ uint32_t hist[kDigits];
    hist[threadIdx.x] = 0;
    __syncthreads();
    const int64_t begin = blockIdx.x * p.per, end = min(begin + p.per, p.n);
    for (int64_t base = begin; base < end; base += kThreads) {
        const int64_t i = base + threadIdx.x;
        count_digit(hist, digit_of(i < end ? p.in[i] : 0, p.shift), i < end);
    }
    __syncthreads();
    p.counts[threadIdx.x * p.blocks + blockIdx.x] = hist[threadIdx.x];
}

// Sum of the values of the threads before this one, and of all.
__device__ __forceinline__ uint32_t sum_before(uint32_t v, uint32_t* waves, uint32_t& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t x = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    if (lane == 63) waves[wave] = x;
    __syncthreads();
    uint32_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
        const uint32_t s = waves[w];
        if (w < wave) before += s;
        total += s;
    }
    __syncthreads();
    return before + x - v;
}

// A block for each digit: its counts become sums over the blocks before.
__global__ void __launch_bounds__(kThreads) embedding_scan_kernel(SortArgs p, Zeros z) {
    if (zero_share(z)) return;
    __shared__ uint32_t waves[kThreads / 64];
    uint32_t* c = p.counts + (int64_t)blockIdx.x * p.blocks;
    uint32_t carry = 0;
    for (int base = 0; base < p.blocks; base += kThreads) {
        const int i = base + threadIdx.x;
        uint32_t total;
        const uint32_t before = sum_before(i < p.blocks ? c[i] : 0u, waves, total);
        if (i < p.blocks) c[i] = carry + before;
        carry += total;
    }
    if (threadIdx.x == 0) p.totals[blockIdx.x] = carry;
}

__global__ void __launch_bounds__(kThreads) embedding_place_kernel(SortArgs p, Zeros z) {
    if (zero_share(z)) return;
    constexpr int WAVES = kThreads / 64;
    __shared__ uint32_t waves[WAVES], place[WAVES][kDigits];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, d0 = threadIdx.x;
    uint32_t total;
    // the next place of digit d0's items of this block
    uint32_t next = sum_before(p.totals[d0], waves, total) + p.counts[d0 * p.blocks + blockIdx.x];
    const int64_t begin = blockIdx.x * p.per, end = min(begin + p.per, p.n);
    const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
    for (int64_t tile = begin; tile < end; tile += kSortTile) {
#pragma unroll
        for (int w = 0; w < WAVES; ++w) place[w][d0] = 0;
        uint64_t word[kItems];
        uint32_t rank[kItems];
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int64_t i = tile + wave * (64 * kItems) + j * 64 + lane;
            word[j] = p.in[min(i, end - 1)];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const bool valid = tile + wave * (64 * kItems) + j * 64 + lane < end;
            const uint32_t d = digit_of(word[j], p.shift);
            const uint64_t peers = same_digit(d, valid);
            const uint32_t prior = place[wave][d], mine = (uint32_t)__popcll(peers & below);
            // the lowest lane of a digit advances the wave's count
            if (valid && mine == 0) place[wave][d] = prior + (uint32_t)__popcll(peers);
            rank[j] = prior + mine;
            wave_lds_sync();
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const uint32_t c = place[w][d0];
            place[w][d0] = next;
            next += c;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            if (tile + wave * (64 * kItems) + j * 64 + lane >= end) continue;
            const uint32_t to = place[wave][digit_of(word[j], p.shift)] + rank[j];
            if (to < p.n) p.out[to] = word[j];
        }
        __syncthreads();
    }
}

// All passes of up to 4,096 items in one block, in LDS.
constexpr int kSmallThreads = 1024;
constexpr int kSmallItems = 4;
constexpr int kSmall = kSmallThreads * kSmallItems;

template <typename I>
__global__ void __launch_bounds__(kSmallThreads) embedding_small_sort_kernel(const I* index, int64_t istride, int n,
                                                                             int64_t entries, int bits, uint64_t* out,
                                                                             uint32_t* listed, Zeros z) {
    if (zero_share(z)) return;
    constexpr int WAVES = kSmallThreads / 64;
    __shared__ uint64_t items[kSmall];
    __shared__ uint32_t place[WAVES][kDigits], waves[kDigits / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
    if (threadIdx.x == 0) listed[0] = 0;
    uint64_t word[kSmallItems];
    const int used = (n + 64 * kSmallItems - 1) / (64 * kSmallItems);  // waves with items
#pragma unroll
    for (int j = 0; j < kSmallItems; ++j) {
        const int i = wave * (64 * kSmallItems) + j * 64 + lane;
        // past the end: as rows without an entry, behind them all
        word[j] = i < n ? word_of(index, istride, i, entries) : (uint64_t)entries << 32 | (uint32_t)i;
    }
    for (int shift = 32; shift < 32 + bits; shift += 8) {
        for (int k = threadIdx.x; k < WAVES * kDigits; k += kSmallThreads) place[k / kDigits][k % kDigits] = 0;
        __syncthreads();
        uint32_t rank[kSmallItems];
        if (wave < used) {
#pragma unroll
            for (int j = 0; j < kSmallItems; ++j) {
                const uint32_t d = digit_of(word[j], shift);
                const uint64_t peers = same_digit(d, true);
                const uint32_t prior = place[wave][d], mine = (uint32_t)__popcll(peers & below);
                if (mine == 0) place[wave][d] = prior + (uint32_t)__popcll(peers);
                rank[j] = prior + mine;
                wave_lds_sync();
            }
        }
        __syncthreads();
        uint32_t sum = 0, x = 0;
        if (threadIdx.x < kDigits) {
            for (int w = 0; w < used; ++w) sum += place[w][threadIdx.x];
            x = sum;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const uint32_t y = __shfl_up(x, d);
                if (lane >= d) x += y;
            }
            if (lane == 63) waves[wave] = x;
        }
        __syncthreads();
        if (threadIdx.x < kDigits) {
            uint32_t next = x - sum;
            for (int w = 0; w < wave; ++w) next += waves[w];
            for (int w = 0; w < used; ++w) {
                const uint32_t c = place[w][threadIdx.x];
                place[w][threadIdx.x] = next;
                next += c;
            }
        }
        __syncthreads();
        if (wave < used) {
#pragma unroll
            for (int j = 0; j < kSmallItems; ++j) items[place[wave][digit_of(word[j], shift)] + rank[j]] = word[j];
        }
        __syncthreads();
        if (wave < used) {
#pragma unroll
            for (int j = 0; j < kSmallItems; ++j) word[j] = items[wave * (64 * kSmallItems) + j * 64 + lane];
        }
    }
#pragma unroll
    for (int j = 0; j < kSmallItems; ++j) {
        const int i = wave * (64 * kSmallItems) + j * 64 + lane;
        if (i < n) out[i] = word[j];
    }
}

struct SumArgs {
    const uint64_t* words;
    int64_t n;
    uint32_t entries, dim;
    int lanes;        // lanes of a group: a power of two up to 64
    int tile;         // sorted rows that a group starts from
    int64_t slices;   // groups side by side over the columns
    int64_t tiles;
    int64_t block0;   // first of the launch
    float factor;
    float* grad;      // [entries][dim], zeros
    float* part;      // [tiles][2][dim]: sums of a long entry's rows in a tile, at its end (0) and at its start (1)
    uint32_t* listed; // [0] how many, then the tiles where a long entry starts
};

constexpr int kAhead = 8;  // rows in flight

// Four consecutive values; `count` of them exist.
template <typename T>
__device__ __forceinline__ floatx4 load4(const T* p, int64_t count) {
    floatx4 v;
    if (count >= 4) {
        T t[4];
        __builtin_memcpy(t, p, sizeof(t));
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = (float)t[j];
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = j < count ? (float)p[j] : 0.0f;
    }
    return v;
}
__device__ __forceinline__ void store4(float* p, int64_t count, floatx4 v) {
    if (count >= 4) {
        __builtin_memcpy(p, &v, 16);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < count) p[j] = v[j];
    }
}

// Four values of a row, loaded at once and without a branch, which would make every
// load wait for itself: rows of a multiple of four values, of other numbers from
// four on (the last lane's values are loaded from the row's end and shifted), or of
// fewer.
enum Rows { kQuads, kRagged, kNarrow };
template <typename T, Rows ROWS>
struct Quad {
    T t[4];

    // values c .. c + 3 of a row of dim; c < dim, or any four of it
    __device__ __forceinline__ void load(const T* row, int64_t c, int64_t dim) {
        if (ROWS == kNarrow) {
#pragma unroll
            for (int j = 0; j < 4; ++j) t[j] = row[min(c + j, dim - 1)];
        } else {
            __builtin_memcpy(t, row + min(c, dim - 4), sizeof(t));
        }
    }
    // as floats, zero past the row's end
    __device__ __forceinline__ floatx4 get(int64_t c, int64_t dim) const {
        floatx4 v = {(float)t[0], (float)t[1], (float)t[2], (float)t[3]};
        if (ROWS == kNarrow) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = c + j < dim ? v[j] : 0.0f;
        }
        if (ROWS == kRagged) {
            const int by = (int)(max(c, dim - 4) - (dim - 4));
            if (by & 1) v = floatx4{v[1], v[2], v[3], 0.0f};
            if (by & 2) v = floatx4{v[2], v[3], 0.0f, 0.0f};
        }
        return v;
    }
};

// A group of lanes walks the sorted rows from a tile's start, adding rows until
// the index changes; a lane has QUADS times four columns, so that the group writes
// whole lines.  An entry belongs to the tile in which its rows start; that tile's
// group follows it into the next tile, so most entries are written once and whole.
// An entry that also reaches the tile after the next is long: every tile leaves the
// sum of its own rows, and the join adds those in order.  The words of a block's
// tiles pass through LDS, and which rows a group needs is known before they are
// loaded: no row of dy is read twice.  131,071 rows of 512 bf16 values into 50,021
// entries: 43 us for 134 MB of rows read in any order and about 60 MB of sums written
// (4.5 TB/s).  Each load converted behind a branch on the row's end took twice that.
template <typename T, bool DROP, int QUADS, Rows ROWS>
__global__ void __launch_bounds__(256) embedding_sums_kernel(const T* dy, int64_t lddy, SumArgs p, DropArgs a) {
    extern __shared__ uint64_t s_words[];  // from a tile and a word before the first tile to two tiles past the last one's start
    const int groups = 256 / p.lanes, group = threadIdx.x / p.lanes, lane = threadIdx.x % p.lanes;
    const int64_t block = p.block0 + blockIdx.x, unit = block * groups + group;
    const int64_t tile0 = block * groups / p.slices;
    const int before = p.tile + 1;
    {
        const int64_t from = tile0 * p.tile - before;
        const int count = (int)(((block + 1) * groups - 1) / p.slices - tile0 + 2) * p.tile + before + 1;
        for (int i = threadIdx.x; i < count; i += 256) s_words[i] = p.words[min(max(from + i, (int64_t)0), p.n - 1)];
        __syncthreads();
    }
    const int64_t tile = unit / p.slices, slice = unit - tile * p.slices;
    if (tile >= p.tiles) return;
    const uint64_t* const words = s_words + (int)(tile - tile0) * p.tile + before;  // of the tile's rows
    const int64_t t0 = tile * p.tile;
    const int left = (int)min(p.n - t0, (int64_t)INT_MAX), own = min(left, p.tile);  // rows from here on, of the tile
    const uint32_t head = key_of(words[0]), last = key_of(words[own - 1]);
    if (head >= p.entries) return;  // rows without an entry only
    const int64_t c0 = (slice * p.lanes * QUADS + lane) * 4;  // and every 4 lanes columns from there
    const bool first = slice == 0 && lane == 0;
    const Dropper drop(a);

    // the first rows' entry starts in an earlier tile; it is long, the last rows' entry is long
    const bool carried = t0 > 0 && key_of(words[-1]) == head;
    const bool head_long = carried && ((t0 > p.tile && key_of(words[-p.tile - 1]) == head) ||
                                       (own < left && key_of(words[own]) == head));
    const bool tail_long = !(carried && last == head) && last < p.entries && own + p.tile < left &&
                           key_of(words[own + p.tile]) == last;
    if (tail_long && first) p.listed[1 + atomicAdd(p.listed, 1u)] = (uint32_t)tile;

    floatx4 acc[QUADS] = {};
    int at = 0;
    if (carried && !head_long) {  // the rows of another tile's entry
        while (at < own && key_of(words[at]) == head) ++at;
        if (at == own) return;
    }
    bool mine = !carried || at > 0, done = false;
    uint32_t cur = key_of(words[at]);
    if (cur >= p.entries) return;
    for (; !done; at += kAhead) {
        // what the rows' loop below will do, from their words alone
        int64_t row[kAhead];
        uint32_t key[kAhead];
        bool ends[kAhead];  // the rows of `cur` end before this one
        {
            uint32_t k = cur;
            bool m = mine, d = false;
            const int64_t row0 = (int64_t)(uint32_t)words[min(at, own + p.tile)];  // for none
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = at + u;
                const uint64_t w = words[min(i, own + p.tile)];
                const bool past = i >= own;
                key[u] = key_of(w);
                ends[u] = i >= left || (past && (!m || tail_long)) || key[u] != k;
                d = d || (ends[u] && (i >= left || past || key[u] >= p.entries));
                m = m || ends[u];
                k = ends[u] ? key[u] : k;
                row[u] = d ? row0 : (int64_t)(uint32_t)w;
            }
        }
        Quad<T, ROWS> x[kAhead][QUADS];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int q = 0; q < QUADS; ++q) x[u][q].load(dy + row[u] * lddy, c0 + 4 * q * p.lanes, p.dim);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (done) continue;
            if (ends[u]) {
                const bool past = at + u >= own, partial = mine ? past && tail_long : head_long;
                if (mine || head_long) {
                    const float f = partial ? 1.0f : p.factor;
                    float* out = partial ? p.part + (2 * tile + (mine ? 0 : 1)) * (int64_t)p.dim : p.grad + (int64_t)cur * p.dim;
#pragma unroll
                    for (int q = 0; q < QUADS; ++q) {
                        const int64_t c = c0 + 4 * q * p.lanes;
                        store4(out + c, (int64_t)p.dim - c, acc[q] * f);
                    }
                }
                done = at + u >= left || past || key[u] >= p.entries;
                cur = key[u];
                mine = true;
#pragma unroll
                for (int q = 0; q < QUADS; ++q) acc[q] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
            }
#pragma unroll
            for (int q = 0; q < QUADS; ++q) {
                floatx4 v = x[u][q].get(c0 + 4 * q * p.lanes, p.dim);
                if (DROP) drop.apply(v, (uint32_t)row[u], (uint32_t)(c0 + 4 * q * p.lanes));
                acc[q] += v;
            }
        }
    }
}

// Long entries: the sums that their tiles left, added in double in a fixed order.
// Bound by latency: a block waits for its entry, its words and its sums in turn (370
// entries of up to 12,000 rows of 512: 11 us with 4,096 blocks, 21 with 512).
__global__ void __launch_bounds__(256) embedding_join_kernel(SumArgs p) {
    constexpr int COLS = 64, WAYS = 16;  // columns of a block's pass, tiles side by side
    __shared__ double s_sum[WAYS][COLS];
    const int way = threadIdx.x / (COLS / 4), q = threadIdx.x % (COLS / 4);
    const int64_t across = ((int64_t)p.dim + COLS - 1) / COLS, items = (int64_t)p.listed[0] * across;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t tile = p.listed[1 + it / across], c = (it % across) * COLS + 4 * q;
        const uint32_t key = key_of(p.words[(tile + 1) * p.tile - 1]);
        int64_t more = 0;  // tiles behind this one that begin with the entry
        for (int found = 256; found == 256; more += found) {
            const int64_t t = (tile + 1 + more + threadIdx.x) * p.tile;
            found = __syncthreads_count(t < p.n && key_of(p.words[t < p.n ? t : 0]) == key);
        }
        double sum[4] = {};
#pragma unroll 8
        for (int64_t k = way; k <= more; k += WAYS) {
            const floatx4 v = load4(p.part + (2 * (tile + k) + (k == 0 ? 0 : 1)) * (int64_t)p.dim + c, (int64_t)p.dim - c);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] += (double)v[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) s_sum[way][4 * q + j] = sum[j];
        __syncthreads();
        const int64_t col = (it % across) * COLS + threadIdx.x;
        if (threadIdx.x < COLS && col < p.dim) {
            double v = 0.0;
#pragma unroll
            for (int k = 0; k < WAYS; ++k) v += s_sum[k][threadIdx.x];
            p.grad[(int64_t)key * p.dim + col] = (float)(v * (double)p.factor);
        }
        __syncthreads();
    }
}

// How the sums are laid over the chip: a lane has four columns, or eight of wide
// rows; a tile is 16 sorted rows, 32 where that is more than 16 waves a SIMD (so that no
// more than 64 rows are added one after the other).
struct SumShape {
    int lanes, quads, tile;
    int64_t slices, tiles;
};
SumShape sum_shape(int64_t n, int64_t dim) {
    SumShape s{};
    s.quads = dim > 256 ? 2 : 1;
    s.lanes = 1;
    while (s.lanes < 64 && s.lanes * 4 * s.quads < dim) s.lanes *= 2;
    s.slices = ceil_div(dim, s.lanes * 4 * s.quads);
    s.tile = 16;
    while (s.tile < 32 && s.lanes > 1 && ceil_div(n, s.tile) * s.slices * s.lanes > (int64_t)64 * 16384) s.tile *= 2;
    s.tiles = ceil_div(n, s.tile);
    return s;
}

struct GradLayout {
    size_t words0, words1, counts, totals, listed, part, total;
};
GradLayout grad_layout(int64_t n, int64_t dim) {
    const SumShape shape = sum_shape(n, dim);
    GradLayout l{};
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t here = at;
        at += round_up(bytes);
        return here;
    };
    l.words0 = take(8 * (size_t)n);
    l.words1 = take(8 * (size_t)n);
    l.counts = take(4 * kDigits * (size_t)kSortBlocks);
    l.totals = take(4 * kDigits);
    l.listed = take(4 * (size_t)(shape.tiles + 1));
    l.part = take(2 * 4 * (size_t)shape.tiles * (size_t)dim);
    l.total = at;
    return l;
}

__global__ void __launch_bounds__(kThreads) embedding_zero_kernel(Zeros z) { zero_share(z); }

template <typename T, int QUADS, Rows ROWS>
hipError_t launch_sums(const T* dy, int64_t lddy, const SumArgs& a, const DropArgs* d, hipStream_t s) {
    SumArgs p = a;
    const int groups = 256 / p.lanes;
    // the tiles of a block, the one before and two behind
    const size_t lds = 8 * ((size_t)(ceil_div(groups - 1, p.slices) + 3) * p.tile + p.tile + 2);
    const int64_t blocks = ceil_div(p.tiles * p.slices, groups), most = 1 << 23;  // a grid has less than 2^32 threads
    for (p.block0 = 0; p.block0 < blocks; p.block0 += most) {
        const dim3 grid((unsigned)std::min(most, blocks - p.block0));
        if (d)
            IA_LAUNCH("embedding_sums_kernel", (embedding_sums_kernel<T, true, QUADS, ROWS>), grid, dim3(256), lds, s, dy, lddy,
                      p, *d);
        else
            IA_LAUNCH("embedding_sums_kernel", (embedding_sums_kernel<T, false, QUADS, ROWS>), grid, dim3(256), lds, s, dy,
                      lddy, p, DropArgs{});
    }
    return hipGetLastError();
}
template <typename T>
hipError_t sums(const void* dy, int64_t lddy, int quads, const SumArgs& p, const DropArgs* d, hipStream_t s) {
    const T* const t = (const T*)dy;
    if (p.dim < 4) return launch_sums<T, 1, kNarrow>(t, lddy, p, d, s);
    if (p.dim % 4 != 0)
        return quads == 2 ? launch_sums<T, 2, kRagged>(t, lddy, p, d, s) : launch_sums<T, 1, kRagged>(t, lddy, p, d, s);
    return quads == 2 ? launch_sums<T, 2, kQuads>(t, lddy, p, d, s) : launch_sums<T, 1, kQuads>(t, lddy, p, d, s);
}

// Sorts the rows by index and clears the gradient; the buffer with the result.
template <typename I>
const uint64_t* sort_rows(const Indices& ix, int64_t entries, float* grad, int64_t values, char* w, const GradLayout& l,
                          hipStream_t s) {
    uint64_t* const buf[2] = {(uint64_t*)(w + l.words0), (uint64_t*)(w + l.words1)};
    uint32_t* const listed = (uint32_t*)(w + l.listed);
    int bits = 1;
    while ((entries >> bits) != 0) ++bits;
    // the zeros go along with the sort, in equal shares, at most 1,024 blocks of them
    const auto zeros = [&](int first, int part, int parts) {
        const int64_t want = ceil_div(values, (int64_t)parts * kThreads * 16);
        return Zeros{grad, values, first, (int)(want < 1024 ? want : 1024), part, parts};
    };
    if (ix.n <= kSmall) {
        const Zeros z = zeros(1, 0, 1);
        IA_LAUNCH("embedding_small_sort_kernel", embedding_small_sort_kernel<I>, dim3((unsigned)(1 + z.blocks)),
                  dim3(kSmallThreads), 0, s, (const I*)ix.index, ix.stride, (int)ix.n, entries, bits, buf[0], listed, z);
        return buf[0];
    }
    const int passes = (bits + 7) / 8;
    SortArgs p{};
    p.n = ix.n;
    p.per = ceil_div(ceil_div(ix.n, kSortTile), kSortBlocks) * kSortTile;
    p.blocks = (int)ceil_div(ix.n, p.per);
    p.counts = (uint32_t*)(w + l.counts);
    p.totals = (uint32_t*)(w + l.totals);
    int cur = 0, part = 0;
    for (int pass = 0; pass < passes; ++pass, cur ^= 1) {
        p.in = buf[cur];
        p.out = buf[cur ^ 1];
        p.shift = 32 + 8 * pass;
        Zeros z = zeros(p.blocks, part++, 3 * passes);
        const dim3 grid((unsigned)(p.blocks + z.blocks)), block(kThreads);
        if (pass == 0)
            IA_LAUNCH("embedding_keys_kernel", embedding_keys_kernel<I>, grid, block, 0, s, (const I*)ix.index, ix.stride,
                      entries, buf[0], p, listed, z);
        else
            IA_LAUNCH("embedding_count_kernel", embedding_count_kernel, grid, block, 0, s, p, z);
        z = zeros(kDigits, part++, 3 * passes);
        IA_LAUNCH("embedding_scan_kernel", embedding_scan_kernel, dim3((unsigned)(kDigits + z.blocks)), block, 0, s, p, z);
        z = zeros(p.blocks, part++, 3 * passes);
        IA_LAUNCH("embedding_place_kernel", embedding_place_kernel, grid, block, 0, s, p, z);
    }
    return buf[cur];
}

}  // namespace

hipError_t launch_embedding(const void* table, int32_t dtype, int64_t entries, int64_t dim, int64_t ld, const Indices& ix,
                            float factor, const DropArgs* drop, int32_t out_dtype, void* out, int64_t ldo, hipStream_t s) {
    if (ix.n == 0 || dim == 0) return hipSuccess;
    const LookupArgs p{ix.index, ix.stride, ix.n, entries, dim, ix.bytes, factor, out, ldo, drop, s};
    return IA_BY_DTYPE(dtype, lookup_dense, table, ld, out_dtype, p);
}

hipError_t launch_embedding_mx4(const Mx4View& t, const Indices& ix, float factor, const DropArgs* drop, int32_t out_dtype,
                                void* out, int64_t ldo, hipStream_t s) {
    if (ix.n == 0 || t.cols == 0) return hipSuccess;
    const LookupArgs p{ix.index, ix.stride, ix.n, t.rows, t.cols, ix.bytes, factor, out, ldo, drop, s};
    const Mx4Table table{(const uint32_t*)t.codes, t.scales, mx4_blocks(t.cols)};
    return IA_BY_DTYPE(out_dtype, lookup, table, p);
}

size_t embedding_backward_workspace(int64_t n, int64_t entries, int64_t dim) {
    return n == 0 || entries == 0 || dim == 0 ? 0 : grad_layout(n, dim).total;
}

hipError_t launch_embedding_backward(const void* dy, int32_t dtype, int64_t dim, int64_t lddy, const Indices& ix,
                                     int64_t entries, float factor, const DropArgs* drop, float* grad, void* ws,
                                     hipStream_t s) {
    if (entries == 0 || dim == 0) return hipSuccess;
    if (ix.n == 0) {
        const int64_t blocks = ceil_div(entries * dim, kThreads * 16);
        const Zeros z{grad, entries * dim, 0, (int)(blocks < 2048 ? blocks : 2048), 0, 1};
        IA_LAUNCH("embedding_zero_kernel", embedding_zero_kernel, dim3(z.blocks), dim3(kThreads), 0, s, z);
        return hipGetLastError();
    }
    const GradLayout l = grad_layout(ix.n, dim);
    char* const w = (char*)ws;
    const uint64_t* words = ix.bytes == 8 ? sort_rows<int64_t>(ix, entries, grad, entries * dim, w, l, s)
                                          : sort_rows<int32_t>(ix, entries, grad, entries * dim, w, l, s);
    const SumShape shape = sum_shape(ix.n, dim);
    SumArgs p{};
    p.words = words;
    p.n = ix.n;
    p.entries = (uint32_t)entries;
    p.dim = (uint32_t)dim;
    p.lanes = shape.lanes;
    p.tile = shape.tile;
    p.slices = shape.slices;
    p.tiles = shape.tiles;
    p.factor = factor;
    p.grad = grad;
    p.part = (float*)(w + l.part);
    p.listed = (uint32_t*)(w + l.listed);
    hipError_t e = IA_BY_DTYPE(dtype, sums, dy, lddy, shape.quads, p, drop, s);
    if (e != hipSuccess || shape.tiles < 3) return e;  // no entry reaches a third tile
    // blocks for every long entry there can be, 4,096 at most
    const int64_t most = ceil_div(ix.n, 2 * shape.tile) * ceil_div(dim, 64);
    IA_LAUNCH("embedding_join_kernel", embedding_join_kernel, dim3((unsigned)(most < 4096 ? most : 4096)), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace ia
