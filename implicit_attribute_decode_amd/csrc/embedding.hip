// Rows of a table picked by index, scaled, with dropout where asked, and the
// table's gradient.
//
// The gradient of entry v is the sum of the rows of dy whose index is v.  The
// rows' numbers are sorted by index (stable, so the rows of an entry stay in
// order), then each entry's rows are added in that order in fp32: the sums are
// the same on every run, no floating-point atomics take part.
#include <hip/hip_runtime.h>

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

    // values c .. c + 7 of entry v
    __device__ __forceinline__ void load(int64_t v, uint32_t c, float (&x)[8]) const {
        load8(t + v * ld + c, (int64_t)dim - c, x);
    }
};

// A quarter of a block of 32 codes and the block's scale; values past the row's
// end are whatever the codes there say and are not stored.
struct Mx4Table {
    const uint32_t* codes;
    const uint8_t* scales;
    int64_t blocks;

    __device__ __forceinline__ void load(int64_t v, uint32_t c, float (&x)[8]) const {
        const int64_t block = v * blocks + (c >> 5);
        const uint32_t q = codes[4 * block + ((c >> 3) & 3)], byte = scales[block];
        const float s = __builtin_bit_cast(float, byte << 23);
        typedef float pair __attribute__((ext_vector_type(2)));
        const pair p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 1);
        const pair p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 3);
        const pair p[4] = {p0, p1, p2, p3};
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = byte == (uint32_t)kNaNByte ? __builtin_nanf("") : (float)p[j >> 1][j & 1];
    }
};

// Eight values of a row a thread.  An index outside [0, entries) gives zeros.
template <typename Table, typename I, typename O, bool DROP>
__global__ void __launch_bounds__(256) embedding_kernel(Table t, const I* index, int64_t istride, int64_t n, int64_t entries,
                                                        uint32_t dim, float factor, O* out, int64_t ldo, DropArgs a) {
    const uint32_t chunks = (dim + 7) / 8;
    const int64_t total = n * chunks;
    const Dropper drop(a);
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < total; k += (int64_t)gridDim.x * 256) {
        const uint32_t r = (uint32_t)(k / chunks), c = (uint32_t)(k - (int64_t)r * chunks) * 8;
        const int64_t v = (int64_t)index[(int64_t)r * istride];
        float x[8] = {};
        if (v >= 0 && v < entries) {
            t.load(v, c, x);
            if (DROP) {
                drop.apply(x, r, c, factor);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= factor;
            }
        }
        store8(out + (int64_t)r * ldo + c, (int64_t)dim - c, x);
    }
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

template <typename O, typename Table, typename I, bool DROP>
hipError_t launch_lookup(const Table& t, const LookupArgs& p) {
    IA_LAUNCH("embedding_kernel", (embedding_kernel<Table, I, O, DROP>), dim3(grid_for(p.n * ceil_div(p.dim, 8))),
              dim3(256), 0, p.s, t, (const I*)p.index, p.istride, p.n, p.entries, (uint32_t)p.dim, p.factor, (O*)p.out,
              p.ldo, p.drop ? *p.drop : DropArgs{});
    return hipGetLastError();
}
template <typename O, typename Table>
hipError_t lookup(const Table& t, const LookupArgs& p) {
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
constexpr int kTile = 32;   // sorted rows that a group of lanes starts from
constexpr int kAhead = 8;   // rows in flight
constexpr int kLane = 8;    // columns of a lane

// Sort words, the sort's count, and the marks and the list cleared.
template <typename I>
__global__ void __launch_bounds__(256) embedding_keys_kernel(const I* index, int64_t istride, int64_t n, int64_t entries,
                                                             uint64_t* words, uint64_t* count, uint32_t* marks,
                                                             int64_t mark_words, uint32_t* listed) {
    const int64_t stride = (int64_t)gridDim.x * 256, at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at == 0) {
        count[0] = (uint64_t)n;
        listed[0] = 0;
    }
    for (int64_t i = at; i < n; i += stride) {
        const int64_t v = (int64_t)index[i * istride];
        words[i] = ((uint64_t)(v >= 0 && v < entries ? v : entries) << 32) | (uint32_t)i;
    }
    for (int64_t i = at; i < mark_words; i += stride) marks[i] = 0;
}

struct SumArgs {
    const uint64_t* words;
    int64_t n;
    uint32_t entries, dim;
    int lanes;        // lanes of a group: a power of two up to 64
    int64_t slices;   // groups side by side over the columns
    int64_t tiles;
    float factor;
    float* grad;      // [entries][dim]
    uint8_t* marks;   // [entries]: the entry has rows
    float* part;      // [tiles][2][dim]: sums of a long entry's rows in a tile, at its end (0) and at its start (1)
    uint32_t* listed; // [0] how many, then the tiles where a long entry starts
};

__device__ __forceinline__ uint32_t key_of(uint64_t w) { return (uint32_t)(w >> 32); }

// A group of lanes walks the sorted rows from a tile's start, adding rows until
// the index changes.  An entry belongs to the tile in which its rows start; that
// tile's group follows it into the next tile, so most entries are written once
// and whole.  An entry that also reaches the tile after the next is long: every
// tile leaves the sum of its own rows, and the join adds those in order.
template <typename T, bool DROP>
__global__ void __launch_bounds__(256) embedding_sums_kernel(const T* dy, int64_t lddy, SumArgs p, DropArgs a) {
    const int group = threadIdx.x / p.lanes, lane = threadIdx.x % p.lanes, groups = 256 / p.lanes;
    const int64_t unit = (int64_t)blockIdx.x * groups + group;
    const int64_t tile = unit / p.slices, slice = unit - tile * p.slices;
    if (tile >= p.tiles) return;
    const int64_t t0 = tile * kTile, t1 = min(t0 + kTile, p.n);
    const uint32_t head = key_of(p.words[t0]), last = key_of(p.words[t1 - 1]);
    if (head >= p.entries) return;  // rows without an entry only
    const int64_t c = (slice * p.lanes + lane) * kLane, left = (int64_t)p.dim - c;
    const bool first = slice == 0 && lane == 0;
    const Dropper drop(a);

    // the first rows' entry starts in an earlier tile; it is long, the last rows' entry is long
    const bool carried = t0 > 0 && key_of(p.words[t0 - 1]) == head;
    const bool head_long = carried && ((t0 > kTile && key_of(p.words[t0 - kTile - 1]) == head) ||
                                       (t1 < p.n && key_of(p.words[t1]) == head));
    const bool tail_long = !(carried && last == head) && last < p.entries && t1 + kTile < p.n &&
                           key_of(p.words[t1 + kTile]) == last;
    if (tail_long && first) p.listed[1 + atomicAdd(p.listed, 1u)] = (uint32_t)tile;

    float acc[kLane] = {};
    uint32_t cur = head;
    bool mine = !carried, done = false;
    for (int64_t at = t0; !done; at += kAhead) {
        uint64_t w[kAhead];
        float x[kAhead][kLane];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) w[u] = p.words[min(at + u, p.n - 1)];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) load8(dy + (int64_t)(uint32_t)w[u] * lddy + c, left, x[u]);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (done) continue;
            const uint32_t key = key_of(w[u]);
            const bool past = at + u >= t1;
            // the rows are at an end, or those of this tile are and the entry is another tile's or long
            const bool stop = at + u >= p.n || (past && (!mine || tail_long));
            if (stop || key != cur) {
                const bool partial = mine ? past && tail_long : head_long;
                if (mine && first) p.marks[cur] = 1;
                if (mine || head_long) {
                    const float f = partial ? 1.0f : p.factor;
                    float* out = partial ? p.part + (2 * tile + (mine ? 0 : 1)) * (int64_t)p.dim : p.grad + (int64_t)cur * p.dim;
#pragma unroll
                    for (int j = 0; j < kLane; ++j) acc[j] *= f;
                    store8(out + c, left, acc);
                }
                done = stop || past || key >= p.entries;
                cur = key;
                mine = true;
#pragma unroll
                for (int j = 0; j < kLane; ++j) acc[j] = 0.0f;
            }
            if (DROP) drop.apply(x[u], (uint32_t)w[u], (uint32_t)c, 1.0f);
#pragma unroll
            for (int j = 0; j < kLane; ++j) acc[j] += x[u][j];
        }
    }
}

// Long entries: the sums that their tiles left, added in double in a fixed
// order; then zeros for the entries without rows.
__global__ void __launch_bounds__(256) embedding_join_kernel(SumArgs p) {
    constexpr int COLS = 64, WAYS = 16;  // columns of a block's pass, tiles side by side
    __shared__ double s_sum[WAYS][COLS];
    const int way = threadIdx.x / (COLS / 4), q = threadIdx.x % (COLS / 4);
    const int64_t across = ((int64_t)p.dim + COLS - 1) / COLS, items = (int64_t)p.listed[0] * across;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t tile = p.listed[1 + it / across], c = (it % across) * COLS + 4 * q;
        const uint32_t key = key_of(p.words[(tile + 1) * kTile - 1]);
        int64_t more = 0;  // tiles behind this one that begin with the entry
        for (int found = 256; found == 256; more += found) {
            const int64_t t = (tile + 1 + more + threadIdx.x) * kTile;
            found = __syncthreads_count(t < p.n && key_of(p.words[t < p.n ? t : 0]) == key);
        }
        double sum[4] = {};
        for (int64_t k = way; k <= more; k += WAYS) {
            const float* from = p.part + (2 * (tile + k) + (k == 0 ? 0 : 1)) * (int64_t)p.dim + c;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < p.dim) sum[j] += (double)from[j];
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
    const int64_t chunks = ((int64_t)p.dim + kLane - 1) / kLane, total = (int64_t)p.entries * chunks;
    const float zeros[8] = {};
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t v = i / chunks, c = (i - v * chunks) * kLane;
        if (p.marks[v] == 0) store8(p.grad + v * p.dim + c, (int64_t)p.dim - c, zeros);
    }
}

struct GradLayout {
    size_t words0, words1, count, counts, digits, marks, listed, part, total;
};
GradLayout grad_layout(int64_t n, int64_t entries, int64_t dim) {
    const int64_t tiles = ceil_div(n, kTile);
    GradLayout l{};
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t here = at;
        at += round_up(bytes);
        return here;
    };
    l.words0 = take(8 * (size_t)n);
    l.words1 = take(8 * (size_t)n);
    l.count = take(8);
    l.counts = take(radix_sort_counts_bytes(radix_sort_blocks(n)));
    l.digits = take(4096);
    l.marks = take((size_t)entries);
    l.listed = take(4 * (size_t)(tiles + 1));
    l.part = take(2 * 4 * (size_t)tiles * (size_t)dim);
    l.total = at;
    return l;
}

template <typename I>
void launch_keys(const void* index, int64_t istride, int64_t n, int64_t entries, uint64_t* words, uint64_t* count,
                 uint32_t* marks, int64_t mark_words, uint32_t* listed, hipStream_t s) {
    IA_LAUNCH("embedding_keys_kernel", embedding_keys_kernel<I>, dim3(grid_for(n > mark_words ? n : mark_words)), dim3(256),
              0, s, (const I*)index, istride, n, entries, words, count, marks, mark_words, listed);
}

template <typename T>
hipError_t launch_sums(const void* dy, int64_t lddy, const SumArgs& p, const DropArgs* d, hipStream_t s) {
    const dim3 grid((unsigned)ceil_div(p.tiles * p.slices, 256 / p.lanes));
    if (d)
        IA_LAUNCH("embedding_sums_kernel", (embedding_sums_kernel<T, true>), grid, dim3(256), 0, s, (const T*)dy, lddy, p, *d);
    else
        IA_LAUNCH("embedding_sums_kernel", (embedding_sums_kernel<T, false>), grid, dim3(256), 0, s, (const T*)dy, lddy, p,
                  DropArgs{});
    return hipGetLastError();
}

__global__ void __launch_bounds__(256) embedding_zero_kernel(float* grad, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) grad[i] = 0.0f;
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
    return n == 0 || entries == 0 || dim == 0 ? 0 : grad_layout(n, entries, dim).total;
}

hipError_t launch_embedding_backward(const void* dy, int32_t dtype, int64_t dim, int64_t lddy, const Indices& ix,
                                     int64_t entries, float factor, const DropArgs* drop, float* grad, void* ws,
                                     hipStream_t s) {
    if (entries == 0 || dim == 0) return hipSuccess;
    if (ix.n == 0) {
        IA_LAUNCH("embedding_zero_kernel", embedding_zero_kernel, dim3(grid_for(entries * dim)), dim3(256), 0, s, grad,
                  entries * dim);
        return hipGetLastError();
    }
    const GradLayout l = grad_layout(ix.n, entries, dim);
    char* const w = (char*)ws;
    uint64_t* buf[2] = {(uint64_t*)(w + l.words0), (uint64_t*)(w + l.words1)};
    uint64_t* const count = (uint64_t*)(w + l.count);
    const int64_t mark_words = ceil_div(entries, 4);
    if (ix.bytes == 8)
        launch_keys<int64_t>(ix.index, ix.stride, ix.n, entries, buf[0], count, (uint32_t*)(w + l.marks), mark_words,
                             (uint32_t*)(w + l.listed), s);
    else
        launch_keys<int32_t>(ix.index, ix.stride, ix.n, entries, buf[0], count, (uint32_t*)(w + l.marks), mark_words,
                             (uint32_t*)(w + l.listed), s);
    int bits = 1;
    while ((entries >> bits) != 0) ++bits;
    const int at = radix_sort_u64(buf, count, (uint64_t)ix.n, 32, bits, radix_sort_blocks(ix.n), (uint32_t*)(w + l.counts),
                                  (uint32_t*)(w + l.digits), s);
    SumArgs p{};
    p.words = buf[at];
    p.n = ix.n;
    p.entries = (uint32_t)entries;
    p.dim = (uint32_t)dim;
    p.lanes = 1;
    while (p.lanes < 64 && p.lanes * kLane < dim) p.lanes *= 2;
    p.slices = ceil_div(dim, p.lanes * kLane);
    p.tiles = ceil_div(ix.n, kTile);
    p.factor = factor;
    p.grad = grad;
    p.marks = (uint8_t*)(w + l.marks);
    p.part = (float*)(w + l.part);
    p.listed = (uint32_t*)(w + l.listed);
    hipError_t e = IA_BY_DTYPE(dtype, launch_sums, dy, lddy, p, drop, s);
    if (e != hipSuccess) return e;
    const int64_t work = ceil_div(entries * ceil_div(dim, kLane), 256);
    const unsigned grid = (unsigned)(work < 256 ? 256 : work < 2048 ? work : 2048);
    IA_LAUNCH("embedding_join_kernel", embedding_join_kernel, dim3(grid), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace ia
