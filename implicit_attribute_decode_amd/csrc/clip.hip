// Global gradient norm over many tensors, clipping by it (Pascanu, Mikolov &
// Bengio, "On the difficulty of training recurrent neural networks", 2013,
// §3.2: scale every gradient by max_norm / norm when the norm exceeds it),
// and the Adam step over every parameter group that applies the factor while
// it reads the gradients.
//
//   norm = sqrt(sum over tensors and elements of g^2)
//   factor = max_norm / norm if norm > max_norm, else 1
//
// All three are bound by memory: a call reads each gradient once for the norm
// and once for its use.  Tensors are cut into chunks of kChunk elements, and
// as many tensors as their descriptors fit into 4 KB of kernel arguments go
// into one launch (kNormTensors, kScaleTensors, kGroups), so that a decoder's
// fourteen groups take one and no table has to be uploaded.  Squares are
// summed in double (fp32 squares overflow from 1.8e19 on; the conversions and
// double multiply-adds hide behind the loads), per block.  Every block of the
// pass that uses the factor adds the blocks' sums itself, all in one order:
// the norm is the same on every run, and no third launch stands between.
#include <hip/hip_runtime.h>

#include "adam_common.h"
#include "ia_internal.h"

namespace ia {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 4096;      // elements
constexpr int kNormBlocks = 1024;  // most blocks of a norm launch (each leaves one sum)
constexpr int kUseBlocks = 2048;   // of a launch that uses the factor
constexpr int kMostParts = 2048;   // sums that every block adds by itself
constexpr int kNormTensors = 240;
constexpr int kScaleTensors = 160;
constexpr int kStridedTensors = 80;
constexpr int kGroups = 48;

// A dense tensor to read: its size is its chunks, less `slack` elements of the
// last one.
struct Dense {
    const void* src;
    uint32_t dtype_slack;  // dtype | slack << 2
    int32_t first;         // its first chunk in the launch
};
struct DenseArgs {
    int32_t count, chunks;
    Dense t[kNormTensors];
};
static_assert(sizeof(DenseArgs) <= 3968, "descriptors and the other arguments fit 4 KB");

// A dense tensor to scale.
struct Scaled {
    const void* src;
    void* dst;
    uint32_t dtype_slack;
    int32_t first;
};
struct ScaledArgs {
    int32_t count, chunks;
    Scaled t[kScaleTensors];
};
static_assert(sizeof(ScaledArgs) <= 3968, "descriptors and the other arguments fit 4 KB");

// Rows of dim elements, sstride (dstride) apart.
struct Strided {
    const void* src;
    void* dst;
    int64_t n;
    int32_t dim, sstride, dstride;
    int32_t dtype;
    int32_t first;
    int32_t pad;
};
struct StridedArgs {
    int32_t count, chunks;
    Strided t[kStridedTensors];
};
static_assert(sizeof(StridedArgs) <= 3968, "descriptors and the other arguments fit 4 KB");

struct Group {
    float* p;
    const float* g;
    float* m;
    float* v;
    uint16_t* p16;
    int64_t n;
    int32_t dim, stride;  // the parameter's rows (dim == stride: dense)
    float step_size;
    int32_t first;
};
struct GroupArgs {
    int32_t count, chunks;
    Group t[kGroups];
};
static_assert(sizeof(GroupArgs) <= 3900, "descriptors and the other arguments fit 4 KB");

// The tensor that holds chunk c (uniform over the block), at or after `from`.
template <typename A>
__device__ __forceinline__ int find(const A& a, int c, int from) {
    int lo = from, hi = a.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.t[mid].first <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// 16 bytes from an address that is aligned to T only (one global_load_dwordx4;
// views into a bucket start at any element).
template <typename T>
struct Vec {
    static constexpr int N = 16 / (int)sizeof(T);
    T e[N];
};

template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T* p) {
    Vec<T> v;
    __builtin_memcpy(&v, p, sizeof(v));
    return v;
}

template <typename T>
__device__ __forceinline__ void store_vec(T* p, const Vec<T>& v) {
    __builtin_memcpy(p, &v, sizeof(v));
}

// The same for data that this call reads or writes once: it does not displace
// what the memory-side cache holds (the gradients, between their two readings).
// Parameters and moments so: an Adam step over 16.8M, 50M and 158M parameters
// 113 -> 104, 340 -> 295 and 1072 -> 1036 us; clipped copies so: 16.8M and 67M
// gradients 40 -> 35 and 151 -> 135 us.  The gradients themselves are read in
// the ordinary way: read once only, the norm is faster (149 -> 110 us at 158M)
// and the step slower by as much or more (295 -> 325 us in all at 50M).
typedef uint32_t uintx4 __attribute__((ext_vector_type(4)));
typedef uint32_t loose_uintx4 __attribute__((ext_vector_type(4), aligned(2)));
template <typename T>
__device__ __forceinline__ Vec<T> load_once(const T* p) {
    Vec<T> v;
    const uintx4 w = __builtin_nontemporal_load(reinterpret_cast<const loose_uintx4*>(p));
    __builtin_memcpy(&v, &w, sizeof(v));
    return v;
}
template <typename T>
__device__ __forceinline__ void store_once(T* p, const Vec<T>& v) {
    uintx4 w;
    __builtin_memcpy(&w, &v, sizeof(w));
    __builtin_nontemporal_store(w, reinterpret_cast<loose_uintx4*>(p));
}

__device__ __forceinline__ double square(float g) {
    const double d = (double)g;
    return d * d;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* src, int n) {
    constexpr int E = Vec<T>::N, V = kChunk / (kThreads * E);
    const int nv = n / E;
    Vec<T> v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = j * kThreads + (int)threadIdx.x;
        if (i < nv) v[j] = load_vec(src + (size_t)i * E);
    }
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (j * kThreads + (int)threadIdx.x < nv) {
#pragma unroll
            for (int e = 0; e < E; ++e) s += square((float)v[j].e[e]);
        }
    const int r = nv * E + (int)threadIdx.x;
    if (r < n) s += square((float)src[r]);
    return s;
}

template <typename T>
__device__ double chunk_squares_strided(const T* src, int64_t i0, int n, int dim, int stride) {
    double s = 0.0;
    for (int k = threadIdx.x; k < n; k += kThreads) {
        const int64_t row = (i0 + k) / dim;
        s += square((float)src[row * stride + (i0 + k - row * dim)]);
    }
    return s;
}

// Elements of chunk c of the tensor with descriptor word w and chunks up to
// `next`.
__device__ __forceinline__ int elements(uint32_t w, int c, int next) { return c + 1 == next ? kChunk - (int)(w >> 2) : kChunk; }

// The sum over the block, on all threads.
__device__ __forceinline__ double block_sum(double s) {
    __shared__ double red[kThreads / 64];
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(DenseArgs a, double* part) {
    double s = 0.0;
    int k = 0;
    for (int c = blockIdx.x; c < a.chunks; c += gridDim.x) {
        k = find(a, c, k);
        const uint32_t w = a.t[k].dtype_slack;
        const int n = elements(w, c, k + 1 < a.count ? a.t[k + 1].first : a.chunks);
        const int64_t i0 = (int64_t)(c - a.t[k].first) * kChunk;
        if ((w & 3) == IA_DTYPE_F32)
            s += chunk_squares(reinterpret_cast<const float*>(a.t[k].src) + i0, n);
        else if ((w & 3) == IA_DTYPE_F16)
            s += chunk_squares(reinterpret_cast<const _Float16*>(a.t[k].src) + i0, n);
        else
            s += chunk_squares(reinterpret_cast<const __bf16*>(a.t[k].src) + i0, n);
    }
    s = block_sum(s);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads) grad_norm_strided_kernel(StridedArgs a, double* part) {
    double s = 0.0;
    int k = 0;
    for (int c = blockIdx.x; c < a.chunks; c += gridDim.x) {
        k = find(a, c, k);
        const Strided& t = a.t[k];
        const int64_t i0 = (int64_t)(c - t.first) * kChunk;
        const int n = (int)min((int64_t)kChunk, t.n - i0);
        if (t.dtype == IA_DTYPE_F32)
            s += chunk_squares_strided(reinterpret_cast<const float*>(t.src), i0, n, t.dim, t.sstride);
        else if (t.dtype == IA_DTYPE_F16)
            s += chunk_squares_strided(reinterpret_cast<const _Float16*>(t.src), i0, n, t.dim, t.sstride);
        else
            s += chunk_squares_strided(reinterpret_cast<const __bf16*>(t.src), i0, n, t.dim, t.sstride);
    }
    s = block_sum(s);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The norm launches' sums and what comes of them.
struct Norm {
    const double* part;
    int32_t parts;
    float max_norm;
    float* stats;  // {norm, factor, 1 if the norm is finite else 0}
};

// The factor, on all threads; the first block writes stats, each value rounded
// once from double.
__device__ __forceinline__ float clip_factor(const Norm& m, bool& finite) {
    double s = 0.0;
    for (int i = threadIdx.x; i < m.parts; i += kThreads) s += m.part[i];
    const double norm = sqrt(block_sum(s)), most = (double)m.max_norm;
    // a NaN norm passes NaN on; an infinite one gives 0
    const float f = (float)(norm > most ? most / norm : (norm == norm ? 1.0 : norm));
    finite = isfinite(norm);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        m.stats[0] = (float)norm;
        m.stats[1] = f;
        m.stats[2] = finite ? 1.0f : 0.0f;
    }
    return f;
}

__global__ void __launch_bounds__(kThreads) norm_collect_kernel(double* part, int32_t parts) {
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) s += part[i];
    s = block_sum(s);
    if (threadIdx.x == 0) part[0] = s;
}

__global__ void __launch_bounds__(kThreads) norm_finish_kernel(Norm m) {
    bool finite;
    (void)clip_factor(m, finite);
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const T* src, T* dst, int n, float f) {
    constexpr int E = Vec<T>::N, V = kChunk / (kThreads * E);
    const int nv = n / E;
    Vec<T> v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = j * kThreads + (int)threadIdx.x;
        if (i < nv) v[j] = load_vec(src + (size_t)i * E);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = j * kThreads + (int)threadIdx.x;
        if (i < nv) {
#pragma unroll
            for (int e = 0; e < E; ++e) v[j].e[e] = (T)((float)v[j].e[e] * f);
            if (src == dst)
                store_vec(dst + (size_t)i * E, v[j]);
            else
                store_once(dst + (size_t)i * E, v[j]);
        }
    }
    const int r = nv * E + (int)threadIdx.x;
    if (r < n) dst[r] = (T)((float)src[r] * f);
}

__global__ void __launch_bounds__(kThreads) grad_scale_kernel(ScaledArgs a, Norm m) {
    bool finite;
    const float f = clip_factor(m, finite);
    int k = 0;
    for (int c = blockIdx.x; c < a.chunks; c += gridDim.x) {
        k = find(a, c, k);
        const void* src = a.t[k].src;
        void* dst = a.t[k].dst;
        if (f == 1.0f && src == dst) continue;  // in place: every product is its own value
        const uint32_t w = a.t[k].dtype_slack;
        const int n = elements(w, c, k + 1 < a.count ? a.t[k + 1].first : a.chunks);
        const int64_t i0 = (int64_t)(c - a.t[k].first) * kChunk;
        if ((w & 3) == IA_DTYPE_F32)
            scale_chunk(reinterpret_cast<const float*>(src) + i0, reinterpret_cast<float*>(dst) + i0, n, f);
        else if ((w & 3) == IA_DTYPE_F16)
            scale_chunk(reinterpret_cast<const _Float16*>(src) + i0, reinterpret_cast<_Float16*>(dst) + i0, n, f);
        else
            scale_chunk(reinterpret_cast<const __bf16*>(src) + i0, reinterpret_cast<__bf16*>(dst) + i0, n, f);
    }
}

template <typename T>
__device__ __forceinline__ void scale_strided(const Strided& t, int64_t i0, int n, float f) {
    const T* src = reinterpret_cast<const T*>(t.src);
    T* dst = reinterpret_cast<T*>(t.dst);
    for (int k = threadIdx.x; k < n; k += kThreads) {
        const int64_t row = (i0 + k) / t.dim, col = i0 + k - row * t.dim;
        dst[row * t.dstride + col] = (T)((float)src[row * t.sstride + col] * f);
    }
}

__global__ void __launch_bounds__(kThreads) grad_scale_strided_kernel(StridedArgs a, Norm m) {
    bool finite;
    const float f = clip_factor(m, finite);
    int k = 0;
    for (int c = blockIdx.x; c < a.chunks; c += gridDim.x) {
        k = find(a, c, k);
        const Strided& t = a.t[k];
        if (f == 1.0f && t.src == t.dst) continue;
        const int64_t i0 = (int64_t)(c - t.first) * kChunk;
        const int n = (int)min((int64_t)kChunk, t.n - i0);
        if (t.dtype == IA_DTYPE_F32)
            scale_strided<float>(t, i0, n, f);
        else if (t.dtype == IA_DTYPE_F16)
            scale_strided<_Float16>(t, i0, n, f);
        else
            scale_strided<__bf16>(t, i0, n, f);
    }
}

// Steps that the call before this one left out (device count or null): the bias
// corrections are those of the steps applied.
struct Skips {
    int32_t* count;
    int32_t step;   // this call's, those left out included
    int32_t first;  // the first launch of the call counts
};

// 1 - b^t
__device__ __forceinline__ double bias_correction(double b, int t) {
    double p = 1.0;
    for (; t > 0; t >>= 1, b *= b)
        if (t & 1) p *= b;
    return 1.0 - p;
}

__device__ __forceinline__ void adam_chunk(const Group& t, int64_t i0, int n, float f, float step_size,
                                           const AdamConsts& c) {
    const float* g = t.g + i0;
    float* m = t.m + i0;
    float* v = t.v + i0;
    uint16_t* p16 = t.p16 ? t.p16 + i0 : nullptr;
    if (t.dim != t.stride) {
        for (int k = threadIdx.x; k < n; k += kThreads) {
            const int64_t row = (i0 + k) / t.dim;
            float* p = t.p + row * t.stride + (i0 + k - row * t.dim);
            float mi = m[k], vi = v[k];
            const float pi = adam_element(*p, g[k] * f, mi, vi, c, step_size);
            m[k] = mi;
            v[k] = vi;
            *p = pi;
            if (p16) p16[k] = __builtin_bit_cast(uint16_t, (_Float16)pi);
        }
        return;
    }
    float* p = t.p + i0;
    const int nv = n / 4;
    for (int i = threadIdx.x; i < nv; i += kThreads) {
        Vec<float> pv = load_once(p + 4 * i), mv = load_once(m + 4 * i), vv = load_once(v + 4 * i);
        const Vec<float> gv = load_vec(g + 4 * i);
        uint16_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            pv.e[e] = adam_element(pv.e[e], gv.e[e] * f, mv.e[e], vv.e[e], c, step_size);
            h[e] = __builtin_bit_cast(uint16_t, (_Float16)pv.e[e]);
        }
        store_once(p + 4 * i, pv);
        store_once(m + 4 * i, mv);
        store_once(v + 4 * i, vv);
        if (p16) __builtin_memcpy(p16 + 4 * i, h, 8);
    }
    const int k = nv * 4 + (int)threadIdx.x;
    if (k < n) {
        float mi = m[k], vi = v[k];
        const float pi = adam_element(p[k], g[k] * f, mi, vi, c, step_size);
        m[k] = mi;
        v[k] = vi;
        p[k] = pi;
        if (p16) p16[k] = __builtin_bit_cast(uint16_t, (_Float16)pi);
    }
}

__global__ void __launch_bounds__(kThreads) adam_clip_kernel(GroupArgs a, AdamConsts c, Norm m, Skips left_out) {
    bool finite;
    const float f = clip_factor(m, finite);
    if (!finite) {  // gradients that are not finite change nothing
        if (left_out.count && left_out.first && blockIdx.x == 0 && threadIdx.x == 0) *left_out.count += 1;
        return;
    }
    float rate = 1.0f;
    if (const int skipped = left_out.count ? *left_out.count : 0; skipped > 0) {
        const int t = max(left_out.step - skipped, 1);
        rate = (float)(bias_correction((double)c.b1, left_out.step) / bias_correction((double)c.b1, t));
        c.v_scale = (float)(1.0 / bias_correction((double)c.b2, t));
    }
    int t = 0;
    for (int k = blockIdx.x; k < a.chunks; k += gridDim.x) {
        t = find(a, k, t);
        const int64_t i0 = (int64_t)(k - a.t[t].first) * kChunk;
        adam_chunk(a.t[t], i0, (int)min((int64_t)kChunk, a.t[t].n - i0), f, a.t[t].step_size * rate, c);
    }
}

int64_t chunks(int64_t n) { return (n + kChunk - 1) / kChunk; }
uint32_t dtype_slack(int32_t dtype, int64_t n) { return (uint32_t)dtype | (uint32_t)(chunks(n) * kChunk - n) << 2; }

// Calls launch(args, blocks) for consecutive runs of tensors that fit one
// launch's descriptors; fill(k, args.t[i]) describes tensor k and returns its
// size (0: it is left out).
template <typename A, typename Fill, typename Launch>
hipError_t each_launch(int count, int capacity, int most, Fill fill, Launch launch) {
    A a;
    a.count = a.chunks = 0;
    for (int k = 0; k <= count; ++k) {
        if (k < count) {
            const int64_t n = fill(k, a.t[a.count]);
            if (n > 0) {
                a.t[a.count].first = a.chunks;
                a.chunks += (int32_t)chunks(n);
                ++a.count;
            }
        }
        if (a.count > 0 && (a.count == capacity || k == count)) {
            launch(a, a.chunks < most ? a.chunks : most);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            a.count = a.chunks = 0;
        }
    }
    return hipSuccess;
}

bool is_dense(const ia_grad& g) { return g.stride == g.dim && (!g.out || g.out_stride == g.dim); }

int64_t fill_strided(const ia_grad& g, Strided& t) {
    if (is_dense(g)) return 0;
    t = Strided{g.data, g.out ? g.out : g.data, g.rows * g.dim, g.dim, g.stride, g.out ? g.out_stride : g.stride, g.dtype,
                0, 0};
    return t.n;
}

int64_t fill_dense(const void* src, int32_t dtype, int64_t n, Dense& t) {
    t.src = src;
    t.dtype_slack = dtype_slack(dtype, n);
    return n;
}

// Leaves every block's sum in part; returns how many through m.parts.
hipError_t norm_passes(const ia_grad* grads, int count, double* part, Norm& m, hipStream_t s) {
    hipError_t e = each_launch<DenseArgs>(
        count, kNormTensors, kNormBlocks,
        [&](int k, Dense& t) {
            return is_dense(grads[k]) ? fill_dense(grads[k].data, grads[k].dtype, grads[k].rows * grads[k].dim, t) : 0;
        },
        [&](const DenseArgs& a, int blocks) {
            IA_LAUNCH("grad_norm_kernel", grad_norm_kernel, dim3(blocks), dim3(kThreads), 0, s, a, part + m.parts);
            m.parts += blocks;
        });
    if (e != hipSuccess) return e;
    return each_launch<StridedArgs>(
        count, kStridedTensors, kNormBlocks, [&](int k, Strided& t) { return fill_strided(grads[k], t); },
        [&](const StridedArgs& a, int blocks) {
            IA_LAUNCH("grad_norm_strided_kernel", grad_norm_strided_kernel, dim3(blocks), dim3(kThreads), 0, s, a,
                      part + m.parts);
            m.parts += blocks;
        });
}

// Very many tensors leave so many sums that adding them in every block would
// cost more than a launch: one block joins them first.
hipError_t collect(double* part, Norm& m, hipStream_t s) {
    if (m.parts <= kMostParts) return hipSuccess;
    IA_LAUNCH("norm_collect_kernel", norm_collect_kernel, dim3(1), dim3(kThreads), 0, s, part, m.parts);
    m.parts = 1;
    return hipGetLastError();
}

hipError_t finish(const Norm& m, hipStream_t s) {
    IA_LAUNCH("norm_finish_kernel", norm_finish_kernel, dim3(1), dim3(kThreads), 0, s, m);
    return hipGetLastError();
}

}  // namespace

// One double per block of every norm launch: tensors of more than
// kNormTensors, or strided ones between dense ones, take several.
size_t clip_workspace(int32_t tensors) {
    return ((size_t)tensors / kNormTensors + (size_t)tensors / kStridedTensors + 2) * kNormBlocks * sizeof(double);
}

hipError_t launch_grad_norm(const ia_grad* grads, int32_t count, float max_norm, void* ws, float* stats,
                            hipStream_t s) {
    double* part = reinterpret_cast<double*>(ws);
    Norm m{part, 0, max_norm, stats};
    hipError_t e = norm_passes(grads, count, part, m, s);
    return e != hipSuccess ? e : finish(m, s);
}

hipError_t launch_clip_grad_norm(const ia_grad* grads, int32_t count, float max_norm, void* ws, float* stats,
                                 hipStream_t s) {
    double* part = reinterpret_cast<double*>(ws);
    Norm m{part, 0, max_norm, stats};
    hipError_t e = norm_passes(grads, count, part, m, s);
    if (e == hipSuccess) e = collect(part, m, s);
    if (e != hipSuccess) return e;
    if (m.parts == 0) return finish(m, s);
    e = each_launch<ScaledArgs>(
        count, kScaleTensors, kUseBlocks,
        [&](int k, Scaled& t) {
            const ia_grad& g = grads[k];
            if (!is_dense(g)) return (int64_t)0;
            t.src = g.data;
            t.dst = g.out ? g.out : g.data;
            t.dtype_slack = dtype_slack(g.dtype, g.rows * g.dim);
            return g.rows * g.dim;
        },
        [&](const ScaledArgs& a, int blocks) {
            IA_LAUNCH("grad_scale_kernel", grad_scale_kernel, dim3(blocks), dim3(kThreads), 0, s, a, m);
        });
    if (e != hipSuccess) return e;
    return each_launch<StridedArgs>(
        count, kStridedTensors, kUseBlocks, [&](int k, Strided& t) { return fill_strided(grads[k], t); },
        [&](const StridedArgs& a, int blocks) {
            IA_LAUNCH("grad_scale_strided_kernel", grad_scale_strided_kernel, dim3(blocks), dim3(kThreads), 0, s, a, m);
        });
}

hipError_t launch_adam_clip(const ia_adam_group* groups, int32_t count, float max_norm, float beta1, float beta2,
                            float eps, int32_t step, void* ws, int32_t* skipped, float* stats, hipStream_t s) {
    double* part = reinterpret_cast<double*>(ws);
    Norm m{part, 0, max_norm, stats};
    hipError_t e = each_launch<DenseArgs>(
        count, kNormTensors, kNormBlocks,
        [&](int k, Dense& t) { return fill_dense(groups[k].grad, IA_DTYPE_F32, groups[k].rows * groups[k].dim, t); },
        [&](const DenseArgs& a, int blocks) {
            IA_LAUNCH("grad_norm_kernel", grad_norm_kernel, dim3(blocks), dim3(kThreads), 0, s, a, part + m.parts);
            m.parts += blocks;
        });
    if (e == hipSuccess) e = collect(part, m, s);
    if (e != hipSuccess) return e;
    if (m.parts == 0) return finish(m, s);
    Skips left_out{skipped, step, 1};
    const AdamConsts c{beta1, beta2, eps, (float)(1.0 / (1.0 - pow((double)beta2, (double)step)))};
    const double correction = 1.0 - pow((double)beta1, (double)step);
    return each_launch<GroupArgs>(
        count, kGroups, kUseBlocks,
        [&](int k, Group& t) {
            const ia_adam_group& g = groups[k];
            const bool dense = g.dim == g.param_stride;
            t = Group{g.param, g.grad, g.m, g.v, g.param_f16, g.rows * g.dim, dense ? 1 : g.dim,
                      dense ? 1 : g.param_stride, (float)((double)g.lr / correction), 0};
            return t.n;
        },
        [&](const GroupArgs& a, int blocks) {
            IA_LAUNCH("adam_clip_kernel", adam_clip_kernel, dim3(blocks), dim3(kThreads), 0, s, a, c, m, left_out);
            left_out.first = 0;
        });
}

}  // namespace ia
