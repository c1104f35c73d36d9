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
// and once for its use.  Tensors are cut into chunks of kChunk elements; one
// launch covers up to kNormTensors (kScaleTensors, kAdamGroups) tensors, whose
// descriptors travel as kernel arguments, so that a decoder's fourteen groups
// take one launch and no table has to be uploaded.  Squares are summed in
// double (fp32 squares overflow from 1.8e19 on; the conversions and double
// multiply-adds hide behind the loads), per block, then over the blocks in a
// fixed order: the norm is the same on every run.
#include <hip/hip_runtime.h>

#include "adam_common.h"
#include "ia_internal.h"

namespace ia {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 4096;      // elements
constexpr int kMaxBlocks = 2048;  // 8 blocks per CU
constexpr int kTensors = 80;      // descriptors in 4 KB of kernel arguments
constexpr int kGroups = 48;

struct Tensor {
    const void* src;
    void* dst;
    int64_t n;
    int32_t dim, sstride, dstride;  // rows of dim elements stride apart (dim == stride: dense)
    int32_t dtype;
};

struct TensorArgs {
    int32_t count;
    int32_t first[kTensors + 1];  // first chunk of each tensor, then the number of chunks
    Tensor t[kTensors];
};
static_assert(sizeof(TensorArgs) <= 3900, "descriptors and the other arguments fit 4 KB");

struct Group {
    float* p;
    const float* g;
    float* m;
    float* v;
    uint16_t* p16;
    int64_t n;
    int32_t dim, stride;
    float step_size;
    int32_t pad;
};

struct GroupArgs {
    int32_t count;
    int32_t first[kGroups + 1];
    Group t[kGroups];
};
static_assert(sizeof(GroupArgs) <= 3900, "descriptors and the other arguments fit 4 KB");

// The tensor that holds chunk c (uniform over the block).
template <typename A>
__device__ __forceinline__ int find(const A& a, int c) {
    int lo = 0, hi = a.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.first[mid] <= c)
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

template <typename T>
__device__ __forceinline__ double squares(const Tensor& t, int64_t i0, int n) {
    const T* src = reinterpret_cast<const T*>(t.src);
    if (t.dim == t.sstride) return chunk_squares(src + i0, n);
    return chunk_squares_strided(src, i0, n, t.dim, t.sstride);
}

__device__ __forceinline__ double block_sum(double s) {
    __shared__ double red[kThreads / 64];
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(TensorArgs a, double* part) {
    double s = 0.0;
    for (int c = blockIdx.x; c < a.first[a.count]; c += gridDim.x) {
        const int k = find(a, c);
        const Tensor& t = a.t[k];
        const int64_t i0 = (int64_t)(c - a.first[k]) * kChunk;
        const int n = (int)min((int64_t)kChunk, t.n - i0);
        if (t.dtype == IA_DTYPE_F32)
            s += squares<float>(t, i0, n);
        else if (t.dtype == IA_DTYPE_F16)
            s += squares<_Float16>(t, i0, n);
        else
            s += squares<__bf16>(t, i0, n);
    }
    s = block_sum(s);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// One block: the partial sums added in a fixed order.  stats = {norm, factor,
// 1 if the norm is finite else 0}, rounded once from double.
__global__ void __launch_bounds__(kThreads) norm_finish_kernel(const double* part, int n, float max_norm,
                                                               float* stats) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) s += part[i];
    s = block_sum(s);
    if (threadIdx.x == 0) {
        const double norm = sqrt(s);
        // a NaN norm passes NaN on; an infinite one gives 0
        const double f = norm > (double)max_norm ? (double)max_norm / norm : (norm == norm ? 1.0 : norm);
        stats[0] = (float)norm;
        stats[1] = (float)f;
        stats[2] = isfinite(norm) ? 1.0f : 0.0f;
    }
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const Tensor& t, int64_t i0, int n, float f) {
    constexpr int E = Vec<T>::N, V = kChunk / (kThreads * E);
    const T* src = reinterpret_cast<const T*>(t.src);
    T* dst = reinterpret_cast<T*>(t.dst);
    if (t.dim != t.sstride || t.dim != t.dstride) {
        for (int k = threadIdx.x; k < n; k += kThreads) {
            const int64_t row = (i0 + k) / t.dim, col = i0 + k - row * t.dim;
            dst[row * t.dstride + col] = (T)((float)src[row * t.sstride + col] * f);
        }
        return;
    }
    src += i0;
    dst += i0;
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
            store_vec(dst + (size_t)i * E, v[j]);
        }
    }
    const int r = nv * E + (int)threadIdx.x;
    if (r < n) dst[r] = (T)((float)src[r] * f);
}

__global__ void __launch_bounds__(kThreads) grad_scale_kernel(TensorArgs a, const float* stats) {
    const float f = stats[1];
    for (int c = blockIdx.x; c < a.first[a.count]; c += gridDim.x) {
        const int k = find(a, c);
        const Tensor& t = a.t[k];
        if (f == 1.0f && t.src == t.dst) continue;  // in place: every product is its own value
        const int64_t i0 = (int64_t)(c - a.first[k]) * kChunk;
        const int n = (int)min((int64_t)kChunk, t.n - i0);
        if (t.dtype == IA_DTYPE_F32)
            scale_chunk<float>(t, i0, n, f);
        else if (t.dtype == IA_DTYPE_F16)
            scale_chunk<_Float16>(t, i0, n, f);
        else
            scale_chunk<__bf16>(t, i0, n, f);
    }
}

__device__ __forceinline__ void adam_chunk(const Group& t, int64_t i0, int n, float f, const AdamConsts& c) {
    const float* g = t.g + i0;
    float* m = t.m + i0;
    float* v = t.v + i0;
    uint16_t* p16 = t.p16 ? t.p16 + i0 : nullptr;
    if (t.dim != t.stride) {
        for (int k = threadIdx.x; k < n; k += kThreads) {
            const int64_t row = (i0 + k) / t.dim;
            float* p = t.p + row * t.stride + (i0 + k - row * t.dim);
            float mi = m[k], vi = v[k];
            const float pi = adam_element(*p, g[k] * f, mi, vi, c, t.step_size);
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
        Vec<float> pv = load_vec(p + 4 * i), mv = load_vec(m + 4 * i), vv = load_vec(v + 4 * i);
        const Vec<float> gv = load_vec(g + 4 * i);
        uint16_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            pv.e[e] = adam_element(pv.e[e], gv.e[e] * f, mv.e[e], vv.e[e], c, t.step_size);
            h[e] = __builtin_bit_cast(uint16_t, (_Float16)pv.e[e]);
        }
        store_vec(p + 4 * i, pv);
        store_vec(m + 4 * i, mv);
        store_vec(v + 4 * i, vv);
        if (p16) __builtin_memcpy(p16 + 4 * i, h, 8);
    }
    const int k = nv * 4 + (int)threadIdx.x;
    if (k < n) {
        float mi = m[k], vi = v[k];
        const float pi = adam_element(p[k], g[k] * f, mi, vi, c, t.step_size);
        m[k] = mi;
        v[k] = vi;
        p[k] = pi;
        if (p16) p16[k] = __builtin_bit_cast(uint16_t, (_Float16)pi);
    }
}

__global__ void __launch_bounds__(kThreads) adam_clip_kernel(GroupArgs a, AdamConsts c, const float* stats) {
    const float f = stats[1];
    if (stats[2] == 0.0f) return;  // gradients that are not finite change nothing
    for (int k = blockIdx.x; k < a.first[a.count]; k += gridDim.x) {
        const int t = find(a, k);
        const int64_t i0 = (int64_t)(k - a.first[t]) * kChunk;
        adam_chunk(a.t[t], i0, (int)min((int64_t)kChunk, a.t[t].n - i0), f, c);
    }
}

int chunks(int64_t n) { return (int)((n + kChunk - 1) / kChunk); }

// Calls launch(args, blocks) for consecutive runs of tensors that fit one
// launch's descriptors; fill(k, args.t[i]) describes tensor k and returns its
// size.  Empty tensors are left out.
template <typename A, typename Fill, typename Launch>
hipError_t each_launch(int count, int capacity, Fill fill, Launch launch) {
    A a;
    a.count = 0;
    a.first[0] = 0;
    for (int k = 0; k <= count; ++k) {
        if (k < count) {
            const int64_t n = fill(k, a.t[a.count]);
            if (n == 0) continue;
            a.first[a.count + 1] = a.first[a.count] + chunks(n);
            ++a.count;
        }
        if (a.count == capacity || (k == count && a.count > 0)) {
            const int c = a.first[a.count];
            launch(a, c < kMaxBlocks ? c : kMaxBlocks);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            a.count = 0;
        }
    }
    return hipSuccess;
}

int64_t fill_tensor(const ia_grad& g, Tensor& t) {
    const bool dense = g.stride == g.dim && (!g.out || g.out_stride == g.dim);
    t.src = g.data;
    t.dst = g.out ? g.out : g.data;
    t.n = g.rows * g.dim;
    t.dim = dense ? 1 : g.dim;
    t.sstride = dense ? 1 : g.stride;
    t.dstride = dense ? 1 : (g.out ? g.out_stride : g.stride);
    t.dtype = g.dtype;
    return t.n;
}

hipError_t norm_passes(const ia_grad* grads, int count, float max_norm, double* part, float* stats, hipStream_t s) {
    int parts = 0;
    hipError_t e = each_launch<TensorArgs>(
        count, kTensors, [&](int k, Tensor& t) { return fill_tensor(grads[k], t); },
        [&](const TensorArgs& a, int blocks) {
            IA_LAUNCH("grad_norm_kernel", grad_norm_kernel, dim3(blocks), dim3(kThreads), 0, s, a, part + parts);
            parts += blocks;
        });
    if (e != hipSuccess) return e;
    IA_LAUNCH("norm_finish_kernel", norm_finish_kernel, dim3(1), dim3(kThreads), 0, s, (const double*)part, parts,
              max_norm, stats);
    return hipGetLastError();
}

}  // namespace

// One double per block of every norm launch
size_t clip_workspace(int32_t tensors) {
    return ((size_t)tensors / kTensors + 1) * kMaxBlocks * sizeof(double);
}

int64_t clip_chunk() { return kChunk; }

hipError_t launch_grad_norm(const ia_grad* grads, int32_t count, float max_norm, void* ws, float* stats,
                            hipStream_t s) {
    return norm_passes(grads, count, max_norm, reinterpret_cast<double*>(ws), stats, s);
}

hipError_t launch_clip_grad_norm(const ia_grad* grads, int32_t count, float max_norm, void* ws, float* stats,
                                 hipStream_t s) {
    hipError_t e = norm_passes(grads, count, max_norm, reinterpret_cast<double*>(ws), stats, s);
    if (e != hipSuccess) return e;
    return each_launch<TensorArgs>(
        count, kTensors, [&](int k, Tensor& t) { return fill_tensor(grads[k], t); },
        [&](const TensorArgs& a, int blocks) {
            IA_LAUNCH("grad_scale_kernel", grad_scale_kernel, dim3(blocks), dim3(kThreads), 0, s, a,
                      (const float*)stats);
        });
}

hipError_t launch_adam_clip(const ia_adam_group* groups, int32_t count, float max_norm, float beta1, float beta2,
                            float eps, int32_t step, void* ws, float* stats, hipStream_t s) {
    double* part = reinterpret_cast<double*>(ws);
    int parts = 0;
    hipError_t e = each_launch<TensorArgs>(
        count, kTensors,
        [&](int k, Tensor& t) {
            const int64_t n = groups[k].rows * groups[k].dim;
            t = Tensor{groups[k].grad, nullptr, n, 1, 1, 1, IA_DTYPE_F32};
            return n;
        },
        [&](const TensorArgs& a, int blocks) {
            IA_LAUNCH("grad_norm_kernel", grad_norm_kernel, dim3(blocks), dim3(kThreads), 0, s, a, part + parts);
            parts += blocks;
        });
    if (e != hipSuccess) return e;
    IA_LAUNCH("norm_finish_kernel", norm_finish_kernel, dim3(1), dim3(kThreads), 0, s, (const double*)part, parts,
              max_norm, stats);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const AdamConsts c{beta1, beta2, eps, (float)(1.0 / (1.0 - pow((double)beta2, (double)step)))};
    const double correction = 1.0 - pow((double)beta1, (double)step);
    return each_launch<GroupArgs>(
        count, kGroups,
        [&](int k, Group& t) {
            const ia_adam_group& g = groups[k];
            const bool dense = g.dim == g.param_stride;
            t = Group{g.param, g.grad, g.m, g.v, g.param_f16, g.rows * g.dim, dense ? 1 : g.dim,
                      dense ? 1 : g.param_stride, (float)((double)g.lr / correction), 0};
            return t.n;
        },
        [&](const GroupArgs& a, int blocks) {
            IA_LAUNCH("adam_clip_kernel", adam_clip_kernel, dim3(blocks), dim3(kThreads), 0, s, a, c,
                      (const float*)stats);
        });
}

}  // namespace ia
