// Global gradient norm and clipping on gfx950.
//
//   S = sum over all listed tensors of g^2,   norm = sqrt(S),
//   coef = min(1, max_norm / (norm + 1e-6)),  dst = coef * src.
//
// The sum is held in float64 from the first element on: the square of a
// float32 is exact there, nothing overflows or underflows (a float32 sum of
// squares leaves its range at |g| > 1.8e19 and below 1e-19), and billions of
// terms keep all digits that the float32 result can show.  A float64 fused
// multiply-add runs at the float32 rate on gfx950, so the kernel stays bound by
// HBM reads all the same.
//
// Sums have one order whatever runs first: thread, wave, workgroup, then the
// partials by slot.  No atomics.
#include "clip_internal.h"
#include "k_common.h"

#pragma clang fp contract(off)

namespace muon {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

typedef uint32_t u32x4_stream __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int64_t meta_numel(uint64_t m) { return int64_t(m & ((uint64_t(1) << 35) - 1)); }
__device__ __forceinline__ int meta_src(uint64_t m) { return int(m >> 35) & 1; }
__device__ __forceinline__ int meta_dst(uint64_t m) { return int(m >> 36) & 1; }
__device__ __forceinline__ int meta_unit(uint64_t m) { return int(m >> 37); }

// Tensor that owns unit u: the last one whose first unit is <= u (every tensor
// owns at least one unit).
__device__ __forceinline__ int tensor_of(const uint64_t* meta, int n, int u) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (meta_unit(meta[mid]) <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Sum over the workgroup, in a fixed order; thread 0 has it.  The barriers
// make `lds` free again on return.
__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = lds[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) t += lds[w];
    __syncthreads();
    return t;
}

__device__ __forceinline__ double square_add(double acc, float x) {
    const double d = x;
    return __builtin_fma(d, d, acc);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ float element(const float* p) { return *p; }
__device__ __forceinline__ float element(const uint16_t* p) { return bf16_to_f32(*p); }

__device__ __forceinline__ void add_vector(u32x4_stream q, const float*, double acc[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = square_add(acc[k], __uint_as_float(q[k]));
}
__device__ __forceinline__ void add_vector(u32x4_stream q, const uint16_t*, double acc[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        acc[k] = square_add(acc[k], bf16_lo(q[k]));
        acc[k] = square_add(acc[k], bf16_hi(q[k]));
    }
}

// This thread's share of the sum of squares of p[begin, end): elements before
// the first and behind the last 16-byte boundary one by one, whole vectors
// between them.
template <typename T>
__device__ __forceinline__ double sum_squares(const T* __restrict__ p, int64_t begin, int64_t end) {
    constexpr int V = 16 / sizeof(T);
    const T* first = p + begin;
    const int64_t count = end - begin;
    int64_t head = int64_t((16 - (reinterpret_cast<uintptr_t>(first) & 15)) & 15) / int64_t(sizeof(T));
    if (head > count) head = count;
    const int64_t nvec = (count - head) / V;
    double acc[4] = {0., 0., 0., 0.};
    const u32x4_stream* v = reinterpret_cast<const u32x4_stream*>(first + head);
    int64_t i = threadIdx.x;
    for (; i + 3 * kThreads < nvec; i += 4 * kThreads) {
        u32x4_stream q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = __builtin_nontemporal_load(v + i + k * kThreads);
#pragma unroll
        for (int k = 0; k < 4; ++k) add_vector(q[k], p, acc);
    }
    for (; i < nvec; i += kThreads) add_vector(__builtin_nontemporal_load(v + i), p, acc);
    if (int64_t(threadIdx.x) < head) acc[0] = square_add(acc[0], element(first + threadIdx.x));
    const int64_t tail = head + nvec * V + threadIdx.x;
    if (tail < count) acc[1] = square_add(acc[1], element(first + tail));
    return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

// Workgroup w takes units [w span, (w + 1) span) and leaves its sum over
// tensor t in slot w + t.  Going from one (w, t) to the next raises w or t by
// one, or both where a workgroup ends with a tensor: that workgroup clears the
// slot between.
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const NormArgs a) {
    __shared__ double lds[kWaves];
    const int w = blockIdx.x;
    int u = w * a.span;
    const int u_end = min(u + a.span, a.units);
    int t = tensor_of(a.meta, a.n, u);
    while (u < u_end) {
        const uint64_t meta = a.meta[t];
        const int t_begin = meta_unit(meta);
        const int t_end = t + 1 < a.n ? meta_unit(a.meta[t + 1]) : a.units;
        const int stop = min(t_end, u_end);
        const int64_t numel = meta_numel(meta);
        const int64_t begin = int64_t(u - t_begin) * kClipUnit;
        const int64_t end = min(int64_t(stop - t_begin) * kClipUnit, numel);
        double s = 0.;
        if (begin < end) {
            if (meta_src(meta))
                s = sum_squares(static_cast<const uint16_t*>(a.data[t]), begin, end);
            else
                s = sum_squares(static_cast<const float*>(a.data[t]), begin, end);
        }
        s = block_sum(s, lds);
        if (threadIdx.x == 0) {
            a.partial[w + t] = s;
            if (stop == u_end && stop == t_end && t + 1 < a.n) a.partial[w + t + 1] = 0.;
        }
        u = stop;
        ++t;
    }
}

// norm and coefficient from the sum of squares, each rounded once from
// float64.  NaN stays NaN (min() would drop it).
__device__ __forceinline__ void finish(muon_clip_t* clip, double sumsq, float max_norm) {
    const double norm = sqrt(sumsq);
    const double c = double(max_norm) / (norm + 1e-6);
    clip->sumsq = sumsq;
    clip->norm = float(norm);
    clip->coef = c > 1. ? 1.f : float(c);
}

__global__ __launch_bounds__(kThreads) void norm_finish_kernel(const double* __restrict__ slots,
                                                               int count, float max_norm,
                                                               muon_clip_t* clip) {
    __shared__ double lds[kWaves];
    double s = 0.;
    for (int i = threadIdx.x; i < count; i += kThreads) s += slots[i];
    s = block_sum(s, lds);
    if (threadIdx.x == 0) finish(clip, s, max_norm);
}

// One wave sums the slots of one tensor.
__global__ __launch_bounds__(kThreads) void tensor_norms_kernel(const NormArgs a,
                                                                float* __restrict__ norms) {
    const int t = blockIdx.x * kWaves + (threadIdx.x >> 6);
    if (t >= a.n) return;
    const int first = meta_unit(a.meta[t]);
    const int last = (t + 1 < a.n ? meta_unit(a.meta[t + 1]) : a.units) - 1;
    const int lo = first / a.span + t, hi = last / a.span + t;
    double s = 0.;
    for (int i = lo + int(threadIdx.x & 63); i <= hi; i += 64) s += a.partial[i];
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
    if ((threadIdx.x & 63) == 0) norms[a.base + t] = float(sqrt(s));
}

__global__ void clip_finish_kernel(muon_clip_t* clip, float max_norm) {
    finish(clip, clip->sumsq, max_norm);
}

// ------------------------------------------------------------------- clipping

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = bf16_rne(v); }

template <int V>
__device__ __forceinline__ void load_v(const float* p, float v[V]) {
#pragma unroll
    for (int k = 0; k < V; k += 4) {
        const float4 q = load4_stream(p + k);
        v[k] = q.x, v[k + 1] = q.y, v[k + 2] = q.z, v[k + 3] = q.w;
    }
}
template <int V>
__device__ __forceinline__ void load_v(const uint16_t* p, float v[V]) {
    static_assert(V == 8, "16 bytes");
    const u32x4_stream q = __builtin_nontemporal_load(reinterpret_cast<const u32x4_stream*>(p));
#pragma unroll
    for (int k = 0; k < 4; ++k) v[2 * k] = bf16_lo(q[k]), v[2 * k + 1] = bf16_hi(q[k]);
}
template <int V>
__device__ __forceinline__ void store_v(float* p, const float v[V]) {
#pragma unroll
    for (int k = 0; k < V; k += 4) store4_stream(p + k, make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]));
}
template <int V>
__device__ __forceinline__ void store_v(uint16_t* p, const float v[V]) {
    static_assert(V == 8, "16 bytes");
    u32x4_stream q;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        q[k] = uint32_t(bf16_rne(v[2 * k])) | uint32_t(bf16_rne(v[2 * k + 1])) << 16;
    __builtin_nontemporal_store(q, reinterpret_cast<u32x4_stream*>(p));
}

// dst[i] = coef * src[i] for [begin, end).  Vectors of 16 bytes of the narrower
// type where source and destination come to their 16-byte boundaries at the same
// element, else one element after the other.  src may be dst.
template <typename TS, typename TD>
__device__ __forceinline__ void scale(const TS* src, TD* dst, int64_t begin, int64_t end,
                                      float coef) {
    constexpr int V = (sizeof(TS) == 2 || sizeof(TD) == 2) ? 8 : 4;
    const int64_t count = end - begin;
    src += begin, dst += begin;
    const int sp = int((16 - (reinterpret_cast<uintptr_t>(src) & 15)) & 15) / int(sizeof(TS));
    const int dp = int((16 - (reinterpret_cast<uintptr_t>(dst) & 15)) & 15) / int(sizeof(TD));
    // elements up to a boundary of both: the phase of the narrower type decides
    const int head0 = sizeof(TS) == 2 ? sp : dp;
    const bool together = sp % int(16 / sizeof(TS)) == head0 % int(16 / sizeof(TS)) &&
                          dp % int(16 / sizeof(TD)) == head0 % int(16 / sizeof(TD));
    const int64_t head = together ? min(int64_t(head0), count) : count;
    const int64_t nvec = (count - head) / V;
    for (int64_t i = threadIdx.x; i < nvec; i += kThreads) {
        float v[V];
        load_v<V>(src + head + i * V, v);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = coef * v[k];
        store_v<V>(dst + head + i * V, v);
    }
    for (int64_t i = threadIdx.x; i < head; i += kThreads) put(dst + i, coef * element(src + i));
    const int64_t tail = head + nvec * V + threadIdx.x;
    if (tail < count) put(dst + tail, coef * element(src + tail));
}

__global__ __launch_bounds__(kThreads) void clip_kernel(const ClipArgs a) {
    const float coef = a.clip->coef;
    for (int u = blockIdx.x; u < a.units; u += int(gridDim.x)) {
        const int t = tensor_of(a.meta, a.n, u);
        const uint64_t meta = a.meta[t];
        const void* src = a.src[t];
        void* dst = a.dst[t];
        // times 1 in place changes nothing
        if (src == dst && coef == 1.f) continue;
        const int64_t begin = int64_t(u - meta_unit(meta)) * kClipUnit;
        const int64_t end = min(begin + kClipUnit, meta_numel(meta));
        if (begin >= end) continue;
        if (meta_src(meta)) {
            if (meta_dst(meta))
                scale(static_cast<const uint16_t*>(src), static_cast<uint16_t*>(dst), begin, end, coef);
            else
                scale(static_cast<const uint16_t*>(src), static_cast<float*>(dst), begin, end, coef);
        } else {
            if (meta_dst(meta))
                scale(static_cast<const float*>(src), static_cast<uint16_t*>(dst), begin, end, coef);
            else
                scale(static_cast<const float*>(src), static_cast<float*>(dst), begin, end, coef);
        }
    }
}

// The launches of a tensor list: f(first tensor, count, units).
template <typename F>
void for_each_batch(const muon_tensor_t* t, int64_t n, int most, F f) {
    for (int64_t i = 0; i < n; i += most) {
        const int64_t m = std::min<int64_t>(most, n - i);
        int64_t units = 0;
        for (int64_t k = i; k < i + m; ++k) units += clip_units(t[k].numel);
        f(i, int(m), units);
    }
}

int span_of(int64_t units) { return int((units + kNormGroups - 1) / kNormGroups); }
int groups_of(int64_t units) {
    const int span = span_of(units);
    return int((units + span - 1) / span);
}

}  // namespace

int64_t norm_slots(const muon_tensor_t* t, int64_t n) {
    int64_t slots = 0;
    for_each_batch(t, n, kNormTensors,
                   [&](int64_t, int m, int64_t units) { slots += groups_of(units) + m - 1; });
    return slots;
}

hipError_t launch_grad_norm(const muon_tensor_t* t, int64_t n, float max_norm, muon_clip_t* clip,
                            float* tensor_norms, double* slots, hipStream_t s) {
    hipError_t err = hipSuccess;
    int64_t at = 0;
    for_each_batch(t, n, kNormTensors, [&](int64_t i, int m, int64_t units) {
        if (err != hipSuccess) return;
        NormArgs a;
        int64_t u = 0;
        for (int k = 0; k < m; ++k) {
            a.data[k] = t[i + k].data;
            a.meta[k] = clip_meta(t[i + k].numel, t[i + k].dtype == MUON_DTYPE_BF16, 0, u);
            u += clip_units(t[i + k].numel);
        }
        a.partial = slots + at;
        a.n = m, a.units = int32_t(units), a.span = span_of(units), a.base = int32_t(i);
        const int groups = groups_of(units);
        {
            LaunchTimer timer("grad_norm", s);
            grad_norm_kernel<<<dim3(unsigned(groups)), dim3(kThreads), 0, s>>>(a);
        }
        if ((err = hipGetLastError()) != hipSuccess) return;
        if (tensor_norms != nullptr) {
            LaunchTimer timer("tensor_norms", s);
            tensor_norms_kernel<<<dim3(unsigned((m + kWaves - 1) / kWaves)), dim3(kThreads), 0, s>>>(
                a, tensor_norms);
            err = hipGetLastError();
        }
        at += groups + m - 1;
    });
    if (err != hipSuccess) return err;
    LaunchTimer timer("norm_finish", s);
    norm_finish_kernel<<<dim3(1), dim3(kThreads), 0, s>>>(slots, int(at), max_norm, clip);
    return hipGetLastError();
}

hipError_t launch_clip_finish(muon_clip_t* clip, float max_norm, hipStream_t s) {
    LaunchTimer timer("clip_finish", s);
    clip_finish_kernel<<<dim3(1), dim3(1), 0, s>>>(clip, max_norm);
    return hipGetLastError();
}

hipError_t launch_clip(const muon_tensor_t* src, const muon_tensor_t* dst, int64_t n,
                       const muon_clip_t* clip, hipStream_t s) {
    hipError_t err = hipSuccess;
    for_each_batch(src, n, kClipTensors, [&](int64_t i, int m, int64_t units) {
        if (err != hipSuccess) return;
        ClipArgs a;
        int64_t u = 0;
        for (int k = 0; k < m; ++k) {
            a.src[k] = src[i + k].data;
            a.dst[k] = dst[i + k].data;
            a.meta[k] = clip_meta(src[i + k].numel, src[i + k].dtype == MUON_DTYPE_BF16,
                                  dst[i + k].dtype == MUON_DTYPE_BF16, u);
            u += clip_units(src[i + k].numel);
        }
        a.clip = clip, a.n = m, a.units = int32_t(units);
        const int64_t grid = std::min<int64_t>(units, int64_t(1) << 23);
        LaunchTimer timer("clip", s);
        clip_kernel<<<dim3(unsigned(grid)), dim3(kThreads), 0, s>>>(a);
        err = hipGetLastError();
    });
    return err;
}

}  // namespace muon
