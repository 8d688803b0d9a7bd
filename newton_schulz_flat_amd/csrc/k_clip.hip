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

// The norm: 1024 workgroups of 256 threads, 8 vectors of 16 bytes in flight per
// thread.  7 G float32 elements 3.98 ms (7.0 TB/s), 218 M bfloat16 65 us (6.7).  Of 512 to
// 16384 workgroups, 128 to 1024 threads and 2 to 8 vectors the ones near this lie
// within 1%; half the vectors with double the workgroups 1.5% more, 2 vectors
// 5% more, 8192 workgroups (more partials, less of each tensor) 3% more.  Plain
// instead of nontemporal loads: 6.2 TB/s.
constexpr int kThreads = 256;
constexpr int kFlight = 8;
constexpr int kWaves = kThreads / 64;
// One workgroup of this size reads up to kSoloUnits units of kSoloUnit elements by
// itself and saves the second launch.  A tensor takes a unit at least, a run of
// adjacent tensors counts as one.  Time of a call among others, alone in brackets, one
// workgroup against two launches, float32: 1000 elements 5.4 (16.1) against 8.1 us
// (20.1); one run of 64 Ki 5.4 (17.6) against 8.0 (18.6), of 96 Ki, the longest taken,
// 6.6 (18.7) against 8.0 (19.3), of 128 Ki 8.0 (20.1) against 8.0 (18.6).  Tensors
// that lie apart are dearer: 40 of 100 elements 6.3 (18.5) against 8.2 (19.4), 48 of 1024
// 8.1 (20.4) against 8.2 (19.1), 48 of 2048 9.4 (21.6) against 8.2 (19.3), 64 of 1024
// 10.2 (22.4) against 8.3 (19.4).  So the limit, one number of units for both, suits runs
// well and is at or past the crossing for its 48 separate tensors.
// Units of 512 or 1024 elements: 9.5 and 6.4 us at 64 Ki.
constexpr int kFinishThreads = 1024;
constexpr int kSoloThreads = 1024;
constexpr int64_t kSoloUnit = 2048;
constexpr int kSoloUnits = 48;
// Clipping: 128 threads, 2 vectors of 4 elements in flight per thread.  2.1 G float32
// elements into another buffer 2.75 ms (6.2 TB/s); 64 threads x 2 3.38 ms, 128 x 4
// 3.00, 256 x 2 2.84.
constexpr int kScaleThreads = 128;

typedef uint32_t u32x4_stream __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int64_t meta_numel(uint64_t m) { return int64_t(m & ((uint64_t(1) << 35) - 1)); }
__host__ __device__ __forceinline__ int meta_src(uint64_t m) { return int(m >> 35) & 1; }
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

// Sum over the workgroup, in a fixed order, for every thread.  The barriers make
// `lds` free again on return.
template <int kCount>
__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = lds[0];
#pragma unroll
    for (int w = 1; w < kCount; ++w) t += lds[w];
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

template <bool kStream>
__device__ __forceinline__ u32x4_stream load_vector(const u32x4_stream* v) {
    if constexpr (kStream) return __builtin_nontemporal_load(v);
    return *v;
}

// Share of thread `me` of kStep in the sum of squares of p[begin, end): elements
// before the first and behind the last 16-byte boundary one by one, whole
// vectors between them.
template <int kStep, int kLoads, bool kStream, typename T>
__device__ __forceinline__ double sum_squares(const T* __restrict__ p, int64_t begin, int64_t end,
                                              int me) {
    constexpr int V = 16 / sizeof(T);
    const T* first = p + begin;
    const int64_t count = end - begin;
    int64_t head = int64_t((16 - (reinterpret_cast<uintptr_t>(first) & 15)) & 15) / int64_t(sizeof(T));
    if (head > count) head = count;
    const int64_t nvec = (count - head) / V;
    double acc[4] = {0., 0., 0., 0.};
    const u32x4_stream* v = reinterpret_cast<const u32x4_stream*>(first + head);
    int64_t i = me;
    for (; i + (kLoads - 1) * kStep < nvec; i += kLoads * kStep) {
        u32x4_stream q[kLoads];
#pragma unroll
        for (int k = 0; k < kLoads; ++k) q[k] = load_vector<kStream>(v + i + k * kStep);
#pragma unroll
        for (int k = 0; k < kLoads; ++k) add_vector(q[k], p, acc);
    }
    for (; i < nvec; i += kStep) add_vector(load_vector<kStream>(v + i), p, acc);
    if (me < head) acc[0] = square_add(acc[0], element(first + me));
    const int64_t tail = head + nvec * V + me;
    if (tail < count) acc[1] = square_add(acc[1], element(first + tail));
    return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

// Workgroup w takes units [w span, (w + 1) span) and leaves its sum over
// tensor t in slot w + t.  Going from one (w, t) to the next raises w or t by
// one, or both where a workgroup ends with a tensor: that workgroup clears the
// slot between.
template <bool kStream>
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
        const int64_t begin = int64_t(u - t_begin) * kNormUnit;
        const int64_t end = min(int64_t(stop - t_begin) * kNormUnit, numel);
        double s = 0.;
        if (begin < end) {
            if (meta_src(meta))
                s = sum_squares<kThreads, kFlight, kStream>(
                    static_cast<const uint16_t*>(a.data[t]), begin, end, threadIdx.x);
            else
                s = sum_squares<kThreads, kFlight, kStream>(static_cast<const float*>(a.data[t]),
                                                            begin, end, threadIdx.x);
        }
        s = block_sum<kWaves>(s, lds);
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

// The record from all partials.  One workgroup as wide as they come, so that
// each thread waits for one load (two launches' worth of partials: for two).
__device__ __forceinline__ void finish_all(const double* __restrict__ slots, int count,
                                           float max_norm, muon_clip_t* clip, double* lds) {
    double s = 0.;
    for (int i = threadIdx.x; i < count; i += kFinishThreads) s += slots[i];
    s = block_sum<kFinishThreads / 64>(s, lds);
    if (threadIdx.x == 0) finish(clip, s, max_norm);
}

__global__ __launch_bounds__(kFinishThreads) void norm_finish_kernel(
    const double* __restrict__ slots, int count, float max_norm, muon_clip_t* clip) {
    __shared__ double lds[kFinishThreads / 64];
    finish_all(slots, count, max_norm, clip, lds);
}

// The norms of a launch's tensors, one wave for each, and, from the list's last
// launch (clip not null), the record by workgroup 0.
__global__ __launch_bounds__(kFinishThreads) void tensor_norms_kernel(
    const NormArgs a, float* __restrict__ norms, const double* __restrict__ slots, int count,
    float max_norm, muon_clip_t* clip) {
    __shared__ double lds[kFinishThreads / 64];
    if (blockIdx.x == 0) {
        if (clip != nullptr) finish_all(slots, count, max_norm, clip, lds);
        return;
    }
    const int t = (int(blockIdx.x) - 1) * (kFinishThreads / 64) + int(threadIdx.x >> 6);
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

// Short lists, in one launch: the waves of one workgroup take units of kSoloUnit
// elements in turn, and the workgroup ends with the record.
__global__ __launch_bounds__(kSoloThreads) void norm_solo_kernel(const NormArgs a, float max_norm,
                                                                 muon_clip_t* clip) {
    constexpr int kSoloWaves = kSoloThreads / 64;
    __shared__ double lds[kSoloWaves];
    double s = 0.;
    for (int u = int(threadIdx.x) / 64; u < a.units; u += kSoloWaves) {
        const int t = tensor_of(a.meta, a.n, u);
        const uint64_t meta = a.meta[t];
        const int64_t begin = int64_t(u - meta_unit(meta)) * kSoloUnit;
        const int64_t end = min(begin + kSoloUnit, meta_numel(meta));
        if (begin >= end) continue;
        if (meta_src(meta))
            s += sum_squares<64, 2, false>(static_cast<const uint16_t*>(a.data[t]), begin, end,
                                           threadIdx.x & 63);
        else
            s += sum_squares<64, 4, false>(static_cast<const float*>(a.data[t]), begin, end,
                                           threadIdx.x & 63);
    }
    s = block_sum<kSoloWaves>(s, lds);
    if (threadIdx.x == 0) finish(clip, s, max_norm);
}

__global__ void clip_finish_kernel(muon_clip_t* clip, float max_norm) {
    finish(clip, clip->sumsq, max_norm);
}

// ------------------------------------------------------------------- clipping

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = bf16_rne(v); }

// V consecutive elements, aligned to V elements.
template <int V, bool kStream>
__device__ __forceinline__ void load_v(const float* p, float v[V]) {
    static_assert(V == 4, "16 bytes");
    const u32x4_stream q = load_vector<kStream>(reinterpret_cast<const u32x4_stream*>(p));
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __uint_as_float(q[k]);
}
template <int V, bool kStream>
__device__ __forceinline__ void load_v(const uint16_t* p, float v[V]) {
    if constexpr (V == 8) {
        const u32x4_stream q = load_vector<kStream>(reinterpret_cast<const u32x4_stream*>(p));
#pragma unroll
        for (int k = 0; k < 4; ++k) v[2 * k] = bf16_lo(q[k]), v[2 * k + 1] = bf16_hi(q[k]);
    } else {
        const uint2* at = reinterpret_cast<const uint2*>(p);
        const uint2 q = kStream ? load2_stream(at) : *at;
        v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
    }
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    return uint32_t(bf16_rne(lo)) | uint32_t(bf16_rne(hi)) << 16;
}
template <int V>
__device__ __forceinline__ void store_v(float* p, const float v[V]) {
    static_assert(V == 4, "16 bytes");
    store4_stream(p, make_float4(v[0], v[1], v[2], v[3]));
}
template <int V>
__device__ __forceinline__ void store_v(uint16_t* p, const float v[V]) {
    if constexpr (V == 8) {
        u32x4_stream q;
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = bf16_pair(v[2 * k], v[2 * k + 1]);
        __builtin_nontemporal_store(q, reinterpret_cast<u32x4_stream*>(p));
    } else {
        store2_stream(reinterpret_cast<uint2*>(p),
                      make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])));
    }
}

// Unit k of dst = coef * src.  Where source and destination come to their vector
// boundaries at the same element (`head` elements in), units are whole vectors
// counted from there, unit 0 takes the head as well and the last one the tail;
// elsewhere they are plain runs of elements.  src may be dst.
//
// Vectors against single elements, 218 M of them in TB/s: float32 to float32 6.3 against
// 4.7, bfloat16 to float32 6.3 and 3.2, float32 to bfloat16 6.6 and 3.9, bfloat16 to
// bfloat16 6.0 and 2.6.
//
// A thread's vector is 4 elements (8 where both sides are bfloat16), so that
// neighbouring lanes meet without a gap on the wider side too: 8 bfloat16 read
// and two times 16 bytes of float32 stored by each lane took 1.6 times as long.
template <bool kStream, typename TS, typename TD>
__device__ __forceinline__ void scale_unit(const TS* src, TD* dst, int64_t numel, int64_t k,
                                           float coef) {
    constexpr int V = (sizeof(TS) == 2 && sizeof(TD) == 2) ? 8 : 4;
    constexpr int kIters = int(kScaleUnit / (kScaleThreads * V));
    static_assert(kScaleUnit == kIters * kScaleThreads * V, "whole passes of a workgroup");
    const int head = int(-(reinterpret_cast<uintptr_t>(src) / sizeof(TS)) & (V - 1));
    const bool together = head == int(-(reinterpret_cast<uintptr_t>(dst) / sizeof(TD)) & (V - 1));
    const int64_t begin = k * kScaleUnit + (together ? head : 0);
    if (together && begin + kScaleUnit <= numel) {
        float v[kIters][V];
#pragma unroll
        for (int it = 0; it < kIters; ++it)
            load_v<V, kStream>(src + begin + (it * kScaleThreads + int(threadIdx.x)) * V, v[it]);
#pragma unroll
        for (int it = 0; it < kIters; ++it) {
#pragma unroll
            for (int j = 0; j < V; ++j) v[it][j] = coef * v[it][j];
            store_v<V>(dst + begin + (it * kScaleThreads + int(threadIdx.x)) * V, v[it]);
        }
    } else {
        const int64_t end = min(begin + kScaleUnit, numel);
        for (int64_t i = begin + threadIdx.x; i < end; i += kScaleThreads)
            put(dst + i, coef * element(src + i));
    }
    if (k == 0 && together && int(threadIdx.x) < head && int64_t(threadIdx.x) < numel)
        put(dst + threadIdx.x, coef * element(src + threadIdx.x));
}

template <bool kStream>
__global__ __launch_bounds__(kScaleThreads) void clip_kernel(const ClipArgs a) {
    const float coef = a.clip->coef;
    // times 1 in place changes nothing
    if (a.in_place && coef == 1.f) return;
    for (int b = blockIdx.x; b < a.units; b += int(gridDim.x)) {
        const int t = tensor_of(a.meta, a.n, b);
        const uint64_t meta = a.meta[t];
        const void* src = a.src[t];
        void* dst = a.dst[t];
        const int64_t numel = meta_numel(meta), k = b - meta_unit(meta);
        const float* sf = static_cast<const float*>(src);
        const uint16_t* sb = static_cast<const uint16_t*>(src);
        float* df = static_cast<float*>(dst);
        uint16_t* db = static_cast<uint16_t*>(dst);
        if (meta_src(meta)) {
            if (meta_dst(meta))
                scale_unit<kStream>(sb, db, numel, k, coef);
            else
                scale_unit<kStream>(sb, df, numel, k, coef);
        } else {
            if (meta_dst(meta))
                scale_unit<kStream>(sf, db, numel, k, coef);
            else
                scale_unit<kStream>(sf, df, numel, k, coef);
        }
    }
}

// A grid counts at most 2^32 - 1 work-items; longer lists loop.
constexpr int64_t kMaxGrid = int64_t(1) << 24;
static_assert(kMaxGrid * kScaleThreads < (int64_t(1) << 32), "grid");

int span_of(int64_t units) { return int((units + kNormGroups - 1) / kNormGroups); }
int groups_of(int64_t units) {
    const int span = span_of(units);
    return int((units + span - 1) / span);
}

size_t type_bytes(int dtype) { return dtype == MUON_DTYPE_BF16 ? 2 : 4; }

// Whether y begins where x ends, so that one entry can stand for both.
bool adjacent(const muon_tensor_t& x, const muon_tensor_t& y) {
    return x.dtype == y.dtype && x.numel + y.numel <= kMaxNumel &&
           static_cast<const char*>(x.data) + size_t(x.numel) * type_bytes(x.dtype) == y.data;
}

// Lists up to this size are read with plain loads, which leave them in the
// cache behind HBM for the pass that follows the norm; longer ones, which it
// could not hold for long, with nontemporal ones.  Norm and clipping of float32
// into another buffer, plain against nontemporal: 32 MiB 20.8 against 23.1 us, 64 MiB
// 34.4 against 38.5 (the norm alone 14.3 against 14.8); at 96 MiB clipping still
// gains 7%, but the norm alone loses 4%, and 14% at 128 MiB.
constexpr size_t kKeepBytes = size_t(64) << 20;
bool keep_cached(const muon_tensor_t* t, int64_t n) {
    size_t bytes = 0;
    for (int64_t i = 0; i < n; ++i) bytes += size_t(t[i].numel) * type_bytes(t[i].dtype);
    return bytes <= kKeepBytes;
}

}  // namespace

int64_t norm_slots(const muon_tensor_t* t, int64_t n) {
    int64_t units = 0;
    for (int64_t i = 0; i < n; ++i) units += units_of(t[i].numel, kNormUnit);
    return (n + kNormTensors - 1) / kNormTensors * std::min<int64_t>(units, kNormGroups) + n;
}

hipError_t launch_grad_norm(const muon_tensor_t* t, int64_t n, float max_norm, muon_clip_t* clip,
                            float* tensor_norms, double* slots, hipStream_t s) {
    const bool keep = keep_cached(t, n);
    int64_t at = 0;
    for (int64_t i = 0; i < n;) {
        NormArgs a;
        a.base = int32_t(i);
        int m = 0;
        int64_t numel[kNormTensors];
        int64_t units = 0, solo_units = 0;
        while (i < n && m < kNormTensors) {
            // a run of adjacent tensors is one, unless each one's norm is asked for
            muon_tensor_t x = t[i++];
            while (tensor_norms == nullptr && i < n && adjacent(x, t[i])) x.numel += t[i++].numel;
            a.data[m] = x.data;
            a.meta[m] = clip_meta(x.numel, x.dtype == MUON_DTYPE_BF16, 0, units);
            numel[m] = x.numel;
            units += units_of(x.numel, kNormUnit);
            solo_units += units_of(x.numel, kSoloUnit);
            ++m;
        }
        a.partial = slots + at;
        a.n = m;
        if (a.base == 0 && i == n && tensor_norms == nullptr && solo_units <= kSoloUnits) {
            a.units = int32_t(solo_units);
            solo_units = 0;
            for (int k = 0; k < m; ++k) {
                a.meta[k] = clip_meta(numel[k], meta_src(a.meta[k]), 0, solo_units);
                solo_units += units_of(numel[k], kSoloUnit);
            }
            LaunchTimer timer("norm_solo", s);
            norm_solo_kernel<<<dim3(1), dim3(kSoloThreads), 0, s>>>(a, max_norm, clip);
            return hipGetLastError();
        }
        a.units = int32_t(units), a.span = span_of(units);
        const int groups = groups_of(units);
        {
            LaunchTimer timer("grad_norm", s);
            const auto kernel = keep ? grad_norm_kernel<false> : grad_norm_kernel<true>;
            kernel<<<dim3(unsigned(groups)), dim3(kThreads), 0, s>>>(a);
        }
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        at += groups + m - 1;
        if (tensor_norms != nullptr) {
            constexpr int kTensors = kFinishThreads / 64;  // of one workgroup
            LaunchTimer timer("tensor_norms", s);
            tensor_norms_kernel<<<dim3(unsigned(1 + (m + kTensors - 1) / kTensors)),
                                  dim3(kFinishThreads), 0, s>>>(a, tensor_norms, slots, int(at),
                                                                max_norm, i == n ? clip : nullptr);
            if ((e = hipGetLastError()) != hipSuccess || i == n) return e;
        }
    }
    LaunchTimer timer("norm_finish", s);
    norm_finish_kernel<<<dim3(1), dim3(kFinishThreads), 0, s>>>(slots, int(at), max_norm, clip);
    return hipGetLastError();
}

hipError_t launch_clip_finish(muon_clip_t* clip, float max_norm, hipStream_t s) {
    LaunchTimer timer("clip_finish", s);
    clip_finish_kernel<<<dim3(1), dim3(1), 0, s>>>(clip, max_norm);
    return hipGetLastError();
}

hipError_t launch_clip(const muon_tensor_t* src, const muon_tensor_t* dst, int64_t n,
                       const muon_clip_t* clip, hipStream_t s) {
    const bool keep = keep_cached(src, n);
    for (int64_t i = 0; i < n;) {
        ClipArgs a;
        int64_t units = 0;
        int m = 0;
        int32_t in_place = 1;
        while (i < n && m < kClipTensors) {
            // a run of tensors adjacent on both sides is one
            muon_tensor_t x = src[i], y = dst[i];
            ++i;
            while (i < n && adjacent(x, src[i]) && adjacent(y, dst[i])) {
                x.numel += src[i].numel;
                y.numel = x.numel;
                ++i;
            }
            if (x.numel > 0 && x.data != y.data) in_place = 0;
            a.src[m] = x.data;
            a.dst[m] = y.data;
            a.meta[m] = clip_meta(x.numel, x.dtype == MUON_DTYPE_BF16, y.dtype == MUON_DTYPE_BF16,
                                  units);
            units += units_of(x.numel, kScaleUnit);
            ++m;
        }
        a.clip = clip, a.n = m, a.units = int32_t(units), a.in_place = in_place;
        const int64_t grid = std::min<int64_t>(units, kMaxGrid);
        LaunchTimer timer("clip", s);
        const auto kernel = keep ? clip_kernel<false> : clip_kernel<true>;
        kernel<<<dim3(unsigned(grid)), dim3(kScaleThreads), 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace muon
