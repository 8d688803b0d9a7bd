// AdamW on gfx950: the optimizer of the parameters that the Muon step does not
// take (embeddings, output heads, norm weights, biases), on the same flat
// buffers, with the clipping coefficient applied to the gradient as it is read.
//
//   g' = fl(coef g)                         (g itself without a clip record)
//   m  = fl(fl(b1 m) + fl((1 - b1) g'))
//   v  = fl(fl(b2 v) + fl(fl((1 - b2) g') g'))
//   w1 = fl(w f),  f = fl(1 - fl(lr wd))
//   w  = fl(w1 - fl(a fl(m / fl(fl(sqrt(v) r) + eps))))
//   a  = fl(lr / (1 - b1^t)),  r = fl(1 / sqrt(1 - b2^t))
//
// float32 throughout, each operation rounded on its own; a and r come from
// float64 (1 - b2^t loses all its digits in float32 while t is small).  It is an
// HBM stream of 22 to 30 bytes per element.
#include "clip_internal.h"
#include "k_common.h"

#pragma clang fp contract(off)

namespace muon {

namespace {

// One wave per workgroup, one vector of every stream per thread.  Seven or
// eight streams are open at once; the fewer bytes of each are in flight, the
// better HBM keeps up (of 64 to 512 threads and 1 to 4 vectors).  float32
// weights with a bfloat16 copy, 1.05 G elements: 64 threads x 1 vector 5.93
// TB/s, 128 x 1 5.70, 256 x 1 5.75, 256 x 2 5.30; plain instead of nontemporal
// loads or stores cost 4 to 11% more time.
constexpr int kThreads = 64;
constexpr int kVec = 4;
constexpr int kIters = int(kAdamwUnit / (kThreads * kVec));
static_assert(kAdamwUnit <= 256, "the missing elements fit 8 bits");
static_assert(kAdamwUnit == kIters * kThreads * kVec, "whole passes of a workgroup");

// b^t by repeated squaring.  t = 0 gives 1 (and with it an infinite step
// size: steps count from 1).
__device__ __forceinline__ double power(double b, uint64_t t) {
    double p = 1.;
    for (; t != 0; t >>= 1) {
        if (t & 1) p *= b;
        b *= b;
    }
    return p;
}

struct Step {
    float coef, b1, c1, b2, c2, decay, a, r, eps;
};
__device__ __forceinline__ Step step_of(const muon_adamw_group_t& g, const muon_clip_t* clip) {
    Step s;
    s.coef = clip != nullptr ? clip->coef : 1.f;
    s.b1 = g.beta1, s.c1 = 1.f - g.beta1;
    s.b2 = g.beta2, s.c2 = 1.f - g.beta2;
    const float lrwd = g.lr * g.weight_decay;
    s.decay = 1.f - lrwd;
    s.a = float(double(g.lr) / (1. - power(double(g.beta1), uint64_t(g.step))));
    s.r = float(1. / sqrt(1. - power(double(g.beta2), uint64_t(g.step))));
    s.eps = g.eps;
    return s;
}

__device__ __forceinline__ void update(const Step& s, float g, float& m, float& v, float& w) {
    const float gc = s.coef * g;
    m = s.b1 * m + s.c1 * gc;
    v = s.b2 * v + (s.c2 * gc) * gc;
    const float d = sqrtf(v) * s.r + s.eps;
    const float q = m / d;
    w = w * s.decay - s.a * q;
}

__device__ __forceinline__ float4 load4(const float* p) { return load4_stream(p); }
__device__ __forceinline__ float4 load4(const uint16_t* p) {
    const uint2 b = load2_stream(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u),
                       __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { store4_stream(p, v); }
__device__ __forceinline__ void store4(uint16_t* p, float4 v) {
    store2_stream(reinterpret_cast<uint2*>(p),
                  make_uint2(uint32_t(bf16_rne(v.x)) | uint32_t(bf16_rne(v.y)) << 16,
                             uint32_t(bf16_rne(v.z)) | uint32_t(bf16_rne(v.w)) << 16));
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = bf16_rne(v); }

constexpr uint64_t kOffsetBits = (uint64_t(1) << 34) - 1;
__device__ __forceinline__ int unit_begin(const AdamwRange& r) { return int(r.to >> 34); }

// Unit of workgroup b.  Workgroups go to the 8 XCDs in turn; each XCD gets runs
// of kRun consecutive units (64 Ki elements), so that it walks through pages of
// its own instead of sharing every page with the seven others: 6.15 against 5.98
// TB/s in the geometric mean over seven sets of 131 M to 1.05 G elements (runs of
// 32 to 384 units: 5.70 to 6.09).  What is left behind the last whole round, and
// with it any small set, goes in plain order.
constexpr int kXcds = 8, kRun = 256;
__device__ __forceinline__ int unit_of(int b, int units) {
    const int whole = units / (kXcds * kRun) * (kXcds * kRun);
    if (b >= whole) return b;
    const int q = b / kXcds;
    return q / kRun * (kXcds * kRun) + b % kXcds * kRun + q % kRun;
}

template <typename TW, typename TG>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const AdamwArgs a) {
    for (int b = blockIdx.x; b < a.units; b += int(gridDim.x)) {
        const int u = unit_of(b, a.units);
        int lo = 0, hi = a.n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (unit_begin(a.range[mid]) <= u)
                lo = mid;
            else
                hi = mid - 1;
        }
        const AdamwRange range = a.range[lo];
        const int next = lo + 1 < a.n ? unit_begin(a.range[lo + 1]) : a.units;
        const int64_t numel = int64_t(next - unit_begin(range)) * kAdamwUnit -
                              int64_t((range.at >> 50) & 255);
        const int64_t base = int64_t(u - unit_begin(range)) * kAdamwUnit;
        const int64_t off = int64_t(range.at & kOffsetBits) * 4;
        const int64_t poff = int64_t(range.to & kOffsetBits) * 4;
        const int group = int(range.at >> 34) & 0xffff;
        const TG* g = static_cast<const TG*>(a.grads) + off;
        float* m = a.m + off;
        float* v = a.v + off;
        TW* w = static_cast<TW*>(a.params) + poff;
        uint16_t* copy = a.copy != nullptr ? a.copy + poff : nullptr;
        if (base + kAdamwUnit <= numel) {
            // whole unit: every load goes out before the first wait; the step's scalars
            // (some hundred cycles of float64) are worked out while they are on their way
            float4 g4[kIters], m4[kIters], v4[kIters], w4[kIters];
#pragma unroll
            for (int it = 0; it < kIters; ++it) {
                const int64_t e = base + (int64_t(it) * kThreads + threadIdx.x) * kVec;
                g4[it] = load4(g + e);
                m4[it] = load4(m + e);
                v4[it] = load4(v + e);
                w4[it] = load4(w + e);
            }
            const Step s = step_of(a.groups[group], a.clip);
#pragma unroll
            for (int it = 0; it < kIters; ++it) {
                const int64_t e = base + (int64_t(it) * kThreads + threadIdx.x) * kVec;
                update(s, g4[it].x, m4[it].x, v4[it].x, w4[it].x);
                update(s, g4[it].y, m4[it].y, v4[it].y, w4[it].y);
                update(s, g4[it].z, m4[it].z, v4[it].z, w4[it].z);
                update(s, g4[it].w, m4[it].w, v4[it].w, w4[it].w);
                store4(m + e, m4[it]);
                store4(v + e, v4[it]);
                store4(w + e, w4[it]);
                if (copy != nullptr) store4(copy + e, w4[it]);
            }
        } else {
            const Step s = step_of(a.groups[group], a.clip);
            for (int64_t k = base + threadIdx.x; k < numel; k += kThreads) {
                float m1 = m[k], v1 = v[k], w1 = load1(w + k);
                update(s, load1(g + k), m1, v1, w1);
                m[k] = m1;
                v[k] = v1;
                store1(w + k, w1);
                if (copy != nullptr) store1(copy + k, w1);
            }
        }
    }
}

// A grid counts at most 2^32 - 1 work-items; longer sets loop.
constexpr int64_t kMaxGrid = int64_t(1) << 25;
static_assert(kMaxGrid * kThreads < (int64_t(1) << 32), "grid");

template <typename TW, typename TG>
hipError_t enqueue(const AdamwArgs& a, hipStream_t s) {
    const int64_t grid = std::min<int64_t>(a.units, kMaxGrid);
    LaunchTimer timer("adamw", s);
    adamw_kernel<TW, TG><<<dim3(unsigned(grid)), dim3(kThreads), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_adamw(void* params, int param_dtype, void* model_copy, const void* grads,
                        int grad_dtype, float* exp_avg, float* exp_avg_sq,
                        const muon_range_t* ranges, int64_t n, const muon_adamw_group_t* groups,
                        const muon_clip_t* clip, hipStream_t s) {
    AdamwArgs a;
    a.params = params, a.copy = static_cast<uint16_t*>(model_copy), a.grads = grads;
    a.m = exp_avg, a.v = exp_avg_sq, a.groups = groups, a.clip = clip;
    for (int64_t i = 0; i < n;) {
        int64_t units = 0;
        int m = 0;
        while (i < n && m < kAdamwRanges) {
            muon_range_t q = ranges[i++];
            if (q.numel == 0) continue;
            // a run of ranges of one group, adjacent in the state and in params, is one
            for (; i < n && ranges[i].group == q.group && ranges[i].offset == q.offset + q.numel &&
                   ranges[i].param_offset == q.param_offset + q.numel &&
                   q.numel + ranges[i].numel <= kMaxNumel;
                 ++i)
                q.numel += ranges[i].numel;
            const int64_t mine = (q.numel + kAdamwUnit - 1) / kAdamwUnit;
            a.range[m].at = uint64_t(q.offset / 4) | uint64_t(q.group) << 34 |
                            uint64_t(mine * kAdamwUnit - q.numel) << 50;
            a.range[m].to = uint64_t(q.param_offset / 4) | uint64_t(units) << 34;
            units += mine;
            ++m;
        }
        if (m == 0) break;
        a.n = m, a.units = int32_t(units);
        hipError_t e;
        if (param_dtype == MUON_DTYPE_BF16)
            e = grad_dtype == MUON_DTYPE_BF16 ? enqueue<uint16_t, uint16_t>(a, s)
                                              : enqueue<uint16_t, float>(a, s);
        else
            e = grad_dtype == MUON_DTYPE_BF16 ? enqueue<float, uint16_t>(a, s)
                                              : enqueue<float, float>(a, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace muon
