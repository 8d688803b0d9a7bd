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

constexpr int kThreads = 256;
constexpr int kVec = 4;
static_assert(kAdamwUnit % (kThreads * kVec) == 0, "whole passes of a workgroup");

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

__device__ __forceinline__ int unit_begin(uint64_t meta) { return int(meta >> 36); }
__device__ __forceinline__ int64_t meta_numel(uint64_t meta) {
    return int64_t(meta & ((uint64_t(1) << 36) - 1));
}

template <typename TW, typename TG>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const AdamwArgs a) {
    for (int u = blockIdx.x; u < a.units; u += int(gridDim.x)) {
        int lo = 0, hi = a.n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (unit_begin(a.meta[mid]) <= u)
                lo = mid;
            else
                hi = mid - 1;
        }
        const Step s = step_of(a.groups[a.group[lo]], a.clip);
        const uint64_t meta = a.meta[lo];
        const int64_t numel = meta_numel(meta);
        const int64_t base = int64_t(u - unit_begin(meta)) * kAdamwUnit;
        const TG* g = static_cast<const TG*>(a.grads) + a.off[lo];
        float* m = a.m + a.off[lo];
        float* v = a.v + a.off[lo];
        TW* w = static_cast<TW*>(a.params) + a.poff[lo];
        uint16_t* copy = a.copy != nullptr ? a.copy + a.poff[lo] : nullptr;
#pragma unroll
        for (int it = 0; it < int(kAdamwUnit / (kThreads * kVec)); ++it) {
            const int64_t e = base + (int64_t(it) * kThreads + threadIdx.x) * kVec;
            if (e + kVec <= numel) {
                const float4 g4 = load4(g + e);
                float4 m4 = load4(m + e), v4 = load4(v + e), w4 = load4(w + e);
                update(s, g4.x, m4.x, v4.x, w4.x);
                update(s, g4.y, m4.y, v4.y, w4.y);
                update(s, g4.z, m4.z, v4.z, w4.z);
                update(s, g4.w, m4.w, v4.w, w4.w);
                store4(m + e, m4);
                store4(v + e, v4);
                store4(w + e, w4);
                if (copy != nullptr) store4(copy + e, w4);
            } else {
                for (int64_t k = e; k < numel && k < e + kVec; ++k) {
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
}

template <typename TW, typename TG>
hipError_t enqueue(const AdamwArgs& a, hipStream_t s) {
    const int64_t grid = std::min<int64_t>(a.units, int64_t(1) << 23);
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
    int64_t i = 0;
    while (i < n) {
        int64_t units = 0;
        int m = 0;
        for (; i < n && m < kAdamwRanges; ++i) {
            const int64_t numel = ranges[i].numel;
            if (numel == 0) continue;
            a.off[m] = ranges[i].offset;
            a.poff[m] = ranges[i].param_offset;
            a.meta[m] = uint64_t(numel) | uint64_t(units) << 36;
            a.group[m] = uint16_t(ranges[i].group);
            units += (numel + kAdamwUnit - 1) / kAdamwUnit;
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
