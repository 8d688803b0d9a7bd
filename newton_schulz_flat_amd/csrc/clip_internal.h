// Internal declarations of the gradient norm, clipping and AdamW: the tables
// that a launch carries in its kernel arguments, and the launchers.
//
// These operators keep no plan: what a kernel has to know about its tensors
// (address, length, type) is passed by value, so that a first call costs what
// every call costs, nothing is cached by address, and a call can be captured
// into a HIP graph at once.  A launch carries as many tensors as fit 4 KB of
// kernel arguments; longer lists take several launches.
#pragma once

#include <algorithm>

#include "muon_internal.h"

namespace muon {

// Elements of one unit of work of the norm and of the clipping kernel.  A tensor
// of numel elements is cut into max(1, ceil(numel / unit)) units (its last one
// short); units of a launch's tensors are numbered through in list order.
constexpr int64_t kNormUnit = 8192;
constexpr int64_t kScaleUnit = 1024;
// Workgroups of one launch of the norm kernel, at most: each takes a
// contiguous run of units, so that it leaves one partial sum for each tensor
// it meets and the partials of a launch number at most workgroups + tensors.
constexpr int kNormGroups = 1024;

inline int64_t units_of(int64_t numel, int64_t unit) {
    return std::max<int64_t>(1, (numel + unit - 1) / unit);
}

// A tensor's length, type(s) and first unit in one word: bits 0-34 numel
// (<= 2^34), bit 35 the source's type, bit 36 the destination's (1: bfloat16),
// bits 37-63 the first unit (below 2^27: a launch's tensors hold at most
// 2^36 elements and number at most 248).
inline uint64_t clip_meta(int64_t numel, int src_bf16, int dst_bf16, int64_t unit) {
    return uint64_t(numel) | uint64_t(src_bf16) << 35 | uint64_t(dst_bf16) << 36 |
           uint64_t(unit) << 37;
}
static_assert((kMaxSetNumel / kScaleUnit + 256) < (int64_t(1) << 27), "unit number");

constexpr int kNormTensors = 248;
struct NormArgs {
    const void* data[kNormTensors];
    uint64_t meta[kNormTensors];
    double* partial;  // slot w + t holds workgroup w's sum over tensor t
    int32_t n;
    int32_t units;  // of all n tensors
    int32_t span;   // units of one workgroup
    int32_t base;   // number of the first tensor in the whole list
};
static_assert(sizeof(NormArgs) <= 4096, "kernel arguments");

constexpr int kClipTensors = 169;
struct ClipArgs {
    const void* src[kClipTensors];
    void* dst[kClipTensors];
    uint64_t meta[kClipTensors];
    const muon_clip_t* clip;
    int32_t n;
    int32_t units;
    int32_t in_place;  // every dst is its src
};
static_assert(sizeof(ClipArgs) <= 4096, "kernel arguments");

// Elements of one unit of the AdamW kernel.
constexpr int64_t kAdamwUnit = 256;
static_assert(kMaxSetNumel / kAdamwUnit + 256 < (int64_t(1) << 29), "unit number");
constexpr int kAdamwRanges = 240;
// A range in two words.  Offsets are multiples of 4 below kMaxSetNumel; the
// length follows from the units that the range takes and what its last one lacks.
struct AdamwRange {
    uint64_t at;  // bits 0-33 offset / 4, 34-49 group, 50-57 elements missing in the last unit
    uint64_t to;  // bits 0-33 param_offset / 4, 34-63 first unit
};
struct AdamwArgs {
    AdamwRange range[kAdamwRanges];
    void* params;
    uint16_t* copy;
    const void* grads;
    float* m;
    float* v;
    const muon_adamw_group_t* groups;
    const muon_clip_t* clip;
    int32_t n;
    int32_t units;
};
static_assert(sizeof(AdamwArgs) <= 4096, "kernel arguments");

// Slots of partial sums that a list of tensors takes over all its launches, at
// most: as many launches as its length asks for, each with all the workgroups
// that its units could fill.
int64_t norm_slots(const muon_tensor_t* t, int64_t n);
// Sums of squares of the listed tensors into `slots`, then the record (and
// with tensor_norms every tensor's own norm).
hipError_t launch_grad_norm(const muon_tensor_t* t, int64_t n, float max_norm, muon_clip_t* clip,
                            float* tensor_norms, double* slots, hipStream_t s);
hipError_t launch_clip_finish(muon_clip_t* clip, float max_norm, hipStream_t s);
hipError_t launch_clip(const muon_tensor_t* src, const muon_tensor_t* dst, int64_t n,
                       const muon_clip_t* clip, hipStream_t s);
hipError_t launch_adamw(void* params, int param_dtype, void* model_copy, const void* grads,
                        int grad_dtype, float* exp_avg, float* exp_avg_sq,
                        const muon_range_t* ranges, int64_t n, const muon_adamw_group_t* groups,
                        const muon_clip_t* clip, hipStream_t s);

}  // namespace muon
