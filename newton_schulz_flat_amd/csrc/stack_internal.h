// Internal declarations of the orthogonalization of stacks.
#pragma once

#include <algorithm>
#include <cmath>

#include <hip/hip_runtime.h>

#include "muon_internal.h"

namespace muon {

constexpr int64_t kStackMaxCount = int64_t(1) << 20;
constexpr int64_t kStackMaxNumel = int64_t(1) << 31;
// Bound on the iterate's largest singular value, under which its float16 pairs keep
// their digits.
constexpr float kStackMaxNorm = 16777216.f;

// Coefficients of one step.
struct StackStep {
    float a, b, c;
};

// Exponents with which one step's matrices are stored: X 2^sx, A 2^sa, B 2^sb.
struct StackScale {
    int16_t sx, sa, sb, reserved;
};

// The exponent that brings magnitudes of up to `top` to at most 2^15, half of
// float16's range.  For a `top` below 2^least it is that of 2^least: an X is scaled by 2^127 at most,
// a float32, which gives the smallest one (2^-126, of a U of the smallest subnormal number) all its digits.
constexpr int kStackLeastX = -112, kStackLeastPoly = -120;
__host__ __device__ inline int stack_exponent(float top, int least) {
    int e = least;
    if (top > 0.f) {
        const uint32_t bits = __builtin_bit_cast(uint32_t, top);
        e = int(bits >> 23) - 126;  // top < 2^e (subnormal ones: 2^-126)
    }
    return 15 - (e > least ? e : least);
}

// v 2^e, for any e: exponents of factors leave float32's range (down to -500) where the product does not, or
// where it is lost beside its sum's other term.
__host__ __device__ inline float stack_scaled(float v, int e) { return __builtin_ldexpf(v, e); }

// The largest |a x + b x^3 + c x^5| on [0, top]: at an end or where the derivative
// a + 3 b x^2 + 5 c x^4 is zero.  Worked out for x = top sqrt(z), z up to 1, and coefficients of at most 1, so
// that nothing leaves float32's range that the result does not; the roots without a difference of
// numbers that may be alike (where c is small beside b, one of them).
__host__ __device__ inline float stack_largest(const StackStep& k, float top) {
    float a = k.a, b = k.b * top * top, c = k.c * top * top * top * top;
    const float most_of = fmaxf(fabsf(a), fmaxf(fabsf(b), fabsf(c)));
    if (!(most_of > 0.f)) return 0.f;
    a /= most_of, b /= most_of, c /= most_of;
    const auto value = [&](float z) { return fabsf(sqrtf(z) * (a + z * (b + c * z))); };
    float most = value(1.f);
    const float d = 9.f * b * b - 20.f * a * c;
    if (d >= 0.f) {
        const float q = -0.5f * (3.f * b + copysignf(sqrtf(d), b));
        for (float z : {q / (5.f * c), a / q})  // (c = 0: one of them infinite, or no number)
            if (z > 0.f && z < 1.f) most = fmaxf(most, value(z));
    }
    return most * most_of * top;
}

// One step: the exponents of its matrices where the largest singular value (and with it every
// entry) of X is at most `top`, and that bound for the next X.  Roundings, these of the
// bound included, add a part in a thousand at most.  The largest entry of A is at most top^2; where
// that leaves float32's range the exponent follows from top's.
__host__ __device__ inline StackScale stack_scale(const StackStep& k, float& top) {
    const int sx = stack_exponent(top, kStackLeastX), sa = 2 * sx - 15;
    const float poly = fabsf(k.b) + fabsf(k.c) * top * top;
    const StackScale s = {int16_t(sx), int16_t(sa), int16_t(sa - (15 - stack_exponent(poly, kStackLeastPoly))), 0};
    top = 1.001f * stack_largest(k, top);
    return s;
}

// What a stage's sums (down) and the matrix that is added to them (own) are multiplied by, each with
// the exponents of what it reads and of what is written; x_factors: the result once more, by after.
struct StackFactors {
    float own, down, after;
};
__host__ __device__ inline float stack_a_factor(const StackScale& s) { return stack_scaled(1.f, s.sa - 2 * s.sx); }
__host__ __device__ inline StackFactors stack_b_factors(const StackStep& k, const StackScale& s) {
    return {stack_scaled(k.b, s.sb - s.sa), stack_scaled(k.c, s.sb - 2 * s.sa), 1.f};
}
// `next`: the next X's exponent.  Results of the last step are those of the call, times `scale`; where X
// is small, 2^64 of its 2^-sx waits for the end, so that own and down, which are rounded, stay normal numbers.
__host__ __device__ inline StackFactors stack_x_factors(const StackStep& k, const StackScale& s, int next, bool last,
                                                        float scale) {
    const bool late = last && s.sx > 32;
    const int to = late ? 64 : last ? 0 : next;
    StackFactors f = {stack_scaled(k.a, to - s.sx), stack_scaled(1.f, to - s.sx - s.sb), 1.f};
    if (late)
        f.after = stack_scaled(scale, -64);
    else if (last)
        f.own *= scale, f.down *= scale;
    return f;
}

// The shape as the iteration sees it: r <= c, sides padded to whole blocks.
struct StackShape {
    int64_t r, c, rp, cp;
    bool tall;
};

// Sides are padded to this many elements, a shorter one of up to 32 to 32.
constexpr int64_t kStackPad = 64;
// Partial sums of squares of one matrix, and the room for them.
constexpr int64_t kStackPartials = 1024;
inline int64_t stack_parts(int64_t r, int64_t c) { return std::min(kStackPartials, (r * c + 8191) / 8192); }
inline int64_t stack_part_slots(int64_t r, int64_t c) { return (stack_parts(r, c) + 31) / 32 * 32; }
// Entries of one matrix's table of exponents: one a step, and the last X's; a multiple of 32.
constexpr int kStackScales = (kMaxNsSteps + 1 + 31) / 32 * 32;

StackShape stack_shape(int64_t rows, int64_t cols);

// The steps of a call with their exponents for a bound of 1 on the first iterate, which is
// every matrix's but those whose norm is not far above 1e-7: these, below kStackSmallBound, have
// theirs worked out by the kernels.
struct StackPlan {
    StackStep steps[kMaxNsSteps];
    StackScale scales[kMaxNsSteps + 1];
    int32_t n;
};
constexpr float kStackSmallBound = 0.5f;

// LDS of a matrix that one workgroup takes as a whole: X, A and B (whose rows are 256 bytes at
// least).
inline size_t stack_whole_lds(const StackShape& s) {
    // (of 32 rows, A's tiles are summed in four shares: three places of 4 KB)
    return s.r > 64 ? ~size_t(0) : size_t(s.rp * s.cp * 4 + 2 * s.rp * 256 + (s.rp == 32 ? 3 * 4096 : 0));
}
constexpr size_t kStackWholeLds = 156 * 1024;
bool stack_is_whole(const StackShape& s);
hipError_t launch_stack_whole(const muon_stack_t& stack, const StackShape& s, const StackPlan& plan,
                              float scale, hipStream_t stream);
// Workspace bytes of one matrix of a stack of `count`.
size_t stack_matrix_bytes(const StackShape& s, int64_t count);

// How a stage's products run, for every matrix of a stack of `count`: tiles, and the workgroups
// that share one matrix's K steps.
enum StackStage { kStageA = 0, kStageB = 1, kStageX = 2 };
struct StackTiling {
    int tile;
    int64_t tiles;    // of one matrix
    int64_t steps;    // K steps of a tile
    int64_t workers;  // workgroups of one matrix; tiles where each takes one tile
    int64_t per;      // K steps of a workgroup
    int64_t slots() const { return workers == tiles ? 0 : workers + tiles; }
    size_t slot_bytes() const { return size_t(tile) * tile * 4; }
};
StackTiling stack_tiling(int stage, const StackShape& s, int64_t count);
hipError_t launch_stack(const muon_stack_t& stack, const StackPlan& plan, float scale,
                        void* workspace, size_t workspace_bytes, hipStream_t s);

}  // namespace muon
