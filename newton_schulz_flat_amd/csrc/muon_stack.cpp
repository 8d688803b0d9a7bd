// extern "C" entry points of the orthogonalization of stacks (declared, with their
// contracts, in include/muon_step.h), and the exponents of its float16 pairs.
#include <algorithm>
#include <cmath>

#include "abi_checks.h"
#include "stack_internal.h"

namespace muon {

StackShape stack_shape(int64_t rows, int64_t cols) {
    StackShape s;
    s.tall = rows > cols;
    s.r = std::min(rows, cols), s.c = std::max(rows, cols);
    s.rp = s.r <= 32 ? 32 : (s.r + kStackPad - 1) / kStackPad * kStackPad;
    s.cp = (s.c + kStackPad - 1) / kStackPad * kStackPad;
    return s;
}

// About how many microseconds a stage takes, from measurements of 14 stacks (256 x 256 to 4096 x 4096,
// 64 x 256 x 256, 1024 x 8192) in every tile with and without shared K steps: a K step lasts the
// longer where two workgroups share a CU, and where workgroups share tiles: these are at different K
// steps, so that L2 serves none of them twice.  Every tile ends with its epilogue, or a second
// pass adds the sums.  Off by 15% as a rule.  Stage A of 4096 x 4096: 256-tiles
// shared by 256 workgroups 201 us, a workgroup a tile 243, 64-tiles 328; of 512 x 512: 10, 50 and 10.
static double stack_estimate(const StackTiling& t, int64_t count) {
    const double most = t.tile == 256 ? 1 : 2;
    const bool shared = t.slots() > 0;
    const double first = t.tile == 256 ? 2.3 : t.tile == 128 ? (shared ? 0.8 : 0.72) : shared ? 0.45 : 0.21;
    const double both = t.tile == 256 ? 2.3 : t.tile == 128 ? (shared ? 2.0 : 1.3) : shared ? 0.86 : 0.47;
    const double end = t.tile == 256 ? 16 : t.tile == 128 ? 5 : 2;
    const double load = double(t.workers) * double(count) / 256, rounds = std::floor(load / most);
    const double rest = load - rounds * most;
    const double step = rounds * both + (rest > 1 ? both : rest > 0 ? first : 0);
    double us = 4 + double(t.per) * step;
    if (!shared) return us + end * (rounds + (rest > 0 ? 1 : 0));
    us += end * (1 + double(t.tiles) / double(t.workers));
    return us + 3 + double(t.slots()) * double(count) * double(t.slot_bytes()) * 2 / 6e6;
}

StackTiling stack_tiling(int stage, const StackShape& s, int64_t count) {
    StackTiling best{};
    double least = 0;
    for (int tile : {256, 128, 64}) {
        const int64_t tm = (s.rp + tile - 1) / tile, tn = (s.cp + tile - 1) / tile;
        StackTiling t{tile, stage == kStageX ? tm * tn : tm * (tm + 1) / 2, (stage == kStageA ? s.cp : s.rp) / 32,
                      0, 0};
        const int64_t resident = tile == 256 ? 256 : 512;
        for (int64_t workers : {t.tiles, 256 / count, resident / count, 2 * resident / count}) {
            // (a tile's steps are shared where there are few tiles, and not below 4 steps each)
            if (workers != t.tiles && (workers <= t.tiles / 4 || workers * 4 > t.tiles * t.steps || workers < 2))
                continue;
            t.workers = workers;
            t.per = workers == t.tiles ? t.steps : (t.tiles * t.steps + workers - 1) / workers;
            const double us = stack_estimate(t, count);
            if (best.tile == 0 || us < least) least = us, best = t;
        }
    }
    return best;
}

// Two iterates, A and B, 4 bytes an element, the partial sums of squares, the exponents, and the
// sums of tiles that several workgroups share.
size_t stack_matrix_bytes(const StackShape& s, int64_t count) {
    size_t shared = size_t(s.rp * s.cp) * 4;  // r <= 128: Gram matrices
    if (s.r > 128)
        for (int stage : {kStageA, kStageB, kStageX}) {
            const StackTiling t = stack_tiling(stage, s, count);
            shared = std::max(stage == kStageA ? 0 : shared, size_t(t.slots()) * t.slot_bytes());
        }
    return size_t(2 * s.rp * s.cp + 2 * s.rp * s.rp) * 4 + size_t(stack_part_slots(s.r, s.c)) * sizeof(double) +
           kStackScales * sizeof(StackScale) + shared;
}

namespace {

int check_stack(const muon_stack_t* s, Status* st) {
    if (s == nullptr) return fail(st, MUON_ERR_NULL_POINTER, "stack is NULL");
    if (s->count < 0 || s->count > kStackMaxCount)
        return fail(st, MUON_ERR_BAD_ARG, "count %lld is outside [0, %lld]", (long long)s->count,
                    (long long)kStackMaxCount);
    if (s->rows < 1 || s->cols < 1 || s->rows > kMaxSide || s->cols > kMaxSide ||
        s->rows * s->cols > kStackMaxNumel)
        return fail(st, MUON_ERR_BAD_SHAPE, "%lld x %lld has a side outside [1, %lld] or more than %lld "
                    "elements", (long long)s->rows, (long long)s->cols, (long long)kMaxSide,
                    (long long)kStackMaxNumel);
    if (!known_dtype(s->in_dtype) || !known_dtype(s->out_dtype))
        return fail(st, MUON_ERR_BAD_ARG, "in_dtype %d or out_dtype %d is not MUON_DTYPE_F32 or _BF16",
                    s->in_dtype, s->out_dtype);
    return MUON_OK;
}

// Strides of in (or out); matrices of out lie apart.
int check_strides(const muon_stack_t& s, int64_t stride, int64_t row, bool apart, const char* name,
                  Status* st) {
    const int64_t most = int64_t(1) << 40;
    if (s.rows > 1 && (row < s.cols || row > kStackMaxNumel))
        return fail(st, MUON_ERR_BAD_SHAPE, "%s_row %lld is outside [cols = %lld, %lld]", name,
                    (long long)row, (long long)s.cols, (long long)kStackMaxNumel);
    if (s.count > 1 && (stride < 0 || stride > most))
        return fail(st, MUON_ERR_BAD_SHAPE, "%s_stride %lld is outside [0, 2^40]", name,
                    (long long)stride);
    if (!apart || s.count <= 1) return MUON_OK;
    // matrices one behind the other, or side by side within longer rows
    const int64_t span = s.rows > 1 ? (s.rows - 1) * row + s.cols : s.cols;
    const bool beside = stride >= s.cols && (s.rows == 1 || (s.count - 1) * stride + s.cols <= row);
    if (stride < span && !beside)
        return fail(st, MUON_ERR_OVERLAP, "%s_stride %lld lets matrices of %lld elements overlap", name,
                    (long long)stride, (long long)span);
    return MUON_OK;
}

Range span_of(const muon_stack_t& s, const void* p, int64_t stride, int64_t row, int dtype,
              const char* name) {
    const int64_t last = (s.count > 1 ? (s.count - 1) * stride : 0) + (s.rows > 1 ? (s.rows - 1) * row : 0);
    return {p, size_t(last + s.cols) * dtype_bytes(dtype), name};
}

// Coefficients are finite, and the bound on the largest singular value, which is 1 at first,
// stays where float32 holds everything that is worked out from it.  (The kernels work the
// same bounds out from a matrix's own norm where that is small.)
int plan_steps(const float* k, int n, StackPlan* plan, Status* st) {
    float top = 1.001f;
    plan->n = n;
    for (int t = 0; t < n; ++t) {
        StackStep& s = plan->steps[t];
        s.a = k[3 * t], s.b = k[3 * t + 1], s.c = k[3 * t + 2];
        for (float v : {s.a, s.b, s.c})
            if (!std::isfinite(v))
                return fail(st, MUON_ERR_BAD_ARG, "coefficients of step %d are not finite", t);
        const double gram = double(top) * top;
        const double poly = std::fabs(double(s.a)) + std::fabs(double(s.b)) * gram +
                            std::fabs(double(s.c)) * gram * gram;
        plan->scales[t] = stack_scale(s, top);
        if (!(top < kStackMaxNorm) || !(poly < kStackMaxNorm))
            return fail(st, MUON_ERR_BAD_ARG,
                        "coefficients of step %d let singular values grow beyond 2^24", t);
    }
    plan->scales[n] = {int16_t(stack_exponent(top, kStackLeastX)), 0, 0, 0};
    return MUON_OK;
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" {

int muon_stack_workspace_bytes(const muon_stack_t* stack, size_t* out_bytes) {
    return guarded([&](Status& st) {
        if (out_bytes == nullptr) return fail(&st, MUON_ERR_NULL_POINTER, "out_bytes is NULL");
        TRY(check_stack(stack, &st));
        *out_bytes = size_t(stack->count) *
                     stack_matrix_bytes(stack_shape(stack->rows, stack->cols), std::max<int64_t>(stack->count, 1));
        return int(MUON_OK);
    });
}

int muon_orthogonalize_stack(const muon_stack_t* stack, const float* coefficients, int n_steps,
                             float scale, void* workspace, size_t workspace_bytes,
                             hipStream_t stream) {
    return guarded([&](Status& st) {
        TRY(check_stack(stack, &st));
        if (n_steps < 0 || n_steps > kMaxNsSteps)
            return fail(&st, MUON_ERR_BAD_ARG, "n_steps = %d is outside [0, %d]", n_steps, kMaxNsSteps);
        if (n_steps > 0 && coefficients == nullptr)
            return fail(&st, MUON_ERR_NULL_POINTER, "coefficients is NULL");
        TRY(check_scalar(scale, "scale", &st));
        StackPlan plan;
        TRY(plan_steps(coefficients, n_steps, &plan, &st));
        const muon_stack_t& s = *stack;
        if (s.count == 0) return int(MUON_OK);
        TRY(check_strides(s, s.in_stride, s.in_row, false, "in", &st));
        TRY(check_strides(s, s.out_stride, s.out_row, true, "out", &st));
        TRY(check_pointer(s.in, "in", dtype_bytes(s.in_dtype), &st));
        TRY(check_pointer(s.out, "out", dtype_bytes(s.out_dtype), &st));
        TRY(check_pointer(workspace, "workspace", kWsAlign, &st));
        const size_t one = stack_matrix_bytes(stack_shape(s.rows, s.cols), s.count);
        if (workspace_bytes < one)
            return fail(&st, MUON_ERR_WORKSPACE_TOO_SMALL,
                        "workspace has %zu bytes; one matrix needs %zu", workspace_bytes, one);
        const size_t used = std::min(workspace_bytes, size_t(s.count) * one);
        const Range all[3] = {span_of(s, s.in, s.in_stride, s.in_row, s.in_dtype, "in"),
                              span_of(s, s.out, s.out_stride, s.out_row, s.out_dtype, "out"),
                              {workspace, used, "workspace"}};
        TRY(check_no_alias(all, 3, &st));
        return hip_status(launch_stack(s, plan, scale, workspace, used, stream),
                          "orthogonalize stack", &st);
    });
}

}  // extern "C"
