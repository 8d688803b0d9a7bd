// extern "C" entry points of the gradient norm, clipping and AdamW (declared,
// with their contracts, in include/muon_step.h).  As for the step, everything
// is checked on the host before anything is enqueued, and nothing is thrown
// across the ABI.
#include <algorithm>
#include <cmath>
#include <vector>

#include "abi_checks.h"
#include "clip_internal.h"

namespace muon {

namespace {

int check_count(int64_t n, const void* list, const char* name, Status* st) {
    if (n < 0) return fail(st, MUON_ERR_BAD_ARG, "%s count n = %lld < 0", name, (long long)n);
    if (n > (int64_t(1) << 24))
        return fail(st, MUON_ERR_BAD_ARG, "%s count n = %lld is too large", name, (long long)n);
    if (n > 0 && list == nullptr) return fail(st, MUON_ERR_NULL_POINTER, "%s is NULL", name);
    return MUON_OK;
}

int check_tensors(const muon_tensor_t* t, int64_t n, const char* name, Status* st) {
    if (check_count(n, t, name, st) != MUON_OK) return st->code;
    int64_t total = 0;
    for (int64_t i = 0; i < n; ++i) {
        if (!known_dtype(t[i].dtype))
            return fail(st, MUON_ERR_BAD_ARG, "%s[%lld]: dtype %d is not MUON_DTYPE_F32 or _BF16",
                        name, (long long)i, t[i].dtype);
        if (t[i].numel < 0 || t[i].numel > kMaxNumel)
            return fail(st, MUON_ERR_BAD_SHAPE, "%s[%lld]: numel %lld is outside [0, %lld]", name,
                        (long long)i, (long long)t[i].numel, (long long)kMaxNumel);
        total += t[i].numel;
        if (total > kMaxSetNumel)
            return fail(st, MUON_ERR_BAD_SHAPE, "%s[0..%lld] hold more than %lld elements in total",
                        name, (long long)i, (long long)kMaxSetNumel);
        if (t[i].numel > 0 && t[i].data == nullptr)
            return fail(st, MUON_ERR_NULL_POINTER, "%s[%lld]: data is NULL", name, (long long)i);
        if (reinterpret_cast<uintptr_t>(t[i].data) % dtype_bytes(t[i].dtype) != 0)
            return fail(st, MUON_ERR_MISALIGNED, "%s[%lld]: data is not aligned to its elements",
                        name, (long long)i);
    }
    return MUON_OK;
}

// Bytes (or elements) of one entry of a list.
struct Span {
    uintptr_t begin, end;
    int64_t entry;
};

std::vector<Span> spans_of(const muon_tensor_t* t, int64_t n) {
    std::vector<Span> s;
    s.reserve(size_t(n));
    for (int64_t i = 0; i < n; ++i) {
        if (t[i].numel == 0) continue;
        const uintptr_t a = reinterpret_cast<uintptr_t>(t[i].data);
        s.push_back({a, a + size_t(t[i].numel) * dtype_bytes(t[i].dtype), i});
    }
    return s;
}

// Lists come in address order as a rule: a look is cheaper than a sort.
void sort_spans(std::vector<Span>& s) {
    const auto before = [](const Span& a, const Span& b) { return a.begin < b.begin; };
    if (!std::is_sorted(s.begin(), s.end(), before)) std::sort(s.begin(), s.end(), before);
}

int check_disjoint(std::vector<Span>& s, const char* what, Status* st) {
    sort_spans(s);
    for (size_t i = 1; i < s.size(); ++i)
        if (s[i].begin < s[i - 1].end)
            return fail(st, MUON_ERR_OVERLAP, "%s[%lld] and %s[%lld] overlap", what,
                        (long long)s[i - 1].entry, what, (long long)s[i].entry);
    return MUON_OK;
}

int check_apart(const muon_tensor_t* t, int64_t n, const char* name, const Range& r, Status* st) {
    if (r.ptr == nullptr || r.bytes == 0) return MUON_OK;
    const uintptr_t a = reinterpret_cast<uintptr_t>(r.ptr), b = a + r.bytes;
    for (int64_t i = 0; i < n; ++i) {
        if (t[i].numel == 0) continue;
        const uintptr_t c = reinterpret_cast<uintptr_t>(t[i].data);
        const uintptr_t d = c + size_t(t[i].numel) * dtype_bytes(t[i].dtype);
        if (c < b && a < d)
            return fail(st, MUON_ERR_ALIAS, "%s[%lld] and %s overlap in memory", name,
                        (long long)i, r.name);
    }
    return MUON_OK;
}

// Every destination is its own source (in place: same address and type) or
// lies apart from all sources.
int check_in_place(const muon_tensor_t* src, const muon_tensor_t* dst, int64_t n,
                   const std::vector<Span>& out, Status* st) {
    std::vector<Span> in;
    for (const Span& s : spans_of(src, n))
        if (src[s.entry].data != dst[s.entry].data || src[s.entry].dtype != dst[s.entry].dtype)
            in.push_back(s);
    sort_spans(in);
    // no source that is read into another place may meet any destination
    size_t k = 0;
    uintptr_t reach = 0;  // sources may overlap each other: the furthest end so far
    int64_t who = 0;
    for (const Span& o : out) {
        for (; k < in.size() && in[k].begin < o.end; ++k)
            if (in[k].end > reach) reach = in[k].end, who = in[k].entry;
        if (reach > o.begin)
            return fail(st, MUON_ERR_ALIAS, "src[%lld] and dst[%lld] overlap in memory",
                        (long long)who, (long long)o.entry);
    }
    return MUON_OK;
}

int check_max_norm(float v, Status* st) {
    if (!(v >= 0.f))  // NaN too
        return fail(st, MUON_ERR_BAD_ARG, "max_norm = %g is not a number >= 0", v);
    return MUON_OK;
}

size_t workspace_need(const muon_tensor_t* t, int64_t n) {
    const size_t bytes = size_t(norm_slots(t, n)) * sizeof(double);
    return (bytes + kWsAlign - 1) / kWsAlign * kWsAlign;
}

int check_ranges(const muon_range_t* r, int64_t n, int64_t n_groups, int64_t n_state,
                 int64_t n_params, int param_dtype, Status* st) {
    const int64_t align = param_dtype == MUON_DTYPE_F32 ? 4 : 8;  // 16 bytes
    int64_t total = 0;
    std::vector<Span> state, params;
    state.reserve(size_t(n));
    params.reserve(size_t(n));
    for (int64_t i = 0; i < n; ++i) {
        const muon_range_t& q = r[i];
        if (q.numel < 0 || q.numel > kMaxNumel)
            return fail(st, MUON_ERR_BAD_SHAPE, "ranges[%lld]: numel %lld is outside [0, %lld]",
                        (long long)i, (long long)q.numel, (long long)kMaxNumel);
        total += q.numel;
        if (total > kMaxSetNumel)
            return fail(st, MUON_ERR_BAD_SHAPE, "ranges[0..%lld] hold more than %lld elements in total",
                        (long long)i, (long long)kMaxSetNumel);
        if (q.group < 0 || q.group >= n_groups)
            return fail(st, MUON_ERR_BAD_ARG, "ranges[%lld]: group %d outside [0, %lld)",
                        (long long)i, q.group, (long long)n_groups);
        if (q.offset < 0 || q.offset > n_state - q.numel)
            return fail(st, MUON_ERR_OUT_OF_BOUNDS,
                        "ranges[%lld]: offset %lld, numel %lld are outside the state buffers of %lld "
                        "elements",
                        (long long)i, (long long)q.offset, (long long)q.numel, (long long)n_state);
        if (q.param_offset < 0 || q.param_offset > n_params - q.numel)
            return fail(st, MUON_ERR_OUT_OF_BOUNDS,
                        "ranges[%lld]: param_offset %lld, numel %lld are outside params (%lld elements)",
                        (long long)i, (long long)q.param_offset, (long long)q.numel,
                        (long long)n_params);
        if (q.offset >= kMaxSetNumel || q.param_offset >= kMaxSetNumel)
            return fail(st, MUON_ERR_BAD_SHAPE,
                        "ranges[%lld]: offset %lld or param_offset %lld is not below %lld",
                        (long long)i, (long long)q.offset, (long long)q.param_offset,
                        (long long)kMaxSetNumel);
        if (q.offset % 4 != 0)
            return fail(st, MUON_ERR_MISALIGNED, "ranges[%lld]: offset %lld is not a multiple of 4",
                        (long long)i, (long long)q.offset);
        if (q.param_offset % align != 0)
            return fail(st, MUON_ERR_MISALIGNED,
                        "ranges[%lld]: param_offset %lld is not 16-byte aligned", (long long)i,
                        (long long)q.param_offset);
        if (q.numel == 0) continue;
        state.push_back({uintptr_t(q.offset), uintptr_t(q.offset + q.numel), i});
        params.push_back({uintptr_t(q.param_offset), uintptr_t(q.param_offset + q.numel), i});
    }
    if (check_disjoint(state, "state of ranges", st) != MUON_OK) return st->code;
    return check_disjoint(params, "params of ranges", st);
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" {

int muon_clip_workspace_bytes(const muon_tensor_t* tensors, int64_t n, size_t* out_bytes) {
    return guarded([&](Status& st) {
        if (out_bytes == nullptr) return fail(&st, MUON_ERR_NULL_POINTER, "out_bytes is NULL");
        TRY(check_tensors(tensors, n, "tensors", &st));
        *out_bytes = workspace_need(tensors, n);
        return int(MUON_OK);
    });
}

int muon_grad_norm(const muon_tensor_t* tensors, int64_t n, float max_norm, muon_clip_t* clip,
                   float* tensor_norms, void* workspace, size_t workspace_bytes,
                   hipStream_t stream) {
    return guarded([&](Status& st) {
        TRY(check_tensors(tensors, n, "tensors", &st));
        TRY(check_max_norm(max_norm, &st));
        TRY(check_pointer(clip, "clip", alignof(muon_clip_t), &st));
        if (tensor_norms != nullptr)
            TRY(check_pointer(tensor_norms, "tensor_norms", sizeof(float), &st));
        const size_t need = workspace_need(tensors, n);
        if (need > 0) TRY(check_pointer(workspace, "workspace", kWsAlign, &st));
        if (workspace_bytes < need)
            return fail(&st, MUON_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes; %zu are needed",
                        workspace_bytes, need);
        const Range own[3] = {
            {clip, sizeof(muon_clip_t), "clip"},
            {tensor_norms, tensor_norms ? size_t(n) * sizeof(float) : 0, "tensor_norms"},
            {workspace, need, "workspace"}};
        TRY(check_no_alias(own, 3, &st));
        for (const Range& r : own) TRY(check_apart(tensors, n, "tensors", r, &st));
        return hip_status(launch_grad_norm(tensors, n, max_norm, clip, tensor_norms,
                                           static_cast<double*>(workspace), stream),
                          "grad norm", &st);
    });
}

int muon_clip_finish(muon_clip_t* clip, float max_norm, hipStream_t stream) {
    return guarded([&](Status& st) {
        TRY(check_pointer(clip, "clip", alignof(muon_clip_t), &st));
        TRY(check_max_norm(max_norm, &st));
        return hip_status(launch_clip_finish(clip, max_norm, stream), "clip finish", &st);
    });
}

int muon_clip_grads(const muon_tensor_t* src, const muon_tensor_t* dst, int64_t n,
                    const muon_clip_t* clip, hipStream_t stream) {
    return guarded([&](Status& st) {
        TRY(check_tensors(src, n, "src", &st));
        TRY(check_tensors(dst, n, "dst", &st));
        if (n == 0) return int(MUON_OK);
        TRY(check_pointer(clip, "clip", alignof(muon_clip_t), &st));
        for (int64_t i = 0; i < n; ++i)
            if (src[i].numel != dst[i].numel)
                return fail(&st, MUON_ERR_BAD_SHAPE, "src[%lld] has %lld elements, dst[%lld] %lld",
                            (long long)i, (long long)src[i].numel, (long long)i,
                            (long long)dst[i].numel);
        std::vector<Span> out = spans_of(dst, n);
        TRY(check_disjoint(out, "dst", &st));
        TRY(check_in_place(src, dst, n, out, &st));
        const Range record{clip, sizeof(muon_clip_t), "clip"};
        TRY(check_apart(dst, n, "dst", record, &st));
        return hip_status(launch_clip(src, dst, n, clip, stream), "clip", &st);
    });
}

int muon_adamw(void* params, int param_dtype, int64_t n_param_elems, void* model_copy,
               const void* grads, int grad_dtype, float* exp_avg, float* exp_avg_sq,
               int64_t n_state_elems, const muon_range_t* ranges, int64_t n,
               const muon_adamw_group_t* groups, int32_t n_groups, const muon_clip_t* clip,
               hipStream_t stream) {
    return guarded([&](Status& st) {
        TRY(check_count(n, ranges, "ranges", &st));
        if (!known_dtype(param_dtype))
            return fail(&st, MUON_ERR_BAD_ARG, "param_dtype %d is not MUON_DTYPE_F32 or _BF16",
                        param_dtype);
        if (!known_dtype(grad_dtype))
            return fail(&st, MUON_ERR_BAD_ARG, "grad_dtype %d is not MUON_DTYPE_F32 or _BF16",
                        grad_dtype);
        if (model_copy != nullptr && param_dtype != MUON_DTYPE_F32)
            return fail(&st, MUON_ERR_BAD_ARG, "model_copy needs float32 params (param_dtype %d)",
                        param_dtype);
        if (n_groups < 1 || n_groups > kMaxGroups)
            return fail(&st, MUON_ERR_BAD_ARG, "n_groups = %d is outside [1, %d]", n_groups,
                        kMaxGroups);
        if (n_param_elems < 0 || n_state_elems < 0)
            return fail(&st, MUON_ERR_BAD_ARG, "n_param_elems or n_state_elems < 0");
        TRY(check_ranges(ranges, n, n_groups, n_state_elems, n_param_elems, param_dtype, &st));
        bool any = false;
        for (int64_t i = 0; i < n && !any; ++i) any = ranges[i].numel > 0;
        if (!any) return int(MUON_OK);
        TRY(check_pointer(params, "params", 16, &st));
        TRY(check_pointer(grads, "grads", 16, &st));
        TRY(check_pointer(exp_avg, "exp_avg", 16, &st));
        TRY(check_pointer(exp_avg_sq, "exp_avg_sq", 16, &st));
        TRY(check_pointer(groups, "groups", alignof(muon_adamw_group_t), &st));
        if (model_copy != nullptr) TRY(check_pointer(model_copy, "model_copy", 16, &st));
        if (clip != nullptr) TRY(check_pointer(clip, "clip", alignof(muon_clip_t), &st));
        const Range all[7] = {
            {params, size_t(n_param_elems) * dtype_bytes(param_dtype), "params"},
            {model_copy, model_copy ? size_t(n_param_elems) * 2 : 0, "model_copy"},
            {grads, size_t(n_state_elems) * dtype_bytes(grad_dtype), "grads"},
            {exp_avg, size_t(n_state_elems) * 4, "exp_avg"},
            {exp_avg_sq, size_t(n_state_elems) * 4, "exp_avg_sq"},
            {groups, size_t(n_groups) * sizeof(muon_adamw_group_t), "groups"},
            {clip, clip ? sizeof(muon_clip_t) : 0, "clip"}};
        TRY(check_no_alias(all, 7, &st));
        return hip_status(launch_adamw(params, param_dtype, model_copy, grads, grad_dtype, exp_avg,
                                       exp_avg_sq, ranges, n, groups, clip, stream),
                          "adamw", &st);
    });
}

}  // extern "C"
