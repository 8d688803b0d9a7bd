// extern "C" entry points of the 8-bit casts and products (declared, with their
// contracts, in include/muon_step.h).  Everything is checked on the host before
// anything is enqueued, and nothing is thrown across the ABI.
#include "abi_checks.h"
#include "fp8_internal.h"

namespace muon {

namespace {

int check_sides(int64_t rows, int64_t cols, const char* name, Status* st) {
    if (rows < 0 || cols < 0 || rows > kFp8MaxSide || cols > kFp8MaxSide || rows * cols > kMaxNumel)
        return fail(st, MUON_ERR_BAD_SHAPE,
                    "%s: %lld x %lld has a side outside [0, %lld] or more than %lld elements", name,
                    (long long)rows, (long long)cols, (long long)kFp8MaxSide, (long long)kMaxNumel);
    return MUON_OK;
}

// (With rows of up to 2^24 a matrix's last one ends within 2^50 elements of its start.)
int check_row_stride(int64_t rows, int64_t cols, int64_t stride, const char* name, Status* st) {
    if (rows > 1 && (stride < cols || stride > (int64_t(1) << 26)))
        return fail(st, MUON_ERR_BAD_SHAPE, "%s: row stride %lld is outside [cols = %lld, 2^26]", name,
                    (long long)stride, (long long)cols);
    return MUON_OK;
}

int64_t extent(int64_t rows, int64_t cols, int64_t stride) {
    return rows == 0 || cols == 0 ? 0 : (rows - 1) * stride + cols;
}

int check_matrix(const muon_fp8_t& m, const char* name, Status* st) {
    if (check_sides(m.rows, m.cols, name, st) != MUON_OK) return st->code;
    if (m.format != MUON_FP8_E4M3 && m.format != MUON_FP8_E5M2)
        return fail(st, MUON_ERR_BAD_ARG, "%s: format %d is not MUON_FP8_E4M3 or _E5M2", name, m.format);
    if (m.block_rows != 1 && m.block_rows != kFp8Block)
        return fail(st, MUON_ERR_BAD_ARG, "%s: block_rows %d is not 1 or 128", name, m.block_rows);
    if (m.rows == 0 || m.cols == 0) return MUON_OK;
    if (check_row_stride(m.rows, m.cols, m.row_stride, name, st) != MUON_OK) return st->code;
    if (check_pointer(m.codes, name, 1, st) != MUON_OK) return st->code;
    if (m.scales == nullptr) return fail(st, MUON_ERR_NULL_POINTER, "%s: scales is NULL", name);
    if (reinterpret_cast<uintptr_t>(m.scales) % sizeof(float) != 0)
        return fail(st, MUON_ERR_MISALIGNED, "%s: scales is not 4-byte aligned", name);
    // scales of different blocks lie apart, with either direction outermost
    const int64_t nr = m.block_rows == 1 ? m.rows : fp8_blocks(m.rows), nc = fp8_blocks(m.cols);
    const int64_t r = m.scale_row, c = m.scale_col, most = int64_t(1) << 32;
    const bool apart = (nr == 1 || (r >= 1 && r <= most)) && (nc == 1 || (c >= 1 && c <= most)) &&
                       (nr == 1 || nc == 1 || r >= c * nc || c >= r * nr);
    if (!apart)
        return fail(st, MUON_ERR_BAD_SHAPE,
                    "%s: scale strides %lld, %lld let %lld x %lld scales overlap, or are above 2^32",
                    name, (long long)r, (long long)c, (long long)nr, (long long)nc);
    return MUON_OK;
}

Range codes_range(const muon_fp8_t& m, const char* name) {
    return {m.codes, size_t(extent(m.rows, m.cols, m.row_stride)), name};
}

Range scales_range(const muon_fp8_t& m, const char* name) {
    if (m.rows == 0 || m.cols == 0) return {m.scales, 0, name};
    const int64_t nr = m.block_rows == 1 ? m.rows : fp8_blocks(m.rows), nc = fp8_blocks(m.cols);
    const int64_t last = (nr > 1 ? (nr - 1) * m.scale_row : 0) + (nc > 1 ? (nc - 1) * m.scale_col : 0);
    return {m.scales, size_t(last + 1) * sizeof(float), name};
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" {

int muon_fp8_cast(const void* x, int dtype, int64_t rows, int64_t cols, int64_t row_stride,
                  const muon_fp8_t* out, const muon_fp8_t* out_t, hipStream_t stream) {
    return guarded([&](Status& st) {
        if (!known_dtype(dtype))
            return fail(&st, MUON_ERR_BAD_ARG, "dtype %d is not MUON_DTYPE_F32 or _BF16", dtype);
        TRY(check_sides(rows, cols, "x", &st));
        if (out == nullptr && out_t == nullptr)
            return fail(&st, MUON_ERR_NULL_POINTER, "out and out_t are NULL");
        if (out != nullptr) {
            TRY(check_matrix(*out, "out", &st));
            if (out->rows != rows || out->cols != cols)
                return fail(&st, MUON_ERR_BAD_SHAPE, "out is %lld x %lld, x %lld x %lld",
                            (long long)out->rows, (long long)out->cols, (long long)rows, (long long)cols);
        }
        if (out_t != nullptr) {
            TRY(check_matrix(*out_t, "out_t", &st));
            if (out_t->rows != cols || out_t->cols != rows)
                return fail(&st, MUON_ERR_BAD_SHAPE, "out_t is %lld x %lld, x %lld x %lld",
                            (long long)out_t->rows, (long long)out_t->cols, (long long)rows,
                            (long long)cols);
        }
        if (out != nullptr && out_t != nullptr &&
            (out->format != out_t->format || out->block_rows != out_t->block_rows))
            return fail(&st, MUON_ERR_BAD_ARG, "out and out_t differ in format or block_rows");
        if (rows == 0 || cols == 0) return int(MUON_OK);
        TRY(check_row_stride(rows, cols, row_stride, "x", &st));
        TRY(check_pointer(x, "x", dtype_bytes(dtype), &st));
        const Range none{nullptr, 0, ""};
        const Range all[5] = {{x, size_t(extent(rows, cols, row_stride)) * dtype_bytes(dtype), "x"},
                              out ? codes_range(*out, "out's codes") : none,
                              out ? scales_range(*out, "out's scales") : none,
                              out_t ? codes_range(*out_t, "out_t's codes") : none,
                              out_t ? scales_range(*out_t, "out_t's scales") : none};
        TRY(check_no_alias(all, 5, &st));
        return hip_status(launch_fp8_cast(x, dtype, rows, cols, row_stride, out, out_t, stream),
                          "fp8 cast", &st);
    });
}

int muon_fp8_workspace_bytes(int64_t m, int64_t n, int64_t k, size_t* out_bytes) {
    return guarded([&](Status& st) {
        if (out_bytes == nullptr) return fail(&st, MUON_ERR_NULL_POINTER, "out_bytes is NULL");
        TRY(check_sides(m, k, "a", &st));
        TRY(check_sides(n, k, "b", &st));
        *out_bytes = fp8_workspace_bytes(m, n, k);
        return int(MUON_OK);
    });
}

int muon_fp8_matmul(const muon_fp8_t* a, const muon_fp8_t* b, void* out, int out_dtype,
                    int64_t out_row_stride, int accumulate, void* workspace,
                    size_t workspace_bytes, hipStream_t stream) {
    return guarded([&](Status& st) {
        if (a == nullptr || b == nullptr)
            return fail(&st, MUON_ERR_NULL_POINTER, "%s is NULL", a == nullptr ? "a" : "b");
        TRY(check_matrix(*a, "a", &st));
        TRY(check_matrix(*b, "b", &st));
        if (a->cols != b->cols)
            return fail(&st, MUON_ERR_BAD_SHAPE, "a has %lld columns, b %lld", (long long)a->cols,
                        (long long)b->cols);
        if (!known_dtype(out_dtype))
            return fail(&st, MUON_ERR_BAD_ARG, "out_dtype %d is not MUON_DTYPE_F32 or _BF16", out_dtype);
        if (accumulate != 0 && accumulate != 1)
            return fail(&st, MUON_ERR_BAD_ARG, "accumulate = %d is not 0 or 1", accumulate);
        if (accumulate != 0 && out_dtype != MUON_DTYPE_F32)
            return fail(&st, MUON_ERR_BAD_ARG, "accumulate needs a float32 out");
        const int64_t m = a->rows, n = b->rows;
        if (m == 0 || n == 0) return int(MUON_OK);
        if (m * n > kFp8MaxOut)
            return fail(&st, MUON_ERR_BAD_SHAPE, "out: %lld x %lld has more than %lld elements",
                        (long long)m, (long long)n, (long long)kFp8MaxOut);
        TRY(check_row_stride(m, n, out_row_stride, "out", &st));
        TRY(check_pointer(out, "out", dtype_bytes(out_dtype), &st));
        const size_t need = fp8_workspace_bytes(m, n, a->cols);
        if (need > 0) TRY(check_pointer(workspace, "workspace", kWsAlign, &st));
        if (workspace_bytes < need)
            return fail(&st, MUON_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes; %zu are needed",
                        workspace_bytes, need);
        const Range written[2] = {
            {out, size_t(extent(m, n, out_row_stride)) * dtype_bytes(out_dtype), "out"},
            {workspace, need, "workspace"}};
        const Range read[4] = {codes_range(*a, "a's codes"), scales_range(*a, "a's scales"),
                               codes_range(*b, "b's codes"), scales_range(*b, "b's scales")};
        TRY(check_no_alias(written, 2, &st));
        for (const Range& w : written)
            for (const Range& r : read) {
                const Range pair[2] = {w, r};
                TRY(check_no_alias(pair, 2, &st));
            }
        return hip_status(launch_fp8_matmul(*a, *b, out, out_dtype, out_row_stride, accumulate != 0,
                                            workspace, stream),
                          "fp8 matmul", &st);
    });
}

}  // extern "C"
