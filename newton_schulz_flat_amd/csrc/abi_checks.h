// What the entry points without plans share: failing with a message, running a
// body as an entry point, and the checks of types and pointers.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "muon_internal.h"

namespace muon {

namespace {

__attribute__((format(printf, 3, 4))) inline int fail(Status* st, int code, const char* fmt, ...) {
    st->code = code;
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(st->msg, sizeof(st->msg), fmt, ap);
    va_end(ap);
    return code;
}

// Runs an entry point's body and reports its status.
template <typename F>
int guarded(F body) try {
    Status st{MUON_OK, ""};
    return body(st) == MUON_OK ? int(MUON_OK) : report(st);
}
MUON_CATCH

#define TRY(expr)                              \
    do {                                       \
        if ((expr) != MUON_OK) return st.code; \
    } while (0)

inline bool known_dtype(int dtype) { return dtype == MUON_DTYPE_F32 || dtype == MUON_DTYPE_BF16; }
inline size_t dtype_bytes(int dtype) { return dtype == MUON_DTYPE_BF16 ? 2 : 4; }

inline int check_pointer(const void* p, const char* name, size_t align, Status* st) {
    if (p == nullptr) return fail(st, MUON_ERR_NULL_POINTER, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % align != 0)
        return fail(st, MUON_ERR_MISALIGNED, "%s is not %zu-byte aligned", name, align);
    return MUON_OK;
}

inline int hip_status(hipError_t e, const char* what, Status* st) {
    if (e == hipSuccess) return MUON_OK;
    return fail(st, MUON_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

}  // namespace

}  // namespace muon
