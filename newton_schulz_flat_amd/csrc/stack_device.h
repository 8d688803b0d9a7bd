// Device helpers of the orthogonalization of stacks: pairs of float16, their products, loads to
// LDS, and where a matrix begins and ends.
#pragma once

#include "k_common.h"
#include "stack_internal.h"

namespace muon {

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_one(uint16_t* p, float v) { *p = bf16_rne(v); }

// v 2^s as a pair, where v is already scaled.
struct Pair {
    _Float16 hi, lo;
};
__device__ __forceinline__ Pair split(float v) {
    const _Float16 hi = static_cast<_Float16>(v);
    return {hi, static_cast<_Float16>(v - static_cast<float>(hi))};
}
// Element (i, j) of a matrix of pairs with rp rows (padded): its high half; the low one lies 32
// further on.  Blocks of 32 columns lie one behind the other, each rp rows of 128 bytes: a K step of
// a tile is one contiguous piece, whatever the matrix's width.  (Row after row, a K step of a tile
// of 14336 columns is 256 lines 57344 bytes apart; that measured the same, 10.3 ms, and needs an
// address for every row.)
__device__ __forceinline__ int64_t pair_at(int64_t i, int j, int64_t rp) {
    return ((j >> 5) * rp + i) * 64 + (j & 31);
}

// 16 bytes from memory at base + offset to LDS at lds + 16 * lane, without passing
// through registers.  Written as assembly because the compiler cannot tell the two halves
// of the double buffer apart and would wait for the load before every LDS read; it has no
// output registers, and the kernel waits for it (wait_loads) before the barrier.
__device__ __forceinline__ void load_to_lds(const void* base, uint32_t offset, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(offset), "s"(base), "s"(lds)
                 : "memory", "m0");
}
// Waits until at most N loads are on their way.
template <int N = 0>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

typedef __attribute__((address_space(3))) unsigned char lds_byte;
__device__ __forceinline__ uint32_t lds_address(const unsigned char* p) {
    return uint32_t(reinterpret_cast<uintptr_t>((const lds_byte*)p));
}

// Transposing LDS read: within 16 lanes, lane g points at 4 neighbouring elements of row
// g / 4 of a 4 x 16 block, at column 4 (g % 4), and receives column g.
__device__ __forceinline__ uint2 read_turned(const unsigned char* p) {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
    return __builtin_bit_cast(
        uint2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(const_cast<unsigned char*>(p))));
}

__device__ __forceinline__ f32x4 mfma(f16x8 q, f16x8 p, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(q, p, c, 0, 0, 0);
}

__device__ __forceinline__ void store_pairs(_Float16* p, const float v[4]) {
    f16x4 hi, lo;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const Pair s = split(v[t]);
        hi[t] = s.hi, lo[t] = s.lo;
    }
    *reinterpret_cast<f16x4*>(p) = hi;
    *reinterpret_cast<f16x4*>(p + 32) = lo;
}

// Four neighbouring elements (i, j..j+3) of a matrix in the iteration's orientation to O in its
// own: o, rows x cols with out_row elements between rows.
template <typename T>
__device__ __forceinline__ void store_result(T* o, int64_t out_row, bool tall, int rows, int cols, int i,
                                             int j, const float v[4]) {
    if (tall) {
        // O's rows are the iterate's columns
        if (i < cols)
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (j + t < rows) store_one(o + int64_t(j + t) * out_row + i, v[t]);
    } else if (i < rows) {
        o += int64_t(i) * out_row + j;
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (j + t < cols) store_one(o + t, v[t]);
    }
}

}  // namespace

struct InArgs {
    const void* in;
    void* out;  // split with no steps: the result itself
    int64_t in_stride, in_row, out_stride, out_row;
    double* partial;  // [matrix][part_slots]
    _Float16* x;      // first iterate, [matrix][cp / 32][rp][64]
    int32_t rows, cols;
    int32_t rp, cp;
    int32_t parts, part_slots;  // partial sums of one matrix, and their room
    float scale;
    StackScale* scales;  // [matrix][kStackScales]
    StackPlan plan;
};
static_assert(sizeof(InArgs) + 256 <= 4096, "kernel arguments");

namespace {

// ||U|| of a matrix from its partial sums: every wave adds them by itself, in the same order.
__device__ __forceinline__ double matrix_norm(const double* partial, int parts) {
    double sum = 0.;
    for (int p = threadIdx.x & 63; p < parts; p += 64) sum += partial[p];
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    return sqrt(sum);
}
// 2^64 / (||U|| + 1e-7): without the 2^64, norms above 2^126 (of finite matrices) would make it a
// subnormal number and cost its digits.  U times it is 2^64 at most.  An infinite norm makes the whole
// matrix NaN, like a NaN does.
constexpr int kInverseUp = 64;
__device__ __forceinline__ float inverse_of(double norm) {
    return norm > 1.7e308 ? __uint_as_float(0x7fc00000u) : float(0x1p64 / (norm + 1e-7));
}
// The bound on the largest singular value of U / (||U|| + 1e-7) (a NaN: any will do).
__device__ __forceinline__ float first_bound(double norm) {
    return norm <= 1.7e308 ? 1.001f * float(norm / (norm + 1e-7)) : 1.f;
}

}  // namespace

// Shorter side up to 128: all steps, from the partial sums of squares on.  `count` matrices of the
// stack; gram0, gram1: room for rp * cp floats a matrix each.
hipError_t launch_stack_strips(const muon_stack_t& stack, const StackShape& s, int64_t count, const InArgs& in,
                               void* x, void* gram0, void* gram1, void* b, const StackPlan& plan, float scale,
                               hipStream_t stream);

}  // namespace muon
