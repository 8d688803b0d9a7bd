// Casts into 8-bit floats with a scale for each 1 x 128 or 128 x 128 block, of a
// matrix and of its transpose in one pass.
//
//   m = max(largest magnitude of the block, 2^-100),  s = fl(m / L),  code = rne8(x L / m)
//
// with L the format's largest number.  The code is that of the quotient itself.  L / m is held in two
// float32 (high and rest), so that y = x high + x rest is x L / m with one float32 rounding and before
// it an error below 2^-30 (2^-47 unless m is above 2^100).  Middles between codes are float32 numbers,
// and a quotient that is not one lies at least 2^-29 beside it (7 X and D M, integers of 27 and
// 29 bits, differ by one at least), so y is on the quotient's side of every middle or on the middle
// itself; where it is on it, x L and y m, both exact in float64, tell the side.  (Without that
// look 28 of 58.7 million float32 elements get the farther of two codes, with fl(x fl(1 / s)) 42;
// it costs 1% of the time.)
// Magnitudes are compared as bit patterns, in which a NaN is above infinity: a block that holds
// one gets the scale NaN.
//
// A workgroup takes a 128 x 128 tile, a thread an 8 x 8 block of it, held in
// registers: 16 neighbouring lanes read one row's 128 elements.  Row blocks
// reduce over these 16 lanes (DPP), column blocks over the 16 threads of a column
// group (lanes, then LDS).  Each block's divisions are made by one lane (of a row's 16, the
// row's; of the workgroup, the column's) and handed round.  The transposed codes go through LDS
// so that each row of the transpose leaves as 128 contiguous bytes.  It is an HBM stream: 14336 x
// 4096 float32 in 128 x 128 blocks, both ways, take 70 us (5.0 TB/s), one way 45 (6.5); 8192 x 4096 bfloat16
// in rows, both ways, 28 (4.8).
#include <type_traits>

#include "fp8_internal.h"
#include "k_common.h"

#pragma clang fp contract(off)

namespace muon {

namespace {

constexpr int kThreads = 256;

struct CastSide {
    uint8_t* codes;  // null: not asked for
    float* scales;
    int64_t row_stride, scale_row, scale_col;
};

struct CastArgs {
    const void* x;
    int64_t row_stride;
    int32_t rows, cols, col_tiles;
    CastSide out, out_t;
};

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

// Eight consecutive elements, of which the first `left` exist; the rest are 0.
__device__ __forceinline__ void load8(const float* p, int left, float v[8]) {
    if (left >= 8) {
        const f32x4_any a = *reinterpret_cast<const f32x4_any*>(p);
        const f32x4_any b = *reinterpret_cast<const f32x4_any*>(p + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < left ? p[j] : 0.f;
    }
}
__device__ __forceinline__ void load8(const uint16_t* p, int left, float v[8]) {
    if (left >= 8) {
        const u32x4_any a = *reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(a[j] << 16);
            v[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < left ? bf16_to_f32(p[j]) : 0.f;
    }
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Maximum over the 16 lanes of a DPP row, in all of them.
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x128, 0xF, 0xF, true)));
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x124, 0xF, 0xF, true)));
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x122, 0xF, 0xF, true)));
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x121, 0xF, 0xF, true)));
    return x;
}

// What a block's values are multiplied by: high + rest = L / m.
struct Factor {
    float high, rest;
    __device__ __forceinline__ float of(float x) const { return __builtin_fmaf(x, high, x * rest); }
};
template <bool E5M2>
constexpr float kTop = E5M2 ? 57344.f : 448.f;
__device__ __forceinline__ float held_max(uint32_t largest) {
    return __uint_as_float(max(largest, 27u << 23));  // 2^-100
}
template <bool E5M2>
__device__ __forceinline__ Factor factor_of(uint32_t largest, float* scale) {
    const float m = held_max(largest);
    const float top = kTop<E5M2>;
    *scale = m / top;
    float high = top / m;
    // not above L / m: a negative rest would turn -0 into 0
    if (__builtin_fmaf(-high, m, top) < 0.f) high = __uint_as_float(__float_as_uint(high) - 1);
    return {high, __builtin_fmaf(-high, m, top) / m};
}
// Lane n's value in all 16 lanes of its DPP row.
template <int N>
__device__ __forceinline__ float row_value(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x150 + N, 0xF, 0xF, true));
}

template <bool E5M2>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    int w = 0;
    if constexpr (E5M2) {
        w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
        w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
    } else {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    }
    return uint32_t(w);
}

// Eight codes.  EXACT: a y on a middle is looked at again.  Middles of normal codes have the bit below
// the code's last one and none behind it; of subnormal codes, which are rare, every y but 0 is looked
// at.  m(): the block's held_max, called by whole waves.  (bfloat16 x and m have 8 bits: a quotient
// that is no middle lies 2^-14 beside it at least, so y is never on one by rounding.)
template <bool E5M2, bool EXACT, typename M>
__device__ __forceinline__ uint2 encode8(const Factor& f, const float (&x)[8], M&& m) {
    constexpr int kBehind = E5M2 ? 11 : 12;  // shift that leaves that bit and those behind it
    constexpr uint32_t kNormal = (E5M2 ? 127 - 14 : 127 - 6) << 23;
    float y[8];
    uint32_t middle = ~0u, small = ~0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        y[j] = f.of(x[j]);
        if constexpr (EXACT) {
            const uint32_t bits = __float_as_uint(y[j]);
            middle = min(middle, (bits << kBehind) + 0x80000000u);
            small = min(small, (bits << 1) - 2);  // (0: the largest)
        }
    }
    if constexpr (EXACT) {
        if (__builtin_amdgcn_ballot_w64(middle == 0 || small < (kNormal << 1) - 2) != 0) {
            const double top = double(kTop<E5M2>), held = double(m());
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t bits = __float_as_uint(y[j]);
                const double exact = fabs(double(x[j]) * top), here = fabs(double(y[j]) * held);
                if (bits << (kBehind + 1) == 0 && y[j] != 0.f && exact != here)
                    y[j] = __uint_as_float(exact > here ? bits + 1 : bits - 1);
            }
        }
    }
    return {encode4<E5M2>(y[0], y[1], y[2], y[3]), encode4<E5M2>(y[4], y[5], y[6], y[7])};
}

// The first `left` of eight codes.
__device__ __forceinline__ void store8(uint8_t* p, int left, uint2 w) {
    if (left >= 8) {
        u32x2_any t = {w.x, w.y};
        *reinterpret_cast<u32x2_any*>(p) = t;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) p[j] = uint8_t((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
    }
}

// f(0), ..., f(7) with the number as a constant.
template <typename F>
__device__ __forceinline__ void for_eight(F&& f) {
    f(std::integral_constant<int, 0>{}), f(std::integral_constant<int, 1>{});
    f(std::integral_constant<int, 2>{}), f(std::integral_constant<int, 3>{});
    f(std::integral_constant<int, 4>{}), f(std::integral_constant<int, 5>{});
    f(std::integral_constant<int, 6>{}), f(std::integral_constant<int, 7>{});
}

template <typename T, bool SQUARE, bool E5M2>
__global__ __launch_bounds__(kThreads) void fp8_cast_kernel(const CastArgs a) {
    __shared__ uint32_t col_max[4][kFp8Block];
    __shared__ Factor factors[kFp8Block];
    __shared__ float held[kFp8Block];
    __shared__ uint2 turned[kFp8Block * 16];
    constexpr bool kExact = std::is_same_v<T, float>;
    const int tr = blockIdx.x / a.col_tiles, tc = blockIdx.x % a.col_tiles;
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;  // 8-column and 8-row group
    const int r0 = tr * kFp8Block + rg * 8, c0 = tc * kFp8Block + cg * 8;
    const int rows_left = a.rows - r0, cols_left = a.cols - c0;

    float v[8][8];
    const T* x = static_cast<const T*>(a.x) + int64_t(r0) * a.row_stride + c0;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        if (p < rows_left)
            load8(x + p * a.row_stride, cols_left, v[p]);
        else
#pragma unroll
            for (int j = 0; j < 8; ++j) v[p][j] = 0.f;
    }

    Factor all = {0.f, 0.f};
    float all_held = 0.f;
    if constexpr (SQUARE) {
        uint32_t top = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p)
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max(top, magnitude(v[p][j]));
        top = row_max(top);
        if (cg == 0) col_max[0][rg] = top;
        __syncthreads();
        float scale;
        top = row_max(col_max[0][cg]);
        all = factor_of<E5M2>(top, &scale), all_held = held_max(top);
        if (threadIdx.x == 0) {
            if (a.out.codes != nullptr)
                a.out.scales[tr * a.out.scale_row + tc * a.out.scale_col] = scale;
            if (a.out_t.codes != nullptr)
                a.out_t.scales[tc * a.out_t.scale_row + tr * a.out_t.scale_col] = scale;
        }
    }

    if (a.out.codes != nullptr) {
        float scale = 0.f;
        Factor mine = {0.f, 0.f};  // of row cg % 8 of this thread's 8
        float mine_held = 0.f;
        if constexpr (!SQUARE) {
            uint32_t my_top = 0;
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) top = max(top, magnitude(v[p][j]));
                top = row_max(top);
                if ((cg & 7) == p) my_top = top;
            }
            mine = factor_of<E5M2>(my_top, &scale), mine_held = held_max(my_top);
            if (cg < rows_left && cg < 8)
                a.out.scales[(r0 + cg) * a.out.scale_row + tc * a.out.scale_col] = scale;
        }
        uint8_t* q = a.out.codes + int64_t(r0) * a.out.row_stride + c0;
        for_eight([&](auto index) {
            constexpr int p = decltype(index)::value;
            const Factor f = SQUARE ? all : Factor{row_value<p>(mine.high), row_value<p>(mine.rest)};
            const uint2 w = encode8<E5M2, kExact>(f, v[p], [&] { return SQUARE ? all_held : row_value<p>(mine_held); });
            if (p < rows_left) store8(q + p * a.out.row_stride, cols_left, w);
        });
    }

    if (a.out_t.codes == nullptr) return;
    if constexpr (!SQUARE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t top = 0;
#pragma unroll
            for (int p = 0; p < 8; ++p) top = max(top, magnitude(v[p][j]));
            top = max(top, uint32_t(__shfl_xor(int(top), 16)));
            top = max(top, uint32_t(__shfl_xor(int(top), 32)));
            if ((threadIdx.x & 63) < 16) col_max[threadIdx.x >> 6][cg * 8 + j] = top;
        }
        __syncthreads();
        if (threadIdx.x < kFp8Block) {
            const int c = threadIdx.x, col = tc * kFp8Block + c;
            float scale;
            const uint32_t top = max(max(col_max[0][c], col_max[1][c]), max(col_max[2][c], col_max[3][c]));
            factors[c] = factor_of<E5M2>(top, &scale), held[c] = held_max(top);
            if (col < a.cols) a.out_t.scales[col * a.out_t.scale_row + tr * a.out_t.scale_col] = scale;
        }
        __syncthreads();
    }
    // 8-byte chunk (column c, rows of group g) lies at c * 16 + (g ^ (c / 8)): lanes that write
    // together meet 16 different chunks
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const Factor f = SQUARE ? all : factors[cg * 8 + j];
        const float column[8] = {v[0][j], v[1][j], v[2][j], v[3][j], v[4][j], v[5][j], v[6][j], v[7][j]};
        turned[(cg * 8 + j) * 16 + (rg ^ cg)] =
            encode8<E5M2, kExact>(f, column, [&] { return SQUARE ? all_held : held[cg * 8 + j]; });
    }
    __syncthreads();
    const int left = a.rows - tr * kFp8Block - cg * 8;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int c = p * 16 + rg;
        const int col = tc * kFp8Block + c;
        if (col < a.cols)
            store8(a.out_t.codes + int64_t(col) * a.out_t.row_stride + tr * kFp8Block + cg * 8, left,
                   turned[c * 16 + (cg ^ (c >> 3))]);
    }
}

CastSide side_of(const muon_fp8_t* m) {
    if (m == nullptr) return {nullptr, nullptr, 0, 0, 0};
    return {static_cast<uint8_t*>(m->codes), m->scales, m->row_stride, m->scale_row, m->scale_col};
}

template <typename T>
void enqueue(const CastArgs& a, int64_t tiles, bool square, bool e5m2, hipStream_t s) {
    const dim3 grid = dim3(unsigned(tiles)), block = dim3(kThreads);
    if (square)
        e5m2 ? fp8_cast_kernel<T, true, true><<<grid, block, 0, s>>>(a)
             : fp8_cast_kernel<T, true, false><<<grid, block, 0, s>>>(a);
    else
        e5m2 ? fp8_cast_kernel<T, false, true><<<grid, block, 0, s>>>(a)
             : fp8_cast_kernel<T, false, false><<<grid, block, 0, s>>>(a);
}

}  // namespace

hipError_t launch_fp8_cast(const void* x, int dtype, int64_t rows, int64_t cols, int64_t row_stride,
                           const muon_fp8_t* out, const muon_fp8_t* out_t, hipStream_t s) {
    const muon_fp8_t& any = out != nullptr ? *out : *out_t;
    CastArgs a;
    a.x = x, a.row_stride = row_stride;
    a.rows = int32_t(rows), a.cols = int32_t(cols);
    a.col_tiles = int32_t(fp8_blocks(cols));
    a.out = side_of(out), a.out_t = side_of(out_t);
    // at most 2^21: rows * cols <= 2^34 and both sides <= 2^24
    const int64_t tiles = fp8_blocks(rows) * a.col_tiles;
    LaunchTimer timer("fp8_cast", s);
    if (dtype == MUON_DTYPE_BF16)
        enqueue<uint16_t>(a, tiles, any.block_rows != 1, any.format == MUON_FP8_E5M2, s);
    else
        enqueue<float>(a, tiles, any.block_rows != 1, any.format == MUON_FP8_E5M2, s);
    return hipGetLastError();
}

}  // namespace muon
