// Products of 8-bit matrices with a scale for each block of 128 along k.
//
//   out[i, j] (+)= sum over blocks kb of  sa[i, kb] sb[j, kb] sum over k in kb of a[i, k] b[j, k]
//
// The inner sums run on the matrix cores, the outer one in float32 on the vector
// unit: each block's result is multiplied by its two scales and added.  The
// instruction's operands are b's rows and then a's, so that a lane holds four
// neighbouring columns of one row of out.
//
// Two kinds of inner sum, by the type of out.  For bfloat16, one
// v_mfma_f32_16x16x128_f8f6f4 is a block of 128 of a 16 x 16 tile.  That
// instruction adds the products of 8 neighbouring elements after cutting each at 2^-13
// of the largest of the 8 (measured: of 2^16 + 2^2 the second term is lost, of 2^16 + 2^3
// not, within a group of 8 only): 1.5e-5 relative over Gaussian operands, 100 times below
// the rounding of out to bfloat16 (1.7e-3), but not float32.  For float32 the codes
// are widened to bfloat16, which is exact, and four v_mfma_f32_16x16x32_bf16 sum
// the block in float32 (6e-8 over the same operands), at half the rate.
#include "fp8_internal.h"
#include "k_common.h"

namespace muon {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));

struct Operand {
    const uint8_t* codes;
    const float* scales;
    int64_t row_stride, scale_row, scale_col;
    int32_t rows;
    int32_t shift;  // row >> shift is its row of blocks: 0 or 7
};

struct ProductArgs {
    Operand a, b;
    void* out;
    int64_t out_row;
    int32_t k;
    int32_t tiles_m, tiles_n;
    int32_t out_bf16, accumulate;
};

// 16 bytes of a row of codes from byte `at` on, those from byte k on as zeros.
__device__ __forceinline__ i32x4 load_chunk(const uint8_t* row, int at, int k) {
    if (at + 16 <= k) return i32x4(*reinterpret_cast<const u32x4_any*>(row + at));
    i32x4 w = {0, 0, 0, 0};
    for (int j = 0; j < 16; ++j)
        if (at + j < k) {
            const int byte = int(uint32_t(row[at + j]) << (8 * (j & 3)));
            w.x |= j < 4 ? byte : 0;
            w.y |= (j >> 2) == 1 ? byte : 0;
            w.z |= (j >> 2) == 2 ? byte : 0;
            w.w |= j >= 12 ? byte : 0;
        }
    return w;
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight codes (two words) as bfloat16; F: the format's number in the instructions (0: e4m3,
// 1: e5m2).
template <int F>
__device__ __forceinline__ bf16x8 widen8(uint32_t lo, uint32_t hi) {
    bf16x2 w[4];
    if constexpr (F == 0) {
        w[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false);
        w[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
        w[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false);
        w[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
    } else {
        w[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.f, false);
        w[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.f, true);
        w[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.f, false);
        w[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.f, true);
    }
    return {w[0].x, w[0].y, w[1].x, w[1].y, w[2].x, w[2].y, w[3].x, w[3].y};
}

// One 16 x 16 product over a block of 128.
template <int FA, int FB, bool EXACT>
__device__ __forceinline__ f32x4 block_product(const i32x8& a, const i32x8& b) {
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    if constexpr (EXACT) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<FA>(a[2 * t], a[2 * t + 1]),
                                                          widen8<FB>(b[2 * t], b[2 * t + 1]), sum, 0, 0, 0);
        return sum;
    } else {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, sum, FA, FB, 0, 0, 0, 0);
    }
}

__device__ __forceinline__ i32x8 join(i32x4 lo, i32x4 hi) {
    return {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
}

// Four neighbouring results of row i, from column j on.
__device__ __forceinline__ void store_result(const ProductArgs& g, int i, int j, f32x4 v) {
    if (i >= g.a.rows || j >= g.b.rows) return;
    const int left = g.b.rows - j;
    if (g.out_bf16) {
        uint16_t* p = static_cast<uint16_t*>(g.out) + int64_t(i) * g.out_row + j;
        const uint16_t h[4] = {bf16_rne(v.x), bf16_rne(v.y), bf16_rne(v.z), bf16_rne(v.w)};
        if (left >= 4) {
            u32x2_any w = {uint32_t(h[0]) | uint32_t(h[1]) << 16, uint32_t(h[2]) | uint32_t(h[3]) << 16};
            *reinterpret_cast<u32x2_any*>(p) = w;
        } else {
#pragma unroll
            for (int t = 0; t < 3; ++t)
                if (t < left) p[t] = h[t];
        }
    } else {
        float* p = static_cast<float*>(g.out) + int64_t(i) * g.out_row + j;
        if (left >= 4) {
            f32x4_any w = v;
            if (g.accumulate) w += *reinterpret_cast<const f32x4_any*>(p);
            *reinterpret_cast<f32x4_any*>(p) = w;
        } else {
#pragma unroll
            for (int t = 0; t < 3; ++t)
                if (t < left) p[t] = g.accumulate ? v[t] + p[t] : v[t];
        }
    }
}

// Any alignment and length: 128 x 128 tiles, operands through registers into
// double-buffered LDS.  Row r's 16-byte chunk c lies at chunk c ^ (r / 2 mod 8), so that the
// fragment reads of 16 rows meet every bank.
constexpr int kTile = 128;
constexpr int kOpBytes = kTile * kFp8Block;

template <int FA, int FB, bool EXACT>
__global__ __launch_bounds__(256) void fp8_any_kernel(const ProductArgs g) {
    __shared__ __attribute__((aligned(16))) unsigned char lds[2][2 * kOpBytes];
    __shared__ __attribute__((aligned(16))) float scales[2][2 * kTile];
    const int m0 = blockIdx.x / g.tiles_n * kTile, n0 = blockIdx.x % g.tiles_n * kTile;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;

    // this thread's chunks: rows tid / 8 + 32 p, chunk tid % 8; rows behind the last read the last
    const int chunk = tid & 7;
    const uint8_t *pa[4], *pb[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int r = (tid >> 3) + 32 * p;
        pa[p] = g.a.codes + int64_t(min(m0 + r, g.a.rows - 1)) * g.a.row_stride;
        pb[p] = g.b.codes + int64_t(min(n0 + r, g.b.rows - 1)) * g.b.row_stride;
    }
    const float* ps;
    int64_t ps_step;
    {
        const Operand& o = tid < kTile ? g.a : g.b;
        const int r = min((tid < kTile ? m0 : n0) + (tid & (kTile - 1)), o.rows - 1);
        ps = o.scales + int64_t(r >> o.shift) * o.scale_row;
        ps_step = o.scale_col;
    }

    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = {0.f, 0.f, 0.f, 0.f};

    i32x4 ra[4], rb[4];
    float rs;
    auto fetch = [&](int kb) {
        const int at = kb * kFp8Block + chunk * 16;
#pragma unroll
        for (int p = 0; p < 4; ++p) ra[p] = load_chunk(pa[p], at, g.k), rb[p] = load_chunk(pb[p], at, g.k);
        rs = ps[kb * ps_step];
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int r = (tid >> 3) + 32 * p;
            const int at = r * kFp8Block + ((chunk ^ ((r >> 1) & 7)) << 4);
            *reinterpret_cast<i32x4*>(&lds[buf][at]) = ra[p];
            *reinterpret_cast<i32x4*>(&lds[buf][kOpBytes + at]) = rb[p];
        }
        scales[buf][tid] = rs;
    };
    auto fragment = [&](const unsigned char* op, int row0) {
        const int r = row0 + (lane & 15), q = lane >> 4, x = (r >> 1) & 7;
        return join(*reinterpret_cast<const i32x4*>(op + r * kFp8Block + ((q ^ x) << 4)),
                    *reinterpret_cast<const i32x4*>(op + r * kFp8Block + (((q + 4) ^ x) << 4)));
    };

    const int nk = (g.k + kFp8Block - 1) / kFp8Block;
    fetch(0);
    put(0);
    __syncthreads();
    for (int kb = 0; kb < nk; ++kb) {
        const int buf = kb & 1;
        if (kb + 1 < nk) fetch(kb + 1);
        i32x8 fb[4];
        f32x4 sb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            fb[j] = fragment(lds[buf] + kOpBytes, wn + 16 * j);
            sb[j] = *reinterpret_cast<const f32x4*>(&scales[buf][kTile + wn + 16 * j + 4 * (lane >> 4)]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const i32x8 fa = fragment(lds[buf], wm + 16 * i);
            const float sa = scales[buf][wm + 16 * i + (lane & 15)];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] += block_product<FB, FA, EXACT>(fb[j], fa) * (sb[j] * sa);
        }
        if (kb + 1 < nk) put(buf ^ 1);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            store_result(g, m0 + wm + 16 * i + (lane & 15), n0 + wn + 16 * j + 4 * (lane >> 4), acc[i][j]);
}

// out of k = 0: zeros.
__global__ __launch_bounds__(256) void fp8_zero_kernel(const ProductArgs g) {
    const int64_t groups = int64_t(g.a.rows) * ((g.b.rows + 3) / 4);
    for (int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x; t < groups; t += int64_t(gridDim.x) * 256) {
        const int per = (g.b.rows + 3) / 4;
        store_result(g, int(t / per), int(t % per) * 4, f32x4{0.f, 0.f, 0.f, 0.f});
    }
}

Operand operand_of(const muon_fp8_t& m) {
    return {static_cast<const uint8_t*>(m.codes), m.scales, m.row_stride, m.scale_row, m.scale_col,
            int32_t(m.rows), m.block_rows == 1 ? 0 : 7};
}

template <int FA, int FB>
hipError_t enqueue(ProductArgs g, hipStream_t s) {
    LaunchTimer timer("fp8_matmul", s);
    g.tiles_m = (g.a.rows + kTile - 1) / kTile, g.tiles_n = (g.b.rows + kTile - 1) / kTile;
    const dim3 grid = dim3(unsigned(int64_t(g.tiles_m) * g.tiles_n));
    g.out_bf16 ? fp8_any_kernel<FA, FB, false><<<grid, dim3(256), 0, s>>>(g)
               : fp8_any_kernel<FA, FB, true><<<grid, dim3(256), 0, s>>>(g);
    return hipGetLastError();
}

}  // namespace

size_t fp8_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_fp8_matmul(const muon_fp8_t& a, const muon_fp8_t& b, void* out, int out_dtype,
                             int64_t out_row_stride, bool accumulate, void*, hipStream_t s) {
    ProductArgs g{};
    g.a = operand_of(a), g.b = operand_of(b);
    g.out = out, g.out_row = out_row_stride, g.k = int32_t(a.cols);
    g.out_bf16 = out_dtype == MUON_DTYPE_BF16, g.accumulate = accumulate;
    if (g.k == 0) {
        if (accumulate) return hipSuccess;
        LaunchTimer timer("fp8_matmul", s);
        fp8_zero_kernel<<<dim3(1024), dim3(256), 0, s>>>(g);
        return hipGetLastError();
    }
    if (a.format == MUON_FP8_E5M2)
        return b.format == MUON_FP8_E5M2 ? enqueue<1, 1>(g, s) : enqueue<1, 0>(g, s);
    return b.format == MUON_FP8_E5M2 ? enqueue<0, 1>(g, s) : enqueue<0, 0>(g, s);
}

}  // namespace muon
