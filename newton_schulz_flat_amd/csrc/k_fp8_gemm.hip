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
#include <algorithm>
#include <cmath>
#include <type_traits>

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
    float* partial;  // [split][m][n] where the blocks of k are split, else null
    int32_t k;
    int32_t tiles_m, tiles_n;
    int32_t splits, per_split;  // of the blocks of k
    int32_t out_bf16, accumulate;
};

// 16 bytes of a row of codes from byte `at` on, those from byte k on as zeros.  At the end of
// a row its last 16 bytes are read and shifted, so that nothing behind it is touched.
__device__ __forceinline__ i32x4 load_chunk(const uint8_t* row, int at, int k) {
    if (at + 16 <= k) return i32x4(*reinterpret_cast<const u32x4_any*>(row + at));
    if (at >= k) return {0, 0, 0, 0};
    uint64_t lo = 0, hi = 0;
    if (k >= 16) {
        const u32x4_any t = *reinterpret_cast<const u32x4_any*>(row + k - 16);
        lo = t.x | uint64_t(t.y) << 32, hi = t.z | uint64_t(t.w) << 32;
        int drop = 8 * (at + 16 - k);  // bits, 8 to 120
        if (drop >= 64) lo = hi, hi = 0, drop -= 64;
        if (drop > 0) lo = lo >> drop | hi << (64 - drop), hi >>= drop;
    } else {
#pragma unroll 1
        for (int j = k - 1; j >= at; --j) hi = hi << 8 | lo >> 56, lo = lo << 8 | row[j];
    }
    return {int(uint32_t(lo)), int(lo >> 32), int(uint32_t(hi)), int(hi >> 32)};
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

// A lane's 32 codes of one row and block, as the inner sum takes them.
template <int F, bool EXACT>
struct Wide {
    std::conditional_t<EXACT, bf16x8[4], i32x8> v;
    __device__ __forceinline__ void set(const i32x8& codes) {
        if constexpr (EXACT) {
#pragma unroll
            for (int t = 0; t < 4; ++t) v[t] = widen8<F>(codes[2 * t], codes[2 * t + 1]);
        } else {
            v = codes;
        }
    }
};

// N 16 x 16 products over a block of 128.
template <int N, int FA, int FB, bool EXACT>
__device__ __forceinline__ void block_products(const Wide<FA, EXACT>* a, const Wide<FB, EXACT>& b, f32x4* sum) {
#pragma unroll
    for (int q = 0; q < N; ++q) sum[q] = {0.f, 0.f, 0.f, 0.f};
    if constexpr (EXACT) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int q = 0; q < N; ++q)
                sum[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[q].v[t], b.v[t], sum[q], 0, 0, 0);
    } else {
#pragma unroll
        for (int q = 0; q < N; ++q)
            sum[q] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[q].v, b.v, sum[q], FA, FB, 0, 0, 0, 0);
    }
}

__device__ __forceinline__ i32x8 join(i32x4 lo, i32x4 hi) {
    return {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
}

// A sum is multiplied by the product p of its two scales.  p leaves float32's normal numbers where both
// scales are very small or very large, which the result, the sum times both, need not do; such elements
// take the scales by parts.  Two multiplications a sum would do for most of them, but not all, and the
// vector unit is half of what bounds a tile: instead a tile looks at its scales as they pass (8192 x 14336
// over 4096 into bfloat16 within 1%, into float32 801 us to 819) and is made again where it has to be.
__device__ __forceinline__ bool is_normal(float p) { return __builtin_amdgcn_classf(p, 0x108); }
// A scale's mantissa (0.5 to 1; a zero, an infinity or a NaN itself) and exponent.
struct Parts {
    float mantissa;
    int exponent;
    __device__ __forceinline__ explicit Parts(float s)
        : mantissa(__builtin_amdgcn_frexp_mantf(s)), exponent(__builtin_amdgcn_frexp_expf(s)) {}
};
// acc + sum * a's scale * b's: the same bits as sum * p + acc where p is a normal number, else rounded
// once more.  (A sum of zero stays away from an infinite product of finite scales.)
__device__ __forceinline__ float add_by_parts(float acc, float sum, float sa, float sb) {
    const float p = sb * sa;
    if (is_normal(p)) return __builtin_fmaf(sum, p, acc);
    const Parts a(sa), b(sb);
    return acc + __builtin_ldexpf(sum * (a.mantissa * b.mantissa), a.exponent + b.exponent);
}

// Four neighbouring results of row i, from column j on; of one split of k where there are several.
__device__ __forceinline__ void store_result(const ProductArgs& g, int split, int i, int j, f32x4 v) {
    if (i >= g.a.rows || j >= g.b.rows) return;
    const int left = g.b.rows - j;
    if (g.partial != nullptr) {
        float* p = g.partial + (int64_t(split) * g.a.rows + i) * g.b.rows + j;
        if (left >= 4) {
            *reinterpret_cast<f32x4_any*>(p) = v;
        } else {
#pragma unroll
            for (int t = 0; t < 3; ++t)
                if (t < left) p[t] = v[t];
        }
    } else if (g.out_bf16) {
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

// ------------------------------------------------------------------- tiles

template <int TILE>
struct Geo {
    static constexpr int kWaves = TILE == 256 ? 8 : 4;
    static constexpr int kThreads = kWaves * 64;
    static constexpr int kWm = TILE / 2, kWn = TILE / (kWaves / 2);  // of a wave
    static constexpr int kMi = kWm / 16, kNj = kWn / 16;
    static constexpr int kOp = TILE * kFp8Block;          // bytes of one operand's block
    static constexpr int kLoads = kOp / (kThreads * 16);  // 16-byte loads of a thread
    // Direct loads go as many blocks ahead as LDS has stages (less one), loads through registers as
    // many as there are sets of them: a 64-tile's block is too short to cover a load.
    static constexpr int kStages = TILE == 64 ? 4 : 2, kSets = TILE == 64 ? 2 : 1;
    static constexpr int kScales = TILE == 64 ? kThreads : 2 * TILE;  // one of a thread
};

// 16 bytes to LDS at lds + 16 * lane from base + offset, or 4 bytes at lds + 4 * lane from p,
// without passing through registers.  Written as assembly because the compiler
// cannot tell the two halves of the double buffer apart and would wait for the load
// before every LDS read; it has no output registers, and the kernel waits for it
// (wait_loads) before the barrier.
__device__ __forceinline__ void load16_to_lds(const void* base, uint32_t offset, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(offset), "s"(base), "s"(lds)
                 : "memory", "m0");
}
__device__ __forceinline__ void load16_to_lds(const void* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :
                 : "v"(p), "s"(lds)
                 : "memory", "m0");
}
__device__ __forceinline__ void load4_to_lds(const void* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
                 :
                 : "v"(p), "s"(lds)
                 : "memory", "m0");
}
// Waits until at most N loads are on their way.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

typedef __attribute__((address_space(3))) unsigned char lds_byte;
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return uint32_t(reinterpret_cast<uintptr_t>((const lds_byte*)p));
}

// What lies behind the last column of a row of codes.
__device__ const uint32_t zeros[4] = {0, 0, 0, 0};

// The tile of workgroup b of `tiles`: workgroups go to the 8 XCDs in turn, and each XCD
// takes a contiguous run of tiles, in bands of 4 tile rows, column by column, so that
// the 32 tiles it works on at once share 12 panels of a and b in its L2.
__device__ __forceinline__ void tile_of(int b, int tiles_m, int tiles_n, int& ti, int& tj) {
    const int tiles = tiles_m * tiles_n, x = b & 7, low = tiles >> 3, more = tiles & 7;
    const int t = x * low + min(x, more) + (b >> 3);
    const int band = t / (4 * tiles_n), rest = t - band * 4 * tiles_n;
    const int high = min(4, tiles_m - band * 4);
    ti = band * 4 + rest % high, tj = rest / high;
}

// Scales from 2^-63 to 2^63, of which no product of two leaves the normal numbers.
__device__ __forceinline__ bool is_plain(float scale) {
    return (__float_as_uint(scale) << 1) - (64u << 24) < (126u << 24);
}
// The least (but zeros) and the largest finite one of the scales of a row.
struct Sizes {
    uint32_t least = (255u << 23) - 1, most = 0;  // bits; least: less one, so that zeros are the largest
    __device__ __forceinline__ void meet(float scale) {
        const uint32_t bits = __float_as_uint(scale) & 0x7fffffffu;
        least = min(least, bits - 1), most = max(most, bits < 255u << 23 ? bits : 0u);
    }
};
// No product of a scale of a and one of b leaves the normal numbers, by the sizes of a tile's scales: the
// first half of every `rows` threads has those of a's rows.  The same in all threads.
template <int WAVES>
__device__ __forceinline__ bool products_are_normal(const Sizes& s, uint2* met, int rows) {
    uint32_t least = s.least, most = s.most;
    for (int d = 32; d > 0; d >>= 1) {
        least = min(least, uint32_t(__shfl_xor(int(least), d)));
        most = max(most, uint32_t(__shfl_xor(int(most), d)));
    }
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if ((threadIdx.x & 63) == 0) met[wave] = {least, most};
    __syncthreads();
    uint2 a = {(255u << 23) - 1, 0}, b = a;
    for (int w = 0; w < WAVES; ++w) {
        uint2& o = (w * 64 & (rows - 1)) < rows / 2 ? a : b;
        o.x = min(o.x, met[w].x), o.y = max(o.y, met[w].y);
    }
    __syncthreads();
    const float low = __uint_as_float(a.x + 1) * __uint_as_float(b.x + 1);
    const float high = __uint_as_float(a.y) * __uint_as_float(b.y);
    return __builtin_amdgcn_ballot_w64(!(low >= 0x1p-126f && high <= 3.4028235e38f)) == 0;
}

// A wave's MI x NJ tiles of 16 x 16 with their scales by parts, from row m0 of a and n0 of b on, one after the
// other and straight from memory: what a tile is made of again where products of its scales leave the normal
// numbers.  Rolled, and a tile at a time: what it holds, the main loop cannot (256-tiles with widened codes keep 8
// bytes in scratch across their loop as it is, unaligned 128-tiles 16).  It is 10 to 20 times slower
// (8192 x 14336 over 4096 with all scales near 2^-70: 11 ms), for products that are otherwise lost.
template <int MI, int NJ, int FA, int FB, bool EXACT>
__device__ __forceinline__ void tiles_by_parts(const ProductArgs& g, int split, int m0, int n0, int first, int last) {
    const int lane = threadIdx.x & 63, q = lane >> 4;
#pragma unroll 1
    for (int tile = 0; tile < MI * NJ; ++tile) {
        const int m = m0 + tile / NJ * 16, n = n0 + tile % NJ * 16;
        const int ar = min(m + (lane & 15), g.a.rows - 1), br = min(n + (lane & 15), g.b.rows - 1);
        const uint8_t* pa = g.a.codes + int64_t(ar) * g.a.row_stride;
        const uint8_t* pb = g.b.codes + int64_t(br) * g.b.row_stride;
        const float* sa = g.a.scales + int64_t(ar >> g.a.shift) * g.a.scale_row;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int kb = first; kb < last; ++kb) {
            const int at = kb * kFp8Block + q * 16;
            Wide<FA, EXACT> wa;
            Wide<FB, EXACT> wb;
            wa.set(join(load_chunk(pa, at, g.k), load_chunk(pa, at + 64, g.k)));
            wb.set(join(load_chunk(pb, at, g.k), load_chunk(pb, at + 64, g.k)));
            f32x4 sum;
            block_products<1>(&wb, wa, &sum);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int r = min(n + 4 * q + t, g.b.rows - 1) >> g.b.shift;
                acc[t] = add_by_parts(acc[t], sum[t], sa[kb * g.a.scale_col],
                                      g.b.scales[int64_t(r) * g.b.scale_row + kb * g.b.scale_col]);
            }
        }
        store_result(g, split, m + (lane & 15), n + 4 * q, acc);
    }
}

// One TILE x TILE tile of out over a range of blocks of k.  Row r's 16-byte chunk c lies at
// chunk c ^ (r / 2 mod 8), so that the fragment reads of 16 rows meet every bank.  DIRECT (rows of codes that start at multiples of 16
// bytes and hold a multiple of 16): loads go from memory to LDS directly; else through
// registers, by bytes at the end of a row.  Rows behind the last one read the last.
// SQUARE: b's blocks are 128 x 128, and a wave's columns (64 or fewer, within 128) share one
// scale.
// What bounds it (8192 x 14336 over 4096 into bfloat16, 450 to 500 us by machine, 1.9 to 2.1 PFLOP/s): matrix
// instructions are busy 44% of the cycles, the vector unit 41%, with little of one beside the other. Of 470 us,
// 395 were left without the scaling, 313 without the matrix instructions, 395 without loads.
template <int TILE, bool DIRECT, int FA, int FB, bool EXACT, bool SQUARE>
__global__ __launch_bounds__(Geo<TILE>::kThreads, 2) void fp8_tile_kernel(const ProductArgs g) {
    using G = Geo<TILE>;
    constexpr int kStages = DIRECT ? G::kStages : 2;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[kStages][2 * G::kOp];
    __shared__ __attribute__((aligned(16))) float scales[kStages][G::kScales];
    __shared__ int not_plain[G::kWaves];
    __shared__ uint2 met[G::kWaves];
    const int tiles = g.tiles_m * g.tiles_n;
    const int split = blockIdx.x / tiles;
    int ti, tj;
    tile_of(blockIdx.x - split * tiles, g.tiles_m, g.tiles_n, ti, tj);
    const int m0 = ti * TILE, n0 = tj * TILE;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = (wave / (G::kWaves / 2)) * G::kWm, wn = (wave % (G::kWaves / 2)) * G::kWn;
    const int nk = (g.k + kFp8Block - 1) / kFp8Block;
    const int first = split * g.per_split, last = min(nk, first + g.per_split);

    // chunk tid % 8 of rows tid / 8 + p * rows of a pass (a multiple of 16: the swizzle is the
    // same in every pass); direct loads put their chunks one behind the other, so they
    // fetch the chunk that belongs there
    constexpr int kRows = G::kThreads / 8;
    const int lr = tid >> 3, x = (lr >> 1) & 7;
    const int chunk = DIRECT ? (tid & 7) ^ x : tid & 7;
    const uint8_t* a_base = g.a.codes + int64_t(m0) * g.a.row_stride;
    const uint8_t* b_base = g.b.codes + int64_t(n0) * g.b.row_stride;
    const auto a_row = [&](int p) { return min(lr + p * kRows, g.a.rows - 1 - m0); };
    const auto b_row = [&](int p) { return min(lr + p * kRows, g.b.rows - 1 - n0); };

    // the scales of a block: a's by the first TILE threads of 2 TILE, b's by the others (of a
    // 64-tile's 256 threads two waves load them once more, so that every wave has as many loads)
    const float* ps;
    int64_t ps_step;
    {
        const int t = tid & (2 * TILE - 1);
        const Operand& o = t < TILE ? g.a : g.b;
        const int r = min((t < TILE ? m0 : n0) + (t & (TILE - 1)), o.rows - 1);
        ps = o.scales + int64_t(r >> o.shift) * o.scale_row;
        ps_step = o.scale_col;
    }

    uint32_t a_off[G::kLoads], b_off[G::kLoads];
    i32x4 ra[G::kSets][G::kLoads], rb[G::kSets][G::kLoads];
    float rs[G::kSets];
    if constexpr (DIRECT) {
#pragma unroll
        for (int p = 0; p < G::kLoads; ++p) {
            a_off[p] = uint32_t(a_row(p)) * uint32_t(g.a.row_stride) + chunk * 16;
            b_off[p] = uint32_t(b_row(p)) * uint32_t(g.b.row_stride) + chunk * 16;
        }
    }
    const uint32_t lds0 = lds_address(lds), scales0 = lds_address(scales);
    // starts the loads of block kb: DIRECT into a stage, else into a set of registers
    auto fetch = [&](int kb, int to_stage, auto set) {
        const int at = kb * kFp8Block;
        if constexpr (DIRECT) {
            const uint32_t to = lds0 + to_stage * 2 * G::kOp + wave * 1024;
            if (at + kFp8Block <= g.k) {
#pragma unroll
                for (int p = 0; p < G::kLoads; ++p) {
                    load16_to_lds(a_base + at, a_off[p], to + p * G::kThreads * 16);
                    load16_to_lds(b_base + at, b_off[p], to + G::kOp + p * G::kThreads * 16);
                }
            } else {
                const bool there = at + chunk * 16 < g.k;
#pragma unroll
                for (int p = 0; p < G::kLoads; ++p) {
                    load16_to_lds(there ? a_base + at + a_off[p] : reinterpret_cast<const uint8_t*>(zeros),
                                  to + p * G::kThreads * 16);
                    load16_to_lds(there ? b_base + at + b_off[p] : reinterpret_cast<const uint8_t*>(zeros),
                                  to + G::kOp + p * G::kThreads * 16);
                }
            }
            load4_to_lds(ps + kb * ps_step, scales0 + to_stage * G::kScales * 4 + wave * 256);
        } else {
            constexpr int kSet = decltype(set)::value;
#pragma unroll
            for (int p = 0; p < G::kLoads; ++p) {
                ra[kSet][p] = load_chunk(a_base + a_row(p) * g.a.row_stride, at + chunk * 16, g.k);
                rb[kSet][p] = load_chunk(b_base + b_row(p) * g.b.row_stride, at + chunk * 16, g.k);
            }
            rs[kSet] = ps[kb * ps_step];
        }
    };
    uint64_t others = 0;  // lanes that met scales that are not plain
    auto put = [&](int to_stage, auto set) {
        if constexpr (!DIRECT) {
            constexpr int kSet = decltype(set)::value;
#pragma unroll
            for (int p = 0; p < G::kLoads; ++p) {
                const int at = (lr + p * kRows) * kFp8Block + ((chunk ^ x) << 4);
                *reinterpret_cast<i32x4*>(&lds[to_stage][at]) = ra[kSet][p];
                *reinterpret_cast<i32x4*>(&lds[to_stage][G::kOp + at]) = rb[kSet][p];
            }
            scales[to_stage][tid] = rs[kSet];
            others |= __builtin_amdgcn_ballot_w64(!is_plain(rs[kSet]));
        }
    };
    auto fragment = [&](const unsigned char* op, int row0) {
        const int r = row0 + (lane & 15), q = lane >> 4, y = (r >> 1) & 7;
        return join(*reinterpret_cast<const i32x4*>(op + r * kFp8Block + ((q ^ y) << 4)),
                    *reinterpret_cast<const i32x4*>(op + r * kFp8Block + (((q + 4) ^ y) << 4)));
    };

    f32x4 acc[G::kMi][G::kNj];
#pragma unroll
    for (int i = 0; i < G::kMi; ++i)
#pragma unroll
        for (int j = 0; j < G::kNj; ++j) acc[i][j] = {0.f, 0.f, 0.f, 0.f};

    int stage = 0, ahead = kStages - 1;
    // DEALT: a's and b's loads of the next block, a whole one, among the products: issued all at once
    // they hold up the first of these (8192 x 14336 over 4096 484 us to 464, 600 x 2048 over 7168 25.3 to
    // 24.6; of 256-tiles those with more registers at work lose 1 to 3%)
    constexpr bool kDeals = DIRECT && kStages == 2 && (TILE == 128 || (SQUARE && !EXACT));
    auto step = [&](int kb, auto set, auto dealt) {
        constexpr bool kDealt = decltype(dealt)::value;
        if constexpr (DIRECT)
            wait_loads<(kStages - 2) * (2 * G::kLoads + 1)>();
        else
            put(stage, set);
        __syncthreads();
        const int buf = stage;
        // a's first rows before b's: LDS returns in order, and the first products wait for two reads only
        // (600 x 2048 over 7168 26.4 us to 25.7, the weight gradient 1029 to 995).  The 256-tile that
        // keeps codes and one scale of b has the registers, but the compiler then spreads its
        // reads worse: 505 us for 480
        constexpr bool kEarly = TILE < 256 || EXACT || !SQUARE;
        i32x8 early;
        float early_sa;
        if constexpr (kEarly) early = fragment(lds[buf], wm), early_sa = scales[buf][wm + (lane & 15)];
        Wide<FB, EXACT> fb[G::kNj];
#pragma unroll
        for (int j = 0; j < G::kNj; ++j) fb[j].set(fragment(lds[buf] + G::kOp, wn + 16 * j));
        // (behind these reads, not before them: 1 to 3% on every shape.)  With more than two stages
        // the last block is loaded once more at the end, so that as many loads are on their way
        if constexpr (kDealt)
            load4_to_lds(ps + (kb + 1) * ps_step, scales0 + ahead * G::kScales * 4 + wave * 256);
        else if constexpr (DIRECT && kStages > 2)
            fetch(min(kb + kStages - 1, last - 1), ahead, set);
        else if (kb + (DIRECT ? 1 : G::kSets) < last)
            fetch(kb + (DIRECT ? 1 : G::kSets), ahead, set);
        const float sb1 = scales[buf][TILE + wn];
#pragma unroll
        for (int i = 0; i < G::kMi; ++i) {
            Wide<FA, EXACT> fa;
            fa.set(kEarly && i == 0 ? early : fragment(lds[buf], wm + 16 * i));
            const float sa = kEarly && i == 0 ? early_sa : scales[buf][wm + 16 * i + (lane & 15)];
            if constexpr (kDealt) {
                constexpr int kEach = 2 * G::kLoads / G::kMi;
                static_assert(kEach * G::kMi == 2 * G::kLoads, "loads of a row of tiles");
                const uint32_t to = lds0 + ahead * 2 * G::kOp + wave * 1024;
                const int next = (kb + 1) * kFp8Block;
#pragma unroll
                for (int q = i * kEach; q < (i + 1) * kEach; ++q) {
                    const int p = q / 2;
                    if (q % 2 == 0)
                        load16_to_lds(a_base + next, a_off[p], to + p * G::kThreads * 16);
                    else
                        load16_to_lds(b_base + next, b_off[p], to + G::kOp + p * G::kThreads * 16);
                }
            }
            // b's scales of single rows are read anew for every i: held, they cost the 256-tile
            // with widened codes 44 spilled registers and twice the time
            int at = TILE + wn + 4 * (lane >> 4);
            if constexpr (!SQUARE && EXACT) asm volatile("" : "+v"(at));
            // two tiles at once: of widened codes an inner sum is a chain of four instructions (846
            // against 819 us, 8192 x 14336 over 4096; with scales of single rows there are no
            // registers left for it)
            constexpr int kAtOnce = EXACT && !SQUARE ? 1 : 2;
#pragma unroll
            for (int j = 0; j < G::kNj; j += kAtOnce) {
                f32x4 sum[kAtOnce];
                block_products<kAtOnce>(fb + j, fa, sum);
#pragma unroll
                for (int q = 0; q < kAtOnce; ++q) {
                    if constexpr (SQUARE)
                        acc[i][j + q] += sum[q] * (sb1 * sa);
                    else
                        acc[i][j + q] +=
                            sum[q] * (*reinterpret_cast<const f32x4*>(&scales[buf][at + 16 * (j + q)]) * sa);
                }
            }
        }
        if constexpr (DIRECT) others |= __builtin_amdgcn_ballot_w64(!is_plain(scales[buf][tid & (2 * TILE - 1)]));
        stage = stage + 1 == kStages ? 0 : stage + 1;
        ahead = ahead + 1 == kStages ? 0 : ahead + 1;
    };
    using Set0 = std::integral_constant<int, 0>;
    using Set1 = std::integral_constant<int, !DIRECT && G::kSets == 2 ? 1 : 0>;
    if constexpr (DIRECT) {
#pragma unroll
        for (int p = 0; p < kStages - 1; ++p) fetch(min(first + p, last - 1), p, Set0{});
    } else {
        fetch(first, 0, Set0{});
        if (G::kSets == 2 && first + 1 < last) fetch(first + 1, 0, Set1{});
    }
    if constexpr (!DIRECT && G::kSets == 2) {
        for (int kb = first; kb < last; kb += 2) {
            step(kb, Set0{}, std::false_type{});
            if (kb + 1 < last) step(kb + 1, Set1{}, std::false_type{});
        }
    } else {
        int kb = first;
        if constexpr (kDeals)
            for (; kb + 1 < last && (kb + 2) * kFp8Block <= g.k; ++kb) step(kb, Set0{}, std::true_type{});
        for (; kb < last; ++kb) step(kb, Set0{}, std::false_type{});
    }
    if constexpr (DIRECT && kStages > 2) wait_loads<0>();  // the repeated ones: LDS must be left alone
    if (lane == 0) not_plain[wave] = others != 0;
    __syncthreads();
    if (__builtin_amdgcn_ballot_w64(lane < G::kWaves && not_plain[lane & (G::kWaves - 1)]) != 0) {
        // (a gradient's rows may be that small, without any product of their scales being so)
        Sizes all;
#pragma unroll 4
        for (int kb = first; kb < last; ++kb) all.meet(ps[kb * ps_step]);
        bool normal = products_are_normal<G::kWaves>(all, met, 2 * TILE);
        if (!normal) {
            // blocks of zeros have scales near 2^-109, but their sums are zero too, and zero times a
            // small product is right: without them
            const int t = tid & (2 * TILE - 1);
            const Operand& o = t < TILE ? g.a : g.b;
            const int r = min((t < TILE ? m0 : n0) + (t & (TILE - 1)), o.rows - 1);
            const uint8_t* row = o.codes + int64_t(r) * o.row_stride;
            Sizes nonzero;
#pragma unroll 1
            for (int kb = first; kb < last; ++kb) {
                const float scale = ps[kb * ps_step];
                if (fabsf(scale) < 0x1p-63f) {
                    i32x4 any = {0, 0, 0, 0};
#pragma unroll 1
                    for (int c = 0; c < kFp8Block; c += 16) any |= load_chunk(row, kb * kFp8Block + c, g.k);
                    if (((any.x | any.y | any.z | any.w) & 0x7f7f7f7f) == 0) continue;
                }
                nonzero.meet(scale);
            }
            normal = products_are_normal<G::kWaves>(nonzero, met, 2 * TILE);
        }
        if (!normal) {
            tiles_by_parts<G::kMi, G::kNj, FA, FB, EXACT>(g, split, m0 + wm, n0 + wn, first, last);
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < G::kMi; ++i)
#pragma unroll
        for (int j = 0; j < G::kNj; ++j)
            store_result(g, split, m0 + wm + 16 * i + (lane & 15), n0 + wn + 16 * j + 4 * (lane >> 4),
                         acc[i][j]);
}

// ------------------------------------------------------------ few rows of a

// At most 16 rows of a against 16 rows of b a workgroup: b is read once, straight into the
// instruction's registers, each of 16 waves taking a share of k's blocks; the waves'
// sums are added through LDS in wave order.  Bound by b's bytes once it runs: one row over 14336,
// 4096 rows of b (58.7 MB, cold) takes 13.7 us, where 1024 rows over 4096 (4 MB) take 5.2.  2
// blocks on their way a wave; 4 take 14.8, 8 waves 15.7 (4 blocks) and 17.9 (8), 4 waves 20.7 and more,
// nontemporal loads 15.1.
constexpr int kFewWaves = 16, kFewAhead = 2, kFewRows = 16;

template <int FA, int FB, bool EXACT, bool SQUARE>
__global__ __launch_bounds__(kFewWaves * 64) void fp8_few_kernel(const ProductArgs g) {
    __shared__ f32x4 sums[kFewWaves][64];
    const int split = blockIdx.x / g.tiles_n, n0 = (blockIdx.x - split * g.tiles_n) * 16;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int nk = (g.k + kFp8Block - 1) / kFp8Block;
    const int first = split * g.per_split, last = min(nk, first + g.per_split);
    const int q = lane >> 4, ar = min(lane & 15, g.a.rows - 1), br = min(n0 + (lane & 15), g.b.rows - 1);

    const uint8_t* pa = g.a.codes + int64_t(ar) * g.a.row_stride;
    const uint8_t* pb = g.b.codes + int64_t(br) * g.b.row_stride;
    const float* sa = g.a.scales + int64_t(ar >> g.a.shift) * g.a.scale_row;
    const float* sb[SQUARE ? 1 : 4];
    if constexpr (SQUARE) {
        sb[0] = g.b.scales + int64_t(n0 >> 7) * g.b.scale_row;
    } else {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            sb[t] = g.b.scales + int64_t(min(n0 + 4 * q + t, g.b.rows - 1)) * g.b.scale_row;
    }
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int kb0 = first + wave; kb0 < last; kb0 += kFewWaves * kFewAhead) {
        i32x8 fb[kFewAhead], fa[kFewAhead];
        float sa_at[kFewAhead], sb_at[kFewAhead][SQUARE ? 1 : 4];
#pragma unroll
        for (int u = 0; u < kFewAhead; ++u) {
            const int kb = kb0 + u * kFewWaves;
            if (kb >= last) continue;
            const int at = kb * kFp8Block + q * 16;
            fb[u] = join(load_chunk(pb, at, g.k), load_chunk(pb, at + 64, g.k));
            fa[u] = join(load_chunk(pa, at, g.k), load_chunk(pa, at + 64, g.k));
            sa_at[u] = sa[kb * g.a.scale_col];
#pragma unroll
            for (int t = 0; t < (SQUARE ? 1 : 4); ++t) sb_at[u][t] = sb[t][kb * g.b.scale_col];
        }
#pragma unroll
        for (int u = 0; u < kFewAhead; ++u) {
            if (kb0 + u * kFewWaves >= last) continue;
            Wide<FB, EXACT> wb;
            Wide<FA, EXACT> wa;
            wb.set(fb[u]), wa.set(fa[u]);
            f32x4 sum;
            block_products<1>(&wb, wa, &sum);
            f32x4 scale;
            bool plain = true;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                scale[t] = sa_at[u] * sb_at[u][SQUARE ? 0 : t];
                plain &= is_normal(scale[t]);
            }
            if (__builtin_amdgcn_ballot_w64(!plain) == 0)
                acc += sum * scale;
            else
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    acc[t] = add_by_parts(acc[t], sum[t], sa_at[u], sb_at[u][SQUARE ? 0 : t]);
        }
    }
    sums[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
        for (int w = 1; w < kFewWaves; ++w) acc += sums[w][lane];
        store_result(g, split, lane & 15, n0 + 4 * q, acc);
    }
}

// out (+)= the splits' sums, in their order; zeros where there are none (k = 0).
__global__ __launch_bounds__(256) void fp8_join_kernel(ProductArgs g) {
    const float* partial = g.partial;
    g.partial = nullptr;
    const int per = (g.b.rows + 3) / 4;
    const int64_t groups = int64_t(g.a.rows) * per, all = int64_t(g.a.rows) * g.b.rows;
    for (int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x; t < groups; t += int64_t(gridDim.x) * 256) {
        const int i = int(t / per), j = int(t - int64_t(i) * per) * 4, left = g.b.rows - j;
        const float* p = partial + int64_t(i) * g.b.rows + j;
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < g.splits; ++k, p += all) {
            if (left >= 4) {
                sum += f32x4(*reinterpret_cast<const f32x4_any*>(p));
            } else {
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (e < left) sum[e] += p[e];
            }
        }
        store_result(g, 0, i, j, sum);
    }
}

Operand operand_of(const muon_fp8_t& m) {
    return {static_cast<const uint8_t*>(m.codes), m.scales, m.row_stride, m.scale_row, m.scale_col,
            int32_t(m.rows), m.block_rows == 1 ? 0 : 7};
}

// How a product runs.
struct Shape {
    int tile;        // 0: few rows of a
    int64_t tiles;   // workgroups of one split
    int splits, per_split;
};

// About how many microseconds a product takes in `tiles` workgroups of one size and `splits`
// splits of its nk blocks of k, from measurements of 21 shapes (100 x 700 over 300 to 8192 x
// 4096 over 4096): a block takes the longer the more workgroups share a CU, up to `most` of them.
// What it chooses takes at most 15% more than the best there, where 256-tiles throughout
// take up to 3.5 times the best (512 x 512 over 512: 16.8 and 4.8 us) and 64-tiles 1.8 times (4096^3: 124
// and 68).
float estimate(int64_t m, int64_t n, int64_t nk, int tile, int64_t tiles, int64_t splits) {
    const float most = tile == 256 ? 1.f : 2.f;
    const float first = tile == 256 ? 2.f : tile == 128 ? 0.82f : 0.36f;
    const float full = tile == 256 ? 2.f : tile == 128 ? 1.12f : 0.5f;
    const float load = float(tiles * splits) / 256.f, rounds = std::floor(load / most);  // a CU
    const float rest = load - rounds * most;
    const float block = rounds * full + (rest > 1.f ? full : rest > 0.f ? first : 0.f);
    const float join = splits > 1 ? 5.f + float(splits * m) * float(n) * 1e-6f : 0.f;
    return 2.5f + block * float((nk + splits - 1) / splits) + join;
}

Shape shape_of(int64_t m, int64_t n, int64_t k) {
    const int64_t nk = fp8_blocks(k);
    Shape best{};
    if (m <= kFewRows) {
        best.tiles = (n + 15) / 16;
        // 1024 rows of b over k = 14336: 7.5 us in 4 splits, 10.5 in one; over 4096 6.2 and 5.0
        const int64_t splits = std::clamp<int64_t>(std::min(256 / best.tiles, nk / 28), 1, 4);
        best.per_split = int((nk + splits - 1) / splits);
    } else {
        float least = 0.f;
        for (int tile : {256, 128, 64}) {
            const int64_t tiles = ((m + tile - 1) / tile) * ((n + tile - 1) / tile);
            for (int64_t splits : {1, 2, 3, 4, 6, 8, 12, 16}) {
                if (splits > 1 && (tiles * splits > 1024 || nk < 4 * splits)) break;
                const float t = estimate(m, n, nk, tile, tiles, splits);
                if (best.tiles == 0 || t < least)
                    least = t, best = {tile, tiles, int(splits), int((nk + splits - 1) / splits)};
            }
        }
    }
    best.splits = int((nk + best.per_split - 1) / std::max(best.per_split, 1));
    return best;
}

template <int FA, int FB, bool EXACT>
void enqueue(const Shape& sh, const ProductArgs& g, bool direct, hipStream_t s) {
    const dim3 grid = dim3(unsigned(sh.tiles * sh.splits));
    const bool square = g.b.shift != 0;
    if (sh.tile == 0) {
        const dim3 block = dim3(kFewWaves * 64);
        square ? fp8_few_kernel<FA, FB, EXACT, true><<<grid, block, 0, s>>>(g)
               : fp8_few_kernel<FA, FB, EXACT, false><<<grid, block, 0, s>>>(g);
        return;
    }
    const auto run = [&](auto tile) {
        constexpr int kTile = decltype(tile)::value;
        const dim3 block = dim3(Geo<kTile>::kThreads);
        if (direct)
            square ? fp8_tile_kernel<kTile, true, FA, FB, EXACT, true><<<grid, block, 0, s>>>(g)
                   : fp8_tile_kernel<kTile, true, FA, FB, EXACT, false><<<grid, block, 0, s>>>(g);
        else if constexpr (kTile != 256)
            fp8_tile_kernel<kTile, false, FA, FB, EXACT, false><<<grid, block, 0, s>>>(g);
    };
    if (sh.tile == 256)
        run(std::integral_constant<int, 256>{});
    else if (sh.tile == 128)
        run(std::integral_constant<int, 128>{});
    else
        run(std::integral_constant<int, 64>{});
}

template <int FA, int FB>
void enqueue(const Shape& sh, const ProductArgs& g, bool direct, hipStream_t s) {
    g.out_bf16 ? enqueue<FA, FB, false>(sh, g, direct, s) : enqueue<FA, FB, true>(sh, g, direct, s);
}

// Rows of codes that direct loads take.
bool direct_rows(const muon_fp8_t& m) {
    return reinterpret_cast<uintptr_t>(m.codes) % 16 == 0 && m.cols % 16 == 0 &&
           (m.rows == 1 || (m.row_stride % 16 == 0 && m.row_stride < (int64_t(1) << 24)));
}

}  // namespace

size_t fp8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (m == 0 || n == 0 || k == 0) return 0;
    const Shape s = shape_of(m, n, k);
    if (s.splits == 1) return 0;
    return (size_t(s.splits) * m * n * sizeof(float) + kWsAlign - 1) / kWsAlign * kWsAlign;
}

hipError_t launch_fp8_matmul(const muon_fp8_t& a, const muon_fp8_t& b, void* out, int out_dtype,
                             int64_t out_row_stride, bool accumulate, void* workspace, hipStream_t s) {
    ProductArgs g{};
    g.a = operand_of(a), g.b = operand_of(b);
    g.out = out, g.out_row = out_row_stride, g.k = int32_t(a.cols);
    g.out_bf16 = out_dtype == MUON_DTYPE_BF16, g.accumulate = accumulate;
    const int64_t groups = a.rows * ((b.rows + 3) / 4);
    const dim3 join_grid = dim3(unsigned(std::min<int64_t>((groups + 255) / 256, 1 << 16)));
    if (g.k == 0) {
        if (accumulate) return hipSuccess;
        LaunchTimer timer("fp8_join", s);
        fp8_join_kernel<<<join_grid, dim3(256), 0, s>>>(g);
        return hipGetLastError();
    }
    Shape sh = shape_of(a.rows, b.rows, a.cols);
    const bool direct = direct_rows(a) && direct_rows(b);
    if (sh.tile == 256 && !direct) {
        // loads through registers have none to spare at this size
        sh.tile = 128;
        sh.tiles = ((a.rows + 127) / 128) * ((b.rows + 127) / 128);
    }
    g.tiles_m = sh.tile ? int32_t((a.rows + sh.tile - 1) / sh.tile) : 1;
    g.tiles_n = int32_t(sh.tile ? (b.rows + sh.tile - 1) / sh.tile : sh.tiles);
    g.splits = sh.splits, g.per_split = sh.per_split;
    g.partial = sh.splits > 1 ? static_cast<float*>(workspace) : nullptr;
    {
        LaunchTimer timer("fp8_matmul", s);
        if (a.format == MUON_FP8_E5M2)
            b.format == MUON_FP8_E5M2 ? enqueue<1, 1>(sh, g, direct, s) : enqueue<1, 0>(sh, g, direct, s);
        else
            b.format == MUON_FP8_E5M2 ? enqueue<0, 1>(sh, g, direct, s) : enqueue<0, 0>(sh, g, direct, s);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || sh.splits == 1) return e;
    LaunchTimer timer("fp8_join", s);
    fp8_join_kernel<<<join_grid, dim3(256), 0, s>>>(g);
    return hipGetLastError();
}

}  // namespace muon
