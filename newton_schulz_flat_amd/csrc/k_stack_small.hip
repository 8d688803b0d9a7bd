// Newton-Schulz of stacks of matrices with a short side, on the pairs of float16 of k_stack.hip.
//
// stack_whole: matrices that fit a CU's LDS (shorter side up to 64).  One workgroup and one
// launch a matrix: norm, split, all iterations and the result, X and A and B in LDS.  Bound by the
// latency of 15 products that follow each other: 16 matrices of 48 x 64 take 18.1 us, 512 of 64 x 64 42.
//
// stack_strip and stack_poly: shorter side up to 128.  B (r x r) is small, so one pass over X
// makes the next iterate and its Gram matrix at once: a workgroup takes strips of 64
// columns, X <- a X + B X in place, and adds X X^T of the strip to its own partial
// Gram matrix; stack_poly adds a matrix's partial ones in order and makes B = b A + c A A of
// them.  Two launches and one read and write of X a step, where the stages of k_stack.hip take
// three and two reads.  A strip of 128 rows takes 5 us of which 1.4 are matrix instructions: three
// barriers a strip and one workgroup a CU.  (Two tiles below each other of the strip a wave, for
// fewer LDS reads, spilled: 234 us of 5 steps for 206; Gram tiles on and above the diagonal only: 194.)
#include <algorithm>
#include <type_traits>

#include "stack_device.h"

namespace muon {

namespace {

// Where a matrix of pairs lies in LDS: rows of row_bytes (a multiple of 256), chunk c (16 bytes) of
// row r at chunk c ^ turn(r).  A 16-byte read of 16 rows at two neighbouring chunks is served in
// groups of rows 0-3 and 12-15 of one with 4-11 of the other: turn leaves out bit 2, which the chunk
// makes up for.  A transposing read takes rows 0-3 and 8-11 mod 16, or these + 4, to 32 bytes each, which
// turn, always even, leaves together and sends to all 256.  (A turn of all four bits: half of the
// reads' cycles were conflicts.)
__device__ __forceinline__ int turn(int r) { return (r & 3) << 1 | (r >> 3 & 1) << 3; }

// A lane's part of the addresses in a matrix with rows of row_bytes.  What a call adds to it (K
// step, half, place of the tile) it adds as constants: those below 256 bytes by exclusive or, like
// turn itself.  Worked out anew for every operand, addresses took more time than the products.
struct Place {
    int row_bytes, rows, turned, quad;
    __device__ __forceinline__ explicit Place(int bytes) : row_bytes(bytes) {
        const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4, k = g * 8 + (l >> 2);
        rows = l * bytes + ((g ^ turn(l)) << 4);
        turned = k * bytes + ((((l & 3) >> 1) ^ turn(k & 15)) << 4) + (l & 1) * 8;
        quad = l * bytes + (((g >> 1) ^ turn(l)) << 4) + (g & 1) * 8;
    }
};

// Operand of 16 rows from row0 on, K step ks (32 columns), half 0 (high) or 1.
__device__ __forceinline__ f16x8 rows_operand(const unsigned char* m, const Place& p, int row0, int ks, int half) {
    return *reinterpret_cast<const f16x8*>(m + (p.rows ^ ((ks & 1) * 128 + half * 64)) + (ks >> 1) * 256 +
                                           row0 * p.row_bytes);
}
// Operand of 16 columns from 16 * tile on, K step ks (32 rows).
__device__ __forceinline__ f16x8 turned_operand(const unsigned char* m, const Place& p, int tile, int ks, int half) {
    const int low = ((tile >> 1) & 1) * 128 + half * 64 + (tile & 1) * 32;
    const unsigned char* at = m + (tile >> 2) * 256 + ks * 32 * p.row_bytes;
    // the second read's rows are 4 further on, where turn is the same
    const uint2 lo = read_turned(at + (p.turned ^ low));
    const uint2 hi = read_turned(at + (p.turned ^ low) + 4 * p.row_bytes);
    return __builtin_bit_cast(f16x8, u32x4{lo.x, lo.y, hi.x, hi.y});
}
// This lane's four neighbouring elements of the 16 x 16 tile (ti, tj): row lane % 16, columns
// from 4 (lane / 16) on.
__device__ __forceinline__ unsigned char* quad_at(unsigned char* m, const Place& p, int ti, int tj, int half) {
    return m + (p.quad ^ (((tj >> 1) & 1) * 128 + half * 64 + (tj & 1) * 32)) + (tj >> 2) * 256 +
           ti * 16 * p.row_bytes;
}
__device__ __forceinline__ void put_quad(unsigned char* m, const Place& p, int ti, int tj, const float v[4]) {
    f16x4 hi, lo;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const Pair s = split(v[t]);
        hi[t] = s.hi, lo[t] = s.lo;
    }
    *reinterpret_cast<f16x4*>(quad_at(m, p, ti, tj, 0)) = hi;
    *reinterpret_cast<f16x4*>(quad_at(m, p, ti, tj, 1)) = lo;
}
__device__ __forceinline__ void get_quad(unsigned char* m, const Place& p, int ti, int tj, float v[4]) {
    const f16x4 hi = *reinterpret_cast<const f16x4*>(quad_at(m, p, ti, tj, 0));
    const f16x4 lo = *reinterpret_cast<const f16x4*>(quad_at(m, p, ti, tj, 1));
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = float(hi[t]) + float(lo[t]);
}
// One element (i, j) of either half.
__device__ __forceinline__ _Float16* element_at(unsigned char* m, int row_bytes, int i, int j, int half) {
    const int c = (j >> 5) * 8 + half * 4 + ((j & 31) >> 3);
    return reinterpret_cast<_Float16*>(m + i * row_bytes + ((c ^ turn(i)) << 4)) + (j & 7);
}
// acc += the three products of the halves.
__device__ __forceinline__ f32x4 product(f16x8 qh, f16x8 ql, f16x8 ph, f16x8 pl, f32x4 acc) {
    acc = mfma(ql, ph, acc);
    acc = mfma(qh, pl, acc);
    return mfma(qh, ph, acc);
}

// -------------------------------------------------------- one workgroup a matrix

struct WholeArgs {
    InArgs in;
    int32_t out_bf16, tall;
};

// RP: rows, padded (32 or 64).  16 waves: A and B in tiles of 16 x 16, a wave each (of 32 rows
// there are 4 tiles, and four waves share A's K steps); X in blocks of 16 tiles, which are all read
// before they are renewed in place.  The matrices are small: what counts is the number
// of waves that wait for LDS at once (64 x 64, five steps: 4 waves 24 us, 16 waves 19).
constexpr int kWholeThreads = 1024;

template <int RP, typename T>
__global__ __launch_bounds__(kWholeThreads) void stack_whole_kernel(const WholeArgs w) {
    extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
    __shared__ double sums[16];
    const InArgs& g = w.in;
    constexpr int kSquare = 256;  // bytes of a row of A and B
    constexpr int kF = RP / 16, kSteps = RP / 32, kShare = 16 / (kF * kF);
    const int x_row = g.cp * 4;
    unsigned char *x = lds, *a = x + RP * x_row, *b = a + RP * kSquare;
    const int matrix = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const T* u = static_cast<const T*>(g.in) + matrix * g.in_stride;

    // rows of U in turn to the waves, 64 columns at a time, or several short rows at once
    const int wide = g.cols >= 64 ? 6 : 32 - __builtin_clz(g.cols - 1 | 1), at_once = 64 >> wide;
    const int i0 = wave * at_once + (lane >> wide), j0 = lane & ((1 << wide) - 1);
    double sum = 0.;
#pragma unroll 4
    for (int i = i0; i < g.rows; i += 16 * at_once)
#pragma unroll 4
        for (int j = j0; j < g.cols; j += 64) {
            const double v = load_one(u + int64_t(i) * g.in_row + j);
            sum = fma(v, v, sum);
        }
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    if (lane == 0) sums[wave] = sum;
    // zeros everywhere, for the padding
    for (int at = tid * 16; at < RP * (x_row + 2 * kSquare); at += kWholeThreads * 16)
        *reinterpret_cast<u32x4*>(lds + at) = u32x4{0, 0, 0, 0};
    __syncthreads();
    double norm = 0.;
#pragma unroll
    for (int k = 0; k < 16; ++k) norm += sums[k];
    norm = sqrt(norm);
    const float inv = inverse_of(norm);
    float top = first_bound(norm);
    const bool small = top < kStackSmallBound;
    int sx = small ? stack_exponent(top, kStackLeastX) : g.plan.scales[0].sx;
    const float up = stack_scaled(1.f, sx - kInverseUp);
#pragma unroll 4
    for (int i = i0; i < g.rows; i += 16 * at_once)
#pragma unroll 4
        for (int j = j0; j < g.cols; j += 64) {
            const Pair p = split(load_one(u + int64_t(i) * g.in_row + j) * inv * up);
            const int m = w.tall ? j : i, n = w.tall ? i : j;
            *element_at(x, x_row, m, n, 0) = p.hi;
            *element_at(x, x_row, m, n, 1) = p.lo;
        }
    __syncthreads();

    const int k_steps = g.cp / 32;
    // this wave's tile of A and B, and its share of A's K steps; its row of tiles of X
    const int tile = wave % (kF * kF), share = wave / (kF * kF), fi = tile / kF, fj = tile % kF;
    const Place in_x(x_row), in_square(kSquare);
    constexpr int kBlock = 16 * 16 / kF;  // columns of a block of 16 tiles of X
    for (int t = 0; t < g.plan.n; ++t) {
        const StackStep step = g.plan.steps[t];
        const StackScale s = small ? stack_scale(step, top) : g.plan.scales[t];
        // A = X X^T
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
        for (int ks = share; ks < k_steps; ks += kShare)
            acc = product(rows_operand(x, in_x, fj * 16, ks, 0), rows_operand(x, in_x, fj * 16, ks, 1),
                          rows_operand(x, in_x, fi * 16, ks, 0), rows_operand(x, in_x, fi * 16, ks, 1), acc);
        if constexpr (kShare > 1) {
            // the first wave of a tile adds the others' sums in their order
            f32x4* sums_a = reinterpret_cast<f32x4*>(b + RP * kSquare);
            if (share > 0) sums_a[(tile * (kShare - 1) + share - 1) * 64 + lane] = acc;
            __syncthreads();
            if (share == 0)
#pragma unroll
                for (int k = 0; k < kShare - 1; ++k) acc += sums_a[(tile * (kShare - 1) + k) * 64 + lane];
        }
        const float down_a = stack_a_factor(s);
        const auto put = [&](unsigned char* to) {
            const float v[4] = {acc.x, acc.y, acc.z, acc.w};
            put_quad(to, in_square, fi, fj, v);
        };
        acc *= down_a;
        if (share == 0) put(a);
        __syncthreads();
        // B = b A + c A A, with this wave's tile of A still in registers
        if (share == 0) {
            const StackFactors fb = stack_b_factors(step, s);
            f32x4 aa = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks)
                aa = product(rows_operand(a, in_square, fj * 16, ks, 0), rows_operand(a, in_square, fj * 16, ks, 1),
                             rows_operand(a, in_square, fi * 16, ks, 0), rows_operand(a, in_square, fi * 16, ks, 1), aa);
            acc = acc * fb.own + aa * fb.down;
            put(b);
        }
        __syncthreads();
        // X <- a X + B X
        const bool last = t + 1 == g.plan.n;
        const int next = small ? stack_exponent(top, kStackLeastX) : g.plan.scales[t + 1].sx;
        const StackFactors fx = stack_x_factors(step, s, next, last, g.scale);
        const int xi = wave % kF, xm = xi * 16 + (lane & 15);
        f16x8 bh[kSteps], bl[kSteps];
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
            bh[ks] = rows_operand(b, in_square, xi * 16, ks, 0);
            bl[ks] = rows_operand(b, in_square, xi * 16, ks, 1);
        }
        for (int at = 0; at < g.cp; at += kBlock) {
            const int xj = at / 16 + wave / kF, col = xj * 16, n = col + 4 * (lane >> 4);
            float v[4];
            if (col < g.cp) {
                f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks)
                    y = product(turned_operand(x, in_x, xj, ks, 0), turned_operand(x, in_x, xj, ks, 1), bh[ks],
                                bl[ks], y);
                get_quad(x, in_x, xi, xj, v);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = fx.own * v[e] + fx.down * y[e];
            }
            if (!last) {
                __syncthreads();
                if (col < g.cp) put_quad(x, in_x, xi, xj, v);
            } else if (col < g.cp) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] *= fx.after;
                if (w.out_bf16)
                    store_result(static_cast<uint16_t*>(g.out) + matrix * g.out_stride, g.out_row, w.tall, g.rows,
                                 g.cols, xm, n, v);
                else
                    store_result(static_cast<float*>(g.out) + matrix * g.out_stride, g.out_row, w.tall, g.rows,
                                 g.cols, xm, n, v);
            }
        }
        sx = next;
        __syncthreads();
    }
}

// ------------------------------------------------------------- strips of 64 columns

struct StripArgs {
    InArgs in;
    _Float16* x;    // [matrix][cp / 32][rp][64]
    const float* gram;  // [matrix][part][tile of 16 x 16][lane][4]
    float* gram_next;   // of the next iterate
    _Float16* b;    // [matrix][row tile][K step][half][lane][8]
    const StackScale* scales;  // this step's, of matrix 0
    StackStep step;
    void* out;
    int64_t out_stride, out_row;
    int32_t cp, parts, per;  // strips of 64 columns of one part
    int32_t rows, cols, tall, out_bf16, last;
    float scale;
};

// Waves in 2 columns of RP / 16: each has one row of 16 x 16 tiles, of the strip 2 of its 4 tiles,
// of the Gram matrix half.
template <int RP>
struct StripGeo {
    static constexpr int kF = RP / 16, kSteps = RP / 32;
    static constexpr int kWaves = 2 * kF, kThreads = kWaves * 64;
    static constexpr int kGn = kF / 2;
    static constexpr int kOp = RP * 256;  // bytes of a strip
    // Half of the waves load strips, the other half stores them: one counter covers a wave's
    // loads and stores, and waiting for the next strip must not wait for the last one's stores.
    static constexpr int kMovers = kThreads / 2;
    static constexpr int kLoads = kOp / (kMovers * 16);
    static constexpr int kStages = 3;  // strips in LDS: two on their way
};

// B = b A + c A A of a matrix, A the sum of its partial Gram matrices, in their order: WAVES waves, each
// with tiles of one row of tiles, A in LDS at a.  Returns this wave's tiles of B, stored 2^sb.
template <int RP, int WAVES>
struct Poly {
    static constexpr int kRow = RP == 32 ? 256 : RP * 4, kBytes = RP * kRow;
    static constexpr int kF = RP / 16, kSteps = RP / 32, kMine = kF * kF / WAVES;
    static_assert(kMine >= 1 && kF % kMine == 0, "tiles of one row");
    f32x4 b[kMine];
    int fi, fj;

    __device__ __forceinline__ void run(const StripArgs& g, int matrix, const StackScale& s, unsigned char* a) {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        fi = wave * kMine / kF, fj = wave * kMine % kF;
        const f32x4* from = reinterpret_cast<const f32x4*>(g.gram) + int64_t(matrix) * g.parts * (RP * RP / 4) +
                            wave * kMine * 64 + lane;
        f32x4 acc[kMine];
#pragma unroll
        for (int q = 0; q < kMine; ++q) acc[q] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int p = 0; p < g.parts; ++p)
#pragma unroll
            for (int q = 0; q < kMine; ++q) acc[q] += from[p * (RP * RP / 4) + q * 64];
        const Place in_a(kRow);
        const float down_a = stack_a_factor(s);
#pragma unroll
        for (int q = 0; q < kMine; ++q) {
            acc[q] *= down_a;
            put(a, in_a, q, acc[q]);
        }
        __syncthreads();
        const StackFactors f = stack_b_factors(g.step, s);
#pragma unroll
        for (int q = 0; q < kMine; ++q) b[q] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
            const f16x8 ph = rows_operand(a, in_a, fi * 16, ks, 0), pl = rows_operand(a, in_a, fi * 16, ks, 1);
#pragma unroll
            for (int q = 0; q < kMine; ++q)
                b[q] = product(rows_operand(a, in_a, (fj + q) * 16, ks, 0),
                               rows_operand(a, in_a, (fj + q) * 16, ks, 1), ph, pl, b[q]);
        }
#pragma unroll
        for (int q = 0; q < kMine; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) b[q][e] = __builtin_fmaf(acc[q][e], f.own, b[q][e] * f.down);
    }
    __device__ __forceinline__ void put(unsigned char* m, const Place& place, int q, const f32x4& t) const {
        const float v[4] = {t.x, t.y, t.z, t.w};
        put_quad(m, place, fi, fj + q, v);
    }
};

// Eight neighbouring elements of U as they are in memory, zeros behind the first `left`.
template <typename T>
struct Eight {
    uint32_t w[2 * sizeof(T)];
    __device__ __forceinline__ void load(const T* p, int left) {
        typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
        if (left >= 8) {
#pragma unroll
            for (int k = 0; k < int(sizeof(T)) / 2; ++k) {
                const u32x4_any t = reinterpret_cast<const u32x4_any*>(p)[k];
                w[4 * k] = t.x, w[4 * k + 1] = t.y, w[4 * k + 2] = t.z, w[4 * k + 3] = t.w;
            }
        } else {
#pragma unroll
            for (int k = 0; k < int(2 * sizeof(T)); ++k) w[k] = 0;
#pragma unroll
            for (int k = 0; k < 7; ++k)
                if (k < left) {
                    if constexpr (sizeof(T) == 4)
                        w[k] = __float_as_uint(p[k]);
                    else
                        w[k / 2] |= uint32_t(p[k]) << (16 * (k & 1));
                }
        }
    }
    __device__ __forceinline__ float operator[](int k) const {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[k]);
        else
            return __uint_as_float(k & 1 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
    }
};
struct Nothing {};

// MODE kGram: the Gram matrix of the first iterate.  kStep: B comes from
// stack_poly_kernel.  kWholeStep: the workgroup makes B of the partial Gram matrices itself, which
// saves a launch where they are few (2 x 128 x 512, 4 of them: 92 us, with stack_poly 100), but is work
// done by every workgroup (64 x 128 x 1024, 4 of them: 212 and 206; 32 x 128 x 4096, 8: 362 and 302).
// Both give the same bits: fused sums are written out, since the compiler's choice differs.
// T: U's type, where the iterate is the first one; it is made of U anew in kGram and in the first step
// (32 x 128 x 4096, bfloat16: 277 us, with a launch that stores it once 303).  void: X.
enum StripMode { kGram, kStep, kWholeStep };

template <int RP, int MODE, typename T>
__global__ __launch_bounds__(StripGeo<RP>::kThreads) void stack_strip_kernel(const StripArgs g) {
    using G = StripGeo<RP>;
    constexpr bool FIRST = MODE == kGram, FROM_U = !std::is_void_v<T>;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[G::kStages][G::kOp];
    const int matrix = blockIdx.x / g.parts, part = blockIdx.x % g.parts;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int strips = g.cp / 64, first = part * g.per, end = min(strips, first + g.per);
    unsigned char* x = reinterpret_cast<unsigned char*>(g.x) + int64_t(matrix) * RP * g.cp * 4;
    const uint32_t lds0 = lds_address(lds[0]);
    const int wr = wave % G::kF, wc = wave / G::kF;
    const Place in_strip(256);

    // a mover's chunks: chunk tid % 16 of rows tid / 16 + p * rows of a pass
    constexpr int kRows = G::kMovers / 16;
    const bool loads = wave < G::kWaves / 2;
    const int mover = loads ? tid : tid - G::kMovers;
    uint32_t off[G::kLoads];
#pragma unroll
    for (int p = 0; p < G::kLoads; ++p) {
        const int r = (mover >> 4) + p * kRows, c = (mover & 15) ^ turn(r);
        off[p] = (c >> 3) * RP * 128 + r * 128 + (c & 7) * 16;
    }
    // eight neighbours in a row of U: in a row of the strip, or (tall) in a column, where 4 lanes take
    // 32 neighbours, 16 columns side by side (16 lanes a column: 8 of them meet in a bank)
    static_assert(RP * 64 == 8 * G::kThreads, "eight elements a thread");
    const int across = g.tall ? (wave % (RP / 32) * 4 + (lane & 3)) * 8 : tid % 8 * 8;
    const int down_to = g.tall ? wave / (RP / 32) * 16 + (lane >> 2) : tid / 8;
    std::conditional_t<FROM_U, Eight<std::conditional_t<FROM_U, T, float>>, Nothing> u;
    float inv = 0.f, up = 0.f;
    const auto take = [&](int strip) {
        if constexpr (FROM_U) {
            const int i = g.tall ? strip * 64 + down_to : down_to, j = g.tall ? across : strip * 64 + across;
            const T* from = static_cast<const T*>(g.in.in) + matrix * g.in.in_stride + int64_t(i) * g.in.in_row + j;
            u.load(from, i < g.rows ? g.cols - j : 0);
        }
    };
    const auto place = [&](unsigned char* m) {
        if constexpr (FROM_U) {
            f16x8 hi, lo;
            // (places are worked out for every strip: held, they cost spilled registers)
            int col = across, row = down_to;
            asm volatile("" : "+v"(col), "+v"(row));
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const Pair p = split(u[k] * inv * up);
                hi[k] = p.hi, lo[k] = p.lo;
            }
            if (g.tall) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    *element_at(m, 256, col + k, row, 0) = hi[k];
                    *element_at(m, 256, col + k, row, 1) = lo[k];
                }
            } else {
                *reinterpret_cast<f16x8*>(element_at(m, 256, row, col, 0)) = hi;
                *reinterpret_cast<f16x8*>(element_at(m, 256, row, col, 1)) = lo;
            }
        }
    };
    const auto fetch = [&](int strip, int stage) {
        if (FROM_U || !loads) return;
#pragma unroll
        for (int p = 0; p < G::kLoads; ++p)
            load_to_lds(x + int64_t(strip) * G::kOp, off[p],
                        lds0 + stage * G::kOp + p * G::kMovers * 16 + wave * 1024);
    };

    take(first);
    if constexpr (FROM_U) {
        const double norm = matrix_norm(g.in.partial + int64_t(matrix) * g.in.part_slots, g.in.parts);
        inv = inverse_of(norm);
        float top = first_bound(norm);
        const bool small = top < kStackSmallBound;
        up = stack_scaled(1.f, (small ? stack_exponent(top, kStackLeastX) : g.in.plan.scales[0].sx) - kInverseUp);
        if (FIRST && part == 0) {
            // the matrix's exponents
            StackScale* ex = g.in.scales + int64_t(matrix) * kStackScales;
            if (!small) {
                if (tid <= g.in.plan.n) ex[tid] = g.in.plan.scales[tid];
            } else if (tid == 0) {
                for (int k = 0; k < g.in.plan.n; ++k) ex[k] = stack_scale(g.in.plan.steps[k], top);
                ex[g.in.plan.n] = {int16_t(stack_exponent(top, kStackLeastX)), 0, 0, 0};
            }
        }
    }
    StackScale s{};
    StackFactors f = {0.f, 0.f, 1.f};
    f16x8 bh[G::kSteps], bl[G::kSteps];
    if constexpr (!FIRST) {
        const StackScale* ex = g.scales + int64_t(matrix) * kStackScales;
        s = ex[0];
        f = stack_x_factors(g.step, s, ex[1].sx, g.last, g.scale);
    }
    if constexpr (MODE == kStep) {
        const f16x8* b = reinterpret_cast<const f16x8*>(g.b) + int64_t(matrix) * RP * RP / 4;
#pragma unroll
        for (int ks = 0; ks < G::kSteps; ++ks) {
            const f16x8* q = b + ((wr * G::kSteps + ks) * 2) * 64 + lane;
            bh[ks] = q[0], bl[ks] = q[64];
        }
    }
    f32x4 gram[G::kGn];
#pragma unroll
    for (int j = 0; j < G::kGn; ++j) gram[j] = {0.f, 0.f, 0.f, 0.f};

    fetch(first, 0);
    if constexpr (MODE == kWholeStep) {
        // A and then B where the later strips will lie
        using P = Poly<RP, G::kWaves>;
        static_assert(P::kBytes <= 2 * G::kOp, "two strips");
        P poly;
        poly.run(g, matrix, s, lds[1]);
        __syncthreads();
        const Place in_b(P::kRow);
#pragma unroll
        for (int q = 0; q < P::kMine; ++q) poly.put(lds[1], in_b, q, poly.b[q]);
        __syncthreads();
#pragma unroll
        for (int ks = 0; ks < G::kSteps; ++ks) {
            bh[ks] = rows_operand(lds[1], in_b, wr * 16, ks, 0);
            bl[ks] = rows_operand(lds[1], in_b, wr * 16, ks, 1);
        }
        __syncthreads();
    }
    if (first + 1 < end) fetch(first + 1, 1);
    int stage = 0;
    for (int strip = first; strip < end; ++strip) {
        unsigned char* m = lds[stage];
        if constexpr (FROM_U) {
            place(m);
            if (strip + 1 < end) take(strip + 1);
        } else if (loads) {
            // all but the next strip's loads (and, of the results' stores, none: loads return in
            // their order, so what is left are these)
            if (strip + 1 < end)
                wait_loads<G::kLoads>();
            else
                wait_loads<0>();
        }
        __syncthreads();
        const int row = wr * 16 + (lane & 15);
        float v[2][4];
        if constexpr (!FIRST) {
            f32x4 y[2];
            y[0] = y[1] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < G::kSteps; ++ks)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    y[j] = product(turned_operand(m, in_strip, wc * 2 + j, ks, 0),
                                   turned_operand(m, in_strip, wc * 2 + j, ks, 1), bh[ks], bl[ks], y[j]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = (wc * 2 + j) * 16;
                get_quad(m, in_strip, wr, wc * 2 + j, v[j]);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[j][e] = __builtin_fmaf(f.own, v[j][e], f.down * y[j][e]);
                if (g.last) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[j][e] *= f.after;
                    if (g.out_bf16)
                        store_result(static_cast<uint16_t*>(g.out) + matrix * g.out_stride, g.out_row, g.tall,
                                     g.rows, g.cols, row, strip * 64 + col + 4 * (lane >> 4), v[j]);
                    else
                        store_result(static_cast<float*>(g.out) + matrix * g.out_stride, g.out_row, g.tall,
                                     g.rows, g.cols, row, strip * 64 + col + 4 * (lane >> 4), v[j]);
                }
            }
            if (!g.last) {
                __syncthreads();  // every wave has read the old strip
#pragma unroll
                for (int j = 0; j < 2; ++j) put_quad(m, in_strip, wr, wc * 2 + j, v[j]);
                __syncthreads();
                // back to memory as it was read
                if (!loads)
#pragma unroll
                    for (int p = 0; p < G::kLoads; ++p)
                        *reinterpret_cast<u32x4*>(x + int64_t(strip) * G::kOp + off[p]) =
                            *reinterpret_cast<const u32x4*>(m + (p * G::kMovers + mover) * 16);
            }
        }
        if (strip + 2 < end) fetch(strip + 2, stage == 0 ? 2 : stage - 1);
        if (FIRST || !g.last) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const f16x8 ph = rows_operand(m, in_strip, wr * 16, ks, 0), pl = rows_operand(m, in_strip, wr * 16, ks, 1);
#pragma unroll
                for (int j = 0; j < G::kGn; ++j)
                    gram[j] = product(rows_operand(m, in_strip, (wc * G::kGn + j) * 16, ks, 0),
                                      rows_operand(m, in_strip, (wc * G::kGn + j) * 16, ks, 1), ph, pl, gram[j]);
            }
        }
        stage = stage == 2 ? 0 : stage + 1;
    }
    if (!FIRST && g.last) return;
    f32x4* to = reinterpret_cast<f32x4*>(g.gram_next) + (int64_t(matrix) * g.parts + part) * (RP * RP / 4);
#pragma unroll
    for (int j = 0; j < G::kGn; ++j) to[(wr * G::kF + wc * G::kGn + j) * 64 + lane] = gram[j];
}

// B of a matrix, in the order in which stack_strip_kernel's lanes take it.
template <int RP>
constexpr int kPolyThreads = RP == 32 ? 256 : 1024;

template <int RP>
__global__ __launch_bounds__(kPolyThreads<RP>) void stack_poly_kernel(const StripArgs g) {
    using P = Poly<RP, kPolyThreads<RP> / 64>;
    __shared__ __attribute__((aligned(1024))) unsigned char a[P::kBytes];
    const int matrix = blockIdx.x, lane = threadIdx.x & 63;
    P poly;
    poly.run(g, matrix, g.scales[int64_t(matrix) * kStackScales], a);
    unsigned char* b = reinterpret_cast<unsigned char*>(g.b) + int64_t(matrix) * RP * RP * 4;
#pragma unroll
    for (int q = 0; q < P::kMine; ++q) {
        const int m = lane & 15, n = (poly.fj + q) * 16 + 4 * (lane >> 4);  // elements (m, n..n+3)
        f16x4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const Pair p = split(poly.b[q][e]);
            hi[e] = p.hi, lo[e] = p.lo;
        }
        unsigned char* at = b +
                            (((poly.fi * P::kSteps + (n >> 5)) * 2) * 64 + ((n & 31) >> 3) * 16 + m) * 16 + (n & 4) * 2;
        *reinterpret_cast<f16x4*>(at) = hi;
        *reinterpret_cast<f16x4*>(at + 1024) = lo;
    }
}

}  // namespace

bool stack_is_whole(const StackShape& sh) { return stack_whole_lds(sh) <= kStackWholeLds; }

hipError_t launch_stack_whole(const muon_stack_t& st, const StackShape& sh, const StackPlan& plan,
                              float scale, hipStream_t s) {
    WholeArgs w{};
    InArgs& in = w.in;
    in.in = st.in, in.out = st.out;
    in.in_stride = st.in_stride, in.in_row = st.in_row;
    in.out_stride = st.out_stride, in.out_row = st.out_row;
    in.rows = int32_t(st.rows), in.cols = int32_t(st.cols);
    in.cp = int32_t(sh.cp), in.plan = plan, in.scale = scale;
    w.tall = sh.tall, w.out_bf16 = st.out_dtype == MUON_DTYPE_BF16;
    const size_t lds = stack_whole_lds(sh);
    const dim3 grid = dim3(unsigned(st.count)), block = dim3(kWholeThreads);
    const auto run = [&](auto kernel) {
        if (lds > 64 * 1024) {
            // has to be told
            const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize,
                                                     int(kStackWholeLds));
            if (e != hipSuccess) return e;
        }
        LaunchTimer timer("stack_whole", s);
        kernel<<<grid, block, lds, s>>>(w);
        return hipGetLastError();
    };
    const bool bf16 = st.in_dtype == MUON_DTYPE_BF16;
    if (sh.r <= 32) return bf16 ? run(stack_whole_kernel<32, uint16_t>) : run(stack_whole_kernel<32, float>);
    return bf16 ? run(stack_whole_kernel<64, uint16_t>) : run(stack_whole_kernel<64, float>);
}

namespace {

template <int RP, typename T>
hipError_t run_strips(StripArgs g, float* const (&gram)[2], int64_t count, const StackScale* scales,
                      const StackPlan& plan, hipStream_t s) {
    const dim3 grid = dim3(unsigned(g.parts * count)), block = dim3(StripGeo<RP>::kThreads);
    const bool whole = g.parts <= (g.parts * count <= 64 ? 4 : 2);
    {
        LaunchTimer timer("stack_gram", s);
        g.gram_next = gram[0];
        stack_strip_kernel<RP, kGram, T><<<grid, block, 0, s>>>(g);
    }
    hipError_t e = hipGetLastError();
    for (int t = 0; t < plan.n && e == hipSuccess; ++t) {
        g.scales = scales + t, g.step = plan.steps[t], g.last = t + 1 == plan.n;
        g.gram = gram[t & 1], g.gram_next = gram[(t + 1) & 1];
        if (!whole) {
            LaunchTimer timer("stack_poly", s);
            stack_poly_kernel<RP><<<dim3(unsigned(count)), dim3(kPolyThreads<RP>), 0, s>>>(g);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        LaunchTimer timer("stack_strip", s);
        if (t == 0)
            whole ? stack_strip_kernel<RP, kWholeStep, T><<<grid, block, 0, s>>>(g)
                  : stack_strip_kernel<RP, kStep, T><<<grid, block, 0, s>>>(g);
        else
            whole ? stack_strip_kernel<RP, kWholeStep, void><<<grid, block, 0, s>>>(g)
                  : stack_strip_kernel<RP, kStep, void><<<grid, block, 0, s>>>(g);
        e = hipGetLastError();
    }
    return e;
}

template <typename T>
hipError_t run_strips(int64_t rp, const StripArgs& g, float* const (&gram)[2], int64_t count,
                      const StackScale* scales, const StackPlan& plan, hipStream_t s) {
    if (rp == 32) return run_strips<32, T>(g, gram, count, scales, plan, s);
    return rp == 64 ? run_strips<64, T>(g, gram, count, scales, plan, s)
                    : run_strips<128, T>(g, gram, count, scales, plan, s);
}

}  // namespace

hipError_t launch_stack_strips(const muon_stack_t& st, const StackShape& sh, int64_t count, const InArgs& in,
                               void* x, void* gram0, void* gram1, void* b, const StackPlan& plan, float scale,
                               hipStream_t s) {
    StripArgs g{};
    g.in = in;
    g.x = static_cast<_Float16*>(x), g.b = static_cast<_Float16*>(b);
    float* const gram[2] = {static_cast<float*>(gram0), static_cast<float*>(gram1)};
    g.out = in.out, g.out_stride = st.out_stride, g.out_row = st.out_row;
    g.cp = int32_t(sh.cp), g.rows = int32_t(st.rows), g.cols = int32_t(st.cols);
    g.tall = sh.tall, g.out_bf16 = st.out_dtype == MUON_DTYPE_BF16, g.scale = scale;
    // about a workgroup a CU for the whole stack (not for `count`, so that groups make the same
    // sums), and no more partial Gram matrices than the second iterate's place holds
    const int64_t strips = sh.cp / 64, resident = sh.rp == 128 ? 256 : 768;
    const int64_t want = std::max<int64_t>(1, resident / st.count);
    const int64_t parts = std::min({strips, want, sh.cp / sh.rp, int64_t(32)});
    g.per = int32_t((strips + parts - 1) / parts);
    g.parts = int32_t((strips + g.per - 1) / g.per);
    return st.in_dtype == MUON_DTYPE_BF16 ? run_strips<uint16_t>(sh.rp, g, gram, count, in.scales, plan, s)
                                          : run_strips<float>(sh.rp, g, gram, count, in.scales, plan, s);
}

}  // namespace muon
