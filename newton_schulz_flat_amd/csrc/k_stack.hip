// Newton-Schulz orthogonalization of a stack of equal matrices in float32 accuracy.
//
//   A = X X^T,  B = b A + c A A,  X <- a X + B X        (X is r x c, r <= c)
//
// Every matrix is held as pairs of float16: v 2^s = hi + lo with hi the nearest float16
// and lo that of what hi lacks, 22 bits together.  s is worked out for each matrix of the stack
// and each step from a bound on the matrix's largest singular value, ||U|| / (||U|| + 1e-7) at
// first, so that nothing overflows and small entries keep their digits.  A product takes three of
// the four products of the halves,
//   hi hi + hi lo + lo hi,
// on the float16 matrix cores with float32 sums; lo lo is below 2^-22 of the largest
// term, the pairs' own rounding.  Three 16-bit products at 16 times the rate of a float32
// one: about a third of the 16-bit rate, in float32 accuracy.
//
// Layout: along a row, each 32 elements are 128 bytes, 32 highs and then 32 lows, so that
// one K step of 32 is one 128-byte line of both halves; blocks of 32 columns lie one behind the
// other.  All products are of the form C = P Q^T with P and Q rows along K; stage X's Q = X^T is
// read from X's rows with transposing LDS reads.  Stages A and B are symmetric: tiles on and above the
// diagonal only, mirrored by the epilogue.
//
// Main loop: K steps of 32, two of them in LDS (64-tiles: four), filled by loads that go from memory to
// LDS directly (global_load_lds, 16 bytes a lane), one barrier a step.  The
// instruction's first operand is Q's rows, so that a lane holds four neighbouring elements of
// a row of C.
//
// Five steps of 14336 x 4096 take 9.9 to 10.3 ms by machine, 1.15 to 1.19 PFLOP/s of float16 operations (a large
// library product reaches 1.31): matrix instructions are busy 63 to 70% of the cycles at 1.8 GHz.
#include <algorithm>
#include <type_traits>

#include "stack_device.h"

namespace muon {

namespace {

// ------------------------------------------------------------- norm and split

// Four neighbouring elements of which the first `left` exist.
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
__device__ __forceinline__ void load_four(const float* p, int left, float v[4]) {
    if (left >= 4) {
        const f32x4_any t = *reinterpret_cast<const f32x4_any*>(p);
        v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = k < left ? p[k] : 0.f;
    }
}
__device__ __forceinline__ void load_four(const uint16_t* p, int left, float v[4]) {
    if (left >= 4) {
        const u32x2_any t = *reinterpret_cast<const u32x2_any*>(p);
        v[0] = __uint_as_float(t.x << 16), v[1] = __uint_as_float(t.x & 0xffff0000u);
        v[2] = __uint_as_float(t.y << 16), v[3] = __uint_as_float(t.y & 0xffff0000u);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = k < left ? load_one(p + k) : 0.f;
    }
}

// Sum of squares in float64 (squares of float32 are exact there): part b % parts of matrix
// b / parts, a contiguous run of its groups of four elements, then over the workgroup in fixed order.
template <typename T>
__global__ __launch_bounds__(256) void stack_norm_kernel(const InArgs a) {
    __shared__ double sums[4];
    const int matrix = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
    const T* u = static_cast<const T*>(a.in) + matrix * a.in_stride;
    const uint32_t per = uint32_t(a.cols + 3) / 4, groups = uint32_t(a.rows) * per;
    const uint32_t run = (groups + a.parts - 1) / a.parts, end = min(groups, (part + 1) * run);
    double sum = 0.;
#pragma unroll 4
    for (uint32_t e = part * run + threadIdx.x; e < end; e += 256) {
        const uint32_t i = e / per, j = (e - i * per) * 4;
        float v[4];
        load_four(u + int64_t(i) * a.in_row + j, a.cols - int(j), v);
#pragma unroll
        for (int k = 0; k < 4; ++k) sum = fma(double(v[k]), double(v[k]), sum);
    }
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0)
        a.partial[int64_t(matrix) * a.part_slots + part] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// X = U / (||U|| + 1e-7) in the iteration's orientation, zero in the padding, 64 x 64 tiles.
// A matrix's first tile also works out its exponents.
template <typename T, bool TALL>
__global__ __launch_bounds__(256) void stack_split_kernel(const InArgs a) {
    __shared__ float tile[64][65];
    const int across = a.cp / 64, per = (a.rp + 63) / 64 * across;
    const int matrix = blockIdx.x / per, t = blockIdx.x % per;
    const int i0 = t / across * 64, j0 = t % across * 64;  // in the iteration's orientation
    const double norm = matrix_norm(a.partial + int64_t(matrix) * a.part_slots, a.parts);
    const float inv = inverse_of(norm);
    float top = first_bound(norm);
    const int sx = top < kStackSmallBound ? stack_exponent(top, kStackLeastX) : a.plan.scales[0].sx;
    const float up = stack_scaled(1.f, sx - kInverseUp);
    if (t == 0 && threadIdx.x == 0) {
        StackScale* out = a.scales + int64_t(matrix) * kStackScales;
        if (top < kStackSmallBound) {
            for (int k = 0; k < a.plan.n; ++k) out[k] = stack_scale(a.plan.steps[k], top);
            out[a.plan.n] = {int16_t(stack_exponent(top, kStackLeastX)), 0, 0, 0};
        }
    }
    if (t == 0 && !(first_bound(norm) < kStackSmallBound) && int(threadIdx.x) <= a.plan.n)
        a.scales[int64_t(matrix) * kStackScales + threadIdx.x] = a.plan.scales[threadIdx.x];
    const T* u = static_cast<const T*>(a.in) + matrix * a.in_stride;
    const int x = threadIdx.x & 63;
    for (int y = threadIdx.x >> 6; y < 64; y += 4) {
        const int i = TALL ? j0 + y : i0 + y, j = TALL ? i0 + x : j0 + x;
        const bool there = i < a.rows && j < a.cols;
        tile[y][x] = there ? load_one(u + int64_t(i) * a.in_row + j) * inv : 0.f;
    }
    __syncthreads();
    _Float16* out = a.x + int64_t(matrix) * a.rp * 2 * a.cp;
    for (int y = threadIdx.x >> 6; y < min(64, a.rp - i0); y += 4) {
        const Pair p = split((TALL ? tile[x][y] : tile[y][x]) * up);
        _Float16* q = out + pair_at(i0 + y, j0 + x, a.rp);
        q[0] = p.hi, q[32] = p.lo;
    }
}

template <typename TI, typename TO>
__global__ __launch_bounds__(256) void stack_scaled_kernel(const InArgs a) {
    const int matrix = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
    const float inv = inverse_of(matrix_norm(a.partial + int64_t(matrix) * a.part_slots, a.parts));
    const TI* u = static_cast<const TI*>(a.in) + matrix * a.in_stride;
    TO* o = static_cast<TO*>(a.out) + matrix * a.out_stride;
    const uint32_t numel = uint32_t(a.rows) * uint32_t(a.cols);
    for (uint64_t e = uint64_t(part) * 256 + threadIdx.x; e < numel; e += uint64_t(a.parts) * 256) {
        const uint32_t i = uint32_t(e) / uint32_t(a.cols), j = uint32_t(e) - i * uint32_t(a.cols);
        store_one(o + int64_t(i) * a.out_row + j,
                  stack_scaled(load_one(u + int64_t(i) * a.in_row + j) * inv, -kInverseUp) * a.scale);
    }
}

// ------------------------------------------------------------------ products

struct ProductArgs {
    const _Float16* x;  // [matrix][cp / 32][rp][64]
    _Float16* x_next;
    _Float16* a;        // [matrix][rp / 32][rp][64]
    _Float16* b;
    float* shared;      // [matrix][slot][tile of 16 x 16][thread][4]
    void* out;          // last stage X: the result
    int64_t out_stride, out_row;
    int32_t rp, cp;
    int32_t rows, cols;  // of the result
    int32_t tiles, workers;
    int64_t per;         // K steps of a workgroup
    int32_t tall, out_bf16, last;
    const StackScale* scales;  // this step's, of matrix 0
    StackStep step;
    float scale;
};

// Loads go as many K steps ahead as LDS has stages (less one): a 64-tile's step is too
// short to cover a load.
template <int TILE>
struct Geo {
    static constexpr int kWaves = TILE == 256 ? 8 : 4;
    static constexpr int kThreads = kWaves * 64;
    static constexpr int kWm = TILE / 2, kWn = TILE / (kWaves / 2);  // of a wave
    static constexpr int kMi = kWm / 16, kNj = kWn / 16;
    static constexpr int kOp = TILE * 128;  // bytes of one operand's K step
    static constexpr int kLoads = kOp / (kThreads * 16);
    static constexpr int kStages = TILE == 64 ? 4 : 2;
    static constexpr int kLds = kStages * 2 * kOp;
    static constexpr int kMinWaves = 2;
};

// Tile t of a matrix: stage X in bands of 4 tile rows, column by column; the others those
// on and above the diagonal, column by column.
template <int STAGE>
__device__ __forceinline__ void place_of(int t, int tm, int tn, int& ti, int& tj) {
    if constexpr (STAGE == kStageX) {
        const int band = t / (4 * tn), rest = t - band * 4 * tn, high = min(4, tm - band * 4);
        ti = band * 4 + rest % high, tj = rest / high;
    } else {
        tj = int((sqrtf(8.f * float(t) + 1.f) - 1.f) * 0.5f);
        while (tj * (tj + 1) / 2 > t) --tj;
        while ((tj + 1) * (tj + 2) / 2 <= t) ++tj;
        ti = t - tj * (tj + 1) / 2;
    }
}

// C (or O) = own * (the axpy's operand as stored) + down * (the sums); N rows of 16 x 16 tiles of each
// wave, from row i0 on.
template <int TILE, int STAGE, int N>
__device__ __forceinline__ void finish(const ProductArgs& g, int matrix, int ti, int tj, int i0,
                                       const f32x4 (&acc)[N][Geo<TILE>::kNj]) {
    using G = Geo<TILE>;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m0 = ti * TILE + (wave / (G::kWaves / 2)) * G::kWm, n0 = tj * TILE + (wave % (G::kWaves / 2)) * G::kWn;
    const int64_t x_at = int64_t(matrix) * g.rp * 2 * g.cp, a_at = int64_t(matrix) * g.rp * 2 * g.rp;
    const StackScale* ex = g.scales + int64_t(matrix) * kStackScales;
    StackFactors f = {0.f, 0.f, 1.f};
    if constexpr (STAGE == kStageA)
        f.down = stack_a_factor(ex[0]);
    else if constexpr (STAGE == kStageB)
        f = stack_b_factors(g.step, ex[0]);
    else
        f = stack_x_factors(g.step, ex[0], ex[1].sx, g.last, g.scale);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int m = m0 + 16 * (i0 + i) + (lane & 15);
#pragma unroll
        for (int j = 0; j < G::kNj; ++j) {
            const int n = n0 + 16 * j + 4 * (lane >> 4);
            if (m >= g.rp || n >= (STAGE == kStageX ? g.cp : g.rp)) continue;
            float v[4];
#pragma unroll
            for (int t4 = 0; t4 < 4; ++t4) v[t4] = acc[i][j][t4] * f.down;
            if constexpr (STAGE != kStageA) {
                const _Float16* w = (STAGE == kStageX ? g.x + x_at : g.a + a_at) + pair_at(m, n, g.rp);
                const f16x4 hi = *reinterpret_cast<const f16x4*>(w);
                const f16x4 lo = *reinterpret_cast<const f16x4*>(w + 32);
#pragma unroll
                for (int t4 = 0; t4 < 4; ++t4) v[t4] += f.own * (float(hi[t4]) + float(lo[t4]));
            }
            if constexpr (STAGE == kStageX) {
                if (g.last) {
#pragma unroll
                    for (int t4 = 0; t4 < 4; ++t4) v[t4] *= f.after;
                    if (g.out_bf16)
                        store_result(static_cast<uint16_t*>(g.out) + matrix * g.out_stride, g.out_row, g.tall,
                                     g.rows, g.cols, m, n, v);
                    else
                        store_result(static_cast<float*>(g.out) + matrix * g.out_stride, g.out_row, g.tall,
                                     g.rows, g.cols, m, n, v);
                    continue;
                }
                store_pairs(g.x_next + x_at + pair_at(m, n, g.rp), v);
            } else {
                _Float16* c = (STAGE == kStageA ? g.a : g.b) + a_at;
                store_pairs(c + pair_at(m, n, g.rp), v);
                if (ti != tj)
#pragma unroll
                    for (int t4 = 0; t4 < 4; ++t4) {
                        const Pair s = split(v[t4]);
                        _Float16* q = c + pair_at(n + t4, m, g.rp);
                        q[0] = s.hi, q[32] = s.lo;
                    }
            }
        }
    }
}

// A workgroup takes g.per K steps of its matrix's tiles, tile after tile: whole tiles are finished
// at once, of the others the sums are left in a slot for stack_join_kernel.  Worker w's sum
// over tile t lies in slot w + t (one of the two grows from one piece to the next).
template <int TILE, int STAGE>
__global__ __launch_bounds__(Geo<TILE>::kThreads, Geo<TILE>::kMinWaves) void stack_gemm_kernel(
    const ProductArgs g) {
    using G = Geo<TILE>;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[G::kLds];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int matrix = blockIdx.x / g.workers;
    // workgroups go to the 8 XCDs in turn; each XCD takes a contiguous run of a matrix's work
    const int b = blockIdx.x - matrix * g.workers, low = g.workers >> 3, more = g.workers & 7;
    const int worker = (b & 7) * low + min(b & 7, more) + (b >> 3);
    const int tm = (g.rp + TILE - 1) / TILE, tn = (g.cp + TILE - 1) / TILE;
    const int64_t x_at = int64_t(matrix) * g.rp * 2 * g.cp, a_at = int64_t(matrix) * g.rp * 2 * g.rp;

    // operands: blocks of 32 columns of rp rows of 128 bytes.  P and, but for stage X, Q take one a
    // K step; stage X's Q takes 32 rows of TILE / 32 of them
    const unsigned char* p_base = reinterpret_cast<const unsigned char*>(
        STAGE == kStageA ? g.x + x_at : STAGE == kStageB ? g.a + a_at : g.b + a_at);
    const unsigned char* q_base = reinterpret_cast<const unsigned char*>(
        STAGE == kStageB ? g.a + a_at : g.x + x_at);
    const int k_steps = (STAGE == kStageA ? g.cp : g.rp) / 32;
    const int64_t block = int64_t(g.rp) * 128;
    const int64_t q_step = STAGE == kStageX ? 32 * 128 : block;
    const uint32_t lds0 = lds_address(lds);

    // Rows along K: a thread loads chunk (tid % 8) ^ (row / 2 % 8) of rows tid / 8 + p * rows of a pass; with
    // rows of a pass a multiple of 16 the swizzle is the same in every pass.  Rows behind
    // the last one (sides are padded to 64, tiles may be longer) repeat a row that exists.
    constexpr int kRows = G::kThreads / 8;
    const int lr = tid >> 3;
    const uint32_t lc = uint32_t((tid & 7) ^ ((lr >> 1) & 7)) * 16;
    const int wm = (wave / (G::kWaves / 2)) * G::kWm, wn = (wave % (G::kWaves / 2)) * G::kWn;
    auto rows_fragment = [&](const unsigned char* op, int row0, int half) {
        const int r = row0 + (lane & 15);
        return *reinterpret_cast<const f16x8*>(
            op + r * 128 + ((((lane >> 4) + 4 * half) ^ ((r >> 1) & 7)) << 4));
    };
    auto turned_fragment = [&](const unsigned char* op, int col0, int half) {
        const int l = lane & 15, k = (lane >> 4) * 8 + (l >> 2);
        const int c = (col0 >> 5) * 8 + half * 4 + ((col0 >> 4) & 1) * 2 + ((l & 3) >> 1);
        const int f = 2 * ((k & 3) | ((k >> 3) & 1) << 2);
        const unsigned char* at = op + k * (TILE * 4) + ((c ^ f) << 4) + (l & 1) * 8;
        // the second read's rows are 4 further on, where the swizzle is the same
        const uint2 lo = read_turned(at), hi = read_turned(at + 4 * TILE * 4);
        return __builtin_bit_cast(f16x8, u32x4{lo.x, lo.y, hi.x, hi.y});
    };

    const int64_t end = min(int64_t(g.tiles) * k_steps, (worker + 1) * g.per);
    for (int64_t at = worker * g.per; at < end;) {
        const int t = int(at / k_steps), k0 = int(at - int64_t(t) * k_steps);
        const int k1 = int(min(int64_t(k_steps), k0 + (end - at)));
        int ti, tj;
        place_of<STAGE>(t, tm, tn, ti, tj);
        const int m0 = ti * TILE, n0 = tj * TILE;
        uint32_t p_off[G::kLoads], q_off[G::kLoads];
#pragma unroll
        for (int p = 0; p < G::kLoads; ++p) {
            p_off[p] = uint32_t(min(lr + p * kRows, g.rp - 1 - m0)) * 128 + lc;
            if constexpr (STAGE == kStageX) {
                // K rows of TILE columns: TILE / 4 chunks a row; columns behind the last block
                // of 32 repeat the last one
                constexpr int kAcross = TILE / 4;
                const int pos = tid + p * G::kThreads, k = pos / kAcross;
                const int f = 2 * ((k & 3) | ((k >> 3) & 1) << 2);
                const int c = (pos % kAcross) ^ f;
                q_off[p] = uint32_t(min(c >> 3, (g.cp - n0) / 32 - 1) * block) + uint32_t(k * 128 + (c & 7) * 16);
            } else {
                q_off[p] = uint32_t(min(lr + p * kRows, g.rp - 1 - n0)) * 128 + lc;
            }
        }
        const unsigned char* p_at = p_base + int64_t(m0) * 128 + k0 * block;
        const unsigned char* q_at = q_base + (STAGE == kStageX ? n0 / 32 * block : int64_t(n0) * 128) + k0 * q_step;
        // the loads of the next K step into a stage; behind the last step its own once more, so that
        // the number on their way stays the same
        int fetched = k0;
        auto fetch = [&](int stage) {
            const uint32_t to = lds0 + stage * 2 * G::kOp + wave * 1024;
#pragma unroll
            for (int p = 0; p < G::kLoads; ++p) {
                load_to_lds(p_at, p_off[p], to + p * G::kThreads * 16);
                load_to_lds(q_at, q_off[p], to + G::kOp + p * G::kThreads * 16);
            }
            if (++fetched < k1) p_at += block, q_at += q_step;
        };

        f32x4 acc[G::kMi][G::kNj];
#pragma unroll
        for (int i = 0; i < G::kMi; ++i)
#pragma unroll
            for (int j = 0; j < G::kNj; ++j) acc[i][j] = {0.f, 0.f, 0.f, 0.f};

#pragma unroll
        for (int p = 0; p < G::kStages - 1; ++p) fetch(p);
        int stage = 0, ahead = G::kStages - 1;
        for (int ks = k0; ks < k1; ++ks) {
            wait_loads<(G::kStages - 2) * 2 * G::kLoads>();
            __syncthreads();
            const unsigned char* p_lds = lds + stage * 2 * G::kOp;
            const unsigned char* q_lds = p_lds + G::kOp;
            // P's first rows before Q's: LDS returns in order, and the first products wait for fewer reads
            // (1024 x 1024 196 us to 188; larger tiles have steps that are long enough, 1% slower)
            constexpr bool kEarly = TILE == 64;
            f16x8 early_h, early_l;
            if constexpr (kEarly) early_h = rows_fragment(p_lds, wm, 0), early_l = rows_fragment(p_lds, wm, 1);
            f16x8 qh[G::kNj], ql[G::kNj];
#pragma unroll
            for (int j = 0; j < G::kNj; ++j) {
                if constexpr (STAGE == kStageX) {
                    qh[j] = turned_fragment(q_lds, wn + 16 * j, 0);
                    ql[j] = turned_fragment(q_lds, wn + 16 * j, 1);
                } else {
                    qh[j] = rows_fragment(q_lds, wn + 16 * j, 0);
                    ql[j] = rows_fragment(q_lds, wn + 16 * j, 1);
                }
            }
            if (G::kStages > 2 || ks + 1 < k1) fetch(ahead);
#pragma unroll
            for (int i = 0; i < G::kMi; ++i) {
                const f16x8 ph = kEarly && i == 0 ? early_h : rows_fragment(p_lds, wm + 16 * i, 0);
                const f16x8 pl = kEarly && i == 0 ? early_l : rows_fragment(p_lds, wm + 16 * i, 1);
#pragma unroll
                for (int j = 0; j < G::kNj; ++j) acc[i][j] = mfma(ql[j], ph, acc[i][j]);
#pragma unroll
                for (int j = 0; j < G::kNj; ++j) acc[i][j] = mfma(qh[j], pl, acc[i][j]);
#pragma unroll
                for (int j = 0; j < G::kNj; ++j) acc[i][j] = mfma(qh[j], ph, acc[i][j]);
            }
            stage = stage + 1 == G::kStages ? 0 : stage + 1;
            ahead = ahead + 1 == G::kStages ? 0 : ahead + 1;
        }
        wait_loads();     // the repeated ones: LDS must be left alone
        __syncthreads();  // the next piece's loads go where this one's were
        if (k0 == 0 && k1 == k_steps) {
            finish<TILE, STAGE, G::kMi>(g, matrix, ti, tj, 0, acc);
        } else {
            f32x4* to = reinterpret_cast<f32x4*>(g.shared) +
                        (int64_t(matrix) * (g.workers + g.tiles) + worker + t) * (TILE * TILE / 4) + tid;
#pragma unroll
            for (int i = 0; i < G::kMi; ++i)
#pragma unroll
                for (int j = 0; j < G::kNj; ++j) to[(i * G::kNj + j) * G::kThreads] = acc[i][j];
        }
        at += k1 - k0;
    }
}

// Tiles whose K steps several workers share: their sums in the workers' order, and the rest.  A
// workgroup takes one row of 16 x 16 tiles of each wave.
template <int TILE, int STAGE>
__global__ __launch_bounds__(Geo<TILE>::kThreads) void stack_join_kernel(const ProductArgs g) {
    using G = Geo<TILE>;
    const int i = blockIdx.x % G::kMi;
    const int matrix = blockIdx.x / G::kMi / g.tiles, t = blockIdx.x / G::kMi % g.tiles;
    const int k_steps = (STAGE == kStageA ? g.cp : g.rp) / 32;
    const int first = int(int64_t(t) * k_steps / g.per), last = int((int64_t(t + 1) * k_steps - 1) / g.per);
    if (first == last) return;
    const f32x4* from = reinterpret_cast<const f32x4*>(g.shared) +
                        (int64_t(matrix) * (g.workers + g.tiles) + first + t) * (TILE * TILE / 4) +
                        i * G::kNj * G::kThreads + threadIdx.x;
    f32x4 acc[1][G::kNj];
#pragma unroll
    for (int j = 0; j < G::kNj; ++j) acc[0][j] = from[j * G::kThreads];
#pragma unroll 2
    for (int w = first + 1; w <= last; ++w) {
        from += TILE * TILE / 4;
#pragma unroll
        for (int j = 0; j < G::kNj; ++j) acc[0][j] += from[j * G::kThreads];
    }
    int ti, tj;
    place_of<STAGE>(t, (g.rp + TILE - 1) / TILE, (g.cp + TILE - 1) / TILE, ti, tj);
    finish<TILE, STAGE, 1>(g, matrix, ti, tj, i, acc);
}

template <int TILE, int STAGE>
hipError_t enqueue_stage(const ProductArgs& g, int64_t count, hipStream_t s) {
    const dim3 block = dim3(Geo<TILE>::kThreads);
    {
        LaunchTimer timer(STAGE == kStageA ? "stack_a" : STAGE == kStageB ? "stack_b" : "stack_x", s);
        stack_gemm_kernel<TILE, STAGE><<<dim3(unsigned(g.workers * count)), block, 0, s>>>(g);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || g.workers == g.tiles) return e;
    LaunchTimer timer("stack_join", s);
    stack_join_kernel<TILE, STAGE>
        <<<dim3(unsigned(int64_t(g.tiles) * Geo<TILE>::kMi * count)), block, 0, s>>>(g);
    return hipGetLastError();
}

template <int STAGE>
hipError_t run_stage(ProductArgs g, const StackShape& sh, int64_t count, int64_t all, hipStream_t s) {
    // by the whole stack's count, so that groups of it are summed in the same order
    const StackTiling t = stack_tiling(STAGE, sh, all);
    g.tiles = int32_t(t.tiles), g.workers = int32_t(t.workers), g.per = t.per;
    switch (t.tile) {
        case 256: return enqueue_stage<256, STAGE>(g, count, s);
        case 128: return enqueue_stage<128, STAGE>(g, count, s);
        default: return enqueue_stage<64, STAGE>(g, count, s);
    }
}

// `count` matrices whose intermediates fit the workspace.
hipError_t run_group(const muon_stack_t& st, const StackShape& sh, int64_t first, int64_t count,
                     const StackPlan& plan, float scale, void* workspace, hipStream_t s) {
    const size_t in_es = st.in_dtype == MUON_DTYPE_BF16 ? 2 : 4, out_es = st.out_dtype == MUON_DTYPE_BF16 ? 2 : 4;
    unsigned char* w = static_cast<unsigned char*>(workspace);
    double* partial = reinterpret_cast<double*>(w);
    w += size_t(count) * size_t(stack_part_slots(sh.r, sh.c)) * sizeof(double);
    StackScale* scales = reinterpret_cast<StackScale*>(w);
    w += size_t(count) * kStackScales * sizeof(StackScale);
    const size_t x_bytes = size_t(count) * sh.rp * sh.cp * 4, a_bytes = size_t(count) * sh.rp * sh.rp * 4;
    _Float16* x[2] = {reinterpret_cast<_Float16*>(w), reinterpret_cast<_Float16*>(w + x_bytes)};
    _Float16* a = reinterpret_cast<_Float16*>(w + 2 * x_bytes);
    _Float16* b = reinterpret_cast<_Float16*>(w + 2 * x_bytes + a_bytes);

    InArgs in;
    in.in = static_cast<const unsigned char*>(st.in) + size_t(first * st.in_stride) * in_es;
    in.out = static_cast<unsigned char*>(st.out) + size_t(first * st.out_stride) * out_es;
    in.in_stride = st.in_stride, in.in_row = st.in_row;
    in.out_stride = st.out_stride, in.out_row = st.out_row;
    in.partial = partial, in.x = x[0];
    in.rows = int32_t(st.rows), in.cols = int32_t(st.cols);
    in.rp = int32_t(sh.rp), in.cp = int32_t(sh.cp);
    in.parts = int32_t(stack_parts(sh.r, sh.c)), in.part_slots = int32_t(stack_part_slots(sh.r, sh.c));
    in.scale = scale, in.scales = scales, in.plan = plan;
    const int n = plan.n;
    const bool bf16 = st.in_dtype == MUON_DTYPE_BF16;
    {
        LaunchTimer timer("stack_norm", s);
        const dim3 grid = dim3(unsigned(in.parts * count));
        if (bf16)
            stack_norm_kernel<uint16_t><<<grid, dim3(256), 0, s>>>(in);
        else
            stack_norm_kernel<float><<<grid, dim3(256), 0, s>>>(in);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (n == 0) {
        LaunchTimer timer("stack_scaled", s);
        const dim3 grid = dim3(unsigned(in.parts * count));
        const bool to16 = st.out_dtype == MUON_DTYPE_BF16;
        if (bf16)
            to16 ? stack_scaled_kernel<uint16_t, uint16_t><<<grid, dim3(256), 0, s>>>(in)
                 : stack_scaled_kernel<uint16_t, float><<<grid, dim3(256), 0, s>>>(in);
        else
            to16 ? stack_scaled_kernel<float, uint16_t><<<grid, dim3(256), 0, s>>>(in)
                 : stack_scaled_kernel<float, float><<<grid, dim3(256), 0, s>>>(in);
        return hipGetLastError();
    }
    if (sh.r <= 128)
        return launch_stack_strips(st, sh, count, in, x[0], x[1], reinterpret_cast<unsigned char*>(b) + a_bytes, b,
                                   plan, scale, s);
    {
        LaunchTimer timer("stack_split", s);
        const dim3 grid = dim3(unsigned((sh.rp + 63) / 64 * (sh.cp / 64) * count));
        if (bf16)
            sh.tall ? stack_split_kernel<uint16_t, true><<<grid, dim3(256), 0, s>>>(in)
                    : stack_split_kernel<uint16_t, false><<<grid, dim3(256), 0, s>>>(in);
        else
            sh.tall ? stack_split_kernel<float, true><<<grid, dim3(256), 0, s>>>(in)
                    : stack_split_kernel<float, false><<<grid, dim3(256), 0, s>>>(in);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;

    for (int t = 0; t < n; ++t) {
        ProductArgs g{};
        g.x = x[t & 1], g.x_next = x[(t + 1) & 1], g.a = a, g.b = b;
        g.out = in.out, g.out_stride = st.out_stride, g.out_row = st.out_row;
        g.rp = in.rp, g.cp = in.cp, g.rows = in.rows, g.cols = in.cols;
        g.tall = sh.tall, g.out_bf16 = st.out_dtype == MUON_DTYPE_BF16, g.last = t + 1 == n;
        g.scales = scales + t, g.step = plan.steps[t], g.scale = scale;
        g.shared = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(b) + a_bytes);
        if ((e = run_stage<kStageA>(g, sh, count, st.count, s)) != hipSuccess) return e;
        if ((e = run_stage<kStageB>(g, sh, count, st.count, s)) != hipSuccess) return e;
        if ((e = run_stage<kStageX>(g, sh, count, st.count, s)) != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_stack(const muon_stack_t& stack, const StackPlan& plan, float scale,
                        void* workspace, size_t workspace_bytes, hipStream_t s) {
    const StackShape sh = stack_shape(stack.rows, stack.cols);
    if (plan.n > 0 && stack_is_whole(sh)) return launch_stack_whole(stack, sh, plan, scale, s);
    // a grid counts below 2^32 work-items: at most 2^22 tiles of 64 x 64 in a group
    const int64_t per = (sh.rp + 63) / 64 * (sh.cp / 64);
    const int64_t held = int64_t(workspace_bytes / stack_matrix_bytes(sh, stack.count));
    const int64_t most = (int64_t(1) << 22) / std::max<int64_t>(per, kStackPartials);
    const int64_t fit = std::max<int64_t>(1, std::min(held, most));
    for (int64_t at = 0; at < stack.count; at += fit) {
        const hipError_t e = run_group(stack, sh, at, std::min(fit, stack.count - at), plan, scale, workspace,
                                       s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace muon
