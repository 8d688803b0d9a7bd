// Newton-Schulz orthogonalization of a stack of equal matrices in float32 accuracy.
//
//   A = X X^T,  B = b A + c A A,  X <- a X + B X        (X is r x c, r <= c)
//
// Every matrix is held as pairs of float16: v 2^s = hi + lo with hi the nearest float16
// and lo that of what hi lacks, 22 bits together.  s is worked out for each matrix of the stack
// and each step from a bound on the matrix's largest singular value, ||U|| / (||U|| + 1e-7) at
// first, so that nothing overflows and small entries keep their digits.  A product takes three of the four products of the halves,
//   hi hi + hi lo + lo hi,
// on the float16 matrix cores with float32 sums; lo lo is below 2^-22 of the largest
// term, the pairs' own rounding.  Three 16-bit products at 16 times the rate of a float32
// one: about a third of the 16-bit rate, in float32 accuracy.
//
// Layout: along a row, each 32 elements are 128 bytes, 32 highs and then 32 lows, so that
// one K step of 32 is one 128-byte line of both halves.  All products are of the form
// C = P Q^T with P and Q rows along K; stage X's Q = X^T is read from X's rows
// with transposing LDS reads.  Stages A and B are symmetric: tiles on and above the diagonal
// only, mirrored by the epilogue.
//
// Main loop: K steps of 32, double-buffered in LDS, filled by loads that go from memory to
// LDS directly (global_load_lds, 16 bytes a lane), one barrier a step.  The
// instruction's first operand is Q's rows, so that a lane holds four neighbouring elements of
// a row of C.
#include <algorithm>
#include <type_traits>

#include "stack_device.h"

namespace muon {

namespace {

enum Stage { kA = 0, kB = 1, kX = 2 };

// ------------------------------------------------------------- norm and split

// Sum of squares in float64 (squares of float32 are exact there): part b % parts of matrix
// b / parts, rows in turn, then over the workgroup in fixed order.
template <typename T>
__global__ __launch_bounds__(256) void stack_norm_kernel(const InArgs a) {
    __shared__ double sums[4];
    const int matrix = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
    const T* u = static_cast<const T*>(a.in) + matrix * a.in_stride;
    const uint32_t numel = uint32_t(a.rows) * uint32_t(a.cols);
    double sum = 0.;
    for (uint64_t e = uint64_t(part) * 256 + threadIdx.x; e < numel; e += uint64_t(a.parts) * 256) {
        const uint32_t i = uint32_t(e) / uint32_t(a.cols), j = uint32_t(e) - i * uint32_t(a.cols);
        const double v = load_one(u + int64_t(i) * a.in_row + j);
        sum = fma(v, v, sum);
    }
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0)
        a.partial[int64_t(matrix) * kStackPartials + part] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// X = U / (||U|| + 1e-7) in the iteration's orientation, zero in the padding, 64 x 64 tiles.
// A matrix's first tile also works out its exponents.
template <typename T, bool TALL>
__global__ __launch_bounds__(256) void stack_split_kernel(const InArgs a) {
    __shared__ float tile[64][65];
    const int across = a.cp / 64, per = a.rp / 64 * across;
    const int matrix = blockIdx.x / per, t = blockIdx.x % per;
    const int i0 = t / across * 64, j0 = t % across * 64;  // in the iteration's orientation
    const double norm = matrix_norm(a.partial + int64_t(matrix) * kStackPartials, a.parts);
    const float inv = inverse_of(norm);
    float top = first_bound(norm);
    const float up = power_of_two(stack_exponent(top, 0));
    if (t == 0 && threadIdx.x == 0) {
        StackScale* out = a.scales + int64_t(matrix) * kStackScales;
        for (int k = 0; k < a.n_steps; ++k) out[k] = stack_scale(a.steps[k], top);
        out[a.n_steps] = {stack_exponent(top, 0), 0, 0, 0};
    }
    const T* u = static_cast<const T*>(a.in) + matrix * a.in_stride;
    const int x = threadIdx.x & 63;
    for (int y = threadIdx.x >> 6; y < 64; y += 4) {
        const int i = TALL ? j0 + y : i0 + y, j = TALL ? i0 + x : j0 + x;
        const bool there = i < a.rows && j < a.cols;
        tile[y][x] = there ? load_one(u + int64_t(i) * a.in_row + j) * inv : 0.f;
    }
    __syncthreads();
    _Float16* out = a.x + int64_t(matrix) * a.rp * 2 * a.cp;
    for (int y = threadIdx.x >> 6; y < 64; y += 4) {
        const Pair p = split((TALL ? tile[x][y] : tile[y][x]) * up);
        _Float16* q = out + pair_at(i0 + y, j0 + x, a.cp);
        q[0] = p.hi, q[32] = p.lo;
    }
}

template <typename TI, typename TO>
__global__ __launch_bounds__(256) void stack_scaled_kernel(const InArgs a) {
    const int matrix = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
    const float inv = inverse_of(matrix_norm(a.partial + int64_t(matrix) * kStackPartials, a.parts));
    const TI* u = static_cast<const TI*>(a.in) + matrix * a.in_stride;
    TO* o = static_cast<TO*>(a.out) + matrix * a.out_stride;
    const uint32_t numel = uint32_t(a.rows) * uint32_t(a.cols);
    for (uint64_t e = uint64_t(part) * 256 + threadIdx.x; e < numel; e += uint64_t(a.parts) * 256) {
        const uint32_t i = uint32_t(e) / uint32_t(a.cols), j = uint32_t(e) - i * uint32_t(a.cols);
        store_one(o + int64_t(i) * a.out_row + j,
                  load_one(u + int64_t(i) * a.in_row + j) * inv * a.scale);
    }
}

// ------------------------------------------------------------------ products

struct ProductArgs {
    const _Float16* x;  // [matrix][rp][2 cp]
    _Float16* x_next;
    _Float16* a;        // [matrix][rp][2 rp]
    _Float16* b;
    void* out;          // last stage X: the result
    int64_t out_stride, out_row;
    int32_t rp, cp;
    int32_t rows, cols;  // of the result
    int32_t tiles;       // of one matrix
    int32_t tall, out_bf16, last;
    const StackScale* scales;  // this step's, of matrix 0
    StackStep step;
    float scale;
};

template <int TILE>
struct Geo {
    static constexpr int kWaves = TILE == 256 ? 8 : 4;
    static constexpr int kThreads = kWaves * 64;
    static constexpr int kWm = TILE / 2, kWn = TILE / (kWaves / 2);  // of a wave
    static constexpr int kMi = kWm / 16, kNj = kWn / 16;
    static constexpr int kOp = TILE * 128;           // bytes of one operand's K step
    static constexpr int kLoads = kOp / (kThreads * 16);
    static constexpr int kLds = 4 * kOp;
    static constexpr int kMinWaves = TILE == 256 ? 2 : TILE == 128 ? 2 : 4;
};

template <int TILE, int STAGE>
__global__ __launch_bounds__(Geo<TILE>::kThreads, Geo<TILE>::kMinWaves) void stack_gemm_kernel(
    const ProductArgs g) {
    using G = Geo<TILE>;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[G::kLds];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int matrix = blockIdx.x / g.tiles, t = blockIdx.x % g.tiles;
    const int tm = (g.rp + TILE - 1) / TILE;
    int ti, tj;
    if constexpr (STAGE == kX) {
        ti = t % tm, tj = t / tm;
    } else {
        // t counts the tiles on and above the diagonal, column by column
        tj = int((sqrtf(8.f * float(t) + 1.f) - 1.f) * 0.5f);
        while (tj * (tj + 1) / 2 > t) --tj;
        while ((tj + 1) * (tj + 2) / 2 <= t) ++tj;
        ti = t - tj * (tj + 1) / 2;
    }
    const int m0 = ti * TILE, n0 = tj * TILE;
    const int64_t x_at = int64_t(matrix) * g.rp * 2 * g.cp, a_at = int64_t(matrix) * g.rp * 2 * g.rp;

    // operands: rows of p_row bytes
    const unsigned char* p_base = reinterpret_cast<const unsigned char*>(
        STAGE == kA ? g.x + x_at : STAGE == kB ? g.a + a_at : g.b + a_at);
    const unsigned char* q_base = reinterpret_cast<const unsigned char*>(
        STAGE == kB ? g.a + a_at : g.x + x_at);
    const int64_t p_row = int64_t(STAGE == kA ? g.cp : g.rp) * 4, q_row = int64_t(STAGE == kB ? g.rp : g.cp) * 4;
    const int k_steps = (STAGE == kA ? g.cp : g.rp) / 32;
    const uint32_t lds0 = lds_address(lds);

    // Rows along K: a thread loads chunk (tid % 8) ^ (row / 2 % 8) of rows tid / 8 + p * rows of a pass; with
    // rows of a pass a multiple of 16 the swizzle is the same in every pass.  Rows behind
    // the last one (sides are padded to 64, tiles may be longer) repeat a row that exists.
    constexpr int kRows = G::kThreads / 8;
    const int lr = tid >> 3;
    const uint32_t lc = uint32_t((tid & 7) ^ ((lr >> 1) & 7)) * 16;
    uint32_t p_off[G::kLoads], q_off[G::kLoads];
#pragma unroll
    for (int p = 0; p < G::kLoads; ++p) {
        p_off[p] = uint32_t(min(lr + p * kRows, g.rp - 1 - m0) * p_row) + lc;
        if constexpr (STAGE == kX) {
            // K rows of TILE columns: TILE / 4 chunks a row; columns behind the last block
            // of 32 repeat the last one
            constexpr int kAcross = TILE / 4;
            const int pos = tid + p * G::kThreads, k = pos / kAcross;
            const int f = 2 * ((k & 3) | ((k >> 3) & 1) << 2);
            const int c = (pos % kAcross) ^ f;
            const int block = min(c >> 3, (g.cp - n0) / 32 - 1);
            q_off[p] = uint32_t(k * q_row) + uint32_t(block * 128 + (c & 7) * 16);
        } else {
            q_off[p] = uint32_t(min(lr + p * kRows, g.rp - 1 - n0) * q_row) + lc;
        }
    }
    const unsigned char* p_at = p_base + int64_t(m0) * p_row;
    const unsigned char* q_at = STAGE == kX ? q_base + int64_t(n0) * 4 : q_base + int64_t(n0) * q_row;
    const int64_t q_step = STAGE == kX ? 32 * q_row : 128;
    auto fetch = [&](int buf) {
        const uint32_t to = lds0 + buf * 2 * G::kOp + wave * 1024;
#pragma unroll
        for (int p = 0; p < G::kLoads; ++p) {
            load_to_lds(p_at, p_off[p], to + p * G::kThreads * 16);
            load_to_lds(q_at, q_off[p], to + G::kOp + p * G::kThreads * 16);
        }
        p_at += 128, q_at += q_step;
    };

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

    f32x4 acc[G::kMi][G::kNj];
#pragma unroll
    for (int i = 0; i < G::kMi; ++i)
#pragma unroll
        for (int j = 0; j < G::kNj; ++j) acc[i][j] = {0.f, 0.f, 0.f, 0.f};

    fetch(0);
    for (int ks = 0; ks < k_steps; ++ks) {
        wait_loads();
        __syncthreads();
        if (ks + 1 < k_steps) fetch((ks + 1) & 1);
        const unsigned char* p_lds = lds + (ks & 1) * 2 * G::kOp;
        const unsigned char* q_lds = p_lds + G::kOp;
        f16x8 qh[G::kNj], ql[G::kNj];
#pragma unroll
        for (int j = 0; j < G::kNj; ++j) {
            if constexpr (STAGE == kX) {
                qh[j] = turned_fragment(q_lds, wn + 16 * j, 0);
                ql[j] = turned_fragment(q_lds, wn + 16 * j, 1);
            } else {
                qh[j] = rows_fragment(q_lds, wn + 16 * j, 0);
                ql[j] = rows_fragment(q_lds, wn + 16 * j, 1);
            }
        }
#pragma unroll
        for (int i = 0; i < G::kMi; ++i) {
            const f16x8 ph = rows_fragment(p_lds, wm + 16 * i, 0);
            const f16x8 pl = rows_fragment(p_lds, wm + 16 * i, 1);
#pragma unroll
            for (int j = 0; j < G::kNj; ++j) acc[i][j] = mfma(ql[j], ph, acc[i][j]);
#pragma unroll
            for (int j = 0; j < G::kNj; ++j) acc[i][j] = mfma(qh[j], pl, acc[i][j]);
#pragma unroll
            for (int j = 0; j < G::kNj; ++j) acc[i][j] = mfma(qh[j], ph, acc[i][j]);
        }
    }

    // C (or O) = own * (the axpy's operand as stored) + down * (the sums), each with the exponents
    // of what it reads and of what is written
    const StackScale* ex = g.scales + int64_t(matrix) * kStackScales;
    const int to = STAGE == kA ? ex[0].sa : STAGE == kB ? ex[0].sb : g.last ? 0 : ex[1].sx;
    float down, own = 0.f;
    if constexpr (STAGE == kA) {
        down = power_of_two(to - 2 * ex[0].sx);
    } else if constexpr (STAGE == kB) {
        down = g.step.c * power_of_two(to - 2 * ex[0].sa), own = g.step.b * power_of_two(to - ex[0].sa);
    } else {
        down = power_of_two(to - ex[0].sx - ex[0].sb), own = g.step.a * power_of_two(to - ex[0].sx);
        if (g.last) down *= g.scale, own *= g.scale;
    }
#pragma unroll
    for (int i = 0; i < G::kMi; ++i) {
        const int m = m0 + wm + 16 * i + (lane & 15);
#pragma unroll
        for (int j = 0; j < G::kNj; ++j) {
            const int n = n0 + wn + 16 * j + 4 * (lane >> 4);
            if (m >= g.rp || n >= (STAGE == kX ? g.cp : g.rp)) continue;
            float v[4];
#pragma unroll
            for (int t4 = 0; t4 < 4; ++t4) v[t4] = acc[i][j][t4] * down;
            if constexpr (STAGE != kA) {
                const int64_t cp = STAGE == kX ? g.cp : g.rp;
                const _Float16* w = (STAGE == kX ? g.x + x_at : g.a + a_at) + pair_at(m, n, cp);
                const f16x4 hi = *reinterpret_cast<const f16x4*>(w);
                const f16x4 lo = *reinterpret_cast<const f16x4*>(w + 32);
#pragma unroll
                for (int t4 = 0; t4 < 4; ++t4) v[t4] += own * (float(hi[t4]) + float(lo[t4]));
            }
            if constexpr (STAGE == kX) {
                if (g.last) {
                    if (g.out_bf16)
                        store_result(static_cast<uint16_t*>(g.out) + matrix * g.out_stride, g.out_row, g.tall,
                                     g.rows, g.cols, m, n, v);
                    else
                        store_result(static_cast<float*>(g.out) + matrix * g.out_stride, g.out_row, g.tall,
                                     g.rows, g.cols, m, n, v);
                    continue;
                }
            }
            if constexpr (STAGE == kX) {
                store_pairs(g.x_next + x_at + pair_at(m, n, g.cp), v);
            } else {
                _Float16* c = (STAGE == kA ? g.a : g.b) + a_at;
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

template <int TILE>
hipError_t enqueue_stage(int stage, ProductArgs g, int64_t count, hipStream_t s) {
    const int64_t tm = (g.rp + TILE - 1) / TILE, tn = (g.cp + TILE - 1) / TILE;
    g.tiles = int32_t(stage == kX ? tm * tn : tm * (tm + 1) / 2);
    const dim3 grid = dim3(unsigned(g.tiles * count)), block = dim3(Geo<TILE>::kThreads);
    LaunchTimer timer(stage == kA ? "stack_a" : stage == kB ? "stack_b" : "stack_x", s);
    if (stage == kA)
        stack_gemm_kernel<TILE, kA><<<grid, block, 0, s>>>(g);
    else if (stage == kB)
        stack_gemm_kernel<TILE, kB><<<grid, block, 0, s>>>(g);
    else
        stack_gemm_kernel<TILE, kX><<<grid, block, 0, s>>>(g);
    return hipGetLastError();
}

// The largest tile of which a stage has enough to fill the chip.
int tile_for(int stage, int64_t rp, int64_t cp, int64_t count) {
    for (int tile : {256, 128}) {
        const int64_t tm = (rp + tile - 1) / tile, tn = (cp + tile - 1) / tile;
        if ((stage == kX ? tm * tn : tm * (tm + 1) / 2) * count >= 192) return tile;
    }
    return 64;
}

// The tile goes by the whole stack's count, so that groups of it are summed in the same order.
hipError_t run_stage(int stage, const ProductArgs& g, int64_t count, int64_t all, hipStream_t s) {
    switch (tile_for(stage, g.rp, g.cp, all)) {
        case 256: return enqueue_stage<256>(stage, g, count, s);
        case 128: return enqueue_stage<128>(stage, g, count, s);
        default: return enqueue_stage<64>(stage, g, count, s);
    }
}

// `count` matrices whose intermediates fit the workspace.
hipError_t run_group(const muon_stack_t& st, const StackShape& sh, int64_t first, int64_t count,
                     const StackStep* steps, int n, float scale, void* workspace, hipStream_t s) {
    const size_t in_es = st.in_dtype == MUON_DTYPE_BF16 ? 2 : 4, out_es = st.out_dtype == MUON_DTYPE_BF16 ? 2 : 4;
    unsigned char* w = static_cast<unsigned char*>(workspace);
    double* partial = reinterpret_cast<double*>(w);
    w += size_t(count) * kStackPartials * sizeof(double);
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
    in.parts = int32_t(std::min<int64_t>(kStackPartials, (sh.r * sh.c + 4095) / 4096));
    in.scale = scale, in.scales = scales, in.n_steps = n;
    std::copy(steps, steps + n, in.steps);
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
    {
        LaunchTimer timer("stack_split", s);
        const dim3 grid = dim3(unsigned(sh.rp / 64 * (sh.cp / 64) * count));
        if (bf16)
            sh.tall ? stack_split_kernel<uint16_t, true><<<grid, dim3(256), 0, s>>>(in)
                    : stack_split_kernel<uint16_t, false><<<grid, dim3(256), 0, s>>>(in);
        else
            sh.tall ? stack_split_kernel<float, true><<<grid, dim3(256), 0, s>>>(in)
                    : stack_split_kernel<float, false><<<grid, dim3(256), 0, s>>>(in);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;

    if (sh.r <= 128)
        return launch_stack_strips(st, sh, count, in.out, x[0], x[1], b, scales, steps, n, scale, s);
    for (int t = 0; t < n; ++t) {
        ProductArgs g{};
        g.x = x[t & 1], g.x_next = x[(t + 1) & 1], g.a = a, g.b = b;
        g.out = in.out, g.out_stride = st.out_stride, g.out_row = st.out_row;
        g.rp = in.rp, g.cp = in.cp, g.rows = in.rows, g.cols = in.cols;
        g.tall = sh.tall, g.out_bf16 = st.out_dtype == MUON_DTYPE_BF16, g.last = t + 1 == n;
        g.scales = scales + t, g.step = steps[t], g.scale = scale;
        for (int stage : {kA, kB, kX})
            if ((e = run_stage(stage, g, count, st.count, s)) != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_stack(const muon_stack_t& stack, const StackStep* steps, int n_steps, float scale,
                        void* workspace, size_t workspace_bytes, hipStream_t s) {
    const StackShape sh = stack_shape(stack.rows, stack.cols);
    if (n_steps > 0 && stack_is_whole(sh)) return launch_stack_whole(stack, sh, steps, n_steps, scale, s);
    // a grid counts below 2^32 work-items: at most 2^22 tiles of 64 x 64 in a group
    const int64_t per = sh.rp / 64 * (sh.cp / 64);
    const int64_t fit = std::max<int64_t>(1, std::min<int64_t>(int64_t(workspace_bytes / stack_matrix_bytes(sh)),
                                                               (int64_t(1) << 22) / std::max<int64_t>(per, 64)));
    for (int64_t at = 0; at < stack.count; at += fit) {
        const hipError_t e = run_group(stack, sh, at, std::min(fit, stack.count - at), steps, n_steps, scale,
                                       workspace, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace muon
