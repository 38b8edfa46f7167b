// int8.cuh -- matrices in 8-bit integers with one scale a row: the quantiser
// (rows, or columns stored transposed), and the product.  Included into asr.cu
// (inside its anonymous namespace), after muon.cuh.
//
//   scale_i = max_j |x_ij| / 127
//   q_ij    = rint(y), y = x_ij * (127 / max_j |x_ij|)            (nearest)
//           = floor(y) + [65536 (y - floor(y)) > r_ij]            (stochastic)
//   C_ij    = (sum_k a_ik b_jk) * sa_i * sb_j
//
// r_ij: the low 16 bits of the Philox word of x_ij's index, i * cols + j from
// the call's base index, whichever way the matrix is stored; y in binary32, the
// comparison exact.  The sum of integers is exact.  sm_103a's tensor memory instructions have no 8-bit
// integer kind; an 8-bit integer is exact in f16, a product of two in binary32,
// and so is any sum of 1,024 of them (1,024 * 128^2 = 2^24).  So the operands
// are widened to f16 in the workspace, int8_product.cuh sums chunks of 1,024 in
// tensor memory at the f16 rate, and its epilogue adds the chunks in int32 (the
// gradients' sums over more than 131,071 in int64).  With few rows of A the weight is read as it is (int8_few.cuh).
//
// Widening costs three bytes' traffic an element, once: 52 us of 610 for tokens
// 8,192 x 4,096 and a weight 14,336 x 4,096 (310 MB, 6.0 TB/s).  Widening inside
// the product instead would cost shared memory two bytes written and one read an
// element and tile next to the 64 bytes a cycle that the products read, more than
// its 128.  The gradients' operands are quantised where they lie and read across,
// in two streams: maxima (4,096 tokens, 8,192 x 2,048: 117 MB, 24 us), then the
// integers, dy's by rows and by columns from one read and one set of random bits
// (301 MB, 66 us; bound by instructions: 15 an element for Philox, 5 for each
// rounding; 64 registers, which leave 36 bytes of spilled loads a thread).
//
// The quantiser on its own, 14,336 x 4,096 bf16 (26 us of bytes): rows 48 us, 91
// stochastically (a row a block, read twice, the second time out of the cache;
// bound by instructions); columns 112 and 159 us (maxima, then 64 x 64 tiles turned
// in shared memory and stored a byte a thread, which bounds it; then the scales).

namespace int8 {

constexpr int kThreads = 256;
constexpr uint64_t kMaxK = prod::kMaxIntSum;
constexpr uint32_t kChunk = 1024 / prod::kBK;

struct WidenParams {
    const int8_t *src[2];
    __half *dst[2];
    uint64_t rows[2], src_ld[2];
    uint64_t cols, dst_ld;                      // dst_ld: cols up to a multiple of 16
    uint32_t vec[2];
};

// 8-bit integers to f16, block `block` of `blocks`: a warp a span of 512
// columns, 16 a lane.
__device__ __forceinline__ void widen_block(const WidenParams &P, uint32_t block, uint32_t blocks)
{
    const uint32_t lane = threadIdx.x & 31;
    muon::Walk k(P.rows[0] + P.rows[1], (P.cols + 1) / 2, block * 8ull + (threadIdx.x >> 5), blocks * 8ull);
    for (; k.more(); k.next()) {
        const int which = k.row >= P.rows[0];
        const uint64_t row = which ? k.row - P.rows[0] : k.row, col = k.span * 512ull + lane * 16;
        if (col >= P.cols) continue;
        const int8_t *src = P.src[which] + row * P.src_ld[which] + col;
        uint32_t a[4] = {0, 0, 0, 0};
        if (P.vec[which] && P.cols - col >= 16) {
            const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(src));
            a[0] = w.x, a[1] = w.y, a[2] = w.z, a[3] = w.w;
        } else {
            const int live = P.cols - col < 16 ? static_cast<int>(P.cols - col) : 16;
#pragma unroll
            for (int q = 0; q < 16; ++q)
                if (q < live) a[q >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(src[q])) << (8 * (q & 3));
        }
        uint32_t h[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) int8few::widen4(a[q], h[2 * q], h[2 * q + 1]);
        gemm::st_global_v8(P.dst[which] + row * P.dst_ld + col, h);
    }
}

__global__ void __launch_bounds__(kThreads) widen_kernel(const __grid_constant__ WidenParams P)
{
    widen_block(P, blockIdx.x, gridDim.x);
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t *part)
{
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[0];
    for (int w = 1; w < kThreads / 32; ++w) v = max(v, part[w]);
    return v;
}

// 65535 less the random words (their low halves) of elements e .. e+7.
__device__ __forceinline__ void words8(uint64_t base, uint64_t e, uint32_t step, const RoundKeys &K, uint32_t r[8])
{
    if (((base + e) & 3u) == 0) unit_words<true>(base, e, step, K, r);
    else unit_words<false>(base, e, step, K, r);
#pragma unroll
    for (int q = 0; q < 8; ++q) r[q] = ~r[q] & 0xFFFFu;
}

struct RowParams {
    const void *x;
    void *q;                                    // int8, or f16 rows a multiple of 16 apart (WIDE)
    float *scale;
    uint64_t rows, cols, x_ld, q_ld;
    uint64_t base;
    uint32_t dtype, step;
    uint32_t vec;                               // 8-element units of x are 16-byte aligned
    RoundKeys keys;
    WidenParams w;                              // WIDE: the other operand, widened by the blocks past `rows`
};

// Rows: one block each, the second pass over the row out of the cache.
template <bool SR, bool WIDE>
__global__ void __launch_bounds__(kThreads) quantise_rows_kernel(const __grid_constant__ RowParams P, uint32_t row_blocks)
{
    // the product that follows may start on what does not depend on this
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (WIDE && blockIdx.x >= row_blocks) {
        widen_block(P.w, blockIdx.x - row_blocks, gridDim.x - row_blocks);
        return;
    }
    __shared__ uint32_t part[kThreads / 32];
    for (uint64_t row = blockIdx.x; row < P.rows; row += row_blocks) {
        uint32_t top = 0;                       // the order of non-negative floats is that of their bits; a NaN is above all
        for (uint64_t col = threadIdx.x * 8ull; col < P.cols; col += kThreads * 8ull) {
            const int live = P.cols - col < 8 ? static_cast<int>(P.cols - col) : 8;
            float x[8];
            muon::load8(P.x, P.dtype, row * P.x_ld + col, live, P.vec, x);
#pragma unroll
            for (int q = 0; q < 8; ++q) top = max(top, absbits(x[q]));
        }
        const float amax = __uint_as_float(block_max(top, part));
        const Levels L = levels_of(amax);
        if (threadIdx.x == 0) P.scale[row] = __fdiv_rn(amax, 127.0f);
        for (uint64_t col = threadIdx.x * 8ull; col < P.cols; col += kThreads * 8ull) {
            const int live = P.cols - col < 8 ? static_cast<int>(P.cols - col) : 8;
            float x[8];
            muon::load8(P.x, P.dtype, row * P.x_ld + col, live, P.vec, x);
            uint32_t r[8];
            if (SR) words8(P.base, row * P.cols + col, P.step, P.keys, r);
            uint32_t v[4];
            quantise8<SR>(x, L, r, v);
            if (WIDE) *reinterpret_cast<uint4 *>(static_cast<__half *>(P.q) + row * P.q_ld + col) = halves_of(v);
            else store_int8(static_cast<int8_t *>(P.q) + row * P.q_ld + col, v, live);
        }
        __syncthreads();
    }
}

// What the product with few rows needs before it: the tokens widened (quantised
// here from f32 or bf16, or given as integers), their scales, and zeros in its
// sums.  Blocks below `rows` take a row each, a few units a thread held in
// registers between the two passes; the others zero.
constexpr int kPrepThreads = 1024;
constexpr int kFewUnits = 4;                    // rows of up to 4 * 8 * 1,024 values stay in registers

struct FewPrepParams {
    const void *x;
    __half *out;
    float *scale;                               // null: x is int8
    uint4 *zero;
    uint64_t rows, cols, x_ld, out_ld, zero_units;
    uint32_t dtype, vec;
};

__global__ void __launch_bounds__(kPrepThreads) few_prep_kernel(const __grid_constant__ FewPrepParams P)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x >= P.rows) {
        for (uint64_t i = (blockIdx.x - P.rows) * kPrepThreads + threadIdx.x; i < P.zero_units;
             i += (gridDim.x - P.rows) * kPrepThreads)
            P.zero[i] = make_uint4(0, 0, 0, 0);
        return;
    }
    const uint64_t row = blockIdx.x;
    __half *out = P.out + row * P.out_ld;
    if (!P.scale) {
        const int8_t *src = static_cast<const int8_t *>(P.x) + row * P.x_ld;
        for (uint64_t col = threadIdx.x * 8ull; col < P.out_ld; col += kPrepThreads * 8ull) {
            uint32_t e[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int lo = col + 2 * q < P.cols ? src[col + 2 * q] : 0, hi = col + 2 * q + 1 < P.cols ? src[col + 2 * q + 1] : 0;
                e[q] = __byte_perm(static_cast<uint32_t>(lo + 0x6480), static_cast<uint32_t>(hi + 0x6480), 0x5410);
            }
            *reinterpret_cast<uint4 *>(out + col) = halves_of(e);
        }
        return;
    }
    __shared__ uint32_t part[kPrepThreads / 32];
    float x[kFewUnits][8];
    uint32_t top = 0;
    auto fetch = [&](uint64_t col, float v[8]) {
        const int live = col >= P.cols ? 0 : P.cols - col < 8 ? static_cast<int>(P.cols - col) : 8;
        muon::load8(P.x, P.dtype, row * P.x_ld + col, live, P.vec, v);
    };
#pragma unroll
    for (int u = 0; u < kFewUnits; ++u) {
        fetch((u * kPrepThreads + threadIdx.x) * 8ull, x[u]);
#pragma unroll
        for (int q = 0; q < 8; ++q) top = max(top, absbits(x[u][q]));
    }
    for (uint64_t col = (kFewUnits * kPrepThreads + threadIdx.x) * 8ull; col < P.cols; col += kPrepThreads * 8ull) {
        float v[8];
        fetch(col, v);
#pragma unroll
        for (int q = 0; q < 8; ++q) top = max(top, absbits(v[q]));
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
    const float amax = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, part[threadIdx.x & 31]));
    const Levels L = levels_of(amax);
    if (threadIdx.x == 0) P.scale[row] = __fdiv_rn(amax, 127.0f);
#pragma unroll
    for (int u = 0; u < kFewUnits; ++u) {
        const uint64_t col = (u * kPrepThreads + threadIdx.x) * 8ull;
        uint32_t q[4];
        quantise8<false>(x[u], L, nullptr, q);
        if (col < P.out_ld) *reinterpret_cast<uint4 *>(out + col) = halves_of(q);
    }
    for (uint64_t col = (kFewUnits * kPrepThreads + threadIdx.x) * 8ull; col < P.out_ld; col += kPrepThreads * 8ull) {
        float v[8];
        fetch(col, v);
        uint32_t q[4];
        quantise8<false>(v, L, nullptr, q);
        *reinterpret_cast<uint4 *>(out + col) = halves_of(q);
    }
}

__global__ void __launch_bounds__(kThreads) zero_kernel(uint32_t *p, uint64_t n)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint64_t i = blockIdx.x * static_cast<uint64_t>(kThreads) + threadIdx.x;
    if (i < n) p[i] = 0;
}

// Maxima along columns, or along both, of up to three matrices in one launch:
// blocks of 8 * `deep` rows x 256 columns, a warp `deep` rows, eight columns a
// lane.  `row_max` and `col_max` hold bits of non-negative floats, zero at the
// start; integer maxima are the same whatever their order.
constexpr int kDeep = 32;                       // rows a warp, at most, eight loads ahead

struct Side {
    const void *x;
    uint64_t rows, cols, x_ld;
    uint32_t *row_max, *col_max;                // row_max may be null
    uint32_t vec, dtype;
    uint32_t tiles_x, first;                    // first block of this matrix
    // what becomes of it in `wide_kernel`: f16 integers in place, scaled by columns and (with row_max) by rows
    __half *by_row, *by_col;
    float *row_scale, *col_scale;
    uint64_t q_ld;
};

struct SideParams {
    Side s[3];
    uint32_t count, blocks, deep;
    uint32_t step;
    RoundKeys keys;
};

__device__ __forceinline__ const Side &side_of(const SideParams &P, uint32_t block)
{
    return P.s[P.count > 2 && block >= P.s[2].first ? 2 : P.count > 1 && block >= P.s[1].first ? 1 : 0];
}

__global__ void __launch_bounds__(kThreads) max_kernel(const __grid_constant__ SideParams P)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ uint32_t part[8][8 * 33];
    const Side &S = side_of(P, blockIdx.x);
    const uint32_t tile = blockIdx.x - S.first, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t r0 = (static_cast<uint64_t>(tile / S.tiles_x) * 8 + warp) * P.deep;
    const uint64_t c0 = static_cast<uint64_t>(tile % S.tiles_x) * 256, col = c0 + lane * 8;
    const int live = col >= S.cols ? 0 : S.cols - col < 8 ? static_cast<int>(S.cols - col) : 8;
    const uint32_t rows = r0 >= S.rows ? 0 : S.rows - r0 < P.deep ? static_cast<uint32_t>(S.rows - r0) : P.deep;
    uint32_t top[8] = {};
    const bool packed = S.dtype == ASR_BF16 && S.vec && live == 8;      // the first lanes of a warp, or none
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, packed);
    if (packed) {
        // two values a word: sixteen-bit maxima of the bits without signs
        const uint16_t *p = static_cast<const uint16_t *>(S.x) + r0 * S.x_ld + col;
        uint32_t t[4] = {};
        for (uint32_t i0 = 0; i0 < rows; i0 += 8) {
            uint4 w[8];
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i)
                w[i] = i0 + i < rows ? *reinterpret_cast<const uint4 *>(p + (i0 + i) * S.x_ld) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) {
                const uint32_t a[4] = {w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu, w[i].z & 0x7FFF7FFFu,
                                       w[i].w & 0x7FFF7FFFu};
#pragma unroll
                for (int q = 0; q < 4; ++q) t[q] = __vmaxu2(t[q], a[q]);
                if (S.row_max && i0 + i < rows) {
                    uint32_t most = __vmaxu2(__vmaxu2(a[0], a[1]), __vmaxu2(a[2], a[3]));
                    most = max(most << 16, most & 0xFFFF0000u);
                    most = __reduce_max_sync(mask, most);
                    if (lane == 0) atomicMax(S.row_max + r0 + i0 + i, most);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) top[2 * q] = t[q] << 16, top[2 * q + 1] = t[q] & 0xFFFF0000u;
    } else {
        for (uint32_t i = 0; i < rows; ++i) {
            uint32_t most = 0;
            if (live) {
                float x[8];
                muon::load8(S.x, S.dtype, (r0 + i) * S.x_ld + col, live, S.vec, x);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const uint32_t b = absbits(x[q]);
                    top[q] = max(top[q], b);
                    most = max(most, b);
                }
            }
            if (S.row_max) {
                most = __reduce_max_sync(~mask, most);
                if (lane == static_cast<uint32_t>(__ffs(~mask) - 1)) atomicMax(S.row_max + r0 + i, most);
            }
        }
    }
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 8; ++q) part[warp][q * 33 + lane] = top[q];     // column lane * 8 + q
    __syncthreads();
    const uint32_t at = (threadIdx.x & 7) * 33 + (threadIdx.x >> 3);
    uint32_t v = part[0][at];
#pragma unroll
    for (int w = 1; w < 8; ++w) v = max(v, part[w][at]);
    const uint64_t c = c0 + threadIdx.x;
    if (c < S.cols) atomicMax(S.col_max + c, v);
}

// Rows r0 on of a lane's eight columns (`live` of them), for wide_kernel.
// inv_rows: the rows' scales times 65536.
template <bool RANDOM>
__device__ __forceinline__ void wide_rows(const SideParams &P, const Side &S, uint64_t r0, uint32_t rows, uint64_t col,
                                          int live, const float *inv_rows)
{
    float inv[8];
    bool odd = false;
    auto column = [&](int q) { return levels_of(q < live ? __uint_as_float(S.col_max[col + q]) : 0.0f); };
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const Levels L = column(q);
        inv[q] = RANDOM ? __fmul_rn(L.inv, 65536.0f) : L.inv;
        odd |= L.odd && q < live;
    }
    __half *by_row = RANDOM && S.by_row ? S.by_row + r0 * S.q_ld + col : nullptr;
    __half *by_col = S.by_col ? S.by_col + r0 * S.q_ld + col : nullptr;
    uint64_t e = r0 * S.cols + col;
    auto one = [&](uint32_t i, float x[8]) {
        uint32_t v[4], r[8];
        if (RANDOM) {
            words8(0, e, P.step, P.keys, r);
            e += S.cols;
            if (by_row) {
                float f = inv_rows[i], z[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) z[q] = x[q];
                if (f < 0.0f) {
                    const Levels L = levels_of(__uint_as_float(S.row_max[r0 + i]));
                    f = __fmul_rn(L.inv, 65536.0f);
#pragma unroll
                    for (int q = 0; q < 8; ++q) z[q] = regular(x[q], L);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = random2(z[2 * q], z[2 * q + 1], f, f, r[2 * q], r[2 * q + 1]);
                *reinterpret_cast<uint4 *>(by_row) = halves_of(v);
                by_row += S.q_ld;
            }
        }
        if (!by_col) return;
        if (odd) {
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = regular(x[q], column(q));
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            v[q] = RANDOM ? random2(x[2 * q], x[2 * q + 1], inv[2 * q], inv[2 * q + 1], r[2 * q], r[2 * q + 1])
                          : nearest2(x[2 * q], x[2 * q + 1], inv[2 * q], inv[2 * q + 1]);
        // past the last column: zeros (their loads gave zeros)
        *reinterpret_cast<uint4 *>(by_col) = halves_of(v);
        by_col += S.q_ld;
    };
    if (S.dtype == ASR_BF16 && S.vec && live == 8) {
        const uint16_t *p = static_cast<const uint16_t *>(S.x) + r0 * S.x_ld + col;
        // two rows at a time: four do not fit the registers (gradients of the size above 258 us; one 262)
        for (uint32_t i = 0; i < rows; i += 2) {
            uint4 w[2];
            w[0] = *reinterpret_cast<const uint4 *>(p);
            w[1] = i + 1 < rows ? *reinterpret_cast<const uint4 *>(p + S.x_ld) : make_uint4(0, 0, 0, 0);
            p += 2 * S.x_ld;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (i + j >= rows) break;
                float x[8] = {bf16_lo(w[j].x), bf16_hi(w[j].x), bf16_lo(w[j].y), bf16_hi(w[j].y),
                              bf16_lo(w[j].z), bf16_hi(w[j].z), bf16_lo(w[j].w), bf16_hi(w[j].w)};
                one(i + j, x);
            }
        }
    } else {
        for (uint32_t i = 0; i < rows; ++i) {
            float x[8];
            muon::load8(S.x, S.dtype, (r0 + i) * S.x_ld + col, live, S.vec, x);
            one(i, x);
        }
    }
}

// The integers of every matrix of the call, as f16, where they lie (the
// products read them across): side 0 (dy) stochastically, by its rows' and by
// its columns' maxima with the same random bits; the others to nearest, by
// columns.  The first tiles write the scales.
__global__ void __launch_bounds__(kThreads, 4) wide_kernel(const __grid_constant__ SideParams P)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Side &S = side_of(P, blockIdx.x);
    const uint32_t tile = blockIdx.x - S.first, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t t0 = static_cast<uint64_t>(tile / S.tiles_x) * 8 * P.deep, r0 = t0 + warp * P.deep;
    const uint64_t c0 = static_cast<uint64_t>(tile % S.tiles_x) * 256, col = c0 + lane * 8;
    const int live = col >= S.cols ? 0 : S.cols - col < 8 ? static_cast<int>(S.cols - col) : 8;
    if (t0 == 0 && c0 + threadIdx.x < S.cols)
        S.col_scale[c0 + threadIdx.x] = __fdiv_rn(__uint_as_float(S.col_max[c0 + threadIdx.x]), 127.0f);
    if (S.row_max && c0 == 0 && threadIdx.x < 8 * P.deep && t0 + threadIdx.x < S.rows)
        S.row_scale[t0 + threadIdx.x] = __fdiv_rn(__uint_as_float(S.row_max[t0 + threadIdx.x]), 127.0f);
    // the block's rows' scales, once; -1 for an odd row
    __shared__ float by_row[8 * kDeep];
    if (S.row_max && threadIdx.x < 8 * P.deep && t0 + threadIdx.x < S.rows) {
        const Levels L = levels_of(__uint_as_float(S.row_max[t0 + threadIdx.x]));
        by_row[threadIdx.x] = L.odd ? -1.0f : __fmul_rn(L.inv, 65536.0f);
    }
    __syncthreads();
    if (!live || r0 >= S.rows) return;
    const uint32_t rows = S.rows - r0 < P.deep ? static_cast<uint32_t>(S.rows - r0) : P.deep;
    if (S.row_max) wide_rows<true>(P, S, r0, rows, col, live, by_row + warp * P.deep);
    else wide_rows<false>(P, S, r0, rows, col, live, nullptr);
}

struct ColumnParams {
    const void *x;
    int8_t *q;
    const uint32_t *col_max;                    // in `scale`, until the scales are written
    uint64_t rows, cols, x_ld, q_ld;
    uint64_t base;
    uint32_t dtype, step, vec;
    RoundKeys keys;
};

// Columns, stored transposed: 64 x 64 tiles turned in shared memory.
template <bool SR>
__global__ void __launch_bounds__(kThreads) quantise_columns_kernel(const __grid_constant__ ColumnParams P)
{
    __shared__ int8_t tile[64][68];
    const uint64_t r0 = blockIdx.y * 64ull, c0 = blockIdx.x * 64ull;
    const uint64_t col = c0 + (threadIdx.x & 7) * 8;
    const int live = col >= P.cols ? 0 : P.cols - col < 8 ? static_cast<int>(P.cols - col) : 8;
    Levels L[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) L[q] = levels_of(q < live ? __uint_as_float(P.col_max[col + q]) : 0.0f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int tr = (threadIdx.x >> 3) + i * 32;
        const uint64_t row = r0 + tr;
        if (row >= P.rows || !live) continue;
        float x[8];
        muon::load8(P.x, P.dtype, row * P.x_ld + col, live, P.vec, x);
        uint32_t r[8];
        if (SR) words8(P.base, row * P.cols + col, P.step, P.keys, r);
        uint32_t e[4];
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = regular(x[q], L[q]);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            e[q] = SR ? random2(x[2 * q], x[2 * q + 1], __fmul_rn(L[2 * q].inv, 65536.0f),
                                __fmul_rn(L[2 * q + 1].inv, 65536.0f), r[2 * q], r[2 * q + 1])
                      : nearest2(x[2 * q], x[2 * q + 1], L[2 * q].inv, L[2 * q + 1].inv);
        const uint2 w = bytes_of(e);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            tile[(threadIdx.x & 7) * 8 + q][tr] = static_cast<int8_t>((q < 4 ? w.x : w.y) >> (8 * (q & 3)));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * 64; i += kThreads) {
        const uint64_t c = c0 + (i >> 6), row = r0 + (i & 63);
        if (row < P.rows && c < P.cols) P.q[c * P.q_ld + row] = tile[i >> 6][i & 63];
    }
}

__global__ void __launch_bounds__(kThreads) column_scale_kernel(float *scale, uint64_t n)
{
    const uint64_t i = blockIdx.x * static_cast<uint64_t>(kThreads) + threadIdx.x;
    if (i < n) scale[i] = __fdiv_rn(scale[i], 127.0f);
}

// ------------------------------------------------------------------ host

unsigned blocks_for(uint64_t units, uint64_t per_block, uint64_t most)
{
    const uint64_t b = (units + per_block - 1) / per_block;
    return static_cast<unsigned>(b < 1 ? 1 : b < most ? b : most);
}

bool pitch_ok(uint64_t ld, uint64_t least) { return ld >= least && ld <= (1ull << 32); }

// A row and column range of the tiles that the column kernels walk must be countable in a launch.
bool quantisable(uint64_t rows, uint64_t cols)
{
    return rows <= (1u << 30) && cols <= (1u << 30) &&
           ((rows + 7) / 8) * ((cols + 255) / 256) < (1ull << 28);
}

Side side(const void *x, int32_t dtype, uint64_t rows, uint64_t cols, uint64_t ld)
{
    Side S;
    std::memset(&S, 0, sizeof(S));
    S.x = x;
    S.rows = rows;
    S.cols = cols;
    S.x_ld = ld;
    S.vec = muon::units_aligned(x, ld, 0);
    S.dtype = static_cast<uint32_t>(dtype);
    S.tiles_x = static_cast<uint32_t>((cols + 255) / 256);
    return S;
}

// Lays the sides' blocks end to end: as many rows a warp as leave the GPU full
// (four blocks an SM).
void lay_out(SideParams &M)
{
    for (M.deep = kDeep;; M.deep /= 2) {
        M.blocks = 0;
        for (uint32_t i = 0; i < M.count; ++i) {
            Side &S = M.s[i];
            S.first = M.blocks;
            M.blocks += static_cast<uint32_t>((S.rows + 8 * M.deep - 1) / (8 * M.deep)) * S.tiles_x;
        }
        if (M.blocks >= 608 || M.deep == 1) return;
    }
}

// The sides' maxima, which lie in the `words` words from `zero` on.
asr_status maxima(SideParams &M, uint32_t *zero, uint64_t words, cudaStream_t stream)
{
    lay_out(M);
    zero_kernel<<<static_cast<unsigned>((words + kThreads - 1) / kThreads), kThreads, 0, stream>>>(zero, words);
    const asr_status st = launched(ASR_KERNEL_QUANTIZE);
    if (st != ASR_OK) return st;
    return prod::launch_early(ASR_KERNEL_QUANTIZE, max_kernel, dim3(M.blocks), kThreads, M, stream);
}

// Every kernel of this file and of the products ready on the device, whichever a call takes.
asr_status setup()
{
    static std::atomic<uint64_t> ready{0};
    int pairs = 0, sms = 0, dev = 0;
    asr_status st = prod::int8_setup(&pairs);
    if (st == ASR_OK) st = int8few::setup(&sms);
    if (st != ASR_OK) return st;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (e == cudaSuccess && (ready.load(std::memory_order_acquire) & bit)) return ASR_OK;
    if (e == cudaSuccess) e = prod::load_kernel(zero_kernel);
    if (e == cudaSuccess) e = prod::load_kernel(few_prep_kernel);
    if (e == cudaSuccess) e = prod::load_kernel(quantise_rows_kernel<false, false>);
    if (e == cudaSuccess) e = prod::load_kernel(quantise_rows_kernel<true, false>);
    if (e == cudaSuccess) e = prod::load_kernel(quantise_rows_kernel<false, true>);
    if (e == cudaSuccess) e = prod::load_kernel(quantise_columns_kernel<false>);
    if (e == cudaSuccess) e = prod::load_kernel(quantise_columns_kernel<true>);
    if (e == cudaSuccess) e = prod::load_kernel(column_scale_kernel);
    if (e == cudaSuccess) e = prod::load_kernel(widen_kernel);
    if (e == cudaSuccess) e = prod::load_kernel(max_kernel);
    if (e == cudaSuccess) e = prod::load_kernel(wide_kernel);
    if (e != cudaSuccess) return cuda_fail(e);
    ready.fetch_or(bit, std::memory_order_release);
    return ASR_OK;
}

asr_status quantize(const void *x, int32_t dtype, uint64_t rows, uint64_t cols, uint64_t x_ld, int32_t axis, int8_t *q,
                    uint64_t q_ld, float *scale, uint32_t rounding, uint64_t base, uint32_t step, uint64_t seed,
                    cudaStream_t stream)
{
    if (dtype != ASR_F32 && dtype != ASR_BF16) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (rounding != ASR_ROUND_SR && rounding != ASR_ROUND_RNE) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (axis != ASR_ROWS && axis != ASR_COLUMNS) return ASR_ERR_INVALID_VALUE;
    const uint64_t scales = axis == ASR_ROWS ? rows : cols;
    if (scales == 0) return ASR_OK;
    if (rows == 0 || cols == 0) {                   // rows of no elements: scales of zero
        if (!scale || !muon::element_aligned(scale, ASR_F32) || scales > (1u << 30)) return ASR_ERR_INVALID_VALUE;
        const asr_status st = setup();
        if (st != ASR_OK) return st;
        zero_kernel<<<static_cast<unsigned>((scales + kThreads - 1) / kThreads), kThreads, 0, stream>>>(
            reinterpret_cast<uint32_t *>(scale), scales);
        return launched(ASR_KERNEL_QUANTIZE);
    }
    if (!x || !q || !scale || !muon::element_aligned(x, dtype) || !muon::element_aligned(scale, ASR_F32))
        return ASR_ERR_INVALID_VALUE;
    if (!quantisable(rows, cols) || !pitch_ok(x_ld, cols) || !pitch_ok(q_ld, axis == ASR_ROWS ? cols : rows) ||
        base > UINT64_MAX - rows * cols || (axis == ASR_COLUMNS && (rows + 63) / 64 > 65535))
        return ASR_ERR_INVALID_VALUE;
    asr_status st = setup();
    if (st != ASR_OK) return st;
    const bool sr = rounding == ASR_ROUND_SR;
    if (axis == ASR_ROWS) {
        RowParams P;
        std::memset(&P, 0, sizeof(P));
        P.x = x;
        P.q = q;
        P.scale = scale;
        P.rows = rows;
        P.cols = cols;
        P.x_ld = x_ld;
        P.q_ld = q_ld;
        P.base = base;
        P.dtype = static_cast<uint32_t>(dtype);
        P.step = step;
        P.vec = muon::units_aligned(x, x_ld, 0);
        P.keys = make_keys(seed);
        const unsigned grid = blocks_for(rows, 1, 65536);
        if (sr) quantise_rows_kernel<true, false><<<grid, kThreads, 0, stream>>>(P, grid);
        else quantise_rows_kernel<false, false><<<grid, kThreads, 0, stream>>>(P, grid);
        return launched(ASR_KERNEL_QUANTIZE);
    }
    SideParams M;
    std::memset(&M, 0, sizeof(M));
    M.s[0] = side(x, dtype, rows, cols, x_ld);
    M.s[0].col_max = reinterpret_cast<uint32_t *>(scale);
    M.count = 1;
    st = maxima(M, M.s[0].col_max, cols, stream);
    if (st != ASR_OK) return st;
    ColumnParams P;
    P.x = x;
    P.q = q;
    P.col_max = reinterpret_cast<const uint32_t *>(scale);
    P.rows = rows;
    P.cols = cols;
    P.x_ld = x_ld;
    P.q_ld = q_ld;
    P.base = base;
    P.dtype = static_cast<uint32_t>(dtype);
    P.step = step;
    P.vec = muon::units_aligned(x, x_ld, 0);
    P.keys = make_keys(seed);
    const dim3 grid(static_cast<unsigned>((cols + 63) / 64), static_cast<unsigned>((rows + 63) / 64));
    if (sr) quantise_columns_kernel<true><<<grid, kThreads, 0, stream>>>(P);
    else quantise_columns_kernel<false><<<grid, kThreads, 0, stream>>>(P);
    st = launched(ASR_KERNEL_QUANTIZE);
    if (st != ASR_OK) return st;
    column_scale_kernel<<<static_cast<unsigned>((cols + kThreads - 1) / kThreads), kThreads, 0, stream>>>(scale, cols);
    return launched(ASR_KERNEL_QUANTIZE);
}

bool sizes_ok(uint64_t m, uint64_t n, uint64_t k)
{
    return m <= (1u << 24) && n <= (1u << 24) && k <= kMaxK;
}

// Whether the weight is read as it is (int8_few.cuh) or widened first.  Reading it
// costs more with every token (int32 sums of n x tokens through memory: 0.1 to 0.3
// us a token), widening 0.84 us a million values of the weight, and the product
// that follows does not share out K (2.2 us a thousand), so the choice goes by
// tokens against K.  Measured, us, weight as it is / widened: 1,024 x 1,024: 16
// tokens 8.8 / 9.8, 32 9.9 / 9.4; 2,048 x 2,048: 48 12.1 / 13.5, 64 14.0 / 13.7, 128
// 20.2 / 13.9; 4,096 x 4,096: 64 19.7 / 23.5, 128 30.7 / 24.1; 14,336 x 4,096: 128
// 39.5 / 62.7, 160 58.9 / 62.8, 256 75 / 64; 4,096 x 14,336: 256 71 / 84, 384 99 / 97;
// 28,672 x 8,192: 256 163 / 224; 8,192 x 512: 16 11.2 / 13.2, 32 14.4 / 13.0.
bool few(uint64_t m, uint64_t n, uint64_t k)
{
    const uint64_t most = k / 32 < 16 ? 16 : k / 32 < 256 ? k / 32 : 256;
    return m <= most || int8few::dots(m, n, k);
}

// Workspace: with few rows of A the widened rows, their scales and the sums;
// otherwise the scales and both operands, widened.
struct Layout {
    uint64_t scale, zero, zero_bytes, counts, a, b, bytes, ld;
};

Layout layout(uint64_t m, uint64_t n, uint64_t k)
{
    Layout L{};
    L.ld = muon::up(k, 16);
    if (int8few::dots(m, n, k)) return L;     // none
    L.scale = 0;
    L.zero = muon::up(m * sizeof(float), 256);
    L.zero_bytes = 0;
    L.counts = L.zero;
    const bool narrow = few(m, n, k);
    if (narrow) {
        const uint64_t tiles = (n + int8few::kRows - 1) / int8few::kRows;
        L.counts = L.zero + tiles * m * int8few::kRows * sizeof(int32_t);
        L.zero_bytes = muon::up(L.counts - L.zero + tiles * int8few::passes(m) * sizeof(uint32_t), 256);
    }
    L.a = L.zero + L.zero_bytes;
    L.b = L.a + muon::up(m * L.ld * 2, 256);
    L.bytes = narrow ? L.b : L.b + muon::up(n * L.ld * 2, 256);
    return L;
}

struct Output {
    void *c;
    uint64_t ld;
    int32_t dtype;
    uint32_t rounding, step;
    uint64_t seed;
};

bool output_ok(const Output &o, uint64_t n)
{
    return o.c && pitch_ok(o.ld, n) && muon::element_aligned(o.c, o.dtype);
}

asr_status output_kind(const Output &o)
{
    if (o.dtype != ASR_F32 && o.dtype != ASR_BF16) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (o.rounding != ASR_ROUND_SR && o.rounding != ASR_ROUND_RNE) return ASR_ERR_UNSUPPORTED_DTYPE;
    return ASR_OK;
}

// The output's fields of a product of widened operands.
prod::Params product_params(const float *sa, const float *sb, const Output &o)
{
    prod::Params P;
    std::memset(&P, 0, sizeof(P));
    P.out_ld = o.ld;
    P.out_dtype = static_cast<uint32_t>(o.dtype);
    P.rounding = o.rounding;
    P.vec = muon::aligned32(o.c) && o.ld % 16 == 0;
    P.step = o.step;
    P.row_scale = sa;
    P.col_scale = sb;
    P.keys = make_keys(o.seed);
    P.slot[0].ptr = o.c;
    return P;
}

asr_status product(const prod::Stored &a, const prod::Stored &b, const float *sa, const float *sb, const Output &o,
                   cudaStream_t stream)
{
    prod::Int8Products L;
    prod::Stored operands[4];
    std::memset(&L, 0, sizeof(L));
    prod::int8_add(L, operands, a, false, b, false, product_params(sa, sb, o));
    return prod::int8_launch(L, operands, kChunk, stream);
}

prod::Stored stored(__half *p, uint64_t rows, uint64_t cols, uint64_t ld)
{
    return prod::Stored{p, rows, cols, ld, muon::up(rows * ld * 2, 256) / 2};
}

// The product with few rows: x is the tokens (quantised here), or, with `sa`,
// 8-bit integers with those scales.
asr_status few_rows(const void *x, int32_t x_dtype, uint64_t x_ld, const float *sa, const int8_t *b, uint64_t ldb,
                    const float *sb, const Output &o, uint64_t m, uint64_t n, uint64_t k, char *ws, const Layout &L,
                    cudaStream_t stream)
{
    if (int8few::dots(m, n, k)) {
        int8few::DotParams D;
        std::memset(&D, 0, sizeof(D));
        D.a = x;
        D.b = b;
        D.row_scale = sa;
        D.col_scale = sb;
        D.c = o.c;
        D.lda = x_ld;
        D.ldb = ldb;
        D.ldc = o.ld;
        D.m = static_cast<uint32_t>(m);
        D.n = static_cast<uint32_t>(n);
        D.k = static_cast<uint32_t>(k);
        D.a_dtype = static_cast<uint32_t>(x_dtype);
        D.a_vec = !sa && muon::units_aligned(x, x_ld, 0);
        D.b_vec = aligned16(b) && ldb % 16 == 0;
        D.c_dtype = static_cast<uint32_t>(o.dtype);
        D.rounding = o.rounding;
        D.step = o.step;
        D.keys = make_keys(o.seed);
        return int8few::run_dots(D, !sa, stream);
    }
    FewPrepParams F;
    std::memset(&F, 0, sizeof(F));
    F.x = x;
    F.out = reinterpret_cast<__half *>(ws + L.a);
    F.scale = sa ? nullptr : reinterpret_cast<float *>(ws + L.scale);
    F.zero = reinterpret_cast<uint4 *>(ws + L.zero);
    F.rows = m;
    F.cols = k;
    F.x_ld = x_ld;
    F.out_ld = L.ld;
    F.zero_units = L.zero_bytes / 16;
    F.dtype = static_cast<uint32_t>(x_dtype);
    F.vec = !sa && muon::units_aligned(x, x_ld, 0);
    const unsigned blocks = static_cast<unsigned>(m) + blocks_for(F.zero_units, 4 * kPrepThreads, 64);
    few_prep_kernel<<<blocks, kPrepThreads, 0, stream>>>(F);
    asr_status st = launched(ASR_KERNEL_QUANTIZE);
    if (st != ASR_OK) return st;
    int8few::Params P;
    std::memset(&P, 0, sizeof(P));
    P.a = F.out;
    P.b = b;
    P.row_scale = sa ? sa : F.scale;
    P.col_scale = sb;
    P.c = o.c;
    P.sums = reinterpret_cast<int32_t *>(ws + L.zero);
    P.counts = reinterpret_cast<uint32_t *>(ws + L.counts);
    P.lda = L.ld;
    P.ldb = ldb;
    P.ldc = o.ld;
    P.m = static_cast<uint32_t>(m);
    P.n = static_cast<uint32_t>(n);
    P.k = static_cast<uint32_t>(k);
    P.b_vec = aligned16(b) && ldb % 16 == 0;
    P.c_dtype = static_cast<uint32_t>(o.dtype);
    P.rounding = o.rounding;
    P.step = o.step;
    P.keys = make_keys(o.seed);
    return int8few::run(P, stream);
}

asr_status gemm(const int8_t *a, uint64_t lda, const int8_t *b, uint64_t ldb, const float *sa, const float *sb,
                const Output &o, uint64_t m, uint64_t n, uint64_t k, void *ws, uint64_t ws_bytes, cudaStream_t stream)
{
    asr_status st = output_kind(o);
    if (st != ASR_OK) return st;
    if (m == 0 || n == 0) return ASR_OK;
    if (!sizes_ok(m, n, k) || k == 0) return ASR_ERR_INVALID_VALUE;
    if (!a || !b || !sa || !sb || !pitch_ok(lda, k) || !pitch_ok(ldb, k) || !output_ok(o, n) ||
        !muon::element_aligned(sa, ASR_F32) || !muon::element_aligned(sb, ASR_F32))
        return ASR_ERR_INVALID_VALUE;
    const Layout L = layout(m, n, k);
    if (L.bytes && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < L.bytes)) return ASR_ERR_INVALID_VALUE;
    st = setup();
    if (st != ASR_OK) return st;
    char *w = static_cast<char *>(ws);
    if (few(m, n, k)) return few_rows(a, 0, lda, sa, b, ldb, sb, o, m, n, k, w, L, stream);
    WidenParams W;
    std::memset(&W, 0, sizeof(W));
    W.src[0] = a;
    W.src[1] = b;
    W.dst[0] = reinterpret_cast<__half *>(w + L.a);
    W.dst[1] = reinterpret_cast<__half *>(w + L.b);
    W.rows[0] = m;
    W.rows[1] = n;
    W.src_ld[0] = lda;
    W.src_ld[1] = ldb;
    W.cols = k;
    W.dst_ld = L.ld;
    W.vec[0] = aligned16(a) && lda % 16 == 0;
    W.vec[1] = aligned16(b) && ldb % 16 == 0;
    widen_kernel<<<blocks_for((m + n) * ((k + 511) / 512), 8, 1216), kThreads, 0, stream>>>(W);
    st = launched(ASR_KERNEL_QUANTIZE);
    if (st != ASR_OK) return st;
    return product(stored(W.dst[0], m, k, L.ld), stored(W.dst[1], n, k, L.ld), sa, sb, o, stream);
}

// ---- the linear layer's calls

asr_status linear(const void *x, int32_t x_dtype, uint64_t x_ld, const int8_t *qw, uint64_t ldw, const float *sw,
                  const Output &o, uint64_t m, uint64_t n, uint64_t k, void *ws, uint64_t ws_bytes,
                  cudaStream_t stream)
{
    if (x_dtype != ASR_F32 && x_dtype != ASR_BF16) return ASR_ERR_UNSUPPORTED_DTYPE;
    asr_status st = output_kind(o);
    if (st != ASR_OK) return st;
    if (m == 0 || n == 0) return ASR_OK;
    if (!sizes_ok(m, n, k) || k == 0) return ASR_ERR_INVALID_VALUE;
    if (!x || !qw || !sw || !pitch_ok(x_ld, k) || !pitch_ok(ldw, k) || !output_ok(o, n) ||
        !muon::element_aligned(x, x_dtype) || !muon::element_aligned(sw, ASR_F32))
        return ASR_ERR_INVALID_VALUE;
    const Layout L = layout(m, n, k);
    if (L.bytes && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < L.bytes)) return ASR_ERR_INVALID_VALUE;
    st = setup();
    if (st != ASR_OK) return st;
    char *w = static_cast<char *>(ws);
    if (few(m, n, k)) return few_rows(x, x_dtype, x_ld, nullptr, qw, ldw, sw, o, m, n, k, w, L, stream);
    RowParams P;
    std::memset(&P, 0, sizeof(P));
    P.x = x;
    P.q = w + L.a;
    P.scale = reinterpret_cast<float *>(w + L.scale);
    P.rows = m;
    P.cols = k;
    P.x_ld = x_ld;
    P.q_ld = L.ld;
    P.dtype = static_cast<uint32_t>(x_dtype);
    P.vec = muon::units_aligned(x, x_ld, 0);
    const unsigned row_blocks = blocks_for(m, 1, 65536);
    P.w.src[0] = qw;
    P.w.dst[0] = reinterpret_cast<__half *>(w + L.b);
    P.w.rows[0] = n;
    P.w.src_ld[0] = ldw;
    P.w.cols = k;
    P.w.dst_ld = L.ld;
    P.w.vec[0] = aligned16(qw) && ldw % 16 == 0;
    const unsigned more = blocks_for(n * ((k + 511) / 512), 8, 1216);
    quantise_rows_kernel<false, true><<<row_blocks + more, kThreads, 0, stream>>>(P, row_blocks);
    st = launched(ASR_KERNEL_QUANTIZE);
    if (st != ASR_OK) return st;
    return product(stored(static_cast<__half *>(P.q), m, k, L.ld), stored(P.w.dst[0], n, k, L.ld),
                                 P.scale, sw, o, stream);
}

struct GradLayout {
    // maxima (zeroed together), scales, and the widened matrices
    uint64_t max_row, max_dy, max_w, max_x, zeroed;
    uint64_t row, col_dy, col_w, col_x;
    uint64_t dy_row, dy_col, w, x, bytes, ldn, ldk;
};

GradLayout grad_layout(uint64_t t, uint64_t n, uint64_t k, bool dx, bool dw)
{
    GradLayout L;
    L.ldn = muon::up(n, 16);
    L.ldk = muon::up(k, 16);
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t was = at;
        at += muon::up(bytes, 256);
        return was;
    };
    L.max_row = take(t * 4);
    L.max_dy = take(n * 4);
    L.max_w = take(dx ? k * 4 : 0);
    L.max_x = take(dw ? k * 4 : 0);
    L.zeroed = at;
    L.row = take(t * 4);
    L.col_dy = take(n * 4);
    L.col_w = take(dx ? k * 4 : 0);
    L.col_x = take(dw ? k * 4 : 0);
    L.dy_row = take(dx ? t * L.ldn * 2 : 0);
    L.dy_col = take(dw ? t * L.ldn * 2 : 0);
    L.w = take(dx ? n * L.ldk * 2 : 0);
    L.x = take(dw ? t * L.ldk * 2 : 0);
    L.bytes = at;
    return L;
}

bool grad_sizes_ok(uint64_t t, uint64_t n, uint64_t k)
{
    return sizes_ok(t, n, k) && quantisable(t, n) && quantisable(n, k) && quantisable(t, k);
}

struct GradSource {
    const void *p;
    uint64_t ld;
    int32_t dtype;
};

asr_status grads(const GradSource &dy, const GradSource &x, const GradSource &w, uint16_t *dx, uint64_t dx_ld,
                 uint16_t *dw, uint64_t dw_ld, uint64_t t, uint64_t n, uint64_t k, uint32_t step, uint64_t seed,
                 void *ws, uint64_t ws_bytes, cudaStream_t stream)
{
    auto known = [](const GradSource &s) { return s.dtype == ASR_F32 || s.dtype == ASR_BF16; };
    if (!known(dy) || (dw && !known(x)) || (dx && !known(w))) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (!dx && !dw) return ASR_OK;
    if (t == 0 || n == 0 || k == 0 || !grad_sizes_ok(t, n, k)) return ASR_ERR_INVALID_VALUE;
    const Output ox{dx, dx_ld, ASR_BF16, ASR_ROUND_RNE, 0, 0}, ow{dw, dw_ld, ASR_BF16, ASR_ROUND_RNE, 0, 0};
    if (!dy.p || !pitch_ok(dy.ld, n) || !muon::element_aligned(dy.p, dy.dtype)) return ASR_ERR_INVALID_VALUE;
    if (dx && (!w.p || !pitch_ok(w.ld, k) || !muon::element_aligned(w.p, w.dtype) || !output_ok(ox, k)))
        return ASR_ERR_INVALID_VALUE;
    if (dw && (!x.p || !pitch_ok(x.ld, k) || !muon::element_aligned(x.p, x.dtype) || !output_ok(ow, k)))
        return ASR_ERR_INVALID_VALUE;
    const GradLayout L = grad_layout(t, n, k, dx != nullptr, dw != nullptr);
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < L.bytes) return ASR_ERR_INVALID_VALUE;
    asr_status st = setup();
    if (st != ASR_OK) return st;
    char *b = static_cast<char *>(ws);
    auto words = [&](uint64_t at) { return reinterpret_cast<uint32_t *>(b + at); };
    auto floats = [&](uint64_t at) { return reinterpret_cast<float *>(b + at); };
    auto halves = [&](uint64_t at) { return reinterpret_cast<__half *>(b + at); };
    SideParams M;
    std::memset(&M, 0, sizeof(M));
    M.step = step;
    M.keys = make_keys(seed);
    Side &D = M.s[M.count++];
    D = side(dy.p, dy.dtype, t, n, dy.ld);
    D.row_max = words(L.max_row);
    D.col_max = words(L.max_dy);
    D.row_scale = floats(L.row);
    D.col_scale = floats(L.col_dy);
    D.by_row = dx ? halves(L.dy_row) : nullptr;
    D.by_col = dw ? halves(L.dy_col) : nullptr;
    D.q_ld = L.ldn;
    if (dx) {
        Side &W = M.s[M.count++];
        W = side(w.p, w.dtype, n, k, w.ld);
        W.col_max = words(L.max_w);
        W.col_scale = floats(L.col_w);
        W.by_col = halves(L.w);
        W.q_ld = L.ldk;
    }
    if (dw) {
        Side &X = M.s[M.count++];
        X = side(x.p, x.dtype, t, k, x.ld);
        X.col_max = words(L.max_x);
        X.col_scale = floats(L.col_x);
        X.by_col = halves(L.x);
        X.q_ld = L.ldk;
    }
    st = maxima(M, words(0), L.zeroed / sizeof(uint32_t), stream);
    if (st != ASR_OK) return st;
    st = prod::launch_early(ASR_KERNEL_QUANTIZE, wide_kernel, dim3(M.blocks), kThreads, M, stream);
    if (st != ASR_OK) return st;
    prod::Int8Products P;
    prod::Stored operands[4];
    std::memset(&P, 0, sizeof(P));
    if (dx)
        prod::int8_add(P, operands, stored(halves(L.dy_row), t, n, L.ldn), false, stored(halves(L.w), n, k, L.ldk), true,
                       product_params(floats(L.row), floats(L.col_w), ox));
    if (dw)
        prod::int8_add(P, operands, stored(halves(L.dy_col), t, n, L.ldn), true, stored(halves(L.x), t, k, L.ldk), true,
                       product_params(floats(L.col_dy), floats(L.col_x), ow));
    return prod::int8_launch(P, operands, kChunk, stream);
}

}  // namespace int8
