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
// the call's base index, whichever way the matrix is stored.  The sum of
// integers is exact.  sm_103a's tensor memory instructions have no 8-bit
// integer kind; an 8-bit integer is exact in f16, a product of two in binary32,
// and so is any sum of 1,024 of them (1,024 * 128^2 = 2^24).  So the operands
// are widened to f16 in the workspace, product.cuh sums chunks of 1,024 in
// tensor memory at the f16 rate, and its epilogue adds the chunks in int32.

namespace int8 {

constexpr int kThreads = 256;
constexpr uint64_t kMaxK = 131071;              // 128^2 K < 2^31
constexpr uint32_t kChunk = 1024 / prod::kBK;

struct QuantParams {
    const void *x;
    int8_t *q;
    float *scale;
    uint64_t rows, cols, x_ld, q_ld;
    uint64_t base;
    uint32_t dtype, rounding, step;
    uint32_t vec;                               // 8-element units of x are 16-byte aligned
    RoundKeys keys;
};

// How a row's values become integers: y = (x * pre) * inv.  A row whose largest
// value is so small that 127 / max would overflow is raised by 2^64 first (exact);
// a row that holds an infinity or a NaN gives zeros, and its scale, not finite,
// marks every product of the row.
struct Levels {
    float pre, inv;
};

__device__ __forceinline__ Levels levels_of(float top)
{
    Levels L;
    L.pre = top < 0x1p-64f ? 0x1p64f : 1.0f;
    L.inv = top > 0.0f && top <= 3.402823466e38f ? __fdiv_rn(127.0f, __fmul_rn(top, L.pre)) : 0.0f;
    return L;
}

template <bool SR>
__device__ __forceinline__ int quantise(float x, const Levels &L, uint32_t r)
{
    const float y = __fmul_rn(__fmul_rn(x, L.pre), L.inv);
    if (!SR) {
        const int q = __float2int_rn(y);
        return L.inv == 0.0f ? 0 : q;           // |y| <= 127 (1 + 2^-23): rounds to at most 127
    }
    const float low = floorf(y);
    const int q = static_cast<int>(low) + (__fmul_rn(__fsub_rn(y, low), 65536.0f) > static_cast<float>(r & 0xFFFFu));
    return L.inv == 0.0f ? 0 : max(-127, min(127, q));
}

__device__ __forceinline__ uint32_t absbits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t *part)
{
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[0];
    for (int w = 1; w < kThreads / 32; ++w) v = max(v, part[w]);
    return v;
}

// One block a row.
template <bool SR>
__global__ void __launch_bounds__(kThreads) quantise_rows_kernel(const __grid_constant__ QuantParams P)
{
    __shared__ uint32_t part[kThreads / 32];
    for (uint64_t row = blockIdx.x; row < P.rows; row += gridDim.x) {
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
            if (SR) unit_words<false>(P.base + row * P.cols, col, P.step, P.keys, r);
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int q = 0; q < 8; ++q)
                w[q >> 2] |= static_cast<uint32_t>(quantise<SR>(x[q], L, SR ? r[q] : 0u) & 0xFF) << (8 * (q & 3));
            int8_t *dst = P.q + row * P.q_ld + col;
            if (live == 8 && (reinterpret_cast<uintptr_t>(dst) & 7u) == 0) {
                *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
            } else {
                for (int q = 0; q < live; ++q) dst[q] = static_cast<int8_t>(w[q >> 2] >> (8 * (q & 3)));
            }
        }
        __syncthreads();
    }
}

// Columns: the largest value of each (bits, in `scale`, zeroed before) ...
__global__ void __launch_bounds__(kThreads) column_max_kernel(const __grid_constant__ QuantParams P)
{
    const uint64_t col = (blockIdx.x * 32ull + (threadIdx.x & 31)) * 8;
    if (col >= P.cols) return;
    const int live = P.cols - col < 8 ? static_cast<int>(P.cols - col) : 8;
    uint32_t top[8] = {};
    for (uint64_t row = blockIdx.y * 8ull + (threadIdx.x >> 5); row < P.rows; row += gridDim.y * 8ull) {
        float x[8];
        muon::load8(P.x, P.dtype, row * P.x_ld + col, live, P.vec, x);
#pragma unroll
        for (int q = 0; q < 8; ++q) top[q] = max(top[q], absbits(x[q]));
    }
    // integer maxima: the same whatever their order
    for (int q = 0; q < live; ++q) atomicMax(reinterpret_cast<uint32_t *>(P.scale) + col + q, top[q]);
}

// ... the integers, 64 x 64 tiles turned in shared memory ...
template <bool SR>
__global__ void __launch_bounds__(kThreads) quantise_columns_kernel(const __grid_constant__ QuantParams P)
{
    __shared__ int8_t tile[64][68];
    const uint64_t r0 = blockIdx.y * 64ull, c0 = blockIdx.x * 64ull;
    for (int i = threadIdx.x; i < 64 * 8; i += kThreads) {
        const uint64_t row = r0 + (i >> 3), col = c0 + (i & 7) * 8;
        if (row >= P.rows || col >= P.cols) continue;
        const int live = P.cols - col < 8 ? static_cast<int>(P.cols - col) : 8;
        float x[8];
        muon::load8(P.x, P.dtype, row * P.x_ld + col, live, P.vec, x);
        uint32_t r[8];
        if (SR) unit_words<false>(P.base + row * P.cols, col, P.step, P.keys, r);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (q < live)
                tile[(i & 7) * 8 + q][i >> 3] =
                    static_cast<int8_t>(quantise<SR>(x[q], levels_of(P.scale[col + q]), SR ? r[q] : 0u));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * 64; i += kThreads) {
        const uint64_t col = c0 + (i >> 6), row = r0 + (i & 63);
        if (row < P.rows && col < P.cols) P.q[col * P.q_ld + row] = tile[i >> 6][i & 63];
    }
}

// ... and the scales.
__global__ void __launch_bounds__(kThreads) column_scale_kernel(float *scale, uint64_t n)
{
    const uint64_t i = blockIdx.x * static_cast<uint64_t>(kThreads) + threadIdx.x;
    if (i < n) scale[i] = __fdiv_rn(scale[i], 127.0f);
}

struct WidenParams {
    const int8_t *src[2];
    __half *dst[2];
    uint64_t rows[2], src_ld[2];
    uint64_t cols, dst_ld;                      // dst_ld: cols up to a multiple of 16
    uint32_t vec[2];
};

__device__ __forceinline__ uint32_t widen2(int lo, int hi)
{
    const __half2 h = __halves2half2(__int2half_rn(lo), __int2half_rn(hi));
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 8-bit integers to f16: 16 a thread.
__global__ void __launch_bounds__(kThreads) widen_kernel(const __grid_constant__ WidenParams P)
{
    const uint64_t per_row = P.dst_ld / 16, first = P.rows[0] * per_row, units = first + P.rows[1] * per_row;
    for (uint64_t u = blockIdx.x * static_cast<uint64_t>(kThreads) + threadIdx.x; u < units;
         u += static_cast<uint64_t>(gridDim.x) * kThreads) {
        const int which = u >= first;
        const uint64_t v = which ? u - first : u;
        const uint64_t row = v / per_row, col = (v - row * per_row) * 16;
        const int live = P.cols - col < 16 ? static_cast<int>(P.cols - col) : 16;
        const int8_t *src = P.src[which] + row * P.src_ld[which] + col;
        int x[16];
        if (P.vec[which] && live == 16) {
            const int4 w = *reinterpret_cast<const int4 *>(src);
            const int a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int q = 0; q < 16; ++q) x[q] = static_cast<int8_t>(a[q >> 2] >> (8 * (q & 3)));
        } else {
#pragma unroll
            for (int q = 0; q < 16; ++q) x[q] = q < live ? src[q] : 0;
        }
        uint4 *dst = reinterpret_cast<uint4 *>(P.dst[which] + row * P.dst_ld + col);
        dst[0] = make_uint4(widen2(x[0], x[1]), widen2(x[2], x[3]), widen2(x[4], x[5]), widen2(x[6], x[7]));
        dst[1] = make_uint4(widen2(x[8], x[9]), widen2(x[10], x[11]), widen2(x[12], x[13]), widen2(x[14], x[15]));
    }
}

// ------------------------------------------------------------------ host

asr_status quantize(const void *x, int32_t dtype, uint64_t rows, uint64_t cols, uint64_t x_ld, int32_t axis, int8_t *q,
                    uint64_t q_ld, float *scale, uint32_t rounding, uint64_t base, uint32_t step, uint64_t seed,
                    cudaStream_t stream)
{
    if (dtype != ASR_F32 && dtype != ASR_BF16) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (rounding != ASR_ROUND_SR && rounding != ASR_ROUND_RNE) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (axis != ASR_ROWS && axis != ASR_COLUMNS) return ASR_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0) return ASR_OK;
    if (!x || !q || !scale || !muon::element_aligned(x, dtype) || !muon::element_aligned(scale, ASR_F32))
        return ASR_ERR_INVALID_VALUE;
    if (rows > (1u << 30) || cols > (1u << 30) || x_ld < cols || x_ld > (1ull << 32) || q_ld > (1ull << 32) ||
        q_ld < (axis == ASR_ROWS ? cols : rows) || base > UINT64_MAX - rows * cols)
        return ASR_ERR_INVALID_VALUE;
    QuantParams P;
    P.x = x;
    P.q = q;
    P.scale = scale;
    P.rows = rows;
    P.cols = cols;
    P.x_ld = x_ld;
    P.q_ld = q_ld;
    P.base = base;
    P.dtype = static_cast<uint32_t>(dtype);
    P.rounding = rounding;
    P.step = step;
    P.vec = muon::units_aligned(x, x_ld, 0);
    P.keys = make_keys(seed);
    const bool sr = rounding == ASR_ROUND_SR;
    if (axis == ASR_ROWS) {
        const unsigned grid = static_cast<unsigned>(rows < 65536 ? rows : 65536);
        if (sr) quantise_rows_kernel<true><<<grid, kThreads, 0, stream>>>(P);
        else quantise_rows_kernel<false><<<grid, kThreads, 0, stream>>>(P);
        return launched(ASR_KERNEL_QUANTIZE);
    }
    if ((rows + 63) / 64 > 65535) return ASR_ERR_INVALID_VALUE;
    cudaError_t e = cudaMemsetAsync(scale, 0, cols * sizeof(float), stream);
    if (e != cudaSuccess) return cuda_fail(e);
    const uint64_t strips = (cols + 255) / 256, chunks = (rows + 63) / 64;
    column_max_kernel<<<dim3(static_cast<unsigned>(strips), static_cast<unsigned>(chunks)), kThreads, 0, stream>>>(P);
    asr_status st = launched(ASR_KERNEL_QUANTIZE);
    if (st != ASR_OK) return st;
    const dim3 grid(static_cast<unsigned>((cols + 63) / 64), static_cast<unsigned>((rows + 63) / 64));
    if (sr) quantise_columns_kernel<true><<<grid, kThreads, 0, stream>>>(P);
    else quantise_columns_kernel<false><<<grid, kThreads, 0, stream>>>(P);
    st = launched(ASR_KERNEL_QUANTIZE);
    if (st != ASR_OK) return st;
    column_scale_kernel<<<static_cast<unsigned>((cols + kThreads - 1) / kThreads), kThreads, 0, stream>>>(scale, cols);
    return launched(ASR_KERNEL_QUANTIZE);
}

struct Layout {
    uint64_t a, b, bytes, ld;
};

Layout layout(uint64_t m, uint64_t n, uint64_t k)
{
    Layout L;
    L.ld = muon::up(k, 16);
    L.a = 0;
    L.b = muon::up(m * L.ld * 2, 256);
    L.bytes = L.b + muon::up(n * L.ld * 2, 256);
    return L;
}

bool sizes_ok(uint64_t m, uint64_t n, uint64_t k)
{
    return m <= (1u << 24) && n <= (1u << 24) && k <= kMaxK;
}

asr_status gemm(const int8_t *a, uint64_t lda, const int8_t *b, uint64_t ldb, const float *sa, const float *sb, void *c,
                uint64_t ldc, int32_t c_dtype, uint64_t m, uint64_t n, uint64_t k, uint32_t rounding, uint32_t step,
                uint64_t seed, void *ws, uint64_t ws_bytes, cudaStream_t stream)
{
    if (c_dtype != ASR_F32 && c_dtype != ASR_BF16) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (rounding != ASR_ROUND_SR && rounding != ASR_ROUND_RNE) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (m == 0 || n == 0) return ASR_OK;
    if (!sizes_ok(m, n, k) || k == 0) return ASR_ERR_INVALID_VALUE;
    if (!a || !b || !sa || !sb || !c || lda < k || ldb < k || ldc < n || lda > (1ull << 32) || ldb > (1ull << 32) ||
        ldc > (1ull << 32))
        return ASR_ERR_INVALID_VALUE;
    if (!muon::element_aligned(sa, ASR_F32) || !muon::element_aligned(sb, ASR_F32) ||
        !muon::element_aligned(c, c_dtype))
        return ASR_ERR_INVALID_VALUE;
    const Layout L = layout(m, n, k);
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < L.bytes) return ASR_ERR_INVALID_VALUE;
    int pairs = 0;
    asr_status st = prod::setup(&pairs);
    if (st != ASR_OK) return st;
    char *w = static_cast<char *>(ws);
    WidenParams W;
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
    const uint64_t blocks = ((m + n) * (L.ld / 16) + kThreads - 1) / kThreads;
    widen_kernel<<<static_cast<unsigned>(blocks < 65536 ? blocks : 65536), kThreads, 0, stream>>>(W);
    st = launched(ASR_KERNEL_QUANTIZE);
    if (st != ASR_OK) return st;
    prod::Params P;
    std::memset(&P, 0, sizeof(P));
    P.batch = 1;
    P.chunk = kChunk;
    P.out_ld = ldc;
    P.out_dtype = static_cast<uint32_t>(c_dtype);
    P.rounding = rounding;
    P.vec = muon::aligned32(c) && ldc % 16 == 0;
    P.step = step;
    P.row_scale = sa;
    P.col_scale = sb;
    P.keys = make_keys(seed);
    P.slot[0].ptr = c;
    const prod::Stored A{W.dst[0], m, k, L.ld, muon::up(m * L.ld * 2, 256) / 2};
    const prod::Stored B{W.dst[1], n, k, L.ld, muon::up(n * L.ld * 2, 256) / 2};
    return prod::launch<false, false, prod::kInt8>(A, B, P, ASR_KERNEL_PRODUCT, stream);
}

}  // namespace int8
