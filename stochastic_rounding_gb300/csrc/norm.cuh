// norm.cuh -- layer norm and the norm by the root mean square, and their backward
// pass with the weight's and the bias's gradients.  Included into asr.cu (inside
// its anonymous namespace), after checkpoint.cuh.
//
//   mean = sum x / n (centred) or 0;   rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
//   h = (x - mean) rstd;   y = h w + b
//   g = dy w;   dx = rstd (g - [sum g / n] - h sum (g h) / n)
//   dw = sum over rows of dy h;   db = sum over rows of dy
//
// A row is held in registers, 16 values a thread, by a warp or by a block, so it is
// read once.  Its sums: each warp's own mean and its squares about that, then the
// warps' joined (the squares of a warp's mean about the row's added), so nothing
// cancels.  The backward kernel's blocks walk over rows and keep their columns'
// sums for dw and db in registers; a second kernel adds the blocks' sums up, in one
// order.  Rows that do not fit a block of 1,024 threads are read anew for each sum.

namespace norm {

using kept::live_of;

constexpr int kUnits = 2;                       // of eight values, a thread
constexpr uint64_t kWarpCols = 32 * 8 * kUnits; // a warp's row at most
constexpr uint64_t kBlockCols = 1024 * 8 * kUnits;
constexpr int kWarpThreads = 256;               // eight rows a block where a warp has one

struct Params {
    kept::Matrix x, dy;
    kept::Out y, dx;
    const void *w, *b;                          // may be null
    float *mean, *rstd;                         // forward: may be null
    uint64_t rows, cols;
    float eps, over_n;                          // 1 / n
    uint32_t w_dtype, b_dtype, w_vec, b_vec;
    uint32_t centred;
    uint32_t sr;
    kept::Store to;
    kept::Source from;
    float *partial;                             // backward: [groups of threads][2][cols]
    uint32_t sums;                              // whether it is wanted
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

// Eight of the weight or the bias; ones or zeros where there is none.
__device__ __forceinline__ void params8(const void *p, uint32_t dtype, uint64_t col, int live, uint32_t vec, float none,
                                        float v[8])
{
    if (p) {
        muon::load8(p, dtype, col, live, vec, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = none;
    }
}

// A row's place: a warp's, or a block's.
template <bool WARP>
struct Place {
    uint64_t first, stride, group;              // rows; which group of threads this is
    uint32_t at, threads;                       // within the group
    __device__ Place()
    {
        if (WARP) {
            group = blockIdx.x * static_cast<uint64_t>(kWarpThreads / 32) + (threadIdx.x >> 5);
            stride = gridDim.x * static_cast<uint64_t>(kWarpThreads / 32);
            at = threadIdx.x & 31;
            threads = 32;
        } else {
            group = blockIdx.x;
            stride = gridDim.x;
            at = threadIdx.x;
            threads = blockDim.x;
        }
        first = group;
    }
};

// The values' places in a row, for one thread.
struct Unit {
    uint64_t col[kUnits];
    int live[kUnits];
};

__device__ __forceinline__ Unit units_of(uint32_t at, uint32_t threads, uint64_t cols)
{
    Unit U;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        U.col[u] = (static_cast<uint64_t>(u) * threads + at) * 8;
        U.live[u] = live_of(cols, U.col[u]);
    }
    return U;
}

// How many of a row's values the caller's warp holds.
__device__ __forceinline__ float warp_count(const Unit &U)
{
    int n = 0;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) n += U.live[u];
    return static_cast<float>(__reduce_add_sync(0xFFFFFFFFu, n));
}

// The row's mean and sum of squares about it from each warp's; `part` is used by
// turns, so that one barrier a row is enough.
template <bool WARP>
__device__ __forceinline__ void join_moments(float sum, float squares, float count, const Params &P, float3 *part,
                                             float &mean, float &total)
{
    // `sum`, `squares`: of the warp; the squares about its own mean (centred), or about zero
    if (WARP) {
        mean = P.centred ? __fmul_rn(sum, P.over_n) : 0.0f;
        total = squares;
        return;
    }
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if (lane == 0) part[warp] = make_float3(sum, squares, count);
    __syncthreads();
    const float3 p = lane < warps ? part[lane] : make_float3(0.0f, 0.0f, 0.0f);
    mean = P.centred ? __fmul_rn(warp_sum(p.x), P.over_n) : 0.0f;
    float q = p.y;
    if (P.centred && p.z > 0.0f) {
        const float d = __fsub_rn(__fdiv_rn(p.x, p.z), mean);
        q = __fmaf_rn(__fmul_rn(d, d), p.z, q);
    }
    total = warp_sum(q);
}

template <int DT, bool WARP, bool KEEP>
__global__ void __launch_bounds__(WARP ? kWarpThreads : 1024) forward_kernel(const __grid_constant__ Params P)
{
    __shared__ float3 part[2][32];
    const Place<WARP> at;
    const Unit U = units_of(at.at, at.threads, P.cols);
    const float count = warp_count(U);
    uint32_t turn = 0;
    for (uint64_t row = at.first; row < P.rows; row += at.stride, turn ^= 1) {
        float x[kUnits][8], sum = 0.0f, squares = 0.0f;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            muon::load8(P.x.p, DT, row * P.x.ld + U.col[u], U.live[u], P.x.vec, x[u]);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = __fadd_rn(sum, x[u][i]);
        }
        float middle = 0.0f;
        if (P.centred) {
            sum = warp_sum(sum);
            middle = count > 0.0f ? __fdiv_rn(sum, count) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = i < U.live[u] ? __fsub_rn(x[u][i], middle) : 0.0f;
                squares = __fmaf_rn(d, d, squares);
            }
        squares = warp_sum(squares);
        float mean, total;
        join_moments<WARP>(sum, squares, count, P, part[turn], mean, total);
        const float rstd = __frsqrt_rn(__fmaf_rn(total, P.over_n, P.eps));
        if (at.at == 0 && P.rstd) {
            P.rstd[row] = rstd;
            if (P.mean) P.mean[row] = mean;
        }
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            if (KEEP) {
                if (P.sr) kept::keep8<true>(P.to, row, U.col[u], U.live[u], x[u]);
                else kept::keep8<false>(P.to, row, U.col[u], U.live[u], x[u]);
            }
            if (U.live[u] == 0) continue;
            float w[8], b[8];
            params8(P.w, P.w_dtype, U.col[u], U.live[u], P.w_vec, 1.0f, w);
            params8(P.b, P.b_dtype, U.col[u], U.live[u], P.b_vec, 0.0f, b);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[u][i] = __fmaf_rn(__fmul_rn(__fsub_rn(x[u][i], mean), rstd), w[i], b[i]);
            kept::store8<DT>(P.y.p, row * P.y.ld + U.col[u], U.live[u], P.y.vec, x[u]);
        }
    }
}

// Sums over a block's threads, the same in all of them.
__device__ __forceinline__ float block_sum(float v, float *part)
{
    const uint32_t lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    v = warp_sum(v);
    __syncthreads();
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < warps ? part[lane] : 0.0f);
}

// Rows that do not fit: a block each, read three times.
constexpr int kLongThreads = 1024;

template <int DT, bool KEEP>
__global__ void __launch_bounds__(kLongThreads) forward_long_kernel(const __grid_constant__ Params P)
{
    __shared__ float part[32];
    const uint64_t end = (P.cols + 255) / 256 * 256;        // whole warps take part, for the groups
    for (uint64_t row = blockIdx.x; row < P.rows; row += gridDim.x) {
        float sum = 0.0f, squares = 0.0f, x[8];
        if (P.centred)
            for (uint64_t col = threadIdx.x * 8ull; col < P.cols; col += kLongThreads * 8ull) {
                muon::load8(P.x.p, DT, row * P.x.ld + col, live_of(P.cols, col), P.x.vec, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum = __fadd_rn(sum, x[i]);
            }
        const float mean = P.centred ? __fmul_rn(block_sum(sum, part), P.over_n) : 0.0f;
        for (uint64_t col = threadIdx.x * 8ull; col < P.cols; col += kLongThreads * 8ull) {
            const int live = live_of(P.cols, col);
            muon::load8(P.x.p, DT, row * P.x.ld + col, live, P.x.vec, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = i < live ? __fsub_rn(x[i], mean) : 0.0f;
                squares = __fmaf_rn(d, d, squares);
            }
        }
        const float rstd = __frsqrt_rn(__fmaf_rn(block_sum(squares, part), P.over_n, P.eps));
        if (threadIdx.x == 0 && P.rstd) {
            P.rstd[row] = rstd;
            if (P.mean) P.mean[row] = mean;
        }
        for (uint64_t col = threadIdx.x * 8ull; col < end; col += kLongThreads * 8ull) {
            const int live = live_of(P.cols, col);
            muon::load8(P.x.p, DT, row * P.x.ld + col, live, P.x.vec, x);
            if (KEEP) {
                if (P.sr) kept::keep8<true>(P.to, row, col, live, x);
                else kept::keep8<false>(P.to, row, col, live, x);
            }
            if (live == 0) continue;
            float w[8], b[8];
            params8(P.w, P.w_dtype, col, live, P.w_vec, 1.0f, w);
            params8(P.b, P.b_dtype, col, live, P.b_vec, 0.0f, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __fmaf_rn(__fmul_rn(__fsub_rn(x[i], mean), rstd), w[i], b[i]);
            kept::store8<DT>(P.y.p, row * P.y.ld + col, live, P.y.vec, x);
        }
    }
}

// ---- backward

template <int DT, bool KEPT>
__device__ __forceinline__ void input8(const Params &P, uint64_t row, uint64_t col, int live, float x[8])
{
    if (KEPT) kept::values8(kept::fetch8(P.from, row, col, live), x);
    else muon::load8(P.x.p, DT, row * P.x.ld + col, live, P.x.vec, x);
}

template <int DT, bool WARP, bool KEPT, int THREADS>
__global__ void __launch_bounds__(THREADS) backward_kernel(const __grid_constant__ Params P)
{
    __shared__ float2 part[2][32];
    const Place<WARP> at;
    const Unit U = units_of(at.at, at.threads, P.cols);
    float dw[kUnits][8] = {}, db[kUnits][8] = {};
    uint32_t turn = 0;
    for (uint64_t row = at.first; row < P.rows; row += at.stride, turn ^= 1) {
        float h[kUnits][8], g[kUnits][8], along = 0.0f, sum = 0.0f;
        const float mean = P.centred ? P.mean[row] : 0.0f, rstd = P.rstd[row];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            muon::load8(P.dy.p, DT, row * P.dy.ld + U.col[u], U.live[u], P.dy.vec, g[u]);
            input8<DT, KEPT>(P, row, U.col[u], U.live[u], h[u]);
        }
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            float w[8];
            params8(P.w, P.w_dtype, U.col[u], U.live[u], P.w_vec, 1.0f, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[u][i] = __fmul_rn(__fsub_rn(h[u][i], mean), rstd);
                dw[u][i] = __fmaf_rn(g[u][i], h[u][i], dw[u][i]);
                db[u][i] = __fadd_rn(db[u][i], g[u][i]);
                g[u][i] = __fmul_rn(g[u][i], w[i]);
                sum = __fadd_rn(sum, g[u][i]);
                along = __fmaf_rn(g[u][i], h[u][i], along);
            }
        }
        if (!P.dx.p) continue;
        if (P.centred) sum = warp_sum(sum);
        along = warp_sum(along);
        if (!WARP) {
            const uint32_t lane = threadIdx.x & 31, warps = blockDim.x >> 5;
            if (lane == 0) part[turn][threadIdx.x >> 5] = make_float2(sum, along);
            __syncthreads();
            const float2 p = lane < warps ? part[turn][lane] : make_float2(0.0f, 0.0f);
            if (P.centred) sum = warp_sum(p.x);
            along = warp_sum(p.y);
        }
        sum = P.centred ? __fmul_rn(sum, P.over_n) : 0.0f;
        along = __fmul_rn(along, P.over_n);
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                g[u][i] = __fmul_rn(__fmaf_rn(-h[u][i], along, __fsub_rn(g[u][i], sum)), rstd);
            kept::store8<DT>(P.dx.p, row * P.dx.ld + U.col[u], U.live[u], P.dx.vec, g[u]);
        }
    }
    if (!P.sums) return;
    float *to = P.partial + at.group * 2 * P.cols;
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < U.live[u]) {
                to[U.col[u] + i] = dw[u][i];
                to[P.cols + U.col[u] + i] = db[u][i];
            }
}

// Rows that do not fit: dx, a block a row, read twice.
template <int DT, bool KEPT>
__global__ void __launch_bounds__(kLongThreads) backward_long_kernel(const __grid_constant__ Params P)
{
    __shared__ float part[32];
    for (uint64_t row = blockIdx.x; row < P.rows; row += gridDim.x) {
        const float mean = P.centred ? P.mean[row] : 0.0f, rstd = P.rstd[row];
        float sum = 0.0f, along = 0.0f, g[8], h[8], w[8];
        for (uint64_t col = threadIdx.x * 8ull; col < P.cols; col += kLongThreads * 8ull) {
            const int live = live_of(P.cols, col);
            muon::load8(P.dy.p, DT, row * P.dy.ld + col, live, P.dy.vec, g);
            input8<DT, KEPT>(P, row, col, live, h);
            params8(P.w, P.w_dtype, col, live, P.w_vec, 1.0f, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                g[i] = __fmul_rn(g[i], w[i]);
                sum = __fadd_rn(sum, g[i]);
                along = __fmaf_rn(g[i], __fmul_rn(__fsub_rn(h[i], mean), rstd), along);
            }
        }
        sum = P.centred ? __fmul_rn(block_sum(sum, part), P.over_n) : 0.0f;
        along = __fmul_rn(block_sum(along, part), P.over_n);
        for (uint64_t col = threadIdx.x * 8ull; col < P.cols; col += kLongThreads * 8ull) {
            const int live = live_of(P.cols, col);
            muon::load8(P.dy.p, DT, row * P.dy.ld + col, live, P.dy.vec, g);
            input8<DT, KEPT>(P, row, col, live, h);
            params8(P.w, P.w_dtype, col, live, P.w_vec, 1.0f, w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                g[i] = __fmul_rn(__fmaf_rn(-__fmul_rn(__fsub_rn(h[i], mean), rstd), along,
                                           __fsub_rn(__fmul_rn(g[i], w[i]), sum)), rstd);
            kept::store8<DT>(P.dx.p, row * P.dx.ld + col, live, P.dx.vec, g);
        }
    }
}

// Their columns' sums: a block 2,048 columns of every gridDim.y-th row.
template <int DT, bool KEPT>
__global__ void __launch_bounds__(256) columns_kernel(const __grid_constant__ Params P)
{
    const uint64_t col = (blockIdx.x * 256ull + threadIdx.x) * 8;
    const int live = live_of(P.cols, col);
    float dw[8] = {}, db[8] = {}, g[8], h[8];
    for (uint64_t row = blockIdx.y; row < P.rows; row += gridDim.y) {
        const float mean = P.centred ? P.mean[row] : 0.0f, rstd = P.rstd[row];
        muon::load8(P.dy.p, DT, row * P.dy.ld + col, live, P.dy.vec, g);
        input8<DT, KEPT>(P, row, col, live, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dw[i] = __fmaf_rn(g[i], __fmul_rn(__fsub_rn(h[i], mean), rstd), dw[i]);
            db[i] = __fadd_rn(db[i], g[i]);
        }
    }
    float *to = P.partial + blockIdx.y * 2 * P.cols;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < live) {
            to[col + i] = dw[i];
            to[P.cols + col + i] = db[i];
        }
}

struct SumParams {
    const float *partial;
    uint64_t cols, groups;
    void *out[2];                               // dw, db; null where not wanted
    uint32_t dtype[2];
};

// Adds the groups' sums of a column up in one order: a block 32 columns, of dw or of
// db, every sixteenth group a warp.
constexpr int kSumWarps = 16;

__global__ void __launch_bounds__(kSumWarps * 32) sum_kernel(const __grid_constant__ SumParams P)
{
    __shared__ float part[kSumWarps][32];
    const int which = blockIdx.y;
    if (!P.out[which]) return;
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t col = blockIdx.x * 32ull + lane;
    float sum = 0.0f;
    if (col < P.cols)
        for (uint64_t g = warp; g < P.groups; g += kSumWarps) sum = __fadd_rn(sum, P.partial[(g * 2 + which) * P.cols + col]);
    part[warp][lane] = sum;
    __syncthreads();
    if (warp || col >= P.cols) return;
    for (int w = 1; w < kSumWarps; ++w) sum = __fadd_rn(sum, part[w][lane]);
    if (P.dtype[which] == ASR_BF16) static_cast<uint16_t *>(P.out[which])[col] = static_cast<uint16_t>(round_rne(sum));
    else static_cast<float *>(P.out[which])[col] = sum;
}

// ------------------------------------------------------------------ host

using Kernel = void (*)(const Params);

enum { kWarp = 0, kBlock = 1, kLong = 2 };      // who holds a row

int shape_of(uint64_t cols) { return cols <= kWarpCols ? kWarp : cols <= kBlockCols ? kBlock : kLong; }

unsigned block_threads(uint64_t cols) { return static_cast<unsigned>((cols + kWarpCols - 1) / kWarpCols * 32); }

template <int DT, bool KEEP>
Kernel forward_of(int shape)
{
    return shape == kWarp ? forward_kernel<DT, true, KEEP> : shape == kBlock ? forward_kernel<DT, false, KEEP>
                                                                             : forward_long_kernel<DT, KEEP>;
}

Kernel forward_of(int32_t dtype, int shape, bool keep)
{
    if (dtype == ASR_BF16) return keep ? forward_of<ASR_BF16, true>(shape) : forward_of<ASR_BF16, false>(shape);
    return keep ? forward_of<ASR_F32, true>(shape) : forward_of<ASR_F32, false>(shape);
}

// Threads that a block's registers are budgeted for: more a thread in smaller blocks.
template <int DT, bool KEPT>
Kernel backward_of(int shape, unsigned threads)
{
    if (shape == kWarp) return backward_kernel<DT, true, KEPT, kWarpThreads>;
    if (shape == kLong) return backward_long_kernel<DT, KEPT>;
    return threads <= 256 ? backward_kernel<DT, false, KEPT, 256> : threads <= 512 ? backward_kernel<DT, false, KEPT, 512>
                                                                                   : backward_kernel<DT, false, KEPT, 1024>;
}

Kernel backward_of(int32_t dtype, bool codes, int shape, unsigned threads)
{
    if (dtype == ASR_BF16)
        return codes ? backward_of<ASR_BF16, true>(shape, threads) : backward_of<ASR_BF16, false>(shape, threads);
    return codes ? backward_of<ASR_F32, true>(shape, threads) : backward_of<ASR_F32, false>(shape, threads);
}

template <int DT>
Kernel columns_of(bool codes)
{
    return codes ? columns_kernel<DT, true> : columns_kernel<DT, false>;
}

Kernel columns_of(int32_t dtype, bool codes)
{
    return dtype == ASR_BF16 ? columns_of<ASR_BF16>(codes) : columns_of<ASR_F32>(codes);
}

asr_status setup()
{
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (e == cudaSuccess && (ready.load(std::memory_order_acquire) & bit)) return ASR_OK;
    if (e == cudaSuccess) e = prod::load_kernel(sum_kernel);
    for (int32_t dtype : {ASR_F32, ASR_BF16})
        for (int kept = 0; kept < 2; ++kept) {
            if (e == cudaSuccess) e = prod::load_kernel(columns_of(dtype, kept != 0));
            for (int shape : {kWarp, kBlock, kLong}) {
                if (e == cudaSuccess) e = prod::load_kernel(forward_of(dtype, shape, kept != 0));
                for (unsigned threads : {256u, 512u, 1024u})
                    if (e == cudaSuccess) e = prod::load_kernel(backward_of(dtype, kept != 0, shape, threads));
            }
        }
    if (e != cudaSuccess) return cuda_fail(e);
    ready.fetch_or(bit, std::memory_order_release);
    return ASR_OK;
}

asr_status common_ok(const asr_norm_params *p)
{
    if (!p) return ASR_ERR_INVALID_VALUE;
    if (!kept::dtype_ok(p->dtype) || (p->weight && !kept::dtype_ok(p->weight_dtype)) ||
        (p->bias && !kept::dtype_ok(p->bias_dtype)))
        return ASR_ERR_UNSUPPORTED_DTYPE;
    if (!(std::isfinite(p->eps) && p->eps >= 0.0) || p->centred > 1 || p->reserved) return ASR_ERR_INVALID_VALUE;
    return ASR_OK;
}

bool params_ok(const asr_norm_params *p)
{
    return (!p->weight || muon::element_aligned(p->weight, p->weight_dtype)) &&
           (!p->bias || muon::element_aligned(p->bias, p->bias_dtype));
}

Params common(const asr_norm_params *p)
{
    Params P;
    std::memset(&P, 0, sizeof(P));
    P.w = p->weight;
    P.b = p->bias;
    P.rows = p->rows;
    P.cols = p->cols;
    P.eps = static_cast<float>(p->eps);
    P.over_n = static_cast<float>(1.0 / static_cast<double>(p->cols));
    P.w_dtype = static_cast<uint32_t>(p->weight_dtype);
    P.b_dtype = static_cast<uint32_t>(p->bias_dtype);
    P.w_vec = aligned16(p->weight);
    P.b_vec = aligned16(p->bias);
    P.centred = p->centred;
    return P;
}

asr_status forward(const asr_norm_params *p, const void *x, uint64_t x_ld, void *y, uint64_t y_ld, float *mean, float *rstd,
                   const asr_checkpoint *to, cudaStream_t stream)
{
    asr_status st = common_ok(p);
    if (st == ASR_OK && to && to->rounding != ASR_ROUND_SR && to->rounding != ASR_ROUND_RNE) st = ASR_ERR_UNSUPPORTED_DTYPE;
    if (st != ASR_OK || p->rows == 0 || p->cols == 0) return st;
    if (!kept::sizes_ok(p->rows, p->cols) || !kept::matrix_ok(x, p->dtype, x_ld, p->cols) ||
        !kept::matrix_ok(y, p->dtype, y_ld, p->cols) || !params_ok(p) || (mean && !rstd) ||
        !muon::element_aligned(mean, ASR_F32) || !muon::element_aligned(rstd, ASR_F32))
        return ASR_ERR_INVALID_VALUE;
    if (to) st = kept::writable(*to, p->rows, p->cols);
    if (st == ASR_OK) st = setup();
    if (st != ASR_OK) return st;
    Params P = common(p);
    P.x = kept::matrix(x, x_ld);
    P.y = kept::out(y, y_ld);
    P.mean = mean;
    P.rstd = rstd;
    if (to) {
        P.to = kept::store(*to, p->cols);
        P.sr = to->rounding == ASR_ROUND_SR;
    }
    const int shape = shape_of(p->cols);
    const unsigned threads = shape == kWarp ? kWarpThreads : shape == kBlock ? block_threads(p->cols) : kLongThreads;
    const unsigned grid = int8::blocks_for(p->rows, shape == kWarp ? kWarpThreads / 32 : 1, 1u << 20);
    forward_of(p->dtype, shape, to != nullptr)<<<grid, threads, 0, stream>>>(P);
    return launched(ASR_KERNEL_NORM);
}

// Groups of threads that walk over the rows of a backward pass: enough to fill the
// GPU, and eight rows each where there are fewer, since each leaves 2 x cols sums.
constexpr uint64_t kMostGroups = 152 * 4;

uint64_t groups_of(uint64_t rows, uint64_t cols)
{
    const uint64_t most = shape_of(cols) == kWarp ? kMostGroups * (kWarpThreads / 32) : kMostGroups;
    const uint64_t want = shape_of(cols) == kLong ? (rows + 31) / 32 : (rows + 7) / 8;
    const uint64_t g = want < most ? want : most;
    return shape_of(cols) == kWarp ? (g + 7) / 8 * 8 : shape_of(cols) == kLong && g > 64 ? 64 : g;
}

uint64_t workspace_of(uint64_t rows, uint64_t cols) { return groups_of(rows, cols) * 2 * cols * sizeof(float); }

asr_status backward(const asr_norm_params *p, const void *dy, uint64_t dy_ld, const void *x, uint64_t x_ld,
                    const asr_checkpoint *from, const float *mean, const float *rstd, void *dx, uint64_t dx_ld, void *dweight,
                    int32_t dweight_dtype, void *dbias, int32_t dbias_dtype, void *ws, uint64_t ws_bytes, cudaStream_t stream)
{
    asr_status st = common_ok(p);
    if (st != ASR_OK) return st;
    if ((dweight && !kept::dtype_ok(dweight_dtype)) || (dbias && !kept::dtype_ok(dbias_dtype))) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (x && from) return ASR_ERR_INVALID_VALUE;
    if (p->cols == 0 || (!dx && !dweight && !dbias)) return ASR_OK;
    const bool sums = dweight || dbias;
    if ((dweight && !muon::element_aligned(dweight, dweight_dtype)) || (dbias && !muon::element_aligned(dbias, dbias_dtype)) ||
        !kept::sizes_ok(p->rows, p->cols))
        return ASR_ERR_INVALID_VALUE;
    const uint64_t groups = groups_of(p->rows, p->cols);
    if (p->rows) {
        if (!kept::matrix_ok(dy, p->dtype, dy_ld, p->cols) || (dx && !kept::matrix_ok(dx, p->dtype, dx_ld, p->cols)) ||
            !params_ok(p) || !rstd || (p->centred && !mean) || !muon::element_aligned(mean, ASR_F32) ||
            !muon::element_aligned(rstd, ASR_F32))
            return ASR_ERR_INVALID_VALUE;
        if (from) st = kept::readable(*from, p->cols);
        else if (!kept::matrix_ok(x, p->dtype, x_ld, p->cols)) st = ASR_ERR_INVALID_VALUE;
        if (st != ASR_OK) return st;
        if (sums && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < workspace_of(p->rows, p->cols)))
            return ASR_ERR_INVALID_VALUE;
    }
    st = setup();
    if (st != ASR_OK) return st;
    if (p->rows) {
        Params P = common(p);
        P.dy = kept::matrix(dy, dy_ld);
        if (dx) P.dx = kept::out(dx, dx_ld);
        if (from) P.from = kept::source(*from);
        else P.x = kept::matrix(x, x_ld);
        P.mean = const_cast<float *>(mean);
        P.rstd = const_cast<float *>(rstd);
        P.partial = static_cast<float *>(ws);
        P.sums = sums;
        const int shape = shape_of(p->cols);
        const unsigned threads = shape == kWarp ? kWarpThreads : shape == kBlock ? block_threads(p->cols) : kLongThreads;
        if (shape != kLong || dx) {
            const unsigned grid = shape == kWarp ? static_cast<unsigned>(groups / 8) :
                                  shape == kBlock ? static_cast<unsigned>(groups) : int8::blocks_for(p->rows, 1, 1u << 20);
            backward_of(p->dtype, from != nullptr, shape, threads)<<<grid, threads, 0, stream>>>(P);
            st = launched(ASR_KERNEL_NORM);
        }
        if (st == ASR_OK && shape == kLong && sums) {
            const dim3 grid(static_cast<unsigned>((p->cols + 2047) / 2048), static_cast<unsigned>(groups));
            columns_of(p->dtype, from != nullptr)<<<grid, 256, 0, stream>>>(P);
            st = launched(ASR_KERNEL_NORM);
        }
        if (st != ASR_OK) return st;
    }
    if (!sums) return ASR_OK;
    SumParams S;
    S.partial = static_cast<const float *>(ws);
    S.cols = p->cols;
    S.groups = p->rows ? groups : 0;
    S.out[0] = dweight;
    S.out[1] = dbias;
    S.dtype[0] = static_cast<uint32_t>(dweight_dtype);
    S.dtype[1] = static_cast<uint32_t>(dbias_dtype);
    const dim3 grid(static_cast<unsigned>((p->cols + 31) / 32), dbias ? 2 : 1);
    sum_kernel<<<grid, kSumWarps * 32, 0, stream>>>(S);
    return launched(ASR_KERNEL_NORM);
}

}  // namespace norm
