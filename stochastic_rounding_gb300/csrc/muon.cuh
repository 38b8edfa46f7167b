// muon.cuh -- orthogonalising an update by Newton-Schulz products, and the Muon
// step around it.  Included into asr.cu (inside its anonymous namespace), after
// product.cuh.
//
//   X_0 = G / max(|G|_F, eps)
//   S   = X X^T (rows <= cols) or X^T X
//   X'  = a X + (b S + c S S) X, or X (..) on the other side;   `steps` times
//
// Matrices whose smaller side is at most 128 (the larger at most 4,096) take one
// launch (skinny.cuh).  The others are streamed once each by two kernels: sums of
// squares (and the momentum, for Muon), then the scaled f16 copy (8 x 2,048^2,
// Muon: 55 and 50 us for 335 and 268 MB, 6.0 and 5.4 TB/s); the products are
// product.cuh's, all matrices of one shape in each launch, and the last one's
// epilogue writes the caller's matrix -- the bf16 result, or the parameter
// itself, decayed, stepped and rounded with its own random bits.  With P = a I + b S + c S S formed by the
// epilogue of S S, a step is three products: S and S S (symmetric: half the
// tiles), and P X.  m = min(rows, cols), n = max: 3 m^2 n + m^3 multiplications
// and additions a step.
//
// Number format.  Every matrix between the products is f16 at 2^12 times its
// value.  Singular values start at or below 1 and the polynomial keeps them
// small (checked on the host for the coefficients of the call), an entry is
// never larger than the largest singular value, so 2^12 leaves a factor of 16
// to f16's largest number and puts its smallest normal number at 1.5e-8 --
// below the entries of S (about n^-1.5) that a matrix of any practical size
// has.  f16 keeps three more bits than bf16 at the same tensor rate, which the
// iteration needs: it raises small singular values by a^steps (485 for the
// usual coefficients), and the rounding of X's entries with them.  Sums, norms
// and momentum are binary32 or wider.
//
// Diagonals.  Where singular values bunch (a short and wide matrix), S and P are
// nearly multiples of I, and the rounding of their diagonals is the same for
// all rows: not noise but a factor, up to 2^-11 a step and matrix.  So S's
// diagonal is kept in binary32 as well and P's made from it, and each row of P X is
// multiplied by P's diagonal over its rounded value (the rest of the row takes
// the same factor, within its own rounding).  Error of the bf16 result against
// 64 bits, without and with: 137 x 7,674 0.0028 and 0.0018, 16 x 300 0.0027 and
// 0.0022, 512 x 2,048 0.0019 and 0.0018; of the exact result rounded to bf16
// 0.0017.  It costs 1.5 us of 27 for 96 x 160 and nothing that shows above that.

namespace muon {

constexpr int kThreads = 256;
constexpr int kPartBlocks = 1024;           // partial sums a matrix at most
constexpr int kSpan = 256;                  // columns a warp takes at a time, eight a lane
constexpr float kStore = 4096.0f;
constexpr double kLargest = 8.0;            // bound of every stored value / 2^12

struct Matrix {                             // one matrix of a stack
    const void *src;                        // G, or the gradient
    float *momentum;                        // Muon: updated in place
};

struct PrepParams {
    uint64_t rows, cols, src_ld;
    uint32_t src_dtype;                     // asr_dtype
    uint32_t vec;                           // 8-element units of the source and momentum are 16-byte aligned
    uint32_t blocks;                        // per matrix
    uint32_t nesterov;
    float mu, omu;                          // momentum, 1 - momentum
    float eps;
    float2 *partial;                        // [batch][blocks]
    __half *out;                            // [batch][rows][ld], 2^12 X
    uint64_t out_ld, out_stride;
    Matrix m[prod::kMaxBatch];
};

// Units of 8 columns; a row's last unit may be short.
__device__ __forceinline__ void load8(const void *src, uint32_t dtype, uint64_t at, int live, bool vec, float x[8])
{
    if (dtype == ASR_BF16) {
        const uint16_t *p = static_cast<const uint16_t *>(src) + at;
        if (vec && live == 8) {
            const uint4 w = *reinterpret_cast<const uint4 *>(p);
            x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
            x[4] = bf16_lo(w.z), x[5] = bf16_hi(w.z), x[6] = bf16_lo(w.w), x[7] = bf16_hi(w.w);
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = q < live ? bf16_lo(p[q]) : 0.0f;
        }
    } else {
        const float *p = static_cast<const float *>(src) + at;
        if (vec && live == 8) {
            const float4 u = reinterpret_cast<const float4 *>(p)[0], v = reinterpret_cast<const float4 *>(p)[1];
            x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = q < live ? p[q] : 0.0f;
        }
    }
}

// u = what is orthogonalised, from the gradient and the new momentum.
__device__ __forceinline__ float update_of(const PrepParams &P, float g, float m)
{
    return P.nesterov ? __fadd_rn(g, __fmul_rn(P.mu, __fsub_rn(m, g))) : m;
}

// A sum of squares of x, and of 2^64 x.  The first is used unless it is below
// 2^-60; squares below 2^-126, which binary32 loses, do not matter in one that is
// not.  If it is, every x is below 2^-30 and the second does not overflow.
// (Squares alone: entries of 1e-23 come out as zeros, and 2^12 x / eps past f16.)
struct Squares {
    float plain, raised;
};

__device__ __forceinline__ void add_square(Squares &s, float x)
{
    s.plain = fmaf(x, x, s.plain);
    const float y = __fmul_rn(x, 0x1p64f);
    s.raised = fmaf(y, y, s.raised);
}

__device__ __forceinline__ void add_squares(Squares &s, float plain, float raised)
{
    s.plain += plain;
    s.raised += raised;
}

// Over a warp, in every lane.
__device__ __forceinline__ void add_warp(Squares &s)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        add_squares(s, __shfl_xor_sync(0xFFFFFFFFu, s.plain, o), __shfl_xor_sync(0xFFFFFFFFu, s.raised, o));
}

// What X_0 = G / max(norm, eps) is multiplied with to be stored.  A norm that is
// not finite makes every entry NaN, so that a gradient holding an infinity or a
// NaN shows in the whole result.
__device__ __forceinline__ float factor_of(const Squares &s, float eps)
{
    const float norm = s.plain < 0x1p-60f ? __fmul_rn(__fsqrt_rn(s.raised), 0x1p-64f) : __fsqrt_rn(s.plain);
    return norm <= 3.402823466e38f ? __fdiv_rn(kStore, fmaxf(norm, eps)) : __int_as_float(0x7FC00000);
}

// A warp's way through a matrix in spans of kSpan columns: span `at` counted
// along the rows, then every `stride`-th.  One division at the start instead of
// one an element.
struct Walk {
    uint64_t row, rows;
    uint32_t span, spans, dspan;
    uint64_t drow;
    __device__ Walk(uint64_t rows_, uint64_t cols, uint64_t at, uint64_t stride)
    {
        rows = rows_;
        spans = static_cast<uint32_t>((cols + kSpan - 1) / kSpan);
        row = at / spans;
        span = static_cast<uint32_t>(at % spans);
        drow = stride / spans;
        dspan = static_cast<uint32_t>(stride % spans);
    }
    __device__ bool more() const { return row < rows; }
    __device__ void next()
    {
        row += drow;
        span += dspan;
        if (span >= spans) {
            span -= spans;
            ++row;
        }
    }
};

// First pass: m <- m + (1 - mu)(g - m) (MUON), and each block's sums of squares.
template <bool MUON>
__global__ void __launch_bounds__(kThreads) square_sum_kernel(const __grid_constant__ PrepParams P)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Matrix M = P.m[blockIdx.y];
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Squares sum = {0.0f, 0.0f};
    for (Walk k(P.rows, P.cols, blockIdx.x * 8ull + warp, P.blocks * 8ull); k.more(); k.next()) {
        const uint64_t row = k.row, col = k.span * static_cast<uint64_t>(kSpan) + lane * 8;
        if (col >= P.cols) continue;
        const int live = P.cols - col < 8 ? static_cast<int>(P.cols - col) : 8;
        float x[8];
        load8(M.src, P.src_dtype, row * P.src_ld + col, live, P.vec, x);
        if (MUON) {
            float m[8];
            const uint64_t at = row * P.cols + col;
            load8(M.momentum, ASR_F32, at, live, P.vec, m);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                m[q] = __fadd_rn(m[q], __fmul_rn(P.omu, __fsub_rn(x[q], m[q])));
                x[q] = update_of(P, x[q], m[q]);
            }
            if (P.vec && live == 8) {
                reinterpret_cast<float4 *>(M.momentum + at)[0] = make_float4(m[0], m[1], m[2], m[3]);
                reinterpret_cast<float4 *>(M.momentum + at)[1] = make_float4(m[4], m[5], m[6], m[7]);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q < live) M.momentum[at + q] = m[q];
            }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) add_square(sum, x[q]);
    }
    add_warp(sum);
    __shared__ Squares part[kThreads / 32];
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) add_squares(sum, part[w].plain, part[w].raised);
        P.partial[blockIdx.y * P.blocks + blockIdx.x] = make_float2(sum.plain, sum.raised);
    }
}

// Second pass: X_0 in f16.  Each block adds the matrix's partial sums again, in
// one order.
template <bool MUON>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ PrepParams P)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Matrix M = P.m[blockIdx.y];
    __shared__ Squares part[kThreads / 32];
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Squares sum = {0.0f, 0.0f};
    for (uint32_t i = threadIdx.x; i < P.blocks; i += kThreads) {
        const float2 v = P.partial[blockIdx.y * P.blocks + i];
        add_squares(sum, v.x, v.y);
    }
    add_warp(sum);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    sum = {0.0f, 0.0f};
    for (int w = 0; w < kThreads / 32; ++w) add_squares(sum, part[w].plain, part[w].raised);
    const float f = factor_of(sum, P.eps);
    __half *out = P.out + blockIdx.y * P.out_stride;
    for (Walk k(P.rows, P.cols, blockIdx.x * 8ull + warp, gridDim.x * 8ull); k.more(); k.next()) {
        const uint64_t row = k.row, col = k.span * static_cast<uint64_t>(kSpan) + lane * 8;
        if (col >= P.cols) continue;
        const int live = P.cols - col < 8 ? static_cast<int>(P.cols - col) : 8;
        float x[8];
        load8(M.src, P.src_dtype, row * P.src_ld + col, live, P.vec, x);
        if (MUON) {
            float m[8];
            load8(M.momentum, ASR_F32, row * P.cols + col, live, P.vec, m);
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = update_of(P, x[q], m[q]);
        }
        // the row's padding (rows are a multiple of 16 values apart) takes the zeros of a short unit
        *reinterpret_cast<uint4 *>(out + row * P.out_ld + col) =
            make_uint4(prod::pack_f16(x[0] * f, x[1] * f), prod::pack_f16(x[2] * f, x[3] * f),
                       prod::pack_f16(x[4] * f, x[5] * f), prod::pack_f16(x[6] * f, x[7] * f));
    }
}

#include "skinny.cuh"

// ------------------------------------------------------------------ host

uint64_t up(uint64_t x, uint64_t to) { return (x + to - 1) / to * to; }

// The bound that the number format needs: with singular values in [0, s], the
// next ones are at most max |a x + b x^3 + c x^5|, and P's largest entry is at
// most max |a + b t + c t^2| over t = x^2.
bool coefficients_fit(double a, double b, double c, uint32_t steps)
{
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
    double s = 1.001;
    for (uint32_t i = 0; i < steps; ++i) {
        const double t1 = s * s;
        double p = std::max(std::fabs(a), std::fabs(a + b * t1 + c * t1 * t1));
        double next = s * std::fabs(a + b * t1 + c * t1 * t1);
        if (c != 0.0) {
            const double v = -b / (2.0 * c);
            if (v > 0.0 && v < t1) p = std::max(p, std::fabs(a + b * v + c * v * v));
        }
        // stationary points of a x + b x^3 + c x^5: 5 c t^2 + 3 b t + a = 0
        double roots[2];
        int n = 0;
        if (c != 0.0) {
            const double disc = 9.0 * b * b - 20.0 * a * c;
            if (disc >= 0.0) {
                roots[n++] = (-3.0 * b + std::sqrt(disc)) / (10.0 * c);
                roots[n++] = (-3.0 * b - std::sqrt(disc)) / (10.0 * c);
            }
        } else if (b != 0.0) {
            roots[n++] = -a / (3.0 * b);
        }
        for (int r = 0; r < n; ++r)
            if (roots[r] > 0.0 && roots[r] < t1)
                next = std::max(next, std::sqrt(roots[r]) * std::fabs(a + roots[r] * (b + c * roots[r])));
        // S S goes unstored; P, X' and S' = X' X'^T are stored
        if (!(p <= kLargest) || !(next <= kLargest) || !(next * next <= kLargest) || !(t1 * t1 * std::fabs(c) <= 1e6))
            return false;
        s = next * 1.001;
    }
    return true;
}

struct NsParams {
    double a, b, c, eps;
    uint32_t steps;
};

struct Group {                              // a launch's stack: up to kMaxBatch matrices of one shape
    uint64_t rows, cols, src_ld, out_ld;
    uint32_t src_dtype, out_dtype;
    bool vec_in, vec_out;
    uint32_t batch;
    Matrix m[prod::kMaxBatch];
    prod::Slot out[prod::kMaxBatch];
};

struct Layout {                             // a group's part of the workspace
    uint64_t partial, diag, gain, x0, x1, s, p, bytes;
    uint64_t ldx, lds, m;
};

Layout layout(uint64_t rows, uint64_t cols, uint64_t batch)
{
    Layout L{};
    if (skinny_fits(rows, cols)) {              // everything in shared memory
        L.bytes = 256;
        return L;
    }
    L.m = rows < cols ? rows : cols;
    L.ldx = up(cols, 16);
    L.lds = up(L.m, 16);
    const uint64_t x = up(rows * L.ldx * 2, 256) * batch, s = up(L.m * L.lds * 2, 256) * batch;
    L.partial = 0;
    L.diag = up(batch * kPartBlocks * sizeof(float2), 256);
    L.gain = L.diag + up(batch * L.lds * sizeof(float), 256);
    L.x0 = L.gain + up(batch * L.lds * sizeof(float), 256);
    L.x1 = L.x0 + x;
    L.s = L.x1 + x;
    L.p = L.s + s;
    L.bytes = L.p + s;
    return L;
}

// Matrices a launch: as many as fill the GPU a few times over; more would only
// grow the workspace (kept to 2 GB, or one matrix).
uint32_t batch_limit(uint64_t rows, uint64_t cols)
{
    const uint64_t one = layout(rows, cols, 1).bytes;
    const uint64_t fit = (2ull << 30) / one;
    return static_cast<uint32_t>(fit < 1 ? 1 : fit < prod::kMaxBatch ? fit : prod::kMaxBatch);
}

void prep_params(PrepParams &P, const Group &G, const NsParams &ns, float mu, bool nesterov)
{
    P.rows = G.rows;
    P.cols = G.cols;
    P.src_ld = G.src_ld;
    P.src_dtype = G.src_dtype;
    P.vec = G.vec_in;
    P.nesterov = nesterov;
    P.mu = mu;
    P.omu = static_cast<float>(1.0 - static_cast<double>(mu));
    P.eps = static_cast<float>(ns.eps);
    std::memcpy(P.m, G.m, sizeof(Matrix) * G.batch);
}

template <bool MUON>
asr_status prep(const Group &G, const NsParams &ns, const Layout &L, char *ws, float mu, bool nesterov,
                cudaStream_t stream)
{
    PrepParams P;
    std::memset(&P, 0, sizeof(P));
    prep_params(P, G, ns, mu, nesterov);
    // eight spans a block at least, and no more blocks than fill the GPU (152
    // SMs, eight a SM) or make enough partial sums
    const uint64_t want = (G.rows * ((G.cols + kSpan - 1) / kSpan) + 7) / 8;
    const uint64_t fill = std::max<uint64_t>(16, std::min<uint64_t>(kPartBlocks, 1216 / G.batch));
    P.blocks = static_cast<uint32_t>(want < fill ? want : fill);
    P.partial = reinterpret_cast<float2 *>(ws + L.partial);
    P.out = reinterpret_cast<__half *>(ws + L.x0);
    P.out_ld = L.ldx;
    P.out_stride = up(G.rows * L.ldx * 2, 256) / 2;
    const dim3 grid(P.blocks, G.batch, 1);
    square_sum_kernel<MUON><<<grid, kThreads, 0, stream>>>(P);
    const asr_status st = launched(ASR_KERNEL_MATRIX_PREP);
    if (st != ASR_OK) return st;
    return prod::launch_early(ASR_KERNEL_MATRIX_PREP, scale_kernel<MUON>, grid, kThreads, P, stream);
}

// A group whose matrices' smaller side is at most 128: one launch.
std::mutex g_skinny_mu;
bool g_skinny_ready[kMaxDevices];

// Every kernel of this file and of the products ready on the device.
asr_status setup()
{
    int pairs = 0;
    const asr_status st = prod::setup(&pairs);
    if (st != ASR_OK) return st;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev < 0 || dev >= kMaxDevices) return ASR_ERR_INVALID_VALUE;
    std::lock_guard<std::mutex> lk(g_skinny_mu);
    if (!g_skinny_ready[dev]) {
        e = cudaFuncSetAttribute(skinny_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSkinnySmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(skinny_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSkinnySmem);
        if (e == cudaSuccess) e = prod::load_kernel(square_sum_kernel<false>);
        if (e == cudaSuccess) e = prod::load_kernel(square_sum_kernel<true>);
        if (e == cudaSuccess) e = prod::load_kernel(scale_kernel<false>);
        if (e == cudaSuccess) e = prod::load_kernel(scale_kernel<true>);
        if (e != cudaSuccess) return cuda_fail(e);
        g_skinny_ready[dev] = true;
    }
    return ASR_OK;
}

template <bool MUON>
asr_status skinny(const Group &G, const NsParams &ns, const prod::Params &last, float mu, bool nesterov,
                  cudaStream_t stream)
{
    SkinnyParams P;
    std::memset(&P, 0, sizeof(P));
    prep_params(P.in, G, ns, mu, nesterov);
    P.out = last;
    P.out.m = static_cast<uint32_t>(G.rows);
    P.out.n = static_cast<uint32_t>(G.cols);
    P.out.alpha = last.alpha / kStore / kStore;
    P.tall = G.rows > G.cols;
    P.m = static_cast<uint32_t>(P.tall ? G.cols : G.rows);
    P.n = static_cast<uint32_t>(P.tall ? G.rows : G.cols);
    P.steps = ns.steps;
    P.a = static_cast<float>(ns.a);
    P.b = static_cast<float>(ns.b);
    P.c = static_cast<float>(ns.c);
    uint32_t ctas = 1;
    while (ctas * kSkinnyCols < P.n) ctas *= 2;
    P.share = (P.n + 64 * ctas - 1) / (64 * ctas) * 64;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(G.batch * ctas, 1, 1);
    cfg.blockDim = dim3(kSkinnyThreads, 1, 1);
    cfg.dynamicSmemBytes = kSkinnySmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const uint64_t limit = kWaitLimitNs;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, skinny_kernel<MUON>, P, limit);
    if (e != cudaSuccess) return cuda_fail(e);
    return launched(ASR_KERNEL_PRODUCT);
}

// The products of a group.  `last` holds the fields of the last product's
// epilogue (kOut or kParam), whose alpha is per unit of the result.
template <int LAST>
asr_status iterate(const Group &G, const NsParams &ns, const Layout &L, char *ws, const prod::Params &last,
                   cudaStream_t stream)
{
    using prod::Stored;
    const bool tall = G.rows > G.cols;
    const uint64_t xs = up(G.rows * L.ldx * 2, 256) / 2, ss = up(L.m * L.lds * 2, 256) / 2;
    Stored x{reinterpret_cast<__half *>(ws + L.x0), G.rows, G.cols, L.ldx, xs};
    Stored y{reinterpret_cast<__half *>(ws + L.x1), G.rows, G.cols, L.ldx, xs};
    const Stored S{reinterpret_cast<__half *>(ws + L.s), L.m, L.m, L.lds, ss};
    const Stored Q{reinterpret_cast<__half *>(ws + L.p), L.m, L.m, L.lds, ss};
    const float down = 1.0f / kStore;               // a product of two stored matrices, stored
    asr_status st = ASR_OK;
    for (uint32_t i = 0; st == ASR_OK && i < ns.steps; ++i) {
        prod::Params P = last;
        P.batch = G.batch;
        P.alpha = down;
        P.ld = static_cast<uint32_t>(S.ld);
        P.stride = S.stride;
        P.out = S.ptr;
        P.diag = reinterpret_cast<float *>(ws + L.diag);
        P.gain = reinterpret_cast<float *>(ws + L.gain);
        P.side = static_cast<uint32_t>(L.lds);
        st = tall ? prod::launch<true, true, prod::kGram>(x, x, P, stream)
                  : prod::launch<false, false, prod::kGram>(x, x, P, stream);
        if (st != ASR_OK) break;
        P.alpha = static_cast<float>(ns.c) * down;
        P.beta = static_cast<float>(ns.b);
        P.shift = static_cast<float>(ns.a) * kStore;
        P.aux = S.ptr;
        P.out = Q.ptr;
        st = prod::launch<false, false, prod::kPoly>(S, S, P, stream);
        if (st != ASR_OK) break;
        if (i + 1 < ns.steps) {
            P.alpha = down;
            P.ld = static_cast<uint32_t>(y.ld);
            P.stride = y.stride;
            P.out = y.ptr;
            st = tall ? prod::launch<false, false, prod::kNext>(x, Q, P, stream)
                      : prod::launch<false, true, prod::kNext>(Q, x, P, stream);
            std::swap(x, y);
        } else {
            P.alpha = last.alpha * down * down;
            P.beta = last.beta;
            st = tall ? prod::launch<false, false, LAST>(x, Q, P, stream)
                      : prod::launch<false, true, LAST>(Q, x, P, stream);
        }
    }
    return st;
}

bool ns_ok(const NsParams &ns)
{
    return ns.steps >= 1 && ns.steps <= 100 && finite_nonneg(ns.eps) && ns.eps >= 1e-30 && ns.eps <= 1e30 &&
           coefficients_fit(ns.a, ns.b, ns.c, ns.steps);
}

constexpr uint64_t kMaxSide = 1u << 20;

bool shape_ok(uint64_t count, uint64_t rows, uint64_t cols)
{
    return rows <= kMaxSide && cols <= kMaxSide && count <= (1u << 24);
}

// Whether 8-element units (16 or 32 bytes) start on 16-byte boundaries.
bool units_aligned(const void *p, uint64_t ld, uint64_t stride)
{
    return aligned16(p) && ld % 8 == 0 && stride % 8 == 0;
}

bool aligned32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

bool element_aligned(const void *p, int32_t dtype)
{
    return (reinterpret_cast<uintptr_t>(p) & (dtype == ASR_BF16 ? 1u : 3u)) == 0;
}

// Every matrix of a table, in table order, in stacks of one shape and type
// that follow one another: F(group) for each full or last stack.
struct Flat {
    uint64_t rows, cols, src_ld, out_ld;
    int32_t src_dtype, out_dtype;
    bool vec_in, vec_out;
    Matrix m;
    prod::Slot out;
    bool same(const Flat &o) const
    {
        return rows == o.rows && cols == o.cols && src_ld == o.src_ld && out_ld == o.out_ld &&
               src_dtype == o.src_dtype && out_dtype == o.out_dtype && vec_in == o.vec_in && vec_out == o.vec_out;
    }
};

template <typename F>
asr_status for_groups(std::vector<Flat> &flat, F f)
{
    // a stable grouping: matrices of one kind together, kinds in order of first appearance
    std::vector<uint32_t> kind(flat.size());
    std::vector<uint32_t> first;
    for (size_t i = 0; i < flat.size(); ++i) {
        uint32_t k = 0;
        while (k < first.size() && !flat[first[k]].same(flat[i])) ++k;
        if (k == first.size()) first.push_back(static_cast<uint32_t>(i));
        kind[i] = k;
    }
    std::unique_ptr<Group> G(new Group);
    for (uint32_t k = 0; k < first.size(); ++k) {
        const Flat &T = flat[first[k]];
        G->rows = T.rows;
        G->cols = T.cols;
        G->src_ld = T.src_ld;
        G->out_ld = T.out_ld;
        G->src_dtype = static_cast<uint32_t>(T.src_dtype);
        G->out_dtype = static_cast<uint32_t>(T.out_dtype);
        G->vec_in = T.vec_in;
        G->vec_out = T.vec_out;
        G->batch = 0;
        const uint32_t limit = batch_limit(T.rows, T.cols);
        for (size_t i = first[k]; i < flat.size(); ++i) {
            if (kind[i] != k) continue;
            G->m[G->batch] = flat[i].m;
            G->out[G->batch] = flat[i].out;
            if (++G->batch == limit) {
                const asr_status st = f(*G);
                if (st != ASR_OK) return st;
                G->batch = 0;
            }
        }
        if (G->batch) {
            const asr_status st = f(*G);
            if (st != ASR_OK) return st;
        }
    }
    return ASR_OK;
}

const void *element(const void *p, int32_t dtype, uint64_t at)
{
    return static_cast<const char *>(p) + at * (dtype == ASR_BF16 ? 2 : 4);
}

asr_status flatten(const asr_matrix_desc *table, int32_t n, std::vector<Flat> &flat)
{
    if (n < 0 || (n > 0 && !table)) return ASR_ERR_INVALID_VALUE;
    for (int32_t i = 0; i < n; ++i) {
        const asr_matrix_desc &d = table[i];
        if (d.x_dtype != ASR_F32 && d.x_dtype != ASR_BF16) return ASR_ERR_UNSUPPORTED_DTYPE;
        if (d.count == 0 || d.rows == 0 || d.cols == 0) continue;
        if (!shape_ok(d.count, d.rows, d.cols) || d.x_ld < d.cols || d.out_ld < d.cols || d.x_ld > (1ull << 32) ||
            d.out_ld > (1ull << 32) || d.x_stride > (1ull << 48) || d.out_stride > (1ull << 48))
            return ASR_ERR_INVALID_VALUE;
        if (!d.x || !d.out || !element_aligned(d.x, d.x_dtype) || !element_aligned(d.out, ASR_BF16))
            return ASR_ERR_INVALID_VALUE;
        if (flat.size() + d.count > (1u << 24)) return ASR_ERR_INVALID_VALUE;
        Flat f;
        f.rows = d.rows;
        f.cols = d.cols;
        f.src_ld = d.x_ld;
        f.out_ld = d.out_ld;
        f.src_dtype = d.x_dtype;
        f.out_dtype = ASR_BF16;
        for (uint64_t z = 0; z < d.count; ++z) {
            f.m.src = element(d.x, d.x_dtype, z * d.x_stride);
            f.m.momentum = nullptr;
            f.out.ptr = d.out + z * d.out_stride;
            f.out.base = 0;
            f.vec_in = units_aligned(f.m.src, d.x_ld, 0);
            f.vec_out = aligned32(f.out.ptr) && d.out_ld % 16 == 0;
            flat.push_back(f);
        }
    }
    return ASR_OK;
}

asr_status flatten(const asr_muon_desc *table, int32_t n, std::vector<Flat> &flat)
{
    if (n < 0 || (n > 0 && !table)) return ASR_ERR_INVALID_VALUE;
    for (int32_t i = 0; i < n; ++i) {
        const asr_muon_desc &d = table[i];
        if (d.param_dtype != ASR_F32 && d.param_dtype != ASR_BF16) return ASR_ERR_UNSUPPORTED_DTYPE;
        if (d.grad_dtype != ASR_F32 && d.grad_dtype != ASR_BF16) return ASR_ERR_UNSUPPORTED_DTYPE;
        if (d.count == 0 || d.rows == 0 || d.cols == 0) continue;
        if (!shape_ok(d.count, d.rows, d.cols)) return ASR_ERR_INVALID_VALUE;
        const uint64_t size = d.rows * d.cols;
        if (!d.param || !d.grad || !d.momentum || !element_aligned(d.param, d.param_dtype) ||
            !element_aligned(d.grad, d.grad_dtype) || !element_aligned(d.momentum, ASR_F32))
            return ASR_ERR_INVALID_VALUE;
        if (d.base_index > UINT64_MAX - size * d.count) return ASR_ERR_INVALID_VALUE;
        if (flat.size() + d.count > (1u << 24)) return ASR_ERR_INVALID_VALUE;
        Flat f;
        f.rows = d.rows;
        f.cols = d.cols;
        f.src_ld = f.out_ld = d.cols;
        f.src_dtype = d.grad_dtype;
        f.out_dtype = d.param_dtype;
        for (uint64_t z = 0; z < d.count; ++z) {
            f.m.src = element(d.grad, d.grad_dtype, z * size);
            f.m.momentum = d.momentum + z * size;
            f.out.ptr = const_cast<void *>(element(d.param, d.param_dtype, z * size));
            f.out.base = d.base_index + z * size;
            f.vec_in = units_aligned(f.m.src, d.cols, 0) && aligned16(f.m.momentum);
            f.vec_out = aligned32(f.out.ptr) && d.cols % 16 == 0;
            flat.push_back(f);
        }
    }
    return ASR_OK;
}

uint64_t workspace(std::vector<Flat> &flat)
{
    uint64_t most = 0;
    for_groups(flat, [&](const Group &G) {
        const uint64_t b = layout(G.rows, G.cols, G.batch).bytes;
        if (b > most) most = b;
        return ASR_OK;
    });
    return most;
}

template <typename D>
asr_status workspace_of(const D *table, int32_t n, uint64_t *bytes)
{
    if (!bytes) return ASR_ERR_INVALID_VALUE;
    std::vector<Flat> flat;
    const asr_status st = flatten(table, n, flat);
    if (st == ASR_OK) *bytes = workspace(flat);
    return st;
}

prod::Params last_params(const Group &G)
{
    prod::Params P;
    std::memset(&P, 0, sizeof(P));
    P.out_ld = G.out_ld;
    P.out_dtype = G.out_dtype;
    P.rounding = ASR_ROUND_RNE;
    P.vec = G.vec_out;
    std::memcpy(P.slot, G.out, sizeof(prod::Slot) * G.batch);
    return P;
}

asr_status newton_schulz(const asr_matrix_desc *table, int32_t n, const asr_ns_params *p, void *ws, uint64_t ws_bytes,
                         cudaStream_t stream)
{
    if (!p) return ASR_ERR_INVALID_VALUE;
    const NsParams ns{p->a, p->b, p->c, p->eps, p->steps};
    if (!ns_ok(ns)) return ASR_ERR_INVALID_VALUE;
    std::vector<Flat> flat;
    asr_status st = flatten(table, n, flat);
    if (st != ASR_OK || flat.empty()) return st;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < workspace(flat)) return ASR_ERR_INVALID_VALUE;
    st = setup();
    if (st != ASR_OK) return st;
    return for_groups(flat, [&](const Group &G) {
        const Layout L = layout(G.rows, G.cols, G.batch);
        char *w = static_cast<char *>(ws);
        prod::Params last = last_params(G);
        last.alpha = 1.0f;
        if (skinny_fits(G.rows, G.cols)) return skinny<false>(G, ns, last, 0.0f, false, stream);
        asr_status s = prep<false>(G, ns, L, w, 0.0f, false, stream);
        if (s != ASR_OK) return s;
        return iterate<prod::kOut>(G, ns, L, w, last, stream);
    });
}

asr_status check_hparams(const asr_muon_hparams *hp)
{
    if (!hp) return ASR_ERR_INVALID_VALUE;
    if (hp->rounding != ASR_ROUND_SR && hp->rounding != ASR_ROUND_RNE) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (hp->step == 0 || hp->adjust > ASR_MUON_ADJUST_RMS || hp->nesterov > 1) return ASR_ERR_INVALID_VALUE;
    if (!finite_nonneg(hp->lr) || !finite_nonneg(hp->weight_decay)) return ASR_ERR_INVALID_VALUE;
    if (!(hp->momentum >= 0.0 && hp->momentum < 1.0)) return ASR_ERR_INVALID_VALUE;
    const NsParams ns{hp->ns.a, hp->ns.b, hp->ns.c, hp->ns.eps, hp->ns.steps};
    return ns_ok(ns) ? ASR_OK : ASR_ERR_INVALID_VALUE;
}

asr_status step(const asr_muon_desc *table, int32_t n, const asr_muon_hparams *hp, void *ws, uint64_t ws_bytes,
                cudaStream_t stream)
{
    asr_status st = check_hparams(hp);
    if (st != ASR_OK) return st;
    const NsParams ns{hp->ns.a, hp->ns.b, hp->ns.c, hp->ns.eps, hp->ns.steps};
    std::vector<Flat> flat;
    st = flatten(table, n, flat);
    if (st != ASR_OK || flat.empty()) return st;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < workspace(flat)) return ASR_ERR_INVALID_VALUE;
    st = setup();
    if (st != ASR_OK) return st;
    return for_groups(flat, [&](const Group &G) {
        const Layout L = layout(G.rows, G.cols, G.batch);
        char *w = static_cast<char *>(ws);
        const double r = static_cast<double>(G.rows), c = static_cast<double>(G.cols);
        const double adjust = hp->adjust == ASR_MUON_ADJUST_RMS ? 0.2 * std::sqrt(std::max(r, c))
                              : hp->adjust == ASR_MUON_ADJUST_SPECTRAL ? std::sqrt(std::max(1.0, r / c)) : 1.0;
        prod::Params last = last_params(G);
        last.alpha = static_cast<float>(hp->lr * adjust);
        last.beta = static_cast<float>(1.0 - hp->lr * hp->weight_decay);
        last.rounding = hp->rounding;
        last.step = hp->step;
        last.keys = make_keys(hp->seed);
        if (skinny_fits(G.rows, G.cols))
            return skinny<true>(G, ns, last, static_cast<float>(hp->momentum), hp->nesterov != 0, stream);
        asr_status s = prep<true>(G, ns, L, w, static_cast<float>(hp->momentum), hp->nesterov != 0, stream);
        if (s != ASR_OK) return s;
        return iterate<prod::kParam>(G, ns, L, w, last, stream);
    });
}

}  // namespace muon
