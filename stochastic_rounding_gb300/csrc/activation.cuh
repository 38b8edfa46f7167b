// activation.cuh -- a layer's activation and its backward pass, the input kept as
// it is or in 8 bits (checkpoint.cuh) between them.  Included into asr.cu (inside
// its anonymous namespace), after checkpoint.cuh.
//
//   f(a) = a s(u),  s(u) = 1 / (1 + e^-u):   u = a                          (silu)
//                                            u = sqrt(8/pi) (a + 0.044715 a^3)  (gelu, its tanh form)
//   f'(a) = s(u) (1 + a u' s(-u))
//   y = f(a), or gated, x = [a | b]:  y = f(a) b,  da = dy f'(a) b,  db = dy f(a)
//
// s from t = e^-|u|, as 1 / (1 + t) or t / (1 + t): no cancellation on either side,
// and no overflow.  bf16 results take the hardware's exponential and division,
// whose error (below 2^-16 where e^-|u| is a normal number) their rounding hides;
// f32 results take the library's.
//
// Bound by bytes: an element of x and y each once, the kept form on the way.

namespace act {

using kept::Codes;
using kept::live_of;
constexpr int kThreads = kept::kThreads;

struct Params {
    kept::Matrix x, dy;
    kept::Out y, dx;
    uint64_t rows, cols;                        // of y
    uint32_t gelu;
    kept::Store to;                             // forward
    kept::Source from;                          // backward
};

constexpr float kSlope = 1.5957691216057308f;   // sqrt(8 / pi)
constexpr float kCube = 0.044715f;

struct Sigmoid {
    float plus, minus;                          // s(u), s(-u)
};

template <int DT>
__device__ __forceinline__ Sigmoid sigmoid(float u)
{
    float t, big, small;
    if (DT == ASR_BF16) {
        t = __expf(-fabsf(u));
        big = __fdividef(1.0f, __fadd_rn(1.0f, t));
        small = __fmul_rn(t, big);
    } else {
        t = expf(-fabsf(u));
        big = __fdiv_rn(1.0f, __fadd_rn(1.0f, t));
        small = __fdiv_rn(t, __fadd_rn(1.0f, t));
    }
    return u >= 0.0f ? Sigmoid{big, small} : u < 0.0f ? Sigmoid{small, big} : Sigmoid{u + big, u + big};
}

__device__ __forceinline__ float argument(float a, bool gelu)
{
    return gelu ? __fmul_rn(kSlope, __fmaf_rn(__fmul_rn(__fmul_rn(a, a), a), kCube, a)) : a;
}

// f(a), and f'(a).  Where s(-u) is zero, so is what it multiplies, whatever the size.
template <int DT>
__device__ __forceinline__ float value(float a, bool gelu)
{
    return __fmul_rn(a, sigmoid<DT>(argument(a, gelu)).plus);
}

template <int DT>
__device__ __forceinline__ void value_and_slope(float a, bool gelu, float &f, float &df)
{
    const Sigmoid s = sigmoid<DT>(argument(a, gelu));
    float r = a;                                // a u'
    if (gelu) r = __fmul_rn(__fmul_rn(a, kSlope), __fmaf_rn(__fmul_rn(a, a), 3.0f * kCube, 1.0f));
    f = __fmul_rn(a, s.plus);
    df = s.minus == 0.0f ? s.plus : __fmul_rn(s.plus, __fmaf_rn(r, s.minus, 1.0f));
}

// KEEP: 0 nothing, 1 to nearest, 2 stochastically.  A warp a span of 256 columns
// of y, gated, or 512, two units of eight values of x a lane either way.
template <int DT, bool GATED, int KEEP>
__global__ void __launch_bounds__(kThreads) forward_kernel(const __grid_constant__ Params P)
{
    constexpr int kUnits = GATED ? 1 : 2;
    const uint32_t lane = threadIdx.x & 31;
    const bool gelu = P.gelu;
    muon::Walk k(P.rows, (P.cols + kUnits - 1) / kUnits, blockIdx.x * 8ull + (threadIdx.x >> 5), gridDim.x * 8ull);
    for (; k.more(); k.next()) {
        float x[2][8];
        uint64_t col[2];                        // of x
        int live[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint64_t c = k.span * (256ull * kUnits) + (GATED ? 0 : u * 256) + lane * 8;
            live[u] = live_of(P.cols, c);
            col[u] = GATED && u ? P.cols + c : c;
            muon::load8(P.x.p, DT, k.row * P.x.ld + col[u], live[u], P.x.vec && (!GATED || !u || P.cols % 8 == 0), x[u]);
        }
        float y[2][8];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[u][i] = value<DT>(x[u][i], gelu);
                if (GATED) y[u][i] = __fmul_rn(y[u][i], x[1][i]);
            }
            kept::store8<DT>(P.y.p, k.row * P.y.ld + col[u], live[u], P.y.vec, y[u]);
        }
        if (KEEP) {
#pragma unroll
            for (int u = 0; u < 2; ++u) kept::keep8<KEEP == 2>(P.to, k.row, col[u], live[u], x[u]);
        }
    }
}

// KEPT: 0 from x, 1 from its codes, 2 from codes whose groups do not begin anew with
// the gating half (cols not a multiple of 32).
template <int DT, bool GATED, int KEPT>
__global__ void __launch_bounds__(kThreads) backward_kernel(const __grid_constant__ Params P)
{
    constexpr int kUnits = GATED ? 1 : 2;
    const uint32_t lane = threadIdx.x & 31;
    const bool gelu = P.gelu;
    muon::Walk k(P.rows, (P.cols + kUnits - 1) / kUnits, blockIdx.x * 8ull + (threadIdx.x >> 5), gridDim.x * 8ull);
    for (; k.more(); k.next()) {
        float x[2][8], g[kUnits][8];
        Codes c[2];
        uint64_t col[2];
        int live[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint64_t at = k.span * (256ull * kUnits) + (GATED ? 0 : u * 256) + lane * 8;
            live[u] = live_of(P.cols, at);
            col[u] = GATED && u ? P.cols + at : at;
            if (KEPT == 2 && u == 1) kept::values_across(P.from, k.row, col[u], live[u], x[u]);
            else if (KEPT) c[u] = kept::fetch8(P.from, k.row, col[u], live[u]);
            else muon::load8(P.x.p, DT, k.row * P.x.ld + col[u], live[u], P.x.vec && (!GATED || !u || P.cols % 8 == 0), x[u]);
            if (u < kUnits) muon::load8(P.dy.p, DT, k.row * P.dy.ld + col[u], live[u], P.dy.vec, g[u]);
        }
        if (KEPT) {
#pragma unroll
            for (int u = 0; u < (KEPT == 2 ? 1 : 2); ++u) kept::values8(c[u], x[u]);
        }
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            float da[8], db[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float f, df;
                value_and_slope<DT>(x[u][i], gelu, f, df);
                da[i] = __fmul_rn(g[u][i], df);
                if (GATED) {
                    da[i] = __fmul_rn(da[i], x[1][i]);
                    db[i] = __fmul_rn(g[u][i], f);
                }
            }
            kept::store8<DT>(P.dx.p, k.row * P.dx.ld + col[u], live[u], P.dx.vec, da);
            if (GATED) kept::store8<DT>(P.dx.p, k.row * P.dx.ld + col[1], live[1], P.dx.vec && P.cols % 8 == 0, db);
        }
    }
}

// ------------------------------------------------------------------ host

using Kernel = void (*)(const Params);

template <int DT, bool GATED>
Kernel forward_of(int keep)
{
    return keep == 2 ? forward_kernel<DT, GATED, 2> : keep ? forward_kernel<DT, GATED, 1> : forward_kernel<DT, GATED, 0>;
}

Kernel forward_of(int32_t dtype, bool gated, int keep)
{
    if (dtype == ASR_BF16) return gated ? forward_of<ASR_BF16, true>(keep) : forward_of<ASR_BF16, false>(keep);
    return gated ? forward_of<ASR_F32, true>(keep) : forward_of<ASR_F32, false>(keep);
}

template <int DT>
Kernel backward_of(bool gated, int codes)
{
    if (gated)
        return codes == 2 ? backward_kernel<DT, true, 2> : codes ? backward_kernel<DT, true, 1> : backward_kernel<DT, true, 0>;
    return codes ? backward_kernel<DT, false, 1> : backward_kernel<DT, false, 0>;
}

Kernel backward_of(int32_t dtype, bool gated, int codes)
{
    return dtype == ASR_BF16 ? backward_of<ASR_BF16>(gated, codes) : backward_of<ASR_F32>(gated, codes);
}

asr_status setup()
{
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (e == cudaSuccess && (ready.load(std::memory_order_acquire) & bit)) return ASR_OK;
    for (int32_t dtype : {ASR_F32, ASR_BF16})
        for (int gated = 0; gated < 2; ++gated) {
            for (int keep = 0; keep < 3; ++keep)
                if (e == cudaSuccess) e = prod::load_kernel(forward_of(dtype, gated != 0, keep));
            for (int codes = 0; codes < 3; ++codes)
                if (e == cudaSuccess) e = prod::load_kernel(backward_of(dtype, gated != 0, codes));
        }
    if (e != cudaSuccess) return cuda_fail(e);
    ready.fetch_or(bit, std::memory_order_release);
    return ASR_OK;
}

asr_status kind_ok(int32_t dtype, uint32_t function)
{
    return kept::dtype_ok(dtype) && (function == ASR_SILU || function == ASR_GELU) ? ASR_OK : ASR_ERR_UNSUPPORTED_DTYPE;
}

unsigned blocks(uint64_t rows, uint64_t cols, bool gated)
{
    const uint64_t span = gated ? 256 : 512;
    return int8::blocks_for(rows * ((cols + span - 1) / span), 8, 1u << 20);
}

asr_status forward(const void *x, uint64_t x_ld, void *y, uint64_t y_ld, int32_t dtype, uint64_t rows, uint64_t cols,
                   uint32_t function, uint32_t gated, const asr_checkpoint *to, cudaStream_t stream)
{
    asr_status st = kind_ok(dtype, function);
    if (st == ASR_OK && to && to->rounding != ASR_ROUND_SR && to->rounding != ASR_ROUND_RNE) st = ASR_ERR_UNSUPPORTED_DTYPE;
    if (st == ASR_OK && gated > 1) st = ASR_ERR_INVALID_VALUE;
    if (st != ASR_OK || rows == 0 || cols == 0) return st;
    const uint64_t width = gated ? 2 * cols : cols;
    if (!kept::sizes_ok(rows, cols) || !kept::matrix_ok(x, dtype, x_ld, width) || !kept::matrix_ok(y, dtype, y_ld, cols))
        return ASR_ERR_INVALID_VALUE;
    if (to) st = kept::writable(*to, rows, width);
    if (st == ASR_OK) st = setup();
    if (st == ASR_OK && to) st = kept::setup();
    if (st != ASR_OK) return st;
    Params P;
    std::memset(&P, 0, sizeof(P));
    P.x = kept::matrix(x, x_ld);
    P.y = kept::out(y, y_ld);
    P.rows = rows;
    P.cols = cols;
    P.gelu = function == ASR_GELU;
    // the kernel's lanes hold whole groups of both halves where they begin with the halves
    const bool apart = to && gated && cols % kept::kGroup != 0;
    int keep = 0;
    if (to && !apart) {
        P.to = kept::store(*to, width);
        keep = to->rounding == ASR_ROUND_SR ? 2 : 1;
    }
    forward_of(dtype, gated != 0, keep)<<<blocks(rows, cols, gated != 0), kThreads, 0, stream>>>(P);
    st = launched(ASR_KERNEL_ACTIVATION);
    if (st == ASR_OK && apart) st = kept::pack(x, dtype, rows, width, x_ld, to, stream);
    return st;
}

asr_status backward(const void *dy, uint64_t dy_ld, const void *x, uint64_t x_ld, const asr_checkpoint *from, void *dx,
                    uint64_t dx_ld, int32_t dtype, uint64_t rows, uint64_t cols, uint32_t function, uint32_t gated,
                    cudaStream_t stream)
{
    asr_status st = kind_ok(dtype, function);
    if (st == ASR_OK && (gated > 1 || (x != nullptr && from != nullptr))) st = ASR_ERR_INVALID_VALUE;
    if (st != ASR_OK || rows == 0 || cols == 0) return st;
    const uint64_t width = gated ? 2 * cols : cols;
    if (!kept::sizes_ok(rows, cols) || !kept::matrix_ok(dy, dtype, dy_ld, cols) || !kept::matrix_ok(dx, dtype, dx_ld, width))
        return ASR_ERR_INVALID_VALUE;
    if (from) st = kept::readable(*from, width);
    else if (!kept::matrix_ok(x, dtype, x_ld, width)) st = ASR_ERR_INVALID_VALUE;
    if (st == ASR_OK) st = setup();
    if (st != ASR_OK) return st;
    Params P;
    std::memset(&P, 0, sizeof(P));
    P.dy = kept::matrix(dy, dy_ld);
    P.dx = kept::out(dx, dx_ld);
    if (from) P.from = kept::source(*from);
    else P.x = kept::matrix(x, x_ld);
    P.rows = rows;
    P.cols = cols;
    P.gelu = function == ASR_GELU;
    const int codes = !from ? 0 : gated && cols % kept::kGroup != 0 ? 2 : 1;
    backward_of(dtype, gated != 0, codes)<<<blocks(rows, cols, gated != 0), kThreads, 0, stream>>>(P);
    return launched(ASR_KERNEL_ACTIVATION);
}

}  // namespace act
