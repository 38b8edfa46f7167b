// activation.cuh -- a layer's activation and its backward pass, the input kept as
// it is or in 8 bits (checkpoint.cuh) between them.  Included into asr.cu (inside
// its anonymous namespace), after checkpoint.cuh.
//
//   f(a) = a s(u),  s(u) = 1 / (1 + e^-u):   u = a                          (silu)
//                                            u = sqrt(8/pi) (a + 0.044715 a^3)  (gelu, its tanh form)
//   f'(a) = s(u) (1 + a u' s(-u))
//   y = f(a), or gated, x = [a | b]:  y = f(a) b,  da = dy f'(a) b,  db = dy f(a)
//
// bf16 results take the hardware's exponential and reciprocal, whose errors (a few
// 2^-24, and |u| 2^-24 from the exponent's rounding) are far below their rounding;
// f32 results take the library's.  Below u = -87, where e^-u leaves binary32, s is 0.
//
// Bound by bytes: an element of x and y each once, the kept form on the way (x is read once
// more where a gated half is no whole number of groups); kept stochastically, by
// instructions, 2.5 times as many (issue 62 %, memory 51).  Gated silu of 8,192 x 14,336
// bf16, one launch after another, with the time of its bytes at 6,697 GB/s: 105 us (105),
// codes to nearest 153 (141), stochastic 204 (141), backward 181 (175), from codes 147.5
// (141).

namespace act {

using kept::Codes;
using kept::live_of;
constexpr int kThreads = kept::kThreads;

struct Params {
    kept::Matrix x, dy;
    kept::Out y, dx;
    uint32_t rows, cols;                        // of y
    uint32_t gelu;
    kept::Store to;                             // forward
    kept::Source from;                          // backward
};

constexpr float kSlope = 1.5957691216057308f;   // sqrt(8 / pi)
constexpr float kCube = 0.044715f;
constexpr float kLog2e = 1.4426950408889634f;

// s(u), and s(-u) from e^-u.
template <int DT>
__device__ __forceinline__ float sigmoid(float u, float &minus)
{
    float s;
    if (DT == ASR_BF16) {
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(u, -kLog2e)));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(__fadd_rn(1.0f, e)));
        minus = __fsub_rn(1.0f, s);             // what is lost near u = 25 is added to 1
    } else {
        const float e = expf(-u);
        s = __frcp_rn(__fadd_rn(1.0f, e));
        minus = e <= 3.402823466e38f ? __fmul_rn(e, s) : 1.0f;
    }
    return s;
}

__device__ __forceinline__ float argument(float a, bool gelu)
{
    return gelu ? __fmul_rn(kSlope, __fmaf_rn(__fmul_rn(__fmul_rn(a, a), a), kCube, a)) : a;
}

template <int DT>
__device__ __forceinline__ float value(float a, bool gelu)
{
    float minus;
    return __fmul_rn(a, sigmoid<DT>(argument(a, gelu), minus));
}

template <int DT>
__device__ __forceinline__ void value_and_slope(float a, bool gelu, float &f, float &df)
{
    float minus;
    const float s = sigmoid<DT>(argument(a, gelu), minus);
    f = __fmul_rn(a, s);
    // a u', finite: from |a| = 128 on s s(-u) is 0, as the product is whatever a
    float r = fminf(fmaxf(a, -128.0f), 128.0f);
    if (gelu) r = __fmul_rn(__fmul_rn(r, kSlope), __fmaf_rn(__fmul_rn(r, r), 3.0f * kCube, 1.0f));
    df = __fmaf_rn(__fmul_rn(s, minus), r, s);
}

// How the gating half's rows begin, `cols` values behind the others.
__device__ __forceinline__ uint32_t half_vec(uint32_t vec, uint32_t cols)
{
    return cols % 16 == 0 ? vec : cols % 8 == 0 && vec ? 1 : 0;
}

// KEEP: 0 nothing, 1 to nearest, 2 stochastically.  A span is 512 columns of y; the
// next one's values are fetched before the current one's are worked on.  Registers for
// four blocks an SM, for three where Philox's come on top, for two of f32 with its values
// twice as wide; the gated bf16 ones with codes spill 12 to 60 bytes at that.
template <int DT, bool GATED, int KEEP, bool FULL>
__global__ void __launch_bounds__(kThreads, DT == ASR_F32 ? 2 : GATED && KEEP == 2 ? 3 : 4) forward_kernel(const __grid_constant__ Params P, uint32_t spans)
{
    constexpr int kHalves = GATED ? 2 : 1;      // of x
    __shared__ kept::Stage stages[FULL ? 1 : kThreads / 32];
    kept::Stage &stage = stages[FULL ? 0 : threadIdx.x >> 5];
    const bool gelu = P.gelu;
    const uint32_t vec1 = half_vec(P.x.vec, P.cols), lane = (threadIdx.x & 31) * 16;
    kept::Pair<DT> next[kHalves];
    auto load = [&](const kept::Walk &k) {
        if (!k.more()) return;
        const uint32_t col = k.span * kept::kSpan + lane;
        next[0] = kept::fetch16<DT, FULL>(P.x, k.row, col, P.cols, P.x.vec, stage);
        if (GATED) next[kHalves - 1] = kept::fetch16<DT, FULL>(P.x, k.row, P.cols + col, 2 * P.cols, vec1, stage);
    };
    kept::Walk k(P.rows, spans);
    load(k);
    while (k.more()) {
        kept::Pair<DT> raw[kHalves];
#pragma unroll
        for (int u = 0; u < kHalves; ++u) raw[u] = next[u];
        const uint32_t row = k.row, col = k.span * kept::kSpan + lane;
        const int live = FULL ? 16 : live_of(P.cols, col, 16);
        k.next();
        load(k);
        if (KEEP) {
#pragma unroll
            for (int u = 0; u < kHalves; ++u) kept::keep16<KEEP == 2, DT, FULL>(P.to, row, u * P.cols + col, live, raw[u]);
        }
        float y[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float b[8];
            kept::values(raw[0].h[h], y[h]);
            if (GATED) kept::values(raw[kHalves - 1].h[h], b);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[h][i] = value<DT>(y[h][i], gelu);
                if (GATED) y[h][i] = __fmul_rn(y[h][i], b[i]);
            }
        }
        kept::store16<DT, FULL>(P.y, row, col, P.cols, P.y.vec, y, stage);
    }
}

// KEPT: 0 from x, 1 from its codes, 2 from codes whose groups do not begin anew with
// the gating half (cols not a multiple of 32).
template <int DT, bool GATED, int KEPT, bool FULL>
__global__ void __launch_bounds__(kThreads) backward_kernel(const __grid_constant__ Params P, uint32_t spans)
{
    constexpr int kHalves = GATED ? 2 : 1;
    __shared__ kept::Stage stages[FULL ? 1 : kThreads / 32];
    kept::Stage &stage = stages[FULL ? 0 : threadIdx.x >> 5];
    const bool gelu = P.gelu;
    const uint32_t in1 = half_vec(P.x.vec, P.cols), out1 = half_vec(P.dx.vec, P.cols), lane = (threadIdx.x & 31) * 16;
    kept::Pair<DT> raw[kHalves], grad;
    kept::Codes16 codes[kHalves];
    kept::CodesAcross across;
    auto load = [&](const kept::Walk &k) {
        if (!k.more()) return;
        const uint32_t col = k.span * kept::kSpan + lane;
        const int live = FULL ? 16 : live_of(P.cols, col, 16);
#pragma unroll
        for (int u = 0; u < kHalves; ++u) {
            if (!KEPT) raw[u] = kept::fetch16<DT, FULL>(P.x, k.row, u * P.cols + col, (u + 1) * P.cols, u ? in1 : P.x.vec, stage);
            else if (KEPT == 1 || u == 0) codes[u] = kept::fetch_codes16<FULL>(P.from, k.row, u * P.cols + col, live);
            else across = kept::fetch_across(P.from, k.row, P.cols + col, 2 * P.cols, stage);
        }
        grad = kept::fetch16<DT, FULL>(P.dy, k.row, col, P.cols, P.dy.vec, stage);
    };
    kept::Walk k(P.rows, spans);
    load(k);
    while (k.more()) {
        const uint32_t row = k.row, col = k.span * kept::kSpan + lane;
        kept::Pair<DT> x0[kHalves], g0 = grad;
        kept::Codes16 c0[kHalves];
        const kept::CodesAcross across0 = across;
#pragma unroll
        for (int u = 0; u < kHalves; ++u) {
            if (!KEPT) x0[u] = raw[u];
            else c0[u] = codes[u];
        }
        k.next();
        load(k);
        float da[2][8], db[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x[2][8];
            kept::values(g0.h[h], da[h]);
#pragma unroll
            for (int u = 0; u < kHalves; ++u) {
                if (!KEPT) kept::values(x0[u].h[h], x[u]);
                else if (KEPT == 1 || u == 0) kept::values(Codes{c0[u].h[h], c0[u].b}, x[u]);
                else kept::values(across0, h, x[u]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float f, df;
                value_and_slope<DT>(x[0][i], gelu, f, df);
                if (GATED) {
                    db[h][i] = __fmul_rn(da[h][i], f);
                    df = __fmul_rn(df, x[1][i]);
                }
                da[h][i] = __fmul_rn(da[h][i], df);
            }
        }
        kept::store16<DT, FULL>(P.dx, row, col, P.cols, P.dx.vec, da, stage);
        if (GATED) kept::store16<DT, FULL>(P.dx, row, P.cols + col, 2 * P.cols, out1, db, stage);
    }
}

// Rows off alignment, nothing kept.
template <int DT, bool GATED>
__global__ void __launch_bounds__(kThreads) forward_loose_kernel(const __grid_constant__ Params P, uint32_t spans)
{
    const bool gelu = P.gelu;
    for (kept::Walk k(P.rows, spans); k.more(); k.next()) {
        const uint32_t first = k.span * kept::kSpan;
        float a[kept::kLoose], b[kept::kLoose];
        kept::fetch_loose<DT>(P.x, k.row, first, P.cols, a);
        if (GATED) kept::fetch_loose<DT>(P.x, k.row, P.cols + first, 2 * P.cols, b);
#pragma unroll
        for (int i = 0; i < kept::kLoose; ++i) {
            a[i] = value<DT>(a[i], gelu);
            if (GATED) a[i] = __fmul_rn(a[i], b[i]);
            kept::store_loose1<DT>(P.y, k.row, first, P.cols, i, a[i]);
        }
    }
}

template <int DT, bool GATED>
__global__ void __launch_bounds__(kThreads) backward_loose_kernel(const __grid_constant__ Params P, uint32_t spans)
{
    const bool gelu = P.gelu;
    for (kept::Walk k(P.rows, spans); k.more(); k.next()) {
        const uint32_t first = k.span * kept::kSpan;
        float a[kept::kLoose], b[kept::kLoose], g[kept::kLoose];
        kept::fetch_loose<DT>(P.dy, k.row, first, P.cols, g);
        kept::fetch_loose<DT>(P.x, k.row, first, P.cols, a);
        if (GATED) kept::fetch_loose<DT>(P.x, k.row, P.cols + first, 2 * P.cols, b);
#pragma unroll
        for (int i = 0; i < kept::kLoose; ++i) {
            float f, df;
            value_and_slope<DT>(a[i], gelu, f, df);
            if (GATED) df = __fmul_rn(df, b[i]);
            kept::store_loose1<DT>(P.dx, k.row, first, P.cols, i, __fmul_rn(g[i], df));
            if (GATED) kept::store_loose1<DT>(P.dx, k.row, P.cols + first, 2 * P.cols, i, __fmul_rn(g[i], f));
        }
    }
}

// ------------------------------------------------------------------ host

using Kernel = void (*)(const Params, uint32_t);

template <int DT, bool GATED, bool FULL>
Kernel forward_of(int keep)
{
    return keep == 2 ? forward_kernel<DT, GATED, 2, FULL> : keep ? forward_kernel<DT, GATED, 1, FULL>
                                                                 : forward_kernel<DT, GATED, 0, FULL>;
}

enum { kGeneral = 0, kFull = 1, kOff = 2 };     // how rows lie: whole and aligned, or off alignment

Kernel forward_of(int32_t dtype, bool gated, int keep, int how)
{
    if (how == kOff && !keep) {
        if (dtype == ASR_BF16) return gated ? forward_loose_kernel<ASR_BF16, true> : forward_loose_kernel<ASR_BF16, false>;
        return gated ? forward_loose_kernel<ASR_F32, true> : forward_loose_kernel<ASR_F32, false>;
    }
    if (dtype != ASR_BF16) return gated ? forward_of<ASR_F32, true, false>(keep) : forward_of<ASR_F32, false, false>(keep);
    if (how == kFull) return gated ? forward_of<ASR_BF16, true, true>(keep) : forward_of<ASR_BF16, false, true>(keep);
    return gated ? forward_of<ASR_BF16, true, false>(keep) : forward_of<ASR_BF16, false, false>(keep);
}

template <int DT, bool FULL>
Kernel backward_of(bool gated, int codes)
{
    if (!gated) return codes ? backward_kernel<DT, false, 1, FULL> : backward_kernel<DT, false, 0, FULL>;
    if (codes == 2) return backward_kernel<DT, true, 2, false>;
    return codes ? backward_kernel<DT, true, 1, FULL> : backward_kernel<DT, true, 0, FULL>;
}

Kernel backward_of(int32_t dtype, bool gated, int codes, int how)
{
    if (how == kOff && !codes) {
        if (dtype == ASR_BF16) return gated ? backward_loose_kernel<ASR_BF16, true> : backward_loose_kernel<ASR_BF16, false>;
        return gated ? backward_loose_kernel<ASR_F32, true> : backward_loose_kernel<ASR_F32, false>;
    }
    if (dtype != ASR_BF16) return backward_of<ASR_F32, false>(gated, codes);
    return how == kFull ? backward_of<ASR_BF16, true>(gated, codes) : backward_of<ASR_BF16, false>(gated, codes);
}

asr_status setup()
{
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (e == cudaSuccess && (ready.load(std::memory_order_acquire) & bit)) return ASR_OK;
    for (int32_t dtype : {ASR_F32, ASR_BF16})
        for (int how : {kGeneral, kFull, kOff})
            for (int gated = 0; gated < 2; ++gated)
                for (int form = 0; form < 3; ++form) {
                    if (e == cudaSuccess) e = prod::load_kernel(forward_of(dtype, gated != 0, form, how));
                    if (e == cudaSuccess) e = prod::load_kernel(backward_of(dtype, gated != 0, form, how));
                }
    if (e != cudaSuccess) return cuda_fail(e);
    ready.fetch_or(bit, std::memory_order_release);
    return ASR_OK;
}

asr_status kind_ok(int32_t dtype, uint32_t function)
{
    return kept::dtype_ok(dtype) && (function == ASR_SILU || function == ASR_GELU) ? ASR_OK : ASR_ERR_UNSUPPORTED_DTYPE;
}

// Blocks an SM at most (kept::walk), of bf16 where rows are whole spans; us of 8,192 rows,
// capped and as many as fit (four):
//                                 4,096          8,192          14,336         28,672 (4,096 rows)
//   gated, 3                      33.3 / 33.2    61.8 / 63.5    104.9 / 111.4  105.0 / 111.4
//   gated, codes to nearest, 2    47.6 / 51.0    89.9 / 98.7    152.6 / 170.1  152.1 / 169.7
//   not gated, codes to nearest, 3  30.7 / 30.0  55.6 / 61.6    94.0 / 105.3   94.0 / 105.4
// (1,024 x 14,336, 0.1 to 2 us the other way).  Rows that end inside a span leave lanes
// idle, for which more warps make up: 16,384 x 2,752 57.8 / 45.1, 90.1 / 70.8 and 56.0 /
// 42.8, 8,192 x 6,912 55.4 / 54.1, 102.4 / 82.1 and 51.2 / 47.8, 8,192 x 11,008 83.9 / 85.0,
// 156.8 / 127.3 and 77.0 / 77.8.  Kept stochastically, or not gated and not kept, as many
// as fit.
int forward_limit(int32_t dtype, bool gated, int keep, int how)
{
    if (dtype != ASR_BF16 || how != kFull || keep == 2 || (!gated && !keep)) return 32;
    return gated && keep ? 2 : 3;
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
    P.x = kept::matrix(x, x_ld, dtype);
    P.y = kept::out(y, y_ld, dtype);
    P.rows = static_cast<uint32_t>(rows);
    P.cols = static_cast<uint32_t>(cols);
    P.gelu = function == ASR_GELU;
    // the kernel's lanes hold whole groups of both halves where they begin with the halves
    const bool apart = to && gated && cols % kept::kGroup != 0;
    int keep = 0;
    if (to && !apart) {
        P.to = kept::store(*to, width);
        keep = to->rounding == ASR_ROUND_SR ? 2 : 1;
    }
    const bool full = cols % kept::kSpan == 0 && P.x.vec == 2 && P.y.vec == 2 && (!keep || P.to.vec == 2);
    const bool off = !P.x.vec || !P.y.vec || (gated && cols % 8 != 0);
    const int how = full ? kFull : off ? kOff : kGeneral;
    st = kept::walk(ASR_KERNEL_ACTIVATION, forward_of(dtype, gated != 0, keep, how), P, rows, cols, kept::kSpan, stream,
                    forward_limit(dtype, gated != 0, keep, how));
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
    P.dy = kept::matrix(dy, dy_ld, dtype);
    P.dx = kept::out(dx, dx_ld, dtype);
    if (from) P.from = kept::source(*from);
    else P.x = kept::matrix(x, x_ld, dtype);
    P.rows = static_cast<uint32_t>(rows);
    P.cols = static_cast<uint32_t>(cols);
    P.gelu = function == ASR_GELU;
    const int codes = !from ? 0 : gated && cols % kept::kGroup != 0 ? 2 : 1;
    const bool full = cols % kept::kSpan == 0 && P.dy.vec == 2 && P.dx.vec == 2 && (from ? P.from.vec : P.x.vec) == 2;
    const bool off = !P.dy.vec || !P.dx.vec || (!from && !P.x.vec) || (gated && cols % 8 != 0);
    const int how = full ? kFull : off ? kOff : kGeneral;
    // gated from x, bf16, rows that end inside a span: two blocks and three, 8,192 x 11,008 137.5 and 159 us, 8,192 x 6,912
    // 90.2 and 100, 16,384 x 2,752 79.8 and 94.7, 1,024 x 11,008 22.4 and 21.5; of whole rows either gives the same
    const int limit = dtype == ASR_BF16 && gated && !from && how == kGeneral ? 2 : 32;
    return kept::walk(ASR_KERNEL_ACTIVATION, backward_of(dtype, gated != 0, codes, how), P, rows, cols, kept::kSpan, stream, limit);
}

}  // namespace act
