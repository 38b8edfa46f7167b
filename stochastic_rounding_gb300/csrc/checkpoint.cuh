// checkpoint.cuh -- what a layer keeps of its input for the backward pass, in 8
// bits: making it and reading it, as kernels of their own and as what the
// activation's (activation.cuh) and the norm's (norm.cuh) kernels do on the way.
// Included into asr.cu (inside its anonymous namespace), after int8.cuh.
//
//   32 values of a row share a power of two, 2^e, the least (at least 2^-127)
//   with max |x| <= 127 2^e;   y = x 2^-e, exact;
//   q = rint(y)                              (nearest)
//     = floor(y) + [65536 (y - floor(y)) > r]  (stochastic)
//
// A power of two, and not max / 127, because everything about it is then exact --
// y, which neighbour a value goes to, the value that is read back, in bf16 too --
// at one byte for 32 values.  It costs up to a bit where the largest value is just
// above 127 2^e; 32 values rather than a row keep a strong channel from costing the
// others theirs.
//
// Random bits: eight values to a Philox counter, sixteen bits each, where the
// optimizers take four: the generator is a third of the stochastic form's
// instructions, and the third counter word sets these numbers apart from theirs.

namespace kept {

constexpr int kThreads = 256;
constexpr int kGroup = 32;
constexpr uint32_t kStream = 1;                 // last counter word

struct Store {                                  // where it goes
    int8_t *q;
    uint8_t *power;                             // e + 127; 255: the group holds an infinity or a NaN
    uint64_t q_ld, power_ld;
    uint64_t base, across;                      // first counter; counters a row
    uint32_t vec;                               // eight codes are 8-byte aligned
    uint32_t step;
    RoundKeys keys;
};

struct Source {
    const int8_t *q;
    const uint8_t *power;
    uint64_t q_ld, power_ld;
    uint32_t vec;
};

__device__ __forceinline__ int live_of(uint64_t cols, uint64_t col)
{
    return col >= cols ? 0 : cols - col < 8 ? static_cast<int>(cols - col) : 8;
}

// e + 127 for the bits of a largest value, 127 being 1.984375 * 2^6.
__device__ __forceinline__ uint32_t power_of(uint32_t top)
{
    const int b = static_cast<int>((top + 0x1FFFFu) >> 23) - 6;
    return top >= 0x7F800000u ? 255u : b > 0 ? static_cast<uint32_t>(b) : 0u;
}

__device__ __forceinline__ float scale_of(uint32_t b)
{
    return __uint_as_float(b == 255u ? 0x7FC00000u : b ? b << 23 : 0x00400000u);
}

// Eight values of a row from `col` on, a multiple of 8, of which `live` are the
// row's.  All lanes of a warp call this together; four in a row hold a group.
template <bool SR>
__device__ __forceinline__ void keep8(const Store &S, uint64_t row, uint64_t col, int live, const float x[8])
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const uint32_t b = power_of(top);
    const float up = __uint_as_float((254u - b) << 23);
    uint32_t c[8], w[4];
    if (SR) {
        const uint64_t at = S.base + row * S.across + (col >> 3);
        philox4x32_10(static_cast<uint32_t>(at), static_cast<uint32_t>(at >> 32), S.step, kStream, S.keys, w);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float y = __fmul_rn(x[i], up);
        if (SR) {
            // the high half of ceil(65536 y) + 65535 - r; |y| <= 127, so the sum stays below 128 * 65536
            const uint32_t not_r = (i & 1) ? ~w[i >> 1] >> 16 : ~w[i >> 1] & 0xFFFFu;
            c[i] = static_cast<uint32_t>(__float2int_ru(__fmul_rn(y, 65536.0f))) + not_r;
        } else {
            c[i] = __float_as_uint(__fadd_rn(y, 12582912.0f));      // its low byte
        }
    }
    constexpr uint32_t kPick = SR ? 0x0062 : 0x0040;
    uint2 v = make_uint2(__byte_perm(__byte_perm(c[0], c[1], kPick), __byte_perm(c[2], c[3], kPick), 0x5410),
                         __byte_perm(__byte_perm(c[4], c[5], kPick), __byte_perm(c[6], c[7], kPick), 0x5410));
    if (b == 255u) v = make_uint2(0, 0);
    int8_t *q = S.q + row * S.q_ld + col;
    if (live == 8 && S.vec) {
        *reinterpret_cast<uint2 *>(q) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) q[i] = static_cast<int8_t>((i < 4 ? v.x : v.y) >> (8 * (i & 3)));
    }
    if (live > 0 && (threadIdx.x & 3) == 0) S.power[row * S.power_ld + (col >> 5)] = static_cast<uint8_t>(b);
}

// Codes and scale of eight values, to be loaded ahead of their use.
struct Codes {
    uint2 v;
    uint32_t b;
};

__device__ __forceinline__ Codes fetch8(const Source &S, uint64_t row, uint64_t col, int live)
{
    Codes c{make_uint2(0, 0), 0};
    if (live <= 0) return c;
    const int8_t *q = S.q + row * S.q_ld + col;
    if (live == 8 && S.vec) {
        c.v = *reinterpret_cast<const uint2 *>(q);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) (i < 4 ? c.v.x : c.v.y) |= static_cast<uint32_t>(static_cast<uint8_t>(q[i])) << (8 * (i & 3));
    }
    c.b = S.power[row * S.power_ld + (col >> 5)];
    return c;
}

__device__ __forceinline__ void values8(const Codes &c, float x[8])
{
    const float scale = scale_of(c.b);
    const uint32_t lo = c.v.x ^ 0x80808080u, hi = c.v.y ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 8; ++i)     // 2^23 + 128 + q
        x[i] = __fmul_rn(__fsub_rn(__uint_as_float(__byte_perm(i < 4 ? lo : hi, 0x4B000000u, 0x7440 + (i & 3))),
                                   8388736.0f), scale);
}

// Eight values from any column on, whose group may end among them.
__device__ __forceinline__ void values_across(const Source &S, uint64_t row, uint64_t col, int live, float x[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = i < live ? __fmul_rn(static_cast<float>(S.q[row * S.q_ld + col + i]),
                                    scale_of(S.power[row * S.power_ld + ((col + i) >> 5)])) : 0.0f;
}

// Eight values out, `live` of them, to nearest where they are bf16.
template <int DT>
__device__ __forceinline__ void store8(void *dst, uint64_t at, int live, bool vec, const float v[8])
{
    if (DT == ASR_BF16) {
        uint16_t *p = static_cast<uint16_t *>(dst) + at;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        if (vec && live == 8) {
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < live) p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
        }
    } else {
        float *p = static_cast<float *>(dst) + at;
        if (vec && live == 8) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < live) p[i] = v[i];
        }
    }
}

// A matrix of f32 or bf16 values, rows `ld` apart.
struct Matrix {
    const void *p;
    uint64_t ld;
    uint32_t vec;                               // units of eight are 16-byte aligned
};

struct Out {
    void *p;
    uint64_t ld;
    uint32_t vec;
};

struct PackParams {
    Matrix x;
    uint64_t rows, cols;
    Store to;
};

// A warp a span of 512 columns, two units of eight a lane.
template <bool SR, int DT>
__global__ void __launch_bounds__(kThreads) pack_kernel(const __grid_constant__ PackParams P)
{
    const uint32_t lane = threadIdx.x & 31;
    muon::Walk k(P.rows, (P.cols + 1) / 2, blockIdx.x * 8ull + (threadIdx.x >> 5), gridDim.x * 8ull);
    for (; k.more(); k.next()) {
        float x[2][8];
        int live[2];
        uint64_t col[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            col[u] = k.span * 512ull + u * 256 + lane * 8;
            live[u] = live_of(P.cols, col[u]);
            muon::load8(P.x.p, DT, k.row * P.x.ld + col[u], live[u], P.x.vec, x[u]);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) keep8<SR>(P.to, k.row, col[u], live[u], x[u]);
    }
}

struct UnpackParams {
    Source from;
    Out out;
    uint64_t rows, cols;
};

template <int DT>
__global__ void __launch_bounds__(kThreads) unpack_kernel(const __grid_constant__ UnpackParams P)
{
    const uint32_t lane = threadIdx.x & 31;
    muon::Walk k(P.rows, (P.cols + 1) / 2, blockIdx.x * 8ull + (threadIdx.x >> 5), gridDim.x * 8ull);
    for (; k.more(); k.next()) {
        Codes c[2];
        int live[2];
        uint64_t col[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            col[u] = k.span * 512ull + u * 256 + lane * 8;
            live[u] = live_of(P.cols, col[u]);
            c[u] = fetch8(P.from, k.row, col[u], live[u]);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float v[8];
            values8(c[u], v);
            store8<DT>(P.out.p, k.row * P.out.ld + col[u], live[u], P.out.vec, v);
        }
    }
}

// ------------------------------------------------------------------ host

constexpr uint64_t kMaxRows = 1ull << 30, kMaxCols = 1ull << 24;

bool sizes_ok(uint64_t rows, uint64_t cols) { return rows <= kMaxRows && cols <= kMaxCols; }

bool dtype_ok(int32_t dtype) { return dtype == ASR_F32 || dtype == ASR_BF16; }

bool matrix_ok(const void *p, int32_t dtype, uint64_t ld, uint64_t cols)
{
    return p && muon::element_aligned(p, dtype) && int8::pitch_ok(ld, cols);
}

Matrix matrix(const void *p, uint64_t ld) { return Matrix{p, ld, muon::units_aligned(p, ld, 0) ? 1u : 0u}; }

Out out(void *p, uint64_t ld) { return Out{p, ld, muon::units_aligned(p, ld, 0) ? 1u : 0u}; }

bool aligned8(const void *p, uint64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0 && ld % 8 == 0; }

uint64_t groups(uint64_t cols) { return (cols + kGroup - 1) / kGroup; }

// Whether a checkpoint of rows x cols can be read.
asr_status readable(const asr_checkpoint &c, uint64_t cols)
{
    return c.q && c.power && int8::pitch_ok(c.q_ld, cols) && int8::pitch_ok(c.power_ld, groups(cols))
               ? ASR_OK : ASR_ERR_INVALID_VALUE;
}

// And written, its random bits with it.
asr_status writable(const asr_checkpoint &c, uint64_t rows, uint64_t cols)
{
    if (c.rounding != ASR_ROUND_SR && c.rounding != ASR_ROUND_RNE) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (c.base_index % kGroup || c.base_index > UINT64_MAX - rows * groups(cols) * kGroup) return ASR_ERR_INVALID_VALUE;
    return readable(c, cols);
}

Source source(const asr_checkpoint &c)
{
    return Source{c.q, c.power, c.q_ld, c.power_ld, aligned8(c.q, c.q_ld) ? 1u : 0u};
}

Store store(const asr_checkpoint &c, uint64_t cols)
{
    Store S;
    S.q = c.q;
    S.power = c.power;
    S.q_ld = c.q_ld;
    S.power_ld = c.power_ld;
    S.base = c.base_index / 8;
    S.across = groups(cols) * (kGroup / 8);
    S.vec = aligned8(c.q, c.q_ld);
    S.step = c.step;
    S.keys = make_keys(c.seed);
    return S;
}

// Loads every kernel of a list on the current device once, so that any later call
// of them may be captured into a graph.
template <typename... K>
asr_status load_once(std::atomic<uint64_t> &ready, K... kernels)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (e == cudaSuccess && (ready.load(std::memory_order_acquire) & bit)) return ASR_OK;
    (void)std::initializer_list<int>{(e = e == cudaSuccess ? prod::load_kernel(kernels) : e, 0)...};
    if (e != cudaSuccess) return cuda_fail(e);
    ready.fetch_or(bit, std::memory_order_release);
    return ASR_OK;
}

// Blocks of eight warps for spans of 512 columns.
unsigned span_blocks(uint64_t rows, uint64_t cols)
{
    return int8::blocks_for(rows * ((cols + 511) / 512), 8, 1u << 20);
}

asr_status setup()
{
    static std::atomic<uint64_t> ready{0};
    return load_once(ready, pack_kernel<false, ASR_F32>, pack_kernel<false, ASR_BF16>, pack_kernel<true, ASR_F32>,
                     pack_kernel<true, ASR_BF16>, unpack_kernel<ASR_F32>, unpack_kernel<ASR_BF16>);
}

asr_status pack(const void *x, int32_t dtype, uint64_t rows, uint64_t cols, uint64_t x_ld, const asr_checkpoint *to,
                cudaStream_t stream)
{
    if (!dtype_ok(dtype)) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (!to) return ASR_ERR_INVALID_VALUE;
    if (to->rounding != ASR_ROUND_SR && to->rounding != ASR_ROUND_RNE) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (rows == 0 || cols == 0) return ASR_OK;
    if (!sizes_ok(rows, cols) || !matrix_ok(x, dtype, x_ld, cols)) return ASR_ERR_INVALID_VALUE;
    asr_status st = writable(*to, rows, cols);
    if (st == ASR_OK) st = setup();
    if (st != ASR_OK) return st;
    PackParams P;
    P.x = matrix(x, x_ld);
    P.rows = rows;
    P.cols = cols;
    P.to = store(*to, cols);
    const bool sr = to->rounding == ASR_ROUND_SR, bf = dtype == ASR_BF16;
    auto kernel = sr ? (bf ? pack_kernel<true, ASR_BF16> : pack_kernel<true, ASR_F32>)
                     : (bf ? pack_kernel<false, ASR_BF16> : pack_kernel<false, ASR_F32>);
    kernel<<<span_blocks(rows, cols), kThreads, 0, stream>>>(P);
    return launched(ASR_KERNEL_CHECKPOINT);
}

asr_status unpack(const asr_checkpoint *from, uint64_t rows, uint64_t cols, void *dst, int32_t dtype, uint64_t ld,
                  cudaStream_t stream)
{
    if (!dtype_ok(dtype)) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (!from) return ASR_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0) return ASR_OK;
    if (!sizes_ok(rows, cols) || !matrix_ok(dst, dtype, ld, cols)) return ASR_ERR_INVALID_VALUE;
    asr_status st = readable(*from, cols);
    if (st == ASR_OK) st = setup();
    if (st != ASR_OK) return st;
    UnpackParams P;
    P.from = source(*from);
    P.out = out(dst, ld);
    P.rows = rows;
    P.cols = cols;
    auto kernel = dtype == ASR_BF16 ? unpack_kernel<ASR_BF16> : unpack_kernel<ASR_F32>;
    kernel<<<span_blocks(rows, cols), kThreads, 0, stream>>>(P);
    return launched(ASR_KERNEL_CHECKPOINT);
}

}  // namespace kept
