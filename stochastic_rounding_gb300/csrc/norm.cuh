// norm.cuh -- layer norm and the norm by the root mean square, and their backward
// pass with the weight's and the bias's gradients.  Included into asr.cu (inside
// its anonymous namespace), after checkpoint.cuh.
//
//   mean = sum x / n (centred) or 0;   rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
//   h = (x - mean) rstd;   y = h w + b
//   g = dy w;   dx = rstd (g - [sum g / n] - h sum (g h) / n)
//   dw = sum over rows of dy h;   db = sum over rows of dy
//
// A row is held in registers, 16 values a thread, so it is read once: by 4 to 32
// lanes where it has up to 512 values, else by a block.  Its sums: each warp's own
// mean and its squares about that, then the warps' joined (the squares of a warp's
// mean about the row's added), so nothing cancels.  Blocks walk over rows, the next
// row's values fetched before the current one's are worked on.
//
// The backward kernel keeps its columns' sums for dw and db in registers (up to 1,216
// blocks leave theirs, and a second kernel adds them up, in one order), which leaves
// too few warps to hide memory behind: each thread copies its own values of the next
// rows into shared memory, asynchronously, and reads them back itself, so the ring
// needs no barrier but the warp's.  Rows that do not fit a block of 1,024 threads are
// read anew for each sum.
//
// bf16 8,192 x 4,096, one launch after another, with the time of its bytes at 6,697 GB/s:
// norm 26.6 us (20.0), layer norm 30.8, with codes 32.7 and 39.1 (25.2); backward from x
// 37.0 and 37.8 (30.1), from codes 35.1 and 39.1 (25.2), of which the sums of dw take 4.
// Bound forward by instructions, 16 a value, 23 with a mean and 31 with codes too: issue
// slots are 69 to 73 % full with the memory at 35 to 47 %.  Backward by waiting: two blocks
// an SM (23 % of its warps) issue in 43 to 52 % of cycles, held up by shared memory and
// the row's barrier.  f32 from x, 8,192 x 4,096, 104 us (60), by the ring: two rows of it
// fit, and issue is at 26 %, what is waited for being memory.

namespace norm {

using kept::live_of;

constexpr int kUnits = 2;                       // of eight values, a thread
constexpr uint64_t kWarpCols = 32 * 8 * kUnits; // a warp's row at most
constexpr uint64_t kBlockCols = 1024 * 8 * kUnits;
constexpr int kWarpThreads = 256;               // where lanes have rows

struct Params {
    kept::Matrix x, dy;
    kept::Out y, dx;
    const void *w, *b;                          // may be null
    float *mean, *rstd;                         // forward: may be null
    uint32_t rows, cols;
    float eps, over_n;                          // 1 / n
    uint32_t w_dtype, b_dtype, w_vec, b_vec;
    uint32_t centred;
    uint32_t sr;
    uint32_t lanes;                             // of a row, where lanes have rows
    kept::Store to;
    kept::Source from;
    float *partial;                             // backward: [blocks][dw, db][pitch]
    uint64_t pitch;                             // cols up to a multiple of eight
    uint32_t dw, db;                            // which are wanted
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

// Over `lanes` neighbours, a power of two.
__device__ __forceinline__ float lane_sum(float v, uint32_t lanes)
{
    for (uint32_t d = lanes / 2; d; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
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

// Which rows a thread works on, and which values of them.  All threads of a warp make
// the same number of steps; `row` may lie past the last row.
template <bool WARP, bool FULL>
struct Place {
    uint32_t base, stride, col[kUnits];
    uint32_t sub, at;                           // row of a step; place in the row's threads
    int live[kUnits];
    __device__ explicit Place(const Params &P)
    {
        uint32_t threads;
        if (WARP) {
            const uint32_t lane = threadIdx.x & 31, rows = 32 / P.lanes;
            base = (blockIdx.x * (kWarpThreads / 32) + (threadIdx.x >> 5)) * rows;
            stride = gridDim.x * (kWarpThreads / 32) * rows;
            sub = lane / P.lanes;
            at = lane % P.lanes;
            threads = P.lanes;
        } else {
            base = blockIdx.x;
            stride = gridDim.x;
            sub = 0;
            at = threadIdx.x;
            threads = blockDim.x;
        }
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            col[u] = (u * threads + at) * 8;
            live[u] = FULL ? 8 : live_of(P.cols, col[u]);
        }
    }
    // where value e of the warp's 256 of unit u lies in a matrix, null where there is none; `first`: the warp's first row
    template <int DT, typename T>
    __device__ T *value(const Params &P, T *matrix, uint32_t ld, int u, uint32_t first, uint32_t e) const
    {
        using Char = typename std::conditional<std::is_const<T>::value, const char, char>::type;
        const uint32_t lane = e >> 3, lanes = WARP ? P.lanes : 32, r = WARP ? first + lane / lanes : first;
        const uint32_t c = col[u] - at8() + lane % lanes * 8 + (e & 7);
        return r < P.rows && c < P.cols ? static_cast<Char *>(matrix) + kept::place(r, ld, c) * (DT == ASR_BF16 ? 2 : 4) : nullptr;
    }
    // the caller's place among its warp's columns of a row
    __device__ uint32_t at8() const { return (WARP ? at : at & 31) * 8; }
    __device__ uint32_t row() const { return base + sub; }
    __device__ int of(int u, uint32_t row, uint32_t rows) const
    {
        return FULL && !WARP ? 8 : row < rows ? live[u] : 0;
    }
};

// For rows off alignment: a warp's 256 values (the first half of a kept::Stage).
struct __align__(16) HalfStage {
    uint4 w[64];
};

// Two sums over a warp: lanes below 16 get the first, the others the second.
__device__ __forceinline__ float half_sums(float a, float b)
{
    const bool high = threadIdx.x & 16;
    float v = __fadd_rn(high ? b : a, __shfl_xor_sync(0xFFFFFFFFu, high ? a : b, 16));
#pragma unroll
    for (int d = 8; d; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

// Sums of a block's warps, two of each; `turn` says which half a row uses, so that one
// barrier a row is enough.
struct Parts {
    float v[2][2][32];
};

// Every lane gets warp `lane`'s two.
__device__ __forceinline__ float2 exchange(Parts &parts, uint32_t turn, float2 mine)
{
    const uint32_t lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) {
        parts.v[turn][0][threadIdx.x >> 5] = mine.x;
        parts.v[turn][1][threadIdx.x >> 5] = mine.y;
    }
    __syncthreads();
    return lane < warps ? make_float2(parts.v[turn][0][lane], parts.v[turn][1][lane]) : make_float2(0.0f, 0.0f);
}

// Two sums over a block, of what its threads hold: half the shuffles of one after the
// other, and as many steps as one takes.
__device__ __forceinline__ float2 block_sums(Parts &parts, uint32_t turn, float a, float b)
{
    const uint32_t lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    float v = half_sums(a, b);
    if ((lane & 15) == 0) parts.v[turn][lane >> 4][threadIdx.x >> 5] = v;
    __syncthreads();
    const float *part = parts.v[turn][lane >> 4];
    v = (lane & 15) < warps ? part[lane & 15] : 0.0f;
    if (warps > 16) v = __fadd_rn(v, (lane & 15) + 16 < warps ? part[(lane & 15) + 16] : 0.0f);
#pragma unroll
    for (int d = 8; d; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    const float other = __shfl_xor_sync(0xFFFFFFFFu, v, 16);
    return lane & 16 ? make_float2(other, v) : make_float2(v, other);
}

// How many of a row's values warp `lane` of the block holds.
__device__ __forceinline__ float count_of(uint32_t cols)
{
    const uint32_t first = (threadIdx.x & 31) * 256;
    float n = 0.0f;
    if ((threadIdx.x & 31) < blockDim.x >> 5)
        for (int u = 0; u < kUnits; ++u) {
            const uint32_t col = first + u * blockDim.x * 8;
            n += col >= cols ? 0.0f : static_cast<float>(cols - col < 256 ? cols - col : 256);
        }
    return n;
}

template <int DT, bool WARP, bool KEEP, bool FULL>
__global__ void __launch_bounds__(WARP ? kWarpThreads : 1024) forward_kernel(const __grid_constant__ Params P)
{
    __shared__ Parts parts;
    extern __shared__ HalfStage stages[];       // one a warp, where rows are off alignment
    kept::Stage &stage = reinterpret_cast<kept::Stage &>(stages[threadIdx.x >> 5]);
    Place<WARP, FULL> at(P);
    float counts = 0.0f, own = 0.0f;            // of warp `lane`, of the caller's
    if (!WARP) {
        counts = count_of(P.cols);
        own = __shfl_sync(0xFFFFFFFFu, counts, threadIdx.x >> 5);
    }
    const float over_own = own > 0.0f ? __frcp_rn(own) : 0.0f, over_counts = counts > 0.0f ? __frcp_rn(counts) : 0.0f;
    kept::Raw<DT> next[kUnits];
    auto load = [&]() {
        if (at.base >= P.rows) return;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int live = at.of(u, at.row(), P.rows);
            if (!FULL && P.x.vec == 0) {
                kept::stage_in<DT, 8>(stage, [&](uint32_t e) { return at.template value<DT>(P, P.x.p, P.x.ld, u, at.base, e); });
                next[u] = kept::staged<DT>(stage, threadIdx.x & 31);
            } else {
                next[u] = kept::fetch<DT, FULL && !WARP>(P.x, at.row(), at.col[u], live, P.x.vec);
            }
        }
    };
    load();
    for (uint32_t turn = 0; at.base < P.rows; turn ^= 1) {
        const uint32_t row = at.row();
        kept::Raw<DT> raw[kUnits];
        float x[kUnits][8], sum = 0.0f, squares = 0.0f, mean = 0.0f;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            raw[u] = next[u];
            kept::values(raw[u], x[u]);
        }
        at.base += at.stride;
        load();
        float2 two = kept::both(0.0f);
        if (P.centred) {
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
#pragma unroll
                for (int i = 0; i < 8; i += 2) two = kept::add2(two, make_float2(x[u][i], x[u][i + 1]));
            sum = __fadd_rn(two.x, two.y);
            sum = WARP ? lane_sum(sum, P.lanes) : warp_sum(sum);
            mean = __fmul_rn(sum, WARP ? P.over_n : over_own);
            two = kept::both(0.0f);
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    float2 d = kept::add2(make_float2(x[u][i], x[u][i + 1]), kept::both(-mean));
                    if (!FULL) d = make_float2(i < at.live[u] ? d.x : 0.0f, i + 1 < at.live[u] ? d.y : 0.0f);
                    two = kept::fma2(d, d, two);
                }
        } else {
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float2 d = make_float2(x[u][i], x[u][i + 1]);
                    two = kept::fma2(d, d, two);
                }
        }
        squares = __fadd_rn(two.x, two.y);
        squares = WARP ? lane_sum(squares, P.lanes) : warp_sum(squares);
        if (!WARP) {
            const float2 p = exchange(parts, turn, make_float2(sum, squares));
            squares = p.y;
            if (P.centred) {
                mean = __fmul_rn(warp_sum(p.x), P.over_n);
                const float d = counts > 0.0f ? __fsub_rn(__fmul_rn(p.x, over_counts), mean) : 0.0f;    // the warp's own mean again
                squares = __fmaf_rn(__fmul_rn(d, d), counts, squares);
            }
            squares = warp_sum(squares);
        }
        const float rstd = __frsqrt_rn(__fmaf_rn(squares, P.over_n, P.eps));
        if (at.at == 0 && P.rstd && row < P.rows) {
            P.rstd[row] = rstd;
            if (P.mean) P.mean[row] = mean;
        }
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int live = at.of(u, row, P.rows);
            if (KEEP) {
                if (P.sr) kept::keep8<true, DT, FULL && !WARP>(P.to, row, at.col[u], live, raw[u]);
                else kept::keep8<false, DT, FULL && !WARP>(P.to, row, at.col[u], live, raw[u]);
            }
            if ((FULL || P.y.vec) && !(FULL && !WARP) && live == 0) continue;
            float w[8], b[8];
            params8(P.w, P.w_dtype, at.col[u], live, P.w_vec, 1.0f, w);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                float2 &h = reinterpret_cast<float2 &>(x[u][i]);
                h = kept::mul2(kept::add2(h, kept::both(-mean)), kept::both(rstd));
                h = kept::mul2(h, make_float2(w[i], w[i + 1]));
            }
            if (P.b) {                          // behind the weight, and not with it, for want of registers
                muon::load8(P.b, P.b_dtype, at.col[u], live, P.b_vec, b);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[u][i] = __fadd_rn(x[u][i], b[i]);
            }
            if (!FULL && P.y.vec == 0) {
                __syncwarp();
                kept::put_staged<DT>(stage, threadIdx.x & 31, kept::rounded<DT>(x[u]));
                kept::stage_out<DT, 8>(stage, [&](uint32_t e) { return at.template value<DT>(P, P.y.p, P.y.ld, u, row - at.sub, e); });
            } else {
                kept::store8<DT, FULL && !WARP>(P.y, row, at.col[u], live, P.y.vec, x[u]);
            }
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
    const uint32_t end = (P.cols + 255) / 256 * 256;        // whole warps take part, for the groups
    for (uint32_t row = blockIdx.x; row < P.rows; row += gridDim.x) {
        float sum = 0.0f, squares = 0.0f, x[8];
        if (P.centred)
            for (uint32_t col = threadIdx.x * 8; col < P.cols; col += kLongThreads * 8) {
                kept::values(kept::fetch<DT>(P.x, row, col, live_of(P.cols, col), P.x.vec), x);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum = __fadd_rn(sum, x[i]);
            }
        const float mean = P.centred ? __fmul_rn(block_sum(sum, part), P.over_n) : 0.0f;
        for (uint32_t col = threadIdx.x * 8; col < P.cols; col += kLongThreads * 8) {
            const int live = live_of(P.cols, col);
            kept::values(kept::fetch<DT>(P.x, row, col, live, P.x.vec), x);
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
        for (uint32_t col = threadIdx.x * 8; col < end; col += kLongThreads * 8) {
            const int live = live_of(P.cols, col);
            const kept::Raw<DT> raw = kept::fetch<DT>(P.x, row, col, live, P.x.vec);
            kept::values(raw, x);
            if (KEEP) {
                if (P.sr) kept::keep8<true, DT, false>(P.to, row, col, live, raw);
                else kept::keep8<false, DT, false>(P.to, row, col, live, raw);
            }
            if (live == 0) continue;
            float w[8], b[8];
            params8(P.w, P.w_dtype, col, live, P.w_vec, 1.0f, w);
            params8(P.b, P.b_dtype, col, live, P.b_vec, 0.0f, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __fmaf_rn(__fmul_rn(__fsub_rn(x[i], mean), rstd), w[i], b[i]);
            kept::store8<DT>(P.y, row, col, live, P.y.vec, x);
        }
    }
}

// ---- backward

template <int DT, bool KEPT>
__device__ __forceinline__ void input8(const Params &P, uint32_t row, uint32_t col, int live, float x[8])
{
    if (KEPT) kept::values(kept::fetch_codes(P.from, row, col, live), x);
    else kept::values(kept::fetch<DT>(P.x, row, col, live, P.x.vec), x);
}

template <int BYTES>
__device__ __forceinline__ void copy_async(void *to, const void *from)
{
    if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_addr(to)), "l"(from), "n"(BYTES) : "memory");
}

// Eight values of a matrix, from memory to a thread's place in shared memory (words
// `step` apart for 16 bytes each), asynchronously in 16 bytes; of a row's last ones f32
// by one, bf16 at once.
template <int DT, bool FULL>
__device__ __forceinline__ void bring(uint4 *to, uint32_t step, const kept::Matrix &M, uint32_t row, uint32_t col, int live)
{
    const char *from = static_cast<const char *>(M.p) + kept::place(row, M.ld, col) * (DT == ASR_BF16 ? 2 : 4);
    if (FULL || (M.vec && live == 8)) {
#pragma unroll
        for (int i = 0; i < (DT == ASR_BF16 ? 1 : 2); ++i) copy_async<16>(to + i * step, from + 16 * i);
    } else if (DT == ASR_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t *w = reinterpret_cast<uint32_t *>(to + (i >> 2) * step) + (i & 3);
            if (i < live) copy_async<4>(w, from + 4 * i);
            else *w = 0;
        }
    } else {
        const kept::Raw<DT> r = kept::fetch<DT>(M, row, col, live, 0);
        to[0] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    }
}

template <int DT>
__device__ __forceinline__ void taken(const uint4 *from, uint32_t step, float x[8])
{
    kept::Raw<DT> r;
#pragma unroll
    for (int i = 0; i < (DT == ASR_BF16 ? 1 : 2); ++i) {
        const uint4 v = from[i * step];
        r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
    }
    kept::values(r, x);
}

// A thread's share of a stage, in words of 16 bytes: dy, then x or its codes.
template <int DT, bool KEPT>
struct Stage {
    static constexpr int kDy = (DT == ASR_BF16 ? 1 : 2) * kUnits;
    static constexpr int kX = KEPT ? 1 : kDy;               // codes: 8 bytes a unit
    static constexpr int kWords = kDy + kX;
};
static_assert(kUnits == 2, "codes of two units fill a word");

// Stages of the ring: four, fewer where a block's values and weight would not leave
// room (227 KB) for them.
template <int DT, bool KEPT, int THREADS>
struct Ring {
    static constexpr int kRoom = 220 * 1024 - THREADS * 64;
    static constexpr int kFit = kRoom / (THREADS * Stage<DT, KEPT>::kWords * 16);
    static constexpr int kStages = kFit < 1 ? 1 : kFit > 4 ? 4 : kFit;
    static size_t bytes(unsigned threads) { return ((static_cast<size_t>(kStages) * Stage<DT, KEPT>::kWords + 4) * 16 + kStages) * threads; }
};

// LEAN: without a mean and a bias's gradient, with fewer instructions, for up to 512
// threads (bf16 from codes, one launch after another: 8,192 x 4,096 38.9 -> 35.0 us,
// 4,096 x 8,192 42.6 -> 38.9; from x it gains nothing, 37.0 and 37.3).
template <int DT, bool WARP, bool KEPT, int THREADS, bool FULL, bool LEAN = false>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 2 : 1) backward_kernel(const __grid_constant__ Params P)
{
    using S = Stage<DT, KEPT>;
    constexpr bool kPower = KEPT && !WARP && FULL;           // whole words of powers
    constexpr int kStages = Ring<DT, KEPT, THREADS>::kStages;
    extern __shared__ __align__(16) uint4 ring[];           // [weight: 4 | stages' words][thread], [stage][warp][8]
    __shared__ Parts parts;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Place<WARP, FULL> at(P);
    const uint32_t step = blockDim.x;
    uint4 *const mine = ring + threadIdx.x;
    // Rows off alignment: value e of the warp's 256 of unit u, in words of 16 bytes that
    // its lanes have side by side.
    auto word_of = [&](uint4 *to, uint32_t e) {
        uint4 *const warp = to - (threadIdx.x & 31);
        return reinterpret_cast<uint32_t *>(warp + (e >> 2 & 1) * step + (e >> 3)) + (e & 3);
    };
    auto bring_off = [&](uint4 *to, const kept::Matrix &M, uint32_t first) {
        if (DT == ASR_BF16) {                   // nothing smaller than four bytes is copied asynchronously
            uint16_t v[kUnits][8];
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const void *from = at.template value<DT>(P, M.p, M.ld, u, first, 32 * i + (threadIdx.x & 31));
                    v[u][i] = from ? *static_cast<const uint16_t *>(from) : static_cast<uint16_t>(0);
                }
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    reinterpret_cast<uint16_t *>(to + u * step - (threadIdx.x & 31))[32 * i + (threadIdx.x & 31)] = v[u][i];
        } else {
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t e = 32 * i + (threadIdx.x & 31);
                    uint32_t *w = word_of(to + 2 * u * step, e);
                    const void *from = at.template value<DT>(P, M.p, M.ld, u, first, e);
                    if (from) copy_async<4>(w, from);
                    else *w = 0;
                }
        }
    };
    // A row's rstd, mean and words of powers come through the ring too, a lane a word of
    // the warp's: in registers, a row ahead, they came too late (8,192 x 4,096 bf16 from x
    // 44.5 -> 40.4 us, from codes 44.0 -> 37.0).
    const uint32_t lane = threadIdx.x & 31;
    const char *stat = nullptr;
    uint32_t stat_step = 4;
    if (!WARP) {
        if (lane == 0) stat = reinterpret_cast<const char *>(P.rstd);
        if (!LEAN && lane == 1 && P.centred) stat = reinterpret_cast<const char *>(P.mean);
        if (kPower && lane >= 2 && lane < 6) {
            stat = reinterpret_cast<const char *>(P.from.power) + ((lane >= 4 ? at.col[1] : at.col[0]) - at.at8()) / 32 + (lane & 1) * 4;
            stat_step = P.from.power_ld;
        }
    }
    auto rest_of = [&](uint32_t slot) {
        return reinterpret_cast<uint32_t *>(ring + (4 + kStages * S::kWords) * step) + (slot * (step >> 5) + (threadIdx.x >> 5)) * 8;
    };
    // `first`: the warp's first row
    auto bring_row = [&](uint32_t first, uint32_t slot) {
        const uint32_t row = first + at.sub;
        uint4 *to = mine + (4 + slot * S::kWords) * step;
        if (!(FULL && WARP)) __syncwarp();      // lanes may write for one another what was read a row ago
        if (!FULL && first < P.rows) {
            if (P.dy.vec == 0) bring_off(to, P.dy, first);
            if (!KEPT && P.x.vec == 0) bring_off(to + S::kDy * step, P.x, first);
        }
        if (first < P.rows)
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int live = at.of(u, row, P.rows);
            if (!(FULL && !WARP) && live == 0) continue;
            if (FULL || P.dy.vec) bring<DT, FULL>(to + u * (S::kDy / kUnits) * step, step, P.dy, row, at.col[u], live);
            if (!KEPT) {
                if (FULL || P.x.vec)
                    bring<DT, FULL>(to + (S::kDy + u * (S::kDy / kUnits)) * step, step, P.x, row, at.col[u], live);
            } else {
                uint2 *q = reinterpret_cast<uint2 *>(to + S::kDy * step) + u;
                if (FULL || (P.from.vec && live == 8)) copy_async<8>(q, P.from.q + kept::place(row, P.from.q_ld, at.col[u]));
                else *q = kept::fetch_codes(P.from, row, at.col[u], live).v;
            }
        }
        if (!WARP && stat && row < P.rows) copy_async<4>(rest_of(slot) + lane, stat + static_cast<uint64_t>(row) * stat_step);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // what does not come through the ring is fetched a row ahead
    float mean = 0.0f, rstd = 0.0f;
    uint32_t power[kUnits] = {};
    auto fetch_rest = [&](uint32_t row) {
        if (row >= P.rows) return;
        if (WARP) {
            rstd = P.rstd[row];
            if (P.centred) mean = P.mean[row];
        }
        if (KEPT && !kPower)
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
                if (FULL || at.live[u]) power[u] = P.from.power[kept::place(row, P.from.power_ld, at.col[u] >> 5)];
    };
    if constexpr (kStages > 1) {
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) bring_row(at.base + s * at.stride, s);
    }
    fetch_rest(at.row());
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        float w[8];
        params8(P.w, P.w_dtype, at.col[u], at.live[u], P.w_vec, 1.0f, w);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float4 *>(mine + (2 * u + i) * step) = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    float dw[kUnits][8] = {}, db[kUnits][8] = {};
    uint32_t slot = 0;
    for (uint32_t turn = 0; at.base < P.rows; turn ^= 1) {
        const uint32_t row = at.row();
        bring_row(at.base + (kStages - 1) * at.stride, slot ? slot - 1 : kStages - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        if (!(FULL && WARP)) __syncwarp();
        const uint4 *from = mine + (4 + slot * S::kWords) * step;
        float m = mean, r = rstd;
        uint32_t b[kUnits] = {power[0], power[1]};
        if (!WARP) {
            const uint32_t *rest = rest_of(slot);
            r = __uint_as_float(rest[0]);
            m = !LEAN && P.centred ? __uint_as_float(rest[1]) : 0.0f;
            if (kPower)
#pragma unroll
                for (int u = 0; u < kUnits; ++u) b[u] = rest[2 + 2 * u + (lane >> 4)] >> (lane * 2 & 24) & 255;
        }
        slot = slot + 1 == kStages ? 0 : slot + 1;
        at.base += at.stride;
        fetch_rest(at.row());
        float h[kUnits][8], g[kUnits][8];
        float2 along2 = kept::both(0.0f), sum2 = kept::both(0.0f);
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            if (at.of(u, row, P.rows) == 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) h[u][i] = g[u][i] = 0.0f;
                continue;
            }
            taken<DT>(from + u * (S::kDy / kUnits) * step, step, g[u]);
            if (KEPT) kept::values(kept::Codes{*(reinterpret_cast<const uint2 *>(from + S::kDy * step) + u), b[u]}, h[u]);
            else taken<DT>(from + (S::kDy + u * (S::kDy / kUnits)) * step, step, h[u]);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float4 w4 = *reinterpret_cast<const float4 *>(mine + (2 * u + (i >> 2)) * step);
                float2 &h2 = reinterpret_cast<float2 &>(h[u][i]), &g2 = reinterpret_cast<float2 &>(g[u][i]);
                float2 &dw2 = reinterpret_cast<float2 &>(dw[u][i]), &db2 = reinterpret_cast<float2 &>(db[u][i]);
                if (!LEAN) h2 = kept::add2(h2, kept::both(-m));
                h2 = kept::mul2(h2, kept::both(r));
                dw2 = kept::fma2(g2, h2, dw2);
                if (!LEAN) db2 = kept::add2(db2, g2);
                g2 = kept::mul2(g2, i & 2 ? make_float2(w4.z, w4.w) : make_float2(w4.x, w4.y));
                if (!LEAN) sum2 = kept::add2(sum2, g2);
                along2 = kept::fma2(g2, h2, along2);
            }
        }
        float along = __fadd_rn(along2.x, along2.y), sum = __fadd_rn(sum2.x, sum2.y);
        if (!P.dx.p) continue;
        if (WARP) {
            sum = lane_sum(sum, P.lanes);
            along = lane_sum(along, P.lanes);
        } else {
            const float2 p = block_sums(parts, turn, sum, along);
            sum = p.x;
            along = p.y;
        }
        sum = LEAN || !P.centred ? 0.0f : __fmul_rn(__fmul_rn(sum, P.over_n), r);
        along = __fmul_rn(__fmul_rn(along, P.over_n), r);
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int live = at.of(u, row, P.rows);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                float2 &g2 = reinterpret_cast<float2 &>(g[u][i]);
                const float2 h2 = reinterpret_cast<const float2 &>(h[u][i]);
                g2 = LEAN ? kept::mul2(g2, kept::both(r)) : kept::fma2(g2, kept::both(r), kept::both(-sum));
                g2 = kept::fma2(h2, kept::both(-along), g2);
            }
            if (!FULL && P.dx.vec == 0) {
                // through the words that this row's dy came in
                uint4 *const mine_dy = const_cast<uint4 *>(from) + u * (S::kDy / kUnits) * step, *const warp = mine_dy - (threadIdx.x & 31);
                const kept::Raw<DT> v = kept::rounded<DT>(g[u]);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < S::kDy / kUnits; ++i)
                    mine_dy[i * step] = make_uint4(v.w[4 * i], v.w[4 * i + 1], v.w[4 * i + 2], v.w[4 * i + 3]);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t e = 32 * i + (threadIdx.x & 31);
                    void *dst = at.template value<DT>(P, P.dx.p, P.dx.ld, u, row - at.sub, e);
                    if (!dst) continue;
                    if (DT == ASR_BF16) *static_cast<uint16_t *>(dst) = reinterpret_cast<const uint16_t *>(warp)[e];
                    else *static_cast<uint32_t *>(dst) = *word_of(mine_dy, e);
                }
            } else if ((FULL && !WARP) || live) {
                kept::store8<DT, FULL && !WARP>(P.dx, row, at.col[u], live, P.dx.vec, g[u]);
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!P.dw && !P.db) return;
    float *to = P.partial + blockIdx.x * 2 * P.pitch;
    if constexpr (WARP) {
        // a row's lanes, then the warps, one after another, in the first rows of the ring
        float *const sums = reinterpret_cast<float *>(ring);
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                for (uint32_t d = P.lanes; d < 32; d <<= 1) {
                    dw[u][i] = __fadd_rn(dw[u][i], __shfl_xor_sync(0xFFFFFFFFu, dw[u][i], d));
                    db[u][i] = __fadd_rn(db[u][i], __shfl_xor_sync(0xFFFFFFFFu, db[u][i], d));
                }
        for (uint32_t w = 0; w < kWarpThreads / 32; ++w) {
            __syncthreads();
            if (threadIdx.x >> 5 == w && lane < P.lanes)
#pragma unroll
                for (int u = 0; u < kUnits; ++u)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float *p = sums + at.col[u] + i;
                        p[0] = w ? __fadd_rn(p[0], dw[u][i]) : dw[u][i];
                        p[kWarpCols] = w ? __fadd_rn(p[kWarpCols], db[u][i]) : db[u][i];
                    }
        }
        __syncthreads();
        for (uint64_t c = threadIdx.x; c < P.cols; c += kWarpThreads) {
            to[c] = sums[c];
            if (P.db) to[P.pitch + c] = sums[kWarpCols + c];
        }
    } else {
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            if (at.live[u] == 0) continue;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float4 *p = reinterpret_cast<float4 *>(to + at.col[u]) + i;
                *p = make_float4(dw[u][4 * i], dw[u][4 * i + 1], dw[u][4 * i + 2], dw[u][4 * i + 3]);
                if (!LEAN && P.db) p[P.pitch / 4] = make_float4(db[u][4 * i], db[u][4 * i + 1], db[u][4 * i + 2], db[u][4 * i + 3]);
            }
        }
    }
}

// Rows that do not fit: dx, a block a row, read twice.
template <int DT, bool KEPT>
__global__ void __launch_bounds__(kLongThreads) backward_long_kernel(const __grid_constant__ Params P)
{
    __shared__ float part[32];
    for (uint32_t row = blockIdx.x; row < P.rows; row += gridDim.x) {
        const float mean = P.centred ? P.mean[row] : 0.0f, rstd = P.rstd[row];
        float sum = 0.0f, along = 0.0f, g[8], h[8], w[8];
        for (uint32_t col = threadIdx.x * 8; col < P.cols; col += kLongThreads * 8) {
            const int live = live_of(P.cols, col);
            kept::values(kept::fetch<DT>(P.dy, row, col, live, P.dy.vec), g);
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
        for (uint32_t col = threadIdx.x * 8; col < P.cols; col += kLongThreads * 8) {
            const int live = live_of(P.cols, col);
            kept::values(kept::fetch<DT>(P.dy, row, col, live, P.dy.vec), g);
            input8<DT, KEPT>(P, row, col, live, h);
            params8(P.w, P.w_dtype, col, live, P.w_vec, 1.0f, w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                g[i] = __fmul_rn(__fmaf_rn(-__fmul_rn(__fsub_rn(h[i], mean), rstd), along,
                                           __fsub_rn(__fmul_rn(g[i], w[i]), sum)), rstd);
            kept::store8<DT>(P.dx, row, col, live, P.dx.vec, g);
        }
    }
}

// Their columns' sums: a block 2,048 columns of every gridDim.y-th row.
template <int DT, bool KEPT>
__global__ void __launch_bounds__(256) columns_kernel(const __grid_constant__ Params P)
{
    const uint32_t col = (blockIdx.x * 256 + threadIdx.x) * 8;
    const int live = live_of(P.cols, col);
    float dw[8] = {}, db[8] = {}, g[8], h[8];
    for (uint32_t row = blockIdx.y; row < P.rows; row += gridDim.y) {
        const float mean = P.centred ? P.mean[row] : 0.0f, rstd = P.rstd[row];
        kept::values(kept::fetch<DT>(P.dy, row, col, live, P.dy.vec), g);
        input8<DT, KEPT>(P, row, col, live, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dw[i] = __fmaf_rn(g[i], __fmul_rn(__fsub_rn(h[i], mean), rstd), dw[i]);
            db[i] = __fadd_rn(db[i], g[i]);
        }
    }
    float *to = P.partial + blockIdx.y * 2 * P.pitch;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < live) {
            to[col + i] = dw[i];
            to[P.pitch + col + i] = db[i];
        }
}

struct SumParams {
    const float *partial;
    uint64_t cols, pitch;
    uint32_t groups;
    void *out[2];                               // dw, db; null where not wanted
    uint32_t dtype[2];
};

// Adds the blocks' sums of a column up in one order: a block 32 columns, of dw or of
// db, every sixteenth sum a warp.
constexpr int kSumWarps = 16;

__global__ void __launch_bounds__(kSumWarps * 32) sum_kernel(const __grid_constant__ SumParams P)
{
    __shared__ float part[kSumWarps][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int which = P.out[blockIdx.y] ? blockIdx.y : 1;       // db alone comes in the grid's only row
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t col = blockIdx.x * 32ull + lane;
    float sum = 0.0f;
    if (col < P.cols)
#pragma unroll 8
        for (uint32_t g = warp; g < P.groups; g += kSumWarps)
            sum = __fadd_rn(sum, P.partial[(g * 2ull + which) * P.pitch + col]);
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

unsigned threads_of(uint64_t cols)
{
    const int shape = shape_of(cols);
    return shape == kWarp ? kWarpThreads : shape == kBlock ? block_threads(cols) : kLongThreads;
}

// Lanes of a row of up to 512 values, 16 each.
uint32_t lanes_of(uint64_t cols)
{
    uint32_t n = 4;
    while (n * 8 * kUnits < cols && n < 32) n *= 2;
    return n;
}

template <int DT, bool KEEP, bool FULL>
Kernel forward_of(int shape)
{
    return shape == kWarp ? forward_kernel<DT, true, KEEP, FULL> : shape == kBlock ? forward_kernel<DT, false, KEEP, FULL>
                                                                                   : forward_long_kernel<DT, KEEP>;
}

Kernel forward_of(int32_t dtype, int shape, bool keep, bool full)
{
    if (dtype != ASR_BF16) return keep ? forward_of<ASR_F32, true, false>(shape) : forward_of<ASR_F32, false, false>(shape);
    if (full) return keep ? forward_of<ASR_BF16, true, true>(shape) : forward_of<ASR_BF16, false, true>(shape);
    return keep ? forward_of<ASR_BF16, true, false>(shape) : forward_of<ASR_BF16, false, false>(shape);
}

// Whether every thread of a row's has its sixteen values.
bool whole(uint64_t cols)
{
    const int shape = shape_of(cols);
    return shape == kWarp ? cols == lanes_of(cols) * 8 * kUnits : shape == kBlock && cols % kWarpCols == 0;
}

// A backward kernel and its shared memory, the registers of its blocks budgeted for
// their size: fewer a thread in larger ones.
struct Backward {
    Kernel kernel;
    size_t smem;
};

template <int DT, bool KEPT, bool WARP, int THREADS, bool FULL>
Backward backward_at(unsigned threads)
{
    return Backward{backward_kernel<DT, WARP, KEPT, THREADS, FULL>, Ring<DT, KEPT, THREADS>::bytes(threads)};
}

template <int DT, bool KEPT, bool FULL>
Backward backward_of(int shape, unsigned threads, bool lean)
{
    if constexpr (FULL && KEPT) {
        if (lean && shape == kBlock && threads <= 512)
            return Backward{backward_kernel<DT, false, true, 512, true, true>, Ring<DT, true, 512>::bytes(threads)};
    }
    if (shape == kWarp) return backward_at<DT, KEPT, true, kWarpThreads, FULL>(threads);
    if (shape == kLong) return Backward{backward_long_kernel<DT, KEPT>, 0};
    return threads <= 512 ? backward_at<DT, KEPT, false, 512, FULL>(threads) : backward_at<DT, KEPT, false, 1024, FULL>(threads);
}

template <bool KEPT>
Backward backward_of(int32_t dtype, int shape, unsigned threads, bool full, bool lean)
{
    if (dtype != ASR_BF16) return backward_of<ASR_F32, KEPT, false>(shape, threads, lean);
    return full ? backward_of<ASR_BF16, KEPT, true>(shape, threads, lean) : backward_of<ASR_BF16, KEPT, false>(shape, threads, lean);
}

Backward backward_of(int32_t dtype, bool codes, int shape, unsigned threads, bool full, bool lean)
{
    return codes ? backward_of<true>(dtype, shape, threads, full, lean) : backward_of<false>(dtype, shape, threads, full, lean);
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
            for (int form = 0; form < 6; ++form) {
                const int shape = form % 3;
                const bool full = form >= 3;
                if (e == cudaSuccess) e = prod::load_kernel(forward_of(dtype, shape, kept != 0, full));
                for (int block = 0; block < 3; ++block) {
                    const unsigned threads = shape == kWarp ? kWarpThreads : block == 2 ? 1024 : 512;
                    const Backward k = backward_of(dtype, kept != 0, shape, threads, full, block == 1);
                    if (e == cudaSuccess && k.smem)
                        e = cudaFuncSetAttribute(k.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(k.smem));
                    if (e == cudaSuccess) e = prod::load_kernel(k.kernel);
                }
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
    P.rows = static_cast<uint32_t>(p->rows);
    P.cols = static_cast<uint32_t>(p->cols);
    P.eps = static_cast<float>(p->eps);
    P.over_n = static_cast<float>(1.0 / static_cast<double>(p->cols));
    P.w_dtype = static_cast<uint32_t>(p->weight_dtype);
    P.b_dtype = static_cast<uint32_t>(p->bias_dtype);
    P.w_vec = aligned16(p->weight);
    P.b_vec = aligned16(p->bias);
    P.centred = p->centred;
    P.lanes = lanes_of(p->cols);
    P.pitch = muon::up(p->cols, 8);
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
    P.x = kept::matrix(x, x_ld, p->dtype);
    P.y = kept::out(y, y_ld, p->dtype);
    P.mean = mean;
    P.rstd = rstd;
    if (to) {
        P.to = kept::store(*to, p->cols);
        P.sr = to->rounding == ASR_ROUND_SR;
    }
    const int shape = shape_of(p->cols);
    const unsigned threads = threads_of(p->cols);
    const bool full = whole(p->cols) && P.x.vec && P.y.vec && (!to || P.to.vec);
    auto kernel = forward_of(p->dtype, shape, to != nullptr, full);
    const size_t smem = shape != kLong && (!P.x.vec || !P.y.vec) ? threads / 32 * sizeof(HalfStage) : 0;
    int most = 0;
    st = kept::resident(kernel, threads, smem, &most);
    if (st != ASR_OK) return st;
    const unsigned grid = int8::blocks_for(p->rows, shape == kWarp ? kWarpThreads / P.lanes : 1, static_cast<uint64_t>(most));
    kernel<<<grid, threads, smem, stream>>>(P);
    return launched(ASR_KERNEL_NORM);
}

// Blocks that leave sums of a backward pass at most: enough to fill the GPU, more where
// they are small, and four steps' rows each where there are fewer, since each leaves
// 2 x cols of them.  Of rows that do not fit, 64, with 32 rows each.
uint64_t groups_of(uint64_t rows, uint64_t cols)
{
    const int shape = shape_of(cols);
    const uint64_t each = shape == kLong ? 32 : 4 * (shape == kWarp ? kWarpThreads / lanes_of(cols) : 1);
    const uint64_t per_sm = threads_of(cols) < 128 ? 512 / threads_of(cols) : 4;
    const uint64_t want = (rows + each - 1) / each, most = shape == kLong ? 64 : 152 * per_sm;
    return want < most ? want : most;
}

uint64_t workspace_of(uint64_t rows, uint64_t cols) { return groups_of(rows, cols) * 2 * muon::up(cols, 8) * sizeof(float); }

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
    uint64_t groups = groups_of(p->rows, p->cols);
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
        P.dy = kept::matrix(dy, dy_ld, p->dtype);
        if (dx) P.dx = kept::out(dx, dx_ld, p->dtype);
        if (from) P.from = kept::source(*from);
        else P.x = kept::matrix(x, x_ld, p->dtype);
        P.mean = const_cast<float *>(mean);
        P.rstd = const_cast<float *>(rstd);
        P.partial = static_cast<float *>(ws);
        P.dw = dweight != nullptr;
        P.db = dbias != nullptr;
        const int shape = shape_of(p->cols);
        const unsigned threads = threads_of(p->cols);
        const bool full = whole(p->cols) && P.dy.vec && (!dx || P.dx.vec) && (from ? P.from.vec && kept::powers_whole(*from, p->cols) : P.x.vec);
        const Backward k = backward_of(p->dtype, from != nullptr, shape, threads, full, !p->centred && !dbias);
        int most = 0;
        st = kept::resident(k.kernel, static_cast<int>(threads), k.smem, &most);
        if (st != ASR_OK) return st;
        if (shape != kLong && groups > static_cast<uint64_t>(most)) groups = static_cast<uint64_t>(most);
        if (shape != kLong || dx) {
            const unsigned grid = shape == kLong ? int8::blocks_for(p->rows, 1, static_cast<uint64_t>(most)) : static_cast<unsigned>(groups);
            k.kernel<<<grid, threads, k.smem, stream>>>(P);
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
    S.pitch = muon::up(p->cols, 8);
    S.groups = p->rows ? static_cast<uint32_t>(groups) : 0;
    S.out[0] = dweight;
    S.out[1] = dbias;
    S.dtype[0] = static_cast<uint32_t>(dweight_dtype);
    S.dtype[1] = static_cast<uint32_t>(dbias_dtype);
    const dim3 grid(static_cast<unsigned>((p->cols + 31) / 32), dweight && dbias ? 2 : 1);
    return prod::launch_early(ASR_KERNEL_NORM, sum_kernel, grid, kSumWarps * 32, S, stream);
}

}  // namespace norm
