// int8_few.cuh -- the 8-bit integer product with few rows of A (tokens): what
// bounds it is reading B (the weight) once.  Included into asr.cu (inside its
// anonymous namespace), before int8.cuh.
//
// The work is cut into slabs, 128 rows of B by 512 of K, and every CTA (one on
// each SM) takes the same number of consecutive slabs, across row blocks where
// they end: all SMs read the same share of the weight, whatever its shape.
// Sixteen warps: four blocks of 32 rows, four quarters of a slab's K.  A warp
// streams its rows from global memory straight into registers, 16 bytes a lane
// and row, a slab ahead, and widens them to f16 there; the tokens (f16 already)
// come into shared memory by asynchronous copies, two slabs ahead.  The sums of
// a row block's part are added up over the warps in shared memory, in int32,
// and where several CTAs share the block, over them in the workspace: the CTA
// that completes the block's count of slabs writes the outputs.  Integer sums
// are the same in every order, and nobody waits for anybody.
//
// The products are mma.sync m16n8k16 (f16, binary32 sums): B's rows are the 16,
// tokens the 8.  Measured on GB300, an SM does one in two cycles; with up to 48
// tokens (6 products for 256 bytes of B, so 23 bytes a cycle) that keeps pace
// with the SM's share of the memory rate (23 bytes a cycle), and with operands
// in registers the weight never passes through shared memory, where widening it
// for tcgen05 would cost three bytes' traffic for each.  The order of K inside a
// product is free, so a lane's 16 contiguous bytes serve as its fragments of
// four consecutive steps.  At most 1,024 products are added in binary32, which
// is exact.

namespace int8few {

constexpr int kThreads = 512;
constexpr int kRows = 128;                  // rows of B a slab
constexpr int kSlab = 512;                  // K a slab, a quarter of it a warp
constexpr int kPitch = kSlab * 2 + 16;      // bytes between tokens in shared memory: 8 lanes' 16 bytes never collide
constexpr int kSumPitch = kRows + 4;        // words between tokens' sums
constexpr int kMaxTokens = 48;              // of a pass over B
constexpr uint32_t kMaxRun = 1024 / (kSlab / 4);    // slabs added up in binary32
constexpr int kStages = 3;                  // slabs of tokens in shared memory

struct Params {
    const __half *a;                        // tokens, widened: m x k, rows a multiple of 32 bytes apart
    const int8_t *b;                        // weight, n x k
    const float *row_scale, *col_scale;
    void *c;
    int32_t *sums;                          // [row block][token][128], zero at the start
    uint32_t *counts;                       // [token group][row block], zero at the start
    uint64_t lda, ldb, ldc;
    uint32_t m, n, k, tiles, slabs;         // row blocks, slabs of each
    uint32_t b_vec;                         // rows of B in 16-byte aligned units
    uint32_t c_dtype, rounding, step;
    uint32_t early;                         // B may be read before the previous kernel has finished
    RoundKeys keys;
};

// Four 8-bit integers (bytes of w) to f16, exact: 1,024 + (x + 128), less 1,152.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), bias);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), bias);
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
}

// 16 bytes of a row from column k on, zeros past its end.
__device__ __noinline__ uint4 load16_slow(const int8_t *p, uint32_t count)
{
    uint32_t w[4] = {0, 0, 0, 0};
    for (uint32_t q = 0; q < 16 && q < count; ++q) {
        const uint32_t v = static_cast<uint32_t>(static_cast<uint8_t>(p[q])) << (8 * (q & 3));
        if (q < 4) w[0] |= v;
        else if (q < 8) w[1] |= v;
        else if (q < 12) w[2] |= v;
        else w[3] |= v;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void mma16816(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int NB>
constexpr int smem_bytes()
{
    return kStages * 8 * NB * kPitch + 8 * NB * kSumPitch * 4;
}

// One output from its integer sum.
__device__ __forceinline__ void store_output(const Params &P, uint32_t token, uint32_t col, int32_t sum)
{
    const float y = __fmul_rn(__fmul_rn(__int2float_rn(sum), P.row_scale[token]), __ldg(P.col_scale + col));
    const uint64_t dst = token * P.ldc + col;
    if (P.c_dtype == ASR_F32) {
        static_cast<float *>(P.c)[dst] = y;
        return;
    }
    uint32_t h;
    if (P.rounding == ASR_ROUND_SR) {
        const uint64_t e = static_cast<uint64_t>(token) * P.n + col;
        uint32_t r[4];
        philox_q(e >> 2, P.step, P.keys, r);
        const uint32_t sel = static_cast<uint32_t>(e & 3u);
        h = round_sr(y, sel == 0 ? r[0] : sel == 1 ? r[1] : sel == 2 ? r[2] : r[3]);
    } else {
        h = round_rne(y);
    }
    static_cast<uint16_t *>(P.c)[dst] = static_cast<uint16_t>(h);
}

// Tokens 8 * NB * blockIdx.y and on.
template <int NB>
__global__ void __launch_bounds__(kThreads, 1) few_rows_kernel(const __grid_constant__ Params P)
{
    constexpr int kTokens = 8 * NB;
    extern __shared__ __align__(128) unsigned char smem[];
    int32_t *sums = reinterpret_cast<int32_t *>(smem + kStages * kTokens * kPitch);   // [kTokens][kSumPitch]
    __shared__ uint32_t done;
    const uint32_t xs = smem_addr(smem);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3, quarter = warp & 3, wr = warp >> 2;
    const uint32_t token0 = blockIdx.y * kTokens, tokens = min(static_cast<uint32_t>(kTokens), P.m - token0);
    const uint32_t total = P.tiles * P.slabs;
    const uint32_t first = static_cast<uint32_t>(static_cast<uint64_t>(total) * blockIdx.x / gridDim.x);
    const uint32_t end = static_cast<uint32_t>(static_cast<uint64_t>(total) * (blockIdx.x + 1) / gridDim.x);

    if (!P.early) asm volatile("griddepcontrol.wait;" ::: "memory");

    // the weight of slab (tile, s): rows g, g + 8, g + 16, g + 24 of the warp's 32, two 64-wide pieces
    uint4 w[2][4];
    auto weight = [&](uint32_t tile, uint32_t s, int i) {
        const uint32_t row = tile * kRows + wr * 32 + g, k = s * kSlab + quarter * (kSlab / 4) + i * 64 + t * 16;
        const int8_t *p = P.b + row * P.ldb + k;
#pragma unroll
        for (int r = 0; r < 4; ++r, p += 8 * P.ldb) {
            w[i][r] = make_uint4(0, 0, 0, 0);
            if (row + 8 * r < P.n && k < P.k) {
                if (P.b_vec && k + 16 <= P.k) w[i][r] = __ldcs(reinterpret_cast<const uint4 *>(p));
                else w[i][r] = load16_slow(p, P.k - k);
            }
        }
    };
    // the tokens of a slab: copies of 16 bytes, zeros past their end (rows are padded to 16 values, the last
    // unit's padding is zero)
    auto fetch = [&](uint32_t s, uint32_t stage) {
#pragma unroll
        for (int q = 0; q < NB; ++q) {
            const uint32_t u = q * kThreads + threadIdx.x, token = u >> 6, k = s * kSlab + (u & 63) * 8;
            const bool in = token < tokens && k < P.k;
            const __half *src = P.a + (in ? static_cast<uint64_t>(token0 + token) * P.lda + k : 0);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(xs + (stage * kTokens + token) * kPitch +
                                                                               (u & 63) * 16),
                         "l"(src), "r"(in ? 16 : 0)
                         : "memory");
        }
    };

    uint32_t tile = first / P.slabs, s = first % P.slabs;
    if (first < end) {
        weight(tile, s, 0);
        weight(tile, s, 1);
    }
    if (P.early) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    for (int i = threadIdx.x; i < kTokens * kSumPitch; i += kThreads) sums[i] = 0;
    // slab numbers of the copies run ahead of those of the products
    uint32_t fs = s, fetched = first;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        if (fetched < end) fetch(fs, static_cast<uint32_t>(i));
        ++fetched;
        fs = fs + 1 == P.slabs ? 0 : fs + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    float acc[2][NB][4];
#pragma unroll
    for (int mb = 0; mb < 2; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[mb][nb][q] = 0.0f;

    uint32_t run = 0, stage = 0, ahead = kStages - 1;
    for (uint32_t at = first; at < end; ++at) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncthreads();                        // this slab's tokens are here, and the stage two ahead is free
        if (fetched < end) fetch(fs, ahead);
        ++fetched;
        fs = fs + 1 == P.slabs ? 0 : fs + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
        const uint32_t ns = s + 1 == P.slabs ? 0 : s + 1, nt = s + 1 == P.slabs ? tile + 1 : tile;
        const unsigned char *x = smem + (stage * kTokens + g) * kPitch + quarter * (kSlab / 2) + t * 32;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t v[4][4];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r][0] = w[i][r].x, v[r][1] = w[i][r].y, v[r][2] = w[i][r].z, v[r][3] = w[i][r].w;
            if (at + 1 < end) weight(nt, ns, i);
#pragma unroll
            for (int h = 0; h < 2; ++h) {        // two steps of 16
                uint32_t a[2][2][4];             // [step][row block][fragment]
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int r = 0; r < 4; ++r) widen4(v[r][2 * h + q], a[q][r >> 1][r & 1], a[q][r >> 1][(r & 1) + 2]);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const uint4 b = *reinterpret_cast<const uint4 *>(x + nb * 8 * kPitch + i * 128 + h * 16);
                    mma16816(acc[0][nb], a[0][0], b.x, b.y);
                    mma16816(acc[1][nb], a[0][1], b.x, b.y);
                    mma16816(acc[0][nb], a[1][0], b.z, b.w);
                    mma16816(acc[1][nb], a[1][1], b.z, b.w);
                }
            }
        }
        ++run;
        if (at + 1 == end || s + 1 == P.slabs || run == kMaxRun) {
            // add the warps' sums up
#pragma unroll
            for (int mb = 0; mb < 2; ++mb)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int token = nb * 8 + 2 * t + (q & 1), row = wr * 32 + mb * 16 + g + (q >> 1) * 8;
                        atomicAdd(sums + token * kSumPitch + row, __float2int_rn(acc[mb][nb][q]));
                        acc[mb][nb][q] = 0.0f;
                    }
            __syncthreads();
            const bool whole = run == P.slabs;      // the block's only part
            const uint32_t row = threadIdx.x % kRows, col = tile * kRows + row;
            for (uint32_t token = threadIdx.x / kRows; token < tokens; token += kThreads / kRows) {
                int32_t *p = sums + token * kSumPitch + row;
                const int32_t sum = *p;
                *p = 0;
                if (whole) {
                    if (col < P.n) store_output(P, token0 + token, col, sum);
                } else {
                    atomicAdd(P.sums + (static_cast<uint64_t>(tile) * P.m + token0 + token) * kRows + row, sum);
                }
            }
            if (!whole) {
                __threadfence();
                __syncthreads();
                if (threadIdx.x == 0) done = atomicAdd(P.counts + blockIdx.y * P.tiles + tile, run) + run;
                __syncthreads();
                if (done == P.slabs) {
                    __threadfence();
                    for (uint32_t token = threadIdx.x / kRows; token < tokens; token += kThreads / kRows)
                        if (col < P.n)
                            store_output(P, token0 + token, col,
                                         __ldcg(P.sums + (static_cast<uint64_t>(tile) * P.m + token0 + token) * kRows + row));
                }
            }
            run = 0;
            // the sums are zero again before any warp adds to them: the next slab begins with a barrier, and
            // they are added to at its end
        }
        s = ns;
        tile = nt;
        stage = stage + 1 == kStages ? 0 : stage + 1;
        ahead = ahead + 1 == kStages ? 0 : ahead + 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// ------------------------------------------------------------------ host

std::mutex g_few_mu;
int g_few_sms[kMaxDevices];

template <int NB>
cudaError_t opt_in()
{
    return cudaFuncSetAttribute(few_rows_kernel<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<NB>());
}

asr_status setup(int *sms)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev < 0 || dev >= kMaxDevices) return ASR_ERR_INVALID_VALUE;
    std::lock_guard<std::mutex> lk(g_few_mu);
    if (!g_few_sms[dev]) {
        int n = 0;
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = opt_in<1>();
        if (e == cudaSuccess) e = opt_in<2>();
        if (e == cudaSuccess) e = opt_in<3>();
        if (e == cudaSuccess) e = opt_in<4>();
        if (e == cudaSuccess) e = opt_in<5>();
        if (e == cudaSuccess) e = opt_in<6>();
        if (e != cudaSuccess) return cuda_fail(e);
        g_few_sms[dev] = n;
    }
    *sms = g_few_sms[dev];
    return ASR_OK;
}

uint32_t groups(uint64_t m) { return static_cast<uint32_t>((m + kMaxTokens - 1) / kMaxTokens); }

template <int NB>
asr_status launch_few(Params &P, int sms, cudaStream_t stream)
{
    const uint32_t count = (P.m + 8 * NB - 1) / (8 * NB), total = P.tiles * P.slabs;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(total < static_cast<uint32_t>(sms) ? total : static_cast<uint32_t>(sms), count, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes<NB>();
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, few_rows_kernel<NB>, P);
    if (e != cudaSuccess) return cuda_fail(e);
    return launched(ASR_KERNEL_INT8_FEW_ROWS);
}

// P.m tokens in groups of equal size, at most kMaxTokens each.
asr_status run(Params &P, cudaStream_t stream)
{
    int sms = 0;
    const asr_status st = setup(&sms);
    if (st != ASR_OK) return st;
    P.tiles = (P.n + kRows - 1) / kRows;
    P.slabs = (P.k + kSlab - 1) / kSlab;
    if (static_cast<uint64_t>(P.tiles) * P.slabs >= (1ull << 31)) return ASR_ERR_INVALID_VALUE;
    const uint32_t g = groups(P.m), each = (P.m + g - 1) / g, nb = (each + 7) / 8;
    switch (nb) {
    case 1: return launch_few<1>(P, sms, stream);
    case 2: return launch_few<2>(P, sms, stream);
    case 3: return launch_few<3>(P, sms, stream);
    case 4: return launch_few<4>(P, sms, stream);
    case 5: return launch_few<5>(P, sms, stream);
    default: return launch_few<6>(P, sms, stream);
    }
}

}  // namespace int8few
